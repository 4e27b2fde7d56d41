"""The operators over sequences and AdamW without a GPU: the headers, the sizes, and the refusals, which come
before anything touches the device."""
import ctypes
import os
import re

import pytest
import torch

import cnn_convolution_conv2d_b200 as cb
from cnn_convolution_conv2d_b200 import optimizer, sequence
import sequence_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TABLES = {"sequence_b200.h": sequence.SIGNATURES, "optimizer_b200.h": optimizer.SIGNATURES}


BF, F = cb.CONV_BF16, cb.CONV_F32


@pytest.fixture(scope="module")
def lib():
    from cnn_convolution_conv2d_b200 import build
    build.build()
    return cb.load()


@pytest.mark.parametrize("header", sorted(TABLES))
def test_headers_and_signatures_agree(lib, header):
    text = open(os.path.join(ROOT, "include", header), encoding="utf-8").read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    decls = {n: len(a.split(",")) for n, a in re.findall(r"^int\s+(\w+)\s*\(([^)]*)\)\s*;", text, flags=re.M)}
    assert set(decls) == set(TABLES[header])
    for name, count in decls.items():
        assert len(TABLES[header][name][0]) == count, name
        assert hasattr(lib, name)


def test_adamw_struct_matches_the_header():
    # seven pointers and a long long: no padding on a 64-bit machine
    assert ctypes.sizeof(optimizer.AdamWTensor) == 64


def test_sizes(lib):
    assert cb.conv1d_causal_backward_workspace_size(0, 64, 4) == 0
    # without a device strips are 64 rows, four to a block: 1000 rows are 4 blocks of (K + 1) C sums
    if not torch.cuda.is_available():
        assert cb.conv1d_causal_backward_workspace_size(1000, 64, 4) == 4 * 5 * 64 * 4
    # one chunk (forward 256 rows in bf16, 128 in fp32; backward 128 and 96): nothing to join; otherwise three values for
    # each chunk and channel (rounded up to 32), and a rate; backward also a sum for each
    forward, backward, saved = (cb.gated_recurrence_workspace_size, cb.gated_recurrence_backward_workspace_size,
                                cb.gated_recurrence_saved_size)
    assert forward(1, 0, 256, 100, BF) == 0 and forward(1, 128, 128, 100, F) == 0
    assert forward(1, 0, 257, 100, BF) == 256 + 2 * 128 * 12 + 128 * 4
    assert forward(9, 0, 257, 100, F) == 256 + 3 * 128 * 12 + 128 * 4
    assert backward(1, 0, 128, 100, BF) == 128 * 4
    assert backward(1, 0, 129, 100, BF) == 256 + 2 * 128 * 16 + 128 * 4
    assert backward(1, 0, 97, 100, F) == 256 + 2 * 128 * 16 + 128 * 4
    # a saved state for every 8 rows that have begun; sequences of a few chunks have chunks and states of their own
    assert saved(1, 129, 129, 100, BF) == saved(3, 0, 129, 100, F) == 17 * 128 * 4
    assert saved(3, 129, 387, 100, BF) == 3 * 17 * 128 * 4 and forward(3, 129, 387, 100, BF) == 256 + 3 * 128 * 12 + 128 * 4
    assert saved(30, 10, 300, 100, BF) == 38 * 128 * 4      # shorter than half a chunk: one after the other
    for bad in ((1, 0, -1, 4, BF), (1, 0, 5, 0, BF), (1, 0, 5, 4, 7), (0, 0, 5, 4, BF), (2, 3, 5, 4, BF), (1, -1, 5, 4, BF)):
        with pytest.raises(cb.Conv2dError) as err:
            saved(*bad)
        assert err.value.status == cb.CONV_ERR_INVALID_ARG
    with pytest.raises(cb.Conv2dError) as err:
        cb.gated_recurrence_workspace_size(1, 0, 2 ** 31, 4, BF)
    assert err.value.status == cb.CONV_ERR_UNSUPPORTED
    for size in (lambda C: saved(1, 0, 1, C, BF), lambda C: forward(1, 0, 1, C, F), lambda C: backward(1, 0, 1, C, F),
                 lambda C: cb.conv1d_causal_backward_workspace_size(1, C, 4)):
        size(2 ** 30)
        with pytest.raises(cb.Conv2dError) as err:
            size(2 ** 30 + 1)
        assert err.value.status == cb.CONV_ERR_UNSUPPORTED
    for K in (1, 9):
        with pytest.raises(cb.Conv2dError):
            cb.conv1d_causal_backward_workspace_size(8, 8, K)


INVALID, UNSUPPORTED = cb.CONV_ERR_INVALID_ARG, cb.CONV_ERR_UNSUPPORTED


def conv_forward(lib, x=16, w=16, bias=None, y=64, state=None, final=None, off=None, nseq=2, T=4, rows=8, C=8, K=4, act=0,
                 ldx=8, ldy=8, dtype=BF):
    return lib.conv1d_causal_forward(x, w, bias, y, state, final, off, nseq, T, rows, C, K, act, ldx, ldy, dtype, None)


@pytest.mark.parametrize("change, status", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(y=16), INVALID),
    (dict(nseq=0), INVALID), (dict(T=3), INVALID), (dict(rows=-1), INVALID), (dict(C=0), INVALID), (dict(K=1), INVALID),
    (dict(K=9), INVALID), (dict(act=2), INVALID), (dict(ldx=-1), INVALID), (dict(ldy=7), INVALID), (dict(dtype=5), INVALID),
    (dict(state=128, final=128), INVALID), (dict(x=17), UNSUPPORTED), (dict(off=18), UNSUPPORTED),
    (dict(rows=2 ** 31, T=2 ** 30), UNSUPPORTED),
], ids=str)
def test_convolution_refusals(lib, change, status):
    assert conv_forward(lib, **change) == status
    assert cb.conv2d_last_error()


def test_convolution_backward_refusals(lib):
    def call(x=16, w=16, dy=32, dx=64, dw=96, ldx=8, dfinal=None, dstate=None, ws=None, nbytes=0, K=4):
        return lib.conv1d_causal_backward(x, w, None, dy, None, dfinal, dx, dw, None, dstate, None, 2, 4, 8, 8, K, 0, ldx, 8, 8, BF,
                                          ws, nbytes, None)
    for change in (dict(dy=None), dict(dx=None), dict(dw=None), dict(dx=32), dict(ldx=-8), dict(K=12),
                   dict(dfinal=128, dstate=128)):
        assert call(**change) == INVALID, change
    assert call(dy=33) == UNSUPPORTED


def test_step_refusals(lib):
    def conv(x=16, w=16, y=64, state=128, slots=None, B=2, pool=2, C=8, K=4, act=0, ldx=8, ldy=8, dtype=BF):
        return lib.conv1d_causal_step(x, w, None, y, state, slots, B, pool, C, K, act, ldx, ldy, dtype, None)
    for change in (dict(x=None), dict(w=None), dict(y=None), dict(state=None), dict(B=0), dict(pool=0), dict(pool=1),
                   dict(C=0), dict(K=1), dict(act=-1), dict(ldy=4), dict(y=16), dict(state=64), dict(dtype=9)):
        assert conv(**change) == INVALID, change
    assert conv(slots=129) == UNSUPPORTED

    def rec(x=16, ga=16, gx=16, decay=16, kappa=8.0, y=64, state=128, slots=None, B=2, pool=2, C=8, ldy=8, dtype=BF):
        return lib.gated_recurrence_step(x, ga, gx, decay, kappa, y, state, slots, B, pool, C, 8, 8, 8, ldy, dtype, None)
    for change in (dict(x=None), dict(ga=None), dict(gx=None), dict(decay=None), dict(kappa=0.0), dict(kappa=float("inf")),
                   dict(kappa=float("nan")), dict(state=None), dict(B=0), dict(pool=1), dict(ldy=7), dict(state=64)):
        assert rec(**change) == INVALID, change
    assert rec(decay=18) == UNSUPPORTED


def test_recurrence_refusals(lib):
    def forward(x=16, ga=32, gx=48, decay=16, kappa=8.0, y=64, state=None, final=None, off=None, nseq=2, T=4, rows=8, C=8,
                lda=8, ldy=8, dtype=BF, ws=None, nbytes=0):
        return lib.gated_recurrence_forward(x, ga, gx, decay, kappa, y, state, final, None, off, nseq, T, rows, C, 8, lda, 8,
                                            ldy, dtype, ws, nbytes, None)
    for change in (dict(x=None), dict(ga=None), dict(gx=None), dict(decay=None), dict(y=None), dict(y=32), dict(kappa=-1.0),
                   dict(nseq=0), dict(T=5), dict(C=0), dict(lda=-2), dict(ldy=4), dict(dtype=3), dict(state=96, final=96)):
        assert forward(**change) == INVALID, change
    assert forward(gx=49) == UNSUPPORTED
    # more than one chunk: the workspace is checked, before any device is asked for
    assert forward(T=128, rows=256) == cb.CONV_ERR_WORKSPACE
    assert forward(T=128, rows=256, ws=256, nbytes=100) == cb.CONV_ERR_WORKSPACE
    assert forward(T=128, rows=256, ws=264, nbytes=1 << 20) == UNSUPPORTED

    def backward(saved=256, dx=64, dga=128, dgx=192, ddecay=16, ws=None, nbytes=0):
        return lib.gated_recurrence_backward(16, 32, 48, 512, 8.0, 56, saved, None, None, dx, dga, dgx, ddecay, None, None, 2, 4,
                                             8, 8, 8, 8, 8, 8, 8, 8, 8, BF, ws, nbytes, None)
    for change in (dict(saved=None), dict(dx=None), dict(dga=None), dict(dgx=None), dict(ddecay=None), dict(dga=64),
                   dict(dx=56), dict(ddecay=512)):
        assert backward(**change) == INVALID, change
    assert backward() == cb.CONV_ERR_WORKSPACE


def adamw(lib, entries=None, count=None, pd=F, gd=F, bits=32, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.0, step=1,
          step_device=None, scale=None):
    rows = entries if entries is not None else [dict()]
    table = (optimizer.AdamWTensor * max(1, len(rows)))()
    for t, e in zip(table, rows):
        e = dict(dict(param=4096, master=None, grad=64, exp_avg=128, exp_avg_sq=192, exp_avg_scale=None, exp_avg_sq_scale=None,
                      numel=8), **e)
        for k, v in e.items():
            setattr(t, k, v)
    return lib.adamw_step(table, len(rows) if count is None else count, pd, gd, bits, lr, b1, b2, eps, wd, step, step_device,
                          scale, 0, None)


@pytest.mark.parametrize("change, status", [
    (dict(count=-1), INVALID), (dict(pd=4), INVALID), (dict(gd=-1), INVALID), (dict(bits=16), INVALID), (dict(lr=-1.0), INVALID),
    (dict(lr=float("nan")), INVALID), (dict(b1=1.0), INVALID), (dict(b2=-0.1), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(wd=-1.0), INVALID), (dict(step=0), INVALID), (dict(entries=[dict(param=None)]), INVALID),
    (dict(entries=[dict(grad=None)]), INVALID), (dict(entries=[dict(exp_avg=None)]), INVALID),
    (dict(entries=[dict(exp_avg_sq=None)]), INVALID), (dict(entries=[dict(numel=-1)]), INVALID),
    (dict(bits=8), INVALID), (dict(entries=[dict(master=256)]), INVALID),
    (dict(pd=BF, entries=[dict(master=256), dict(param=8192)]), INVALID),
    (dict(entries=[dict(), dict()]), INVALID), (dict(entries=[dict(), dict(param=4112)]), INVALID),
    (dict(entries=[dict(param=4100)]), UNSUPPORTED), (dict(entries=[dict(grad=72)]), UNSUPPORTED),
    (dict(entries=[dict(numel=2 ** 41 + 1)]), UNSUPPORTED), (dict(step_device=4), UNSUPPORTED), (dict(scale=2), UNSUPPORTED),
], ids=str)
def test_adamw_refusals(lib, change, status):
    assert adamw(lib, **change) == status
    assert cb.conv2d_last_error()


def table_of(*entries):
    table = (optimizer.AdamWTensor * len(entries))()
    for i, (t, e) in enumerate(zip(table, entries)):
        e = dict(dict(param=(i + 1) << 48, grad=64, exp_avg=128, exp_avg_sq=192, exp_avg_scale=256, exp_avg_sq_scale=320, numel=8), **e)
        for k, v in e.items():
            setattr(t, k, v)
    return table


def test_adamw_launches(lib):
    """Tensors without elements are passed over whatever they hold: they do not choose the kernel, but keep their place."""
    plan = cb.adamw_describe_plan(table_of(dict(), dict(numel=0, master=4096), dict(numel=1025)), BF, 32, 148)
    assert plan == {"master": 0, "batches": 1, "launches": [{"first": 0, "count": 3, "blocks": 3}]}
    plan = cb.adamw_describe_plan(table_of(dict(numel=0), dict(master=4096)), BF, 32, 148)
    assert plan["master"] == 1 and plan["launches"] == [{"first": 0, "count": 2, "blocks": 1}]
    assert cb.adamw_describe_plan(table_of(*[dict(numel=0, master=16, param=None)] * 3), BF, 8, 148)["launches"] == []
    # 48 tensors of a launch, those without elements among them
    plan = cb.adamw_describe_plan(table_of(*[dict(numel=n % 2 * 1024) for n in range(100)]), F, 32, 148)
    assert plan["launches"] == [{"first": 0, "count": 48, "blocks": 24}, {"first": 48, "count": 48, "blocks": 24},
                                {"first": 96, "count": 4, "blocks": 2}]
    # more batches a block with 8-bit states: 8 blocks an SM are left
    plan = cb.adamw_describe_plan(table_of(dict(numel=1024 * 8 * 148 * 3)), F, 8, 148)
    assert plan["batches"] == 3 and plan["launches"][0]["blocks"] == 8 * 148
    for bad in (lambda t: lib.adamw_describe_plan(t, 1, F, 32, 148, None, 0),
                lambda t: lib.adamw_describe_plan(t, 1, F, 32, 148, ctypes.create_string_buffer(8), 8),
                lambda t: lib.adamw_describe_plan(t, -1, F, 32, 148, ctypes.create_string_buffer(99), 99),
                lambda t: lib.adamw_describe_plan(t, 1, F, 16, 148, ctypes.create_string_buffer(99), 99),
                lambda t: lib.adamw_describe_plan(t, 1, 4, 32, 148, ctypes.create_string_buffer(99), 99)):
        assert bad(table_of(dict())) == INVALID


def test_the_largest_tensor_of_adamw(lib):
    """One that needs all the blocks of a launch is taken by itself; one element more is refused, by the plan as by the step."""
    most = (2 ** 31 - 1) * 1024
    plan = cb.adamw_describe_plan(table_of(dict(), dict(numel=most)), F, 32, 148)
    assert plan["launches"] == [{"first": 0, "count": 1, "blocks": 1}, {"first": 1, "count": 1, "blocks": 2 ** 31 - 1}]
    for numel in (most + 1, 2 ** 41):
        assert adamw(lib, entries=[dict(numel=numel)]) == UNSUPPORTED
        with pytest.raises(cb.Conv2dError) as err:
            cb.adamw_describe_plan(table_of(dict(numel=numel)), F, 32, 148)
        assert err.value.status == UNSUPPORTED


def test_layers_refuse_on_the_host(lib):
    w = torch.zeros(6, 4)
    for bad in (lambda: cb.CausalConv1dB200(torch.zeros(6)), lambda: cb.CausalConv1dB200(torch.zeros(6, 1)),
                lambda: cb.CausalConv1dB200(torch.zeros(6, 9)), lambda: cb.CausalConv1dB200(w, activation="relu"),
                lambda: cb.CausalConv1dB200(w, torch.zeros(5)), lambda: cb.CausalConv1dB200(torch.zeros(4, 6).t()),
                lambda: cb.GatedRecurrenceB200(torch.zeros(2, 3))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: cb.CausalConv1dB200(w.half()), lambda: cb.CausalConv1dB200(w, torch.zeros(6).bfloat16()),
                lambda: cb.GatedRecurrenceB200(torch.zeros(3).bfloat16())):
        with pytest.raises(TypeError):
            bad()
    conv, rec = cb.CausalConv1dB200(w), cb.GatedRecurrenceB200(torch.zeros(6))
    x = torch.zeros(2, 3, 6)
    for bad in (lambda: conv(x), lambda: conv(torch.zeros(2, 3, 5)), lambda: rec(x, x, x), lambda: conv.step(x, x),
                lambda: cb.AdamWB200([w]), lambda: cb.AdamWB200([])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        conv(x.bfloat16())


def test_layers_look_at_weights_whose_memory_was_replaced(lib):
    """Another type or size behind the same tensor is refused before anything reads it; the same kind is taken."""
    w, b, decay = torch.zeros(6, 4), torch.zeros(6), torch.zeros(6)
    conv, rec = cb.CausalConv1dB200(w, b), cb.GatedRecurrenceB200(decay)
    x, window, state = torch.zeros(2, 3, 6), torch.zeros(2, 3, 6), torch.zeros(2, 6)
    row, saved = x[:, 0].contiguous(), rec.saved_states(x)
    conv_calls = (lambda: conv(x), lambda: conv.backward(x, x), lambda: conv.step(row, window))
    rec_calls = (lambda: rec(x, x, x), lambda: rec.backward(x, x, x, x, saved), lambda: rec.step(row, row, row, state))
    for t, calls, bad in ((w, conv_calls, [torch.zeros(6, 4).bfloat16(), torch.zeros(6, 3), torch.zeros(4, 6).t()]),
                          (b, conv_calls, [torch.zeros(6).bfloat16(), torch.zeros(3)]),
                          (decay, rec_calls, [torch.zeros(6).bfloat16(), torch.zeros(5)])):
        good = t.data
        for other in bad:
            t.data = other
            for call in calls:
                with pytest.raises(TypeError if other.dtype != torch.float32 else ValueError) as err:
                    call()
                assert "CUDA" not in str(err.value)
        for other in (good.clone(), good):
            t.data = other
            for call in calls:
                with pytest.raises(ValueError, match="CUDA"):       # as far as a call gets without a device
                    call()


def test_layers_look_at_weights_that_changed_in_the_same_memory(lib):
    """Memory that was freed in between may come back at the same address for another type or shape."""
    w, decay = torch.zeros(6, 4), torch.zeros(6)
    conv, rec = cb.CausalConv1dB200(w), cb.GatedRecurrenceB200(decay)
    x = torch.zeros(2, 3, 6)
    for t, call, others in ((w, lambda: conv(x), [w.data.view(torch.bfloat16), w.data[:3], w.data.view(4, 6).t()]),
                            (decay, lambda: rec(x, x, x), [decay.data.view(torch.bfloat16), decay.data[:3], decay.data[:1].expand(6)])):
        good = t.data
        for other in others:
            assert other.data_ptr() == good.data_ptr()
            t.data = other
            with pytest.raises(TypeError if other.dtype != torch.float32 else ValueError) as err:
                call()
            assert "CUDA" not in str(err.value)
        t.data = good


def test_reference_gradients_against_differences():
    """The 64-bit reference's own gradients, against central differences of its loss."""
    gen = torch.Generator().manual_seed(3)
    normal = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    seqs, C, K = [(0, 3), (3, 0), (3, 5)], 2, 3
    x, ga, gx, decay, h0 = normal(8, C), normal(8, C), normal(8, C), normal(C), normal(3, C)
    w, b, s0 = normal(C, K), normal(C), normal(3, K - 1, C)
    cy, cf, hy, hf = normal(8, C), normal(3, K - 1, C), normal(8, C), normal(3, C)

    def conv_loss(x, w, b, s0):
        y, final, _ = ref.conv1d(x, w, b, True, seqs, s0)
        return (y * cy).sum() + (final * cf).sum()

    def rec_loss(x, ga, gx, decay, h0):
        h, final, _ = ref.recurrence(x, ga, gx, decay, 8.0, seqs, h0)
        return (h * hy).sum() + (final * hf).sum()

    for loss, args in ((conv_loss, (x, w, b, s0)), (rec_loss, (x, ga, gx, decay, h0))):
        args = [a.clone().requires_grad_() for a in args]
        grads = torch.autograd.grad(loss(*args), args)
        for i, g in enumerate(grads):
            d = normal(*g.shape)
            at = lambda e: loss(*[a.detach() + (e * d if j == i else 0) for j, a in enumerate(args)])  # noqa: E731, B023
            # the difference is off by eps^2 times a third derivative of order 100, and 1e-15/eps
            assert abs((at(1e-5) - at(-1e-5)) / 2e-5 - (g * d).sum()) <= 1e-7 * (1 + g.abs().sum())
