"""The causal convolution over time and the gated recurrence on a B200, against the 64-bit loops of
sequence_reference.py, whose tolerances apply."""
import pytest
import torch

import cnn_convolution_conv2d_b200 as cb
import sequence_reference as ref

pytestmark = pytest.mark.gpu
KAPPA = 8.0


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    assert torch.cuda.is_available(), "these tests need a CUDA device"
    from cnn_convolution_conv2d_b200 import build
    build.build()
    cb.load()
    cb.conv2d_debug_set_watchdog(0, False)
    yield
    cb.conv2d_sync_status()


class Draw:
    """Seeded tensors: the values a kernel sees, and the same in 64 bits on the CPU."""

    def __init__(self, seed, dtype):
        self.gen, self.dtype = torch.Generator().manual_seed(seed), dtype

    def __call__(self, *shape, dtype=None, scale=1.0):
        t = (torch.randn(*shape, generator=self.gen) * scale).to(dtype or self.dtype)
        return t.cuda(), t.double()


def dev(offsets):
    return None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")


def shape_of(B, T, C, offsets, rows):
    return (rows if rows is not None else offsets[-1], C) if offsets else (B, T, C)


CASES = [  # B, T, offsets, rows (behind the last sequence), C, K, silu, carried state
    (1, 1, None, None, 1, 2, True, False),
    (2, 3, None, None, 5, 8, True, True),           # sequences shorter than the window
    (3, 130, None, None, 66, 4, True, True),        # chunks of the recurrence across sequences; ragged channels
    (1, 300, None, None, 130, 3, False, False),
    (2, 128, None, None, 128, 4, True, True),       # wide accesses
    (2, 257, None, None, 40, 6, True, True),
    (1, 0, None, None, 8, 4, True, True),           # no rows
    (3, 56, None, None, 24, 2, False, True),        # sequences that end with their chunks
    (1, 2100, None, None, 4, 4, True, True),        # a carry over many chunks
    (2, 2050, None, None, 16, 3, False, True),      # sequences with chunks of their own
    (5, 0, [0, 0, 1, 1, 140, 141], None, 72, 4, True, True),
    (4, 0, [0, 7, 7, 300, 300], 333, 64, 5, False, True),   # empty ones, and rows of no sequence
    (3, 0, [0, 128, 256, 384], 384, 64, 4, True, False),    # ... that end at multiples of runs
    (40, 0, list(range(0, 123, 3)), 122, 33, 7, True, True),  # many short ones
    (2, 0, [0, 0, 0], 9, 16, 4, True, True),        # rows, but none of a sequence
    (2, 512, None, None, 40, 4, True, True),        # chunks that begin and end with their sequences, forward,
    (3, 672, None, None, 33, 2, False, True),       # ... backward (672 is 7 x 96, 384 is 3 x 128 and 4 x 96),
    (2, 384, None, None, 33, 2, False, True),
    (4, 0, [0, 256, 256, 928, 1600], 1700, 48, 3, True, True),  # ... and packed
]
IDS = [f"B{c[0]}-T{c[1] if c[2] is None else 'packed'}-C{c[4]}-K{c[5]}" for c in CASES]
both = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
cases = pytest.mark.parametrize("case", CASES, ids=IDS)


def leaf(t):
    return None if t is None else t.clone().requires_grad_()


def conv_inputs(case, dtype, seed=1):
    B, T, offsets, rows, C, K, silu, carry = case
    d = Draw(seed, dtype)
    shape = shape_of(B, T, C, offsets, rows)
    return dict(x=d(*shape), dy=d(*shape), w=d(C, K, scale=K ** -0.5), bias=d(C, scale=0.2),
                state=d(B, K - 1, C) if carry else (None, None), dfinal=d(B, K - 1, C) if carry else (None, None))


def outside(shape, offsets):
    """Which rows belong to no sequence."""
    mask = torch.zeros(shape[0] if offsets else shape[0] * shape[1], dtype=torch.bool)
    if offsets:
        mask[offsets[-1]:] = True
    return mask


@both
@cases
def test_convolution(case, dtype):
    B, T, offsets, rows, C, K, silu, carry = case
    t = conv_inputs(case, dtype)
    x, w, bias, state = (leaf(t[k][1]) for k in ("x", "w", "bias", "state"))
    seqs = ref.pieces(x.shape, offsets)
    y, final, sizes = ref.conv1d(x.reshape(-1, C), w, bias, silu, seqs, state)
    skip = outside(x.shape, offsets)
    layer = cb.CausalConv1dB200(t["w"][0], t["bias"][0], "silu" if silu else None)
    got = torch.full_like(t["x"][0], 7.0)
    got_final = torch.full((B, K - 1, C), 7.0, dtype=dtype, device="cuda")
    out = layer(t["x"][0], y=got, offsets=dev(offsets), initial_state=t["state"][0], final_state=got_final)
    assert out is got
    flat = got.reshape(-1, C)
    assert bool((flat[skip.cuda()] == 7.0).all())
    # z is off by (K + 2) u sizes; y = z sigmoid(z) by at most 1.1 times that, and 16 u of itself
    ref.close(flat[~skip.cuda()], y[~skip], dtype, 1.1 * (K + 2) * ref.U * sizes[~skip] + 16 * ref.U * y.detach()[~skip].abs(), "y")
    ref.close(got_final, final, dtype, 0.0, "final state")
    # gradients
    loss = (y[~skip] * t["dy"][1].reshape(-1, C)[~skip]).sum() + (0 if not carry else (final * t["dfinal"][1]).sum())
    wanted = torch.autograd.grad(loss + 0 * sum(v.sum() for v in (x, w, bias)), [x, w, bias] + ([state] if carry else []))
    gx = torch.full_like(t["x"][0], 7.0)
    dx, dw, db, ds = layer.backward(t["x"][0], t["dy"][0], offsets=dev(offsets), initial_state=t["state"][0],
                                    d_final_state=t["dfinal"][0], dx=gx)
    cb.conv2d_sync_status()
    assert bool((dx.reshape(-1, C)[skip.cuda()] == 7.0).all())
    ref.grad_close(dx.reshape(-1, C)[~skip.cuda()], wanted[0].reshape(-1, C)[~skip], dtype, "dx")
    ref.grad_close(dw, wanted[1], dtype, "dw")
    ref.grad_close(db, wanted[2], dtype, "db")
    assert (ds is not None) == carry
    if carry:
        ref.grad_close(ds, wanted[3], dtype, "d_initial_state")


def rec_inputs(case, dtype, seed=2):
    B, T, offsets, rows, C, _, _, carry = case
    d = Draw(seed, dtype)
    shape = shape_of(B, T, C, offsets, rows)
    f32 = torch.float32
    # softplus(decay) between about 0.002 and 0.4: a between 0.04 and 0.998
    return dict(x=d(*shape), dy=d(*shape), ga=d(*shape), gx=d(*shape),
                decay=tuple(v - 3.5 for v in d(C, dtype=f32)),
                state=d(B, C, dtype=f32) if carry else (None, None), dfinal=d(B, C, dtype=f32) if carry else (None, None))


@both
@cases
def test_recurrence(case, dtype):
    B, T, offsets, rows, C, _, _, carry = case
    t = rec_inputs(case, dtype)
    x, ga, gx, decay, state = (leaf(t[k][1]) for k in ("x", "ga", "gx", "decay", "state"))
    decay = leaf(t["decay"][0].cpu().double())
    seqs = ref.pieces(x.shape, offsets)
    flatten = lambda v: v.reshape(-1, C)  # noqa: E731
    h, final, error = ref.recurrence(flatten(x), flatten(ga), flatten(gx), decay, KAPPA, seqs, state)
    skip = outside(x.shape, offsets)
    layer = cb.GatedRecurrenceB200(t["decay"][0], KAPPA)
    xs = [t[k][0] for k in ("x", "ga", "gx")]
    got = torch.full_like(xs[0], 7.0)
    got_final = torch.full((B, C), 7.0, device="cuda")
    saved = layer.saved_states(xs[0])
    layer(*xs, y=got, offsets=dev(offsets), initial_state=t["state"][0], final_state=got_final, saved=saved)
    flat = got.reshape(-1, C)
    assert bool((flat[skip.cuda()] == 7.0).all())
    ref.close(flat[~skip.cuda()], h[~skip], dtype, error[~skip], "y")
    last = torch.stack([error[first + n - 1] if n else torch.zeros(C) for first, n in seqs])
    ref.close(got_final, final, torch.float32, last, "final state")
    loss = (h[~skip] * flatten(t["dy"][1])[~skip]).sum() + (0 if not carry else (final * t["dfinal"][1]).sum())
    wanted = torch.autograd.grad(loss + 0 * sum(v.sum() for v in (x, ga, gx, decay)),
                                 [x, ga, gx, decay] + ([state] if carry else []))
    grads = [torch.full_like(xs[0], 7.0) for _ in range(3)]
    dx, dga, dgx, dd, ds = layer.backward(*xs, t["dy"][0], saved, offsets=dev(offsets), initial_state=t["state"][0],
                                          d_final_state=t["dfinal"][0], dx=grads[0], d_gate_a=grads[1], d_gate_x=grads[2])
    cb.conv2d_sync_status()
    for name, g, w in zip(("dx", "d_gate_a", "d_gate_x"), (dx, dga, dgx), wanted):
        assert bool((flatten(g)[skip.cuda()] == 7.0).all()), name
        ref.grad_close(flatten(g)[~skip.cuda()], flatten(w)[~skip], dtype, name)
    ref.grad_close(dd, wanted[3], torch.float32, "d_decay")
    assert (ds is not None) == carry
    if carry:
        ref.grad_close(ds, wanted[4], torch.float32, "d_initial_state")


@both
@pytest.mark.parametrize("B, C, K", [(1, 1, 2), (3, 70, 4), (5, 256, 8), (2, 4100, 4), (300, 8, 3)])
def test_steps_continue_a_forward_pass(B, C, K, dtype):
    """Tokens one by one, in slots of a larger pool with rows of no sequence among them, against the whole."""
    T = 5
    d = Draw(4, dtype)
    x, w, bias = d(B, T, C), d(C, K, scale=K ** -0.5), d(C)
    ga, gx, decay = d(B, T, C), d(B, T, C), d(C, dtype=torch.float32)
    pool = B + 3
    conv = cb.CausalConv1dB200(w[0], bias[0], "silu")
    rec = cb.GatedRecurrenceB200(decay[0], KAPPA)
    seqs = [(b * T, T) for b in range(B)]
    y, final, sizes = ref.conv1d(x[1].reshape(-1, C), w[1], bias[1], True, seqs)
    h, last, error = ref.recurrence(*(v[1].reshape(-1, C) for v in (x, ga, gx)), decay[1], KAPPA, seqs)
    order = torch.randperm(pool, generator=torch.Generator().manual_seed(1))[:B].to(torch.int32).cuda()
    # two rows without a sequence, in front and behind
    slots = torch.cat([torch.tensor([-1], dtype=torch.int32, device="cuda"), order,
                       torch.tensor([pool], dtype=torch.int32, device="cuda")])
    window = torch.zeros(pool, K - 1, C, dtype=dtype, device="cuda")
    state = torch.zeros(pool, C, device="cuda")
    pad = lambda v, t: torch.cat([v[:1, 0], v[:, t], v[:1, 0]])  # noqa: E731
    y, sizes = y.view(B, T, C), sizes.view(B, T, C)
    h, error = h.view(B, T, C), error.view(B, T, C)
    for t in range(T):
        got = torch.full((B + 2, C), 7.0, dtype=dtype, device="cuda")
        conv.step(pad(x[0], t), window, slots=slots, y=got)
        assert bool((got[[0, -1]] == 7.0).all())
        ref.close(got[1:-1], y[:, t], dtype, 1.1 * (K + 2) * ref.U * sizes[:, t] + 16 * ref.U * y[:, t].abs(), "conv step")
        got = torch.full((B + 2, C), 7.0, dtype=dtype, device="cuda")
        rec.step(pad(x[0], t), pad(ga[0], t), pad(gx[0], t), state, slots=slots, y=got)
        assert bool((got[[0, -1]] == 7.0).all())
        ref.close(got[1:-1], h[:, t], dtype, error[:, t], "recurrence step")
    ref.close(window[order.long()], final, dtype, 0.0, "window")
    ref.close(state[order.long()], last, torch.float32, error[:, -1], "state")
    rest = torch.ones(pool, dtype=torch.bool)
    rest[order.long().cpu()] = False
    assert bool((window[rest.cuda()] == 0).all()) and bool((state[rest.cuda()] == 0).all())
    # without slots row b has state b
    direct = torch.zeros(B, C, device="cuda")
    one = rec.step(x[0][:, 0], ga[0][:, 0], gx[0][:, 0], direct)
    ref.close(one, h[:, 0], dtype, error[:, 0], "without slots")
    cb.conv2d_sync_status()


def test_a_slot_named_twice_is_reported_and_the_later_row_left_out():
    rec = cb.GatedRecurrenceB200(torch.zeros(8, device="cuda"))
    conv = cb.CausalConv1dB200(torch.ones(8, 2, device="cuda"))
    x = torch.ones(3, 8, device="cuda")
    slots = torch.tensor([1, 0, 1], dtype=torch.int32, device="cuda")
    for step, state in ((lambda s, y: rec.step(x, x, x, s, slots=slots, y=y), torch.zeros(2, 8, device="cuda")),
                        (lambda s, y: conv.step(x, s, slots=slots, y=y), torch.zeros(2, 1, 8, device="cuda"))):
        y = torch.full((3, 8), 7.0, device="cuda")
        step(state, y)
        with pytest.raises(cb.Conv2dError) as err:
            cb.conv2d_sync_status()
        assert err.value.status == cb.CONV_ERR_INVALID_ARG and "slot" in str(err.value)
        assert bool((y[2] == 7.0).all()) and bool((y[:2] != 7.0).all()) and bool((state[0] == state[1]).all())
        cb.conv2d_sync_status()


@pytest.mark.parametrize("offsets", [[0, 9, 5, 12], [1, 4, 12], [0, 4, 13], [0, -3, 12]], ids=str)
def test_bad_offsets_are_reported(offsets):
    x = torch.ones(12, 8, device="cuda")
    rec, conv = cb.GatedRecurrenceB200(torch.zeros(8, device="cuda")), cb.CausalConv1dB200(torch.ones(8, 3, device="cuda"))
    saved = rec.saved_states(x)
    n = len(offsets) - 1
    for call in (lambda: conv(x, offsets=dev(offsets), final_state=torch.zeros(n, 2, 8, device="cuda")),
                 lambda: conv.backward(x, x, offsets=dev(offsets), initial_state=torch.zeros(n, 2, 8, device="cuda")),
                 lambda: rec(x, x, x, offsets=dev(offsets), final_state=torch.zeros(n, 8, device="cuda"), saved=saved),
                 lambda: rec.backward(x, x, x, x, saved, offsets=dev(offsets), initial_state=torch.zeros(n, 8, device="cuda"))):
        call()
        with pytest.raises(cb.Conv2dError) as err:
            cb.conv2d_sync_status()
        assert err.value.status == cb.CONV_ERR_INVALID_ARG and "offsets" in str(err.value)


@both
@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_what_one_sequence_holds_stays_there(poison, dtype):
    """NaN and infinities of one sequence, and of the rows behind the last one, reach no other."""
    offsets, rows, C, K = [0, 100, 260, 400], 450, 64, 4
    d = Draw(6, dtype)
    x, ga, gx, dy = (d(rows, C)[0] for _ in range(4))
    conv = cb.CausalConv1dB200(d(C, K)[0], None, "silu")
    rec = cb.GatedRecurrenceB200(d(C, dtype=torch.float32)[0])
    off = dev(offsets)

    def run(x, ga, gx, dy):
        new = lambda: torch.zeros(rows, C, dtype=dtype, device="cuda")  # noqa: E731
        saved = rec.saved_states(x)
        out = [conv(x, y=new(), offsets=off), conv.backward(x, dy, offsets=off, dx=new())[0],
               rec(x, ga, gx, y=new(), offsets=off, saved=saved)]
        out += rec.backward(x, ga, gx, dy, saved, offsets=off, dx=new(), d_gate_a=new(), d_gate_x=new())[:3]
        return out

    clean = run(x, ga, gx, dy)
    for bad in (slice(100, 260), slice(400, 450)):
        spoilt = [t.clone() for t in (x, ga, gx, dy)]
        for t in spoilt:
            t[bad] = poison
        for a, b in zip(clean, run(*spoilt)):
            keep = torch.ones(rows, dtype=torch.bool, device="cuda")
            keep[bad] = False
            assert torch.equal(a[keep], b[keep])
    cb.conv2d_sync_status()


@both
def test_rows_of_no_sequence_leave_the_sums_as_they_are(dtype):
    """NaN behind the last sequence, in every input, and in a window of an empty one: the weights' gradients are the same bits."""
    offsets, rows, C, K = [0, 0, 140, 400], 450, 72, 4
    d = Draw(15, dtype)
    x, ga, gx, dy = (d(rows, C)[0] for _ in range(4))
    conv = cb.CausalConv1dB200(d(C, K)[0], d(C)[0], "silu")
    rec = cb.GatedRecurrenceB200(d(C, dtype=torch.float32)[0])
    window, state, off = d(3, K - 1, C)[0], d(3, C, dtype=torch.float32)[0], dev(offsets)

    def run():
        saved = rec.saved_states(x)
        rec(x, ga, gx, offsets=off, saved=saved, initial_state=state)
        return [*conv.backward(x, dy, offsets=off, initial_state=window)[1:3],
                rec.backward(x, ga, gx, dy, saved, offsets=off, initial_state=state)[3]]

    clean = run()
    for t in (x, ga, gx, dy):
        t[400:] = float("nan")
    window[0], state[0] = float("nan"), float("nan")
    for a, b in zip(clean, run()):
        assert bool(a.isfinite().all()) and torch.equal(a, b)
    cb.conv2d_sync_status()


@both
@pytest.mark.parametrize("offsets", [None, [0, 3, 400, 600]], ids=["dense", "packed"])
@pytest.mark.parametrize("decay", [-3.5, 3.0], ids=["slow", "fast"])
def test_nan_reaches_the_later_rows_of_its_sequence(decay, offsets, dtype):
    """A NaN in any input of a row makes every later state of its sequence NaN, however small the decays' products;
    one in dy every earlier gradient.  Infinities leave no finite state either."""
    d = Draw(12, dtype)
    C, rows, at, first, last = 64, 600, 77, 3 if offsets else 0, 400 if offsets else 600
    x, ga, gx, dy = (d(rows, C)[0] if offsets else d(1, rows, C)[0] for _ in range(4))
    rec, off = cb.GatedRecurrenceB200(torch.full((C,), decay, device="cuda")), dev(offsets)
    flat = lambda t: t.view(rows, C)  # noqa: E731
    for which, bad in [(i, float("nan")) for i in range(3)] + [(0, float("inf"))]:
        t = [v.clone() for v in (x, ga, gx)]
        flat(t[which])[at, 5] = bad
        y = flat(rec(*t, offsets=off))
        assert not bool(y[at:last, 5].isfinite().any())
        if bad != bad:
            assert bool(y[at:last, 5].isnan().all())
        y[at:last, 5] = 0
        assert bool(y.isfinite().all())
    state = torch.zeros(len(offsets) - 1 if offsets else 1, C, device="cuda")
    state[1 if offsets else 0, 5] = float("nan")
    y = flat(rec(x, ga, gx, offsets=off, initial_state=state))
    assert bool(y[first:last, 5].isnan().all())
    y[first:last, 5] = 0
    assert bool(y.isfinite().all())
    saved = rec.saved_states(x)
    rec(x, ga, gx, offsets=off, saved=saved)
    bad = dy.clone()
    flat(bad)[at, 5] = float("nan")
    for g in rec.backward(x, ga, gx, bad, saved, offsets=off)[:3]:
        g = flat(g)
        assert bool(g[first:at + 1, 5].isnan().all())
        g[first:at + 1, 5] = 0
        assert bool(g.isfinite().all())
    cb.conv2d_sync_status()


@both
def test_masked_gates_keep_the_state(dtype):
    """gate_a of the lowest value or -infinity: the row adds nothing, has no gradient, and the state passes."""
    C, T = 64, 200
    d = Draw(7, dtype)
    x, ga, gx, dy = (d(1, T, C)[0] for _ in range(4))
    ga[:, 50:] = float("-inf")
    ga[:, 120:] = torch.finfo(dtype).min
    decay = d(C, dtype=torch.float32)
    rec = cb.GatedRecurrenceB200(decay[0])
    saved = rec.saved_states(x)
    final = torch.zeros(1, C, device="cuda")
    h = rec(x, ga, gx, saved=saved, final_state=final)
    # From row 49 on the exact state is one value; each row is within the recurrence's error of it (and half a step of its type), so
    # a row behind a split of the time axis may differ from the row before it by twice that.  Rows of the second chunk
    # (from 128 on) are reached through decays of exactly 1 and contributions of exactly 0: they are equal.
    wide = [t[0].double().cpu() for t in (x, ga, gx)]
    exact, _, error = ref.recurrence(wide[0][:50], wide[1][:50], wide[2][:50], decay[1], KAPPA, [(0, 50)])
    ref.close(h[0, 49:], exact[49:].expand(T - 49, -1), dtype, error[49:].expand(T - 49, -1), "kept state")
    assert torch.equal(h[:, 128:], h[:, 128:129].expand(-1, T - 128, -1))
    ref.close(final[0], exact[49], torch.float32, error[49], "final state")
    dx, dga, dgx, dd, _ = rec.backward(x, ga, gx, dy, saved)
    for g in (dx, dga, dgx):
        assert bool((g[:, 50:] == 0).all()) and bool(g.isfinite().all())
    assert bool(dd.isfinite().all())


@both
@pytest.mark.parametrize("C, shift", [(64, 0), (64, 1), (63, 0), (66, 2)])
def test_strided_rows_and_unaligned_pointers(C, shift, dtype):
    """Slices of wider rows give the bits that whole tensors give; what lies between them stays."""
    B, T = 2, 150
    d = Draw(8, dtype)
    wide = d(B, T, 5 * C + shift)[0]
    x, ga, gx, dy = (wide[..., shift + i * C:shift + (i + 1) * C] for i in range(4))
    conv, rec = cb.CausalConv1dB200(d(C, 4)[0], d(C)[0], "silu"), cb.GatedRecurrenceB200(d(C, dtype=torch.float32)[0])

    def run(x, ga, gx, dy, new):
        saved = rec.saved_states(x)
        first = [conv(x, y=new(0)), rec(x, ga, gx, y=new(1), saved=saved)]
        return first + [conv.backward(x, dy, dx=new(2))[0]] + list(
            rec.backward(x, ga, gx, dy, saved, dx=new(3), d_gate_a=new(4), d_gate_x=new(5))[:3])

    whole = run(*(t.contiguous() for t in (x, ga, gx, dy)), lambda i: None)
    out = torch.full((B, T, 7 * C + shift), 7.0, dtype=dtype, device="cuda")
    part = run(x, ga, gx, dy, lambda i: out[..., shift + i * C:shift + (i + 1) * C])
    for a, b in zip(whole, part):
        assert torch.equal(a, b)
    assert bool((out[..., 6 * C + shift:] == 7.0).all()) and bool((out[..., :shift] == 7.0).all())
    # one row for every place: a broadcast input (row stride 0)
    one = x[:1, :1].contiguous().expand(1, T, C)
    assert torch.equal(conv(one), conv(one.contiguous()))
    with pytest.raises(ValueError):
        conv(wide[:, ::2, :C].transpose(0, 1))


def test_equal_inputs_give_equal_bits():
    """Long time axes with few channels: the order in which chunks find their carries changes from run to run."""
    d = Draw(9, torch.bfloat16)
    x, ga, gx, dy = (d(1, 20000, 64)[0] for _ in range(4))
    rec, conv = cb.GatedRecurrenceB200(d(64, dtype=torch.float32)[0]), cb.CausalConv1dB200(d(64, 4)[0], d(64)[0])

    def run():
        saved = rec.saved_states(x)
        y = rec(x, ga, gx, saved=saved)
        return [y, *rec.backward(x, ga, gx, dy, saved)[:4], conv(x), *conv.backward(x, dy)[:3]]

    first = run()
    for _ in range(5):
        for a, b in zip(first, run()):
            assert torch.equal(a, b)


def test_streams_and_captured_graphs():
    """Calls on two streams at once, and two captured graphs replayed in turn, share nothing."""
    d = Draw(10, torch.bfloat16)
    layers = [(cb.GatedRecurrenceB200(d(128, dtype=torch.float32)[0]), [d(2, 700, 128)[0] for _ in range(4)]) for _ in range(2)]

    def run(layer, t, stream=None):
        saved = layer.saved_states(t[0])
        y = layer(*t[:3], saved=saved, stream=stream)
        return [y, *layer.backward(*t, saved, stream=stream)[:4]]

    want = [run(*l) for l in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(3):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        got = [run(*l, stream=s) for l, s in zip(layers, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
    graphs, outs = [], []
    for l in layers:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(*l))
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            for u in o:
                u.fill_(7.0)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
    cb.conv2d_sync_status()
    with pytest.raises(ValueError):
        layers[0][0](layers[0][1][0], layers[0][1][1].cpu(), layers[0][1][2])


def test_convolution_on_streams_and_in_captured_graphs():
    """Forward, backward and tokens of two layers at once, eager and replayed, give what they give alone."""
    d = Draw(13, torch.bfloat16)
    offsets = dev([0, 5, 5, 333, 600])
    layers = [(cb.CausalConv1dB200(d(136, K)[0], d(136)[0], "silu"), d(610, 136)[0], d(610, 136)[0], d(4, K - 1, 136)[0])
              for K in (4, 7)]

    def run(layer, x, dy, state, stream=None):
        final, window = torch.zeros_like(state), state.clone()
        out = [layer(x, y=torch.zeros_like(x), offsets=offsets, initial_state=state, final_state=final, stream=stream), final]
        out += layer.backward(x, dy, offsets=offsets, initial_state=state, d_final_state=state, dx=torch.zeros_like(x), stream=stream)
        return out + [layer.step(x[:4], window, stream=stream), window]

    want = [run(*l) for l in layers]
    torch.cuda.synchronize()
    streams, graphs, outs = [torch.cuda.Stream() for _ in layers], [], []
    for l in layers:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(*l))
        graphs.append(g)
    for _ in range(3):
        for s, g in zip(streams, graphs):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        got = []
        for l, s in zip(layers, streams):
            with torch.cuda.stream(s):
                got.append(run(*l))
        torch.cuda.synchronize()
        for a, b, c in zip(want, got, outs):
            assert all(torch.equal(u, v) and torch.equal(u, w) for u, v, w in zip(a, b, c))
    cb.conv2d_sync_status()


def test_many_items_for_every_block():
    """More items than blocks take at once, each kind of copy, packed and dense, twice the same bits and near one another:
    the same rows as one batch and packed differ by the roundings of other chunks only."""
    d = Draw(14, torch.bfloat16)
    B, T, C = 3, 2600, 1024
    x, ga, gx, dy = (d(B, T, C)[0] for _ in range(4))
    rec = cb.GatedRecurrenceB200(d(C, dtype=torch.float32)[0] - 3.5)
    offsets = dev([0, T, 2 * T, 3 * T])
    wide = torch.empty(B, T, C + 1, dtype=torch.bfloat16, device="cuda")    # rows of 2050 bytes: no bulk copies
    wide[..., :C] = x

    def run(x, **kw):
        flat = lambda t: t.reshape(B * T, -1) if kw else t  # noqa: E731
        shaped = x.flatten(0, 1) if kw else x
        saved = rec.saved_states(shaped)
        y = rec(shaped, flat(ga), flat(gx), saved=saved, **kw)
        return [t.reshape(B, T, C) for t in (y, *rec.backward(shaped, flat(ga), flat(gx), flat(dy), saved, **kw)[:3])]

    dense, again, strided, packed = run(x), run(x), run(wide[..., :C]), run(x, offsets=offsets)
    for a, b, c, e in zip(dense, again, strided, packed):
        assert torch.equal(a, b) and torch.equal(a, c)
        # both are within half a step of bf16 of fp32 results that differ by rounding errors, 2^-24 times some hundreds of terms
        size = torch.maximum(a.float().abs(), e.float().abs())
        assert bool(((a.float() - e.float()).abs() <= 2 ** -7 * size + 2 ** -24 * 1000 * a.float().abs().max()).all())
    cb.conv2d_sync_status()


def test_a_carry_that_never_comes_ends_in_a_timeout():
    x = torch.zeros(1, 300, 64, device="cuda")
    rec = cb.GatedRecurrenceB200(torch.zeros(64, device="cuda"))
    try:
        cb.conv2d_debug_set_watchdog(2_000_000, True)   # 2 ms, and no chunk publishes its carry
        rec(x, x, x)
        with pytest.raises(cb.Conv2dError) as err:
            cb.conv2d_sync_status()
        assert err.value.status == cb.CONV_ERR_TIMEOUT
    finally:
        cb.conv2d_debug_set_watchdog(0, False)
    assert bool((rec(x, x, x) == 0).all())
    cb.conv2d_sync_status()


def test_a_block_waits_once_for_carries_that_never_come():
    """Six items for each block, each without its carry: the first wait takes the limit, the others next to nothing."""
    x = torch.zeros(1, 100_000, 64, device="cuda")
    rec = cb.GatedRecurrenceB200(torch.zeros(64, device="cuda"))
    rec(x, x, x)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    try:
        cb.conv2d_debug_set_watchdog(200_000_000, True)   # 200 ms
        begin.record()
        rec(x, x, x)
        end.record()
        with pytest.raises(cb.Conv2dError) as err:
            cb.conv2d_sync_status()
        assert err.value.status == cb.CONV_ERR_TIMEOUT
    finally:
        cb.conv2d_debug_set_watchdog(0, False)
    assert 150 < begin.elapsed_time(end) < 600
    assert bool((rec(x, x, x) == 0).all())
    cb.conv2d_sync_status()


def test_long_offsets_pass_32_bits():
    """Rows whose byte offsets (and element offsets) pass 2^32: a strided view whose last rows lie far out."""
    rows, C, stride = 300, 64, 1 << 24
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of free device memory")
    big = torch.empty(rows * stride, dtype=torch.bfloat16, device="cuda")
    x = big.view(rows, stride)[:, :C]
    d = Draw(11, torch.bfloat16)
    small = d(rows, C)[0]
    x.copy_(small)
    y = big.view(rows, stride)[:, C:2 * C]
    off = dev([0, 200, 300])
    conv, rec = cb.CausalConv1dB200(d(C, 4)[0]), cb.GatedRecurrenceB200(d(C, dtype=torch.float32)[0])
    assert torch.equal(conv(x, y=y, offsets=off), conv(small, offsets=off))
    assert torch.equal(rec(x, x, x, y=y, offsets=off), rec(small, small, small, offsets=off))
    cb.conv2d_sync_status()


@both
def test_tiles_are_read_before_they_are_loaded_again(dtype):
    """Sequences that leave the last chunk of each part empty, many for every block: a tile's last reads are those of its
    rows by themselves, and the loads of a later item into its place wait for them.  Rows of other strides take copies by
    the warps; both give the same bits, run after run."""
    d = Draw(16, dtype)
    B, T, C = 96, 250, 1024     # (chunks of its own for each sequence: of 256 and 2 x 128 rows in bf16, 2 x 128 and 3 x 96 in fp32)
    x, ga, gx, dy = (d(B, T, C)[0] for _ in range(4))
    rec = cb.GatedRecurrenceB200(d(C, dtype=torch.float32)[0] - 3.5)
    state = d(B, C, dtype=torch.float32)[0]
    wide = torch.empty(B, T, C + 1, dtype=dtype, device="cuda")
    wide[..., :C] = x

    def run(x):
        saved, final = rec.saved_states(x), torch.zeros(B, C, device="cuda")
        y = rec(x, ga, gx, initial_state=state, final_state=final, saved=saved)
        return [y, final, *rec.backward(x, ga, gx, dy, saved, initial_state=state, d_final_state=state)]

    want = run(wide[..., :C])
    for _ in range(5):
        for a, b in zip(want, run(x)):
            assert torch.equal(a, b)
    cb.conv2d_sync_status()


@both
@pytest.mark.parametrize("case", [
    (2, 300, None, None, 128, 7, True, True), (3, 130, None, None, 192, 8, False, True), (1, 257, None, None, 72, 5, True, False),
    (4, 0, [0, 5, 5, 300, 333], 340, 64, 8, True, True), (3, 0, [0, 3, 9, 150], None, 130, 6, True, True),
], ids=str)
def test_convolution_with_long_kernels(case, dtype):
    """K of 5 to 8 in rows that travel by bulk copies (channels a multiple of 8), and one whose rows do not in bf16."""
    test_convolution(case, dtype)


@both
def test_masked_gates_across_chunks(dtype):
    """The state passes chunks (of 256 rows at most) of nothing but masked rows unchanged, and so does its gradient."""
    C, T = 64, 700
    d = Draw(17, dtype)
    x, ga, gx, dy = (d(1, T, C) for _ in range(4))
    decay, state = d(C, dtype=torch.float32), d(1, C, dtype=torch.float32)
    for t in ga:
        t[:, 50:] = float("-inf")
    rec = cb.GatedRecurrenceB200(decay[0])
    saved, final = rec.saved_states(x[0]), torch.zeros(1, C, device="cuda")
    h = rec(x[0], ga[0], gx[0], initial_state=state[0], saved=saved, final_state=final)
    dx, dga, dgx, dd, ds = rec.backward(x[0], ga[0], gx[0], dy[0], saved, initial_state=state[0])
    cb.conv2d_sync_status()
    wide = state[1].requires_grad_()
    want, last, error = ref.recurrence(*(t[1][0] for t in (x, ga, gx)), decay[1], KAPPA, [(0, T)], wide)
    ref.close(h[0], want, dtype, error, "y")
    ref.close(final, last, torch.float32, error[-1], "final state")
    # behind the first chunk the decays' products are 1 and what they add is 0: every row has the same bits
    assert torch.equal(h[:, 256:], h[:, 256:257].expand(-1, T - 256, -1))
    for g in (dx, dga, dgx):
        assert bool((g[:, 50:] == 0).all()) and bool(g.isfinite().all())
    assert bool(dd.isfinite().all())
    ref.grad_close(ds, torch.autograd.grad((want * dy[1][0]).sum(), wide)[0], torch.float32, "d_initial_state")
