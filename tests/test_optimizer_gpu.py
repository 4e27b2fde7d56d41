"""AdamW on a B200, and the layers and the optimizer as they are used together: a training step of a
convolution layer and of a sequence block, and the block's tokens after its training.

A weight in fp32 (or its master) is off from the 64-bit step by the roundings of its own value, and by its update's:
2 u |p| + 16 u lr (|m^| / (sqrt(v^) + eps) + decay |p|); u = 2^-24.  m and v: three products and a sum, 4 u of the sum of
their terms' sizes.  bf16 adds half a step, 2^-8 of the value."""
import pytest
import torch

import cnn_convolution_conv2d_b200 as cb
import sequence_reference as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    assert torch.cuda.is_available(), "these tests need a CUDA device"
    from cnn_convolution_conv2d_b200 import build
    build.build()
    cb.load()
    yield
    cb.conv2d_sync_status()


SHAPES = [(64, 3, 7, 7), (1,), (255,), (256,), (257,), (2049,), (0,), (512, 16, 3, 3), (5,)]


def normal(shape, seed, scale=1.0, dtype=F32):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * scale).to(dtype).cuda()


@pytest.mark.parametrize("dtype, master, gtype", [(F32, False, F32), (F32, False, BF), (BF, False, BF), (BF, True, BF), (BF, True, F32)],
                         ids=["f32", "f32-gbf16", "bf16", "master", "master-gf32"])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("copies", [1, 7])     # 63 tensors: more than one launch takes
def test_steps(dtype, master, gtype, bits, copies):
    shapes = SHAPES * copies
    params = [normal(s, i, 0.1, dtype) for i, s in enumerate(shapes)]
    masters = [normal(s, 100 + i, 0.1) for i, s in enumerate(shapes)] if master else None
    opt = cb.AdamWB200(params, lr=1e-2, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.1, state_bits=bits, masters=masters, seed=5)
    scale = torch.tensor([0.5], device="cuda")
    lr, (b1, b2), eps, wd = 1e-2, (0.9, 0.99), 1e-6, 0.1
    for step in (1, 2, 3):
        grads = [normal(s, 1000 * step + i, 1.0, gtype) for i, s in enumerate(shapes)]
        held = lambda i, name: held_state(opt, i, name)  # noqa: E731
        before = [((masters or params)[i].double().cpu().flatten(), held(i, "m"), held(i, "v")) for i in range(len(shapes))]
        opt.step(grads, grad_scale=scale if step == 3 else None)
        for i, (p0, m0, v0) in enumerate(before):
            g = grads[i].double().cpu().flatten() * (0.5 if step == 3 else 1.0)
            p, m, v = ref.adamw(p0, g, m0, v0, lr, b1, b2, eps, wd, step)
            update = (m0.abs() * b1 + g.abs() * (1 - b1)) / (1 - b1 ** step) / ((v / (1 - b2 ** step)).sqrt() + eps)
            atol = 2 * ref.U * p0.abs() + 16 * ref.U * lr * (update + wd * p0.abs())
            if master:
                ref.close(masters[i].flatten(), p, F32, atol, f"master {i}")
                assert torch.equal(masters[i].to(BF), params[i])
            else:
                ref.close(params[i].flatten(), p, dtype, atol, f"weight {i}")
            terms = b1 * m0.abs() + (1 - b1) * g.abs()
            if bits == 32:
                ref.close(opt.exp_avg[i], m, F32, 4 * ref.U * terms, f"m {i}")
                ref.close(opt.exp_avg_sq[i], v, F32, 4 * ref.U * v, f"v {i}")
            else:
                # held between the two codes around the value: less than one step, an eighth of a value in e4m3 and a
                # quarter in e5m2, or one of the equal steps below the smallest normal number
                check_codes(opt, i, m, v, terms)
    cb.conv2d_sync_status()


def held_state(opt, i, name):
    """The values that a tensor's state stands for, in 64 bits."""
    t = (opt.exp_avg if name == "m" else opt.exp_avg_sq)[i].double().cpu()
    if opt.state_bits == 32 or not t.numel():
        return t
    start = (t.data_ptr() * 0 + (opt.exp_avg if name == "m" else opt.exp_avg_sq)[i].storage_offset()) // 256
    scale = opt.flat[name + "_scale"][start:start + -(-t.numel() // 256)].double().cpu()
    return t * scale.repeat_interleave(256)[:t.numel()]


def check_codes(opt, i, m, v, terms):
    for name, value, top, least, rel, sizes in (("m", m, 7, 2.0 ** -9, 2.0 ** -3, terms), ("v", v, 14, 2.0 ** -16, 2.0 ** -2, v)):
        got = held_state(opt, i, name)
        if not got.numel():
            continue
        start = (opt.exp_avg if name == "m" else opt.exp_avg_sq)[i].storage_offset() // 256
        scale = opt.flat[name + "_scale"][start:start + -(-got.numel() // 256)].double().cpu()
        assert bool((torch.log2(scale) == torch.log2(scale).round()).all())
        # the scale is that of the largest fp32 value, which is off by 4 u of its terms (which may cancel: then it says nothing)
        block = lambda t: torch.nn.functional.pad(t.abs(), (0, -t.numel() % 256)).view(-1, 256).amax(1)  # noqa: E731
        big, slack = block(value), 4 * ref.U * block(sizes)
        inside = ((big >= scale * 2.0 ** top - slack) & (big < scale * 2.0 ** (top + 1) + slack)) | (big <= slack)
        assert bool(inside.all()), (name, i)
        wide = scale.repeat_interleave(256)[:got.numel()]
        allowed = torch.maximum(rel * value.abs(), least * wide) * (1 + 1e-6) + 4 * ref.U * sizes
        assert bool(((got - value).abs() <= allowed).all()), (name, i)
        if name == "v":
            assert bool((got[value > 0] > 0).all())


def test_rounding_by_chance_keeps_the_mean():
    """With beta2 = 0.999 a constant gradient moves v by a thousandth a step: rounding to nearest would leave it; by chance
    its mean follows.  v after n steps is 1 - beta2^n; a step of chance is a random move of at most a quarter of v, so the mean
    of N elements is off by less than 6 standard deviations, 6 * 0.25 * sqrt(n / N), of v."""
    N, n = 1 << 16, 400
    p = torch.zeros(N, device="cuda")
    opt = cb.AdamWB200([p], lr=0.0, weight_decay=0.0, state_bits=8, seed=9)
    g = [torch.ones(N, device="cuda")]
    for _ in range(n):
        opt.step(g)
    v = held_state(opt, 0, "v").mean().item()
    want = 1 - 0.999 ** n
    assert abs(v - want) <= 6 * 0.25 * (n / N) ** 0.5 * want
    m = held_state(opt, 0, "m").mean().item()
    assert abs(m - 1) <= 6 * 0.125 * (n / N) ** 0.5


def scrambled(h):
    """The header's mix, of 32-bit numbers held in 64."""
    h = ((h ^ (h >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    h = ((h ^ (h >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


def held_in_8_bits(x, bits, top, small, keep):
    """(values, scales) of fp32 x: the scale brings the largest of 256 into [2^top, 2^(top+1)); then `keep` fraction bits, or steps of
    2^(small-keep) below 2^small, up where the fraction of a step and the 16 random bits in units of 2^-16 come to one."""
    big = torch.nn.functional.pad(x.abs(), (0, -x.numel() % 256)).view(-1, 256).amax(1)
    scale = torch.where(big > 0, 2.0 ** (torch.frexp(big)[1] - 1 - top).double(), torch.ones_like(big).double())
    wide = scale.repeat_interleave(256)[:x.numel()]
    y = x.double() / wide
    size = y.abs()
    step = 2.0 ** ((torch.frexp(size)[1] - 1).clamp(min=small) - keep).double()
    # the fraction counts in units of 2^-16 of a step and below; the bits of an fp32 sum above 2^small hold it
    size = torch.where(size < 2.0 ** small, (size.float() + 2.0 ** small).double() - 2.0 ** small, size)
    held = torch.floor(size / step + bits.double() / 65536) * step
    return torch.copysign(held, y), scale


@pytest.mark.parametrize("gtype", [F32, BF], ids=["f32", "bf16"])
def test_8_bit_states_are_what_the_header_says(gtype):
    """Bit for bit: m and v in fp32, each product and sum rounded by itself, then rounded by the hash of seed, step, place and
    element; more tensors than one launch takes, one of them without elements, sizes that are no multiples of 256."""
    shapes = [(n,) for n in (1, 255, 257, 0, 1000, 2049)] * 9
    params = [normal(s, i) for i, s in enumerate(shapes)]
    b1, b2, seed = 0.9, 0.999, 77
    opt = cb.AdamWB200(params, betas=(b1, b2), state_bits=8, seed=seed)
    one = lambda v: torch.tensor(v, dtype=torch.float64).float()  # noqa: E731
    held = [(torch.zeros(s), torch.zeros(s)) for s in shapes]
    for step in (1, 2, 3):
        # sizes over many binades, so that some values fall below the smallest normal number of a block
        grads = [(normal(s, 100 * step + i) * torch.exp2(normal(s, 500 + i, 4.0))).to(gtype) for i, s in enumerate(shapes)]
        opt.step(grads)
        for i, (g, (m, v)) in enumerate(zip(grads, held)):
            if not g.numel():
                continue
            g = g.float().cpu()
            m = m * one(b1) + g * one(1 - b1)
            v = v * one(b2) + (g * g) * one(1 - b2)
            key = scrambled(torch.tensor((seed + 0x9E3779B9 * step) & 0xFFFFFFFF)) + 0x85EBCA77 * (i + 1)
            h = scrambled((torch.arange(g.numel()) * 0x9E3779B1 + scrambled(key & 0xFFFFFFFF)) & 0xFFFFFFFF)
            hm, scale_m = held_in_8_bits(m, h & 0xFFFF, 7, -6, 3)
            hv, scale_v = held_in_8_bits(v, h >> 16, 14, -14, 2)
            hv = torch.where((v > 0) & (hv == 0), torch.tensor(2.0 ** -16, dtype=torch.float64), hv)
            start, blocks = opt.exp_avg[i].storage_offset() // 256, -(-g.numel() // 256)
            assert torch.equal(opt.flat["m_scale"][start:start + blocks].double().cpu(), scale_m), (step, i)
            assert torch.equal(opt.flat["v_scale"][start:start + blocks].double().cpu(), scale_v), (step, i)
            assert torch.equal(opt.exp_avg[i].double().cpu(), hm), (step, i)
            assert torch.equal(opt.exp_avg_sq[i].double().cpu(), hv), (step, i)
            expand = lambda t: t.repeat_interleave(256)[:g.numel()]  # noqa: E731, B023
            held[i] = (hm * expand(scale_m)).float(), (hv * expand(scale_v)).float()
    cb.conv2d_sync_status()


def test_the_mean_of_rounding_by_chance():
    """A constant gradient, v = 1 - beta2^n.  A step moves v by d = (1 - beta2) (1 - v), less than a code step s <= v / 4 of which it
    is taken whole with the chance d / s: a variance of at most s d.  They add up to less than the sum of v (1 - beta2) / 4; the
    mean of N elements is held to 6 deviations, and to the 2^-16 of a code step by which 16 random bits may round the chance."""
    N, n, beta2 = 1 << 16, 400, 0.999
    p = torch.zeros(N, device="cuda")
    opt = cb.AdamWB200([p], lr=0.0, weight_decay=0.0, state_bits=8, seed=11)
    g = [torch.ones(N, device="cuda")]
    variance = 0.0
    for step in range(1, n + 1):
        opt.step(g)
        variance += (1 - beta2 ** step) / 4 * (1 - beta2)
    want = 1 - beta2 ** n
    v = held_state(opt, 0, "v").mean().item()
    assert abs(v - want) <= 6 * (variance / N) ** 0.5 + n * 2.0 ** -16 * want / 4


def test_equal_seeds_give_equal_bits_and_the_device_counter_the_same_steps():
    def run(seed, device_counter, graph=False):
        params = [normal((300, 40), 1), normal((77,), 2)]
        grads = [normal((300, 40), 3), normal((77,), 4)]
        counter = torch.ones(1, dtype=torch.int64, device="cuda") if device_counter else None
        opt = cb.AdamWB200(params, state_bits=8, seed=seed, step_device=counter)
        if graph:
            opt.step(grads)                     # step 1, and the first launch outside the capture
            counter += 1
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                opt.step(grads)
                counter.add_(1)
            for _ in range(2):
                g.replay()
        else:
            for _ in range(3):
                opt.step(grads)
                if device_counter:
                    counter += 1
        torch.cuda.synchronize()
        return [t.clone() for t in params] + [t.view(torch.uint8).clone() for t in (opt.flat["m"], opt.flat["v"])]

    one, two, other = run(1, False), run(1, False), run(2, False)
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    assert not torch.equal(one[3], other[3])
    assert all(torch.equal(a, b) for a, b in zip(one, run(1, True)))
    assert all(torch.equal(a, b) for a, b in zip(one, run(1, True, graph=True)))


@pytest.mark.parametrize("bits", [32, 8])
def test_what_is_not_finite(bits):
    p = normal((1000,), 1)
    opt = cb.AdamWB200([p], state_bits=bits)
    g = normal((1000,), 2)
    for bad in (0.0, -1.0, float("nan"), float("inf")):      # a scale that is no scale: nothing changes
        kept = p.clone()
        opt.step([g], grad_scale=torch.tensor([bad], device="cuda"))
        assert torch.equal(p, kept) and bool((opt.flat["m"].float() == 0).all())
    clean = cb.AdamWB200([normal((1000,), 1)], state_bits=bits)
    clean.step_count = opt.step_count
    clean.step([g])
    spoilt = g.clone()
    spoilt[300], spoilt[301] = float("nan"), float("inf")
    opt.step([spoilt])
    mask = torch.ones(1000, dtype=torch.bool, device="cuda")
    mask[300:302] = False
    assert bool(p[300:302].isnan().all()) and torch.equal(p[mask], clean.params[0][mask])
    assert bool(opt.exp_avg[0].float()[300:302].isnan().all() if bits == 8 else ~opt.exp_avg[0][300:302].isfinite().any())
    # the spoilt elements leave the scale to the others
    assert torch.equal(opt.exp_avg[0].float()[:256], clean.exp_avg[0].float()[:256])
    assert bool(opt.exp_avg[0].float()[mask].isfinite().all()) and bool(opt.exp_avg_sq[0].float()[mask].isfinite().all())


@pytest.mark.parametrize("bits", [32, 8])
def test_small_gradients_count_without_eps(bits):
    """g near 1e-18, so v near 1e-39, below the smallest normal number: m^ / sqrt(v^) is still 1 in size after one step.
    v's products are off by half a unit of 2^-149 each, 7e-7 of the smallest v here: 2e-6 of the update is wide."""
    p, g = normal((999,), 1, 0.1), (normal((999,), 2).abs() + 1) * 1e-18
    p0 = p.double()
    opt = cb.AdamWB200([p], lr=1e-2, eps=0.0, weight_decay=0.0, state_bits=bits)
    opt.step([g])
    want = p0 - 1e-2
    assert bool(((p.double() - want).abs() <= 2 * ref.U * p0.abs() + 1e-2 * (2e-6 + 16 * ref.U)).all())


def test_a_step_number_below_one_is_reported():
    p = normal((300,), 1)
    kept = p.clone()
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")
    opt = cb.AdamWB200([p], step_device=counter)
    opt.step([normal((300,), 2)])
    with pytest.raises(cb.Conv2dError) as err:
        cb.conv2d_sync_status()
    assert err.value.status == cb.CONV_ERR_INVALID_ARG and "step" in str(err.value)
    assert torch.equal(p, kept) and bool((opt.flat["m"] == 0).all())
    counter += 1
    opt.step([normal((300,), 2)])
    cb.conv2d_sync_status()
    assert not torch.equal(p, kept)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_tensor_without_elements_does_not_choose_the_kernel(bits):
    """Through the C entry: an entry without elements that names master weights, beside weights that have none."""
    p, g = normal((300,), 1, 0.1, BF), normal((300,), 2, 1.0, BF)
    opt, alone = cb.AdamWB200([p, p[:0]], state_bits=bits), cb.AdamWB200([p.clone()], state_bits=bits)
    decoy = torch.full((4,), 7.0, device="cuda")
    opt._table[1].master = decoy.data_ptr()
    opt.step([g, g[:0]])
    alone.step([g])
    assert torch.equal(p, alone.params[0]) and bool((decoy == 7.0).all())
    cb.conv2d_sync_status()


def test_refusals():
    p = [torch.zeros(16, device="cuda"), torch.zeros(16, device="cuda")]
    for bad in (lambda: cb.AdamWB200([p[0], p[0]]), lambda: cb.AdamWB200([p[0], p[0][4:12]]), lambda: cb.AdamWB200(p, state_bits=4),
                lambda: cb.AdamWB200(p, masters=True), lambda: cb.AdamWB200([torch.zeros(4, 4, device="cuda").t()]),
                lambda: cb.AdamWB200(p, step_device=torch.zeros(1, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    opt = cb.AdamWB200(p)
    for bad in ([p[0]], [p[0], torch.zeros(15, device="cuda")], [p[0], torch.zeros(16)], [p[0], torch.zeros(16, device="cuda", dtype=BF)]):
        with pytest.raises(ValueError):
            opt.step(bad)
    with pytest.raises(TypeError):
        cb.AdamWB200([p[0], torch.zeros(4, device="cuda", dtype=BF)])
    with pytest.raises(cb.Conv2dError) as err:
        opt.step(p, lr=-1.0)
    assert err.value.status == cb.CONV_ERR_INVALID_ARG
    assert opt.step_count == 0
    unaligned = cb.AdamWB200([torch.zeros(40, device="cuda")[1:33]])
    with pytest.raises(cb.Conv2dError) as err:
        unaligned.step([p[0].repeat(2)])
    assert err.value.status == cb.CONV_ERR_UNSUPPORTED


@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_works_on_the_memory_of_now(bits):
    """Weights whose data was replaced, other masters, restored states: the step takes them, and leaves the old ones alone."""
    def make():
        params = [normal((300, 7), 1, 0.1, BF), normal((70,), 2, 0.1, BF)]
        return cb.AdamWB200(params, state_bits=bits, masters=True, seed=3)

    grads = [normal((300, 7), 3, 1.0, BF), normal((70,), 4, 1.0, BF)]
    opt, want = make(), make()
    for o in (opt, want):
        o.step(grads)
    old = [opt.params[0].data, opt.masters[1], *opt.flat.values()]      # (alive, so that nothing else gets their memory)
    kept = [t.clone() for t in old]
    opt.params[0].data = opt.params[0].data.clone()
    opt.masters[1] = opt.masters[1].clone()
    opt.flat = {name: t.clone() for name, t in opt.flat.items()}
    for o in (opt, want):
        o.step(grads)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(old, kept))
    for a, b in zip(opt.params + opt.masters + list(opt.flat.values()) + opt.exp_avg + opt.exp_avg_sq,
                    want.params + want.masters + list(want.flat.values()) + want.exp_avg + want.exp_avg_sq):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    good = opt.params[0].data
    for bad, error in ((good[:100].clone(), ValueError), (good.float(), TypeError), (good.t().contiguous().t(), ValueError),
                       (good.cpu(), ValueError)):
        opt.params[0] = bad
        with pytest.raises(error):
            opt.step(grads)
    opt.params[0] = good
    kind = opt.params[0].data
    for other, error in ((kind.view(torch.float16), TypeError), (kind.view(7, 300).t(), ValueError)):     # in the same memory
        assert other.data_ptr() == kind.data_ptr()
        opt.params[0] = other
        with pytest.raises(error):
            opt.step(grads)
    opt.params[0] = kind
    for name, bad in (("m", opt.flat["m"][:256].clone()), ("v", opt.flat["v"].float().half()), ("other", good)):
        flat = opt.flat
        opt.flat = dict(flat, **{name: bad})
        with pytest.raises((ValueError, TypeError)):
            opt.step(grads)
        opt.flat = flat
    assert opt.step_count == 2
    opt.step(grads)
    cb.conv2d_sync_status()


def test_training_a_convolution_layer():
    """Forward, backward, AdamW and again: the layer's own gradients update the weights it packs."""
    w, b = normal((16, 8, 3, 3), 1, 0.1), normal((16,), 2, 0.1)
    x, dy = normal((2, 8, 9, 9), 3), normal((2, 16, 9, 9), 4)
    layer = cb.Conv2dB200(w, b, pad=1, layout="nchw")
    opt = cb.AdamWB200([w, b], lr=1e-2)
    dx0 = layer.backward_data(dy, 9, 9)
    dw, db = layer.backward_weight(x, dy)
    before = [t.double().cpu().flatten() for t in (w, b, dw, db)]
    opt.step([dw, db])
    for t, p, g in ((w, before[0], before[2]), (b, before[1], before[3])):
        want, _, _ = ref.adamw(p, g, 0 * g, 0 * g, 1e-2, 0.9, 0.999, 1e-8, 1e-2, 1)
        ref.close(t.flatten(), want, F32, 2 * ref.U * p.abs() + 16 * ref.U * 1e-2 * (1 + 1e-2 * p.abs()))
    layer.repack()
    fresh = cb.Conv2dB200(w.clone(), b.clone(), pad=1, layout="nchw")
    assert torch.equal(layer(x), fresh(x))
    dx1 = layer.backward_data(dy, 9, 9)
    assert torch.equal(dx1, fresh.backward_data(dy, 9, 9)) and not torch.equal(dx0, dx1)
    cb.conv2d_sync_status()


@pytest.mark.parametrize("other_stream", [False, True], ids=["current", "other"])
@pytest.mark.parametrize("which", ["channels_last", "slice", "transposed", "contiguous"])
def test_repacking_follows_the_callers_tensors(which, other_stream):
    """Weights that are not contiguous and a bias of another dtype, updated in place: the layer's copies are made again."""
    make = {"channels_last": lambda: normal((16, 8, 3, 3), 1, 0.1, BF).to(memory_format=torch.channels_last),
            "slice": lambda: normal((16, 20, 3, 3), 1, 0.1, BF)[:, 4:12],
            "transposed": lambda: normal((8, 16, 3, 3), 1, 0.1, BF).transpose(0, 1), "contiguous": lambda: normal((16, 8, 3, 3), 1, 0.1, BF)}
    w, b = make[which](), normal((16,), 2, 0.1)
    x, dy = normal((2, 8, 9, 9), 3, 1.0, BF), normal((2, 16, 9, 9), 4, 1.0, BF)
    layer = cb.Conv2dB200(w, b, pad=1, layout="nchw")
    for step in range(2):       # without and with the transposed kernel, which the first backward pass packs
        before = layer(x)
        w.mul_(-0.5)
        b.add_(1.0)
        stream = torch.cuda.Stream() if other_stream else None
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        layer.repack(stream=stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        fresh = cb.Conv2dB200(w.clone().contiguous(), b.to(BF), pad=1, layout="nchw")
        assert torch.equal(layer(x), fresh(x)) and not torch.equal(layer(x), before), step
        assert torch.equal(layer.backward_data(dy, 9, 9), fresh.backward_data(dy, 9, 9)), step
    cb.conv2d_sync_status()


def test_repacking_refuses_a_weight_of_another_size_or_type():
    w, x = normal((16, 8, 3, 3), 1, 0.1), normal((2, 8, 9, 9), 3)
    layer = cb.Conv2dB200(w, None, pad=1, layout="nchw")
    good, y = w.data, layer(x)
    for bad in (normal((32, 8, 3, 3), 1), normal((16, 8, 5, 5), 1), normal((16, 8, 3, 3), 1, 0.1, BF)):
        w.data = bad
        with pytest.raises(ValueError):
            layer.repack()
    w.data = good.clone()
    layer.repack()
    assert torch.equal(layer(x), y)


def test_a_sequence_block_from_training_to_tokens():
    """Convolution, recurrence, their gradients and AdamW as a training step uses them, on packed sequences; then a prompt
    and single tokens with the trained weights, against one pass over all of it."""
    C, K, off = 96, 4, [0, 70, 70, 300]
    x, dh = normal((300, C), 1), normal((300, C), 2)
    gates = normal((300, 2 * C), 3)
    w, b, decay = normal((C, K), 4, 0.5), normal((C,), 5), normal((C,), 6) - 3
    conv, rec = cb.CausalConv1dB200(w, b, "silu"), cb.GatedRecurrenceB200(decay)
    opt = cb.AdamWB200([w, b, decay], lr=1e-2, state_bits=32)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    ga, gx = gates[:, :C], gates[:, C:]
    wide = [t.double().cpu().requires_grad_() for t in (w, b, decay)]
    for step in (1, 2):
        y = conv(x, offsets=offsets)
        saved = rec.saved_states(y)
        rec(y, ga, gx, offsets=offsets, saved=saved)
        dy, _, _, ddecay, _ = rec.backward(y, ga, gx, dh, saved, offsets=offsets)
        _, dw, db, _ = conv.backward(x, dy, offsets=offsets)
        wide = [t.double().cpu().requires_grad_() for t in (w, b, decay)]
        seqs = ref.pieces(x.shape, off)
        yy, _, _ = ref.conv1d(x.double().cpu(), wide[0], wide[1], True, seqs)
        hh, _, _ = ref.recurrence(yy, ga.double().cpu(), gx.double().cpu(), wide[2], 8.0, seqs)
        wanted = torch.autograd.grad((hh * dh.double().cpu()).sum(), wide)
        for name, got, want in zip(("dw", "db", "ddecay"), (dw, db, ddecay), wanted):
            # two operators in a row: twice the bar of one
            ref.close(got, want, F32, 2 * ref.GRAD * want.abs().max().item(), name)
        opt.step([dw, db, ddecay])
    # the layers read the updated weights: a prompt of 50 rows each, then one token at a time
    xs, gs = normal((2, 60, C), 7), normal((2, 60, 2 * C), 8)
    whole = rec(conv(xs), gs[..., :C], gs[..., C:])
    window, state = torch.zeros(2, K - 1, C, device="cuda"), torch.zeros(2, C, device="cuda")
    y = conv(xs[:, :50].contiguous(), final_state=window)
    rec(y, gs[:, :50, :C].contiguous(), gs[:, :50, C:].contiguous(), final_state=state)
    for t in range(50, 60):
        y = conv.step(xs[:, t], window)
        h = rec.step(y, gs[:, t, :C], gs[:, t, C:], state)
        scale = whole[:, t].abs().max().item()
        ref.close(h, whole[:, t].double().cpu(), F32, ref.GRAD * scale, f"token {t}")
    cb.conv2d_sync_status()
