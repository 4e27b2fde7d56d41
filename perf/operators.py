"""Cases, plain forms and exact values of the sequence operators and of the weight update.

Three operators, each with the calls that a program makes of it:

- ``conv``: the causal depthwise convolution over time (``CausalConv1dB200``): forward over whole
  or packed sequences, forward + backward, and one token for each of a batch of sequences;
- ``rec``: the gated linear recurrence (``GatedRecurrenceB200``): the same three;
- ``adamw``: one AdamW step over many tensors (``AdamWB200``), states in 32 or 8 bits.

``run`` computes the plain form with elementary torch operations where ``own`` is false, and makes
the framework's calls where it is true."""
import math
import random

import torch

own = False

KAPPA = 8.0
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
LR, BETA1, BETA2, EPS, DECAY = 1e-3, 0.9, 0.999, 1e-8, 0.01
QBLOCK = 256       # elements of one scale of an 8-bit state
STEP = 100         # steps already taken when a case begins


# ------------------------------------------------------------------- cases ---
def listed():
    return [
        # a prompt batch of ragged sequences, packed one behind the other, the first layer of a sequence block
        {"name": "conv_prefill_packed_bf16", "op": "conv", "mode": "forward", "dtype": "bf16", "B": 12, "T": 16384, "packed": True,
         "C": 4096, "K": 4, "silu": True, "carry": False},
        # a training step of that layer
        {"name": "conv_train_bf16", "op": "conv", "mode": "train", "dtype": "bf16", "B": 4, "T": 4096, "packed": False,
         "C": 4096, "K": 4, "silu": True, "carry": False},
        # fp32, odd length and width, no activation, continued from carried windows (truncated backpropagation)
        {"name": "conv_train_odd_f32", "op": "conv", "mode": "train", "dtype": "f32", "B": 3, "T": 1021, "packed": False,
         "C": 1000, "K": 3, "silu": False, "carry": True},
        # one decoded token for each of 64 running sequences, their windows in slots of a larger pool
        {"name": "conv_step_bf16", "op": "conv", "mode": "step", "dtype": "bf16", "B": 64, "T": 1, "packed": False,
         "C": 4096, "K": 4, "silu": True, "carry": True},
        # one long document: few channels in flight, so the time axis has to be split
        {"name": "rec_prefill_long_bf16", "op": "rec", "mode": "forward", "dtype": "bf16", "B": 1, "T": 32768, "packed": False,
         "C": 2048, "K": 0, "silu": False, "carry": False},
        # ragged prompts continued from cached states, packed
        {"name": "rec_prefill_packed_bf16", "op": "rec", "mode": "forward", "dtype": "bf16", "B": 12, "T": 16384, "packed": True,
         "C": 2560, "K": 0, "silu": False, "carry": True},
        # a training step
        {"name": "rec_train_bf16", "op": "rec", "mode": "train", "dtype": "bf16", "B": 4, "T": 4096, "packed": False,
         "C": 4096, "K": 0, "silu": False, "carry": False},
        # fp32, odd length and width, with gradients of the carried state
        {"name": "rec_train_odd_f32", "op": "rec", "mode": "train", "dtype": "f32", "B": 3, "T": 777, "packed": False,
         "C": 1001, "K": 0, "silu": False, "carry": True},
        # one decoded token of one sequence: the smallest call
        {"name": "rec_step_one_bf16", "op": "rec", "mode": "step", "dtype": "bf16", "B": 1, "T": 1, "packed": False,
         "C": 2048, "K": 0, "silu": False, "carry": True},
        # the weights and biases of this repository's benchmark layers, fp32
        {"name": "adamw_conv_layers_f32", "op": "adamw", "dtype": "f32", "master": False, "bits": 32, "layers": 0, "width": 0},
        # a stack of blocks trained in bf16 with fp32 master weights
        {"name": "adamw_blocks_master", "op": "adamw", "dtype": "bf16", "master": True, "bits": 32, "layers": 6, "width": 2048},
        # the same in little memory: bf16 weights, 8-bit states
        {"name": "adamw_blocks_8bit", "op": "adamw", "dtype": "bf16", "master": False, "bits": 8, "layers": 6, "width": 2048},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["conv", "conv", "rec", "rec", "adamw"])
    if op == "adamw":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        return {"op": op, "dtype": dtype, "master": dtype == "bf16" and rng.random() < 0.5, "bits": rng.choice([8, 32]),
                "layers": rng.randint(1, 6), "width": _log_int(rng, 32, 2048)}
    mode = rng.choice(["forward", "train", "train", "step"])
    C = _log_int(rng, 33, 4096)
    C = C if rng.random() < 0.3 else max(8, C // 8 * 8)
    B = _log_int(rng, 1, 256) if mode == "step" else _log_int(rng, 1, 16)
    if mode == "step":
        T = 1
    else:
        T = _log_int(rng, 1, max(1, min(32768, (60_000_000 if mode == "forward" else 30_000_000) // (B * C))))
    packed = mode != "step" and rng.random() < 0.5
    return {"op": op, "mode": mode, "dtype": rng.choice(["bf16", "bf16", "f32"]), "B": B, "T": B * T if packed else T, "packed": packed,
            "C": C, "K": rng.randint(2, 8) if op == "conv" else 0, "silu": op == "conv" and rng.random() < 0.6,
            "carry": mode == "step" or rng.random() < 0.5}


def _lengths(case):
    """Lengths of the packed sequences (T rows in all): uneven ones, some of them empty."""
    rng = random.Random(case["B"] * 7919 + case["T"])
    cuts = sorted(rng.randint(0, case["T"]) for _ in range(case["B"] - 1))
    if case["B"] > 3:
        cuts[1] = cuts[0]      # an empty sequence
    return [b - a for a, b in zip([0] + cuts, cuts + [case["T"]])]


def _shapes(case):
    """The tensors of an adamw case."""
    if case["layers"] == 0:    # the weights (OIHW) and biases of this repository's benchmark layers
        return [(64, 3, 7, 7), (64,), (256, 256, 3, 3), (1024, 256, 1, 1), (1024,), (512, 16, 3, 3), (512,), (512, 512, 7, 7), (512,)]
    w = case["width"]
    return [s for _ in range(case["layers"]) for s in ((w,), (2 * w, w), (w, 4), (w,), (w, w + 1), (w, w), (w,))]


def _numel(shape):
    return math.prod(shape)


# ----------------------------------------------------------------- prepare ---
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    if case["op"] == "adamw":
        return _prepare_adamw(case, normal, gen)
    C, B, mode = case["C"], case["B"], case["mode"]
    packed = case["packed"]
    shape = (B, C) if mode == "step" else (case["T"], C) if packed else (B, case["T"], C)
    s = {"case": case, "x": normal(*shape), "offsets": None}
    if packed:
        ends = [0]
        for n in _lengths(case):
            ends.append(ends[-1] + n)
        s["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    if mode == "step":         # the running sequences' states lie in slots of a larger pool
        s["slots"] = torch.randperm(B + B // 2 + 1, generator=gen, device="cuda")[:B].to(torch.int32)
    pool = B + B // 2 + 1 if mode == "step" else B
    if case["op"] == "conv":
        K = case["K"]
        s["w"] = normal(C, K, scale=1 / math.sqrt(K))
        s["bias"] = normal(C, scale=0.1)
        s["state"] = normal(pool, K - 1, C) if case["carry"] else None
        s["final"] = torch.zeros(pool, K - 1, C, dtype=dt, device="cuda")
        if mode == "train":
            s["dy"] = normal(*shape)
            s["dfinal"] = normal(pool, K - 1, C) if case["carry"] else None
        if own:
            import cnn_convolution_conv2d_b200 as cb
            s["layer"] = cb.CausalConv1dB200(s["w"], s["bias"], "silu" if case["silu"] else None)
    else:
        # the two gates come from one projection of x: rows of 2C, a gate's rows are strided
        s["gates"] = normal(*shape[:-1], 2 * C)
        s["gate_a"], s["gate_x"] = s["gates"][..., :C], s["gates"][..., C:]
        u = torch.rand(C, generator=gen, device="cuda") * 0.099 + 0.9
        s["decay"] = torch.log(torch.expm1(-torch.log(u)))   # softplus(decay) = -log(u)
        s["state"] = normal(pool, C, dtype=torch.float32) if case["carry"] else None
        s["final"] = torch.zeros(pool, C, dtype=torch.float32, device="cuda")
        if mode == "train":
            s["dy"] = normal(*shape)
            s["dfinal"] = normal(pool, C, dtype=torch.float32) if case["carry"] else None
        if own:
            import cnn_convolution_conv2d_b200 as cb
            s["layer"] = cb.GatedRecurrenceB200(s["decay"], KAPPA)
    return s


def _views(flat, case):
    """The tensors of a case in one buffer, each at a multiple of QBLOCK elements."""
    out, at = [], 0
    for shape in _shapes(case):
        out.append(flat[at:at + _numel(shape)].view(shape))
        at += -(-_numel(shape) // QBLOCK) * QBLOCK
    return out


def _prepare_adamw(case, normal, gen):
    dt = DTYPES[case["dtype"]]
    sizes = [_numel(s) for s in _shapes(case)]
    total = sum(-(-n // QBLOCK) * QBLOCK for n in sizes)
    # the elements behind a tensor's end, up to the next multiple of QBLOCK, belong to none
    inside = torch.zeros(total, dtype=torch.bool, device="cuda")
    for view in _views(inside, case):
        view.fill_(True)
    weight = normal(total, scale=0.02, dtype=torch.float32) * inside
    grad = (normal(total, scale=1e-3, dtype=torch.float32) * inside).to(dt)
    m = normal(total, scale=2e-4, dtype=torch.float32) * inside
    v = (torch.rand(total, generator=gen, device="cuda") * 1e-6 + 1e-8) * (1 - BETA2 ** STEP) * inside
    s = {"case": case, "p": weight.to(dt), "grad": grad, "scale": torch.full((1,), 0.7, device="cuda"), "seed": 1234,
         "step": STEP, "master": weight if case["master"] else None, "sizes": sizes}
    if case["bits"] == 8:
        # states as earlier steps left them: held in 8 bits with a power of two for each block
        for name, value, top, kind in (("m", m, 7, torch.float8_e4m3fn), ("v", v, 14, torch.float8_e5m2)):
            scale = _block_scale(value, top)
            s[name + "_scale"] = scale
            s[name] = (value.view(-1, QBLOCK) / scale[:, None]).to(kind).view(-1)
    else:
        s["m"], s["v"] = m, v
    if own:
        import cnn_convolution_conv2d_b200 as cb
        opt = cb.AdamWB200(_views(s["p"], case), lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY, state_bits=case["bits"],
                           masters=_views(weight, case) if case["master"] else None, seed=s["seed"])
        for name in ("m", "v") + (("m_scale", "v_scale") if case["bits"] == 8 else ()):
            opt.flat[name].copy_(s[name])
            s[name] = opt.flat[name]
        opt.step_count = STEP
        s["opt"], s["grads"] = opt, _views(grad, case)
    return s


def _block_scale(x, top):
    """A power of two for each QBLOCK elements: it brings the largest of them into [2^top, 2^(top+1))."""
    big = x.view(-1, QBLOCK).abs().amax(1)
    exponent = (big.view(torch.int32) >> 23).clamp(min=top + 1)      # biased; also keeps the scale a normal number
    scale = ((exponent - top) << 23).view(torch.float32)
    return torch.where(big > 0, scale, torch.ones_like(scale))


# --------------------------------------------------------------------- run ---
def run(s):
    case = s["case"]
    if case["op"] == "adamw":
        return _adamw_own(s) if own else _adamw_plain(s)
    if own:
        return _own(s)
    return (_conv_plain if case["op"] == "conv" else _rec_plain)(s)


def _own(s):
    case, layer = s["case"], s["layer"]
    gates = (s["gate_a"], s["gate_x"]) if case["op"] == "rec" else ()
    if case["mode"] == "step":
        y = layer.step(s["x"], *gates, s["state"], slots=s["slots"])
        return {"y": y, "state": s["state"]}
    if case["mode"] == "forward":
        y = layer(s["x"], *gates, offsets=s["offsets"], initial_state=s["state"], final_state=s["final"])
        return {"y": y, "final": s["final"]}
    if case["op"] == "conv":
        y = layer(s["x"], offsets=s["offsets"], initial_state=s["state"], final_state=s["final"])
        dx, dw, db, dstate = layer.backward(s["x"], s["dy"], offsets=s["offsets"], initial_state=s["state"],
                                            d_final_state=s["dfinal"])
        return {"y": y, "final": s["final"], "dx": dx, "dw": dw, "db": db, "dstate": dstate}
    saved = layer.saved_states(s["x"])
    y = layer(s["x"], *gates, offsets=s["offsets"], initial_state=s["state"], final_state=s["final"], saved=saved)
    dx, da, dg, ddecay, dstate = layer.backward(s["x"], *gates, s["dy"], saved, offsets=s["offsets"], initial_state=s["state"],
                                                d_final_state=s["dfinal"])
    return {"y": y, "final": s["final"], "dx": dx, "dgate_a": da, "dgate_x": dg, "ddecay": ddecay, "dstate": dstate}


def _adamw_own(s):
    s["opt"].step(s["grads"], grad_scale=s["scale"])
    return {k: s[k] for k in ("p", "master", "m", "v", "m_scale", "v_scale") if s.get(k) is not None}


def _rows(s, shape_rows):
    """For every row: its sequence, its place there, and how many rows follow in the sequence."""
    case = s["case"]
    row = torch.arange(shape_rows, device="cuda")
    if case["packed"]:
        off = s["offsets"].long()
        seq = torch.searchsorted(off, row, right=True) - 1
        return seq, row - off[seq], off[seq + 1] - 1 - row
    return row // case["T"], row % case["T"], case["T"] - 1 - row % case["T"]


def _ends(s):
    """First row and length of each sequence."""
    case = s["case"]
    if case["packed"]:
        off = s["offsets"].long()
        return off[:-1], off[1:] - off[:-1]
    first = torch.arange(case["B"], device="cuda") * case["T"]
    return first, torch.full_like(first, case["T"])


def _earlier(x, k, state, seq, at):
    """x k rows earlier in its sequence; before the beginning the carried window's rows, or zeros."""
    if k == 0:
        return x
    back = torch.zeros_like(x)
    back[k:] = x[:-k]
    before = torch.zeros_like(x) if state is None else state[seq, (at - k + state.shape[1]).clamp(0, state.shape[1] - 1)]
    return torch.where((at >= k)[:, None], back, before)


def _sigmoid(z):
    return 1 / (1 + torch.exp(-z))


def _conv_plain(s):
    case = s["case"]
    C, K, dt = case["C"], case["K"], s["x"].dtype
    w, bias = s["w"].float(), s["bias"].float()
    if case["mode"] == "step":
        slots = s["slots"].long()
        window = torch.cat([s["state"][slots].float(), s["x"].float()[:, None]], 1)       # (B, K, C)
        z = (window * w.t()[None]).sum(1) + bias
        s["state"][slots] = window[:, 1:].to(dt)
        return {"y": (z * _sigmoid(z) if case["silu"] else z).to(dt), "state": s["state"]}
    x = s["x"].reshape(-1, C).float()
    seq, at, left = _rows(s, x.shape[0])
    first, length = _ends(s)
    state = None if s["state"] is None else s["state"].float()
    z = bias.expand_as(x)
    for k in range(K):
        z = z + _earlier(x, K - 1 - k, state, seq, at) * w[:, k]
    y = z * _sigmoid(z) if case["silu"] else z
    # the last K-1 rows of (window, x): for short sequences rows of the window itself
    place = length[:, None] - (K - 1) + torch.arange(K - 1, device="cuda")                # (B, K-1), negative: in the window
    here = x[(first[:, None] + place).clamp(0, max(0, x.shape[0] - 1))]
    if state is not None:
        old = torch.gather(state, 1, (place + K - 1).clamp(0, K - 2)[..., None].expand(-1, -1, C))
    else:
        old = torch.zeros_like(here)
    final = torch.where((place >= 0)[..., None], here, old)
    s["final"].copy_(final)
    out = {"y": y.to(dt).view(s["x"].shape), "final": s["final"]}
    if case["mode"] == "forward":
        return out
    dy = s["dy"].reshape(-1, C).float()
    dz = dy
    if case["silu"]:
        sig = _sigmoid(z)
        dz = dy * sig * (1 + z * (1 - sig))
    dx = torch.zeros_like(x)
    dw = torch.empty(C, K, device="cuda")
    dstate = None if state is None else torch.zeros_like(state)
    for k in range(K):
        j = K - 1 - k
        dw[:, k] = (dz * _earlier(x, j, state, seq, at)).sum(0, dtype=torch.float64)
        later = torch.zeros_like(dz)
        later[:dz.shape[0] - j] = dz[j:]
        dx = dx + torch.where((left >= j)[:, None], later, torch.zeros_like(later)) * w[:, k]
        if dstate is not None and j:
            # window row q (q - (K-1) rows before the first) meets tap k at row q - k
            q = torch.arange(k, K - 1, device="cuda")
            use = (q - k)[None] < length[:, None]
            got = dz[(first[:, None] + (q - k)[None]).clamp(0, max(0, x.shape[0] - 1))] * w[:, k]
            dstate[:, k:K - 1] += torch.where(use[..., None], got, torch.zeros_like(got))
    if s["dfinal"] is not None:
        df = s["dfinal"].float()
        dx.index_put_(((first[:, None] + place)[place >= 0],), df[place >= 0], accumulate=True)
        grid = torch.arange(case["B"], device="cuda")[:, None].expand_as(place)
        dstate.index_put_((grid[place < 0], (place + K - 1)[place < 0]), df[place < 0], accumulate=True)
    out.update(dx=dx.to(dt).view(s["x"].shape), dw=dw.to(dt), db=dz.sum(0, dtype=torch.float64).to(dt),
               dstate=None if dstate is None else dstate.to(dt))
    return out


def _scan(a, b):
    """h[t] = a[t] h[t-1] + b[t] over the rows, by doubling the distance: log2(rows) passes over the data."""
    a, b, d = a.clone(), b.clone(), 1
    while d < a.shape[0]:
        b[d:] = b[d:] + a[d:] * b[:-d].clone()
        a[d:] = a[d:] * a[:-d].clone()
        d *= 2
    return b


def _rec_plain(s):
    case = s["case"]
    C, dt = case["C"], s["x"].dtype
    x, ga, gx = (s[k].reshape(-1, C).float() for k in ("x", "gate_a", "gate_x"))
    rate = KAPPA * torch.log1p(torch.exp(s["decay"]))
    ra, rx = _sigmoid(ga), _sigmoid(gx)
    la = -rate * ra
    a, beta = torch.exp(la), torch.sqrt(-torch.expm1(2 * la))
    b = beta * rx * x
    if case["mode"] == "step":
        slots = s["slots"].long()
        h = a * s["state"][slots] + b
        s["state"][slots] = h
        return {"y": h.to(dt), "state": s["state"]}
    seq, at, left = _rows(s, x.shape[0])
    first, length = _ends(s)
    begins, ends = (at == 0)[:, None], (left == 0)[:, None]
    zero = torch.zeros((), device="cuda")
    before = zero if s["state"] is None else s["state"][seq]
    h = _scan(torch.where(begins, zero, a), torch.where(begins, b + a * before, b))
    last = h[(first + length - 1).clamp(0, x.shape[0] - 1)]
    s["final"].copy_(torch.where((length > 0)[:, None], last, zero if s["state"] is None else s["state"]))
    out = {"y": h.to(dt).view(s["x"].shape), "final": s["final"]}
    if case["mode"] == "forward":
        return out
    earlier = torch.zeros_like(h)
    earlier[1:] = h[:-1]
    earlier = torch.where(begins, before, earlier)
    dy = s["dy"].reshape(-1, C).float()
    if s["dfinal"] is not None:
        dy = torch.where(ends, dy + s["dfinal"][seq], dy)
    later = torch.zeros_like(a)
    later[:-1] = a[1:]
    g = _scan(torch.where(ends, zero, later).flip(0), dy.flip(0)).flip(0)
    dla = a * g * (earlier - a * rx * x / beta)
    dstate = None
    if s["state"] is not None:
        start = (a * g)[first.clamp(0, x.shape[0] - 1)]
        kept = zero if s["dfinal"] is None else s["dfinal"]
        dstate = torch.where((length > 0)[:, None], start, kept)
    ddecay = -KAPPA * _sigmoid(s["decay"]) * (dla * ra).sum(0, dtype=torch.float64)
    out.update(dx=(g * beta * rx).to(dt).view(s["x"].shape), dgate_a=(la * dla * (1 - ra)).to(dt).view(s["x"].shape),
               dgate_x=(g * beta * x * rx * (1 - rx)).to(dt).view(s["x"].shape), ddecay=ddecay.float(), dstate=dstate)
    return out


def _mix(h):
    """Scrambles 32-bit whole numbers held in 64 (Appleby's public-domain finaliser)."""
    h = ((h ^ (h >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    h = ((h ^ (h >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _round_random(x, bits, kind, smallest, keep):
    """x rounded up or down to 8 bits by chance: `bits` are 16 random ones, `smallest` the exponent of the smallest normal
    number of `kind`, `keep` the fraction bits it has."""
    size = x.abs()
    lift = torch.where(size < 2.0 ** smallest, 2.0 ** smallest, 0.0)    # below it the steps stay equal
    low = 23 - keep
    whole = (size + lift).view(torch.int32) + (bits << (low - 16)).int()
    size = (whole >> low << low).view(torch.float32) - lift
    return torch.copysign(size, x).to(kind)


def _adamw_plain(s):
    case = s["case"]
    eight = case["bits"] == 8
    s["step"] += 1
    step = s["step"]
    g = s["grad"].float() * s["scale"]
    m, v = s["m"].float(), s["v"].float()
    if eight:
        m = (m.view(-1, QBLOCK) * s["m_scale"][:, None]).view(-1)
        v = (v.view(-1, QBLOCK) * s["v_scale"][:, None]).view(-1)
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + (g * g) * (1 - BETA2)
    p = s["p"].float() if s["master"] is None else s["master"]
    p = p * (1 - LR * DECAY) - (LR / (1 - BETA1 ** step)) * m / (torch.sqrt(v / (1 - BETA2 ** step)) + EPS)
    if s["master"] is not None:
        s["master"].copy_(p)
    s["p"].copy_(p)
    if eight:
        # one 32-bit hash for each element, from the seed, the step, the tensor and the element's place
        size = torch.tensor(s["sizes"], device="cuda")
        room = (size + QBLOCK - 1) // QBLOCK * QBLOCK
        total = s["p"].shape[0]
        which = torch.repeat_interleave(torch.arange(len(size), device="cuda"), room, output_size=total)
        place = torch.arange(total, device="cuda") - (torch.cumsum(room, 0) - room)[which]
        key = _mix((_mix(torch.tensor((s["seed"] + 0x9E3779B9 * step) & 0xFFFFFFFF, device="cuda")) + 0x85EBCA77 * (which + 1)) & 0xFFFFFFFF)
        h = _mix((place * 0x9E3779B1 + key) & 0xFFFFFFFF)
        for name, x, top, kind, smallest, keep, bits in (("m", m, 7, torch.float8_e4m3fn, -6, 3, h & 0xFFFF),
                                                         ("v", v, 14, torch.float8_e5m2, -14, 2, h >> 16)):
            scale = _block_scale(x, top)
            code = _round_random((x.view(-1, QBLOCK) / scale[:, None]).view(-1), bits, kind, smallest, keep)
            if name == "v":    # a second moment above zero is held above zero
                code = torch.where((x > 0) & (code.float() == 0), torch.tensor(2.0 ** -16, device="cuda").to(kind).float(), code.float()).to(kind)
            s[name].copy_(code)
            s[name + "_scale"].copy_(scale)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return {k: s[k] for k in ("p", "master", "m", "v", "m_scale", "v_scale") if s.get(k) is not None}


# -------------------------------------------------------------------- work ---
def work(case):
    s = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "adamw":
        n = sum(_numel(x) for x in _shapes(case))
        weight = s + s if not case["master"] else s + 8
        state = 4 * (1 + 1 / 64 * 2) if case["bits"] == 8 else 16
        return {"bytes": n * (s + weight + state), "flops": n * 16}
    C, B = case["C"], case["B"]
    rows = B if case["mode"] == "step" else case["T"] if case["packed"] else B * case["T"]
    n = rows * C
    if case["op"] == "conv":
        K = case["K"]
        weights = (K + 1) * C * s
        window = B * (K - 1) * C * s
        fwd = {"bytes": 2 * n * s + weights + window * (2 if case["carry"] else 1), "flops": n * (2 * K + (5 if case["silu"] else 0))}
        if case["mode"] != "train":
            return fwd
        return {"bytes": fwd["bytes"] + 3 * n * s + 2 * weights + (3 * window if case["carry"] else 0),
                "flops": fwd["flops"] + n * (6 * K + (12 if case["silu"] else 0))}
    window = B * C * 4
    fwd = {"bytes": 4 * n * s + 4 * C + window * (2 if case["carry"] else 1), "flops": n * 24}
    if case["mode"] != "train":
        return fwd
    return {"bytes": fwd["bytes"] + 7 * n * s + 8 * C + (3 * window if case["carry"] else 0), "flops": fwd["flops"] + n * 48}


# ------------------------------------------------------------------- exact ---
def exact(case, seed):
    """The outputs from the definitions, in 64 bits: one sequence after the other, one row after the other."""
    global own
    if case["op"] == "rec" and (case["T"] if case["packed"] else case["B"] * case["T"]) > 300_000:
        return None        # row after row, this would take too long
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    with torch.no_grad():
        return {"adamw": _adamw_exact, "conv": _conv_exact, "rec": _rec_exact}[case["op"]](s)


def _pieces(s):
    """(sequence, rows) of each sequence that has rows; rows index the flattened input."""
    case = s["case"]
    lengths = _lengths(case) if case["packed"] else [case["T"]] * case["B"]
    at = 0
    for b, n in enumerate(lengths):
        yield b, slice(at, at + n), n
        at += n


def _conv_exact(s):
    case = s["case"]
    C, K = case["C"], case["K"]
    w, bias = s["w"].double(), s["bias"].double()
    kernel = w[:, None]                                            # (C, 1, K): a grouped correlation

    def act(z):
        return z * torch.special.expit(z) if case["silu"] else z

    if case["mode"] == "step":
        state, y = s["state"].double().clone(), []
        for b, slot in enumerate(s["slots"].tolist()):
            window = torch.cat([state[slot], s["x"][b:b + 1].double()])
            y.append(act((window.t() * w).sum(1) + bias))
            state[slot] = window[1:]
        return {"y": torch.stack(y), "state": state}
    x = s["x"].reshape(-1, C).double()
    train = case["mode"] == "train"
    y, dx = torch.empty_like(x), torch.zeros_like(x)
    final = torch.zeros(case["B"], K - 1, C, dtype=torch.float64, device="cuda")
    dstate = torch.zeros_like(final)
    dw, db = torch.zeros_like(w), torch.zeros_like(bias)
    for b, rows, n in _pieces(s):
        head = s["state"][b].double() if case["carry"] else torch.zeros(K - 1, C, dtype=torch.float64, device="cuda")
        whole = torch.cat([head, x[rows]])                          # K-1+n rows
        final[b] = whole[n:]
        dwhole = torch.zeros_like(whole)
        if n:
            windows = whole.unfold(0, K, 1)                         # (n, C, K)
            z = torch.einsum("nck,ck->nc", windows, w) + bias
            y[rows] = act(z)
            if train:
                dz = s["dy"].reshape(-1, C)[rows].double()
                if case["silu"]:
                    e = torch.special.expit(z)
                    dz = dz * (e + z * e * (1 - e))
                dw += torch.einsum("nck,nc->ck", windows, dz)
                db += dz.sum(0)
                dwhole = torch.nn.functional.conv_transpose1d(dz.t()[None], kernel, groups=C)[0].t().clone()
        if train:
            if s["dfinal"] is not None:
                dwhole[n:] += s["dfinal"][b].double()
            dstate[b] = dwhole[:K - 1]
            dx[rows] = dwhole[K - 1:]
    out = {"y": y.view(s["x"].shape), "final": final}
    if train:
        out.update(dx=dx.view(s["x"].shape), dw=dw, db=db, dstate=dstate if case["carry"] else None)
    return out


def _rec_exact(s):
    case = s["case"]
    C = case["C"]
    x, ga, gx = (s[k].reshape(-1, C).double() for k in ("x", "gate_a", "gate_x"))
    lam = s["decay"].double()
    rate = KAPPA * torch.nn.functional.softplus(lam, threshold=1000.0)
    ra, rx = torch.special.expit(ga), torch.special.expit(gx)
    la = -ra * rate
    a, beta = la.exp(), (-torch.expm1(la + la)).sqrt()
    u = beta * (rx * x)
    if case["mode"] == "step":
        state = s["state"].double().clone()
        h = torch.stack([a[b] * state[slot] + u[b] for b, slot in enumerate(s["slots"].tolist())])
        for b, slot in enumerate(s["slots"].tolist()):
            state[slot] = h[b]
        return {"y": h, "state": state}
    train = case["mode"] == "train"
    h, before, g = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    final = torch.zeros(case["B"], C, dtype=torch.float64, device="cuda")
    dstate = torch.zeros_like(final)
    dy = s["dy"].reshape(-1, C).double() if train else None
    for b, rows, n in _pieces(s):
        cur = s["state"][b].double() if case["carry"] else torch.zeros(C, dtype=torch.float64, device="cuda")
        for t in range(rows.start, rows.stop):
            before[t] = cur
            cur = torch.addcmul(u[t], a[t], cur)
            h[t] = cur
        final[b] = cur
        if train:
            back = s["dfinal"][b].double() if s["dfinal"] is not None else torch.zeros_like(cur)
            for t in range(rows.stop - 1, rows.start - 1, -1):
                g[t] = dy[t] + back
                back = a[t] * g[t]
            dstate[b] = back
    out = {"y": h.view(s["x"].shape), "final": final}
    if train:
        # beta = sqrt(1 - a^2), a = exp(la): d beta / d la = -a^2 / beta
        dla = g * before * a - g * rx * x * a.square() / beta
        out.update(dx=(g * beta * rx).view(s["x"].shape), dgate_a=(dla * la * (1 - ra)).view(s["x"].shape),
                   dgate_x=(g * beta * x * rx * (1 - rx)).view(s["x"].shape),
                   ddecay=(dla * -ra).sum(0) * KAPPA * torch.special.expit(lam), dstate=dstate if case["carry"] else None)
    return out


def _adamw_exact(s):
    case = s["case"]
    wide = lambda name: s[name].double() if case["bits"] == 32 else s[name].double() * s[name + "_scale"].double().repeat_interleave(QBLOCK)  # noqa: E731
    g = s["grad"].double() * s["scale"].double()
    m, v = wide("m").lerp(g, 1 - BETA1), wide("v").lerp(g.square(), 1 - BETA2)
    t = STEP + 1
    p = s["p"].double() if s["master"] is None else s["master"].double()
    p = p - LR * (DECAY * p + m / (1 - BETA1 ** t) / ((v / (1 - BETA2 ** t)).sqrt() + EPS))
    kept = case["bits"] == 32      # 8 bits hold a rounding by chance of m and v: it has no value in 64 bits
    return {"p": p, "master": p if case["master"] else None, "m": m if kept else None, "v": v if kept else None}
