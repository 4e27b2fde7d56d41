"""The gated recurrence where the decay is strong (a between 1e-11 and 0.6), entry by entry, on a B200.

Every entry of y, the states and the gradients is held to a bound of its own, relative to the sums of its terms' sizes, not to the
largest entry of its tensor: where a is small, so are the entries that it multiplies, and they have to be right too.

The bounds (u = 2^-24, half a step of fp32 relative to the value; CUDA gives expf 2 units of the last place, 4 u, and log1pf
1 unit, 2 u).  They run beside the recurrence, on the absolute values (capital letters) of what it adds:

- rate = kappa softplus(decay) log2(e): expf 4 u, log1pf 2 u, a sum, a constant, two products: 10 u.  sigmoids for |z| <= 8: 15 u
  (sequence_reference.py).  log a is their product, off by 26 u of itself, so a by eps = (26 |log a| + 2) u of itself.
- p = a - 1 is off by 26 u |log a| a / (1 - a) <= 26 u, and 2 u; 1 - a^2 = -p (2 + p) by 30 u, its root (or one over it) by
  17 u; b = beta rx x by 17 + 15 + 3 = 35 u.
- h: S = a S + |b|;  E = a E + (eps + u) a S' + 36 u |b| + 4 u S (a row's own rounding, and those of joining its run and its chunk).
- g = dy + a' g' against time: the same, without b's 35 u.
- ra a g (h' - a rx x / beta) = w: ra (E_ag M + AG E_M) + 18 u W, with M = S' + a rx |x| / beta and
  E_M = E' + (eps + 36 u) a rx |x| / beta + u M.
- 1 - sigmoid is off by 16 u; d_gate_a = -kappa softplus(decay) w (1 - ra) adds 14 u, and the factor's error.
- d_decay: a chunk's rows are summed in fp32 by eights, then the warps' sums: 24 u of the sum of sizes; the chunks' in 64 bits.

A result in bf16 adds half its step.  1e-37 stands for values below the smallest normal number.

The 64-bit values come from loops of their own: sequence_reference.py takes beta as sqrt(-expm1(2 log a)), whose
automatic derivative is -expm1 + 1 in 64 bits, 0 where a^2 is below 1e-16.  sqrt(1 - exp(2 log a)) has the derivative's exponential
itself, and a stays below 0.9 here, so 1 - a^2 is exact to 1e-15."""
import pytest
import torch

import cnn_convolution_conv2d_b200 as cb
import sequence_reference as ref

pytestmark = pytest.mark.gpu
KAPPA, U, LEAST = 8.0, ref.U, 1e-37


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    assert torch.cuda.is_available(), "these tests need a CUDA device"
    from cnn_convolution_conv2d_b200 import build
    build.build()
    cb.load()
    yield
    cb.conv2d_sync_status()


def gates(ga, gx, decay):
    la = -KAPPA * torch.nn.functional.softplus(decay, threshold=1e9) * torch.sigmoid(ga)
    return la, torch.exp(la), torch.sqrt(1 - torch.exp(2 * la)), torch.sigmoid(gx)


def recurrence(x, ga, gx, decay, seqs, state):
    """(states of all rows of a sequence, the last of each), in 64 bits."""
    la, a, beta, rx = gates(ga, gx, decay)
    b, rows, finals = beta * rx * x, [], []
    for s, (first, n) in enumerate(seqs):
        h = state[s]
        for t in range(first, first + n):
            h = a[t] * h + b[t]
            rows.append(h)
        finals.append(h)
    return torch.stack(rows), torch.stack(finals)


def bounds(x, ga, gx, decay, dy, seqs, state, dfinal):
    """The bounds of the docstring, for one-dimensional lists of rows in 64 bits."""
    la, a, beta, rx = gates(ga, gx, decay)
    ra, rate = torch.sigmoid(ga), KAPPA * torch.nn.functional.softplus(decay, threshold=1e9)
    eps, b = (26 * la.abs() + 2) * U, (beta * rx * x).abs()
    zero = torch.zeros_like(x)
    S, E, S0, E0, G, EG, AG, EAG = (zero.clone() for _ in range(8))
    for s, (first, n) in enumerate(seqs):
        size, err = state[s].abs(), torch.zeros_like(state[s])
        for t in range(first, first + n):
            S0[t], E0[t] = size, err
            err = a[t] * err + (eps[t] + U) * a[t] * size + 36 * U * b[t]
            size = a[t] * size + b[t]
            err = err + 4 * U * size
            S[t], E[t] = size, err
        size, err = dfinal[s].abs(), torch.zeros_like(state[s])
        for t in reversed(range(first, first + n)):
            G[t] = dy[t].abs() + size
            EG[t] = err + 4 * U * G[t]
            err = EAG[t] = a[t] * EG[t] + (eps[t] + U) * a[t] * G[t]
            size = AG[t] = a[t] * G[t]
    part = a * rx * x.abs() / beta
    M = S0 + part
    EM = E0 + (eps + 36 * U) * part + U * M
    W = ra * AG * M
    EW = ra * (EAG * M + AG * EM) + 18 * U * W
    DX = G * beta * rx
    EDX = EG * beta * rx + 35 * U * DX
    return dict(y=E, dx=EDX, d_gate_x=(EDX + DX * (18 * U + 16 * U / (1 - rx))) * x.abs() * (1 - rx),
                d_gate_a=rate * (1 - ra) * (EW + W * (14 * U + 16 * U / (1 - ra))),
                d_decay=KAPPA * torch.sigmoid(decay) * (EW.sum(0) + 26 * U * W.sum(0)), back=EAG)


FORMS = {"tiles": (96, None, 2, 300), "copies": (33, None, 2, 300), "packed": (64, [0, 200, 200, 204, 600], 4, 620)}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("decay, gate, zero", [(0.0, 0.0, False), (3.0, 0.0, False), (2.0, 2.0, False), (3.0, 2.0, False),
                                               (3.0, 2.0, True), (3.0, -4.0, False)], ids=str)
def test_strong_decays(decay, gate, zero, form, dtype):
    """gate 2: shut almost always, -4: open; `zero`: x = 0, so nothing but the decayed state is there."""
    C, offsets, B, T = FORMS[form]
    gen = torch.Generator().manual_seed(int(10 * decay + gate) + C)
    normal = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    shape = (T, C) if offsets else (B, T, C)
    x, ga, gx, dy = (normal(*shape).to(dtype), (0.5 * normal(*shape) + gate).to(dtype), normal(*shape).to(dtype),
                     normal(*shape).to(dtype))
    if zero:
        x.zero_()
    lam, state, dfinal = 0.1 * normal(C) + decay, normal(B, C), normal(B, C)
    wide = [t.double().reshape(-1, C) if t.dim() > 1 else t.double() for t in (x, ga, gx, lam)]
    wx, wa, wg, wl = (t.requires_grad_() for t in wide)
    ws = state.double().requires_grad_()
    seqs = ref.pieces(shape, offsets)
    h, final = recurrence(wx, wa, wg, wl, seqs, ws)
    rows = sum(n for _, n in seqs)
    flat_dy = dy.double().reshape(-1, C)
    want = torch.autograd.grad((h * flat_dy[:rows]).sum() + (final * dfinal.double()).sum(), [wx, wa, wg, wl, ws])
    with torch.no_grad():
        tol = bounds(wx, wa, wg, wl, flat_dy, seqs, ws, dfinal.double())
    rec = cb.GatedRecurrenceB200(lam.cuda(), KAPPA)
    t = [v.cuda() for v in (x, ga, gx)]
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    got_final, saved = torch.zeros(B, C, device="cuda"), rec.saved_states(t[0])
    y = rec(*t, offsets=off, initial_state=state.cuda(), final_state=got_final, saved=saved)
    dx, dga, dgx, dd, ds = rec.backward(*t, dy.cuda(), saved, offsets=off, initial_state=state.cuda(), d_final_state=dfinal.cuda())
    cb.conv2d_sync_status()
    cut = lambda v: v.reshape(-1, C)[:rows]  # noqa: E731
    f32 = torch.float32
    for name, g, w in (("y", y, h), ("dx", dx, want[0]), ("d_gate_a", dga, want[1]), ("d_gate_x", dgx, want[2])):
        ref.close(cut(g), w[:rows], dtype, tol[name][:rows] + LEAST, name)
    ref.close(dd, want[3], f32, tol["d_decay"] + LEAST, "d_decay")
    ends = torch.stack([tol["y"][first + n - 1] if n else torch.zeros(C) for first, n in seqs])
    starts = torch.stack([tol["back"][first] if n else torch.zeros(C) for first, n in seqs])
    ref.close(got_final, final, f32, ends + LEAST, "final state")
    ref.close(ds, want[4], f32, starts + LEAST, "d_initial_state")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_a_token_with_a_strong_decay(dtype):
    gen = torch.Generator().manual_seed(3)
    B, C = 5, 300
    ga, lam, state = (torch.randn(B, C, generator=gen) + 2).to(dtype), torch.randn(C, generator=gen) + 2, torch.randn(B, C, generator=gen)
    x = torch.zeros(B, C, dtype=dtype)
    la, a, _, _ = gates(ga.double(), x.double(), lam.double())
    want, tol = a * state.double(), (26 * la.abs() + 4) * U * a * state.double().abs()
    held = state.cuda()
    y = cb.GatedRecurrenceB200(lam.cuda(), KAPPA).step(x.cuda(), ga.cuda(), x.cuda(), held)
    ref.close(held, want, torch.float32, tol, "state")
    ref.close(y, want, dtype, tol, "y")
    cb.conv2d_sync_status()
