"""The operators over sequences and AdamW in 64 bits on the CPU, one sequence and one row at a time,
written from their formulas; gradients by automatic differentiation of those loops.

Tolerances (u = 2^-24, half a step of fp32 relative to the value; half a step of bf16 is 2^-8):

- convolution, fp32: a sum of K products and a bias is off by at most (K + 2) u times the sum of
  the sizes of its terms; the sigmoid adds 16 u of the result (below).  bf16 adds the one rounding
  of the result, 2^-8 of its size.
- sigmoid: the approximate exponential is off by 2^-22 of itself (4 u) plus the rounding of its
  argument (|z| log2(e) u in the exponent, ln 2 of that in the result: at most 8 u for |z| <= 8), the
  sum and the approximate reciprocal by 1 u and 2 u: at most 15 u.
- recurrence: log a is then off by at most 18 u of itself, a by 18 |log a| a u and its own
  rounding (2 u, with the 2e-8 of its polynomial), b = beta rx x by 32 u (beta: half of 1 - a^2's
  22 u, and 2 u; rx: 15 u; three products).  So the error e of h obeys
  e[t] <= a e[t-1] + |h[t-1]| (18 |log a| a + 2) u + 32 u |b| + u |h[t]|,
  which `recurrence_error` runs beside h.  bf16 adds 2^-8 |h| in y only.
- gradients are sums of such products; they are held to GRAD of the largest entry of their tensor
  (the library's bar for fp32), plus 2^-8 of the entry in bf16."""
from __future__ import annotations

import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
GRAD = 1e-5


def pieces(shape, offsets):
    """(first row, rows) of each sequence of an input of this shape, rows counted in the flattened input."""
    if offsets is None:
        return [(b * shape[1], shape[1]) for b in range(shape[0])]
    return [(a, b - a) for a, b in zip(offsets[:-1], offsets[1:])]


def conv1d(x, w, bias, silu, seqs, state=None):
    """(y, final, sizes): x (rows, C) in float64; `sizes` the sums of the terms' sizes.  Rows of no sequence are NaN."""
    K = w.shape[1]
    ys, finals = [torch.full_like(x, float("nan"))], []
    out = torch.full_like(x, float("nan"))
    sizes = torch.zeros_like(x)
    for s, (first, n) in enumerate(seqs):
        head = x.new_zeros(K - 1, x.shape[1]) if state is None else state[s]
        whole = torch.cat([head, x[first:first + n]])
        finals.append(whole[n:])
        if n:
            terms = torch.stack([whole[k:k + n] * w[:, k] for k in range(K)])
            b = 0 if bias is None else bias
            z = terms.sum(0) + b
            y = z * torch.sigmoid(z) if silu else z
            out = out.index_put((torch.arange(first, first + n),), y)
            sizes[first:first + n] = (terms.abs().sum(0) + abs(b)).detach()
    del ys
    return out, torch.stack(finals), sizes


def gates(gate_a, gate_x, decay, kappa):
    ra, rx = torch.sigmoid(gate_a), torch.sigmoid(gate_x)
    la = -kappa * torch.nn.functional.softplus(decay, threshold=1e9) * ra
    return la, torch.exp(la), torch.sqrt(-torch.expm1(2 * la)), rx


def recurrence(x, gate_a, gate_x, decay, kappa, seqs, state=None):
    """(h, final, error): the states of all rows (NaN where there is no sequence), the last of each sequence, and the
    bound of the module's docstring."""
    la, a, beta, rx = gates(gate_a, gate_x, decay, kappa)
    b = beta * rx * x
    rows, finals = {}, []
    error = torch.zeros_like(x)
    for s, (first, n) in enumerate(seqs):
        h = x.new_zeros(x.shape[1]) if state is None else state[s]
        e = torch.zeros_like(h)
        for t in range(first, first + n):
            before = h
            h = a[t] * h + b[t]
            rows[t] = h
            with torch.no_grad():
                e = a[t] * e + before.abs() * (18 * la[t].abs() * a[t] + 2) * U + (32 * b[t].abs() + h.abs()) * U
                error[t] = e
        finals.append(h)
    none = x.new_full((x.shape[1],), float("nan"))
    out = torch.stack([rows.get(t, none) for t in range(x.shape[0])]) if x.shape[0] else x
    return out, torch.stack(finals), error


def adamw(p, g, m, v, lr, beta1, beta2, eps, decay, step):
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    update = (m / (1 - beta1 ** step)) / ((v / (1 - beta2 ** step)).sqrt() + eps)
    return p * (1 - lr * decay) - lr * update, m, v


def close(got, want, dtype, atol, what=""):
    """got within half a step of its type plus atol (a number, or one for each entry) of the 64-bit values."""
    got, want = got.detach().double().cpu().reshape(want.shape), want.detach()
    atol = torch.as_tensor(atol, dtype=torch.float64)
    ok = ((got - want).abs() <= HALF[dtype] * want.abs() + atol) | (got == want) | (got.isnan() & want.isnan())
    if not bool(ok.all()):
        bad = (~ok).nonzero()[0].tolist()
        raise AssertionError(f"{what}: {int((~ok).sum())} of {ok.numel()} off, first at {bad}: got "
                             f"{got[tuple(bad)].item()!r}, want {want[tuple(bad)].item()!r}")


def grad_close(got, want, dtype, what=""):
    scale = want.detach().abs().max().item() if want.numel() else 0.0
    close(got, want, dtype, GRAD * scale, what)
