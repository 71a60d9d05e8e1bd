"""Plain 64-bit definitions of the prompt, rotary and row-moving operators, with the largest error
their kernels may make, for the tests."""
import math

import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # half a step, relative
EPS32 = 2.0 ** -24


def attention(q, k, v, lens, scale, start=0):
    """out, lse and their error bounds for packed prompts: q [T, hq, d], k, v [T, hkv, d], sequence
    by sequence and head by head, each row over the rows up to it alone (hidden rows are cut off,
    never multiplied).

    Bounds, to first order.  A score is a sum of d products in 32 bits: off by at most (d + 4) EPS32
    A, A the largest sum of |q k| scale of the row; that and the exponential's error (4 EPS32) move
    a probability by `dp` relative to it; sums over n keys in 32 bits add n EPS32.  16-bit rows round
    each unnormalised probability once (HALF) and every result once (HALF)."""
    T, hq, d = q.shape
    hkv = k.shape[1]
    half = HALF[q.dtype]
    out = torch.zeros(T, hq, d, dtype=torch.float64, device=q.device)
    lse = torch.zeros(T, hq, dtype=torch.float64, device=q.device)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    at = start
    for n in lens:
        for h in range(hq if n else 0):
            Q, K, V = (x[at:at + n, i].double() for x, i in ((q, h), (k, h // (hq // hkv)), (v, h // (hq // hkv))))
            hidden = torch.ones(n, n, dtype=torch.bool, device=q.device).triu(1)
            Kf, Vf, Qf = (torch.nan_to_num(x, 0.0, 0.0, 0.0) for x in (K, V, Q))
            s = (Q @ Kf.t()) * scale
            bad = (~torch.isfinite(K)).any(1)
            for j in bad.nonzero().flatten().tolist():           # a non-finite key, for the rows that see it
                s[:, j] = (Q @ K[j]) * scale
            s.masked_fill_(hidden, -math.inf)
            m = s.amax(1, keepdim=True)
            e = torch.exp(s - m)
            z = e.sum(1, keepdim=True)
            P = e / z
            o = P @ Vf
            for j in (~torch.isfinite(V)).any(1).nonzero().flatten().tolist():
                o[j:] += torch.where(torch.isfinite(V[j]), 0.0, V[j])
            out[at:at + n, h], lse[at:at + n, h] = o, (m + z.log())[:, 0]
            A = ((Qf.abs() @ Kf.abs().t()) * abs(scale)).masked_fill(hidden, 0).amax(1, keepdim=True)
            dp = 2 * (d + 4) * EPS32 * A + (n + 8) * EPS32 + 8 * EPS32 + 2 * EPS32 * (m.abs().nan_to_num(0, 0, 0) + 8)
            rounded = half if q.dtype != torch.float32 else 0.0
            tol_o[at:at + n, h] = (P.nan_to_num(0) @ Vf.abs()) * (dp + rounded) * 1.01 + o.abs().nan_to_num(0, 0, 0) * (half + 4 * EPS32)
            tol_l[at:at + n, h] = (dp + EPS32 * (lse[at:at + n, h, None].abs().nan_to_num(0, 0, 0) + 8))[:, 0]
        at += n
    return out, lse, tol_o, tol_l


def close(got, want, tol, what=""):
    got = got.double()
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(got)), f"{what}: finite in other places"
    assert torch.equal(torch.isnan(want), torch.isnan(got)), f"{what}: NaN in other places"
    other = ~fine & ~torch.isnan(want)
    assert torch.equal(got[other], want[other]), f"{what}: infinities differ"
    over = ((got - want).abs() - tol)[fine]
    assert over.numel() == 0 or over.max() <= 0, f"{what}: {over.max():.3e} over its bound"


def axis_of_pair(sections, cyclic):
    out, left = [], list(sections)
    if not cyclic:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    a = 0
    while any(left):
        if left[a]:
            out.append(a)
            left[a] -= 1
        a = (a + 1) % len(left)
    return out


def rotate(x, positions, sections, freq, cyclic=False, interleaved=False):
    """x [T, h, d] turned, in 64 bits, and the error bound of a kernel in 32 bits."""
    half = sum(sections)
    ax = torch.tensor(axis_of_pair(sections, cyclic), device=x.device)
    ang = positions.double()[ax].t() * freq.double()             # [T, half]
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    X = x.double()
    out, tol = X.clone(), torch.zeros_like(X)
    i = torch.arange(half, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = X[..., ia], X[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    # the angle: 2^-25 turn, 2^-52 of it in each of the two roundings here and there; then sincospif
    # (1 ulp) and two rounded products
    da = (2 * math.pi * 2.0 ** -25 + ang.abs() * 2.0 ** -50 + 6 * EPS32)[:, None]
    tol[..., ia] = tol[..., ib] = (a.abs() + b.abs()) * da
    return out, tol + out.abs() * HALF[x.dtype] * (1 if x.dtype != torch.float32 else 2)
