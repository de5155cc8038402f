"""fp64 definitions of linear attention with a head decay and of token trees over
cached states, with the magnitudes that rounding errors scale with.

Every function takes CPU or GPU tensors and computes in fp64 on the CPU, token by
token.  Beside each value it returns its magnitude: the same recursion with every
term replaced by its absolute value.  A computation that rounds each of its
operations by at most u (relative) is off by at most (operations in a row) * u *
magnitude, which is what ``gamma`` counts.
"""
from __future__ import annotations

import torch

U32 = 2.0 ** -24   # half a step of fp32
UB16 = 2.0 ** -8   # half a step of bf16


def d64(x):
    return None if x is None else x.detach().to("cpu", torch.float64)


def gamma(Dk, depth, split=0.0, extra=16):
    """Relative error bound of a path of ``depth`` updates: each has dot products of
    Dk terms (tensor cores may cut instead of round a partial sum: 2 u an
    addition) and ``extra`` other roundings, on operands off by ``split``."""
    return (depth + 1) * (2 * (Dk + extra) * U32 + split)


def tree(q, k, v, g, beta, parent, S0, scale=1.0, raw=False):
    """One sequence.  q, k [M, Hqk, Dk]; v [M, Hv, Dv]; g, beta [M, Hv], or beta
    None and g [Hv]; parent list of M ints; S0 [Hv, Dv, Dk].  Returns
    (o [M, Hv, Dv], its magnitude, {node: state}, {node: state magnitude},
    {node: depth}); rows of padding nodes are zero."""
    q, k, v, g, beta, S0 = (d64(x) for x in (q, k, v, g, beta, S0))
    M, Hv, Dv = v.shape
    rep = torch.arange(Hv) // (Hv // k.shape[1])
    if raw:
        unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-300)  # noqa: E731
        q, k = unit(q), unit(k)
        g, beta = -torch.nn.functional.softplus(g), torch.sigmoid(beta)
    q, k = q[:, rep], k[:, rep]
    o, om = torch.zeros_like(v), torch.zeros_like(v)
    S, Sm, depth = {-1: S0}, {-1: S0.abs()}, {-1: 0}
    for i in range(M):
        p = parent[i]
        if p < -1:
            continue
        a = (g if beta is None else g[i]).exp()[:, None, None]
        b = torch.ones(Hv, dtype=torch.float64) if beta is None else beta[i]
        ki, vi = k[i], v[i]
        Sp, Spm = a * S[p], a * Sm[p]
        w, wm = vi, vi.abs()
        if beta is not None:
            w = vi - torch.einsum("hvd,hd->hv", Sp, ki)
            wm = vi.abs() + torch.einsum("hvd,hd->hv", Spm, ki.abs())
        S[i] = Sp + (b[:, None] * w)[:, :, None] * ki[:, None, :]
        Sm[i] = Spm + (b[:, None] * wm)[:, :, None] * ki.abs()[:, None, :]
        depth[i] = depth[p] + 1
        o[i] = scale * torch.einsum("hvd,hd->hv", S[i], q[i])
        om[i] = abs(scale) * torch.einsum("hvd,hd->hv", Sm[i], q[i].abs())
    return o, om, S, Sm, depth


def scan(q, k, v, g, cu, S0=None, scale=1.0):
    """Linear attention over packed sequences: (o, its magnitude, final states, theirs)."""
    q, k, v, g, S0 = (d64(x) for x in (q, k, v, g, S0))
    T, Hv, Dv = v.shape
    N, Dk = len(cu) - 1, k.shape[2]
    rep = torch.arange(Hv) // (Hv // k.shape[1])
    q, k = q[:, rep], k[:, rep]
    lam = g.clamp_min(-30.0).exp()[:, None, None]
    o, om = torch.zeros_like(v), torch.zeros_like(v)
    F = torch.zeros(N, Hv, Dv, Dk, dtype=torch.float64)
    Fm = torch.zeros_like(F)
    for n in range(N):
        S = torch.zeros(Hv, Dv, Dk, dtype=torch.float64) if S0 is None else S0[n]
        Sm = S.abs()
        for t in range(cu[n], cu[n + 1]):
            S = lam * S + v[t, :, :, None] * k[t, :, None, :]
            Sm = lam * Sm + (v[t, :, :, None] * k[t, :, None, :]).abs()
            o[t] = scale * torch.einsum("hvd,hd->hv", S, q[t])
            om[t] = abs(scale) * torch.einsum("hvd,hd->hv", Sm, q[t].abs())
        F[n], Fm[n] = S, Sm
    return o, om, F, Fm


def check(x, ref, mag, rel, what, stored=0.0):
    """|x - ref| <= rel * mag + stored * |ref| (+ the least normal fp32), element by
    element; ``stored`` is half a step of the type x is stored in."""
    x = d64(x)
    bound = rel * mag * (1 + stored) + stored * ref.abs() + 2.0 ** -126
    err = (x - ref).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst ratio "
                           f"{float((err / bound).nan_to_num(float('inf')).max()):.3g}")


def scan_grads(q, k, v, g, cu, S0, do, dsf, scale=1.0):
    """Gradients of ``scan``'s o and final states, given theirs: ((dq, dk, dv, dS0),
    the magnitudes of the same), token by token from the formulas."""
    q, k, v, g, do, S0, dsf = (d64(x) for x in (q, k, v, g, do, S0, dsf))
    T, Hv, Dv = v.shape
    N, Hqk, Dk = len(cu) - 1, *k.shape[1:]
    rep = torch.arange(Hv) // (Hv // Hqk)
    zero = torch.zeros(N, Hv, Dv, Dk, dtype=torch.float64)
    S0, dsf = zero if S0 is None else S0, zero if dsf is None else dsf
    lam = g.clamp_min(-30.0).exp()[:, None, None]
    out = []
    for q, k, v, do, S0, dsf, s in ((q, k, v, do, S0, dsf, scale),
                                    (q.abs(), k.abs(), v.abs(), do.abs(), S0.abs(), dsf.abs(), abs(scale))):
        q, k = q[:, rep], k[:, rep]
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        dS0 = dsf.clone()
        for n in range(N):
            S, D = S0[n], dsf[n]
            for t in range(cu[n], cu[n + 1]):
                S = lam * S + v[t, :, :, None] * k[t, :, None, :]
                dq[t] = s * torch.einsum("hvd,hv->hd", S, do[t])
            for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
                D = D + s * do[t, :, :, None] * q[t, :, None, :]
                dk[t] = torch.einsum("hvd,hv->hd", D, v[t])
                dv[t] = torch.einsum("hvd,hd->hv", D, k[t])
                D = lam * D
            dS0[n] = D
        dq, dk = (x.unflatten(1, (Hqk, Hv // Hqk)).sum(2) for x in (dq, dk))
        out.append((dq, dk, dv, dS0))
    return out
