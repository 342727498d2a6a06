"""Plain fp64 forms of the operators on packed sequences, with elementwise error bounds.

attend() computes one sequence from the definition and, beside every output, the bound that its
roundings allow a kernel with bf16 values and fp32 sums (u = 2^-8 is half a bf16 step, relative):
  o     P is rounded to bf16 before its product and o at the store: u sum_j p |v| + u |o|; the
        exponentials and the fp32 sums add less than 2^-12 of the first term.
  lse   fp32 throughout: 1e-3, the bound of every forward here.
  dv    as o, over queries: u sum_i p |dout| + u |dv|.
  dS    = p (dP - D): rounded to bf16 (u |dS|); D comes from the rounded o, so it is off by at most
        sum_d |dout_d| tol_o_d; P comes from lse and fp32 scores (relative 2^-12).
  dq, dk  the dS bound times |k| or |q| and the scale, plus u |dq| or u |dk|.
"""
import math

import torch

U = 2.0 ** -8     # half a step of bf16, relative
EXP = 2.0 ** -12  # exponentials, fp32 scores and fp32 sums, relative to the probabilities
TINY = 2.0 ** -100


def attend(q, k, v, causal, window, scale=None, dout=None):
    """q [n, Hq, D] are the last n positions of k, v [m, Hkv, D]. Returns a dict of fp64 tensors and, under
    the same name + '_tol', their bounds."""
    n, Hq, D = q.shape
    m, Hkv = k.shape[0], k.shape[1]
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    q, k, v = q.double(), k.double(), v.double()
    kh, vh = (x.repeat_interleave(G, dim=1) for x in (k, v))
    i = torch.arange(m - n, m, device=q.device)[:, None]
    j = torch.arange(m, device=q.device)[None]
    ok = torch.ones(n, m, dtype=torch.bool, device=q.device)
    if causal:
        ok &= j <= i
    if window > 0:
        ok &= j > i - window
    s = torch.einsum("ihd,jhd->hij", q, kh) * scale
    s = s.masked_fill(~ok, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = (s - lse[..., None]).exp()
    o = torch.einsum("hij,jhd->ihd", p, vh)
    r = {"o": o, "lse": lse, "lse_tol": torch.full_like(lse, 1e-3)}
    r["o_tol"] = (U + EXP) * torch.einsum("hij,jhd->ihd", p, vh.abs()) + U * o.abs() + TINY
    if dout is None:
        return r
    g = dout.double()
    ds = p * (torch.einsum("ihd,jhd->hij", g, vh) - (g * o).sum(-1).t()[..., None])
    ds_tol = p * (g.abs() * r["o_tol"]).sum(-1).t()[..., None] + (U + EXP) * ds.abs() + \
        EXP * p * torch.einsum("ihd,jhd->hij", g.abs(), vh.abs())
    share = lambda x: x.view(m, Hkv, G, D).sum(2)
    r["dq"] = torch.einsum("hij,jhd->ihd", ds, kh) * scale
    r["dk"] = share(torch.einsum("hij,ihd->jhd", ds, q)) * scale
    r["dv"] = share(torch.einsum("hij,ihd->jhd", p, g))
    r["dq_tol"] = torch.einsum("hij,jhd->ihd", ds_tol, kh.abs()) * scale + U * r["dq"].abs() + TINY
    r["dk_tol"] = share(torch.einsum("hij,ihd->jhd", ds_tol, q.abs())) * scale + U * r["dk"].abs() + TINY
    r["dv_tol"] = (U + EXP) * share(torch.einsum("hij,ihd->jhd", p, g.abs())) + U * r["dv"].abs() + TINY
    return r


def packed(q, k, v, starts, causal, window, scale=None, dout=None):
    """attend() over every sequence of a packed batch: starts = offsets, a list. Rows outside the sequences
    are NaN. lse is [Hq, T]."""
    T = q.shape[0]
    out = {}
    for a, b in zip(starts, starts[1:]):
        if a == b:
            continue
        one = attend(q[a:b], k[a:b], v[a:b], causal, window, scale, None if dout is None else dout[a:b])
        for name, x in one.items():
            lse = name.startswith("lse")
            if name not in out:
                shape = (x.shape[0], T) if lse else (T,) + x.shape[1:]
                out[name] = torch.full(shape, math.nan, dtype=torch.float64, device=q.device)
            (out[name].t() if lse else out[name])[a:b] = x.t() if lse else x
    return out


def check(name, got, ref):
    """got against ref[name] within ref[name + '_tol'], where ref is not NaN."""
    want, tol = ref[name], ref[name + "_tol"]
    inside = ~torch.isnan(want)
    err = (got.double() - want).abs()
    assert bool(torch.isfinite(got[inside]).all()), "%s: non-finite" % name
    worst = (err / tol)[inside].max().item() if bool(inside.any()) else 0.0
    assert worst <= 1.0, "%s: error %.3f of its bound" % (name, worst)
    return worst


def rope_axes(x, positions, sections, interleave, per_axis, half, base, pos_scale=1.0, inverse=False):
    """y and its bound: x [T, H, D], positions [axes, T]. The angle is formed in fp64 by four roundings, here
    and in the kernel alike (2^-50 of it together); the reduced angle, sin and cos are fp32 (2^-23 each), and so
    are products and sum: (2^-21 + 2^-50 |angle|) (|x0| + |x1|). One rounding to bf16: half a step of y (u |y|)."""
    n, R2 = len(sections), sum(sections)
    owner, left = [], list(sections)
    for i in range(R2):
        a = 0
        if interleave:
            a = i % n if i % n and i // n < sections[i % n] else 0
        else:
            while left[a] == 0:
                a += 1
        left[a] -= 1
        owner.append(a)
    seen, expo = [0] * n, []
    for i, a in enumerate(owner):
        expo.append(seen[a] / sections[a] if per_axis else i / R2)
        seen[a] += 1
    theta = torch.tensor([float(base) ** -e for e in expo], dtype=torch.float64, device=x.device)
    ang = positions.double()[owner].t() / pos_scale * theta * (-1.0 if inverse else 1.0)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    z = x.double().clone()
    tol = torch.zeros_like(z)
    first, second = (slice(0, R2), slice(R2, 2 * R2)) if half else (slice(0, 2 * R2, 2), slice(1, 2 * R2, 2))
    x0, x1 = x.double()[..., first], x.double()[..., second]
    off = 2.0 ** -21 + 2.0 ** -50 * ang.abs()[:, None]
    z[..., first], z[..., second] = x0 * c - x1 * s, x0 * s + x1 * c
    for part in (first, second):
        tol[..., part] = U * z[..., part].abs() + off * (x0.abs() + x1.abs()) + TINY
    return z, tol
