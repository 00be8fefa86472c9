"""64-bit references of the packed attention and the 8-bit cache, with bounds on what rounding may do.

u = 2^-8 is the largest relative error of one rounding to bf16, h = 2^-11 to fp16.  The kernels round
P (bf16 or fp16), dS, and the outputs; everything else is fp32, whose error enters the scores:
a score is off by at most e_s = (d + 16) 2^-24 S, S = scale * sum |q||k| (its products, its sum,
the multiplication and subtraction before the exponential, 2^-22 of the exponential itself), so an
unnormalised probability by (e_s + 2^-22) relative, and a normalised one by twice that at most.
"""
import math

import torch

U, H16 = 2.0 ** -8, 2.0 ** -11


def cu_of(lengths, device="cuda"):
    return torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device=device)


def visible(nq, nk, causal, device):
    i, j = torch.arange(nq, device=device)[:, None], torch.arange(nk, device=device)[None]
    return (j <= i + nk - nq) if causal else torch.ones(nq, nk, dtype=torch.bool, device=device)


def one_sequence(q, k, v, causal, scale, dout=None, p_step=U, v_unit=None):
    """q, dout [G, n, d], k and v [m, d] of one sequence and key head.  Returns a dict of 64-bit results and the
    bound on each's error (name + "_tol")."""
    q, k, v = q.double(), k.double(), v.double()
    n, m, d = q.shape[1], k.shape[0], q.shape[2]
    ok = visible(n, m, causal, q.device)[None]
    # a NaN in V reaches the queries that see it, and only its own column
    lost = torch.einsum("gnm,md->gnd", ok.double().expand(q.shape[0], -1, -1), v.isnan().double()) > 0
    v = v.nan_to_num(0.0, math.inf, -math.inf)
    x = scale * torch.einsum("gnd,md->gnm", q, k)
    x = torch.where(ok, x, -math.inf)
    top = x.amax(-1, keepdim=True) if m else torch.full((*x.shape[:2], 1), -math.inf, dtype=x.dtype, device=x.device)
    e = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    l = e.sum(-1, keepdim=True)
    lse = (torch.log(l) + torch.where(top == -math.inf, 0.0, top))[..., 0]
    p = e / torch.where(l > 0, l, 1.0)
    o = torch.einsum("gnm,md->gnd", p, v)
    big = scale * torch.where(ok, torch.einsum("gnd,md->gnm", q.abs(), k.abs()), 0.0)
    big = big.amax(-1) if m else torch.zeros_like(lse)
    es = (d + 16 + m * 2.0 ** -6) * 2.0 ** -24 * big + 2.0 ** -21 + m * 2.0 ** -24
    spread = torch.einsum("gnm,md->gnd", p, v.abs())
    o = torch.where(lost, math.nan, o)
    r = {"o": o, "lse": lse, "lse_tol": es + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0)}
    r["o_tol"] = U * o.abs() + (p_step + 2 * es[..., None]) * (1 + U) * spread + 1e-30
    if v_unit is not None and m:  # fp16 products below the smallest subnormal: half of 2^-24 of the largest contribution
        r["o_tol"] += m * 2.0 ** -25 * 448.0 * (p * v_unit.double()[None, None]).amax(-1, keepdim=True)
    if dout is None:
        return r
    do = dout.double()
    dp = torch.einsum("gnd,md->gnm", do, v)
    dsum = (do * o).sum(-1, keepdim=True)
    ds = p * (dp - dsum)
    mag = p * (torch.einsum("gnd,md->gnm", do.abs(), v.abs()) + (do.abs() * spread).sum(-1, keepdim=True))
    # D from the bf16 output: off by sum |dO| times the output's own error
    d_err = (do.abs() * r["o_tol"]).sum(-1, keepdim=True)
    ds_err = U * ds.abs() + p * d_err + (2 * es[..., None] + (d + 4) * 2.0 ** -23) * mag
    ds_err = ds_err * (1 + U)
    for name, eq, a, err, b, mul in (("dq", "gnm,md->gnd", ds, ds_err, k, scale), ("dk", "gnm,gnd->md", ds, ds_err, q, scale),
                                     ("dv", "gnm,gnd->md", p, p * (U + 2 * es[..., None]), do, 1.0)):
        want = mul * torch.einsum(eq, a, b)
        r[name] = want
        r[name + "_tol"] = U * want.abs() + (1 + U) * mul * torch.einsum(eq, err + 2.0 ** -18 * a.abs(), b.abs()) + 1e-30
    return r


def packed(q, k, v, lens_q, lens_k, causal, scale, dout=None):
    """Reference of the packed calls: dict of 64-bit tensors and bounds shaped like the outputs (lse [heads, tokens]);
    rows behind the last sequence are zeros (lse -inf)."""
    T, H, d = q.shape
    K = k.shape[1]
    G = H // K
    out = {n: torch.zeros(T, H, d, dtype=torch.float64, device=q.device) for n in ("o", "o_tol", "dq", "dq_tol")}
    out.update({n: torch.zeros(k.shape, dtype=torch.float64, device=q.device) for n in ("dk", "dk_tol", "dv", "dv_tol")})
    out["lse"] = torch.full((H, T), -math.inf, dtype=torch.float64, device=q.device)
    out["lse_tol"] = torch.zeros_like(out["lse"])
    a = b = 0
    for n, m in zip(lens_q, lens_k):
        for h in range(K):
            hs = slice(h * G, h * G + G)
            r = one_sequence(q[a:a + n, hs].transpose(0, 1), k[b:b + m, h], v[b:b + m, h], causal, scale,
                             None if dout is None else dout[a:a + n, hs].transpose(0, 1))
            for name, t in r.items():
                if name.startswith("lse"):
                    out[name][hs, a:a + n] = t
                elif name.startswith(("dk", "dv")):
                    out[name][b:b + m, h] = t
                else:
                    out[name][a:a + n, hs] = t.transpose(0, 1)
        a, b = a + n, b + m
    return out


def check(got, ref, name, rows=None):
    """`got` within `ref`'s bound, infinities and NaN where `ref` has them."""
    want, tol = ref[name], ref[name + "_tol"]
    g = got.double()
    if rows is not None:
        want, tol, g = want[..., rows], tol[..., rows], g[..., rows]
    same = (g == want) | ((g - want).abs() <= tol) | (g.isnan() & want.isnan())
    assert bool(same.all()), (name, int((~same).sum()), float(((g - want).abs() / tol.clamp(min=1e-30))[~same].max()))


def e4m3(x):
    """Nearest e4m3 value of x (|x| <= 448), ties to even, in 64 bits."""
    x = x.double()
    e = (torch.frexp(x)[1] - 1).clamp(min=-6)
    step = torch.ldexp(torch.ones_like(x), e - 3)
    return torch.round(x / step) * step


def scale_of(amax):
    """The smallest 2^e, -60 <= e <= 120, with amax <= 448 * 2^e."""
    for e in range(-60, 121):
        if amax <= 448.0 * 2.0 ** e:
            return 2.0 ** e
    return 2.0 ** 120
