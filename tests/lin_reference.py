"""fp64 definitions of linear attention with a decay per head and of attention over a paged cache,
token by token and row by row, and the error bounds the GPU tests hold the kernels to.

Bounds.  Each result is a sum of products; A is the same sum over the products' absolute values.
 - States and fp32 outputs: fp32 sums of at most 64 terms a chunk and one step per chunk, each step
   off by at most 2^-23 of what it holds (tensor-core sums may truncate), plus a few roundings of
   the factors: within 256 * 2^-23 A = 2^-15 A for the lengths tested here.
 - bf16 outputs: the same, the scores' and states' 16-bit copies (a rounded half and the rounded
   rest, 2^-16 of each product, for two factors at most) within 2^-14 A in all, and the rounding
   of the result itself, 2^-8 |o|.
 - Attention: a score is off by (d + 8) 2^-23 scale sum_i |q_i k_ti|, its exponential by as much
   again and 2^-20, the weights' 16-bit copies by 2^-16, in the sum and in what it is divided by.
"""
import math

import torch

U_OUT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
C_OUT = {torch.float32: 2.0 ** -15, torch.bfloat16: 2.0 ** -14}
C_STATE = 2.0 ** -15


def _cpu(t):
    return None if t is None else t.detach().cpu().double()


def lin_forward(q, k, v, g=None, head_g=None, s0=None, cu=None):
    """(out, final, |out| sums, |final| sums) in fp64 on the CPU."""
    q, k, v, g, head_g, s0 = (_cpu(x) for x in (q, k, v, g, head_g, s0))
    B, T, H, dv = v.shape
    rep = H // q.shape[2]
    q, k = q.repeat_interleave(rep, 2), k.repeat_interleave(rep, 2)
    dk = q.shape[-1]
    if cu is None:
        spans = [(b, 0, T) for b in range(B)]
    else:
        c = cu.cpu().tolist()
        spans = [(0, c[i], c[i + 1]) for i in range(len(c) - 1)]
    out, oabs = torch.zeros_like(v), torch.zeros_like(v)
    fin = torch.zeros(len(spans), H, dk, dv, dtype=torch.float64)
    fabs = torch.zeros_like(fin)
    for n, (b, lo, hi) in enumerate(spans):
        S = torch.zeros(H, dk, dv, dtype=torch.float64) if s0 is None else s0[n].clone()
        A = S.abs()
        for t in range(lo, hi):
            lg = torch.zeros(H, dtype=torch.float64)
            if g is not None:
                lg = lg + g[b, t]
            if head_g is not None:
                lg = lg + head_g
            a = lg.exp()[:, None, None]
            kv = k[b, t][:, :, None] * v[b, t][:, None, :]
            S, A = a * S + kv, a * A + kv.abs()
            out[b, t] = torch.einsum("hij,hi->hj", S, q[b, t])
            oabs[b, t] = torch.einsum("hij,hi->hj", A, q[b, t].abs())
        fin[n], fabs[n] = S, A
    return out, fin, oabs, fabs


def check_lin(out, final, ref):
    ro, rs, ao, as_ = ref
    err = (out.detach().cpu().double() - ro).abs()
    assert bool((err <= U_OUT[out.dtype] * ro.abs() + C_OUT[out.dtype] * ao + 1e-37).all()), float((err / (ao + 1e-30)).max())
    if final is not None:
        err = (final.detach().cpu().double() - rs).abs()
        assert bool((err <= C_STATE * as_ + 1e-37).all()), float((err / (as_ + 1e-30)).max())


def paged_forward(q, kc, vc, table, lens, scale):
    """(out, lse, bound on the error of out, of lse) in fp64 on the CPU; pages outside the pool are left out."""
    dt = q.dtype
    q, kc, vc = _cpu(q), _cpu(kc), _cpu(vc)
    N, Hq, d = q.shape
    pages, ps, Hkv = kc.shape[:3]
    rep = Hq // Hkv
    out = torch.zeros(N, Hq, d, dtype=torch.float64)
    lse = torch.full((N, Hq), -math.inf, dtype=torch.float64)
    tol, tol_l = torch.zeros_like(out), torch.zeros(N, Hq, dtype=torch.float64)
    table = table.cpu()
    for n in range(N):
        length = max(0, min(int(lens[n]), table.shape[1] * ps))
        at = [(int(table[n, t // ps]), t % ps) for t in range(length)]
        at = [x for x in at if 0 <= x[0] < pages]
        if not at:
            continue
        pg, off = (torch.tensor(x) for x in zip(*at))
        k, v = (x[pg, off].repeat_interleave(rep, 1) for x in (kc, vc))      # [L, Hq, d]
        s = torch.einsum("hd,lhd->hl", q[n], k) * scale
        m = s.amax(-1, keepdim=True)
        fine = m.isfinite()
        p = torch.where(fine, (s - torch.where(fine, m, 0.0)).exp(), 0.0)
        tot = p.sum(-1, keepdim=True)
        p = p / tot.clamp_min(1e-300)
        out[n] = torch.einsum("hl,lhd->hd", p, v)
        lse[n] = (m + tot.log())[:, 0]
        k0 = torch.where(k.isfinite(), k, 0.0)
        ds = (d + 8) * 2.0 ** -23 * abs(scale) * torch.einsum("hd,lhd->hl", q[n].abs(), k0.abs()).amax(-1, keepdim=True)
        rel = 2 * ds + 2.0 ** -19 + 2.0 ** -15
        tol[n] = rel * torch.einsum("hl,lhd->hd", p, v.abs()) + U_OUT[dt] * out[n].abs()
        tol_l[n] = (ds + 2.0 ** -19)[:, 0] + 2.0 ** -22 * torch.where(lse[n].isfinite(), lse[n].abs(), 0.0)
    return out, lse, tol, tol_l


def check_paged(out, lse, ref):
    ro, rl, tol, tol_l = ref
    err = (out.detach().cpu().double() - ro).abs()
    assert bool((err <= tol + 1e-37).all()), float((err - tol).max())
    if lse is not None:
        got = lse.detach().cpu().double()
        assert torch.equal(got == -math.inf, rl == -math.inf)
        fine = rl > -math.inf
        assert bool(((got - rl).abs()[fine] <= tol_l[fine]).all()), float((got - rl).abs()[fine].max())
