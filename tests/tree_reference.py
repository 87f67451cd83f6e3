"""fp64 definitions of the calls for branching decode, token by token, and the bounds that the GPU tests hold the
kernels to.

Bounds.  Each result is a sum of products; A is the same sum over the products' absolute values, with D tokens on a path.
 - KDA outputs: a coefficient or product with the state is a sum of fp32 terms in at most 64 steps (16 channels of a
   lane, 3 joins, 16 steps of the tensor cores, which may truncate: 2^-23), its decays a product of at most D
   factors that are off by 2^-22 + 2^-24 each, and a path adds up at most D such errors:
   (D + 1)(64 + 8 D) 2^-24 A.  bf16 calls round both factors of the products with the state to 11 bits: 2 * 2^-11 A
   more, and the result, 2^-8 |o|.
 - States: per token the decay (2^-22 + 2^-24), a sum of dk / 8 + 3 steps and four more roundings: D (dk / 8 + 16) 2^-24 A.
 - L2-normalised rows: a sum of dk / 8 + 3 steps, rsqrt 2^-22, one product: 32 * 2^-24 of each factor (k twice).
 - Attention: as for one token per row (tests/lin_reference.py).
Copies and whole numbers are exact.
"""
import math
import random

import torch

from tests.lin_reference import U_OUT, _cpu


def tree(rng, m, kind="tree"):
    """parents of m drafted tokens."""
    if kind == "chain":
        return [i - 1 for i in range(m)]
    if kind == "star":
        return [-1] * m
    return [rng.randint(-1, i - 1) for i in range(m)]


def path(parents, i):
    p = []
    while i >= 0:
        p.append(i)
        i = parents[i]
    return p[::-1]


def drafts(seed, N, T, kind="tree", num=None):
    """(parents per row, int32 [N, T] tensor of them with anything behind a row's count)."""
    rng = random.Random(seed)
    m = [T] * N if num is None else num
    rows = [tree(rng, min(max(x, 0), T), kind) for x in m]
    full = [p + [rng.choice([-7, 0, T, 1 << 30]) for _ in range(T - len(p))] for p in rows]
    return rows, torch.tensor(full, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ KDA
def _normal(x, eps):
    den = x.square().sum(-1, keepdim=True) + eps
    return torch.where(den > 0, x / den.clamp_min(1e-300).sqrt(), torch.zeros_like(x))


def recurrent(q, k, v, g, beta, state, rows, idx=None, eps=None):
    """Per row, {token: (S, A)} of the state behind it (-1: the row's own), and outputs with their A; rows: parents per
    row; a slot outside the pool gives None."""
    q, k, v, g, beta, state = (_cpu(x) for x in (q, k, v, g, beta, state))
    if eps is not None:
        k = _normal(k, eps)
        q = None if q is None else _normal(q, eps)
    kept, out = [], torch.zeros_like(v)
    oabs = torch.zeros_like(v)
    for n, parents in enumerate(rows):
        slot = n if idx is None else int(idx[n])
        if not 0 <= slot < state.shape[0]:
            kept.append(None)
            continue
        S = {-1: (state[slot], state[slot].abs())}
        for i, p in enumerate(parents):
            a = g[n, i].exp()[:, :, None]
            kk, b = k[n, i][:, :, None], beta[n, i][:, None, None]
            s, A = a * S[p][0], a * S[p][1]
            e = v[n, i][:, None] - (kk * s).sum(1, keepdim=True)
            u = v[n, i][:, None].abs() + (kk.abs() * A).sum(1, keepdim=True)
            S[i] = s + b * kk * e, A + b.abs() * kk.abs() * u
            if q is not None:
                out[n, i] = torch.einsum("hij,hi->hj", S[i][0], q[n, i])
                oabs[n, i] = torch.einsum("hij,hi->hj", S[i][1], q[n, i].abs())
        kept.append(S)
    return kept, out, oabs


def depth(rows):
    return max((len(path(p, i)) for p in rows for i in range(len(p))), default=1)


def check_outputs(out, ref, oabs, rows, eps=None):
    D = depth(rows)
    c = (D + 1) * (64 + 8 * D) * 2.0 ** -24
    if out.dtype == torch.bfloat16:
        c += 2.0 ** -10
    if eps is not None:
        c += (D + 1) * 96 * 2.0 ** -24
    err = (out.detach().cpu().double() - ref).abs()
    bound = U_OUT[out.dtype] * ref.abs() + c * oabs + 1e-37
    assert bool((err <= bound).all()), float((err / bound).max())


def check_state(got, ref, A, D, dk, eps=None):
    c = D * (dk / 8 + 16 + (96 if eps is not None else 0)) * 2.0 ** -24
    err = (got.detach().cpu().double() - ref).abs()
    assert bool((err <= c * A + 1e-37).all()), float((err / (A + 1e-30)).max())


# ------------------------------------------------------------------ attention
def attention(q, kc, vc, table, lens, rows, scale):
    """(out, lse, bound on the error of out, of lse); rows: parents per row."""
    dt = q.dtype
    q, kc, vc = _cpu(q), _cpu(kc), _cpu(vc)
    N, T, Hq, d = q.shape
    pages, ps, Hkv = kc.shape[:3]
    rep = Hq // Hkv
    out = torch.zeros(N, T, Hq, d, dtype=torch.float64)
    lse = torch.full((N, T, Hq), -math.inf, dtype=torch.float64)
    tol, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    table = table.cpu()
    width = table.shape[1] * ps
    for n, parents in enumerate(rows):
        length = max(0, min(int(lens[n]), width))
        for i in range(len(parents)):
            pos = list(range(length)) + [length + j for j in path(parents, i)]
            at = [(int(table[n, t // ps]), t % ps) for t in pos if t < width]
            at = [x for x in at if 0 <= x[0] < pages]
            if not at:
                continue
            pg, off = (torch.tensor(x) for x in zip(*at))
            k, v = (x[pg, off].repeat_interleave(rep, 1) for x in (kc, vc))
            s = torch.einsum("hd,lhd->hl", q[n, i], k) * scale
            m = s.amax(-1, keepdim=True)
            fine = m.isfinite()
            p = torch.where(fine, (s - torch.where(fine, m, 0.0)).exp(), 0.0)
            tot = p.sum(-1, keepdim=True)
            p = p / tot.clamp_min(1e-300)
            out[n, i] = torch.einsum("hl,lhd->hd", p, v)
            lse[n, i] = (m + tot.log())[:, 0]
            ds = (d + 8) * 2.0 ** -23 * abs(scale) * torch.einsum("hd,lhd->hl", q[n, i].abs(), torch.where(k.isfinite(), k, 0.0).abs()).amax(-1, keepdim=True)
            tol[n, i] = (2 * ds + 2.0 ** -19 + 2.0 ** -15) * torch.einsum("hl,lhd->hd", p, v.abs()) + U_OUT[dt] * out[n, i].abs()
            tol_l[n, i] = (ds + 2.0 ** -19)[:, 0] + 2.0 ** -22 * torch.where(lse[n, i].isfinite(), lse[n, i].abs(), 0.0)
    return out, lse, tol, tol_l


# ------------------------------------------------------------------ pages
def fork(table, lens, refs, sources, new, ps):
    """(table, lens, refs, copies, short) as lists."""
    W, pages, N = len(table[0]), len(refs), len(table)
    free = [p for p, r in enumerate(refs) if r == 0]
    ok = lambda p: 0 <= p < pages  # noqa: E731
    after, rows, length, copies, seen, asked = list(refs), [], [], [], set(), 0
    for row in table:
        for p in row:
            if ok(p):
                after[p] -= 1
    for n in range(N):
        s, row, x, copy = sources[n], [-1] * W, 0, (-1, -1)
        if 0 <= s < N:
            x = min(max(lens[s], 0), W * ps)
            full, part = divmod(x, ps)
            heir = s not in seen
            seen.add(s)
            held = W if heir else full + (part > 0)
            row[:held] = [p if ok(p) else -1 for p in table[s][:held]]
            for e in range(full + (part > 0), held):     # room to write to: the row's own pages alone
                row[e] = row[e] if row[e] >= 0 and refs[row[e]] == 1 else -1
            need = min(W, -(-(x + max(0, new[n] if new else 0)) // ps))
            for e in range(W):
                shared = part > 0 and e == full and row[e] >= 0 and not (heir and refs[row[e]] == 1)
                if shared or (e < need and row[e] < 0):
                    p = free[asked] if asked < len(free) else -1
                    asked += 1
                    if shared:
                        copy = (row[e], p)
                    row[e] = p
        rows.append(row)
        length.append(x)
        copies.append(copy)
    if asked > len(free):
        return [list(r) for r in table], list(lens), list(refs), [(-1, -1)] * N, asked - len(free)
    for row in rows:
        for p in row:
            if ok(p):
                after[p] += 1
    return rows, length, after, copies, 0


def compact(table, refs):
    pages = len(refs)
    used = sum(r != 0 for r in refs)
    holes = [p for p in range(used) if refs[p] == 0]
    new, to, copies = list(refs), {}, []
    for p in range(used, pages):
        if refs[p]:
            to[p] = holes[len(copies)]
            copies.append((p, to[p]))
            new[to[p]], new[p] = refs[p], 0
    table = [[to.get(p, p) if 0 <= p < pages else -1 for p in row] for row in table]
    return table, new, copies + [(-1, -1)] * (pages // 2 - len(copies))
