"""Workloads of branching decode: a tree of drafted tokens verified at once by a hybrid stack's layers
(softmax attention over a paged cache, KDA on a pool of states), the accepted path kept, and rows that
fork, reorder and end on shared pages.

A case is a dict of plain values.  ``run`` computes one pass: in its plain form from elementary
torch operations in 32 bits, or, with ``own`` set, through the library's calls.  ``exact`` is the
operators' definition in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}


# ----------------------------------------------------------------------------- cases
def _attend(name, dtype, N, lo, hi, T, least, chain, Hq, Hkv, d, ps):
    """least .. T drafted tokens for each of N rows of lo .. hi cached tokens."""
    return dict(name=name, op="attend", dtype=dtype, N=N, lo=lo, hi=hi, T=T, least=least, chain=chain, Hq=Hq, Hkv=Hkv,
                d=d, ps=ps)


def _tree(name, op, dtype, N, T, least, chain, H, dk, dv, slots, none=0):
    """least .. T drafted tokens for each of N rows on a pool of states: `verify` gives every token's
    output, `replay` brings the accepted path into the state (`none` rows accept nothing)."""
    return dict(name=name, op=op, dtype=dtype, N=N, T=T, least=least, chain=chain, H=H, dk=dk, dv=dv, slots=slots, none=none)


def _keep(name, dtype, N, lo, hi, T, least, chain, Hkv, d, ps, none=0):
    """The accepted path's keys and values moved to the end of each row's cached tokens."""
    return dict(name=name, op="keep", dtype=dtype, N=N, lo=lo, hi=hi, T=T, least=least, chain=chain, Hkv=Hkv, d=d, ps=ps,
                none=none)


def _fork(name, dtype, N, lo, hi, group, new, spare, Hkv, d, ps):
    """N rows of lo .. hi tokens, `group` of them on one prompt's pages, continued by rows of their
    group, ended, or given room for `new` tokens; `spare` free pages; then one layer's copies."""
    return dict(name=name, op="fork", dtype=dtype, N=N, lo=lo, hi=hi, group=group, new=new, spare=spare, Hkv=Hkv, d=d, ps=ps)


def _compact(name, dtype, N, lo, hi, spare, Hkv, d, ps):
    """A pool with `spare` free pages among those of N rows of lo .. hi tokens, closed up; one layer's copies."""
    return dict(name=name, op="compact", dtype=dtype, N=N, lo=lo, hi=hi, spare=spare, Hkv=Hkv, d=d, ps=ps)


def listed():
    return [
        # one short conversation, a small draft: latency
        _attend("attend_one_small", "bf16", 1, 777, 777, 8, 8, False, 32, 8, 128, 16),
        # a serving batch of very different lengths and drafts
        _attend("attend_batch", "bf16", 32, 200, 16384, 32, 8, False, 32, 8, 128, 16),
        # one very long conversation, a large draft, alone on the GPU
        _attend("attend_long", "bf16", 1, 131071, 131071, 64, 64, False, 64, 8, 128, 64),
        # one conversation's draft through a KDA layer: latency
        _tree("verify_one", "verify", "bf16", 1, 8, 8, False, 32, 128, 128, 3),
        # a serving batch's drafts through a KDA layer
        _tree("verify_batch", "verify", "bf16", 64, 32, 8, False, 64, 128, 128, 80),
        # the accepted paths of the benchmark's decode batch, some rows with nothing accepted
        _tree("replay_batch", "replay", "bf16", 256, 16, 1, False, 64, 128, 128, 256, none=20),
        # one conversation in the fp32 checking mode: latency
        _keep("keep_one_fp32", "fp32", 1, 900, 900, 13, 13, False, 8, 64, 13),
        # a serving batch's accepted paths, pages cut anywhere
        _keep("keep_batch", "bf16", 256, 33, 2048, 32, 8, False, 8, 128, 16, none=20),
        # eight beams on one prompt, reordered for the next token: latency
        _fork("fork_beams", "bf16", 8, 700, 700, 8, 1, 64, 8, 128, 16),
        # a serving batch of sampled groups, some rows ended, all given room for a draft
        _fork("fork_batch", "bf16", 256, 100, 8000, 8, 32, 3000, 8, 128, 16),
        # a small pool in the fp32 checking mode: latency
        _compact("compact_small_fp32", "fp32", 4, 1, 900, 100, 2, 64, 7),
        # a pool of half-empty memory closed up before it shrinks
        _compact("compact_pool", "bf16", 128, 100, 8000, 12000, 8, 128, 16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "verify", "verify", "replay", "keep", "fork", "compact"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    T = _log(rng, 1, 64)
    least, chain = rng.choice([1, (T + 1) // 2, T]), rng.random() < 0.2
    if op in ("verify", "replay"):
        H, N = _log(rng, 1, 64), _log(rng, 1, 256)
        N = max(1, min(N, (64 * 64 * 32) // (H * max(T, 8))))       # rows x heads x tokens
        return dict(op=op, dtype=dtype, N=N, T=T, least=least, chain=chain, H=H, dk=rng.choice([128, 128, 64]),
                    dv=rng.choice([128, 128, 64]), slots=N + rng.choice([0, 1, 7]),
                    none=min(N - 1, rng.choice([0, 1, N // 4])) if op == "replay" else 0)
    Hkv, d, ps = rng.choice([1, 2, 4, 8, 8, 16]), rng.choice([128, 128, 64]), rng.choice([1, 7, 16, 16, 32, 64, 100, 256])
    if op == "attend":
        N, hi, rep = _log(rng, 1, 128), _log(rng, 1, 131072), rng.choice([1, 2, 4, 4, 5, 8, 16])
        cells = (1 << 29) // (2 if dtype == "fp32" else 1)          # scores
        most = (1 << 20) // (2 if dtype == "fp32" else 1)           # cached tokens x key/value heads, of N rows of hi
        hi = max(1, min(hi, most // (N * Hkv), cells // (N * Hkv * rep * T)))
        return dict(op=op, dtype=dtype, N=N, lo=min(hi, rng.choice([0, 1, 1 + hi // 10, hi])), hi=hi, T=T, least=least,
                    chain=chain, Hq=Hkv * rep, Hkv=Hkv, d=d, ps=ps)
    N, hi = _log(rng, 1, 256), _log(rng, 1, 8192)
    if op == "keep":
        hi = max(1, min(hi, (1 << 19) // N))
        return dict(op=op, dtype=dtype, N=N, lo=rng.choice([0, hi // 10, hi]), hi=hi, T=T, least=least, chain=chain, Hkv=Hkv,
                    d=d, ps=ps, none=min(N - 1, rng.choice([0, 1, N // 4])))
    hi = max(1, min(hi, (1 << 18) // (N * max(1, Hkv // 4))))
    lo = rng.choice([0, hi // 10, hi])
    held = N * -(-hi // ps)
    if op == "fork":
        new = rng.choice([0, 1, 1, T])
        return dict(op=op, dtype=dtype, N=N, lo=lo, hi=hi, group=rng.choice([1, 2, 4, 8]), new=new,
                    spare=rng.choice([0, N // 2, 2 * N + N * (new // ps), 1 + held // 2]), Hkv=Hkv, d=d, ps=ps)
    return dict(op=op, dtype=dtype, N=N, lo=lo, hi=hi, spare=1 + rng.choice([0, held // 4, held]), Hkv=Hkv, d=d, ps=ps)


def _spread(n, lo, hi):
    """n whole numbers spread over [lo, hi], evenly over their logarithm, the ends among them."""
    if n == 1 or lo == hi:
        return [hi] * n
    a, b = math.log(lo + 1), math.log(hi + 1)
    return [int(round(math.exp(a + (b - a) * i / (n - 1)))) - 1 for i in range(n)]


def _drafts(case):
    """Each row's drafted tokens: their number and the token each one continues (-1: the row itself)."""
    rng = random.Random(case["N"] * 1000 + case["T"])
    m = _spread(case["N"], case["least"], case["T"])
    rng.shuffle(m)
    chain = case["chain"]
    return m, [[i - 1 if chain else rng.randint(-1, i - 1) for i in range(n)] for n in m]


def _path(parents, i):
    """The tokens from the first drafted one to token i."""
    path = []
    while i >= 0:
        path.append(i)
        i = parents[i]
    return path[::-1]


def _accepted(case):
    """The last accepted token of each row (-1: none), as a sampler may leave it: anywhere in the tree, late tokens
    rather than early ones."""
    m, parents = _drafts(case)
    rng = random.Random(case["N"] + case["T"])
    return [-1 if n < case["none"] else max(rng.randrange(m[n]), rng.randrange(m[n])) for n in range(case["N"])], parents


def work(case):
    es, N = SIZE[case["dtype"]], case["N"]
    if case["op"] in ("verify", "replay"):
        H, dk, dv = case["H"], case["dk"], case["dv"]
        state = H * dk * dv * 4
        if case["op"] == "replay":
            last, parents = _accepted(case)
            tokens = sum(len(_path(p, i)) for p, i in zip(parents, last))
            return {"bytes": 2 * state * (N - case["none"]) + tokens * H * es * (2 * dk + dv + 1), "flops": tokens * H * 4 * dk * dv}
        m, parents = _drafts(case)
        tokens, pairs = sum(m), sum(len(_path(p, i)) for p in parents for i in range(len(p)))
        return {"bytes": state * N + tokens * H * es * (3 * dk + 2 * dv + 1), "flops": H * (tokens * 4 * dk * dv + pairs * 4 * (dk + dv))}
    row = case["Hkv"] * case["d"] * es
    if case["op"] == "attend":
        m, parents = _drafts(case)
        n = _spread(N, case["lo"], case["hi"])
        n = [n[i] for i in _order(case)]
        cells = sum(a * b for a, b in zip(m, n)) + sum(len(_path(p, i)) for p in parents for i in range(len(p)))
        return {"bytes": 2 * (sum(n) + sum(m)) * row + sum(m) * case["Hq"] * (2 * case["d"] * es + 4), "flops": cells * case["Hq"] * 4 * case["d"]}
    if case["op"] == "keep":
        last, parents = _accepted(case)
        # a token that stays where it is need not be moved
        moved = sum(sum(a != r for r, a in enumerate(_path(p, i))) for p, i in zip(parents, last))
        return {"bytes": 4 * moved * row + 4 * N * case["T"], "flops": 0}
    pages, width, copies = _pool_size(case)
    return {"bytes": 4 * copies * case["ps"] * row + 8 * (N * width + pages), "flops": 0}


def _order(case):
    """Which of the spread lengths each row has."""
    order = list(range(case["N"]))
    random.Random(case["N"] + 7).shuffle(order)
    return order


# ----------------------------------------------------------------------------- inputs
def _unit(x):
    return x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)


def _held(case):
    """How the rows hold pages: (row lengths, the row each one shares its first pages with, how many)."""
    n = _spread(case["N"], case["lo"], case["hi"])
    group, ps = case.get("group", 1), case["ps"]
    n = [n[i // group * group] + i % group * (n[i // group * group] > 0) for i in range(case["N"])]
    lead = [i // group * group for i in range(case["N"])]
    return n, lead, [0 if lead[i] == i else n[lead[i]] // ps for i in range(case["N"])]


def _sources(case):
    """The row that each row continues (-1: it ends): its own, or one of its group's best."""
    rng = random.Random(case["N"] + case["hi"])
    g, N = case["group"], case["N"]
    return [-1 if g > 1 and rng.random() < 0.1 else i // g * g + rng.randrange(min(g, N - i // g * g)) if rng.random() < 0.5 else i
            for i in range(N)]


def _pool_size(case):
    """(pages of the pool, width of the block table, pages copied)."""
    n, _, shared = _held(case)
    ps = case["ps"]
    c = [-(-x // ps) for x in n]
    used = sum(c) - sum(shared)
    pages = max(1, used + case["spare"])
    width = max(1, -(-(max(n) + case.get("new", 0)) // ps))
    if case["op"] == "compact":
        return pages, width, sum(_in_use(case, pages, used)[used:])
    src = _sources(case)
    first = {}
    for i, s in enumerate(src):
        first.setdefault(s, i)
    copied = sum(s >= 0 and n[s] % ps > 0 and first[s] != i for i, s in enumerate(src))
    asked = copied + sum(max(0, -(-(n[s] + case["new"]) // ps) - c[s]) for s in src if s >= 0)
    return pages, width, copied if asked <= case["spare"] else 0


def _in_use(case, pages, used):
    """Which pages are in use."""
    return [x < used for x in random.Random(pages).sample(range(pages), pages)]


def _prepare_pool(case, gen, dev):
    n, lead, shared = _held(case)
    ps, N = case["ps"], case["N"]
    pages, width, _ = _pool_size(case)
    c = [-(-x // ps) for x in n]
    used = sum(c) - sum(shared)
    mask = torch.tensor(_in_use(case, pages, used), device=dev)
    at = mask.nonzero()[:, 0]
    at = at[torch.randperm(used, generator=gen, device=dev)].tolist()
    table = [[-1] * width for _ in range(N)]
    for i in range(N):
        table[i][: shared[i]] = table[lead[i]][: shared[i]]
        k = c[i] - shared[i]
        table[i][shared[i]: c[i]] = at[:k]
        del at[:k]
    st = {"table": torch.tensor(table, dtype=torch.int32, device=dev)}
    valid = st["table"][st["table"] >= 0].long()
    st["refs"] = torch.bincount(valid, minlength=pages).to(torch.int32)
    st["lens"] = torch.tensor(n, dtype=torch.int32, device=dev)
    if case["op"] == "fork":
        st["sources"] = torch.tensor(_sources(case), dtype=torch.int32, device=dev)
        st["new"] = torch.full((N,), case["new"], dtype=torch.int32, device=dev) if case["new"] else None
    return st, pages


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    rnd = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    st = {"case": case}
    N = case["N"]
    if "T" in case:
        T = case["T"]
        m, parents = _drafts(case)
        st["num"] = None if min(m) == T else i32(m)
        # what lies behind a row's tokens says nothing
        st["parents"] = None if case["chain"] else i32([p + [-1] * (T - len(p)) for p in parents])
        if "none" in case:
            st["accepted"] = i32(_accepted(case)[0])
    if case["op"] in ("verify", "replay"):
        H, dk, dv = case["H"], case["dk"], case["dv"]
        st["q"], st["k"] = _unit(rnd(N, T, H, dk)).to(dt), _unit(rnd(N, T, H, dk)).to(dt)
        st["v"] = rnd(N, T, H, dv).to(dt)
        st["g"] = (-5 * torch.sigmoid(2 * rnd(N, T, H, dk) - 3)).to(dt)
        st["beta"] = torch.sigmoid(rnd(N, T, H)).to(dt)
        st["state"] = 0.1 * rnd(case["slots"], H, dk, dv)
        st["rows"] = torch.randperm(case["slots"], generator=gen, device=dev)[:N].to(torch.int32)
        return st
    Hkv, d, ps = case["Hkv"], case["d"], case["ps"]
    if case["op"] in ("fork", "compact"):
        more, pages = _prepare_pool(case, gen, dev)
        st.update(more)
    else:
        n = _spread(N, case["lo"], case["hi"])
        st["lens"] = i32([n[i] for i in _order(case)])
        width = -(-(case["hi"] + T) // ps)
        pages = N * width + 3
        st["table"] = torch.randperm(pages, generator=gen, device=dev)[: N * width].view(N, width).to(torch.int32)
    st["k_cache"], st["v_cache"] = (torch.empty((pages, ps, Hkv, d), dtype=dt, device=dev).normal_(generator=gen) for _ in range(2))
    if case["op"] == "attend":
        st["q"] = (1.5 * rnd(N, T, case["Hq"], d)).to(dt)
        st["scale"] = d ** -0.5
    return st


# ----------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    return {"attend": _plain_attend, "verify": _plain_verify, "replay": _plain_replay, "keep": _plain_keep, "fork": _plain_fork,
            "compact": _plain_compact}[op](state)


def _own(op, s):
    from linear_attention_fwd_gb300 import kda
    if op == "attend":
        out, lse = kda.kda_paged_tree_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["parents"], s["scale"],
                                                s["num"])
        return {"out": out, "lse": lse}
    if op == "verify":
        return {"out": kda.kda_recurrent_tree(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["parents"], s["rows"], s["num"])}
    if op == "replay":
        kda.kda_recurrent_tree_commit(s["k"], s["v"], s["g"], s["beta"], s["state"], s["parents"], s["accepted"], s["rows"], s["num"])
        return {"state": s["state"]}
    if op == "keep":
        lens = kda.kda_paged_tree_commit(s["k_cache"], s["v_cache"], s["table"], s["lens"], s["parents"], s["accepted"], s["num"])
        return {"lens": lens, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "fork":
        table, lens, refs, copies, short = kda.kda_paged_fork(s["table"], s["lens"], s["refs"], s["sources"], s["new"],
                                                              page_size=s["case"]["ps"])
        kda.kda_paged_copy(s["k_cache"], s["v_cache"], copies)
        return {"table": table, "lens": lens, "refs": refs, "copies": copies, "short": short, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    table, refs, copies = kda.kda_paged_compact(s["table"], s["refs"])
    kda.kda_paged_copy(s["k_cache"], s["v_cache"], copies)
    return {"table": table, "refs": refs, "copies": copies, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _square(x):
    """Reach over twice as many steps."""
    return ((x @ x) > 0).float()


def _ancestors(s):
    """fp32 [N, T, T], 1 where token j lies on the path to token i (i itself among them), and the tokens' own mask [N, T]."""
    c = s["case"]
    T, dev = c["T"], s["lens" if "lens" in s else "rows"].device
    i = torch.arange(T, device=dev)
    up = s["parents"].long() if s["parents"] is not None else (i - 1).expand(c["N"], T)
    step = (up[:, :, None] == i).float() + torch.eye(T, device=dev)
    reach = _square(_square(_square(_square(_square(_square(step))))))
    here = i < s["num"][:, None] if s["num"] is not None else torch.ones(c["N"], T, dtype=torch.bool, device=dev)
    return reach * here[:, :, None] * here[:, None, :], here


def _places(s, pos):
    """Index of each position [N, L] of the rows in a cache of single tokens, and where there is one."""
    ps, table = s["case"]["ps"], s["table"].long()
    inside = (pos >= 0) & (pos < table.shape[1] * ps)
    pos = pos.clamp(0, table.shape[1] * ps - 1)
    page = table.gather(1, pos // ps)
    inside &= (page >= 0) & (page < s["k_cache"].shape[0])
    return page.clamp(0, s["k_cache"].shape[0] - 1) * ps + pos % ps, inside


def _plain_attend(s):
    c = s["case"]
    N, T, Hkv, d = c["N"], c["T"], c["Hkv"], c["d"]
    reach, here = _ancestors(s)
    t = torch.arange(c["hi"], device=s["q"].device)
    lens = s["lens"].long()
    pos = torch.cat([t.expand(N, -1), lens[:, None] + torch.arange(T, device=t.device)], 1)
    at, inside = _places(s, pos)                                                                        # [N, L]
    past = ((t < lens[:, None])[:, None, :] & here[:, :, None])
    see = (torch.cat([past, reach > 0], 2) & inside[:, None, :])[:, None, :, None]                      # [N, 1, T, 1, L]
    k, v = (s[x].view(-1, Hkv, d)[at].float().transpose(1, 2) for x in ("k_cache", "v_cache"))          # [N, Hkv, L, d]
    q = s["q"].float().view(N, T, Hkv, -1, d).transpose(1, 2)                                           # [N, Hkv, T, rep, d]
    score = (q.flatten(2, 3) @ k.transpose(-1, -2)).view(N, Hkv, T, -1, pos.shape[1]) * s["scale"]
    score = score.masked_fill(~see, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - top.clamp_min(-3e38)).exp()
    total = p.sum(-1, keepdim=True)
    out = (p.flatten(2, 3) @ v).view(N, Hkv, T, -1, d) / total.clamp_min(1e-38)
    lse = (top + total.log())[..., 0]
    return {"out": out.transpose(1, 2).reshape(N, T, -1, d).to(s["q"].dtype), "lse": lse.transpose(1, 2).reshape(N, T, -1)}


def _inverse(a):
    """(1 + a)^-1 of strictly lower triangular a, of at most 64 rows."""
    one = torch.eye(a.shape[-1], device=a.device)
    b = a @ a
    inv = (one - a) @ (one + b)
    b = b @ b
    inv = inv @ (one + b)
    b = b @ b
    inv = inv @ (one + b)
    b = b @ b
    inv = inv @ (one + b)
    b = b @ b
    return inv @ (one + b)


def _corrections(s, reach, S):
    """What each token writes, u [N, H, T, dv] (S_i = E_i S + sum_j E_ij k_j u_j^T), E_ij k_j [N, H, T, T, dk] and E_i [N, H, T, dk]:
    the decays on the path from j (excluded), or from the row's state, to i."""
    k, v = (s[x].float().transpose(1, 2) for x in ("k", "v"))
    beta = s["beta"].float().transpose(1, 2)[..., None]
    G = reach[:, None].double() @ s["g"].double().transpose(1, 2)                                       # sums along each path
    before = (reach * (1 - torch.eye(reach.shape[-1], device=S.device)))[:, None, :, :, None]
    between = (G[:, :, :, None] - G[:, :, None]).float().masked_fill(reach[:, None, :, :, None] == 0, -math.inf).exp()
    ek = between * k[:, :, None]
    first = G.float().exp()
    a = beta * (ek * before * k[:, :, :, None]).sum(-1)
    return _inverse(a) @ (beta * (v - (k * first) @ S)), ek, first


def _plain_verify(s):
    reach, here = _ancestors(s)
    S = s["state"][s["rows"].long()]
    u, ek, first = _corrections(s, reach, S)
    q = s["q"].float().transpose(1, 2)
    out = (q * first) @ S + (ek * q[:, :, :, None]).sum(-1) @ u
    return {"out": (out * here[:, None, :, None]).transpose(1, 2).to(s["q"].dtype).contiguous()}


def _plain_replay(s):
    reach, _ = _ancestors(s)
    rows = s["rows"].long()
    S = s["state"][rows]
    u, ek, first = _corrections(s, reach, S)
    n = torch.arange(rows.shape[0], device=S.device)
    last = s["accepted"].long()
    some = (last >= 0)[:, None, None, None]
    last = last.clamp_min(0)
    new = first[n, :, last][..., None] * S + ek[n, :, last].transpose(-1, -2) @ u
    s["state"][rows] = torch.where(some, new, S)
    return {"state": s["state"]}


def _plain_keep(s):
    c = s["case"]
    reach, _ = _ancestors(s)
    T = c["T"]
    lens, last = s["lens"].long(), s["accepted"].long()
    path = (reach[torch.arange(c["N"], device=lens.device), last.clamp_min(0)] > 0) & (last >= 0)[:, None]
    rank = path.cumsum(1) - 1
    frm, a = _places(s, lens[:, None] + torch.arange(T, device=lens.device))
    to, b = _places(s, lens[:, None] + rank)
    do = path & a & b
    frm, to = frm[do], to[do]
    k, v = (s[x].view(-1, c["Hkv"], c["d"]) for x in ("k_cache", "v_cache"))
    k[to], v[to] = k[frm], v[frm]
    return {"lens": (lens + path.sum(1)).to(torch.int32), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _copy_pages(s, copies):
    done = copies[copies[:, 0] >= 0].long()
    s["k_cache"][done[:, 1]] = s["k_cache"][done[:, 0]]
    s["v_cache"][done[:, 1]] = s["v_cache"][done[:, 0]]


def _plain_fork(s):
    ps, table, lens, refs = s["case"]["ps"], s["table"].long(), s["lens"].long(), s["refs"].long()
    (N, W), pages, dev = table.shape, refs.shape[0], table.device
    i = torch.arange(N, device=dev)
    src = s["sources"].long()
    live = (src >= 0) & (src < N)
    at = src.clamp(0, N - 1)
    length = torch.where(live, lens.clamp(0, W * ps)[at], 0)
    first = torch.full((N + 1,), N, device=dev).scatter_reduce(0, torch.where(live, at, N), i, "amin")
    heir = live & (first[at] == i)
    full, part = length // ps, length % ps > 0
    e = torch.arange(W, device=dev)
    rows = torch.where(live[:, None] & (heir[:, None] | (e < (full + part)[:, None])), table[at], -1)
    last = rows.gather(1, full.clamp_max(W - 1)[:, None])[:, 0]
    shared = part & (last >= 0) & (last < pages) & ~(heir & (refs[last.clamp(0, pages - 1)] == 1))
    new = s["new"].long().clamp_min(0) if s["new"] is not None else torch.zeros_like(lens)
    need = torch.where(live, -((-(length + new)) // ps), 0).clamp_max(W)
    wanted = (e < need[:, None]) & ((rows < 0) | (rows >= pages)) | (shared[:, None] & (e == full[:, None]))
    free = torch.sort((refs != 0).int(), stable=True)[1]
    missing = (wanted.sum() - (refs == 0).sum()).clamp_min(0)
    given = free[(wanted.flatten().cumsum(0) - 1).clamp(0, pages - 1)].view(N, W)
    ok = missing == 0
    out = torch.where(ok, torch.where(wanted, given, rows), table)
    count = lambda x: torch.zeros(pages + 1, dtype=torch.long, device=dev).index_add_(  # noqa: E731
        0, torch.where((x >= 0) & (x < pages), x, pages).flatten(), torch.ones(N * W, dtype=torch.long, device=dev))[:pages]
    copies = torch.stack([last, out.gather(1, full.clamp_max(W - 1)[:, None])[:, 0]], 1)
    copies = torch.where((ok & shared)[:, None], copies, -1).to(torch.int32)
    _copy_pages(s, copies)
    return {"table": out.to(torch.int32), "lens": torch.where(ok, length, lens).to(torch.int32), "refs": (refs - count(table) + count(out)).to(torch.int32),
            "copies": copies, "short": missing.to(torch.int32).view(1), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_compact(s):
    table, refs = s["table"].long(), s["refs"]
    pages, dev = refs.shape[0], refs.device
    p = torch.arange(pages, device=dev)
    used = refs != 0
    front = p < used.sum()
    moved, hole = used & ~front, ~used & front
    most = pages // 2
    slot = lambda mask: torch.where(mask, mask.cumsum(0) - 1, most)  # noqa: E731
    copies = torch.full((most + 1, 2), -1, device=dev)
    copies[slot(moved), 0] = p
    copies[slot(hole), 1] = p
    to = torch.cat([copies[:, 1], p.new_zeros(1)])[torch.where(moved, moved.cumsum(0) - 1, 0)]
    to = torch.where(moved, to, p)
    inside = (table >= 0) & (table < pages)
    out = torch.where(inside, to[table.clamp(0, pages - 1)], table).to(torch.int32)
    new = torch.zeros_like(refs)
    new[to[used]] = refs[used]
    copies = copies[:most].to(torch.int32).contiguous()
    _copy_pages(s, copies)
    return {"table": out, "refs": new, "copies": copies, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# ----------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "verify": _exact_tree, "replay": _exact_tree, "keep": _exact_keep, "fork": _exact_fork,
            "compact": _exact_compact}[case["op"]](case, s)


def _exact_attend(case, s):
    N, T, Hq, Hkv, d, ps = (case[x] for x in ("N", "T", "Hq", "Hkv", "d", "ps"))
    m, parents = _drafts(case)
    out = torch.zeros(N, T, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((N, T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for n, length in enumerate(s["lens"].tolist()):
        end = length + m[n]
        pages = s["table"][n, : -(-end // ps)].long()
        k, v = (s[x][pages].flatten(0, 1)[:end].double() for x in ("k_cache", "v_cache"))
        q = s["q"][n, : m[n]].double().view(m[n], Hkv, Hq // Hkv, d)
        score = torch.einsum("thgd,lhd->thgl", q, k) * s["scale"]
        for i in range(m[n]):
            out_of_path = [length + j for j in range(m[n]) if j not in _path(parents[n], i)]
            score[i, :, :, out_of_path] = -math.inf
        lse[n, : m[n]] = torch.logsumexp(score, -1).flatten(1)
        out[n, : m[n]] = torch.einsum("thgl,lhd->thgd", torch.softmax(score, -1), v).reshape(m[n], Hq, d)
    return {"out": out, "lse": lse}


def _exact_tree(case, s):
    m, parents = _drafts(case)
    replay = case["op"] == "replay"
    last = s["accepted"].tolist() if replay else None
    out = torch.zeros(case["N"], case["T"], case["H"], case["dv"], dtype=torch.float64, device="cuda")
    state = s["state"].double()
    for n, slot in enumerate(s["rows"].tolist()):
        start = state[slot]
        kept = {-1: start}
        for i in (_path(parents[n], last[n]) if replay else range(m[n])):
            k, v, g, beta = (s[x][n, i].double() for x in ("k", "v", "g", "beta"))
            S = g.exp()[:, :, None] * kept[parents[n][i]]
            e = v - torch.einsum("hij,hi->hj", S, k)
            S = S + beta[:, None, None] * k[:, :, None] * e[:, None, :]
            kept[i] = S
            if not replay:
                out[n, i] = torch.einsum("hij,hi->hj", S, s["q"][n, i].double())
        if replay:
            state[slot] = kept[last[n]]
    return {"state": state} if replay else {"out": out}


def _exact_keep(case, s):
    last, parents = _accepted(case)
    lens = s["lens"].tolist()
    table, ps = s["table"].tolist(), case["ps"]
    place = lambda n, pos: table[n][pos // ps] * ps + pos % ps  # noqa: E731
    frm, to = [], []
    for n in range(case["N"]):
        path = _path(parents[n], last[n])
        frm += [place(n, lens[n] + a) for a in path]
        to += [place(n, lens[n] + r) for r in range(len(path))]
        lens[n] += len(path)
    frm, to = (torch.tensor(x, dtype=torch.long, device="cuda") for x in (frm, to))
    for x in ("k_cache", "v_cache"):
        flat = s[x].view(-1, case["Hkv"], case["d"])
        flat[to] = flat[frm]
    return {"lens": torch.tensor(lens, dtype=torch.int32), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _exact_copies(s, copies):
    for a, b in copies:
        if a >= 0:
            s["k_cache"][b], s["v_cache"][b] = s["k_cache"][a].clone(), s["v_cache"][a].clone()


def _exact_fork(case, s):
    ps, new = case["ps"], case["new"]
    table, lens, refs, src = (s[x].tolist() for x in ("table", "lens", "refs", "sources"))
    W = len(table[0])
    free = [p for p, r in enumerate(refs) if r == 0]
    after, rows, length, copies, seen, wanted = list(refs), [], [], [], set(), 0
    for row in table:
        for p in row:
            if p >= 0:
                after[p] -= 1
    for n, a in enumerate(src):
        row, x, copy = [-1] * W, 0, (-1, -1)
        if a >= 0:
            x = lens[a]
            full, part = divmod(x, ps)
            keeps = a not in seen
            seen.add(a)
            row[: full + (part > 0)] = table[a][: full + (part > 0)]
            if keeps:
                row = list(table[a])
            if part and not (keeps and refs[row[full]] == 1):
                copy = (row[full], free[wanted] if wanted < len(free) else -1)
                row[full] = copy[1]
                wanted += 1
            for e in range(min(W, -(-(x + new) // ps))):
                if row[e] == -1:
                    row[e] = free[wanted] if wanted < len(free) else -1
                    wanted += 1
        rows.append(row)
        length.append(x)
        copies.append(copy)
        for p in row:
            if p >= 0:
                after[p] += 1
    short = max(0, wanted - len(free))
    if short:
        rows, length, after, copies = table, lens, refs, [(-1, -1)] * len(src)
    _exact_copies(s, copies)
    whole = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return {"table": whole(rows), "lens": whole(length), "refs": whole(after), "copies": whole(copies), "short": whole([short]),
            "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _exact_compact(case, s):
    refs = s["refs"].tolist()
    pages = len(refs)
    used = sum(r != 0 for r in refs)
    holes = [p for p in range(used) if refs[p] == 0]
    to, copies = list(range(pages)), []
    for p in range(used, pages):
        if refs[p] != 0:
            to[p] = holes[len(copies)]
            copies.append((p, to[p]))
            refs[to[p]], refs[p] = refs[p], 0
    _exact_copies(s, copies)
    copies += [(-1, -1)] * (pages // 2 - len(copies))
    table = [[to[p] if p >= 0 else p for p in row] for row in s["table"].tolist()]
    whole = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return {"table": whole(table), "refs": whole(refs), "copies": whole(copies).view(-1, 2), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
