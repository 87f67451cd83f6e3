"""Workloads of the serving operators beside Kimi Delta Attention: linear attention with a decay
for each head (prompts in chunks, single tokens on a state pool) and a paged key-value cache
(append, and attention of one new token per row).

A case is a dict of plain values.  ``run`` computes one pass: in its plain form from elementary
torch operations in 32 bits, or, with ``own`` set, through the library's calls.  ``exact`` is the
operators' definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}


# ----------------------------------------------------------------------------- cases
def _chunk(name, dtype, B, T, H, Hk, dk, dv, decay, init, N=0, lo=0):
    """Prompts: dense [B, T], or with N > 0 packed: N sequences of lo .. T tokens."""
    return dict(name=name, op="chunk", dtype=dtype, B=B, T=T, H=H, Hk=Hk, dk=dk, dv=dv,
                decay=decay, init=init, N=N, lo=lo)


def _step(name, dtype, N, H, Hk, dk, dv, decay, slots):
    """One token for each of N rows on a pool of `slots` states."""
    return dict(name=name, op="step", dtype=dtype, N=N, H=H, Hk=Hk, dk=dk, dv=dv, decay=decay,
                slots=slots)


def _append(name, dtype, N, lo, hi, past, Hkv, d, ps):
    """lo .. hi new tokens for each of N rows that hold up to `past` tokens (hi = 1: decode)."""
    return dict(name=name, op="append", dtype=dtype, N=N, lo=lo, hi=hi, past=past, Hkv=Hkv, d=d, ps=ps)


def _attend(name, dtype, N, lo, hi, Hq, Hkv, d, ps, empty=0):
    """One query token for each of N rows of lo .. hi cached tokens, `empty` of them without any."""
    return dict(name=name, op="attend", dtype=dtype, N=N, lo=lo, hi=hi, Hq=Hq, Hkv=Hkv, d=d, ps=ps,
                empty=empty)


def listed():
    return [
        # a short prompt in the fp32 checking mode: one call's latency
        _chunk("chunk_short_fp32", "fp32", 1, 256, 2, 2, 64, 64, "head", False),
        # the prefill workload of the benchmark, with a decay that depends on the token
        _chunk("chunk_prefill", "bf16", 4, 8192, 32, 32, 128, 128, "token", False),
        # one long prompt, few heads: fewer (sequence, head) pairs than SMs
        _chunk("chunk_long_few_heads", "bf16", 1, 32767, 8, 8, 128, 128, "token", True),
        # packed prompts of very different lengths resumed from cached states, q and k shared by 4 heads
        _chunk("chunk_packed_resume", "bf16", 1, 8192, 32, 8, 128, 128, "both", True, N=16, lo=100),
        # one conversation's next token: latency
        _step("step_one_row", "bf16", 1, 32, 32, 128, 128, "token", 3),
        # the decode workload of the benchmark
        _step("step_batch", "bf16", 256, 64, 64, 128, 128, "token", 256),
        # every conversation's new token into its last page
        _append("append_decode", "bf16", 256, 1, 1, 2048, 8, 128, 16),
        # ragged prompts written in one call, pages cut anywhere
        _append("append_prompts", "bf16", 12, 33, 8191, 500, 8, 128, 64),
        # one short conversation: latency
        _attend("attend_one_short", "bf16", 1, 777, 777, 32, 8, 128, 16),
        # one very long conversation, alone on the GPU
        _attend("attend_one_long", "bf16", 1, 131071, 131071, 64, 8, 128, 64),
        # a serving batch of very different lengths, one row still empty
        _attend("attend_batch", "bf16", 64, 200, 16384, 32, 8, 128, 16, empty=1),
        # fp32 checking mode, a head of keys for each query head, pages of an odd size
        _attend("attend_fp32_odd_pages", "fp32", 5, 3, 2500, 8, 8, 64, 13),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "step", "append", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op == "chunk":
        Hk = _log(rng, 1, 32)
        rep = rng.choice([1, 1, 2, 4])
        H, N, B, lo = Hk * rep, 0, 1, 0
        T = _log(rng, 1, 32768)
        if rng.random() < 0.4:
            N, lo = _log(rng, 2, 24), rng.choice([0, 1, 1 + T // 20])
            lo = min(lo, T)
        else:
            B = _log(rng, 1, 8)
        most = (1 << 20) if dtype == "bf16" else (1 << 16)      # tokens x heads
        T = max(1, min(T, most // (H * max(B, N))))
        lo = min(lo, T)
        return dict(op=op, dtype=dtype, B=B, T=T, H=H, Hk=Hk, dk=rng.choice([128, 128, 64]),
                    dv=rng.choice([128, 128, 64]), decay=rng.choice(["token", "head", "both", "none"]),
                    init=rng.random() < 0.5, N=N, lo=lo)
    if op == "step":
        N, Hk, rep = _log(rng, 1, 256), _log(rng, 1, 32), rng.choice([1, 1, 2])
        return dict(op=op, dtype=dtype, N=N, H=Hk * rep, Hk=Hk, dk=rng.choice([128, 128, 64]),
                    dv=rng.choice([128, 128, 64]), decay=rng.choice(["token", "head", "both", "none"]),
                    slots=N + rng.choice([0, 1, 7]))
    Hkv, d, ps = rng.choice([1, 2, 4, 8, 8, 16]), rng.choice([128, 128, 64]), rng.choice([1, 7, 16, 16, 32, 64, 100, 256])
    if op == "append":
        N = _log(rng, 1, 300)
        hi = 1 if rng.random() < 0.5 else _log(rng, 2, 8192)
        hi = max(1, min(hi, 65536 // N))
        return dict(op=op, dtype=dtype, N=N, lo=1 if hi == 1 else rng.randint(0, min(40, hi)), hi=hi,
                    past=_log(rng, 1, 2048), Hkv=Hkv, d=d, ps=ps)
    N, hi = _log(rng, 1, 200), _log(rng, 1, 131072)
    rep = rng.choice([1, 2, 4, 4, 5, 8, 12, 16])
    most = (1 << 22) // (Hkv * (2 if dtype == "fp32" else 1))   # cached tokens, N rows of hi
    hi = max(1, min(hi, most // N, most // (N * max(1, rep // 8))))
    return dict(op=op, dtype=dtype, N=N, lo=min(hi, rng.choice([1, 1 + hi // 10, hi])), hi=hi, Hq=Hkv * rep,
                Hkv=Hkv, d=d, ps=ps, empty=min(N - 1, rng.choice([0, 0, 1])))


def _spread(n, lo, hi):
    """n lengths spread over [lo, hi], evenly over their logarithm, the ends among them."""
    if n == 1 or lo == hi:
        return [hi] * n
    a, b = math.log(lo + 1), math.log(hi + 1)
    return [int(round(math.exp(a + (b - a) * i / (n - 1)))) - 1 for i in range(n)]


def _lengths(case):
    """The rows' lengths (their order comes from the seed)."""
    n = _spread(case["N"], case["lo"], case["T"] if case["op"] == "chunk" else case["hi"])
    for i in range(case.get("empty", 0)):
        n[i] = 0
    return n


def work(case):
    es = SIZE[case["dtype"]]
    if case["op"] in ("chunk", "step"):
        H, Hk, dk, dv = case["H"], case["Hk"], case["dk"], case["dv"]
        if case["op"] == "step":
            tokens, states = case["N"], 2 * case["N"]
        else:
            seqs = case["N"] or case["B"]
            tokens = sum(_lengths(case)) if case["N"] else case["B"] * case["T"]
            states = seqs * (2 if case["init"] else 1)
        per = es * (2 * Hk * dk + 2 * H * dv) + (4 * H if case["decay"] in ("token", "both") else 0)
        # the recurrence's least work a token and head: the state's update and its read-out
        return {"bytes": tokens * per + states * H * dk * dv * 4, "flops": tokens * H * 4 * dk * dv}
    row = case["Hkv"] * case["d"] * es
    tokens = sum(_lengths(case))
    if case["op"] == "append":
        return {"bytes": 4 * tokens * row, "flops": 0}
    q = case["N"] * case["Hq"]
    return {"bytes": 2 * tokens * row + q * (2 * case["d"] * es + 4), "flops": tokens * case["Hq"] * 4 * case["d"]}


# ----------------------------------------------------------------------------- inputs
def _unit(x):
    return x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)


def _decays(case, gen, dev, shape):
    """Log decays: of each token (softplus of its input, heads from slow to fast), and of each head."""
    H = case["H"]
    g = head = None
    if case["decay"] in ("token", "both"):
        rate = torch.exp(torch.linspace(math.log(2e-3), 0.0, H, device=dev))
        g = -rate * torch.nn.functional.softplus(torch.randn(shape, generator=gen, device=dev))
    if case["decay"] in ("head", "both"):
        head = -torch.exp2(-torch.linspace(1.0, 9.0, H, device=dev)) * (0.9 + 0.2 * torch.rand(H, generator=gen, device=dev))
    return g, head


def _shuffled(n, gen, dev):
    order = torch.randperm(len(n), generator=gen, device=dev)
    return torch.tensor(n, dtype=torch.int64, device=dev)[order]


def _offsets(n):
    return torch.nn.functional.pad(torch.cumsum(n, 0), (1, 0)).to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    rnd = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    st = {"case": case}
    if case["op"] in ("chunk", "step"):
        H, Hk, dk, dv = case["H"], case["Hk"], case["dk"], case["dv"]
        cu = None
        if case["op"] == "step":
            lead = (case["N"],)
        elif case["N"]:
            n = _shuffled(_lengths(case), gen, dev)
            cu = _offsets(n)
            lead = (1, sum(_lengths(case)))
        else:
            lead = (case["B"], case["T"])
        st["q"], st["k"] = _unit(rnd(*lead, Hk, dk)).to(dt), _unit(rnd(*lead, Hk, dk)).to(dt)
        st["v"] = rnd(*lead, H, dv).to(dt)
        st["g"], st["head_g"] = _decays(case, gen, dev, (*lead, H))
        if case["op"] == "step":
            st["state"] = 0.02 * rnd(case["slots"], H, dk, dv)
            st["rows"] = torch.randperm(case["slots"], generator=gen, device=dev)[: case["N"]].to(torch.int32)
        else:
            st["cu"] = cu
            seqs = case["N"] or case["B"]
            st["initial_state"] = 0.02 * rnd(seqs, H, dk, dv) if case["init"] else None
        return st
    N, Hkv, d, ps = case["N"], case["Hkv"], case["d"], case["ps"]
    n = _shuffled(_lengths(case), gen, dev)
    longest = case["hi"] + case.get("past", 0)
    width = -(-longest // ps)
    pages = N * width + 3
    st["table"] = torch.randperm(pages, generator=gen, device=dev)[: N * width].view(N, width).to(torch.int32)
    if case["op"] == "append":
        st["k_cache"], st["v_cache"] = (torch.zeros((pages, ps, Hkv, d), dtype=dt, device=dev) for _ in range(2))
        st["positions"] = torch.randint(0, case["past"] + 1, (N,), generator=gen, device=dev, dtype=torch.int32)
        st["cu"] = None if case["hi"] == 1 and case["lo"] == 1 else _offsets(n)
        tokens = sum(_lengths(case))
        st["k"], st["v"] = rnd(tokens, Hkv, d).to(dt), rnd(tokens, Hkv, d).to(dt)
        return st
    st["k_cache"], st["v_cache"] = (torch.empty((pages, ps, Hkv, d), dtype=dt, device=dev).normal_(generator=gen) for _ in range(2))
    st["q"] = (1.5 * rnd(N, case["Hq"], d)).to(dt)
    st["lens"] = n.to(torch.int32)
    st["scale"] = d ** -0.5
    return st


# ----------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    return {"chunk": _plain_chunk, "step": _plain_step, "append": _plain_append, "attend": _plain_attend}[op](state)


def _own(op, s):
    from linear_attention_fwd_gb300 import kda
    if op == "chunk":
        out, final = kda.kda_lin_chunk_fwd(s["q"], s["k"], s["v"], s["g"], s["head_g"], s["initial_state"], s["cu"])
        return {"out": out, "final_state": final}
    if op == "step":
        out = kda.kda_lin_recurrent_step(s["q"], s["k"], s["v"], s["g"], s["head_g"], s["state"], s["rows"])
        return {"out": out, "state": s["state"]}
    if op == "append":
        kda.kda_paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["positions"], s["cu"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    out, lse = kda.kda_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["scale"])
    return {"out": out, "lse": lse}


def _log_decay(g, head_g, shape, dev):
    """fp64 log decay [..., H]: the token's and the head's, either may be missing."""
    total = torch.zeros(shape, dtype=torch.float64, device=dev)
    if g is not None:
        total = total + g.double()
    if head_g is not None:
        total = total + head_g.double()
    return total


CHUNK = 64


def _dense_chunks(q, k, v, g, s0):
    """All chunks at once.  q, k [B, T, H, dk], v [B, T, H, dv] fp32, g [B, T, H] fp64 (sums of
    log decays are taken in fp64, their exponentials in fp32), s0 [B, H, dk, dv] or None."""
    B, T, H, dk = q.shape
    n = -(-T // CHUNK)
    pad = n * CHUNK - T
    split = lambda x: torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad)).view(B, n, CHUNK, H, -1).permute(0, 3, 1, 2, 4)  # noqa: E731
    q, k, v = split(q), split(k), split(v)
    G = torch.cumsum(split(g[..., None])[..., 0], -1)                 # [B, H, n, C]
    dev = q.device
    causal = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
    mask = (G[..., :, None] - G[..., None, :]).masked_fill(~causal, -math.inf).exp().float()
    out = ((q @ k.transpose(-1, -2)) * mask) @ v
    last = G[..., -1:]
    local = (k * (last - G).exp().float()[..., None]).transpose(-1, -2) @ v     # [B, H, n, dk, dv]
    E = torch.nn.functional.pad(torch.cumsum(last[..., 0], -1), (1, 0))         # before chunk c, 0 .. n
    before = torch.ones(n + 1, n, dtype=torch.bool, device=dev).tril(-1)
    D = (E[..., :, None] - E[..., None, 1:]).masked_fill(~before, -math.inf).exp().float()
    start = (D @ local.flatten(-2)).view(B, H, n + 1, dk, -1)
    if s0 is not None:
        start = start + E.exp().float()[..., None, None] * s0[:, :, None]
    out = out + G.exp().float()[..., None] * (q @ start[:, :, :-1])
    out = out.permute(0, 2, 3, 1, 4).reshape(B, n * CHUNK, H, -1)[:, :T]
    return out, start[:, :, -1]


def _plain_chunk(s):
    c, dt = s["case"], s["q"].dtype
    rep = c["H"] // c["Hk"]
    q, k = (s[x].float().repeat_interleave(rep, 2) for x in ("q", "k"))
    v = s["v"].float()
    g = _log_decay(s["g"], s["head_g"], (*v.shape[:2], c["H"]), v.device)
    if s["cu"] is None:
        out, final = _dense_chunks(q, k, v, g, s["initial_state"])
        return {"out": out.to(dt), "final_state": final}
    # packed sequences as rows of the longest one's length: zeros past a row's end, without decay
    cu = s["cu"].long()
    t = torch.arange(c["T"], device=v.device)
    at = cu[:-1, None] + t
    inside = at < cu[1:, None]
    at = at.clamp_max(v.shape[1] - 1)
    rows = lambda x: x[0][at] * inside[..., None, None]  # noqa: E731
    out, final = _dense_chunks(rows(q), rows(k), rows(v), rows(g[..., None])[..., 0], s["initial_state"])
    token = torch.arange(v.shape[1], device=v.device)
    seq = torch.searchsorted(cu[1:], token, right=True)
    return {"out": out[seq, token - cu[seq]][None].to(dt), "final_state": final}


def _plain_step(s):
    c = s["case"]
    rep = c["H"] // c["Hk"]
    q, k = (s[x].float().repeat_interleave(rep, 1) for x in ("q", "k"))
    v = s["v"].float()
    a = _log_decay(s["g"], s["head_g"], (c["N"], c["H"]), v.device).exp().float()
    rows = s["rows"].long()
    S = s["state"][rows] * a[..., None, None] + k[..., :, None] * v[..., None, :]
    s["state"][rows] = S
    return {"out": (q[..., None, :] @ S)[..., 0, :].to(s["q"].dtype), "state": s["state"]}


def _plain_append(s):
    c = s["case"]
    tokens, ps = s["k"].shape[0], c["ps"]
    u = torch.arange(tokens, device=s["k"].device)
    row, p = u, s["positions"].long()
    if s["cu"] is not None:
        cu = s["cu"].long()
        row = torch.searchsorted(cu[1:], u, right=True)
        p = s["positions"].long()[row] + u - cu[row]
    at = s["table"].long()[row, p // ps] * ps + p % ps
    s["k_cache"].view(-1, c["Hkv"], c["d"])[at] = s["k"]
    s["v_cache"].view(-1, c["Hkv"], c["d"])[at] = s["v"]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attend(s):
    c = s["case"]
    N, Hkv, d, ps = c["N"], c["Hkv"], c["d"], c["ps"]
    t = torch.arange(c["hi"], device=s["q"].device)
    at = s["table"].long()[:, t // ps] * ps + t % ps                       # [N, L]
    k, v = (s[x].view(-1, Hkv, d)[at].float().transpose(1, 2) for x in ("k_cache", "v_cache"))   # [N, Hkv, L, d]
    q = s["q"].float().view(N, Hkv, -1, d)
    score = (q @ k.transpose(-1, -2)) * s["scale"]
    score = score.masked_fill((t >= s["lens"][:, None])[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - top.clamp_min(-3e38)).exp()
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / total.clamp_min(1e-38)
    lse = (top + total.log())[..., 0]
    return {"out": out.reshape(N, -1, d).to(s["q"].dtype), "lse": lse.reshape(N, -1)}


# ----------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        for x in ("k", "v"):
            cache = s[x + "_cache"]
            for row, first in enumerate(s["positions"].tolist()):
                b, e = (row, row + 1) if s["cu"] is None else s["cu"][row: row + 2].tolist()
                pos = torch.arange(first, first + e - b, device=cache.device)
                cache[s["table"][row].long()[pos // case["ps"]], pos % case["ps"]] = s[x][b:e]
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if case["op"] == "attend":
        return _exact_attend(case, s)
    rep = case["H"] // case["Hk"]
    head = lambda x, dim: x.double().repeat_interleave(rep, dim)  # noqa: E731
    if case["op"] == "step":
        out = torch.empty(s["v"].shape, dtype=torch.float64, device="cuda")
        for n, slot in enumerate(s["rows"].tolist()):
            lg = torch.zeros(case["H"], dtype=torch.float64, device="cuda")
            lg = lg if s["g"] is None else lg + s["g"][n].double()
            lg = lg if s["head_g"] is None else lg + s["head_g"].double()
            S = lg.exp()[:, None, None] * s["state"][slot].double() + torch.einsum("hi,hj->hij", head(s["k"][n], 0), s["v"][n].double())
            out[n] = torch.einsum("hij,hi->hj", S, head(s["q"][n], 0))
            s["state"][slot] = S.float()
        return {"out": out, "state": s["state"].double()}
    # prompts: block by block, the state carried from one to the next
    H, dk, dv = case["H"], case["dk"], case["dv"]
    tokens = s["v"].shape[1]
    batch = s["cu"] is None
    cu = [0, tokens] if batch else s["cu"].tolist()
    seqs = case["B"] if batch else case["N"]
    out = torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
    final = torch.zeros(seqs, H, dk, dv, dtype=torch.float64, device="cuda")
    if s["initial_state"] is not None:
        final += s["initial_state"]
    step = 256
    for i, (b, e) in enumerate(zip(cu[:-1], cu[1:])):
        S = final if batch else final[i: i + 1]
        for t0 in range(b, e, step):
            t1 = min(e, t0 + step)
            q, k = head(s["q"][:, t0:t1], 2).transpose(1, 2), head(s["k"][:, t0:t1], 2).transpose(1, 2)
            v = s["v"][:, t0:t1].double().transpose(1, 2)
            lg = torch.zeros(v.shape[0], H, t1 - t0, dtype=torch.float64, device="cuda")
            lg = lg if s["g"] is None else lg + s["g"][:, t0:t1].double().transpose(1, 2)
            lg = lg if s["head_g"] is None else lg + s["head_g"].double()[None, :, None]
            G = lg.cumsum(-1)
            between = torch.exp((G[..., None] - G[..., None, :]).clamp_max(0)).tril()
            o = torch.einsum("bhij,bhjc->bhic", torch.einsum("bhid,bhjd->bhij", q, k) * between, v)
            o += torch.einsum("bhid,bhdc->bhic", q * G.exp()[..., None], S)
            out[:, t0:t1] = o.transpose(1, 2)
            S = G[..., -1].exp()[..., None, None] * S + torch.einsum("bhjd,bhjc->bhdc", k * (G[..., -1:] - G).exp()[..., None], v)
        if batch:
            final = S
        else:
            final[i] = S[0]
    return {"out": out, "final_state": final}


def _exact_attend(case, s):
    N, Hq, Hkv, d, ps = case["N"], case["Hq"], case["Hkv"], case["d"], case["ps"]
    out = torch.zeros(N, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((N, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for n, length in enumerate(s["lens"].tolist()):
        if length == 0:
            continue
        pages = s["table"][n, : -(-length // ps)].long()
        k, v = (s[x][pages].flatten(0, 1)[:length].double() for x in ("k_cache", "v_cache"))
        q = s["q"][n].double().view(Hkv, Hq // Hkv, d)
        score = torch.einsum("hgd,lhd->hgl", q, k) * s["scale"]
        lse[n] = torch.logsumexp(score, -1).flatten()
        out[n] = torch.einsum("hgl,lhd->hgd", torch.softmax(score, -1), v).reshape(Hq, d)
    return {"out": out, "lse": lse}
