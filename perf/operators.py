"""The token mixers of hybrid models next to the selective scan, as cases to measure: linear attention with a decay per
head (prompt and single token), attention of one new token over a paged key-value cache, and eviction from that cache by
accumulated attention weight.

``run`` computes each operator in its plain form (float32 torch operations, rounded once at the end), or, where ``own``
is true, through the library's entry points.  ``exact`` computes the same from the definitions in float64, in another
form: token by token, sequence by sequence.

Definitions.

Linear attention, per batch entry b and head h (q, k of head h / (H / Hk)), state S of P x N (values by keys)::

    S_t   = exp(g[b,h,t]) S_{t-1} + v_t k_t^T          g: log decay, per head or per head and token
    out_t = scale * S_t q_t                             tokens at or past seq_lens[b] are not there

Attention of one new token over a paged cache: token t of sequence b lies in row t % page of page table[b, t // page];
a page index outside the pool holds no tokens::

    p[t] = softmax over t < seq_lens[b] of scale * q . k_t,     out = sum_t p[t] v_t
    weights_out[b,hk,t] = weights[b,hk,t] + sum over the query heads of hk of p[t]        (where asked for)

Eviction keeps min(keep, length) tokens of each sequence and key-value head: its last `recent` tokens and, of the
others, those of the largest accumulated weight (the lowest position first among equals), copied in order of position
into the pages of another table.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_ES = {"f32": 4, "f16": 2, "bf16": 2}
_CHUNK = 64  # tokens per chunk of the plain form of the prompt


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # a short prompt of one user, where launches and latency count
        dict(name="linattn prompt short", op="prompt", io="bf16", B=1, H=8, Hk=8, L=100, N=64, P=64,
             decay="head", ragged=False),
        # the batch and length of the prefill benchmark, the head sizes of the Mamba-2 layout, decay per head
        dict(name="linattn prompt batch", op="prompt", io="bf16", B=4, H=32, Hk=32, L=2048, N=128, P=128,
             decay="head", ragged=False),
        # a long document of one user; keys shared by groups of heads, a decay gate per token
        dict(name="linattn prompt long", op="prompt", io="f16", B=1, H=32, Hk=8, L=16384, N=128, P=128,
             decay="token", ragged=False),
        # a padded batch of prompts of different lengths, odd head sizes
        dict(name="linattn prompt padded", op="prompt", io="bf16", B=7, H=12, Hk=12, L=1013, N=96, P=72,
             decay="token", ragged=True),
        # single precision, as a numerics check or a small model runs it
        dict(name="linattn prompt f32", op="prompt", io="f32", B=2, H=16, Hk=16, L=1024, N=64, P=64,
             decay="head", ragged=False),
        # one user's decode step: one token, latency
        dict(name="linattn step one", op="step", io="bf16", state="f32", B=1, H=32, Hk=32, N=128, P=128,
             slots=1, decay="head"),
        # continuous batching at the concurrency of the decode benchmark, slots in a larger pool
        dict(name="linattn step batch", op="step", io="bf16", state="f32", B=245, H=32, Hk=8, N=128, P=128,
             slots=300, decay="token"),
        # one user's decode step over a few thousand cached tokens
        dict(name="paged one", op="paged", io="bf16", B=1, Hq=32, Hkv=8, D=128, page=16, longest=4001,
             lens="equal", weights=False),
        # a served batch of sequences of different lengths
        dict(name="paged batch", op="paged", io="bf16", B=64, Hq=32, Hkv=8, D=128, page=64, longest=8192,
             lens="ragged", weights=False),
        # the same with the accumulated weights that eviction goes by, small heads
        dict(name="paged weighted", op="paged", io="f16", B=16, Hq=32, Hkv=8, D=64, page=32, longest=12000,
             lens="ragged", weights=True),
        # a short cache cut to a budget
        dict(name="evict small", op="evict", io="bf16", B=1, Hkv=8, D=64, page=16, longest=1000, keep=500,
             recent=64, lens="equal"),
        # a served batch of long caches cut to half
        dict(name="evict batch", op="evict", io="bf16", B=16, Hkv=8, D=128, page=32, longest=16000, keep=6000,
             recent=512, lens="ragged"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def _draw_one(rng):
    op = rng.choice(("prompt", "prompt", "step", "paged", "paged", "evict"))
    io = rng.choice(("bf16", "bf16", "f16", "f16", "f32"))
    if op == "prompt":
        H = rng.randint(1, 32)
        Hk = rng.choice([d for d in range(1, H + 1) if H % d == 0])
        return dict(op=op, io=io, B=_log_int(rng, 1, 8), H=H, Hk=Hk,
                    L=_log_int(rng, 1, 2048 if io == "f32" else 16384), N=8 * rng.randint(2, 16),
                    P=8 * rng.randint(2, 16), decay=rng.choice(("head", "token")), ragged=rng.random() < 0.5)
    if op == "step":
        H = rng.randint(1, 32)
        Hk = rng.choice([d for d in range(1, H + 1) if H % d == 0])
        B = _log_int(rng, 1, 245)
        return dict(op=op, io=io, state=rng.choice(("f32", io)), B=B, H=H, Hk=Hk, N=8 * rng.randint(2, 32),
                    P=rng.randint(8, 200), slots=B + rng.randint(0, 20), decay=rng.choice(("head", "token")))
    if op == "paged":
        Hkv = rng.randint(1, 8)
        return dict(op=op, io=io, B=_log_int(rng, 1, 64), Hq=Hkv * rng.randint(1, 16), Hkv=Hkv,
                    D=rng.choice((64, 128, 64, 128, 96, 80)), page=rng.choice((16, 32, 64, 128, 24)),
                    longest=_log_int(rng, 1, 32768), lens=rng.choice(("equal", "ragged")),
                    weights=rng.random() < 0.4)
    longest = _log_int(rng, 16, 32768)
    keep = rng.randint(1, longest)
    return dict(op=op, io=io, B=_log_int(rng, 1, 32), Hkv=rng.randint(1, 8), D=rng.choice((64, 128, 96)),
                page=rng.choice((16, 32, 64, 24)), longest=longest, keep=keep, recent=rng.randint(0, keep),
                lens=rng.choice(("equal", "ragged")))


def draw(rng):
    # at least 2^17 bytes, and no more than the largest listed case of its operator
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), work(c)["bytes"])
    while True:
        c = _draw_one(rng)
        w = work(c)
        if (1 << 17) <= w["bytes"] <= most[c["op"]] and (c["io"] != "f32" or w["flops"] < 3e10):
            return c


# ----------------------------------------------------------------- inputs --
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _normal(g, shape, dt, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(_DT[dt])


def _lengths(case):
    """The lengths of the sequences: part of the case, so that the work is the same for every seed."""
    B, top = case["B"], case["longest"] if "longest" in case else case["L"]
    if case.get("lens") == "ragged" or case.get("ragged"):
        # the longest one, then lengths spread over (0, top] in a fixed irregular order
        return [top] + [max(1, (top * (((i * 37) % 101) + 1)) // 102) for i in range(1, B)]
    return [top] * B


def _log_decay(g, case, shape_tokens):
    """Decay per head: memories of 2 to 256 tokens over the heads.  Per token: a gate's logarithm, mostly close to 0."""
    H = case["H"]
    slope = torch.exp2(-1.0 - 7.0 * torch.arange(H, device="cuda") / max(H - 1, 1))
    if case["decay"] == "head":
        return -slope * (0.9 + 0.2 * torch.rand(H, generator=g, device="cuda"))
    gate = torch.nn.functional.softplus(torch.randn(shape_tokens, generator=g, device="cuda") - 1.0)
    return -gate * slope.view((1, H) + (1,) * (len(shape_tokens) - 2))


def _table(g, B, pages_each, pool):
    """Distinct pages of the pool for every sequence, in random order."""
    return torch.randperm(pool, generator=g, device="cuda")[: B * pages_each].view(B, pages_each).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "prompt":
        B, H, Hk, L, N, P = (case[x] for x in ("B", "H", "Hk", "L", "N", "P"))
        # as a token-major projection writes them: (B, L, heads, size), seen as (B, heads, L, size)
        q = _normal(g, (B, L, Hk, N), case["io"]).transpose(1, 2)
        k = _normal(g, (B, L, Hk, N), case["io"], std=N ** -0.5).transpose(1, 2)
        v = _normal(g, (B, L, H, P), case["io"]).transpose(1, 2)
        lens = torch.tensor(_lengths(case), device="cuda", dtype=torch.int32) if case["ragged"] else None
        return dict(case=case, q=q, k=k, v=v, scale=1.0, log_decay=_log_decay(g, case, (B, H, L)),
                    state=torch.randn((B, H, P, N), generator=g, device="cuda"), lens=lens,
                    state_out=torch.zeros((B, H, P, N), device="cuda"),
                    out=torch.zeros((B, L, H, P), device="cuda", dtype=_DT[case["io"]]).transpose(1, 2))
    if op == "step":
        B, H, Hk, N, P = (case[x] for x in ("B", "H", "Hk", "N", "P"))
        state = _normal(g, (case["slots"], H, P, N), case["state"])
        slots = torch.randperm(case["slots"], generator=g, device="cuda")[:B].to(torch.int32)
        return dict(case=case, q=_normal(g, (B, Hk, N), case["io"]), k=_normal(g, (B, Hk, N), case["io"], std=N ** -0.5),
                    v=_normal(g, (B, H, P), case["io"]), scale=1.0, log_decay=_log_decay(g, case, (B, H)),
                    state=state, state_out=torch.zeros_like(state), slots=slots)
    B, Hkv, D, page = (case[x] for x in ("B", "Hkv", "D", "page"))
    lens = torch.tensor(_lengths(case), device="cuda", dtype=torch.int32)
    each = -(-case["longest"] // page)
    if op == "paged":
        Hq = case["Hq"]
        pool = B * each + 3
        s = dict(case=case, q=_normal(g, (B, Hq, D), case["io"]), k=_normal(g, (pool, page, Hkv, D), case["io"]),
                 v=_normal(g, (pool, page, Hkv, D), case["io"]), table=_table(g, B, each, pool), lens=lens,
                 scale=D ** -0.5)
        if case["weights"]:
            s["weights"] = torch.rand((B, Hkv, each * page), generator=g, device="cuda")
            s["weights_out"] = torch.zeros_like(s["weights"])
        return s
    new_each = -(-case["keep"] // page)
    pool = B * (each + new_each) + 3
    every = _table(g, B, each + new_each, pool)
    # sums of softmax weights: many small ones, a few large ones, some never attended to (equal to one another)
    w = torch.rand((B, Hkv, each * page), generator=g, device="cuda").pow(6)
    w = torch.where(w < 0.001, torch.zeros_like(w), w)
    return dict(case=case, k=_normal(g, (pool, page, Hkv, D), case["io"]), v=_normal(g, (pool, page, Hkv, D), case["io"]),
                table=every[:, :each].contiguous(), new_table=every[:, each:].contiguous(), lens=lens, weights=w)


# ------------------------------------------------------------------- work --
def work(case):
    op, es = case["op"], _ES[case["io"]]
    if op == "prompt":
        H, Hk, N, P = (case[x] for x in ("H", "Hk", "N", "P"))
        tokens = sum(_lengths(case))
        decay = 4 * H * tokens if case["decay"] == "token" else 4 * H
        return {"bytes": tokens * es * (2 * Hk * N + 2 * H * P) + decay + 2 * 4 * case["B"] * H * P * N,
                "flops": 4 * tokens * H * N * P}
    if op == "step":
        B, H, Hk, N, P = (case[x] for x in ("B", "H", "Hk", "N", "P"))
        return {"bytes": B * (2 * _ES[case["state"]] * H * P * N + es * (2 * Hk * N + 2 * H * P) + 4 * H),
                "flops": 5 * B * H * P * N}
    B, Hkv, D = (case[x] for x in ("B", "Hkv", "D"))
    tokens = sum(_lengths(case))
    if op == "paged":
        Hq = case["Hq"]
        extra = 8 * tokens * Hkv if case["weights"] else 0
        return {"bytes": 2 * tokens * Hkv * D * es + 2 * B * Hq * D * es + extra + 4 * tokens // case["page"],
                "flops": 4 * tokens * Hq * D}
    kept = sum(min(n, case["keep"]) for n in _lengths(case))
    return {"bytes": 4 * tokens * Hkv + 4 * kept * Hkv * D * es + 8 * kept * Hkv, "flops": tokens * Hkv}


# ------------------------------------------------------------ plain forms --
def _prompt(s):
    """Chunks of _CHUNK tokens: inside a chunk the masked product of queries and keys, between chunks their states."""
    q, k, v = (s[x].float() for x in ("q", "k", "v"))
    B, H, L, P = v.shape
    N, C = q.shape[-1], _CHUNK
    nc = -(-L // C)
    pad = nc * C - L
    there = torch.arange(nc * C, device=q.device)[None, :] < (s["lens"][:, None] if s["lens"] is not None else L)  # (B|1, L')
    there = there[:, None, :].expand(B, H, nc * C)
    g = s["log_decay"].double()
    g = g.view(1, H, 1).expand(B, H, L) if g.dim() == 1 else g
    g = torch.where(there, torch.nn.functional.pad(g, (0, pad)), torch.zeros((), dtype=g.dtype, device=g.device))

    def cut(x):
        x = torch.nn.functional.pad(x.repeat_interleave(H // x.shape[1], dim=1), (0, 0, 0, pad))
        return torch.where(there[..., None], x, torch.zeros((), device=x.device)).view(B, H, nc, C, -1)

    q, k, v = cut(q), cut(k), cut(v)
    G = g.view(B, H, nc, C).cumsum(-1)                                        # log decay from the chunk's start
    low = torch.tril(torch.ones(C, C, dtype=torch.bool, device=q.device))
    D = torch.where(low, (G[..., :, None] - G[..., None, :]).float(), -torch.inf).exp()
    inside = ((q @ k.transpose(-1, -2)) * D) @ v
    ends = (v * (G[..., -1:] - G).float().exp()[..., None]).transpose(-1, -2) @ k  # (B, H, nc, P, N)
    # the state before chunk i: the initial state and the ends of chunks j < i, each decayed to chunk i's start
    T = torch.nn.functional.pad(G[..., -1].cumsum(-1), (1, 0))                # (B, H, nc + 1)
    before = torch.tril(torch.ones(nc + 1, nc, dtype=torch.bool, device=q.device), -1)
    M = torch.where(before, (T[..., :, None] - T[..., None, 1:]).float(), -torch.inf).exp()
    S = (M @ ends.flatten(-2)).view(B, H, nc + 1, P, N) + T.float().exp()[..., None, None] * s["state"][:, :, None]
    across = (q * G.float().exp()[..., None]) @ S[:, :, :nc].transpose(-1, -2)
    o = ((inside + across) * s["scale"]).view(B, H, nc * C, P)[:, :, :L].to(s["v"].dtype)
    s["out"].copy_(torch.where(there[:, :, :L, None], o, s["out"]))
    s["state_out"].copy_(S[:, :, nc])
    return s["out"], s["state_out"]


def _step(s):
    q, k, v = (s[x].float() for x in ("q", "k", "v"))
    H = v.shape[1]
    q, k = (x.repeat_interleave(H // x.shape[1], dim=1) for x in (q, k))
    at = s["slots"].long()
    S = s["state"][at].float() * s["log_decay"].float().exp().view(-1, H, 1, 1) + v[..., None] * k[:, :, None, :]
    s["state_out"][at] = S.to(s["state_out"].dtype)
    return ((S * q[:, :, None, :]).sum(-1) * s["scale"]).to(s["v"].dtype), s["state_out"]


def _paged(s):
    q, table = s["q"].float(), s["table"].long()
    B, Hq, D = q.shape
    page, Hkv = s["k"].shape[1:3]
    T = table.shape[1] * page
    k, v = (s[x][table].float().view(B, T, Hkv, D).transpose(1, 2) for x in ("k", "v"))
    there = (torch.arange(T, device=q.device)[None] < s["lens"][:, None])[:, None, None, :]
    x = (q.view(B, Hkv, Hq // Hkv, D) @ k.transpose(-1, -2)) * s["scale"]
    x = torch.where(there, x, -torch.inf)
    p = torch.where(there, (x - x.amax(-1, keepdim=True)).exp(), torch.zeros((), device=q.device))
    p = p / p.sum(-1, keepdim=True)
    out = (p @ v).view(B, Hq, D).to(s["q"].dtype)
    if "weights" not in s:
        return out
    s["weights_out"].copy_(torch.where(there[:, :, 0], s["weights"] + p.sum(2), s["weights_out"]))
    return out, s["weights_out"]


def _evict(s):
    c, w = s["case"], s["weights"]
    B, Hkv, T = w.shape
    page, keep = c["page"], c["keep"]
    t = torch.arange(T, device=w.device)
    n = s["lens"].long()[:, None, None]
    w1 = torch.where(t >= n, -torch.inf, torch.where(t >= n - c["recent"], torch.inf, w))
    first = torch.sort(w1, dim=-1, descending=True, stable=True).indices[..., :keep]
    j = torch.arange(keep, device=w.device)
    there = (j < n).expand(B, Hkv, keep)
    kept = torch.sort(torch.where(there, first, T), dim=-1).values
    src = torch.where(there, kept, 0)
    b, h, jj = torch.nonzero(there, as_tuple=True)
    at = src[b, h, jj]
    from_page, to_page = s["table"].long()[b, at // page], s["new_table"].long()[b, jj // page]
    s["k"][to_page, jj % page, h] = s["k"][from_page, at % page, h]
    s["v"][to_page, jj % page, h] = s["v"][from_page, at % page, h]
    new_w = torch.where(there, torch.gather(w, -1, src), torch.zeros((), device=w.device))
    return s["lens"].clamp(max=keep), torch.where(there, kept, -1).to(torch.int32), new_w, s["k"], s["v"]


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"prompt": _prompt, "step": _step, "paged": _paged, "evict": _evict}[op](s)
    import state_space_model_causal_b200 as lib
    if op == "prompt":
        lib.ssm_linear_attention_fwd(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"], state=s["state"],
                                     state_out=s["state_out"], seq_lens=s["lens"], out=s["out"])
        return s["out"], s["state_out"]
    if op == "step":
        out = lib.ssm_linear_attention_update(s["state"], s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"],
                                              state_batch_indices=s["slots"], state_out=s["state_out"])
        return out, s["state_out"]
    if op == "paged":
        if "weights" not in s:
            return lib.ssm_paged_attention_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], scale=s["scale"])
        out = lib.ssm_paged_attention_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], scale=s["scale"],
                                             weights=s["weights"], weights_out=s["weights_out"])
        return out, s["weights_out"]
    new_lens, kept, new_w = lib.ssm_kv_cache_evict(s["k"], s["v"], s["weights"], s["table"], s["lens"], s["new_table"],
                                                   s["case"]["keep"], recent=s["case"]["recent"])
    return new_lens, kept, new_w, s["k"], s["v"]


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "prompt":  # the recurrence, token by token
        rep = case["H"] // case["Hk"]
        q, k = (s[x].double().repeat_interleave(rep, dim=1) for x in ("q", "k"))
        v, S, lam = s["v"].double(), s["state"].double(), s["log_decay"].double().exp()
        out = s["out"].double()
        for t in range(case["L"]):
            lt = lam[None, :] if lam.dim() == 1 else lam[:, :, t]
            new = S * lt[..., None, None] + v[:, :, t, :, None] * k[:, :, t, None, :]
            o = torch.einsum("bhpn,bhn->bhp", new, q[:, :, t]) * s["scale"]
            if s["lens"] is None:
                S, out[:, :, t] = new, o
            else:
                live = (t < s["lens"])[:, None, None]
                S = torch.where(live[..., None], new, S)
                out[:, :, t] = torch.where(live, o, out[:, :, t])
        return out, S
    if op == "step":  # slot by slot
        out = torch.empty_like(s["v"], dtype=torch.float64)
        after = s["state_out"].double()
        rep = case["H"] // case["Hk"]
        for b, slot in enumerate(s["slots"].tolist()):
            lam = (s["log_decay"] if s["log_decay"].dim() == 1 else s["log_decay"][b]).double().exp()
            kb, qb = (s[x][b].double().repeat_interleave(rep, dim=0) for x in ("k", "q"))
            after[slot] = s["state"][slot].double() * lam[:, None, None] + torch.einsum("hp,hn->hpn", s["v"][b].double(), kb)
            out[b] = torch.einsum("hpn,hn->hp", after[slot], qb) * s["scale"]
        return out, after
    page = case["page"]
    if op == "paged":  # sequence by sequence
        out = torch.empty_like(s["q"], dtype=torch.float64)
        w = s["weights_out"].double() if case["weights"] else None
        rep = case["Hq"] // case["Hkv"]
        for b, n in enumerate(_lengths(case)):
            pages = s["table"][b, : -(-n // page)].long()
            k, v = (s[x][pages].double().flatten(0, 1)[:n].repeat_interleave(rep, dim=1) for x in ("k", "v"))
            p = torch.softmax(torch.einsum("hd,thd->ht", s["q"][b].double(), k) * s["scale"], dim=-1)
            out[b] = torch.einsum("ht,thd->hd", p, v)
            if w is not None:
                w[b, :, :n] = s["weights"][b, :, :n].double() + p.view(case["Hkv"], rep, n).sum(1)
        return out if w is None else (out, w)
    # eviction, head by head on the host
    B, Hkv, keep = case["B"], case["Hkv"], case["keep"]
    K, V = s["k"].double(), s["v"].double()
    w = s["weights"].double().cpu()
    kept = torch.full((B, Hkv, keep), -1, dtype=torch.int32)
    new_w = torch.zeros((B, Hkv, keep), dtype=torch.float64)
    lens = _lengths(case)
    for b, n in enumerate(lens):
        forced = max(0, n - case["recent"])
        m = min(keep, n)
        for h in range(Hkv):
            free = w[b, h, :forced]
            order = torch.argsort(-free, stable=True)[: m - (n - forced)]
            idx = torch.cat([order.sort().values, torch.arange(forced, n)])
            kept[b, h, :m], new_w[b, h, :m] = idx.to(torch.int32), w[b, h, idx]
            at, to = idx.cuda(), torch.arange(m, device="cuda")
            src, dst = s["table"][b].long()[at // page], s["new_table"][b].long()[to // page]
            K[dst, to % page, h] = s["k"][src, at % page, h].double()
            V[dst, to % page, h] = s["v"][src, at % page, h].double()
    return torch.tensor(lens, dtype=torch.int32).clamp(max=keep), kept, new_w, K, V
