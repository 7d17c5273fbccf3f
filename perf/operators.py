"""The cached-attention operators: what they compute, on which sizes, and what they cannot do without.

Two operators share one paged cache of keys and values, k_cache and v_cache [pages, kv_heads, page_size, head_dim]:

* rope: every head of the queries and keys is normalised and rotated, the queries are returned, the keys and values
  go to their places in the cache.
* attn: queries of ragged sequences attend to their sequence's cached keys: the first `sinks` tokens and a sliding
  window, causal by chunks of tokens that see one another (chunk = 1: plain causal).

A case holds "op" and plain sizes; lengths that differ between sequences are drawn from its "shape" number.
"""
import math
import random

import torch

own = False

EPS = 1e-6
THETA = 10000.0


def listed():
    return [
        # one generated token for each of 8 sequences
        dict(name="rope_step", op="rope", N=8, H=32, Hkv=8, hd=128, page=64, neox=True, pad=0, shape=1),
        # the image tokens of one diffusion step, as many key heads as query heads
        dict(name="rope_image", op="rope", N=4216, H=32, Hkv=32, hd=128, page=128, neox=False, pad=0, shape=2),
        # an odd number of tokens with padding among them, short heads, small pages
        dict(name="rope_ragged", op="rope", N=5003, H=20, Hkv=4, hd=64, page=16, neox=True, pad=301, shape=3),
        # a long prompt
        dict(name="rope_long", op="rope", N=65536, H=32, Hkv=8, hd=128, page=64, neox=True, pad=0, shape=4),
        # one sequence's next token in a rolling window: latency
        dict(name="attn_step_one", op="attn", S=1, q_min=1, q_max=1, kv_min=4216, kv_max=4216, H=32, Hkv=8, hd=128,
             page=64, window=1024, sinks=4, chunk=1, pad=0, shape=11),
        # the next token of 64 sequences of unlike length, all their keys visible: the cache's bandwidth
        dict(name="attn_step_batch", op="attn", S=64, q_min=1, q_max=1, kv_min=100, kv_max=32768, H=32, Hkv=8, hd=128,
             page=64, window=32768, sinks=0, chunk=1, pad=0, shape=12),
        # one to three drafted tokens for each of 96 sequences, short heads, an odd group, small pages
        dict(name="attn_draft", op="attn", S=96, q_min=1, q_max=3, kv_min=3, kv_max=8192, H=40, Hkv=8, hd=64, page=16,
             window=2048, sinks=64, chunk=1, pad=0, shape=13),
        # a prompt of 4216 tokens
        dict(name="attn_prefill", op="attn", S=1, q_min=4216, q_max=4216, kv_min=4216, kv_max=4216, H=32, Hkv=8,
             hd=128, page=64, window=4216, sinks=0, chunk=1, pad=0, shape=14),
        # a long prompt in a sliding window with first tokens kept
        dict(name="attn_prefill_window", op="attn", S=1, q_min=8192, q_max=8192, kv_min=8192, kv_max=8192, H=32,
             Hkv=8, hd=128, page=128, window=1024, sinks=16, chunk=1, pad=0, shape=15),
        # the next chunk of three generated videos: tokens of one chunk see one another, the prompt and two chunks before
        dict(name="attn_chunk", op="attn", S=3, q_min=1054, q_max=1054, kv_min=2108, kv_max=5270, H=32, Hkv=32,
             hd=128, page=128, window=2109, sinks=256, chunk=1054, pad=0, shape=16),
        # prompts and single tokens mixed, some sequences empty, rows behind the last one, short heads
        dict(name="attn_mixed", op="attn", S=24, q_min=0, q_max=700, kv_min=0, kv_max=6000, H=24, Hkv=8, hd=64,
             page=16, window=4096, sinks=4, chunk=1, pad=37, shape=17),
        # a few new tokens over long caches: the keys have to be split
        dict(name="attn_long", op="attn", S=2, q_min=48, q_max=48, kv_min=30011, kv_max=32768, H=32, Hkv=8, hd=128,
             page=64, window=32768, sinks=0, chunk=1, pad=0, shape=18),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    Hkv = rng.choice([1, 2, 3, 4, 8])
    hd = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    if rng.random() < 1 / 3:
        N = _log(rng, 1, 40000)
        return dict(op="rope", N=N, H=Hkv * rng.choice([1, 2, 3, 4, 5, 8]), Hkv=Hkv, hd=hd, page=page,
                    neox=rng.random() < 0.5, pad=rng.randint(0, N // 8), shape=rng.randrange(1 << 30))
    g = rng.choice([1, 2, 3, 4, 5, 8, 16])
    kind = rng.choice(["step", "draft", "prefill", "chunk", "mixed", "few"])
    window, sinks, chunk, pad = _log(rng, 64, 8192), rng.choice([0, 0, 4, rng.randint(1, 300)]), 1, 0
    if kind == "step":
        S, q0, q1, k1 = _log(rng, 1, 64), 1, 1, _log(rng, 64, 16384)
        k0 = rng.randint(1, k1)
    elif kind == "draft":
        S, q0, q1, k1 = _log(rng, 1, 64), 1, rng.randint(2, 6), _log(rng, 64, 8192)
        k0 = rng.randint(6, k1)
    elif kind == "prefill":
        S, q1 = 1, _log(rng, 33, 4216)
        q0, k0 = q1, q1 + rng.choice([0, rng.randint(0, 1000)])
        k1 = k0
    elif kind == "chunk":
        S, chunk = rng.randint(1, 3), rng.randint(100, 1054)
        q0 = q1 = chunk
        k0, k1 = chunk, 4 * chunk
        window = 1 + chunk * rng.randint(0, 3)
    elif kind == "mixed":
        S, q0, q1, k0, pad = rng.randint(2, 16), 0, _log(rng, 20, 500), 0, rng.randint(0, 50)
        k1 = q1 + _log(rng, 64, 4000)
    else:
        S, q0, q1, k1 = rng.randint(1, 4), rng.randint(2, 16), rng.randint(17, 64), _log(rng, 500, 24000)
        k0 = rng.randint(100, k1)
    return dict(op="attn", S=S, q_min=q0, q_max=q1, kv_min=k0, kv_max=k1, H=Hkv * g, Hkv=Hkv, hd=hd, page=page,
                window=window, sinks=sinks, chunk=chunk, pad=pad, shape=rng.randrange(1 << 30))


# ------------------------------------------------------------------ sizes

def _lengths(c):
    """(query lengths, key lengths) of the sequences; every query token has its own key in the cache."""
    rng = random.Random(c["shape"])
    q, kv = [], []
    for s in range(c["S"]):
        n = rng.randint(c["q_min"], c["q_max"])
        if c["chunk"] > 1:  # a whole number of chunks in the cache, the new one last
            L = c["chunk"] * rng.randint(c["kv_min"] // c["chunk"], c["kv_max"] // c["chunk"])
        else:
            L = rng.randint(c["kv_min"], c["kv_max"])
        if s == 0 and c["S"] > 1:
            n, L = c["q_max"], c["kv_max"] // c["chunk"] * c["chunk"]
        if c["q_min"] == 0 and s % 4 == 1:
            n = rng.choice([0, 1, 1])
        q.append(n)
        kv.append(max(L, n))
    return q, kv


def _seen(c, n, L):
    """([first, end) of the window over all query tokens, visible (query, key) pairs) of one sequence."""
    ch, W, sinks = c["chunk"], c["window"], c["sinks"]
    lo_all, pairs = L, 0
    for p in range(L - n, L):
        first = p // ch * ch
        end = min(first + ch, L)
        lo = min(end, max(0, first + 1 - W))
        lo_all = min(lo_all, lo)
        pairs += end - lo + min(lo, sinks)
    return lo_all, pairs


def work(case):
    c = case
    if c["op"] == "rope":
        heads, live = c["H"] + 2 * c["Hkv"], c["N"] - c["pad"]
        moved = (c["N"] * c["H"] + live * 2 * c["Hkv"]) * c["hd"] * 2 * 2
        return {"bytes": moved + c["N"] * (c["hd"] * 4 + 8) + c["hd"] * 4,
                "flops": c["N"] * heads * c["hd"] * 8}
    q, kv = _lengths(c)
    rows, keys, pairs = sum(q), 0, 0
    for n, L in zip(q, kv):
        if n:
            lo, p = _seen(c, n, L)
            keys += L - lo + min(lo, c["sinks"])
            pairs += p
    return {"bytes": rows * c["H"] * (c["hd"] * 4 + 4) + keys * c["Hkv"] * c["hd"] * 4,
            "flops": pairs * c["H"] * c["hd"] * 4}


# ----------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, g, std=1.0, mean=0.0):
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)
    return x.add_(mean) if mean else x


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _rope_table(P, hd):
    inv = THETA ** (-torch.arange(hd // 2, dtype=torch.float64, device="cuda") * 2 / hd)
    a = torch.arange(P, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def prepare(case, seed):
    c, g = case, _gen(seed)
    rng = random.Random(seed * 1000003 + c["shape"])
    H, Hkv, hd, page = c["H"], c["Hkv"], c["hd"], c["page"]
    if c["op"] == "rope":
        N, live = c["N"], c["N"] - c["pad"]
        pages = -(-live // page) + 3
        # a packed projection: queries, keys and values are its column slices; one channel in a hundred is large
        qkv = _normal((N, (H + 2 * Hkv) * hd), g)
        big = torch.rand(qkv.shape[1], device="cuda", generator=g) < 0.01
        qkv[:, big] *= 20
        order = torch.randperm(pages * page, generator=g, device="cuda")[:live]
        keep = torch.randperm(N, generator=g, device="cuda")[:live].sort().values
        slots = torch.full((N,), -1, dtype=torch.int32, device="cuda")
        if N >= 64:  # tokens of a prompt fill pages in order, the pages lie anywhere
            where = torch.randperm(pages, generator=g, device="cuda")
            t = torch.arange(live, device="cuda")
            order = where[t // page] * page + t % page
        slots[keep] = order.int()
        P = max(8192, N)
        pos = torch.arange(N, device="cuda") if N >= 64 else torch.randint(P, (N,), generator=g, device="cuda")
        return dict(c=c, q=qkv[:, :H * hd], k=qkv[:, H * hd:(H + Hkv) * hd], v=qkv[:, (H + Hkv) * hd:],
                    wq=_normal((hd,), g, 0.05, 1.0), wk=_normal((hd,), g, 0.05, 1.0), rope=_rope_table(P, hd),
                    positions=pos.int(), slots=slots, keep=keep,
                    k_cache=_normal((pages, Hkv, page, hd), g), v_cache=_normal((pages, Hkv, page, hd), g))
    q, kv = _lengths(c)
    rows = sum(q) + c["pad"]
    M = max(1, -(-max(kv) // page))
    table, used = [], 0
    for n, L in zip(q, kv):  # pages behind the window and the sinks are given back: -1
        lo = _seen(c, n, L)[0] if n else 0
        row = []
        for i in range(M):
            live = i * page < L and (i * page < c["sinks"] or (i + 1) * page > lo)
            row.append(used if live else -1)
            used += live
        table.append(row)
    pages = used + 2
    where = list(range(pages))
    rng.shuffle(where)
    table = [[where[i] if i >= 0 else -1 for i in row] for row in table]
    starts = [0]
    for n in q:
        starts.append(starts[-1] + n)
    return dict(c=c, rows=sum(q), qmax=max(1, max(q)), q=_normal((rows, H, hd), g),
                k_cache=_normal((pages, Hkv, page, hd), g), v_cache=_normal((pages, Hkv, page, hd), g),
                table=_ints(table), q_start=_ints(starts), kv_len=_ints(kv),
                out=torch.zeros((rows, H, hd), dtype=torch.bfloat16, device="cuda"),
                lse=torch.zeros((rows, H), dtype=torch.float32, device="cuda"))


# -------------------------------------------------------------------- run

def run(state):
    s = state
    c = s["c"]
    if own:
        from dit_adaln_norm_gb300 import ops
        if c["op"] == "rope":
            q = ops.qk_norm_rope_cache(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["rope"], s["positions"], s["slots"],
                                       s["k_cache"], s["v_cache"], EPS, neox=c["neox"])
            return q, s["k_cache"], s["v_cache"]
        return ops.window_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["q_start"], s["kv_len"],
                                    c["window"], sinks=c["sinks"], chunk=c["chunk"], max_q=s["qmax"], out=s["out"],
                                    lse=s["lse"])
    if c["op"] == "rope":
        return _plain_rope(s, c)
    return _plain_attention(s, c)


def _plain_rope(s, c):
    hd, page, half = c["hd"], c["page"], c["hd"] // 2
    row = s["rope"][s["positions"].long()]
    cos, sin = row[:, None, :half], row[:, None, half:]

    def turn(x, w):
        x = x.float().view(c["N"], -1, hd)
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        if c["neox"]:
            a, b = x[..., :half], x[..., half:]
            return torch.cat([a * cos - b * sin, a * sin + b * cos], -1).bfloat16()
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2).bfloat16()

    q, k = turn(s["q"], s["wq"]), turn(s["k"], s["wk"])
    at = s["slots"][s["keep"]].long()
    s["k_cache"][at // page, :, at % page] = k[s["keep"]]
    s["v_cache"][at // page, :, at % page] = s["v"].reshape(c["N"], -1, hd)[s["keep"]]
    return q, s["k_cache"], s["v_cache"]


def _plain_attention(s, c):
    S, H, Hkv, hd, T, nq = c["S"], c["H"], c["Hkv"], c["hd"], s["rows"], s["qmax"]
    g, dev = H // Hkv, s["q"].device
    starts, L = s["q_start"].long(), s["kv_len"].long()
    n = starts[1:] - starts[:-1]
    t = torch.arange(T, device=dev)
    seq = torch.searchsorted(starts[1:], t, right=True)
    i = t - starts[seq]
    q = torch.zeros((S, nq, H, hd), device=dev)
    q[seq, i] = s["q"][:T].float()
    q = q.view(S, nq, Hkv, g, hd).permute(0, 2, 3, 1, 4).reshape(S, Hkv, g * nq, hd)
    pages = s["table"].clamp(min=0).long()
    k = s["k_cache"][pages].transpose(1, 2).reshape(S, Hkv, -1, hd).float()
    p = (L - n)[:, None] + torch.arange(nq, device=dev)  # [S, nq] positions of the query tokens
    first = p // c["chunk"] * c["chunk"]
    j = torch.arange(k.shape[2], device=dev)
    end = torch.minimum(first + c["chunk"], L[:, None])
    see = (j < end[..., None]) & ((j < c["sinks"]) | (j > (first - c["window"])[..., None]))  # [S, nq, keys]
    x = (q @ k.transpose(-1, -2)).mul_(hd ** -0.5).view(S, Hkv, g, nq, -1)
    x.masked_fill_(~see[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    v = s["v_cache"][pages].transpose(1, 2).reshape(S, Hkv, -1, hd).float()
    o = (x.view(S, Hkv, g * nq, -1) @ v).view(S, Hkv, g, nq, hd) / total
    lse = (top + total.log())[..., 0]
    s["out"][:T] = o.permute(0, 3, 1, 2, 4).reshape(S, nq, H, hd)[seq, i].bfloat16()
    s["lse"][:T] = lse.permute(0, 3, 1, 2).reshape(S, nq, H)[seq, i]
    return s["out"], s["lse"]


# ------------------------------------------------------------------ exact

def exact(case, seed):
    s, c = prepare(case, seed), case
    hd, page = c["hd"], c["page"]
    if c["op"] == "rope":
        ang = s["rope"].double()[s["positions"].long()]
        kc, vc = s["k_cache"].double(), s["v_cache"].double()

        def heads(x, w):
            out = []
            for h in range(x.shape[1] // hd):
                y = x[:, h * hd:(h + 1) * hd].double()
                y = y / torch.sqrt((y * y).sum(1, keepdim=True) / hd + EPS) * w.double()
                z = torch.empty_like(y)
                for m in range(hd // 2):
                    a, b = (m, m + hd // 2) if c["neox"] else (2 * m, 2 * m + 1)
                    co, si = ang[:, m], ang[:, hd // 2 + m]
                    z[:, a] = co * y[:, a] - si * y[:, b]
                    z[:, b] = si * y[:, a] + co * y[:, b]
                out.append(z)
            return torch.stack(out, 1)

        q, k = heads(s["q"], s["wq"]), heads(s["k"], s["wk"])
        at = s["slots"].long()
        live = at >= 0
        v = s["v"].double().reshape(c["N"], c["Hkv"], hd)
        kc[at[live] // page, :, at[live] % page] = k[live]
        vc[at[live] // page, :, at[live] % page] = v[live]
        return q, kc, vc
    H, Hkv = c["H"], c["Hkv"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    lens, t0 = _lengths(c), 0
    if work(c)["flops"] > 4e11:
        return None
    for b, (n, L) in enumerate(zip(*lens)):
        if n == 0:
            continue
        row = s["table"][b, :-(-L // page)].long().clamp(min=0)
        K = s["k_cache"][row].double().permute(1, 0, 2, 3).reshape(Hkv, -1, hd)[:, :L]
        V = s["v_cache"][row].double().permute(1, 0, 2, 3).reshape(Hkv, -1, hd)[:, :L]
        j = torch.arange(L, device="cuda")
        for i0 in range(0, n, 256):
            i1 = min(n, i0 + 256)
            p = torch.arange(L - n + i0, L - n + i1, device="cuda")[:, None]
            start = p - p % c["chunk"]
            hidden = (j >= start + c["chunk"]) | ((j >= c["sinks"]) & (j < start + 1 - c["window"]))
            lo = 0 if c["sinks"] else max(0, int(start[0, 0]) + 1 - c["window"])
            hi = min(L, int(start[-1, 0]) + c["chunk"])
            for h in range(H):
                u = h // (H // Hkv)
                x = s["q"][t0 + i0:t0 + i1, h].double() @ K[u, lo:hi].T / math.sqrt(hd)
                x = x.masked_fill(hidden[:, lo:hi], -math.inf)
                z = torch.logsumexp(x, 1)
                out[t0 + i0:t0 + i1, h] = torch.exp(x - z[:, None]) @ V[u, lo:hi]
                lse[t0 + i0:t0 + i1, h] = z
        t0 += n
    return out, lse
