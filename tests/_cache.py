"""Problems and 64-bit references for the paged-cache operators' tests.

A problem's cache is poisoned: every key and value slot that no query of its
sequence sees is NaN, page-table entries that cover only such slots are -1 or
far out of range, and output rows outside the sequences hold a sentinel."""
import math
import random

import torch

BF16 = 2.0 ** -8   # half a step of bf16 relative to the value
SENTINEL = -77.0


def seen(p, L, window, sinks, chunk):
    """Keys that the query at position p sees, as a sorted list of ranges."""
    if p < 0:
        return []
    p0 = p - p % chunk
    hi = min(L, p0 + chunk)
    lo = max(0, p0 + 1 - window) if window else hi
    lo, s = min(lo, hi), min(sinks, hi)
    return [(0, hi)] if lo <= s else [r for r in ((0, s), (lo, hi)) if r[0] < r[1]]


class Problem:
    def __init__(self, q_lens, kv_lens, H=4, Hkv=2, hd=128, page=16, window=1 << 20, sinks=0,
                 chunk=1, seed=0, pad=0, spare=3, scale=None, dev="cuda", q_std=1.0, poison=True,
                 v_mean=0.0):
        g = torch.Generator(device=dev).manual_seed(seed)
        rng = random.Random(seed)
        self.q_lens, self.kv_lens = list(q_lens), list(kv_lens)
        self.H, self.Hkv, self.hd, self.page = H, Hkv, hd, page
        self.window, self.sinks, self.chunk = window, sinks, chunk
        self.scale = hd ** -0.5 if scale is None else scale
        S, rows = len(q_lens), sum(q_lens)
        self.rows, self.N = rows, rows + pad
        normal = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
        # packed projection: q is a strided view
        self.qkv = (normal(self.N, (H + 2 * Hkv) * hd) * q_std).bfloat16()
        self.q = self.qkv[:, :H * hd].unflatten(1, (H, hd)) if self.N else \
            torch.empty((0, H, hd), dtype=torch.bfloat16, device=dev)
        M = max(1, max((-(-L // page) for L in kv_lens), default=1))
        self.K = [normal(Hkv, L, hd).bfloat16() for L in kv_lens]
        self.V = [(normal(Hkv, L, hd) + v_mean).bfloat16() for L in kv_lens]
        vis = []
        for n, L in zip(q_lens, kv_lens):
            m = torch.zeros(L, dtype=torch.bool)
            for p in range(L - n, L):
                for a, b in seen(p, L, window, sinks, chunk):
                    m[a:b] = True
            vis.append(m)
        need = [(s, i) for s, m in enumerate(vis) for i in range(-(-len(m) // page))
                if m[i * page:(i + 1) * page].any()]
        pages = len(need) + spare
        ids = list(range(pages))
        rng.shuffle(ids)
        fill = float("nan") if poison else 0.0
        self.k_cache = torch.full((pages, Hkv, page, hd), fill, dtype=torch.bfloat16, device=dev)
        self.v_cache = torch.full_like(self.k_cache, fill)
        table = [[rng.choice([-1, -5, 1 << 30]) for _ in range(M + 2)] for _ in range(S)]
        for pid, (s, i) in zip(ids, need):
            table[s][i] = pid
            a, b = i * page, min((i + 1) * page, kv_lens[s])
            live = vis[s][a:b].to(dev)
            kk, vv = self.K[s][:, a:b].clone(), self.V[s][:, a:b].clone()
            if poison:
                kk[:, ~live] = float("nan")
                vv[:, ~live] = float("inf")
            self.k_cache[pid, :, :b - a] = kk
            self.v_cache[pid, :, :b - a] = vv
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
        self.table_full = i32(table).reshape(S, M + 2)
        self.table = self.table_full[:, :M]  # strided rows
        starts = [0]
        for n in q_lens:
            starts.append(starts[-1] + n)
        self.q_start, self.kv_len = i32(starts), i32(self.kv_lens)

    def call(self, ops, max_q=None, out=None, lse=None, q=None):
        dev = self.k_cache.device
        if out is None:
            out = torch.full((self.N, self.H, self.hd), SENTINEL, dtype=torch.bfloat16, device=dev)
        if lse is None:
            lse = torch.full((self.N, self.H), SENTINEL, device=dev)
        return ops.window_attention(self.q if q is None else q, self.k_cache, self.v_cache, self.table,
                                    self.q_start, self.kv_len, self.window, sinks=self.sinks,
                                    chunk=self.chunk, scale=self.scale, max_q=max_q, out=out, lse=lse)

    def reference(self):
        """(out, lse, out's tolerance, lse's tolerance) in 64 bits.

        Tolerances, from the arithmetic alone.  A score's sum of hd products in
        fp32 is off by at most 2^-20 of sum |q||k| (hd/16 partial sums, each
        within 2^-23 and truncated at worst); its probability by that times
        scale, by 2^-21 for the exponential and by 2^-8 for its rounding to
        bf16, which only the product with V sees; L fp32 additions of
        probabilities are off by L 2^-23 at worst, far less in practice; the
        output is rounded once more to bf16."""
        dev = self.k_cache.device
        out = torch.full((self.N, self.H, self.hd), SENTINEL, dtype=torch.float64, device=dev)
        lse = torch.full((self.N, self.H), SENTINEL, dtype=torch.float64, device=dev)
        otol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
        t0, g = 0, self.H // self.Hkv
        for s, (n, L) in enumerate(zip(self.q_lens, self.kv_lens)):
            if n == 0:
                continue
            mask = torch.zeros(n, L, dtype=torch.bool)
            for i in range(n):
                for a, b in seen(L - n + i, L, self.window, self.sinks, self.chunk):
                    mask[i, a:b] = True
            mask = mask.to(dev)
            K = self.K[s].double().repeat_interleave(g, 0)
            V = self.V[s].double().repeat_interleave(g, 0)
            q = self.q[t0:t0 + n].double().transpose(0, 1)
            x = (q @ K.transpose(1, 2) * self.scale).masked_fill(~mask, -math.inf)
            size = (q.abs() @ K.abs().transpose(1, 2) * self.scale).masked_fill(~mask, 0).amax(-1) \
                if L else torch.zeros(self.H, n, dtype=torch.float64, device=dev)
            empty = ~mask.any(-1)
            z = torch.logsumexp(x, -1) if L else torch.full_like(size, -math.inf)
            P = torch.exp(x - torch.where(z.isfinite(), z, torch.zeros_like(z))[..., None])
            o, mag = P @ V, P @ V.abs()
            rel = 2.0 ** -20 * (1 + size) + 2.0 ** -21 + (L + 64) * 2.0 ** -23
            tol = (BF16 * 1.01 + 2 * rel)[..., None] * mag + BF16 * o.abs() if L else torch.zeros_like(o)
            o[:, empty] = 0
            out[t0:t0 + n], lse[t0:t0 + n] = o.transpose(0, 1), z.transpose(0, 1)
            otol[t0:t0 + n] = tol.transpose(0, 1)
            ltol[t0:t0 + n] = (rel + 2.0 ** -22 * torch.where(z.isfinite(), z.abs(), 0)).transpose(0, 1)
            t0 += n
        return out, lse, otol, ltol

    def check(self, got, what=""):
        out, lse = got
        want, wlse, otol, ltol = self.reference()
        err = (out.double() - want).abs()
        bad = ~(err <= otol)
        assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outputs off, first at "
                               f"{bad.nonzero()[0].tolist()}: {out[tuple(bad.nonzero()[0])]} for "
                               f"{want[tuple(bad.nonzero()[0])]} +- {otol[tuple(bad.nonzero()[0])]}")
        lbad = ~(((lse.double() - wlse).abs() <= ltol) | (lse.double() == wlse))
        assert not lbad.any(), (f"{what}: {int(lbad.sum())} statistics off, first at "
                                f"{lbad.nonzero()[0].tolist()}: {lse[tuple(lbad.nonzero()[0])]} for "
                                f"{wlse[tuple(lbad.nonzero()[0])]}")
