"""GPU tests of the paged-cache operators: values against 64-bit references
with tolerances from the arithmetic (tests/_cache.py), the rotation bit for
bit against single fp32 steps, untouched rows and slots, index checks, batch
invariance, graphs, streams, and both operators together over several steps."""
import random

import numpy as np
import pytest
import torch

from dit_adaln_norm_gb300 import ops, synth
from _cache import SENTINEL, Problem

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _setup():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    ops.load()


@pytest.fixture(autouse=True)
def _no_status_left():
    ops.device_status()
    yield
    torch.cuda.synchronize()
    assert ops.device_status() == 0


# ------------------------------------------------------- rotation + cache

def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def rotate_steps(x, w, table, pos, eps, neox):
    """The documented fp32 steps on heads x [N, heads, hd] (float32 arrays)."""
    f = np.float32
    N, H, hd = x.shape
    part = np.zeros((N, H, hd // 8), f)
    for e in range(8):
        part = part + x[..., e::8] * x[..., e::8]
    while part.shape[-1] > 1:
        part = part[..., 0::2] + part[..., 1::2]
    r = f(1) / np.sqrt(part / f(hd) + f(eps))
    n = (x * r) * w
    c, s = table[pos][:, None, :hd // 2], table[pos][:, None, hd // 2:]
    out = np.empty_like(n)
    a, b = (n[..., :hd // 2], n[..., hd // 2:]) if neox else (n[..., 0::2], n[..., 1::2])
    ra, rb = a * c - b * s, a * s + b * c
    if neox:
        out[..., :hd // 2], out[..., hd // 2:] = ra, rb
    else:
        out[..., 0::2], out[..., 1::2] = ra, rb
    return synth.to_bf16_bits(out)


def rope_problem(N, H, Hkv, hd, page, seed, pad=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    qkv = (torch.randn(N, (H + 2 * Hkv) * hd + 8, generator=g, device="cuda") * std).bfloat16()
    w = (1 + 0.1 * torch.randn(2, hd, generator=g, device="cuda")).bfloat16()
    pages = -(-max(N, 1) // page) + 2
    slots = rng.permutation(pages * page)[:N].astype(np.int32)
    slots[rng.permutation(N)[:pad]] = -1 - rng.integers(0, 5, pad)
    pos = rng.integers(0, 500, N).astype(np.int32)
    caches = [torch.full((pages, Hkv, page, hd), v, dtype=torch.bfloat16, device="cuda") for v in (3.5, -2.5)]
    table = synth.rope_table(500, hd)
    return dict(q=qkv[:, :H * hd], k=qkv[:, H * hd:(H + Hkv) * hd], v=qkv[:, (H + Hkv) * hd:-8], w=w,
                table=table, pos=pos, slots=slots, caches=caches)


def rope_call(p, neox, q_out=None):
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    return ops.qk_norm_rope_cache(p["q"], p["k"], p["v"], p["w"][0], p["w"][1], dev(p["table"]),
                                  dev(p["pos"]), dev(p["slots"]), *p["caches"], EPS, neox=neox, q_out=q_out)


def rope_check(p, got, neox, q_in=None, k_in=None, v_in=None):
    kc, vc = p["caches"]
    pages, Hkv, page, hd = kc.shape
    N = len(p["pos"])
    x = lambda t: t.float().cpu().numpy().reshape(N, -1, hd)  # noqa: E731
    wq, wk = (p["w"][i].float().cpu().numpy() for i in (0, 1))
    q_in = p["q"] if q_in is None else q_in
    with np.errstate(invalid="ignore", over="ignore"):
        wantq = rotate_steps(x(q_in), wq, p["table"], p["pos"], EPS, neox)
        wantk = rotate_steps(x(p["k"]), wk, p["table"], p["pos"], EPS, neox)
    nan = lambda b: (b & 0x7FFF) > 0x7F80  # noqa: E731
    gq = bits(got)
    assert ((gq == wantq) | (nan(gq) & nan(wantq))).all()
    ek = np.full((pages * page, Hkv, hd), bits(torch.tensor([3.5]).bfloat16())[0], np.uint16)
    ev = np.full((pages * page, Hkv, hd), bits(torch.tensor([-2.5]).bfloat16())[0], np.uint16)
    live = p["slots"] >= 0
    ek[p["slots"][live]] = wantk[live]
    ev[p["slots"][live]] = bits(p["v"]).reshape(N, Hkv, hd)[live]
    gk = bits(kc).reshape(pages, Hkv, page, hd).transpose(0, 2, 1, 3).reshape(pages * page, Hkv, hd)
    gv = bits(vc).reshape(pages, Hkv, page, hd).transpose(0, 2, 1, 3).reshape(pages * page, Hkv, hd)
    assert ((gk == ek) | (nan(gk) & nan(ek))).all()
    assert (gv == ev).all()


@pytest.mark.parametrize("hd,neox", [(128, False), (128, True), (64, False), (64, True)])
@pytest.mark.parametrize("N,H,Hkv,page", [(1, 1, 1, 16), (1, 32, 8, 64), (3, 6, 2, 32), (37, 20, 4, 16),
                                          (130, 5, 5, 128), (515, 32, 8, 64)])
def test_rope_cache(N, H, Hkv, page, hd, neox):
    p = rope_problem(N, H, Hkv, hd, page, 7 * N + H + hd, pad=N // 5)
    rope_check(p, rope_call(p, neox), neox)


@pytest.mark.parametrize("hd,neox", [(128, False), (128, True), (64, False), (64, True)])
@pytest.mark.parametrize("N,H,Hkv,page", [(5003, 1, 1, 16), (1751, 32, 8, 64), (2600, 9, 3, 128)])
def test_rope_cache_many_tokens(N, H, Hkv, page, hd, neox):
    """Enough units of work for the persistent form, several a warp."""
    p = rope_problem(N, H, Hkv, hd, page, N + H + hd, pad=N // 7)
    p["pos"][17] = 499
    rope_check(p, rope_call(p, neox), neox)


def ring_tokens(units, H, Hkv, hd):
    """Tokens that give each of the persistent form's warps (16 an SM) `units` units of work."""
    per_token = -(-(H + 2 * Hkv) // (2048 // hd))
    return -(-units * 16 * torch.cuda.get_device_properties(0).multi_processor_count // per_token)


@pytest.mark.parametrize("hd,neox", [(128, False), (128, True), (64, False), (64, True)])
@pytest.mark.parametrize("more", [-1, 0, 1])
def test_rope_cache_where_the_persistent_form_begins(hd, neox, more):
    N = ring_tokens(2, 1, 1, hd) + more
    p = rope_problem(N, 1, 1, hd, 16, N + hd, pad=N // 9)
    rope_check(p, rope_call(p, neox), neox)


@pytest.mark.parametrize("hd,neox", [(128, False), (128, True), (64, False), (64, True)])
@pytest.mark.parametrize("one,in_place", [(True, False), (True, True), (False, False), (False, True)])
def test_rope_cache_slots_are_refilled(hd, neox, one, in_place):
    """36 units a warp: its three slots are filled again and again, their barriers' phases
    come round, and the positions and slots of its units are looked up twice (32 at a time);
    with one unit a token, and with two (the second one of values too)."""
    H, Hkv = (1, 1) if one else (2048 // hd - 4, 4)
    N = ring_tokens(36, H, Hkv, hd) + 5
    p = rope_problem(N, H, Hkv, hd, 64, N + hd, pad=N // 7)
    q_in = p["q"].clone()
    got = rope_call(p, neox, q_out=p["q"] if in_place else None)
    rope_check(p, got, neox, q_in=q_in)


def test_rope_cache_many_tokens_in_place_and_bad_indices():
    p = rope_problem(6000, 4, 2, 128, 64, 40)
    q_in, out_of = p["q"].clone(), [5, 4999, 5999]
    p["pos"][out_of] = [-1, 500, 1 << 30]
    p["slots"][11] = p["caches"][0].shape[0] * 64
    got = rope_call(p, True, q_out=p["q"])
    torch.cuda.synchronize()
    assert ops.device_status() == 8
    assert torch.equal(p["q"][out_of].view(torch.int16), q_in[out_of].view(torch.int16))
    keep = np.ones(6000, bool)
    keep[out_of] = False
    pos = np.where(keep, p["pos"], 0).astype(np.int32)
    want = rotate_steps(q_in.float().cpu().numpy().reshape(6000, -1, 128), p["w"][0].float().cpu().numpy(),
                        p["table"], pos, EPS, True)
    assert (bits(got)[keep] == want[keep]).all()
    slots = p["slots"].copy()
    slots[out_of + [11]] = -1
    full = bits(got).copy()
    full[~keep] = want[~keep]
    rope_check(dict(p, pos=pos, slots=slots), torch.from_numpy(full.view(np.int16)).view(torch.bfloat16).cuda(),
               True, q_in=q_in)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("neox", [False, True])
def test_rope_cache_extreme_values(neox, many):
    p = rope_problem(5000 if many else 64, 4, 2, 128, 16, 5)
    p["q"][0], p["k"][0] = 0.0, 0.0
    p["q"][1], p["k"][1] = 1e-38, -1e-38
    p["q"][2], p["k"][2] = 3e38, 3e38            # squares overflow
    p["q"][3, 5], p["k"][3, 7], p["v"][3, 1] = float("inf"), float("nan"), float("nan")
    p["q"][4, ::2] = -0.0
    rope_check(p, rope_call(p, neox), neox)


@pytest.mark.parametrize("neox", [False, True])
def test_rope_cache_in_place_beside_k_and_v(neox):
    p = rope_problem(70, 6, 2, 128, 32, 6)
    q_in = p["q"].clone()
    got = rope_call(p, neox, q_out=p["q"])
    assert got.data_ptr() == p["q"].data_ptr()
    rope_check(p, got, neox, q_in=q_in)


@pytest.mark.parametrize("order", ["kvq", "kqv"])
@pytest.mark.parametrize("N", [70, 5000])
def test_rope_cache_in_place_behind_k_and_v(N, order):
    p = rope_problem(N, 6, 2, 128, 32, 6)
    parts = {n: p[n] for n in "qkv"}
    packed = torch.cat([parts[n] for n in order], 1)
    at = 0
    for n in order:
        p[n] = packed[:, at:at + parts[n].shape[1]]
        at += parts[n].shape[1]
    got = rope_call(p, True, q_out=p["q"])
    assert got.data_ptr() == p["q"].data_ptr()
    rope_check(p, got, True, q_in=parts["q"].clone())


def test_rope_cache_bad_indices_are_left_out():
    p = rope_problem(40, 4, 2, 64, 16, 8)
    total = p["caches"][0].shape[0] * 16
    p["pos"][3], p["pos"][4], p["slots"][5], p["slots"][6] = -1, 500, total, 0x7FFFFFFF
    out = torch.full((40, 4, 64), SENTINEL, dtype=torch.bfloat16, device="cuda")
    rope_call(p, True, q_out=out)
    torch.cuda.synchronize()
    assert ops.device_status() == 8
    assert (out[3:5] == SENTINEL).all()
    good = np.ones(40, bool)
    good[3:5] = False
    p["pos"][3:5] = 0
    x = p["q"].float().cpu().numpy().reshape(40, -1, 64)
    want = rotate_steps(x, p["w"][0].float().cpu().numpy(), p["table"], p["pos"], EPS, True)
    assert (bits(out)[good] == want[good]).all()
    slots = p["slots"].copy()
    slots[3:7] = -1  # none of the four stored anything
    p2 = dict(p, slots=slots)
    rope_check(p2, torch.from_numpy(want.view(np.int16)).view(torch.bfloat16).cuda(), True)


@pytest.mark.parametrize("number", [np.float32, np.float64, torch.tensor, float])
def test_numbers_of_any_kind(number):
    """eps and scale as the other entry points take theirs: what float() takes."""
    p = rope_problem(9, 2, 1, 64, 16, 10)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    args = (p["q"], p["k"], p["v"], p["w"][0], p["w"][1], dev(p["table"]), dev(p["pos"]), dev(p["slots"]))
    want = ops.qk_norm_rope_cache(*args, *p["caches"], 0.25)
    assert same(ops.qk_norm_rope_cache(*args, *p["caches"], number(0.25)), want)
    a = Problem([1, 20], [30, 40], 2, 1, 64, 16, seed=44, scale=0.25)
    want = [t.clone() for t in a.call(ops)]
    a.scale = number(0.25)
    assert all(torch.equal(x, y) for x, y in zip(a.call(ops), want))


def test_rope_cache_empty_call():
    p = rope_problem(0, 4, 2, 64, 16, 9)
    assert rope_call(p, True).shape == (0, 4, 64)


# -------------------------------------------------------------- attention

def run(p, what="", **kw):
    p.check(p.call(ops, **kw), what)


GROUPS = [(1, 1), (4, 2), (8, 1), (6, 2), (16, 1), (32, 1), (5, 5)]


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("H,Hkv", GROUPS)
def test_single_tokens(H, Hkv, hd):
    lens = [1, 2, 15, 16, 17, 63, 255, 256, 257, 300, 777, 1030]
    run(Problem([1] * len(lens), lens, H, Hkv, hd, page=16, seed=H + hd), max_q=1)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (17, 0), (100, 4), (256, 64), (0, 5), (0, 0), (5, 1000),
                                          (300, 130)])
def test_step_windows_and_sinks(window, sinks, page):
    lens = [1, 5, 6, 64, 129, 400, 1000]
    run(Problem([1] * len(lens), lens, 8, 2, 128, page, window, sinks, seed=window + page), max_q=1)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("H,Hkv", GROUPS)
def test_drafted_tokens(H, Hkv, hd):
    q = [1, 2, 3, 4, 0, 5, 1, 16]
    kv = [1, 2, 300, 64, 0, 5, 700, 1029]
    run(Problem(q, kv, H, Hkv, hd, 32, 200, 7, seed=H * hd, pad=3))


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("q,kv", [(17, 17), (40, 40), (128, 128), (129, 200), (255, 1000), (300, 300),
                                  (513, 513), (700, 1500)])
def test_prefill(q, kv, hd):
    run(Problem([q], [kv], 4, 2, hd, 16, seed=q + kv))


@pytest.mark.parametrize("window,sinks,chunk", [(1, 0, 1), (50, 0, 1), (128, 4, 1), (129, 130, 1), (0, 9, 1),
                                                (0, 0, 1), (1, 0, 100), (201, 37, 100), (64, 3, 7),
                                                (0, 5, 33), (1 << 30, 0, 1 << 30), (1000, 300, 256)])
@pytest.mark.parametrize("H,Hkv,hd,page", [(4, 4, 128, 64), (6, 2, 64, 16), (8, 1, 128, 128)])
def test_prefill_masks(window, sinks, chunk, H, Hkv, hd, page):
    run(Problem([400, 90, 300], [400, 1000, 333], H, Hkv, hd, page, window, sinks, chunk,
                seed=window + chunk + hd))


@pytest.mark.parametrize("H,Hkv", [(128, 1), (100, 1), (24, 1), (17, 1), (66, 2)])
@pytest.mark.parametrize("hd", [64, 128])
def test_wide_groups(H, Hkv, hd):
    """Groups of query heads that fill a row tile, or leave rows of it over."""
    run(Problem([1, 5, 33], [300, 5, 200], H, Hkv, hd, 32, 150, 3, seed=H + hd))


def test_most_heads():
    run(Problem([1, 3], [40, 60], 1024, 8, 64, 16, seed=30))
    run(Problem([1, 3], [40, 60], 1024, 1024, 64, 16, seed=31))


def test_mixed_batch_with_empty_sequences_and_rows_behind():
    run(Problem([0, 1, 300, 0, 2, 70, 1, 0], [0, 1, 500, 40, 900, 70, 1300, 0], 8, 2, 128, 32, 250, 5,
                seed=3, pad=9))


def test_queries_before_the_first_key_give_zeros():
    # kv_len < n: the first rows have negative positions
    run(Problem([5, 40, 3], [2, 30, 0], 4, 2, 64, 16, seed=4))


@pytest.mark.parametrize("max_q", [None, 300])
def test_max_q_bound_is_only_a_hint(max_q):
    run(Problem([1, 300, 7], [50, 300, 1000], 4, 2, 128, 16, seed=5), max_q=max_q)


@pytest.mark.parametrize("q", [1, 60])
def test_large_scores_and_values(q):
    run(Problem([q, q], [400, 257], 4, 2, 128, 16, seed=6, q_std=30.0, v_mean=1000.0))
    run(Problem([q, q], [400, 257], 4, 2, 128, 16, seed=7, q_std=1e-3, scale=3.0))


@pytest.mark.parametrize("q", [1, 40])
def test_huge_values(q):
    """Value rows near the type's largest: sums of probabilities stay small enough."""
    p = Problem([q], [600], 4, 2, 64, 16, seed=32, q_std=3.0, v_mean=1e30)
    run(p)


@pytest.mark.parametrize("first", [0.0, 2.0, 200.0])
@pytest.mark.parametrize("q", [1, 40])
def test_jump_after_the_first_block(q, first):
    """Scores of the first keys are `first` lower than the others': the reference
    they set has to rise, a little, by a power of two, or far at once."""
    p = Problem([q], [640], 2, 1, 64, 16, seed=33)
    u = torch.ones(64, device="cuda") / 8
    base = p.q.float() * 0.3
    p.q.copy_((base + u * 8).bfloat16())
    p.K[0] = (p.K[0].float() * 0.3).bfloat16()
    p.K[0][:, 200:] += (u * first).bfloat16()
    for b in range(40):
        pid = int(p.table[0, b])
        if 0 <= pid < p.k_cache.shape[0]:
            p.k_cache[pid] = p.K[0][:, 16 * b:16 * b + 16]
    run(p)


def jump(p, first, V=None):
    """Make the scores of keys 0..199 of the one sequence `first` lower than the others',
    and its values V, in the problem and in its cache."""
    u = torch.ones(p.hd, device="cuda") / 8
    p.q.copy_((p.q.float() * 0.3 + u * 8 * 64 / p.hd).bfloat16())
    p.K[0] = (p.K[0].float() * 0.3).bfloat16()
    p.K[0][:, 200:] += (u * first).bfloat16()
    if V is not None:
        p.V[0] = V.bfloat16()
    L = p.kv_lens[0]
    for b in range(-(-L // p.page)):
        pid, a, e = int(p.table[0, b]), p.page * b, min(L, p.page * b + p.page)
        if 0 <= pid < p.k_cache.shape[0]:
            p.k_cache[pid, :, :e - a] = p.K[0][:, a:e]
            p.v_cache[pid, :, :e - a] = p.V[0][:, a:e]


@pytest.mark.parametrize("first", [0.0, 4.0, 9.0, 11.0, 12.0, 13.0, 16.0, 200.0])
@pytest.mark.parametrize("q,kv,hd", [(1, 640, 64), (40, 640, 64), (40, 640, 128), (48, 9000, 128)])
def test_values_up_to_the_documented_largest(q, kv, hd, first):
    """All of one sign and within a factor of two below 2^99, under scores that rise after the
    first block by what moves its reference late (a block's sum just below 2^24), or far."""
    p = Problem([q], [kv], 4, 1, hd, 16, seed=34, poison=False)
    g = torch.Generator(device="cuda").manual_seed(35)
    V = (torch.rand(p.V[0].shape, generator=g, device="cuda") * 0.49 + 0.5) * 2.0 ** 99
    jump(p, first, V)
    assert p.V[0].isfinite().all() and p.V[0].max() <= 2.0 ** 99
    run(p)


@pytest.mark.parametrize("q", [1, 50])
def test_rising_scores_rescale(q):
    """Keys that grow along the sequence: the running maximum moves at every block."""
    p = Problem([q], [900], 4, 2, 64, 16, seed=8)
    ramp = torch.linspace(0.01, 4, 900, device="cuda")[None, :, None]
    p2 = Problem([q], [900], 4, 2, 64, 16, seed=8)
    for b in range(-(-900 // 16)):
        a, e = 16 * b, min(900, 16 * b + 16)
        pid = int(p2.table[0, b])
        if pid < 0 or pid >= p2.k_cache.shape[0]:
            continue
        p2.k_cache[pid, :, :e - a] = (p.K[0][:, a:e].float() * ramp[:, a:e]).bfloat16()
    p2.K[0] = (p.K[0].float() * ramp).bfloat16()
    run(p2)


@pytest.mark.parametrize("q", [1, 40])
def test_visible_nan_and_infinite_keys_reach_only_their_rows(q):
    p = Problem([q], [200], 2, 1, 64, 16, window=60, seed=9)
    base = [t.clone() for t in p.call(ops)]
    pid = int(p.table[0, 150 // 16])
    p.k_cache[pid, 0, 150 % 16, 3] = float("nan")
    got = p.call(ops)
    torch.cuda.synchronize()
    for i in range(q):
        pos = 200 - q + i
        hit = pos - 60 < 150 <= pos
        assert got[0][i].isnan().all() == hit and got[1][i].isnan().all() == hit
        if not hit:
            assert torch.equal(got[0][i], base[0][i]) and torch.equal(got[1][i], base[1][i])


@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
@pytest.mark.parametrize("q", [1, 40])
@pytest.mark.parametrize("at", [3, 150, 190])
def test_infinite_keys(q, at, value):
    """A key with an infinite element has a score of +infinity, and its row NaN, where the
    query's element is of its sign, and a score of -infinity, and no weight, where it is not."""
    p = Problem([q], [200], 2, 1, 64, 16, seed=9, poison=False)
    pid = int(p.table[0, at // 16])
    p.k_cache[pid, 0, at % 16, 3] = value
    p.K[0][0, at, 3] = value
    out, lse = p.call(ops)
    sign = p.q[..., 3].float() * (1.0 if value > 0 else -1.0)   # [rows, heads]
    sees = (torch.arange(200 - q, 200, device="cuda") >= at)[:, None]
    gone = sees & (sign > 0)
    assert (sign != 0).all() and (q == 1 or (gone.any() and (sees & ~gone).any()))
    assert out[gone].isnan().all() and lse[gone].isnan().all()
    want, wlse, otol, ltol = p.reference()   # NaN where the formula's is; weights of 0 elsewhere
    err, lerr = (out.double() - want).abs(), (lse.double() - wlse).abs()
    # a score's tolerance goes by its largest seen product, which is infinite here: the same
    # problem's without that key's element
    p.K[0][0, at, 3] = 0.0
    _, _, otol, ltol = p.reference()
    assert (err[~gone] <= otol[~gone]).all() and (lerr[~gone] <= ltol[~gone]).all()


def test_long_context_split():
    run(Problem([1, 1, 2], [20000, 9000, 12345], 4, 1, 128, 64, seed=10), max_q=2)
    run(Problem([48, 20], [9000, 5000], 4, 1, 128, 64, seed=11))


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("window,sinks,chunk", [(3000, 700, 1), (1, 6000, 1), (2500, 0, 900), (16, 1, 5000),
                                                (769, 0, 1), (1, 0, 800)])
def test_windows_in_long_tables(window, sinks, chunk, hd):
    """Few of a long table's keys are seen: the launch covers those."""
    run(Problem([1, 3, 2, 4], [20000, 15001, 2, 9999], 4, 1, hd, 16, window, sinks, chunk, seed=hd + window))


def test_lse_is_optional_and_out_is_made():
    p = Problem([3, 20], [50, 60], 4, 2, 64, 16, seed=12)
    out = ops.window_attention(p.q, p.k_cache, p.v_cache, p.table, p.q_start, p.kv_len, p.window)
    both = ops.window_attention(p.q, p.k_cache, p.v_cache, p.table, p.q_start, p.kv_len, p.window, lse=True)
    assert torch.equal(out, both[0])
    p.check(both)


def test_bad_indices_leave_their_sequence_out():
    p = Problem([1, 1, 1, 1], [40, 40, 40, 40], 4, 2, 64, 16, seed=13, poison=False)
    want = p.call(ops)[0].clone()
    p.table[1, 1] = p.k_cache.shape[0]       # one past the last page
    got = p.call(ops)[0]
    torch.cuda.synchronize()
    assert ops.device_status() == 8
    keep = [0, 2, 3]
    assert torch.equal(got[keep], want[keep]) and got[1].isfinite().all()
    p.table[1, 1] = -1
    p.call(ops)
    torch.cuda.synchronize()
    assert ops.device_status() == 8


@pytest.mark.parametrize("starts", [[0, 2, 1, 3, 4], [0, 1, 2, 3, 5], [-1, 1, 2, 3, 4], [0, 1, 2, 3, 1 << 30]])
def test_bad_query_starts_leave_their_sequence_out(starts):
    p = Problem([1] * 4, [40] * 4, 4, 2, 64, 16, seed=14)
    want = p.call(ops)[0].clone()
    p.q_start.copy_(torch.tensor(starts, dtype=torch.int32))
    out = p.call(ops)[0]
    torch.cuda.synchronize()
    assert ops.device_status() == 8
    if starts[:3] == [0, 1, 2]:
        assert torch.equal(out[:3], want[:3]) and (out[3] == SENTINEL).all()


def test_bad_lengths_and_max_q():
    p = Problem([1, 1, 20], [40, 40, 40], 4, 2, 64, 16, seed=15, poison=False)
    p.kv_len.copy_(torch.tensor([-5, 40, 1 << 30], dtype=torch.int32))
    out, lse = p.call(ops, max_q=19)
    torch.cuda.synchronize()
    assert ops.device_status() == 8
    assert (out[0] == 0).all() and (lse[0] == float("-inf")).all()   # no keys
    assert (out[2:] == SENTINEL).all()                               # more than max_q rows
    assert not (out[1] == SENTINEL).any()


def test_sequences_that_overlap_are_safe():
    """Query starts that go back and forth name more rows than there are: what
    does not fit the work lists is left out, and nothing else is touched."""
    p = Problem([300], [300], 8, 1, 64, 16, seed=21, poison=False)
    S = 4001
    starts = torch.tensor([0 if i % 2 == 0 else 300 for i in range(S + 1)], dtype=torch.int32, device="cuda")
    guard = torch.full((300 + 64, 8, 64), SENTINEL, dtype=torch.bfloat16, device="cuda")
    ops.window_attention(p.q, p.k_cache, p.v_cache, p.table.expand(S, -1).contiguous(), starts,
                         p.kv_len.expand(S).contiguous(), 1 << 20, scale=p.scale, out=guard[32:-32])
    torch.cuda.synchronize()
    assert ops.device_status() == 8
    assert (guard[:32] == SENTINEL).all() and (guard[-32:] == SENTINEL).all()


def guarded_call(p, table, starts, kv_len, max_q, window=1 << 20, sinks=0, chunk=1):
    """A call through the C entry with a workspace of exactly the bytes asked for, which, like
    out and lse, lies between guards that have to stay as they were."""
    lib, (S, M), H, hd = ops.load(), table.shape, p.H, p.hd
    need = lib.dan_window_attention_workspace(p.N, S, H, p.Hkv, hd, M, p.page, window, sinks, chunk, max_q)
    buf = torch.full((256 + need + 65536,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((p.N + 64, H, hd), SENTINEL, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((p.N + 64, H), SENTINEL, device="cuda")
    st = lib.dan_window_attention(
        p.q.data_ptr(), p.N, p.q.stride(0), p.k_cache.data_ptr(), p.v_cache.data_ptr(), p.k_cache.shape[0], p.page,
        table.data_ptr(), table.stride(0), M, starts.data_ptr(), kv_len.data_ptr(), S, H, p.Hkv, hd, window, sinks,
        chunk, max_q, p.scale, out[32:].data_ptr(), lse[32:].data_ptr(), buf.data_ptr() + 256, need,
        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0
    assert (buf[:256] == 0xA5).all() and (buf[256 + need:] == 0xA5).all()
    for t in (out, lse):
        assert (t[:32] == SENTINEL).all() and (t[-32:] == SENTINEL).all()
    return out[32:-32], lse[32:-32]


def test_sequences_that_share_rows_are_left_out():
    """The first sequence's rows are its own, whatever later ones name the same rows."""
    p = Problem([300], [300], 8, 1, 64, 16, seed=21, poison=False)
    S = 4001
    starts = torch.tensor([0 if i % 2 == 0 else 300 for i in range(S + 1)], dtype=torch.int32, device="cuda")
    kv_len = torch.full((S,), 150, dtype=torch.int32, device="cuda")
    kv_len[0] = 300
    got = guarded_call(p, p.table.expand(S, -1).contiguous(), starts, kv_len, 300)
    assert ops.device_status() == 8
    p.check(got)


@pytest.mark.parametrize("at", [3, 127, 128, 150])
def test_a_start_that_goes_back_far_behind(at):
    """Sequence `at` + 1 and the next lie on the rows of the first; the last has its own."""
    p = Problem([300, 30], [300, 77], 8, 1, 64, 16, seed=26, poison=False)
    S = 200
    starts = [0] + [300] * at + [100, 180] + [300] * (S - at - 3) + [330]
    kv_len = torch.full((S,), 150, dtype=torch.int32, device="cuda")
    kv_len[0], kv_len[-1] = 300, 77
    table = p.table[:1].expand(S, -1).contiguous()
    table[-1] = p.table[1]
    starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
    assert starts.shape == (S + 1,) and starts[at + 1] == 100
    got = guarded_call(p, table, starts, kv_len, 330)
    assert ops.device_status() == 8
    p.check(got)


@pytest.mark.parametrize("H,Hkv,hd", [(32, 8, 128), (16, 4, 64), (8, 1, 128)])
def test_split_sequences_of_both_kernels_in_a_large_batch(H, Hkv, hd):
    """256 sequences over one long cache, half of them a few rows and half a tile, all split:
    each row has the bits of a call of its sequence alone, and the workspace, which keeps the
    two kernels' partial results apart, is exactly what is asked for."""
    g, few = H // Hkv, 16 * Hkv // H
    q_lens = [few if s % 2 else 32 - few for s in range(256)]
    p = Problem([sum(q_lens)], [16384], H, Hkv, hd, 64, seed=25, poison=False)
    starts = torch.tensor([sum(q_lens[:s]) for s in range(257)], dtype=torch.int32, device="cuda")
    kv = [16384 - 61 * (s % 7) for s in range(256)]
    kv_len = torch.tensor(kv, dtype=torch.int32, device="cuda")
    out, lse = guarded_call(p, p.table.expand(256, -1).contiguous(), starts, kv_len, 32)
    assert (lse != SENTINEL).all()
    for s in [*range(0, 256, 37), 1, 254, 255]:
        a, b = int(starts[s]), int(starts[s + 1])
        o1, l1 = torch.empty_like(out[a:b]), torch.empty_like(lse[a:b])
        ops.window_attention(p.q[a:b], p.k_cache, p.v_cache, p.table, torch.tensor(
            [0, b - a], dtype=torch.int32, device="cuda"), kv_len[s:s + 1], 1 << 20, scale=p.scale, out=o1, lse=l1)
        assert same(o1, out[a:b]) and torch.equal(l1, lse[a:b]), s
    for s in (0, 1):  # and those of the formula
        one = Problem([q_lens[s]], [kv[s]], H, Hkv, hd, 64, seed=25, poison=False)
        a, b = int(starts[s]), int(starts[s + 1])
        one.q, one.K, one.V = p.q[a:b], [p.K[0][:, :kv[s]]], [p.V[0][:, :kv[s]]]
        one.check((out[a:b], lse[a:b]), str(s))


def test_more_shared_rows_than_32_bits_count():
    """2^19 sequences name the same 8192 rows of 128 heads, 4096 tiles each: 2^31 tiles in all."""
    p = Problem([8192], [16], 128, 1, 64, 16, seed=23, poison=False)
    S = 1 << 20
    starts = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    starts[1::2] = 8192
    kv_len = torch.full((S,), 5, dtype=torch.int32, device="cuda")
    kv_len[0] = 16
    out, lse = guarded_call(p, p.table.expand(S, -1).contiguous(), starts, kv_len, 8192)
    assert ops.device_status() == 8
    assert (out[:8176] == 0).all() and (lse[:8176] == float("-inf")).all()  # before the first key
    tail = Problem([16], [16], 128, 1, 64, 16, seed=23, poison=False)
    tail.q, tail.K, tail.V = p.q[8176:], p.K, p.V
    tail.check((out[8176:], lse[8176:]))


@pytest.mark.parametrize("behind", [False, True])
def test_a_sequence_after_a_bad_one_keeps_its_rows(behind):
    """A sequence that is left out (its start lies past its end, or its rows past N) takes no rows."""
    p = Problem([40, 0, 50, 30], [40, 10, 90, 30], 4, 2, 64, 16, seed=24, poison=False)
    want = [t.clone() for t in p.call(ops)]
    p.q_start.copy_(torch.tensor([0, 1 << 30 if behind else 40, 40, 90, 120], dtype=torch.int32))
    got = p.call(ops)
    torch.cuda.synchronize()
    assert ops.device_status() == (8 if behind else 0)
    assert same(got[0][40:], want[0][40:]) and torch.equal(got[1][40:], want[1][40:])


def test_two_streams_at_once():
    ps = [Problem([1, 300, 3], [700, 900, 64], 8, 2, 128, 32, 400, 4, seed=22 + i) for i in range(2)]
    want = [[t.clone() for t in p.call(ops)] for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    for _ in range(5):
        got = []
        for p, s in zip(ps, streams):
            with torch.cuda.stream(s):
                got.append(p.call(ops))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


@pytest.mark.parametrize("S", [127, 128, 129, 300])
def test_many_sequences(S):
    """More sequences than the plan's block looks at together, of every length."""
    rng = random.Random(S)
    q = [rng.choice([0, 1, 1, 3, 9, 20, 70]) for _ in range(S)]
    run(Problem(q, [n + rng.randint(0, 300) for n in q], 6, 2, 64, 16, 90, 3, seed=S))


@pytest.mark.parametrize("H,Hkv,hd", [(8, 2, 64), (24, 1, 128)])
def test_very_many_sequences(H, Hkv, hd):
    """Twelve turns of the plan's block, with sequences of no rows, a few, one tile and two."""
    rng = random.Random(50)
    q = [rng.choice([0, 1, 1, 2, 4, 5, 17, 40, 70]) for _ in range(1500)]
    run(Problem(q, [max(0, n + rng.randint(-3, 60)) for n in q], H, Hkv, hd, 16, 33, 2, seed=51, pad=7))


def test_most_heads_rotated():
    p = rope_problem(5, 1024, 1024, 64, 16, 41)
    rope_check(p, rope_call(p, True), True)


def test_sequences_share_pages():
    """A prefix's pages in two sequences' tables, as after a fork."""
    p = Problem([1, 40, 1], [200, 240, 200], 8, 2, 128, 32, seed=42)
    p.table[2, :7] = p.table[0, :7]
    p.K[2], p.V[2] = p.K[0], p.V[0]
    run(p)


@pytest.mark.parametrize("many", [False, True])
def test_decode_step_in_a_graph(many):
    """Both operators captured once and replayed as the sequences grow, lengths,
    positions, slots and inputs rewritten in place between replays."""
    H, Hkv, hd, page, S, M = 8, 2, 128, 16, 3, 12
    add = 25 if many else 1
    g = torch.Generator(device="cuda").manual_seed(43)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.randperm(S * M, generator=g, device="cuda").int().view(S, M)
    kc, vc = (torch.zeros((S * M, Hkv, page, hd), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rope = torch.from_numpy(synth.rope_table(256, hd)).cuda()
    w = torch.ones(hd, dtype=torch.bfloat16, device="cuda")
    qkv = torch.zeros(S * add, (H + 2 * Hkv) * hd, dtype=torch.bfloat16, device="cuda")
    pos, slots, lens = i32([0] * S * add), i32([-1] * S * add), i32([add] * S)
    starts = i32([add * s for s in range(S + 1)])

    def step(kc, vc):
        q = ops.qk_norm_rope_cache(qkv[:, :H * hd], qkv[:, H * hd:(H + Hkv) * hd], qkv[:, (H + Hkv) * hd:],
                                   w, w, rope, pos, slots, kc, vc, EPS)
        return ops.window_attention(q, kc, vc, table, starts, lens, 60, sinks=2, max_q=add)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(kc, vc)
    kc2, vc2 = kc.clone(), vc.clone()
    for t in range(6):
        qkv.copy_(torch.randn(qkv.shape, generator=g, device="cuda"))
        at = [(s, t * add + i) for s in range(S) for i in range(add)]
        pos.copy_(i32([p for _, p in at]))
        slots.copy_(i32([int(table[s, p // page]) * page + p % page for s, p in at]))
        lens.fill_((t + 1) * add)
        graph.replay()
        want = step(kc2, vc2)
        torch.cuda.synchronize()
        assert same(out, want) and same(kc, kc2) and same(vc, vc2), t


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("hd", [64, 128])
def test_batch_invariance(hd):
    """A sequence's bits are the same alone, in a batch, with another page size
    and with another bound."""
    q, kv = [1, 300, 3, 40, 1], [777, 900, 2000, 1500, 5000]
    kw = dict(H=8, Hkv=2, hd=hd, window=1100, sinks=20, seed=16)
    p = Problem(q, kv, page=16, **kw)
    out, lse = p.call(ops)
    p2 = Problem(q, kv, page=128, **kw)
    out2, lse2 = p2.call(ops, max_q=300)
    assert same(out, out2) and torch.equal(lse, lse2)
    t0 = 0
    for s, n in enumerate(q):
        o1 = torch.empty_like(out[t0:t0 + n])
        l1 = torch.empty_like(lse[t0:t0 + n])
        ops.window_attention(p.q[t0:t0 + n], p.k_cache, p.v_cache, p.table[s:s + 1],
                             torch.tensor([0, n], dtype=torch.int32, device="cuda"), p.kv_len[s:s + 1],
                             1100, sinks=20, scale=p.scale, max_q=n, out=o1, lse=l1)
        assert same(o1, out[t0:t0 + n]) and torch.equal(l1, lse[t0:t0 + n]), s
        t0 += n


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(4, 4), (16, 2), (6, 1)])
@pytest.mark.parametrize("window,sinks,chunk", [(0, 1500, 1), (200, 4, 1), (700, 100, 33), (1600, 40, 128),
                                                (1 << 20, 0, 1)])
def test_workspace_is_as_large_as_is_used(hd, H, Hkv, window, sinks, chunk):
    """With exactly the bytes asked for, between guards that stay as they were."""
    p = Problem([1, 2, 130, 300, 1], [2600, 2000, 2500, 2111, 40], H, Hkv, hd, 32, window, sinks, chunk,
                seed=window + hd + H)
    want = p.call(ops)
    lib, (S, M) = ops.load(), p.table.shape
    need = lib.dan_window_attention_workspace(p.N, S, H, Hkv, hd, M, 32, window, sinks, chunk, 300)
    buf = torch.full((256 + need + 65536,), 0xA5, dtype=torch.uint8, device="cuda")
    out, lse = torch.full_like(want[0], SENTINEL), torch.full((p.N, H), SENTINEL, device="cuda")
    st = lib.dan_window_attention(
        p.q.data_ptr(), p.N, p.q.stride(0), p.k_cache.data_ptr(), p.v_cache.data_ptr(), p.k_cache.shape[0], 32,
        p.table.data_ptr(), p.table.stride(0), M, p.q_start.data_ptr(), p.kv_len.data_ptr(), S, H, Hkv, hd,
        window, sinks, chunk, 300, p.scale, out.data_ptr(), lse.data_ptr(), buf.data_ptr() + 256, need,
        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and same(out, want[0]) and torch.equal(lse, want[1])
    assert (buf[:256] == 0xA5).all() and (buf[256 + need:] == 0xA5).all()


@pytest.mark.parametrize("q,kv", [([1] * 5, [700, 1, 64, 5000, 333]), ([1, 200, 30], [900, 300, 4000])])
def test_graph_replay_and_other_stream(q, kv):
    p = Problem(q, kv, 8, 2, 128, 32, 800, 4, seed=17)
    want = [t.clone() for t in p.call(ops)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = p.call(ops)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs = [torch.zeros_like(want[0]), torch.zeros_like(want[1])]
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            p.call(ops, out=outs[0], lse=outs[1])
        graphs.append(gr)
    for gr in graphs + graphs:
        outs[0].fill_(SENTINEL)
        outs[1].fill_(SENTINEL)
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("chunk,window,sinks", [(1, 40, 4), (1, 1 << 20, 0), (24, 49, 10)])
def test_steps_with_the_cache_writer(chunk, window, sinks):
    """Both operators as a model uses them: two sequences advance by prompts,
    single tokens or chunks; every output against the attention of the whole
    sequence so far in 64 bits, keys as the cache holds them."""
    H, Hkv, hd, page, S, M = 4, 2, 64, 16, 2, 20
    rng = random.Random(18)
    g = torch.Generator(device="cuda").manual_seed(18)
    pages = list(range(S * M))
    rng.shuffle(pages)
    table = torch.tensor(pages, dtype=torch.int32, device="cuda").view(S, M)
    kc, vc = (torch.full((S * M, Hkv, page, hd), float("nan"), dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    rope = torch.from_numpy(synth.rope_table(512, hd)).cuda()
    w = (1 + 0.1 * torch.randn(2, hd, generator=g, device="cuda")).bfloat16()
    lens = [0, 0]
    keep_k, keep_v = [[], []], [[], []]
    steps = [(48, 24), (24, 24), (24, 24), (24, 48)] if chunk > 1 else [(70, 3), (1, 1), (1, 1), (2, 30), (1, 1)]
    for add in steps:
        N = sum(add)
        qkv = torch.randn(N, (H + 2 * Hkv) * hd, generator=g, device="cuda").bfloat16()
        pos = [lens[s] + i for s in range(S) for i in range(add[s])]
        slot = [int(table[s, (lens[s] + i) // page]) * page + (lens[s] + i) % page
                for s in range(S) for i in range(add[s])]
        lens = [a + b for a, b in zip(lens, add)]
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        q = ops.qk_norm_rope_cache(qkv[:, :H * hd], qkv[:, H * hd:(H + Hkv) * hd], qkv[:, (H + Hkv) * hd:],
                                   w[0], w[1], rope, i32(pos), i32(slot), kc, vc, EPS, neox=True)
        out, lse = ops.window_attention(q, kc, vc, table, i32([0, add[0], N]), i32(lens), window,
                                        sinks=sinks, chunk=chunk, lse=True)
        p = Problem(add, lens, H, Hkv, hd, page, window, sinks, chunk, seed=0, poison=False)
        p.q = q
        for s in range(S):
            ids = table[s, :-(-lens[s] // page)].long()
            p.K[s] = kc[ids].transpose(0, 1).reshape(Hkv, -1, hd)[:, :lens[s]]
            p.V[s] = vc[ids].transpose(0, 1).reshape(Hkv, -1, hd)[:, :lens[s]]
            assert p.K[s].isfinite().all() and p.V[s].isfinite().all()
        p.check((out, lse), f"after {lens}")


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes whose used pages lie at its end."""
    hd, page, Hkv = 128, 64, 8
    pages = (1 << 32) // (Hkv * page * hd * 2) + 40
    kc = torch.zeros((pages, Hkv, page, hd), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    p = Problem([1, 30], [500, 100], 16, Hkv, hd, page, seed=19)
    n = p.k_cache.shape[0]
    kc[-n:], vc[-n:] = p.k_cache, p.v_cache
    live = (p.table >= 0) & (p.table < n)
    p.table.copy_(torch.where(live, p.table + (pages - n), p.table))
    p.k_cache, p.v_cache = kc, vc
    run(p)
    r = rope_problem(20, 16, Hkv, hd, page, 20)
    small = r["caches"][0].shape[0]
    kc[-small:], vc[-small:] = r["caches"][0], r["caches"][1]
    first = dict(r, caches=[kc, vc], slots=(r["slots"] + (pages - small) * page).astype(np.int32))
    got = rope_call(first, True)
    rope_check(dict(r, caches=[kc[-small:].clone(), vc[-small:].clone()]), got, True)


def test_row_offsets_past_32_bits():
    """Queries, outputs and rotated rows more than 2^31 elements into their buffers."""
    H, Hkv, hd = 64, 8, 128
    N = (1 << 31) // (H * hd) + 400
    p = Problem([300, 1, 40], [300, 900, 6000], H, Hkv, hd, 64, seed=45)
    q = torch.zeros((N, H, hd), dtype=torch.bfloat16, device="cuda")
    q[-p.N:] = p.q
    out = torch.full_like(q, SENTINEL)
    lse = torch.full((N, H), SENTINEL, device="cuda")
    ops.window_attention(q, p.k_cache, p.v_cache, p.table, p.q_start + (N - p.N), p.kv_len, p.window,
                         scale=p.scale, max_q=300, out=out, lse=lse)
    p.check((out[-p.N:], lse[-p.N:]))
    assert (out[:-p.N] == SENTINEL).all() and (lse[:-p.N] == SENTINEL).all()
    del out, lse

    # the last 50 tokens of as many, all padding but those
    r = rope_problem(50, H, 1, hd, 64, 46)
    kv = torch.zeros((N, 2 * hd), dtype=torch.bfloat16, device="cuda")
    q[-50:], kv[-50:, :hd], kv[-50:, hd:] = r["q"].reshape(50, H, hd), r["k"], r["v"]
    pos, slots = np.zeros(N, np.int32), np.full(N, -1, np.int32)
    pos[-50:], slots[-50:] = r["pos"], r["slots"]
    got = rope_call(dict(r, q=q, k=kv[:, :hd], v=kv[:, hd:], pos=pos, slots=slots), True, q_out=q)
    rope_check(r, got[-50:], True)
    assert (q[:-50 - p.N] == 0).all()


def test_no_rows_allowed():
    """max_q = 0: every sequence that has rows is left out."""
    p = Problem([1, 0, 30], [9, 5, 30], 2, 1, 64, 16, seed=47)
    out, lse = p.call(ops, max_q=0)
    torch.cuda.synchronize()
    assert ops.device_status() == 8
    assert (out == SENTINEL).all() and (lse == SENTINEL).all()


def test_a_page_twice_in_one_sequence():
    """Repeated tokens: two entries of a table row name one page."""
    p = Problem([1, 40], [200, 240], 8, 2, 128, 32, seed=48)
    for s in (0, 1):
        p.table[s, 4] = p.table[s, 1]
        p.K[s][:, 128:160], p.V[s][:, 128:160] = p.K[s][:, 32:64].clone(), p.V[s][:, 32:64].clone()
    run(p)


def refuses(error, call, **changed):
    with pytest.raises(error) as e:
        call(**changed)
    if error is ops.DanError:
        assert e.value.status in (ops.DAN_EINVAL, ops.DAN_EALIGN, ops.DAN_EALIAS, ops.DAN_EUNSUPPORTED)


def test_rope_cache_refusals():
    """Each by its type, before anything is written."""
    p = rope_problem(6, 4, 2, 64, 16, 49)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    good = dict(q=p["q"], k=p["k"], v=p["v"], wq=p["w"][0], wk=p["w"][1], rope=dev(p["table"]),
                positions=dev(p["pos"]), slots=dev(p["slots"]), k_cache=p["caches"][0], v_cache=p["caches"][1])
    before = [c.clone() for c in p["caches"]]
    call = lambda **kw: ops.qk_norm_rope_cache(**{**good, "eps": EPS, **kw})  # noqa: E731
    for name in good:
        refuses(TypeError, call, **{name: good[name].cpu()})
        refuses(TypeError, call, **{name: good[name].double()})
        refuses(TypeError, call, **{name: None})
    for name in ("positions", "slots"):
        refuses(TypeError, call, **{name: good[name].long()})
        refuses(ValueError, call, **{name: good[name][:5]})
        refuses(ValueError, call, **{name: torch.stack([good[name]] * 2, 1)[:, 0]})
    refuses(ValueError, call, q=good["q"][:, :-1])
    refuses(ValueError, call, k=good["k"][:, :64])
    refuses(ValueError, call, v=good["v"].clone())            # another row stride than k's
    refuses(ValueError, call, q=good["q"].t().contiguous().t())
    refuses(ValueError, call, wq=good["wq"][:32])
    refuses(ValueError, call, rope=good["rope"][:, :32])
    refuses(ValueError, call, k_cache=good["k_cache"][:, :1])
    refuses(ValueError, call, k_cache=good["k_cache"].transpose(1, 2))
    refuses(ValueError, call, q_out=torch.empty((6, 4, 32), dtype=torch.bfloat16, device="cuda"))
    refuses(ops.DanError, call, eps=-1.0)
    refuses(ops.DanError, call, eps=float("nan"))
    refuses(ops.DanError, call, q=torch.zeros(6, 4 * 64 + 4, dtype=torch.bfloat16, device="cuda")[:, 4:])
    refuses(ops.DanError, call, q_out=good["q"].as_strided((6, 4, 64), (good["q"].stride(0), 64, 1),
                                                           good["q"].storage_offset() + 64))
    refuses(ops.DanError, call, v_cache=good["k_cache"])
    refuses(ops.DanError, call, q=good["q"][:, :3 * 64])       # 3 heads on 2 key heads
    small = [torch.zeros((9, 2, 8, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    refuses(ops.DanError, call, k_cache=small[0], v_cache=small[1])
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(p["caches"], before))
    call()


def test_attention_refusals():
    p = Problem([1, 20], [30, 40], 4, 2, 64, 16, seed=50, poison=False)
    good = dict(q=p.q, k_cache=p.k_cache, v_cache=p.v_cache, page_table=p.table, q_start=p.q_start, kv_len=p.kv_len)
    out = torch.full((21, 4, 64), SENTINEL, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((21, 4), SENTINEL, device="cuda")
    call = lambda **kw: ops.window_attention(**{**good, "window": 9, "out": out, "lse": lse, **kw})  # noqa: E731
    for name in good:
        refuses(TypeError, call, **{name: good[name].cpu()})
        refuses(TypeError, call, **{name: good[name].double()})
        refuses(TypeError, call, **{name: None})
    for name in ("page_table", "q_start", "kv_len"):
        refuses(TypeError, call, **{name: good[name].long()})
    refuses(ValueError, call, q=p.q.flatten(1))
    refuses(ValueError, call, q=p.q[..., :32])
    refuses(ValueError, call, q=p.q.transpose(1, 2).contiguous().transpose(1, 2))
    refuses(ValueError, call, page_table=p.table.t().contiguous().t())
    refuses(ValueError, call, page_table=p.table[0])
    refuses(ValueError, call, q_start=p.q_start[:2])
    refuses(ValueError, call, kv_len=p.kv_len[:1])
    refuses(ValueError, call, out=out[:20])
    refuses(ValueError, call, lse=lse[:, :3])
    refuses(TypeError, call, out=out.float())
    refuses(TypeError, call, lse=lse.bfloat16())
    for name in ("window", "sinks", "chunk", "max_q"):
        refuses(ValueError, call, **{name: -1})
        refuses(ValueError, call, **{name: 1 << 31})
    refuses(ops.DanError, call, chunk=0)
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        refuses(ops.DanError, call, scale=scale)
    refuses(ops.DanError, call, q=torch.zeros((21, 3, 64), dtype=torch.bfloat16, device="cuda"),
            out=torch.empty((21, 3, 64), dtype=torch.bfloat16, device="cuda"), lse=None)
    refuses(ops.DanError, call, page_table=p.table[:1].expand(2, -1))   # rows on one another
    both = p.q.contiguous()
    refuses(ops.DanError, call, q=both, out=both)
    torch.cuda.synchronize()
    assert (out == SENTINEL).all() and (lse == SENTINEL).all()
    call()
