"""The training operators over the whole of the ranges that they take: the narrowest rows, the
shortest batches, many images, levels far above the spread, buffers of exactly their size; against
64-bit references (tests/_train.py), the oracle's bits, and the plain form's time."""
import numpy as np
import pytest
import torch

import _train as ref
from _gpu import from_dev
from dit_adaln_norm_gb300 import ops

pytestmark = pytest.mark.gpu
BF16, FP16, FP32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.uint8
EPS = 1e-6


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, std=1.0, mean=0.0, dtype=BF16):
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)


@pytest.fixture(autouse=True)
def no_bad_status():
    yield
    torch.cuda.synchronize()
    assert ops.device_status() == 0


def device_us(f, reps=5):
    """The least device time of a call, in microseconds."""
    f()
    times = []
    for _ in range(reps):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 1e3)
    return min(times)


def same_bits(a, b):
    a, b = a.contiguous().view(torch.int32), b.contiguous().view(torch.int32)
    nan = lambda t: (t & 0x7FFFFFFF) > 0x7F800000  # noqa: E731
    return bool(((a == b) | (nan(a) & nan(b))).all())


# ------------------------------------------------------------- LayerNorm of short rows

SHORT = [8, 16, 24, 32, 40, 64, 72, 128, 136, 256, 264, 504, 512, 520, 768, 776, 1016, 1024, 1032]


@pytest.mark.parametrize("D", SHORT)
def test_short_rows_have_the_oracles_statistics(orc, D):
    """Mean and 1/std of ln_modulate's definition bit for bit, whatever is in a row; the codes and
    scales of the format, y within its rounding."""
    B, T = 3, 67
    g = gen(D)
    x = normal(g, B, T, D, mean=0.5)
    x[:, 1] *= 1e4
    x[:, 2] = 0
    x[:, 3] = -0.0
    x[:, 4] = 1e-40
    x[0, 5, -1], x[0, 6, 0], x[0, 7, D // 2], x[0, 8, :8] = float("nan"), float("inf"), float("-inf"), 3e38
    emb = normal(g, B, 3 * D, std=0.3)
    scale, shift = emb[:, :D], emb[:, 2 * D:]
    for checkpoint in (True, False):
        y, (stats, codes, scales) = ops.ln_modulate_save(x, scale, shift, EPS, checkpoint=checkpoint)
        _, st = orc.ln_modulate(from_dev(x), from_dev(scale), from_dev(shift), EPS, with_stats=True)
        want = torch.from_numpy(st[:, [0, 2]].copy()).view(B, T, 2).cuda()
        assert same_bits(stats, want)
        fine = [i for i in range(T) if not 5 <= i <= 8]
        w, _, e, _ = ref.ln_forward(x[:, fine], scale, shift, EPS)
        ref.assert_near(y[:, fine], w, e, "y")
        assert bool(y[0, 5:8].isnan().all()) and bool(y[1:].isfinite().all())
    c, s = ref.checkpoint(x)
    codes, scales = ops.ln_modulate_save(x, scale, shift, EPS)[1][1:]
    nan = (c & 0x7F == 0x7F) & (codes & 0x7F == 0x7F)
    assert bool(((codes == c) | nan).all()) and torch.equal(scales, s)


@pytest.mark.parametrize("B,T,D", [(1, 1, 8), (1, 50000, 8), (7, 1, 16), (5000, 1, 24), (3, 9001, 40), (1001, 3, 64),
                                   (2, 33, 256), (11, 31, 264), (400, 7, 1000)])
def test_short_rows_of_any_batches(B, T, D):
    """Batches of one row, of fewer rows than a warp takes, and of many; in place too."""
    g = gen(1)
    x, emb = normal(g, B, T, D, mean=0.5), normal(g, B, 2 * D, std=0.3)
    y, saved = ops.ln_modulate_save(x, emb[:, :D], emb[:, D:], EPS)
    want, st, ey, est = ref.ln_forward(x, emb[:, :D], emb[:, D:], EPS)
    ref.assert_near(y, want, ey, "y")
    ref.assert_near(saved[0], st, est, "stats")
    c, s = ref.checkpoint(x)
    assert torch.equal(saved[1], c) and torch.equal(saved[2], s)
    z = x.clone()
    assert ops.ln_modulate_save(z, emb[:, :D], emb[:, D:], EPS, out=z)[0] is z and torch.equal(z, y)


@pytest.mark.parametrize("rows,D", [(500000, 8), (500000, 16), (300000, 64), (150000, 128)])
def test_many_short_rows_take_less_than_torch(rows, D):
    """A warp a row, one at a time, took 1.3 to 13 times as long as these five torch operations."""
    g = gen(2)
    x, scale, shift = normal(g, 1, rows, D), normal(g, 1, D), normal(g, 1, D)

    def plain():
        v = x.float()
        d = v - v.mean(-1, keepdim=True)
        r = (d.square().mean(-1, keepdim=True) + EPS).rsqrt()
        return (d * r * (1 + scale.float()[:, None]) + shift.float()[:, None]).bfloat16()

    for checkpoint in (False, True):
        assert device_us(lambda: ops.ln_modulate_save(x, scale, shift, EPS, checkpoint=checkpoint)) < device_us(plain)


# ------------------------------------------------------------------------- group norm

@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("N,S", [(1, 0), (2, 0), (5, 0), (0, 4), (0, 0)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_gradients_of_nothing_are_zeros_whatever_the_parameters(dtype, N, S, bad):
    """Sums of no terms; the parameters are not looked at."""
    C, groups = 320, 32
    e = torch.empty((N, S, C), dtype=dtype, device="cuda")
    w, b = (torch.full((C,), bad, dtype=dtype, device="cuda") for _ in range(2))
    s, t = (torch.full((N, C), bad, dtype=dtype, device="cuda") for _ in range(2))
    saved = (torch.full((N, groups, 2), bad, device="cuda"), None, None)
    for act in (None, "silu"):
        got = ops.group_norm_backward(e, e, groups, w, b, saved, act=act, scale=s, shift=t)
        assert got[0].shape == e.shape
        for g, like in zip(got[1:], (w, b, s, t)):
            assert g.shape == like.shape and g.dtype is dtype and not g.any()
        dw, db = ops.group_norm_backward(e, e, groups, w.float(), b.float(), saved, act=act)[1:3]
        assert dw.dtype is FP32 and not dw.any() and not db.any()


# (N, S, C, groups): one CTA's slab, clusters, few chunks and many, whole tiles and narrow groups
CUTS = [(2, 64, 320, 32), (1, 3, 96, 4), (1, 1000, 1280, 32), (2, 777, 640, 16), (1, 6000, 512, 8), (2, 9001, 96, 3),
        (1, 100001, 64, 32), (1, 70000, 24, 1), (1, 300001, 16, 2)]


@pytest.mark.parametrize("N,S,C,groups", CUTS)
@pytest.mark.parametrize("level", [1000.1, -3001.7, 1.7e20])
def test_equal_values_have_no_spread(N, S, C, groups, level):
    """Whatever the bits of their level: the mean is exact, and what is normalised zero."""
    x = torch.full((N, S, C), level, dtype=FP32, device="cuda")
    x += torch.arange(groups, device="cuda").repeat_interleave(C // groups) * 0.7   # each group its own
    y, saved = ops.group_norm_save(x, groups, None, None, EPS, checkpoint=False)
    assert torch.equal(saved[0][..., 0], x[:, 0, ::C // groups])
    assert not y.any() and bool((saved[0][..., 1].double() - EPS ** -0.5).abs().max() < 1e-3 * EPS ** -0.5)


@pytest.mark.parametrize("N,S,C,groups", CUTS)
def test_means_of_a_level_far_above_the_spread(N, S, C, groups):
    """A mean is off by the roundings of the level at its three joins (a thread's values, a CTA's, the
    image's), half a step each, and by the differences' own sums."""
    x = normal(gen(4), N, S, C, mean=1e5, dtype=FP32)
    mean, rstd = ops.group_norm_save(x, groups, None, None, EPS, checkpoint=False)[1][0].double().unbind(-1)
    v = x.double().unflatten(2, (groups, -1))
    want = v.mean((1, 3))
    far = (v - want[:, None, :, None]).abs().amax((1, 3))
    lim = 3 * 2.0 ** -24 * 2.0 ** 17 + ref.E * far          # (1e5 < 2^17)
    assert bool(((mean - want).abs() <= lim).all())
    std = (v - want[:, None, :, None]).square().mean((1, 3)).add(EPS).sqrt()
    # each join's means are off by so much at most, and what they add to the squares too
    assert bool(((rstd * std - 1).abs() <= 2 * lim * rstd + ref.E * (1 + far * rstd)).all())


# ------------------------------------------------------------- LayerNorm gradients

def ln_back_case(B, T, D, ckpt, res, seed=0):
    g = gen(seed)
    x, emb = normal(g, B, T, D, mean=0.5), normal(g, B, 3 * D, std=0.3)
    saved = ops.ln_modulate_save(x, emb[:, :D], emb[:, D:2 * D], EPS, checkpoint=ckpt)[1]
    dy = normal(g, B, T, D, std=0.1, mean=0.02)
    return x, emb[:, :D], saved, dy, normal(g, B, T, D, std=0.1) if res else None


def check_ln_back(got, x, scale, saved, dy, dres):
    B, T, D = dy.shape
    v = x.double() if saved[1] is None else ref.restore(*saved[1:])
    want, err = ref.ln_backward(dy, v, saved[0], scale, dres, min(T, -(-B * T // min(max(B * T, 1), 148))))
    for a, w, e, name in zip(got, want, err, ("dx", "dscale", "dshift")):
        ref.assert_near(a, w, e, name)


# a width of each cut: several rows a warp, one to five fragments a lane, teams of three to eight warps
CUT_WIDTHS = [8, 16, 40, 136, 256, 264, 520, 776, 1032, 1280, 1288, 2048, 2056, 3064, 3080, 4096, 4104, 6152, 8192]


@pytest.mark.parametrize("D", CUT_WIDTHS)
@pytest.mark.parametrize("ckpt,res", [(True, False), (False, True), (True, True), (False, False)])
def test_many_short_batches(D, ckpt, res):
    """Of one row each, of three, and of none, the gradients' places as slices of one embedding."""
    for B, T in ((700, 1), (401, 3), (350, 0)):
        x, scale, saved, dy, dres = ln_back_case(B, T, D, ckpt, res)
        demb = torch.full((B, 4 * D), 77, dtype=BF16, device="cuda")
        got = ops.ln_modulate_backward(dy, None if ckpt else x, scale, saved, dres=dres, dscale=demb[:, 2 * D:3 * D],
                                       dshift=demb[:, D:2 * D])
        check_ln_back(got, x, scale, saved, dy, dres)
        assert bool((demb[:, :D] == 77).all()) and bool((demb[:, 3 * D:] == 77).all())


@pytest.mark.parametrize("D", CUT_WIDTHS)
@pytest.mark.parametrize("ckpt", [True, False])
def test_a_rows_dx_is_its_own_at_every_width(D, ckpt):
    """The same bits alone, among the rows of a long batch and of short ones, in place too; a bad
    row spoils no other."""
    x, scale, saved, dy, dres = ln_back_case(1, 900, D, ckpt, True)
    keep = lambda s, at: tuple(None if t is None else t[:, at].contiguous() for t in s)  # noqa: E731
    dx = ops.ln_modulate_backward(dy, None if ckpt else x, scale, saved, dres=dres)[0]
    for at in (slice(0, 1), slice(17, 40), slice(899, 900), slice(100, 700)):
        cut = lambda t: t[:, at].contiguous()  # noqa: E731
        one = ops.ln_modulate_backward(cut(dy), None if ckpt else cut(x), scale, keep(saved, at), dres=cut(dres))[0]
        assert torch.equal(one, dx[:, at]), at
    for B, T in ((900, 1), (450, 2), (300, 3), (30, 30)):
        as_batches = lambda t: None if t is None else t.view(B, T, -1)  # noqa: E731
        d = as_batches(dy.clone())
        got = ops.ln_modulate_backward(d, None if ckpt else as_batches(x), scale.expand(B, D).contiguous(),
                                       tuple(map(as_batches, saved)), dres=as_batches(dres), dx=d)[0]
        assert torch.equal(got.view(1, 900, D), dx), (B, T)
        bad = as_batches(dy.clone())
        bad[-1, 0, 3], bad[11, -1, D - 1] = float("nan"), float("inf")
        got = ops.ln_modulate_backward(bad, None if ckpt else as_batches(x), scale.expand(B, D).contiguous(),
                                       tuple(map(as_batches, saved)), dres=as_batches(dres))[0].view(1, 900, D)
        rows = [i for i in range(900) if i not in ((B - 1) * T, 12 * T - 1)]
        assert torch.equal(got[:, rows], dx[:, rows])


@pytest.mark.parametrize("B", [2, 9, 11, 16, 50, 52, 153, 290, 310])
@pytest.mark.parametrize("T,D", [(40, 264), (7, 4096), (300, 40)])
def test_batches_of_few_and_many_partials(B, T, D):
    """The joins of 64, of 8 and of one thread a column."""
    case = ln_back_case(B, T, D, True, False)
    check_ln_back(ops.ln_modulate_backward(case[3], None, case[1], case[2]), *case)


@pytest.mark.parametrize("B,T,D", [(20000, 1, 64), (4000, 8, 64), (8000, 1, 1024), (1953, 8, 1024), (3906, 1, 4096),
                                   (488, 8, 4096), (61, 64, 4096)])
def test_short_batches_take_less_than_torch(B, T, D):
    """A join of 64 threads a column and batch took up to nine times as long as these operations."""
    x, scale, saved, dy, _ = ln_back_case(B, T, D, False, False)

    def plain():
        n = (x.float() - saved[0][..., :1]) * saved[0][..., 1:]
        d = dy.float()
        g = d * (1 + scale.float()[:, None])
        dx = saved[0][..., 1:] * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True))
        return dx.bfloat16(), (d * n).sum(1).bfloat16(), d.sum(1).bfloat16()

    assert device_us(lambda: ops.ln_modulate_backward(dy, x, scale, saved)) < device_us(plain)


# ------------------------------------------------------------- group norms of many images

@pytest.mark.parametrize("N,S,C,groups", [(255, 2, 64, 8), (256, 1, 40, 5), (257, 3, 32, 4), (1000, 1, 96, 3),
                                          (65537, 1, 16, 2), (70000, 2, 8, 1), (300, 700, 24, 3)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_parameter_gradients_of_many_images(N, S, C, groups, dtype):
    """Sums of 256 images at a time; the same bits every time."""
    g = gen(6)
    x, dy = normal(g, N, S, C, mean=0.5, dtype=dtype), normal(g, N, S, C, std=0.1, mean=0.02, dtype=dtype)
    w, b = normal(g, C, std=0.3, mean=1.0, dtype=dtype), normal(g, C, std=0.3, dtype=dtype)
    emb = normal(g, N, 2 * C, std=0.3, dtype=dtype)
    s, t = emb[:, :C], emb[:, C:]
    saved = ops.group_norm_save(x, groups, w, b, 0.1, act="silu", scale=s, shift=t, checkpoint=False)[1]
    got = ops.group_norm_backward(dy, x, groups, w, b, saved, act="silu", scale=s, shift=t)
    want, err = ref.gn_backward(dy, x.double(), groups, w, b, saved[0], "silu", s, t)
    for a, u, e, name in zip(got, want, err, ("dx", "dweight", "dbias", "dscale", "dshift")):
        ref.assert_near(a, u, e, name)
    again = ops.group_norm_backward(dy, x, groups, w, b, saved, act="silu", scale=s, shift=t)
    assert all(torch.equal(u, v) for u, v in zip(got, again))


def plain_group_norm_backward(dy, x, groups, w, b, saved):
    """The formulas in elementary torch operations."""
    N, S, C = x.shape
    mean, rstd = (saved[0][:, None, :, i].repeat_interleave(C // groups, 2) for i in range(2))
    n = (x.float() - mean) * rstd
    z = n * w.float() + b.float()
    p = 1 / (1 + (-z).exp())
    dz = dy.float() * (p * (1 + z * (1 - p)))
    g = dz * w.float()
    avg = lambda v: v.unflatten(2, (groups, -1)).mean((1, 3)).repeat_interleave(C // groups, 1)[:, None]  # noqa: E731
    dx = (rstd * (g - avg(g) - n * avg(g * n))).to(x.dtype)
    return dx, (dz * n).sum((0, 1)).to(w.dtype), dz.sum((0, 1)).to(b.dtype)


@pytest.mark.parametrize("N,S,C,groups", [(65536, 1, 64, 8), (4096, 16, 320, 32)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_gradients_of_many_images_take_less_than_torch(N, S, C, groups, dtype):
    """A chain of N / 8 loads for each parameter took six times as long as these operations."""
    g = gen(7)
    x, dy = normal(g, N, S, C, dtype=dtype), normal(g, N, S, C, dtype=dtype)
    w, b = normal(g, C, dtype=dtype), normal(g, C, dtype=dtype)
    saved = ops.group_norm_save(x, groups, w, b, EPS, checkpoint=False)[1]
    assert device_us(lambda: ops.group_norm_backward(dy, x, groups, w, b, saved, act="silu")) < \
        device_us(lambda: plain_group_norm_backward(dy, x, groups, w, b, saved))


@pytest.mark.parametrize("N,S,C,groups", [(16384, 1, 1024, 32), (65536, 1, 64, 8), (8192, 2, 1024, 32)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_many_images_of_few_positions_take_less_than_torch(N, S, C, groups, dtype):
    """CTAs of eight live threads took up to 1.5 times as long as these operations."""
    g = gen(8)
    x = normal(g, N, S, C, dtype=dtype)
    w, b = normal(g, C, dtype=dtype), normal(g, C, dtype=dtype)

    def plain():
        v = x.float().unflatten(2, (groups, -1))
        d = v - v.mean((1, 3), keepdim=True)
        n = (d * (d.square().mean((1, 3), keepdim=True) + EPS).rsqrt()).flatten(2)
        z = n * w.float() + b.float()
        return (z / (1 + (-z).exp())).to(dtype)

    assert device_us(lambda: ops.group_norm(x, groups, w, b, EPS, act="silu")) < device_us(plain)


@pytest.mark.parametrize("S", [1, 2, 3, 4, 7])
@pytest.mark.parametrize("C,groups", [(8, 1), (24, 3), (96, 3), (320, 32), (640, 32), (1024, 32), (4096, 1), (8192, 32),
                                      (40, 8), (2560, 2)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_group_norm_of_few_positions(S, C, groups, dtype):
    N = 37
    g = gen(9)
    x = normal(g, N, S, C, mean=0.5, dtype=dtype)
    w, b = normal(g, C, std=0.3, mean=1.0, dtype=dtype), normal(g, C, std=0.3, dtype=dtype)
    ckpt = C % 32 == 0
    y, (stats, codes, scales) = ops.group_norm_save(x, groups, w, b, 0.1, act="silu", checkpoint=ckpt)
    want, st, ey, est = ref.gn_forward(x, groups, w, b, 0.1, "silu", None, None)
    ref.assert_near(y, want, ey, "y")
    ref.assert_near(stats, st, est, "stats")
    if ckpt:
        c, s = ref.checkpoint(x)
        assert torch.equal(codes, c) and torch.equal(scales, s)
    one = ops.group_norm_save(x[5:6], groups, w, b, 0.1, act="silu", checkpoint=ckpt)
    assert torch.equal(one[0], y[5:6]) and torch.equal(one[1][0], stats[5:6])


@pytest.mark.parametrize("groups", [65, 1 << 40, (1 << 64) + 8, 0, -8])
def test_more_groups_than_channels_are_refused(groups):
    """By their number alone, with nothing allocated for them."""
    x = normal(gen(0), 4, 100, 64)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    for call in (lambda: ops.group_norm_save(x, groups, None, None, EPS, checkpoint=False),
                 lambda: ops.group_norm(x, groups, None, None, EPS)):
        with pytest.raises(ops.DanError):
            call()
    assert torch.cuda.max_memory_allocated() == before


def gn_case(N, S, C, dtype, mod, seed=0):
    g = gen(seed)
    x = normal(g, N, S, C, mean=0.5, dtype=dtype)
    x *= torch.exp(0.3 * torch.randn(C, generator=g, device="cuda")).to(dtype)
    w, b = normal(g, C, std=0.3, mean=1.0, dtype=dtype), normal(g, C, std=0.3, dtype=dtype)
    emb = normal(g, N, 2 * C, std=0.3, dtype=dtype)
    s, t = (emb[:, :C], emb[:, C:]) if mod else (None, None)
    return x, w, b, s, t, normal(g, N, S, C, std=0.1, mean=0.02, dtype=dtype)


def check_gn_case(x, groups, w, b, s, t, dy, ckpt, terms=128):
    """Both directions; `terms`: the roundings of a sum's longest chain."""
    k = terms / 128
    y, saved = ops.group_norm_save(x, groups, w, b, EPS, act="silu", scale=s, shift=t, checkpoint=ckpt)
    want, st, ey, est = ref.gn_forward(x, groups, w, b, EPS, "silu", s, t)
    ref.assert_near(y, want, k * ey, "y")
    ref.assert_near(saved[0], st, k * est, "stats")
    if ckpt:
        c, q = ref.checkpoint(x)
        assert torch.equal(saved[1], c) and torch.equal(saved[2], q)
    del y, want, ey
    v = ref.restore(*saved[1:]) if ckpt else x.double()
    got = ops.group_norm_backward(dy, None if ckpt else x, groups, w, b, saved, act="silu", scale=s, shift=t)
    want, err = ref.gn_backward(dy, v, groups, w, b, saved[0], "silu", s, t)
    for a, u, e, name in zip(got, want, err, ("dx", "dweight", "dbias", "dscale", "dshift")):
        if u is not None:
            ref.assert_near(a, u, k * e, name)


# in passes, with tiles of 250 and 230 fragments (fp32), 250 and 70, 240, 240 and 40, 255 and 225; in slabs
# whose last one is narrower
@pytest.mark.parametrize("N,S,C,groups", [(1, 20000, 1920, 48), (2, 9000, 2560, 32), (1, 6000, 4160, 13),
                                          (1, 7001, 3840, 32), (1, 5000, 2600, 13), (3, 50, 2600, 13), (2, 300, 1000, 25),
                                          (2, 70, 416, 13)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_tiles_whose_last_one_is_narrower(N, S, C, groups, dtype):
    for ckpt in (True, False) if C % 32 == 0 else (False,):
        x, w, b, s, t, dy = gn_case(N, S, C, dtype, ckpt)
        check_gn_case(x, groups, w, b, s, t, dy, ckpt)


@pytest.mark.parametrize("ckpt", [True, False])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_large_images_in_64_bits(dtype, ckpt):
    """Rows as wide as a CTA and so many that a thread adds some 165 of them in turn, in the gradients
    330 (608 and 304 chunks), and a join as many chunks."""
    x, w, b, s, t, dy = gn_case(1, 100000, 1024 if dtype is FP32 else 2048, dtype, True)
    check_gn_case(x, 32, w, b, s, t, dy, ckpt, terms=330 + 128)


class Buffers:
    """Buffers of exactly the bytes that a call needs, between bytes that it must not write."""

    def __init__(self):
        self.all = []

    def out(self, nbytes, align=16, pad=1024):
        buf = torch.full((nbytes + 2 * pad + align,), 0xA5, dtype=U8, device="cuda")
        at = pad + align if align < 16 else pad          # no better aligned than it needs
        self.all.append((buf, at, nbytes))
        assert (buf.data_ptr() + at) % align == 0
        return buf.data_ptr() + at

    def check(self):
        torch.cuda.synchronize()
        for buf, at, n in self.all:
            assert bool((buf[:at] == 0xA5).all()) and bool((buf[at + n:] == 0xA5).all()), (n, at)


@pytest.mark.parametrize("B,T,D", [(1, 1, 8), (3, 41, 24), (2, 67, 1160), (500, 3, 40), (1, 333, 4104), (2, 9, 1016),
                                   (16, 40, 520), (60, 7, 2056), (1, 200, 1024)])
def test_ln_calls_stay_in_buffers_of_their_size(B, T, D):
    x, scale, _, dy, _ = ln_back_case(B, T, D, False, False)
    scale = scale.contiguous()
    rows, blocks, lib = B * T, (D + 31) // 32, ops.load()
    b = Buffers()
    y, stats, codes, scales = b.out(rows * D * 2), b.out(rows * 8, 8), b.out(rows * D, 8), b.out(rows * blocks, 1)
    ops._on(0, "dan_ln_modulate_save", x.data_ptr(), scale.data_ptr(), scale.data_ptr(), D, y, stats, codes, scales,
            B, T, D, EPS)
    b.check()
    size = lib.dan_ln_modulate_backward_workspace(B, T, D)
    for from_x in (False, True):
        dx, dscale, dshift, work = b.out(rows * D * 2), b.out(B * D * 2), b.out(B * D * 2), b.out(size)
        ops._on(0, "dan_ln_modulate_backward", dy.data_ptr(), x.data_ptr() if from_x else None,
                None if from_x else codes, None if from_x else scales, stats, scale.data_ptr(), D, None, dx, dscale,
                dshift, D, B, T, D, work if size else None, size)
        b.check()


@pytest.mark.parametrize("N,S,C,groups", [(1, 1, 8, 1), (3, 5, 96, 3), (2, 77, 320, 32), (300, 2, 64, 8), (1, 20001, 64, 8),
                                          (2, 9001, 96, 3), (1, 5003, 2560, 32), (3, 3001, 1056, 33), (1, 300001, 8, 8)])
@pytest.mark.parametrize("ty,dtype", [(0, BF16), (1, FP16), (2, FP32)])
def test_gn_calls_stay_in_buffers_of_their_size(N, S, C, groups, ty, dtype):
    x, w, b_, s, t, dy = gn_case(N, S, C, dtype, True)
    s, t = s.contiguous(), t.contiguous()
    es, lib, n = x.element_size(), ops.load(), N * S * C
    ckpt = C % 32 == 0
    b = Buffers()
    y, stats = b.out(n * es), b.out(N * groups * 8, 8)
    codes, scales = (b.out(n, 8), b.out(n // 32, 1)) if ckpt else (None, None)
    size = lib.dan_group_norm_workspace(N, S, C, groups, ty, int(ckpt))
    ops._on(0, "dan_group_norm", x.data_ptr(), ty, w.data_ptr(), b_.data_ptr(), ty, s.data_ptr(), t.data_ptr(), C, 1, y,
            stats, codes, scales, N, S, C, groups, EPS, b.out(size) if size else None, size)
    b.check()
    for from_x in (True, False) if ckpt else (True,):
        size = lib.dan_group_norm_backward_workspace(N, S, C, groups, ty, int(not from_x))
        dx, dw, db, ds, dt = b.out(n * es), b.out(C * es), b.out(C * es), b.out(N * C * es), b.out(N * C * es)
        ops._on(0, "dan_group_norm_backward", dy.data_ptr(), x.data_ptr() if from_x else None, ty,
                None if from_x else codes, None if from_x else scales, stats, w.data_ptr(), b_.data_ptr(), ty, s.data_ptr(),
                t.data_ptr(), C, 1, dx, dw, db, ds, dt, C, N, S, C, groups, b.out(size) if size else None, size)
        b.check()


def test_gradients_of_narrow_rows_take_about_as_long_as_of_wide_ones():
    """Of as many bytes, replayed.  A hint to the L2 for each row at a call's start made it three times."""
    times = []
    for T, D in ((1 << 17, 8), (1 << 10, 1024)):
        x, scale, saved, dy, dres = ln_back_case(1, T, D, False, True)
        ops.ln_modulate_backward(dy, x, scale, saved, dres=dres)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(20):
                ops.ln_modulate_backward(dy, x, scale, saved, dres=dres)
        times.append(device_us(graph.replay))
    assert times[0] < 1.8 * times[1], times


@pytest.mark.parametrize("per", [1, 2, 3, 4, 7, 8, 12, 16, 17, 32, 33, 40])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_gradients_of_small_images_in_groups_of_any_width(per, dtype):
    """In one launch: lanes of a warp a group, or a warp; an image's are its own."""
    groups = 8 if per > 4 else 40
    for N, S in ((5, 9), (2, 200)):
        x, w, b, s, t, dy = gn_case(N, S, groups * per, dtype, True)
        check_gn_case(x, groups, w, b, s, t, dy, False)
        saved = ops.group_norm_save(x, groups, w, b, EPS, checkpoint=False)[1]
        got = ops.group_norm_backward(dy, x, groups, w, b, saved)[0]
        one = ops.group_norm_backward(dy[1:2], x[1:2], groups, w, b, (saved[0][1:2], None, None))[0]
        assert torch.equal(one, got[1:2])


def test_gradients_in_groups_of_one_channel_take_less_than_torch():
    N, S, C = 15184, 2, 200
    x, w, b, _, _, dy = gn_case(N, S, C, FP32, False)
    saved = ops.group_norm_save(x, C, w, b, EPS, checkpoint=False)[1]

    def plain():
        n = (x - saved[0][:, None, :, 0]) * saved[0][:, None, :, 1]
        g = dy * w
        dx = saved[0][:, None, :, 1] * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
        return dx, (dy * n).sum((0, 1)), dy.sum((0, 1))

    assert device_us(lambda: ops.group_norm_backward(dy, x, C, w, b, saved)) < device_us(plain)


@pytest.mark.parametrize("N,S,C,groups", [(47088, 1, 112, 112), (300000, 7, 8, 4), (65536, 1, 64, 8)])
def test_many_images_of_a_warp_take_less_than_torch(N, S, C, groups):
    """Images of up to 32 fragments in CTAs of two warps took up to 1.2 times as long as these operations."""
    x, w, b, _, _, _ = gn_case(N, S, C, FP16, False)

    def plain():
        v = x.float().unflatten(2, (groups, -1))
        d = v - v.mean((1, 3), keepdim=True)
        n = (d * (d.square().mean((1, 3), keepdim=True) + EPS).rsqrt()).flatten(2)
        z = n * w.float() + b.float()
        return (z / (1 + (-z).exp())).to(x.dtype)

    assert device_us(lambda: ops.group_norm(x, groups, w, b, EPS, act="silu")) < device_us(plain)


@pytest.mark.parametrize("N,S,C,groups", [(3000, 2, 16, 16), (1000, 1, 24, 3), (500, 4, 32, 4), (700, 3, 8, 1), (300, 8, 32, 1)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_images_of_a_warp(N, S, C, groups, dtype):
    x, w, b, s, t, dy = gn_case(N, S, C, dtype, True)
    g = groups
    for ckpt in (True, False) if C % 32 == 0 else (False,):
        k = dict(act="silu", scale=s, shift=t)
        y, saved = ops.group_norm_save(x, g, w, b, 0.1, checkpoint=ckpt, **k)
        want, st, ey, est = ref.gn_forward(x, g, w, b, 0.1, "silu", s, t)
        ref.assert_near(y, want, ey, "y")
        ref.assert_near(saved[0], st, est, "stats")
        got = ops.group_norm_backward(dy, None if ckpt else x, g, w, b, saved, **k)
        v = ref.restore(*saved[1:]) if ckpt else x.double()
        want, err = ref.gn_backward(dy, v, g, w, b, saved[0], "silu", s, t)
        for a, u, e, name in zip(got, want, err, ("dx", "dweight", "dbias", "dscale", "dshift")):
            ref.assert_near(a, u, e, name)


# ------------------------------------------------------------------ streams and graphs

def calls_of_the_ranges():
    """Calls that take the forms for narrow rows, short batches, many images and no positions."""
    x, scale, saved, dy, dres = ln_back_case(700, 2, 40, True, True)
    u, w, b, s, t, du = gn_case(600, 2, 64, BF16, True)
    kept = ops.group_norm_save(u, 8, w, b, EPS, act="silu", scale=s, shift=t)[1]
    none = u[:, :0]
    small, sw, sb, _, _, ds = gn_case(3, 30, 40, BF16, False)
    keep = ops.group_norm_save(small, 40, sw, sb, EPS, checkpoint=False)[1]
    wide = ln_back_case(20, 9, 4096, True, False)
    return [lambda: ops.ln_modulate_save(x, scale, scale, EPS)[0],
            lambda: ops.ln_modulate_backward(dy, None, scale, saved, dres=dres),
            lambda: ops.ln_modulate_backward(wide[3], None, wide[1], wide[2]),
            lambda: ops.group_norm(u, 8, w, b, EPS, act="silu", scale=s, shift=t),
            lambda: ops.group_norm_backward(du, None, 8, w, b, kept, act="silu", scale=s, shift=t),
            lambda: ops.group_norm_backward(none, none, 8, w, b, (kept[0], None, None), scale=s, shift=t),
            lambda: ops.group_norm_backward(ds, small, 40, sw, sb, keep)]


def tensors(v):
    return [v] if isinstance(v, torch.Tensor) else [t for t in v if t is not None]


def test_the_ranges_ends_on_streams_and_in_graphs():
    """The same bits on three streams at once, and from two graphs replayed in turn."""
    calls = calls_of_the_ranges()
    want = [tensors(f()) for f in calls]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(3)], []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append([tensors(f()) for f in calls])
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = [tensors(f()) for f in calls]
        graphs.append((graph, outs))
    for _ in range(2):
        for _, outs in graphs:
            for run in outs:
                for v in run:
                    v.fill_(3)
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        got += [[[v.clone() for v in run] for run in outs] for _, outs in graphs]
    for run in got:
        for a, b in zip(run, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_a_call_follows_what_the_stream_does_before_it():
    """Zeros for no positions, and short forms, on inputs that the kernel before still writes."""
    x, scale, saved, dy, _ = ln_back_case(20000, 1, 64, False, False)
    want = tensors(ops.ln_modulate_backward(dy, x, scale, saved))
    y = ops.ln_modulate_save(x, scale, scale, EPS)[0]
    src = [dy.clone(), x.clone(), scale.clone()]
    for _ in range(5):
        for v in (dy, x, scale):
            v.fill_(float("nan"))
        torch.cuda.synchronize()
        torch.cuda._sleep(200000)
        for v, k in zip((dy, x, scale), src):
            v.copy_(k)
        a = ops.ln_modulate_save(x, scale, scale, EPS)[0]
        b = tensors(ops.ln_modulate_backward(dy, x, scale, saved))
        assert torch.equal(a, y) and all(torch.equal(u, v) for u, v in zip(b, want))


@pytest.mark.parametrize("N,S,C,groups", [(3, 40, 64, 8), (2, 9000, 320, 32), (300, 1, 96, 3), (4, 0, 64, 8), (1, 70, 32, 4)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_group_norm_gradients_into_slices(N, S, C, groups, dtype):
    """dscale and dshift as slices of one embedding's gradient, the rest of it left as it was."""
    x, w, b, s, t, dy = gn_case(N, S, C, dtype, True)
    saved = ops.group_norm_save(x, groups, w, b, EPS, act="silu", scale=s, shift=t, checkpoint=False)[1]
    k = dict(act="silu", scale=s, shift=t)
    want = ops.group_norm_backward(dy, x, groups, w, b, saved, **k)
    demb = torch.full((N, 5 * C), 77, dtype=dtype, device="cuda")
    a, c = demb[:, 3 * C:4 * C], demb[:, C:2 * C]
    got = ops.group_norm_backward(dy, x, groups, w, b, saved, dscale=a, dshift=c, **k)
    assert got[3] is a and got[4] is c and all(torch.equal(u, v) for u, v in zip(got, want))
    rest = [i for i in range(5 * C) if not (C <= i < 2 * C or 3 * C <= i < 4 * C)]
    assert bool((demb[:, rest] == 77).all())


def test_group_norm_gradients_into_slices_refuse():
    x, w, b, s, t, dy = gn_case(2, 10, 64, BF16, True)
    saved = ops.group_norm_save(x, 8, w, b, EPS, scale=s, shift=t, checkpoint=False)[1]
    d = torch.zeros((2, 256), dtype=BF16, device="cuda")
    f = lambda scale=s, shift=t, **k: ops.group_norm_backward(dy, x, 8, w, b, saved, scale=scale, shift=shift, **k)  # noqa: E731
    for bad in (dict(dscale=d[:, :64]), dict(dshift=d[:, :64]), dict(dscale=d[:, :64], dshift=d[:, :32]),
                dict(dscale=d[:, :64], dshift=torch.zeros_like(d[:, :64])),
                dict(scale=None, shift=None, dscale=d[:, :64], dshift=d[:, 64:128])):
        with pytest.raises(ValueError):
            f(**bad)
    with pytest.raises(TypeError):
        f(dscale=d[:, :64].float(), dshift=d[:, 64:128].float())
    with pytest.raises(ops.DanError):
        f(dscale=d[:, :64], dshift=d[:, 32:96])               # they overlap
    with pytest.raises(ops.DanError):
        f(dscale=d[:, 4:68], dshift=d[:, 128:192])            # not on 16 bytes
    assert not d.any()
