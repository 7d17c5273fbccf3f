"""The training operators on the GPU against 64-bit references (tests/_train.py), at the sizes and
values where they can go wrong."""
import math

import pytest
import torch

import _train as ref
from dit_adaln_norm_gb300 import ops

pytestmark = pytest.mark.gpu
BF16, FP16, FP32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.uint8
EPS = 1e-6
TYPES = [BF16, FP16, FP32]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, std=1.0, mean=0.0, dtype=BF16):
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)


def guarded(shape, dtype, pad=4096):
    """(whole buffer, view) of an output with a sentinel on both sides."""
    n = math.prod(shape)
    buf = torch.full((n + 2 * pad,), 77, dtype=dtype, device="cuda")
    return buf, buf[pad:pad + n].view(shape)


def untouched(buf, pad=4096):
    return bool((buf[:pad] == 77).all()) and bool((buf[-pad:] == 77).all())


@pytest.fixture(autouse=True)
def no_bad_status():
    yield
    torch.cuda.synchronize()
    assert ops.device_status() == 0


# -------------------------------------------------------------------- LN forward

LN_SHAPES = [(1, 1, 8), (2, 3, 24), (1, 128, 2048), (2, 37, 1160), (1, 700, 1024), (3, 65, 4096), (1, 5000, 40),
             (2, 9, 8192), (1, 33, 6152), (700, 1, 264), (1, 4000, 4096)]


def ln_inputs(B, T, D, seed=0, level=0.5):
    g = gen(seed)
    x = normal(g, B, T, D, mean=level)
    x[..., :: max(D // 3, 1)] *= 20
    emb = normal(g, B, 6 * D, std=0.3)
    return g, x, emb[:, D:2 * D], emb[:, 4 * D:5 * D]


@pytest.mark.parametrize("B,T,D", LN_SHAPES)
@pytest.mark.parametrize("checkpoint", [True, False])
def test_ln_save(B, T, D, checkpoint):
    g, x, scale, shift = ln_inputs(B, T, D)
    y, (stats, codes, scales) = ops.ln_modulate_save(x, scale, shift, EPS, checkpoint=checkpoint)
    want, st, ey, est = ref.ln_forward(x, scale, shift, EPS)
    ref.assert_near(y, want, ey, "y")
    ref.assert_near(stats, st, est, "stats")
    if not checkpoint:
        assert codes is None and scales is None
        return
    c, s = ref.checkpoint(x)
    assert torch.equal(codes, c) and torch.equal(scales, s)


@pytest.mark.parametrize("D", [2048, 4096, 1160, 8192])
def test_ln_save_statistics_are_those_of_ln_modulate(D):
    """ln_modulate's chain of roundings from the kept mean and 1/std gives its bits."""
    _, x, scale, shift = ln_inputs(2, 150, D)
    mean, rstd = ops.ln_modulate_save(x, scale, shift, EPS)[1][0].split(1, -1)
    n = ((x.float() - mean) * rstd).to(BF16)
    assert torch.equal(ops.ln_modulate(x, scale, shift, EPS), n * (1 + scale)[:, None] + shift[:, None])


@pytest.mark.parametrize("B,T,D", [(2, 300, 1160), (1, 100, 2048), (1, 4216, 4096), (2, 9, 8192)])
def test_ln_save_in_place(B, T, D):
    _, x, scale, shift = ln_inputs(B, T, D)
    y, saved = ops.ln_modulate_save(x, scale, shift, EPS)
    z = x.clone()
    got, kept = ops.ln_modulate_save(z, scale, shift, EPS, out=z)
    assert got is z and torch.equal(z, y) and all(torch.equal(u, v) for u, v in zip(kept, saved))


def test_ln_save_level_far_above_the_spread():
    _, x, scale, shift = ln_inputs(1, 40, 2048, level=300.0)
    y, (stats, _, _) = ops.ln_modulate_save(x, scale, shift, EPS)
    want, st, ey, est = ref.ln_forward(x, scale, shift, EPS)
    ref.assert_near(y, want, ey)
    ref.assert_near(stats, st, est)


def special_rows(D, dtype):
    """Rows whose blocks are zero, at the scales' borders, huge, tiny, infinite and not a number."""
    g = gen(3)
    big = 60000.0 if dtype is FP16 else 3e38
    x = normal(g, 16, D, dtype=FP32)
    x[1] = 0
    x[2, :32], x[3, :32] = 448, 449
    x[2, 32:], x[3, 32:] = 0.875, -0.8755
    x[4] *= big / 8
    x[5] *= 1e-38
    x[6] *= 1e-44
    x[7, 3] = 1e-30
    x[8, ::2] = 0
    x[9] = -big
    return x.to(dtype)


def test_checkpoint_borders():
    D = 264
    x = special_rows(D, BF16)[None]
    zero = torch.zeros(D, dtype=BF16, device="cuda")
    _, (_, codes, scales) = ops.ln_modulate_save(x, zero, zero, EPS)
    c, s = ref.checkpoint(x)
    assert torch.equal(scales, s) and torch.equal(codes, c)


@pytest.mark.parametrize("dtype", TYPES)
def test_gn_checkpoint_borders(dtype):
    x = special_rows(320, dtype)[None]
    _, (_, codes, scales) = ops.group_norm_save(x, 10, None, None, EPS)
    c, s = ref.checkpoint(x)
    assert torch.equal(scales, s) and torch.equal(codes, c)


def test_checkpoint_of_infinities_and_nan():
    """Codes of what is not a number or infinite; the other rows are what they were."""
    D = 320
    g = gen(5)
    x = normal(g, 1, 6, D)
    x[0, 1, 7], x[0, 3, 40], x[0, 3, 41], x[0, 4, 0] = float("nan"), float("inf"), 5.0, float("-inf")
    zero = torch.zeros(D, dtype=BF16, device="cuda")
    for y, (stats, codes, scales) in (ops.ln_modulate_save(x, zero, zero, EPS),
                                      ops.group_norm_save(x.view(6, 1, D), 10, None, None, EPS)):
        c, s = ref.checkpoint(x)
        assert torch.equal(scales.view(-1), s.view(-1))
        nan = c & 0x7F == 0x7F
        assert bool(((codes.view_as(c) == c) | (nan & (codes.view_as(c) & 0x7F == 0x7F))).all())
        y = y.view(6, D)
        assert bool(y[[0, 2, 5]].isfinite().all())
    assert bool(ops.ln_modulate_save(x, zero, zero, EPS)[0][0, [1, 3, 4]].isnan().all())


# ------------------------------------------------------------------- LN backward

def ln_back_case(B, T, D, ckpt, res, seed=0):
    g, x, scale, shift = ln_inputs(B, T, D, seed)
    saved = ops.ln_modulate_save(x, scale, shift, EPS, checkpoint=ckpt)[1]
    dy = normal(g, B, T, D, std=0.1, mean=0.02)
    dres = normal(g, B, T, D, std=0.1) if res else None
    return x, scale, saved, dy, dres


def check_ln_back(got, x, scale, saved, dy, dres):
    B, T, D = dy.shape
    stats, codes, scales = saved
    v = x.double() if codes is None else ref.restore(codes, scales)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    want, err = ref.ln_backward(dy, v, stats, scale, dres, -(-B * T // min(B * T, sms)))
    for a, w, e, name in zip(got, want, err, ("dx", "dscale", "dshift")):
        ref.assert_near(a, w, e, name)


@pytest.mark.parametrize("B,T,D", LN_SHAPES + [(3, 1, 8), (16, 300, 16), (5, 77, 136), (1, 1, 8192), (2, 400, 2056),
                                               (4, 190, 32), (1, 152, 512), (2, 153, 520)])
@pytest.mark.parametrize("ckpt", [True, False])
@pytest.mark.parametrize("res", [True, False])
def test_ln_backward(B, T, D, ckpt, res):
    x, scale, saved, dy, dres = ln_back_case(B, T, D, ckpt, res)
    got = ops.ln_modulate_backward(dy, None if ckpt else x, scale, saved, dres=dres)
    check_ln_back(got, x, scale, saved, dy, dres)


def test_ln_backward_of_x_beside_a_checkpoint():
    """x given: the checkpoint is not looked at."""
    x, scale, saved, dy, _ = ln_back_case(1, 50, 264, True, False)
    a = ops.ln_modulate_backward(dy, x, scale, saved)
    b = ops.ln_modulate_backward(dy, x, scale, (saved[0], None, None))
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def shifted(t, by):
    """The same bytes `by` bytes behind a 16-byte boundary."""
    buf = torch.empty(t.numel() + 32, dtype=U8, device="cuda")
    v = buf[by:by + t.numel()]
    assert v.data_ptr() % 16 == by
    return v.copy_(t.reshape(-1))


@pytest.mark.parametrize("D", [64, 1160, 4096])
def test_checkpoints_at_their_least_alignment(D):
    """Codes on 8 bytes, scales on any."""
    x, scale, saved, dy, _ = ln_back_case(2, 50, D, True, False)
    kept = (saved[0], shifted(saved[1], 8).view(2, 50, D), shifted(saved[2], 5).view(2, 50, -1))
    for u, v in zip(ops.ln_modulate_backward(dy, None, scale, kept), ops.ln_modulate_backward(dy, None, scale, saved)):
        assert torch.equal(u, v)
    for dtype in TYPES:
        for S in (40, 9000):
            C = 64
            g, x, w, b, _, _ = gn_inputs(2, S, C, dtype, dtype, False)
            saved = ops.group_norm_save(x, 8, w, b, EPS, act="silu")[1]
            kept = (saved[0], shifted(saved[1], 8).view(2, S, C), shifted(saved[2], 5).view(2, S, C // 32))
            for u, v in zip(ops.group_norm_backward(x, None, 8, w, b, kept, act="silu")[:3],
                            ops.group_norm_backward(x, None, 8, w, b, saved, act="silu")[:3]):
                assert torch.equal(u, v)


@pytest.mark.parametrize("ckpt", [True, False])
def test_ln_backward_in_place_and_into_slices(ckpt):
    B, T, D = 3, 50, 1160
    x, scale, saved, dy, dres = ln_back_case(B, T, D, ckpt, True)
    kept = None if ckpt else x
    want = ops.ln_modulate_backward(dy, kept, scale, saved, dres=dres)
    buf, demb = guarded((B, 6 * D), BF16)
    a, b = dy.clone(), dres.clone()
    got = ops.ln_modulate_backward(a, kept, scale, saved, dres=dres, dx=a, dscale=demb[:, 2 * D:3 * D],
                                   dshift=demb[:, D:2 * D])
    assert got[0] is a and all(torch.equal(u, v) for u, v in zip(got, want))
    rest = [i for i in range(6 * D) if not D <= i < 3 * D]
    assert bool((demb[:, rest] == 77).all()) and untouched(buf)
    got = ops.ln_modulate_backward(dy, kept, scale, saved, dres=b, dx=b)
    assert got[0] is b and all(torch.equal(u, v) for u, v in zip(got, want))


def test_ln_outputs_stay_in_bounds():
    B, T, D = 2, 61, 1160
    x, scale, saved, dy, _ = ln_back_case(B, T, D, True, False)
    by, y = guarded((B, T, D), BF16)
    ops.ln_modulate_save(x, scale, scale, EPS, out=y)
    bx, dx = guarded((B, T, D), BF16)
    ops.ln_modulate_backward(dy, None, scale, saved, dx=dx)
    assert untouched(by) and untouched(bx)


def test_ln_rows_do_not_follow_the_batch():
    """y, the statistics and dx of a row are its own; a bad row spoils no other."""
    x, scale, saved, dy, _ = ln_back_case(1, 300, 1160, True, False)
    y, (stats, codes, scales) = ops.ln_modulate_save(x, scale, scale, EPS)
    dx = ops.ln_modulate_backward(dy, None, scale, saved)[0]
    for a, b in ((0, 1), (17, 40), (299, 300)):
        part = x[:, a:b].contiguous()
        y1, s1 = ops.ln_modulate_save(part, scale, scale, EPS)
        assert torch.equal(y1, y[:, a:b])
        assert all(torch.equal(u, v[:, a:b]) for u, v in zip(s1, (stats, codes, scales)))
        d1 = ops.ln_modulate_backward(dy[:, a:b].contiguous(), None, scale, s1)[0]
        assert torch.equal(d1, dx[:, a:b])
    bad = dy.clone()
    bad[0, 5, 3], bad[0, 90, 1000] = float("nan"), float("inf")
    d2 = ops.ln_modulate_backward(bad, None, scale, saved)[0]
    keep = [i for i in range(300) if i not in (5, 90)]
    assert torch.equal(d2[:, keep], dx[:, keep]) and bool(d2[0, [5, 90]].isnan().any(-1).all())


def test_ln_no_rows():
    D = 264
    e = lambda B, T: torch.empty((B, T, D), dtype=BF16, device="cuda")  # noqa: E731
    scale = torch.zeros((2, D), dtype=BF16, device="cuda")
    y, saved = ops.ln_modulate_save(e(2, 0), scale, scale, EPS)
    assert y.shape == (2, 0, D) and saved[0].shape == (2, 0, 2)
    dscale, dshift = (torch.full((2, D), 5.0, dtype=BF16, device="cuda") for _ in range(2))
    dx, *_ = ops.ln_modulate_backward(e(2, 0), None, scale, saved, dscale=dscale, dshift=dshift)
    assert dx.shape == (2, 0, D) and not dscale.any() and not dshift.any()
    assert ops.ln_modulate_backward(e(0, 4), e(0, 4), scale[:0], (torch.empty((0, 4, 2), device="cuda"), None,
                                                                  None))[1].shape == (0, D)


# -------------------------------------------------------------------- group norm

# (N, S, C, groups)
GN_SHAPES = [(1, 1, 8, 1), (2, 1, 64, 8), (1, 64, 1280, 32), (3, 77, 320, 32), (2, 5673, 40, 8), (1, 1000, 8, 8),
             (2, 300, 96, 3), (1, 2000, 2048, 32), (1, 70, 4096, 1), (2, 33, 2560, 2), (1, 40, 8192, 32),
             (5, 129, 160, 16), (1, 50000, 64, 32), (1, 300, 1920, 48), (1, 200001, 16, 2), (2, 4096, 512, 32),
             (1, 16384, 256, 32), (2, 17, 24, 1), (1, 5000, 4096, 1),
             (3, 9000, 96, 3)]


def gn_inputs(N, S, C, dtype, wtype, mod, seed=0, level=0.5):
    g = gen(seed)
    x = normal(g, N, S, C, mean=level, dtype=dtype)
    x *= torch.exp(0.3 * torch.randn(C, generator=g, device="cuda")).to(dtype)
    w, b = (normal(g, C, std=0.3, mean=m, dtype=wtype) for m in (1.0, 0.0))
    s = t = None
    if mod:
        emb = normal(g, N, 3 * C, std=0.3, dtype=dtype)
        s, t = emb[:, C:2 * C], emb[:, 2 * C:]
    return g, x, w, b, s, t


def check_gn(y, saved, x, groups, w, b, act, s, t, checkpoint, eps=EPS):
    want, st, ey, est = ref.gn_forward(x, groups, w, b, eps, act, s, t)
    ref.assert_near(ref.rows(y), want, ey, "y")
    if saved is None:
        return
    stats, codes, scales = saved
    ref.assert_near(stats, st, est, "stats")
    if checkpoint:
        c, k = ref.checkpoint(ref.rows(x))
        assert torch.equal(ref.rows(codes), c) and torch.equal(ref.rows(scales), k)


@pytest.mark.parametrize("N,S,C,groups", GN_SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_group_norm(N, S, C, groups, dtype):
    for k, (wtype, act, mod) in enumerate(((dtype, "silu", False), (FP32, None, True), (FP32, "silu", True))):
        g, x, w, b, s, t = gn_inputs(N, S, C, dtype, wtype, mod, k)
        y = ops.group_norm(x, groups, w, b, EPS, act=act, scale=s, shift=t)
        check_gn(y, None, x, groups, w, b, act, s, t, False)
        ckpt = C % 32 == 0 and k != 1
        y2, saved = ops.group_norm_save(x, groups, w, b, EPS, act=act, scale=s, shift=t, checkpoint=ckpt)
        check_gn(y2, saved, x, groups, w, b, act, s, t, ckpt)


@pytest.mark.parametrize("N,S,C,groups", GN_SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_group_norm_backward(N, S, C, groups, dtype):
    for k, (wtype, act, mod) in enumerate(((dtype, "silu", False), (FP32, None, True), (FP32, "silu", True))):
        g, x, w, b, s, t = gn_inputs(N, S, C, dtype, wtype, mod, k)
        ckpt = C % 32 == 0 and k != 1
        stats, codes, scales = saved = ops.group_norm_save(x, groups, w, b, EPS, act=act, scale=s, shift=t,
                                                           checkpoint=ckpt)[1]
        dy = normal(g, N, S, C, std=0.1, mean=0.02, dtype=dtype)
        got = ops.group_norm_backward(dy, None if ckpt else x, groups, w, b, saved, act=act, scale=s, shift=t)
        v = ref.restore(codes, scales) if ckpt else x.double()
        want, err = ref.gn_backward(dy, v, groups, w, b, stats, act, s, t)
        for a, u, e, name in zip(got, want, err, ("dx", "dweight", "dbias", "dscale", "dshift")):
            if u is None:
                assert a is None
            else:
                ref.assert_near(a, u, e, name)


@pytest.mark.parametrize("dtype", TYPES)
def test_group_norm_of_torch_images(dtype):
    """channels_last tensors of two and three dimensions; the same bits as their rows."""
    for shape in ((2, 64, 9, 7), (1, 96, 3, 5, 4), (3, 32, 1, 1)):
        g = gen(1)
        C = shape[1]
        fmt = torch.channels_last if len(shape) == 4 else torch.channels_last_3d
        x = normal(g, *shape, dtype=dtype).contiguous(memory_format=fmt)
        dy = normal(g, *shape, dtype=dtype).contiguous(memory_format=fmt)
        w, b = normal(g, C, mean=1.0, dtype=dtype), normal(g, C, dtype=dtype)
        y, saved = ops.group_norm_save(x, 8, w, b, EPS, act="silu")
        assert y.shape == x.shape and y.stride() == x.stride() and saved[1].stride() == x.stride()
        assert saved[2].shape == (shape[0], C // 32, *shape[2:])
        r = ref.rows(x).contiguous()
        y2, saved2 = ops.group_norm_save(r, 8, w, b, EPS, act="silu")
        assert torch.equal(ref.rows(y), y2) and torch.equal(ref.rows(saved[1]), saved2[1])
        assert torch.equal(ref.rows(saved[2]), saved2[2])
        check_gn(y, saved, x, 8, w, b, "silu", None, None, True)
        got = ops.group_norm_backward(dy, None, 8, w, b, saved, act="silu")
        want = ops.group_norm_backward(ref.rows(dy).contiguous(), None, 8, w, b, saved2, act="silu")
        assert got[0].stride() == x.stride() and torch.equal(ref.rows(got[0]), want[0])
        assert all(torch.equal(u, v) for u, v in zip(got[1:3], want[1:3]))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("S", [30, 4096, 70000])
def test_group_norm_without_parameters_and_in_place(dtype, S):
    N, C, groups = 2, 64, 16
    g, x, w, b, s, t = gn_inputs(N, S, C, dtype, dtype, True)
    y, saved = ops.group_norm_save(x, groups, None, None, EPS, checkpoint=False)
    check_gn(y, saved, x, groups, None, None, None, None, None, False)
    z = x.clone()
    assert ops.group_norm(z, groups, w, b, EPS, act="silu", scale=s, shift=t, out=z) is z
    assert torch.equal(z, ops.group_norm(x, groups, w, b, EPS, act="silu", scale=s, shift=t))
    dy = normal(g, N, S, C, dtype=dtype)
    want = ops.group_norm_backward(dy, x, groups, None, None, saved)
    assert want[1:] == (None,) * 4
    d = dy.clone()
    assert ops.group_norm_backward(d, x, groups, None, None, saved, dx=d)[0] is d and torch.equal(d, want[0])


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_group_norm_level_far_above_the_spread(dtype):
    """Squares of the values themselves would lose the variance."""
    for S in (200, 30000):
        g, x, w, b, _, _ = gn_inputs(1, S, 64, dtype, dtype, False, level=300.0)
        y, saved = ops.group_norm_save(x, 8, w, b, EPS, checkpoint=False)
        check_gn(y, saved, x, 8, w, b, None, None, None, False)
    x = torch.full((1, S, 64), 7.5, dtype=dtype, device="cuda")   # no spread at all
    y, saved = ops.group_norm_save(x, 8, None, None, EPS, checkpoint=False)
    assert not y.any() and bool((saved[0][..., 0] == 7.5).all())


@pytest.mark.parametrize("S", [50, 6000, 100000])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_group_norm_first_rows_far_off(S, dtype):
    """Pivots that say nothing of the rest: the first rows of an image, and its middle ones, 3000
    times the others' spread away."""
    for rows in (slice(0, 1), slice(0, 40), slice(S // 2, S // 2 + 1)):
        g, x, w, b, _, _ = gn_inputs(2, S, 512, dtype, dtype, False)
        x[1, rows] += 3000
        y, saved = ops.group_norm_save(x, 8, w, b, EPS, act="silu", checkpoint=False)
        check_gn(y, saved, x, 8, w, b, "silu", None, None, False)
        assert torch.equal(y[:1], ops.group_norm(x[:1], 8, w, b, EPS, act="silu"))


@pytest.mark.parametrize("S,C,groups", [(100, 320, 32), (5000, 64, 8), (6000, 512, 8), (70000, 32, 4)])
def test_images_do_not_follow_the_batch(S, C, groups):
    N = 5
    g, x, w, b, s, t = gn_inputs(N, S, C, BF16, BF16, True)
    dy = normal(g, N, S, C)
    kw = dict(act="silu")
    y, (stats, codes, scales) = ops.group_norm_save(x, groups, w, b, EPS, scale=s, shift=t, **kw)
    grads = ops.group_norm_backward(dy, x, groups, w, b, (stats, codes, scales), scale=s, shift=t, **kw)
    i = slice(3, 4)
    y1, saved = ops.group_norm_save(x[i], groups, w, b, EPS, scale=s[i], shift=t[i], **kw)
    assert torch.equal(y1, y[i]) and all(torch.equal(u, v[i]) for u, v in zip(saved, (stats, codes, scales)))
    g1 = ops.group_norm_backward(dy[i], x[i], groups, w, b, saved, scale=s[i], shift=t[i], **kw)
    assert torch.equal(g1[0], grads[0][i]) and torch.equal(g1[3], grads[3][i]) and torch.equal(g1[4], grads[4][i])
    # a bad value spoils its image's group, and no other
    per = C // groups
    x[2, S // 2, per * 3] = float("nan")
    y2 = ops.group_norm_save(x, groups, w, b, EPS, scale=s, shift=t, **kw)[0]
    bad = torch.zeros((N, S, C), dtype=torch.bool, device="cuda")
    bad[2, :, per * 3:per * 4] = True
    assert bool(y2[bad].isnan().all()) and torch.equal(y2[~bad], y[~bad])


@pytest.mark.parametrize("S,C,groups", [(100, 320, 32), (3000, 40, 40), (5000, 64, 8), (6000, 512, 8), (70000, 32, 4),
                                        (400000, 32, 4)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_an_infinity_spoils_its_group(S, C, groups, dtype):
    """Its group's outputs are not numbers, wherever the infinity lies, and the others are what they were."""
    _, x, w, b, _, _ = gn_inputs(2, S, C, dtype, dtype, False)
    y = ops.group_norm(x, groups, w, b, EPS)
    per = C // groups
    bad = torch.zeros((2, S, C), dtype=torch.bool, device="cuda")
    bad[1, :, per:2 * per] = True
    for row in (0, S // 2, S - 1):
        z = x.clone()
        z[1, row, 2 * per - 1] = float("-inf")
        y2, (stats, _, _) = ops.group_norm_save(z, groups, w, b, EPS, checkpoint=False)
        assert bool(y2[bad].isnan().all()) and torch.equal(y2[~bad], y[~bad]), row
        assert bool(stats[1, 1, 1].isnan()), row


def test_group_norm_no_positions():
    C = 40
    w = torch.ones(C, dtype=BF16, device="cuda")
    s = torch.ones((2, C), dtype=BF16, device="cuda")
    for N, S in ((2, 0), (1, 0), (0, 5)):
        x = torch.empty((N, S, C), dtype=BF16, device="cuda")
        y, saved = ops.group_norm_save(x, 5, w, w, EPS, scale=s[:N], shift=s[:N], checkpoint=False)
        assert y.shape == x.shape
        dx, *grads = ops.group_norm_backward(x, x, 5, w, w, saved, scale=s[:N], shift=s[:N])
        assert dx.shape == x.shape and [tuple(v.shape) for v in grads] == [(C,), (C,), (N, C), (N, C)]
        assert not any(v.any() for v in grads)


def test_group_norm_outputs_stay_in_bounds():
    for N, S, C, groups in ((2, 77, 320, 32), (1, 20001, 64, 8)):
        g, x, w, b, s, t = gn_inputs(N, S, C, BF16, BF16, False)
        by, y = guarded((N, S, C), BF16)
        bx, dx = guarded((N, S, C), BF16)
        _, saved = ops.group_norm_save(x, groups, w, b, EPS, act="silu", out=y)
        ops.group_norm_backward(normal(g, N, S, C), x, groups, w, b, saved, act="silu", dx=dx)
        assert untouched(by) and untouched(bx)


@pytest.mark.parametrize("S", [50, 20000])
def test_gradient_agrees_with_differences(S):
    """The fp32 group norm's gradients against differences of its own outputs, along directions
    that change the loss by far more than its rounding."""
    N, C, groups = 2, 64, 8
    g, x, w, b, s, t = gn_inputs(N, S, C, FP32, FP32, True)
    s, t = s.contiguous(), t.contiguous()
    dy = normal(g, N, S, C, mean=0.3, dtype=FP32)
    saved = ops.group_norm_save(x, groups, w, b, EPS, act="silu", scale=s, shift=t, checkpoint=False)[1]
    grads = ops.group_norm_backward(dy, x, groups, w, b, saved, act="silu", scale=s, shift=t)
    args = (x, w, b, s, t)
    for i, grad in enumerate(grads):
        d = grad / grad.norm()
        h = 0.05 * math.sqrt(N * S * C) if i == 0 else 0.05

        def at(k):
            a = [v + k * h * d if j == i else v for j, v in enumerate(args)]
            y = ops.group_norm(a[0], groups, a[1], a[2], EPS, act="silu", scale=a[3], shift=a[4])
            return float((y.double() * dy.double()).sum())

        # the fourth-order difference: its own error falls with h^4
        slope = (8 * (at(1) - at(-1)) - (at(2) - at(-2))) / (12 * h)
        assert abs(slope - float(grad.double().norm())) < 2e-3 * abs(slope), i


def test_ln_offsets_past_2_31_elements():
    """The last rows of more than 2^31 elements, against those rows alone."""
    T, D, n = (1 << 31) // 8192 + 40, 8192, 60
    g = gen(0)
    x = torch.empty((1, T, D), dtype=BF16, device="cuda").normal_(generator=g)
    scale = normal(g, D, std=0.3)
    y, saved = ops.ln_modulate_save(x, scale, scale, EPS)
    dx = ops.ln_modulate_backward(y, None, scale, saved, dres=x)[0]
    part = x[:, -n:].contiguous()
    y1, saved1 = ops.ln_modulate_save(part, scale, scale, EPS)
    assert torch.equal(y[:, -n:], y1) and all(torch.equal(u[:, -n:], v) for u, v in zip(saved, saved1))
    assert torch.equal(dx[:, -n:], ops.ln_modulate_backward(y1, None, scale, saved1, dres=part)[0])


@pytest.mark.parametrize("N,S,C,groups", [(2, 1 << 20, 1040, 8), (70000, 16, 2048, 32)])
def test_gn_offsets_past_2_31_elements(N, S, C, groups):
    """The last image of more than 2^31 elements, against that image alone."""
    g = gen(0)
    x = torch.empty((N, S, C), dtype=BF16, device="cuda").normal_(generator=g)
    w, b = normal(g, C, mean=1.0), normal(g, C)
    kw = dict(act="silu")
    y, saved = ops.group_norm_save(x, groups, w, b, EPS, checkpoint=C % 32 == 0, **kw)
    kept = None if C % 32 == 0 else x
    dx, dw, db, *_ = ops.group_norm_backward(y, kept, groups, w, b, saved, **kw)
    i = slice(N - 1, N)
    y1, saved1 = ops.group_norm_save(x[i], groups, w, b, EPS, checkpoint=C % 32 == 0, **kw)
    assert torch.equal(y[i], y1)
    assert all(u is None and v is None or torch.equal(u[i], v) for u, v in zip(saved, saved1))
    dx1 = ops.group_norm_backward(y1, None if kept is None else x[i], groups, w, b, saved1, **kw)[0]
    assert torch.equal(dx[i], dx1)
    # dbias: sums of dy * silu'(z); of its size, and the same every time
    again = ops.group_norm_backward(y, kept, groups, w, b, saved, **kw)
    assert bool(dw.isfinite().all()) and torch.equal(again[1], dw) and torch.equal(again[2], db)


# ------------------------------------------------------- together, streams, graphs

class GroupNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, b, groups):
        y, saved = ops.group_norm_save(x, groups, w, b, EPS, act="silu")
        ctx.save_for_backward(w, b, *saved)
        ctx.groups = groups
        return y

    @staticmethod
    def backward(ctx, dy):
        w, b, *saved = ctx.saved_tensors
        return *ops.group_norm_backward(dy.contiguous(), None, ctx.groups, w, b, saved, act="silu")[:3], None


class Modulate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, emb):
        D = x.shape[-1]
        y, saved = ops.ln_modulate_save(x, emb[:, :D], emb[:, D:], EPS)
        ctx.save_for_backward(emb, *saved)
        return y

    @staticmethod
    def backward(ctx, dy):
        emb, *saved = ctx.saved_tensors
        D = dy.shape[-1]
        demb = torch.empty_like(emb)
        dx, _, _ = ops.ln_modulate_backward(dy.contiguous(), None, emb[:, :D], saved, dscale=demb[:, :D],
                                            dshift=demb[:, D:])
        return dx, demb


def test_a_training_step_through_both():
    """Group norm, a projection, LayerNorm + modulate: gradients of all parameters against autograd
    in 64 bits.  The checkpoints' rounding (at most 1/16 of a value) is in them: a loose bound, on
    norms."""
    N, S, C, D = 2, 256, 64, 128
    g = gen(0)
    x = normal(g, N, S, C)
    leaves = [normal(g, C, std=0.2, mean=1.0), normal(g, C, std=0.2), normal(g, C, D, std=C ** -0.5),
              normal(g, N, 2 * D, std=0.2)]
    seed = normal(g, N, S, D, mean=0.3)
    a = [t.clone().requires_grad_() for t in leaves]
    y = Modulate.apply(GroupNorm.apply(x, a[0], a[1], 8) @ a[2], a[3])
    y.backward(seed)
    d = [t.double().requires_grad_() for t in leaves]
    v = x.double().unflatten(2, (8, -1))
    n = ((v - v.mean((1, 3), keepdim=True)) / (v.var((1, 3), keepdim=True, correction=0) + EPS).sqrt()).flatten(2)
    h = torch.nn.functional.silu(n * d[0] + d[1]) @ d[2]
    n = (h - h.mean(-1, keepdim=True)) / (h.var(-1, keepdim=True, correction=0) + EPS).sqrt()
    z = n * (1 + d[3][:, None, :D]) + d[3][:, None, D:]
    z.backward(seed.double())
    assert float((y.detach().double() - z.detach()).norm() / z.detach().norm()) < 0.02
    for u, w in zip(a, d):
        assert float((u.grad.double() - w.grad).norm() / w.grad.norm()) < 0.06


def all_operators(k=0):
    """A call of each operator, as functions of nothing, with their outputs' expected values."""
    x, scale, saved, dy, dres = ln_back_case(2, 333, 1160, True, True, seed=k)
    g, xi, w, b, s, t = gn_inputs(3, 1000, 320, BF16, FP32, True, seed=k)
    di = normal(g, 3, 1000, 320)
    kept = ops.group_norm_save(xi, 32, w, b, EPS, act="silu", scale=s, shift=t)[1]
    big = normal(g, 1, 60000, 64)
    keep_big = ops.group_norm_save(big, 16, None, None, EPS, checkpoint=False)[1]
    return [lambda: ops.ln_modulate_save(x, scale, scale, EPS)[0],
            lambda: ops.ln_modulate_backward(dy, None, scale, saved, dres=dres),
            lambda: ops.group_norm(xi, 32, w, b, EPS, act="silu", scale=s, shift=t),
            lambda: ops.group_norm_backward(di, None, 32, w, b, kept, act="silu", scale=s, shift=t),
            lambda: ops.group_norm(big, 16, None, None, EPS),
            lambda: ops.group_norm_backward(big, big, 16, None, None, keep_big)[0]]


def flat(v):
    return [v] if isinstance(v, torch.Tensor) else [t for t in v if t is not None]


def test_same_bits_every_time_and_on_other_streams():
    calls = all_operators()
    want = [flat(f()) for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append([flat(f()) for f in calls])
    torch.cuda.synchronize()
    for run in got:
        for a, b in zip(run, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_captured_and_replayed():
    """All of them in one graph, replayed on new inputs in the same buffers; two graphs alive."""
    graphs = []
    for k in range(2):
        calls = all_operators(k)
        want = [[v.clone() for v in flat(f())] for f in calls]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = [flat(f()) for f in calls]
        graphs.append((graph, outs, want, calls))  # the calls hold the inputs
    for _ in range(3):
        for _, outs, _, _ in graphs:
            for run in outs:
                for v in run:
                    v.zero_()
        for graph, *_ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, outs, want, _ in graphs:
            for a, b in zip(outs, want):
                assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_replayed_on_new_inputs():
    x, scale, saved, dy, _ = ln_back_case(1, 100, 520, True, False)
    f = lambda: ops.ln_modulate_backward(dy, None, scale, saved)  # noqa: E731
    f()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = f()
    dy.copy_(normal(gen(9), 1, 100, 520))
    graph.replay()
    assert all(torch.equal(u, v) for u, v in zip(outs, f()))


def test_binding_refuses():
    x, scale, saved, dy, _ = ln_back_case(2, 10, 64, True, False)
    with pytest.raises(ValueError):
        ops.ln_modulate_backward(dy, None, scale, (saved[0], None, None))
    with pytest.raises(TypeError):
        ops.ln_modulate_backward(dy, None, scale, saved[0])
    with pytest.raises(TypeError):
        ops.ln_modulate_backward(dy, None, scale, (saved[0].double(), *saved[1:]))
    with pytest.raises(ValueError):
        ops.ln_modulate_backward(dy, None, scale, (saved[0], saved[1][:, :5], saved[2]))
    with pytest.raises(ValueError):
        ops.ln_modulate_backward(dy, x[:, :5].contiguous(), scale, saved)
    with pytest.raises(ValueError):
        ops.ln_modulate_backward(dy, x, scale, saved, dscale=torch.empty_like(scale))
    with pytest.raises(ops.DanError):
        ops.ln_modulate_backward(dy, x, scale, saved, dx=x)           # x is not to be overwritten
    with pytest.raises(ValueError):
        ops.ln_modulate_save(x, scale, scale[:1], EPS)
    img = normal(gen(0), 2, 64, 5, 6)
    w = normal(gen(0), 64)
    with pytest.raises(ValueError):
        ops.group_norm(img, 8, w, w, EPS)                              # channels first in memory
    img = img.contiguous(memory_format=torch.channels_last)
    with pytest.raises(ValueError):
        ops.group_norm(img, 8, w, None, EPS)
    with pytest.raises(ValueError):
        ops.group_norm(img, 8, w, w, EPS, scale=torch.zeros(2, 64, dtype=BF16, device="cuda"))
    with pytest.raises(ValueError):
        ops.group_norm(img, 8, w, w, EPS, act="gelu")
    with pytest.raises(TypeError):
        ops.group_norm(img, 8, w.half(), w.half(), EPS)
    with pytest.raises(TypeError):
        ops.group_norm(img.double(), 8, w, w, EPS)
    with pytest.raises(ops.DanError):
        ops.group_norm(img, 7, w, w, EPS)
    with pytest.raises(ops.DanError):
        ops.group_norm(img, 0, w, w, EPS)
    with pytest.raises(ops.DanError):
        ops.group_norm(img, 8, w, w, -1.0)
    with pytest.raises(ValueError):
        ops.group_norm_save(normal(gen(0), 1, 4, 40), 5, None, None, EPS)   # no whole blocks
    _, kept = ops.group_norm_save(img, 8, w, w, EPS)
    with pytest.raises(ValueError):
        ops.group_norm_backward(img, None, 8, w, w, (kept[0], None, None))
    with pytest.raises(ValueError):
        ops.group_norm_backward(img, None, 4, w, w, kept)              # other groups
    with pytest.raises(ValueError):
        ops.group_norm_backward(img, None, 8, w, w, (kept[0], kept[1].contiguous(), kept[2]))
    with pytest.raises(ops.DanError):
        ops.group_norm_backward(torch.ones_like(img), img, 8, w, w, kept, dx=img)   # x is not to be overwritten
