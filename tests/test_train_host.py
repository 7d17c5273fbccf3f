"""Host-side tests of the training operators (no GPU): the library exports what
include/dan_train.h declares, every dan_can_use_* returns the documented status (fake addresses
that validation never dereferences), the binding refuses what is not a CUDA tensor, and the tests'
64-bit references agree with differences of the forward formulas."""
import pytest
import torch

import _train as ref
from dit_adaln_norm_gb300 import build as dan_build
from dit_adaln_norm_gb300 import ops

OK, EINVAL, EUNSUP, EALIGN, EALIAS, ECUDA = range(6)
GB = 1 << 30
EPS = 1e-6
(X, Y, SC, SH, ST, CO, BS, DY, DX, DR, G1, G2, WK, W, B_) = (0x100000000 + i * 64 * GB for i in range(15))
BF, HF, F32 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    dan_build.build()
    return ops.load()


def test_exports_every_declared_symbol(lib):
    names = ops.declared_symbols(ops.TRAIN_HEADER)
    assert len(names) == 11
    for n in names:
        assert hasattr(lib, n), n
        assert n in ops._SIGS, n


def test_save_validation(lib):
    def f(x=X, sc=SC, sh=SH, vs=4096, y=Y, st=ST, co=CO, bs=BS, B=1, T=4216, D=4096, eps=EPS):
        return lib.dan_can_use_ln_modulate_save(x, sc, sh, vs, y, st, co, bs, B, T, D, eps)

    assert f() == OK and f(co=None, bs=None) == OK and f(y=X) == OK
    for D in (8, 24, 1160, 8192):
        assert f(D=D, vs=D) == OK, D
    for D in (0, 4, 12, 8200):
        assert f(D=D, vs=max(D, 8)) == EUNSUP, D
    assert f(co=None) == EINVAL and f(bs=None) == EINVAL and f(st=None) == EINVAL and f(x=None) == EINVAL
    assert f(B=-1) == EINVAL and f(T=-1) == EINVAL and f(T=1 << 40) == EINVAL
    for eps in (-1e-6, float("nan"), float("inf")):
        assert f(eps=eps) == EINVAL
    assert f(B=2, vs=4088) == EINVAL and f(B=2, vs=4100) == EALIGN and f(B=2, vs=6 * 4096) == OK
    assert f(x=X + 8) == EALIGN and f(st=ST + 4) == EALIGN and f(co=CO + 4) == EALIGN
    assert f(st=ST + 8) == OK and f(co=CO + 8) == OK and f(bs=BS + 1) == OK
    for over in (dict(y=X + 16), dict(st=X), dict(co=X), dict(bs=SC), dict(co=Y), dict(bs=CO), dict(st=Y)):
        assert f(**over) == EALIAS, over
    assert f(T=0, x=None, y=None, st=None) == OK and f(B=0) == OK


def ln_back(lib, dy=DY, x=None, co=CO, bs=BS, st=ST, sc=SC, vs=4096, dr=None, dx=DX, g1=G1, g2=G2, gs=4096, B=1,
            T=4216, D=4096, wk=WK, size=None):
    if size is None:
        size = lib.dan_ln_modulate_backward_workspace(B, T, D)
    return lib.dan_can_use_ln_modulate_backward(dy, x, co, bs, st, sc, vs, dr, dx, g1, g2, gs, B, T, D, wk, size)


def test_ln_backward_validation(lib):
    f = lambda **k: ln_back(lib, **k)  # noqa: E731
    assert f() == OK and f(x=X, co=None, bs=None) == OK and f(dr=DR) == OK
    assert f(x=X, co=1, bs=3) == OK                          # not looked at beside x
    assert f(co=None) == EINVAL and f(bs=None) == EINVAL and f(st=None) == EINVAL and f(sc=None) == EINVAL
    assert f(dx=DY) == OK and f(dx=DR, dr=DR) == OK          # in place
    assert f(dx=DY + 16) == EALIAS and f(x=X, dx=X) == EALIAS and f(dx=CO) == EALIAS and f(dx=ST) == EALIAS
    assert f(g1=DX) == EALIAS and f(g2=DY) == EALIAS and f(g2=G1) == EALIAS and f(wk=G2) == EALIAS
    # the two gradients as slices of one [B, 6 * D] buffer, side by side in either order
    assert f(B=2, gs=6 * 4096, g2=G1 + 4096 * 2) == OK and f(B=2, gs=6 * 4096, g1=G2 + 4096 * 2) == OK
    assert f(B=2, gs=6 * 4096, g2=G1 + 4096 * 10) == OK and f(B=2, gs=6 * 4096, g2=G1 + 4088 * 2) == EALIAS
    assert f(B=2, gs=6 * 4096, g2=G1 + (5 * 4096 + 8) * 2) == EALIAS
    assert f(B=2, gs=4088) == EINVAL and f(B=2, gs=4100) == EALIGN and f(B=2, vs=4100) == EALIGN
    for name, base in (("dy", DY), ("dx", DX), ("g1", G1), ("g2", G2), ("sc", SC), ("wk", WK)):
        assert f(**{name: base + 8}) == EALIGN, name
    assert f(co=CO + 4) == EALIGN and f(st=ST + 4) == EALIGN and f(bs=BS + 1) == OK
    need = lib.dan_ln_modulate_backward_workspace(1, 4216, 4096)
    assert need > 0 and f(size=need - 1) == EINVAL and f(wk=None) == EINVAL
    assert f(D=12) == EUNSUP and f(D=8200) == EUNSUP and f(T=-1, size=0) == EINVAL
    assert f(B=(1 << 27) + 1, T=0, D=8, vs=8, gs=8) == EUNSUP
    assert f(B=0, dy=None, dx=None, g1=None, wk=None) == OK
    # rows of no tokens: the gradients are still written
    assert f(T=0, dy=None, dx=None, co=None, bs=None, st=None, sc=None, wk=None) == OK
    assert f(T=0, g1=None) == EINVAL
    assert lib.dan_ln_modulate_backward_workspace(1, 1, 12) == 0


def gn(lib, x=X, ty=BF, w=W, b=B_, pt=BF, sc=None, sh=None, vs=512, act=1, y=Y, st=None, co=None, bs=None, N=1,
       S=4096, C=512, G=32, eps=EPS, wk=WK, size=None):
    if size is None:
        size = lib.dan_group_norm_workspace(N, S, C, G, ty, 1 if co else 0)
    return lib.dan_can_use_group_norm(x, ty, w, b, pt, sc, sh, vs, act, y, st, co, bs, N, S, C, G, eps, wk, size)


def test_slabs_of_the_widest_images_fit_a_grid(lib):
    """65536 slabs of 64 bytes a row are more than a grid has in y: such images go in passes, which
    need a workspace; one step narrower, and with slabs of 128 bytes, they are slabs."""
    forward, backward = lib.dan_group_norm_workspace, lib.dan_group_norm_backward_workspace
    C = 1 << 20
    for S in (5200, 8192):
        assert forward(1, S, C, C // 4, F32, 0) > 0 and forward(1, S, C - 16, C // 4 - 4, F32, 0) == 0
    assert forward(1, 4096, C, C // 4, F32, 0) == 0
    for S in (2600, 4096):
        assert backward(1, S, C, C // 4, F32, 0) > 0 and backward(1, S, C - 16, C // 4 - 4, F32, 0) == 0


def test_group_norm_validation(lib):
    f = lambda **k: gn(lib, **k)  # noqa: E731
    assert f() == OK and f(w=None, b=None) == OK and f(sc=SC, sh=SH) == OK and f(st=ST, co=CO, bs=BS) == OK
    for ty in (BF, HF, F32):
        assert f(ty=ty, pt=ty) == OK and f(ty=ty, pt=F32) == OK
    assert f(ty=BF, pt=HF) == EINVAL and f(ty=F32, pt=BF) == EINVAL and f(ty=3) == EINVAL and f(ty=-1) == EINVAL
    assert f(act=2) == EINVAL and f(act=0) == OK and f(w=None) == EINVAL and f(sc=SC) == EINVAL
    assert f(co=CO, bs=BS) == EINVAL and f(st=ST, co=CO) == EINVAL      # codes need stats and scales
    for C, G in ((320, 32), (8, 1), (8, 8), (40, 5), (4096, 1), (16384, 4), (1 << 20, 1 << 10)):
        assert f(C=C, G=G) == OK, (C, G)
    assert f(C=12, G=1) == EUNSUP and f(C=320, G=33) == EUNSUP and f(C=320, G=0) == EINVAL
    assert f(C=8192, G=1) == EUNSUP and f(C=8 * 1025, G=8) == EUNSUP and f(C=(1 << 20) + 8, G=8) == EUNSUP
    assert f(C=40, G=5, st=ST, co=CO, bs=BS) == EUNSUP                  # blocks of 32 channels
    assert f(S=1 << 31) == EUNSUP and f(N=1 << 28, S=1) == EUNSUP and f(N=1 << 27, S=1) == EUNSUP and f(N=1 << 20, S=1 << 20) == EINVAL
    assert f(y=X) == OK and f(y=X + 16) == EALIAS and f(st=X) == EALIAS and f(S=1 << 20, wk=Y) == EALIAS
    assert f(S=1 << 20, wk=X) == EALIAS and f(st=ST, co=Y, bs=BS) == EALIAS and f(y=W) == EALIAS
    assert f(x=X + 8) == EALIGN and f(w=W + 2) == EALIGN and f(st=ST + 4) == EALIGN
    assert f(N=2, sc=SC, sh=SH, vs=516) == EALIGN and f(N=2, sc=SC, sh=SH, vs=504) == EINVAL
    assert f(N=2, ty=F32, pt=F32, sc=SC, sh=SH, vs=516) == OK
    assert f(eps=-1.0) == EINVAL and f(eps=float("nan")) == EINVAL
    need = lib.dan_group_norm_workspace(1, 1 << 20, 512, 32, BF, 0)
    assert need > 0 and f(S=1 << 20, size=need - 1) == EINVAL and f(S=1 << 20, wk=None) == EINVAL
    assert f(S=0, x=None, y=None) == OK and f(N=0, x=None) == OK
    assert lib.dan_group_norm_workspace(1, 16, 12, 1, BF, 0) == 0


def gn_back(lib, dy=DY, x=X, ty=BF, co=None, bs=None, st=ST, w=W, b=B_, pt=BF, sc=None, sh=None, vs=512, act=1,
            dx=DX, dw=Y, db=Y + GB, dsc=None, dsh=None, gs=512, N=1, S=4096, C=512, G=32, wk=WK, size=None):
    if size is None:
        size = lib.dan_group_norm_backward_workspace(N, S, C, G, ty, 0 if x else 1)
    return lib.dan_can_use_group_norm_backward(dy, x, ty, co, bs, st, w, b, pt, sc, sh, vs, act, dx, dw, db, dsc,
                                               dsh, gs, N, S, C, G, wk, size)


def test_group_norm_backward_validation(lib):
    f = lambda **k: gn_back(lib, **k)  # noqa: E731
    mod = dict(sc=SC, sh=SH, dsc=G1, dsh=G2)
    assert f() == OK and f(**mod) == OK and f(x=None, co=CO, bs=BS) == OK and f(dx=DY) == OK
    assert f(w=None, b=None, dw=None, db=None) == OK
    # each gradient with its parameter
    assert f(dw=None) == EINVAL and f(w=None, b=None) == EINVAL and f(sc=SC, sh=SH) == EINVAL
    assert f(dsc=G1, dsh=G2) == EINVAL and f(**{**mod, "dsh": None}) == EINVAL
    assert f(x=None) == EINVAL and f(x=None, co=CO) == EINVAL and f(st=None) == EINVAL
    assert f(x=None, co=CO, bs=BS, C=40, G=5) == EUNSUP and f(C=40, G=5) == OK
    assert f(dx=X) == EALIAS and f(dx=DY + 16) == EALIAS and f(dw=W) == EALIAS and f(db=Y) == EALIAS
    assert f(**{**mod, "dsh": G1}) == EALIAS and f(**{**mod, "dsc": DX}) == EALIAS and f(N=2, wk=DX) == EALIAS
    assert f(**mod, N=2, gs=1024) == OK and f(**{**mod, "dsh": G1 + 1024}, N=2, gs=1024) == OK
    assert f(**{**mod, "dsh": G1 + 512}, N=2, gs=1024) == EALIAS
    assert f(**mod, N=2, gs=516) == EALIGN and f(**mod, N=2, gs=504) == EINVAL
    assert f(dy=DY + 8) == EALIGN and f(x=None, co=CO + 4, bs=BS) == EALIGN
    for n, s in ((1, 1 << 20), (2, 4096)):
        need = lib.dan_group_norm_backward_workspace(n, s, 512, 32, BF, 0)
        assert need > 0 and f(N=n, S=s, db=Y + 8 * GB) == OK
        assert f(N=n, S=s, size=need - 1) == EINVAL and f(N=n, S=s, wk=None) == EINVAL
    assert f(S=0, dy=None, x=16, dx=None, st=None) == OK and f(S=0, dw=None) == EINVAL


def test_cuts_do_not_follow_the_batch(lib):
    """What a call asks for grows with the images, so that each is cut up alike."""
    for size, k in ((lib.dan_group_norm_workspace, 0), (lib.dan_group_norm_backward_workspace, 0)):
        for S, C, G in ((1 << 16, 128, 32), (77, 320, 32), (1, 8, 8)):
            assert size(14, S, C, G, BF, k) == 2 * size(7, S, C, G, BF, k)


def test_binding_refuses_without_cuda_tensors():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    saved = (z(1, 2, 2, dt=torch.float32), None, None)
    with pytest.raises(TypeError):
        ops.ln_modulate_save(z(1, 2, 64), z(64), z(64), EPS)
    with pytest.raises(TypeError):
        ops.ln_modulate_backward(z(1, 2, 64), z(1, 2, 64), z(64), saved)
    with pytest.raises(TypeError):
        ops.group_norm(z(1, 4, 32), 4, z(32), z(32), EPS)
    with pytest.raises(TypeError):
        ops.group_norm_save(z(1, 4, 32), 4, None, None, EPS)
    with pytest.raises(TypeError):
        ops.group_norm_backward(z(1, 4, 32), z(1, 4, 32), 4, None, None, saved)


def directional(f, args, grads, seed, h=1e-5):
    """The derivative of f along a random direction of its arguments, and by the gradients."""
    g = torch.Generator().manual_seed(seed)
    ds = [None if a is None else torch.randn(a.shape, generator=g, dtype=torch.float64) for a in args]
    at = lambda t: f(*(a if d is None else a + t * d for a, d in zip(args, ds)))  # noqa: E731
    return float(at(h) - at(-h)) / (2 * h), sum(float((d * k).sum()) for d, k in zip(ds, grads) if d is not None)


def test_ln_reference_agrees_with_differences():
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, scale, shift, dy = r(2, 5, 24) + 0.5, r(2, 24), r(2, 24), r(2, 5, 24)
    f = lambda x, s, t: (ref.ln_forward(x, s, t, 1e-3)[0] * dy).sum()  # noqa: E731
    stats = ref.ln_forward(x, scale, shift, 1e-3)[1]
    grads, _ = ref.ln_backward(dy, x, stats, scale, None, 0)
    a, b = directional(f, (x, scale, shift), grads, 1)
    assert abs(a - b) < 1e-7 * (1 + abs(b))


@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("mod", [False, True])
def test_gn_reference_agrees_with_differences(act, mod):
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, b, dy = r(2, 6, 24) + 0.5, r(24), r(24), r(2, 6, 24)
    s, t = (r(2, 24), r(2, 24)) if mod else (None, None)
    f = lambda x, w, b, s, t: (ref.gn_forward(x, 3, w, b, 1e-3, act, s, t)[0] * dy).sum()  # noqa: E731
    stats = ref.gn_forward(x, 3, w, b, 1e-3, act, s, t)[1]
    grads, _ = ref.gn_backward(dy, x, 3, w, b, stats, act, s, t)
    a, b = directional(f, (x, w, b, s, t), grads, 1)
    assert abs(a - b) < 1e-7 * (1 + abs(b))


def test_checkpoint_reference():
    """The reference against the format: codes within half a step, and the scale the least one."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn(64, 96, generator=g) * torch.exp2(torch.randint(-130, 120, (64, 1), generator=g).float())
    x[0], x[1, :32], x[2, 0], x[3, 5], x[4, :32] = 0, 448, float("inf"), float("nan"), 449
    codes, scales = ref.checkpoint(x)
    v, k = ref.restore(codes, scales), scales.to(torch.int64) - 127
    fine = x.isfinite()
    step = torch.maximum(x.double().abs() / 16, ref.power(k - 10).repeat_interleave(32, 1))
    assert bool(((v - x.double()).abs() <= step)[fine & ~x.isinf().any(1, keepdim=True)].all())
    assert int(k[0, 0]) == -126 and int(k[1, 0]) == 0 and int(k[4, 0]) == 1 and int(k[2, 0]) == 120
    assert int(codes[3, 5]) & 0x7F == 0x7F
    top = torch.where(fine, x.double().abs(), 0.0).view(64, 3, 32).amax(-1)
    least = (top > 448 * ref.power((k - 1).clamp(min=-127))) | (k == -126) | (k == 120)
    assert bool((top <= 448 * ref.power(k)).all()) and bool(least.all())
