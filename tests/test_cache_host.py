"""Host-side tests of the paged-cache operators (no GPU): exported symbols,
the documented status of every refused call, workspace sizes, and the checks
of the Python binding.  Pointers are fake addresses that validation only
compares."""
import pytest
import torch

from dit_adaln_norm_gb300 import build as dan_build
from dit_adaln_norm_gb300 import ops

OK, EINVAL, EUNSUP, EALIGN, EALIAS, ECUDA = range(6)
GB = 1 << 30
Q, K, V, WQ, WK, ROPE, POS, SLOT, QO, KC, VC, TAB, QS, KL, OUT, LSE, WORK = (
    0x1000000000 + i * 64 * GB for i in range(17))


@pytest.fixture(scope="module")
def lib():
    dan_build.build()
    return ops.load()


def test_exports_every_declared_symbol(lib):
    names = ops.declared_symbols(ops.CACHE_HEADER)
    assert names == sorted(["dan_qk_norm_rope_cache", "dan_can_use_qk_norm_rope_cache",
                            "dan_window_attention", "dan_can_use_window_attention",
                            "dan_window_attention_workspace"])
    for n in names:
        assert hasattr(lib, n), n


def rope(lib, q=Q, k=K, v=V, N=100, qs=6144, ks=6144, H=32, Hkv=8, hd=128, wq=WQ, wk=WK, r=ROPE,
         P=8192, pos=POS, slot=SLOT, eps=1e-6, qo=QO, os=4096, kc=KC, vc=VC, pages=50, page=64):
    return lib.dan_can_use_qk_norm_rope_cache(q, k, v, N, qs, ks, H, Hkv, hd, wq, wk, r, P, pos, slot,
                                              eps, 1, qo, os, kc, vc, pages, page)


def test_rope_cache_validation(lib):
    f = lambda **k: rope(lib, **k)  # noqa: E731
    assert f() == OK
    for page in (16, 32, 64, 128):
        assert f(page=page) == OK
    for page in (0, 1, 8, 48, 256):
        assert f(page=page) == EUNSUP
    assert f(hd=64) == OK and f(hd=96) == EUNSUP and f(hd=256) == EUNSUP
    assert f(H=30) == EINVAL                      # not a multiple of kv_heads
    assert f(Hkv=0) == EINVAL and f(H=0) == EINVAL and f(pages=0) == EINVAL
    assert f(H=2048, Hkv=2048, qs=1 << 20, ks=1 << 20, os=1 << 20) == EUNSUP
    assert f(N=-1) == EINVAL and f(P=0) == EINVAL and f(P=1 << 31) == EINVAL
    assert f(eps=-1.0) == EINVAL and f(eps=float("nan")) == EINVAL and f(eps=float("inf")) == EINVAL
    assert f(qs=4088) == EINVAL and f(ks=1016) == EINVAL and f(os=4088) == EINVAL
    assert f(qs=6148) == EALIGN and f(ks=6148) == EALIGN and f(os=4100) == EALIGN
    for name in ("q", "k", "v", "wq", "wk", "r", "qo", "kc", "vc"):
        assert f(**{name: None}) == EINVAL, name
        base = dict(q=Q, k=K, v=V, wq=WQ, wk=WK, r=ROPE, qo=QO, kc=KC, vc=VC)[name]
        assert f(**{name: base + 8}) == EALIGN, name
    assert f(pos=None) == EINVAL and f(slot=None) == EINVAL
    assert f(pos=POS + 4) == OK and f(pos=POS + 2) == EALIGN and f(slot=SLOT + 1) == EALIGN
    assert f(N=0, q=None, k=None, v=None, pos=None, slot=None, qo=None) == OK
    # caches beyond 2^31 - 256 token rows of one head are refused, below are taken
    assert f(pages=(1 << 31) // (64 * 8)) == EUNSUP
    assert f(pages=(1 << 31) // (64 * 8) - 1, kc=1 << 45, vc=1 << 46) == OK
    assert f(N=1 << 40) == EINVAL


def test_rope_cache_aliases(lib):
    f = lambda **k: rope(lib, **k)  # noqa: E731
    assert f(kc=VC) == EALIAS and f(qo=KC) == EALIAS and f(qo=K) == EALIAS
    assert f(qo=Q + 64) == EALIAS                 # partial overlap
    assert f(qo=Q, os=6144) == OK                 # in place
    assert f(qo=Q) == EALIAS                      # same start, another stride
    # one packed projection, q rotated in place beside k and v
    assert f(qo=Q, os=6144, k=Q + 4096 * 2, v=Q + 5120 * 2) == OK
    assert f(qo=Q, os=6144, k=Q + 4088 * 2, v=Q + 5120 * 2) == EALIAS  # k starts inside q's row
    assert f(qo=Q, os=6144, k=Q + 5128 * 2, v=Q + 4096 * 2) == EALIAS  # k runs into the next row
    assert f(kc=Q) == EALIAS and f(vc=V) == EALIAS and f(kc=ROPE) == EALIAS and f(vc=SLOT) == EALIAS


def test_rope_cache_in_place_in_a_packed_projection(lib):
    """q, k and v as the columns of one buffer in any order; rows that cross are refused."""
    f = lambda q, k, v, **kw: rope(lib, q=Q + q * 2, qo=Q + q * 2, os=6144, k=Q + k * 2, v=Q + v * 2, **kw)  # noqa: E731
    assert f(0, 4096, 5120) == f(1024, 0, 5120) == f(2048, 0, 1024) == f(2048, 1024, 0) == OK
    # the same columns some rows further on or back, which share no element either
    assert f(2048, 6144 * 3, 1024) == f(6144 * 50, 6144 * 3 + 4096, 5120) == OK
    assert f(2048, 1032, 0) == EALIAS      # k's rows run into q's
    assert f(2048, 6144 - 8, 0) == EALIAS  # k's rows begin inside q's
    assert f(1024, 1024, 0) == EALIAS and f(1024, 2048, 0) == EALIAS
    assert rope(lib, q=Q + 4096, qo=Q + 4096, os=6144, k=Q, v=Q + 2048, ks=6152) == EALIAS  # other strides


def attn(lib, q=Q, N=100, qs=4096, kc=KC, vc=VC, pages=50, page=64, tab=TAB, ts=70, M=66, q_start=QS,
         kl=KL, S=8, H=32, Hkv=8, hd=128, window=1000, sinks=4, chunk=1, max_q=100, scale=0.1, out=OUT,
         lse=LSE, work=WORK, size=None):
    if size is None:
        size = lib.dan_window_attention_workspace(N, S, H, Hkv, hd, M, page, window, sinks, chunk, max_q)
    return lib.dan_can_use_window_attention(q, N, qs, kc, vc, pages, page, tab, ts, M, q_start, kl, S,
                                            H, Hkv, hd, window, sinks, chunk, max_q, scale, out, lse,
                                            work, size)


def test_attention_validation(lib):
    f = lambda **k: attn(lib, **k)  # noqa: E731
    assert f() == OK and f(lse=None) == OK and f(hd=64) == OK
    for page in (16, 32, 128):
        assert f(page=page) == OK
    assert f(page=24) == EUNSUP and f(hd=80) == EUNSUP and f(H=33) == EINVAL
    assert f(N=-1) == EINVAL and f(S=-1) == EINVAL and f(M=0) == EINVAL and f(max_q=-1) == EINVAL
    assert f(window=-1) == EINVAL and f(sinks=-1) == EINVAL and f(chunk=0) == EINVAL
    assert f(window=0) == OK and f(window=0x7FFFFFFF, sinks=0x7FFFFFFF, chunk=0x7FFFFFFF) == OK
    assert f(window=1 << 31) == EINVAL and f(sinks=1 << 31) == EINVAL and f(chunk=1 << 31) == EINVAL
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert f(scale=s) == EINVAL
    assert f(ts=65) == EINVAL and f(qs=4088) == EINVAL and f(qs=4100) == EALIGN
    assert f(S=(1 << 20) + 1, size=1 << 50) == EUNSUP
    assert f(M=(1 << 24) + 1, ts=1 << 25, size=1 << 50) == EUNSUP
    assert f(N=(1 << 30) + 1, size=1 << 50) == EUNSUP
    for name in ("q", "kc", "vc", "tab", "q_start", "kl", "out"):
        assert f(**{name: None}) == EINVAL, name
    for name, base in (("q", Q), ("kc", KC), ("vc", VC), ("out", OUT), ("work", WORK)):
        assert f(**{name: base + 8}) == EALIGN, name
    for name, base in (("tab", TAB), ("q_start", QS), ("kl", KL), ("lse", LSE)):
        assert f(**{name: base + 4}) == OK and f(**{name: base + 2}) == EALIGN, name
    assert f(N=0, q=None, out=None) == OK and f(S=0, tab=None, kl=None) == OK
    for over in (dict(out=Q), dict(out=KC + 4096), dict(lse=OUT), dict(work=OUT), dict(work=VC),
                 dict(lse=TAB), dict(out=QS), dict(work=KL), dict(lse=WORK)):
        assert f(**over) == EALIAS, over


def test_workspace(lib):
    size = lambda N=64, S=64, H=32, Hkv=8, hd=128, M=512, page=64, window=1000, sinks=4, chunk=1, \
        max_q=1: lib.dan_window_attention_workspace(N, S, H, Hkv, hd, M, page, window, sinks, chunk, max_q)  # noqa: E731
    need = size()
    assert need > 0 and attn(lib, N=64, S=64, M=512, ts=512, max_q=1, size=need) == OK
    assert attn(lib, N=64, S=64, M=512, ts=512, max_q=1, size=need - 1) == EINVAL
    assert attn(lib, N=64, S=64, M=512, ts=512, max_q=1, work=None) == EINVAL
    assert size(N=0) == 0 and size(S=0) == 0
    assert size(hd=80) == 0 and size(M=0) == 0 and size(N=-1) == 0  # refused by the call
    assert size(window=-1) == 0 and size(sinks=1 << 31) == 0 and size(chunk=0) == 0
    # what a wider window needs is no less, up to the whole table
    grows = [size(window=w) for w in (0, 1, 200, 1000, 5000, 40000, 0x7FFFFFFF)]
    assert grows == sorted(grows) and grows[-1] == grows[-2]
    assert size(window=100, sinks=4) == 0 and attn(lib, N=64, S=64, M=512, ts=512, max_q=1, window=100,
                                                   work=None) == OK
    # a prompt always has its work list
    assert size(N=500, S=1, max_q=500, window=100) > 0
    # a table that holds fewer keys than two splits needs none, and none may be passed
    assert size(M=1) == 0 and attn(lib, N=64, S=64, M=1, ts=1, max_q=1, work=None) == OK


def test_workspace_is_bounded_by_each_kernel(lib):
    """A sequence is split by one kernel or the other, each with rows and splits of its own: a
    large batch over long caches asks for what both can use, not for the larger of each."""
    size = lambda N, S, H=32, Hkv=8, hd=128, M=512, page=64, window=1 << 30, sinks=0, chunk=1, max_q=None: \
        lib.dan_window_attention_workspace(N, S, H, Hkv, hd, M, page, window, sinks, chunk,
                                           N if max_q is None else max_q)  # noqa: E731
    MiB = 1 << 20
    # 256 sequences of up to 16 rows and 32 splits, 4096 rows of up to 8 splits, 520 bytes each
    assert size(4096, 256) < 1100 * MiB
    assert size(8192, 1024) < 3200 * MiB
    assert size(4096, 256, max_q=28) < 1000 * MiB
    # a group of more than 16 query heads leaves the step kernel no sequence: no room for it
    assert size(64, 64, H=32, Hkv=1, max_q=1) <= 64 * 32 * 16 * 520 + (8 + 64 * 65) * 80 + 64 * 33 * 8 + 16
    # tokens that the step kernel alone takes: their own rows, 32 splits each
    assert size(64, 64, max_q=1) == 64 * 32 * 32 * 520
    # prompts too long to be split have work lists alone, where the bound says so
    assert size(65536, 64, H=8, Hkv=8, hd=64, M=4, max_q=1024) < MiB


def test_binding_refuses_without_cuda_tensors():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    with pytest.raises(TypeError):
        ops.qk_norm_rope_cache(z(2, 256), z(2, 128), z(2, 128), z(128), z(128),
                               z(8, 128, dt=torch.float32), z(2, dt=torch.int32),
                               z(2, dt=torch.int32), z(1, 1, 16, 128), z(1, 1, 16, 128), 1e-6)
    with pytest.raises(TypeError):
        ops.window_attention(z(2, 2, 128), z(1, 1, 16, 128), z(1, 1, 16, 128),
                             z(1, 1, dt=torch.int32), z(2, dt=torch.int32), z(1, dt=torch.int32), 16)
