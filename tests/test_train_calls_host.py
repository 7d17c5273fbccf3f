"""Host paths of the training operators with a fake CUDA runtime (no GPU): which kernels a call
launches, how an image is cut, and that a call that cannot launch them all launches none."""
import pytest

from test_cache_calls_host import fake  # noqa: F401 (a fixture)

OK, EINVAL, EUNSUP, EALIGN, EALIAS, ECUDA = range(6)

CALLS = r"""
for name in ("dan_ln_modulate_backward_workspace", "dan_group_norm_workspace", "dan_group_norm_backward_workspace"):
    getattr(lib, name).restype = I
N32 = ctypes.c_int
lib.dan_ln_modulate_backward_workspace.argtypes = [I] * 3
lib.dan_group_norm_workspace.argtypes = lib.dan_group_norm_backward_workspace.argtypes = [I] * 4 + [N32] * 2
lib.dan_ln_modulate_save.argtypes = [P, P, P, I, P, P, P, P, I, I, I, F, P]
lib.dan_ln_modulate_backward.argtypes = [P] * 6 + [I, P, P, P, P, I, I, I, I, P, I, P]
lib.dan_group_norm.argtypes = [P, N32, P, P, N32, P, P, I, N32, P, P, P, P, I, I, I, I, F, P, I, P]
lib.dan_group_norm_backward.argtypes = [P, P, N32, P, P, P, P, P, N32, P, P, I, N32] + [P] * 5 + [I] * 5 + [P, I, P]
at = [0x1000000000 * (i + 1) for i in range(16)]
def launched(call):
    before = ctypes.c_int.in_dll(fake, "launches").value
    st = call()
    grids = (ctypes.c_uint * 4 * 64).in_dll(fake, "grids")
    return st, [list(grids[i]) for i in range(before, ctypes.c_int.in_dll(fake, "launches").value)]
def save(B=1, T=4216, D=4096):
    return launched(lambda: lib.dan_ln_modulate_save(at[0], at[1], at[2], D, at[3], at[4], at[5], at[6], B, T, D, 1e-6, None))
def ln_back(B=1, T=4216, D=4096):
    size = lib.dan_ln_modulate_backward_workspace(B, T, D)
    return launched(lambda: lib.dan_ln_modulate_backward(at[0], None, at[1], at[2], at[3], at[4], D, None, at[5], at[6],
                                                         at[7], D, B, T, D, at[8], size, None))
def gn(N=1, S=4096, C=512, G=32):
    size = lib.dan_group_norm_workspace(N, S, C, G, 0, 0)
    return launched(lambda: lib.dan_group_norm(at[0], 0, at[1], at[2], 0, None, None, C, 1, at[3], None, None, None, N, S, C,
                                               G, 1e-6, at[4], size, None))
def gn_back(N=1, S=4096, C=512, G=32):
    size = lib.dan_group_norm_backward_workspace(N, S, C, G, 0, 0)
    return launched(lambda: lib.dan_group_norm_backward(at[0], at[1], 0, None, None, at[2], at[3], at[4], 0, None, None, C, 1,
                                                        at[5], at[6], at[7], None, None, C, N, S, C, G, at[8], size, None))
"""


def test_kernels_of_a_call(fake):
    """One launch, the rows' and the join; a slab (and its images' sum); the passes and theirs, the
    second one joining few chunks itself."""
    s, b, small, many, large, back, pair, passes, nothing, few = fake(CALLS + """
print(json.dumps([save(), ln_back(), gn(S=64), gn(N=7, S=64), gn(S=1 << 18), gn_back(S=64), gn_back(N=3, S=64),
                  gn_back(N=3, S=1 << 18), ln_back(T=0), gn(S=6000, G=8)]))""")
    assert all(r[0] == OK for r in (s, b, small, many, large, back, pair, passes, nothing, few))
    assert [len(r[1]) for r in (s, b, small, many, large, back, pair, passes, nothing, few)] == \
        [1, 2, 1, 1, 3, 1, 2, 4, 1, 2]
    # a slab's launch has the images along x and is cut the same for each
    assert many[1][0][0] == 7 * small[1][0][0] and many[1][0][1:] == small[1][0][1:]
    # the passes' first wave: a CTA in each of an SM's four places (two for the gradients)
    assert 0.85 * 608 <= large[1][0][0] * large[1][0][1] <= 608 and large[1][0][3] > 228 * 1024 // 5 - 1024
    assert large[1][2][3] > 228 * 1024 // 5 - 1024 and passes[1][0][3] > 228 * 1024 // 3 - 1024


@pytest.mark.parametrize("call,sets", [("ln_back()", 3), ("gn(S=1 << 18)", 3), ("gn_back(N=3, S=1 << 18)", 6)])
def test_a_call_that_cannot_run_whole_launches_nothing(fake, call, sets):
    """Each attribute that a call sets fails once: DAN_ECUDA and no kernel, and the next call is good."""
    for n in range(1, sets + 1):
        first, counted, again = fake(CALLS + f"fail_at[SET] = {n}\na = {call}\n"
                                     f"print(json.dumps([a, count[SET], {call}]))")
        assert first == [ECUDA, []] and counted == n, n
        assert again[0] == OK and len(again[1]) >= 2


def test_no_exception_leaves_a_call(fake):
    for call in ("save()", "ln_back()", "gn()", "gn_back()"):
        first, again = fake(CALLS + "fail_at[SET] = 1\nctypes.c_int.in_dll(fake, 'throws').value = 1\n"
                            f"print(json.dumps([{call}, {call}]))")
        assert first == [ECUDA, []] and again[0] == OK, call
