"""Host paths of the training operators at the ends of their ranges, with a fake CUDA runtime (no
GPU): the kernels that a call launches there, and calls that cannot launch them all."""
import pytest

from test_cache_calls_host import fake  # noqa: F401 (a fixture)
from test_train_calls_host import CALLS, ECUDA, OK


def test_short_rows_share_a_warp(fake):
    """Rows of fewer than 1024 columns that are many: three CTAs an SM, of as many rows at once as
    their lanes hold; 1024 and more go by the row kernel."""
    narrow, few, widest, row = fake(CALLS + """
print(json.dumps([save(T=1 << 20, D=16), save(T=100, D=16), save(T=1 << 20, D=1016), save(T=1 << 20, D=1024)]))""")
    assert [r[0] for r in (narrow, few, widest, row)] == [OK] * 4
    assert narrow[1][0][:3] == [3 * 152, 1, 256] == widest[1][0][:3]
    assert few[1][0][:3] == [1, 1, 256]             # 128 lanes' worth of two lanes a row, four rows each
    assert row[1][0][0] == 152


@pytest.mark.parametrize("D", [8, 264, 1016])
def test_short_rows_that_cannot_run_launch_nothing(fake, D):
    for fail in ("SET", "LAUNCH"):
        first, again = fake(CALLS + f"fail_at[{fail}] = 1\nprint(json.dumps([save(D={D}), save(D={D})]))")
        assert first == [ECUDA, []] and again[0] == OK and len(again[1]) == 1


def test_gradients_of_nothing(fake):
    """One kernel that needs no workspace, and none where it cannot run."""
    for sizes in ("N=1, S=0", "N=3, S=0", "N=0, S=7"):
        call = f"gn_back({sizes})"
        good, size = fake(CALLS + f"print(json.dumps([{call}, lib.dan_group_norm_backward_workspace(3, 0, 512, 32, 0, 0)]))")
        assert good[0] == OK and len(good[1]) == 1 and size == 0
        assert fake(CALLS + f"fail_at[SET] = 1\nprint(json.dumps({call}))") == [ECUDA, []]


def test_gradients_of_short_and_long_batches(fake):
    """Many short batches: one kernel without a workspace; else the rows' and a join whose blocks have
    as many threads a column as a batch can have partials."""
    sizes = [(65536, 1, 64), (1953, 8, 1024), (700, 0, 4096), (488, 32, 1024), (1, 4216, 4096), (16, 256, 4096),
             (61, 64, 4096)]
    calls = "".join(f"ln_back(B={b}, T={t}, D={d}), " for b, t, d in sizes)
    works = "".join(f"lib.dan_ln_modulate_backward_workspace({b}, {t}, {d}), " for b, t, d in sizes)
    got, work = fake(CALLS + f"print(json.dumps([[{calls}], [{works}]]))")
    assert all(st == OK for st, _ in got)
    assert [len(grids) for _, grids in got] == [1, 1, 1, 2, 2, 2, 2]
    assert [w > 0 for w in work] == [False] * 3 + [True] * 4
    assert got[0][1][0][0] == 3 * 152
    # blocks of the join: 4, 32 and 256 columns' quads of [dscale | dshift] each
    assert [grids[1][0] for _, grids in got[4:]] == [512, 16 * 64, 61 * 8]


@pytest.mark.parametrize("call,sets", [("ln_back(B=4000, T=1, D=64)", 1), ("ln_back(B=61, T=64, D=4096)", 3)])
def test_gradients_that_cannot_run_whole_launch_nothing(fake, call, sets):
    for n in range(1, sets + 1):
        first, counted, again = fake(CALLS + f"fail_at[SET] = {n}\na = {call}\nprint(json.dumps([a, count[SET], {call}]))")
        assert first == [ECUDA, []] and counted == n and again[0] == OK, n


def test_parameter_gradients_of_many_images(fake):
    """A launch more for each further factor of 256 images; where one cannot be made ready, none."""
    got = fake(CALLS + "print(json.dumps([gn_back(N=n, S=1) for n in (1, 2, 256, 257, 65536, 65537)]))")
    assert all(st == OK for st, _ in got) and [len(grids) for _, grids in got] == [1, 2, 2, 3, 3, 4]
    assert all(grids[-1][:2] == [1, 16] for _, grids in got[1:])
    for n in range(1, 4):
        first, counted, again = fake(CALLS + f"fail_at[SET] = {n}\na = gn_back(N=300, S=1)\n"
                                     "print(json.dumps([a, count[SET], gn_back(N=300, S=1)]))")
        assert first == [ECUDA, []] and counted == n and again[0] == OK and len(again[1]) == 3


def test_slabs_of_few_positions(fake):
    """A fragment for each thread of the smallest CTA, whole groups; cut alike for any number of
    images."""
    got = fake(CALLS + "print(json.dumps([gn(N=n, S=s, C=1024) for s in (1, 2, 8, 64) for n in (1, 500)]))")
    assert all(st == OK and len(grids) == 1 for st, grids in got)
    # fragments of a row: 128
    assert [grids[0][:3] for _, grids in got[::2]] == [[1, 2, 64], [1, 4, 64], [1, 16, 64], [1, 16, 64]]
    assert all(b[1][0][0] == 500 * a[1][0][0] and b[1][0][1:] == a[1][0][1:] for a, b in zip(got[::2], got[1::2]))
