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
