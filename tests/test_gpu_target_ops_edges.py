"""Calls of the target-side operators that their documentation allows at its
edges: pages that a window has left behind, strides of one entry, workspaces
sized ahead, status words."""
import pytest
import torch

from tests.test_gpu_target_ops import Batch, check_attention, i32, ref_paged, run_paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,lens,hq", [([16], [3000], 4), ([1, 5], [900, 2000], 8), ([200, 90], [900, 700], 4),
                                          ([1, 1, 1], [30011, 700, 16384], 8), ([300, 2, 150], [2100, 3000, 150], 8)])
def test_pages_behind_the_window_may_be_gone(dtype, rows, lens, hq):
    """A server gives the pages back that no row's window reaches any more: their table entries name no page, and
    that is not an error, although a tile of keys begins in front of the window."""
    W = 100
    B = Batch(dtype, hq, 2, 64, 16, rows, lens, seed=2)
    ref = ref_paged(B, True, W)
    B.kp, B.vp = B.appended()
    for b, (n, L) in enumerate(zip(rows, lens)):
        B.table[b, :max(0, L - n - W + 1) // 16] = -1
    status = i32([0])
    out, lse, _, _ = run_paged(B, True, W, append=False, status=status)
    check_attention(out, lse, ref, B.starts[-1])
    assert int(status.item()) == 0
    b = max(range(len(lens)), key=lambda i: lens[i])   # one page further: the first new row sees its last slots
    B.table[b, (lens[b] - rows[b] - W + 1) // 16] = -1
    run_paged(B, True, W, append=False, status=status)
    assert int(status.item()) == 4
