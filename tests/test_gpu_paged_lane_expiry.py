"""A bounded wait that runs out in some lanes of a warp only (a tile that lands just as the
limit expires), without a GPU fault: the test-only build makes every wait of a whole warp run
out in its odd lanes where the status word asks for it.  The warp then gives up as one: the
call returns, reports GVA_DEVERR_WAIT, and the regular library attends the same inputs."""
import ctypes
import time

import pytest
import torch

from compressed_kv_cache_gva_b200 import _build, gva
from test_gpu_paged import A, B24, BF, C128, F32, Batch

pytestmark = pytest.mark.gpu

CASES = [(A, [40, 30], [1, 1], F32), (A, [9000, 30], [1, 2], F32), (A, [300, 40], [4, 3], BF),
         (C128, [300, 40], [2, 1], BF), (A, [300, 40], [40, 9], BF), (A, [9000, 60], [40, 40], F32),
         (B24, [400, 90], [5, 5], BF), (C128, [300, 150], [20, 20], BF), (C128, [300, 150], [20, 1], F32)]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_a_wait_that_half_a_warp_sees_expire(case):
    heads, lens, new, out = CASES[case]
    _build.build_wait_test()
    L = gva.load(_build.WAIT_TEST_LIB)
    x = Batch(heads, 64 if heads is not B24 else 32, lens, new, seed=case)
    t, sh = x.device(), x.shape(out)
    ws = gva.new_paged_workspace(sh, x.page, x.rows, x.max_new, x.total)
    ws[:4].view(torch.int32).fill_(_build.LANE_EXPIRY)
    o = torch.zeros(x.rows, x.H, x.d_h, dtype=out, device="cuda")
    torch.cuda.synchronize()
    t0 = time.time()
    st = L.gva_paged_attention(ctypes.byref(sh), x.page, t["q"].data_ptr(), t["V"].data_ptr(), t["kr"].data_ptr(),
                               t["V"].shape[0], t["table"].data_ptr(), t["table"].shape[1], t["table"].stride(0),
                               t["q_start"].data_ptr(), t["L"].data_ptr(), x.rows, x.max_new, x.total, o.data_ptr(), None,
                               ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == 0, L.gva_last_error()
    torch.cuda.synchronize()
    assert time.time() - t0 < 30
    assert gva.workspace_status(ws) == gva.DEVERR_WAIT | _build.LANE_EXPIRY
    x.check(x.run(out), x.reference(), out, 2.0 ** -8 if out == BF else 2.0 ** -16)
