"""Failure detection of the paged attention kernels without a GPU fault: in the test-only
build (50 ms wait limit) the producer of either kernel never requests the second tile of a
CTA, so bounded waits run out.  The call returns, reports GVA_DEVERR_WAIT, frees its tensor
memory and leaves the context usable: the regular library then attends the same inputs."""
import ctypes
import time

import pytest
import torch

from compressed_kv_cache_gva_b200 import _build, gva
from test_gpu_paged import A, BF, C128, F32, Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,new,out", [(A, [1, 1], F32), (A, [40, 40], BF), (C128, [20, 20], BF), (A, [5, 5], F32)])
def test_withheld_tile_is_reported(heads, new, out):
    _build.build_wait_test()
    L = gva.load(_build.WAIT_TEST_LIB)
    x = Batch(heads, 64, [40000, 30000] if new == [1, 1] else [9000, 6000], new, seed=1)
    t, sh = x.device(), x.shape(out)
    ws = gva.new_paged_workspace(sh, 64, x.rows, x.max_new, x.total)
    o = torch.zeros(x.rows, x.H, x.d_h, dtype=out, device="cuda")
    torch.cuda.synchronize()
    t0 = time.time()
    st = L.gva_paged_attention(ctypes.byref(sh), 64, t["q"].data_ptr(), t["V"].data_ptr(), t["kr"].data_ptr(),
                               t["V"].shape[0], t["table"].data_ptr(), t["table"].shape[1], t["table"].stride(0),
                               t["q_start"].data_ptr(), t["L"].data_ptr(), x.rows, x.max_new, x.total, o.data_ptr(), None,
                               ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == 0, L.gva_last_error()
    torch.cuda.synchronize()
    assert time.time() - t0 < 30
    assert gva.workspace_status(ws) == gva.DEVERR_WAIT
    # the regular library, in the same process
    got = x.run(out)
    assert abs(got[0]).max() < 10 and torch.isfinite(torch.from_numpy(got[1])).all()
    again = x.run(out)
    assert (got[0] == again[0]).all() and (got[1] == again[1]).all()
