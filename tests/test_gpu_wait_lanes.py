"""The decode and prefill kernels of the contiguous cache, with waits that run out in the odd
lanes of a warp only (test-only build; the status word asks for it): the warp gives up as one,
the call returns and reports GVA_DEVERR_WAIT, and the regular library is unaffected."""
import ctypes
import time

import numpy as np
import pytest
import torch

from compressed_kv_cache_gva_b200 import _build, gva
from compressed_kv_cache_gva_b200.synth import WORKLOADS, make_decode_inputs
from gpu_helpers import assert_close, dev, oracle_gva, run_gva, shape_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths", [[40, 17], [16384, 300]])
@pytest.mark.parametrize("flags,Q", [(0, 1), (gva.FLAG_TCGEN05_PATH, 1), (0, 16)])
def test_a_wait_that_half_a_warp_sees_expire(flags, Q, lengths):
    _build.build_wait_test()
    L = gva.load(_build.WAIT_TEST_LIB)
    wl = WORKLOADS["350m_b8_t4096"]
    di = make_decode_inputs(wl, extra_slots=1, lengths=np.array(lengths))
    sh = shape_of(di, flags=flags)
    B, total = 2, di.total_tokens
    q_abs = torch.randn(B, Q, wl.H, wl.d_h + wl.d_r, device="cuda")
    V, KR, soff, slen = dev(di.V), dev(di.k_rope), dev(di.seq_offset), dev(di.seq_len)
    ws = torch.zeros(gva.decode_workspace_size_multi(sh, Q, total), dtype=torch.uint8, device="cuda")
    ws[:4].view(torch.int32).fill_(_build.LANE_EXPIRY)
    out = torch.zeros(B, Q, wl.H, wl.d_h, device="cuda")
    torch.cuda.synchronize()
    t0 = time.time()
    st = L.gva_decode_attention_multi(ctypes.byref(sh), Q, q_abs.data_ptr(), V.data_ptr(), KR.data_ptr(),
                                      soff.data_ptr(), slen.data_ptr(), total, V.shape[0], out.data_ptr(), None,
                                      ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == 0, L.gva_last_error()
    torch.cuda.synchronize()
    assert time.time() - t0 < 30
    assert gva.workspace_status(ws) & gva.DEVERR_WAIT
    got, _, _, status = run_gva(di, flags=flags)
    assert status == 0
    assert_close(got, oracle_gva(di)[0], wl.dtype, "decode after waits that half a warp saw expire")
