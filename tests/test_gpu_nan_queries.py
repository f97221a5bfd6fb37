"""Queries that hold a NaN on the contiguous cache: NaN outputs and lse for their row, however
the sequence is cut between CTAs, every other row bit by bit as without them; and the merge of
states over parts of a sequence passes NaN on."""
import numpy as np
import pytest
import torch

from compressed_kv_cache_gva_b200 import gva
from compressed_kv_cache_gva_b200.synth import WORKLOADS, make_decode_inputs
from gpu_helpers import dev, shape_of

pytestmark = pytest.mark.gpu


def attend(di, sh, Q, q_abs, out_dtype):
    wl, total = di.wl, max(di.total_tokens, 1)
    B = len(di.seq_len)
    ws = torch.zeros(gva.decode_workspace_size_multi(sh, Q, total), dtype=torch.uint8, device="cuda")
    out = torch.empty(B, Q, wl.H, wl.d_h, dtype=out_dtype, device="cuda")
    lse = torch.empty(B, Q, wl.H, device="cuda")
    gva.decode_attention_multi(sh, Q, q_abs, dev(di.V), dev(di.k_rope), dev(di.seq_offset), dev(di.seq_len), total, out, lse,
                               ws)
    torch.cuda.synchronize()
    assert gva.workspace_status(ws) == 0
    return out.float(), lse


BF16 = [("350m_b8_t4096", [40, 17]), ("350m_b8_t4096", [16384, 300]), ("d128_b1_t131072", [9000, 40])]
KINDS = [(0, 1), (gva.FLAG_TCGEN05_PATH, 1), (gva.FLAG_FMA_PATH, 1), (0, 2), (0, 16)]   # flags, new tokens
CASES = [(*c, *k) for c in BF16 for k in KINDS] + [("tiny_fp32_t64", [700, 90], 0, 1)]


@pytest.mark.parametrize("name,lengths,flags,Q", CASES)
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_rows_of_a_nan_query(name, lengths, flags, Q, out_dtype):
    wl = WORKLOADS[name]
    di = make_decode_inputs(wl, extra_slots=1, lengths=np.array(lengths))
    sh = shape_of(di, out_dtype=out_dtype, flags=flags)
    torch.manual_seed(1)
    q = torch.randn(2, Q, wl.H, wl.d_h + wl.d_r, device="cuda") * 0.2
    want, want_l = attend(di, sh, Q, q, out_dtype)
    hit = torch.zeros(2, Q, wl.H, dtype=torch.bool, device="cuda")
    for b, i, h, c in ((0, 0, 0, 3), (0, Q - 1, wl.H - 1, wl.d_h + wl.d_r - 1), (1, Q - 1, 1, 0)):
        q[b, i, h, c] = float("nan")
        hit[b, i, h] = True
    out, lse = attend(di, sh, Q, q, out_dtype)
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], want_l[~hit])


def test_an_empty_sequence_stays_empty():
    wl = WORKLOADS["350m_b8_t4096"]
    di = make_decode_inputs(wl, extra_slots=1, lengths=np.array([30, 5]))
    di.seq_len[1] = 0
    for flags in (0, gva.FLAG_TCGEN05_PATH, gva.FLAG_FMA_PATH):
        q = torch.full((2, 1, wl.H, wl.d_h + wl.d_r), float("nan"), device="cuda")
        out, lse = attend(di, shape_of(di, flags=flags), 1, q, torch.float32)
        assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
        assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()


def test_merged_states():
    nan, inf = float("nan"), float("inf")
    sh = gva.make_shape(1, 4, 2, 64, 64, 16)
    lses = torch.tensor([[nan, nan, -inf, 1.0], [nan, 2.0, -inf, -inf]], device="cuda").reshape(2, 1, 4)
    outs = torch.ones(2, 1, 4, 64, device="cuda")
    outs[:, :, 0] = nan
    outs[0, :, 1] = nan
    out, lse = torch.empty(1, 4, 64, device="cuda"), torch.empty(1, 4, device="cuda")
    gva.merge_states(sh, outs, lses, out, lse)
    assert torch.isnan(out[0, :2]).all() and torch.isnan(lse[0, :2]).all()
    assert (out[0, 2] == 0).all() and lse[0, 2] == -inf
    assert (out[0, 3] == 1).all() and lse[0, 3] == 1.0
