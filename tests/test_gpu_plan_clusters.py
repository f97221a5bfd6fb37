"""The page plan of a large step where the GPU (a partition of it) holds no cluster of 16
blocks: the largest that fits is launched, with the same results.  The test-only build takes
the bound from the environment."""
import numpy as np
import pytest
import torch

from compressed_kv_cache_gva_b200 import _build, gva
from test_plan_pages import make, want

pytestmark = pytest.mark.gpu
I32 = torch.int32


def run(L, s, in_place):
    dev = lambda x: torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()
    B, width = s["table"].shape
    z = lambda k: torch.full((k,), 77, dtype=I32, device="cuda")
    table, free, held_in, count_in = dev(s["table"]), dev(s["free"]), dev(s["held"]), dev([s["count"]])
    held, count = (held_in, count_in) if in_place else (z(B), z(1))
    o = dict(q_start=z(B + 1), seq_len=z(B), n_granted=z(B), slot=z(s["room"]), pos=z(s["room"]))
    kept, n, err = dev(s["kept"]), dev(s["n"]), dev([0])
    p = lambda t: t.data_ptr()
    st = L.gva_plan_pages(B, s["page"], s["num_pages"], width, width, s["room"], p(kept), p(n), p(held_in), p(held), p(free),
                          p(count_in), p(count), p(table), p(o["q_start"]), p(o["seq_len"]), p(o["n_granted"]), p(o["slot"]),
                          p(o["pos"]), p(err), torch.cuda.current_stream().cuda_stream)
    assert st == 0, L.gva_last_error()
    torch.cuda.synchronize()
    o = {k: v.tolist() for k, v in o.items()}
    o.update(held=held.tolist(), free=free.tolist(), count=int(count), table=table.tolist(), err=int(err))
    return o


@pytest.mark.parametrize("limit", [16, 8, 5, 4, 2, 1])
@pytest.mark.parametrize("in_place", [False, True])
def test_smaller_clusters(monkeypatch, limit, in_place):
    _build.build_wait_test()
    L = gva.load(_build.WAIT_TEST_LIB)
    monkeypatch.setenv("GVA_TEST_CLUSTER_LIMIT", str(limit))
    for B, page, max_len, n_hi, spare in ((513, 8, 60, 70, 200), (2048, 16, 500, 8, 600), (4096, 16, 100, 6, 900),
                                          (7, 16, 5000, 9000, 4000)):
        s = make(B, page, max_len, n_hi, spare, seed=limit)
        got, ref = run(L, s, in_place), want(s)
        for k in ref:
            assert got[k] == ref[k], (B, k)
