"""A paged workspace sized for the largest step of a server serves every smaller one: fewer
requests, rows, new tokens per request or cached tokens, though those may take other kernels."""
import ctypes
import random
import re

import numpy as np
import pytest
import torch

from compressed_kv_cache_gva_b200 import gva
from test_gpu_paged import A, BF, C128, D32, F32, MHA, WIDE, Batch

pytestmark = pytest.mark.gpu
FAKE = 1 << 20
HEADS = [A, C128, (8, 2, 32, 8), MHA, WIDE, (16, 4, 32, 24), (8, 2, 128, 16), (12, 4, 64, 8), (20, 2, 64, 16),
         (16, 4, 128, 16), (24, 1, 64, 16), (5 * 8, 8, 64, 0), (6, 2, 40, 4)]


def shape(heads, B, cache=BF, out=BF, flags=0, ctas=0):
    H, G, d_h, d_r = heads
    return gva.make_shape(B, H, G, d_h, d_h, d_r, cache_dtype=cache, out_dtype=out, flags=flags, ctas_per_sm=ctas)


def required(sh, page, rows, most, total):
    """The bytes that a call of these bounds asks for, from its refusal of one byte (nothing is
    launched and no pointer read)."""
    L = gva.lib()
    st = L.gva_paged_attention(ctypes.byref(sh), page, FAKE, FAKE, FAKE, 1024 * page, FAKE, 8, 8, FAKE, FAKE, rows, most,
                               total, FAKE, None, FAKE, 1, None)
    assert st == 3, L.gva_last_error()
    return int(re.search(r"required (\d+)", L.gva_last_error().decode()).group(1))


def test_sizes_cover_every_smaller_step():
    rng = random.Random(1)
    log = lambda lo, hi: int(round(2 ** rng.uniform(np.log2(lo), np.log2(hi))))
    for _ in range(1500):
        heads = rng.choice(HEADS)
        narrow = heads[2] % 8 or heads[3] % 8
        kw = dict(cache=F32 if narrow else rng.choice([BF, BF, BF, F32]), out=rng.choice([BF, F32]),
                  flags=rng.choice([0, 0, 0, gva.FLAG_FMA_PATH]), ctas=rng.choice([0, 0, 0, 1, 2]))
        page = rng.choice([1, 8, 12, 16, 64])
        B, most = log(1, 4096), log(1, 600)
        rows, total = log(1, B * most), log(1, 1 << 22)
        size = gva.paged_workspace_size(shape(heads, B, **kw), page, rows, most, total)
        assert size > 0
        for k in range(8):
            b = B if k % 2 else log(1, B)
            r, m, t = log(1, rows), log(1, most), log(1, total)
            if k == 0:
                b, r, m, t = B, rows, most, total
            assert required(shape(heads, b, **kw), page, r, m, t) <= size, (heads, kw, page, B, rows, most, total, b, r, m, t)


@pytest.mark.parametrize("heads,B,page,large,small", [
    (A, 2048, 16, (16384, 512, 1 << 20), (16384, 4, 1 << 20)),
    (A, 64, 16, (4096, 64, 64 * 8192), (127, 64, 64 * 4000)),
    (C128, 1024, 16, (8192, 8, 1 << 20), (2048, 2, 1 << 20))])
def test_prompts_then_single_tokens(heads, B, page, large, small):
    sh = shape(heads, B)
    assert required(sh, page, *small) <= gva.paged_workspace_size(sh, page, *large)


@pytest.mark.parametrize("heads", [A, C128, D32])
def test_one_workspace_for_all_steps(heads):
    """A server of 40 requests, its workspace made once for the largest step."""
    cache = F32 if heads is D32 else BF
    B, most, rows, total = 40, 64, 40 * 64, 40 * 200
    lens = [1 + 5 * i for i in range(B)]
    x = Batch(heads, 16, lens, [min(most, L) for L in lens], cache=cache, seed=1)
    big = gva.new_paged_workspace(x.shape(BF), 16, rows, most, total)
    big[256:] = 0xff
    for i, new in enumerate([[min(most, L) for L in lens], [1] * B, [min(4, L) for L in lens], [1, 2, 0, 1] * 10,
                             [1] * (B - 1) + [64]]):
        y = Batch(heads, 16, lens, new, cache=cache, seed=i, pad=i % 2)
        t, sh = y.device(), y.shape(BF)
        for bounds in ((most, total), (y.max_new, y.total)):
            o = torch.full((y.rows, y.H, y.d_h), 3.25, dtype=BF, device="cuda")
            lse = torch.full((y.rows, y.H), 3.25, device="cuda")
            gva.paged_attention(sh, 16, t["q"], t["V"], t["kr"], t["table"], t["q_start"], t["L"], *bounds, o, lse, big)
            torch.cuda.synchronize()
            assert gva.workspace_status(big) == 0
            y.check((o.float().cpu().double().numpy(), lse.cpu().double().numpy()), y.reference(), BF, 2.0 ** -8,
                    q_round=0.0 if heads is D32 else 2.0 ** -16)
