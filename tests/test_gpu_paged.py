"""Paged attention against the float64 oracle, element by element.

Tolerances are worst-case bounds of the arithmetic, computed from the inputs.  With
A = sum p |v| of an output element, S = max over a row's keys of sum_i |q_i v_i|:
  - tensor-core kernels split the fp32 query in two bf16 parts, each rounding off at most
    2^-8 of its operand: |ds| <= 2^-16 S (natural units: times ln 2); the CUDA-core kernel
    uses it whole;
  - products accumulate in fp32: |ds| <= (d + 2) 2^-24 S, and the sums over L keys
    (L + 64) 2^-24 of the sum of magnitudes (probabilities' sum and value sum alike);
  - an exponential is off by 2^-21 of itself (ex2.approx and its fp32 argument);
  - a probability is rounded to 2^-8 of itself (bf16 outputs of the tcgen05 kernel) or to
    2^-16 (two bf16 parts, the other tensor-core kernels);
  - the output is rounded once: 2^-8 |o| (bf16) or 2^-24 |o|.
So |o - ref| <= A (exp(2 e) - 1 + p + 2 (L + 64) 2^-24 + 2^-20) + out |ref| with e the
score error, and |lse - ref| <= e + (L + 64) 2^-24 + 2^-20 + 2^-23 |ref|.
"""
import numpy as np
import pytest
import torch

from compressed_kv_cache_gva_b200 import gva
from oracle import serving_oracle

pytestmark = pytest.mark.gpu
I32 = torch.int32
BF, F32 = torch.bfloat16, torch.float32


class Batch:
    """Requests of given lengths and new tokens in a paged cache with pages dealt at random."""

    def __init__(self, heads, page, lens, new, cache=BF, pad=0, seed=0, extra_pages=2, scale=1.0, stride=0):
        self.H, self.G, self.d_h, self.d_r = H, G, d_h, d_r = heads
        self.page, self.lens, self.new, self.cache = page, list(lens), list(new), cache
        g = torch.Generator().manual_seed(seed)
        pages = [-(-L // page) for L in lens]
        self.num_pages = sum(pages) + extra_pages
        ids = torch.randperm(self.num_pages, generator=g).tolist()
        width = max(pages + [1])
        # behind a request's pages the table holds ids that must not be read
        self.table = np.full((len(lens), width + stride), 2 ** 30, dtype=np.int32)
        at = 0
        for b, k in enumerate(pages):
            self.table[b, :k] = ids[at:at + k]
            at += k
        self.width = width
        n = self.num_pages * page
        self.V = torch.randn(n, G, d_h, generator=g).to(cache)
        self.kr = torch.randn(n, d_r, generator=g).to(cache)
        used = np.zeros(n, dtype=bool)
        for b, L in enumerate(lens):
            for t in range(L):
                used[self.table[b, t // page] * page + t % page] = True
        for b, x in enumerate((self.V, self.kr)):       # slots of no token hold NaN and infinities
            x[torch.from_numpy(~used)] = float("nan") if b == 0 else float("inf")
        self.q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.rows = int(self.q_start[-1]) + pad
        c = scale * 1.4426950408889634 / np.sqrt(d_h)
        self.q = torch.randn(self.rows, H, d_h + d_r, generator=g) * c
        self.max_new, self.total = max(new + [1]), max(sum(lens), 1)

    def shape(self, out=F32, flags=0, ctas=0):
        return gva.make_shape(len(self.lens), self.H, self.G, self.d_h, self.d_h, self.d_r, cache_dtype=self.cache,
                              out_dtype=out, flags=flags, ctas_per_sm=ctas)

    def device(self):
        d = lambda x: torch.as_tensor(x).cuda()
        table = d(self.table)[:, :self.width]
        return dict(q=d(self.q), V=d(self.V), kr=d(self.kr) if self.d_r else None, table=table,
                    q_start=d(self.q_start), L=d(np.asarray(self.lens, dtype=np.int32)))

    def run(self, out=F32, flags=0, ctas=0, max_new=None, total=None, status=0, on=None):
        sh, t = self.shape(out, flags, ctas), on or self.device()
        max_new, total = max_new or self.max_new, total or self.total
        ws = gva.new_paged_workspace(sh, self.page, self.rows, max_new, total)
        ws[256:] = 0xff                                   # stale partials: NaN
        o = torch.full((self.rows, self.H, self.d_h), 3.25, dtype=out, device="cuda")
        lse = torch.full((self.rows, self.H), 3.25, device="cuda")
        gva.paged_attention(sh, self.page, t["q"], t["V"], t["kr"], t["table"], t["q_start"], t["L"], max_new, total, o,
                            lse, ws)
        torch.cuda.synchronize()
        assert gva.workspace_status(ws) == status
        return o.float().cpu().double().numpy(), lse.cpu().double().numpy()

    def reference(self):
        return serving_oracle.paged_attention(self.q.numpy(), self.V.double().numpy(), self.kr.double().numpy(),
                                              self.table[:, :self.width], self.page, self.q_start, self.lens, self.G)

    def check(self, got, ref, out, p_round, q_round=2.0 ** -16):
        o, lse = got
        ro, rl, mag = ref
        live = ~np.isnan(rl)
        assert np.all(o[~live] == 3.25) and np.all(lse[~live] == 3.25)     # rows of no request
        V = self.V.double().abs()
        V = torch.where(torch.isfinite(V), V, 0.0)
        K = self.kr.double().abs()
        K = torch.where(torch.isfinite(K), K, 0.0)
        q = self.q.double().abs()
        big = V.amax(0)                                                     # [G, d_h], over all slots
        S = torch.einsum("nhd,hd->nh", q[..., :self.d_h], big.repeat_interleave(self.H // self.G, 0)).numpy()
        if self.d_r:
            S = S + torch.einsum("nhr,r->nh", q[..., self.d_h:], K.amax(0)).numpy()
        e = np.log(2) * S * (q_round + (self.d_h + self.d_r + 2) * 2.0 ** -24)
        n = (max(self.lens) + 64) * 2.0 ** -24
        rel = np.exp(2 * e) - 1 + p_round + 2 * n + 2.0 ** -20
        half = 2.0 ** -8 if out == BF else 2.0 ** -24
        tol = mag * rel[..., None] + half * np.abs(ro) + 1e-30
        live3 = np.broadcast_to(live[..., None], ro.shape)
        assert np.all(np.isfinite(o[live3]))
        assert np.all(np.abs(o - ro)[live3] <= (tol * (1 + 2.0 ** -7))[live3])
        empty = live & np.isneginf(rl)
        assert np.all(np.isneginf(lse[empty])) and np.all(o[empty] == 0)
        seen = live & ~empty
        assert np.all(np.abs(lse[seen] - rl[seen]) <= e[seen] + n + 2.0 ** -20 + 2.0 ** -23 * np.abs(rl[seen]))


A, B24, C128, D32 = (16, 4, 64, 16), (16, 4, 64, 24), (32, 8, 128, 16), (8, 2, 32, 8)
MHA, WIDE, NOPE, R32 = (8, 8, 64, 16), (16, 2, 64, 32), (16, 4, 64, 0), (16, 8, 128, 32)
FMA = gva.FLAG_FMA_PATH

# new tokens fit 8 columns per group: the split-KV kernel
FEW = [
    (A, 16, [1, 15, 16, 17, 100], [1] * 5),
    (A, 8, [300, 41], [1, 1]), (A, 24, [300, 41, 47], [1, 1, 1]),          # 8-row boxes
    (A, 32, [700, 33, 64], [1, 0, 1]), (A, 256, [700, 33, 64], [1, 1, 1]),
    (A, 16, [0, 5, 0, 9], [1, 1, 0, 1]),                                   # a new token that sees nothing
    (A, 16, [1, 2, 3, 1], [2, 2, 2, 1]),                                   # 8 columns; the first token sees nothing
    (B24, 64, [1000, 2], [2, 1]), (C128, 16, [500, 129], [1, 1]), (C128, 128, [500, 129], [2, 1]),
    (D32, 16, [70, 200], [1, 2]), (MHA, 16, [90, 300], [1, 8]), (MHA, 16, [90, 300], [3, 1]),
    (WIDE, 16, [333], [1]), (NOPE, 16, [200, 31], [1, 2]), (R32, 48, [200, 31], [2, 1]),
    (A, 16, [37] * 40, [1] * 40), (A, 16, list(range(0, 99)), [1, 2, 0] * 33),
]


@pytest.mark.parametrize("case", range(len(FEW)))
@pytest.mark.parametrize("out", [F32, BF])
def test_few_new_tokens(case, out):
    x = Batch(*FEW[case], pad=case % 3, seed=case, stride=case % 2)
    ref = x.reference()
    x.check(x.run(out), ref, out, 2.0 ** -16)
    x.check(x.run(out, ctas=1), ref, out, 2.0 ** -16)        # another cut of the batch


# wide blocks: the tcgen05 kernel, alone (all requests alike) or beside the split-KV one
WIDE_BLOCKS = [
    (A, 16, [300], [3]), (A, 16, [130, 40], [32, 32]), (A, 8, [129, 200], [33, 33]),
    (A, 64, [500, 64, 63], [40, 40, 40]), (A, 24, [100], [100]),
    (A, 16, [300, 20, 7, 55], [1, 20, 0, 3]),                              # mixed with single tokens
    (B24, 32, [400, 90], [5, 5]), (B24, 32, [400, 90, 33], [5, 1, 33]),
    (C128, 64, [300, 150], [16, 16]), (C128, 16, [300, 150, 90], [40, 1, 7]), (R32, 128, [260], [64]),
    (MHA, 16, [200, 150], [130, 9]), (WIDE, 16, [64, 65, 66], [2, 2, 2]), (NOPE, 16, [90, 91], [30, 31]),
    (A, 16, [2, 0, 9], [5, 5, 5]),                                         # requests shorter than their chunk
    (A, 16, [12, 0, 9], [4, 5, 1]),
    (A, 256, [2000], [3]),                                                 # one block, split over the keys
    ((12, 4, 64, 8), 16, [100, 50], [50, 30]),                             # H/G = 3: rows straddle tokens
    ((20, 2, 64, 16), 16, [150, 60], [14, 1]),                             # H/G = 10: no split-KV kernel
]


@pytest.mark.parametrize("case", range(len(WIDE_BLOCKS)))
@pytest.mark.parametrize("out", [F32, BF])
def test_row_blocks(case, out):
    x = Batch(*WIDE_BLOCKS[case], pad=case % 3, seed=case, stride=case % 2)
    ref = x.reference()
    p = 2.0 ** -8 if out == BF else 2.0 ** -16
    x.check(x.run(out), ref, out, p)


# any shape on the CUDA cores
ANY = [
    (A, 16, [40, 0, 33], [1, 1, 7], BF), (C128, 16, [70, 32], [3, 20], BF), (A, 5, [40, 33], [1, 7], BF),
    (A, 1, [20, 3], [2, 3], BF), ((4, 2, 32, 8), 16, [64, 1, 100], [1, 2, 0], F32), ((4, 2, 32, 8), 3, [64, 9], [5, 9], F32),
    ((6, 2, 40, 4), 7, [50, 21], [4, 1], F32), ((6, 6, 12, 0), 16, [50], [17], F32), ((2, 1, 512, 128), 16, [40], [3], F32),
    ((24, 1, 64, 16), 16, [90], [2], BF), ((16, 4, 64, 48), 16, [40, 50], [1, 3], BF),
]


@pytest.mark.parametrize("case", range(len(ANY)))
@pytest.mark.parametrize("out", [F32, BF])
def test_cuda_cores(case, out):
    heads, page, lens, new, cache = ANY[case]
    x = Batch(heads, page, lens, new, cache=cache, pad=case % 3, seed=case)
    x.check(x.run(out, flags=FMA), x.reference(), out, 0.0, q_round=0.0)


def test_long_request_over_every_cta():
    for heads, page, n in ((A, 16, 1), (A, 64, 6), (C128, 16, 1)):
        x = Batch(heads, page, [20000], [n], seed=3)
        x.check(x.run(), x.reference(), F32, 2.0 ** -16)


def test_far_apart_scores():
    """Large scores: the running maximum moves by more than the lazy rescale's bound."""
    for new in ([1, 1], [20, 20]):
        x = Batch(A, 16, [400, 70], new, seed=4, scale=12.0)
        x.check(x.run(), x.reference(), F32, 2.0 ** -16)


def test_pages_outside_the_cache_read_as_zero():
    for new, flags in (([1, 1], 0), ([20, 3], 0), ([2, 3], FMA)):
        x = Batch(A, 16, [100, 70], new, seed=5)
        x.table[0, 2], x.table[1, 0], x.table[1, 4] = -1, x.num_pages, 2 ** 31 - 1
        ref = x.reference()
        got = x.run(flags=flags, status=gva.DEVERR_RANGE)
        x.check(got, ref, F32, 2.0 ** -16)


def test_request_longer_than_its_table_row():
    for new in ([1, 1], [20, 3]):
        x = Batch(A, 16, [112, 70], new, seed=6)              # whole pages: all 112 slots hold tokens
        x.lens = [120, 70]
        ref = x.reference()
        x.check(x.run(status=gva.DEVERR_RANGE), ref, F32, 2.0 ** -16)


def test_inconsistent_row_ranges_are_skipped():
    for new, flags in (([1, 2, 1], 0), ([20, 3, 9], 0), ([2, 3, 1], FMA)):
        x = Batch(A, 16, [50, 60, 40], new, seed=7)
        ref = x.reference()
        r0, r1 = x.q_start[1], x.q_start[2]
        for b in range(3):
            ref[b][r0:r1] = np.nan
        keep = x.q_start.copy()
        for length in (-3, x.num_pages * x.page + 1, 2 ** 31 - 1):   # negative; above all slots
            on = x.device()
            on["L"][1] = length
            x.check(x.run(flags=flags, status=gva.DEVERR_RANGE, on=on), ref, F32, 2.0 ** -16)
        on = x.device()
        on["q_start"][3] = x.rows + 1                         # leaves the buffers
        ref2 = x.reference()
        for b in range(3):
            ref2[b][keep[2]:] = np.nan
        x.check(x.run(flags=flags, status=gva.DEVERR_RANGE, on=on), ref2, F32, 2.0 ** -16)


def test_more_new_tokens_than_the_host_said():
    x = Batch(A, 16, [50, 60], [2, 1], seed=8)
    ref = x.reference()
    for b in range(3):
        ref[b][:2] = np.nan
    x.check(x.run(max_new=1, status=gva.DEVERR_RANGE), ref, F32, 2.0 ** -16)


def test_token_bound_far_from_the_batch():
    """A bound far above or below the batch's tokens changes the cut only."""
    for new in ([1, 2, 1], [20, 3, 20]):
        x = Batch(A, 16, [500, 60, 333], new, seed=9)
        ref = x.reference()
        for total in (10, 300000):
            x.check(x.run(total=total, max_new=64), ref, F32, 2.0 ** -16)


def test_cache_beyond_32_bit_offsets():
    """Pages in the last slots of a 9 GB cache: byte and element offsets pass 2^32."""
    page, n = 64, 1 << 24
    for new in ([1, 1], [20, 20]):
        x = Batch(A, page, [200, 70], new, seed=10)
        small = x.device()
        V = torch.empty(n + x.num_pages * page, 4, 64, dtype=BF, device="cuda")
        kr = torch.empty(n + x.num_pages * page, 16, dtype=BF, device="cuda")
        V[n:], kr[n:] = small["V"], small["kr"]
        small.update(V=V, kr=kr, table=small["table"] + n // page)
        x.check(x.run(on=small), x.reference(), F32, 2.0 ** -16)
        del V, kr, small


def test_same_result_every_time_and_in_graphs():
    """Bitwise: repeated calls, a captured call replayed on new lengths, other workspaces."""
    for new in ([1] * 6, [30, 1, 2, 9, 0, 30]):
        x = Batch(A, 16, [900, 31, 500, 64, 77, 300], new, pad=4, seed=11)
        t, sh = x.device(), x.shape(BF)
        o1, l1 = x.run(BF, on=t)
        o2, l2 = x.run(BF, on=t)
        assert np.array_equal(o1, o2) and np.array_equal(l1, l2)
        ws = gva.new_paged_workspace(sh, 16, x.rows, 32, 4000)
        out, lse = torch.zeros(x.rows, 16, 64, dtype=BF, device="cuda"), torch.zeros(x.rows, 16, device="cuda")
        go = lambda: gva.paged_attention(sh, 16, t["q"], t["V"], t["kr"], t["table"], t["q_start"], t["L"], 32, 4000, out,
                                         lse, ws)
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
            go()
        for cut in (0, 7, 25):
            y = Batch(A, 16, [900, 31, 500, 64, 77, 300], new, pad=4, seed=11)
            y.lens = [max(L - cut, 0) for L in y.lens]
            t["L"].copy_(torch.tensor(y.lens, dtype=I32))
            out.fill_(3.25)
            lse.fill_(3.25)
            graph.replay()
            torch.cuda.synchronize()
            y.check((out.float().cpu().double().numpy(), lse.cpu().double().numpy()), y.reference(), BF, 2.0 ** -8)
            assert gva.workspace_status(ws) == 0


def test_two_streams_at_once():
    """Two calls that may overlap, each with its own workspace."""
    xs = [Batch(A, 16, [3000, 500], n, seed=12 + i) for i, n in enumerate(([1, 1], [40, 40]))]
    ts = [x.device() for x in xs]
    shs = [x.shape(F32) for x in xs]
    wss = [gva.new_paged_workspace(s, 16, x.rows, x.max_new, x.total) for s, x in zip(shs, xs)]
    outs = [torch.zeros(x.rows, 16, 64, device="cuda") for x in xs]
    lses = [torch.zeros(x.rows, 16, device="cuda") for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, x in enumerate(xs):
            gva.paged_attention(shs[i], 16, ts[i]["q"], ts[i]["V"], ts[i]["kr"], ts[i]["table"], ts[i]["q_start"], ts[i]["L"],
                                x.max_new, x.total, outs[i], lses[i], wss[i], stream=streams[i])
    torch.cuda.synchronize()
    for x, o, l in zip(xs, outs, lses):
        x.check((o.cpu().double().numpy(), l.cpu().double().numpy()), x.reference(), F32, 2.0 ** -16)
