"""Paged attention by ways that ordinary steps take and the cases of test_gpu_paged do not:
more than 32 requests in the row-block kernels (prefixes of the whole batch in shared memory),
the split-KV kernel beside the CUDA cores, shapes that fall to the CUDA cores by themselves, one
value group, many heads per group.  Bounds as in test_gpu_paged."""
import pytest
import torch

from compressed_kv_cache_gva_b200 import gva
from test_gpu_paged import A, B24, BF, C128, D32, F32, MHA, NOPE, WIDE, Batch
from test_gpu_paged_columns import SIXTEEN

pytestmark = pytest.mark.gpu
G1, G1W, TWELVE, TEN = (8, 1, 64, 16), (4, 1, 128, 16), (24, 2, 64, 16), (20, 2, 128, 16)

# new tokens that fill whole blocks of their request, that straddle blocks, none
MANY = [
    (A, 16, [20 + 3 * i for i in range(64)], [5] * 64),                     # drafts, row blocks alone
    (A, 16, [1 + 7 * i for i in range(33)], [min(1 + 7 * i, 40) for i in range(33)]),
    (B24, 32, [50 + i for i in range(100)], [5, 1, 0, 9] * 25),             # beside the split-KV kernel
    (C128, 64, [30 + 2 * i for i in range(40)], [20, 1, 3, 0] * 10),
    (NOPE, 8, [9 + i for i in range(70)], [9] * 70), (A, 16, [0, 5, 700] * 20, [0, 5, 40] * 20),
    (G1, 16, [30, 200, 7], [1, 2, 3]), (G1, 16, [40 + i for i in range(50)], [1, 17] * 25),
    (G1W, 64, [300, 41], [33, 1]), (G1W, 16, [20 + i for i in range(35)], [3] * 35),
    (TWELVE, 16, [300, 50], [1, 20]), (TWELVE, 16, [12 + i for i in range(60)], [1, 2, 11] * 20),
    (TEN, 16, [60 + i for i in range(45)], [1, 13, 0] * 15),
    ((6, 3, 64, 16), 16, [90, 20], [2, 5]),                                 # three groups: row blocks only
]


@pytest.mark.parametrize("case", range(len(MANY)))
@pytest.mark.parametrize("out", [F32, BF])
def test_row_blocks_of_many_requests(case, out):
    x = Batch(*MANY[case], pad=case % 3, seed=case, stride=case % 2)
    ref = x.reference()
    x.check(x.run(out), ref, out, 2.0 ** -8 if out == BF else 2.0 ** -16)
    x.check(x.run(out, ctas=1), ref, out, 2.0 ** -8 if out == BF else 2.0 ** -16)


# more than four blocks of a request, whose tiles are counted in closed form: heads per group
# odd and even, tiles of 64 keys (float32 output of d_h = 64) and of 128
CHUNKS = [(A, 16, [500, 41], [200, 41]), ((12, 4, 64, 8), 16, [600, 300], [300, 201]), ((10, 2, 64, 0), 32, [450], [333]),
          ((6, 2, 128, 16), 64, [700, 400], [300, 260]), ((8, 1, 128, 16), 16, [333], [150]), ((7, 1, 64, 8), 16, [333], [151])]


@pytest.mark.parametrize("case", range(len(CHUNKS)))
@pytest.mark.parametrize("out", [F32, BF])
def test_chunks_of_many_blocks(case, out):
    x = Batch(*CHUNKS[case], pad=case % 2, seed=case)
    x.check(x.run(out), x.reference(), out, 2.0 ** -8 if out == BF else 2.0 ** -16)


@pytest.mark.parametrize("heads,new", [((4, 1, 64, 16), [3, 4, 2, 0]), ((8, 2, 64, 16), [1] * 7 + [9])])
def test_the_largest_batch(heads, new):
    B = 4096
    new = (new * B)[:B]
    x = Batch(heads, 8, [max(n, i % 23) for i, n in enumerate(new)], new, seed=1)
    x.check(x.run(BF), x.reference(), BF, 2.0 ** -8)


# no flag: the shape, the type or the page leads to the CUDA cores
CORES = [
    ((4, 2, 32, 8), 16, [5 + 4 * i for i in range(40)], [1, 2, 0, 5] * 10, F32),
    ((4, 2, 64, 8), 16, [300, 17], [1, 16], F32), ((16, 4, 64, 16), 12, [100, 33], [1, 5], BF),
    ((16, 4, 64, 16), 1, [40, 33], [2, 9], BF), ((16, 4, 64, 16), 4, [30 + i for i in range(36)], [1, 3] * 18, BF),
    ((8, 4, 96, 16), 16, [90, 20], [1, 20], BF), ((4, 2, 256, 32), 16, [70, 33], [1, 7], BF),
    ((16, 4, 64, 40), 16, [90, 20], [1, 20], BF), ((10, 1, 32, 8), 16, [90, 20], [2, 5], BF),
]


@pytest.mark.parametrize("case", range(len(CORES)))
@pytest.mark.parametrize("out", [F32, BF])
def test_cuda_cores_without_the_flag(case, out):
    heads, page, lens, new, cache = CORES[case]
    x = Batch(heads, page, lens, new, cache=cache, pad=case % 3, seed=case)
    x.check(x.run(out), x.reference(), out, 0.0, q_round=0.0)


# d_h = 32 of a bf16 cache: no tcgen05 blocks, so chunks run on the CUDA cores beside the
# single tokens on the split-KV kernel
BESIDE = [
    ((8, 2, 32, 8), 16, [90, 200, 33, 64], [1, 40, 1, 0]), ((16, 4, 32, 24), 16, [90, 200, 33, 64], [2, 30, 1, 6]),
    ((8, 8, 32, 0), 8, [50 + i for i in range(40)], [1, 9, 1, 0] * 10), ((16, 2, 32, 16), 64, [4000, 300], [1, 5]),
]


@pytest.mark.parametrize("case", range(len(BESIDE)))
@pytest.mark.parametrize("out", [F32, BF])
def test_split_kv_beside_the_cuda_cores(case, out):
    x = Batch(*BESIDE[case], pad=case % 3, seed=case, stride=case % 2)
    ref = x.reference()
    a = x.run(out)
    x.check(a, ref, out, 2.0 ** -16)
    b = x.run(out)
    assert (a[0] == b[0]).all() and (a[1] == b[1]).all()


@pytest.mark.parametrize("case", range(len(SIXTEEN)))
def test_two_warps_per_group_keep_p_in_two_parts(case):
    """The bf16 output of 9 to 16 columns, to the bound of probabilities in two bf16 parts."""
    x = Batch(*SIXTEEN[case], pad=case % 3, seed=case, stride=case % 2)
    x.check(x.run(BF), x.reference(), BF, 2.0 ** -16)


@pytest.mark.parametrize("new,out", [([1, 1, 2], F32), ([20, 20, 1], BF)])
def test_requests_that_share_pages(new, out):
    """A common prefix: two requests name the same pages, a third the first of them."""
    x = Batch(A, 16, [100, 100, 64], new, seed=2)
    x.table[1] = x.table[0]
    x.table[2, :4] = x.table[0, :4]
    x.q[new[0]:2 * new[0]] = x.q[:new[0]]
    got = x.run(out)
    x.check(got, x.reference(), out, 2.0 ** -8 if out == BF else 2.0 ** -16)
