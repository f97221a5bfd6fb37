"""Paged attention of 9 to 16 query columns per value group (a few drafts per request): two
warps per group of the split-KV kernel, the second of them without work for requests of up to
8 columns.  Bounds as in test_gpu_paged; and row blocks at 17 columns and more, alone, ragged
and cut over the keys."""
import pytest
import torch

from test_gpu_paged import A, B24, BF, C128, D32, F32, MHA, NOPE, WIDE, Batch

pytestmark = pytest.mark.gpu

# d_h = 128 in two groups, H/G = 3 (columns straddle tokens and warps), H/G = 8, H/G = 1
G2, THREE, EIGHT, ONE = (8, 2, 128, 16), (12, 4, 64, 8), (16, 2, 64, 32), (4, 4, 64, 16)
SIXTEEN = [
    (A, 16, [300], [3]), (A, 16, [1, 15, 16, 17, 100], [1, 3, 4, 4, 4]), (A, 64, [700, 33, 64], [4, 1, 4]),
    (A, 16, [2, 0, 9, 3], [4, 3, 1, 4]),                                   # requests shorter than their drafts
    (A, 16, [37] * 40, [4] * 40), (A, 16, list(range(0, 99)), [1, 4, 0] * 33), (A, 256, [9000], [4]),
    (B24, 32, [400, 90], [3, 4]), (B24, 8, [401, 93, 64], [1, 3, 2]), (NOPE, 24, [90, 91], [3, 4]),
    (G2, 16, [300, 1000, 5], [4, 1, 4]), (G2, 128, [513, 40], [3, 3]), (D32, 16, [70, 200], [4, 3]),
    ((16, 4, 32, 0), 16, [70, 200, 1], [4, 3, 1]), ((16, 4, 32, 24), 40, [70, 200, 1], [4, 3, 1]),
    (THREE, 16, [100, 50, 64], [5, 4, 3]), (EIGHT, 16, [100, 50], [2, 1]), (ONE, 16, [90, 300], [16, 9]),
]


@pytest.mark.parametrize("case", range(len(SIXTEEN)))
@pytest.mark.parametrize("out", [F32, BF])
def test_nine_to_sixteen_columns(case, out):
    x = Batch(*SIXTEEN[case], pad=case % 3, seed=case, stride=case % 2)
    ref = x.reference()
    p = 2.0 ** -8 if out == BF else 2.0 ** -16
    got = x.run(out)
    x.check(got, ref, out, p)
    x.check(x.run(out, ctas=1), ref, out, p)                               # another cut of the batch
    again = x.run(out)
    assert (got[0] == again[0]).all() and (got[1] == again[1]).all()


# one more token than the split-KV kernel takes: 128-row blocks
BEYOND = [(A, 256, [2000], [5]), (A, 16, [300, 40], [5, 5]), (B24, 32, [400, 90], [5, 5]), (C128, 64, [3000], [3]),
          ((16, 4, 128, 16), 64, [900, 100], [3, 4]), (MHA, 16, [200, 150], [9, 16]), (WIDE, 16, [64, 65, 66], [3, 3, 3])]


@pytest.mark.parametrize("case", range(len(BEYOND)))
@pytest.mark.parametrize("out", [F32, BF])
def test_row_blocks_of_few_rows(case, out):
    x = Batch(*BEYOND[case], pad=case % 3, seed=case, stride=case % 2)
    x.check(x.run(out), x.reference(), out, 2.0 ** -8 if out == BF else 2.0 ** -16)


def test_one_bound_more_gives_the_same_rows():
    """The kernel is chosen by the host's bound on new tokens: a looser one sends drafts to
    row blocks, the results agree to both kernels' bounds."""
    x = Batch(A, 16, [500, 333, 64, 2], [4, 2, 3, 4], seed=5)
    ref = x.reference()
    for bound in (4, 5, 9):
        x.check(x.run(BF, max_new=bound), ref, BF, 2.0 ** -8)


def test_a_long_batch_of_mostly_single_tokens():
    """Above 96 MB of cache rows such a batch goes to two kernels side by side: the host's
    bound on tokens decides, so a bound that is far too large reaches that choice too."""
    x = Batch(A, 16, [37, 200, 64, 90, 1, 5], [1, 4, 1, 1, 1, 0], seed=6)
    ref = x.reference()
    for total in (None, 1 << 18):
        x.check(x.run(BF, total=total), ref, BF, 2.0 ** -8)
