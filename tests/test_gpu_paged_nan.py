"""Paged attention of queries that hold a NaN or an infinity: their rows of out and lse are
NaN whether or not the request is cut between CTAs, and every other row is what it is without
them, bit by bit.  A row that sees no key stays 0 and -inf whatever its query holds."""
import numpy as np
import pytest

from test_gpu_paged import A, BF, C128, D32, F32, FMA, Batch

pytestmark = pytest.mark.gpu

# (heads, page, lengths, new tokens, cache, flags): short requests, which one CTA covers, and
# long ones, which are cut
CASES = [
    (A, 16, [40, 30], [1, 1], BF, 0), (A, 64, [9000, 700], [1, 2], BF, 0), (A, 64, [9000, 700], [4, 3], BF, 0),
    (C128, 64, [4000, 40], [1, 2], BF, 0), (A, 16, [40, 30], [20, 9], BF, 0), (A, 64, [5000, 700], [5, 5], BF, 0),
    (A, 64, [3000, 700], [70, 1], BF, 0), (C128, 64, [3000, 700], [20, 1], BF, 0),
    (D32, 16, [700, 90], [1, 3], F32, 0), (A, 16, [700, 90], [3, 20], BF, FMA),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("out", [F32, BF])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_rows_of_a_nan_or_infinite_query(case, out, value):
    heads, page, lens, new, cache, flags = CASES[case]
    x = Batch(heads, page, lens, new, cache=cache, pad=1, seed=case)
    H, dq = x.H, x.d_h + x.d_r
    want_o, want_l = x.run(out, flags=flags)
    hit = np.zeros((x.rows, H), dtype=bool)
    # two heads of one group, one in another group, in the first and the last new token; the
    # value slice of the query and, where there is one, the positional slice
    for row, head, col in ((0, 0, 3), (0, H - 1, dq - 1), (x.rows - 2, 1, 0)):
        x.q[row, head, col] = value
        hit[row, head] = True
    o, lse = x.run(out, flags=flags)
    assert np.all(np.isnan(o[hit])) and np.all(np.isnan(lse[hit]))
    assert np.array_equal(o[~hit], want_o[~hit]) and np.array_equal(lse[~hit], want_l[~hit])


@pytest.mark.parametrize("new,lens,flags", [([4, 1], [2, 9], 0), ([40, 9], [3, 50], 0), ([4, 20], [2, 50], FMA)])
def test_a_nan_query_that_sees_no_key(new, lens, flags):
    x = Batch(A, 16, lens, new, seed=1)
    x.q[0] = float("nan")                 # the request counts fewer tokens than it brings
    o, lse = x.run(flags=flags)
    assert np.all(o[0] == 0) and np.all(np.isneginf(lse[0]))
