"""The piece walk of test_paged_model at the cut of the d_h = 128 row blocks (tiles of 128 keys,
a piece's fixed cost of four tiles) and over batches of more than 32 requests."""
import numpy as np
import pytest

from test_paged_model import cta_of, tiles, units, walk


@pytest.mark.parametrize("M,TK,OV", [(128, 128, 4), (128, 128, 3), (128, 64, 3), (16, 32, 1)])
@pytest.mark.parametrize("seed", range(12))
def test_every_tile_once_and_every_piece_merged(M, TK, OV, seed):
    rng = np.random.default_rng(100 * OV + seed)
    G, hpr = int(rng.choice([1, 2, 4, 8])), int(rng.choice([1, 3, 4, 10]))
    grid = int(rng.choice([1, 3, 148, 296]))
    hi = int(rng.choice([1, 5, 200]))
    B = int(rng.choice([3, 20, 80]))
    seqs = [(int(rng.integers(0, hi + 1)), int(rng.integers(0, 3000))) for _ in range(B)]
    NT = sum(units(n, L, G, hpr, M, TK, OV) for n, L in seqs)
    seen, slots, meta, blocks = {}, {}, {}, {}
    for cta, item, k0, k1, nt, u in walk(seqs, G, hpr, M, TK, OV, grid):
        assert 0 <= k0 < k1 <= nt
        blocks[item] = nt
        for k in range(k0, k1):
            assert (item, k) not in seen
            seen[item, k] = cta
        if k1 - k0 < nt:
            slot = 2 * cta + (1 if k0 == 0 else 0)
            assert slot not in slots and slot < 2 * grid
            slots[slot] = (item, k0, k1)
            if k0 == 0:
                assert cta not in meta
                meta[cta] = (cta_of(u + OV + nt - 1, NT, grid) - cta + 1, item, nt)
    want = {(b, g, rb): tiles(*seqs[b], hpr, rb, M, TK)
            for b, (n, L) in enumerate(seqs) for g in range(G) for rb in range(-(-n * hpr // M))}
    assert blocks == want and len(seen) == sum(want.values())
    merged = set()
    for i, (count, item, nt) in meta.items():
        at = 0
        for c in range(count):
            s = 2 * i + 1 if c == 0 else 2 * (i + c)
            it, k0, k1 = slots[s]
            assert it == item and k0 == at
            at = k1
            merged.add(s)
        assert at == nt
    assert merged == set(slots)


def steps_below(x, h):
    q = x // h
    return h * (q * (q - 1) // 2) + q * (x - q * h)


def line_floors(M, TK, n, h, b):
    """Sum over i < n of (M i + b) // (h TK), in the kernels' closed form."""
    if TK % M == 0:
        c, p = b // M, h * (TK // M)
        return steps_below(c + n, p) - steps_below(c, p)
    c = b // TK
    if h % 2 == 0:
        return steps_below(c // 2 + n, h // 2) - steps_below(c // 2, h // 2)
    last, y0, p = c + 2 * n, 0 if c % 2 else h, 2 * h
    higher = (last + p - y0) // p - (c + p - y0) // p
    total = steps_below(last, h) - steps_below(c, h) - higher
    assert total % 2 == 0
    return total // 2


@pytest.mark.parametrize("M,TK", [(128, 64), (128, 128), (16, 32)])
@pytest.mark.parametrize("h", [1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 33, 64])
def test_tiles_of_a_sequence_without_a_loop(M, TK, h):
    rng = np.random.default_rng(h)
    for _ in range(150):
        n = int(rng.integers(1, 3000))
        L = n + int(rng.integers(0, 20000))
        nb = -(-n * h // M)
        got = line_floors(M, TK, nb - 1, h, M - 1 + h * (L - n + TK))
        assert got == sum(tiles(n, L, h, rb, M, TK) for rb in range(nb - 1))
        b, k = int(rng.integers(0, 10 ** 6)), int(rng.integers(0, 200))
        assert line_floors(M, TK, k, h, b) == sum((M * i + b) // (h * TK) for i in range(k))
