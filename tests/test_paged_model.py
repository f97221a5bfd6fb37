"""The paged kernels' work list, restated on the CPU: every tile of every row block is
processed once, a CTA leaves at most one block it did not start and one it does not end,
and the merge finds exactly the pieces that were written."""
import numpy as np
import pytest


def kv_end(n, L, hpr, rb, M):
    return max(0, L - n + min(n - 1, ((rb + 1) * M - 1) // hpr) + 1)


def tiles(n, L, hpr, rb, M, TK):
    return max(1, -(-kv_end(n, L, hpr, rb, M) // TK))


def first(i, NT, grid):
    g = min(grid, NT) if NT > 0 else 1
    return min(i, g) * NT // g


def cta_of(u, NT, grid):
    g = min(grid, NT)
    return ((u + 1) * g - 1) // NT


def units(n, L, G, hpr, M, TK, OV):
    return G * sum(tiles(n, L, hpr, rb, M, TK) + OV for rb in range(-(-n * hpr // M)))


def walk(seqs, G, hpr, M, TK, OV, grid):
    """(cta, item, k0, k1, nt, u) of every piece, following the kernel's walk: a block counts
    OV + nt units from u on, its tiles the last nt of them."""
    prefix = [0]
    for n, L in seqs:
        prefix.append(prefix[-1] + units(n, L, G, hpr, M, TK, OV))
    NT = prefix[-1]
    for cta in range(grid):
        at, end = first(cta, NT, grid), first(cta + 1, NT, grid)
        if at >= end:
            continue
        b = next(i for i in range(len(seqs)) if prefix[i + 1] > at)
        rem, rb = at - prefix[b], 0
        while True:
            nt = tiles(*seqs[b], hpr, rb, M, TK)
            if rem < G * (nt + OV):
                break
            rem, rb = rem - G * (nt + OV), rb + 1
        g, rem = rem // (nt + OV), rem % (nt + OV)
        u, k0 = at - rem, max(0, rem - OV)
        while True:
            k1 = min(nt, end - u - OV)
            if k1 <= k0:
                break
            yield cta, (b, g, rb), k0, k1, nt, u
            u += OV + nt
            if u >= end:
                break
            k0, g = 0, g + 1
            if g == G:
                g, rb = 0, rb + 1
                if rb == -(-seqs[b][0] * hpr // M):
                    rb, b = 0, b + 1
                    while seqs[b][0] == 0:
                        b += 1
                nt = tiles(*seqs[b], hpr, rb, M, TK)


@pytest.mark.parametrize("seed", range(40))
def test_row_blocks_and_pieces(seed):
    rng = np.random.default_rng(seed)
    G, hpr = int(rng.choice([1, 2, 4, 8])), int(rng.choice([1, 3, 4, 10]))
    M, TK, OV = [(128, 64, 3), (128, 128, 3), (16, 32, 1)][seed % 3]
    grid = int(rng.choice([1, 3, 148, 296]))
    hi = int(rng.choice([1, 5, 200]))
    seqs = [(int(rng.integers(0, hi + 1)), int(rng.integers(0, 4000))) for _ in range(int(rng.integers(1, 20)))]
    seen, slots, meta, blocks = {}, {}, {}, {}
    NT = sum(units(n, L, G, hpr, M, TK, OV) for n, L in seqs)
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
    want = {(b, g, rb) for b, (n, L) in enumerate(seqs) for g in range(G) for rb in range(-(-n * hpr // M))}
    assert set(blocks) == want
    assert len(seen) == sum(blocks.values())
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


def test_every_query_row_and_key_is_in_a_block():
    for n, hpr, M in ((1, 4, 128), (32, 4, 128), (33, 4, 128), (50, 3, 128), (14, 10, 16), (7, 1, 16)):
        for L in (0, 1, n - 1, n, n + 1, 500):
            rows = set()
            for rb in range(-(-n * hpr // M)):
                end = kv_end(n, L, hpr, rb, M)
                assert end <= max(L, 0)
                for r in range(min(M, n * hpr - rb * M)):
                    R = rb * M + r
                    rows.add(R)
                    assert L - n + R // hpr + 1 <= max(end, 0)   # the row's keys lie in the block's
            assert rows == set(range(n * hpr))


def floor_sum(n, m, a, b):
    """Sum over i < n of (a i + b) // m, by the kernel's recursion."""
    s = 0
    while True:
        if a >= m:
            s += n * (n - 1) // 2 * (a // m)
            a %= m
        if b >= m:
            s += n * (b // m)
            b %= m
        y = a * n + b
        if y < m:
            return s
        n, b, m, a = y // m, y % m, a, m


@pytest.mark.parametrize("hpr", [1, 3, 4, 10, 64])
def test_tiles_of_a_sequence_in_closed_form(hpr):
    rng = np.random.default_rng(hpr)
    for _ in range(300):
        M, TK = [(128, 64), (128, 128), (16, 32)][int(rng.integers(3))]
        n = int(rng.integers(1, 3000))
        L = n + int(rng.integers(0, 20000))
        nb = -(-n * hpr // M)
        got = floor_sum(nb - 1, hpr * TK, M, M - 1 + hpr * (L - n + TK)) if nb > 1 else 0
        assert got == sum(tiles(n, L, hpr, rb, M, TK) for rb in range(nb - 1))


@pytest.mark.parametrize("page", [8, 16, 24, 32, 40, 64, 128, 256])
@pytest.mark.parametrize("tile", [16, 32, 64, 128])
def test_boxes_stay_in_their_page(page, tile):
    log2 = 0
    while (2 << log2) <= tile and page % (2 << log2) == 0:
        log2 += 1
    box = 1 << log2
    assert box >= 8 and tile % box == 0 and page % box == 0 and 32 % (tile // box) == 0
    for i in range(4 * tile // box * 33):
        t = i << log2
        assert t // page == (t + box - 1) // page      # one page per box
