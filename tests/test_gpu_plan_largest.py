"""The page plan at the largest counts its arguments allow: 2^31 - 1 pages of one token, all
taken by one request and all returned, and as many token slots.  Loop counters pass 2^31 on
their last step."""
import pytest
import torch

from compressed_kv_cache_gva_b200 import gva

pytestmark = pytest.mark.gpu
I32, N, GUARD = torch.int32, 2 ** 31 - 1, 64


def guarded(n):
    """n words between guard words."""
    whole = torch.full((n + 2 * GUARD,), 77, dtype=I32, device="cuda")
    return whole, whole[GUARD:GUARD + n]


def pieces(n, step=1 << 28):
    return [(a, min(a + step, n)) for a in range(0, n, step)]


def counting(a, b):
    return torch.arange(a, b, dtype=I32, device="cuda")


def test_all_pages_taken_and_returned():
    i = lambda *v: torch.tensor(v, dtype=I32, device="cuda")
    (f_all, free), (s_all, slot), (p_all, pos), (t_all, table) = (guarded(N) for _ in range(4))
    for a, b in pieces(N):
        free[a:b] = counting(a, b)
    z = lambda k: torch.zeros(k, dtype=I32, device="cuda")
    held, count, q_start, seq_len, got, err = i(0), i(N), z(2), z(1), z(1), z(1)
    gva.plan_pages(1, N, i(0), i(N), held, held, free, count, count, table[None], q_start, seq_len, got, slot, pos, err)
    assert [t.tolist() for t in (held, count, q_start, seq_len, got, err)] == [[N], [0], [0, N], [N], [N], [0]]
    for a, b in pieces(N):
        want = N - 1 - counting(a, b)                       # taken from the top of the list
        assert torch.equal(table[a:b], want) and torch.equal(slot[a:b], want)
        assert torch.equal(pos[a:b], counting(a, b))
    # the request ends; room for 5000 tokens, none of which come
    s2, p2 = slot[:5000], pos[:5000]
    free.fill_(-9)
    gva.plan_pages(1, N, i(0), i(0), held, held, free, count, count, table[None], q_start, seq_len, got, s2, p2, err)
    assert [t.tolist() for t in (held, count, q_start, seq_len, got, err)] == [[0], [N], [0, 0], [0], [0], [0]]
    assert (s2 == -1).all() and (p2 == -1).all()
    for a, b in pieces(N):
        assert torch.equal(free[a:b], N - 1 - counting(a, b))
    for whole in (f_all, s_all, p_all, t_all):
        assert (whole[:GUARD] == 77).all() and (whole[-GUARD:] == 77).all()


def test_room_for_far_more_tokens_than_come():
    i = lambda *v: torch.tensor(v, dtype=I32, device="cuda")
    (s_all, slot), (p_all, pos) = guarded(N), guarded(N)
    z = lambda k: torch.zeros(k, dtype=I32, device="cuda")
    q_start, seq_len, got, err, table = z(4), z(3), z(3), z(1), z((3, 2)) - 1
    gva.plan_pages(4, 6, i(0, 0, 0), i(5, 0, 3), z(3), z(3), counting(0, 6), i(6), z(1), table, q_start, seq_len, got, slot,
                   pos, err)
    assert slot[:8].tolist() == [20, 21, 22, 23, 16, 12, 13, 14] and pos[:8].tolist() == [0, 1, 2, 3, 4, 0, 1, 2]
    assert int(err) == 0
    for a, b in pieces(N):
        a = max(a, 8)
        assert (slot[a:b] == -1).all() and (pos[a:b] == -1).all()
    for whole in (s_all, p_all):
        assert (whole[:GUARD] == 77).all() and (whole[-GUARD:] == 77).all()
