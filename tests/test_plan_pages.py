"""The page plan against the request-by-request oracle: whole numbers, so every output
is equal, entry by entry."""
import numpy as np
import pytest
import torch

from compressed_kv_cache_gva_b200 import gva
from oracle import serving_oracle

I32 = torch.int32


def make(B, page, max_len, n_hi, spare, room=None, seed=0, max_pages=None, n_lo=0, idle=0.2):
    """A server's state before a step: requests of random lengths, pages dealt at random."""
    g = np.random.default_rng(seed)
    kept = g.integers(0, max_len + 1, B)
    n = np.where(g.random(B) < idle, 0, g.integers(n_lo, n_hi + 1, B))
    held = -(-(kept + g.integers(0, 2 * page + 3, B)) // page)
    width = max_pages or int(-(-(max_len + max(n_hi, 2 * page + 3)) // page))
    held = np.minimum(held, width)
    kept = np.minimum(kept, held * page)
    used = int(held.sum())
    ids = g.permutation(used + spare).astype(np.int32)
    table = np.full((B, width), -7, dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = np.full(used + spare, -9, dtype=np.int32)
    free[:spare] = ids[used:]
    return dict(page=page, num_pages=used + spare, kept=kept.tolist(), n=n.tolist(), held=held.tolist(), free=free,
                count=spare, table=table, room=int(n.sum()) if room is None else room)


def run(s, in_place=False, stride=0, err=0):
    dev = lambda x: torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()
    B, width = s["table"].shape
    wide = torch.full((B, width + stride), -5, dtype=I32, device="cuda")
    wide[:, :width] = dev(s["table"])
    table = wide[:, :width]
    free, held_in, count_in = dev(s["free"]), dev(s["held"]), dev([s["count"]])
    z = lambda k: torch.full((k,), 77, dtype=I32, device="cuda")
    held = held_in if in_place else z(B)
    count = count_in if in_place else z(1)
    o = dict(q_start=z(B + 1), seq_len=z(B), n_granted=z(B), slot=z(s["room"]), pos=z(s["room"]))
    flag = torch.full((1,), err, dtype=I32, device="cuda")
    gva.plan_pages(s["page"], s["num_pages"], dev(s["kept"]), dev(s["n"]), held_in, held, free, count_in, count,
                   table, o["q_start"], o["seq_len"], o["n_granted"], o["slot"], o["pos"], flag)
    torch.cuda.synchronize()
    if stride:
        assert bool((wide[:, width:] == -5).all())   # between the rows nothing is written
    o = {k: v.tolist() for k, v in o.items()}
    o.update(held=held.tolist(), free=free.tolist(), count=int(count), table=table.tolist(), err=int(flag))
    return o


def want(s):
    return serving_oracle.plan_pages(s["page"], s["num_pages"], s["kept"], s["n"], s["held"], s["free"].tolist(),
                                     s["count"], s["table"].tolist(), s["room"])


def same(s, **kw):
    got, ref = run(s, **kw), want(s)
    for k in ref:
        assert got[k] == ref[k], k
    return ref


CASES = [
    # B, page, longest kept, most new tokens, free pages
    (1, 16, 100, 1, 1),
    (3, 1, 9, 4, 30),            # one token per page
    (5, 12, 200, 40, 25),        # a page size that is no power of two
    (31, 16, 500, 3, 40), (33, 16, 500, 3, 40),
    (64, 64, 1000, 130, 10),     # the list runs out
    (300, 16, 3000, 8, 300), (513, 8, 60, 70, 200), (1025, 32, 800, 9, 400), (4096, 16, 100, 6, 900),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_matches_oracle(case, in_place):
    B, page, max_len, n_hi, spare = case
    for seed in range(3):
        same(make(B, page, max_len, n_hi, spare, seed=seed), in_place=in_place, stride=3 * seed)


@pytest.mark.gpu
def test_many_new_tokens():
    ref = same(make(7, 16, 5000, 9000, 4000, seed=4, idle=0.0))
    assert len(ref["slot"]) > 4096


@pytest.mark.gpu
@pytest.mark.parametrize("B", [40, 700])
def test_denied_requests_keep_what_they_hold(B):
    s = make(B, 16, 300, 50, 3, seed=1)
    ref = same(s)
    assert ref["err"] == gva.DEVERR_PAGES and any(n and not g for n, g in zip(s["n"], ref["n_granted"]))
    s = make(B, 16, 300, 50, 500, seed=2, room=B * 10)   # pages enough, token room short
    ref = same(s)
    assert ref["err"] == gva.DEVERR_PAGES


@pytest.mark.gpu
@pytest.mark.parametrize("B", [4, 600])
def test_inconsistent_requests(B):
    s = make(B, 16, 100, 4, 4 * B, seed=3)
    s["kept"][0] = -1
    s["n"][1] = -2
    s["kept"][2] = s["held"][2] * 16 + 1             # more tokens than its pages hold
    s["n"][3] = s["table"].shape[1] * 16 + 1         # longer than its table row
    s["room"] = sum(n for b, n in enumerate(s["n"]) if b > 3)
    ref = same(s)
    assert ref["err"] == gva.DEVERR_RANGE
    assert run(s, err=2)["err"] == gva.DEVERR_RANGE | 2      # or-ed, never cleared


@pytest.mark.gpu
@pytest.mark.parametrize("count", [-1, 10 ** 6])
def test_free_list_that_cannot_be_right(count):
    s = make(20, 16, 100, 4, 30, seed=5)
    s["count"] = count
    ref = same(s)
    assert ref["err"] & gva.DEVERR_RANGE and not any(ref["n_granted"])


@pytest.mark.gpu
def test_bad_page_ids_give_no_slot():
    s = make(6, 16, 200, 5, 40, seed=6, idle=0.0, n_lo=1)
    s["table"][:] = np.where(s["table"] >= 0, s["num_pages"] + 3, s["table"])
    s["free"][:s["count"]] = -4
    ref = same(s)
    assert ref["err"] & gva.DEVERR_RANGE and set(ref["slot"]) == {-1}


@pytest.mark.gpu
def test_release_everything_and_empty_batch():
    s = make(50, 16, 400, 4, 0, seed=7)
    s["kept"], s["n"], s["room"] = [0] * 50, [0] * 50, 5
    ref = same(s)
    assert ref["count"] == s["num_pages"] and not any(ref["held"])
    assert sorted(ref["free"]) == list(range(s["num_pages"]))
    one = torch.zeros(1, dtype=I32, device="cuda")
    none = torch.zeros(0, dtype=I32, device="cuda")
    q, slot, pos, count = one + 9, torch.zeros(3, dtype=I32, device="cuda"), torch.zeros(3, dtype=I32, device="cuda"), one + 9
    gva.plan_pages(16, 4, none, none, none, none, torch.zeros(4, dtype=I32, device="cuda"), one + 2, count,
                   torch.zeros(0, 1, dtype=I32, device="cuda"), q, none, none, slot, pos)
    assert q.tolist() == [0] and slot.tolist() == pos.tolist() == [-1] * 3 and count.tolist() == [2]


@pytest.mark.gpu
def test_steps_in_a_captured_graph():
    """Plan in place, drafts rejected, plan again, replayed: pages are conserved."""
    s = make(48, 16, 600, 6, 400, seed=8)
    dev = lambda x: torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()
    B, room = 48, 512
    kept, n, held = dev(s["kept"]), dev(s["n"]), dev(s["held"])
    free, count, table = dev(s["free"]), dev([s["count"]]), dev(s["table"])
    z = lambda k: torch.zeros(k, dtype=I32, device="cuda")
    q_start, seq_len, granted, slot, pos, err = z(B + 1), z(B), z(B), z(room), z(room), z(1)
    go = lambda: gva.plan_pages(16, s["num_pages"], kept, n, held, held, free, count, count, table, q_start, seq_len,
                                granted, slot, pos, err)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            go()
    rng = np.random.default_rng(0)
    state = dict(s)
    for step in range(6):
        state["kept"] = [min(k, h * 16) for k, h in zip(state["kept"], state["held"])]
        state["n"] = rng.integers(0, 8, B).tolist()
        state["room"] = room
        kept.copy_(dev(state["kept"]))
        n.copy_(dev(state["n"]))
        graph.replay()
        torch.cuda.synchronize()
        ref = want(state)
        assert slot.tolist() == ref["slot"] and table.tolist() == ref["table"] and int(count) == ref["count"]
        assert held.tolist() == ref["held"] and free.tolist()[:ref["count"]] == ref["free"][:ref["count"]]
        owned = [p for b, r in enumerate(ref["table"]) for p in r[:ref["held"][b]]]
        assert sorted(owned + ref["free"][:ref["count"]]) == list(range(s["num_pages"]))
        state.update(held=ref["held"], free=np.asarray(ref["free"]), count=ref["count"], table=np.asarray(ref["table"]),
                     kept=[max(0, L - int(x)) for L, x in zip(ref["seq_len"], rng.integers(0, 3, B))])
