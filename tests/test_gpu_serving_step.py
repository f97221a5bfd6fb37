"""A server's steps over a paged cache, as a user strings the calls together: plan pages,
append, absorb, attend, verify drafts, plan again.  Every step's outputs are compared with
the float64 oracle on a contiguous copy of each request's cache (keys materialised, no
pages, no absorption), eagerly and as one captured graph replayed."""
import numpy as np
import pytest
import torch

import oracle
from oracle import serving_oracle
from compressed_kv_cache_gva_b200 import gva
from gpu_helpers import assert_close, lse_close

pytestmark = pytest.mark.gpu
I32, BF = torch.int32, torch.bfloat16
H, G, d_h, d_n, d_r, BASE = 16, 4, 64, 48, 16, 10000.0
PAGE, VOCAB = 16, 1003


class Server:
    """Device state of B requests, and the host's copy of what each has cached."""

    def __init__(self, B, pages, width, room, most, seed):
        self.B, self.room, self.most, self.g = B, room, most, torch.Generator().manual_seed(seed)
        z = lambda *s: torch.zeros(*s, dtype=I32, device="cuda")
        self.kept, self.n_new, self.held, self.table = z(B), z(B), z(B), z(B, width) - 1
        self.free, self.count = torch.arange(pages, dtype=I32, device="cuda"), z(1) + pages
        self.q_start, self.seq_len, self.granted = z(B + 1), z(B), z(B)
        self.slot, self.pos, self.err = z(room), z(room), z(1)
        self.pages = pages
        self.V = torch.full((pages * PAGE, G, d_h), float("nan"), dtype=BF, device="cuda")
        self.kr = torch.full((pages * PAGE, d_r), float("nan"), dtype=BF, device="cuda")
        self.M = (torch.randn(H, d_h, d_n, generator=self.g) / 8).to(BF)
        self.Md = self.M.cuda()
        f = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")
        self.q, self.v, self.kpe = f(room, H, d_n + d_r, dt=BF), f(room, G, d_h, dt=BF), f(room, d_r, dt=BF)
        self.q_abs, self.out, self.lse = f(room, H, d_h + d_r), f(room, H, d_h), f(room, H)
        self.tokens, self.out_tokens, self.acc = z(room), z(room), z(B)
        self.target, self.draft, self.u, self.us = f(room, VOCAB), f(room, VOCAB), f(room), f(B)
        self.sh = gva.make_shape(B, H, G, d_h, d_n, d_r)
        self.rows = gva.make_shape(room, H, G, d_h, d_n, d_r)
        self.ws = gva.new_paged_workspace(self.sh, PAGE, room, most, B * width * PAGE)
        self.bound = B * width * PAGE
        self.cached = [(np.zeros((0, G, d_h)), np.zeros((0, d_r))) for _ in range(B)]

    def calls(self):
        gva.plan_pages(PAGE, self.pages, self.kept, self.n_new, self.held, self.held, self.free, self.count, self.count,
                       self.table, self.q_start, self.seq_len, self.granted, self.slot, self.pos, self.err)
        gva.append_cache(self.sh, self.v, self.kpe, self.slot, self.pos, self.V, self.kr)
        gva.absorb_query(self.rows, self.q, self.Md, self.pos, self.q_abs)
        gva.paged_attention(self.sh, PAGE, self.q_abs, self.V, self.kr, self.table, self.q_start, self.seq_len, self.most,
                            self.bound, self.out, self.lse, self.ws)
        gva.verify_draft(VOCAB, self.tokens, self.q_start, self.target, self.draft, self.u, self.us, self.out_tokens,
                         self.acc, self.seq_len, self.kept, self.err)

    def draw(self, n_new):
        """New tokens' values, keys and queries, and the models' probabilities, for this step.
        Steps with a prompt keep all of their tokens (random numbers 0 accept every draft)."""
        g, r = self.g, self.room
        rnd = lambda t: t.copy_(torch.randn(t.shape, generator=g))
        for t in (self.q, self.v, self.kpe):
            rnd(t)
        logits = torch.randn(r, VOCAB, generator=g) * 2
        self.target.copy_(torch.softmax(logits, -1))
        dr = torch.softmax(logits + torch.randn(r, VOCAB, generator=g) * 0.4, -1)
        self.draft.copy_(dr)
        tok = torch.randint(0, VOCAB, (r,), generator=g)
        tok[1:] = torch.multinomial(dr, 1, generator=g)[:-1, 0]
        self.tokens.copy_(tok)
        self.u.copy_(torch.rand(r, generator=g) * (max(n_new) <= 8))
        self.us.copy_(torch.rand(self.B, generator=g))
        self.n_new.copy_(torch.tensor(n_new, dtype=I32))
        self.out.fill_(3.25)

    def check(self, before):
        """The step's outputs against the oracle; moves the host's copy on."""
        torch.cuda.synchronize()
        assert gva.workspace_status(self.ws) == 0 and int(self.err) & gva.DEVERR_RANGE == 0
        starts, got = self.q_start.tolist(), self.granted.tolist()
        f64 = lambda t: t.float().cpu().double().numpy()
        q, v, kpe, out, lse = f64(self.q), f64(self.v), f64(self.kpe), f64(self.out), f64(self.lse)
        for b in range(self.B):
            n, r0 = got[b], starts[b]
            V, K = (x[:before[b]] for x in self.cached[b])
            if n:
                slots = np.arange(before[b], before[b] + n, dtype=np.int32)
                pad = np.zeros((n,) + V.shape[1:]), np.zeros((n, d_r))
                V, K, _ = oracle.append_cache(np.concatenate([V, pad[0]]), np.concatenate([K, pad[1]]), v[r0:r0 + n],
                                              kpe[r0:r0 + n], slots, slots, BASE, "bf16")
                pos = np.arange(before[b], before[b] + n)[None]
                ref, rl = oracle.gva_decode_multi(q[None, r0:r0 + n], f64(self.M), pos, V, K, np.array([0]),
                                                  np.array([len(V)]), d_n, d_r, BASE)
                assert_close(out[r0:r0 + n], ref[0], "bf16", f"request {b}")
                lse_close(lse[r0:r0 + n], rl[0], f"request {b}")
            self.cached[b] = (V, K)
        assert np.all(out[starts[-1]:] == 3.25)
        ref, acc, delta = serving_oracle.verify_draft(VOCAB, self.tokens.tolist(), starts, f64(self.target),
                                                      f64(self.draft), self.u.tolist(), self.us.tolist())
        assert self.acc.tolist() == acc
        assert [t for t, r in zip(self.out_tokens.tolist(), ref) if r is not None] == [r for r in ref if r is not None]
        assert self.kept.tolist() == [L + d for L, d in zip(self.seq_len.tolist(), delta)]
        owned = [p for row, h in zip(self.table.tolist(), self.held.tolist()) for p in row[:h]]
        assert sorted(owned + self.free.tolist()[:int(self.count)]) == list(range(self.pages))
        for b, kept in enumerate(self.kept.tolist()):
            self.cached[b] = tuple(x[:kept] for x in self.cached[b])


STEPS = [
    [90, 40, 0, 5, 1],          # prompts
    [1, 1, 33, 1, 1],           # decode beside a prompt
    [5, 1, 4, 0, 3],            # drafts
    [1, 1, 1, 1, 1],
    [6, 6, 6, 6, 6],
]


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("pages,denied", [(60, False), (12, True)])
def test_steps_of_a_server(graph, pages, denied):
    s = Server(5, pages, 12, 160, 90, seed=3)
    g = None
    if graph:
        s.calls()               # attributes are set outside the capture; no request has tokens yet
        torch.cuda.synchronize()
        side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
            s.calls()
    seen = 0
    for n_new in STEPS:
        s.draw(n_new)
        s.err.zero_()
        before = s.kept.tolist()
        g.replay() if graph else s.calls()
        s.check(before)
        seen |= int(s.err) & gva.DEVERR_PAGES
    assert bool(seen) == denied
    # every request ends: all pages come back
    s.kept.zero_()
    s.n_new.zero_()
    gva.plan_pages(PAGE, s.pages, s.kept, s.n_new, s.held, s.held, s.free, s.count, s.count, s.table, s.q_start, s.seq_len,
                   s.granted, s.slot, s.pos, s.err)
    assert int(s.count) == s.pages and sorted(s.free.tolist()) == list(range(s.pages))
