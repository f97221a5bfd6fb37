"""Draft verification against the request-by-request oracle: tokens and counts are whole
numbers and equal.  Sums are in 64 bits on both sides, so a drawn token could differ only
where u * sum lies within ~1e-15 of a running sum; the seeded inputs have no such row."""
import numpy as np
import pytest
import torch

from compressed_kv_cache_gva_b200 import gva
from oracle import serving_oracle

I32 = torch.int32


def make(ks, vocab, row, dtype=torch.float32, draft=True, seed=0, pad=0, sharp=2.0, near=0.5):
    """Probabilities of a target and a draft model near to it; drafts drawn from the draft."""
    g = torch.Generator().manual_seed(seed)
    n = torch.tensor([k + 1 for k in ks])   # k = -1: a request without rows
    q_start = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)])
    N = int(q_start[-1]) + pad
    logits = torch.randn(N, row, generator=g) * sharp
    target = torch.softmax(logits, -1).to(dtype)
    dr = torch.softmax(logits + near * torch.randn(N, row, generator=g), -1).to(dtype)
    race = torch.empty(N, row).exponential_(generator=g)
    drawn = (dr.float() / race)[:, :vocab].argmax(-1)
    tokens = torch.randint(0, vocab, (N,), generator=g)
    tokens[1:] = drawn[:-1]
    return dict(vocab=vocab, tokens=tokens.to(I32), q_start=q_start.to(I32), target=target,
                draft=dr if draft else None, u=torch.rand(N, generator=g), us=torch.rand(len(ks), generator=g),
                seq_len=torch.randint(50, 999, (len(ks),), generator=g).to(I32))


def run(s, err=0):
    d = lambda t: None if t is None else t.cuda()
    N, B = len(s["tokens"]), len(s["us"])
    out = torch.full((N,), -99, dtype=I32, device="cuda")
    acc, kept = torch.full((B,), 7, dtype=I32, device="cuda"), torch.full((B,), 7, dtype=I32, device="cuda")
    flag = torch.full((1,), err, dtype=I32, device="cuda")
    cols = s["target"].shape[1]
    target = d(s["target"])
    gva.verify_draft(s["vocab"], d(s["tokens"]), d(s["q_start"]), target, d(s["draft"]), d(s["u"]), d(s["us"]), out,
                     acc, d(s["seq_len"]), kept, flag)
    torch.cuda.synchronize()
    assert target.shape[1] == cols
    return out.tolist(), acc.tolist(), kept.tolist(), int(flag)


def same(s, err=0):
    out, acc, kept, flag = run(s)
    ref, racc, delta = serving_oracle.verify_draft(
        s["vocab"], s["tokens"].tolist(), s["q_start"].tolist(), s["target"].double().numpy(),
        None if s["draft"] is None else s["draft"].double().numpy(), s["u"].tolist(), s["us"].tolist())
    assert acc == racc
    assert out == [-99 if r is None else r for r in ref]     # rows of no request are left as they were
    assert kept == [int(L) + x for L, x in zip(s["seq_len"], delta)]
    assert flag == err
    return acc


def test_oracle_draws_from_the_target():
    """Over an even grid of the random numbers, the tokens of the oracle follow the target:
    P(x) = sum over drafts of q(d) [accepted and d = x, or redrawn x]."""
    p, q = np.array([0.1, 0.45, 0.05, 0.4]), np.array([0.3, 0.2, 0.25, 0.25])
    n = 400
    mass = np.zeros(4)
    for x in range(4):
        share = np.zeros(4)
        for i in range(n):
            u = (i + 0.5) / n
            if u * q[x] < p[x]:
                share[x] += 1 / n
            else:
                for j in range(50):
                    out, acc, _ = serving_oracle.verify_draft(4, [0, x], [0, 2], [p, p], [q, q], [u, 0], [(j + 0.5) / 50])
                    assert acc == [0]
                    share[out[0]] += 1 / n / 50
        mass += q[x] * share
    assert np.abs(mass - p).max() < 1 / 50 + 2 / n     # the grids' steps


@pytest.mark.parametrize("draft", [True, False])
def test_oracle_edges(draft):
    p = [[0.0, 0.25, 0.25, 0.5], [0.5, 0.5, 0.0, 0.0]]
    q = [[0.0, 1.0, 0.0, 0.0], [0.25] * 4] if draft else None
    # u = 0 accepts what the target can say, and the sample at u = 0.5 is the first token past it
    out, acc, delta = serving_oracle.verify_draft(4, [3, 1], [0, 2], p, q, [0.0, 0.0], [0.5])
    assert (out, acc, delta) == ([1, 1], [1], [0])
    out, acc, delta = serving_oracle.verify_draft(4, [3, 1], [0, 2], p, q, [0.9, 0.0], [0.0])
    assert (out, acc, delta) == ([2, -1], [0], [-1])


VOCABS = [(1, 1), (5, 5), (7, 9), (127, 128), (1000, 1000), (1001, 1003), (4097, 4099), (32768, 32768), (50021, 50048)]


@pytest.mark.gpu
@pytest.mark.parametrize("vocab,row", VOCABS)
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_verify_matches_oracle(vocab, row, draft, dtype):
    ks = [4, 0, 1, -1, 7, 3, 2] if vocab < 30000 else [3, 0, 5]
    same(make(ks, vocab, row, dtype, draft, seed=vocab, pad=2))


@pytest.mark.gpu
def test_batches_of_every_split():
    """From one request (a whole cluster each) to more requests than CTAs fit."""
    accepted = 0
    for B in (1, 2, 60, 170, 400, 1300):
        ks = np.random.default_rng(B).integers(-1, 6, B).tolist()
        accepted += sum(same(make(ks, 331, 332, seed=B)))
    assert accepted > 100


@pytest.mark.gpu
def test_long_drafts():
    same(make([300, 0, 700], 64, 64, seed=5, near=0.0))    # draft = target: everything is accepted


@pytest.mark.gpu
def test_rounds_down_to_no_residual():
    """Equal models refuse nothing with u < 1; where the draft is larger everywhere the token
    comes from the target itself."""
    s = make([2, 2], 40, 40, seed=6)
    s["draft"] = s["target"] * 4
    s["u"][:] = 0.99
    acc = same(s)
    assert acc == [0, 0]


@pytest.mark.gpu
def test_zero_weights_and_ends_of_the_unit_interval():
    s = make([1, 1, 1, 0, 0], 300, 300, seed=7)
    s["target"][:, :100] = 0
    s["target"][:, 200:] = 0
    s["us"][:] = torch.tensor([0.0, 1.0 - 2 ** -24, 1.0, 0.0, 1.0])
    same(s)
    out = run(s)[0]
    assert out[7] == 199                       # u = 1 gives the last token with any weight


@pytest.mark.gpu
def test_exact_borders():
    """Quarters: u * sum meets the running sums exactly, and the next token is taken."""
    s = make([0] * 5, 4, 4, seed=8)
    s["target"][:] = 0.25
    s["us"][:] = torch.tensor([0.0, 0.25, 0.5, 0.75, 0.9])
    same(s)
    assert run(s)[0] == [0, 1, 2, 3, 3]
    s = make([1], 4, 4, seed=9)                # u * q == p refuses
    s["target"][:], s["draft"][:], s["u"][:] = 0.25, 0.5, 0.5
    assert same(s) == [0]


@pytest.mark.gpu
def test_nan_and_negative_weights_count_as_zero():
    s = make([0, 1], 50, 64, seed=10)
    s["target"][:, 50:] = float("nan")         # behind the vocabulary: never read
    s["target"][:, 3] = float("nan")
    s["target"][:, 4] = -1.0
    s["tokens"][2] = 3                         # NaN refuses
    assert same(s) == [0, 0]


@pytest.mark.gpu
def test_flags():
    s = make([2, 2], 40, 40, seed=11)
    s["tokens"][1] = 40                        # outside the vocabulary: refused
    acc = same(s, err=gva.DEVERR_RANGE)
    assert acc[0] == 0
    s = make([0, 0], 40, 40, seed=12)
    s["target"][1] = 0                         # no probability at all
    out, _, _, flag = run(s)
    assert out[1] == 39 and flag == gva.DEVERR_RANGE
    s = make([1, 1], 40, 40, seed=13)
    s["q_start"] = torch.tensor([0, 2, 5], dtype=I32)     # past the rows
    out, acc, kept, flag = run(s)
    assert flag == gva.DEVERR_RANGE and acc[1] == 0 and kept[1] == int(s["seq_len"][1]) and out[2:] == [-99, -99]


@pytest.mark.gpu
def test_without_lengths_and_in_place():
    s = make([3, 2], 500, 500, seed=14)
    ref = run(s)
    d = lambda t: t.cuda()
    out, acc = torch.full((7,), -99, dtype=I32, device="cuda"), torch.zeros(2, dtype=I32, device="cuda")
    gva.verify_draft(500, d(s["tokens"]), d(s["q_start"]), d(s["target"]), d(s["draft"]), d(s["u"]), d(s["us"]), out, acc)
    assert out.tolist() == ref[0] and acc.tolist() == ref[1]
    lens = d(s["seq_len"])
    gva.verify_draft(500, d(s["tokens"]), d(s["q_start"]), d(s["target"]), d(s["draft"]), d(s["u"]), d(s["us"]), out, acc,
                     lens, lens)
    assert lens.tolist() == ref[2]
