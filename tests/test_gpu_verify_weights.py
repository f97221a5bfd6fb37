"""Draft verification of weights that are far from normalised: finite, but with sums of two
above the largest float, or all subnormal.  Tokens equal the oracle's.  Random numbers lie in
the middle of a token's share, so that no rounding of a sum (2^-48 of it) decides."""
import numpy as np
import pytest
import torch

from compressed_kv_cache_gva_b200 import gva
from oracle import serving_oracle

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.mark.parametrize("dtype,big", [(torch.float32, 3.4e38), (torch.bfloat16, 3.3e38), (torch.float32, 1.4e-45),
                                       (torch.bfloat16, 9.2e-41)])
@pytest.mark.parametrize("vocab", [1, 2, 9, 1000, 50021])
@pytest.mark.parametrize("kind", ["all", "residual", "copied"])
def test_finite_weights_of_any_size(dtype, big, vocab, kind):
    g = np.random.default_rng(vocab)
    B = 6
    # requests of two rows: the draft is refused (u = 1 - 2^-24 and a target of 0 there), or one row
    starts = [0]
    for b in range(B):
        starts.append(starts[-1] + (1 if kind == "all" else 2))
    N = starts[-1]
    target = torch.full((N, vocab), big).to(dtype)
    tokens = torch.from_numpy(g.integers(0, vocab, N).astype(np.int32))
    draft = None
    for b in range(B):
        r = starts[b]
        if kind != "all":
            target[r, tokens[r + 1]] = 0
    if kind == "residual":
        draft = torch.zeros(N, vocab, dtype=dtype)
        draft[:, ::3] = target[:, ::3] / 2 if big > 1 else 0    # (halves of powers of two below the largest)
        for b in range(B):
            draft[starts[b], tokens[starts[b] + 1]] = 1
    us = []
    for b in range(B):
        w = target[starts[b]].double().numpy().copy()
        if draft is not None:
            w = np.maximum(w - draft[starts[b]].double().numpy(), 0)
        if not w.any():
            w = target[starts[b]].double().numpy().copy()
        reach = np.cumsum(w)
        if reach[-1] == 0:
            us.append(0.5)
            continue
        v = int(g.choice(np.nonzero(w)[0]))
        us.append((reach[v] - w[v] / 2) / reach[-1])
    u_accept = np.full(N, 1 - 2.0 ** -24, np.float32)
    us = np.array(us, np.float32)
    d = lambda x: x.cuda() if torch.is_tensor(x) else torch.from_numpy(x).cuda()
    out, acc = torch.full((N,), 77, dtype=I32, device="cuda"), torch.zeros(B, dtype=I32, device="cuda")
    gva.verify_draft(vocab, d(tokens), d(np.array(starts, np.int32)), d(target), None if draft is None else d(draft),
                     d(u_accept), d(us), out, acc)
    ref, ref_acc, _ = serving_oracle.verify_draft(vocab, tokens.tolist(), starts, target.double().numpy(),
                                                  None if draft is None else draft.double().numpy(), u_accept.tolist(),
                                                  us.tolist())
    assert acc.tolist() == ref_acc
    assert out.tolist() == ref
