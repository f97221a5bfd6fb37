"""Cases and plain forms of the paged serving operators.

Three operators make up one step of a server that keeps the GVA cache in pages:

  plan    request lengths -> block tables, slots and positions of the new tokens
          (pages are taken from and returned to a free list on the GPU);
  attend  attention of each request's new tokens, one or a chunk, over its pages;
  verify  drafted tokens against the target model's probabilities from given
          random numbers, and the one token that follows them.

`run` computes a case in elementary torch operations, or, with `own`, through the
library.  `exact` computes the definition in 64 bits.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _d(t):
    return t.to("cuda")


def _ints(values):
    return torch.tensor(values, dtype=torch.int32)


# ---------------------------------------------------------------------------- cases

def _plan(name, **kw):
    return dict(name=name, op="plan", **kw)


def _attend(name, **kw):
    return dict(name=name, op="attend", **kw)


def _verify(name, **kw):
    return dict(name=name, op="verify", **kw)


def listed():
    return [
        # the scheduler's work before every decode step of a small batch: one new token each
        _plan("plan_b8", B=8, page=16, max_len=4096, new_lo=1, new_hi=1, long_every=0, long_hi=0, spare=8),
        # a full server: drafts of up to 8 tokens, every 16th request a prompt chunk, and too few
        # free pages for the last of them
        _plan("plan_b2048", B=2048, page=16, max_len=8192, new_lo=1, new_hi=8, long_every=16, long_hi=512,
              spare=1500),
        # one token per request, the 350M-class heads: latency of the smallest step
        _attend("decode_b8_t4096", B=8, H=16, G=4, d_h=64, d_r=16, page=16, len_lo=4096, len_hi=4096,
                new_lo=1, new_hi=1, long_every=0, long_hi=0, pad=0, cache="bf16", out="f32"),
        # ragged serving batch, one token per request, a batch padded to a captured size
        _attend("decode_b64_1k_16k", B=64, H=16, G=4, d_h=64, d_r=16, page=64, len_lo=1024, len_hi=16384,
                new_lo=1, new_hi=1, long_every=0, long_hi=0, pad=5, cache="bf16", out="bf16"),
        # one request with a very long context, large-model heads
        _attend("decode_b1_t131072", B=1, H=32, G=8, d_h=128, d_r=16, page=128, len_lo=131072,
                len_hi=131072, new_lo=1, new_hi=1, long_every=0, long_hi=0, pad=0, cache="bf16", out="f32"),
        # verification of four drafted tokens: five new tokens per request
        _attend("draft_b16_n5", B=16, H=16, G=4, d_h=64, d_r=24, page=32, len_lo=1024, len_hi=8192,
                new_lo=5, new_hi=5, long_every=0, long_hi=0, pad=0, cache="bf16", out="bf16"),
        # a 512-token prompt chunk of every request on 4096 cached tokens
        _attend("chunk_b8_512", B=8, H=16, G=4, d_h=64, d_r=16, page=16, len_lo=4608, len_hi=4608,
                new_lo=512, new_hi=512, long_every=0, long_hi=0, pad=0, cache="bf16", out="bf16"),
        # a mixed step: most requests decode, every fourth brings a chunk; odd lengths, wide heads
        _attend("mixed_b16_d128", B=16, H=32, G=8, d_h=128, d_r=16, page=64, len_lo=1, len_hi=4096,
                new_lo=1, new_hi=1, long_every=4, long_hi=256, pad=3, cache="bf16", out="bf16"),
        # float32 cache, short odd lengths: the correctness configuration
        _attend("decode_f32_b3", B=3, H=4, G=2, d_h=32, d_r=8, page=16, len_lo=1, len_hi=100, new_lo=1,
                new_hi=2, long_every=0, long_hi=0, pad=0, cache="f32", out="f32"),
        # one request, four drafts: latency
        _verify("verify_b1", B=1, drafts_lo=4, drafts_hi=4, vocab=32768, row=32768, draft=True, probs="f32"),
        # a serving batch with a draft model and a large vocabulary
        _verify("verify_b64", B=64, drafts_lo=0, drafts_hi=7, vocab=131072, row=131072, draft=True,
                probs="f32"),
        # drafts copied from the prompt (no draft probabilities), odd vocabulary in padded rows
        _verify("verify_b256_copy", B=256, drafts_lo=1, drafts_hi=4, vocab=50021, row=50048, draft=False,
                probs="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "attend", "attend", "attend", "verify"])
    if op == "plan":
        B = _log(rng, 1, 2048)
        page = rng.choice([1, 8, 12, 16, 16, 32, 64, 128])
        return dict(op=op, B=B, page=page, max_len=_log(rng, 64, 8192), new_lo=rng.choice([0, 1, 1]),
                    new_hi=rng.randint(1, 8), long_every=rng.choice([0, 5, 16]), long_hi=_log(rng, 9, 512),
                    spare=max(1, int(B * rng.uniform(0.02, 2.0) * 16 / page)))
    if op == "verify":
        vocab = _log(rng, 1000, 131072)
        row = vocab + rng.choice([0, 0, 1, 27])
        lo = rng.choice([0, 1, 3])
        return dict(op=op, B=max(1, min(_log(rng, 1, 256), 64 * 131072 // vocab)), drafts_lo=lo,
                    drafts_hi=lo + rng.randint(0, 4), vocab=vocab, row=row, draft=rng.random() < 0.6,
                    probs=rng.choice(["f32", "f32", "bf16"]))
    heads = rng.choice([(16, 4, 64, 16), (16, 4, 64, 24), (32, 8, 128, 16), (16, 2, 64, 32), (8, 8, 64, 0),
                        (4, 2, 32, 8)])
    H, G, d_h, d_r = heads
    kind = rng.choice(["one", "few", "chunk", "mixed"])
    cache = "f32" if d_h == 32 else "bf16"
    page = rng.choice([8, 16, 16, 24, 32, 64, 128, 256])
    hi = _log(rng, 16, 16384)
    B = max(1, min(_log(rng, 1, 64), (131072 if d_h == 128 else 262144) // hi))
    c = dict(op=op, B=B, H=H, G=G, d_h=d_h, d_r=d_r, page=page, len_lo=rng.choice([1, (hi + 1) // 2, hi]),
             len_hi=hi, new_lo=1, new_hi=1, long_every=0, long_hi=0, pad=rng.choice([0, 0, 6]),
             cache=cache, out="f32" if cache == "f32" else rng.choice(["bf16", "bf16", "f32"]))
    if cache == "f32":   # the correctness configuration stays small
        c.update(B=min(B, 4), len_hi=min(hi, 700), len_lo=min(c["len_lo"], min(hi, 700)))
    if kind == "few":
        c.update(new_hi=rng.randint(2, 8))
    if kind in ("chunk", "mixed"):
        # rows x keys no more than the largest listed chunk's
        most = max(2, min(512, c["len_hi"], (4 * 512 * 4608 * 16 * 64) // (c["B"] * c["len_hi"] * H * d_h)))
        n = _log(rng, 2, most)
        c.update(out="f32" if cache == "f32" else "bf16")
        c.update(dict(new_lo=max(1, n - rng.randint(0, n - 1)), new_hi=n) if kind == "chunk" else
                 dict(long_every=rng.randint(2, 5), long_hi=n))
    elif H // G * c["new_hi"] > 8 and cache != "f32":
        c.update(out="bf16")
    return c


# ---------------------------------------------------------------------------- inputs

def _sizes(case):
    """The generator of a case's lengths: they are the same for every seed, which changes the order
    of the requests (so that outputs keep their shapes) and all else."""
    return torch.Generator().manual_seed(1 + case["B"])


def _new_counts(case, g):
    B = case["B"]
    n = torch.randint(case["new_lo"], case["new_hi"] + 1, (B,), generator=g)
    if case["long_every"]:
        big = torch.randint(1, case["long_hi"] + 1, (B,), generator=g)
        n = torch.where(torch.arange(B) % case["long_every"] == case["long_every"] - 1, big, n)
    return n


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case=dict(case))
    st.update({"plan": _prepare_plan, "attend": _prepare_attend, "verify": _prepare_verify}[case["op"]](
        case, g, gd))
    return st


def _prepare_plan(case, g, gd):
    B, page = case["B"], case["page"]
    gs, order = _sizes(case), torch.randperm(B, generator=g)
    kept = torch.randint(0, case["max_len"] + 1, (B,), generator=gs)[order]
    n = _new_counts(case, gs)[order]
    # some requests still hold pages of drafts that were rejected in the step before
    held = (kept + torch.randint(0, 9, (B,), generator=gs)[order] + page - 1) // page
    longest = case["max_len"] + max(case["new_hi"], case["long_hi"], 9)
    max_pages = (longest + page - 1) // page
    num_pages = int(held.sum()) + case["spare"]
    ids = torch.randperm(num_pages, generator=g).to(torch.int32)
    col = torch.arange(max_pages)[None, :]
    own_page = col < held[:, None]
    table = torch.full((B, max_pages), -1, dtype=torch.int32)
    table[own_page] = ids[:int(held.sum())]
    free = torch.full((num_pages,), -1, dtype=torch.int32)
    free[:case["spare"]] = ids[int(held.sum()):]
    room = int(n.sum())
    z = lambda k: torch.zeros(k, dtype=torch.int32, device="cuda")
    return dict(page=page, num_pages=num_pages, kept_len=_d(kept.to(torch.int32)),
                n_new=_d(n.to(torch.int32)), held_in=_d(held.to(torch.int32)), held_out=z(B),
                free_pages=_d(free), free_count_in=_d(_ints([case["spare"]])), free_count_out=z(1),
                block_table=_d(table), q_start=z(B + 1), seq_len=z(B), n_granted=z(B), slot=z(room),
                pos=z(room), err=z(1))


def _prepare_attend(case, g, gd):
    B, H, G, d_h, d_r, page = (case[k] for k in ("B", "H", "G", "d_h", "d_r", "page"))
    dt = DT[case["cache"]]
    gs, order = _sizes(case), torch.randperm(B, generator=g)
    L = torch.randint(case["len_lo"], case["len_hi"] + 1, (B,), generator=gs)[order]
    # the new tokens are the last of each request's; a request may be shorter than its chunk only
    # by a caller's mistake, so lengths count at least the new tokens
    n = _new_counts(case, gs)[order]
    L = torch.maximum(L, n)
    pages = (L + page - 1) // page
    max_pages = int(pages.max())
    used = int(pages.sum())
    num_pages = used + 3
    ids = torch.randperm(num_pages, generator=g).to(torch.int32)
    table = torch.full((B, max_pages), -1, dtype=torch.int32)
    table[torch.arange(max_pages)[None, :] < pages[:, None]] = ids[:used]
    V = torch.randn(num_pages * page, G, d_h, generator=gd, device="cuda", dtype=torch.float32).to(dt)
    kr = torch.randn(num_pages * page, d_r, generator=gd, device="cuda", dtype=torch.float32).to(dt)
    # slots behind the end of a request were never written: whatever they hold must not count
    tail = page * table[torch.arange(B), pages - 1].long()[:, None] + torch.arange(page)[None, :]
    behind = ((pages - 1) * page)[:, None] + torch.arange(page)[None, :] >= L[:, None]
    V[_d(tail[behind])] = float("nan")
    kr[_d(tail[behind])] = float("nan")
    q_start = torch.zeros(B + 1, dtype=torch.int64)
    q_start[1:] = n.cumsum(0)
    rows = int(q_start[-1]) + case["pad"]
    c = math.log2(math.e) / math.sqrt(d_h)
    q_abs = torch.randn(rows, H, d_h + d_r, generator=gd, device="cuda", dtype=torch.float32) * c
    return dict(page=page, q_abs=q_abs, V=V, kr=kr, block_table=_d(table),
                q_start=_d(q_start.to(torch.int32)), seq_len=_d(L.to(torch.int32)), max_new=int(n.max()), max_len=int(L.max()),
                total=int(L.sum()), out=torch.zeros(rows, H, d_h, dtype=DT[case["out"]], device="cuda"),
                lse=torch.zeros(rows, H, dtype=torch.float32, device="cuda"), keep={})


def _prepare_verify(case, g, gd):
    B, vocab, row = case["B"], case["vocab"], case["row"]
    dt = DT[case["probs"]]
    k = torch.randint(case["drafts_lo"], case["drafts_hi"] + 1, (B,), generator=_sizes(case))
    k = k[torch.randperm(B, generator=g)]
    q_start = torch.zeros(B + 1, dtype=torch.int64)
    q_start[1:] = (k + 1).cumsum(0)
    N = int(q_start[-1])
    logits = torch.randn(N, row, generator=gd, device="cuda") * 2.5
    target = torch.softmax(logits, -1).to(dt)
    # the draft model is near to the target; its tokens are drawn from its probabilities
    logits += torch.randn(N, row, generator=gd, device="cuda") * 0.5
    draft = torch.softmax(logits, -1).to(dt)
    race = torch.empty_like(logits).exponential_(generator=gd)
    drawn = (draft[:, :vocab].float() / race[:, :vocab]).argmax(-1).to(torch.int32)
    if not case["draft"]:   # a copied token is often the likeliest one
        drawn = torch.where(torch.rand(N, generator=gd, device="cuda") < 0.7,
                            target[:, :vocab].float().argmax(-1).to(torch.int32), drawn)
    tokens = torch.randint(0, vocab, (N,), generator=gd, device="cuda", dtype=torch.int32)
    tokens[1:] = drawn[:-1]    # fed token j + 1 was drawn from row j
    seq_len = torch.randint(64, 4096, (B,), generator=g).to(torch.int32)
    z = lambda m: torch.zeros(m, dtype=torch.int32, device="cuda")
    return dict(vocab=vocab, most=int(k.max()), tokens=tokens, q_start=_d(q_start.to(torch.int32)),
                target=target, draft=draft if case["draft"] else None,
                u_accept=torch.rand(N, generator=gd, device="cuda"),
                u_sample=torch.rand(B, generator=gd, device="cuda"), seq_len=_d(seq_len), out_tokens=z(N),
                n_accepted=z(B), kept_len=z(B))


# ---------------------------------------------------------------------------- one pass

def run(st):
    op = st["case"]["op"]
    if own:
        return {"plan": _own_plan, "attend": _own_attend, "verify": _own_verify}[op](st)
    return {"plan": _plain_plan, "attend": _plain_attend, "verify": _plain_verify}[op](st)


def _own_plan(st):
    from compressed_kv_cache_gva_b200 import gva
    gva.plan_pages(st["page"], st["num_pages"], st["kept_len"], st["n_new"], st["held_in"], st["held_out"],
                   st["free_pages"], st["free_count_in"], st["free_count_out"], st["block_table"],
                   st["q_start"], st["seq_len"], st["n_granted"], st["slot"], st["pos"], st["err"])
    return {k: st[k] for k in ("held_out", "free_pages", "free_count_out", "block_table", "q_start",
                               "seq_len", "n_granted", "slot", "pos", "err")}


def _own_attend(st):
    from compressed_kv_cache_gva_b200 import gva
    keep = st["keep"]
    if not keep:   # shape and workspace: made once per configuration, as a server does
        c = st["case"]
        keep["shape"] = gva.make_shape(c["B"], c["H"], c["G"], c["d_h"], c["d_h"], c["d_r"],
                                       cache_dtype=DT[c["cache"]], out_dtype=DT[c["out"]])
        keep["ws"] = gva.new_paged_workspace(keep["shape"], st["page"], st["q_abs"].shape[0], st["max_new"],
                                             st["total"])
    gva.paged_attention(keep["shape"], st["page"], st["q_abs"], st["V"], st["kr"], st["block_table"],
                        st["q_start"], st["seq_len"], st["max_new"], st["total"], st["out"], st["lse"],
                        keep["ws"])
    return st["out"], st["lse"]


def _own_verify(st):
    from compressed_kv_cache_gva_b200 import gva
    gva.verify_draft(st["vocab"], st["tokens"], st["q_start"], st["target"], st["draft"], st["u_accept"],
                     st["u_sample"], st["out_tokens"], st["n_accepted"], st["seq_len"], st["kept_len"])
    return st["out_tokens"], st["n_accepted"], st["kept_len"]


def _plain_plan(st):
    page, num_pages, table = st["page"], st["num_pages"], st["block_table"]
    kept, n, held = st["kept_len"].long(), st["n_new"].long(), st["held_in"].long()
    free, count = st["free_pages"], st["free_count_in"].long()
    B, max_pages = table.shape
    dev, room = table.device, st["slot"].numel()
    goal = (kept + n + page - 1) // page
    bad = (kept < 0) | (n < 0) | (held < 0) | (held > max_pages) | (goal > max_pages) | (kept > held * page)
    fits = ~bad & (torch.where(bad, 0, n).cumsum(0) <= room)
    need = torch.where(fits, (goal - held).clamp(min=0), 0)
    back = torch.where(fits, (held - goal).clamp(min=0), 0)
    ok = fits & ((need == 0) | (need.cumsum(0) <= count + back.sum()))
    need, got = torch.where(ok, need, 0), torch.where(ok, n, 0)
    # returned pages go on top of the free list, in the order of the requests
    col = torch.arange(max_pages, device=dev)[None, :]
    freed = (col >= goal[:, None]) & (col < held[:, None]) & ok[:, None]
    at = count + (back.cumsum(0) - back)[:, None] + col - goal[:, None]
    new_free = torch.cat([free, free[:1]])
    new_free[torch.where(freed, at, num_pages)] = table
    new_free = new_free[:num_pages]
    # new pages come from its top
    top = count + back.sum()
    rank = (need.cumsum(0) - need)[:, None] + col - held[:, None]
    new = (col >= held[:, None]) & (col < goal[:, None]) & ok[:, None]
    new_table = torch.where(new, new_free[(top - 1 - rank).clamp(0, num_pages - 1)], table)
    q_start = torch.cat([got.new_zeros(1), got.cumsum(0)])
    i = torch.arange(room, device=dev)
    b = torch.searchsorted(q_start, i, right=True) - 1
    on = b < B
    b = b.clamp(max=B - 1)
    pos = kept[b] + i - q_start[b]
    slot = new_table[b, (pos // page).clamp(max=max_pages - 1)].long() * page + pos % page
    err = torch.where(bad.any(), 1, 0) | torch.where((~ok & ~bad).any(), 4, 0)
    i32 = torch.int32
    return dict(held_out=torch.where(ok, goal, held).to(i32), free_pages=new_free,
                free_count_out=(top - need.sum()).to(i32), block_table=new_table, q_start=q_start.to(i32),
                seq_len=(torch.where(bad, 0, kept) + got).to(i32), n_granted=got.to(i32),
                slot=torch.where(on, slot, -1).to(i32), pos=torch.where(on, pos, -1).to(i32),
                err=err.to(i32).reshape(1))


def _plain_attend(st):
    c, page, table, L = st["case"], st["page"], st["block_table"], st["seq_len"].long()
    B, H, G, d_h, d_r = (c[k] for k in ("B", "H", "G", "d_h", "d_r"))
    hpr, dev = H // G, table.device
    q_start = st["q_start"].long()
    n = q_start[1:] - q_start[:-1]
    Q, T = st["max_new"], st["max_len"]
    j = torch.arange(T, device=dev)
    inside = j[None, :] < L[:, None]
    slot = table.long()[:, j // page].clamp(min=0) * page + (j % page)[None, :]
    V = torch.where(inside[:, :, None, None], st["V"][slot].float(), 0.0).permute(0, 2, 1, 3)   # B G T d
    i = torch.arange(Q, device=dev)
    q = st["q_abs"][(q_start[:-1, None] + i[None, :]).clamp(max=st["q_abs"].shape[0] - 1)]       # B Q H .
    q = q.reshape(B, Q, G, hpr, -1).permute(0, 2, 1, 3, 4).reshape(B, G, Q * hpr, d_h + d_r)
    s = q[..., :d_h] @ V.transpose(2, 3)
    if d_r:
        K = torch.where(inside[:, :, None], st["kr"][slot].float(), 0.0)
        s += q[..., d_h:] @ K.transpose(1, 2)[:, None]
    last = (L - n)[:, None] + i[None, :]                                        # B Q: newest key seen
    seen = inside[:, None, :] & (j[None, None, :] <= last[:, :, None])          # B Q T
    s = s.reshape(B, G, Q, hpr, T).masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp2(s - m.clamp(min=-3e38))
    l = p.sum(-1, keepdim=True)
    o = (p.reshape(B, G, Q * hpr, T) @ V).reshape(B, G, Q, hpr, d_h) / l.clamp(min=1e-38)
    lse = ((m + torch.log2(l)) * math.log(2.0))[..., 0]
    o = o.permute(0, 2, 1, 3, 4).reshape(B, Q, H, d_h)
    lse = lse.permute(0, 2, 1, 3).reshape(B, Q, H)
    r = torch.arange(st["q_abs"].shape[0], device=dev)
    b = torch.searchsorted(q_start, r, right=True) - 1
    on = b < B
    b = b.clamp(max=B - 1)
    at = (r - q_start[b]).clamp(max=Q - 1)
    out = torch.where(on[:, None, None], o[b, at].to(st["out"].dtype), st["out"])
    return out, torch.where(on[:, None], lse[b, at], st["lse"])


def _plain_verify(st):
    x, q_start, vocab, most = st["tokens"].long(), st["q_start"].long(), st["vocab"], st["most"]
    target, draft = st["target"], st["draft"]
    B, N, dev = q_start.numel() - 1, x.numel(), x.device
    k = q_start[1:] - q_start[:-1] - 1
    i = torch.arange(max(most, 1), device=dev)[None, :]
    row = (q_start[:-1, None] + i).clamp(max=N - 1)
    nxt = x[(row + 1).clamp(max=N - 1)]
    p = target[row, nxt].double()
    q = draft[row, nxt].double() if draft is not None else torch.ones_like(p)
    yes = (st["u_accept"][row].double() * q < p) & (i < k[:, None])
    a = yes.long().cumprod(-1).sum(-1)
    row = q_start[:-1] + a
    w = target[row, :vocab].double()
    refused = (a < k)[:, None]
    x_no = x[(row + 1).clamp(max=N - 1)]
    if draft is not None:
        rest = (w - draft[row, :vocab].double()).clamp(min=0)
    else:
        rest = torch.where(torch.arange(vocab, device=dev)[None, :] == x_no[:, None], 0.0, w)
    rest = torch.where(refused, rest, w)
    w = torch.where(rest.sum(-1, keepdim=True) > 0, rest, w)
    total = w.cumsum(-1)
    over = total > st["u_sample"].double()[:, None] * total[:, -1:]
    token = torch.where(over.any(-1), over.to(torch.uint8).argmax(-1), vocab - 1)
    r = torch.arange(N, device=dev)
    b = torch.searchsorted(q_start, r, right=True) - 1
    at = r - q_start[b]
    out = torch.where(at < a[b], x[(r + 1).clamp(max=N - 1)], torch.where(at == a[b], token[b], -1))
    kept = st["seq_len"].long() - (k - a)
    return out.to(torch.int32), a.to(torch.int32), kept.to(torch.int32)


# ---------------------------------------------------------------------------- work and 64 bits

def _mean_new(case):
    n = (case["new_lo"] + case["new_hi"]) / 2
    if case["long_every"]:
        n += ((1 + case["long_hi"]) / 2 - n) / case["long_every"]
    return n


def work(case):
    B = case["B"]
    if case["op"] == "plan":
        # per request three lengths in, four out; each page that changes hands is read and written
        # once; each new token gets a slot and a position
        n = _mean_new(case)
        return {"bytes": B * (7 * 4 + 8 * (n + 4) / case["page"] + 8 * n), "flops": 0}
    if case["op"] == "attend":
        H, G, d_h, d_r = (case[k] for k in ("H", "G", "d_h", "d_r"))
        n, L = _mean_new(case), (case["len_lo"] + case["len_hi"]) / 2
        L = max(L, n)
        e, eo = DT[case["cache"]].itemsize, DT[case["out"]].itemsize
        byts = B * (L * (G * d_h + d_r) * e + n * H * ((d_h + d_r) * 4 + d_h * eo + 4))
        return {"bytes": byts, "flops": B * n * max(L - n / 2, 1) * H * 2 * (2 * d_h + d_r)}
    e = DT[case["probs"]].itemsize
    n = (case["drafts_lo"] + case["drafts_hi"]) / 2 + 1
    return {"bytes": B * (case["vocab"] * e * (2 if case["draft"] else 1) + n * (8 + 3 * e) + 16), "flops": 0}


def exact(case, seed):
    st = prepare(case, seed)
    return {"plan": _exact_plan, "attend": _exact_attend, "verify": _exact_verify}[case["op"]](st)


def _exact_plan(st):
    """The same step request by request, on the host."""
    page, P = st["page"], st["num_pages"]
    kept, n, held = (st[k].tolist() for k in ("kept_len", "n_new", "held_in"))
    free, table = st["free_pages"].tolist(), st["block_table"].tolist()
    room, B, W = st["slot"].numel(), len(kept), st["block_table"].shape[1]
    count = st["free_count_in"].item()
    goal = [-(-(a + b) // page) for a, b in zip(kept, n)]
    bad = [a < 0 or b < 0 or h < 0 or h > W or t > W or a > h * page
           for a, b, h, t in zip(kept, n, held, goal)]
    asked, fits = 0, []
    for b in range(B):
        asked += 0 if bad[b] else n[b]
        fits.append(not bad[b] and asked <= room)
    top = count + sum(max(h - t, 0) for h, t, f in zip(held, goal, fits) if f)
    wanted, ok = 0, []
    for b in range(B):
        need = max(goal[b] - held[b], 0) if fits[b] else 0
        wanted += need
        ok.append(fits[b] and (need == 0 or wanted <= top))
    for b in range(B):
        if ok[b]:
            for t in range(goal[b], held[b]):
                free[count] = table[b][t]
                count += 1
    slot, pos, q_start, seq_len, granted, out_held = [], [], [0], [], [], []
    for b in range(B):
        if ok[b]:
            for t in range(held[b], goal[b]):
                count -= 1
                table[b][t] = free[count]
            for t in range(kept[b], kept[b] + n[b]):
                slot.append(table[b][t // page] * page + t % page)
                pos.append(t)
        granted.append(n[b] if ok[b] else 0)
        seq_len.append((0 if bad[b] else kept[b]) + granted[b])
        out_held.append(goal[b] if ok[b] else held[b])
        q_start.append(len(slot))
    rest = [-1] * (room - len(slot))
    err = (1 if any(bad) else 0) | (4 if any(not o and not x for o, x in zip(ok, bad)) else 0)
    return dict(held_out=_ints(out_held), free_pages=_ints(free), free_count_out=_ints([count]),
                block_table=_ints(table), q_start=_ints(q_start), seq_len=_ints(seq_len),
                n_granted=_ints(granted), slot=_ints(slot + rest), pos=_ints(pos + rest), err=_ints([err]))


def _exact_attend(st):
    c, page = st["case"], st["page"]
    H, G, d_h, d_r = (c[k] for k in ("H", "G", "d_h", "d_r"))
    out, lse = st["out"].double(), st["lse"].double()
    starts, lens = st["q_start"].tolist(), st["seq_len"].tolist()
    for b, L in enumerate(lens):
        n = starts[b + 1] - starts[b]
        ids = st["block_table"][b, :-(-L // page)].long()
        slots = (ids[:, None] * page + torch.arange(page, device=ids.device)).reshape(-1)[:L]
        q = st["q_abs"][starts[b]:starts[b + 1]].double()
        hidden = torch.ones(n, L, dtype=torch.bool, device=ids.device).triu(L - n + 1)
        for g in range(G):
            v = st["V"][slots, g].double()
            h0, h1 = g * H // G, (g + 1) * H // G
            s = torch.einsum("nhd,td->nht", q[:, h0:h1, :d_h], v)
            if d_r:
                s += torch.einsum("nhr,tr->nht", q[:, h0:h1, d_h:], st["kr"][slots].double())
            s = (s * math.log(2.0)).masked_fill(hidden[:, None, :], float("-inf"))
            lse[starts[b]:starts[b + 1], h0:h1] = torch.logsumexp(s, -1)
            out[starts[b]:starts[b + 1], h0:h1] = torch.einsum("nht,td->nhd", torch.softmax(s, -1), v)
    return out, lse


def _exact_verify(st):
    x, starts, vocab = st["tokens"].tolist(), st["q_start"].tolist(), st["vocab"]
    out, acc, kept = [], [], []
    for b, L in enumerate(st["seq_len"].tolist()):
        k, a = starts[b + 1] - starts[b] - 1, 0
        while a < k:
            r = starts[b] + a
            q = float(st["draft"][r, x[r + 1]]) if st["draft"] is not None else 1.0
            if not float(st["u_accept"][r]) * q < float(st["target"][r, x[r + 1]]):
                break
            a += 1
        r = starts[b] + a
        p = st["target"][r, :vocab].double().cpu()
        w = p
        if a < k and st["draft"] is not None:
            w = torch.relu(p - st["draft"][r, :vocab].double().cpu())
        elif a < k:
            w = p.clone()
            w[x[r + 1]] = 0
        if float(w.sum()) == 0:
            w = p
        reach = torch.cumsum(w, 0)
        token = int(torch.searchsorted(reach, float(st["u_sample"][b]) * reach[-1], right=True))
        out += x[starts[b] + 1:r + 1] + [min(token, vocab - 1)] + [-1] * (k - a)
        acc.append(a)
        kept.append(L - (k - a))
    return _ints(out), _ints(acc), _ints(kept)
