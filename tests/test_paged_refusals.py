"""Host-side refusals of the paged calls: a status and a reason, and no launch (CPU: the
pointers are never dereferenced)."""
import ctypes

import pytest
import torch

from compressed_kv_cache_gva_b200 import _build, gva

FAKE = 1 << 20


@pytest.fixture(scope="module")
def L():
    _build.build()
    return gva.lib()


def plan(L, B=4, page=16, pages=100, width=8, stride=8, room=10, **ptr):
    names = ["kept", "new", "held_in", "held_out", "free", "count_in", "count_out", "table", "q_start", "seq_len",
             "granted", "slot", "pos", "err"]
    return L.gva_plan_pages(B, page, pages, width, stride, room, *[ptr.get(n, FAKE) for n in names], None)


@pytest.mark.parametrize("kw,why", [
    (dict(B=-1), "B="), (dict(B=4097), "B="), (dict(page=0), "page_size"), (dict(pages=0), "num_pages"),
    (dict(page=1 << 16, pages=1 << 15), "2^31"), (dict(width=0), "max_pages"), (dict(stride=7), "table_stride"),
    (dict(page=1 << 16, pages=4, width=1 << 15, stride=1 << 15), "2^31"), (dict(room=-1), "max_new_tokens"),
    (dict(kept=None), "NULL"), (dict(free=None), "NULL"), (dict(count_out=None), "NULL"), (dict(table=None), "NULL"),
    (dict(slot=None), "NULL"), (dict(q_start=None), "NULL"), (dict(pos=FAKE + 2), "aligned"), (dict(err=FAKE + 1), "aligned")])
def test_plan_pages(L, kw, why):
    assert plan(L, **kw) == 1 and why in L.gva_last_error().decode()


def attend(L, sh, page=16, q=FAKE, V=FAKE, kr=FAKE, slots=1600, table=FAKE, width=8, stride=8, q_start=FAKE, lens=FAKE,
           rows=4, most=4, total=100, out=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 30):
    return L.gva_paged_attention(ctypes.byref(sh), page, q, V, kr, slots, table, width, stride, q_start, lens, rows, most,
                                 total, out, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,why", [
    (dict(page=0), "page_size"), (dict(page=(1 << 20) + 1), "page_size"), (dict(q=None), "NULL"), (dict(V=None), "NULL"),
    (dict(kr=None), "NULL"), (dict(table=None), "NULL"), (dict(q_start=None), "NULL"), (dict(lens=None), "NULL"),
    (dict(out=None), "NULL"), (dict(ws=None), "NULL"), (dict(q=FAKE + 8), "aligned"), (dict(out=FAKE + 4), "aligned"),
    (dict(lse=FAKE + 4), "aligned"), (dict(table=FAKE + 2), "aligned"), (dict(slots=0), "num_slots"),
    (dict(slots=1601), "num_slots"), (dict(slots=1 << 31), "num_slots"), (dict(width=0), "max_pages"),
    (dict(stride=7), "table_stride"), (dict(rows=-1), "n_rows"), (dict(rows=1 << 28), "n_rows"), (dict(most=0), "max_query_len"),
    (dict(total=-1), "max_total_tokens"), (dict(total=1 << 31), "max_total_tokens")])
def test_paged_attention(L, kw, why):
    sh = gva.make_shape(4, 16, 4, 64, 64, 16)
    assert attend(L, sh, **kw) == 1 and why in L.gva_last_error().decode()


@pytest.mark.parametrize("bad", [dict(H=15), dict(G=0), dict(d_r=15), dict(d_h=0), dict(B=-1), dict(B=5000)])
def test_paged_shapes(L, bad):
    sh = gva.make_shape(**{**dict(B=2, H=16, G=4, d_h=64, d_n=64, d_r=16), **bad})
    assert attend(L, sh) == 1 and L.gva_last_error()
    assert L.gva_paged_workspace_size(ctypes.byref(sh), 16, 4, 4, 100) == 0


def test_cache_rows_of_odd_bytes(L):
    sh = gva.make_shape(2, 4, 2, 64, 64, 6)
    assert attend(L, sh) == 1 and "16 bytes" in L.gva_last_error().decode()


def test_paged_attention_without_rows_is_a_noop(L):
    sh = gva.make_shape(0, 16, 4, 64, 64, 16)
    assert attend(L, sh, q=None, V=None) == 0
    sh = gva.make_shape(4, 16, 4, 64, 64, 16)
    assert attend(L, sh, q=None, rows=0) == 0


def verify(L, B=3, vocab=10, rows=6, dtype=0, tstride=10, dstride=10, **ptr):
    g = lambda n: ptr.get(n, FAKE)
    return L.gva_verify_draft(B, vocab, rows, g("tokens"), g("q_start"), dtype, g("target"), tstride, g("draft"), dstride,
                              g("u"), g("us"), g("out"), g("acc"), g("lens"), g("kept"), g("err"), None)


@pytest.mark.parametrize("kw,why", [
    (dict(B=-1), "B="), (dict(B=65536), "B="), (dict(vocab=0), "vocab"), (dict(rows=-1), "n_rows"), (dict(dtype=2), "probs_dtype"),
    (dict(tstride=9), "strides"), (dict(dstride=9), "strides"), (dict(tokens=None), "NULL"), (dict(target=None), "NULL"),
    (dict(u=None), "NULL"), (dict(us=None), "NULL"), (dict(out=None), "NULL"), (dict(acc=None), "NULL"),
    (dict(kept=None), "together"), (dict(lens=None), "together"), (dict(tokens=FAKE + 2), "aligned"),
    (dict(target=FAKE + 2), "aligned"), (dict(draft=FAKE + 1, dtype=1), "aligned")])
def test_verify_draft(L, kw, why):
    assert verify(L, **kw) == 1 and why in L.gva_last_error().decode()


def test_empty_verification_is_a_noop(L):
    assert verify(L, B=0, tokens=None, q_start=None) == 0


@pytest.mark.gpu
def test_binding_checks_its_tensors():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    f = lambda *s: torch.zeros(*s, device="cuda")
    sh = gva.make_shape(2, 16, 4, 64, 64, 16)
    ws = gva.new_paged_workspace(sh, 16, 2, 1, 100)
    good = dict(q_abs=f(2, 16, 80), V_cache=f(64, 4, 64).bfloat16(), kr_cache=f(64, 16).bfloat16(), block_table=i(2, 4),
                q_start=i(3), seq_len=i(2), max_query_len=1, max_total_tokens=100, out=f(2, 16, 64), lse=f(2, 16),
                workspace=ws)
    gva.paged_attention(sh, 16, **good)
    for k, v in dict(q_abs=f(2, 16, 79), V_cache=f(64, 4, 64), kr_cache=f(32, 16).bfloat16(), block_table=i(3, 4),
                     q_start=i(2), seq_len=i(2).long(), out=f(2, 16, 64).bfloat16(), lse=f(16, 2).t(),
                     workspace=ws.cpu()).items():
        with pytest.raises(ValueError):
            gva.paged_attention(sh, 16, **{**good, k: v})
    with pytest.raises(ValueError):
        gva.paged_attention(sh, 16, **{**good, "block_table": i(2, 8)[:, ::2]})
    with pytest.raises(gva.GVAError):
        gva.paged_attention(sh, 16, **{**good, "workspace": ws[:1024]})
    with pytest.raises(gva.GVAError):
        gva.paged_attention(sh, 48, **good)              # 64 slots are no whole number of pages
    torch.cuda.synchronize()
