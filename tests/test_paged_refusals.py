"""The paged-cache entry points reject invalid arguments on the host, before any
CUDA call (so these run without a GPU), and the oracle they are tested against
agrees with brute force on small inputs."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.paged as oracle
from speech_encoder_attention_b200 import attn

BASE = 0x7F0000000000
STEP = 0x10000000
Q, OUT, KP, VP, TBL, LENS, LSE, WS, W1, W2, KEPT, KP2, VP2, TBL2, LENS2 = (BASE + i * STEP for i in range(15))


def m(ptr, stride):
    return attn.AttnMat(ctypes.c_void_p(ptr), stride)


def cache(k=None, v=None, table=TBL, lens=LENS, num_pages=8, page_size=16, pages_per_seq=4, n_kv_heads=2):
    return attn.AttnPagedKV(k or m(KP, 128), v or m(VP, 128), table, lens, num_pages, page_size, pages_per_seq,
                            n_kv_heads)


def mask(window=0, first=0, causal=1, q_lens=0):
    return attn.AttnPagedMask(window, first, causal, q_lens)


BAD_CACHES = [
    dict(page_size=8), dict(page_size=24), dict(page_size=512), dict(page_size=0), dict(num_pages=0),
    dict(pages_per_seq=0), dict(n_kv_heads=0), dict(table=0), dict(table=TBL + 2), dict(lens=0), dict(lens=LENS + 1),
    dict(k=m(0, 128)), dict(k=m(KP + 8, 128)), dict(k=m(KP, 64)), dict(v=m(VP, 132)), dict(v=m(VP + 2, 128)),
    dict(num_pages=2 ** 27, page_size=16), dict(pages_per_seq=2 ** 20, page_size=256),
]


def call_paged(lib, q=None, c=None, batch=1, t_q=4, heads=4, mk=None, sinks=0, scale=0.125, out=None, lse=0, ws=WS,
               ws_bytes=1 << 30):
    return lib.attn_paged(q or m(Q, 256), c or cache(), batch, t_q, heads, mk or mask(), sinks, scale, out or m(OUT, 256),
                          lse, ws, ws_bytes, None)


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_every_entry_rejects_a_bad_cache(lib, kw):
    bad = cache(**kw)
    assert call_paged(lib, c=bad) == attn.ATTN_ERR_INVALID
    assert lib.attn_paged_append(m(Q, 128), m(OUT, 128), bad, 1, 4, 0, None) == attn.ATTN_ERR_INVALID
    assert lib.attn_paged_weights(m(Q, 256), bad, 1, 4, 4, mask(), LSE, 0.125, W1, W2, WS, 1 << 30, None) == attn.ATTN_ERR_INVALID
    good = cache(k=m(KP2, 128), v=m(VP2, 128), table=TBL2, lens=LENS2)
    assert lib.attn_paged_evict(bad, 1, 16, 0, 0, W1, good, W2, KEPT, None) == attn.ATTN_ERR_INVALID
    assert lib.attn_paged_evict(good, 1, 16, 0, 0, W1, bad, W2, KEPT, None) == attn.ATTN_ERR_INVALID


@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(batch=70000), dict(t_q=0), dict(heads=0), dict(heads=3), dict(heads=2 * 129),
    dict(q=m(0, 256)), dict(q=m(Q, 248)), dict(q=m(Q + 8, 256)), dict(out=m(OUT, 128)), dict(out=m(Q + 64, 256)),
    dict(out=m(KP, 256)), dict(out=m(VP + 128, 256)), dict(scale=0.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(sinks=LSE + 2), dict(lse=LSE + 1), dict(ws=0), dict(ws=WS + 8), dict(ws=0, ws_bytes=16),
    dict(mk=mask(window=-1)), dict(mk=mask(first=2)), dict(mk=mask(window=4, first=-1)), dict(mk=mask(causal=2)),
    dict(mk=mask(q_lens=LSE + 2)),
])
def test_paged_rejects_invalid_arguments(lib, kw):
    assert call_paged(lib, **kw) == attn.ATTN_ERR_INVALID


@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(t=0), dict(k=m(0, 128)), dict(v=m(OUT, 64)), dict(k=m(KP + 256, 128)), dict(v=m(VP, 128)),
    dict(q_lens=LSE + 2),
])
def test_append_rejects_invalid_arguments(lib, kw):
    st = lib.attn_paged_append(kw.get("k", m(Q, 128)), kw.get("v", m(OUT, 128)), cache(), kw.get("batch", 1),
                               kw.get("t", 4), kw.get("q_lens", 0), None)
    assert st == attn.ATTN_ERR_INVALID


@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(t_q=0), dict(heads=3), dict(q=m(Q, 100)), dict(lse=0), dict(lse=LSE + 2), dict(w_out=0),
    dict(w_out=W2 + 1), dict(w_in=W1 + 2), dict(w_in=W2 + 4), dict(w_out=Q), dict(w_out=LSE), dict(w_out=KP),
    dict(scale=-1.0), dict(mk=mask(first=1)), dict(ws=0), dict(ws=WS + 4), dict(heads=2 * 129),
])
def test_weights_rejects_invalid_arguments(lib, kw):
    st = lib.attn_paged_weights(kw.get("q", m(Q, 256)), cache(), kw.get("batch", 1), kw.get("t_q", 4),
                                kw.get("heads", 4), kw.get("mk", mask()), kw.get("lse", LSE), kw.get("scale", 0.125),
                                kw.get("w_in", W1), kw.get("w_out", W2), kw.get("ws", WS), 1 << 30, None)
    assert st == attn.ATTN_ERR_INVALID


DST = dict(k=m(KP2, 128), v=m(VP2, 128), table=TBL2, lens=LENS2)


@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(budget=0), dict(budget=65), dict(first=-1), dict(recent=-1), dict(first=10, recent=7),
    dict(w_in=0), dict(w_in=W1 + 2), dict(w_out=W2 + 2), dict(w_out=W1 + 4), dict(kept=0), dict(kept=KEPT + 2),
    dict(kept=W1), dict(kept=W2), dict(kept=LENS2), dict(dst=dict(DST, page_size=32)),
    dict(dst=dict(DST, n_kv_heads=1)),
    dict(dst=dict(DST, k=m(KP + 128, 128))),                      # pools overlap without being the same
    dict(dst=dict(DST, k=m(VP, 128), v=m(KP, 128))),              # K and V swapped
    dict(dst=dict(k=m(KP, 128), v=m(VP, 128), num_pages=4)),      # the same pools of another size
    dict(dst=dict(DST, lens=LENS + 4), batch=2),                  # lengths overlap without being the same
    dict(dst=dict(DST, pages_per_seq=2), budget=16, w_out=W1),    # one weight buffer for two shapes
])
def test_evict_rejects_invalid_arguments(lib, kw):
    st = lib.attn_paged_evict(cache(), kw.get("batch", 1), kw.get("budget", 16), kw.get("first", 0),
                              kw.get("recent", 0), kw.get("w_in", W1), cache(**kw.get("dst", DST)),
                              kw.get("w_out", W2), kw.get("kept", KEPT), None)
    assert st == attn.ATTN_ERR_INVALID


def test_workspace_size_of_invalid_sizes_is_zero(lib):
    assert lib.attn_paged_workspace_size(cache(), 0, 1, 4, mask()) == 0
    assert lib.attn_paged_workspace_size(cache(), 1, 0, 4, mask()) == 0
    assert lib.attn_paged_workspace_size(cache(n_kv_heads=3), 1, 1, 4, mask()) == 0
    assert lib.attn_paged_workspace_size(cache(n_kv_heads=1), 1, 1, 129, mask()) == 0
    assert lib.attn_paged_weights_workspace_size(cache(), 0, 1, 4) == 0
    assert lib.attn_paged_weights_workspace_size(cache(page_size=24), 1, 1, 4) == 0


def test_binding_refuses_bad_caches():
    k = torch.zeros(32, 128, dtype=torch.float16)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        attn.PagedKV(k, k, table, lens, 16, 2)
    with pytest.raises(ValueError, match="page_size"):
        attn.PagedKV(k, k, table, lens, 24, 2)


# ---------------------------------------------------------------------------
# the oracle against brute force
# ---------------------------------------------------------------------------

def test_oracle_attention_is_contiguous_attention_over_the_gathered_slots():
    import oracle as dense
    rng = np.random.default_rng(0)
    page, t_q, heads, kv_len = 16, 5, 2, 37
    k, v = rng.standard_normal((4 * page, 128)), rng.standard_normal((4 * page, 128))
    table = np.array([[2, 0, 3]], np.int32)
    q = rng.standard_normal((t_q, 128))
    rows = [oracle.slot_row(table[0], j, page, 4) for j in range(kv_len)]
    got, lse = oracle.attention(q, k, v, table, [kv_len], page, t_q, heads, heads)
    want = dense.range_attention(q, k[rows], v[rows], 1, t_q, kv_len, heads, causal=True)
    assert np.abs(got - want).max() < 1e-12
    # constant values come back, the weights of a row sum to one, and a hole is not seen
    w = oracle.weights(q, k, table, [kv_len], lse, page, t_q, heads, heads, np.zeros((1, 48)))
    assert abs(w.sum() - t_q * heads) < 1e-9
    holed = np.array([[2, -1, 3]], np.int32)
    got, _ = oracle.attention(q, k, v, holed, [kv_len], page, t_q, heads, heads, causal=False)
    keep = [r for j, r in enumerate(rows) if j // page != 1]
    want = dense.range_attention(q, k[keep], v[keep], 1, t_q, len(keep), heads)
    assert np.abs(got - want).max() < 1e-12


def test_oracle_evict_keeps_order_ties_and_holes():
    w = np.array([[5, 1, 1, 9, 1, np.nan, 7, 0]], np.float32)
    assert oracle.evict_order([0], 8, w[0], 16, 1, 4, 0, 0) == [0, 1, 3, 6]        # tie at 1: the lowest slot
    assert oracle.evict_order([0], 8, w[0], 16, 1, 4, 2, 2) == [0, 1, 6, 7]
    assert oracle.evict_order([0], 3, w[0], 16, 1, 4, 0, 0) == [0, 1, 2]
    assert oracle.evict_order([-1, 0], 18, np.zeros(32), 16, 1, 4, 2, 1) == [16, 17]


def test_packed_cache_structure_matches_the_c_layout():
    c = attn.AttnPagedKV.from_buffer_copy(attn._PAGED_KV.pack(*range(1, 11)))
    assert ctypes.sizeof(attn.AttnPagedKV) == attn._PAGED_KV.size
    assert (c.k.ptr, c.k.row_stride, c.v.ptr, c.v.row_stride, c.table, c.kv_lens) == (1, 2, 3, 4, 5, 6)
    assert (c.num_pages, c.page_size, c.pages_per_seq, c.n_kv_heads) == (7, 8, 9, 10)
