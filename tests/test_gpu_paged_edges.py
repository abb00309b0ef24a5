"""Edges of the paged-cache operators: what a row sees, and values that are not finite."""
import numpy as np
import pytest
import torch

from paged_util import attention64, check_attention, check_weights, make_cache, weights64
from speech_encoder_attention_b200 import attn

pytestmark = pytest.mark.gpu

NAN = float("nan")
INF = float("inf")


@pytest.fixture(autouse=True)
def no_timeouts():
    yield
    st, word = attn.debug_error_word()
    assert st == attn.ATTN_OK, hex(word)


def queries(rng, rows, heads):
    return torch.from_numpy(rng.standard_normal((rows, heads * 64)).astype(np.float16)).cuda()


def i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32).cuda()


# Not causal, and the first tokens reach past the window of the chunk's earlier rows:
# key tiles behind the window part hold first tokens too. "cut" ones share the line of tiles.
OPEN = {
    "whole": dict(lens=[600, 846], t_q=600, page=16, window=64, first=300),
    "whole_ragged": dict(lens=[846, 600], t_q=600, page=128, window=86, first=839, q_lens=[583, 600], holes=[(0, 2)]),
    "cut": dict(lens=[900, 2000], t_q=400, page=64, window=100, first=850),
    "cut_ragged": dict(lens=[2500, 40, 400], t_q=400, page=256, window=33, first=2000, q_lens=[400, 40, 380]),
    "more_rows_than_slots": dict(lens=[300, 500], t_q=420, page=32, window=64, first=200),
    "all_first": dict(lens=[700], t_q=700, page=16, window=30, first=2 ** 31 - 1),
    "step": dict(lens=[700, 300], t_q=6, page=16, window=30, first=600),
}


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("name", OPEN)
def test_first_tokens_past_the_window_are_seen(name, causal):
    c = OPEN[name]
    rng = np.random.default_rng(31)
    batch, t_q, heads, kv_heads = len(c["lens"]), c["t_q"], 4, 2
    cache = make_cache(rng, c["lens"], kv_heads, c["page"], holes=c.get("holes", ()), garbage=NAN)
    q, q_lens = queries(rng, batch * t_q, heads), c.get("q_lens")
    opts = dict(window=c["window"], first=c["first"], causal=causal)
    if not causal:
        assert (attn.paged_workspace_size(cache, batch, t_q, heads, **opts) > 0) == ("cut" in name)
    got, lse = attn.attn_paged(q, cache, batch, t_q, heads, q_lens=i32(q_lens), return_lse=True, **opts)
    want, want_lse, spread = attention64(q, cache, t_q, heads, q_lens=q_lens, **opts)
    check_attention(got, lse, want, want_lse, spread, max(c["lens"]))
    zero = torch.zeros(batch, cache.slots, device="cuda")
    w = attn.attn_paged_weights(q, cache, lse, batch, t_q, heads, q_lens=i32(q_lens), weights=zero, **opts)
    check_weights(w, weights64(q, cache, lse, t_q, heads, zero, q_lens=q_lens, **opts), zero)
    # each row that sees anything hands out a weight of one: 1e-4 per weight, and the sum's own roundings
    seen = (~torch.isinf(lse)).sum().item()
    assert abs(w.double().sum().item() - seen) <= 2e-4 * seen


# Few slots per sequence: a CTA per unit; more: clusters of CTAs; many: units cut into parts.
@pytest.mark.parametrize("slots", [None, 1500, 14000])
@pytest.mark.parametrize("t_q", [1, 16, 100])
def test_a_nan_query_comes_back_as_nan(t_q, slots):
    """A NaN in one row's query for one head makes NaN of that output and lse, and of no other, on every path."""
    rng = np.random.default_rng(32)
    cache = make_cache(rng, [1000, 300], 2, 16, slots=slots)
    assert slots != 14000 or attn.paged_workspace_size(cache, 2, t_q, 4) > 0
    q = queries(rng, 2 * t_q, 4)
    clean, clean_lse = attn.attn_paged(q, cache, 2, t_q, 4, return_lse=True)
    row, head = t_q // 2, 3
    q[row, head * 64 + 5] = NAN
    sinks = torch.zeros(4, device="cuda")
    got, lse = attn.attn_paged(q, cache, 2, t_q, 4, return_lse=True)
    sunk, sunk_lse = attn.attn_paged(q, cache, 2, t_q, 4, sinks=sinks, return_lse=True)
    for o, l in ((got, lse), (sunk, sunk_lse)):
        assert torch.isnan(o[row, head * 64:]).all() and torch.isnan(l[row, head])
        assert torch.isnan(o).sum() == 64 and torch.isnan(l).sum() == 1
    got[row, head * 64:] = clean[row, head * 64:]
    lse[row, head] = clean_lse[row, head]
    assert torch.equal(got, clean) and torch.equal(lse, clean_lse)


@pytest.mark.parametrize("slots", [None, 1500, 14000])
@pytest.mark.parametrize("t_q", [1, 16, 100])
def test_a_cache_of_nan_keys_comes_back_as_nan(t_q, slots):
    """Every key of one head of one sequence is NaN, or only those of its last key tile."""
    rng = np.random.default_rng(33)
    cache = make_cache(rng, [1000, 300], 2, 16, slots=slots)
    q = queries(rng, 2 * t_q, 4)
    clean, clean_lse = attn.attn_paged(q, cache, 2, t_q, 4, return_lse=True)
    for begin in (896, 0):
        for i in range(begin // 16, 63):
            cache.k[int(cache.table[0, i]) * 16:(int(cache.table[0, i]) + 1) * 16, 64:] = NAN
        got, lse = attn.attn_paged(q, cache, 2, t_q, 4, return_lse=True)
        assert torch.isnan(got[:t_q, 128:]).all() and torch.isnan(lse[:t_q, 2:]).all()
        assert torch.equal(got[:t_q, :128], clean[:t_q, :128]) and torch.equal(got[t_q:], clean[t_q:])
        assert torch.equal(lse[:t_q, :2], clean_lse[:t_q, :2]) and torch.equal(lse[t_q:], clean_lse[t_q:])


def slots_seen(cache, b, t_q, row, window, first, causal):
    """Which of sequence b's slots its row sees, [slots] bool."""
    kv = int(cache.lens[b])
    p = row + kv - t_q
    j = torch.arange(cache.slots, device="cuda")
    see = (j < kv) & (j <= p) if causal else j < kv
    if window:
        see &= ((j - p).abs() < window) | (j < first)
    table = cache.table[b].repeat_interleave(cache.page_size)
    return see & (table >= 0) & (table < cache.k.shape[0] // cache.page_size)


# Few slots per sequence: a CTA or a cluster per key tile; many: shares of the line of items.
@pytest.mark.parametrize("slots", [None, 80000])
@pytest.mark.parametrize("window,first,causal", [(0, 0, True), (50, 3, True), (40, 130, False)])
@pytest.mark.parametrize("t_q", [1, 5, 14, 90, 200])
def test_a_nan_lse_reaches_only_the_slots_its_row_sees(t_q, window, first, causal, slots):
    rng = np.random.default_rng(34)
    batch, heads = 2, 4
    cache = make_cache(rng, [300, 250], 2, 16, slots=slots, holes=[(0, 4)], garbage=NAN)
    q = queries(rng, batch * t_q, heads)
    opts = dict(window=window, first=first, causal=causal)
    assert (attn.paged_weights_workspace_size(cache, batch, t_q, heads) > 0) == (slots is not None)
    _, lse, _ = attention64(q, cache, t_q, heads, **opts)
    lse = lse.float().contiguous()
    w_in = torch.from_numpy(rng.random((batch, cache.slots)).astype(np.float32)).cuda()
    clean = attn.attn_paged_weights(q, cache, lse, batch, t_q, heads, weights=w_in, **opts)
    assert torch.isfinite(clean).all()
    for rows in ([0], [t_q // 2, t_q - 1]):
        bad = lse.clone()
        hit = torch.zeros(cache.slots, dtype=torch.bool, device="cuda")
        for n, i in enumerate(rows):
            bad[i, (1 + 2 * n) % heads] = NAN
            hit |= slots_seen(cache, 0, t_q, i, window, first, causal)
        got = attn.attn_paged_weights(q, cache, bad, batch, t_q, heads, weights=w_in, **opts)
        assert torch.isnan(got[0, hit]).all()
        assert torch.equal(got[0, ~hit], clean[0, ~hit]) and torch.equal(got[1], clean[1])


@pytest.mark.parametrize("slots", [None, 80000])
@pytest.mark.parametrize("t_q", [1, 90])
def test_weights_that_overflow_are_infinite(t_q, slots):
    """An lse far below its row's scores is no NaN: e^(s - lse) is infinite where the row sees a slot."""
    rng = np.random.default_rng(36)
    cache = make_cache(rng, [300, 250], 2, 16, slots=slots)
    q = queries(rng, 2 * t_q, 4)
    lse = torch.full((2 * t_q, 4), 8.0, device="cuda")
    clean = attn.attn_paged_weights(q, cache, lse, 2, t_q, 4, window=50)
    lse[t_q + t_q // 2, 1] = -1000.0
    got = attn.attn_paged_weights(q, cache, lse, 2, t_q, 4, window=50)
    hit = slots_seen(cache, 1, t_q, t_q // 2, 50, 0, True)
    assert (got[1, hit] == INF).all() and torch.equal(got[1, ~hit], clean[1, ~hit]) and torch.equal(got[0], clean[0])
    lse[t_q + t_q // 2, 0] = NAN  # of another head
    got = attn.attn_paged_weights(q, cache, lse, 2, t_q, 4, window=50)
    assert torch.isnan(got[1, hit]).all() and torch.equal(got[1, ~hit], clean[1, ~hit])


@pytest.mark.parametrize("slots", [None, 1500, 14000])
@pytest.mark.parametrize("t_q", [12, 100, 300])
def test_a_nan_key_of_a_chunk_stays_with_the_rows_that_see_it(t_q, slots):
    """The key of one of the chunk's own tokens, causal and with a window: earlier rows and later ones are clean."""
    rng = np.random.default_rng(37)
    cache = make_cache(rng, [400, 300], 2, 16, slots=slots)
    q = queries(rng, 2 * t_q, 4)
    clean, clean_lse = attn.attn_paged(q, cache, 2, t_q, 4, window=5, return_lse=True)
    row = t_q // 2
    slot = row + 400 - t_q
    cache.k[int(cache.table[0, slot // 16]) * 16 + slot % 16, :64] = NAN
    got, lse = attn.attn_paged(q, cache, 2, t_q, 4, window=5, return_lse=True)
    w = attn.attn_paged_weights(q, cache, lse, 2, t_q, 4, window=5)
    hit = torch.zeros_like(lse, dtype=torch.bool)
    hit[row:row + 5, :2] = True
    assert torch.isnan(lse[hit]).all() and torch.equal(lse[~hit], clean_lse[~hit])
    assert torch.isnan(got.view(-1, 4, 64)[hit]).all()
    assert torch.equal(got.view(-1, 4, 64)[~hit], clean.view(-1, 4, 64)[~hit])
    seen = torch.zeros_like(w, dtype=torch.bool)
    for i in range(row, row + 5):
        seen[0] |= slots_seen(cache, 0, t_q, i, 5, 0, True)
    assert torch.isnan(w[seen]).all() and torch.isfinite(w[~seen]).all()
