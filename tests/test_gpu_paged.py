"""The operators on a paged K/V cache against the FP64 oracle on a B200."""
import numpy as np
import pytest
import torch

import oracle.paged as oracle
from paged_util import attention64, check_attention, check_weights, make_cache, parts, weights64
from speech_encoder_attention_b200 import attn

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(autouse=True)
def no_timeouts():
    yield
    st, word = attn.debug_error_word()
    assert st == attn.ATTN_OK, hex(word)


def queries(rng, batch, t_q, heads, wide=0):
    q = torch.from_numpy(rng.standard_normal((batch * t_q, heads * 64 + wide)).astype(np.float16)).cuda()
    return q[:, :heads * 64]


def i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32).cuda()


# batch lengths, t_q, heads, kv heads, page, options
CASES = {
    "one_slot": dict(lens=[1], t_q=1, heads=2, kv=2, page=16),
    "empty": dict(lens=[0, 3], t_q=1, heads=2, kv=1, page=16),
    "step": dict(lens=[37, 128, 129, 255], t_q=1, heads=4, kv=2, page=16),
    "page32": dict(lens=[33, 160], t_q=2, heads=4, kv=4, page=32),
    "page64": dict(lens=[127, 300], t_q=3, heads=5, kv=1, page=64, q_lens=[3, 1]),
    "page128": dict(lens=[131, 260], t_q=1, heads=2, kv=2, page=128),
    "page256": dict(lens=[140, 385, 256], t_q=1, heads=2, kv=1, page=256),
    "block": dict(lens=[100, 64, 17], t_q=16, heads=2, kv=2, page=16, q_lens=[16, 5, 0]),
    "block_open": dict(lens=[100, 150], t_q=16, heads=4, kv=2, page=16, causal=False),
    "window": dict(lens=[300, 40], t_q=1, heads=4, kv=2, page=16, window=30),
    "window_first": dict(lens=[400, 300, 9], t_q=4, heads=4, kv=2, page=16, window=50, first=5),
    "window_one": dict(lens=[200], t_q=8, heads=2, kv=2, page=32, window=1, first=1),
    "window_open": dict(lens=[210, 90], t_q=9, heads=2, kv=2, page=16, window=20, first=3, causal=False),
    "window_wide": dict(lens=[50, 60], t_q=5, heads=2, kv=2, page=16, window=2 ** 31 - 1, first=2 ** 31 - 1),
    "sinks": dict(lens=[70, 0, 200], t_q=2, heads=4, kv=2, page=16, sinks=True),
    "holes": dict(lens=[100, 260], t_q=3, heads=4, kv=2, page=16, holes=[(0, 1), (0, 6), (1, 0), (1, 9), (1, 16)]),
    "all_holes": dict(lens=[30], t_q=2, heads=2, kv=2, page=16, holes=[(0, 0), (0, 1)]),
    "more_rows_than_slots": dict(lens=[3, 7], t_q=12, heads=2, kv=2, page=16),
    "more_rows_open": dict(lens=[3, 140], t_q=12, heads=2, kv=2, page=16, causal=False),
    "chunk": dict(lens=[150, 90], t_q=70, heads=4, kv=2, page=16, q_lens=[70, 33]),
    "chunk_window": dict(lens=[310, 77], t_q=60, heads=2, kv=1, page=32, window=33, first=4),
    "chunk_group": dict(lens=[140], t_q=41, heads=10, kv=2, page=64),
    "chunk_open": dict(lens=[180, 20], t_q=50, heads=2, kv=2, page=128, causal=False, q_lens=[45, 50]),
    "many_heads_on_one": dict(lens=[150, 20], t_q=1, heads=20, kv=1, page=16),
    "group_of_40": dict(lens=[150, 20], t_q=2, heads=40, kv=1, page=16),
    "group_of_128": dict(lens=[130], t_q=3, heads=128, kv=1, page=16),
    "odd_group": dict(lens=[130, 260], t_q=30, heads=7, kv=1, page=16),
}


def inputs(name, slots=None):
    c = CASES[name]
    rng = np.random.default_rng(sum(map(ord, name)))
    cache = make_cache(rng, c["lens"], c["kv"], c["page"], slots=slots, holes=c.get("holes", ()), garbage=NAN,
                       packed=len(name) % 2 == 0)
    batch = len(c["lens"])
    q = queries(rng, batch, c["t_q"], c["heads"], wide=64)
    opts = dict(window=c.get("window", 0), first=c.get("first", 0), causal=c.get("causal", True))
    q_lens = c.get("q_lens")
    if q_lens is not None:  # padding rows hold anything
        for b, n in enumerate(q_lens):
            q[b * c["t_q"] + n:(b + 1) * c["t_q"]] = NAN
    sinks = torch.from_numpy(rng.standard_normal(c["heads"]).astype(np.float32)).cuda() if c.get("sinks") else None
    return c, rng, cache, batch, q, opts, q_lens, sinks


# Few slots per sequence: a CTA or a small cluster per unit; more: eight CTAs; many: units cut into parts.
@pytest.mark.parametrize("slots", [None, 1500, 14000])
@pytest.mark.parametrize("name", CASES)
def test_attention_matches_the_oracle(name, slots):
    c, _, cache, batch, q, opts, q_lens, sinks = inputs(name, slots)
    rows, cols = batch * c["t_q"], c["heads"] * 64
    out = torch.full((rows + 3, cols + 8), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((rows + 3, c["heads"]), 7.0, device="cuda")
    attn.attn_paged(q, cache, batch, c["t_q"], c["heads"], q_lens=i32(q_lens), sinks=sinks, out=out[:rows],
                    lse=lse[:rows], **opts)
    assert (out[:, cols:] == 7.0).all() and (out[rows:] == 7.0).all() and (lse[rows:] == 7.0).all()
    got, lse = out[:rows, :cols], lse[:rows]
    k, v, table, lens = parts(cache)
    args = (table, lens, c["page"], c["t_q"], c["heads"], c["kv"])
    more = dict(q_lens=q_lens, sinks=None if sinks is None else sinks.cpu().numpy().astype(np.float64), **opts)
    qn = q.cpu().numpy()
    want, want_lse = oracle.attention(qn, k, v, *args, **more)
    spread, _ = oracle.attention(qn, k, np.abs(v), *args, **more)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    check_attention(got, lse, dev(want), dev(want_lse), dev(spread), max(c["lens"]))
    # the vectorised form that larger cases are held against says the same
    big, big_lse, _ = attention64(q, cache, c["t_q"], c["heads"], q_lens=q_lens, sinks=sinks, **opts)
    assert (big - dev(want)).abs().max() < 1e-12 and torch.equal(torch.isinf(big_lse), torch.isinf(dev(want_lse)))


# Few slots per sequence: a CTA per key tile; many: shares of the line of items.
@pytest.mark.parametrize("slots", [None, 80000])
@pytest.mark.parametrize("name", [n for n in CASES if "sinks" not in n])
def test_weights_match_the_oracle(name, slots):
    c, rng, cache, batch, q, opts, q_lens, _ = inputs(name, slots)
    assert (attn.paged_weights_workspace_size(cache, batch, c["t_q"], c["heads"]) > 0) == (slots is not None)
    _, lse, _ = attention64(q, cache, c["t_q"], c["heads"], q_lens=q_lens, **opts)
    lse = lse.float().contiguous()
    w_in = torch.from_numpy(rng.random((batch, cache.slots)).astype(np.float32)).cuda()
    got = attn.attn_paged_weights(q, cache, lse, batch, c["t_q"], c["heads"], q_lens=i32(q_lens), weights=w_in, **opts)
    k, _, table, lens = parts(cache)
    want = oracle.weights(q.cpu().numpy(), k, table, lens, lse.cpu().numpy(), c["page"], c["t_q"], c["heads"], c["kv"],
                          w_in.cpu().numpy(), q_lens=q_lens, **opts)
    check_weights(got, torch.from_numpy(want).cuda(), w_in)
    from_zero = attn.attn_paged_weights(q, cache, lse, batch, c["t_q"], c["heads"], q_lens=i32(q_lens), **opts)
    assert (from_zero[torch.from_numpy(want).cuda() == w_in.double()] == 0).all()
    attn.attn_paged_weights(q, cache, lse, batch, c["t_q"], c["heads"], q_lens=i32(q_lens), weights=w_in, out=w_in, **opts)
    assert torch.equal(w_in, got)


LARGE = {
    "step_long": dict(lens=[8191, 3000, 5555, 1, 700], t_q=1, heads=20, kv=20, page=64),
    "step_group": dict(lens=[4097, 12000], t_q=1, heads=20, kv=4, page=16),
    "step_pair": dict(lens=[2500, 1800, 9], t_q=3, heads=20, kv=2, page=32),
    "verify": dict(lens=[1500, 700, 1111, 448, 16], t_q=16, heads=20, kv=20, page=16),
    "prompt": dict(lens=[700, 1500], t_q=1500, heads=4, kv=4, page=64, q_lens=[700, 1500]),
    "prompt_group": dict(lens=[1030], t_q=1030, heads=10, kv=2, page=128),
    "chunk": dict(lens=[3001, 900, 509], t_q=509, heads=20, kv=4, page=128, q_lens=[509, 300, 509]),
    "chunk_window": dict(lens=[4000, 2100], t_q=257, heads=8, kv=8, page=256, window=500, first=4),
    "chunk_open": dict(lens=[1000, 640], t_q=300, heads=6, kv=6, page=16, causal=False),
    "window_step": dict(lens=[16000, 9000, 300], t_q=1, heads=20, kv=5, page=32, window=1024, first=4),
    "many": dict(lens=[5 + 37 * i % 400 for i in range(70)], t_q=2, heads=8, kv=4, page=16),
    "prompt_many": dict(lens=[max(i % 7 * 50, i * 37 % 300) for i in range(31)], t_q=200, heads=20, kv=20, page=64,
                        q_lens=[min(200, max(i % 7 * 50, i * 37 % 300)) for i in range(31)]),
    "many_cut": dict(lens=[5 + 37 * i % 400 for i in range(70)], t_q=2, heads=8, kv=4, page=16, slots=14000),
    "four": dict(lens=[1000, 300, 700], t_q=1, heads=20, kv=20, page=32),
    "two_waves": dict(lens=[200 + 31 * i % 300 for i in range(18)], t_q=1, heads=20, kv=20, page=16),
    "one_cut": dict(lens=[13999, 12001], t_q=1, heads=8, kv=2, page=64, slots=14000),
    "chunk_many_cut": dict(lens=[150 + 37 * i % 400 for i in range(40)], t_q=140, heads=2, kv=1, page=16, slots=4000),
    "chunk_cut": dict(lens=[6001, 900, 2509], t_q=300, heads=20, kv=4, page=128, q_lens=[300, 300, 41]),
    "chunk_many": dict(lens=[150 + 37 * i % 400 for i in range(40)], t_q=140, heads=2, kv=1, page=16),
}


@pytest.mark.parametrize("name", LARGE)
def test_large_attention_and_weights(name):
    c = LARGE[name]
    rng = np.random.default_rng(len(name))
    batch = len(c["lens"])
    cache = make_cache(rng, c["lens"], c["kv"], c["page"], garbage=NAN, slots=c.get("slots"))
    q = queries(rng, batch, c["t_q"], c["heads"])
    q_lens = c.get("q_lens")
    opts = dict(window=c.get("window", 0), first=c.get("first", 0), causal=c.get("causal", True))
    assert "cut" not in name or attn.paged_workspace_size(cache, batch, c["t_q"], c["heads"], **opts) > 0
    got, lse = attn.attn_paged(q, cache, batch, c["t_q"], c["heads"], q_lens=i32(q_lens), return_lse=True, **opts)
    want, want_lse, spread = attention64(q, cache, c["t_q"], c["heads"], q_lens=q_lens, **opts)
    check_attention(got, lse, want, want_lse, spread, max(c["lens"]))
    again, _ = attn.attn_paged(q, cache, batch, c["t_q"], c["heads"], q_lens=i32(q_lens), return_lse=True, **opts)
    assert torch.equal(got, again)
    w_in = torch.from_numpy(rng.random((batch, cache.slots)).astype(np.float32)).cuda()
    w = attn.attn_paged_weights(q, cache, lse, batch, c["t_q"], c["heads"], q_lens=i32(q_lens), weights=w_in, **opts)
    check_weights(w, weights64(q, cache, lse, c["t_q"], c["heads"], w_in, q_lens=q_lens, **opts), w_in)
    assert torch.equal(w, attn.attn_paged_weights(q, cache, lse, batch, c["t_q"], c["heads"], q_lens=i32(q_lens),
                                                  weights=w_in, **opts))


def test_values_of_unseen_slots_do_not_matter():
    """Slots outside the window hold infinities and NaN; the result is that of clean ones."""
    rng = np.random.default_rng(5)
    cache = make_cache(rng, [500], 2, 16)
    q = queries(rng, 1, 1, 2)
    clean = attn.attn_paged(q, cache, 1, 1, 2, window=100, first=3)
    for bad in (NAN, float("inf"), -65504.0):
        for j in list(range(3, 400)) + list(range(500, 512)):
            row = int(cache.table[0, j // 16]) * 16 + j % 16 if j < 500 else None
            if row is not None:
                cache.k[row] = bad
                cache.v[row] = bad
        assert torch.equal(attn.attn_paged(q, cache, 1, 1, 2, window=100, first=3), clean)


def test_large_scores_and_extreme_values():
    """Scores up to about 700 and rows whose max grows through the cache."""
    rng = np.random.default_rng(6)
    cache = make_cache(rng, [700, 260], 2, 16)
    for b, n in enumerate([700, 260]):
        for j in range(n):
            cache.k[int(cache.table[b, j // 16]) * 16 + j % 16] *= 0.02 * (j % 97)
    q = queries(rng, 2, 3, 2) * 8
    got, lse = attn.attn_paged(q, cache, 2, 3, 2, return_lse=True)
    want, want_lse, spread = attention64(q, cache, 3, 2)
    # the exponent's error grows with the products: magnitudes add up to under 64 * 8 * 2 * 16 here
    exponent = 64 * 2.0 ** -24 * 16384 / 8
    assert ((got.double() - want).abs() <= (2.0 ** -10 + 2 * exponent) * (spread + want.abs()) + 1e-3).all()
    assert (lse.double() - want_lse).abs().max() <= exponent + 2.0 ** -22 * want_lse.abs().max()


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("page,t_new,lens,q_lens", [
    (16, 1, [1, 16, 17, 40], None), (32, 5, [5, 64, 3, 33], [5, 2, 0, 5]), (256, 70, [300, 70], None),
    (16, 9, [4, 100], None),  # more rows than slots: the first ones have nowhere to go
])
def test_append_writes_the_slots_and_nothing_else(page, t_new, lens, q_lens, packed):
    rng = np.random.default_rng(page + t_new)
    cache = make_cache(rng, lens, 3, page, packed=packed, holes=[(len(lens) - 1, 0)])
    new = torch.from_numpy(rng.standard_normal((len(lens) * t_new, 3 * 192)).astype(np.float16)).cuda()
    kn, vn = new[:, 192:384], new[:, 384:]
    k, v, table, ln = parts(cache)
    want_k, want_v = oracle.append(kn.cpu().numpy(), vn.cpu().numpy(), k, v, table, ln, page, t_new, q_lens)
    attn.attn_paged_append(kn, vn, cache, len(lens), t_new, q_lens=i32(q_lens))
    assert np.array_equal(cache.k.cpu().numpy(), want_k) and np.array_equal(cache.v.cpu().numpy(), want_v)


EVICT = [
    dict(lens=[40, 100, 8, 0], budget=32, first=4, recent=8, page=16),
    dict(lens=[300, 31], budget=30, first=0, recent=0, page=32),
    dict(lens=[1500, 1100, 700], budget=513, first=3, recent=100, page=64),
    dict(lens=[5000], budget=1000, first=1000, recent=0, page=128),
    dict(lens=[2500, 2048], budget=1024, first=0, recent=1024, page=256),
    dict(lens=[50], budget=1, first=0, recent=0, page=16),
    dict(lens=[20, 90], budget=64, first=2, recent=3, page=16, holes=[(0, 1), (1, 0), (1, 3)]),
    dict(lens=[33], budget=12, first=2, recent=2, page=16, holes=[(0, 0), (0, 1), (0, 2)]),
    dict(lens=[70001], budget=3001, first=7, recent=500, page=256),  # more keys than shared memory holds
]


def weights_of(kind, rng, shape):
    w = rng.random(shape).astype(np.float32)
    if kind == "ties":
        w = np.floor(w * 3).astype(np.float32)
    elif kind == "equal":
        w[:] = 0.25
    elif kind == "odd":
        w = ((w - 0.5) * 1e-3).astype(np.float32)
        pick = rng.random(shape)
        w[pick < 0.1] = np.nan
        w[(pick > 0.1) & (pick < 0.2)] = -np.inf
        w[(pick > 0.2) & (pick < 0.25)] = np.inf
        w[(pick > 0.3) & (pick < 0.4)] = -0.0
        w[(pick > 0.4) & (pick < 0.5)] = 0.0
    return w


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "odd"])
@pytest.mark.parametrize("case", EVICT)
@pytest.mark.parametrize("where", ["other", "pages", "place"])
def test_evict_matches_the_oracle(case, kind, where):
    rng = np.random.default_rng(case["budget"])
    batch, page, budget = len(case["lens"]), case["page"], case["budget"]
    cache = make_cache(rng, case["lens"], 3, page, slots=max(max(case["lens"]), budget), holes=case.get("holes", ()),
                       spare=2 + batch * -(-budget // page))
    w = torch.from_numpy(weights_of(kind, rng, (batch, cache.slots))).cuda()
    k, v, table, lens = parts(cache)
    if where == "place":
        # a destination needs its pages; entries behind the end and holes get unused ones
        free = [i for i in range(len(k) // page) if i not in set(table.reshape(-1).tolist())]
        full = table.copy()
        for b in range(batch):
            for i in range(table.shape[1]):
                if not 0 <= full[b, i] < len(k) // page:
                    full[b, i] = free.pop()
        dst = attn.PagedKV(cache.k, cache.v, torch.from_numpy(full).cuda(), cache.lens, page, 3)
    elif where == "pages":  # other pages of the same pool
        used = set(table.reshape(-1).tolist())
        free = [i for i in range(len(k) // page) if i not in used][:batch * -(-budget // page)]
        dst = attn.PagedKV(cache.k, cache.v, torch.tensor(free, dtype=torch.int32).view(batch, -1).cuda(),
                           torch.zeros(batch, dtype=torch.int32).cuda(), page, 3)
    else:
        dst = make_cache(rng, [budget] * batch, 3, page)
    _, _, out_table, _ = parts(dst)
    k_out, v_out = dst.k.cpu().numpy(), dst.v.cpu().numpy()
    want = oracle.evict(k, v, table, lens, w.cpu().numpy(), page, budget, case["first"], case["recent"], k_out, v_out, out_table)
    w_out = w if where == "place" else None
    kept, w_got = attn.attn_paged_evict(cache, w, budget, case["first"], case["recent"], dst=dst, weights_out=w_out)
    got = (dst.k.cpu().numpy(), dst.v.cpu().numpy(), kept.cpu().numpy(), dst.lens.cpu().numpy(), w_got.cpu().numpy())
    for name, g, x in zip(("k", "v", "kept", "lens", "weights"), got, want):
        assert np.array_equal(g, x, equal_nan=g.dtype.kind == "f"), name


def test_a_decode_loop_with_eviction():
    """Prompt, then decode steps that append, attend, weigh and evict when full, against the oracle."""
    rng = np.random.default_rng(11)
    batch, heads, kv_heads, page, budget, slots = 2, 4, 2, 16, 48, 96
    cache = make_cache(rng, [slots, slots], kv_heads, page)
    lens = np.array([30, 21], np.int32)
    cache.lens.copy_(torch.from_numpy(lens))
    w = torch.zeros(batch, slots, device="cuda")
    steps = [(30, [30, 21])] + [(1, None)] * 45 + [(7, [7, 3])] + [(1, None)] * 25
    evicted = 0
    for n, (t, q_lens) in enumerate(steps):
        if n:
            lens = lens + (np.array(q_lens, np.int32) if q_lens else t)
            cache.lens.copy_(torch.from_numpy(lens.astype(np.int32)))
        qkv = torch.from_numpy(rng.standard_normal((batch * t, 64 * (heads + 2 * kv_heads))).astype(np.float16)).cuda()
        q, kn, vn = qkv[:, :64 * heads], qkv[:, 64 * heads:64 * (heads + kv_heads)], qkv[:, 64 * (heads + kv_heads):]
        k, v, table, ln = parts(cache)
        want_k, want_v = oracle.append(kn.cpu().numpy(), vn.cpu().numpy(), k, v, table, ln, page, t, q_lens)
        attn.attn_paged_append(kn, vn, cache, batch, t, q_lens=i32(q_lens))
        assert np.array_equal(cache.k.cpu().numpy(), want_k) and np.array_equal(cache.v.cpu().numpy(), want_v)
        got, lse = attn.attn_paged(q, cache, batch, t, heads, window=40, first=4, q_lens=i32(q_lens), return_lse=True)
        want, want_lse, spread = attention64(q, cache, t, heads, window=40, first=4, q_lens=q_lens)
        check_attention(got, lse, want, want_lse, spread, slots)
        before = w.clone()
        attn.attn_paged_weights(q, cache, lse, batch, t, heads, window=40, first=4, q_lens=i32(q_lens), weights=w, out=w)
        check_weights(w, weights64(q, cache, lse, t, heads, before, window=40, first=4, q_lens=q_lens), before)
        if lens.max() >= slots - 7:
            k, v, table, ln = parts(cache)
            want = oracle.evict(k, v, table, ln, w.cpu().numpy(), page, budget, 4, 16, k, v, table)
            kept, _ = attn.attn_paged_evict(cache, w, budget, 4, 16, weights_out=w)
            for g, x in zip((cache.k, cache.v, kept, cache.lens, w), want):
                assert np.array_equal(g.cpu().numpy(), x)
            lens, evicted = want[3].copy(), evicted + 1
    assert evicted >= 1


@pytest.mark.parametrize("slots", [400, 16000])
def test_captured_step_follows_its_inputs(slots):
    """One captured decode step replayed while lengths, pages and rows change."""
    rng = np.random.default_rng(12)
    batch, heads, page = 3, 4, 16
    cache = make_cache(rng, [400, 400, 400], 4, page, slots=slots)
    q = queries(rng, batch, 1, heads)
    w = torch.zeros(batch, cache.slots, device="cuda")
    out = torch.empty(batch, heads * 64, dtype=torch.float16, device="cuda")
    lse = torch.empty(batch, heads, device="cuda")
    ws = torch.empty(attn.paged_workspace_size(cache, batch, 1, heads), dtype=torch.uint8, device="cuda")

    def step():
        attn.attn_paged_append(q, q, cache, batch, 1)
        attn.attn_paged(q, cache, batch, 1, heads, out=out, lse=lse, workspace=ws)
        attn.attn_paged_weights(q, cache, lse, batch, 1, heads, out=w)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([1, 200, 400], [399, 0, 17], [128, 129, 16]):
        cache.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        q.copy_(queries(rng, batch, 1, heads))
        graph.replay()
        want, want_lse, spread = attention64(q, cache, 1, heads)
        check_attention(out, lse, want, want_lse, spread, 400)
        check_weights(w, weights64(q, cache, lse, 1, heads, torch.zeros_like(w)), torch.zeros_like(w))


def test_two_streams_at_once():
    rng = np.random.default_rng(13)
    jobs = []
    for i in range(2):
        cache = make_cache(rng, [3000 + i, 1700], 8, 64)
        q = queries(rng, 2, 1 + 39 * i, 8)
        jobs.append((cache, q, 1 + 39 * i, torch.cuda.Stream()))
    alone = [attn.attn_paged(q, c, 2, t, 8) for c, q, t, _ in jobs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [attn.attn_paged(q, c, 2, t, 8, stream=s) for c, q, t, s in jobs]
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert torch.equal(a, b)


def test_pools_beyond_32_bit_offsets():
    """The last pages of a pool of 2^31 values and more (4.3 GB)."""
    page, kv_heads = 256, 20
    pages = 2 ** 31 // (page * 2 * kv_heads * 64) + 3
    buf = torch.empty(pages * page, 2 * kv_heads * 64, dtype=torch.float16, device="cuda")
    rng = np.random.default_rng(14)
    lens = [300, 700]
    table = torch.tensor([[pages - 1, 0, 2 ** 30], [pages - 2, pages - 3, 1]], dtype=torch.int32, device="cuda")
    cache = attn.PagedKV(buf[:, :1280], buf[:, 1280:], table, i32(lens), page, kv_heads)
    for p in (0, 1, pages - 3, pages - 2, pages - 1):
        buf[p * page:(p + 1) * page] = torch.from_numpy(rng.standard_normal((page, 2560)).astype(np.float16)).cuda()
    q = queries(rng, 2, 1, kv_heads)
    attn.attn_paged_append(q, q, cache, 2, 1)
    assert torch.equal(buf[(pages - 1) * page * 0 + 43, :1280], q[0]) and torch.equal(buf[1 * page + 187, 1280:], q[1])
    got, lse = attn.attn_paged(q, cache, 2, 1, kv_heads, return_lse=True)
    check_attention(got, lse, *attention64(q, cache, 1, kv_heads), 700)
    zero = torch.zeros(2, cache.slots, device="cuda")
    w = attn.attn_paged_weights(q, cache, lse, 2, 1, kv_heads, weights=zero)
    check_weights(w, weights64(q, cache, lse, 1, kv_heads, zero), zero)
    rows = lambda b, js: [int(table[b, j // page]) * page + j % page for j in js]  # noqa: E731
    src = buf.index_select(0, torch.tensor(rows(1, range(700)), device="cuda"))
    kept, _ = attn.attn_paged_evict(cache, w, 400, 4, 100)
    assert torch.equal(buf[torch.tensor(rows(1, range(400)), device="cuda")], src[kept[1].long()])


def test_another_device_and_stream_are_refused_or_followed():
    rng = np.random.default_rng(15)
    cache = make_cache(rng, [90], 2, 16)
    q = queries(rng, 1, 1, 2)
    want = attn.attn_paged(q, cache, 1, 1, 2)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = attn.attn_paged(q, cache, 1, 1, 2, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    with pytest.raises(ValueError):
        attn.attn_paged(q[:, :64], cache, 1, 1, 2)
    with pytest.raises(ValueError):
        attn.attn_paged(q, cache, 1, 2, 2)
    with pytest.raises(ValueError):
        attn.attn_paged(q, cache, 2, 1, 2)
    long = make_cache(rng, [90], 2, 16, slots=14000)
    assert attn.paged_workspace_size(cache, 1, 1, 2) == 0 < attn.paged_workspace_size(long, 1, 1, 2)
    with pytest.raises(attn.AttnError):
        attn.attn_paged(q, long, 1, 1, 2, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("t_q", [1, 12, 40])
def test_nan_that_a_row_sees_comes_back_as_nan(t_q):
    """A NaN key makes NaN of the rows that see it, and of no other sequence or head."""
    rng = np.random.default_rng(16)
    cache = make_cache(rng, [200, 90], 2, 16)
    q = queries(rng, 2, t_q, 4)
    clean, clean_lse = attn.attn_paged(q, cache, 2, t_q, 4, return_lse=True)
    cache.k[int(cache.table[0, 3]) * 16 + 2, :64] = NAN
    got, lse = attn.attn_paged(q, cache, 2, t_q, 4, return_lse=True)
    assert torch.isnan(got[:t_q, :128]).all() and torch.isnan(lse[:t_q, :2]).all()
    assert torch.equal(got[:t_q, 128:], clean[:t_q, 128:]) and torch.equal(got[t_q:], clean[t_q:])
    assert torch.equal(lse[t_q:], clean_lse[t_q:])


@pytest.mark.parametrize("slots", [None, 1500, 14000])
@pytest.mark.parametrize("t_q", [1, 40])
def test_sinks_far_above_and_below_the_scores(t_q, slots):
    """A sink of 300 takes all the weight (output 0, lse the sink); one of -300 or -inf takes none."""
    rng = np.random.default_rng(17)
    cache = make_cache(rng, [200, 77], 4, 16, slots=slots)
    q = queries(rng, 2, t_q, 4)
    sinks = torch.tensor([300.0, -300.0, -float("inf"), 2.0], device="cuda")
    got, lse = attn.attn_paged(q, cache, 2, t_q, 4, sinks=sinks, return_lse=True)
    check_attention(got, lse, *attention64(q, cache, t_q, 4, sinks=sinks), 200)
    assert (got[:, :64] == 0).all() and ((lse[:, 0] - 300.0).abs() <= 2.0 ** -14).all()  # 2 roundings of 300


@pytest.mark.parametrize("bad", [dict(budget=2 ** 32 + 8), dict(budget=33), dict(budget=0), dict(budget=-1), dict(first=2 ** 32 + 1),
                                 dict(first=-1), dict(recent=2 ** 32), dict(recent=-2)])
def test_evictions_that_do_not_fit_are_refused(bad):
    rng = np.random.default_rng(19)
    cache = make_cache(rng, [20], 1, 16)
    before = cache.k.clone()
    w = torch.zeros(1, cache.slots, device="cuda")
    fits = all(0 <= x < 2 ** 31 for x in bad.values())  # then the library refuses it
    with pytest.raises(attn.AttnError if fits else ValueError):
        attn.attn_paged_evict(cache, w, **{"budget": 8, **bad})
    assert torch.equal(cache.k, before) and cache.lens.item() == 20
    for t_q, heads in ((2 ** 32 + 1, 1), (1, 2 ** 32 + 1), (0, 1), (1, 0)):
        with pytest.raises(ValueError):
            attn.paged_workspace_size(cache, 1, t_q, heads)
        with pytest.raises(ValueError):
            attn.paged_weights_workspace_size(cache, 1, t_q, heads)


def test_numbers_that_do_not_fit_are_refused():
    rng = np.random.default_rng(18)
    cache = make_cache(rng, [20], 1, 16)
    q = queries(rng, 1, 1, 1)
    for bad in (dict(window=2 ** 32 + 1), dict(window=-1), dict(window=4, first=2 ** 31)):
        with pytest.raises(ValueError):
            attn.attn_paged(q, cache, 1, 1, 1, **bad)
    with pytest.raises(attn.AttnError):
        attn.attn_paged(q, cache, 1, 1, 1, first=3)
    with pytest.raises(attn.AttnError):
        attn.attn_paged_evict(cache, torch.zeros(1, 32, device="cuda"), 33)


@pytest.mark.parametrize("t_q", [1, 20, 50])
def test_lengths_out_of_range_are_clamped(t_q):
    rng = np.random.default_rng(19)
    cache = make_cache(rng, [96, 96, 96], 2, 16)
    q = queries(rng, 3, t_q, 4)
    wild = attn.PagedKV(cache.k, cache.v, cache.table, i32([2 ** 31 - 1, -5, 50]), 16, 2)
    tame = attn.PagedKV(cache.k, cache.v, cache.table, i32([96, 0, 50]), 16, 2)
    got, lse = attn.attn_paged(q, wild, 3, t_q, 4, q_lens=i32([2 ** 31 - 1, 3, -(2 ** 31)]), return_lse=True)
    want, want_lse = attn.attn_paged(q, tame, 3, t_q, 4, q_lens=i32([t_q, 3, 0]), return_lse=True)
    assert torch.equal(got, want) and torch.equal(lse, want_lse) and (got[t_q:] == 0).all()
    w = attn.attn_paged_weights(q, wild, lse, 3, t_q, 4, q_lens=i32([2 ** 31 - 1, 3, -(2 ** 31)]))
    assert torch.equal(w, attn.attn_paged_weights(q, tame, lse, 3, t_q, 4, q_lens=i32([t_q, 3, 0])))


@pytest.mark.parametrize("t_q", [1, 40])
def test_sequences_may_share_pages(t_q):
    """A common prefix held once, and one page twice in a row."""
    rng = np.random.default_rng(20)
    cache = make_cache(rng, [200, 160, 90], 2, 16)
    cache.table[1, :6] = cache.table[0, :6]
    cache.table[2, 3] = cache.table[2, 2]
    q = queries(rng, 3, t_q, 4)
    got, lse = attn.attn_paged(q, cache, 3, t_q, 4, return_lse=True)
    check_attention(got, lse, *attention64(q, cache, t_q, 4), 200)
    zero = torch.zeros(3, cache.slots, device="cuda")
    w = attn.attn_paged_weights(q, cache, lse, 3, t_q, 4, weights=zero)
    check_weights(w, weights64(q, cache, lse, t_q, 4, zero), zero)


def test_captured_eviction_follows_its_inputs():
    rng = np.random.default_rng(21)
    cache = make_cache(rng, [300, 300], 2, 16)
    w = torch.zeros(2, cache.slots, device="cuda")
    kept = torch.empty(2, 64, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        attn.attn_paged_evict(cache, w, 64, 2, 10, kept=kept, weights_out=w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.attn_paged_evict(cache, w, 64, 2, 10, kept=kept, weights_out=w)
    for lens in ([300, 100], [64, 65], [0, 299]):
        cache.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        w.copy_(torch.from_numpy(rng.random((2, cache.slots)).astype(np.float32)))
        k, v, table, ln = parts(cache)
        want = oracle.evict(k, v, table, ln, w.cpu().numpy(), 16, 64, 2, 10, k, v, table)
        graph.replay()
        for g, x in zip((cache.k, cache.v, kept, cache.lens, w), want):
            assert np.array_equal(g.cpu().numpy(), x)


def test_everything_at_once_on_three_streams():
    """Appends, attention, weights and evictions of unrelated caches overlap."""
    rng = np.random.default_rng(22)

    def job(i, stream):
        cache = caches[i]
        attn.attn_paged_append(q[i], q[i], cache, 2, 1 + 40 * i, stream=stream)
        out, lse = attn.attn_paged(q[i], cache, 2, 1 + 40 * i, 4, return_lse=True, stream=stream)
        w = attn.attn_paged_weights(q[i], cache, lse, 2, 1 + 40 * i, 4, stream=stream)
        kept, w2 = attn.attn_paged_evict(cache, w, 500, 4, 100, stream=stream)
        return out, lse, w, kept, w2, cache.k.clone(), cache.v.clone(), cache.lens.clone()

    base = [make_cache(rng, [2000 + i, 1700], 4, 64, slots=16000 if i == 1 else None) for i in range(3)]
    q = [queries(rng, 2, 1 + 40 * i, 4) for i in range(3)]

    def fresh():
        return [attn.PagedKV(c.k.clone(), c.v.clone(), c.table, c.lens.clone(), 64, 4) for c in base]

    caches = fresh()
    alone = []
    for i in range(3):
        alone.append(job(i, None))
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(3):
        caches = fresh()
        torch.cuda.synchronize()
        got = [None] * 3
        for i in range(3):
            with torch.cuda.stream(streams[i]):  # the clones at the end belong to the stream too
                got[i] = job(i, streams[i])
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
