"""Shared helpers of the paged-cache GPU tests: caches with shuffled pages,
garbage where nothing may be read, and a vectorised 64-bit form of the
definitions for sizes the element-wise oracle is too slow for."""
import numpy as np
import torch

from speech_encoder_attention_b200 import attn

D = 64


def make_cache(rng, lens, kv_heads, page, slots=None, spare=2, holes=(), garbage=None, packed=False):
    """A PagedKV on the GPU with the given lengths. Slots behind the end and the
    spare pages hold `garbage` (None: ordinary values); holes: (sequence, page
    index) entries set to -1. packed: K and V are column views of one buffer."""
    batch = len(lens)
    longest = max(max(lens), 1)
    slots = longest if slots is None else slots
    per_seq = -(-slots // page)
    # a table much wider than the sequences has no pages behind their ends
    backed = min(per_seq, -(-2 * longest // page))
    num_pages = batch * backed + spare
    cols = kv_heads * D
    buf = torch.from_numpy(rng.standard_normal((num_pages * page, 2 * cols)).astype(np.float16))
    table = np.full((batch, per_seq), 2 ** 30, np.int32)
    table[:, :backed] = rng.permutation(num_pages)[:batch * backed].reshape(batch, backed)
    for b, i in holes:
        table[b, i] = -1
    if garbage is not None:
        used = np.zeros(num_pages * page, bool)
        for b, n in enumerate(lens):
            for j in range(n):
                if table[b, j // page] >= 0:
                    used[table[b, j // page] * page + j % page] = True
        buf[torch.from_numpy(~used)] = garbage
    # entries behind the end are never looked at
    for b, n in enumerate(lens):
        table[b, -(-n // page):] = 2 ** 30
    buf = buf.cuda()
    if packed:
        k, v = buf[:, :cols], buf[:, cols:]
    else:
        k, v = buf[:, :cols].contiguous(), buf[:, cols:].contiguous()
    return attn.PagedKV(k, v, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), page, kv_heads)


def parts(cache):
    """The cache's host copies: k, v, table, lens."""
    return cache.k.cpu().numpy(), cache.v.cpu().numpy(), cache.table.cpu().numpy(), cache.lens.cpu().numpy()


def attention64(q, cache, t_q, heads, *, window=0, first=0, causal=True, q_lens=None, sinks=None, scale=0.125):
    """(out, lse, spread) in float64 on the GPU; spread = sum_j w_j |v_j|, what a relative
    error of the softmax weights is multiplied by."""
    page, group = cache.page_size, heads // cache.n_kv_heads
    lens, table = cache.lens.tolist(), cache.table.cpu().numpy()
    num_pages = cache.k.shape[0] // page
    batch = len(lens)
    out = torch.zeros(batch * t_q, heads * D, dtype=torch.float64, device="cuda")
    spread = torch.zeros_like(out)
    lse = torch.full((batch * t_q, heads), -np.inf, dtype=torch.float64, device="cuda")
    for b in range(batch):
        kv = min(max(lens[b], 0), cache.slots)
        nq = t_q if q_lens is None else min(max(q_lens[b], 0), t_q)
        if kv == 0 or nq == 0:
            continue
        j = np.arange(kv)
        pages = table[b, j // page]
        j = j[(pages >= 0) & (pages < num_pages)]
        at = torch.from_numpy(table[b, j // page].astype(np.int64) * page + j % page).cuda()
        jj = torch.from_numpy(j).cuda()
        p = (torch.arange(nq, device="cuda") + kv - nq)[:, None]
        see = torch.ones(nq, len(j), dtype=torch.bool, device="cuda")
        if causal:
            see &= jj <= p
        if window:
            see &= ((jj - p).abs() < window) | (jj < first)
        rows = slice(b * t_q, b * t_q + nq)
        for h in range(heads):
            c, g = h * D, h // group * D
            s = q[rows, c:c + D].double() @ cache.k[at, g:g + D].double().T * scale
            s = s.masked_fill(~see, -np.inf)
            if sinks is not None:
                s = torch.cat([s, sinks[h].double().expand(nq, 1)], 1)
            none = ~see.any(1)
            l = torch.where(none, -np.inf, torch.logsumexp(s, 1))
            w = torch.where(none[:, None], 0.0, torch.exp(s - torch.where(none, 0.0, l)[:, None]))[:, :len(j)]
            v = cache.v[at, g:g + D].double()
            out[rows, c:c + D] = w @ v
            spread[rows, c:c + D] = w @ v.abs()
            lse[rows, h] = l
    return out, lse, spread


def weights64(q, cache, lse, t_q, heads, w_in, *, window=0, first=0, causal=True, q_lens=None, scale=0.125):
    """w_in plus the rows' weights, in float64 on the GPU."""
    page, group = cache.page_size, heads // cache.n_kv_heads
    lens, table = cache.lens.tolist(), cache.table.cpu().numpy()
    num_pages = cache.k.shape[0] // page
    w = w_in.double().clone()
    for b, kv in enumerate(lens):
        kv = min(max(kv, 0), cache.slots)
        nq = t_q if q_lens is None else min(max(q_lens[b], 0), t_q)
        if kv == 0 or nq == 0:
            continue
        j = np.arange(kv)
        pages = table[b, j // page]
        j = j[(pages >= 0) & (pages < num_pages)]
        at = torch.from_numpy(table[b, j // page].astype(np.int64) * page + j % page).cuda()
        jj = torch.from_numpy(j).cuda()
        p = (torch.arange(nq, device="cuda") + kv - nq)[:, None]
        see = torch.ones(nq, len(j), dtype=torch.bool, device="cuda")
        if causal:
            see &= jj <= p
        if window:
            see &= ((jj - p).abs() < window) | (jj < first)
        rows = slice(b * t_q, b * t_q + nq)
        for h in range(heads):
            c, g = h * D, h // group * D
            l = lse[rows, h:h + 1].double()
            x = q[rows, c:c + D].double() @ cache.k[at, g:g + D].double().T * scale - torch.where(torch.isinf(l), 0.0, l)
            w[b].index_add_(0, jj, torch.where(see & ~torch.isinf(l), torch.exp(x), 0.0).sum(0))
    return w


def check_attention(got, got_lse, want, lse, spread, n):
    """Element-wise bounds. The softmax weights are rounded to fp16, half a step
    2^-11 of each (2^-25 of the largest where they are subnormal, n of them, times values
    below 6), and so is the output; scores are fp32 sums of 64 products whose
    magnitudes add up to less than 128 here, 64 * 2^-24 * 128 / 8 = 6e-5 in the exponent."""
    got, got_lse = got.double(), got_lse.double()
    assert torch.isfinite(got).all()
    bound = 2.0 ** -11 * (spread + want.abs()) + 2e-4 * spread + n * 6 * 2.0 ** -25 + 2.0 ** -24
    worst = ((got - want).abs() / bound).max().item() if got.numel() else 0.0
    assert worst <= 1.0, f"error is {worst:.2f} of its bound"
    assert torch.equal(torch.isinf(got_lse), torch.isinf(lse))
    seen = ~torch.isinf(lse)
    assert (got_lse[~seen] == -np.inf).all()
    if seen.any():
        assert (got_lse[seen] - lse[seen]).abs().max().item() <= 1e-4


def check_weights(got, want, w_in):
    """Each weight is off by at most the exponent's 6e-5 and a few fp32 roundings."""
    bound = 1e-4 * (want - w_in.double()).abs() + 2.0 ** -22 * want.abs() + 1e-30
    worst = ((got.double() - want).abs() / bound).max().item()
    assert worst <= 1.0, f"error is {worst:.2f} of its bound"
