"""FP64 oracle of the operators on a paged K/V cache, one sequence, one row and
one slot at a time, straight from the definitions. Shares no code with the CUDA
path. Pools are [num_pages * page_size, n_kv_heads * 64]; slot j of sequence b
is pool row table[b, j // page_size] * page_size + j % page_size, and a table
entry outside [0, num_pages) is a hole whose slots hold nothing."""
from __future__ import annotations

import numpy as np

HEAD_DIM = 64


def clamp_len(n, most: int) -> int:
    return min(max(int(n), 0), most)


def slot_row(table_row, j: int, page_size: int, num_pages: int):
    """The pool row of slot j, or None in a hole."""
    page = int(table_row[j // page_size])
    return page * page_size + j % page_size if 0 <= page < num_pages else None


def sees(p: int, j: int, kv: int, window: int, first: int, causal: bool) -> bool:
    """Whether the row at position p sees slot j (holes aside)."""
    if j >= kv or (causal and j > p):
        return False
    return not window or abs(p - j) < window or j < first


def _sequences(table, lens, q_lens, page_size, num_pages, t_q):
    for b in range(len(table)):
        kv = clamp_len(lens[b], table.shape[1] * page_size)
        q = t_q if q_lens is None else clamp_len(q_lens[b], t_q)
        slots = [(j, slot_row(table[b], j, page_size, num_pages)) for j in range(kv)]
        yield b, kv, q, [(j, r) for j, r in slots if r is not None]


def append(k_new, v_new, k, v, table, lens, page_size, t_new, q_lens=None):
    """The pools after the chunk's rows have been written."""
    k, v = k.copy(), v.copy()
    num_pages = len(k) // page_size
    for b, kv, q, _ in _sequences(table, lens, q_lens, page_size, num_pages, t_new):
        for i in range(q):
            j = i + kv - q
            row = slot_row(table[b], j, page_size, num_pages) if j >= 0 else None
            if row is not None:
                k[row] = k_new[b * t_new + i]
                v[row] = v_new[b * t_new + i]
    return k, v


def attention(q, k, v, table, lens, page_size, t_q, n_heads, n_kv_heads, *, window=0, first=0, causal=True, q_lens=None,
              sinks=None, scale=0.125):
    """(out [batch*t_q, H*64], lse [batch*t_q, H]); a row that sees nothing is 0 with lse -inf."""
    batch, group = len(table), n_heads // n_kv_heads
    out = np.zeros((batch * t_q, n_heads * HEAD_DIM))
    lse = np.full((batch * t_q, n_heads), -np.inf)
    for b, kv, nq, slots in _sequences(table, lens, q_lens, page_size, len(k) // page_size, t_q):
        for i in range(nq):
            p = i + kv - nq
            rows = [r for j, r in slots if sees(p, j, kv, window, first, causal)]
            if not rows:
                continue
            for h in range(n_heads):
                c, g = h * HEAD_DIM, h // group * HEAD_DIM
                s = k[rows, g:g + HEAD_DIM].astype(np.float64) @ q[b * t_q + i, c:c + HEAD_DIM].astype(np.float64) * scale
                m = max(s.max(), sinks[h]) if sinks is not None else s.max()
                e = np.exp(s - m)
                total = e.sum() + (np.exp(sinks[h] - m) if sinks is not None else 0.0)
                out[b * t_q + i, c:c + HEAD_DIM] = e @ v[rows, g:g + HEAD_DIM].astype(np.float64) / total
                lse[b * t_q + i, h] = m + np.log(total)
    return out, lse


def weights(q, k, table, lens, lse, page_size, t_q, n_heads, n_kv_heads, w_in, *, window=0, first=0, causal=True,
            q_lens=None, scale=0.125):
    """w_in plus what the rows put on each slot."""
    w, group = np.array(w_in, dtype=np.float64), n_heads // n_kv_heads
    for b, kv, nq, slots in _sequences(table, lens, q_lens, page_size, len(k) // page_size, t_q):
        for i in range(nq):
            p = i + kv - nq
            seen = [(j, r) for j, r in slots if sees(p, j, kv, window, first, causal)]
            if not seen:
                continue
            at, rows = [j for j, _ in seen], [r for _, r in seen]
            for h in range(n_heads):
                if lse[b * t_q + i, h] == -np.inf:
                    continue
                c, g = h * HEAD_DIM, h // group * HEAD_DIM
                s = k[rows, g:g + HEAD_DIM].astype(np.float64) @ q[b * t_q + i, c:c + HEAD_DIM].astype(np.float64) * scale
                w[b, at] += np.exp(s - np.float64(lse[b * t_q + i, h]))
    return w


def evict_order(table_row, kv: int, w_row, page_size: int, num_pages: int, budget: int, first: int, recent: int):
    """The old slots that stay, in order."""
    held = [j for j in range(kv) if slot_row(table_row, j, page_size, num_pages) is not None]
    always = [j for j in held if j < first or j >= kv - recent]
    value = lambda j: -np.inf if np.isnan(w_row[j]) else float(w_row[j])  # noqa: E731
    rest = sorted((j for j in held if not (j < first or j >= kv - recent)), key=lambda j: (-value(j), j))
    return sorted(always + rest[:max(0, budget - len(always))])


def evict(k, v, table, lens, w_in, page_size, budget, first, recent, k_out, v_out, out_table):
    """(k_out, v_out, kept, lens_out, w_out) after the move."""
    num_pages, out_pages = len(k) // page_size, len(k_out) // page_size
    batch = len(table)
    k_out, v_out = k_out.copy(), v_out.copy()
    kept = np.full((batch, budget), -1, np.int32)
    lens_out = np.zeros(batch, np.int32)
    w_out = np.zeros((batch, out_table.shape[1] * page_size), np.float32)
    for b in range(batch):
        kv = clamp_len(lens[b], table.shape[1] * page_size)
        stay = evict_order(table[b], kv, w_in[b], page_size, num_pages, budget, first, recent)
        lens_out[b] = len(stay)
        kept[b, :len(stay)] = stay
        w_out[b, :len(stay)] = w_in[b, stay]
        for n, j in enumerate(stay):
            row = slot_row(out_table[b], n, page_size, out_pages)
            if row is not None:
                old = slot_row(table[b], j, page_size, num_pages)
                k_out[row], v_out[row] = k[old], v[old]
    return k_out, v_out, kept, lens_out, w_out
