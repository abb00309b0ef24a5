"""The operators on a paged K/V cache, as cases to be timed and compared.

A cache is a pool of pages: K and V pools of `num_pages * page_size` rows, a
page table per sequence and the sequences' lengths (new tokens included).
Four operators work on it:

  append   writes a chunk's new K and V rows into their slots
  attend   attention of a chunk of new tokens over the cache, causal, whole or
           within a window plus the first tokens
  weights  adds each slot's attention weight, summed over query rows and heads
  evict    keeps the first, the latest and the heaviest slots up to a budget

`run` takes them in plain torch operations in 32 bits, or, with `own`, through
the package's entry points.
"""
import math

import numpy as np
import torch

own = False

D = 64  # head size


def listed():
    return [
        # one decode step's new rows of 32 streams
        dict(name="append_step", op="append", batch=32, t=1, kv_heads=20, page=16, length=447, ragged=False),
        # the prompt rows of eight windows, read from the packed projection's buffer
        dict(name="append_windows", op="append", batch=8, t=1500, kv_heads=20, page=64, length=1500, ragged=False),
        # one token of one stream over a decoder's 448 slots: latency
        dict(name="attend_one", op="attend", batch=1, t=1, heads=20, kv_heads=20, page=16, length=448, ragged=False,
             window=0, first=0, causal=True),
        # a block of drafted tokens of five beams verified over the cache
        dict(name="attend_verify", op="attend", batch=5, t=16, heads=20, kv_heads=20, page=16, length=1500, ragged=True,
             window=0, first=0, causal=True),
        # one token each of 16 long transcripts: bound by reading the cache
        dict(name="attend_step_long", op="attend", batch=16, t=1, heads=20, kv_heads=20, page=64, length=8191,
             ragged=True, window=0, first=0, causal=True),
        # one token each of 48 streams that see a window and the first tokens; pages in between are given back
        dict(name="attend_step_window", op="attend", batch=48, t=1, heads=20, kv_heads=5, page=32, length=16000,
             ragged=True, window=1024, first=4, causal=True),
        # a chunk of a long prompt over what is there already, grouped heads, ragged chunks
        dict(name="attend_chunk", op="attend", batch=4, t=509, heads=20, kv_heads=4, page=128, length=6007, ragged=True,
             window=0, first=0, causal=True),
        # eight whole prompts: bound by the products and the exponentials
        dict(name="attend_prompt", op="attend", batch=8, t=1500, heads=20, kv_heads=20, page=64, length=1500,
             ragged=False, window=0, first=0, causal=True),
        # a decode step's weights over long caches
        dict(name="weights_step", op="weights", batch=16, t=1, heads=20, kv_heads=20, page=64, length=8191, ragged=True,
             window=0, first=0, causal=True),
        # the weights of whole prompts
        dict(name="weights_prompt", op="weights", batch=4, t=1500, heads=20, kv_heads=20, page=64, length=1500,
             ragged=False, window=0, first=0, causal=True),
        # five beams' caches of 448 slots down to 256
        dict(name="evict_beams", op="evict", batch=5, kv_heads=20, page=16, length=448, ragged=True, budget=256, first=4,
             recent=64),
        # eight long caches down to a quarter
        dict(name="evict_long", op="evict", batch=8, kv_heads=20, page=64, length=16000, ragged=True, budget=4096,
             first=4, recent=1024),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "weights", "evict"])
    page = rng.choice([16, 32, 64, 128, 256])
    heads, kv_heads = rng.choice([(20, 20), (20, 5), (20, 4), (8, 8), (8, 2), (5, 5), (12, 1)])
    ragged = rng.random() < 0.7
    if op == "append":
        t = _log_int(rng, 1, 1500)
        return dict(op=op, batch=_log_int(rng, 1, max(1, min(64, 11000 // t))), t=t, kv_heads=kv_heads, page=page,
                    length=t + rng.randrange(0, 512), ragged=ragged)
    if op == "evict":
        length = _log_int(rng, 64, 16000)
        budget = max(32, int(length * rng.uniform(0.2, 0.9)))
        return dict(op=op, batch=_log_int(rng, 1, 8), kv_heads=kv_heads, page=page, length=length, ragged=ragged,
                    budget=budget, first=rng.randrange(0, 9), recent=rng.randrange(0, max(1, budget // 2)))
    t = rng.choice([1, 1, _log_int(rng, 2, 32), _log_int(rng, 33, 1500)])
    length = max(t, _log_int(rng, 32, 12000 if t <= 32 else 5000))
    most = min(16 * 8191 // (2 * length), 4 * 1500 * 1500 // (t * length))
    batch = _log_int(rng, 1, max(1, min(48, most)))
    window = rng.choice([0, 0, _log_int(rng, 1, 2048)])
    return dict(op=op, batch=batch, t=t, heads=heads, kv_heads=kv_heads, page=page, length=length, ragged=ragged,
                window=window, first=rng.randrange(0, 9) if window else 0, causal=rng.random() < 0.85)


# ---------------------------------------------------------------------------
# sizes that follow from a case
# ---------------------------------------------------------------------------

def _spread(case, b):
    """A fixed fraction in [0, 1) for sequence b; 0 for sequences of one length."""
    return (b * 0.6180339887498949) % 1.0 if case["ragged"] else 0.0


def _lens(case):
    """Slots in use, per sequence: from the full length down to a third of it."""
    n = [max(1, int(case["length"] * (1.0 - 0.66 * _spread(case, b)))) for b in range(case["batch"])]
    return n


def _new(case):
    """New tokens, per sequence (at most the sequence's slots)."""
    return [max(1, min(n, int(math.ceil(case["t"] * (1.0 - 0.5 * _spread(case, b))))))
            for b, n in enumerate(_lens(case))]


def _seen(case):
    """Per sequence: (visible pairs of query row and slot, slots that some row sees)."""
    got = []
    for kv, q in zip(_lens(case), _new(case)):
        p = np.arange(kv - q, kv)
        hi = p + 1 if case["causal"] else np.full_like(p, kv)
        if not case["window"]:
            got.append((int(hi.sum()), int(hi.max())))
            continue
        w = case["window"]
        hi_w = np.minimum(hi, p + w)
        lo = np.maximum(0, p - w + 1)
        head = np.minimum(np.minimum(case["first"], lo), hi)
        any_first = int(min(case["first"], hi.max()))
        got.append((int((hi_w - lo + head).sum()), int(hi_w.max() - min(lo.min(), hi_w.max()) + min(any_first, lo.min()))))
    return got


def work(case):
    lens = _lens(case)
    if case["op"] == "append":
        rows = sum(_new(case))
        return {"bytes": 2.0 * 2 * rows * case["kv_heads"] * D * 2, "flops": 0.0}
    if case["op"] == "evict":
        slots = case["batch"] * _pages(case) * case["page"]
        kept = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": 2.0 * 2 * kept * case["kv_heads"] * D * 2 + 4.0 * (sum(lens) + slots + case["batch"] * case["budget"]),
                "flops": 0.0}
    seen = _seen(case)
    pairs, slots, rows = sum(s[0] for s in seen), sum(s[1] for s in seen), sum(_new(case))
    row = case["heads"] * D * 2
    slot = case["kv_heads"] * D * 2
    if case["op"] == "attend":
        padded = case["batch"] * case["t"]
        return {"bytes": float(rows * row + padded * (row + 4 * case["heads"]) + 2 * slots * slot),
                "flops": 4.0 * D * case["heads"] * pairs}
    return {"bytes": float(rows * (row + 4 * case["heads"]) + slots * (slot + 8)), "flops": 2.0 * D * case["heads"] * pairs}


def _pages(case):
    return (case["length"] + case["page"] - 1) // case["page"]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * (seed + 1) + 17)
    batch, page, cols = case["batch"], case["page"], case["kv_heads"] * D
    per_seq = _pages(case)
    lens = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
    num_pages = batch * per_seq + 3
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda", dtype=torch.float16)  # noqa: E731
    # a program that has run for a while: pages in no order, those behind a sequence's end not handed out
    table = torch.randperm(num_pages, generator=g, device="cuda")[: batch * per_seq].to(torch.int32).view(batch, per_seq)
    place = torch.arange(per_seq, device="cuda") * page
    table = torch.where(place[None, :] < lens[:, None], table, -1)
    s = dict(case=dict(case), batch=batch, page=page, lens=lens, num_pages=num_pages,
             k=normal(num_pages * page, cols), v=normal(num_pages * page, cols))
    if case["op"] == "evict":
        slots = per_seq * page
        # few slots carry most of the weight; some have never been looked at
        w = torch.rand(batch, slots, generator=g, device="cuda") ** 8 * 20.0
        w = torch.where(torch.rand(batch, slots, generator=g, device="cuda") < 0.2, torch.zeros_like(w), w)
        s["weights"] = torch.where(torch.arange(slots, device="cuda")[None, :] < lens[:, None], w, 0.0)
        out_pages = (case["budget"] + page - 1) // page
        s["out_table"] = torch.randperm(batch * out_pages, generator=g, device="cuda").to(torch.int32).view(batch, out_pages)
        s["k_out"] = torch.zeros(batch * out_pages * page, cols, dtype=torch.float16, device="cuda")
        s["v_out"] = torch.zeros_like(s["k_out"])
        s["table"] = table.contiguous()
        return s
    s["t"] = t = case["t"]
    s["q_lens"] = torch.tensor(_new(case), dtype=torch.int32, device="cuda")
    if case["op"] == "append":
        packed = normal(batch * t, 3 * cols)  # the projection's buffer: q, k and v columns
        s["k_new"], s["v_new"] = packed[:, cols: 2 * cols], packed[:, 2 * cols:]
        s["table"] = table.contiguous()
        return s
    if case["window"]:
        # pages that no row sees any more are given back
        lo = (lens - s["q_lens"] - case["window"] + 1)[:, None]
        gone = (place[None, :] + page <= lo) & (place[None, :] >= case["first"])
        table = torch.where(gone, -1, table)
    s["table"] = table.contiguous()
    s["q"] = normal(batch * t, case["heads"] * D)
    s["scale"] = D ** -0.5
    if case["op"] == "weights":
        s["lse"] = _attend(s)[1]
        s["weights"] = torch.rand(batch, per_seq * page, generator=g, device="cuda")
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _gather(s, pool):
    """The sequences' slots in order, [batch, heads, slots, D], with zeros where there is nothing."""
    case, page = s["case"], s["page"]
    rows = (s["table"].clamp_min(0).long()[:, :, None] * page + torch.arange(page, device="cuda")).reshape(s["batch"], -1)
    x = pool[rows].float()
    x = torch.where(_there(s)[:, :, None], x, 0.0)
    return x.view(s["batch"], -1, case["kv_heads"], D).transpose(1, 2)


def _there(s):
    """Slots that hold a token, [batch, slots]."""
    held = ((s["table"] >= 0) & (s["table"] < s["num_pages"])).repeat_interleave(s["page"], dim=1)
    return held & (torch.arange(held.shape[1], device="cuda")[None, :] < s["lens"][:, None])


def _scores(s):
    """Scaled scores with -inf where a row does not see a slot, [batch, kv_heads, group, t, slots]."""
    case, t = s["case"], s["t"]
    group = case["heads"] // case["kv_heads"]
    q = s["q"].float().view(s["batch"], t, case["kv_heads"], group, D).permute(0, 2, 3, 1, 4)
    k = _gather(s, s["k"])
    x = torch.matmul(q.reshape(s["batch"], case["kv_heads"], group * t, D), k.transpose(2, 3)) * s["scale"]
    x = x.view(s["batch"], case["kv_heads"], group, t, -1)
    i = torch.arange(t, device="cuda")
    j = torch.arange(x.shape[-1], device="cuda")
    p = (i[None, :] + (s["lens"] - s["q_lens"])[:, None])[:, :, None]
    see = _there(s)[:, None, :] & (i[None, :] < s["q_lens"][:, None])[:, :, None]
    if case["causal"]:
        see = see & (j <= p)
    if case["window"]:
        see = see & (((p - j).abs() < case["window"]) | (j < case["first"]))
    return x.masked_fill(~see[:, None, None], float("-inf"))


def _attend(s):
    case, t = s["case"], s["t"]
    x = _scores(s)
    m = x.amax(-1, keepdim=True).clamp_min(-1e30)
    e = (x - m).exp()
    total = e.sum(-1, keepdim=True)
    lse = m + total.log()
    shape = e.shape
    o = torch.matmul(e.view(shape[0], shape[1], -1, shape[-1]), _gather(s, s["v"])).view(*shape[:-1], D)
    o = torch.where(total > 0, o / total, 0.0)
    out = o.permute(0, 3, 1, 2, 4).reshape(s["batch"] * t, case["heads"] * D).half()
    return out, lse[..., 0].permute(0, 3, 1, 2).reshape(s["batch"] * t, case["heads"]).contiguous()


def _append(s):
    t, page = s["t"], s["page"]
    i = torch.arange(t, device="cuda")
    p = i[None, :] + (s["lens"] - s["q_lens"])[:, None]
    new = i[None, :] < s["q_lens"][:, None]
    pages = torch.gather(s["table"], 1, (p.clamp(0, s["table"].shape[1] * page - 1) // page).long())
    ok = (new & (pages >= 0)).reshape(-1)
    rows = (pages.long() * page + p % page).reshape(-1)[ok]
    s["k"][rows] = s["k_new"][ok]
    s["v"][rows] = s["v_new"][ok]
    return s["k"], s["v"]


def _weights(s):
    case, t = s["case"], s["t"]
    group = case["heads"] // case["kv_heads"]
    lse = s["lse"].view(s["batch"], t, case["kv_heads"], group).permute(0, 2, 3, 1)[..., None]
    p = (_scores(s) - torch.where(torch.isfinite(lse), lse, 0.0)).exp()
    return s["weights"] + p.sum((1, 2, 3))


def _evict(s):
    case, page, batch = s["case"], s["page"], s["batch"]
    there = _there(s)
    slots = there.shape[1]
    j = torch.arange(slots, device="cuda")
    always = (j[None, :] < case["first"]) | (j[None, :] >= s["lens"][:, None] - case["recent"])
    key = torch.where(always, float("inf"), s["weights"])
    key = torch.where(there, key, float("-inf"))
    order = torch.sort(key, dim=1, descending=True, stable=True)[1]
    rank = torch.empty_like(order).scatter_(1, order, j.expand(batch, slots).contiguous())
    keep = there & (rank < case["budget"])
    count = keep.sum(1).to(torch.int32)
    kept = torch.sort(torch.where(keep, j, slots), dim=1)[0][:, : case["budget"]]
    kept = torch.nn.functional.pad(kept, (0, case["budget"] - kept.shape[1]), value=slots)
    held = kept < slots
    kept = torch.where(held, kept, -1).to(torch.int32)
    old = kept.clamp_min(0).long()
    src = torch.gather(s["table"], 1, old // page).long() * page + old % page
    n = torch.arange(case["budget"], device="cuda")
    dst = s["out_table"][:, n // page].long() * page + n % page
    s["k_out"][dst[held]] = s["k"][src[held]]
    s["v_out"][dst[held]] = s["v"][src[held]]
    out_slots = s["out_table"].shape[1] * page
    weights = torch.zeros(batch, out_slots, device="cuda")
    weights[:, : case["budget"]] = torch.where(held, torch.gather(s["weights"], 1, old), 0.0)
    return s["k_out"], s["v_out"], kept, count, weights


def run(s):
    case = s["case"]
    if own:
        from speech_encoder_attention_b200 import attn
        cache = attn.PagedKV(s["k"], s["v"], s["table"], s["lens"], s["page"], case["kv_heads"])
        if case["op"] == "append":
            attn.attn_paged_append(s["k_new"], s["v_new"], cache, s["batch"], s["t"], q_lens=s["q_lens"])
            return s["k"], s["v"]
        if case["op"] == "attend":
            return attn.attn_paged(s["q"], cache, s["batch"], s["t"], case["heads"], window=case["window"],
                                   first=case["first"], causal=case["causal"], q_lens=s["q_lens"], scale=s["scale"],
                                   return_lse=True)
        if case["op"] == "weights":
            return attn.attn_paged_weights(s["q"], cache, s["lse"], s["batch"], s["t"], case["heads"],
                                           window=case["window"], first=case["first"], causal=case["causal"],
                                           q_lens=s["q_lens"], scale=s["scale"], weights=s["weights"])
        count = torch.empty_like(s["lens"])
        out = attn.PagedKV(s["k_out"], s["v_out"], s["out_table"], count, s["page"], case["kv_heads"])
        kept, weights = attn.attn_paged_evict(cache, s["weights"], case["budget"], first=case["first"],
                                              recent=case["recent"], dst=out)
        return s["k_out"], s["v_out"], kept, count, weights
    if case["op"] == "append":
        return _append(s)
    if case["op"] == "attend":
        return _attend(s)
    if case["op"] == "weights":
        return _weights(s)
    return _evict(s)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one sequence at a time
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    lens, page = _lens(case), case["page"]
    table = s["table"].cpu().numpy()
    if case["op"] == "append":
        k, v = s["k"].double(), s["v"].double()
        for b, (kv, q) in enumerate(zip(lens, _new(case))):
            rows = torch.tensor([int(table[b, p // page]) * page + p % page for p in range(kv - q, kv)], device="cuda")
            k[rows] = s["k_new"][b * case["t"]: b * case["t"] + q].double()
            v[rows] = s["v_new"][b * case["t"]: b * case["t"] + q].double()
        return k, v
    if case["op"] == "evict":
        k, v = s["k_out"].double(), s["v_out"].double()
        out_table = s["out_table"].cpu().numpy()
        all_w = s["weights"].double().cpu().numpy()
        weights = np.zeros((case["batch"], out_table.shape[1] * page))
        for b, kv in enumerate(lens):
            must = set(range(min(case["first"], kv))) | set(range(max(0, kv - case["recent"]), kv))
            rest = sorted((j for j in range(kv) if j not in must), key=lambda j: (-all_w[b, j], j))
            old = sorted(must | set(rest[: max(0, case["budget"] - len(must))]))
            src = torch.tensor([int(table[b, j // page]) * page + j % page for j in old], device="cuda")
            dst = torch.tensor([int(out_table[b, n // page]) * page + n % page for n in range(len(old))], device="cuda")
            k[dst], v[dst] = s["k"][src].double(), s["v"][src].double()
            weights[b, : len(old)] = all_w[b, old]
        return k, v, None, None, torch.from_numpy(weights)
    group, t = case["heads"] // case["kv_heads"], case["t"]
    out = torch.zeros(case["batch"] * t, case["heads"], D, dtype=torch.float64, device="cuda")
    lse = torch.full((case["batch"] * t, case["heads"]), float("-inf"), dtype=torch.float64, device="cuda")
    weights = s["weights"].double() if case["op"] == "weights" else None
    for b, (kv, q) in enumerate(zip(lens, _new(case))):
        held = np.arange(kv)[table[b, np.arange(kv) // page] >= 0]
        at = torch.from_numpy(table[b, held // page].astype(np.int64) * page + held % page).cuda()
        j = torch.from_numpy(held).cuda()
        p = torch.arange(kv - q, kv, device="cuda")[:, None]
        hidden = (j > p) if case["causal"] else torch.zeros(q, len(held), dtype=torch.bool, device="cuda")
        if case["window"]:
            hidden = hidden | (((j - p).abs() >= case["window"]) & (j >= case["first"]))
        rows = slice(b * t, b * t + q)
        for h in range(case["heads"]):
            c = h // group * D
            x = s["q"][rows, h * D: (h + 1) * D].double() @ s["k"][at, c: c + D].double().T * s["scale"]
            x[hidden] = float("-inf")
            if weights is not None:
                weights[b, j] += torch.exp(x - s["lse"][rows, h: h + 1].double()).sum(0)
                continue
            lse[rows, h] = torch.logsumexp(x, 1)
            out[rows, h] = torch.softmax(x, 1) @ s["v"][at, c: c + D].double()
    return weights if weights is not None else (out.view(case["batch"] * t, -1), lse)
