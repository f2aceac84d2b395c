"""Cases of the paged key/value cache operators: appending new tokens' keys and values
(with the position rotation) and the attention of one new token per sequence over the
cache, in full or with a sliding window and always-visible first tokens.

``run`` computes them in plain torch operations, or, where ``own`` is true, with the
framework's kernels. Sizes are per case; see the comments in ``listed``.
"""
import math

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _append(name, rows, pad, seqs, ctx, heads, kv_heads, hd, rot, style, page, dtype, layout):
    return {"name": name, "op": "append", "rows": rows, "pad": pad, "seqs": seqs, "ctx": ctx, "heads": heads,
            "kv_heads": kv_heads, "hd": hd, "rot": rot, "style": style, "page": page, "dtype": dtype,
            "layout": layout}


def _attend(name, seqs, empty, lo, hi, heads, kv_heads, hd, page, window, sinks, dtype, layout):
    return {"name": name, "op": "attend", "seqs": seqs, "empty": empty, "lo": lo, "hi": hi, "heads": heads,
            "kv_heads": kv_heads, "hd": hd, "page": page, "window": window, "sinks": sinks, "dtype": dtype,
            "layout": layout}


def listed():
    return [
        # one generation step of a single request, 12 heads, learned positions (no rotation)
        _append("append_one", 1, 0, 1, 256, 12, 12, 64, 0, "halves", 16, "bf16", "heads"),
        # one step of a batch padded to 64 rows, 53 requests live, grouped heads, full rotation
        _append("append_step_53_of_64", 64, 11, 53, 256, 32, 8, 128, 128, "halves", 16, "bf16", "heads"),
        # a few short prompts in 32 bits, partial rotation of neighbouring pairs, small pages of whole tokens
        _append("append_prompts_f32", 777, 3, 6, 160, 6, 3, 96, 32, "pairs", 8, "f32", "tokens"),
        # a prompt pass over 16 full blocks of 1024 tokens
        _append("append_prompts_16384", 16384, 0, 16, 1024, 12, 12, 64, 64, "halves", 16, "bf16", "heads"),
        # one short request: launch latency
        _attend("attend_one_short", 1, 0, 100, 100, 12, 12, 64, 16, 0, 0, "bf16", "heads"),
        # 16 requests at the full block of 1024 tokens, 12 heads
        _attend("attend_16x1024", 16, 0, 1024, 1024, 12, 12, 64, 16, 0, 0, "bf16", "heads"),
        # 32-bit cache, ragged, three empty slots in the batch
        _attend("attend_ragged_f32", 12, 3, 1, 2000, 8, 4, 32, 32, 0, 0, "f32", "heads"),
        # one request with a very long context, grouped heads
        _attend("attend_long_one", 1, 0, 131071, 131071, 32, 8, 128, 64, 0, 0, "bf16", "heads"),
        # many requests of very different lengths, 25 heads, whole tokens per page row
        _attend("attend_ragged_25_heads", 64, 0, 17, 8191, 25, 25, 64, 16, 0, 0, "bf16", "tokens"),
        # long requests through a window of 1000 tokens with 4 first tokens kept
        _attend("attend_window_sinks", 40, 2, 5, 30000, 16, 2, 128, 32, 1000, 4, "bf16", "heads"),
        # all query heads on one key head
        _attend("attend_one_kv_head", 33, 0, 300, 5000, 16, 1, 64, 128, 0, 0, "bf16", "heads"),
        # a full serving batch
        _attend("attend_128_requests", 128, 0, 512, 8192, 32, 8, 128, 64, 0, 0, "bf16", "heads"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    hd = rng.choice((32, 64, 64, 96, 128, 128))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    layout = rng.choice(("heads", "heads", "tokens"))
    if rng.random() < 0.4:
        seqs = _log_int(rng, 1, 64)
        group = rng.choice((1, 1, 2, 4, 8))
        kv_heads = rng.randint(1, 12)
        per_row = (group + 2) * kv_heads * hd * (2 if dtype == "bf16" else 4)
        rows = seqs if rng.random() < 0.4 else max(seqs, _log_int(rng, 1, max(1, min(16384, 75_000_000 // per_row))))
        ctx = max(16, -(-rows // seqs)) + rng.randint(0, 100)
        pad = rng.choice((0, 0, rng.randint(1, 9)))
        return {"op": "append", "rows": rows + pad, "pad": pad, "seqs": seqs, "ctx": ctx, "heads": group * kv_heads,
                "kv_heads": kv_heads, "hd": hd, "rot": 16 * rng.randint(0, hd // 16),
                "style": rng.choice(("halves", "pairs")), "page": rng.choice((8, 16, 32, 64, 128)), "dtype": dtype,
                "layout": layout}
    seqs = _log_int(rng, 1, 128)
    group = rng.choice((1, 1, 2, 3, 4, 5, 7, 8, 12, 16))
    kv_heads = rng.randint(1, 12)
    most = 128 * 8192 * 8 * 128 // 2 // (seqs * kv_heads * hd)  # half the largest listed batch, padded to the longest
    hi = _log_int(rng, 1, max(1, min(131071, most)))
    lo = _log_int(rng, 1, hi)
    window = rng.choice((0, 0, _log_int(rng, 1, hi + 10)))
    return {"op": "attend", "seqs": seqs, "empty": rng.choice((0, 0, rng.randint(0, seqs - 1))), "lo": lo, "hi": hi,
            "heads": group * kv_heads, "kv_heads": kv_heads, "hd": hd, "page": rng.choice((8, 16, 32, 64, 128)),
            "window": window, "sinks": rng.choice((0, 1, 4, 17)) if window else 0, "dtype": dtype, "layout": layout}


def _lengths(case):
    """Cached tokens of each request: spread evenly in their logarithm, then the empty slots."""
    live = case["seqs"] - case["empty"]
    lo, hi = case["lo"], case["hi"]
    out = [int(round(lo * (hi / lo) ** (i / max(1, live - 1)))) for i in range(live)]
    return out + [0] * case["empty"]


def _visible(case, n):
    lo = max(n - case["window"], 0) if case["window"] else 0
    return min(case["sinks"], lo) + n - lo


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    hd, nh, nkv = case["hd"], case["heads"], case["kv_heads"]
    if case["op"] == "append":
        rows = case["rows"] - case["pad"]
        moved = rows * (nh + 2 * nkv) * hd * es * 2
        positions = min(rows, case["ctx"])  # each row of the rotation table once
        return {"bytes": moved + positions * case["rot"] * 4 + rows * 12, "flops": 3 * rows * (nh + nkv) * case["rot"]}
    vis = [_visible(case, n) for n in _lengths(case)]
    live = len(vis)
    table = sum(-(-v // case["page"]) for v in vis) * 4
    return {"bytes": sum(vis) * nkv * hd * es * 2 + live * nh * (2 * hd * es + 4) + table + 4 * live,
            "flops": 4 * sum(vis) * nh * hd}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _cache(case, pages, g, dtype):
    """A pool of pages with old values in it: logical [page, token, head, element]."""
    p, nkv, hd = case["page"], case["kv_heads"], case["hd"]
    if case["layout"] == "heads":
        return torch.randn(pages, nkv, p, hd, device="cuda", dtype=dtype, generator=g).transpose(1, 2)
    return torch.randn(pages, p, nkv, hd, device="cuda", dtype=dtype, generator=g)


def _tables(per_seq, spare, rs):
    """Pages of each request in the pool's (random) order; unused entries are 0."""
    total = sum(per_seq) + spare
    ids = rs.permutation(total)[: sum(per_seq)].astype(np.int32)
    table = np.zeros((len(per_seq), max(1, max(per_seq))), np.int32)
    at = 0
    for b, n in enumerate(per_seq):
        table[b, :n] = ids[at:at + n]
        at += n
    return torch.from_numpy(table).cuda(), total


def prepare(case, seed):
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(int(seed) + 1)
    rs = np.random.RandomState(int(seed) % (2 ** 31))
    hd, nh, nkv, p = case["hd"], case["heads"], case["kv_heads"], case["page"]
    s = {"case": case}
    if case["op"] == "append":
        rows, valid, seqs, ctx = case["rows"], case["rows"] - case["pad"], case["seqs"], case["ctx"]
        table, pages = _tables([-(-ctx // p)] * seqs, 2, rs)
        # request b gets an equal share of the rows, at consecutive positions after what it holds
        counts = [valid // seqs + (b < valid % seqs) for b in range(seqs)]
        seq = np.concatenate([np.full(n, b) for b, n in enumerate(counts)] + [np.zeros(case["pad"])])
        start = [rs.randint(0, ctx - n + 1) for n in counts]
        pos = np.concatenate([a + np.arange(n) for a, n in zip(start, counts)] + [np.full(case["pad"], -1)])
        # the projections' rows as one tensor: queries, keys, values
        qkv = torch.randn(rows, (nh + 2 * nkv) * hd, device="cuda", dtype=dtype, generator=g)
        s["q"] = qkv[:, : nh * hd].unflatten(1, (nh, hd))
        s["k"] = qkv[:, nh * hd: (nh + nkv) * hd].unflatten(1, (nkv, hd))
        s["v"] = qkv[:, (nh + nkv) * hd:].unflatten(1, (nkv, hd))
        s["q_out"] = torch.randn(rows, nh, hd, device="cuda", dtype=dtype, generator=g)
        s["valid"] = valid
        s["pos"] = torch.from_numpy(pos.astype(np.int32)).cuda()
        s["seq"] = torch.from_numpy(seq.astype(np.int32)).cuda()
        if case["rot"]:
            half = case["rot"] // 2
            angle = np.arange(ctx)[:, None] * 10000.0 ** (-np.arange(half) / half)[None, :]
            s["cos_sin"] = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).cuda()
        else:
            s["cos_sin"] = None
    else:
        lens = np.array(_lengths(case))[rs.permutation(case["seqs"])]
        table, pages = _tables([-(-int(n) // p) for n in lens], 3, rs)
        s["lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
        s["q"] = 1.5 * torch.randn(case["seqs"], nh, hd, device="cuda", dtype=dtype, generator=g)
        s["scale"] = 1.0 / math.sqrt(hd)
    s["k_cache"] = _cache(case, pages, g, dtype)
    s["v_cache"] = _cache(case, pages, g, dtype)
    s["table"] = table
    if own:
        import train_step_b200 as tsb
        s["kv"] = tsb.PagedKV(s["k_cache"], s["v_cache"], table)
        if case["op"] == "attend":
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(case["seqs"], nh, device="cuda")
            s["ws"] = s["kv"].attention_workspace(nh)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _rotate(x, cos, sin, rot, style):
    x = x.float()
    if not rot:
        return x
    if style == "halves":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_append(s):
    case, n = s["case"], s["valid"]
    rot, p = case["rot"], case["page"]
    pos, seq = s["pos"][:n].long(), s["seq"][:n].long()
    cos = sin = None
    if rot:
        cos_sin = s["cos_sin"][pos][:, None, :]
        cos, sin = cos_sin[..., : rot // 2], cos_sin[..., rot // 2:]
    page, slot = s["table"][seq, pos // p].long(), pos % p
    s["k_cache"][page, slot] = _rotate(s["k"][:n], cos, sin, rot, case["style"]).to(s["k"].dtype)
    s["v_cache"][page, slot] = s["v"][:n]
    s["q_out"][:n] = _rotate(s["q"][:n], cos, sin, rot, case["style"]).to(s["q"].dtype)
    return s["k_cache"], s["v_cache"], s["q_out"]


def _plain_attend(s):
    case = s["case"]
    q, table, lens = s["q"], s["table"].long(), s["lens"].long()
    b, nh, hd = q.shape
    nkv, p = case["kv_heads"], case["page"]
    j = torch.arange(table.shape[1] * p, device=q.device)[None, :]
    seen = j < lens[:, None]
    if case["window"]:
        seen = seen & ((j >= lens[:, None] - case["window"]) | (j < case["sinks"]))
    seen = seen[:, None, None, :]
    # each request's pages side by side: [request, head, token, element]
    k = s["k_cache"][table].permute(0, 3, 1, 2, 4).flatten(2, 3).float()
    z = torch.matmul(q.float().view(b, nkv, nh // nkv, hd), k.transpose(-1, -2)) * s["scale"]
    del k
    z = torch.where(seen, z, -torch.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -torch.inf, 0.0, top)  # a request without tokens
    w = torch.exp(z - top)
    total = w.sum(-1, keepdim=True)
    lse = (torch.log(total) + top).view(b, nh)
    w = w / torch.where(total == 0, 1.0, total)
    v = s["v_cache"][table].permute(0, 3, 1, 2, 4).flatten(2, 3).float()
    return torch.matmul(w, v).view(b, nh, hd).to(q.dtype), lse


def run(state):
    if own:
        import train_step_b200 as tsb
        s, case = state, state["case"]
        if case["op"] == "append":
            tsb.paged_kv_append(s["kv"], s["k"], s["v"], s["pos"], s["seq"], q=s["q"], q_out=s["q_out"],
                                cos_sin=s["cos_sin"], interleaved=case["style"] == "pairs")
            return s["k_cache"], s["v_cache"], s["q_out"]
        tsb.paged_attention(s["kv"], s["q"], s["lens"], s["out"], scale=s["scale"], window=case["window"],
                            sinks=case["sinks"], lse=s["lse"], ws=s["ws"])
        return s["out"], s["lse"]
    return _plain_append(state) if state["case"]["op"] == "append" else _plain_attend(state)


# ---------------------------------------------------------------------------
# the definition in 64 bits, row by row
# ---------------------------------------------------------------------------
def _exact_append(s):
    case = s["case"]
    p, rot = case["page"], case["rot"]
    k_cache, v_cache, q_out = s["k_cache"].double(), s["v_cache"].double(), s["q_out"].double()
    if rot:
        index = torch.arange(rot // 2, device="cuda")
        first, second = (index, index + rot // 2) if case["style"] == "halves" else (2 * index, 2 * index + 1)
    where, rows, seqs = s["pos"].tolist(), s["pos"].shape[0], s["seq"].tolist()
    table = s["table"].tolist()
    live = [n for n in range(rows) if where[n] >= 0]
    q, k = s["q"][live].double(), s["k"][live].double()
    if rot:
        at = s["cos_sin"].double()[[where[n] for n in live]]
        for x in (q, k):
            c, sn = at[:, None, : rot // 2], at[:, None, rot // 2:]
            a, b = x[:, :, first].clone(), x[:, :, second].clone()
            x[:, :, first] = a * c - b * sn
            x[:, :, second] = b * c + a * sn
    pages = [table[seqs[n]][where[n] // p] for n in live]
    slots = [where[n] % p for n in live]
    k_cache[pages, slots] = k
    v_cache[pages, slots] = s["v"][live].double()
    q_out[live] = q
    return k_cache, v_cache, q_out


def _exact_attend(s):
    case = s["case"]
    p, nkv = case["page"], case["kv_heads"]
    b, nh, hd = s["q"].shape
    out = torch.zeros(b, nh, hd, device="cuda", dtype=torch.float64)
    lse = torch.full((b, nh), -math.inf, device="cuda", dtype=torch.float64)
    for i, n in enumerate(s["lens"].tolist()):
        if not n:
            continue
        begin = max(0, n - case["window"]) if case["window"] else 0
        keys = torch.cat([torch.arange(min(case["sinks"], begin)), torch.arange(begin, n)]).cuda()
        page, slot = s["table"][i][keys // p].long(), keys % p
        k, v = s["k_cache"][page, slot].double(), s["v_cache"][page, slot].double()
        q = s["q"][i].double().reshape(nkv, nh // nkv, hd)
        z = torch.einsum("hgd,jhd->hgj", q, k) * s["scale"]
        lse[i] = torch.logsumexp(z, -1).reshape(nh)
        out[i] = torch.einsum("hgj,jhd->hgd", torch.softmax(z, -1), v).reshape(nh, hd)
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)
