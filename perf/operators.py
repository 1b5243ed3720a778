"""Cases of the paged-cache operators: a decoding step over a cache of pages, the
same step for a batch whose sequences share a long prefix, and the page
management around them (appending rows, forking sequences, compacting pages).

``run`` computes each operator in its plain form (elementary torch operations,
float32 arithmetic), or, where ``own`` is true, makes the calls a user makes of
the library.  Sizes follow the library's own workloads: 32 query heads over 8
K/V heads of d = 128 against 8192 positions, 8 heads of d = 64 in fp16, and 32
query heads over one K/V head under a window of 1024 plus 64 sinks.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one user's chat answered token by token: latency is all that counts
        {"name": "decode one sequence", "op": "decode", "B": 1, "H": 32, "H_kv": 8, "N_q": 1,
         "d": 128, "page": 16, "len": 517, "window": 0, "n_sink": 0, "causal": True, "dtype": "bf16"},
        # a served batch of ragged lengths, one of its slots empty
        {"name": "decode batch", "op": "decode", "B": 8, "H": 32, "H_kv": 8, "N_q": 1, "d": 128,
         "page": 16, "len": 8192, "window": 0, "n_sink": 0, "causal": True, "dtype": "bf16"},
        # four drafted tokens verified at once, one K/V head, sliding window and sinks
        {"name": "decode drafted window", "op": "decode", "B": 8, "H": 32, "H_kv": 1, "N_q": 4,
         "d": 128, "page": 32, "len": 8192, "window": 1024, "n_sink": 64, "causal": True,
         "dtype": "bf16"},
        # a full batch of long contexts
        {"name": "decode long batch", "op": "decode", "B": 32, "H": 32, "H_kv": 8, "N_q": 1, "d": 128,
         "page": 64, "len": 16384, "window": 0, "n_sink": 0, "causal": True, "dtype": "bf16"},
        # a served batch behind one system prompt, two rows a sequence
        {"name": "shared system prompt", "op": "shared", "B": 32, "H": 8, "H_kv": 8, "N_q": 2,
         "d": 64, "page": 16, "shared": 1024, "len": 513, "causal": True, "dtype": "fp16"},
        # many samples of one long document
        {"name": "shared document", "op": "shared", "B": 128, "H": 32, "H_kv": 8, "N_q": 1, "d": 128,
         "page": 64, "shared": 16384, "len": 1000, "causal": True, "dtype": "bf16"},
        # a decoding step's new rows (three drafted tokens), taken back again
        {"name": "append step", "op": "append", "B": 64, "H_kv": 8, "d": 128, "page": 16,
         "len": 2000, "new": 3, "dtype": "bf16"},
        # ragged prompts written to the cache, and released
        {"name": "append prompts", "op": "append", "B": 16, "H_kv": 8, "d": 128, "page": 64,
         "len": 0, "new": 8192, "dtype": "bf16"},
        # a beam step: losing beams dropped, winners forked, one token for each fork
        {"name": "fork beams", "op": "fork", "B": 16, "H_kv": 8, "d": 64, "page": 16, "len": 777,
         "dtype": "fp16"},
        # sampling many continuations of long sequences
        {"name": "fork samples", "op": "fork", "B": 512, "H_kv": 8, "d": 128, "page": 128,
         "len": 8192, "dtype": "bf16"},
        # a cache that has become sparse, its live pages moved to the front
        {"name": "compact pages", "op": "compact", "B": 64, "H_kv": 8, "d": 128, "page": 64,
         "len": 8192, "live": 0.5, "dtype": "bf16"},
        {"name": "compact small cache", "op": "compact", "B": 8, "H_kv": 8, "d": 64, "page": 16,
         "len": 1000, "live": 0.7, "dtype": "fp16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "shared", "shared", "append", "fork", "compact"])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    page = rng.choice([16, 32, 64, 128, 256])
    H_kv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8, 16, 32])
    # at most 1/2 of the largest listed decoding step's elements
    room = 32 * 16384 * 8 * 128 // 2 // (H_kv * d)
    if op == "decode":
        length = _log_int(rng, 1, 16384)
        B = _log_int(rng, 1, max(1, min(300, room // length)))
        N_q = rng.choice([1, 1, 1, 2, 3, 4])
        window = _log_int(rng, 1, 2 * length) if rng.random() < 0.3 else 0
        n_sink = rng.choice([0, 4, 64, 200]) if window else 0
        return {"op": op, "B": B, "H": G * H_kv, "H_kv": H_kv, "N_q": N_q, "d": d, "page": page,
                "len": length, "window": window, "n_sink": n_sink,
                "causal": True if window else rng.random() < 0.8, "dtype": dtype}
    if op == "shared":
        G = min(G, 8)
        shared = page * max(1, _log_int(rng, 100, 16384) // page)
        length = _log_int(rng, 1, 2000)
        B = _log_int(rng, 2, max(2, min(160, room // length, 100 * 16384 * 32 // (2 * shared * G * H_kv))))
        return {"op": op, "B": B, "H": G * H_kv, "H_kv": H_kv, "N_q": rng.choice([1, 1, 2]), "d": d,
                "page": page, "shared": shared, "len": length, "causal": rng.random() < 0.8,
                "dtype": dtype}
    if op == "append":
        new = _log_int(rng, 1, 4096)
        B = _log_int(rng, 1, max(1, min(300, 16 * 8192 // new)))
        return {"op": op, "B": B, "H_kv": H_kv, "d": d, "page": page,
                "len": _log_int(rng, 1, 4096) if rng.random() < 0.8 else 0, "new": new, "dtype": dtype}
    if op == "fork":
        length = _log_int(rng, 1, 16384)
        return {"op": op, "B": _log_int(rng, 2, max(2, min(512, 2 * room // length))), "H_kv": H_kv,
                "d": d, "page": page, "len": length, "dtype": dtype}
    length = _log_int(rng, 1, 8192)
    return {"op": op, "B": _log_int(rng, 1, max(1, min(200, room // length))), "H_kv": H_kv, "d": d,
            "page": page, "len": length, "live": round(rng.uniform(0.2, 0.95), 2), "dtype": dtype}


# ------------------------------------------------------------------ inputs

def _lengths(B, top, empty=True):
    """Ragged lengths 1..top of a batch by the case alone, one of them the longest;
    from 8 sequences on one slot is empty."""
    got = [1 + int((top - 1) * (0.15 + 0.85 * math.modf((b + 1) * 0.6180339887)[0])) if top else 0
           for b in range(B)]
    got[0] = top
    if empty and B >= 8:
        got[B // 2] = 0
    return got


def _pages(n, page):
    return -(-n // page)


def _forks(B):
    """Rows 0..P-1 are parents, the others their children."""
    P = max(1, B // 4)
    return P, [c % P for c in range(P, B)], list(range(P, B))


def _cache(case, g, lens, columns, spare, live=None):
    """Pages with random contents, and a table that gives every sequence random
    pages of its own.  Rows that no sequence has written hold NaN where attention reads
    around them (bytes of earlier use may be anything)."""
    page, H_kv, d = case["page"], case["H_kv"], case["d"]
    dev, dt = g.device, _DT[case["dtype"]]
    B = len(lens)
    used = sum(_pages(n, page) for n in lens)
    n_pages = used + spare if live is None else max(used + 1, int(used / live))
    ids = torch.randperm(n_pages, generator=g, device=dev)
    l = torch.tensor(lens, device=dev)
    l = l[torch.randperm(B, generator=g, device=dev)]
    have = (l + page - 1) // page
    first = torch.cumsum(have, 0) - have
    col = torch.arange(columns, device=dev)
    on = col < have[:, None]
    table = torch.where(on, ids[(first[:, None] + col).clamp(max=n_pages - 1)], -1)
    refs = torch.zeros(n_pages, dtype=torch.int32, device=dev)
    refs[ids[:used]] = 1
    filled = torch.zeros(n_pages, dtype=torch.long, device=dev)
    filled[table[on]] = (l[:, None] - col * page).clamp(max=page)[on]
    hole = (torch.arange(page, device=dev) >= filled[:, None])[:, None, :, None]

    def data():
        x = torch.empty(n_pages, H_kv, page, d, dtype=dt, device=dev)
        x.normal_(generator=g)
        return x.masked_fill_(hole, float("nan")) if case["op"] in ("decode", "shared") else x

    return {"k": data(), "v": data(), "table": table.int().contiguous(), "lens": l.int(), "refs": refs}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(1000003 * seed + 17)
    dt, op, B, page = _DT[case["dtype"]], case["op"], case["B"], case["page"]

    def normal(*shape):
        return torch.empty(shape, dtype=dt, device=dev).normal_(generator=g)

    if op == "decode":
        s = _cache(case, g, _lengths(B, case["len"]), _pages(case["len"], page), 3)
        s["q"] = normal(B, case["H"], case["N_q"], case["d"])
    elif op == "shared":
        # one sequence's first `shared` positions, in every non-empty row's table
        s = _cache(case, g, _lengths(B, case["len"]), _pages(case["len"], page), 3)
        n0, ns = s["k"].shape[0], case["shared"] // page
        s["k"] = torch.cat([s["k"], normal(ns, case["H_kv"], page, case["d"])])
        s["v"] = torch.cat([s["v"], normal(ns, case["H_kv"], page, case["d"])])
        at = n0 + torch.randperm(ns, generator=g, device=dev)
        row = (s["lens"] > 0)[:, None]
        s["table"] = torch.cat([torch.where(row, at, -1).int(), s["table"]], 1).contiguous()
        s["refs"] = torch.cat([s["refs"], row.sum().int().expand(ns)])
        s["lens"] = torch.where(row[:, 0], s["lens"] + case["shared"], 0).int()
        s["shared_table"] = at.int()
        s["q"] = normal(B, case["H"], case["N_q"], case["d"])
    elif op == "append":
        top = case["len"] + case["new"]
        s = _cache(case, g, _lengths(B, case["len"], False), _pages(top, page),
                   B * (_pages(case["new"], page) + 1))
        s["k_new"] = normal(B, case["H_kv"], case["new"], case["d"])
        s["v_new"] = normal(B, case["H_kv"], case["new"], case["d"])
        s["counts"] = torch.tensor(_lengths(B, case["new"]), device=dev).int()
        s["start"] = s["lens"].clone()
    elif op == "fork":
        P, parents, children = _forks(B)
        lens = _lengths(P, case["len"], False)
        s = _cache(case, g, lens, _pages(case["len"] + 1, page), 2 * B)
        s["table"] = torch.cat([s["table"], s["table"].new_full((B - P, s["table"].shape[1]), -1)])
        s["lens"] = torch.cat([s["lens"], s["lens"].new_zeros(B - P)])
        s["parents"] = torch.tensor(parents, device=dev, dtype=torch.int32)
        s["children"] = torch.tensor(children, device=dev, dtype=torch.int32)
        s["zeros"] = torch.zeros(len(children), device=dev, dtype=torch.int32)
        s["counts"] = torch.tensor([0] * P + [1] * (B - P), device=dev, dtype=torch.int32)
        s["k_new"] = normal(B, case["H_kv"], 1, case["d"])
        s["v_new"] = normal(B, case["H_kv"], 1, case["d"])
    else:
        s = _cache(case, g, _lengths(B, case["len"]), _pages(case["len"], page), 0, case["live"])
        s["table_out"] = torch.empty_like(s["table"])
        s["refs_out"] = torch.empty_like(s["refs"])
    s["case"] = case
    return s


# ------------------------------------------------------------------ plain forms

def _rows(pages, table):
    """[B, H_kv, columns * page, d] float32 rows of every sequence."""
    x = pages[table.long().clamp(min=0)].float()
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _kept(lens, case, N):
    """[B, N_q, N]: which of the first N positions each query row keeps."""
    N_q = case["N_q"]
    l = lens.long()[:, None, None]
    i = l - N_q + torch.arange(N_q, device=lens.device)[None, :, None]
    j = torch.arange(N, device=lens.device)
    keep = (j < l).expand(-1, N_q, -1)
    if case["causal"]:
        keep = keep & (j <= i)
    w = case.get("window", 0)
    if w:
        keep = keep & ((i - j < w) | (j < case["n_sink"]))
    return keep


def _attend(parts, scale, out_dtype):
    """softmax over the positions of all parts (scores [B, H_kv, G, N_q, n], values'
    product, kept); rows that keep nothing give zeros and minus infinity."""
    s = [torch.where(keep[:, None, None], x * scale, -math.inf) for x, _, keep in parts]
    m = torch.stack([x.amax(-1) for x in s]).amax(0)
    m0 = torch.where(m == -math.inf, 0.0, m)
    p = [torch.exp(x - m0[..., None]) for x in s]
    l = sum(x.sum(-1) for x in p)
    o = sum(times(x) for x, (_, times, _) in zip(p, parts))
    o = torch.where(l[..., None] > 0, o / l[..., None], 0.0)
    return o.flatten(1, 2).to(out_dtype), (m + torch.log(l)).flatten(1, 2)


def _own_part(s, case, table, first):
    """Scores and value products against the positions from `first` on, which `table` lists."""
    B, H, N_q, d = s["q"].shape
    q = s["q"].float().unflatten(1, (case["H_kv"], -1))
    k, v = _rows(s["k"], table), _rows(s["v"], table)
    keep = _kept(s["lens"], case, first + k.shape[2])[:, :, first:]
    any_row = keep.any(1)[:, None, :, None]
    k, v = k.masked_fill(~any_row, 0.0), v.masked_fill(~any_row, 0.0)
    return (torch.matmul(q.flatten(2, 3), k.transpose(2, 3)).unflatten(2, (-1, N_q)),
            lambda p: torch.matmul(p.flatten(2, 3), v).unflatten(2, (-1, N_q)), keep)


def _plain_decode(s, case):
    return _attend([_own_part(s, case, s["table"], 0)], 1 / math.sqrt(case["d"]), s["q"].dtype)


def _plain_shared(s, case):
    n, page = case["shared"], case["page"]
    q = s["q"].float().unflatten(1, (case["H_kv"], -1))
    k, v = _rows(s["k"], s["shared_table"][None])[0], _rows(s["v"], s["shared_table"][None])[0]
    prefix = (torch.einsum("bgrid,gnd->bgrin", q, k), lambda p: torch.einsum("bgrin,gnd->bgrid", p, v),
              _kept(s["lens"], case, n))
    return _attend([prefix, _own_part(s, case, s["table"][:, n // page:], n)],
                   1 / math.sqrt(case["d"]), s["q"].dtype)


def _plain_trim(s, rows, new):
    page = s["k"].shape[2]
    old = s["lens"][rows].long()
    new = torch.minimum(old, new.long())
    col = torch.arange(s["table"].shape[1], device=old.device)
    gone = (col >= ((new + page - 1) // page)[:, None]) & (col < ((old + page - 1) // page)[:, None])
    t = s["table"][rows]
    s["refs"].index_add_(0, t[gone].long(), torch.full_like(t[gone], -1))
    s["table"][rows] = torch.where(gone, -1, t)
    s["lens"][rows] = new.int()


def _plain_append(s):
    """Pages go in the order of the sequences, the lowest free ones first; a last,
    partly filled page that others hold too is copied first."""
    k, v, table, refs, page = s["k"], s["v"], s["table"], s["refs"], s["k"].shape[2]
    start, count, N = s["lens"].long(), s["counts"].long(), s["k_new"].shape[2]
    end = start + count
    before, after = (start + page - 1) // page, (end + page - 1) // page
    at = (start // page).clamp(max=table.shape[1] - 1)
    last = table.gather(1, at[:, None])[:, 0].long().clamp(min=0)
    copied = (start % page != 0) & (count > 0) & (refs[last] > 1)
    need = after - before + copied
    upto = torch.cumsum(need, 0)
    free = torch.sort((refs != 0).int(), stable=True).indices
    ok = (need == 0) | (upto <= (refs == 0).sum())
    j = torch.arange(N // page + 2, device=start.device)
    got = free[((upto - need)[:, None] + j).clamp(max=len(free) - 1)]
    on = (j < need[:, None]) & ok[:, None]
    column = torch.where(copied, start // page, before)[:, None] + j
    copied = copied & ok
    src, dst, part = last[copied], got[:, 0][copied], (start % page)[copied]
    old_rows = (torch.arange(page, device=start.device) < part[:, None])[:, None, :, None]
    k[dst] = torch.where(old_rows, k[src], k[dst])
    v[dst] = torch.where(old_rows, v[src], v[dst])
    refs.index_add_(0, src, torch.full_like(src, -1, dtype=refs.dtype))
    refs[got[on]] = 1
    row = torch.arange(len(start), device=start.device)[:, None].expand_as(on)
    table[row[on], column[on]] = got[on].int()
    s["lens"].copy_(torch.where(ok, end, start))
    i = torch.arange(N, device=start.device)
    new = (i < count[:, None]) & ok[:, None]
    pos = start[:, None] + i
    to = table.gather(1, (pos // page).clamp(max=table.shape[1] - 1))[new].long()
    k[to, :, (pos % page)[new]] = s["k_new"].transpose(1, 2)[new]
    v[to, :, (pos % page)[new]] = s["v_new"].transpose(1, 2)[new]


def _plain_fork(s):
    page = s["k"].shape[2]
    p, c = s["parents"].long(), s["children"].long()
    t, l = s["table"][p], s["lens"][p]
    on = torch.arange(t.shape[1], device=t.device) < ((l.long() + page - 1) // page)[:, None]
    s["table"][c] = torch.where(on, t, -1)
    s["lens"][c] = l
    s["refs"].index_add_(0, t[on].long(), torch.ones_like(t[on]))


def _plain_compact(s):
    refs = s["refs"]
    page_id = torch.arange(len(refs), device=refs.device)
    live = refs > 0
    n = live.sum()
    src, dst = page_id[live & (page_id >= n)], page_id[~live & (page_id < n)]
    s["k"][dst], s["v"][dst] = s["k"][src], s["v"][src]
    to = page_id.clone()
    to[src] = dst
    s["table_out"].copy_(torch.where(s["table"] >= 0, to[s["table"].long().clamp(min=0)], -1))
    s["refs_out"].copy_(torch.where(page_id < n, refs, 0))
    s["refs_out"][dst] = refs[src]
    return n.int().reshape(1)


# ------------------------------------------------------------------ one pass

def _handle(s):
    """What a serving program keeps between its steps: the cache's handle and its buffers."""
    import exact_tiled_attention_44_b200 as A
    if "cache" not in s:
        s["cache"] = A.PagedCache(s["k"], s["v"], s["table"], s["lens"], s["refs"])
    return A, s["cache"]


def run(s):
    case = s["case"]
    op = case["op"]
    if op in ("decode", "shared"):
        if not own:
            return _plain_decode(s, case) if op == "decode" else _plain_shared(s, case)
        A, cache = _handle(s)
        if op == "decode":
            return A.decode_paged(s["q"], cache, causal=case["causal"], window=case["window"],
                                  n_sink=case["n_sink"])
        return A.decode_paged(s["q"], cache, causal=case["causal"], shared_len=case["shared"],
                              shared_table=s["shared_table"])
    if op == "append":
        if own:
            A, cache = _handle(s)
            A.pages_append(cache, s["k_new"], s["v_new"], s["counts"])
            A.pages_trim(cache, s["start"])
        else:
            _plain_append(s)
            _plain_trim(s, torch.arange(case["B"], device=s["lens"].device), s["start"])
    elif op == "fork":
        if own:
            A, cache = _handle(s)
            A.pages_trim(cache, s["zeros"], s["children"])
            A.pages_fork(cache, s["parents"], s["children"])
            A.pages_append(cache, s["k_new"], s["v_new"], s["counts"])
        else:
            _plain_trim(s, s["children"].long(), s["zeros"])
            _plain_fork(s)
            _plain_append(s)
    else:
        if own:
            A, cache = _handle(s)
            n = A.pages_compact(cache, table_out=s["table_out"], refs_out=s["refs_out"])
        else:
            n = _plain_compact(s)
        return s["k"], s["v"], s["table_out"], s["refs_out"], n
    return s["k"], s["v"], s["table"], s["lens"], s["refs"]


# ------------------------------------------------------------------ work

def work(case):
    """Bytes: every kept K and V row, q, new rows and moved pages read once, every
    output and moved row written once, the page numbers and lengths that say where they
    are.  Flops: two products of every query row with its kept rows."""
    page, d, H_kv, B = case["page"], case["d"], case["H_kv"], case["B"]
    row = 2 * H_kv * d * 2                       # K and V of one position
    if case["op"] in ("decode", "shared"):
        H, N_q = case["H"], case["N_q"]
        shared = case.get("shared", 0)
        w = case.get("window", 0)
        read = pairs = pages = 0
        for n in _lengths(B, case["len"]):
            if not n:
                continue
            total = n + shared
            kept = [_kept_of(total - N_q + i, total, case["causal"], w, case.get("n_sink", 0))
                    for i in range(N_q)]
            union = total if not w else min(total, w + N_q - 1 + min(case["n_sink"], max(0, total - w - N_q + 1)))
            read += min(n, union)
            pages += _pages(min(n, union), page)
            pairs += sum(kept)
        qo = B * H * N_q * (2 * d * 2 + 4)
        return {"bytes": (read + shared) * row + qo + 4 * (pages + shared // page + B),
                "flops": 4 * d * H * pairs}
    if case["op"] == "append":
        n = sum(_lengths(B, case["new"]))
        return {"bytes": 2 * n * row + 4 * (2 * _pages(n, page) + 4 * B), "flops": 0}
    if case["op"] == "fork":
        P, parents, _ = _forks(B)
        lens = _lengths(P, case["len"], False)
        copied = sum(lens[p] % page for p in parents)
        entries = sum(_pages(lens[p], page) for p in parents)
        return {"bytes": 2 * (copied + len(parents)) * row + 4 * 5 * entries, "flops": 0}
    used = sum(_pages(n, page) for n in _lengths(B, case["len"]))
    n_pages = max(used + 1, int(used / case["live"]))
    moved = used * (1 - used / n_pages)
    return {"bytes": 2 * moved * page * row + 8 * B * _pages(case["len"], page) + 8 * n_pages, "flops": 0}


def _kept_of(i, total, causal, window, n_sink):
    """Kept keys of the query row at position i of a sequence of `total`."""
    n = min(total, i + 1) if causal else total
    if window and n > window:
        n = window + min(n_sink, n - window)
    return max(n, 0)


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The definition, sequence by sequence in float64.  The page operators move
    bytes and count; they compute nothing that could be more exact."""
    if case["op"] not in ("decode", "shared"):
        return None
    s = prepare(case, seed)
    B, H, N_q, d = s["q"].shape
    G, page = H // case["H_kv"], case["page"]
    o = torch.zeros(B, H, N_q, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, N_q), -math.inf, dtype=torch.float64, device="cuda")
    w = case.get("window", 0)
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        ids = s["table"][b, :_pages(n, page)].long()
        pos = torch.arange(n, device="cuda")
        for h in range(case["H_kv"]):
            k = s["k"][ids, h].reshape(-1, d)[:n].double()
            v = s["v"][ids, h].reshape(-1, d)[:n].double()
            for i in range(N_q):
                at = n - N_q + i
                keep = torch.ones_like(pos, dtype=torch.bool)
                if case["causal"]:
                    keep = pos <= at
                if w:
                    keep = keep & ((at - pos < w) | (pos < case["n_sink"]))
                if case["causal"] and at < 0:
                    continue
                x = s["q"][b, h * G:(h + 1) * G, i].double() @ k[keep].T / math.sqrt(d)
                z = torch.logsumexp(x, 1)
                lse[b, h * G:(h + 1) * G, i] = z
                o[b, h * G:(h + 1) * G, i] = torch.exp(x - z[:, None]) @ v[keep]
    return o, lse
