"""What is measured of the operators on a paged key/value cache, and their plain forms.

Five operators, each a kind of case:

  paged    attention of the newest T tokens of each sequence over its pages
  latent   the same over pages of one latent vector a token (absorbed form)
  append   new keys and values written to their pages
  fork     sequences forked (full pages shared, the last one copied), given
           room for the next tokens, and freed again
  compact  live pages moved down into the holes, tables renamed

`run` computes them with elementary torch operations, or, where `own` is
true, with the package's entry points.
"""
import math

import torch

own = False


# ----------------------------------------------------------------- the cases

def _paged(B, Hkv, G, T, d, page, longest, shortest, window, layout):
    return {"kind": "paged", "B": B, "Hkv": Hkv, "G": G, "T": T, "d": d, "page": page,
            "longest": longest, "shortest": shortest, "window": window, "layout": layout}


def _latent(B, H, T, rank, page, longest, shortest):
    return {"kind": "latent", "B": B, "H": H, "T": T, "rank": rank, "page": page,
            "longest": longest, "shortest": shortest}


def _append(B, Hkv, T, d, page, latent, ragged):
    return {"kind": "append", "B": B, "Hkv": Hkv, "T": T, "d": d, "page": page, "latent": latent, "ragged": ragged}


def _fork(parents, forks, longest, room, Hkv, d, page, latent):
    return {"kind": "fork", "parents": parents, "forks": forks, "longest": longest, "room": room, "Hkv": Hkv,
            "d": d, "page": page, "latent": latent}


def _compact(pages, live, rows, width, Hkv, d, page, latent):
    return {"kind": "compact", "pages": pages, "live": live, "rows": rows, "width": width, "Hkv": Hkv, "d": d,
            "page": page, "latent": latent}


def listed():
    return [
        # one short conversation at the smallest head size: latency alone
        {"name": "paged-B1-d64-short"} | _paged(1, 2, 4, 1, 64, 16, 77, 77, -1, "hnd"),
        # the framework's decode workload (64 sequences, 32 query heads on 8
        # key/value heads) as a ragged batch in 16-token pages
        {"name": "paged-B64-ragged"} | _paged(64, 8, 4, 1, 128, 16, 8192, 1000, -1, "hnd"),
        # two long documents, four drafted tokens each, token-major pages:
        # few rows, so the length has to be split
        {"name": "paged-B2-T4-131072"} | _paged(2, 2, 4, 4, 128, 128, 131072, 65500, -1, "nhd"),
        # latent caches: one short sequence with few heads; a ragged batch
        # that the cache's bytes bound; all 128 heads, where the products count
        {"name": "latent-B1-H16-short"} | _latent(1, 16, 1, 512, 16, 333, 333),
        {"name": "latent-B48-H16-ragged"} | _latent(48, 16, 1, 512, 64, 16384, 1500),
        {"name": "latent-B32-H128"} | _latent(32, 128, 1, 512, 64, 8192, 2000),
        # one decode step's rows; a prefill batch's, ragged
        {"name": "append-B64-step"} | _append(64, 8, 1, 128, 16, False, False),
        {"name": "append-B8-prefill"} | _append(8, 8, 4096, 128, 16, False, True),
        # beams of one prompt; many prompts with several samples each
        {"name": "fork-1x4"} | _fork(1, 4, 1000, 8, 8, 128, 16, False),
        {"name": "fork-64x8"} | _fork(64, 8, 4000, 64, 8, 128, 64, False),
        # a small pool; a large one of latent pages that is two thirds full
        {"name": "compact-512"} | _compact(512, 0.7, 16, 40, 8, 128, 16, False),
        {"name": "compact-16384-latent"} | _compact(16384, 0.66, 256, 128, 1, 576, 64, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["paged", "paged", "latent", "latent", "append", "fork", "compact"])
    page = rng.choice([8, 16, 32, 64, 128])
    if kind == "paged":
        d = rng.choice([64, 128])
        B, Hkv = _log(rng, 1, 80), rng.choice([1, 2, 3, 4, 8])
        T = rng.choice([1, 1, 1, 2, 3, 4])
        G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16] if T == 1 else [1, 2, 4, 8])
        longest = _log(rng, 1, min(131072, 270000000 // (B * Hkv * d)))
        return _paged(B, Hkv, G, T, d, page, longest, rng.randint(0, longest),
                      rng.choice([-1, -1, rng.randint(0, longest)]), rng.choice(["hnd", "nhd"]))
    if kind == "latent":
        H, B = rng.choice([8, 16, 20, 32, 64, 128]), _log(rng, 1, 64)
        T = rng.choice([1, 1, 2])
        longest = _log(rng, 1, min(65536, 19000000 // (B * T * max(H, 16))))
        return _latent(B, H, T, rng.choice([256, 512]), page, longest, rng.randint(0, longest))
    latent = rng.random() < 0.3
    Hkv, d = (1, 576) if latent else (rng.choice([1, 2, 4, 8]), rng.choice([64, 128]))
    if kind == "append":
        B = _log(rng, 1, 128)
        return _append(B, Hkv, rng.choice([1, _log(rng, 2, 32000 // B)]), d, page, latent, rng.random() < 0.5)
    if kind == "fork":
        return _fork(_log(rng, 1, 48), rng.randint(1, 8), _log(rng, 1, 4000), rng.randint(1, 64), Hkv, d, page, latent)
    return _compact(_log(rng, 16, min(16384, 300000000 // (page * Hkv * d))), rng.uniform(0.3, 0.95),
                    _log(rng, 1, 200), _log(rng, 1, 100), Hkv, d, page, latent)


# ---------------------------------------------------------------- the inputs

def _lengths(case, n):
    """n lengths from the shortest to the longest, evenly spread."""
    lo, hi = case["shortest"], case["longest"]
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _tables(g, lens, page, width, device):
    """Page tables [n, width] of sequences of these lengths in a pool of
    shuffled pages with an eighth of them unused, and the pool's size."""
    counts = [-(-x // page) for x in lens]
    total = sum(counts)
    pool = total + total // 8 + 1
    ids = torch.randperm(pool, generator=g, device=device)[:total].int()
    held = torch.arange(width, device=device)[None, :] < torch.tensor(counts, device=device)[:, None]
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=device)
    table[held] = ids
    return table, pool


def _pool(g, pages, Hkv, page, d, layout, device):
    if layout == "nhd":
        return torch.randn((pages, page, Hkv, d), generator=g, device=device, dtype=torch.bfloat16).transpose(1, 2)
    return torch.randn((pages, Hkv, page, d), generator=g, device=device, dtype=torch.bfloat16)


def _cache(g, case, pages, device):
    """k_pages and v_pages, or latent pages and None."""
    if case["latent"]:
        return _pool(g, pages, 1, case["page"], case["d"], "hnd", device), None
    k, v = (_pool(g, pages, case["Hkv"], case["page"], case["d"], "hnd", device) for _ in range(2))
    return k, v


def prepare(case, seed):
    device = torch.device("cuda")
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    s = {"kind": case["kind"], "case": dict(case)}
    page = case["page"]
    if case["kind"] in ("paged", "latent"):
        order = torch.randperm(case["B"], generator=g, device=device).tolist()
        spread = _lengths(case, case["B"])
        lens = [spread[i] for i in order]
        s["table"], pool = _tables(g, lens, page, -(-case["longest"] // page) + 1, device)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=device)
        if case["kind"] == "paged":
            H, d = case["Hkv"] * case["G"], case["d"]
            s["q"] = torch.randn((case["B"], H, case["T"], d), generator=g, device=device).mul_(1.5).bfloat16()
            s["k"], s["v"] = (_pool(g, pool, case["Hkv"], page, d, case["layout"], device) for _ in range(2))
            s["scale"] = 1.0 / math.sqrt(d)
        else:
            D = case["rank"] + 64
            s["q"] = torch.randn((case["B"], case["H"], case["T"], D), generator=g, device=device).bfloat16()
            s["c"] = torch.randn((pool, page, D), generator=g, device=device, dtype=torch.bfloat16)
            s["scale"] = 1.5 / math.sqrt(D)
        if own:
            import exact_softmax_attention_04_b200 as attn
            B, T, width = case["B"], case["T"], s["table"].shape[1]
            if case["kind"] == "paged":
                need = attn.decode_paged_workspace_bytes(B, H, case["Hkv"], T, width, page, d)
            else:
                need = attn.decode_latent_workspace_bytes(B, case["H"], T, width, page, case["rank"])
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device=device)
    elif case["kind"] == "append":
        B, T = case["B"], case["T"]
        # the caches hold 0 to 2000 tokens so far
        start = [2000 * (i + 1) // (B + 1) for i in torch.randperm(B, generator=g, device=device).tolist()]
        lens = [x + T for x in start]
        s["table"], pool = _tables(g, lens, page, -(-max(lens) // page), device)
        s["pos"] = torch.tensor(start, dtype=torch.int32, device=device)
        counts = [T - (T // 2) * i // max(1, B - 1) for i in range(B)] if case["ragged"] else [T] * B
        s["count"] = torch.tensor(counts, dtype=torch.int32, device=device)
        s["k"], s["v"] = _cache(g, case, pool, device)
        # as a projection leaves them: token-major
        new = [torch.randn((B, T, s["k"].shape[1], case["d"]), generator=g, device=device,
                           dtype=torch.bfloat16).transpose(1, 2) for _ in range(2)]
        s["new_k"], s["new_v"] = new[0], None if case["latent"] else new[1]
    elif case["kind"] == "fork":
        n, m = case["parents"], case["parents"] * case["forks"]
        lens = [case["longest"] - (case["longest"] // 2) * i // max(1, n - 1) for i in range(n)]
        width = -(-(case["longest"] + case["room"]) // page) + 1
        table, pool = _tables(g, lens, page, width, device)
        pool += m * (2 + case["room"] // page) + 7
        refs = torch.zeros(pool, dtype=torch.int32, device=device)
        refs[table[table >= 0].long()] = 1
        # the parents' pages lie among the free ones
        shuffle = torch.randperm(pool, generator=g, device=device).int()
        s["table"] = torch.full((n + m, width), -1, dtype=torch.int32, device=device)
        s["table"][:n] = torch.where(table >= 0, shuffle[table.clamp(min=0).long()], table)
        s["refs"] = torch.empty_like(refs)
        s["refs"][shuffle.long()] = refs
        s["lens"] = torch.tensor(lens + [0] * m, dtype=torch.int32, device=device)
        s["parents"] = torch.arange(n, device=device, dtype=torch.int32).repeat_interleave(case["forks"])
        s["children"] = torch.randperm(m, generator=g, device=device).int() + n
        s["want"] = torch.tensor(lens, dtype=torch.int32, device=device)[s["parents"].long()] + case["room"]
        s["k"], s["v"] = _cache(g, case, pool, device)
    else:
        P = case["pages"]
        live = min(P, max(1, int(P * case["live"])))
        ids = torch.randperm(P, generator=g, device=device)[:live]
        cells = case["rows"] * case["width"]
        # every live page is some sequence's if the table has room, and some
        # are shared
        table = torch.full((cells,), -1, dtype=torch.int32, device=device)
        used = max(1, cells - cells // 4)
        pick = torch.arange(used, device=device) % live
        table[torch.randperm(cells, generator=g, device=device)[:used]] = ids[pick].int()
        s["table"] = table.view(case["rows"], case["width"])
        s["refs"] = torch.zeros(P, dtype=torch.int32, device=device)
        s["refs"][ids] = 1
        s["refs"].scatter_add_(0, ids[pick[live:]], torch.ones_like(pick[live:], dtype=torch.int32))
        s["k"], s["v"] = _cache(g, case, P, device)
        # renamed tables and counts go to arrays of their own, so that a pass
        # can be repeated; the pages themselves move in place
        s["out"] = (torch.empty_like(s["table"]), torch.empty_like(s["refs"]))
    return s


# ------------------------------------------------------------ the plain forms

def _plain_attention(q, k, v, valid, scale):
    """q [B, Hkv, R, D], k and v [B, Hkv, L, D], valid [B, 1 or Hkv, R, L]."""
    scores = torch.matmul(q.float(), k.float().transpose(-1, -2)) * scale
    scores = scores.masked_fill(~valid, -math.inf)
    top = scores.amax(-1, keepdim=True)
    weights = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = weights.sum(-1, keepdim=True)
    out = torch.matmul(weights, v.float()) / torch.where(total == 0, 1.0, total)
    return out.to(q.dtype), (top + torch.log(total)).squeeze(-1)


def _valid(table, lens, page, T, window, rows):
    """Which positions each of the `rows` query rows sees, [B, 1, rows, L]:
    row r is the new token r % T."""
    L = table.shape[1] * page
    at = torch.arange(L, device=table.device)
    last = (lens[:, None] - T + torch.arange(rows, device=table.device)[None, :] % T)[:, :, None]
    seen = at[None, None, :] <= last
    if window >= 0:
        seen = seen & (at[None, None, :] >= last - window)
    return (seen & (table >= 0).repeat_interleave(page, dim=1)[:, None, :])[:, None]


def _plain_paged(s):
    c, table = s["case"], s["table"]
    B, H, T, d = s["q"].shape
    Hkv, page = c["Hkv"], c["page"]
    at = table.clamp(min=0).long()
    k, v = (x[at].permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, d) for x in (s["k"], s["v"]))
    rows = H // Hkv * T
    valid = _valid(table, s["lens"], page, T, c["window"], rows)
    o, lse = _plain_attention(s["q"].view(B, Hkv, rows, d), k, v, valid, s["scale"])
    return o.view(B, H, T, d), lse.view(B, H, T)


def _plain_latent(s):
    c, table = s["case"], s["table"]
    B, H, T, D = s["q"].shape
    rows = s["c"][table.clamp(min=0).long()].reshape(B, 1, -1, D)
    valid = _valid(table, s["lens"], c["page"], T, -1, H * T)
    o, lse = _plain_attention(s["q"].view(B, 1, H * T, D), rows, rows[..., :c["rank"]], valid, s["scale"])
    return o.view(B, H, T, c["rank"]), lse.view(B, H, T)


def _both(s):
    return [x for x in (s["k"], s["v"]) if x is not None]


def _plain_append(s):
    page, T = s["case"]["page"], s["case"]["T"]
    new = torch.arange(T, device=s["pos"].device)[None, :]
    at = (s["pos"][:, None] + new).long()
    pages = s["table"].gather(1, at // page).long()
    b, u = torch.nonzero(new < s["count"][:, None], as_tuple=True)
    for pool, rows in zip(_both(s), (s["new_k"], s["new_v"])):
        pool[pages[b, u], :, at[b, u] % page] = rows[b, :, u]
    return _both(s)


def _plain_fork(s):
    page, table, lens, refs = s["case"]["page"], s["table"], s["lens"], s["refs"]
    parents, children = s["parents"].long(), s["children"].long()
    width = torch.arange(table.shape[1], device=table.device)[None, :]
    # the lowest free pages go to the forks that need one, in order
    length = lens[parents]
    full, part = length // page, length % page
    free = torch.cumsum(refs == 0, 0)
    asked = torch.cumsum(part > 0, 0)
    needs = (part > 0) & (asked <= free[-1])
    fresh = torch.where(needs, torch.searchsorted(free, asked).clamp(max=refs.numel() - 1), -1).int()
    source = table[parents]
    shared = width < full[:, None]
    last = source.gather(1, full[:, None].long()).squeeze(1)
    table[children] = torch.where(shared, source, torch.where((width == full[:, None]) & needs[:, None],
                                                              fresh[:, None], -1))
    lens[children] = length
    refs.scatter_add_(0, source.clamp(min=0).flatten().long(), shared.flatten().int())
    refs.scatter_add_(0, fresh.clamp(min=0).long(), needs.int())
    move = torch.nonzero(needs).squeeze(1)
    to, frm = fresh[move].long(), last[move].long()
    kept = (torch.arange(page, device=table.device)[None, :] < part[move][:, None])[:, None, :, None]
    for pool in _both(s):
        pool[to] = torch.where(kept, pool[frm], pool[to])
    # room for the next tokens, again the lowest free pages
    row = table[children]
    lacks = (row < 0) & (width < ((s["want"] + page - 1) // page)[:, None])
    asked = torch.cumsum(lacks.flatten(), 0).view_as(lacks)
    free = torch.cumsum(refs == 0, 0)
    got = torch.searchsorted(free, asked.contiguous()).clamp(max=refs.numel() - 1).int()
    row = torch.where(lacks, got, row)
    table[children] = row
    refs.scatter_add_(0, row.clamp(min=0).flatten().long(), lacks.flatten().int())
    batch = table[children]
    # and all of it dropped again
    refs.scatter_add_(0, batch.clamp(min=0).flatten().long(), -(batch >= 0).flatten().int())
    table[children] = -1
    lens[children] = 0
    return [fresh, batch, table, lens, refs] + _both(s)


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    live = refs > 0
    count = live.sum()
    at = torch.arange(refs.numel(), device=refs.device)
    holes = torch.cumsum(~live & (at < count), 0)
    moves = live & (at >= count)
    to = torch.where(moves, torch.searchsorted(holes, torch.cumsum(moves, 0)), at)
    frm = torch.nonzero(moves).squeeze(1)
    for pool in _both(s):
        pool[to[frm]] = pool[frm]
    new_table = torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table)
    new_refs = torch.where(live | (at >= count), refs, 0)
    new_refs[to[frm]] = refs[frm]
    new_refs = torch.where(at < count, new_refs, 0)
    return [new_table, new_refs, count.int().view(1)] + _both(s)


# --------------------------------------------------------- the package's calls

def _run_own(s):
    import exact_softmax_attention_04_b200 as attn
    c = s["case"]
    if s["kind"] == "paged":
        return attn.attn_decode_paged(s["q"], s["k"], s["v"], s["table"], s["lens"], window=c["window"],
                                      scale=s["scale"], workspace=s["workspace"])
    if s["kind"] == "latent":
        return attn.attn_decode_latent(s["q"], s["c"], s["table"], s["lens"], scale=s["scale"],
                                       workspace=s["workspace"])
    if s["kind"] == "append":
        attn.pages_append(s["new_k"], s["new_v"], s["k"], s["v"], s["table"], s["pos"], s["count"])
        return _both(s)
    if s["kind"] == "fork":
        fresh, _ = attn.pages_fork(s["k"], s["v"], s["table"], s["lens"], s["refs"], s["parents"], s["children"])
        attn.pages_reserve(s["table"], s["refs"], s["children"], s["want"], c["page"])
        batch = s["table"][s["children"].long()]
        attn.pages_free(s["table"], s["lens"], s["refs"], s["children"])
        return [fresh, batch, s["table"], s["lens"], s["refs"]] + _both(s)
    count = attn.pages_compact(s["k"], s["v"], s["table"], s["refs"], out=s["out"])
    return [s["out"][0], s["out"][1], count] + _both(s)


def run(state):
    if own:
        return _run_own(state)
    plain = {"paged": _plain_paged, "latent": _plain_latent, "append": _plain_append, "fork": _plain_fork,
             "compact": _plain_compact}
    return plain[state["kind"]](state)


# --------------------------------------------------------- work, and the truth

def work(case):
    kind, page = case["kind"], case["page"]
    if kind in ("paged", "latent"):
        lens = _lengths(case, case["B"])
        window = case.get("window", -1)
        T = case["T"]
        read = [x if window < 0 else min(x, window + T) for x in lens]
        seen = sum(max(0, min(x - T + u + 1, x if window < 0 else window + 1)) for x in lens for u in range(T))
        tables = 4 * (sum(-(-x // page) for x in read) + len(lens))
        if kind == "paged":
            H, d = case["Hkv"] * case["G"], case["d"]
            rows = case["B"] * H * T
            return {"bytes": sum(read) * case["Hkv"] * d * 4 + rows * (4 * d + 4) + tables, "flops": 4 * d * H * seen}
        rank, rows = case["rank"], case["B"] * case["H"] * T
        return {"bytes": sum(read) * (rank + 64) * 2 + rows * (2 * (rank + 64) + 2 * rank + 4) + tables,
                "flops": 2 * case["H"] * seen * (2 * rank + 64)}
    pools = 1 if case["latent"] else 2
    row = case["Hkv"] * case["d"] * 2 * pools
    if kind == "append":
        B, T = case["B"], case["T"]
        counts = [T - (T // 2) * i // max(1, B - 1) for i in range(B)] if case["ragged"] else [T] * B
        return {"bytes": 2 * sum(counts) * row + 4 * sum(2 + -(-x // page) for x in counts), "flops": 0}
    if kind == "fork":
        n, f = case["parents"], case["forks"]
        lens = [case["longest"] - (case["longest"] // 2) * i // max(1, n - 1) for i in range(n)]
        copied = sum(x % page for x in lens) * f
        # a child's table is written, gathered (read and written) and cleared;
        # a share's count is raised and dropped
        entries = sum(-(-(x + case["room"]) // page) for x in lens) * f
        return {"bytes": 2 * copied * row + entries * 4 * (5 + 4), "flops": 0}
    P = case["pages"]
    live = min(P, max(1, int(P * case["live"])))
    moved = live * (P - live) // P
    return {"bytes": 2 * moved * page * row + 8 * (case["rows"] * case["width"] + P), "flops": 0}


def exact(case, seed):
    """Attention in 64 bits, one sequence after the other; what the page
    operators return are copies and whole numbers, which have no such value."""
    if case["kind"] not in ("paged", "latent"):
        return None
    s = prepare(case, seed)
    page, T = case["page"], case["T"]
    q = s["q"].double()
    B, H = q.shape[:2]
    paged = case["kind"] == "paged"
    wide = case["d"] if paged else case["rank"]
    o = torch.zeros((B, H, T, wide), dtype=torch.float64, device=q.device)
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device=q.device)
    for b in range(B):
        n = int(s["lens"][b])
        if n == 0:
            continue
        ids = s["table"][b, : -(-n // page)].long()
        for h in range(case["Hkv"] if paged else 1):
            if paged:
                keys, values = (x[ids][:, h].reshape(-1, wide)[:n].double() for x in (s["k"], s["v"]))
                heads = slice(h * case["G"], (h + 1) * case["G"])
            else:
                keys = s["c"][ids].reshape(-1, q.shape[-1])[:n].double()
                values, heads = keys[:, :wide], slice(0, H)
            for u in range(T):
                end = n - T + u + 1
                begin = max(0, end - 1 - case["window"]) if paged and case["window"] >= 0 else 0
                if end > begin:
                    logits = q[b, heads, u] @ keys[begin:end].T * s["scale"]
                    lse[b, heads, u] = torch.logsumexp(logits, -1)
                    o[b, heads, u] = torch.softmax(logits, -1) @ values[begin:end]
    return o, lse
