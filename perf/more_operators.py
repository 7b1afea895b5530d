"""Workloads of the 8-bit paged cache and of its pages: rows of keys and values stored in 8 bits
with a scale for each block of 32 tokens and head, decode and verify attention over them, and
the pages' life beside the step plan: a row forked into others, pages given back, the pool
compacted, and the copies that forks and compactions ask for.

`own` False computes each in elementary torch operations, True through the library.
"""
import math

import torch

own = False

N_Q, N_KV, GROUP, DIM = 24, 2, 12, 256
BLOCK = 32                                   # tokens of one head that share a scale
E_MIN, E_MAX = -32, 31                       # exponents of the scales


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the new tokens of a decode batch, one a sequence, into blocks that hold tokens already
        {"name": "store_64x1", "op": "store", "n_seq": 64, "new": 1, "page": 64},
        # a long prompt (odd size) stored, then read back for the next chunk's prefill
        {"name": "store_1x40001", "op": "store", "n_seq": 1, "new": 40001, "page": 128},
        # one user, short context, one token: latency
        {"name": "decode_1x1_l300", "op": "verify", "n_seq": 1, "rows": 1, "max_len": 300,
         "page": 64, "ragged": False},
        # a decode batch of ragged lengths
        {"name": "decode_64x1_l8192", "op": "verify", "n_seq": 64, "rows": 1, "max_len": 8192,
         "page": 64, "ragged": True},
        # short verify windows, odd lengths, pages smaller than a key tile
        {"name": "verify_5x6_l12345", "op": "verify", "n_seq": 5, "rows": 6, "max_len": 12345,
         "page": 32, "ragged": True},
        # full verify windows over long caches
        {"name": "verify_8x16_l65536", "op": "verify", "n_seq": 8, "rows": 16, "max_len": 65536,
         "page": 128, "ragged": False},
        # one prompt sampled four times
        {"name": "fork_1x3_l2000", "op": "fork", "parents": 1, "children": 3, "max_len": 2000,
         "page": 64},
        # a batch of prompts, each sampled eight times
        {"name": "fork_32x7_l4096", "op": "fork", "parents": 32, "children": 7, "max_len": 4096,
         "page": 64},
        # a few sequences of a small batch end
        {"name": "release_16_l1000", "op": "release", "parents": 16, "children": 0,
         "max_len": 1000, "page": 64},
        # many end or are cut back at once, most of them branches of shared prompts
        {"name": "release_64x7_l8192", "op": "release", "parents": 64, "children": 7,
         "max_len": 8192, "page": 32},
        # a few pages a step moved down, the budget of a background compaction
        {"name": "compact_512_b16", "op": "compact", "pages": 512, "n_seq": 24, "moves": 16,
         "page": 64},
        # a half-empty pool packed to its front at once
        {"name": "compact_4001_all", "op": "compact", "pages": 4001, "n_seq": 100, "moves": 2000,
         "page": 64},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "verify", "verify", "verify", "fork", "release", "compact"])
    page = rng.choice([32, 64, 96, 128, 256])
    if op == "store":
        n_seq = _log_int(rng, 1, 256)
        return {"op": op, "n_seq": n_seq, "new": _log_int(rng, 1, max(1, 40000 // n_seq)),
                "page": page}
    if op == "verify":
        rows = rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 10, 11, 13, 16])
        n_seq = _log_int(rng, 1, 96)
        max_len = _log_int(rng, 1, min(65536, 8 * 65536 // n_seq))
        return {"op": op, "n_seq": n_seq, "rows": rows, "max_len": max_len, "page": page,
                "ragged": rng.random() < 0.7}
    if op == "compact":
        pages = _log_int(rng, 8, 200000 // page)
        return {"op": op, "pages": pages, "n_seq": _log_int(rng, 1, 256),
                "moves": _log_int(rng, 1, pages // 2 + 1), "page": page}
    parents = _log_int(rng, 1, 64)
    max_len = _log_int(rng, 1, min(16384, 200000 // parents))
    return {"op": op, "parents": parents, "children": rng.choice([1, 2, 3, 4, 7, 8]),
            "max_len": max_len, "page": page}


def _lens(n, m, ragged=True):
    """Cached tokens of each sequence: all m, or spread between none and m."""
    return [m if b == 0 or not ragged else (m * ((b * 37 + 11) % 64)) // 64 for b in range(n)]


def _store_plan(case):
    """(tokens before, tokens added) of each sequence, counted from the beginning of a page."""
    n, new, page = case["n_seq"], case["new"], case["page"]
    old = [0 if n == 1 else (b * 29 + 7) % page for b in range(n)]
    return old, [new if n == 1 else max(1, new - (new * (b % 8)) // 32) for b in range(n)]


def _forks(case):
    """(parent row, child row, tokens shared) of each fork: the children's rows follow the
    parents', a third of the children begin before their parent's end."""
    p, c = case["parents"], case["children"]
    lens = _lens(p, case["max_len"])
    return [(i, p + i * c + j, lens[i] if (i + j) % 3 else lens[i] * 2 // 3)
            for i in range(p) for j in range(c)], lens


def _keeps(case):
    """Tokens that each row keeps: half stay as they are (-1), a sixth are cut back."""
    p, c = case["parents"], case["children"]
    lens = _lens(p, case["max_len"])
    rows = lens + [lens[i] for i in range(p) for _ in range(c)]
    return [-1 if b % 2 else n // 2 if b % 6 == 4 else 0 for b, n in enumerate(rows)], rows


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _bf16(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _empty_pools(n_pages, page):
    s = {}
    for name in ("k", "v"):
        s[name + "_codes"] = torch.zeros(n_pages, N_KV, page, DIM, dtype=torch.uint8, device="cuda")
        s[name + "_scales"] = torch.zeros(n_pages, N_KV, page // BLOCK, dtype=torch.uint8,
                                          device="cuda")
    return s


def _random_pools(g, n_pages, page):
    """Pools of normal rows, a row's magnitude a power of two of its own now and then."""
    s = _empty_pools(n_pages, page)
    step = max(1, 65536 // page)
    for name in ("k", "v"):
        for i in range(0, n_pages, step):
            n = min(step, n_pages - i) * page
            x = _bf16(g, n, N_KV, DIM)
            x *= torch.exp2(-(torch.rand(n, N_KV, 1, generator=g, device="cuda") * 4).floor()).to(torch.bfloat16)
            _store_rows(x, s[name + "_codes"][i:], s[name + "_scales"][i:],
                        torch.arange(n, device="cuda"))
    return s


def _byte_pools(g, n_pages, page):
    return {name + kind: torch.randint(0, 120, (n_pages, N_KV) + tail, dtype=torch.uint8,
                                       generator=g, device="cuda")
            for name in ("k", "v") for kind, tail in (("_codes", (page, DIM)), ("_scales", (page // BLOCK,)))}


def _table(perm, need, width):
    """Rows of page numbers, need[b] of them each, taken from perm in order; -1 after them."""
    nd = torch.tensor(need, device="cuda")
    table = torch.full((len(need), width), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda")[None, :] < nd[:, None]] = perm[:sum(need)]
    return table


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"op": op}
    if op == "store":
        page = case["page"]
        old, new = _store_plan(case)
        need = [-(-(a + b) // page) for a, b in zip(old, new)]
        n_pages = sum(need) + 2
        perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        s.update(_empty_pools(n_pages, page))

        def slots(begin, end):
            table, out = _table(perm, need, max(need)).long(), []
            for b, (i, j) in enumerate(zip(begin, end)):
                t = torch.arange(i, j, device="cuda")
                out.append(table[b][t // page] * page + t % page)
            return torch.cat(out)

        before = slots([0] * len(old), old)
        for name in ("k", "v"):
            _store_rows(_bf16(g, before.numel(), N_KV, DIM), s[name + "_codes"],
                        s[name + "_scales"], before)
        kv = _bf16(g, sum(new), 2, N_KV, DIM)          # the fused projection: V is a strided view
        s.update(k=kv[:, 0].contiguous(), v=kv[:, 1],
                 slots=slots(old, [a + b for a, b in zip(old, new)]).to(torch.int32),
                 read=slots([a // BLOCK * BLOCK for a in old],
                            [a + b for a, b in zip(old, new)]).to(torch.int32))
    elif op == "verify":
        lens, rows, page = _lens(case["n_seq"], case["max_len"], case["ragged"]), case["rows"], case["page"]
        need = [-(-(x + rows) // page) for x in lens]
        n_pages = sum(need) + 2
        s.update(_random_pools(g, n_pages, page))
        perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        s.update(table=_table(perm, need, max(need)).clamp(min=0), seq_len=_i32(lens),
                 q=_bf16(g, len(lens), rows, N_Q, DIM), qg=_bf16(g, len(lens), rows, N_Q, 2 * DIM))
    elif op == "fork":
        forks, lens = _forks(case)
        page = case["page"]
        held = [-(-x // page) for x in lens]
        total = sum(held) + len(forks) + 5
        perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        rows = len(lens) + len(forks)
        s.update(_byte_pools(g, total, page))
        s.update(table=_table(perm, held + [0] * len(forks), max(held) + 2),
                 held=_i32(held + [0] * len(forks)), free=perm[sum(held):].contiguous(),
                 parent=_i32([f[0] for f in forks]), child=_i32([f[1] for f in forks]),
                 lens=_i32([f[2] for f in forks]), page=page)
        s["free"] = torch.cat([s["free"], torch.zeros(sum(held), dtype=torch.int32, device="cuda")])
        s["count"] = _i32([total - sum(held)])
        s["shared"] = torch.zeros(total, dtype=torch.int32, device="cuda")
        s["held_out"] = torch.empty(rows, dtype=torch.int32, device="cuda")
    elif op == "release":
        keeps, lens = _keeps(case)
        p, c, page = case["parents"], case["children"], case["page"]
        held = [-(-x // page) for x in lens]
        # a child shares its parent's whole pages and holds its own last one
        own_pages = held[:p] + [1 if lens[p + i] % page else 0 for i in range(p * c)]
        total = sum(own_pages) + 7
        perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        width = max(held) + 1
        table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
        table[:p] = _table(perm, held[:p], width)
        shared = torch.zeros(total, dtype=torch.int32, device="cuda")
        if c:
            whole = torch.tensor([x // page for x in lens[:p]], device="cuda")
            col = torch.arange(width, device="cuda")[None, :]
            prefix = torch.where(col < whole[:, None], table[:p], -1)
            table[p:] = prefix.repeat_interleave(c, 0)
            shared[prefix[prefix >= 0].long()] = c
            tails = perm[sum(held[:p]):sum(own_pages)]
            at = torch.tensor([i for i in range(p * c) if lens[p + i] % page], dtype=torch.long, device="cuda")
            table[p + at, whole.repeat_interleave(c)[at]] = tails
        s.update(keep=_i32(keeps), table=table, held=_i32(held), shared=shared, page=page,
                 free=torch.cat([perm[sum(own_pages):], torch.zeros(sum(own_pages), dtype=torch.int32, device="cuda")]),
                 count=_i32([7]), held_out=torch.empty(len(lens), dtype=torch.int32, device="cuda"))
    else:
        n, page = case["pages"], case["page"]
        live = n - n // 2
        per = -(-live // case["n_seq"])
        held = [min(per, max(0, live - b * per)) for b in range(case["n_seq"])]
        perm = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
        table = _table(perm, held, per + 1)
        shared = torch.zeros(n, dtype=torch.int32, device="cuda")
        if held[0] and case["n_seq"] > 1 and held[1]:       # the second row begins like the first
            shared[table[0, 0].long()] = 1
            table[1, 1:held[1]] = table[1, :held[1] - 1].clone()
            spare = perm[sum(held[:2]) - 1]
            table[1, 0] = table[0, 0]
            free = torch.cat([perm[live:], spare[None]])
        else:
            free = perm[live:]
        s.update(_byte_pools(g, n, page))
        s.update(table=table, held=_i32(held), shared=shared, page=page, moves=case["moves"],
                 count=_i32([free.numel()]),
                 free=torch.cat([free, torch.zeros(n - free.numel(), dtype=torch.int32, device="cuda")]),
                 table_out=torch.empty_like(table), free_out=torch.empty(n, dtype=torch.int32, device="cuda"),
                 workspace=torch.empty(8 * n + 1024, dtype=torch.uint8, device="cuda"))
    if op in ("fork", "release"):
        s["count_out"] = torch.empty(1, dtype=torch.int32, device="cuda")
    if "shared" in s:
        s["shared_out"] = torch.empty_like(s["shared"])
    return s


POOLS = ("k_codes", "k_scales", "v_codes", "v_scales")


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["op"]
    if own:
        from verify_gated_gqa_gb300 import binding as B

        if op == "store":
            pools = [s[x] for x in POOLS]
            B.ga_kv_quantize_q8(s["k"], s["v"], *pools, slots=s["slots"])
            return B.ga_kv_dequantize_q8(*pools, slots=s["read"])
        if op == "verify":
            return B.ga_attn_verify_q8(s["q"], s["qg"], *(s[x] for x in POOLS), s["table"], s["seq_len"])
        if op == "release":
            info = B.ga_page_release(s["keep"], s["table"], s["held"], s["free"], s["count"], s["shared"],
                                     s["page"], held_out=s["held_out"], free_count_out=s["count_out"],
                                     shared_out=s["shared_out"])
            return s["held_out"], s["free"], s["count_out"], s["shared_out"], info
        pools = [s[x] for x in POOLS]
        if op == "fork":
            src, dst, info = B.ga_page_fork(s["parent"], s["child"], s["lens"], s["table"], s["held"], s["free"],
                                            s["count"], s["shared"], s["page"], held_out=s["held_out"],
                                            free_count_out=s["count_out"], shared_out=s["shared_out"])
            B.ga_page_copy(pools, src, dst)
            return (s["table"], s["held_out"], s["count_out"], s["shared_out"], src, dst, info, *pools)
        src, dst, info = B.ga_page_compact(s["table"], s["held"], s["free"], s["count"], s["shared"], s["moves"],
                                           page_table_out=s["table_out"], free_pages_out=s["free_out"],
                                           shared_out=s["shared_out"], workspace=s["workspace"])
        B.ga_page_copy(pools, src, dst)
        return (s["table_out"], s["free_out"], s["shared_out"], src, dst, info, *pools)
    return {"store": _store, "verify": _verify, "fork": _fork, "release": _release, "compact": _compact}[op](s)


def _e4m3(x):
    """The nearest 8-bit values (ties to even, at most 448) as bytes."""
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _value(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _power(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)


def _store_rows(x, codes, scales, slots):
    """Rows x [n, 2, 256] into their blocks: a block's exponent is the least that holds its new
    rows, and no less than it was unless the block begins anew; codes that were there move to it."""
    if slots.numel() == 0:
        return
    page = codes.shape[2]
    slots = slots.long()
    block, which = torch.unique(slots // BLOCK, return_inverse=True)
    per = page // BLOCK
    at = (block // per, slice(None), block % per)
    x = torch.where(torch.isnan(x), 0, x).float()
    row_max = x.abs().amax(-1)                                            # [n, 2]
    top = torch.zeros(block.numel(), N_KV, device=x.device)
    top = top.scatter_reduce(0, which[:, None].expand(-1, N_KV), row_max, "amax")
    m, e = torch.frexp(top)                                               # 448 = 0.875 x 2^9
    e = torch.where(top > 0, e - 9 + (m > 0.875), E_MIN).clamp(E_MIN, E_MAX)
    fresh = torch.zeros(block.numel(), dtype=torch.bool, device=x.device)
    fresh[which[slots % BLOCK == 0]] = True
    was = (scales[at].int() & 63) + E_MIN                                 # [blocks, 2]
    e = torch.where(fresh[:, None], e, torch.maximum(e, was))
    # the rows of blocks that grew, moved to the new exponent
    grew = ((e > was) & ~fresh[:, None]).any(-1)
    old_at = block[grew][:, None] * BLOCK + torch.arange(BLOCK, device=x.device)
    where = (old_at // page, slice(None), old_at % page)                  # [g, 32, 2, 256]
    moved = codes[where]
    shift = _power((was - e)[grew])[:, None, :, None]
    codes[where] = _e4m3(_value(moved) * shift)
    scales[at] = (e - E_MIN).to(torch.uint8)
    codes[slots // page, :, slots % page] = _e4m3(x * _power(-e)[which][..., None])


def _widen(codes, scales, at):
    """fp32 rows at slots `at` [...]: [..., 2, 256]."""
    page = codes.shape[2]
    e = (scales[at // page, :, at % page // BLOCK].int() & 63) + E_MIN
    return _value(codes[at // page, :, at % page]) * _power(e)[..., None]


def _store(s):
    out = []
    for name in ("k", "v"):
        codes, scales = s[name + "_codes"], s[name + "_scales"]
        _store_rows(s[name], codes, scales, s["slots"])
        out.append(_widen(codes, scales, s["read"].long()).to(torch.bfloat16))
    return tuple(out)


def _verify(s):
    n, rows = s["q"].shape[:2]
    page = s["k_codes"].shape[2]
    at = (s["table"].long()[..., None] * page + torch.arange(page, device=s["q"].device)).flatten(1)
    q = s["q"].float().view(n, rows, N_KV, GROUP, DIM).permute(0, 2, 1, 3, 4).flatten(2, 3)
    k = _widen(s["k_codes"], s["k_scales"], at).transpose(1, 2)            # [n, 2, keys, 256]
    t = q @ k.transpose(-1, -2) / 16                                       # [n, 2, rows * 12, keys]
    del k
    last = s["seq_len"].long()[:, None] + torch.arange(rows, device=t.device)
    seen = torch.arange(t.shape[-1], device=t.device) <= last[..., None]
    seen = seen[:, None].repeat_interleave(GROUP, 2)
    t = t.masked_fill(~seen, -math.inf)
    e = torch.exp(t - t.amax(-1, keepdim=True))
    del t
    o = (e @ _widen(s["v_codes"], s["v_scales"], at).transpose(1, 2)) / e.sum(-1, keepdim=True)
    o = o.view(n, N_KV, rows, GROUP, DIM).permute(0, 2, 1, 3, 4).reshape(n, rows, N_Q, DIM)
    gate = 1 / (1 + torch.exp(-s["qg"][..., DIM:].float()))
    return (o * gate).to(torch.bfloat16).flatten(2)


def _copy_pages(s, src, dst):
    live = src >= 0
    for x in POOLS:
        s[x][dst[live].long()] = s[x][src[live].long()]


def _fork(s):
    """Whole pages of the shared tokens are held by one row more; a page begun is copied to one
    taken from the stack, in order of the forks."""
    parent, child, lens, page = s["parent"].long(), s["child"].long(), s["lens"].long(), s["page"]
    whole, tail = lens // page, (lens % page > 0).long()
    order = tail.cumsum(0) - tail
    fresh = s["free"][(s["count"].long() - 1 - order).clamp(min=0)]
    col = torch.arange(s["table"].shape[1], device=lens.device)[None, :]
    rows = s["table"][parent]
    src = torch.where(tail > 0, rows.gather(1, whole[:, None])[:, 0], -1)
    dst = torch.where(tail > 0, fresh, -1)
    pages = torch.where(col < whole[:, None], rows, s["table"][child])
    s["table"][child] = torch.where((col == whole[:, None]) & (tail > 0)[:, None], fresh[:, None], pages)
    shared = s["shared"] + torch.bincount(rows[col < whole[:, None]].long(), minlength=s["shared"].numel()).int()
    held = s["held"].clone()
    held[child] = (whole + tail).int()
    _copy_pages(s, src, dst)
    info = torch.stack([torch.zeros_like(tail[0]), (parent >= 0).sum(), tail.sum(), whole.sum()]).int()
    return (s["table"], held, s["count"] - tail.sum().int(), shared, src, dst, info, *(s[x] for x in POOLS))


def _release(s):
    """Pages past each row's kept tokens: one holder less, or back on the stack in order of row and
    column where none is left (a page of several rows at its first place)."""
    table, held, page = s["table"], s["held"].long(), s["page"]
    keep = s["keep"].long()
    left = torch.where(keep < 0, held, torch.minimum(held, (keep + page - 1) // page))
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    pages = table[(col >= left[:, None]) & (col < held[:, None])].long()
    shared = s["shared"].long()
    gone = torch.bincount(pages, minlength=shared.numel())
    freed = gone == shared + 1
    index = torch.arange(pages.numel(), device=table.device)
    first = torch.full_like(shared, pages.numel()).scatter_reduce(0, pages, index, "amin")
    back = pages[freed[pages] & (first[pages] == index)]
    free = s["free"].clone()
    n = s["count"].long()
    free[n + torch.arange(back.numel(), device=table.device)] = back.int()
    shared = torch.where(freed, 0, shared - gone)
    rows = ((keep >= 0) & (left < held)).sum()
    info = torch.stack([rows * 0, rows, torch.tensor(back.numel(), device=table.device),
                        torch.tensor(pages.numel(), device=table.device)]).int()
    return left.int(), free, s["count"] + back.numel(), shared.int(), info


def _compact(s):
    """The highest pages in use to the lowest free ones, while that packs the pool."""
    n, count, moves = s["free"].numel(), s["count"].long(), s["moves"]
    dev = s["free"].device
    index = torch.arange(n, device=dev)
    is_free = torch.zeros(n, dtype=torch.bool, device=dev)
    is_free[s["free"][index < count].long()] = True
    live = n - count
    holes = index[is_free & (index < live)]
    movers = index[~is_free & (index >= live)].flip(0)
    k = min(moves, holes.numel())
    src = torch.full((moves,), -1, dtype=torch.int32, device=dev)
    dst = src.clone()
    src[:k], dst[:k] = movers[:k].int(), holes[:k].int()
    to = index.clone()
    to[movers[:k]] = holes[:k]
    mine = torch.arange(s["table"].shape[1], device=dev)[None, :] < s["held"][:, None]
    table = torch.where(mine, to[s["table"].long().clamp(min=0)].int(), s["table"])
    shared = s["shared"].clone()
    shared[holes[:k]], shared[movers[:k]] = shared[movers[:k]], 0
    is_free[holes[:k]], is_free[movers[:k]] = False, True
    free = s["free"].clone()
    left = index[is_free].flip(0).int()
    free[:left.numel()] = left
    _copy_pages(s, src, dst)
    info = torch.stack([live[0] * 0, torch.tensor(k, device=dev), live[0],
                        torch.tensor(holes.numel() - k, device=dev)]).int()
    return (table, free, shared, src, dst, info, *(s[x] for x in POOLS))


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, page = case["op"], case["page"]
    per_page = page * N_KV * DIM * 2 + page // BLOCK * N_KV * 2
    if op == "store":
        old, new = _store_plan(case)
        read = sum(a % BLOCK + b for a, b in zip(old, new))
        # a new token: K and V rows in, codes out; a token read: codes in (those just written are
        # at hand), rows out
        return {"bytes": sum(new) * (4 * DIM * 2 + 4 * DIM + 4) + (read - sum(new)) * 4 * DIM
                + read * (4 * DIM * 2 + 4), "flops": 0}
    if op == "verify":
        lens, rows = _lens(case["n_seq"], case["max_len"], case["ragged"]), case["rows"]
        keys = sum(x + rows for x in lens)
        pairs = sum(x * rows + rows * (rows + 1) // 2 for x in lens)
        # a key: 2 heads x (K and V) x 256 bytes and a scale byte in 32; a query row: query, gate
        # and output
        return {"bytes": keys * 4 * DIM + keys // BLOCK * 4 + len(lens) * rows * N_Q * DIM * 6,
                "flops": pairs * N_Q * DIM * 4}
    if op == "fork":
        forks, lens = _forks(case)
        tails = sum(1 for f in forks if f[2] % page)
        whole = sum(f[2] // page for f in forks)
        total = sum(-(-x // page) for x in lens) + len(forks) + 5
        # a shared page: its number in and out; the counts in and out; a copied page in and out
        return {"bytes": whole * 8 + total * 8 + len(forks) * 20 + tails * (2 * per_page + 8), "flops": 0}
    if op == "release":
        keeps, lens = _keeps(case)
        p, c = case["parents"], case["children"]
        gone = sum(max(0, -(-n // page) + -k // page) for k, n in zip(keeps, lens) if k >= 0)
        total = sum(-(-x // page) for x in lens[:p]) + sum(1 for x in lens[p:] if x % page) + 7
        # a page let go: its number in, its place on the stack out; the counts in and out
        return {"bytes": gone * 8 + total * 8 + len(lens) * 12, "flops": 0}
    n = case["pages"]
    free = n // 2
    moves = min(case["moves"], (n - free) * free // n)
    # the counts, the stack and the table in and out; a moved page in and out
    return {"bytes": n * 16 + (n - free) * 8 + moves * (2 * per_page + 8), "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits
def _decode(codes):
    """Values of 8-bit codes: sign, 4 bits of exponent, 3 of fraction."""
    c = codes.long()
    e, m = (c >> 3) & 15, (c & 7).to(torch.float64)
    v = torch.where(e == 0, m / 512, (8 + m) * torch.exp2((e - 10).to(torch.float64)))
    return torch.where(c >= 128, -v, v)


def _nearest(z):
    """z rounded to 4 significant bits, to multiples of 2^-9 at least, ties to even; at most 448."""
    z = z.clamp(-448.0, 448.0)
    step = torch.exp2((torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3))
    return torch.round(z / step) * step


def exact(case, seed):
    f64 = torch.float64
    if case["op"] not in ("store", "verify"):
        return None                                       # whole numbers and copies of bytes only
    s = prepare(case, seed)
    page = case["page"]
    if case["op"] == "store":
        out = []
        for name in ("k", "v"):
            codes, scales, x = s[name + "_codes"], s[name + "_scales"], s[name].to(f64)
            n_slots = codes.shape[0] * page
            flat = _decode(codes).transpose(1, 2).reshape(n_slots, N_KV, DIM)
            unit = scales.transpose(1, 2).reshape(n_slots // BLOCK, N_KV).to(f64) + E_MIN
            new = torch.zeros(n_slots, dtype=torch.bool, device="cuda")
            rows = torch.zeros(n_slots, N_KV, DIM, dtype=f64, device="cuda")
            new[s["slots"].long()] = True
            rows[s["slots"].long()] = x
            most = rows.view(-1, BLOCK, N_KV, DIM).abs().amax((1, 3))
            need = torch.ceil(torch.log2(most / 448)).clamp(E_MIN, E_MAX)
            anew = new.view(-1, BLOCK)[:, 0, None]
            touched = new.view(-1, BLOCK).any(1)[:, None]
            e = torch.where(anew, need, torch.where(touched, torch.maximum(unit, need), unit))
            per = e.repeat_interleave(BLOCK, 0)[..., None]
            kept = _nearest(flat * torch.exp2(unit.repeat_interleave(BLOCK, 0)[..., None] - per))
            value = torch.where(new[:, None, None], _nearest(rows * torch.exp2(-per)), kept)
            out.append((value * torch.exp2(per))[s["read"].long()])
        return tuple(out)
    rows = case["rows"]
    out = torch.zeros(case["n_seq"], rows, N_Q, DIM, dtype=f64, device="cuda")

    def pull(codes, scales, pages, head, keys):
        e = scales[pages, head].reshape(-1).to(f64) + E_MIN
        v = _decode(codes[pages, head].reshape(-1, DIM)) * torch.exp2(e).repeat_interleave(BLOCK)[:, None]
        return v[:keys]

    for i, length in enumerate(_lens(case["n_seq"], case["max_len"], case["ragged"])):
        keys = length + rows
        pages = s["table"][i, :-(-keys // page)].long()
        for head in range(N_KV):
            k = pull(s["k_codes"], s["k_scales"], pages, head, keys)
            v = pull(s["v_codes"], s["v_scales"], pages, head, keys)
            for r in range(rows):
                q = s["q"][i, r, head * GROUP:(head + 1) * GROUP].to(f64)
                w = torch.softmax((q @ k[:length + r + 1].T) * 0.0625, -1)
                out[i, r, head * GROUP:(head + 1) * GROUP] = w @ v[:length + r + 1]
    return (out * torch.sigmoid(s["qg"][..., DIM:].to(f64))).flatten(2)
