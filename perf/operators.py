"""Workloads of the paged-serving operators: the step plan (page tables, slot maps), the
query/key prologue with positions on several axes, the 4-bit cache rows, and decode / verify
attention over the 4-bit paged cache.

`own` False computes each in elementary torch operations, True through the library.
"""
import math

import torch

own = False

N_Q, N_KV, GROUP, DIM, ROT = 24, 2, 12, 256, 64
EPS = 1e-6
BLOCK = 16                                   # values per 4-bit scale
NIBBLE_DIMS = [0, 2, 4, 6, 1, 3, 5, 7]       # dim of each nibble of a 32-bit word, lowest first


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a full batch: every sequence adds a token, few need a page
        {"name": "plan_256x1", "op": "plan", "n_seq": 256, "new": 1, "max_len": 8192, "page": 64},
        # admission of prompts: 48 sequences add a few thousand tokens each
        {"name": "plan_48x2700", "op": "plan", "n_seq": 48, "new": 2700, "max_len": 500, "page": 32},
        # the new tokens of a decode batch
        {"name": "axes_64", "op": "axes", "n_tok": 64, "interleaved": True},
        # a prompt chunk of text and image tokens, odd size
        {"name": "axes_8191", "op": "axes", "n_tok": 8191, "interleaved": False},
        # a decode batch's rows stored (and read back)
        {"name": "cache_64", "op": "cache", "n_tok": 64, "page": 64},
        # a prompt chunk stored, then widened for the next chunk's prefill
        {"name": "cache_8191", "op": "cache", "n_tok": 8191, "page": 32},
        # a long prefix stored and widened
        {"name": "cache_65536", "op": "cache", "n_tok": 65536, "page": 128},
        # one user, short context, one token: latency
        {"name": "decode_1x1_l300", "op": "verify", "n_seq": 1, "rows": 1, "max_len": 300,
         "page": 64, "ragged": False},
        # one user, long context, one token: the key axis split over the whole device
        {"name": "decode_1x1_l65536", "op": "verify", "n_seq": 1, "rows": 1, "max_len": 65536,
         "page": 128, "ragged": False},
        # a decode batch of ragged lengths
        {"name": "decode_64x1_l8192", "op": "verify", "n_seq": 64, "rows": 1, "max_len": 8192,
         "page": 64, "ragged": True},
        # short verify windows, odd lengths, pages smaller than a key tile
        {"name": "verify_5x6_l12345", "op": "verify", "n_seq": 5, "rows": 6, "max_len": 12345,
         "page": 32, "ragged": True},
        # full verify windows over long caches
        {"name": "verify_8x16_l65536", "op": "verify", "n_seq": 8, "rows": 16, "max_len": 65536,
         "page": 128, "ragged": False},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "axes", "cache", "verify", "verify"])
    page = rng.choice([32, 64, 96, 128, 256])
    if op == "plan":
        n_seq = _log_int(rng, 1, 1024)
        return {"op": op, "n_seq": n_seq, "new": _log_int(rng, 1, max(1, 120000 // n_seq)),
                "max_len": _log_int(rng, 1, 16384), "page": page}
    if op == "axes":
        return {"op": op, "n_tok": _log_int(rng, 1, 8191), "interleaved": rng.random() < 0.5}
    if op == "cache":
        return {"op": op, "n_tok": _log_int(rng, 1, 65536), "page": page}
    rows = rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 10, 11, 13, 16])
    n_seq = _log_int(rng, 1, 96)
    max_len = _log_int(rng, 1, min(65536, 8 * 65536 // n_seq))
    return {"op": op, "n_seq": n_seq, "rows": rows, "max_len": max_len, "page": page,
            "ragged": rng.random() < 0.7}


def _lens(case):
    """Cached tokens of each sequence: all max_len, or spread between none and max_len."""
    n, m = case["n_seq"], case["max_len"]
    if not case.get("ragged", True):
        return [m] * n
    return [m if b == 0 else (m * ((b * 37 + 11) % 64)) // 64 for b in range(n)]


def _news(case):
    """Planned tokens of each sequence: `new`, varied by up to a quarter (a few add none)."""
    n = case["new"]
    return [n if n == 1 else 0 if b % 17 == 5 else max(1, n - (n * (b % 8)) // 32)
            for b in range(case["n_seq"])]


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _bf16(g, *shape, sigma=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * sigma).to(torch.bfloat16)


def _quantize(x):
    """x [..., 256] -> (codes uint8 [..., 128], scale bytes uint8 [..., 16])."""
    v = x.float().unflatten(-1, (DIM // BLOCK, BLOCK))
    a = v.abs().amax(-1)
    a = (a / torch.full_like(a, 7)).clamp(2.0 ** -20, 3840.0)   # a true division: ties matter
    m, e = torch.frexp(a)                                  # a = m 2^e, m in [0.5, 1)
    q = torch.round(m * 16)                                # 4 significant bits, ties to even
    s = torch.ldexp(q / 16, e)
    up = (q == 16).to(torch.int32)
    byte = (e - 1 + up + 20) * 8 + torch.where(q == 16, 0, q - 8).to(torch.int32)
    n = (torch.round(v / s[..., None]).clamp(-8, 7) + 8).to(torch.uint8).flatten(-2)
    nib = n.unflatten(-1, (DIM // 8, 8))[..., NIBBLE_DIMS].unflatten(-1, (4, 2))
    return (nib[..., 0] | (nib[..., 1] << 4)).flatten(-2), byte.to(torch.uint8)


def _widen(codes, scales):
    """The fp32 values [..., 256] of code rows and their scale bytes."""
    nib = torch.stack([codes & 15, codes >> 4], -1).unflatten(-2, (DIM // 8, 4)).flatten(-2)
    order = [NIBBLE_DIMS.index(d) for d in range(8)]
    n = nib[..., order].flatten(-2).to(torch.int32) - 8
    b = scales.to(torch.int32)
    s = torch.ldexp(1 + (b & 7).float() / 8, (b >> 3) - 20)
    return n.float() * s.repeat_interleave(BLOCK, -1)


def _pools(g, n_pages, page):
    """Code and scale pools of n_pages pages of normal rows."""
    codes = torch.empty(n_pages, N_KV, page, DIM // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(n_pages, N_KV, page, DIM // BLOCK, dtype=torch.uint8, device="cuda")
    step = max(1, 65536 // page)
    for i in range(0, n_pages, step):
        x = _bf16(g, min(step, n_pages - i), N_KV, page, DIM)
        codes[i:i + step], scales[i:i + step] = _quantize(x)
    return codes, scales


def _axes_positions(n, interleaved):
    """Positions [3][n] of time, height, width: runs of 256 text tokens (all axes alike), each
    followed by a 24 x 32 grid of image tokens."""
    i = torch.arange(n, device="cuda")
    base, o = (i // 1024) * 288, i % 1024
    q = o - 256
    text = o < 256
    pos = torch.stack([torch.where(text, base + o, base + 256),
                       torch.where(text, base + o, base + 256 + q // 32),
                       torch.where(text, base + o, base + 256 + q % 32)]).to(torch.int32)
    pairs = [i % 3 for i in range(ROT // 2)] if interleaved else [0] * 8 + [1] * 12 + [2] * 12
    return pos.contiguous(), pairs


def prepare(case, seed):
    g = _gen(seed)
    s = {"op": case["op"]}
    if case["op"] == "plan":
        lens, news, page = _lens(case), _news(case), case["page"]
        n = len(lens)
        held = [-(-x // page) for x in lens]
        after = [-(-(x + y) // page) for x, y in zip(lens, news)]
        total = sum(after) + 16
        perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        width = max(after) + 2
        table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
        hd = torch.tensor(held, device="cuda")
        live = torch.arange(width, device="cuda")[None, :] < hd[:, None]
        table[live] = perm[:sum(held)]
        free = perm[sum(held):].contiguous()
        s.update(seq_len=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 new_len=torch.tensor(news, dtype=torch.int32, device="cuda"),
                 table=table, held=hd.to(torch.int32), free=free,
                 free_count=torch.tensor([free.numel()], dtype=torch.int32, device="cuda"),
                 held_out=torch.empty_like(hd, dtype=torch.int32),
                 free_count_out=torch.empty(1, dtype=torch.int32, device="cuda"),
                 delta=torch.randint(-3, 1, (n,), generator=g, device="cuda", dtype=torch.int32),
                 page=page, max_tokens=sum(news) + 5)
    elif case["op"] == "axes":
        n = case["n_tok"]
        pos, pairs = _axes_positions(n, case["interleaved"])
        inv = 1e7 ** (-torch.arange(ROT // 2, device="cuda", dtype=torch.float64) * 2 / ROT)
        rows = (n // 1024 + 1) * 288 + 64
        ang = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * inv
        s.update(k=_bf16(g, n, N_KV, DIM), qg=_bf16(g, n, N_Q, 2 * DIM),
                 w_k=_bf16(g, DIM, sigma=0.1), w_q=_bf16(g, DIM, sigma=0.1), pos=pos,
                 pairs=pairs, pair_index=torch.tensor(pairs, device="cuda"),
                 cos=ang.cos().to(torch.bfloat16), sin=ang.sin().to(torch.bfloat16))
    elif case["op"] == "cache":
        n, page = case["n_tok"], case["page"]
        n_pages = -(-n // page) + 3
        pages = torch.randperm(n_pages, generator=g, device="cuda")
        t = torch.arange(n, device="cuda")
        kv = _bf16(g, n, 2, N_KV, DIM)     # the fused key/value projection: V is a strided view
        s.update(k=kv[:, 0].contiguous(), v=kv[:, 1],
                 slots=(pages[t // page] * page + t % page).to(torch.int32))
        for name in ("k", "v"):
            s[name + "_codes"] = torch.zeros(n_pages, N_KV, page, DIM // 2, dtype=torch.uint8,
                                             device="cuda")
            s[name + "_scales"] = torch.zeros(n_pages, N_KV, page, DIM // BLOCK,
                                              dtype=torch.uint8, device="cuda")
    else:
        lens, rows, page = _lens(case), case["rows"], case["page"]
        need = [-(-(x + rows) // page) for x in lens]
        n_pages = sum(need) + 2
        s["k_codes"], s["k_scales"] = _pools(g, n_pages, page)
        s["v_codes"], s["v_scales"] = _pools(g, n_pages, page)
        perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros(len(lens), max(need), dtype=torch.int32, device="cuda")
        nd = torch.tensor(need, device="cuda")
        table[torch.arange(max(need), device="cuda")[None, :] < nd[:, None]] = perm[:sum(need)]
        s.update(table=table, seq_len=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 q=_bf16(g, len(lens), rows, N_Q, DIM), qg=_bf16(g, len(lens), rows, N_Q, 2 * DIM))
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["op"]
    if own:
        from verify_gated_gqa_gb300 import binding as B

        if op == "plan":
            row_start, slots, pos, info = B.ga_page_plan(
                s["seq_len"], s["new_len"], s["table"], s["held"], s["free"], s["free_count"],
                s["page"], s["max_tokens"], pos_delta=s["delta"], held_out=s["held_out"],
                free_count_out=s["free_count_out"])
            return (s["table"], s["held_out"], s["free_count_out"], row_start, slots, pos, info)
        if op == "axes":
            return B.ga_qk_prologue_axes(s["k"], s["w_k"], s["qg"], s["w_q"], s["pos"], s["pairs"],
                                         s["cos"], s["sin"])
        if op == "cache":
            pools = (s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])
            B.ga_kv_quantize_q4(s["k"], s["v"], *pools, slots=s["slots"])
            return B.ga_kv_dequantize_q4(*pools, slots=s["slots"])
        return B.ga_attn_verify_q4(s["q"], s["qg"], s["k_codes"], s["k_scales"], s["v_codes"],
                                   s["v_scales"], s["table"], s["seq_len"])
    return {"plan": _plan, "axes": _axes, "cache": _cache, "verify": _verify}[op](s)


def _plan(s):
    page, table, dev = s["page"], s["table"], s["table"].device
    n, width = table.shape
    lens, new, held = s["seq_len"].long(), s["new_len"].long(), s["held"].long()
    need = ((lens + new + page - 1) // page - held).clamp(min=0)
    first = need.cumsum(0) - need                       # pages taken before sequence b's
    col = torch.arange(width, device=dev)[None, :]
    fresh = (col >= held[:, None]) & (col < (held + need)[:, None])
    index = s["free_count"].long() - 1 - (first[:, None] + col - held[:, None])
    table.copy_(torch.where(fresh, s["free"][index.clamp(0, s["free"].numel() - 1)], table))
    ends = new.cumsum(0)
    row_start = torch.cat([ends.new_zeros(1), ends])
    t = torch.arange(s["max_tokens"], device=dev)
    live = t < ends[-1]
    b = torch.searchsorted(ends, t, right=True).clamp(max=n - 1)
    p = lens[b] + t - row_start[b]
    slot = table[b, (p // page).clamp(0, width - 1)].long() * page + p % page
    zero = torch.zeros_like(need[:1])
    return (table, (held + need).int(), (s["free_count"] - need.sum()).int(), row_start.int(),
            torch.where(live, slot, -1).int(),
            torch.where(live, p + s["delta"].long()[b], 0).int(),
            torch.cat([zero, ends[-1:], need.sum()[None], zero]).int())


def _axes(s):
    at = s["pos"].long()[s["pair_index"]].T               # [n, 32] table rows
    pair = torch.arange(ROT // 2, device=at.device)
    cos = s["cos"][at, pair].float()[:, None]
    sin = s["sin"][at, pair].float()[:, None]

    def prep(x, w):
        x = x.float()
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * (1 + w.float())
        a, b = y[..., :32], y[..., 32:64]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., 64:]], -1).to(torch.bfloat16)

    return prep(s["k"], s["w_k"]), prep(s["qg"][..., :DIM], s["w_q"])


def _cache(s):
    slots = s["slots"].long()
    out = []
    for name in ("k", "v"):
        codes, scales = s[name + "_codes"], s[name + "_scales"]
        page = codes.shape[2]
        at = (slots // page, slice(None), slots % page)
        codes[at], scales[at] = _quantize(s[name])
        out.append(_widen(codes[at], scales[at]).to(torch.bfloat16))
    return tuple(out)


def _verify(s):
    n, rows = s["q"].shape[:2]
    table = s["table"].long()

    def gather(codes, scales):                            # [n, 2, keys, 256]
        pick = lambda t: t[table].transpose(1, 2).flatten(2, 3)  # noqa: E731
        return _widen(pick(codes), pick(scales))

    q = s["q"].float().view(n, rows, N_KV, GROUP, DIM).permute(0, 2, 1, 3, 4).flatten(2, 3)
    k = gather(s["k_codes"], s["k_scales"])
    t = q @ k.transpose(-1, -2) / 16                      # [n, 2, rows * 12, keys]
    del k
    last = s["seq_len"].long()[:, None] + torch.arange(rows, device=t.device)
    seen = torch.arange(t.shape[-1], device=t.device) <= last[..., None]
    seen = seen[:, None].repeat_interleave(GROUP, 2)
    t = t.masked_fill(~seen, -math.inf)
    e = torch.exp(t - t.amax(-1, keepdim=True))
    del t
    o = (e @ gather(s["v_codes"], s["v_scales"])) / e.sum(-1, keepdim=True)
    o = o.view(n, N_KV, rows, GROUP, DIM).permute(0, 2, 1, 3, 4).reshape(n, rows, N_Q, DIM)
    gate = 1 / (1 + torch.exp(-s["qg"][..., DIM:].float()))
    return (o * gate).to(torch.bfloat16).flatten(2)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "plan":
        lens, news, page = _lens(case), _news(case), case["page"]
        taken = sum(-(-(x + y) // page) - -(-x // page) for x, y in zip(lens, news))
        # lengths, pages held (read, written), offsets and row starts; a page: popped, entered;
        # a token: slot and position
        return {"bytes": 24 * len(lens) + 8 * taken + 8 * (sum(news) + 5), "flops": 0}
    if case["op"] == "axes":
        n = case["n_tok"]
        # 26 rows of 256 values in and out, three positions
        return {"bytes": n * (26 * DIM * 2 * 2 + 12), "flops": n * 26 * DIM * 6}
    if case["op"] == "cache":
        # K and V rows in, code and scale rows out, widened rows out
        return {"bytes": case["n_tok"] * (2 * 1024 + 576 + 2 * 1024 + 4), "flops": 0}
    lens, rows = _lens(case), case["rows"]
    keys = sum(x + rows for x in lens)
    pairs = sum(x * rows + rows * (rows + 1) // 2 for x in lens)
    # a key: 2 heads x (K and V) x 144 bytes; a query row: query, gate and output
    return {"bytes": keys * 576 + len(lens) * rows * N_Q * DIM * 6, "flops": pairs * N_Q * DIM * 4}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    if case["op"] == "plan":
        return None                                       # whole numbers only
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "axes":
        out = []
        for x, w in ((s["k"], s["w_k"]), (s["qg"][..., :DIM], s["w_q"])):
            x = x.to(f64)
            y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / DIM + EPS)
            y = y + y * w.to(f64)
            z = y.clone()
            for i, axis in enumerate(s["pairs"]):
                row = s["pos"][axis].long()
                c, d = s["cos"][row, i].to(f64)[:, None], s["sin"][row, i].to(f64)[:, None]
                z[..., i] = y[..., i] * c - y[..., i + 32] * d
                z[..., i + 32] = y[..., i + 32] * c + y[..., i] * d
            out.append(z)
        return tuple(out)
    if case["op"] == "cache":
        out = []
        for x in (s["k"], s["v"]):
            z = x.to(f64).reshape(*x.shape[:-1], DIM // BLOCK, BLOCK)
            top = z.abs().max(-1, keepdim=True).values
            top = torch.clamp(top.div(torch.tensor(7.0, dtype=f64, device="cuda").expand_as(top)), min=2.0 ** -20, max=3840.0)
            unit = torch.exp2(torch.floor(torch.log2(top)) - 3)
            scale = torch.round(top / unit) * unit
            out.append((torch.clamp(torch.round(z / scale), -8, 7) * scale).reshape(x.shape))
        return tuple(out)
    rows, page = case["rows"], case["page"]
    out = torch.zeros(case["n_seq"], rows, N_Q, DIM, dtype=f64, device="cuda")

    def pull(codes, scales, pages, head, keys):
        c = codes[pages, head].reshape(-1, DIM // 2)[:keys].long()
        b = scales[pages, head].reshape(-1, DIM // BLOCK)[:keys].long()
        word = (c.view(keys, DIM // 8, 4) << torch.tensor([0, 8, 16, 24], device="cuda")).sum(-1)
        shift = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device="cuda")
        n = ((word[..., None] >> shift) & 15).view(keys, DIM // BLOCK, BLOCK) - 8
        scale = (8 + b % 8).to(f64) * torch.exp2((b // 8 - 23).to(f64))
        return (n * scale[..., None]).view(keys, DIM)

    for i, length in enumerate(_lens(case)):
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
