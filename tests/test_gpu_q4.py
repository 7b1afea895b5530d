"""GPU parity of the 4-bit paged serving calls against the float64 oracle: the step plan and
the 4-bit rows value for value, the prologue over position axes bit for bit, the attention
within the error of its two bf16 roundings, and all four run together as a server's steps."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import ga_oracle as O
from tests.parity import SEED, np64
from verify_gated_gqa_gb300 import binding as B
from verify_gated_gqa_gb300 import build as build_mod
from verify_gated_gqa_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_mod.build()
    B.lib()
    yield
    assert B.ga_device_status() == 0


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _pools(n_pages, page, fill=None):
    """Four pools; random bytes unless fill is given (any bytes are finite rows)."""
    make = (lambda k: torch.randint(0, 256, (n_pages, 2, page, k), dtype=torch.uint8, device="cuda")
            if fill is None else torch.full((n_pages, 2, page, k), fill, dtype=torch.uint8,
                                            device="cuda"))
    return make(128), make(16), make(128), make(16)


# ------------------------------------------------------------------ the step plan
def _plan_case(rng, n, page, new, lmax=700, spare=5, release=False):
    L = rng.integers(0, lmax + 1, n)
    a = rng.integers(0, new + 1, n)
    held = -(-L // page) + (rng.integers(0, 3, n) == 0)     # some rows hold a page ahead
    if n > 2:
        L[rng.integers(n)] = -1                             # an unused row
    if release and n > 1:
        a[rng.integers(0, n, 1 + n // 4)] = -1
    need = np.where((a >= 0) & (L >= 0), np.maximum(0, -(-(L + a) // page) - held), 0)
    width = int(max((held + need).max(), 1)) + 1
    total = int(held.sum() + need.sum()) + spare
    perm = rng.permutation(total)
    table = np.full((n, width), -1)
    i = 0
    for b in range(n):
        table[b, :held[b]] = perm[i:i + held[b]]
        i += held[b]
    stack = np.zeros(total, np.int64)
    stack[:total - i] = perm[i:]
    return L, a, table, held, stack, total - i, int(np.where(L >= 0, np.maximum(a, 0), 0).sum())


@pytest.mark.parametrize("n,page,new,pad,release", [
    (1, 32, 1, 0, False), (1, 64, 5000, 3, False), (3, 1, 2, 0, True), (7, 48, 40, 5, True),
    (65, 128, 1, 2, False), (257, 32, 70, 0, True), (1025, 64, 3, 1, True), (2048, 32, 2, 9, True),
    (33, 32, 900, 77, True)])
def test_plan_matches_oracle(n, page, new, pad, release):
    rng = np.random.default_rng(SEED + n)
    L, a, table, held, stack, count, tokens = _plan_case(rng, n, page, new, release=release)
    delta = rng.integers(-5, 50, n)
    mt = tokens + pad
    want = O.page_plan(L, a, table, held, stack, count, page, mt, delta)
    assert want[-1][0] == 0
    for in_place in (False, True):
        t, h, f, c = _i32(table), _i32(held), _i32(stack), _i32([count])
        ho, co = (None, None) if in_place else (torch.empty_like(h), torch.empty_like(c))
        start, slots, pos, info = B.ga_page_plan(_i32(L), _i32(a), t, h, f, c, page, mt,
                                                 pos_delta=_i32(delta), held_out=ho,
                                                 free_count_out=co)
        got = (t, h if in_place else ho, f, c if in_place else co, start, slots, pos, info)
        for name, g, w in zip(("table", "held", "stack", "count", "row_start", "slots",
                               "positions", "info"), got, want):
            assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1)), name


def test_plan_large_step_takes_the_second_launch():
    rng = np.random.default_rng(SEED)
    L, a, table, held, stack, count, tokens = _plan_case(rng, 40, 64, 2000, release=True)
    assert tokens > 8192
    want = O.page_plan(L, a, table, held, stack, count, 64, tokens + 100)
    start, slots, pos, info = B.ga_page_plan(_i32(L), _i32(a), _i32(table), _i32(held), _i32(stack),
                                             _i32([count]), 64, tokens + 100)
    for g, w in zip((start, slots, pos, info), want[4:]):
        assert np.array_equal(g.cpu().numpy(), w)


@pytest.mark.parametrize("kind,status", [("tokens", 1), ("width", 2), ("far", 2), ("pages", 3),
                                         ("held", 4), ("count", 4), ("stack", 4)])
@pytest.mark.parametrize("pad", [0, 9000])
def test_plan_refuses_on_the_device(kind, status, pad):
    page = 32
    L, a = np.array([40, 10, 5]), np.array([4, 30, -1])
    table, held = np.array([[0, 1, -1], [2, -1, -1], [3, -1, -1]]), np.array([2, 1, 1])
    stack, count = np.array([4, 5, 6, 0, 0]), 3
    mt = 34 + pad
    if kind == "tokens":
        a[0], a[1] = mt + 1, 0
        table, L = np.concatenate([table] * 200, 1), np.array([0, 10, 5])
        stack, count = np.arange(600), 500
    elif kind == "width":
        a[0] = 90
    elif kind == "far":
        page, L[0], a[0] = 1 << 20, 1 << 20, 1
    elif kind == "pages":
        count = 0
    elif kind == "held":
        held[1] = 4
    elif kind == "count":
        count = 6
    else:
        count, a[1] = 5, 0
    t, h, f, c = _i32(table), _i32(held), _i32(stack), _i32([count])
    start, slots, pos, info = B.ga_page_plan(_i32(L), _i32(a), t, h, f, c, page, mt)
    want = O.page_plan(L, a, table, held, stack, count, page, mt)
    assert want[-1][0] == status
    for g, w in zip((t, h, f, c, start, slots, pos, info), want):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))


def test_plan_refuses_more_held_pages_than_32_bits_count():
    n, width = 2048, 1 << 21                       # 2^32 pages in all
    table = torch.empty(n, width, dtype=torch.int32, device="cuda")
    held, count = torch.full((n,), width, dtype=torch.int32, device="cuda"), _i32([0])
    stack, lens = torch.full((width,), 7, dtype=torch.int32, device="cuda"), _i32([0] * n)
    start, slots, pos, info = B.ga_page_plan(lens, _i32([-1] * n), table, held, stack, count, 1, 4)
    assert info.tolist() == [4, 0, 0, 0] and count.item() == 0 and slots.tolist() == [-1] * 4
    assert bool((held == width).all()) and bool((stack == 7).all())


def test_plan_without_sequences():
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    start, slots, pos, info = B.ga_page_plan(e, e, torch.zeros(0, 4, dtype=torch.int32, device="cuda"),
                                             e, _i32([3, 4]), _i32([2]), 32, 5)
    assert start.tolist() == [0] and slots.tolist() == [-1] * 5 and pos.tolist() == [0] * 5
    assert info.tolist() == [0, 0, 0, 0]


# ------------------------------------------------------------------ the prologue over axes
def _axes_inputs(n, seed):
    k = synth.normal_bf16(seed, "k", (n, 2, 256)).cuda()
    qg = synth.normal_bf16(seed, "qg", (n, 24, 512)).cuda()
    w_k = synth.normal_bf16(seed, "w_k", (256,), sigma=0.1).cuda()
    w_q = synth.normal_bf16(seed, "w_q", (256,), sigma=0.1).cuda()
    c, s = B.ga_rope_table_host(4096)
    return k, qg, w_k, w_q, c.cuda(), s.cuda()


@pytest.mark.parametrize("n,pairs,ld", [
    (1, [i % 3 for i in range(32)], 1), (77, [0] * 8 + [1] * 12 + [2] * 12, 80),
    (333, [3 - i % 4 for i in range(32)], 333)])
def test_axes_match_oracle(n, pairs, ld):
    k, qg, w_k, w_q, c, s = _axes_inputs(n, SEED + n)
    rng = np.random.default_rng(n)
    na = max(pairs) + 1
    pos = rng.integers(0, 4096, (na, ld))
    pos[0, 0], pos[-1, n - 1] = 4095, 0
    kp, qp = B.ga_qk_prologue_axes(k, w_k, qg, w_q, _i32(pos), pairs, c, s)
    cos, sin = O.rope_tables(4096)
    want_k = O.prep_axes(np64(k), np64(w_k), cos, sin, pos[:, :n], pairs)
    want_q = O.prep_axes(np64(qg)[..., :256], np64(w_q), cos, sin, pos[:, :n], pairs)
    assert np.array_equal(np64(kp), want_k)
    assert np.array_equal(np64(qp), want_q)


def test_axes_equal_positions_are_the_plain_prologue():
    n, base = 515, 1000
    k, qg, w_k, w_q, c, s = _axes_inputs(n, SEED + 3)
    pos = torch.arange(base, base + n, dtype=torch.int32, device="cuda")
    want = B.ga_qk_prologue(k, w_k, qg, w_q, c, s, k_pos_base=base, q_base=base)
    for p, pairs in ((pos, None), (pos[None].repeat(3, 1), [i % 3 for i in range(32)])):
        got = B.ga_qk_prologue_axes(k, w_k, qg, w_q, p, pairs, c, s)
        for g, w in zip(got, want):
            assert torch.equal(g.view(torch.int16), w.view(torch.int16))
    # one side alone, and none of either
    k1, none = B.ga_qk_prologue_axes(k, w_k, None, None, pos, None, c, s)
    assert none is None and torch.equal(k1, want[0])
    none, q1 = B.ga_qk_prologue_axes(None, None, qg, w_q, pos, None, c, s)
    assert none is None and torch.equal(q1, want[1])
    e, _ = B.ga_qk_prologue_axes(k[:0], w_k, None, None, pos, None, c, s)
    assert e.shape[0] == 0


def test_axes_position_outside_the_table_is_recorded():
    n = 9
    k, qg, w_k, w_q, c, s = _axes_inputs(n, SEED + 4)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    bad = pos.clone()
    bad[2], bad[5] = -1, 4096
    fixed = pos.clone()
    fixed[2] = fixed[5] = 0
    got = B.ga_qk_prologue_axes(k, w_k, qg, w_q, bad, None, c, s)
    assert B.ga_device_status() == 4
    want = B.ga_qk_prologue_axes(k, w_k, qg, w_q, fixed, None, c, s)
    assert all(torch.equal(g, w) for g, w in zip(got, want)) and B.ga_device_status() == 0


# ------------------------------------------------------------------ the 4-bit rows
def _special_rows(n, seed):
    """Rows over many magnitudes with zeros, ties, tiny and saturating groups, inf and NaN."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, 2, 256)) * np.exp(rng.uniform(-12, 9, (n, 2, 1)))
    x[0, 0] = 0
    x[0, 1, :16] = np.arange(16) / 2 - 4          # scale boundaries and code ties
    if n > 3:
        x[1, 0, 5] = np.nan
        x[1, 1, 16:32] = np.nan
        x[2, 0, 3], x[2, 0, 4] = np.inf, -np.inf
        x[2, 1] = 1e-30
        x[3, 0] = 3e38
        x[3, 1] = rng.integers(-15, 16, 256) * 0.5
    return torch.tensor(x, dtype=torch.float32).to(torch.bfloat16).cuda()


def _expect_pool(pools, k, v, slots, page):
    """The pools (numpy) after storing the rows of non-negative slots."""
    out = [p.cpu().numpy().copy() for p in pools]
    for x, c, s in ((k, out[0], out[1]), (v, out[2], out[3])):
        codes, byte = O.quantize_q4_rows(np64(x))
        packed = O.pack_q4(codes)
        for t, slot in enumerate(slots):
            if slot >= 0:
                c[slot // page, :, slot % page] = packed[t]
                s[slot // page, :, slot % page] = byte[t]
    return out


@pytest.mark.parametrize("n,page,n_pages", [(1, 32, 1), (77, 96, 3), (500, 64, 9)])
def test_store_and_widen_match_oracle(n, page, n_pages):
    k = _special_rows(n, SEED + n)
    fused = torch.randn(n, 3, 2, 256, device="cuda").to(torch.bfloat16)
    v = fused[:, 1]                                # token stride 1536
    rng = np.random.default_rng(n)
    slots = rng.permutation(n_pages * page)[:n]
    if n > 5:
        slots[4], slots[n - 1] = -1, -7            # padding tokens: not stored
    pools = _pools(n_pages, page)
    want = _expect_pool(pools, k, v, slots, page)
    B.ga_kv_quantize_q4(k, v, *pools, slots=_i32(slots))
    for g, w in zip(pools, want):
        assert np.array_equal(g.cpu().numpy(), w)
    # widened at the same slots; padding rows are left as they were
    ko = torch.full((n, 2, 256), 3.0, dtype=torch.bfloat16, device="cuda")
    vo = torch.full_like(ko, 5.0)
    B.ga_kv_dequantize_q4(*pools, slots=_i32(slots), k_out=ko, v_out=vo)
    for x, o, rest in ((k, ko, 3.0), (v, vo, 5.0)):
        w = O.widen_q4_rows(*O.quantize_q4_rows(np64(x)))
        w[slots < 0] = rest
        assert np.array_equal(np64(o), w)


def test_store_without_slots_and_every_byte_widens():
    page, n_pages = 32, 4
    pools = _pools(n_pages, page)
    kw, vw = B.ga_kv_dequantize_q4(*pools)         # random bytes: the whole pool
    for c, s, o in ((pools[0], pools[1], kw), (pools[2], pools[3], vw)):
        cb = c.transpose(1, 2).reshape(-1, 2, 128).cpu().numpy().astype(np.int64)
        word = cb.reshape(-1, 2, 32, 4) @ np.array([1, 1 << 8, 1 << 16, 1 << 24])
        shift = np.array([0, 16, 4, 20, 8, 24, 12, 28])
        codes = ((word[..., None] >> shift) & 15).reshape(-1, 2, 256)
        sb = s.transpose(1, 2).reshape(-1, 2, 16).cpu().numpy()
        assert np.array_equal(np64(o), O.widen_q4_rows(codes, sb))
    other = _pools(n_pages, page, fill=0)
    B.ga_kv_quantize_q4(kw[:100], vw[:100], *other)
    want = _expect_pool(_pools(n_pages, page, fill=0), kw[:100], vw[:100], range(100), page)
    for g, w in zip(other, want):
        assert np.array_equal(g.cpu().numpy(), w)


def test_slots_outside_the_pool_are_recorded_and_skipped():
    pools = _pools(2, 32)
    before = [p.clone() for p in pools]
    x = torch.randn(3, 2, 256, device="cuda").to(torch.bfloat16)
    B.ga_kv_quantize_q4(x, x, *pools, slots=_i32([64, 2 ** 31 - 1, -1]))
    assert B.ga_device_status() == 3
    assert all(torch.equal(a, b) for a, b in zip(pools, before))
    ko, vo = torch.ones_like(x), torch.ones_like(x)
    B.ga_kv_dequantize_q4(*pools, slots=_i32([64, 2 ** 31 - 1, -1]), k_out=ko, v_out=vo)
    assert B.ga_device_status() == 3 and bool((ko == 1).all()) and bool((vo == 1).all())


@pytest.mark.parametrize("n", [4095, 4096, 4999])
@pytest.mark.parametrize("offset", [0, 8])
def test_store_and_widen_many_tokens(n, offset):
    """Both splits of the work, and rows that begin 16 bytes past a 32-byte boundary."""
    page, n_pages = 96, 60
    flat = torch.zeros(n * 2 * 512 + 8, dtype=torch.bfloat16, device="cuda")
    k = flat[offset:offset + n * 1024].view(n, 2, 2, 256)[:, 0]
    v = flat[offset:offset + n * 1024].view(n, 2, 2, 256)[:, 1]
    k.copy_(_special_rows(n, SEED + n))
    v.copy_(_special_rows(n, SEED + n + 1))
    rng = np.random.default_rng(n)
    slots = rng.permutation(n_pages * page)[:n]
    slots[rng.integers(0, n, 300)] = -1
    pools = _pools(n_pages, page)
    want = _expect_pool(pools, k, v, slots, page)
    B.ga_kv_quantize_q4(k, v, *pools, slots=_i32(slots))
    for g, w in zip(pools, want):
        assert np.array_equal(g.cpu().numpy(), w)
    out = torch.full((2 * n * 512 + 16,), 3.0, dtype=torch.bfloat16, device="cuda")
    ko, vo = (out[offset + i * n * 512:][:n * 512].view(n, 2, 256) for i in (0, 1))
    B.ga_kv_dequantize_q4(*pools, slots=_i32(slots), k_out=ko, v_out=vo)
    for x, o in ((k, ko), (v, vo)):
        w = O.widen_q4_rows(*O.quantize_q4_rows(np64(x)))
        w[slots < 0] = 3.0
        assert np.array_equal(np64(o), w)
    rest = torch.cat((out[:offset], out[offset + 2 * n * 512:]))
    assert bool((rest == 3).all())


def test_store_rows_of_an_odd_stride():
    """Token strides that are multiples of 16 bytes only."""
    n = 70
    k = torch.randn(n, 520, device="cuda").to(torch.bfloat16)[:, :512].unflatten(1, (2, 256))
    v = torch.randn(n, 776, device="cuda").to(torch.bfloat16)[:, 256:768].unflatten(1, (2, 256))
    pools = _pools(3, 32)
    want = _expect_pool(pools, k, v, range(n), 32)
    B.ga_kv_quantize_q4(k, v, *pools)
    for g, w in zip(pools, want):
        assert np.array_equal(g.cpu().numpy(), w)


# ------------------------------------------------------------------ attention
# The tolerance, per element, from the roundings: each weight is rounded to bf16 (at most 2^-8
# of itself) above and below the quotient, so 2 x 2^-8 of sum w |v| times the gate; the output
# is rounded once (2^-8 of itself). A score's fp32 error is at most 32 roundings (16 tensor-core
# steps, two each) of 2^-24 x sum |q k| / 16, under 1.6e-4 for the largest sums here (about 82);
# the exponent's own roundings, exp2 and the sigmoid add under 3e-5; over and under the quotient
# that makes 3.8e-4 < 2^-11 of the same sum, and 2^-10 leaves as much for the sums of P V.
def _check(got, want, mass, seq_len=None):
    g = np64(got).reshape(want.shape)
    tol = (2.0 ** -7 + 2.0 ** -10) * mass + 2.0 ** -8 * np.abs(want) + 1e-30
    live = np.ones(len(want), bool) if seq_len is None else np.asarray(seq_len) >= 0
    bad = ~(np.abs(g - want) <= tol)[live]
    assert not bad.any(), (int(bad.sum()), float(np.nanmax((np.abs(g - want) / tol)[live])))


class Cache:
    """Sequences over random 4-bit pools: pages in random order, unread table entries -1."""

    def __init__(self, lens, rows, page, seed, sigma=1.0, q_sigma=1.0):
        torch.manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.lens, self.rows, self.page = lens, rows, page
        need = [max(0, -(-(L + rows) // page)) if L >= 0 else 0 for L in lens]
        n_pages = sum(need) + 2
        self.pools = _pools(n_pages, page)
        x = (torch.randn(n_pages * page, 2, 2, 256, device="cuda") * sigma).to(torch.bfloat16)
        B.ga_kv_quantize_q4(x[:, 0], x[:, 1], *self.pools)
        self.kw, self.vw = B.ga_kv_dequantize_q4(*self.pools)
        perm = rng.permutation(n_pages)
        self.table = np.full((len(lens), max(max(need), 1)), -1)
        i = 0
        for b, m in enumerate(need):
            self.table[b, :m] = perm[i:i + m]
            i += m
        n = len(lens)
        self.q = (torch.randn(n, rows, 24, 256, device="cuda") * q_sigma).to(torch.bfloat16)
        self.qg = torch.randn(n, rows, 24, 512, device="cuda").to(torch.bfloat16)

    def run(self, **kw):
        return B.ga_attn_verify_q4(self.q, self.qg, *self.pools, _i32(self.table), _i32(self.lens),
                                   **kw)

    def oracle(self, heads=None):
        ks, vs = [], []
        kw, vw = np64(self.kw), np64(self.vw)
        for b, L in enumerate(self.lens):
            t = np.arange(max(L + self.rows, 0))
            at = self.table[b, t // self.page] * self.page + t % self.page
            ks.append(kw[at])
            vs.append(vw[at])
        return O.verify_q4(np64(self.q), np64(self.qg)[..., 256:], ks, vs, self.lens, heads)

    def check(self, **kw):
        _check(self.run(**kw), *self.oracle(), seq_len=self.lens)


@pytest.mark.parametrize("rows", [1, 2, 3, 5, 8, 10, 11, 13, 16])
@pytest.mark.parametrize("lens,page", [
    ([0], 32), ([1, 300], 96), ([127, 128, 129, 0, 31, 112], 128), ([-1, 700, -1, 63, 2], 64)])
def test_attention_matches_oracle(rows, lens, page):
    Cache(lens, rows, page, SEED + rows).check()


@pytest.mark.parametrize("rows,lens,page", [
    (1, [40000], 128), (16, [9000, 100], 64), (4, [5, 12345, 6000, 777], 32), (1, [3000] * 30, 256)])
def test_attention_cut_across_ctas(rows, lens, page):
    """Long streams cut into many parts, and CTAs that end one stream and begin others."""
    Cache(lens, rows, page, SEED + 50 + rows).check()


@pytest.mark.parametrize("rows", [1, 6, 16])
def test_attention_with_peaked_scores(rows):
    """Scores of magnitude 60: maxima that grow from tile to tile by more than the lazy rescale
    lets pass, rows dominated by one key, and parts whose weight vanishes in the merge."""
    Cache([2500, 130], rows, 64, SEED + 60, q_sigma=8.0).check()


def test_attention_growing_scores():
    """One query aligned with keys whose magnitude grows along the cache: the running maximum
    grows in every tile."""
    c = Cache([1500], 1, 32, SEED + 61)
    n = c.kw.shape[0]
    k = torch.ones(n, 2, 256, device="cuda")
    order = torch.empty(n, device="cuda")
    t = np.arange(1501)
    at = c.table[0, t // 32] * 32 + t % 32
    order[torch.tensor(at, device="cuda")] = torch.tensor(t / 1500, device="cuda", dtype=torch.float32)
    k = (k * order[:, None, None] * 4).nan_to_num(0).to(torch.bfloat16)
    B.ga_kv_quantize_q4(k, c.vw, *c.pools)
    c.kw, c.vw = B.ga_kv_dequantize_q4(*c.pools)
    c.q = torch.ones_like(c.q)
    c.check()


def test_attention_many_sequences():
    """More sequences than one launch takes, most of one tile, some unused."""
    rng = np.random.default_rng(7)
    lens = rng.integers(0, 90, 1100)
    lens[rng.integers(0, 1100, 100)] = -1
    c = Cache(list(map(int, lens)), 1, 32, SEED + 70)
    out = torch.full((1100, 1, 24 * 256), 7.0, dtype=torch.bfloat16, device="cuda")
    c.run(out=out)
    assert bool((out[torch.tensor(lens < 0)] == 7).all())       # unused rows left as they were
    want, mass = c.oracle(heads=[0, 11, 12, 23])
    hs = [0, 11, 12, 23]
    _check(out.view(1100, 1, 24, 256)[:, :, hs], want[:, :, hs], mass[:, :, hs], lens)


@pytest.mark.parametrize("rows,lens,page", [
    (8, [12000], 64), (2, [20000, 15], 128),             # more parts than the direct merge takes
    (2, [700] * 90 + [3000] * 3, 64), (1, [40, 6000] + [50] * 80, 32),   # cut among many
    (9, [300] * 40 + [5000], 32), (16, [130] * 60, 96)])
def test_attention_merges_parts(rows, lens, page):
    """Every form of the merge: many parts of one stream, and few parts among many streams."""
    rng = np.random.default_rng(rows + len(lens))
    heads = sorted(map(int, rng.choice(24, 4, replace=False)))
    c = Cache(lens, rows, page, SEED + 80 + rows)
    want, mass = c.oracle(heads=heads)
    got = c.run().view(len(lens), rows, 24, 256)
    _check(got[:, :, heads], want[:, :, heads], mass[:, :, heads])


def test_attention_long_and_short_beyond_one_launch():
    """More sequences than one launch takes, with long ones in each."""
    lens = [int(x) for x in np.random.default_rng(8).integers(0, 60, 300)]
    lens[17], lens[255], lens[256], lens[299] = 3000, 900, 2500, 1111
    c = Cache(lens, 3, 32, SEED + 90)
    heads = [0, 11, 12, 23]
    want, mass = c.oracle(heads=heads)
    _check(c.run().view(300, 3, 24, 256)[:, :, heads], want[:, :, heads], mass[:, :, heads])


@pytest.mark.parametrize("rows", [1, 3, 16])
def test_attention_nan_stays_in_its_row(rows):
    """A NaN or infinite query makes its own head's row NaN and no other element."""
    c = Cache([3000, 40], rows, 32, SEED + 91)
    good = c.run().view(2, rows, 24, 256)
    c.q[0, rows // 2, 5, 77] = float("nan")
    c.q[1, 0, 20, 200] = float("inf")
    c.q[1, rows - 1, 2] = -float("inf")            # every score NaN or infinite
    got = c.run().view(2, rows, 24, 256)
    hit = torch.zeros(2, rows, 24, dtype=torch.bool, device="cuda")
    hit[0, rows // 2, 5] = hit[1, 0, 20] = hit[1, rows - 1, 2] = True
    assert bool(got[hit].isnan().all())
    assert torch.equal(got[~hit], good[~hit])


def test_attention_gates_at_their_limits():
    c = Cache([50, 400], 3, 32, SEED + 71)
    g = c.qg.view(2, 3, 24, 2, 256)[..., 1, :]
    g[0] = -200.0
    g[1, 0] = 200.0
    g[1, 1] = 0.0
    c.check()
    assert bool((c.run()[0] == 0).all())


def test_attention_all_unused_or_empty():
    c = Cache([-1, -5], 2, 32, SEED + 72)
    out = torch.full((2, 2, 6144), 3.0, dtype=torch.bfloat16, device="cuda")
    c.run(out=out)
    assert bool((out == 3).all())
    e = B.ga_attn_verify_q4(c.q[:0], c.qg[:0], *c.pools, _i32(c.table)[:0], _i32([]))
    assert e.shape == (0, 2, 6144)


def test_attention_bad_pages_and_lengths_are_recorded():
    for rows in (1, 4):
        c = Cache([200, 300], rows, 32, SEED + 73)
        good = c.run()
        c.table[0, 3] = 10 ** 6
        c.table[0, 4] = -2
        out = c.run()
        assert B.ga_device_status() == 3
        assert torch.equal(out[1], good[1])             # the other sequence is whole
        c = Cache([200, 300], rows, 32, SEED + 73)
        lens = _i32([c.table.shape[1] * 32 - rows + 1, 300])
        out = torch.full_like(good, 9.0)
        B.ga_attn_verify_q4(c.q, c.qg, *c.pools, _i32(c.table), lens, out=out)
        assert B.ga_device_status() == 4
        assert bool((out[0] == 9).all())
        c.lens = [-1, 300]                              # cut as if sequence 0 were unused
        _check(out, *c.oracle(), seq_len=c.lens)


def test_attention_repeats_bit_for_bit_and_on_another_stream():
    c = Cache([4000, 17, 2222], 7, 64, SEED + 74)
    a = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = c.run()
    s.synchronize()
    assert torch.equal(a, b)
    # a workspace with other contents, and shared pages: two sequences over the same prefix
    ws = torch.full((B.ga_verify_q4_workspace_bytes(),), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(a, c.run(workspace=ws))
    c.table[2, :30] = c.table[0, :30]
    c.check()


@pytest.mark.parametrize("rows", [1, 5])
def test_attention_calls_at_once(rows):
    """Calls on two streams that may run together, each with a workspace of its own, beside a call
    of the other kernel form."""
    a, b = Cache([5000, 30], rows, 32, SEED + 92), Cache([70, 900, 4000], 6 - rows, 64, SEED + 93)
    want = a.run(), b.run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, (c, s) in enumerate(zip((a, b), streams)):
            with torch.cuda.stream(s):
                got[i].append(c.run())
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


@pytest.mark.parametrize("rows", [1, 5, 16])
@pytest.mark.parametrize("graph", [False, True])
def test_attention_calls_in_a_row_see_fresh_data(rows, graph):
    """Calls whose blocks are placed while the kernel before them ends: of two batches in turn over
    one workspace, and with queries, rows, pages and lengths written just before each call."""
    a, b = Cache([9000, 30], rows, 32, SEED + 94), Cache([7000, 900, 4000], rows, 64, SEED + 95)
    want = [a.run(), b.run()]
    ws = torch.empty(B.ga_verify_q4_workspace_bytes(), dtype=torch.uint8, device="cuda")
    got = [[torch.empty_like(w) for w in want] for _ in range(6)]
    live = []
    for c in (a, b):
        bufs = [c.q, c.qg, *c.pools, _i32(c.table), _i32(c.lens)]
        empty = [torch.zeros_like(x) for x in bufs]
        empty[-1].fill_(5)
        live.append((bufs, empty, [torch.empty_like(x) for x in bufs]))

    def body():
        for k in range(6):
            for i, (bufs, empty, use) in enumerate(live):
                if k % 2:           # other contents first, then the call's own
                    for src in (empty, bufs):
                        for to, x in zip(use, src):
                            to.copy_(x)
                        B.ga_attn_verify_q4(*use, out=got[k][i], workspace=ws)
                else:
                    B.ga_attn_verify_q4(*bufs, out=got[k][i], workspace=ws)

    body()
    if graph:
        torch.cuda.synchronize()
        for pair in got:
            for x in pair:
                x.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            body()
        for _ in range(3):
            g.replay()
    torch.cuda.synchronize()
    for pair in got:
        for x, w in zip(pair, want):
            assert torch.equal(x, w)


@pytest.mark.parametrize("rows", [1, 4])
def test_captured_step_follows_its_lengths(rows):
    """One captured graph, replayed as the device lengths change."""
    c = Cache([900, 500, 1200], rows, 64, SEED + 75)
    lens = _i32(c.lens)
    table, ws = _i32(c.table), torch.empty(B.ga_verify_q4_workspace_bytes(), dtype=torch.uint8,
                                           device="cuda")
    out = torch.empty(3, rows, 6144, dtype=torch.bfloat16, device="cuda")
    call = lambda: B.ga_attn_verify_q4(c.q, c.qg, *c.pools, table, lens, out=out,  # noqa: E731
                                       workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for new in ([900, 500, 1200], [3, 0, 1100], [-1, 128, 640]):
        c.lens = new
        lens.copy_(_i32(new))
        g.replay()
        torch.cuda.synchronize()
        _check(out, *c.oracle(), seq_len=new)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("graph", [False, True])
def test_server_steps(graph):
    """Prompts, then decode and verify steps with rejected tokens, a finished sequence and a new
    one in its row: plan, prologue, store, attention, all lengths on the device; each step's
    output against the oracle's attention over the widened rows it should see."""
    n, page, width, rows = 3, 32, 8, 2
    pool = 20
    pools = _pools(pool, page)
    torch.manual_seed(SEED)
    rng = np.random.default_rng(SEED)
    w_k = synth.normal_bf16(SEED, "w_k", (256,), sigma=0.1).cuda()
    w_q = synth.normal_bf16(SEED, "w_q", (256,), sigma=0.1).cuda()
    c, s = (t.cuda() for t in B.ga_rope_table_host(512))
    cos, sin = O.rope_tables(512)
    table, held = _i32(np.full((n, width), -1)), _i32([0] * n)
    free, count = _i32(rng.permutation(pool)), _i32([pool])
    seq_len, new_len = _i32([0] * n), _i32([0] * n)
    model = [dict(k=np.zeros((0, 2, 256)), v=np.zeros((0, 2, 256))) for _ in range(n)]

    def place(new, max_tokens, k, v):
        """Plans and stores the step's packed tokens; their expected rows go to `model`."""
        start, slots, pos, info = B.ga_page_plan(seq_len, new_len, table, held, free, count, page,
                                                 max_tokens)
        kp, _ = B.ga_qk_prologue_axes(k, w_k, None, None, pos, None, c, s)
        B.ga_kv_quantize_q4(kp, v, *pools, slots=slots)
        return info

    def expect(lens, new, k, v):
        t = 0
        for b in range(n):
            if new[b] < 0:
                model[b] = dict(k=np.zeros((0, 2, 256)), v=np.zeros((0, 2, 256)))
                continue
            for i in range(new[b]):
                kp = O.prep_axes(np64(k[t:t + 1]), np64(w_k), cos, sin, [[lens[b] + i]], [0] * 32)
                for key, x in (("k", kp), ("v", np64(v[t:t + 1]))):
                    m = O.widen_q4_rows(*O.quantize_q4_rows(x))
                    model[b][key] = np.concatenate([model[b][key][:lens[b] + i], m])
                t += 1

    # prompts of 40, 7 and 100 tokens
    lens, prompt = [0, 0, 0], [40, 7, 100]
    k = torch.randn(150, 2, 256, device="cuda").to(torch.bfloat16)
    v = torch.randn(150, 2, 256, device="cuda").to(torch.bfloat16)
    new_len.copy_(_i32(prompt))
    info = place(prompt, 150, k, v)
    assert info.tolist() == [0, 147, 2 + 1 + 4, 0]
    expect(lens, prompt, k, v)
    lens = list(prompt)

    # windows of `rows` tokens, captured once; one token of each window may be rejected
    T = n * rows
    kb = torch.empty(T, 2, 256, dtype=torch.bfloat16, device="cuda")
    vb, qg = torch.empty_like(kb), torch.empty(T, 24, 512, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(n, rows, 6144, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(B.ga_verify_q4_workspace_bytes(), dtype=torch.uint8, device="cuda")

    def step():
        start, slots, pos, info = B.ga_page_plan(seq_len, new_len, table, held, free, count, page, T)
        kp, qp = B.ga_qk_prologue_axes(kb, w_k, qg, w_q, pos, None, c, s)
        B.ga_kv_quantize_q4(kp, vb, *pools, slots=slots)
        B.ga_attn_verify_q4(qp.view(n, rows, 24, 256), qg.view(n, rows, 24, 512), *pools, table,
                            seq_len, out=out, workspace=ws)
        return info

    if graph:   # captured with nothing to do: no sequence is planned, so no state changes
        seq_len.copy_(_i32([-1] * n))
        new_len.copy_(_i32([0] * n))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
    for i in range(14):
        kb.copy_(torch.randn(T, 2, 256, device="cuda"))
        vb.copy_(torch.randn(T, 2, 256, device="cuda"))
        qg.copy_(torch.randn(T, 24, 512, device="cuda"))
        seq_len.copy_(_i32(lens))
        new_len.copy_(_i32([rows] * n))
        g.replay() if graph else step()
        torch.cuda.synchronize()
        expect(lens, [rows] * n, kb, vb)
        pos = [[lens[b] + r for b in range(n) for r in range(rows)]]
        q = O.prep_axes(np64(qg)[..., :256], np64(w_q), cos, sin, pos, [0] * 32)
        want = O.verify_q4(q.reshape(n, rows, 24, 256), np64(qg)[..., 256:].reshape(n, rows, 24, 256),
                           [m["k"] for m in model], [m["v"] for m in model], lens)
        _check(out, *want)
        lens = [x + int(rng.integers(1, rows + 1)) for x in lens]
        if i == 6:      # sequence 2 ends, and another starts in its row
            pages = int(held[2].item())
            seq_len.copy_(_i32(lens))
            new_len.copy_(_i32([0, 0, -1]))
            info = B.ga_page_plan(seq_len, new_len, table, held, free, count, page, 0)[3]
            assert info.tolist() == [0, 0, 0, pages]
            lens[2] = 0
            model[2] = dict(k=np.zeros((0, 2, 256)), v=np.zeros((0, 2, 256)))
    used = int(held.sum().item())
    assert int(count.item()) == pool - used
    left = free[:pool - used].tolist() + [int(table[b, j]) for b in range(n)
                                          for j in range(int(held[b]))]
    assert sorted(left) == list(range(pool))       # every page is somewhere, once


def test_widened_prefix_serves_a_prefill():
    """A prefix of a 4-bit cache widened for the bf16 prefill of the next chunk."""
    T, base = 200, 64
    torch.manual_seed(SEED)
    pools = _pools(9, 32)
    slots = _i32(np.random.default_rng(3).permutation(9 * 32)[:T])
    k = torch.randn(T, 2, 256, device="cuda").to(torch.bfloat16)
    v = torch.randn(T, 2, 256, device="cuda").to(torch.bfloat16)
    B.ga_kv_quantize_q4(k, v, *pools, slots=slots)
    kw, vw = B.ga_kv_dequantize_q4(*pools, slots=slots)
    qg = synth.normal_bf16(SEED, "qg", (T - base, 24, 512)).cuda()
    w_q = synth.normal_bf16(SEED, "w_q", (256,), sigma=0.1).cuda()
    c, s = (t.cuda() for t in B.ga_rope_table_host(T))
    out = B.ga_attn_prefill(qg, kw, vw, w_q, c, s, q_base=base, T=T)
    codes = [O.widen_q4_rows(*O.quantize_q4_rows(np64(x))) for x in (k, v)]
    assert np.array_equal(np64(kw), codes[0]) and np.array_equal(np64(vw), codes[1])
    ref = B.ga_attn_prefill(qg, torch.tensor(codes[0], device="cuda").to(torch.bfloat16),
                            torch.tensor(codes[1], device="cuda").to(torch.bfloat16), w_q, c, s,
                            q_base=base, T=T)
    assert torch.equal(out, ref)


def test_calls_refuse_tensors_that_do_not_belong():
    c = Cache([100], 2, 32, SEED + 80)
    kc, ks, vc, vs = c.pools
    t, l = _i32(c.table), _i32(c.lens)
    with pytest.raises(ValueError):
        B.ga_attn_verify_q4(c.q, c.qg, kc, vs[:-1], vc, vs, t, l)
    with pytest.raises(ValueError):
        B.ga_attn_verify_q4(c.q, c.qg, kc, ks, vc, vs, t, l.long())
    with pytest.raises(ValueError):
        B.ga_attn_verify_q4(c.q, c.qg[:, :1], kc, ks, vc, vs, t, l)
    with pytest.raises(ValueError):
        B.ga_attn_verify_q4(c.q.transpose(1, 2), c.qg, kc, ks, vc, vs, t, l)
    with pytest.raises(ValueError):
        B.ga_attn_verify_q4(c.q.cpu(), c.qg, kc, ks, vc, vs, t, l)
    with pytest.raises(ValueError):
        B.ga_kv_quantize_q4(c.kw[..., ::2], c.vw, kc, ks, vc, vs)
    with pytest.raises(ValueError):
        B.ga_kv_quantize_q4(c.kw[:8], c.vw[:8], kc, ks, vc, vs, slots=l)
    with pytest.raises(ValueError):
        B.ga_kv_dequantize_q4(kc, ks, vc, vs, slots=l, n_tok=5)
    with pytest.raises(B.GaError):
        B.ga_attn_verify_q4(c.q, c.qg, kc, ks, vc, vs, t, l, workspace=torch.empty(
            64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        B.ga_page_plan(l, l, t, l, t[0], l, 32, 4, pos_delta=t)
