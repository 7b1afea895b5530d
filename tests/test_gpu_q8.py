"""GPU parity of the 8-bit paged cache against the float64 oracle: stored rows code for code over
any number of calls, widened rows value for value, attention within the error of its roundings."""
import numpy as np
import pytest
import torch

from oracle import ga_oracle as O
from tests.parity import SEED, np64
from tests.q4_bounds import attend64, row_errors
from tests.q8_bounds import ROW_BOUND, allowed, rest_of, score_error
from verify_gated_gqa_gb300 import binding as B
from verify_gated_gqa_gb300 import build as build_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_mod.build()
    B.lib()
    yield
    assert B.ga_device_status() == 0


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(SEED + seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def _pools(n_pages, page, code=0x7F, scale=0xFF):
    """Pools of one byte throughout: by default NaN codes and the largest scale byte."""
    make = lambda fill, *s: torch.full((n_pages, 2) + s, fill, dtype=torch.uint8, device="cuda")  # noqa: E731
    return make(code, page, 256), make(scale, page // 32), make(code, page, 256), make(scale, page // 32)


def _flat(codes, scales):
    """Pools as [head][slot] codes and [head][block] scale bytes."""
    return (codes.transpose(0, 1).flatten(1, 2).cpu().numpy(), scales.transpose(0, 1).flatten(1).cpu().numpy())


class Model:
    """The oracle's cache: values and exponents by (K or V, head)."""

    def __init__(self, n_pages, page):
        n = n_pages * page
        self.values = [[np.zeros((n, 256)) for _ in range(2)] for _ in range(2)]
        self.exps = [[np.full(n // 32, 31) for _ in range(2)] for _ in range(2)]
        self.known = np.zeros(n, bool)

    def store(self, k, v, slots):
        slots = np.asarray(slots)
        anew = {int(s) // 32 for s in slots if s >= 0 and s % 32 == 0}
        for b in anew:
            self.known[32 * b:32 * b + 32] = False
        for i, x in enumerate((np64(k), np64(v))):
            for h in range(2):
                O.q8_store(self.values[i][h], self.exps[i][h], x[:, h], slots)
        self.known[slots[slots >= 0]] = True

    def check(self, pools):
        for i in range(2):
            codes, scales = _flat(pools[2 * i], pools[2 * i + 1])
            for h in range(2):
                at = np.nonzero(self.known)[0]
                assert np.array_equal(codes[h][at], O.e4m3_codes(self.values[i][h][at]))
                b = np.unique(at // 32)
                assert np.array_equal(scales[h][b], self.exps[i][h][b] + 32)


# ------------------------------------------------------------------ storing
@pytest.mark.parametrize("n_seq,page,steps", [
    (1, 32, [1] * 40), (1, 64, [77, 1, 1, 5]), (3, 96, [200, 16, 3]), (64, 64, [20, 1, 1, 1]),
    (5, 32, [1000, 7]), (2, 128, [4097]), (40, 32, [31, 2, 33, 1])])
def test_store_matches_oracle_over_calls(n_seq, page, steps):
    """Sequences fill their pages in several calls; magnitudes grow and shrink from token to token, so
    blocks grow after they hold rows."""
    rng = np.random.default_rng(SEED + n_seq + page)
    g = _gen(page)
    per = -(-sum(steps) // page)
    n_pages = n_seq * per + 1
    table = rng.permutation(n_pages)[:n_seq * per].reshape(n_seq, per)
    pools, m, at = _pools(n_pages, page), Model(n_pages, page), 0
    for step in steps:
        # sequences add up to `step` tokens each, packed; a few skipped tokens between them
        slots = []
        for b in range(n_seq):
            p = at + np.arange(step)
            slots += list(table[b][p // page] * page + p % page)
            if b % 3 == 1:
                slots += [-1]
        n = len(slots)
        kv = _normal(g, n, 2, 2, 256)
        kv *= torch.exp2(torch.randint(-9, 10, (n, 2, 2, 1), generator=g, device="cuda").float()).to(torch.bfloat16)
        k, v = kv[:, 0].contiguous(), kv[:, 1]
        B.ga_kv_quantize_q8(k, v, *pools, slots=_i32(slots))
        m.store(k, v, slots)
        at += step
        m.check(pools)
    # what no token was stored to holds what it held
    codes, _ = _flat(pools[0], pools[1])
    assert (codes[:, ~m.known] == 0x7F).all()
    known = np.nonzero(m.known)[0]
    kw, vw = B.ga_kv_dequantize_q8(*pools, slots=_i32(known))
    for i, w in enumerate((kw, vw)):
        for h in range(2):
            assert np.array_equal(np64(w[:, h]), O.q8_widen(m.values[i][h], m.exps[i][h], known))


@pytest.mark.parametrize("n", [1, 31, 32, 33, 64, 97, 4000])
def test_store_whole_pool_without_slots(n):
    g = _gen(n)
    n_pages = -(-n // 96)
    pools, m = _pools(n_pages, 96), Model(n_pages, 96)
    k, v = _normal(g, n, 2, 256), _normal(g, n, 2, 256)
    B.ga_kv_quantize_q8(k, v, *pools)
    m.store(k, v, np.arange(n))
    m.check(pools)
    kw, vw = B.ga_kv_dequantize_q8(*pools, n_tok=n)
    assert np.array_equal(np64(kw[:, 1]), O.q8_widen(m.values[0][1], m.exps[0][1], np.arange(n)))
    # nearest: half a step of the code's binade, or of the smallest step
    x, w = np64(v[:, 0]), np64(vw[:, 0])
    e = m.exps[1][0][np.arange(n) // 32][:, None]
    assert np.all(np.abs(w - x) <= np.maximum(2.0 ** -4 * np.abs(x), np.ldexp(2.0 ** -10, e)))


def test_store_special_values():
    """NaN, infinities, signed zeros, subnormals, values past both ends of the scales, a tie."""
    rows = torch.zeros(7, 2, 256)
    rows[0, 0, :4] = torch.tensor([float("nan"), 1.0, -0.0, -3.3e38])
    rows[1, 1, :3] = torch.tensor([float("inf"), float("-inf"), 1e30])
    rows[2, 0, :3] = torch.tensor([1e-40, -2.0 ** -42, 2.0 ** -41])
    rows[3, 1, :2] = torch.tensor([448.0, 17.0])
    rows[4, 0, :3] = torch.tensor([float("nan")] * 3)
    rows[5, 0, :2] = torch.tensor([450.0, -19.0])
    rows[6, 1, :3] = torch.tensor([448.0, 2.0 ** -10, 3 * 2.0 ** -10])
    x = rows.to(torch.bfloat16).cuda()
    for slots in (np.arange(7) * 32, np.arange(7) * 32 + 1, [1, 2, 3, 4, 5, 6, 7]):
        pools, m = _pools(8, 32, 0, 0), Model(8, 32)
        for a in range(2):
            for h in range(2):
                m.exps[a][h][:] = -32
        B.ga_kv_quantize_q8(x, -x, *pools, slots=_i32(slots))
        m.store(x, -x, slots)
        m.check(pools)


def test_every_bf16_value_and_every_code():
    """All 65,536 values of a type at every exponent that a block can be given."""
    bits = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    for e in range(-32, 32, 7):
        x = bits.view(256, 1, 256).repeat(1, 2, 1)
        top = 448.0 * 2.0 ** e
        small = torch.where(x.abs() <= top, x, torch.tensor(0.0, dtype=torch.bfloat16, device="cuda"))
        small[::32, :, 0] = top
        pools, m = _pools(4, 64), Model(4, 64)
        B.ga_kv_quantize_q8(small, small, *pools)
        m.store(small, small, np.arange(256))
        assert set(m.exps[0][0].tolist()) == {e}
        m.check(pools)
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(1, 1, 1, 256).repeat(8, 2, 32, 1)
    for byte in range(0, 256, 8):
        s = torch.arange(byte, byte + 8, dtype=torch.uint8, device="cuda").view(8, 1, 1).repeat(1, 2, 1)
        k, v = B.ga_kv_dequantize_q8(codes, s, codes, s)
        c = np.arange(256)
        val = np.where(((c >> 3) & 15) == 0, (c & 7) / 512, (1 + (c & 7) / 8) * 2.0 ** (((c >> 3) & 15) - 7.0))
        val = np.where(c >= 128, -val, val)
        val[[127, 255]] = np.nan
        for i in range(8):
            want = np.ldexp(val, ((byte + i) & 63) - 32)
            assert np.array_equal(np64(k[32 * i + 5, 1]), want, equal_nan=True)
            assert np.array_equal(np64(v[32 * i, 0]), want, equal_nan=True)


def test_store_and_widen_leave_other_rows_and_record_bad_slots():
    g = _gen(3)
    pools = _pools(3, 32, 5, 40)
    k = _normal(g, 4, 2, 256)
    B.ga_kv_quantize_q8(k, k, *pools, slots=_i32([96, -1, 40, 2 ** 31 - 1]))
    assert B.ga_device_status() == 3
    out = [torch.full((4, 2, 256), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    B.ga_kv_dequantize_q8(*pools, slots=_i32([40, 96, -7, 40]), k_out=out[0], v_out=out[1])
    assert B.ga_device_status() == 3
    assert torch.equal(out[0][0], out[0][3]) and bool((out[0][1:3] == 9).all())
    pools[0][1, :, 8] = 5                       # slot 40; its block's exponent may have grown
    assert bool((pools[0][0] == 5).all()) and bool((pools[0][2] == 5).all())


# ------------------------------------------------------------------ attention
def _case(g, lens, rows, page, extra=3, width=None, vary=0):
    """Shuffled pages of stored rows of cached and window tokens; everything else NaN codes."""
    need = [max(0, -(-(x + rows) // page)) if x >= 0 else 0 for x in lens]
    n_pages = sum(need) + extra
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), width or max(max(need), 1) + 1), 2 ** 30, dtype=torch.int32, device="cuda")
    pools = _pools(n_pages, page)
    i = 0
    for b, m in enumerate(need):
        table[b, :m] = perm[i:i + m]
        i += m
        if m == 0:
            continue
        t = torch.arange(lens[b] + rows, device="cuda")
        slots = table[b].long()[t // page] * page + t % page
        k, v = _normal(g, t.numel(), 2, 256), _normal(g, t.numel(), 2, 256)
        if vary:
            block = torch.randint(-vary, vary + 1, (t.numel() // 32 + 1, 1, 1), generator=g, device="cuda")
            v *= torch.exp2(block.float()).to(torch.bfloat16)[t // 32]
        B.ga_kv_quantize_q8(k, v, *pools, slots=slots.to(torch.int32))
    q, qg = _normal(g, len(lens), rows, 24, 256), _normal(g, len(lens), rows, 24, 512)
    return pools, table, q, qg


def _widened(pools, table, b, keys):
    page = pools[0].shape[2]
    t = torch.arange(keys, device="cuda")
    return B.ga_kv_dequantize_q8(*pools, slots=(table[b].long()[t // page] * page + t % page).to(torch.int32))


def _check(out, pools, table, q, qg, lens, only=None):
    rows = q.shape[1]
    for b, length in enumerate(lens):
        if length < 0 or (only is not None and b not in only):
            continue
        k, v = (np64(x) for x in _widened(pools, table, b, length + rows))
        want, mass = O.verify_q4(np64(q[b])[None], np64(qg[b])[None, ..., 256:], [k], [v], [length])
        x = max(score_error(np64(q[b]), k[:, h]) for h in range(2))
        rest = rest_of(np64(q[b]), np64(qg[b])[..., 256:], k, v, length)
        got = np64(out[b]).reshape(want[0].shape)
        assert np.all(np.abs(got - want[0]) <= allowed(want[0], mass[0], x, rest)), (b, length)


@pytest.mark.parametrize("rows", range(1, 17))
def test_attention_rows(rows):
    g = _gen(rows)
    lens = [0, 1, 33, 127, 128, 290, -1, 31 + rows]
    pools, table, q, qg = _case(g, lens, rows, 32 * (1 + rows % 4))
    out = torch.full((len(lens), rows, 6144), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((B.ga_verify_q8_workspace_bytes(),), 0xFF, dtype=torch.uint8, device="cuda")
    B.ga_attn_verify_q8(q, qg, *pools, table, _i32(lens), out=out, workspace=ws)
    assert bool((out[6] == 7).all())
    _check(out, pools, table, q, qg, lens)
    again = B.ga_attn_verify_q8(q, qg, *pools, table, _i32(lens), out=out.clone(), workspace=ws)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("rows", [1, 3, 8, 16])
@pytest.mark.parametrize("length", [0, 1, 30, 31, 32, 95, 96, 111, 112, 126, 127, 128, 129, 255, 500])
def test_attention_lengths(rows, length):
    g = _gen(1000 * rows + length)
    pools, table, q, qg = _case(g, [length], rows, 32)
    out = B.ga_attn_verify_q8(q, qg, *pools, table, _i32([length]))
    _check(out, pools, table, q, qg, [length])


@pytest.mark.parametrize("rows", [1, 5, 12])
def test_attention_value_scales_that_differ(rows):
    """Blocks of values 2^-12 to 2^12 apart: a weight counts by what it multiplies."""
    g = _gen(rows + 50)
    lens = [700, 40, 1300]
    pools, table, q, qg = _case(g, lens, rows, 64, vary=12)
    out = B.ga_attn_verify_q8(q, qg, *pools, table, _i32(lens))
    _check(out, pools, table, q, qg, lens)


@pytest.mark.parametrize("rows", [1, 4, 9])
@pytest.mark.parametrize("kind", ["rising", "falling", "sink", "equal"])
def test_attention_maxima(rows, kind):
    """Scores that grow from tile to tile, fall, have one key far above the rest (with no value of its
    own, so that the others make the output), or are all alike."""
    g = _gen(rows + 70)
    n, page = 900, 64
    pools, table, q, qg = _case(g, [n], rows, page)
    t = torch.arange(n + rows, device="cuda")
    slots = (table[0].long()[t // page] * page + t % page).to(torch.int32)
    k, v = _normal(g, n + rows, 2, 256), _normal(g, n + rows, 2, 256)
    u = _normal(g, 256).float()
    u /= u.norm()
    q[:] = (16 * u + 0.3 * q.float()).to(torch.bfloat16)   # q . (a u) / 16 is about a
    a = {"rising": t * 0.06, "falling": (n - t) * 0.06, "sink": torch.where(t == 5, 25.0, 0.0),
         "equal": t * 0.0}[kind]
    k = (0.2 * k.float() + a[:, None, None] * u).to(torch.bfloat16)
    if kind == "sink":
        k[t == 5] = (25 * u).to(torch.bfloat16)
        v[t == 5] = 0
    B.ga_kv_quantize_q8(k, v, *pools, slots=slots)
    out = B.ga_attn_verify_q8(q, qg, *pools, table, _i32([n]))
    _check(out, pools, table, q, qg, [n])


def test_a_nan_query_stays_in_its_row():
    g = _gen(90)
    lens = [300, 2000, 77]
    for rows in (1, 2, 9):
        pools, table, q, qg = _case(g, lens, rows, 32)
        want = B.ga_attn_verify_q8(q, qg, *pools, table, _i32(lens)).view(3, rows, 24, 256)
        bad = q.clone()
        bad[1, rows - 1, 7, 3] = float("nan")
        bad[2, 0, 20] = float("nan")
        bad[0, 0, 0, 0] = float("inf")
        got = B.ga_attn_verify_q8(bad, qg, *pools, table, _i32(lens)).view(3, rows, 24, 256)
        same = torch.ones(3, rows, 24, dtype=torch.bool, device="cuda")
        same[1, rows - 1, 7] = same[2, 0, 20] = same[0, 0, 0] = False
        assert torch.equal(got[same], want[same])
        assert bool(got[1, rows - 1, 7].isnan().all()) and bool(got[2, 0, 20].isnan().all())


def test_attention_bad_pages_and_lengths_are_recorded():
    g = _gen(91)
    lens = [400, 100, 90]
    pools, table, q, qg = _case(g, lens, 2, 64)
    good = B.ga_attn_verify_q8(q, qg, *pools, table, _i32(lens))
    bad = table.clone()
    bad[0, 2], bad[2, 0] = -1, 2 ** 31 - 1
    out = B.ga_attn_verify_q8(q, qg, *pools, bad, _i32(lens))
    assert B.ga_device_status() == 3
    assert torch.equal(out[1], good[1]) and not bool(out.isnan().any())
    out = torch.full_like(good, 7.0)
    B.ga_attn_verify_q8(q, qg, *pools, table, _i32([400, 64 * table.shape[1] - 1, 90]), out=out)
    assert B.ga_device_status() == 4
    assert bool((out[1] == 7).all())
    _check(out, pools, table, q, qg, lens, only=(0, 2))


@pytest.mark.parametrize("rows,lens,page", [
    (1, [65536], 128), (1, [40001, 5, 300, 9000], 32), (6, [12345, 0, 7777], 32), (16, [30000, 2048], 96),
    (8, [20000], 64), (2, [100] * 300, 32)])
def test_attention_long_rows(rows, lens, page):
    """Long streams, cut among the SMs: a row's 256 outputs together."""
    g = _gen(rows + len(lens))
    pools, table, q, qg = _case(g, lens, rows, page)
    out = B.ga_attn_verify_q8(q, qg, *pools, table, _i32(lens)).view(len(lens), rows, 24, 256)
    for b in range(0, len(lens), 1 if len(lens) < 9 else 37):
        k, v = _widened(pools, table, b, lens[b] + rows)
        for kv in range(2):
            hs = slice(12 * kv, 12 * kv + 12)
            want = attend64(q[b, :, hs], qg[b, :, hs, 256:], k[:, kv], v[:, kv],
                            [lens[b] + r + 1 for r in range(rows)])
            assert float(row_errors(out[b, :, hs], want).max()) <= (ROW_BOUND if lens[b] > 60 else 2 * ROW_BOUND)


def test_pools_past_4_gib():
    """Pages whose bytes lie past 32-bit offsets."""
    g = _gen(95)
    page, n_pages = 1024, 8300                       # 4.3e9 bytes of codes each
    pools = [torch.empty(n_pages, 2, page, 256, dtype=torch.uint8, device="cuda") if i % 2 == 0 else
             torch.empty(n_pages, 2, page // 32, dtype=torch.uint8, device="cuda") for i in range(4)]
    L, rows = 3000, 3
    table = _i32([[n_pages - 1, 0, n_pages - 2]])
    t = torch.arange(L + rows, device="cuda")
    slots = (table[0].long()[t // page] * page + t % page).to(torch.int32)
    k, v = _normal(g, L + rows, 2, 256), _normal(g, L + rows, 2, 256)
    B.ga_kv_quantize_q8(k, v, *pools, slots=slots)
    small = _pools(3, page)
    B.ga_kv_quantize_q8(k, v, *small)
    for x, y in zip(B.ga_kv_dequantize_q8(*pools, slots=slots), B.ga_kv_dequantize_q8(*small, n_tok=L + rows)):
        assert torch.equal(x, y)
    q, qg = _normal(g, 1, rows, 24, 256), _normal(g, 1, rows, 24, 512)
    out = B.ga_attn_verify_q8(q, qg, *pools, table, _i32([L]))
    assert torch.equal(out, B.ga_attn_verify_q8(q, qg, *small, _i32([[0, 1, 2]]), _i32([L])))


def test_empty_calls():
    pools = _pools(2, 32)
    e = torch.zeros(0, 2, 256, dtype=torch.bfloat16, device="cuda")
    B.ga_kv_quantize_q8(e, e, *pools, slots=_i32(np.zeros(0, np.int64)))
    k, v = B.ga_kv_dequantize_q8(*pools, n_tok=0)
    assert k.shape == v.shape == (0, 2, 256)
    q = torch.zeros(0, 3, 24, 256, dtype=torch.bfloat16, device="cuda")
    out = B.ga_attn_verify_q8(q, torch.zeros(0, 3, 24, 512, dtype=torch.bfloat16, device="cuda"), *pools,
                              torch.zeros(0, 2, dtype=torch.int32, device="cuda"), _i32(np.zeros(0, np.int64)))
    assert out.shape == (0, 3, 6144)
