"""The attention over 8-bit caches with scores of any magnitude up to 2^29. Where one key outweighs the
others by far, the output is its value times the gate, whatever its score: the score's own error
reaches the weight and the sum alike."""
import numpy as np
import pytest
import torch

from tests.parity import SEED, np64
from tests.q8_bounds import allowed
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


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def scored_case(g, n, length, rows, power, sign, top):
    """n sequences of `length` cached tokens whose keys `top` [n, m] all have the same largest score with a
    query: sign times 2^power or down to a third of it, with another fraction for every query row. The
    other keys' scores are an eighth of it at most, or (sign < 0) 1.3 to 2.9 times it. Pages of 64 tokens."""
    page, keys = 64, length + rows
    per = -(-keys // page)
    table = torch.randperm(n * per, generator=g, device="cuda").to(torch.int32).view(n, per)
    pools = [torch.full((n * per, 2) + s, 0x7F, dtype=torch.uint8, device="cuda")
             for s in ((page, 256), (page // 32,)) * 2]
    # 256 products of 2^(power - 5) (0.7 .. 1.25) (1 .. 17/16) by 1 .. 1.5, over 16
    q = 2.0 ** (power - 5) * (0.7 + 0.55 * _uniform(g, n, rows, 24, 1)) * (1 + _uniform(g, n, rows, 24, 256) / 16)
    k = 1 + 0.5 * _uniform(g, n, keys, 2, 256)
    far = 2.0 ** -4 if sign > 0 else 2.0
    is_top = torch.zeros(n, keys, dtype=torch.bool, device="cuda").scatter_(1, top, True)
    k = torch.where(is_top[:, :, None, None], k[:, :1], far * k)
    q, k = q.to(torch.bfloat16), (sign * k).to(torch.bfloat16)
    v, qg = _normal(g, n, keys, 2, 256), _normal(g, n, rows, 24, 512)
    t = torch.arange(keys, device="cuda")
    slots = (table.long()[:, t // page] * page + t % page).to(torch.int32)
    B.ga_kv_quantize_q8(k.flatten(0, 1), v.flatten(0, 1), *pools, slots=slots.flatten())
    return pools, table, q, qg, slots


def check_top_values(out, pools, qg, slots, top, rows, only=None):
    """The mean of the top keys' values, times the gate. Equal scores have equal weights, each off by
    2^-9 at most (`mass` is the mean of their values' magnitudes), and no other key has any."""
    n = len(top)
    out, gate = np64(out).reshape(n, rows, 24, 256), 1 / (1 + np.exp(-np64(qg)[..., 256:]))
    for b in only or range(n):
        kw, vw = (np64(x) for x in B.ga_kv_dequantize_q8(*pools, slots=slots[b][top[b]]))
        assert (kw == kw[:1]).all()
        for kv in range(2):
            hs = slice(12 * kv, 12 * kv + 12)
            want, mass = gate[b, :, hs] * vw[:, kv].mean(0), gate[b, :, hs] * np.abs(vw[:, kv]).mean(0)
            bad = np.abs(out[b, :, hs] - want) > allowed(want, mass, 0.0, mass)
            assert not bad.any(), (b, kv, int(bad.sum()))


# the other keys of negative ones are up to 2.9 times as far
POWERS = [(p, s) for p in (8, 16, 20, 21, 22, 23, 24, 25, 26, 27, 28, 29) for s in (1, -1) if s > 0 or p < 28]


@pytest.mark.parametrize("power,sign", POWERS)
@pytest.mark.parametrize("rows", [1, 2, 4, 5, 9, 16])
def test_one_key_far_above_the_rest(rows, power, sign):
    g = _gen(100 * rows + power + 50 * sign)
    top = torch.tensor([[3], [40], [70], [31], [0]], device="cuda")
    pools, table, q, qg, slots = scored_case(g, 5, 100, rows, power, sign, top)
    out = B.ga_attn_verify_q8(q, qg, *pools, table, _i32([100] * 5))
    check_top_values(out, pools, qg, slots, top, rows)


@pytest.mark.parametrize("power", [12, 23, 25, 27, 29])
@pytest.mark.parametrize("rows", [1, 3, 8, 16])
def test_equal_scores_far_above_the_rest(rows, power):
    """Two keys of one block and one of another, alike."""
    g = _gen(1000 * rows + power)
    top = torch.tensor([[3, 30, 70], [33, 95, 64], [90, 65, 0]], device="cuda")
    for sign in (1, -1) if power < 28 else (1,):
        pools, table, q, qg, slots = scored_case(g, 3, 100, rows, power, sign, top)
        out = B.ga_attn_verify_q8(q, qg, *pools, table, _i32([100] * 3))
        check_top_values(out, pools, qg, slots, top, rows)


@pytest.mark.parametrize("power", [4, 20, 25, 29])
def test_a_sequence_of_one_key(power):
    g = _gen(power)
    top = torch.zeros(9, 1, dtype=torch.long, device="cuda")
    for sign in (1, -1):
        pools, table, q, qg, slots = scored_case(g, 9, 0, 1, power, sign, top)
        check_top_values(B.ga_attn_verify_q8(q, qg, *pools, table, _i32([0] * 9)), pools, qg, slots, top, 1)


@pytest.mark.parametrize("power", [12, 21, 23, 25, 27, 29])
@pytest.mark.parametrize("rows", [1, 4, 5, 16])
def test_far_scores_in_long_streams(rows, power):
    """Streams cut into parts, whose references are far apart, and whole ones, whose reference moves when
    the largest score comes by: at the stream's beginning, inside, and in its last whole block."""
    g = _gen(7000 + 100 * rows + power)
    for n, length in ((3, 9000), (160, 1250)):
        top = torch.tensor([[0], [length // 2], [length - 1]], device="cuda").repeat(-(-n // 3), 1)[:n]
        for sign in (1, -1) if power < 28 else (1,):
            pools, table, q, qg, slots = scored_case(g, n, length, rows, power, sign, top)
            out = B.ga_attn_verify_q8(q, qg, *pools, table, _i32([length] * n))
            check_top_values(out, pools, qg, slots, top, rows, None if n == 3 else (0, 1, 2, 76, 77, 78, 157, 158, 159))
