"""The attention over long 4-bit caches, a row at a time: with tests/q4_bounds.py's bound a part of
a stream that is missing, or merged twice, shows in every row (tests/test_q4_bounds.py)."""
import numpy as np
import pytest
import torch

from tests.q4_bounds import ROW_BOUND, attend64, row_errors
from verify_gated_gqa_gb300 import binding as B
from verify_gated_gqa_gb300 import build as build_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_mod.build()
    B.lib()
    yield
    assert B.ga_device_status() == 0


@pytest.mark.parametrize("rows,lens,page", [
    (1, [40000], 128), (1, [65536, 31, -1, 12345], 64), (1, [3000] * 30, 256), (1, [8191] * 80, 32),
    (2, [20000, 15], 128), (4, [5, 12345, 6000, 777], 32), (6, [65000], 64),
    (8, [12000] + [200] * 63, 64), (9, [300] * 40 + [5000], 32), (16, [40000], 128),
    (16, [9000, 100, 30011], 64), (3, [50] * 250 + [20000] + [70] * 49, 32)])
def test_every_part_of_a_long_stream_counts_once(rows, lens, page):
    n = len(lens)
    seed = 5000 + rows + n
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    need = [-(-(L + rows) // page) if L >= 0 else 0 for L in lens]
    n_pages = sum(need) + 1
    perm = np.random.default_rng(seed).permutation(n_pages)
    table = np.full((n, max(need)), -1)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = perm[at:at + m]
        at += m
    pools = []
    for _ in range(2):
        pools += [torch.zeros(n_pages, 2, page, w, dtype=torch.uint8, device="cuda") for w in (128, 16)]
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    B.ga_kv_quantize_q4(normal(n_pages * page, 2, 256), normal(n_pages * page, 2, 256), *pools)
    kw, vw = B.ga_kv_dequantize_q4(*pools)
    q, qg = normal(n, rows, 24, 256), normal(n, rows, 24, 512)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    out = B.ga_attn_verify_q4(q, qg, *pools, i32(table), i32(lens)).view(n, rows, 24, 256)
    worst = 0.0
    for b, L in enumerate(lens):
        if L < 0 or (n > 60 and L < 1000 and b % 16):
            continue
        t = torch.arange(L + rows, device="cuda")
        tab = torch.tensor(table[b], device="cuda")
        slots = tab[t // page] * page + t % page
        for kv in range(2):
            hs = slice(12 * kv, 12 * kv + 12)
            want = attend64(q[b, :, hs], qg[b, :, hs, 256:], kw[slots, kv], vw[slots, kv],
                            [L + r + 1 for r in range(rows)])
            worst = max(worst, float(row_errors(out[b, :, hs], want).max()))
    assert worst <= ROW_BOUND, worst
