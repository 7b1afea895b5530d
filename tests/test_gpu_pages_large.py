"""Compaction of pools of many pages and copies at the sizes where a copy changes its way."""
import numpy as np
import pytest
import torch

from oracle import ga_oracle as O
from tests.parity import SEED
from tests.test_gpu_pages import _compact, _same
from verify_gated_gqa_gb300 import binding as B
from verify_gated_gqa_gb300 import build as build_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_mod.build()
    B.lib()
    yield
    assert B.ga_device_status() == 0


@pytest.mark.parametrize("n_free,width,used", [
    (1, 1, 1), (31, 40, 0.5), (33, 1024, 0.9), (1025, 33, 0.3), (2048, 128, 1.0), (2049, 64, 0.0), (65536, 600, 0.7),
    (65537, 2000, 0.02), (200003, 300, 0.5)])
@pytest.mark.parametrize("part", [1.0, 0.3])
def test_compaction_of_large_pools(n_free, width, used, part):
    """Pages in use at random places; runs of a warp that end inside its 32 pages and beyond the pool."""
    rng = np.random.default_rng(SEED + n_free)
    pages = rng.permutation(n_free)
    live = int(round(used * n_free))
    n = min(2048, max(1, -(-live // max(1, width * 3 // 4))) + 1)
    held = np.zeros(n, np.int64)
    table = rng.integers(-5, n_free + 5, (n, width))   # past `held` entries are not looked at
    left, at = live, 0
    for b in range(n):
        held[b] = min(left, width, rng.integers(0, width + 1) if b + 1 < n else width)
        table[b, :held[b]] = pages[at:at + held[b]]
        at, left = at + held[b], left - held[b]
    stack = rng.integers(-3, n_free, n_free)           # past free_count too
    count = n_free - at
    stack[:count] = pages[at:]
    shared = np.where(np.isin(np.arange(n_free), pages[:at]), rng.integers(0, 9, n_free), 0)
    moves = max(1, int(part * min(n_free, 4 * n_free // 10)))
    want = O.page_compact(table, held, stack, count, shared, moves)
    for in_place in (True, False):
        got = _compact(table, held, stack, count, shared, moves, in_place)
        _same(got, want, (n_free, in_place))


@pytest.mark.parametrize("n_copies", [1, 37, 38, 75, 76, 77, 700])
@pytest.mark.parametrize("sizes", [[4096, 4080], [4112, 2048, 65536], [32768 + 16, 8]])
def test_copies_where_the_way_changes(n_copies, sizes):
    g = torch.Generator(device="cuda")
    g.manual_seed(SEED + n_copies)
    n_pages = 2 * n_copies + 3
    pools = [torch.randint(0, 256, (n_pages, s), generator=g, device="cuda", dtype=torch.uint8) for s in sizes]
    want = [p.clone() for p in pools]
    perm = torch.randperm(n_pages, generator=g, device="cuda")
    src, dst = perm[:n_copies].clone(), perm[n_copies:2 * n_copies].clone()
    if n_copies > 1:
        src[::5] = -1
    for w in want:
        keep = src >= 0
        w[dst[keep]] = w[src[keep]]
    B.ga_page_copy(pools, src.to(torch.int32), dst.to(torch.int32))
    assert all(torch.equal(p, w) for p, w in zip(pools, want))
