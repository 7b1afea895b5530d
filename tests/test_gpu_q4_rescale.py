"""The 4-bit attention's running maximum where it grows inside a segment: O and l, with many keys
in them already, are scaled to the new maximum.

Every row has a key of its own somewhere in the cache whose score is about 8 (11.5 binary
orders) above all others, so that its maximum passes the lazy rescale's 2^8 there, and whose weight
is about that of the 3,000 other keys together: O's old content and the new key both count for the
output, and a factor that is wrong, or that reaches part of O only, shows in every dim. Rows meet
their key at different places, so that warps in which some rows grow, or none, occur too."""
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


def _segment_tiles(n_seq, keys, rows):
    """Tiles of the longest segments, about: a worker's run of the cut without one stream's lead."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tile, lead = (32, 16) if rows == 1 else (128, 6)
    workers = min(sms, 160) // (2 if rows * 12 > 96 else 1)
    units = 2 * n_seq * (-(-keys // tile) + lead)
    return min(-(-units // workers) - lead, -(-keys // tile))


def _case(n_seq, length, rows, page, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    keys = length + rows
    per = -(-keys // page)
    n_pages = n_seq * per + 1
    table = torch.tensor(rng.permutation(n_pages)[:n_seq * per].reshape(n_seq, per),
                         dtype=torch.int32, device="cuda")
    q = normal(n_seq, rows, 24, 256).to(torch.bfloat16)
    qg = normal(n_seq, rows, 24, 512).to(torch.bfloat16)
    k = normal(n_seq, keys, 2, 256) * 0.3
    v = normal(n_seq, keys, 2, 256)
    for b in range(n_seq):
        # one key a row (of either KV head's 12 heads), below every row's last visible key
        for kv in range(2):
            at = torch.tensor(rng.permutation(length)[:12 * rows], device="cuda")
            k[b, at, kv] = 0.5 * q[b, :, 12 * kv:12 * kv + 12].reshape(12 * rows, 256).float()
    pools = [torch.zeros(n_pages, 2, page, w, dtype=torch.uint8, device="cuda")
             for w in (128, 16, 128, 16)]
    t = torch.arange(keys, device="cuda")
    slots = (table.long()[:, t // page] * page + t % page).to(torch.int32).flatten()
    B.ga_kv_quantize_q4(k.flatten(0, 1).to(torch.bfloat16), v.flatten(0, 1).to(torch.bfloat16),
                        *pools, slots=slots)
    kw, vw = (x.view(n_seq, keys, 2, 256) for x in B.ga_kv_dequantize_q4(*pools, slots=slots))
    lens = torch.full((n_seq,), length, dtype=torch.int32, device="cuda")
    return q, qg, pools, table, lens, kw, vw


@pytest.mark.parametrize("rows,n_seq,length,page", [(2, 64, 3001, 64), (6, 64, 3001, 32),
                                                    (8, 70, 2500, 96), (16, 64, 3001, 128)])
def test_rows_grow_inside_segments(rows, n_seq, length, page):
    # segments long enough that most rows meet their key after the first of several tiles
    assert _segment_tiles(n_seq, length + rows, rows) >= 8
    q, qg, pools, table, lens, kw, vw = _case(n_seq, length, rows, page, 4100 + rows)
    out = B.ga_attn_verify_q4(q, qg, *pools, table, lens).view(n_seq, rows, 24, 256)
    worst = 0.0
    for b in range(n_seq):
        for kv in range(2):
            hs = slice(12 * kv, 12 * kv + 12)
            want = attend64(q[b, :, hs], qg[b, :, hs, 256:], kw[b, :, kv], vw[b, :, kv],
                            [length + r + 1 for r in range(rows)])
            worst = max(worst, float(row_errors(out[b, :, hs], want).max()))
    assert worst <= ROW_BOUND, worst
    for _ in range(20):   # the same bits, whichever half of a tile's softmax is ahead
        again = B.ga_attn_verify_q4(q, qg, *pools, table, lens)
        assert torch.equal(again.view_as(out), out)


@pytest.mark.parametrize("n_seq,length,page", [(64, 3001, 64), (150, 2000, 32)])
def test_decoding_rows_grow_inside_segments(n_seq, length, page):
    """One row a sequence: each of eight warps takes every eighth granule of 32 keys and keeps a
    maximum of its own, so the warp that meets the row's key grows and the others do not."""
    assert _segment_tiles(n_seq, length + 1, 1) >= 8 * 3
    q, qg, pools, table, lens, kw, vw = _case(n_seq, length, 1, page, 4200 + n_seq)
    out = B.ga_attn_verify_q4(q, qg, *pools, table, lens).view(n_seq, 1, 24, 256)
    worst = 0.0
    for b in range(n_seq):
        for kv in range(2):
            hs = slice(12 * kv, 12 * kv + 12)
            want = attend64(q[b, :, hs], qg[b, :, hs, 256:], kw[b, :, kv], vw[b, :, kv],
                            [length + 1])
            worst = max(worst, float(row_errors(out[b, :, hs], want).max()))
    assert worst <= ROW_BOUND, worst
    for _ in range(10):
        assert torch.equal(B.ga_attn_verify_q4(q, qg, *pools, table, lens).view_as(out), out)


@pytest.mark.parametrize("rows", [1, 5, 16])
def test_every_tile_grows(rows):
    """Scores that rise by more than 2^8 from one tile (or a warp's granule) to its next, all along
    segments of many: every step scales O and l, and what is left of the older keys is below the
    outputs' rounding, so a step that scales too little shows."""
    n_seq, length, page = 64, 3001, 64
    keys = length + rows
    tile = 32 * 8 if rows == 1 else 128       # keys from one step of a running maximum to its next
    assert _segment_tiles(n_seq, keys, rows) >= (24 if rows == 1 else 8)
    g = torch.Generator(device="cuda")
    g.manual_seed(4300 + rows)
    qg = torch.randn(n_seq, rows, 24, 512, generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn(n_seq * keys, 2, 256, generator=g, device="cuda").to(torch.bfloat16)
    # q is 16 in every dim, a key 1 (widened: 63 / 64) in its first 8 s dims, s its step: each step
    # adds 8 x 16 x 63 / 64 / 16 = 7.9 to the score, 11.4 binary orders
    q = torch.full((n_seq, rows, 24, 256), 16.0, dtype=torch.bfloat16, device="cuda")
    t = torch.arange(keys, device="cuda")
    dims = torch.arange(256, device="cuda")
    k1 = (dims[None] < 8 * (t // tile)[:, None]).to(torch.bfloat16)      # [keys, 256]
    k = k1[None, :, None].expand(n_seq, keys, 2, 256).flatten(0, 1)
    per = -(-keys // page)
    table = torch.randperm(n_seq * per, generator=g, device="cuda").to(torch.int32).view(n_seq, per)
    slots = (table.long()[:, t // page] * page + t % page).to(torch.int32).flatten()
    pools = [torch.zeros(n_seq * per, 2, page, w, dtype=torch.uint8, device="cuda")
             for w in (128, 16, 128, 16)]
    B.ga_kv_quantize_q4(k.contiguous(), v, *pools, slots=slots)
    kw, vw = (x.view(n_seq, keys, 2, 256) for x in B.ga_kv_dequantize_q4(*pools, slots=slots))
    lens = torch.full((n_seq,), length, dtype=torch.int32, device="cuda")
    out = B.ga_attn_verify_q4(q, qg, *pools, table, lens).view(n_seq, rows, 24, 256)
    for b in range(0, n_seq, 7):
        for kv in range(2):
            hs = slice(12 * kv, 12 * kv + 12)
            want = attend64(q[b, :, hs], qg[b, :, hs, 256:], kw[b, :, kv], vw[b, :, kv],
                            [length + r + 1 for r in range(rows)])
            worst = float(row_errors(out[b, :, hs], want).max())
            assert worst <= ROW_BOUND, (b, kv, worst)
