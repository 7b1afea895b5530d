"""Calls queued one behind the other over one buffer of fused query and gate rows that is written
anew before each: the merge of streams that were cut into parts is launched ahead of the parts, and has
to see the gates of its own call."""
import numpy as np
import pytest
import torch

from tests.parity import SEED
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


LENS = {"one": [30000], "few": [3000, 700, 9001], "many": [(b * 37 + 11) % 64 * 60 for b in range(64)]}


@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("rows", [1, 3, 6, 16])
@pytest.mark.parametrize("bits", [4, 8])
def test_gates_written_anew_between_calls(bits, rows, lens):
    g = torch.Generator(device="cuda")
    g.manual_seed(SEED + bits + rows)
    lens, page, versions = LENS[lens], 64, 12
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    width = -(-(max(lens) + rows) // page)
    n_pages = len(lens) * width
    table = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32).view(len(lens), width)
    u8 = lambda *s: torch.zeros(n_pages, 2, *s, dtype=torch.uint8, device="cuda")  # noqa: E731
    if bits == 4:
        pools = [u8(page, 128), u8(page, 16), u8(page, 128), u8(page, 16)]
        store, attend, ws = B.ga_kv_quantize_q4, B.ga_attn_verify_q4, B.ga_verify_q4_workspace_bytes()
    else:
        pools = [u8(page, 256), u8(page // 32), u8(page, 256), u8(page // 32)]
        store, attend, ws = B.ga_kv_quantize_q8, B.ga_attn_verify_q8, B.ga_verify_q8_workspace_bytes()
    store(normal(n_pages * page, 2, 256), normal(n_pages * page, 2, 256), *pools)
    ws = torch.empty(ws, dtype=torch.uint8, device="cuda")
    q, seq_len = normal(len(lens), rows, 24, 256), _i32(lens)
    # version 0 is the buffer of the queued calls; the others' gates are all different
    rows_of = normal(versions + 1, len(lens), rows, 24, 512)
    fresh = [rows_of[i].clone() for i in range(versions + 1)]
    want = [attend(q, x, *pools, table, seq_len) for x in fresh]
    assert not any(torch.equal(want[1], x) for x in want[2:])
    got = [torch.empty_like(want[0]) for _ in want]
    pages, to = _i32(np.arange(versions + 1)), _i32([0])
    torch.cuda.synchronize()
    for by_copy in (False, True):       # by a kernel of torch's, or by one that lets the next begin early
        for i in range(1, versions + 1):
            if by_copy:
                B.ga_page_copy([rows_of], pages[i:i + 1], to)
            else:
                rows_of[0].copy_(fresh[i])
            attend(q, rows_of[0], *pools, table, seq_len, out=got[i], workspace=ws)
        torch.cuda.synchronize()
        for i in range(1, versions + 1):
            assert torch.equal(got[i].view(torch.int16), want[i].view(torch.int16)), (by_copy, i)
            got[i].zero_()
