"""Calls of the 4-bit serving set that its documentation allows, in the ways that a server makes
them: several refusals at once, one position row for all axes."""
import numpy as np
import pytest
import torch

from oracle import ga_oracle as O
from tests.parity import SEED
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


# ------------------------------------------------------------------ the step plan
PLAN = dict(L=[40, 10, 5], a=[4, 30, -1], held=[2, 1, 1], count=3, mt=34)
FAULTS = {   # each by itself: what it changes, its status
    "range": (dict(held=[2, 4, 1]), 4), "far": (dict(a=[90, 30, -1]), 2),
    "room": (dict(count=5, a=[4, 0, -1]), 4), "tokens": (dict(mt=3), 1), "pages": (dict(count=0), 3)}


def _plan_statuses(case, pad):
    table, stack = np.array([[0, 1, -1], [2, -1, -1], [3, -1, -1]]), np.array([4, 5, 6, 0, 0])
    L, a, held, mt = np.array(case["L"]), np.array(case["a"]), np.array(case["held"]), case["mt"] + pad
    want = O.page_plan(L, a, table, held, stack, case["count"], 32, mt)
    t, h, f, c = _i32(table), _i32(held), _i32(stack), _i32([case["count"]])
    start, slots, pos, info = B.ga_page_plan(_i32(L), _i32(a), t, h, f, c, 32, mt)
    for g, w in zip((t, h, f, c, start, slots, pos, info), want):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))
    return int(want[-1][0])


def test_plan_refusals_in_their_order():
    """Two reasons at once: 4 for a range, then 2, then 4 for the stack's room, then 1, then 3."""
    for change, status in FAULTS.values():
        assert _plan_statuses({**PLAN, **change}, 0) == status
    # the far sequence's own pages are left out of the sums that would refuse the stack's room
    assert _plan_statuses({**PLAN, "a": [90, 0, -1], "count": 5}, 0) == 2
    assert _plan_statuses({**PLAN, "a": [90, 0, -1], "count": 5}, 9000) == 2
    assert _plan_statuses({**PLAN, "a": [90, 30, -1], "held": [2, 4, 1]}, 0) == 4
    assert _plan_statuses({**PLAN, "a": [90, 30, -1], "count": 6}, 0) == 4
    assert _plan_statuses({**PLAN, "a": [90, 30, -1], "mt": 3, "count": 0}, 0) == 2
    assert _plan_statuses({**PLAN, "a": [4, 0, -1], "count": 5, "mt": 3}, 0) == 4
    assert _plan_statuses({**PLAN, "mt": 3, "count": 0}, 0) == 1


# ------------------------------------------------------------------ the prologue over axes
@pytest.mark.parametrize("n", [1, 37])
def test_axes_share_one_row_of_positions(n):
    """Text alone: the same positions on every axis, as one row seen three times."""
    k = synth.normal_bf16(SEED, "k", (n, 2, 256)).cuda()
    qg = synth.normal_bf16(SEED, "qg", (n, 24, 512)).cuda()
    w_k = synth.normal_bf16(SEED, "w_k", (256,), sigma=0.1).cuda()
    w_q = synth.normal_bf16(SEED, "w_q", (256,), sigma=0.1).cuda()
    c, s = (t.cuda() for t in B.ga_rope_table_host(512))
    pos = torch.arange(400, 400 + n, dtype=torch.int32, device="cuda")
    pairs = [i % 3 for i in range(32)]
    want = B.ga_qk_prologue_axes(k, w_k, qg, w_q, pos[None].repeat(3, 1), pairs, c, s)
    got = B.ga_qk_prologue_axes(k, w_k, qg, w_q, pos[None].expand(3, n), pairs, c, s)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
