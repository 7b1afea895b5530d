"""Calls of the 4-bit serving set that its documentation allows, in the ways that a server makes
them: several refusals at once, one position row for all axes, a captured step that joins streams,
idle rows at the end of a batch, and the slots of tokens that are cached already."""
import numpy as np
import pytest
import torch

from oracle import ga_oracle as O
from tests.parity import SEED, np64
from tests.q4_bounds import ROW_BOUND, attend64, row_errors
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


# ------------------------------------------------------------------ captured steps
@pytest.mark.parametrize("rows", [1, 4])
def test_captured_attention_after_a_join_of_streams(rows):
    """Keys stored on one stream, queries prepared on another and lengths copied on a third, all
    captured into one graph; the attention follows their join, and another call it."""
    n, page, per = 3, 32, 40
    g = torch.Generator(device="cuda")
    g.manual_seed(SEED + rows)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    table = torch.randperm(n * per, generator=g, device="cuda").to(torch.int32).view(n, per)
    w_q = synth.normal_bf16(SEED, "w_q", (256,), sigma=0.1).cuda()
    c, s = (t.cuda() for t in B.ga_rope_table_host(2048))
    keys = n * per * page
    pos = _i32([1000 + i % rows for i in range(n * rows)])
    live = dict(k=normal(keys, 2, 256), v=normal(keys, 2, 256), qg=normal(n * rows, 24, 512),
                lens=_i32([900, 30, 1100]))
    pools = [torch.zeros(n * per, 2, page, w, dtype=torch.uint8, device="cuda")
             for w in (128, 16, 128, 16)]
    lens = torch.zeros(n, dtype=torch.int32, device="cuda")
    q = torch.empty(n * rows, 24, 256, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(n, rows, 6144, dtype=torch.bfloat16, device="cuda")
    again = torch.empty_like(out)
    ws = torch.empty(B.ga_verify_q4_workspace_bytes(), dtype=torch.uint8, device="cuda")
    side = [torch.cuda.Stream() for _ in range(2)]

    def call(o):
        B.ga_attn_verify_q4(q.view(n, rows, 24, 256), live["qg"].view(n, rows, 24, 512), *pools, table,
                            lens, out=o, workspace=ws)

    def step():
        main = torch.cuda.current_stream()
        for x in side:
            x.wait_stream(main)
        B.ga_kv_quantize_q4(live["k"], live["v"], *pools)
        with torch.cuda.stream(side[0]):
            B.ga_qk_prologue_axes(None, None, live["qg"], w_q, pos, None, c, s, q_prep=q)
        with torch.cuda.stream(side[1]):
            lens.copy_(live["lens"])
        for x in side:
            main.wait_stream(x)
        call(out)
        call(again)

    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step()
    torch.cuda.current_stream().wait_stream(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for new in ([900, 30, 1100], [0, 1200, 5], [31, -1, 1270 - rows]):
        for name in ("k", "v", "qg"):
            live[name].copy_(normal(*live[name].shape))
        live["lens"].copy_(_i32(new))
        lens.fill_(3)
        q.zero_()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, again) or -1 in new
        kw, vw = B.ga_kv_dequantize_q4(*pools)
        for b, L in enumerate(new):
            if L < 0:
                assert bool((out[b] == 0).all())
                continue
            t = torch.arange(L + rows, device="cuda")
            slots = table[b].long()[t // page] * page + t % page
            for kv in range(2):
                hs = slice(12 * kv, 12 * kv + 12)
                want = attend64(q.view(n, rows, 24, 256)[b, :, hs],
                                live["qg"].view(n, rows, 24, 512)[b, :, hs, 256:], kw[slots, kv],
                                vw[slots, kv], [L + r + 1 for r in range(rows)])
                got = out.view(n, rows, 24, 256)[b, :, hs]
                assert float(row_errors(got, want).max()) <= (ROW_BOUND if L > 60 else 2 * ROW_BOUND)


def test_captured_steps_with_idle_rows_at_the_end():
    """A batch of four rows captured once, of which two, three and four are in use: the idle ones, at
    the end, have length -1, and the packed tokens of the plan then lie as the windows do."""
    n, rows, page, width = 4, 2, 32, 4
    T, pool = n * rows, n * width
    g = torch.Generator(device="cuda")
    g.manual_seed(SEED + 9)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    w = synth.normal_bf16(SEED, "w_k", (256,), sigma=0.1).cuda()
    c, s = (t.cuda() for t in B.ga_rope_table_host(512))
    cos, sin = O.rope_tables(512)
    pools = [torch.zeros(pool, 2, page, x, dtype=torch.uint8, device="cuda") for x in (128, 16, 128, 16)]
    table, held = _i32(np.full((n, width), -1)), _i32([0] * n)
    free, count = _i32(np.random.default_rng(4).permutation(pool)), _i32([pool])
    seq_len, new_len = _i32([-1] * n), _i32([0] * n)
    k, v, qg = normal(T, 2, 256), normal(T, 2, 256), normal(T, 24, 512)
    out = torch.zeros(n, rows, 6144, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(B.ga_verify_q4_workspace_bytes(), dtype=torch.uint8, device="cuda")

    def step():
        _, slots, pos, _ = B.ga_page_plan(seq_len, new_len, table, held, free, count, page, T)
        kp, qp = B.ga_qk_prologue_axes(k, w, qg, w, pos, None, c, s)
        B.ga_kv_quantize_q4(kp, v, *pools, slots=slots)
        B.ga_attn_verify_q4(qp.view(n, rows, 24, 256), qg.view(n, rows, 24, 512), *pools, table, seq_len,
                            out=out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    seen = [([], []) for _ in range(n)]
    lens = [0] * n
    for used in (2, 2, 3, 4, 3, 2, 4) + (4,) * 20:
        for x in (k, v, qg):
            x.copy_(normal(*x.shape))
        seq_len.copy_(_i32([lens[b] if b < used else -1 for b in range(n)]))
        new_len.copy_(_i32([rows if b < used else 0 for b in range(n)]))
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        for b in range(n):
            if b >= used:
                assert bool((out[b] == 9).all())
                continue
            at = slice(b * rows, (b + 1) * rows)
            pos = [[lens[b] + r for r in range(rows)]]
            for i, x in enumerate((O.prep_axes(np64(k[at]), np64(w), cos, sin, pos, [0] * 32), np64(v[at]))):
                seen[b][i].append(O.widen_q4_rows(*O.quantize_q4_rows(x)))
            q = O.prep_axes(np64(qg[at])[..., :256], np64(w), cos, sin, pos, [0] * 32)
            want, mass = O.verify_q4(q[None], np64(qg[at])[None, ..., 256:], [np.concatenate(seen[b][0])],
                                     [np.concatenate(seen[b][1])], [lens[b]])
            # per element, as the roundings allow: 2 x 2^-8 of the weighted magnitudes, 2^-8 of itself
            got = np64(out[b]).reshape(want[0].shape)
            assert np.all(np.abs(got - want[0]) <= (2.0 ** -7 + 2.0 ** -10) * mass[0]
                          + 2.0 ** -8 * np.abs(want[0]) + 1e-30)
            lens[b] += rows


# ------------------------------------------------------------------ cached tokens' slots
def test_plan_gives_the_slots_of_cached_tokens():
    """The plan over lengths of 0 and the cached lengths as new tokens takes no page, as the rows hold
    theirs, and lists every cached token's slot: what widening a whole cache for a prefill needs."""
    page, lens, width, bound = 32, [100, 0, 33, 64], 6, 256
    need = [-(-x // page) for x in lens]
    perm = np.random.default_rng(2).permutation(sum(need) + 3)
    table, at = np.full((4, width), -1), 0
    for b, m in enumerate(need):
        table[b, :m] = perm[at:at + m]
        at += m
    free = _i32(np.concatenate([perm[at:], [0] * at]))
    t, held, count = _i32(table), _i32(need), _i32([3])
    start, slots, pos, info = B.ga_page_plan(_i32([0] * 4), _i32(lens), t, held, free, count, page, bound)
    assert info.tolist() == [0, sum(lens), 0, 0] and count.tolist() == [3]
    assert start.tolist() == np.concatenate([[0], np.cumsum(lens)]).tolist()
    assert np.array_equal(t.cpu().numpy(), table) and held.tolist() == need
    want = [table[b, p // page] * page + p % page for b, x in enumerate(lens) for p in range(x)]
    assert slots.tolist() == want + [-1] * (bound - sum(lens))
    pools = [torch.zeros(len(perm), 2, page, w, dtype=torch.uint8, device="cuda")
             for w in (128, 16, 128, 16)]
    x = torch.randn(len(perm) * page, 2, 256, device="cuda").to(torch.bfloat16)
    B.ga_kv_quantize_q4(x, -x, *pools)
    whole = B.ga_kv_dequantize_q4(*pools)
    k, v = (torch.full((bound, 2, 256), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    B.ga_kv_dequantize_q4(*pools, slots=slots, k_out=k, v_out=v)
    for got, all_rows in ((k, whole[0]), (v, whole[1])):
        assert torch.equal(got[:sum(lens)], all_rows[torch.tensor(want, device="cuda")])
        assert bool((got[sum(lens):] == 7).all())
