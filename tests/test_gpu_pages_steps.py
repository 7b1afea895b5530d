"""Whole steps of servers with branches, with their attention's outputs compared: captured and replayed
against plain calls and the float64 oracle, and two servers' steps that overlap on two streams, without
a read by the host between them."""
import numpy as np
import pytest
import torch

from tests.parity import SEED
from tests.q4_bounds import attend64, row_errors
from tests.q8_bounds import ROW_BOUND
from verify_gated_gqa_gb300 import binding as B
from verify_gated_gqa_gb300 import build as build_mod

pytestmark = pytest.mark.gpu
PAGE = 32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_mod.build()
    B.lib()
    yield
    assert B.ga_device_status() == 0


def _i32(x):
    return torch.tensor(np.asarray(x, np.int64), dtype=torch.int32, device="cuda")


def _same_bits(a, b):
    view = torch.int16 if a.dtype == torch.bfloat16 else a.dtype
    return torch.equal(a.view(view), b.view(view))


class State:
    """Page tables, stack and 8-bit pools of n rows."""

    def __init__(self, n, width, pool, seed):
        u8 = lambda *s: torch.full((pool, 2) + s, 0x7F, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.pools = [u8(PAGE, 256), u8(PAGE // 32), u8(PAGE, 256), u8(PAGE // 32)]
        self.table, self.held = _i32(np.full((n, width), -1)), _i32([0] * n)
        self.free, self.count = _i32(np.random.default_rng(seed).permutation(pool)), _i32([pool])
        self.shared = _i32([0] * pool)
        self.ws = torch.empty(B.ga_verify_q8_workspace_bytes(), dtype=torch.uint8, device="cuda")
        self.wc = torch.empty(B.ga_page_compact_workspace_bytes(pool), dtype=torch.uint8, device="cuda")

    def all(self):
        return [self.table, self.held, self.free, self.count, self.shared, *self.pools]

    def append(self, lens, new, total, k, v):
        _, slots, _, info = B.ga_page_plan(lens, new, self.table, self.held, self.free, self.count, PAGE, total)
        B.ga_kv_quantize_q8(k, v, *self.pools, slots=slots)
        return info

    def fork(self, parent, child, lens):
        src, dst, info = B.ga_page_fork(parent, child, lens, self.table, self.held, self.free, self.count,
                                        self.shared, PAGE)
        B.ga_page_copy(self.pools, src, dst)
        return info

    def release(self, keep):
        return B.ga_page_release(keep, self.table, self.held, self.free, self.count, self.shared, PAGE)

    def compact(self, moves):
        src, dst, info = B.ga_page_compact(self.table, self.held, self.free, self.count, self.shared, moves,
                                           workspace=self.wc)
        B.ga_page_copy(self.pools, src, dst)
        return info

    def attend(self, q, qg, lens, out):
        return B.ga_attn_verify_q8(q, qg, *self.pools, self.table, lens, out=out, workspace=self.ws)

    def check_rows(self, q, qg, lens, out):
        """Every row's window against the float64 oracle, from the pages as they are."""
        rows = q.shape[1]
        for b, x in enumerate(lens.tolist()):
            if x < 0:
                continue
            t = torch.arange(x + rows, device="cuda")
            slots = self.table[b].long()[t // PAGE] * PAGE + t % PAGE
            k, v = B.ga_kv_dequantize_q8(*self.pools, slots=slots.to(torch.int32))
            for kv in range(2):
                hs = slice(12 * kv, 12 * kv + 12)
                want = attend64(q[b, :, hs], qg[b, :, hs, 256:], k[:, kv], v[:, kv], [x + r + 1 for r in range(rows)])
                got = out[b].view(rows, 24, 256)[:, hs]
                # few keys: the weights' errors do not average out (under 3 x 2^-8 beside the output's 2^-8)
                assert float(row_errors(got, want).max()) <= (ROW_BOUND if x > 60 else 3 * ROW_BOUND), (b, x)


def _capture(run, warm):
    """A graph of run(); `warm` is run on another stream first."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        result = run()
    return graph, result


# ------------------------------------------------------------------ captured, other rows and lengths
@pytest.mark.parametrize("rows", [1, 3, 6])
def test_captured_steps_attend_to_their_branches(rows):
    n, tokens = 6, max(24, 5 * rows)
    g = torch.Generator(device="cuda")
    g.manual_seed(SEED + rows)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    prompt = normal(227, 2, 256), normal(227, 2, 256)

    def make():
        s = State(n, 12, 60, 5)
        info = s.append(_i32([0, 0] + [-1] * 4), _i32([150, 77] + [0] * 4), 227, *prompt)
        assert info[0].item() == 0
        return s

    plain, graph_side = make(), make()
    io = dict(parent=_i32([-1] * 3), child=_i32([0] * 3), flen=_i32([0] * 3), lens=_i32([-1] * n),
              alens=_i32([-1] * n), new=_i32([0] * n), keep=_i32([-1] * n), k=normal(tokens, 2, 256),
              v=normal(tokens, 2, 256), q=normal(n, rows, 24, 256), qg=normal(n, rows, 24, 512))
    outs = {s: torch.zeros(n, rows, 6144, dtype=torch.bfloat16, device="cuda") for s in (plain, graph_side)}

    def first_half(s):
        return [s.fork(io["parent"], io["child"], io["flen"]),
                s.append(io["lens"], io["new"], tokens, io["k"], io["v"]),
                s.attend(io["q"], io["qg"], io["alens"], outs[s])][:2]

    def second_half(s):
        return [s.release(io["keep"]), s.compact(4)]

    spare = make()
    outs[spare] = torch.zeros_like(outs[plain])
    graph, infos = _capture(lambda: torch.stack(first_half(graph_side) + second_half(graph_side)),
                            lambda: first_half(spare) + second_half(spare))
    lens = [150, 77, -1, -1, -1, -1]
    moves = [(dict(parent=[0, 0, 1], child=[2, 3, 4], flen=[150, 96, 70]), [rows, rows, 0, rows, rows, 0], [-1] * 6),
             (dict(parent=[-1, 2, -1], child=[0, 5, 0], flen=[0, 120, 0]), [rows] * 4 + [0, rows],
              [0, -1, -1, 64, -1, -1]),
             (dict(parent=[3, -1, -1], child=[0, 0, 0], flen=[32, 0, 0]), [rows, 0, rows, 0, rows, 0],
              [-1, 0, 0, -1, 64, -1]),
             (dict(parent=[-1] * 3, child=[0] * 3, flen=[0] * 3), [0] * 6, [0] * 6)]
    for forks, new, keep in moves:
        for c, p, x in zip(forks["child"], forks["parent"], forks["flen"]):
            if p >= 0:
                lens[c] = x
        new = [a if x >= 0 else 0 for a, x in zip(new, lens)]
        assert sum(new) <= tokens
        for name, x in dict(forks, lens=lens, alens=[x if a else -1 for a, x in zip(new, lens)], new=new,
                            keep=keep).items():
            io[name].copy_(_i32(x))
        for name in ("k", "v", "q", "qg"):
            io[name].copy_(normal(*io[name].shape))
        outs[plain].fill_(5.0)
        outs[graph_side].fill_(5.0)
        graph.replay()
        i0, i1 = first_half(plain)
        plain.check_rows(io["q"], io["qg"], io["alens"], outs[plain])
        want = torch.stack([i0, i1] + second_half(plain))
        assert torch.equal(infos, want) and not want[:, 0].any()
        assert _same_bits(outs[graph_side], outs[plain])
        for b, a in enumerate(new):
            assert bool((outs[plain][b] == 5).all()) == (a == 0)
        assert all(torch.equal(a, b) for a, b in zip(graph_side.all(), plain.all()))
        lens = [x + a if x >= 0 else x for x, a in zip(lens, new)]
        lens = [x if k < 0 else -1 if k == 0 else min(x, k) for x, k in zip(lens, keep)]


# ------------------------------------------------------------------ two servers at once
class Cycle:
    """A server's life from an empty pool to an empty pool: a prompt, branches, tokens, attention, rows let
    go, the pool packed, attention again, all finished. Every tensor is made beforehand."""

    def __init__(self, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(SEED + 100 + seed)
        normal = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        self.seed = seed
        self.prompt, self.tokens = (normal(300, 2, 256), normal(300, 2, 256)), (normal(43, 2, 256), normal(43, 2, 256))
        self.q, self.qg = [normal(8, 2, 24, 256) for _ in range(2)], [normal(8, 2, 24, 512) for _ in range(2)]
        self.i = {k: _i32(v) for k, v in dict(
            lens0=[0] + [-1] * 7, new0=[300] + [0] * 7, parent=[0] * 3, child=[1, 2, 3], flen=[300, 64, 100],
            lens1=[300, 300, 64, 100] + [-1] * 4, new1=[1, 40, 1, 1] + [0] * 4,
            alens1=[299, 338, 63, 99] + [-1] * 4, keep=[0, 0, -1, 50] + [-1] * 4,
            alens2=[-1, -1, 63, 48] + [-1] * 4, none=[0] * 8).items()}
        self.zeros = torch.zeros(8, 2, 6144, dtype=torch.bfloat16, device="cuda")

    def state(self):
        return State(8, 20, 120, self.seed)

    def run(self, s, check=False):
        i, outs = self.i, [self.zeros.clone(), self.zeros.clone()]
        infos = [s.append(i["lens0"], i["new0"], 300, *self.prompt), s.fork(i["parent"], i["child"], i["flen"]),
                 s.append(i["lens1"], i["new1"], 43, *self.tokens)]
        s.attend(self.q[0], self.qg[0], i["alens1"], outs[0])
        if check:
            s.check_rows(self.q[0], self.qg[0], i["alens1"], outs[0])
        infos += [s.release(i["keep"]), s.compact(50)]
        s.attend(self.q[1], self.qg[1], i["alens2"], outs[1])
        if check:
            s.check_rows(self.q[1], self.qg[1], i["alens2"], outs[1])
        return outs, torch.stack(infos + [s.release(i["none"])])


@pytest.mark.parametrize("captured", [False, True])
def test_two_servers_overlap_on_two_streams(captured):
    rounds = 12
    cycles = [Cycle(k) for k in range(2)]
    want = []
    for c in cycles:                                    # alone, and read in between
        s = c.state()
        done = [c.run(s, check=k == 0) for k in range(rounds)]
        assert not any(info[:, 0].any() for _, info in done) and s.count.item() == 120 and not s.shared.any()
        want.append((done, s))
    states, streams = [c.state() for c in cycles], [torch.cuda.Stream() for _ in cycles]
    if captured:
        graphs = [_capture(lambda c=c, s=s: c.run(s), lambda c=c: c.run(c.state())) for c, s in zip(cycles, states)]
        wrong = [torch.zeros(1, dtype=torch.int64, device="cuda") for _ in cycles]
    got = [[] for _ in cycles]
    torch.cuda.synchronize()
    for r in range(rounds):                             # nothing below waits on the host
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                if captured:
                    graph, (outs, infos) = graphs[k]
                    graph.replay()
                    w_outs, w_infos = want[k][0][r]
                    for a, b in zip([*outs, infos], [*w_outs, w_infos]):
                        wrong[k] += (a.view(torch.int16) != b.view(torch.int16)).sum()
                else:
                    got[k].append(cycles[k].run(states[k]))
    torch.cuda.synchronize()
    for k, (done, s) in enumerate(want):
        if captured:
            assert wrong[k].item() == 0
        for (outs, infos), (w_outs, w_infos) in zip(got[k], done):
            assert torch.equal(infos, w_infos) and all(_same_bits(a, b) for a, b in zip(outs, w_outs))
        assert all(torch.equal(a, b) for a, b in zip(states[k].all(), s.all()))
