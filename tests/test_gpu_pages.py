"""GPU parity of the calls over pages that several sequences hold (fork, release, compact, copy)
against the oracle, alone, as a server's steps together with the plan and the 8-bit cache, and
captured."""
import numpy as np
import pytest
import torch

from oracle import ga_oracle as O
from tests.parity import SEED, np64
from tests.q4_bounds import attend64, row_errors
from tests.q8_bounds import ROW_BOUND
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
    return torch.tensor(np.asarray(x, np.int64), dtype=torch.int32, device="cuda")


def _same(got, want, what=""):
    for i, (g, w) in enumerate(zip(got, want)):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1)), (what, i)


def _state(rng, n, width, max_len, page, spare, share=0.0):
    """Random rows over a pool, some of whose pages several rows hold (only as first columns)."""
    lens = rng.integers(0, max_len + 1, n)
    held = np.minimum(-(-lens // page), width)
    table = np.full((n, width), -1)
    total = int(held.sum()) + spare
    perm = list(rng.permutation(total))
    shared = np.zeros(total, np.int64)
    for b in range(n):
        k = 0
        if b and rng.random() < share:
            a = int(rng.integers(b))
            k = int(rng.integers(0, min(held[a], held[b]) + 1))
            table[b, :k] = table[a, :k]
            for x in table[a, :k]:
                shared[x] += 1
        for c in range(k, held[b]):
            table[b, c] = perm.pop()
    stack = np.zeros(total, np.int64)
    stack[:len(perm)] = perm
    return lens, table, held, stack, len(perm), shared


# ------------------------------------------------------------------ forks
def _fork(parent, child, lens, table, held, stack, count, shared, page, in_place):
    t, h, f, c, s = _i32(table), _i32(held), _i32(stack), _i32([count]), _i32(shared)
    kw = {} if in_place else dict(held_out=torch.empty_like(h), free_count_out=torch.empty_like(c),
                                  shared_out=torch.empty_like(s))
    src, dst, info = B.ga_page_fork(_i32(parent), _i32(child), _i32(lens), t, h, f, c, s, page, **kw)
    if not in_place:
        _same((h, c, s), (held, [count], shared), "inputs")
    _same((f,), (stack,), "stack")
    return (t, kw.get("held_out", h), kw.get("free_count_out", c), kw.get("shared_out", s), src, dst, info)


@pytest.mark.parametrize("n,forks,page,width,max_len,share", [
    (2, 1, 32, 4, 100, 0), (5, 3, 1, 9, 9, 0.5), (40, 30, 64, 33, 2000, 0.5), (300, 299, 32, 20, 600, 0.3),
    (2048, 2047, 16, 5, 80, 0.5), (64, 63, 32, 1500, 48000, 0.2)])
def test_fork_matches_oracle(n, forks, page, width, max_len, share):
    rng = np.random.default_rng(SEED + n)
    lens, table, held, stack, count, shared = _state(rng, n, width, max_len, page, forks + 2, share)
    children = [int(b) for b in rng.permutation(n)[:forks] if rng.random() < 0.9 or n < 5]
    for c in children:   # empty rows, and their pages on the stack
        back = [x for x in table[c, :held[c]]]
        for x in back:
            if shared[x]:
                shared[x] -= 1
            else:
                stack[count] = x
                count += 1
        held[c] = 0
    parents = [b for b in range(n) if b not in set(children)] or [children.pop()]
    parent = [int(parents[rng.integers(len(parents))]) if rng.random() < 0.95 else -1 for _ in children]
    want_len = [int(rng.integers(0, held[p] * page + 1)) if p >= 0 else 5 for p in parent]
    for i in range(0, len(parent), 4):
        want_len[i] -= want_len[i] % page
    want = O.page_fork(parent, children, want_len, table, held, stack, count, shared, page)
    assert want[-1][0] == 0
    for in_place in (False, True):
        _same(_fork(parent, children, want_len, table, held, stack, count, shared, page, in_place), want)


FORK = dict(parent=[0, 0], child=[1, 2], lens=[70, 64], held=[3, 0, 0, 1], count=3)
FORK_FAULTS = [
    (dict(parent=[4, 0]), 1), (dict(child=[1, -1]), 1), (dict(child=[1, 4]), 1), (dict(child=[0, 2]), 1),
    (dict(child=[2, 2]), 1), (dict(child=[3, 2]), 1), (dict(lens=[97, 0]), 2), (dict(lens=[-1, 0]), 2),
    (dict(parent=[1, 0], child=[2, 1], lens=[1, 0]), 2), (dict(count=0), 3), (dict(count=9), 4),
    (dict(count=-1), 4), (dict(held=[3, 0, 0, 5]), 4), (dict(held=[-1, 0, 0, 1]), 4),
    (dict(child=[2, 2], count=0), 1), (dict(lens=[97, 1], count=0), 2), (dict(lens=[97, 1], count=-3), 4),
    (dict(child=[2, 2], lens=[97, 1]), 1), (dict(child=[2, 2], held=[3, 0, 0, 5]), 4)]


@pytest.mark.parametrize("pad", [0, 2000])
def test_fork_refuses_on_the_device(pad):
    table = np.pad(np.array([[4, 2, 6], [-1] * 3, [-1] * 3, [5, -1, -1]]), ((0, 0), (0, pad)), constant_values=-1)
    stack, shared = np.array([0, 1, 3, 0, 0, 0, 0]), np.arange(7)
    for change, status in FORK_FAULTS:
        a = {**FORK, **change}
        if pad and a["held"][3] == 5:
            a["held"] = [3, 0, 0, 3 + pad + 1]
        want = O.page_fork(a["parent"], a["child"], a["lens"], table, a["held"], stack, a["count"], shared, 32)
        assert want[-1][0] == status
        for in_place in (False, True):
            _same(_fork(a["parent"], a["child"], a["lens"], table, a["held"], stack, a["count"], shared, 32,
                        in_place), want, change)


def test_fork_passes_over_entries_outside_the_pool():
    table = np.array([[4, 9, -5, -1], [-1] * 4])
    got = _fork([0], [1], [80], table, [3, 0], np.array([0, 1, 3, 0, 0, 0]), 3, np.zeros(6), 32, True)
    assert B.ga_device_status() == 3
    t, h, c, s, src, dst, info = got
    assert t[1].tolist() == [4, 9, 3, -1] and h.tolist() == [3, 3] and c.tolist() == [2]
    assert s.tolist() == [0, 0, 0, 0, 1, 0] and src.tolist() == dst.tolist() == [-1]


# ------------------------------------------------------------------ pages given back
def _release(keep, table, held, stack, count, shared, page, in_place):
    t, h, f, c, s = _i32(table), _i32(held), _i32(stack), _i32([count]), _i32(shared)
    kw = {} if in_place else dict(held_out=torch.empty_like(h), free_count_out=torch.empty_like(c),
                                  shared_out=torch.empty_like(s))
    info = B.ga_page_release(_i32(keep), t, h, f, c, s, page, **kw)
    if not in_place:
        _same((h, c, s), (held, [count], shared), "inputs")
    _same((t,), (table,), "table")
    return kw.get("held_out", h), f, kw.get("free_count_out", c), kw.get("shared_out", s), info


@pytest.mark.parametrize("n,page,width,max_len,share", [
    (1, 32, 4, 100, 0), (5, 1, 9, 9, 0.5), (40, 64, 33, 2000, 0.7), (300, 32, 20, 600, 0.9),
    (2048, 16, 5, 80, 0.5), (64, 32, 1500, 48000, 0.5), (700, 16, 100, 1600, 0.9)])
def test_release_matches_oracle(n, page, width, max_len, share):
    rng = np.random.default_rng(SEED + n)
    for part in (0.2, 0.6, 1.1):
        lens, table, held, stack, count, shared = _state(rng, n, width, max_len, page, 3, share)
        keep = [int(rng.choice([0, 0, 2 ** 31 - 1, rng.integers(0, max_len + 1)])) if rng.random() < part else -1
                for _ in range(n)]
        want = O.page_release(keep, table, held, stack, count, shared, page)
        assert want[-1][0] == 0
        for in_place in (False, True):
            _same(_release(keep, table, held, stack, count, shared, page, in_place), want)


@pytest.mark.parametrize("pad", [0, 3000])
def test_release_refuses_on_the_device(pad):
    table = np.pad(np.array([[4, 2, 6], [4, 2, -1], [5, 0, 1]]), ((0, 0), (0, pad)), constant_values=-1)
    held, stack, shared = np.array([3, 2, 1]), np.array([3, 0, 0, 0, 0, 0, 0]), np.array([0, 0, 1, 0, 1, 0, 0])
    cases = [(dict(), 0), (dict(count=8), 4), (dict(count=-1), 4), (dict(held=[3, -1, 1]), 4),
             (dict(held=[3, 2, 4 + pad]), 4), (dict(count=4), 4), (dict(shared=[0] * 7), 5),
             (dict(shared=[0, 0, 1, 0, 0, 0, 0], count=7), 5), (dict(shared=[0, 0, -1, 0, 1, 0, -2 ** 31]), 5),
             (dict(shared=[0] * 7, held=[3, 2, -1]), 4)]
    for change, status in cases:
        a = {**dict(held=held, count=1, shared=shared), **change}
        keep = [0, 0, 0]
        want = O.page_release(keep, table, a["held"], stack, a["count"], a["shared"], 32)
        assert want[-1][0] == status, change
        for in_place in (False, True):
            _same(_release(keep, table, a["held"], stack, a["count"], a["shared"], 32, in_place), want, change)


def test_release_passes_over_entries_outside_the_pool():
    h, f, c, s, info = _release([0, 0], np.array([[4, 9, -5], [1, -1, -1]]), [3, 1], np.array([0, 2, 0, 0, 0]), 2,
                                np.zeros(5), 32, True)
    assert B.ga_device_status() == 3
    assert h.tolist() == [0, 0] and c.tolist() == [4] and f.tolist() == [0, 2, 4, 1, 0]
    assert info.tolist() == [0, 2, 2, 4] and not s.any()


# ------------------------------------------------------------------ compaction
def _compact(table, held, stack, count, shared, moves, in_place):
    t, h, f, c, s = _i32(table), _i32(held), _i32(stack), _i32([count]), _i32(shared)
    kw = {} if in_place else dict(page_table_out=torch.empty_like(t), free_pages_out=torch.empty_like(f),
                                  shared_out=torch.empty_like(s))
    src, dst, info = B.ga_page_compact(t, h, f, c, s, moves, **kw)
    if not in_place:
        _same((t, f, s), (table, stack, shared), "inputs")
    _same((h, c), (held, [count]), "lengths")
    return (kw.get("page_table_out", t), kw.get("free_pages_out", f), kw.get("shared_out", s), src, dst, info)


@pytest.mark.parametrize("n,width,max_len,page,spare", [
    (1, 4, 100, 32, 3), (5, 9, 9, 1, 0), (40, 33, 2000, 64, 900), (300, 20, 600, 32, 3000),
    (2048, 40, 80, 16, 5000), (64, 1500, 48000, 32, 70000), (3, 2, 0, 32, 40)])
def test_compact_matches_oracle(n, width, max_len, page, spare):
    rng = np.random.default_rng(SEED + n)
    lens, table, held, stack, count, shared = _state(rng, n, width, max_len, page, spare, 0.4)
    for moves in (0, 1, 7, len(stack)):
        want = O.page_compact(table, held, stack, count, shared, moves)
        assert want[-1][0] == 0
        for in_place in (False, True):
            _same(_compact(table, held, stack, count, shared, moves, in_place), want)


@pytest.mark.parametrize("pad", [0, 5000])
def test_compact_refuses_on_the_device(pad):
    table, held = np.array([[4, 2, 6], [4, -1, -1]]), np.array([3, 1])
    stack = np.concatenate([[0, 1, 3, 5], np.arange(7, 7 + pad), [0, 0, 0]])
    count = 4 + pad
    shared = np.arange(len(stack)) % 3
    for change in (dict(count=-1), dict(count=len(stack) + 1), dict(held=[4, 1]), dict(held=[3, -1]),
                   dict(at=(2, 1)), dict(at=(0, len(stack))), dict(at=(3, -1))):
        f = stack.copy()
        if "at" in change:
            f[change["at"][0]] = change["at"][1]
        a = {**dict(held=held, count=count), **change}
        want = O.page_compact(table, a["held"], f, a["count"], shared, 5)
        assert want[-1][0] == 4
        for in_place in (False, True):
            _same(_compact(table, a["held"], f, a["count"], shared, 5, in_place), want, change)


# ------------------------------------------------------------------ copies
@pytest.mark.parametrize("sizes", [[1], [16, 2], [4096, 1, 6, 2048], [40000, 8, 65536, 12, 3], [24576, 16384]])
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_copy_moves_whole_pages_only(sizes, offset):
    rng = np.random.default_rng(SEED + len(sizes) + offset)
    n = 37
    raw = [torch.randint(0, 256, (n * s + 32,), dtype=torch.uint8, device="cuda") for s in sizes]
    pools = [x[offset:offset + n * s].view(n, s) for x, s in zip(raw, sizes)]
    order = rng.permutation(n)
    src = np.concatenate([order[:6], order[:3], [-1, 2, -2], [order[0]]])   # some read more than once
    dst = np.concatenate([order[10:16], order[20:23], [1, -1, -3], [order[30]]])
    want = [x.clone() for x in raw]
    for x, s in zip(want, sizes):
        p = x[offset:offset + n * s].view(n, s)
        for a, b in zip(src, dst):
            if a >= 0 and b >= 0:
                p[int(b)] = p[int(a)]
    B.ga_page_copy(pools, _i32(src), _i32(dst))
    assert all(torch.equal(a, b) for a, b in zip(raw, want))


def test_copy_records_pages_outside_the_pool():
    x = torch.arange(40, dtype=torch.int32, device="cuda").view(5, 8)
    B.ga_page_copy([x], _i32([5, 0, 2 ** 31 - 1]), _i32([1, 3, 4]))
    assert B.ga_device_status() == 3
    assert x[3].tolist() == x[0].tolist() == list(range(8)) and x[1, 0].item() == 8 and x[4, 0].item() == 32
    B.ga_page_copy([x], _i32([0]), _i32([5]))
    assert B.ga_device_status() == 3


def test_copy_many_pages_of_several_pools():
    n, m = 3000, 1400
    pools = [torch.randint(0, 255, (n, 2, 64, w), dtype=torch.uint8, device="cuda") for w in (256, 128, 16)]
    pools.append(torch.randn(n, 64, 2, 3, device="cuda"))
    perm = torch.randperm(n, device="cuda").to(torch.int32)
    src, dst = perm[:m].contiguous(), perm[m:2 * m].contiguous()
    want = [x.clone() for x in pools]
    for x in want:
        x[dst.long()] = x[src.long()]
    B.ga_page_copy(pools, src, dst)
    assert all(torch.equal(a, b) for a, b in zip(pools, want))


# ------------------------------------------------------------------ a server's steps
class Server:
    """Branches over an 8-bit cache, with the tokens of every row kept beside it in bf16 as stored."""

    def __init__(self, n, page, width, pool, seed):
        self.n, self.page = n, page
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(SEED + seed)
        u8 = lambda *s: torch.full(s, 0x7F, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.pools = [u8(pool, 2, page, 256), u8(pool, 2, page // 32), u8(pool, 2, page, 256), u8(pool, 2, page // 32)]
        self.table, self.held = _i32(np.full((n, width), -1)), _i32([0] * n)
        self.free, self.count = _i32(np.random.default_rng(seed).permutation(pool)), _i32([pool])
        self.shared, self.lens = _i32([0] * pool), [-1] * n
        self.out = torch.zeros(n, 2, 6144, dtype=torch.bfloat16, device="cuda")

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda").to(torch.bfloat16)

    def widened(self, b):
        t = torch.arange(self.lens[b], device="cuda")
        slots = self.table[b].long()[t // self.page] * self.page + t % self.page
        return B.ga_kv_dequantize_q8(*self.pools, slots=slots.to(torch.int32))

    def append(self, new):
        """new[b] tokens to row b (0 to a row in no use)."""
        total = sum(new)
        _, slots, _, info = B.ga_page_plan(_i32(self.lens), _i32(new), self.table, self.held, self.free,
                                           self.count, self.page, total)
        assert info[0].item() == 0
        B.ga_kv_quantize_q8(self.normal(total, 2, 256), self.normal(total, 2, 256), *self.pools, slots=slots)
        self.lens = [x + a if x >= 0 else x for x, a in zip(self.lens, new)]

    def fork(self, parent, child, lens):
        src, dst, info = B.ga_page_fork(_i32(parent), _i32(child), _i32(lens), self.table, self.held, self.free,
                                        self.count, self.shared, self.page)
        assert info[0].item() == 0
        B.ga_page_copy(self.pools, src, dst)
        for p, c, x in zip(parent, child, lens):
            if p >= 0:
                self.lens[c] = x

    def release(self, keep):
        info = B.ga_page_release(_i32(keep), self.table, self.held, self.free, self.count, self.shared, self.page)
        assert info[0].item() == 0
        self.lens = [x if k < 0 else -1 if k == 0 else min(x, k) for x, k in zip(self.lens, keep)]

    def compact(self, moves):
        src, dst, info = B.ga_page_compact(self.table, self.held, self.free, self.count, self.shared, moves)
        assert info[0].item() == 0
        B.ga_page_copy(self.pools, src, dst)
        return info.tolist()

    def attend(self):
        """A window of two rows over every row's last two tokens."""
        q, qg = self.normal(self.n, 2, 24, 256), self.normal(self.n, 2, 24, 512)
        out = B.ga_attn_verify_q8(q, qg, *self.pools, self.table, _i32([x - 2 if x >= 2 else -1 for x in self.lens]))
        for b, x in enumerate(self.lens):
            if x < 2:
                continue
            k, v = self.widened(b)
            for kv in range(2):
                hs = slice(12 * kv, 12 * kv + 12)
                want = attend64(q[b, :, hs], qg[b, :, hs, 256:], k[:, kv], v[:, kv], [x - 1, x])
                got = out[b].view(2, 24, 256)[:, hs]
                assert float(row_errors(got, want).max()) <= (ROW_BOUND if x > 60 else 3 * ROW_BOUND)

    def check(self):
        """Every page has as many holders as it should; the rest are on the stack once."""
        table, held, count = self.table.cpu().numpy(), self.held.tolist(), self.count.item()
        holders = np.zeros(self.free.numel(), np.int64)
        for b in range(self.n):
            np.add.at(holders, table[b, :held[b]], 1)
        stack = self.free.cpu().numpy()[:count]
        assert len(set(stack)) == count and not holders[stack].any() and (holders > 0).sum() + count == len(holders)
        assert np.array_equal(self.shared.cpu().numpy(), np.maximum(holders - 1, 0))


@pytest.mark.parametrize("page", [32, 96])
def test_branches_of_a_server(page):
    """Prompts, branches at whole and begun pages, tokens to all branches (each to its own pages), rows
    cut back and finished, the pool packed, and on: what each row holds stays what was stored."""
    s = Server(8, page, 30, 100, page)
    s.lens[0] = s.lens[1] = 0
    s.append([700, 333, 0, 0, 0, 0, 0, 0])
    prompt = [x.clone() for x in s.widened(0)]
    s.fork([0, 0, 1, -1], [2, 3, 4, 7], [700, 2 * page, 333, 9])
    s.check()
    for _ in range(3):
        s.append([1, 2, 3, 5, 1, 0, 0, 0])
        s.attend()
    for b, n in ((0, 700), (2, 700), (3, 2 * page)):
        k, v = s.widened(b)
        # a block that went on may have grown; the rest are the prompt's, bit for bit
        n -= n % 32
        assert torch.equal(k[:n], prompt[0][:n]) and torch.equal(v[:n], prompt[1][:n])
    before = {b: [x.clone() for x in s.widened(b)] for b in (1, 3, 4)}
    s.release([0, -1, 0, -1, 330, -1, -1, -1])
    s.check()
    info = s.compact(3)
    while info[3]:
        s.check()
        info = s.compact(3)
    s.check()
    assert s.table[:, :1][s.held > 0].max().item() < info[2]
    for b, (k, v) in before.items():
        x = s.widened(b)
        assert torch.equal(x[0], k[:s.lens[b]]) and torch.equal(x[1], v[:s.lens[b]])
    s.lens[5] = 0
    s.fork([3, 3], [0, 6], [s.lens[3], 70])
    s.append([40, 1, 0, 30, 7, 500, 1, 0])
    s.attend()
    s.check()
    s.release([0] * 8)
    assert s.count.item() == 100 and not s.shared.any()


def test_captured_steps_of_branches():
    """Fork, copy, plan, store, attention, release and compaction captured once and replayed with other
    rows, lengths and forks; the state is the same as by plain calls."""
    def make():
        s = Server(6, 32, 12, 60, 5)
        s.lens[0], s.lens[1] = 0, 0
        s.append([150, 77, 0, 0, 0, 0])
        return s

    plain, graph_side = make(), make()
    io = dict(parent=_i32([-1] * 3), child=_i32([0] * 3), flen=_i32([0] * 3), lens=_i32([-1] * 6), alens=_i32([-1] * 6), new=_i32([0] * 6),
              keep=_i32([-1] * 6), k=plain.normal(24, 2, 256), v=plain.normal(24, 2, 256),
              q=plain.normal(6, 1, 24, 256), qg=plain.normal(6, 1, 24, 512))
    ws = torch.empty(B.ga_verify_q8_workspace_bytes(), dtype=torch.uint8, device="cuda")
    wc = torch.empty(B.ga_page_compact_workspace_bytes(60), dtype=torch.uint8, device="cuda")

    def step(s):
        src, dst, i0 = B.ga_page_fork(io["parent"], io["child"], io["flen"], s.table, s.held, s.free, s.count,
                                      s.shared, 32)
        B.ga_page_copy(s.pools, src, dst)
        _, slots, _, i1 = B.ga_page_plan(io["lens"], io["new"], s.table, s.held, s.free, s.count, 32, 24)
        B.ga_kv_quantize_q8(io["k"], io["v"], *s.pools, slots=slots)
        B.ga_attn_verify_q8(io["q"], io["qg"], *s.pools, s.table, io["alens"], out=s.out[:, :1].contiguous(),
                            workspace=ws)
        i2 = B.ga_page_release(io["keep"], s.table, s.held, s.free, s.count, s.shared, 32)
        src, dst, i3 = B.ga_page_compact(s.table, s.held, s.free, s.count, s.shared, 4, workspace=wc)
        B.ga_page_copy(s.pools, src, dst)
        return torch.stack([i0, i1, i2, i3])

    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step(make())
    torch.cuda.current_stream().wait_stream(warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        infos = step(graph_side)
    lens = [150, 77, -1, -1, -1, -1]
    moves = [(dict(parent=[0, 0, 1], child=[2, 3, 4], flen=[150, 96, 70]), [1, 2, 0, 4, 5, 0], [-1] * 6),
             (dict(parent=[-1, 2, -1], child=[0, 5, 0], flen=[0, 120, 0]), [3, 3, 3, 3, 3, 3], [0, -1, -1, 64, -1, -1]),
             (dict(parent=[3, -1, -1], child=[0, 0, 0], flen=[32, 0, 0]), [1, 1, 1, 1, 1, 1], [-1, 0, 0, -1, 64, -1]),
             (dict(parent=[-1] * 3, child=[0] * 3, flen=[0] * 3), [0] * 6, [0] * 6)]
    for forks, new, keep in moves:
        for c, p, x in zip(forks["child"], forks["parent"], forks["flen"]):
            if p >= 0:
                lens[c] = x
        new = [a if x >= 0 else 0 for a, x in zip(new, lens)]
        alens = [x if a else -1 for a, x in zip(new, lens)]
        for name, x in dict(forks, lens=lens, alens=alens, new=new, keep=keep).items():
            io[name].copy_(_i32(x))
        for name in ("k", "v", "q", "qg"):
            io[name].copy_(plain.normal(*io[name].shape))
        graph.replay()
        want = step(plain)
        assert torch.equal(infos, want) and not want[:, 0].any()
        for a, b in zip((graph_side.table, graph_side.held, graph_side.count, graph_side.shared, *graph_side.pools),
                        (plain.table, plain.held, plain.count, plain.shared, *plain.pools)):
            assert torch.equal(a, b)
        lens = [x + a if x >= 0 else x for x, a in zip(lens, new)]
        lens = [x if k < 0 else -1 if k == 0 else min(x, k) for x, k in zip(lens, keep)]
        for s in (plain, graph_side):
            s.lens = list(lens)
            s.check()


def test_calls_on_two_streams():
    """Two servers of their own, each on a stream, at once."""
    servers = [Server(8, 32, 20, 120, i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, st in zip(servers, streams):
            with torch.cuda.stream(st):
                s.lens[0] = 0
                s.append([300] + [0] * 7)
                s.fork([0] * 3, [1, 2, 3], [300, 64, 100])
                s.append([1, 40, 1, 1, 0, 0, 0, 0])
                s.attend()
                s.release([0, 0, -1, 50] + [-1] * 4)
                s.compact(50)
                s.release([0] * 8)
    for s in servers:
        s.check()
        assert s.count.item() == 120


def test_empty_calls():
    e, one = _i32([]), _i32([2])
    t = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    src, dst, info = B.ga_page_fork(e, e, e, t, e, _i32([0, 1]), one, _i32([0, 0]), 32)
    assert src.numel() == 0 and info.tolist() == [0] * 4 and one.item() == 2
    assert B.ga_page_release(e, t, e, _i32([0, 1]), one, _i32([0, 0]), 32).tolist() == [0] * 4
    src, dst, info = B.ga_page_compact(t, e, _i32([0, 1]), one, _i32([0, 0]), 3)
    assert info.tolist() == [0] * 4 and src.tolist() == dst.tolist() == [-1] * 3
    z = _i32([0])
    src, dst, info = B.ga_page_compact(t, e, e, z, e, 0)
    assert info.tolist() == [0] * 4 and src.numel() == 0
    x = torch.ones(4, 8, device="cuda")
    B.ga_page_copy([x], e, e)
    B.ga_page_copy([x[:0]], _i32([1]), _i32([2]))
