"""The 8-bit paged serving calls and the calls over pages without a GPU: refusals make no CUDA call,
the binding refuses tensors that do not belong together, and the oracle holds by closed forms."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import ga_oracle as O
from verify_gated_gqa_gb300 import binding as B
from verify_gated_gqa_gb300 import build as build_mod

A = 0x10000        # an aligned fake device address (never dereferenced)
MIS = 0x10002


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return B.lib()


def _refused(L, call, want):
    before = L.ga_debug_cuda_calls()
    assert call() == want
    assert L.ga_debug_cuda_calls() == before


# ------------------------------------------------------------------ refusals: rows and attention
def _store(L, **kw):
    a = dict(k=A, ldk=512, v=A, ldv=1024, n=8, slots=A, kc=A, ks=A, vc=A, vs=A, pages=4, page=64)
    a.update(kw)
    return L.ga_kv_quantize_q8(a["k"], a["ldk"], a["v"], a["ldv"], a["n"], a["slots"], a["kc"],
                               a["ks"], a["vc"], a["vs"], a["pages"], a["page"], None)


def _load(L, **kw):
    a = dict(kc=A, ks=A, vc=A, vs=A, pages=4, page=64, slots=A, n=8, k=A, v=A)
    a.update(kw)
    return L.ga_kv_dequantize_q8(a["kc"], a["ks"], a["vc"], a["vs"], a["pages"], a["page"],
                                 a["slots"], a["n"], a["k"], a["v"], None)


POOL_REFUSALS = [
    *[({k: None}, -1) for k in ("k", "v", "kc", "ks", "vc", "vs")],
    (dict(pages=0), -2), (dict(page=0), -2), (dict(n=-1), -2),
    (dict(page=48), -4), (dict(page=1 << 21), -4), (dict(pages=1 << 24), -4),
    (dict(n=(64 << 20) + 1), -4), (dict(slots=None, n=257), -4),
    (dict(slots=MIS), -3), (dict(k=MIS), -3), (dict(v=MIS), -3), (dict(kc=MIS), -3), (dict(vc=MIS), -3),
    (dict(n=0), 0), (dict(n=0, slots=None), 0), (dict(n=0, ks=MIS + 1, vs=MIS + 1), 0),
]


@pytest.mark.parametrize("kw,want", POOL_REFUSALS + [
    (dict(ldk=504), -4), (dict(ldv=0), -4), (dict(ldk=516), -3), (dict(ldv=1028), -3)])
def test_quantize_q8_refusals(L, kw, want):
    _refused(L, lambda: _store(L, **kw), want)


@pytest.mark.parametrize("kw,want", POOL_REFUSALS)
def test_dequantize_q8_refusals(L, kw, want):
    _refused(L, lambda: _load(L, **kw), want)


def _attn(L, **kw):
    a = dict(q=A, qg=A, kc=A, ks=A, vc=A, vs=A, pages=4, page=64, table=A, width=2, lens=A, n=2,
             rows=4, out=A, ws=0x100000, wsb=L.ga_verify_q8_workspace_bytes())
    a.update(kw)
    return L.ga_attn_verify_q8(a["q"], a["qg"], a["kc"], a["ks"], a["vc"], a["vs"], a["pages"],
                               a["page"], a["table"], a["width"], a["lens"], a["n"], a["rows"],
                               a["out"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,want", [
    *[({k: None}, -1) for k in ("q", "qg", "kc", "ks", "vc", "vs", "table", "lens", "out")],
    (dict(n=-1), -2), (dict(rows=-1), -2), (dict(width=0), -2), (dict(pages=0), -2),
    (dict(rows=17), -4), (dict(page=16), -4), (dict(page=100), -4), (dict(pages=1 << 24), -4),
    (dict(n=(1 << 20) + 1), -4),
    (dict(q=MIS), -3), (dict(qg=MIS), -3), (dict(kc=MIS), -3), (dict(out=MIS), -3),
    (dict(table=MIS), -3), (dict(lens=MIS), -3),
    (dict(ws=None), -6), (dict(wsb=1000), -6), (dict(ws=0x100010), -6),
    (dict(n=0), 0), (dict(rows=0), 0),
])
def test_verify_q8_refusals(L, kw, want):
    _refused(L, lambda: _attn(L, **kw), want)


# ------------------------------------------------------------------ refusals: pages
FORK = ("parent", "child", "len", "table", "held", "ho", "free", "fc", "fco", "sh", "sho", "src", "dst", "info")


def _fork(L, **kw):
    a = dict(dict.fromkeys(FORK, A), m=3, n=4, page=64, width=8, nf=100)
    a.update(kw)
    return L.ga_page_fork(a["parent"], a["child"], a["len"], a["m"], a["n"], a["page"], a["table"],
                          a["width"], a["held"], a["ho"], a["free"], a["nf"], a["fc"], a["fco"], a["sh"],
                          a["sho"], a["src"], a["dst"], a["info"], None)


SIZES = [(dict(n=-1), -2), (dict(width=0), -2), (dict(nf=-1), -2), (dict(n=2049), -4),
         (dict(n=2048, width=1 << 20), -4), (dict(nf=1 << 30), -4)]
PAGED = SIZES + [(dict(page=0), -2), (dict(page=1 << 16, width=1 << 15), -4), (dict(nf=1 << 26), -4)]


@pytest.mark.parametrize("kw,want", PAGED + [(dict(m=-1), -2), (dict(m=2049), -4)]
                         + [({k: None}, -1) for k in FORK] + [({k: MIS}, -3) for k in FORK])
def test_fork_refusals(L, kw, want):
    _refused(L, lambda: _fork(L, **kw), want)


RELEASE = ("keep", "table", "held", "ho", "free", "fc", "fco", "sh", "sho", "info")


def _release(L, **kw):
    a = dict(dict.fromkeys(RELEASE, A), n=4, page=64, width=8, nf=100)
    a.update(kw)
    return L.ga_page_release(a["keep"], a["n"], a["page"], a["table"], a["width"], a["held"], a["ho"],
                             a["free"], a["nf"], a["fc"], a["fco"], a["sh"], a["sho"], a["info"], None)


@pytest.mark.parametrize("kw,want", PAGED + [({k: None}, -1) for k in RELEASE]
                         + [({k: MIS}, -3) for k in RELEASE])
def test_release_refusals(L, kw, want):
    _refused(L, lambda: _release(L, **kw), want)


COMPACT = ("table", "to", "held", "free", "fo", "fc", "sh", "sho", "src", "dst", "info")


def _compact(L, **kw):
    a = dict(dict.fromkeys(COMPACT, A), n=4, width=8, nf=100, moves=7, ws=A,
             wsb=L.ga_page_compact_workspace_bytes(100))
    a.update(kw)
    return L.ga_page_compact(a["n"], a["table"], a["to"], a["width"], a["held"], a["free"], a["fo"], a["nf"],
                             a["fc"], a["sh"], a["sho"], a["moves"], a["src"], a["dst"], a["info"], a["ws"],
                             a["wsb"], None)


@pytest.mark.parametrize("kw,want", SIZES + [(dict(moves=-1), -2), (dict(ws=None), -6), (dict(ws=MIS), -6),
                                             (dict(wsb=399), -6)]
                         + [({k: None}, -1) for k in COMPACT] + [({k: MIS}, -3) for k in COMPACT])
def test_compact_refusals(L, kw, want):
    _refused(L, lambda: _compact(L, **kw), want)


def test_compact_workspace(L):
    assert L.ga_page_compact_workspace_bytes(-1) == 0 == L.ga_page_compact_workspace_bytes(0)
    assert all(4 * n <= L.ga_page_compact_workspace_bytes(n) < 4 * n + 256 for n in (1, 63, 64, 65, (1 << 30) - 1))


def _copy(L, **kw):
    a = dict(pools=[A, A], bytes=[64, 2], n=None, pages=4, src=A, dst=A, m=3)
    a.update(kw)
    k = len(a["pools"]) if a["pools"] else 1
    pools = (ctypes.c_void_p * k)(*a["pools"]) if a["pools"] else None
    sizes = (ctypes.c_size_t * max(1, len(a["bytes"])))(*a["bytes"]) if a["bytes"] else None
    return L.ga_page_copy(pools, sizes, k if a["n"] is None else a["n"], a["pages"], a["src"], a["dst"],
                          a["m"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(pools=None), -1), (dict(bytes=None), -1), (dict(pools=[A, None]), -1), (dict(src=None), -1),
    (dict(dst=None), -1), (dict(n=0), -2), (dict(pages=-1), -2), (dict(m=-1), -2), (dict(bytes=[64, 0]), -2),
    (dict(pools=[A] * 17, bytes=[64] * 17), -4), (dict(bytes=[64, (1 << 30) + 1]), -4), (dict(m=1 << 30), -4),
    (dict(src=MIS), -3), (dict(dst=MIS), -3), (dict(m=0), 0), (dict(pages=0), 0)])
def test_copy_refusals(L, kw, want):
    _refused(L, lambda: _copy(L, **kw), want)


def test_binding_refuses_host_tensors():
    c = torch.zeros(2, 2, 32, 256, dtype=torch.uint8)
    s = torch.zeros(2, 2, 1, dtype=torch.uint8)
    x = torch.zeros(4, 2, 256, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    calls = [lambda: B.ga_kv_quantize_q8(x, x, c, s, c, s), lambda: B.ga_kv_dequantize_q8(c, s, c, s),
             lambda: B.ga_attn_verify_q8(x[:, None], x[:, None], c, s, c, s, i[:, None], i),
             lambda: B.ga_page_fork(i, i, i, i[:, None], i, i, i[:1], i, 32),
             lambda: B.ga_page_release(i, i[:, None], i, i, i[:1], i, 32),
             lambda: B.ga_page_compact(i[:, None], i, i, i[:1], i, 4), lambda: B.ga_page_copy([c, s], i, i)]
    for call in calls:
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ the oracle's own pins
def test_q8_exponents():
    e = np.arange(-32, 32)
    assert np.array_equal(O.q8_exponent(448 * 2.0 ** e), e)
    assert np.array_equal(O.q8_exponent(450 * 2.0 ** e), np.minimum(e + 1, 31))
    assert O.q8_exponent(0) == O.q8_exponent(2.0 ** -100) == -32 and O.q8_exponent(np.inf) == 31


def test_q8_codes_name_their_values():
    """All 254 finite codes, and that the two roads to bytes and values agree."""
    c = np.array([x for x in range(256) if x & 127 != 127])
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 512, (1 + m / 8) * 2.0 ** (e - 7)) * np.where(c >= 128, -1.0, 1.0)
    assert np.array_equal(O.e4m3_codes(v), c.astype(np.uint8))
    assert np.array_equal(O.e4m3_sat(v), v) and np.abs(v).max() == 448
    assert O.e4m3_sat(np.nan) == 0 and O.e4m3_sat(1e9) == 448 and O.e4m3_sat(-np.inf) == -448


def test_q8_store_grows_and_keeps():
    """Earlier rows move by powers of two exactly while their codes stay normal."""
    values, exps = np.zeros((64, 256)), np.full(2, -32)
    rows = np.zeros((3, 256))
    rows[0, :3] = [448, 7, 2.0 ** -6]
    rows[1, 0] = 896
    rows[2, 0] = 1
    O.q8_store(values, exps, rows[:1], [32])
    assert exps.tolist() == [-32, 0]
    O.q8_store(values, exps, rows[1:2], [33])
    assert exps[1] == 1 and values[32, :3].tolist() == [224, 3.5, 2.0 ** -7]
    assert np.array_equal(O.q8_widen(values, exps, [32, 33]), rows[:2])
    O.q8_store(values, exps, rows[2:], [34])         # a smaller row does not shrink it
    assert exps[1] == 1 and O.q8_widen(values, exps, [34])[0, 0] == 1
    O.q8_store(values, exps, rows[2:], [32])         # its first slot again: the block begins anew
    assert exps[1] == -8 and values[33, 0] == 448


def test_fork_release_compact_small():
    table = np.array([[4, 2, 7, -1], [-1] * 4, [-1] * 4])
    t, h, count, shared, src, dst, info = O.page_fork([0, -1, 0], [2, 0, 1], [40, 0, 64], table, [3, 0, 0],
                                                      [0, 1, 3, 5, 6, 0, 0, 0], 5, [0] * 8, 32)
    assert t.tolist() == [[4, 2, 7, -1], [4, 2, -1, -1], [4, 6, -1, -1]] and h.tolist() == [3, 2, 2]
    assert count == 4 and src.tolist() == [2, -1, -1] and dst.tolist() == [6, -1, -1]
    assert shared.tolist() == [0, 0, 1, 0, 2, 0, 0, 0] and info.tolist() == [0, 2, 1, 3]
    h, stack, count, shared, info = O.page_release([0, -1, 32], t, h, [0, 1, 3, 5, 0, 0, 0, 0], count, shared, 32)
    assert h.tolist() == [0, 2, 1] and info.tolist() == [0, 2, 2, 4]
    assert stack[:6].tolist() == [0, 1, 3, 5, 7, 6] and shared.tolist() == [0, 0, 0, 0, 1, 0, 0, 0]
    t, stack, shared, src, dst, info = O.page_compact(t, h, stack, count, shared, 1)
    assert src.tolist() == [4] and dst.tolist() == [0] and info.tolist() == [0, 1, 2, 1]
    assert t[1, :2].tolist() == [0, 2] and t[2, 0] == 0 and shared[0] == 1
    assert stack[:count].tolist() == [7, 6, 5, 4, 3, 1]
