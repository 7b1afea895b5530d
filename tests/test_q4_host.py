"""The 4-bit paged serving calls without a GPU: their refusals make no CUDA call, the binding
refuses tensors that do not belong together, and the oracle's 4-bit format and step plan hold
by closed forms."""
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


# ------------------------------------------------------------------ refusals
def _plan(L, **kw):
    a = dict(len=A, new=A, n=4, page=64, table=A, width=8, held=A, ho=A, free=A, nf=100, fc=A, fco=A,
             delta=None, mt=64, rs=A, sm=A, pos=A, info=A)
    a.update(kw)
    return L.ga_page_plan(a["len"], a["new"], a["n"], a["page"], a["table"], a["width"], a["held"],
                          a["ho"], a["free"], a["nf"], a["fc"], a["fco"], a["delta"], a["mt"],
                          a["rs"], a["sm"], a["pos"], a["info"], None)


@pytest.mark.parametrize("kw,want", [
    *[({k: None}, -1) for k in ("len", "new", "table", "held", "ho", "free", "fc", "fco", "rs", "sm",
                                "info")],
    (dict(n=-1), -2), (dict(page=0), -2), (dict(width=0), -2), (dict(nf=-1), -2), (dict(mt=-1), -2),
    (dict(n=2049), -4), (dict(page=1 << 16, width=1 << 15), -4), (dict(nf=1 << 26), -4),
    (dict(mt=1 << 30), -4),
    (dict(len=MIS), -3), (dict(delta=MIS), -3), (dict(pos=MIS), -3), (dict(info=MIS), -3),
])
def test_plan_refusals(L, kw, want):
    _refused(L, lambda: _plan(L, **kw), want)


def _axes(L, **kw):
    a = dict(k=A, wk=A, kp=A, q=A, wq=A, qp=A, n=8, pos=A, ld=8, na=3, ax=[i % 3 for i in range(32)],
             cos=A, sin=A, rows=64)
    a.update(kw)
    ax = None if a["ax"] is None else (ctypes.c_uint8 * 32)(*a["ax"])
    return L.ga_qk_prologue_axes(a["k"], a["wk"], a["kp"], a["q"], a["wq"], a["qp"], a["n"], a["pos"],
                                 a["ld"], a["na"], ax, a["cos"], a["sin"], a["rows"], None)


@pytest.mark.parametrize("kw,want", [
    *[({k: None}, -1) for k in ("k", "wk", "kp", "q", "wq", "qp", "pos", "ax", "cos", "sin")],
    (dict(k=None, wk=None, kp=None, q=None, wq=None, qp=None), -1),
    (dict(n=-1), -2), (dict(na=0), -2), (dict(rows=-1), -2),
    (dict(n=(1 << 20) + 1, ld=1 << 21), -4), (dict(na=5), -4), (dict(ld=7), -4),
    (dict(ax=[3] * 32), -4), (dict(na=1), -4), (dict(rows=0), -5),
    (dict(k=MIS), -3), (dict(qp=MIS), -3), (dict(cos=MIS), -3), (dict(pos=MIS), -3),
    (dict(n=0), 0), (dict(n=0, k=None, wk=None, kp=None), 0),
])
def test_axes_refusals(L, kw, want):
    _refused(L, lambda: _axes(L, **kw), want)


def _store(L, **kw):
    a = dict(k=A, ldk=512, v=A, ldv=1024, n=8, slots=A, kc=A, ks=A, vc=A, vs=A, pages=4, page=64)
    a.update(kw)
    return L.ga_kv_quantize_q4(a["k"], a["ldk"], a["v"], a["ldv"], a["n"], a["slots"], a["kc"],
                               a["ks"], a["vc"], a["vs"], a["pages"], a["page"], None)


def _load(L, **kw):
    a = dict(kc=A, ks=A, vc=A, vs=A, pages=4, page=64, slots=A, n=8, k=A, v=A)
    a.update(kw)
    return L.ga_kv_dequantize_q4(a["kc"], a["ks"], a["vc"], a["vs"], a["pages"], a["page"],
                                 a["slots"], a["n"], a["k"], a["v"], None)


POOL_REFUSALS = [
    *[({k: None}, -1) for k in ("k", "v", "kc", "ks", "vc", "vs")],
    (dict(pages=0), -2), (dict(page=0), -2), (dict(n=-1), -2),
    (dict(page=48), -4), (dict(page=1 << 21), -4), (dict(pages=1 << 24), -4),
    (dict(n=(64 << 20) + 1), -4), (dict(slots=None, n=257), -4),
    (dict(slots=MIS), -3), (dict(k=MIS), -3), (dict(v=MIS), -3), (dict(kc=MIS), -3),
    (dict(vs=MIS), -3), (dict(n=0), 0), (dict(n=0, slots=None), 0),
]


@pytest.mark.parametrize("kw,want", POOL_REFUSALS + [
    (dict(ldk=504), -4), (dict(ldv=0), -4), (dict(ldk=516), -3), (dict(ldv=1028), -3)])
def test_quantize_q4_refusals(L, kw, want):
    _refused(L, lambda: _store(L, **kw), want)


@pytest.mark.parametrize("kw,want", POOL_REFUSALS)
def test_dequantize_q4_refusals(L, kw, want):
    _refused(L, lambda: _load(L, **kw), want)


def _attn(L, **kw):
    a = dict(q=A, qg=A, kc=A, ks=A, vc=A, vs=A, pages=4, page=64, table=A, width=2, lens=A, n=2,
             rows=4, out=A, ws=0x100000, wsb=L.ga_verify_q4_workspace_bytes())
    a.update(kw)
    return L.ga_attn_verify_q4(a["q"], a["qg"], a["kc"], a["ks"], a["vc"], a["vs"], a["pages"],
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
def test_verify_q4_refusals(L, kw, want):
    _refused(L, lambda: _attn(L, **kw), want)


def test_binding_refuses_host_tensors():
    c = torch.zeros(2, 2, 32, 128, dtype=torch.uint8)
    s = torch.zeros(2, 2, 32, 16, dtype=torch.uint8)
    x = torch.zeros(4, 2, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.ga_kv_quantize_q4(x, x, c, s, c, s)
    with pytest.raises(ValueError):
        B.ga_kv_dequantize_q4(c, s, c, s)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.ga_page_plan(i, i, i[:, None], i, i, i[:1], 32, 8)
    with pytest.raises(ValueError):
        B.ga_qk_prologue_axes(x, x[0, 0], None, None, i, None, x[0], x[0])
    with pytest.raises(ValueError):
        B.ga_qk_prologue_axes(None, None, None, None, i, None, x[0], x[0])


# ------------------------------------------------------------------ the oracle's own pins
def test_q4_scale_bytes_cover_the_range():
    # every byte's scale, as the scale that a group of multiples of it picks
    b = np.arange(256)
    s = np.ldexp(1 + (b % 8) / 8, b // 8 - 20)
    x = np.zeros((256, 16))
    x[:, 3] = 7 * s
    codes, byte = O.quantize_q4_rows(x)
    assert np.array_equal(byte[:, 0], b)
    assert np.array_equal(O.widen_q4_rows(codes, byte), x)
    assert np.array_equal(O.bf16(x), x)


def test_q4_rounding_and_specials():
    x = np.zeros((5, 16))
    x[0, :4] = [7, 0.5, 1.5, -2.5]        # scale 1: ties to even
    x[1, :2] = [np.nan, 7]
    x[2, :3] = [np.inf, -np.inf, 3840]
    x[3, 0] = 2.0 ** -25                   # below half a code of the smallest scale
    x[4, :2] = [7.4375, -7.4375]           # 7.4375 / 7 = 1.0625 ties to the even scale 1
    codes, byte = O.quantize_q4_rows(x)
    w = O.widen_q4_rows(codes, byte)
    assert list(w[0, :4]) == [7, 0, 2, -2]
    assert list(w[1, :2]) == [0, 7]
    assert list(w[2, :3]) == [7 * 3840, -8 * 3840, 3840]
    assert w[3, 0] == 0 and byte[3, 0] == 0
    assert list(w[4, :2]) == [7, -7]


def test_q4_error_is_at_most_half_a_step():
    rng = np.random.default_rng(5)
    x = O.bf16(rng.standard_normal((200, 256)) * np.exp(rng.uniform(-6, 6, (200, 1))))
    codes, byte = O.quantize_q4_rows(x)
    s = np.repeat(np.ldexp(1 + (byte % 8) / 8, byte // 8 - 20), 16, -1)
    # the scale is within 1/16 of max / 7, so no value is past 7.5 steps (nothing saturates)
    assert np.all(np.abs(O.widen_q4_rows(codes, byte) - x) <= s / 2)


def test_q4_pack_is_the_documented_word():
    codes = np.arange(16)[None, :256].repeat(1, 0)
    codes = np.tile(codes, 16)
    b = O.pack_q4(codes)
    word = int.from_bytes(bytes(b[0, :4].tolist()), "little")
    assert [(word >> (4 * p)) & 15 for p in range(8)] == [0, 2, 4, 6, 1, 3, 5, 7]


def test_plan_oracle_small_case():
    t, held, stack, count, start, slots, pos, info = O.page_plan(
        [30, -1, 0, 64], [4, 5, 0, -1], [[9, -1], [-1, -1], [-1, -1], [7, 8]], [1, 0, 0, 2],
        [1, 2, 3, 0, 0], 3, 32, 6, pos_delta=[10, 0, 0, 0])
    assert t[0].tolist() == [9, 3] and held.tolist() == [2, 0, 0, 0]
    assert count == 4 and stack[:4].tolist() == [1, 2, 7, 8]
    assert start.tolist() == [0, 4, 4, 4, 4] and info.tolist() == [0, 4, 1, 2]
    assert slots.tolist() == [9 * 32 + 30, 9 * 32 + 31, 3 * 32, 3 * 32 + 1, -1, -1]
    assert pos.tolist() == [40, 41, 42, 43, 0, 0]
