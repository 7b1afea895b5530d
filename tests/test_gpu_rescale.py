"""Rows whose running maximum grows well after their first key tile, in every pass of the bf16 and
e4m3 attention: the accumulated O and l are scaled to the new maximum then.

Every sampled (row, query head) has a key of its own, 256 to 900 positions into the sequence, whose
score is about 8 (11.5 binary orders) above all others: more than the lazy rescale lets pass, and of
about the weight of all the row's other keys together, so that what O held before and what comes
after both count. A factor that is wrong, or that misses part of O, shows in every output."""
import contextlib

import numpy as np
import pytest
import torch

from oracle import ga_oracle as O
from tests.parity import SEED, AttnRef, np64
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


@contextlib.contextmanager
def _pairs(mode):
    prev = B.ga_debug_set_cta_pairs(mode)
    try:
        yield
    finally:
        B.ga_debug_set_cta_pairs(prev)


def _spiked(q_hat, k, rng):
    """Puts 0.5 q_hat of every row and head [n, 24, 256] at keys of their own among 256 .. 899 of
    k [T, 2, 256]."""
    n = q_hat.shape[0]
    for kv in range(2):
        at = torch.tensor(256 + rng.permutation(644)[:12 * n], device=k.device)
        k[at, kv] = (q_hat[:, 12 * kv:12 * kv + 12].float() * 0.5).reshape(-1, 256).to(k.dtype)


T, N_ROWS = 2304, 30


class Problem:
    def __init__(self, seed):
        rng = np.random.default_rng(seed)
        self.qg = synth.normal_bf16(seed, "qg", (T, 24, 512), device="cuda")
        self.w_q = synth.normal_bf16(seed, "w_q", (256,), sigma=0.1, device="cuda")
        self.k = synth.normal_bf16(seed, "k", (T, 2, 256), sigma=0.3, device="cuda")
        self.v = synth.normal_bf16(seed, "v", (T, 2, 256), device="cuda")
        self.c, self.s = (t.cuda() for t in B.ga_rope_table_host(T))
        q_hat = B.ga_q_prologue(self.qg, self.w_q, self.c, self.s)
        self.rows = np.sort(900 + rng.permutation(T - 900)[:N_ROWS])
        _spiked(q_hat.view(T, 24, 256)[torch.tensor(self.rows, device="cuda")], self.k, rng)

    def check(self, out, kind, what, mask=None):
        cos, sin = O.rope_tables(T)
        AttnRef(np64(self.qg), np64(self.k), np64(self.v), np64(self.w_q), cos, sin, 0, T, kind,
                mask, rows=self.rows).check(out[torch.tensor(self.rows, device="cuda")], what=what)


@pytest.fixture(scope="module")
def problem():
    return Problem(SEED + 300)


@pytest.mark.parametrize("causal", [True, False])
def test_prefill_grows(problem, causal):
    p = problem
    run = lambda: B.ga_attn_prefill(p.qg, p.k, p.v, p.w_q, p.c, p.s, causal=causal)  # noqa: E731
    with _pairs(0):
        out = run()
    p.check(out, "causal" if causal else "bidirectional", f"growing maxima, causal={causal}")
    for mode in (0, 2):   # the same bits, in both forms and every time
        with _pairs(mode):
            for _ in range(10):
                assert torch.equal(run(), out)


def test_masked_grows(problem):
    p = problem
    g = torch.Generator()
    g.manual_seed(5)
    mask = ((torch.rand(T, T, generator=g) < 0.7) & torch.tril(torch.ones(T, T, dtype=torch.bool)))
    mask[:, 256:900] |= torch.tril(torch.ones(T, T, dtype=torch.bool))[:, 256:900]
    mask = mask.to(torch.uint8)
    run = lambda: B.ga_attn_masked(p.qg, p.k, p.v, p.w_q, p.c, p.s, mask.cuda())[0]  # noqa: E731
    with _pairs(0):
        out = run()
    p.check(out, "mask", "growing maxima, stored mask", mask=mask.numpy())
    with _pairs(2):
        for _ in range(5):
            assert torch.equal(run(), out)


def test_batch_grows(problem):
    p = problem
    want = B.ga_attn_prefill(p.qg, p.k, p.v, p.w_q, p.c, p.s)
    pages = torch.tensor(np.random.default_rng(1).permutation(T // 128), device="cuda")
    pool = lambda x: torch.empty_like(x).view(T // 128, 128, 2, 256).index_copy_(  # noqa: E731
        0, pages, x.view(T // 128, 128, 2, 256))
    for mode in (0, 2):
        with _pairs(mode):
            out = B.ga_attn_prefill_batch(p.qg, [0, T], [0], pool(p.k), pool(p.v),
                                          pages.to(torch.int32)[None], p.w_q, p.c, p.s)
            assert torch.equal(out, want)


def test_verify_grows():
    n, rows, L, seed = 40, 4, 2000, SEED + 310
    cap = L + rows
    rng = np.random.default_rng(seed)
    w_q = synth.normal_bf16(seed, "w_q", (256,), sigma=0.1, device="cuda")
    c, s = (t.cuda() for t in B.ga_rope_table_host(cap))
    draw = lambda name, shape, **kw: torch.stack([  # noqa: E731
        synth.normal_bf16(seed, name, shape, sub=b, device="cuda", **kw) for b in range(n)])
    qg, v = draw("qg", (rows, 24, 512)), draw("v", (cap, 2, 256))
    k = draw("k", (cap, 2, 256), sigma=0.3)
    ctab, stab = c[L:].contiguous(), s[L:].contiguous()
    for b in range(n):
        _spiked(B.ga_q_prologue(qg[b], w_q, ctab, stab).view(rows, 24, 256), k[b], rng)
    out = B.ga_attn_verify(qg, k, v, [L] * n, w_q, c, s)
    cos, sin = O.rope_tables(cap)
    for b in (0, 17, 39):
        AttnRef(np64(qg[b]), np64(k[b]), np64(v[b]), np64(w_q), cos, sin, L, L + rows,
                "causal").check(out[b], what=f"verify, growing maxima, sequence {b}")
    for _ in range(10):
        assert torch.equal(B.ga_attn_verify(qg, k, v, [L] * n, w_q, c, s), out)
    kc, ks = B.ga_kv_quantize_e4m3(k)
    vc, vs = B.ga_kv_quantize_e4m3(v)
    wide = [B.ga_kv_dequantize_e4m3(*x).view_as(k) for x in ((kc, ks), (vc, vs))]
    want = B.ga_attn_verify(qg, *wide, [L] * n, w_q, c, s)
    for _ in range(10):
        assert torch.equal(B.ga_attn_verify_e4m3(qg, kc, ks, vc, vs, [L] * n, w_q, c, s), want)
