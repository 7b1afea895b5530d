"""The row bound of the 4-bit attention's long tests, on the CPU: the kernel's two roundings stay
inside it, and an expectation that leaves out (or counts twice) one CTA's part of the stream, or one
tile, is outside it in every row."""
import pytest
import torch

from oracle import ga_oracle as O
from tests.q4_bounds import ROW_BOUND, attend64, row_errors


def _stream(n, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, dtype=torch.float32).to(torch.bfloat16)  # noqa: E731
    wide = lambda x: torch.from_numpy(  # noqa: E731
        O.widen_q4_rows(*O.quantize_q4_rows(x.double().numpy())))
    return normal(1, 12, 256), normal(1, 12, 256), wide(normal(n, 256)), wide(normal(n, 256))


def _rounded(q, gate, k, v):
    """The attention with bf16 weights, summed as rounded, and a bf16 output."""
    s = torch.einsum("rhd,jd->rhj", q.double(), k) / 16
    w = torch.exp(s - s.amax(-1, keepdim=True)).to(torch.bfloat16).double()
    o = torch.einsum("rhj,jd->rhd", w, v) / w.sum(-1, keepdim=True)
    return (o * torch.sigmoid(gate.double())).to(torch.bfloat16)


# keys, and a part's: one of 75 CTAs' granules at 40,001 keys, a tile at 12,351 and at 3,001
@pytest.mark.parametrize("n,first,last", [(40001, 10700, 11235), (40001, 39466, 40001),
                                          (12351, 6144, 6272), (3001, 0, 128)])
def test_a_part_left_out_or_counted_twice_is_outside_the_bound(n, first, last):
    q, gate, k, v = _stream(n, n + first)
    want = attend64(q, gate, k, v, [n])
    assert float(row_errors(_rounded(q, gate, k, v), want).max()) <= ROW_BOUND
    without = attend64(q, gate, k, v, [n], without=(first, last))
    assert float(row_errors(without, want).min()) > 2 * ROW_BOUND
    twice = attend64(q, gate, torch.cat([k, k[first:last]]), torch.cat([v, v[first:last]]),
                     [n + last - first])
    assert float(row_errors(twice, want).min()) > 2 * ROW_BOUND
