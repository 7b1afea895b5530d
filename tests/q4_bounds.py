"""What the attention over 4-bit caches may be off by, a whole row at a time, and its definition
in 64 bits.

A bound per element has to allow every weight's rounding to go the same way, which over thousands
of keys is far more than the output itself. A row's 256 outputs together are bound much closer.
With weights w_j (sum 1), values v_j and the gate s (all exact), the attention's row is

    s (sum_j w_j (1 + d_j) v_j) / (sum_j w_j (1 + d_j)) (1 + r),   |d_j| <= 2^-8, |r| <= 2^-8

(bf16 weights, summed as rounded, and one bf16 rounding of each output). Relative to the row's
norm that is off by at most
    2^-8              the outputs' rounding
    2^-8              |sum w_j d_j|, the denominator
    1.5 x 2^-8        sum w_j d_j v_j: where the v_j are drawn independently of the weights, each of
                      its dims has at most 2^-16 of the variance of sum w_j v_j's, and the norms of
                      two such vectors over 256 gated dims have a ratio below 1.5 (a chi variable
                      of 200 degrees of freedom is within 5 % of its mean)
    2^-10             the fp32 sums, exponentials and gates (under 4e-4)
ROW_BOUND = 0.0146. Leaving out n of N keys of like weights is off by about sqrt(n / N): 535 of 40,001
keys 0.116, one tile of 128 of 12,351 keys 0.10.
"""
import torch

ROW_BOUND = 3.5 * 2.0 ** -8 + 2.0 ** -10


def attend64(q, gate, k, v, keys, without=None):
    """Rows q, gate [rows, heads, 256] of ONE KV head over its widened k, v [>= max keys, 256]; row r
    sees keys 0 .. keys[r] - 1, or those of them outside the range `without`. float64."""
    q, gate, k, v = (x.to(torch.float64) for x in (q, gate, k, v))
    rows = q.shape[0]
    n = int(max(keys))
    s = torch.einsum("rhd,jd->rhj", q, k[:n]) / 16
    j = torch.arange(n, device=q.device)
    hidden = j[None, :] >= torch.as_tensor(list(keys), device=q.device)[:, None]
    if without is not None:
        hidden = hidden | ((j >= without[0]) & (j < without[1]))
    assert hidden.shape == (rows, n)
    w = torch.softmax(s.masked_fill(hidden[:, None], -torch.inf), -1)
    return torch.einsum("rhj,jd->rhd", w, v[:n]) * torch.sigmoid(gate)


def row_errors(got, want):
    """|got - want| / |want| of each row of 256."""
    got, want = got.to(torch.float64), want.to(torch.float64)
    return (got - want).norm(dim=-1) / want.norm(dim=-1)
