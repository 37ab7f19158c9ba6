"""Ragged-batch operators where a 16-bit operand's range, an infinity or a NaN can go wrong: weights
far below the largest one, infinite values that a row sees, decays that forget, grow or are not
numbers. Bounds are those of test_gpu_ragged.py; where a test adds to one, its docstring says why.
"""
import numpy as np
import pytest

from test_gpu_ragged import _attn_bound, _hold, _mods, _np, _packed, _status_ok

pytestmark = pytest.mark.gpu


def _sink(q, k, v, rows, sink, gap, dh):
    """Scores 0 at the sink key, -gap (log2) at all others; V 0 at the sink and about 1 elsewhere."""
    q.zero_()
    q[:, ::dh] = 1.0
    k.zero_()
    k[:, ::dh] = -gap * float(np.log(2.0))
    v.abs_().mul_(0.25).add_(0.75)
    for r in sink:
        k[r] = 0.0
        v[r] = 0.0


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gap", [10, 16, 20, 24, 26])
@pytest.mark.parametrize("at", [0, 1500])
def test_packed_attention_long_tail_behind_a_sink(dt, gap, at):
    """One key of V = 0 holds nearly all the weight, the output is what thousands of weights of 2^-gap
    add up to: their half steps are relative to each weight (at 2^-26 fp16's are 2^-10 of it, which
    the bound's factor 2 covers)."""
    torch, hy, rt, code, tdt = _mods()
    H, G, dh, dv, L = 2, 1, 64, 64, 4001
    q, k, v, cu = _packed(dt, [L], H, G, dh, dv, 201, pad=0)
    _sink(q, k, v, L, [at], gap, dh)
    o = torch.zeros(L, H * dv, dtype=tdt[dt], device="cuda")
    rt.attn_prefill_packed(hy.attn_shape(H, G, dh, dv, 0, 0, code[dt], 1.0), q, k, v, cu, o)
    _status_ok(hy, torch)
    rows = np.r_[0:5, 1490:1510, 3990:4001]  # of the output; the oracle's scores are one row's
    kk, vv, qq = _np(k), _np(v), _np(q)
    want = np.zeros((len(rows), H * dv))
    for x, i in enumerate(rows):
        s = qq[i, 0] * kk[:i + 1, 0]
        p = np.exp(s - s.max())
        want[x] = np.tile(p @ vv[:i + 1] / p.sum(), H)
    big = np.full((len(rows), H), 18.1)  # scale |q||k|
    _hold(_np(o)[rows], want, _attn_bound(want, want, big, dt, dh, dv, L, 1.0), f"{dt} 2^-{gap}")
