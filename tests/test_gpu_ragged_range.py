"""Ragged-batch operators where a 16-bit operand's range, an infinity or a NaN can go wrong: weights
far below the largest one, infinite values that a row sees, decays that forget, grow or are not
numbers. Bounds are those of test_gpu_ragged.py; where a test adds to one, its docstring says why.
"""
import numpy as np
import pytest

from oracle import ragged_oracle as ro
from test_gpu_ragged import (TINY, U, _attn_bound, _cache, _decode, _hold, _linear, _linear_bounds, _mods,
                             _np, _offsets, _packed, _run_linear, _status_ok)

pytestmark = pytest.mark.gpu


def _sink(q, k, v, sink, gap, dh):
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
    _sink(q, k, v, [at], gap, dh)
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


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gap", [8, 16, 20, 24, 26])
@pytest.mark.parametrize("at", [0, 700])
def test_decode_paged_long_tail_behind_a_sink(dt, gap, at):
    """As above, one token over the pages, in a batch whose sequences are not split: the warp that meets
    the sink has a quarter of the tail. All sequences share their pages. Weights keep 16 bits or
    more (fp16's at 2^-24 and 2^-26 of the largest 12 and 10, whose half steps lie below 2^-11)."""
    torch, hy, rt, code, tdt = _mods()
    B, H, G, dh, dv, L, page = 160, 8, 8, 64, 64, 1201, 32
    kv = _cache(dt, [L] + [1] * (B - 1), G, dh, dv, page, 202)
    kv.page_table[:] = kv.page_table[0]
    kv.len.fill_(L)
    pages = kv.page_table[0].long()
    k = torch.zeros(L, G * dh, dtype=tdt[dt], device="cuda")
    v = torch.randn(L, G * dv, generator=torch.Generator(device="cuda").manual_seed(203), device="cuda").to(tdt[dt])
    q = torch.zeros(B, H * dh, dtype=tdt[dt], device="cuda")
    _sink(q, k, v, [at], gap, dh)
    pos = torch.arange(L, device="cuda")
    kv.k_pages[pages[pos // page], :, pos % page] = k.view(L, G, dh)
    kv.v_pages[pages[pos // page], :, pos % page] = v.view(L, G, dv)
    q, o = _decode(kv, dt, H, 0, 0, 204, scale=1.0, q=q)
    _status_ok(hy, torch)
    assert (o == o[0]).all()
    want, a, big = ro.paged_attention(_np(q)[:1], _np(kv.k_pages), _np(kv.v_pages), kv.page_table.cpu().numpy(), [L], H,
                                      0, 0, 1.0)
    up = U["f16"] if dt == "f16" and gap > 20 else 2.0 ** -16
    bound = _attn_bound(want, a, big, "f32", dh, dv, L, 1.0) + 2 * a * up + U[dt] * np.abs(want) + TINY[dt]
    _hold(_np(o)[:1], want, bound, f"{dt} 2^-{gap}")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("inf", [float("inf"), float("-inf")])
def test_decode_paged_infinite_values(dt, inf):
    """A visible infinity in V makes its column infinite, whatever its weight (the lower part of a
    weight in two parts may be 0), and nothing else: one key, many, several splits, a key with a small
    weight, heads in two groups."""
    torch, hy, rt, code, tdt = _mods()
    for H, G, lens, page, window in ((4, 2, [1, 300, 40], 16, 0), (25, 5, [2500, 1, 700], 64, 0), (32, 1, [90, 1200, 33], 7, 200)):
        kv = _cache(dt, lens, G, 64, 128, page, 205)
        _, plain = _decode(kv, dt, H, 3, window, 206)
        R = H // G
        for b, pos, g, col in ((0, lens[0] - 1, 0, 5), (1, lens[1] // 2 if window == 0 else lens[1] - 100, G - 1, 127)):
            if pos >= lens[b]:
                continue
            kv.v_pages[int(kv.page_table[b, pos // page]), g, pos % page, col] = inf
        q, o = _decode(kv, dt, H, 3, window, 206)
        _status_ok(hy, torch)
        x, y = _np(o).reshape(3, H, 128), _np(plain).reshape(3, H, 128)
        hit = np.zeros_like(x, dtype=bool)
        hit[0, :R, 5] = True
        hit[1, H - R:, 127] = True
        assert (x[hit] == inf).all(), (H, G, x[hit])
        lens_, want = np.array(lens), None
        vp = kv.v_pages.clone()
        vp[~torch.isfinite(vp)] = 0
        want, a, big = ro.paged_attention(_np(q), _np(kv.k_pages), _np(vp), kv.page_table.cpu().numpy(), lens_, H, 3, window,
                                          64 ** -0.5)
        bound = _attn_bound(want, a, big, dt, 64, 128, max(lens), 64 ** -0.5)
        keep = ~hit.reshape(3, -1)
        _hold(_np(o)[keep], want[keep], bound[keep], f"{dt} {H} heads, other columns")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_packed_attention_infinite_values_of_small_weight(dt):
    """An infinity in V makes its column of every row that sees it infinite, also where its weight is
    far below what the rows' type can hold beside the largest (2^-60), also in key blocks that all
    rows of a tile see."""
    torch, hy, rt, code, tdt = _mods()
    H, G, dh, dv, L, at = 2, 1, 64, 64, 900, 3
    q, k, v, cu = _packed(dt, [L], H, G, dh, dv, 207, pad=0)
    q[:, ::dh] = 8.0
    k[:, 0] = 0.0
    k[at, 0] = -60 * float(np.log(2.0)) / 8.0 * 8.0  # scale 1/8
    k[at, 1:] = 0.0
    v[at, 7] = float("inf")
    o = torch.zeros(L, H * dv, dtype=tdt[dt], device="cuda")
    rt.attn_prefill_packed(hy.attn_shape(H, G, dh, dv, 0, 0, code[dt]), q, k, v, cu, o)
    _status_ok(hy, torch)
    v2 = v.clone()
    v2[at, 7] = 0.0
    want, a, big = ro.packed_attention(_np(q), _np(k), _np(v2), [0, L], H, G, 0, 0, dh ** -0.5)
    hit = np.zeros_like(want, dtype=bool)
    hit[at:, 7::dv] = True
    got = _np(o)
    assert (got[hit] == np.inf).all(), f"{np.count_nonzero(got[hit] != np.inf)} of {hit.sum()}"
    bound = _attn_bound(want, a, big, dt, dh, dv, L, dh ** -0.5)
    _hold(got[~hit], want[~hit], bound[~hit], f"{dt} other columns")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_packed_attention_rows_without_a_score_are_zero(dt):
    """Rows whose visible scores are all -infinity return zeros, whatever V holds."""
    torch, hy, rt, code, tdt = _mods()
    H, G, dh, dv, L = 2, 1, 64, 64, 300
    q, k, v, cu = _packed(dt, [L], H, G, dh, dv, 208, pad=0)
    none = torch.tensor([0, 5, 130, 299], device="cuda")
    k[:, 3] = 1.0
    q[none] = 0.0
    q[none, 3] = float("-inf")
    q[none, dh + 3] = float("-inf")
    k[:, :3], k[:, 4:] = 0.5, 0.5
    v[2, 9] = float("inf")
    v[200, 11] = float("nan")
    o = torch.full((L, H * dv), 7.0, dtype=tdt[dt], device="cuda")
    rt.attn_prefill_packed(hy.attn_shape(H, G, dh, dv, 0, 0, code[dt]), q, k, v, cu, o)
    _status_ok(hy, torch)
    assert (o[none] == 0).all()


ALL_DIMS = [(16, 64), (64, 64), (64, 128), (128, 64)]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dims", ALL_DIMS)
@pytest.mark.parametrize("at", [0, 37, 38, 39, 40, 131])
def test_linear_attention_decay_that_is_no_number(dt, dims, at):
    """NaN or +infinity as one row's log decay: the rows before it and the other sequence keep their
    values, the row and those behind it are not finite."""
    torch, hy, rt, code, tdt = _mods()
    lens, Hk, H, (dk, dv) = [180, 40], 1, 2, dims
    x = _linear(dt, lens, Hk, H, dk, dv, 211)
    q, k, v, g, st, cu = x
    n = sum(lens)
    want, oa, we, ea = ro.linear_attention(*(_np(t)[:n] for t in (q, k, v, g)), _offsets(lens), Hk, H, dk ** -0.5, _np(st))
    ob, eb = _linear_bounds(want, oa, we, ea, dt, max(lens), dk)
    for bad in (float("nan"), float("inf")):
        gg = g.clone()
        gg[at] = bad
        o, end = _run_linear(dt, x, Hk, H, dk, dv, True, g=gg)
        _status_ok(hy, torch)
        got, ge = _np(o)[:n], _np(end)
        sees = np.zeros(n, dtype=bool)
        sees[at:lens[0]] = True
        _hold(got[~sees], want[~sees], ob[~sees], f"{dt} {dims} {bad} at {at}, rows that do not see it")
        assert not np.isfinite(got[sees]).any()
        assert not np.isfinite(ge[0]).any()
        _hold(ge[1], we[1], eb[1], "the other state")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dims", ALL_DIMS)
@pytest.mark.parametrize("at,reset", [(5, 9), (10, 200), (70, 71), (20, 100)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_linear_attention_rows_before_a_reset_are_forgotten(dt, dims, at, reset, bad):
    """A key, value, query or start state that is not finite before a row that forgets everything:
    rows before the one and from the other on, and the state, keep their values."""
    torch, hy, rt, code, tdt = _mods()
    lens, Hk, H, (dk, dv) = [260, 40], 1, 2, dims
    x = _linear(dt, lens, Hk, H, dk, dv, 212, decay=0.05)
    q, k, v, g, st, cu = x
    n = sum(lens)
    g[reset] = float("-inf")
    want, oa, we, ea = ro.linear_attention(*(_np(t)[:n] for t in (q, k, v, g)), _offsets(lens), Hk, H, dk ** -0.5, _np(st))
    ob, eb = _linear_bounds(want, oa, we, ea, dt, max(lens), dk)
    for what in "kvqs":
        y = [t.clone() for t in (q, k, v)]
        s2 = st.clone()
        first = at
        if what == "s":
            s2[0, :, :, 1] = bad
            first = 0
        else:
            y["qkv".index(what)][at] = bad
        o, end = _run_linear(dt, (*y, g, s2, cu), Hk, H, dk, dv, True)
        _status_ok(hy, torch)
        got = _np(o)[:n]
        sees = np.zeros(n, dtype=bool)
        sees[first:at + 1 if what == "q" else reset] = True
        _hold(got[~sees], want[~sees], ob[~sees], f"{dt} {dims} {what}={bad}, rows that do not see it")
        assert not np.isfinite(got[sees]).any(), what
        _hold(_np(end), we, eb, f"{dt} {dims} {what}={bad} states")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dims", ALL_DIMS)
def test_linear_attention_infinities_in_the_state(dt, dims):
    """An infinite key element makes its column of the state infinite, an infinite value its row
    (NaN only where it meets a 0), and the rest of the state stays."""
    torch, hy, rt, code, tdt = _mods()
    lens, Hk, H, (dk, dv), at = [200], 1, 2, dims, 90
    x = _linear(dt, lens, Hk, H, dk, dv, 213, decay=0.05)
    q, k, v, g, st, cu = x
    for what in "kv":
        y = [t.clone() for t in (q, k, v)]
        if what == "k":
            y[1][at, 7] = float("-inf")
        else:
            y[2][at, dv + 9] = float("inf")
        o, end = _run_linear(dt, (*y, g, st, cu), Hk, H, dk, dv, True)
        _status_ok(hy, torch)
        with np.errstate(invalid="ignore"):
            want, oa, we, ea = ro.linear_attention(*(_np(t)[:200] for t in (*y, g)), _offsets(lens), Hk, H, dk ** -0.5, _np(st))
        got, fin = _np(end), np.isfinite(we)
        assert np.count_nonzero(~fin) == (H * dv if what == "k" else dk)
        ob, eb = _linear_bounds(np.where(fin, we, 0), np.where(fin, ea, 0), np.where(fin, we, 0), np.where(fin, ea, 0), dt,
                                200, dk)
        _hold(got[fin], we[fin], eb[fin], f"{dt} {dims} {what}: the rest of the state")
        assert np.array_equal(got[~fin], we[~fin], equal_nan=True), f"{dt} {dims} {what}"
        go, fo = _np(o)[:200], np.isfinite(want)
        ob, _ = _linear_bounds(np.where(fo, want, 0), np.where(fo, oa, 0), we, ea, dt, 200, dk)
        _hold(go[fo], want[fo], ob[fo], f"{dt} {dims} {what}: the rest of the rows")
        assert not np.isfinite(go[~fo]).any()


def _growth(dt, dims, grow):
    """Positive log decays: the state grows by e^(grow x rows); the output's scale brings the last
    rows back near 1."""
    torch, hy, rt, code, tdt = _mods()
    lens, Hk, H, (dk, dv) = [150, 33], 1, 2, dims
    x = _linear(dt, lens, Hk, H, dk, dv, 214)
    q, k, v, g, st, cu = x
    g.copy_(grow * (0.5 + torch.rand(g.shape, generator=torch.Generator(device="cuda").manual_seed(215), device="cuda")))
    scale = float(np.exp(-150 * grow)) * dk ** -0.5
    o, end = _run_linear(dt, x, Hk, H, dk, dv, True, scale=scale)
    _status_ok(hy, torch)
    n = sum(lens)
    want, oa, we, ea = ro.linear_attention(*(_np(t)[:n] for t in (q, k, v, g)), _offsets(lens), Hk, H, scale, _np(st))
    ob, eb = _linear_bounds(want, oa, we, ea, dt, max(lens), dk)
    _hold(_np(o)[:n], want[:n], ob[:n], f"{dt} {dims} o")
    _hold(_np(end), we, eb, f"{dt} {dims} state", 2.0 ** -16)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dims", [(16, 64), (128, 64)])
@pytest.mark.parametrize("grow", [0.04, 0.1, 0.3, 0.45])
def test_linear_attention_growth(dt, dims, grow):
    _growth(dt, dims, grow)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("dk,dv", [(16, 64), (128, 64), (64, 64), (64, 128)])
def test_linear_attention_value_columns_of_different_size(dt, dk, dv):
    """Value columns near 2^13 beside ones near 2^-13, decays of 2^-8 over a chunk: each column of the state
    keeps its own bits."""
    torch, hy, rt, code, tdt = _mods()
    lens, Hk, H = [150, 70], 1, 2
    x = _linear(dt, lens, Hk, H, dk, dv, 216, decay=0.17)
    q, k, v, g, st, cu = x
    v[:, ::2] *= 2.0 ** 11
    v[:, 1::2] *= 2.0 ** -13
    st[..., ::2, :] *= 2.0 ** 11
    st[..., 1::2, :] *= 2.0 ** -13
    scale = 2.0 ** -4
    o, end = _run_linear(dt, x, Hk, H, dk, dv, True, scale=scale)
    _status_ok(hy, torch)
    n = sum(lens)
    want, oa, we, ea = ro.linear_attention(*(_np(t)[:n] for t in (q, k, v, g)), _offsets(lens), Hk, H, scale, _np(st))
    ob, eb = _linear_bounds(want, oa, we, ea, dt, max(lens), dk)
    _hold(_np(o)[:n], want[:n], ob[:n], f"{dt} {dk} o")
    _hold(_np(end), we, eb, f"{dt} {dk} state", 2.0 ** -16)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dv", [64, 128])
@pytest.mark.parametrize("grow", [0.04, 0.1, 0.3, 0.45])
def test_linear_attention_growth_key_dim_64(dt, dv, grow):
    _growth(dt, (64, dv), grow)


def _reset_and_growth(dt, dims):
    """Rows that forget everything, then growth by e^40 and more within the same chunk: what lay
    before them, a NaN among it, does not come back."""
    torch, hy, rt, code, tdt = _mods()
    lens, Hk, H, (dk, dv), at, reset = [60, 130], 1, 2, dims, 3, 6
    x = _linear(dt, lens, Hk, H, dk, dv, 217)
    q, k, v, g, st, cu = x
    n = sum(lens)
    g.fill_(0.8)
    g[60:].fill_(0.4)
    for r in (reset, 60 + reset, 60 + reset + 5):
        g[r] = float("-inf")
    scale = float(np.exp(-40.0)) * dk ** -0.5
    want, oa, we, ea = ro.linear_attention(*(_np(t)[:n] for t in (q, k, v, g)), _offsets(lens), Hk, H, scale, _np(st))
    ob, eb = _linear_bounds(want, oa, we, ea, dt, max(lens), dk)
    for what in "kvs":
        y = [t.clone() for t in (q, k, v)]
        s2 = st.clone()
        if what == "s":
            s2.fill_(float("nan"))
        else:
            for a in (at, 60 + at):
                y["qkv".index(what)][a] = float("nan")
        o, end = _run_linear(dt, (*y, g, s2, cu), Hk, H, dk, dv, True, scale=scale)
        _status_ok(hy, torch)
        got = _np(o)[:n]
        sees = np.zeros(n, dtype=bool)
        first = 0 if what == "s" else at
        sees[first:reset] = sees[60 + first:60 + reset] = True
        _hold(got[~sees], want[~sees], ob[~sees], f"{dt} {dims} {what}, rows that do not see it")
        assert not np.isfinite(got[sees]).any()
        _hold(_np(end), we, eb, f"{dt} {dims} {what} states")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dims", [(16, 64), (128, 64)])
def test_linear_attention_growth_does_not_undo_a_reset(dt, dims):
    _reset_and_growth(dt, dims)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dv", [64, 128])
def test_linear_attention_growth_does_not_undo_a_reset_key_dim_64(dt, dv):
    _reset_and_growth(dt, (64, dv))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dims", [(16, 64), (128, 128)])
def test_linear_attention_decays_of_other_key_dims(dt, dims):
    """As test_linear_attention_decays, for the key dims it does not have, and rows that forget again and again."""
    torch, hy, rt, code, tdt = _mods()
    lens, Hk, H, (dk, dv) = [200, 70], 2, 4, dims
    x = _linear(dt, lens, Hk, H, dk, dv, 53)
    q, k, v, g, st, cu = x
    n = sum(lens)
    per_head = torch.tensor([-1e-3, -0.1, 0.0, -3.0], device="cuda")
    reset = g.clone() * 0.01
    for r in (0, 30, 31, 100, 200, 250):
        reset[r] = float("-inf")
    often = g.clone()
    often[::3] = float("-inf")
    often[1::7] = -90.0
    huge = g.clone() * 0.01
    huge[50] = -1e30
    huge[120] = -5000.0
    for name, gg in (("per head", per_head), ("broadcast", per_head.expand(q.shape[0], H)), ("resets", reset), ("huge", huge),
                     ("often", often)):
        o, end = _run_linear(dt, x, Hk, H, dk, dv, True, g=gg)
        _status_ok(hy, torch)
        full = _np(gg.expand(q.shape[0], H))
        want, oa, we, ea = ro.linear_attention(_np(q), _np(k), _np(v), full, _offsets(lens), Hk, H, dk ** -0.5, _np(st))
        ob, eb = _linear_bounds(want, oa, we, ea, dt, max(lens), dk)
        _hold(_np(o)[:n], want[:n], ob[:n], f"{dt} {name} o", 2 * U[dt] + 2.0 ** -17)
        _hold(_np(end), we, eb, f"{dt} {name} state", 2.0 ** -16)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dims", [(16, 64), (128, 128)])
@pytest.mark.parametrize("spread", [1e-3, 30.0])
def test_linear_attention_small_and_large_values_of_other_key_dims(dt, dims, spread):
    torch, hy, rt, code, tdt = _mods()
    lens, Hk, H, (dk, dv) = [150, 70], 2, 2, dims
    x = _linear(dt, lens, Hk, H, dk, dv, 52, decay=0.05, spread=spread)
    scale = 1.0 if spread < 1 else 1e-4
    q, k, v, g, st, cu = x
    st.mul_(spread * spread)
    o, end = _run_linear(dt, x, Hk, H, dk, dv, True, scale=scale)
    _status_ok(hy, torch)
    want, oa, we, ea = ro.linear_attention(_np(q), _np(k), _np(v), _np(g), _offsets(lens), Hk, H, scale, _np(st))
    ob, eb = _linear_bounds(want, oa, we, ea, dt, max(lens), dk)
    n = sum(lens)
    _hold(_np(o)[:n], want[:n], ob[:n], f"{dt} o")
    _hold(_np(end), we, eb, f"{dt} state", 2.0 ** -16)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("dims", [(16, 64), (128, 64)])
def test_linear_attention_offsets_out_of_order_of_other_key_dims(dt, dims):
    torch, hy, rt, code, tdt = _mods()
    Hk, H, (dk, dv) = 2, 2, dims
    for bad in ([0, 40, 200], [0, 40, 30], [-5, 40, 60]):
        x = list(_linear(dt, [60, 40], Hk, H, dk, dv, 55, pad=0))
        x[5] = torch.tensor(bad, dtype=torch.int32, device="cuda")
        o, end = _run_linear(dt, x, Hk, H, dk, dv, True)
        torch.cuda.synchronize()
        assert hy.hymba_get_device_status(None) == hy.HYMBA_ERR_DEVICE_RANGE
        assert end[0 if bad[0] < 0 else 1].isnan().all(), bad  # not written


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("dims", [(16, 64), (128, 64)])
def test_linear_attention_many_short_prompts_captured_of_other_key_dims(dt, dims):
    """More sequences than a warp has lanes, captured into a graph and replayed on another stream."""
    torch, hy, rt, code, tdt = _mods()
    Hk, H, (dk, dv) = 1, 3, dims
    lens = [(7 * i) % 40 for i in range(70)]
    x = _linear(dt, lens, Hk, H, dk, dv, 59)
    q, k, v, g, st, cu = x
    o, end = _run_linear(dt, x, Hk, H, dk, dv, True)
    want, oa, we, ea = ro.linear_attention(_np(q), _np(k), _np(v), _np(g), _offsets(lens), Hk, H, dk ** -0.5, _np(st))
    ob, eb = _linear_bounds(want, oa, we, ea, dt, max(lens), dk)
    n = sum(lens)
    _hold(_np(o)[:n], want[:n], ob[:n], f"{dt} o", 2 * U[dt] + 2.0 ** -17)
    _hold(_np(end), we, eb, f"{dt} state", 2.0 ** -16)
    s = hy.linattn_shape(Hk, H, dk, dv, code[dt])
    ws = rt.linattn_workspace(s, len(lens), q.shape[0])
    o2, end2 = torch.full_like(o, 7.0), torch.zeros_like(end)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rt.linattn_prefill(s, q, k, v, g, cu, o2, ws, state_in=st, state_out=end2)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        graph.replay()
    _status_ok(hy, torch)
    assert torch.equal(o, o2) and torch.equal(end, end2)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dims", ALL_DIMS)
@pytest.mark.parametrize("at,reset", [(0, 1), (5, 9), (10, 200), (63, 64), (20, 31), (130, 190)])
def test_linear_attention_decay_that_is_no_number_before_a_reset(dt, dims, at, reset):
    """A NaN or +infinity as a log decay reaches no row from the next one on that forgets everything."""
    torch, hy, rt, code, tdt = _mods()
    lens, Hk, H, (dk, dv) = [260, 40], 1, 2, dims
    x = _linear(dt, lens, Hk, H, dk, dv, 218, decay=0.05)
    q, k, v, g, st, cu = x
    n = sum(lens)
    g[reset] = g[reset + 30] = float("-inf")
    want, oa, we, ea = ro.linear_attention(*(_np(t)[:n] for t in (q, k, v, g)), _offsets(lens), Hk, H, dk ** -0.5, _np(st))
    ob, eb = _linear_bounds(want, oa, we, ea, dt, max(lens), dk)
    for bad in (float("nan"), float("inf")):
        gg = g.clone()
        gg[at] = bad
        o, end = _run_linear(dt, x, Hk, H, dk, dv, True, g=gg)
        _status_ok(hy, torch)
        got = _np(o)[:n]
        sees = np.zeros(n, dtype=bool)
        sees[at:reset] = True
        _hold(got[~sees], want[~sees], ob[~sees], f"{dt} {dims} {bad}, rows that do not see it")
        assert not np.isfinite(got[sees]).any()
        _hold(_np(end), we, eb, f"{dt} {dims} {bad} states")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("at,reset", [(400, 600), (600, 601), (600, 1500)])
def test_linear_attention_few_long_prompts_decay_that_is_no_number(dt, at, reset):
    """As above, in one segment of a long prompt and in two."""
    torch, hy, rt, code, tdt = _mods()
    lens, Hk, H, dk, dv = [2500, 30], 2, 2, 64, 64
    x = _linear(dt, lens, Hk, H, dk, dv, 219, decay=0.01)
    q, k, v, g, st, cu = x
    n = sum(lens)
    g[reset] = float("-inf")
    want, oa, we, ea = ro.linear_attention(*(_np(t)[:n] for t in (q, k, v, g)), _offsets(lens), Hk, H, dk ** -0.5, _np(st))
    ob, eb = _linear_bounds(want, oa, we, ea, dt, max(lens), dk)
    for bad in (float("nan"), float("inf")):
        gg = g.clone()
        gg[at] = bad
        o, end = _run_linear(dt, x, Hk, H, dk, dv, True, g=gg)
        _status_ok(hy, torch)
        got = _np(o)[:n]
        sees = np.zeros(n, dtype=bool)
        sees[at:reset] = True
        _hold(got[~sees], want[~sees], ob[~sees], f"{dt} {bad}, rows that do not see it")
        assert not np.isfinite(got[sees]).any()
        _hold(_np(end), we, eb, f"{dt} {bad} states")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("lens", [[2500], [1900, 2100]])
@pytest.mark.parametrize("reset", [None, 777, 1279, 1280])
def test_linear_attention_few_long_prompts_growth(dt, lens, reset):
    """Growth over whole segments, a row that forgets everything within one, at its end and at the next one's
    start; the output's scale brings the last rows back near 1."""
    torch, hy, rt, code, tdt = _mods()
    Hk, H, dk, dv = 1, 1, 64, 64
    x = _linear(dt, lens, Hk, H, dk, dv, 220)
    q, k, v, g, st, cu = x
    g.copy_(0.03 * torch.rand(g.shape, generator=torch.Generator(device="cuda").manual_seed(221), device="cuda"))
    if reset is not None:
        g[reset] = float("-inf")
    scale = float(np.exp(-0.015 * max(lens))) * dk ** -0.5
    o, end = _run_linear(dt, x, Hk, H, dk, dv, True, scale=scale, in_place=True)
    _status_ok(hy, torch)
    n = sum(lens)
    want, oa, we, ea = ro.linear_attention(*(_np(t)[:n] for t in (q, k, v, g)), _offsets(lens), Hk, H, scale, _np(st))
    ob, eb = _linear_bounds(want, oa, we, ea, dt, max(lens), dk)
    _hold(_np(o)[:n], want[:n], ob[:n], f"{dt} o")
    _hold(_np(end), we, eb, f"{dt} state", 2.0 ** -16)
