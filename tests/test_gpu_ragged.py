"""The ragged-batch operators on the GPU against their fp64 oracle: packed-prompt attention,
the paged cache and its decode attention, linear attention (prompts and single tokens), and
runs of them together as a serving loop uses them.

Bounds. u(t) is half a step of type t relative to the value: f32 2^-24, f16 2^-11, bf16 2^-8.
Attention: a score is a sum of dh products scaled by scale log2(e); with accumulation in fp32
(tensor cores may truncate, which doubles the step) it is off by at most (dh + 8) 2^-22 scale
|q||k| =: ds. A weight's relative error is then 2 ds (numerator and denominator) + 2^-20
(exponentials, sums over up to n keys add n 2^-23), plus u(P) where P enters the value product
in 16 bits. So |o - o*| <= sum_j w_j |v_j| (2 ds + 2^-20 + n 2^-23 + u(P)) + u(out) |o*|, with
twice the first factor for the products' second order. Linear attention: every term passes
through at most n decays and sums: |o - o*| <= (sum of |terms|) (u(P) + u(S) + (n + dk) 2^-22) +
u(out) |o*|; the fp32 state has no 16-bit rounding left in it (its products keep 16 bits or
more of the scaled values: 2^-16).
Relative L2: independent roundings add in squares: three of them stay below 2 u(out) + 2^-18.
"""
import ctypes

import numpy as np
import pytest

from gpu_helpers import torch_cuda
from oracle import ragged_oracle as ro

pytestmark = pytest.mark.gpu

U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -126, "f16": 2.0 ** -24, "bf16": 2.0 ** -126}  # steps of the smallest values


def _mods():
    torch = torch_cuda()
    import hybrid_head_ssm_b200 as hy
    from hybrid_head_ssm_b200 import runtime as rt
    code = {"f32": hy.HYMBA_F32, "f16": hy.HYMBA_F16, "bf16": hy.HYMBA_BF16}
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
    return torch, hy, rt, code, dt


def _np(t):
    return t.double().cpu().numpy()


def _status_ok(hy, torch):
    torch.cuda.synchronize()
    assert hy.hymba_get_device_status(None) == hy.HYMBA_OK


def _status_range(hy, torch):
    torch.cuda.synchronize()
    assert hy.hymba_get_device_status(None) == hy.HYMBA_ERR_DEVICE_RANGE


def _hold(got, want, bound, what, rel=None):
    assert np.isfinite(got).all(), f"{what}: {np.count_nonzero(~np.isfinite(got))} values are not finite"
    off = np.abs(got - want) - bound
    at = np.unravel_index(np.argmax(off), off.shape) if off.size else None
    assert off.size == 0 or off[at] <= 0, (f"{what}: at {at} {got[at]:.8g} for {want[at]:.8g}, bound {bound[at]:.3g}; "
                                           f"{np.count_nonzero(off > 0)} of {off.size} off")
    if rel is not None and want.size:
        rl = np.linalg.norm(got - want) / max(np.linalg.norm(want), 1e-30)
        assert rl <= rel, f"{what}: relative L2 {rl:.3g} > {rel:.3g}"


def _attn_bound(o, a, big, dt, dh, dv, n, scale):
    up = 0.0 if dt == "f32" else U[dt]
    ds = np.repeat((dh + 8) * 2.0 ** -22 * big, dv, axis=1)
    return 2 * a * (2 * ds + 2.0 ** -20 + n * 2.0 ** -23 + up) + U[dt] * np.abs(o) + TINY[dt]


def _offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)


def _packed(dt, lens, H, G, dh, dv, seed, gap=0, pad=3, spread=1.0):
    """The columns Q | K | V of one buffer of rows, `gap` unused columns after each, and
    pad rows behind the last sequence."""
    torch, hy, rt, code, tdt = _mods()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows = int(sum(lens)) + pad
    width = (H + G) * dh + G * dv + 3 * gap
    p = (torch.randn(rows, width, generator=gen, device="cuda") * spread).to(tdt[dt])
    a, b = H * dh, H * dh + gap + G * dh
    q, k, v = p[:, :a], p[:, a + gap:b], p[:, b + gap:b + gap + G * dv]
    cu = torch.tensor(_offsets(lens), dtype=torch.int32, device="cuda")
    return q, k, v, cu


# ------------------------------------------------------------------ packed prompts
PREFILL = [
    # lens, heads, dims, meta, window
    ([1], (4, 2), (64, 128), 0, 0),
    ([272, 141], (4, 2), (64, 128), 16, 64),                    # the tiny layer
    ([300, 1, 0, 129, 64], (25, 5), (64, 128), 128, 100),       # the 1.5B layer's heads
    ([257, 255, 256], (8, 8), (64, 64), 0, 0),
    ([130, 5, 513], (8, 1), (128, 128), 7, 33),
    ([385, 2], (6, 3), (128, 64), 130, 1),                      # each row sees itself and the meta rows
    ([640], (5, 1), (64, 128), 200, 128),
    ([3, 2, 1, 1, 0, 0, 4], (4, 4), (64, 64), 2, 2),
    ([700], (2, 2), (128, 128), 0, 0),
    # more key blocks than the kernels keep at a time, last tiles of a pair without a row
    ([1300, 1400, 1537], (2, 1), (64, 128), 0, 0),
    ([1290, 1281], (2, 2), (128, 128), 130, 300),
    ([1665], (3, 1), (64, 64), 140, 700),
    ([1500], (1, 1), (128, 64), 500, 1),
]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens,heads,dims,meta,window", PREFILL)
def test_packed_attention(dt, lens, heads, dims, meta, window):
    torch, hy, rt, code, tdt = _mods()
    (H, G), (dh, dv) = heads, dims
    q, k, v, cu = _packed(dt, lens, H, G, dh, dv, 11, gap=8)
    ob = torch.full((q.shape[0], H * dv + 16), 7.0, dtype=tdt[dt], device="cuda")
    o = ob[:, 8:8 + H * dv]
    rt.attn_prefill_packed(hy.attn_shape(H, G, dh, dv, meta, window, code[dt]), q, k, v, cu, o)
    _status_ok(hy, torch)
    want, a, big = ro.packed_attention(_np(q), _np(k), _np(v), _offsets(lens), H, G, meta, window, dh ** -0.5)
    n = sum(lens)
    _hold(_np(o)[:n], want[:n], _attn_bound(want, a, big, dt, dh, dv, max(lens), dh ** -0.5)[:n],
          f"{dt} {lens} {heads} {dims}", 2 * U[dt] + 2.0 ** -18)
    # the rows behind the last sequence and the columns around o stay as they were
    assert (ob[n:] == 7).all() and (ob[:, :8] == 7).all() and (ob[:, 8 + H * dv:] == 7).all()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("scale,spread", [(1.0, 1.0), (0.02, 4.0), (2.0, 2.0), (1e-3, 1e-3)])
def test_packed_attention_scales(dt, scale, spread):
    """Sharp and flat softmax rows: scores of a few tenths up to hundreds."""
    torch, hy, rt, code, tdt = _mods()
    H, G, dh, dv, lens = 4, 2, 64, 128, [400, 77]
    q, k, v, cu = _packed(dt, lens, H, G, dh, dv, 12, spread=spread)
    o = torch.zeros(q.shape[0], H * dv, dtype=tdt[dt], device="cuda")
    rt.attn_prefill_packed(hy.attn_shape(H, G, dh, dv, 16, 128, code[dt], scale), q, k, v, cu, o)
    _status_ok(hy, torch)
    want, a, big = ro.packed_attention(_np(q), _np(k), _np(v), _offsets(lens), H, G, 16, 128, scale)
    _hold(_np(o), want, _attn_bound(want, a, big, dt, dh, dv, 400, scale), f"{dt} scale {scale}")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("dims", [(64, 128), (128, 64)])
def test_packed_attention_non_finite_values_stay_where_they_are_seen(dt, window, dims):
    """NaN and infinities in K and V of one row: rows that do not see it (earlier ones, later
    ones beyond the window, other sequences) keep their values; rows that see a NaN have
    one. Rows that belong to no sequence hold NaN everywhere."""
    torch, hy, rt, code, tdt = _mods()
    H, G, (dh, dv), lens, meta = 4, 2, dims, [200, 150, 90], 4
    q, k, v, cu = _packed(dt, lens, H, G, dh, dv, 13, pad=140)
    n = sum(lens)
    for t in (q, k, v):
        t[n:] = float("nan")
    s = hy.attn_shape(H, G, dh, dv, meta, window, code[dt])
    want, a, big = ro.packed_attention(*(_np(t[:n]) for t in (q, k, v)), _offsets(lens), H, G, meta, window, dh ** -0.5)
    bound = _attn_bound(want, a, big, dt, dh, dv, 200, dh ** -0.5)
    at = 200 + 60  # row 60 of the second sequence
    sees = np.zeros(n, dtype=bool)
    last = 350 if window == 0 else min(350, at + window)
    sees[at:last] = True
    for what, bad in (("v", float("nan")), ("v", float("inf")), ("k", float("nan"))):
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        {"k": k2, "v": v2}[what][at] = bad
        o = torch.full((q.shape[0], H * dv), 7.0, dtype=tdt[dt], device="cuda")
        rt.attn_prefill_packed(s, q2, k2, v2, cu, o)
        _status_ok(hy, torch)
        got = _np(o)[:n]
        _hold(got[~sees], want[~sees], bound[~sees], f"{dt} {what}={bad}, rows that do not see it")
        assert not np.isfinite(got[sees]).any(), f"{dt} {what}={bad}: rows that see it"
        if what == "v" and bad == float("inf"):
            assert (got[sees] == np.inf).all()
        assert (o[n:] == 7).all()


@pytest.mark.parametrize("dt", ["f32", "f16"])
def test_packed_attention_offsets_out_of_order_are_left_out(dt):
    torch, hy, rt, code, tdt = _mods()
    H, G, dh, dv = 4, 2, 64, 64
    q, k, v, _ = _packed(dt, [100], H, G, dh, dv, 14, pad=0)
    s = hy.attn_shape(H, G, dh, dv, 0, 0, code[dt])
    for bad in ([0, 40, 200], [0, 40, 30], [-5, 40, 60], [0, 1 << 30, 20]):
        o = torch.full((100, H * dv), 7.0, dtype=tdt[dt], device="cuda")
        rt.attn_prefill_packed(s, q, k, v, torch.tensor(bad, dtype=torch.int32, device="cuda"), o)
        _status_range(hy, torch)
    # the sequence before the bad one is computed, rows of none are left
    o = torch.full((100, H * dv), 7.0, dtype=tdt[dt], device="cuda")
    rt.attn_prefill_packed(s, q, k, v, torch.tensor([0, 40, 200], dtype=torch.int32, device="cuda"), o)
    _status_range(hy, torch)
    want, a, big = ro.packed_attention(*(_np(t) for t in (q, k, v)), [0, 40], H, G, 0, 0, dh ** -0.5)
    _hold(_np(o)[:40], want[:40], _attn_bound(want, a, big, dt, dh, dv, 40, dh ** -0.5)[:40], "before the bad one")
    assert (o[40:] == 7).all()


def test_packed_attention_many_short_sequences():
    """1500 sequences of 0 to 9 rows: one work item each, found among all of them."""
    torch, hy, rt, code, tdt = _mods()
    rng = np.random.default_rng(15)
    lens = rng.integers(0, 10, 1500).tolist()
    H, G, dh, dv = 2, 1, 64, 64
    for dt in ("f16", "f32"):
        q, k, v, cu = _packed(dt, lens, H, G, dh, dv, 16)
        o = torch.zeros(q.shape[0], H * dv, dtype=tdt[dt], device="cuda")
        rt.attn_prefill_packed(hy.attn_shape(H, G, dh, dv, 1, 4, code[dt]), q, k, v, cu, o)
        _status_ok(hy, torch)
        want, a, big = ro.packed_attention(_np(q), _np(k), _np(v), _offsets(lens), H, G, 1, 4, dh ** -0.5)
        _hold(_np(o), want, _attn_bound(want, a, big, dt, dh, dv, 9, dh ** -0.5), dt)


def test_packed_attention_offsets_past_32_bits():
    """The only sequence sits behind 2^32 elements of q and o."""
    torch, hy, rt, code, tdt = _mods()
    H, G, dh, dv, L = 32, 1, 64, 128, 140
    rows = (1 << 32) // (H * dv) + 200
    q = torch.empty(rows, H * dh + 2 * dv, dtype=torch.float16, device="cuda")
    o = torch.empty(rows, H * dv, dtype=torch.float16, device="cuda")
    lo = rows - L - 1
    gen = torch.Generator(device="cuda").manual_seed(17)
    q[lo:] = torch.randn(L + 1, q.shape[1], generator=gen, device="cuda").half()
    k, v, qq = q[:, H * dh:H * dh + dh], q[:, H * dh + dv:], q[:, :H * dh]
    cu = torch.tensor([lo, lo + L], dtype=torch.int32, device="cuda")
    rt.attn_prefill_packed(hy.attn_shape(H, G, dh, dv, 0, 0, code["f16"]), qq, k, v, cu, o)
    _status_ok(hy, torch)
    want, a, big = ro.packed_attention(*(_np(t[lo:]) for t in (qq, k, v)), [0, L], H, G, 0, 0, dh ** -0.5)
    _hold(_np(o[lo:lo + L]), want[:L], _attn_bound(want, a, big, "f16", dh, dv, L, dh ** -0.5)[:L], "far rows")


# ------------------------------------------------------------------ pages
def _cache(dt, lens, G, dh, dv, page, seed, extra_pages=2, spread=1.0):
    torch, hy, rt, code, tdt = _mods()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-n // page) for n in lens]
    per = max(1, max(need))
    n_pages = sum(need) + extra_pages
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), per), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = order[at:at + c]
        at += c
    kp = (torch.randn(n_pages, G, page, dh, generator=gen, device="cuda") * spread).to(tdt[dt])
    vp = torch.randn(n_pages, G, page, dv, generator=gen, device="cuda").to(tdt[dt])
    return rt.PagedKV(kp, vp, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))


def _decode(kv, dt, H, meta, window, seed, max_len=0, scale=0.0, q=None, ld_gap=0):
    torch, hy, rt, code, tdt = _mods()
    G, dh, dv, B = kv.s.n_kv_heads, kv.s.head_dim, kv.s.v_head_dim, kv.s.batch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if q is None:
        q = torch.randn(B, H * dh + ld_gap, generator=gen, device="cuda").to(tdt[dt])[:, :H * dh]
    s = hy.attn_shape(H, G, dh, dv, meta, window, code[dt], scale)
    ws = rt.decode_paged_workspace(s, B, max_len or kv.s.max_pages * kv.s.page_size)
    ws.fill_(0xFF)
    ob = torch.full((B, H * dv + ld_gap), float("nan"), dtype=tdt[dt], device="cuda")
    rt.attn_decode_paged(s, q, kv, ob[:, :H * dv], ws, max_len)
    torch.cuda.synchronize()
    assert ob[:, H * dv:].isnan().all()
    return q, ob[:, :H * dv]


def _check_decode(kv, dt, H, meta, window, q, o, what, scale=None, skip=()):
    dh, dv = kv.s.head_dim, kv.s.v_head_dim
    scale = scale or dh ** -0.5
    lens = kv.len.cpu().numpy().copy()
    for b in skip:
        lens[b] = 0
    want, a, big = ro.paged_attention(_np(q), _np(kv.k_pages), _np(kv.v_pages), kv.page_table.cpu().numpy(), lens, H,
                                      meta, window, scale)
    _hold(_np(o), want, _attn_bound(want, a, big, dt, dh, dv, max(1, int(lens.max())), scale), what,
          2 * U[dt] + 2.0 ** -18)


DECODE = [
    # lens, heads, dims, page, meta, window
    ([1], (4, 2), (64, 128), 16, 0, 0),
    ([0, 1, 2, 17, 300], (4, 2), (64, 128), 16, 16, 64),
    ([1153, 700, 64, 129], (25, 5), (64, 128), 64, 128, 1024),
    ([1500, 1, 1281], (25, 5), (64, 128), 24, 128, 200),          # pages that end inside a tile
    ([513, 40], (8, 1), (128, 128), 5, 0, 0),
    ([77, 260, 33], (16, 16), (64, 64), 1, 3, 10),
    ([900, 12], (32, 1), (128, 64), 128, 130, 1),
    ([2500, 2499], (20, 1), (64, 64), 100, 0, 0),
    ([128, 127, 129, 256], (6, 3), (128, 128), 128, 0, 128),
]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens,heads,dims,page,meta,window", DECODE)
def test_decode_paged(dt, lens, heads, dims, page, meta, window):
    torch, hy, rt, code, tdt = _mods()
    (H, G), (dh, dv) = heads, dims
    kv = _cache(dt, lens, G, dh, dv, page, 21)
    q, o = _decode(kv, dt, H, meta, window, 22, ld_gap=8)
    _status_ok(hy, torch)
    _check_decode(kv, dt, H, meta, window, q, o, f"{dt} {lens}")
    # the same with the tightest bound on the lengths: other splits
    q, o = _decode(kv, dt, H, meta, window, 23, max_len=max(1, max(lens)))
    _status_ok(hy, torch)
    _check_decode(kv, dt, H, meta, window, q, o, f"{dt} {lens}, tight bound")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_decode_paged_large_batch_uses_one_split(dt):
    """A batch that fills the GPU: few splits, and sequences that share all their pages."""
    torch, hy, rt, code, tdt = _mods()
    B = 400
    lens = [(37 * b) % 190 for b in range(B)]
    kv = _cache(dt, lens, 4, 64, 64, 16, 24)
    kv.page_table[7] = kv.page_table[5]
    kv.len[7] = kv.len[5]
    q, o = _decode(kv, dt, 8, 2, 0, 25)
    _status_ok(hy, torch)
    _check_decode(kv, dt, 8, 2, 0, q, o, dt)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("scale,spread", [(1.0, 1.0), (0.5, 6.0), (1e-3, 1e-3)])
def test_decode_paged_scales(dt, scale, spread):
    torch, hy, rt, code, tdt = _mods()
    kv = _cache(dt, [700, 90], 2, 64, 128, 32, 26, spread=spread)
    q, o = _decode(kv, dt, 8, 0, 0, 27, scale=scale)
    _status_ok(hy, torch)
    _check_decode(kv, dt, 8, 0, 0, q, o, dt, scale)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_decode_paged_sees_nothing_but_its_keys(dt):
    """NaN in every slot that is not a visible key (the rest of the last page, positions
    beyond the window, other pages), and -1 in the table where no key is visible."""
    torch, hy, rt, code, tdt = _mods()
    lens, page, meta, window, G = [300, 45, 16, 512], 16, 20, 50, 2
    kv = _cache(dt, lens, G, 64, 128, page, 28)
    used = torch.zeros(kv.k_pages.shape[0], page, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        pos = torch.arange(n, device="cuda")
        pos = pos[(pos < meta) | (n - 1 - pos < window)]
        at = kv.page_table[b].long()[pos // page]
        used[at, pos % page] = True
        hidden = torch.ones(kv.page_table.shape[1], dtype=torch.bool, device="cuda")
        hidden[pos // page] = False
        kv.page_table[b, hidden] = -1
    q0 = None
    for t in (kv.k_pages, kv.v_pages):
        t.masked_fill_(~used[:, None, :, None], float("nan"))
    q, o = _decode(kv, dt, 8, meta, window, 29)
    _status_ok(hy, torch)
    _check_decode(kv, dt, 8, meta, window, q, o, dt)
    # a visible NaN reaches its sequence and no other
    kv.v_pages[int(kv.page_table[1, 0]), 0, 3] = float("nan")
    q, o = _decode(kv, dt, 8, meta, window, 29)
    assert o[1, :4 * 128].isnan().all()
    assert not o[[0, 2, 3]].isnan().any() and not o[1, 4 * 128:].isnan().any()


@pytest.mark.parametrize("dt", ["f32", "f16"])
def test_decode_paged_out_of_range(dt):
    """A length past the bound, a negative one, a page outside the pool: zeros for that
    sequence, its neighbours right, the status word set."""
    torch, hy, rt, code, tdt = _mods()
    lens = [300, 200, 250, 100]
    for case in ("length", "negative", "page", "page below 0", "last page"):
        kv = _cache(dt, lens, 2, 64, 128, 16, 30)
        bad = 1
        if case == "length":
            kv.len[bad] = kv.s.max_pages * 16 + 1
        elif case == "negative":
            kv.len[bad] = -3
        elif case == "page":
            kv.page_table[bad, 3] = kv.s.n_pages
        elif case == "page below 0":
            kv.page_table[bad, 0] = -1
        else:
            kv.page_table[bad, 12] = 1 << 30
        q, o = _decode(kv, dt, 4, 0, 0, 31)
        _status_range(hy, torch)
        assert (o[bad] == 0).all(), case
        kv.page_table[bad] = 0
        _check_decode(kv, dt, 4, 0, 0, q, o, case, skip=(bad,))
    # a bound below a length refuses that sequence alone
    kv = _cache(dt, lens, 2, 64, 128, 16, 30)
    q, o = _decode(kv, dt, 4, 0, 0, 31, max_len=260)
    _status_range(hy, torch)
    assert (o[0] == 0).all()
    _check_decode(kv, dt, 4, 0, 0, q, o, "bound", skip=(0,))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("page", [1, 5, 16, 64])
def test_append_paged(dt, page):
    """Several new rows per sequence, none for some, then one for each: exactly the rows,
    exactly there."""
    torch, hy, rt, code, tdt = _mods()
    G, dh, dv = 5, 64, 128
    lens, new = [70, 33, 0, 128, 1, 64], [70, 5, 0, 1, 1, 33]
    kv = _cache(dt, lens, G, dh, dv, page, 41)
    gen = torch.Generator(device="cuda").manual_seed(42)
    p = torch.randn(sum(new) + 4, G * (dh + dv) + 16, generator=gen, device="cuda").to(tdt[dt])
    k, v = p[:, :G * dh], p[:, G * dh + 8:G * dh + 8 + G * dv]
    cu = _offsets(new)
    k0, v0 = _np(kv.k_pages), _np(kv.v_pages)
    table = kv.page_table.cpu().numpy()
    rt.kv_append_paged(kv, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"))
    _status_ok(hy, torch)
    kw, vw = ro.append_pages(k0, v0, table, lens, _np(k), _np(v), cu)
    assert (_np(kv.k_pages) == kw).all() and (_np(kv.v_pages) == vw).all()
    # one row per sequence, without offsets (the empty sequence's row has no place)
    rt.kv_append_paged(kv, k[:6], v[:6])
    _status_range(hy, torch)
    full = [b for b, n in enumerate(lens) if n]
    kw, vw = ro.append_pages(kw, vw, table[full], [lens[b] for b in full], _np(k)[full], _np(v)[full], None)
    assert (_np(kv.k_pages) == kw).all() and (_np(kv.v_pages) == vw).all()


@pytest.mark.parametrize("batch", [33, 1100])
def test_append_paged_many_sequences(batch):
    """More sequences than a warp looks through at once (twice over), every third without new rows,
    rows wider than a warp takes in one go, rows behind the last sequence left alone."""
    torch, hy, rt, code, tdt = _mods()
    G, dh, dv, page = 7, 128, 128, 4
    lens = [1 + (5 * b) % 9 for b in range(batch)]
    new = [0 if b % 3 == 1 else min(n, 1 + b % 2) for b, n in enumerate(lens)]
    kv = _cache("bf16", lens, G, dh, dv, page, 44)
    rows = sum(new) + 5
    k = torch.randn(rows, G * dh, device="cuda").to(torch.bfloat16)
    v = torch.randn(rows, G * dv, device="cuda").to(torch.bfloat16)
    cu = _offsets(new)
    k0, v0, table = _np(kv.k_pages), _np(kv.v_pages), kv.page_table.cpu().numpy()
    rt.kv_append_paged(kv, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"))
    _status_ok(hy, torch)
    kw, vw = ro.append_pages(k0, v0, table, lens, _np(k), _np(v), cu)
    assert (_np(kv.k_pages) == kw).all() and (_np(kv.v_pages) == vw).all()


def test_append_paged_out_of_range():
    """A page outside the pool, more rows than positions, a length past the table, offsets
    out of order: those rows are left out, the others written."""
    torch, hy, rt, code, tdt = _mods()
    G, dh, dv, page = 2, 64, 64, 16
    lens = [40, 40, 40]
    for case in ("page", "rows", "length", "offsets", "negative"):
        kv = _cache("f16", lens, G, dh, dv, page, 43)
        k = torch.ones(60, G * dh, dtype=torch.float16, device="cuda")
        v = torch.ones(60, G * dv, dtype=torch.float16, device="cuda")
        cu = torch.tensor([0, 20, 40, 60], dtype=torch.int32, device="cuda")
        table = kv.page_table.clone()
        first = 20  # sequence 1's rows that stay as they were: positions 20..39
        if case == "page":
            kv.page_table[1] = kv.s.n_pages + 5
        elif case == "rows":
            kv.len[1] = 10  # 20 rows, 10 positions: the first 10 rows have none
            first = 10
        elif case == "length":
            kv.len[1] = 3 * page + 1
        elif case == "negative":
            kv.len[1] = -1
        else:
            cu[2] = 61
        k0, v0 = kv.k_pages.clone(), kv.v_pages.clone()
        rt.kv_append_paged(kv, k, v, cu)
        _status_range(hy, torch)
        for b in range(3):
            for p in range(40):
                at = int(table[b, p // page])
                new = p >= 20 and (b == 0 or (b == 2 and case != "offsets"))
                if b == 1 and case == "rows":
                    new = p < 10
                if new:
                    assert (kv.k_pages[at, :, p % page] == 1).all() and (kv.v_pages[at, :, p % page] == 1).all(), (case, b, p)
                else:
                    assert (kv.k_pages[at, :, p % page] == k0[at, :, p % page]).all(), (case, b, p)
                    assert (kv.v_pages[at, :, p % page] == v0[at, :, p % page]).all(), (case, b, p)


def test_pages_past_32_bits():
    """A pool whose pages lie behind 2^32 elements of V: append and decode there."""
    torch, hy, rt, code, tdt = _mods()
    G, dh, dv, page = 5, 64, 128, 64
    n_pages = (1 << 32) // (G * page * dv) + 20
    kp = torch.empty(n_pages, G, page, dh, dtype=torch.float16, device="cuda")
    vp = torch.empty(n_pages, G, page, dv, dtype=torch.float16, device="cuda")
    L = 300
    per = -(-L // page)
    table = torch.arange(n_pages - per, n_pages, dtype=torch.int32, device="cuda").flip(0).view(1, per).contiguous()
    kv = rt.PagedKV(kp, vp, table, torch.tensor([L], dtype=torch.int32, device="cuda"))
    gen = torch.Generator(device="cuda").manual_seed(44)
    k = torch.randn(L, G * dh, generator=gen, device="cuda").half()
    v = torch.randn(L, G * dv, generator=gen, device="cuda").half()
    rt.kv_append_paged(kv, k, v, torch.tensor([0, L], dtype=torch.int32, device="cuda"))
    q, o = _decode(kv, "f16", 25, 0, 0, 45)
    _status_ok(hy, torch)
    lo = n_pages - per
    want, a, big = ro.paged_attention(_np(q), _np(kp[lo:]), _np(vp[lo:]), (table - lo).cpu().numpy(), [L], 25, 0, 0,
                                      dh ** -0.5)
    _hold(_np(o), want, _attn_bound(want, a, big, "f16", dh, dv, L, dh ** -0.5), "far pages")


# ------------------------------------------------------------------ linear attention
def _linear(dt, lens, Hk, H, dk, dv, seed, pad=3, gap=0, decay=1.0, spread=1.0):
    torch, hy, rt, code, tdt = _mods()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows = int(sum(lens)) + pad
    p = (torch.randn(rows, 2 * Hk * dk + H * dv + 3 * gap, generator=gen, device="cuda") * spread).to(tdt[dt])
    a, b = Hk * dk, 2 * Hk * dk + gap
    q, k, v = p[:, :a], p[:, a + gap:b], p[:, b + gap:b + gap + H * dv]
    g = -torch.rand(rows, H, generator=gen, device="cuda") * decay
    st = torch.randn(len(lens), H, dv, dk, generator=gen, device="cuda")
    cu = torch.tensor(_offsets(lens), dtype=torch.int32, device="cuda")
    return q, k, v, g, st, cu


def _linear_bounds(o, oa, end, enda, dt, n, dk):
    u16 = 0.0 if dt == "f32" else 2 * U[dt]
    f = (n + dk) * 2.0 ** -22
    return (oa * (u16 + f) * 1.01 + U[dt] * np.abs(o) + TINY[dt],
            enda * (f + (0.0 if dt == "f32" else 2.0 ** -16)) + 2.0 ** -126)


LINEAR = [
    # lens, heads, dims, decay, start state
    ([1], (4, 4), (64, 64), 1.0, True),
    ([64, 65, 63], (4, 4), (64, 128), 0.1, True),
    ([130, 0, 1, 40], (25, 25), (64, 128), 0.5, False),
    ([200, 3], (1, 6), (16, 64), 2.0, True),                 # the SSD form's shape: shared keys
    ([257], (2, 4), (128, 128), 0.02, True),
    ([90, 128], (2, 2), (128, 192), 30.0, True),             # decays that leave almost nothing
    ([2, 2, 0, 1, 1], (3, 3), (64, 64), 1.0, False),
    ([700, 129, 640], (1, 2), (64, 128), 0.01, True),        # several chunks of every kernel
    ([515], (1, 1), (64, 64), 0.2, True),
    ([450], (1, 1), (128, 64), 0.05, False),
]


def _run_linear(dt, x, Hk, H, dk, dv, start, scale=0.0, g=None, in_place=False):
    torch, hy, rt, code, tdt = _mods()
    q, k, v, gg, st, cu = x
    s = hy.linattn_shape(Hk, H, dk, dv, code[dt], scale)
    o = torch.full((q.shape[0], H * dv), 7.0, dtype=tdt[dt], device="cuda")
    ws = rt.linattn_workspace(s, cu.numel() - 1, q.shape[0])
    ws.fill_(0xFF)
    end = st.clone() if in_place else torch.full_like(st, float("nan"))
    rt.linattn_prefill(s, q, k, v, gg if g is None else g, cu, o, ws,
                       state_in=(end if in_place else st) if start else None, state_out=end)
    torch.cuda.synchronize()
    return o, end


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens,heads,dims,decay,start", LINEAR)
def test_linear_attention_prompts(dt, lens, heads, dims, decay, start):
    torch, hy, rt, code, tdt = _mods()
    (Hk, H), (dk, dv) = heads, dims
    x = _linear(dt, lens, Hk, H, dk, dv, 51, gap=8, decay=decay)
    o, end = _run_linear(dt, x, Hk, H, dk, dv, start, in_place=start)
    _status_ok(hy, torch)
    q, k, v, g, st, cu = x
    want, oa, we, ea = ro.linear_attention(_np(q), _np(k), _np(v), _np(g), _offsets(lens), Hk, H, dk ** -0.5,
                                           _np(st) if start else None)
    n = sum(lens)
    ob, eb = _linear_bounds(want, oa, we, ea, dt, max(lens), dk)
    _hold(_np(o)[:n], want[:n], ob[:n], f"{dt} {lens} o", 2 * U[dt] + 2.0 ** -17)
    _hold(_np(end), we, eb, f"{dt} {lens} state", 2.0 ** -16)
    assert (o[n:] == 7).all()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("spread", [1e-3, 30.0])
def test_linear_attention_small_and_large_values(dt, spread):
    """Values near the bottom of fp16's full precision, and large ones: nothing is lost to the
    range of a 16-bit operand."""
    torch, hy, rt, code, tdt = _mods()
    lens, Hk, H, dk, dv = [150, 70], 2, 2, 64, 64
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


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_linear_attention_decays(dt):
    """One decay per head for all rows; no decay at all; rows that forget everything (-inf),
    at the first row, inside a chunk and twice in a row, after which the sums' precision is
    what it was."""
    torch, hy, rt, code, tdt = _mods()
    lens, Hk, H, dk, dv = [200, 70], 2, 4, 64, 64
    x = _linear(dt, lens, Hk, H, dk, dv, 53)
    q, k, v, g, st, cu = x
    n = sum(lens)
    per_head = torch.tensor([-1e-3, -0.1, 0.0, -3.0], device="cuda")
    reset = g.clone() * 0.01
    for r in (0, 30, 31, 100, 200, 250):
        reset[r] = float("-inf")
    huge = g.clone() * 0.01
    huge[50] = -1e30
    huge[120] = -5000.0
    for name, gg in (("per head", per_head), ("broadcast", per_head.expand(q.shape[0], H)), ("resets", reset), ("huge", huge)):
        o, end = _run_linear(dt, x, Hk, H, dk, dv, True, g=gg)
        _status_ok(hy, torch)
        full = _np(gg.expand(q.shape[0], H))
        want, oa, we, ea = ro.linear_attention(_np(q), _np(k), _np(v), full, _offsets(lens), Hk, H, dk ** -0.5, _np(st))
        ob, eb = _linear_bounds(want, oa, we, ea, dt, max(lens), dk)
        _hold(_np(o)[:n], want[:n], ob[:n], f"{dt} {name} o", 2 * U[dt] + 2.0 ** -17)
        _hold(_np(end), we, eb, f"{dt} {name} state", 2.0 ** -16)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_linear_attention_non_finite_values_stay_where_they_are_seen(dt):
    """A NaN row: earlier rows of the sequence, other sequences and rows of none keep their
    values; the sequence's later rows and its state have it."""
    torch, hy, rt, code, tdt = _mods()
    lens, Hk, H, dk, dv = [100, 150, 40], 2, 2, 64, 64
    x = _linear(dt, lens, Hk, H, dk, dv, 54, pad=70)
    q, k, v, g, st, cu = x
    n = sum(lens)
    for t in (q, k, v, g):
        t[n:] = float("nan")
    want, oa, we, ea = ro.linear_attention(*(_np(t[:n]) for t in (q, k, v, g)), _offsets(lens), Hk, H, dk ** -0.5, _np(st))
    ob, eb = _linear_bounds(want, oa, we, ea, dt, max(lens), dk)
    at = 100 + 70
    for what in ("k", "v", "q"):
        y = [t.clone() for t in (q, k, v)]
        y["qkv".index(what)][at] = float("nan")
        o, end = _run_linear(dt, (*y, g, st, cu), Hk, H, dk, dv, True)
        _status_ok(hy, torch)
        got, ge = _np(o)[:n], _np(end)
        sees = np.zeros(n, dtype=bool)
        sees[at:250 if what != "q" else at + 1] = True
        _hold(got[~sees], want[~sees], ob[~sees], f"{dt} {what}, rows that do not see it")
        assert np.isnan(got[sees]).all(), f"{dt} {what}: rows that see it"
        keep = [0, 2] if what != "q" else [0, 1, 2]
        _hold(ge[keep], we[keep], eb[keep], f"{dt} {what} states")
        if what != "q":
            assert np.isnan(ge[1]).all()
        assert (o[n:] == 7).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_linear_attention_offsets_out_of_order_are_left_out(dt):
    torch, hy, rt, code, tdt = _mods()
    Hk, H, dk, dv = 2, 2, 64, 64
    for bad in ([0, 40, 200], [0, 40, 30], [-5, 40, 60]):
        x = list(_linear(dt, [60, 40], Hk, H, dk, dv, 55, pad=0))
        x[5] = torch.tensor(bad, dtype=torch.int32, device="cuda")
        o, end = _run_linear(dt, x, Hk, H, dk, dv, True)
        _status_range(hy, torch)
        b = 0 if bad[0] < 0 else 1
        assert end[b].isnan().all(), bad  # not written


# few long prompts, whose rows several blocks share
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("lens,heads,dims", [([1409], (1, 1), (64, 64)), ([0, 1300, 1, 900, 384], (2, 4), (64, 128)),
                                             ([2304, 2305], (3, 3), (64, 192)), ([1152] + [0] * 31, (1, 2), (64, 128)),
                                             ([0, 4100, 1, 900, 384], (1, 2), (64, 64)), ([5, 0, 0, 5000], (2, 2), (64, 128))])
@pytest.mark.parametrize("start", [False, True])
def test_linear_attention_few_long_prompts(dt, lens, heads, dims, start):
    torch, hy, rt, code, tdt = _mods()
    (Hk, H), (dk, dv) = heads, dims
    x = _linear(dt, lens, Hk, H, dk, dv, 56, gap=8, decay=0.01)
    q, k, v, g, st, cu = x
    g[::500] = -400.0  # a segment's whole decay out of fp32's range
    o, end = _run_linear(dt, x, Hk, H, dk, dv, start, in_place=start)
    _status_ok(hy, torch)
    want, oa, we, ea = ro.linear_attention(_np(q), _np(k), _np(v), _np(g), _offsets(lens), Hk, H, dk ** -0.5,
                                           _np(st) if start else None)
    n = sum(lens)
    ob, eb = _linear_bounds(want, oa, we, ea, dt, max(lens), dk)
    _hold(_np(o)[:n], want[:n], ob[:n], f"{dt} {lens} o", 2 * U[dt] + 2.0 ** -17)
    _hold(_np(end), we, eb, f"{dt} {lens} state", 2.0 ** -16)
    assert (o[n:] == 7).all()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_linear_attention_few_long_prompts_non_finite(dt):
    """A NaN in the second segment of a long prompt, and a reset two segments later: rows before
    the one and behind the other keep their values."""
    torch, hy, rt, code, tdt = _mods()
    lens, Hk, H, dk, dv = [2500, 30], 2, 2, 64, 64
    x = _linear(dt, lens, Hk, H, dk, dv, 57, decay=0.01)
    q, k, v, g, st, cu = x
    n, at, reset = sum(lens), 500, 1300
    g[reset] = float("-inf")
    want, oa, we, ea = ro.linear_attention(*(_np(t[:n]) for t in (q, k, v, g)), _offsets(lens), Hk, H, dk ** -0.5, _np(st))
    ob, eb = _linear_bounds(want, oa, we, ea, dt, max(lens), dk)
    for what in ("k", "v"):
        y = [t.clone() for t in (q, k, v)]
        y["qkv".index(what)][at] = float("nan")
        o, end = _run_linear(dt, (*y, g, st, cu), Hk, H, dk, dv, True)
        _status_ok(hy, torch)
        got = _np(o)[:n]
        sees = np.zeros(n, dtype=bool)
        sees[at:reset] = True
        _hold(got[~sees], want[~sees], ob[~sees], f"{dt} {what}, rows that do not see it")
        assert np.isnan(got[sees]).all()
        _hold(_np(end), we, eb, f"{dt} {what} states")


def test_linear_attention_few_long_prompts_offsets_out_of_order():
    """More segments than the offsets may name: nothing outside the buffers is touched."""
    torch, hy, rt, code, tdt = _mods()
    Hk, H, dk, dv = 2, 2, 64, 64
    x = list(_linear("bf16", [5000, 100, 100], Hk, H, dk, dv, 58, pad=0))
    x[5] = torch.tensor([0, 5200, 0, 5200], dtype=torch.int32, device="cuda")
    o, end = _run_linear("bf16", x, Hk, H, dk, dv, True)
    _status_range(hy, torch)
    assert end[1].isnan().all()  # the one with a negative length, not written


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_linear_attention_many_short_prompts(dt):
    """More sequences than a warp has lanes, and none with any row at all."""
    torch, hy, rt, code, tdt = _mods()
    Hk, H, dk, dv = 2, 2, 64, 64
    lens = [(7 * i) % 40 for i in range(70)]
    x = _linear(dt, lens, Hk, H, dk, dv, 59)
    q, k, v, g, st, cu = x
    o, end = _run_linear(dt, x, Hk, H, dk, dv, True, in_place=True)
    _status_ok(hy, torch)
    want, oa, we, ea = ro.linear_attention(_np(q), _np(k), _np(v), _np(g), _offsets(lens), Hk, H, dk ** -0.5, _np(st))
    ob, eb = _linear_bounds(want, oa, we, ea, dt, max(lens), dk)
    n = sum(lens)
    _hold(_np(o)[:n], want[:n], ob[:n], f"{dt} o", 2 * U[dt] + 2.0 ** -17)
    _hold(_np(end), we, eb, f"{dt} state", 2.0 ** -16)
    s = hy.linattn_shape(Hk, H, dk, dv, code[dt])
    none = lambda t: t[:0]
    out = torch.full_like(st, float("nan"))
    rt.linattn_prefill(s, none(q), none(k), none(v), none(g), torch.zeros_like(cu), none(o), rt.linattn_workspace(s, 70, 0),
                       state_in=st, state_out=out)
    _status_ok(hy, torch)
    assert (out == st).all()


@pytest.mark.parametrize("lens", [[1500], [300] * 3])
def test_linear_attention_captured_and_on_two_streams(lens):
    """Two calls at once, each with its own workspace, and a captured one replayed on new inputs,
    equal the call alone bit for bit."""
    torch, hy, rt, code, tdt = _mods()
    Hk, H, dk, dv = 2, 4, 64, 128
    s = hy.linattn_shape(Hk, H, dk, dv, code["bf16"])
    xs = [_linear("bf16", lens, Hk, H, dk, dv, 63 + i, pad=0) for i in range(2)]

    def call(x, ws):
        q, k, v, g, st, cu = x
        o, end = torch.zeros_like(v), torch.zeros_like(st)
        return o, end, lambda: rt.linattn_prefill(s, q, k, v, g, cu, o, ws, state_in=st, state_out=end)

    wss = [rt.linattn_workspace(s, len(lens), sum(lens)) for _ in range(2)]
    alone = []
    for x, ws in zip(xs, wss):
        o, end, f = call(x, ws)
        f()
        alone.append((o, end))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    runs = [call(x, ws) for x, ws in zip(xs, wss)]
    torch.cuda.synchronize()
    for _ in range(3):
        for st, r in zip(streams, runs):
            with torch.cuda.stream(st):
                r[2]()
    torch.cuda.synchronize()
    for (o, end), r in zip(alone, runs):
        assert torch.equal(o, r[0]) and torch.equal(end, r[1])
    buf = tuple(t.clone() for t in xs[0])
    o, end, f = call(buf, wss[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f()
    for x, (wo, we) in zip(xs, alone):
        for to, t in zip(buf, x):
            to.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, wo) and torch.equal(end, we)
    _status_ok(hy, torch)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("batch,heads,dims", [(1, (4, 4), (64, 128)), (7, (1, 50), (16, 64)), (3, (5, 25), (128, 64)),
                                              (40, (2, 2), (64, 512))])
def test_linear_attention_step(dt, batch, heads, dims):
    """Three single tokens in a row, the state in place."""
    torch, hy, rt, code, tdt = _mods()
    (Hk, H), (dk, dv) = heads, dims
    s = hy.linattn_shape(Hk, H, dk, dv, code[dt])
    q, k, v, g, st, _ = _linear(dt, [3] * batch, Hk, H, dk, dv, 61, gap=8, pad=0)
    want, oa, we, ea = ro.linear_attention(_np(q), _np(k), _np(v), _np(g), _offsets([3] * batch), Hk, H, dk ** -0.5,
                                           _np(st))
    outs = []
    for t in range(3):
        o = torch.zeros(batch, H * dv, dtype=tdt[dt], device="cuda")
        rt.linattn_step(s, q[t::3], k[t::3], v[t::3], g[t::3].contiguous(), st, o)
        outs.append(o)
    _status_ok(hy, torch)
    got = _np(torch.stack(outs, 1).reshape(3 * batch, -1))
    ob, eb = _linear_bounds(want, oa, we, ea, dt, 3, dk)
    _hold(got, want, ob, f"{dt} o", 2 * U[dt] + 2.0 ** -18)
    _hold(_np(st), we, ea * (3 + dk) * 2.0 ** -22 + 2.0 ** -126, f"{dt} state", 2.0 ** -20)


def test_linear_attention_step_forgets_what_is_not_finite():
    """A decay of -inf replaces the state, also one that held NaN."""
    torch, hy, rt, code, tdt = _mods()
    s = hy.linattn_shape(2, 2, 64, 64, code["f32"])
    q, k, v, g, st, _ = _linear("f32", [1, 1], 2, 2, 64, 64, 62, pad=0)
    st.fill_(float("nan"))
    g.fill_(float("-inf"))
    o = torch.zeros(2, 128, device="cuda")
    rt.linattn_step(s, q, k, v, g, st, o)
    _status_ok(hy, torch)
    want = torch.einsum("bhv,bhk->bhvk", v.view(2, 2, 64), k.view(2, 2, 64))
    assert (st == want).all() and torch.isfinite(o).all()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_prompts_then_tokens(dt):
    """A serving loop: packed prompts through both head families, their K and V into pages,
    then tokens one by one. Each token's row equals the prompt of the whole text."""
    torch, hy, rt, code, tdt = _mods()
    H, G, dh, dv, meta, window, page, T = 10, 2, 64, 128, 16, 40, 24, 5
    Hk, LH, dk, ldv = 2, 10, 64, 128
    lens = [90, 17, 131, 1]
    full = [n + T for n in lens]
    q, k, v, cu_full = _packed(dt, full, H, G, dh, dv, 71, pad=0)
    lq, lk, lv, lg, st, _ = _linear(dt, full, Hk, LH, dk, ldv, 72, pad=0)
    cu = _offsets(full)
    prompt = np.concatenate([np.arange(a, a + n) for a, n in zip(cu, lens)])
    idx = torch.tensor(prompt, device="cuda")
    cu_p = torch.tensor(_offsets(lens), dtype=torch.int32, device="cuda")
    s = hy.attn_shape(H, G, dh, dv, meta, window, code[dt])
    ls = hy.linattn_shape(Hk, LH, dk, ldv, code[dt])
    o = torch.zeros(len(prompt), H * dv, dtype=tdt[dt], device="cuda")
    lo = torch.zeros(len(prompt), LH * ldv, dtype=tdt[dt], device="cuda")
    kv = _cache(dt, full, G, dh, dv, page, 73)
    kv.len.copy_(torch.tensor(lens, dtype=torch.int32))
    state = st.clone()
    rt.attn_prefill_packed(s, q[idx], k[idx], v[idx], cu_p, o)
    rt.kv_append_paged(kv, k[idx], v[idx], cu_p)
    rt.linattn_prefill(ls, lq[idx], lk[idx], lv[idx], lg[idx], cu_p, lo, rt.linattn_workspace(ls, 4, len(prompt)),
                       state_in=state, state_out=state)
    ws = rt.decode_paged_workspace(s, 4, max(full))
    outs, louts, rows = [o], [lo], [prompt]
    for t in range(T):
        r = cu[:-1] + np.array(lens) + t
        i = torch.tensor(r, device="cuda")
        kv.len.add_(1)
        rt.kv_append_paged(kv, k[i], v[i])
        ot = torch.zeros(4, H * dv, dtype=tdt[dt], device="cuda")
        rt.attn_decode_paged(s, q[i], kv, ot, ws, max(full))
        lot = torch.zeros(4, LH * ldv, dtype=tdt[dt], device="cuda")
        rt.linattn_step(ls, lq[i], lk[i], lv[i], lg[i], state, lot)
        outs.append(ot)
        louts.append(lot)
        rows.append(r)
    _status_ok(hy, torch)
    rows = np.concatenate(rows)
    want, a, big = ro.packed_attention(_np(q), _np(k), _np(v), cu, H, G, meta, window, dh ** -0.5)
    b = _attn_bound(want, a, big, dt, dh, dv, max(full), dh ** -0.5)
    _hold(_np(torch.cat(outs)), want[rows], b[rows], "attention")
    want, oa, we, ea = ro.linear_attention(_np(lq), _np(lk), _np(lv), _np(lg), cu, Hk, LH, dk ** -0.5, _np(st))
    ob, eb = _linear_bounds(want, oa, we, ea, dt, max(full), dk)
    _hold(_np(torch.cat(louts)), want[rows], ob[rows], "linear attention")
    _hold(_np(state), we, eb, "state", 2.0 ** -16)
    # the packed call on the whole text gives the same rows
    o2 = torch.zeros(q.shape[0], H * dv, dtype=tdt[dt], device="cuda")
    rt.attn_prefill_packed(s, q, k, v, cu_full, o2)
    torch.cuda.synchronize()
    assert np.abs(_np(torch.cat(outs)) - _np(o2)[rows]).max() <= 2 * b.max()


@pytest.mark.parametrize("dt", ["f32", "f16"])
def test_captured_and_replayed(dt):
    """A decode step of both head families in a CUDA graph, replayed with new inputs, lengths
    and pages in the same buffers, on another stream than the one it was captured on; then two
    graphs that share one workspace, replayed in turn."""
    torch, hy, rt, code, tdt = _mods()
    H, G, dh, dv = 8, 2, 64, 128
    lens = [700, 30, 257]
    kv = _cache(dt, [n + 10 for n in lens], G, dh, dv, 16, 81)
    kv.len.copy_(torch.tensor(lens, dtype=torch.int32))
    s, ls = hy.attn_shape(H, G, dh, dv, 4, 0, code[dt]), hy.linattn_shape(2, 4, 64, 64, code[dt])
    q, k, v, _ = _packed(dt, [1] * 3, H, G, dh, dv, 82, pad=0)
    lq, lk, lv, lg, st, cu = _linear(dt, [40, 1, 90], 2, 4, 64, 64, 83, pad=0)
    pq, pk, pv, pcu = _packed(dt, [150, 20], H, G, dh, dv, 84, pad=0)
    ws, lws = rt.decode_paged_workspace(s, 3, 710), rt.linattn_workspace(ls, 3, lq.shape[0])
    o = torch.zeros(3, H * dv, dtype=tdt[dt], device="cuda")
    lo = torch.zeros(lq.shape[0], 4 * 64, dtype=tdt[dt], device="cuda")
    end = torch.zeros_like(st)
    po = torch.zeros(pq.shape[0], H * dv, dtype=tdt[dt], device="cuda")

    def step():
        kv.len.add_(1)
        rt.kv_append_paged(kv, k, v)
        rt.attn_decode_paged(s, q, kv, o, ws, 710)
        rt.linattn_prefill(ls, lq, lk, lv, lg, cu, lo, lws, state_in=st, state_out=end)
        rt.attn_prefill_packed(s, pq, pk, pv, pcu, po)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    gen = torch.Generator(device="cuda").manual_seed(85)
    stream = torch.cuda.Stream()
    for r in range(3):
        for t in (q, k, v, lq, lk, lv, pq, pk, pv):
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda").to(t.dtype))
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.current_stream().wait_stream(stream)
        _status_ok(hy, torch)
        assert kv.len.tolist() == [n + r + 1 for n in lens]
        _check_decode(kv, dt, H, 4, 0, q, o, f"replay {r}")
        want, oa, we, ea = ro.linear_attention(_np(lq), _np(lk), _np(lv), _np(lg), [0, 40, 41, 131], 2, 4, 0.125, _np(st))
        ob, eb = _linear_bounds(want, oa, we, ea, dt, 90, 64)
        _hold(_np(lo), want, ob, f"replay {r} o")
        _hold(_np(end), we, eb, f"replay {r} state")
        want, a, big = ro.packed_attention(_np(pq), _np(pk), _np(pv), [0, 150, 170], H, G, 4, 0, 0.125)
        _hold(_np(po), want, _attn_bound(want, a, big, dt, dh, dv, 150, 0.125), f"replay {r} prompts")
    # two graphs on one workspace, one after the other on one stream
    o2, q2 = torch.zeros_like(o), torch.randn(q.shape, generator=gen, device="cuda").to(tdt[dt])
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        rt.attn_decode_paged(s, q, kv, o, ws, 710)
    with torch.cuda.graph(two):
        rt.attn_decode_paged(s, q2, kv, o2, ws, 710)
    for g in (one, two, one, two, two, one):
        g.replay()
    _status_ok(hy, torch)
    _check_decode(kv, dt, H, 4, 0, q, o, "first graph")
    _check_decode(kv, dt, H, 4, 0, q2, o2, "second graph")


def test_calls_on_two_streams_at_once():
    """Each with its own outputs and workspace."""
    torch, hy, rt, code, tdt = _mods()
    dt, H, G, dh, dv = "f16", 25, 5, 64, 128
    s = hy.attn_shape(H, G, dh, dv, 16, 0, code[dt])
    jobs = []
    for i in range(2):
        lens = [2000 + 500 * i, 700, 40]
        kv = _cache(dt, lens, G, dh, dv, 32, 91 + i)
        q = torch.randn(3, H * dh, device="cuda").half()
        jobs.append((kv, q, torch.zeros(3, H * dv, dtype=torch.float16, device="cuda"),
                     rt.decode_paged_workspace(s, 3, max(lens)), max(lens), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for kv, q, o, ws, n, stream in jobs:
            with torch.cuda.stream(stream):
                rt.attn_decode_paged(s, q, kv, o, ws, n)
    _status_ok(hy, torch)
    for kv, q, o, ws, n, stream in jobs:
        _check_decode(kv, dt, H, 16, 0, q, o, "two streams")


def test_results_repeat_bit_for_bit():
    """No sum depends on the order in which blocks finish."""
    torch, hy, rt, code, tdt = _mods()
    for dt in ("f16", "bf16", "f32"):
        kv = _cache(dt, [3000, 511], 5, 64, 128, 16, 95)
        _, first = _decode(kv, dt, 25, 0, 0, 96)
        x = _linear(dt, [300, 65], 5, 5, 64, 128, 97)
        lo, le = _run_linear(dt, x, 5, 5, 64, 128, True)
        q, k, v, cu = _packed(dt, [300, 65], 10, 5, 64, 128, 98)
        s = hy.attn_shape(10, 5, 64, 128, 0, 0, code[dt])
        po = torch.zeros(q.shape[0], 10 * 128, dtype=tdt[dt], device="cuda")
        rt.attn_prefill_packed(s, q, k, v, cu, po)
        for _ in range(3):
            _, again = _decode(kv, dt, 25, 0, 0, 96)
            assert torch.equal(first, again)
            lo2, le2 = _run_linear(dt, x, 5, 5, 64, 128, True)
            assert torch.equal(lo, lo2) and torch.equal(le, le2)
            po2 = torch.zeros_like(po)
            rt.attn_prefill_packed(s, q, k, v, cu, po2)
            assert torch.equal(po, po2)
    _status_ok(hy, torch)
