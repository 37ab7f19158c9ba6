"""The ragged-batch operators without a GPU: their oracle against the mixer's oracle and
closed forms, and every argument check of their entry points (fake addresses, never
dereferenced: the checks run before the device is touched)."""
import ctypes

import numpy as np
import pytest

import oracle
import synth
from oracle import ragged_oracle as ro

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def hy():
    import hybrid_head_ssm_b200 as hy
    return hy


# ------------------------------------------------------------------ the oracle
@pytest.mark.parametrize("window", [0, 3])
def test_oracle_packed_attention_is_each_sequence_alone(window):
    rng = np.random.default_rng(1)
    H, G, dh, dv, m = 4, 2, 8, 6, 2
    lens = [5, 0, 1, 7]
    cu = np.concatenate([[0], np.cumsum(lens)])
    q, k, v = (rng.standard_normal((cu[-1] + 2, w)) for w in (H * dh, G * dh, G * dv))
    o, a, _ = ro.packed_attention(q, k, v, cu, H, G, m, window, dh ** -0.5)
    assert (o[cu[-1]:] == 0).all() and (a >= np.abs(o) - 1e-12).all()
    for lo, hi in zip(cu[:-1], cu[1:]):
        n = hi - lo
        pos = np.arange(n)
        one = oracle.attention(q[lo:hi].reshape(n, H, dh).transpose(1, 0, 2), k[lo:hi].reshape(n, G, dh).transpose(1, 0, 2),
                               v[lo:hi].reshape(n, G, dv).transpose(1, 0, 2),
                               oracle.visibility_mask(pos, pos, m, window)) if n else np.zeros((0, H * dv))
        one = np.asarray(one)
        if one.ndim == 3:
            one = one.transpose(1, 0, 2).reshape(n, H * dv)
        assert np.abs(o[lo:hi] - one).max(initial=0) < 1e-12


@pytest.mark.parametrize("page,window", [(1, 0), (3, 0), (4, 5), (16, 2)])
def test_oracle_pages_give_the_last_row_of_the_prompt(page, window):
    """Rows appended in two parts, then the newest position's attention: the last row of the
    packed prompt."""
    rng = np.random.default_rng(2)
    H, G, dh, dv, m = 4, 2, 8, 6, 2
    lens = [5, 11, 1]
    cu = np.concatenate([[0], np.cumsum(lens)])
    q, k, v = (rng.standard_normal((cu[-1], w)) for w in (H * dh, G * dh, G * dv))
    o, _, _ = ro.packed_attention(q, k, v, cu, H, G, m, window, 0.3)
    per = -(-max(lens) // page)
    table = rng.permutation(3 * per).reshape(3, per)
    kp, vp = np.full((3 * per, G, page, dh), np.nan), np.full((3 * per, G, page, dv), np.nan)
    first = [0] + list(np.cumsum([n - 1 for n in lens]))
    rows = np.concatenate([np.arange(a, b - 1) for a, b in zip(cu[:-1], cu[1:])])
    kp, vp = ro.append_pages(kp, vp, table, [n - 1 for n in lens], k[rows], v[rows], first)
    last = cu[1:] - 1
    kp, vp = ro.append_pages(kp, vp, table, lens, k[last], v[last], None)
    got, _, _ = ro.paged_attention(q[last], kp, vp, table, lens, H, m, window, 0.3)
    assert np.abs(got - o[last]).max() < 1e-12


def test_oracle_linear_attention_matches_the_closed_form_and_the_scan():
    rng = np.random.default_rng(3)
    n, dk, dv = 9, 4, 3
    q, k, v, g = (rng.standard_normal((n, w)) for w in (dk, dk, dv, 1))
    g = -np.abs(g)
    o, oa, end, _ = ro.linear_attention(q, k, v, g, [0, n], 1, 1, 0.5)
    assert np.abs(o - ro.linear_attention_masked(q, k, v, g[:, 0], 0.5)).max() < 1e-12
    assert (oa >= np.abs(o) - 1e-12).all()
    # a hand-worked step: S = 1, decay 1/2, then v k = 6, q = 1
    o1, _, e1, _ = ro.linear_attention(np.array([[1.0]]), np.array([[2.0]]), np.array([[3.0]]),
                                       np.array([[np.log(0.5)]]), [0, 1], 1, 1, 1.0, np.ones((1, 1, 1, 1)))
    assert abs(o1[0, 0] - 6.5) < 1e-12 and abs(e1[0, 0, 0, 0] - 6.5) < 1e-12
    # the selective scan with one scalar A per head: v = Delta xc, k = B, q = C, g = Delta A
    L, N, P = 7, 5, 4
    xc, B, C = rng.standard_normal((L, P)), rng.standard_normal((L, N)), rng.standard_normal((L, N))
    delta, A = np.abs(rng.standard_normal((L, 1))), -0.7
    ref = oracle.selective_scan(xc, np.repeat(delta, P, 1), np.full((P, N), A), B, C, np.zeros(P))
    y, h = ref[0], ref[1]
    o, _, end, _ = ro.linear_attention(C, B, delta * xc, delta * A, [0, L], 1, 1, 1.0)
    assert np.abs(o - y).max() < 1e-12 and np.abs(end[0, 0] - h).max() < 1e-12


# ------------------------------------------------------------------ argument checks
FAKE = 1 << 28


def _shape(hy, **kw):
    a = dict(n_q_heads=4, n_kv_heads=2, head_dim=64, v_head_dim=128, n_meta=16, window=64, dtype=hy.HYMBA_F16)
    a.update(kw)
    return hy.attn_shape(**a)


BAD_ATTN = [(dict(n_q_heads=0), "INVALID_ARG"), (dict(n_kv_heads=0), "INVALID_ARG"), (dict(n_meta=-1), "INVALID_ARG"),
            (dict(dtype=7), "INVALID_ARG"), (dict(scale=-1.0), "INVALID_ARG"), (dict(scale=NAN), "INVALID_ARG"),
            (dict(scale=INF), "INVALID_ARG"), (dict(head_dim=32), "UNSUPPORTED"), (dict(v_head_dim=96), "UNSUPPORTED"),
            (dict(n_kv_heads=3), "UNSUPPORTED"), (dict(n_q_heads=2048, n_kv_heads=2), "UNSUPPORTED")]


def _packed(hy, shape, q=FAKE, ldq=256, k=FAKE, ldk=128, v=FAKE, ldv=256, cu=FAKE, n=2, rows=10, o=FAKE, ldo=512):
    return hy.hymba_attn_prefill_packed(ctypes.byref(shape) if shape else None, q, ldq, k, ldk, v, ldv, cu, n, rows, o,
                                        ldo, None)


@pytest.mark.parametrize("kw,code", BAD_ATTN)
def test_attention_shapes_refused(hy, kw, code):
    want = getattr(hy, "HYMBA_ERR_" + code)
    s = _shape(hy, **kw)
    assert _packed(hy, s, ldq=1 << 20, ldk=1 << 20, ldv=1 << 20, ldo=1 << 20) == want
    assert hy.hymba_attn_decode_paged_workspace(ctypes.byref(s), 2, 100) == 0


@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(cu=None), dict(cu=FAKE + 2),
                                dict(q=FAKE + 2), dict(k=FAKE + 8), dict(v=FAKE + 8), dict(o=FAKE + 8), dict(ldq=255),
                                dict(ldq=260), dict(ldk=120), dict(ldk=132), dict(ldv=248), dict(ldo=504), dict(n=-1),
                                dict(rows=-1), dict(rows=(1 << 30) + 1)])
def test_packed_attention_arguments_refused(hy, kw):
    assert _packed(hy, _shape(hy), **kw) == hy.HYMBA_ERR_INVALID_ARG
    assert _packed(hy, None) == hy.HYMBA_ERR_INVALID_ARG


def test_packed_attention_without_work(hy):
    """No rows or no sequences: nothing to read, nothing launched."""
    before = hy.hymba_launch_count()
    assert _packed(hy, _shape(hy), rows=0, q=None, k=None, v=None, o=None) == hy.HYMBA_OK
    assert _packed(hy, _shape(hy), n=0) == hy.HYMBA_OK
    assert hy.hymba_launch_count() == before


def _kv(hy, **kw):
    a = dict(k_pages=FAKE, v_pages=FAKE, page_table=FAKE, len=FAKE, n_pages=8, page_size=16, max_pages=4, batch=2,
             n_kv_heads=2, head_dim=64, v_head_dim=128, dtype=hy.HYMBA_F16)
    a.update(kw)
    return hy.hymba_paged_kv(**a)


BAD_KV = [(dict(k_pages=None), "INVALID_ARG"), (dict(v_pages=None), "INVALID_ARG"), (dict(page_table=None), "INVALID_ARG"),
          (dict(len=None), "INVALID_ARG"), (dict(n_pages=0), "INVALID_ARG"), (dict(page_size=0), "INVALID_ARG"),
          (dict(max_pages=0), "INVALID_ARG"), (dict(batch=0), "INVALID_ARG"), (dict(n_kv_heads=0), "INVALID_ARG"),
          (dict(dtype=3), "INVALID_ARG"), (dict(k_pages=FAKE + 8), "INVALID_ARG"), (dict(len=FAKE + 1), "INVALID_ARG"),
          (dict(head_dim=80), "UNSUPPORTED"), (dict(v_head_dim=32), "UNSUPPORTED"),
          (dict(max_pages=1 << 20, page_size=1 << 11), "UNSUPPORTED"), (dict(batch=65536), "UNSUPPORTED")]


@pytest.mark.parametrize("kw,code", BAD_KV)
def test_caches_refused(hy, kw, code):
    want = getattr(hy, "HYMBA_ERR_" + code)
    kv = _kv(hy, **kw)
    assert hy.hymba_kv_append_paged(ctypes.byref(kv), FAKE, 1024, FAKE, 1024, FAKE, 3, None) == want
    s = _shape(hy)
    assert hy.hymba_attn_decode_paged(ctypes.byref(s), FAKE, 256, ctypes.byref(kv), 0, FAKE, 512, FAKE, 1 << 30,
                                      None) == want


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(k=FAKE + 4), dict(v=FAKE + 4), dict(ldk=64), dict(ldv=255),
                                dict(ldk=130), dict(rows=-1), dict(rows=3, cu=None), dict(cu=FAKE + 1)])
def test_append_arguments_refused(hy, kw):
    a = dict(k=FAKE, ldk=128, v=FAKE, ldv=256, cu=FAKE, rows=3)
    a.update(kw)
    kv = _kv(hy)
    assert hy.hymba_kv_append_paged(ctypes.byref(kv), a["k"], a["ldk"], a["v"], a["ldv"], a["cu"], a["rows"],
                                    None) == hy.HYMBA_ERR_INVALID_ARG
    assert hy.hymba_kv_append_paged(None, FAKE, 128, FAKE, 256, FAKE, 3, None) == hy.HYMBA_ERR_INVALID_ARG
    assert hy.hymba_kv_append_paged(ctypes.byref(kv), None, 128, None, 256, FAKE, 0, None) == hy.HYMBA_OK


def test_decode_arguments_refused(hy):
    s, kv = _shape(hy), _kv(hy, max_pages=64)
    need = hy.hymba_attn_decode_paged_workspace(ctypes.byref(s), 2, 64 * 16)
    assert need >= 256 and need % 256 == 0

    def call(shape=s, q=FAKE, ldq=256, cache=kv, max_len=0, o=FAKE, ldo=512, ws=FAKE, n=need):
        return hy.hymba_attn_decode_paged(ctypes.byref(shape), q, ldq, ctypes.byref(cache) if cache else None, max_len,
                                          o, ldo, ws, n, None)

    for kw in (dict(q=None), dict(o=None), dict(ws=None), dict(ws=FAKE + 16), dict(q=FAKE + 2), dict(o=FAKE + 8),
               dict(ldq=128), dict(ldo=511), dict(ldq=257), dict(max_len=-1), dict(max_len=64 * 16 + 1), dict(cache=None)):
        assert call(**kw) == hy.HYMBA_ERR_INVALID_ARG, kw
    assert call(n=need - 1) == hy.HYMBA_ERR_WORKSPACE_TOO_SMALL
    for kw in (dict(n_kv_heads=4), dict(head_dim=128), dict(v_head_dim=64), dict(dtype=hy.HYMBA_BF16)):
        assert call(shape=_shape(hy, **kw), ldq=1024, ldo=1024) == hy.HYMBA_ERR_KV_INCOMPATIBLE, kw
    for b, n in ((0, 100), (2, 0), (2, -5), (65536, 100), (2, (1 << 30) + 1)):
        assert hy.hymba_attn_decode_paged_workspace(ctypes.byref(s), b, n) == 0


def test_decode_workspace_of_one_bound_serves_that_bound(hy):
    """The workspace grows with the splits a call may use and stays small where the batch
    fills the GPU by itself."""
    s = hy.attn_shape(25, 5, 64, 128, 128, 0)
    for batch in (1, 7, 64, 1000):
        for n in (1, 128, 129, 1000, 33000, 1 << 20, 1 << 30):
            w = hy.hymba_attn_decode_paged_workspace(ctypes.byref(s), batch, n)
            assert 0 < w <= max(1 << 20, batch * 25 * 132 * 4 * (148 * 16 // batch + 2) + 256), (batch, n, w)


def _lin(hy, **kw):
    a = dict(n_qk_heads=2, n_heads=4, key_dim=64, v_head_dim=128, dtype=hy.HYMBA_F16)
    a.update(kw)
    return hy.linattn_shape(**a)


BAD_LIN = [(dict(n_qk_heads=0), "INVALID_ARG"), (dict(n_heads=0), "INVALID_ARG"), (dict(v_head_dim=0), "INVALID_ARG"),
           (dict(dtype=9), "INVALID_ARG"), (dict(scale=-0.5), "INVALID_ARG"), (dict(scale=NAN), "INVALID_ARG"),
           (dict(key_dim=32), "UNSUPPORTED"), (dict(v_head_dim=96), "UNSUPPORTED"), (dict(v_head_dim=576), "UNSUPPORTED"),
           (dict(n_qk_heads=3), "UNSUPPORTED"), (dict(n_heads=2048), "UNSUPPORTED")]


def _lin_prefill(hy, s, q=FAKE, ldq=128, k=FAKE, ldk=128, v=FAKE, ldv=512, g=FAKE, ldg=4, cu=FAKE, n=2, rows=10,
                 si=None, so=None, o=FAKE, ldo=512, ws=FAKE, nws=1 << 40):
    return hy.hymba_linattn_prefill(ctypes.byref(s), q, ldq, k, ldk, v, ldv, g, ldg, cu, n, rows, si, so, o, ldo, ws,
                                    nws, None)


def _lin_step(hy, s, q=FAKE, ldq=128, k=FAKE, ldk=128, v=FAKE, ldv=512, g=FAKE, ldg=4, st=FAKE, b=2, o=FAKE, ldo=512):
    return hy.hymba_linattn_step(ctypes.byref(s), q, ldq, k, ldk, v, ldv, g, ldg, st, b, o, ldo, None)


@pytest.mark.parametrize("kw,code", BAD_LIN)
def test_linear_attention_shapes_refused(hy, kw, code):
    want = getattr(hy, "HYMBA_ERR_" + code)
    s = _lin(hy, **kw)
    assert _lin_prefill(hy, s, ldq=1 << 20, ldk=1 << 20, ldv=1 << 20, ldo=1 << 20, ldg=1 << 20) == want
    assert _lin_step(hy, s, ldq=1 << 20, ldk=1 << 20, ldv=1 << 20, ldo=1 << 20, ldg=1 << 20) == want
    assert hy.hymba_linattn_workspace(ctypes.byref(s), 2, 10) == 0


ROWS_KW = [dict(q=None), dict(k=None), dict(v=None), dict(g=None), dict(o=None), dict(q=FAKE + 8), dict(k=FAKE + 8),
           dict(v=FAKE + 2), dict(o=FAKE + 4), dict(g=FAKE + 2), dict(ldq=64), dict(ldk=132), dict(ldv=504), dict(ldo=0),
           dict(ldg=3), dict(ldg=-4)]


@pytest.mark.parametrize("kw", ROWS_KW)
def test_linear_attention_rows_refused(hy, kw):
    s = _lin(hy)
    assert _lin_prefill(hy, s, **kw) == hy.HYMBA_ERR_INVALID_ARG
    assert _lin_step(hy, s, **kw) == hy.HYMBA_ERR_INVALID_ARG


def test_linear_attention_arguments_refused(hy):
    s = _lin(hy)
    st = 2 * 4 * 128 * 64 * 4  # bytes of the states of two sequences
    for kw in (dict(cu=None), dict(cu=FAKE + 2), dict(n=-1), dict(rows=-1), dict(rows=(1 << 30) + 1), dict(ws=None),
               dict(ws=FAKE + 128), dict(si=FAKE + 4), dict(so=FAKE + 8), dict(si=FAKE, so=FAKE + st - 16),
               dict(so=FAKE, si=FAKE + 16)):
        assert _lin_prefill(hy, s, **kw) == hy.HYMBA_ERR_INVALID_ARG, kw
    need = hy.hymba_linattn_workspace(ctypes.byref(s), 2, 10)
    assert need >= 256
    assert _lin_prefill(hy, s, nws=need - 1) == hy.HYMBA_ERR_WORKSPACE_TOO_SMALL
    assert _lin_prefill(hy, s, n=0) == hy.HYMBA_OK
    for kw in (dict(st=None), dict(st=FAKE + 8), dict(b=0), dict(b=-3)):
        assert _lin_step(hy, s, **kw) == hy.HYMBA_ERR_INVALID_ARG, kw
    for n, rows in ((0, 10), (-1, 10), (2, -1), (2, (1 << 30) + 1)):
        assert hy.hymba_linattn_workspace(ctypes.byref(s), n, rows) == 0


def test_linear_attention_workspace_of_few_long_prompts(hy):
    """One long prompt of 16-bit rows is cut, and its segments' states need room; short ones, many
    sequences, enough heads, fp32 rows and other key dims need none. A call with too little is
    refused, also where a larger batch would have needed less."""
    ws = lambda s, n, rows: hy.hymba_linattn_workspace(ctypes.byref(s), n, rows)
    H, dk, dv = 4, 64, 128
    state = H * dk * dv * 4
    s = hy.linattn_shape(2, H, dk, dv, hy.HYMBA_BF16)
    for n, rows in ((1, 8192), (3, 5000), (4, 20000)):
        assert 3 * state < ws(s, n, rows) < 148 * (state + H * 4) + 256, (n, rows)
    for n, rows in ((1, 0), (1, 300), (1, 1000), (8, 8000), (33, 100000), (500, 1 << 30)):
        assert ws(s, n, rows) == 256, (n, rows)
    for other in (hy.linattn_shape(2, H, dk, dv, hy.HYMBA_F32), hy.linattn_shape(2, H, 16, dv, hy.HYMBA_BF16),
                  hy.linattn_shape(2, H, 128, dv, hy.HYMBA_F16), hy.linattn_shape(75, 75, dk, dv, hy.HYMBA_F16)):
        assert ws(other, 1, 8192) == 256
    s = _lin(hy, dtype=hy.HYMBA_F16)
    assert _lin_prefill(hy, s, n=1, rows=8192, nws=ws(s, 40, 8192)) == hy.HYMBA_ERR_WORKSPACE_TOO_SMALL
    assert _lin_prefill(hy, s, n=1, rows=8192, nws=ws(s, 1, 8192) - 1) == hy.HYMBA_ERR_WORKSPACE_TOO_SMALL


# ------------------------------------------------------------------ the torch helpers
def test_helpers_refuse_tensors_that_do_not_fit(hy):
    import torch
    from hybrid_head_ssm_b200 import runtime as rt
    s = _shape(hy)
    f16 = torch.float16
    q, k, v, o = (torch.zeros(10, w, dtype=f16) for w in (256, 128, 256, 512))
    cu = torch.zeros(3, dtype=torch.int32)
    for bad in (dict(q=q[:, :128]), dict(q=q.float()), dict(k=k[:9]), dict(v=v.t().contiguous().t()),
                dict(o=o[None]), dict(cu=cu.long()), dict(cu=cu[None])):
        a = dict(q=q, k=k, v=v, cu=cu, o=o)
        a.update(bad)
        with pytest.raises(ValueError):
            rt.attn_prefill_packed(s, a["q"], a["k"], a["v"], a["cu"], a["o"])
    kp, vp = torch.zeros(8, 2, 16, 64, dtype=f16), torch.zeros(8, 2, 16, 128, dtype=f16)
    table, ln = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for bad in (dict(kp=kp.double()), dict(vp=vp.float()), dict(vp=vp[:7]), dict(kp=kp.transpose(0, 1)),
                dict(table=table.long()), dict(table=table[:, ::2]), dict(ln=ln[:1])):
        a = dict(kp=kp, vp=vp, table=table, ln=ln)
        a.update(bad)
        with pytest.raises(ValueError):
            rt.PagedKV(a["kp"], a["vp"], a["table"], a["ln"])
    kv = rt.PagedKV(kp, vp, table, ln)
    with pytest.raises(ValueError):
        rt.kv_append_paged(kv, k[:2], v[:3])
    with pytest.raises(ValueError):
        rt.kv_append_paged(kv, k, v, cu[:2])
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError):
        rt.attn_decode_paged(s, q, kv, o[:2], ws)
    with pytest.raises(ValueError):
        rt.decode_paged_workspace(s, 0, 10)
    ls = _lin(hy)
    lq, lv, lo = torch.zeros(10, 128, dtype=f16), torch.zeros(10, 512, dtype=f16), torch.zeros(10, 512, dtype=f16)
    g, st = torch.zeros(10, 4), torch.zeros(2, 4, 128, 64)
    for bad in (dict(g=g.half()), dict(g=g[:9]), dict(g=g[0, :3]), dict(st=st[:1]), dict(st=st.half()),
                dict(st=st.transpose(2, 3))):
        a = dict(g=g, st=st)
        a.update(bad)
        with pytest.raises(ValueError):
            rt.linattn_prefill(ls, lq, lq, lv, a["g"], cu, lo, ws, a["st"])
    with pytest.raises(ValueError):
        rt.linattn_step(ls, lq, lq, lv, g, st, lo)
    # tensors that fit, but not on a GPU: never handed to a kernel
    table[:] = 1
    for call in (lambda: rt.attn_prefill_packed(s, q, k, v, cu, o), lambda: rt.kv_append_paged(kv, k, v, cu),
                 lambda: rt.attn_decode_paged(s, q[:2], kv, o[:2], ws),
                 lambda: rt.linattn_prefill(ls, lq, lq, lv, g, cu, lo, ws, st, st),
                 lambda: rt.linattn_step(ls, lq[:2], lq[:2], lv[:2], g[:2], st, lo[:2])):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_workload_shapes_are_accepted(hy):
    """The 1.5B layer's heads and its SSD form's (50 heads of 64 channels, 16 states, shared
    keys)."""
    c = synth.hymba15_layer_cfg(1024)
    s = hy.attn_shape(c.n_q_heads, c.n_kv_heads, c.head_dim, c.v_head_dim, c.n_meta, c.window)
    assert hy.hymba_attn_decode_paged_workspace(ctypes.byref(s), 64, 4224) > 0
    assert hy.hymba_linattn_workspace(ctypes.byref(hy.linattn_shape(1, 50, 16, 64)), 8, 8 * 4224) > 0
