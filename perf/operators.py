"""The operators of a ragged batch, as cases to measure: attention over packed prompts, the paged
K/V cache (rows written into it, attention of one new token over it), and linear attention with a
decay per head (whole prompts, single tokens).

`run(state)` computes one pass: with `own` false in elementary torch operations (32 bits, rounded
once at the end), with `own` true through this repository's entry points. `exact` states the same
operators in 64 bits, loop by loop from their definitions.

Sizes are those of the 1.5B layer (25 query heads on 5 KV heads of 64, V heads of 128, 128 meta
tokens, window 1024), of the tiny fp32 layer (4 heads on 2, 16 meta tokens, window 64) and of the
50 SSM heads of the SSD form (16 states, 64 channels, shared keys).
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ESZ = {"f16": 2, "bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------------------------
def _attn(op, dtype, heads, dims, meta, window, seqs, longest, **more):
    return dict(op=op, dtype=dtype, q_heads=heads[0], kv_heads=heads[1], head_dim=dims[0], v_dim=dims[1],
                meta=meta, window=window, seqs=seqs, longest=longest, **more)


def _lin(op, dtype, qk_heads, heads, key_dim, v_dim, seqs, longest=1, start=True):
    return dict(op=op, dtype=dtype, qk_heads=qk_heads, heads=heads, key_dim=key_dim, v_dim=v_dim, seqs=seqs,
                longest=longest, start=start)


def listed():
    big = ((25, 5), (64, 128))
    return [
        # two short prompts of the tiny fp32 layer: the smallest prompt call
        dict(_attn("prefill", "f32", (4, 2), (64, 128), 16, 64, 2, 272), name="prefill_tiny_f32"),
        # a batch of prompts of different lengths through a sliding-window layer
        dict(_attn("prefill", "f16", *big, 128, 1024, 8, 4224), name="prefill_swa_batch"),
        # long prompts through a global layer: the largest amount of arithmetic
        dict(_attn("prefill", "bf16", *big, 128, 0, 3, 8320), name="prefill_global_long"),
        # the K and V of a batch of prompts on their way into the cache
        dict(_attn("append", "f16", *big, 128, 0, 8, 4224, page=64, new=0), name="append_prompts"),
        # one new token of every sequence on its way into the cache
        dict(_attn("append", "f16", *big, 128, 0, 64, 4224, page=16, new=1), name="append_tokens"),
        # a single conversation: latency
        dict(_attn("decode", "f16", *big, 128, 0, 1, 1153, page=16), name="decode_one"),
        # a serving batch in a sliding-window layer
        dict(_attn("decode", "f16", *big, 128, 1024, 64, 4224, page=64), name="decode_swa_batch"),
        # a serving batch of long contexts in a global layer
        dict(_attn("decode", "bf16", *big, 128, 0, 16, 32896, page=32), name="decode_global_long"),
        # one short prompt through the recurrent heads
        dict(_lin("linear", "f16", 25, 25, 64, 128, 1, 185, start=False), name="linear_one_short"),
        # a batch of prompts through the recurrent heads
        dict(_lin("linear", "bf16", 25, 25, 64, 128, 8, 4224), name="linear_batch"),
        # one token of one sequence of the recurrent heads, fp32: latency
        dict(_lin("step", "f32", 25, 25, 64, 128, 1), name="step_one_f32"),
        # one token of every sequence of a serving batch
        dict(_lin("step", "bf16", 25, 25, 64, 128, 256), name="step_batch"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "append", "decode", "decode", "linear", "linear", "step"])
    dtype = rng.choice(["f16", "f16", "bf16", "bf16", "f32"])
    if op in ("linear", "step"):
        qk, heads = rng.choice([(25, 25), (1, 50), (5, 25), (4, 4), (8, 16)])
        key_dim, v_dim = rng.choice([(16, 64), (64, 64), (64, 128), (128, 128), (128, 64)])
        if op == "step":
            return _lin("step", dtype, qk, heads, key_dim, v_dim, _log(rng, 1, 100))
        seqs = _log(rng, 1, 12)
        longest = _log(rng, 1, 1000 if dtype == "f32" else 2000)
        return _lin("linear", dtype, qk, heads, key_dim, v_dim, seqs, longest, rng.random() < 0.5)
    heads = rng.choice([(25, 5), (25, 5), (4, 2), (16, 16), (32, 8), (8, 1)])
    dims = rng.choice([(64, 128), (64, 64), (128, 128)])
    meta = rng.choice([0, 16, 128, rng.randrange(1, 200)])
    window = rng.choice([0, 0, 64, 1024, _log(rng, 1, 2000)])
    if op == "prefill":
        seqs = _log(rng, 1, 12)
        longest = _log(rng, 1, 700 if dtype == "f32" else 2500)
        return _attn("prefill", dtype, heads, dims, meta, window, seqs, longest)
    page = rng.choice([16, 32, 64, 128, rng.randrange(1, 100)])
    seqs = _log(rng, 1, 40)
    longest = _log(rng, 1, 6000)
    if op == "append":
        return _attn("append", dtype, heads, dims, meta, window, seqs, longest, page=page, new=rng.choice([0, 1]))
    return _attn("decode", dtype, heads, dims, meta, window, seqs, longest, page=page)


def _lengths(case):
    """The lengths of the case's sequences: the longest first, then anything from nothing to that
    (linear draws), a single row and an empty one among them."""
    n, longest = case["seqs"], case["longest"]
    rng = random.Random(1000003 * n + longest)
    lens = [longest] + [rng.randint((longest + 1) // 2, longest) if rng.random() < 0.6 else rng.randint(0, longest)
                        for _ in range(n - 1)]
    if n >= 4:
        lens[2] = 1
        lens[3] = 0
    return lens


def _visible(length, meta, window):
    """Keys the newest of `length` positions sees."""
    if length <= 0:
        return 0
    if window <= 0:
        return length
    i = length - 1
    m = min(meta, length)
    return m + max(0, i + 1 - max(meta, i - window + 1))


def work(case):
    e = ESZ[case["dtype"]]
    lens = _lengths(case)
    if case["op"] in ("linear", "step"):
        H, Hk, dk, dv = case["heads"], case["qk_heads"], case["key_dim"], case["v_dim"]
        rows = case["seqs"] if case["op"] == "step" else sum(lens)
        state = 4 * case["seqs"] * H * dk * dv * (2 if case["start"] else 1)
        return {"bytes": rows * (2 * Hk * dk + 2 * H * dv) * e + 4 * rows * H + state,
                "flops": 4.0 * rows * H * dk * dv}
    H, G, dh, dv = case["q_heads"], case["kv_heads"], case["head_dim"], case["v_dim"]
    if case["op"] == "prefill":
        m, w = case["meta"], case["window"]
        pairs = 0
        for n in lens:
            if w <= 0 or n <= m + w:
                pairs += n * (n + 1) // 2
            else:
                short = m + w
                pairs += short * (short + 1) // 2 + (n - short) * (m + w)
        return {"bytes": sum(lens) * (H * (dh + dv) + G * (dh + dv)) * e, "flops": 2.0 * pairs * H * (dh + dv)}
    if case["op"] == "append":
        rows = sum(min(1, n) if case["new"] else n for n in lens)
        return {"bytes": 2 * rows * G * (dh + dv) * e, "flops": 0}
    keys = sum(_visible(n, case["meta"], case["window"]) for n in lens)
    return {"bytes": keys * G * (dh + dv) * e + case["seqs"] * H * (dh + dv) * e, "flops": 2.0 * keys * H * (dh + dv)}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
PAD = 3  # rows behind the last sequence, which every operator leaves as they were


def _offsets(lens, dev):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    lens = _lengths(case)
    n = case["seqs"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dt)

    st = {"case": case, "lens": lens, "kept": {}}
    if case["op"] in ("linear", "step"):
        H, Hk, dk, dv = case["heads"], case["qk_heads"], case["key_dim"], case["v_dim"]
        rows = n if case["op"] == "step" else sum(lens) + PAD
        # one projection's columns: q | k | v; the keys come normalised, as such layers have them
        p = torch.empty(rows, 2 * Hk * dk + H * dv, dtype=dt, device=dev)
        p[:, :Hk * dk] = normal(rows, Hk * dk)
        k = torch.randn(rows, Hk, dk, generator=gen, device=dev)
        p[:, Hk * dk:2 * Hk * dk] = (k / k.norm(dim=2, keepdim=True)).reshape(rows, Hk * dk).to(dt)
        p[:, 2 * Hk * dk:] = normal(rows, H * dv)
        st["q"], st["k"], st["v"] = p[:, :Hk * dk], p[:, Hk * dk:2 * Hk * dk], p[:, 2 * Hk * dk:]
        # log decays: Delta_t * A as in the SSM heads, A = -U[1, 16] per head, Delta in [1e-3, 1e-1]
        a = torch.rand(H, generator=gen, device=dev) * 15 + 1
        d = torch.exp(torch.rand(rows, H, generator=gen, device=dev) * math.log(100) + math.log(1e-3))
        st["g"] = -(a * d)
        st["state"] = torch.randn(n, H, dv, dk, generator=gen, device=dev) if case["start"] else None
        st["end"] = torch.zeros(n, H, dv, dk, device=dev)
        st["o"] = torch.zeros(rows, H * dv, dtype=dt, device=dev)
        if case["op"] == "linear":
            st["cu"] = _offsets(lens, dev)
        return st
    H, G, dh, dv = case["q_heads"], case["kv_heads"], case["head_dim"], case["v_dim"]
    if case["op"] == "prefill":
        rows = sum(lens) + PAD
        p = normal(rows, H * dh + G * (dh + dv))  # the fused projection's columns Q | K | V
        st["q"], st["k"], st["v"] = p[:, :H * dh], p[:, H * dh:(H + G) * dh], p[:, (H + G) * dh:]
        st["cu"] = _offsets(lens, dev)
        st["o"] = torch.zeros(rows, H * dv, dtype=dt, device=dev)
        return st
    page = case["page"]
    need = [-(-x // page) for x in lens]
    per_seq = max(1, max(need))
    n_pages = sum(need) + 2
    order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    table = torch.full((n, per_seq), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = order[at:at + c]
        at += c
    st["table"] = table
    st["len"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    if case["op"] == "decode":
        # sequences that start with the same text share its pages
        if n >= 2:
            shared = min(need[0], need[1]) // 2
            table[1, :shared] = table[0, :shared]
        st["k_pages"], st["v_pages"] = normal(n_pages, G, page, dh), normal(n_pages, G, page, dv)
        st["q"] = normal(n, H * dh)
        st["o"] = torch.zeros(n, H * dv, dtype=dt, device=dev)
        return st
    st["k_pages"] = torch.zeros(n_pages, G, page, dh, dtype=dt, device=dev)
    st["v_pages"] = torch.zeros(n_pages, G, page, dv, dtype=dt, device=dev)
    if case["new"]:
        # one row for each sequence that holds anything
        st["cu"] = _offsets([min(1, x) for x in lens], dev)
        st["new"] = [min(1, x) for x in lens]
    else:
        st["cu"] = _offsets(lens, dev)
        st["new"] = lens
    p = normal(sum(st["new"]) + PAD, G * (dh + dv))
    st["k"], st["v"] = p[:, :G * dh], p[:, G * dh:]
    return st


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"prefill": _own_prefill, "append": _own_append, "decode": _own_decode, "linear": _own_linear,
                "step": _own_step}[op](state)
    return {"prefill": _plain_prefill, "append": _plain_append, "decode": _plain_decode, "linear": _plain_linear,
            "step": _plain_step}[op](state)


def _own_shape(state):
    """The handles a program keeps between calls: shapes, cache and workspace."""
    import hybrid_head_ssm_b200 as hy
    from hybrid_head_ssm_b200 import runtime as rt
    kept, c = state["kept"], state["case"]
    if "rt" in kept:
        return kept
    kept["rt"] = rt
    code = {"f16": hy.HYMBA_F16, "bf16": hy.HYMBA_BF16, "f32": hy.HYMBA_F32}[c["dtype"]]
    if c["op"] in ("linear", "step"):
        kept["shape"] = hy.linattn_shape(n_qk_heads=c["qk_heads"], n_heads=c["heads"], key_dim=c["key_dim"],
                                         v_head_dim=c["v_dim"], dtype=code)
        if c["op"] == "linear":
            kept["ws"] = rt.linattn_workspace(kept["shape"], c["seqs"], state["q"].shape[0])
        return kept
    kept["shape"] = hy.attn_shape(n_q_heads=c["q_heads"], n_kv_heads=c["kv_heads"], head_dim=c["head_dim"],
                                  v_head_dim=c["v_dim"], n_meta=c["meta"], window=c["window"], dtype=code)
    if c["op"] != "prefill":
        kept["kv"] = rt.PagedKV(state["k_pages"], state["v_pages"], state["table"], state["len"])
    if c["op"] == "decode":
        kept["ws"] = rt.decode_paged_workspace(kept["shape"], c["seqs"], c["longest"])
    return kept


def _own_prefill(s):
    h = _own_shape(s)
    h["rt"].attn_prefill_packed(h["shape"], s["q"], s["k"], s["v"], s["cu"], s["o"])
    return s["o"]


def _own_append(s):
    h = _own_shape(s)
    h["rt"].kv_append_paged(h["kv"], s["k"], s["v"], s["cu"])
    return s["k_pages"], s["v_pages"]


def _own_decode(s):
    h = _own_shape(s)
    h["rt"].attn_decode_paged(h["shape"], s["q"], h["kv"], s["o"], h["ws"], s["case"]["longest"])
    return s["o"]


def _own_linear(s):
    h = _own_shape(s)
    h["rt"].linattn_prefill(h["shape"], s["q"], s["k"], s["v"], s["g"], s["cu"], s["o"], h["ws"],
                            state_in=s["state"], state_out=s["end"])
    return s["o"], s["end"]


def _own_step(s):
    h = _own_shape(s)
    h["rt"].linattn_step(h["shape"], s["q"], s["k"], s["v"], s["g"], s["state"], s["o"])
    return s["o"], s["state"]


def _rows(s, longest):
    """Row of (sequence, place), where that is inside the sequence, and back: (sequence, place) of a
    row, and where a row belongs to a sequence."""
    cu = s["cu"].long()
    at = torch.arange(longest, device=cu.device)
    rows = cu[:-1, None] + at
    inside = rows < cu[1:, None]
    r = torch.arange(s["q"].shape[0] if "q" in s else s["k"].shape[0], device=cu.device)
    seq = (torch.searchsorted(cu, r, right=True) - 1).clamp(max=cu.numel() - 2)
    return rows.clamp(max=r.numel() - 1), inside, seq, r - cu[seq], r < cu[-1]


def _plain_prefill(s):
    c = s["case"]
    H, G, dh, dv, n, L = c["q_heads"], c["kv_heads"], c["head_dim"], c["v_dim"], c["seqs"], c["longest"]
    rows, inside, seq, place, real = _rows(s, L)
    q = s["q"][rows].float().view(n, L, G, H // G, dh).permute(0, 2, 3, 1, 4)
    k = s["k"][rows].float().view(n, L, G, 1, dh).permute(0, 2, 3, 4, 1)
    v = s["v"][rows].float().view(n, L, G, 1, dv).permute(0, 2, 3, 1, 4)
    i = torch.arange(L, device=q.device)
    far = i[:, None] - i
    see = far >= 0
    if c["window"] > 0:
        see = see & ((i < c["meta"]) | (far < c["window"]))
    x = torch.matmul(q * (1 / math.sqrt(dh)), k)
    x.masked_fill_(~see, -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(x, v) / x.sum(-1, keepdim=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(n, L, H * dv)[seq, place.clamp(max=L - 1)].to(s["o"].dtype)
    return torch.where(real[:, None], o, s["o"])


def _plain_append(s):
    cu = s["cu"].long()
    n, page, G = s["case"]["seqs"], s["case"]["page"], s["case"]["kv_heads"]
    r = torch.arange(sum(s["new"]), device=cu.device)
    seq = torch.searchsorted(cu, r, right=True) - 1
    pos = s["len"].long()[seq] - (cu[1:] - cu[:-1])[seq] + r - cu[seq]
    to = s["table"].long()[seq, pos // page]
    s["k_pages"][to, :, pos % page] = s["k"][:r.numel()].view(r.numel(), G, -1)
    s["v_pages"][to, :, pos % page] = s["v"][:r.numel()].view(r.numel(), G, -1)
    return s["k_pages"], s["v_pages"]


def _plain_decode(s):
    c = s["case"]
    H, G, dh, dv, n, page = c["q_heads"], c["kv_heads"], c["head_dim"], c["v_dim"], c["seqs"], c["page"]
    most = max(1, max(_visible(x, c["meta"], c["window"]) for x in s["lens"]))
    length = s["len"].long()[:, None]
    j = torch.arange(most, device=length.device)
    if c["window"] > 0:
        m = length.clamp(max=c["meta"])
        lo = (length - c["window"]).clamp(min=c["meta"])
        pos = torch.where(j < m, j, lo + j - m)
    else:
        pos = j.expand(n, most)
    see = pos < length
    pos = torch.where(see, pos, 0)
    at = s["table"].long().gather(1, pos // page).clamp(min=0)
    k = s["k_pages"][at, :, pos % page].float().permute(0, 2, 3, 1)
    v = s["v_pages"][at, :, pos % page].float().permute(0, 2, 1, 3)
    q = s["q"].float().view(n, G, H // G, dh) * (1 / math.sqrt(dh))
    x = torch.matmul(q, k).masked_fill(~see[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = x.sum(-1, keepdim=True)
    o = torch.where(total > 0, torch.matmul(x, v) / total, 0.0)
    return o.reshape(n, H * dv).to(s["o"].dtype)


def _plain_linear(s):
    c = s["case"]
    H, Hk, dk, dv, n, L = c["heads"], c["qk_heads"], c["key_dim"], c["v_dim"], c["seqs"], c["longest"]
    rows, inside, seq, place, real = _rows(s, L)
    q = s["q"][rows].float().view(n, L, Hk, 1, dk).permute(0, 2, 3, 1, 4) * (1 / math.sqrt(dk))
    k = s["k"][rows].float().view(n, L, Hk, 1, dk).permute(0, 2, 3, 1, 4)
    v = s["v"][rows].float().view(n, L, Hk, H // Hk, dv).permute(0, 2, 3, 1, 4)
    g = torch.where(inside[:, :, None], s["g"][rows].double(), 0.0).view(n, L, Hk, H // Hk).permute(0, 2, 3, 1)
    sums = g.cumsum(-1)  # long sums in 64 bits
    i = torch.arange(L, device=q.device)
    fade = (sums[..., :, None] - sums[..., None, :]).float()
    fade.masked_fill_(i[:, None] < i, -math.inf).exp_()
    o = torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * fade, v)
    left = torch.where(inside[:, None, None], torch.exp(sums[..., -1:] - sums), 0.0).float()
    end = torch.matmul((v * left[..., None]).transpose(-1, -2), k)
    if s["state"] is not None:
        first = s["state"].view(n, Hk, H // Hk, dv, dk)
        o = o + torch.matmul(q, first.transpose(-1, -2)) * torch.exp(sums).float()[..., None]
        end = end + first * torch.exp(sums[..., -1:, None]).float()
    o = o.permute(0, 3, 1, 2, 4).reshape(n, L, H * dv)[seq, place.clamp(max=L - 1)].to(s["o"].dtype)
    return torch.where(real[:, None], o, s["o"]), end.reshape(n, H, dv, dk)


def _plain_step(s):
    c = s["case"]
    H, Hk, dk, dv, n = c["heads"], c["qk_heads"], c["key_dim"], c["v_dim"], c["seqs"]
    q = s["q"].float().view(n, Hk, 1, 1, dk) * (1 / math.sqrt(dk))
    k = s["k"].float().view(n, Hk, 1, 1, dk)
    v = s["v"].float().view(n, Hk, H // Hk, dv, 1)
    state = s["state"].view(n, Hk, H // Hk, dv, dk)
    state.mul_(torch.exp(s["g"]).view(n, Hk, H // Hk, 1, 1)).add_(v * k)
    return (state * q).sum(-1).reshape(n, H * dv).to(s["o"].dtype), s["state"]


# ---------------------------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------
def _softmax_rows(q, k, v, see):
    """Weights exp(q.k / sqrt(d)) over the keys each row sees, normalised, on the values."""
    x = (q @ k.T) / math.sqrt(q.shape[1])
    x = x.masked_fill(~see, -math.inf)
    return torch.softmax(x, -1) @ v


def exact(case, seed):
    s = prepare(case, seed)
    lens, dev = s["lens"], "cuda"
    if case["op"] in ("linear", "step"):
        H, Hk, dk, dv, n = case["heads"], case["qk_heads"], case["key_dim"], case["v_dim"], case["seqs"]
        o = s["o"].double()
        S = s["state"].double() if s["state"] is not None else torch.zeros(n, H, dv, dk, dtype=torch.float64, device=dev)
        head = torch.arange(H, device=dev) // (H // Hk)
        if case["op"] == "step":
            start, lens = list(range(n)), [1] * n
        else:
            start = [sum(lens[:b]) for b in range(n)]
        q = s["q"].double().view(-1, Hk, dk)[:, head] / math.sqrt(dk)
        k = s["k"].double().view(-1, Hk, dk)[:, head]
        v = s["v"].double().view(-1, H, dv)
        fade = torch.exp(s["g"].double())
        # S_t = exp(g_t) S_{t-1} + v_t k_t^T, o_t = S_t q_t, all sequences that are that long at a time
        first = torch.tensor(start, device=dev)
        by_len = sorted(range(n), key=lambda b: -lens[b])
        order = torch.tensor(by_len, device=dev)
        S = S[order].contiguous()
        out = o.view(-1, H, dv)
        for t in range(max(lens)):
            m = sum(x > t for x in lens)
            r = first[order[:m]] + t
            S[:m].mul_(fade[r][:, :, None, None]).add_(v[r][..., None] * k[r][:, :, None])
            out[r] = torch.matmul(S[:m], q[r][..., None])[..., 0]
        end = torch.empty_like(S)
        end[order] = S
        return o, end
    H, G, dh, dv = case["q_heads"], case["kv_heads"], case["head_dim"], case["v_dim"]
    meta, window = case["meta"], case["window"]
    if case["op"] == "prefill":
        o = s["o"].double()
        at = 0
        for length in lens:
            i = torch.arange(length, device=dev)
            see = i[None] <= i[:, None]
            if window > 0:
                see &= (i[None] < meta) | (i[:, None] - i[None] < window)
            for h in range(H):
                g = h // (H // G)
                seq = slice(at, at + length)
                if length:
                    o[seq, h * dv:(h + 1) * dv] = _softmax_rows(
                        s["q"][seq, h * dh:(h + 1) * dh].double(), s["k"][seq, g * dh:(g + 1) * dh].double(),
                        s["v"][seq, g * dv:(g + 1) * dv].double(), see)
            at += length
        return o
    page, table = case["page"], s["table"].tolist()
    if case["op"] == "append":
        # numbers that are copied: the pages themselves
        k_pages, v_pages, at = s["k_pages"].double(), s["v_pages"].double(), 0
        for b, new in enumerate(s["new"]):
            first, last = lens[b] - new, lens[b]
            while first < last:
                end = min(last, (first // page + 1) * page)
                p, c0, m = table[b][first // page], first % page, end - first
                k_pages[p, :, c0:c0 + m] = s["k"][at:at + m].double().view(m, G, dh).transpose(0, 1)
                v_pages[p, :, c0:c0 + m] = s["v"][at:at + m].double().view(m, G, dv).transpose(0, 1)
                first, at = end, at + m
        return k_pages, v_pages
    o = torch.zeros(case["seqs"], H * dv, dtype=torch.float64, device=dev)
    for b, length in enumerate(lens):
        if not length:
            continue
        pages = s["table"][b, :-(-length // page)].long()
        k = s["k_pages"][pages].double().transpose(0, 1).reshape(G, -1, dh)[:, :length]
        v = s["v_pages"][pages].double().transpose(0, 1).reshape(G, -1, dv)[:, :length]
        j = torch.arange(length, device=dev)
        see = (j < meta) | (length - 1 - j < window) if window > 0 else j >= 0
        q = s["q"][b].double().view(G, H // G, dh)
        o[b] = torch.cat([_softmax_rows(q[g], k[g], v[g], see[None]) for g in range(G)]).reshape(-1)
    return o
