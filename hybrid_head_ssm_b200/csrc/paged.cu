// Paged K/V cache of a batch of sequences: new rows into pages, and attention of one new
// token per sequence over them ("Lecture 04", section 1: decode reads every cached K and V
// of the span), split over the cache's length and joined.
//
// Pages: k_pages [n_pages, G, page, dh], v_pages [n_pages, G, page, dv]; position p of
// sequence b is slot p mod page of page table[b][p / page]. The newest position len[b] - 1
// sees [0, min(n_meta, len)) and [lo, len), lo = max(n_meta, len - window) (n_meta when
// global): visible key j is position j below the meta end and lo + j - meta end above it.
#include <algorithm>

#include "kernels.h"
#include "ragged.cuh"

namespace hymba {

namespace {

constexpr float LOG2E = 1.4426950408889634f;

// ---------------------------------------------------------------------------
// rows into pages
// ---------------------------------------------------------------------------
struct AppendArgs {
    uint8_t *k_pages, *v_pages;
    const uint8_t *k, *v;
    const int *table, *len, *cu;
    long long ldk, ldv;  // bytes
    int n_pages, page, max_pages, batch, rows, G;
    int kshift, vshift;  // log2 of the 16-byte pieces of one head's row
};

// One warp per row: its sequence by binary search, its slot from the page table, then
// 16-byte pieces from the row into the heads' slots. Bound by HBM: every byte is read
// once and written once.
__global__ void __launch_bounds__(256) kv_append_kernel(const AppendArgs a, int* status) {
    griddep_sync();
    if (a.cu && blockIdx.x == 0)
        for (int s = threadIdx.x; s < a.batch; s += blockDim.x) {
            int st, n;
            if (!ragged::sequence(a.cu, s, a.rows, &st, &n)) set_status(status, HYMBA_ERR_DEVICE_RANGE);
        }
    const long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (r >= a.rows) return;
    int b = (int)r, back = 1;  // the row is position len - back of sequence b
    if (a.cu) {
        int lo = 0, hi = a.batch;  // the last sequence that starts at or before r
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.cu[mid] <= r) lo = mid;
            else hi = mid;
        }
        b = lo;
        int st, n;
        if (!ragged::sequence(a.cu, b, a.rows, &st, &n) || r < st || r >= st + n) return;
        back = (int)(st + n - r);
    }
    const int len = a.len[b];
    const long long pos = (long long)len - back;
    int at = -1;
    if (pos >= 0 && len <= (long long)a.max_pages * a.page)
        at = a.table[(long long)b * a.max_pages + (int)pos / a.page];
    if (at < 0 || at >= a.n_pages) {
        if (lane == 0) set_status(status, HYMBA_ERR_DEVICE_RANGE);
        return;
    }
    const long long slot = (long long)at * a.G * a.page + (int)pos % a.page;  // + g * page: the head's row
    const uint8_t* kr = a.k + r * a.ldk;
    const uint8_t* vr = a.v + r * a.ldv;
    for (int c = lane; c < a.G << a.kshift; c += 32) {
        const int g = c >> a.kshift, e = c & ((1 << a.kshift) - 1);
        *reinterpret_cast<uint4*>(a.k_pages + (((slot + (long long)g * a.page) << a.kshift) + e) * 16) =
            *reinterpret_cast<const uint4*>(kr + c * 16);
    }
    for (int c = lane; c < a.G << a.vshift; c += 32) {
        const int g = c >> a.vshift, e = c & ((1 << a.vshift) - 1);
        *reinterpret_cast<uint4*>(a.v_pages + (((slot + (long long)g * a.page) << a.vshift) + e) * 16) =
            *reinterpret_cast<const uint4*>(vr + c * 16);
    }
}

// ---------------------------------------------------------------------------
// one new token
// ---------------------------------------------------------------------------
template <typename T>
struct DecodeArgs {
    const T *q, *k_pages, *v_pages;
    T* o;
    const int *table, *len;
    long long ldq, ldo;
    float* part;  // [batch, H, n_split, dv + 4]: sum of p v, the max (log2 units), the sum of p (< 0: a bad page)
    int n_pages, page, max_pages, max_len, H, G, n_meta, window, split_keys, n_split;
    float scale_log2;
};

struct View {
    int len, meta, lo, n;  // visible keys: positions [0, meta) and [lo, len)
    __device__ __forceinline__ int pos(int j) const { return j < meta ? j : lo + (j - meta); }
};
// false: the length is out of range
template <typename T>
__device__ __forceinline__ bool view_of(const DecodeArgs<T>& a, int b, View* w) {
    w->len = a.len[b];
    const bool ok = w->len >= 0 && w->len <= a.max_len;
    if (!ok) w->len = 0;
    w->meta = min(a.n_meta, w->len);
    w->lo = a.window > 0 ? max(a.n_meta, w->len - a.window) : a.n_meta;
    w->n = w->meta + max(0, w->len - w->lo);
    return ok;
}
// slot of (page entry, KV head 0): row index of head g is + g * page; -1: a page out of range
template <typename T>
__device__ __forceinline__ long long slot_of(const DecodeArgs<T>& a, int b, int pos) {
    const int at = a.table[(long long)b * a.max_pages + pos / a.page];
    if (at < 0 || at >= a.n_pages) return -1;
    return (long long)at * a.G * a.page + pos % a.page;
}

// CUDA cores (fp32 rows): one 128-thread block per (key split, KV head and group of up to 8
// of its query heads, sequence). Chunks of 128 keys: a thread forms one key's scores, two
// heads' softmax per warp, then a thread owns a column of V.
constexpr int SC = 128, SR = 8;

template <typename T, int DH, int DV>
__global__ void __launch_bounds__(128) decode_paged_simt_kernel(const DecodeArgs<T> a, int* status) {
    griddep_sync();
    __shared__ float qs[SR][DH];
    __shared__ float ps[SR][SC];
    __shared__ long long rows[SC];
    __shared__ float mrun[SR], lrun[SR], fac[SR];
    __shared__ float half[SR][64];
    const int R = a.H / a.G, groups = (R + SR - 1) / SR;
    const int split = blockIdx.x, g = blockIdx.y / groups, grp = blockIdx.y % groups, b = blockIdx.z;
    const int h0 = g * R + grp * SR, nh = min(SR, R - grp * SR);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    View w;
    const bool fine = view_of(a, b, &w);
    if (!fine && split == 0 && tid == 0) set_status(status, HYMBA_ERR_DEVICE_RANGE);
    const int k0 = split * a.split_keys, k1 = min(w.n, k0 + a.split_keys);
    if (k0 >= k1 && split > 0) return;
    for (int j = tid; j < SR * DH; j += 128) {
        const int h = j / DH, e = j % DH;
        qs[h][e] = h < nh ? to_f(a.q[b * a.ldq + (long long)(h0 + h) * DH + e]) * a.scale_log2 : 0.f;
    }
    if (tid < SR) {
        mrun[tid] = -INFINITY;
        lrun[tid] = 0.f;
    }
    const int col = tid % DV, sub = tid / DV;  // DV = 64: two threads per column, alternate keys
    constexpr int NS = 128 / DV;
    float acc[SR];
#pragma unroll
    for (int h = 0; h < SR; ++h) acc[h] = 0.f;
    int bad = 0;
    for (int c0 = k0; c0 < k1; c0 += SC) {
        __syncthreads();
        const int n = min(SC, k1 - c0);
        long long row = -1;
        if (tid < n) {
            row = slot_of(a, b, w.pos(c0 + tid));
            if (row < 0) bad = 1;
            else row += (long long)g * a.page;
        }
        rows[tid] = row;
        float s[SR];
#pragma unroll
        for (int h = 0; h < SR; ++h) s[h] = 0.f;
        if (row >= 0) {
            const T* kp = a.k_pages + row * DH;
#pragma unroll 4
            for (int e = 0; e < DH; e += 8) {
                float x[8];
                ragged::load8(kp + e, x);
#pragma unroll
                for (int h = 0; h < SR; ++h)
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[h] = fmaf(qs[h][e + i], x[i], s[h]);
            }
        }
#pragma unroll
        for (int h = 0; h < SR; ++h) ps[h][tid] = row >= 0 ? s[h] : -INFINITY;
        __syncthreads();
        for (int h = warp; h < nh; h += 4) {
            float mx = -INFINITY;
            for (int j = lane; j < SC; j += 32) mx = fmaxf(mx, ps[h][j]);
#pragma unroll
            for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float m = fmaxf(mrun[h], mx), mu = m == -INFINITY ? 0.f : m;
            float sum = 0.f;
            for (int j = lane; j < SC; j += 32) {
                const float p = exp2f(ps[h][j] - mu);
                ps[h][j] = p;
                sum += p;
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            __syncwarp();
            if (lane == 0) {
                const float f = exp2f(mrun[h] - mu);
                fac[h] = f;
                lrun[h] = lrun[h] * f + sum;
                mrun[h] = m;
            }
        }
        __syncthreads();
#pragma unroll
        for (int h = 0; h < SR; ++h)
            if (h < nh) acc[h] *= fac[h];
        for (int j = sub; j < n; j += NS) {
            const long long rj = rows[j];
            if (rj < 0) continue;
            const float x = to_f(a.v_pages[rj * DV + col]);
#pragma unroll
            for (int h = 0; h < SR; ++h) acc[h] = fmaf(ps[h][j], x, acc[h]);
        }
    }
    bad = __syncthreads_or(bad);
    if (bad && tid == 0) set_status(status, HYMBA_ERR_DEVICE_RANGE);
    if (NS == 2) {
        if (sub == 1)
            for (int h = 0; h < nh; ++h) half[h][col & 63] = acc[h];
        __syncthreads();
        if (sub == 1) return;
#pragma unroll
        for (int h = 0; h < SR; ++h) acc[h] += half[h][col & 63];
    }
    for (int h = 0; h < nh; ++h) {
        const float l = lrun[h];
        if (a.n_split == 1) {
            a.o[b * a.ldo + (long long)(h0 + h) * DV + col] = from_f<T>(bad || l == 0.f ? 0.f : acc[h] / l);
        } else {
            float* p = a.part + (((long long)b * a.H + h0 + h) * a.n_split + split) * (DV + 4);
            p[col] = acc[h];
            if (col == 0) {
                p[DV] = mrun[h];
                p[DV + 1] = bad ? -1.f : l;
            }
        }
    }
}

// Join the key splits of one (query head, sequence): weights 2^(m_s - max m).
template <typename T, int DV>
__global__ void __launch_bounds__(DV) decode_paged_join_kernel(const DecodeArgs<T> a) {
    griddep_sync();
    const int h = blockIdx.x, b = blockIdx.y, col = threadIdx.x;
    View w;
    view_of(a, b, &w);
    const int n = min(a.n_split, max(1, (w.n + a.split_keys - 1) / a.split_keys));
    const float* p = a.part + ((long long)b * a.H + h) * a.n_split * (DV + 4);
    float m = -INFINITY;
    for (int s = 0; s < n; ++s) m = fmaxf(m, p[s * (DV + 4) + DV]);
    const float mu = m == -INFINITY ? 0.f : m;
    float sum = 0.f, l = 0.f;
    bool bad = false;
    for (int s = 0; s < n; ++s) {
        const float ls = p[s * (DV + 4) + DV + 1], f = exp2f(p[s * (DV + 4) + DV] - mu);
        bad |= ls < 0.f;
        l = fmaf(ls, f, l);
        sum = fmaf(p[s * (DV + 4) + col], f, sum);
    }
    a.o[b * a.ldo + (long long)h * DV + col] = from_f<T>(bad || l == 0.f ? 0.f : sum / l);
}

// How the keys are split: a function of the call's host arguments alone, so that the
// workspace has one size. Splits of whole 128-key chunks, enough blocks to fill the GPU's
// 148 SMs several times over.
struct Split {
    int keys, n;
};
Split split_of(const hymba_attn_shape& s, int batch, int max_len) {
    const long long span = s.window > 0 ? std::min<long long>(max_len, (long long)s.n_meta + s.window) : max_len;
    const int R = s.n_q_heads / s.n_kv_heads;
    const long long units = (long long)batch * s.n_kv_heads * ((R + SR - 1) / SR);
    const long long chunks = (span + SC - 1) / SC;
    const long long want = std::max<long long>(1, std::min(chunks, (148 * 8 + units - 1) / units));
    Split r;
    r.keys = (int)((chunks + want - 1) / want) * SC;
    r.n = (int)((span + r.keys - 1) / r.keys);
    return r;
}

template <typename T, int DH, int DV>
int launch_decode_dims(const Ctx& ctx, DecodeArgs<T> a, int batch) {
    const int R = a.H / a.G;
    dim3 grid(a.n_split, a.G * ((R + SR - 1) / SR), batch);
    HYMBA_LAUNCH(ctx, "attn_decode_paged", (decode_paged_simt_kernel<T, DH, DV>), grid, 128, 0, a, ctx.status);
    if (a.n_split > 1)
        HYMBA_LAUNCH(ctx, "attn_decode_paged_join", (decode_paged_join_kernel<T, DV>), dim3(a.H, batch), DV, 0, a);
    return HYMBA_OK;
}

template <typename T>
int launch_decode_type(const Ctx& ctx, const hymba_attn_shape& s, float scale, const void* q, long long ldq,
                       const hymba_paged_kv& kv, int max_len, void* o, long long ldo, void* ws) {
    const Split sp = split_of(s, kv.batch, max_len);
    DecodeArgs<T> a;
    a.q = static_cast<const T*>(q);
    a.k_pages = static_cast<const T*>(kv.k_pages);
    a.v_pages = static_cast<const T*>(kv.v_pages);
    a.o = static_cast<T*>(o);
    a.table = kv.page_table;
    a.len = kv.len;
    a.ldq = ldq;
    a.ldo = ldo;
    a.part = static_cast<float*>(ws);
    a.n_pages = kv.n_pages;
    a.page = kv.page_size;
    a.max_pages = kv.max_pages;
    a.max_len = max_len;
    a.H = s.n_q_heads;
    a.G = s.n_kv_heads;
    a.n_meta = s.n_meta;
    a.window = s.window;
    a.split_keys = sp.keys;
    a.n_split = sp.n;
    a.scale_log2 = scale * LOG2E;
    if (s.head_dim == 64 && s.v_head_dim == 64) return launch_decode_dims<T, 64, 64>(ctx, a, kv.batch);
    if (s.head_dim == 64 && s.v_head_dim == 128) return launch_decode_dims<T, 64, 128>(ctx, a, kv.batch);
    if (s.head_dim == 128 && s.v_head_dim == 64) return launch_decode_dims<T, 128, 64>(ctx, a, kv.batch);
    if (s.head_dim == 128 && s.v_head_dim == 128) return launch_decode_dims<T, 128, 128>(ctx, a, kv.batch);
    return HYMBA_ERR_UNSUPPORTED;
}

}  // namespace

int launch_kv_append(const Ctx& ctx, const hymba_paged_kv& kv, int esz, const void* k, long long ldk, const void* v,
                     long long ldv, const int* cu, int rows) {
    AppendArgs a;
    a.k_pages = static_cast<uint8_t*>(kv.k_pages);
    a.v_pages = static_cast<uint8_t*>(kv.v_pages);
    a.k = static_cast<const uint8_t*>(k);
    a.v = static_cast<const uint8_t*>(v);
    a.table = kv.page_table;
    a.len = kv.len;
    a.cu = cu;
    a.ldk = ldk * esz;
    a.ldv = ldv * esz;
    a.n_pages = kv.n_pages;
    a.page = kv.page_size;
    a.max_pages = kv.max_pages;
    a.batch = kv.batch;
    a.rows = rows;
    a.G = kv.n_kv_heads;
    a.kshift = a.vshift = 0;
    while ((16 << a.kshift) < kv.head_dim * esz) ++a.kshift;
    while ((16 << a.vshift) < kv.v_head_dim * esz) ++a.vshift;
    HYMBA_LAUNCH(ctx, "kv_append_paged", kv_append_kernel, ceil_div(rows, 8), 256, 0, a, ctx.status);
    return HYMBA_OK;
}

size_t decode_paged_bytes(const hymba_attn_shape& s, int batch, int max_len) {
    const Split sp = split_of(s, batch, max_len);
    if (sp.n == 1) return 256;
    return (size_t)round_up((long long)batch * s.n_q_heads * sp.n * (s.v_head_dim + 4) * 4, 256);
}

int launch_decode_paged(const Ctx& ctx, const hymba_attn_shape& s, float scale, const void* q, long long ldq,
                        const hymba_paged_kv& kv, int max_len, void* o, long long ldo, void* ws) {
    if (s.dtype == HYMBA_F32) return launch_decode_type<float>(ctx, s, scale, q, ldq, kv, max_len, o, ldo, ws);
    if (s.dtype == HYMBA_F16) return launch_decode_type<f16>(ctx, s, scale, q, ldq, kv, max_len, o, ldo, ws);
    return launch_decode_type<bf16>(ctx, s, scale, q, ldq, kv, max_len, o, ldo, ws);
}

}  // namespace hymba
