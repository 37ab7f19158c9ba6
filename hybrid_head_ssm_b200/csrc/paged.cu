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

// One row per warp: its first 128 16-byte pieces (four per lane) are on their way while the warp
// finds the row's sequence (32 offsets at a time) and its slot (length, then page table); then the
// pieces go to the heads' slots. Bound by HBM for prompts (every byte is read once and written
// once), by the chain of lookups for single tokens. 19800 rows of 5 heads of 64 and 128 (f16): 14.7 us,
// 79% of the copy rate (17.1 with four rows per warp, 17.8 with eight); 64 tokens 2.7 us.
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
    const uint8_t *krow = a.k + r * a.ldk, *vrow = a.v + r * a.ldv;
    const int nk = a.G << a.kshift, n = nk + (a.G << a.vshift);  // pieces of a row: K's, then V's
    constexpr int U = 4;
    uint4 w[U];
    auto load = [&](int c0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + 32 * u + lane;
            if (c < n) w[u] = __ldg(reinterpret_cast<const uint4*>(c < nk ? krow + c * 16 : vrow + (c - nk) * 16));
        }
    };
    load(0);
    int b = (int)r, back = 1;  // the row is position len - back of sequence b
    if (a.cu) {
        int lo = 0, hi = a.batch;  // the last sequence that starts at or before r
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32, at = lo + lane * step;
            const unsigned m = __ballot_sync(0xffffffffu, at < hi && a.cu[at] <= r) | 1u;
            lo += (31 - __clz(m)) * step;
            hi = min(hi, lo + step);
        }
        b = lo;
        int st, len;
        if (!ragged::sequence(a.cu, b, a.rows, &st, &len) || r < st || r >= st + len) return;
        back = (int)(st + len - r);
    }
    const int len = a.len[b];
    const long long pos = (long long)len - back;
    int at = -1;
    if (pos >= 0 && len <= (long long)a.max_pages * a.page) at = a.table[(long long)b * a.max_pages + (int)pos / a.page];
    if (at < 0 || at >= a.n_pages) {
        if (lane == 0) set_status(status, HYMBA_ERR_DEVICE_RANGE);
        return;
    }
    const long long slot = (long long)at * a.G * a.page + (int)pos % a.page;  // of KV head 0; head g is g * page further
#pragma unroll 1
    for (int c0 = 0; c0 < n; c0 += 32 * U) {
        if (c0 > 0) load(c0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + 32 * u + lane;
            if (c >= n) continue;
            const bool is_k = c < nk;
            const int e = is_k ? c : c - nk, sh = is_k ? a.kshift : a.vshift;
            const int g = e >> sh, f = e & ((1 << sh) - 1);
            *reinterpret_cast<uint4*>((is_k ? a.k_pages : a.v_pages) + (((slot + (long long)g * a.page) << sh) + f) * 16) = w[u];
        }
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
// heads' softmax per warp, then a thread owns a column of V. Bound by latency: nothing is in flight
// across a chunk's barriers. 64 sequences in a window of 1024 236 us, 16 of up to 32896 1287 us (their
// bytes take 40 and 191).
constexpr int SC = 128, SR = 8;
constexpr int MAX_CL = 8;        // splits that join as one cluster
constexpr int MAX_SPLITS = 64;   // splits of one sequence

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

// Tensor cores (16-bit rows): one block of 4 warps per (key split, KV head and group of up
// to 8 NG of its query heads, sequence). Each warp walks every fourth 16-key tile of the split
// with its own ring of cp.async stages and its own running max, so no warp waits for
// another until the split ends; 96 KB of ring per block keeps two blocks per SM and about
// 150 KB per SM in flight. Per tile: S^T = K q^T (keys x heads, K by ldmatrix, q as the B
// operand in registers), p = 2^(s - m) with O rescaled only when a max grows by more than
// 2^4 (fp16) or 2^8 (bf16), and O^T += V^T P^T (V^T by transposing ldmatrix, P^T by an 8 x 8
// register transpose). p enters the product as two 16-bit parts (p = hi + lo), so the weights keep
// 16 bits or more; in fp16 m is the running max less 11, so that they do so down to 2^-20 of the
// largest (below, half of fp16's smallest step: 2^-36 of it). Slots are looked up one tile
// ahead of their copies: lane i holds key i's row. Rows past the split's last key are
// zero-filled by the copy and masked. Bound by HBM: K and V of every visible key once.
constexpr int TK = 16;                 // keys per tile
// m is the running max (log2 units) less LOW; it moves when a score passes it by more than TOP
template <typename T>
struct Weights {
    static constexpr float LOW = std::is_same<T, f16>::value ? 11.f : 0.f;
    static constexpr float TOP = std::is_same<T, f16>::value ? 15.f : 8.f;
};
// Three blocks per SM with 72 KB (64 KB) of rings each where a tile has at most 192 (128)
// dims, two with 96 KB at 256. 64 sequences of the 1.5B heads, window 1024: 33.0 us against 36.0
// with two blocks of four stages; 16 long contexts 100.9 against 115.4.
template <int DH, int DV>
struct Ring {
    static constexpr int KB = TK * DH * 2, VB = TK * DV * 2, BYTES = KB + VB;
    static constexpr int N = DH + DV == 128 ? 4 : 3, SIZE = N * BYTES;  // stages and bytes of one warp's ring
};
constexpr int blocks_per_sm(int dims, int ng) { return dims <= 192 && ng == 1 ? 3 : 2; }

// One warp's sums of p v once more, key by key with fp32 weights, for values of V that are not finite:
// the lower part of a weight may be 0, and 0 x infinity is NaN. m, l: [4][HB] of the block's warps;
// acc: [HB][LD], brought to the block's max like the sums it replaces.
template <typename T, int DH, int DV, int HB, int LD>
__device__ __noinline__ void sums_again(const DecodeArgs<T>& a, const View w, int b, int g, int h0, int nh, int k0, int k1,
                                        const float (*m)[HB], const float (*l)[HB], float* acc) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int h = 0; h < nh; ++h) {
        const float mine = m[warp][h], mu = mine == -INFINITY ? 0.f : mine;
        const float to = fmaxf(fmaxf(m[0][h], m[1][h]), fmaxf(m[2][h], m[3][h]));
        const T* q = a.q + b * a.ldq + (long long)(h0 + h) * DH;
        float sum[DV / 32] = {};
        for (int j0 = k0 + warp * TK; j0 < k1; j0 += 4 * TK)
            for (int j = j0; j < min(j0 + TK, k1); ++j) {
                const long long slot = slot_of(a, b, w.pos(j));
                if (slot < 0) continue;
                const long long row = slot + (long long)g * a.page;
                float s = 0.f;
#pragma unroll
                for (int e = lane; e < DH; e += 32) s = fmaf(to_f(q[e]), to_f(a.k_pages[row * DH + e]), s);
#pragma unroll
                for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                const float p = fast_exp2(fmaf(s, a.scale_log2, -mu));
#pragma unroll
                for (int x = 0; x < DV / 32; ++x) sum[x] = fmaf(p, to_f(a.v_pages[row * DV + lane + 32 * x]), sum[x]);
            }
        float f = mine == -INFINITY ? 0.f : fast_exp2(mine - to);
        if (!(l[warp][h] == l[warp][h])) f = l[warp][h];
#pragma unroll
        for (int x = 0; x < DV / 32; ++x) acc[h * LD + lane + 32 * x] = sum[x] * f;
    }
}

// CL: the splits of one (KV head, sequence) form a thread-block cluster and join over distributed
// shared memory; otherwise they leave partial results for the join kernel.
template <typename T, int DH, int DV, int NG, bool CL>
__global__ void __launch_bounds__(128, blocks_per_sm(DH + DV, NG)) decode_paged_mma_kernel(const __grid_constant__ DecodeArgs<T> a, int* status) {
    using R_ = Ring<DH, DV>;
    griddep_sync();
    extern __shared__ __align__(128) uint8_t decode_raw[];
    __shared__ float ms[4][8 * NG], ls[4][8 * NG];
    const int R = a.H / a.G, groups = (R + 8 * NG - 1) / (8 * NG);
    const int split = blockIdx.x, g = blockIdx.y / groups, grp = blockIdx.y % groups, b = blockIdx.z;
    const int h0 = g * R + grp * 8 * NG, nh = min(8 * NG, R - grp * 8 * NG);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int lg = lane >> 2, lq = lane & 3;
    View w;
    const bool fine = view_of(a, b, &w);
    if (!fine && split == 0 && blockIdx.y == 0 && tid == 0) set_status(status, HYMBA_ERR_DEVICE_RANGE);
    const int k0 = split * a.split_keys, k1 = min(w.n, k0 + a.split_keys);
    if (!CL && k0 >= k1 && split > 0) return;
    const int ntile = k1 > k0 ? (k1 - k0 + TK - 1) / TK : 0;
    uint8_t* ring = decode_raw + warp * R_::SIZE;

    // q as the "col" operand: heads x dims
    uint32_t qf[NG][DH / 16][2];
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk) {
            const int h = n * 8 + lg;
            const uint32_t* qp = reinterpret_cast<const uint32_t*>(a.q + b * a.ldq + (long long)(h0 + min(h, nh - 1)) * DH +
                                                                   kk * 16 + 2 * lq);
            qf[n][kk][0] = h < nh ? qp[0] : 0u;
            qf[n][kk][1] = h < nh ? qp[4] : 0u;
        }
    float ot[NG][DV / 16][4];
    float m[NG][2], l[NG][2];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int t = 0; t < DV / 16; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) ot[n][t][e] = 0.f;
    }

    // the row (head g) of key `lane % 16` of the warp's i-th tile; none past the end
    constexpr uint32_t NONE = 0xffffffffu;
    int bad = 0;
    auto row_of = [&](int i) -> uint32_t {
        const int j = k0 + (warp + 4 * i) * TK + (lane & 15);
        if (j >= k1) return NONE;
        const long long s = slot_of(a, b, w.pos(j));
        if (s < 0) {
            bad = 1;
            return NONE;
        }
        return (uint32_t)(s + (long long)g * a.page);
    };
    const int mine = ntile > warp ? (ntile - warp + 3) / 4 : 0;  // the warp's tiles
    auto issue = [&](int i, uint32_t row) {
        uint8_t* st = ring + (i % R_::N) * R_::BYTES;
        constexpr int KC = DH / 8, VC = DV / 8;  // 16-byte pieces per row
#pragma unroll
        for (int x = 0; x < TK * KC / 32; ++x) {
            const int r = x * (32 / KC) + lane / KC, c = lane % KC;
            const uint32_t rr = __shfl_sync(0xffffffffu, row, r);
            wm::cpa16(st + r * DH * 2 + ((c ^ (r & 7)) * 16), a.k_pages + (rr == NONE ? 0 : (long long)rr * DH) + c * 8,
                      rr == NONE);
        }
#pragma unroll
        for (int x = 0; x < TK * VC / 32; ++x) {
            const int r = x * (32 / VC) + lane / VC, c = lane % VC;
            const uint32_t rr = __shfl_sync(0xffffffffu, row, r);
            wm::cpa16(st + R_::KB + r * DV * 2 + ((c ^ (r & 7)) * 16),
                      a.v_pages + (rr == NONE ? 0 : (long long)rr * DV) + c * 8, rr == NONE);
        }
    };
    {
        uint32_t row[R_::N - 1];
#pragma unroll
        for (int i = 0; i < R_::N - 1; ++i) row[i] = i < mine ? row_of(i) : NONE;
#pragma unroll
        for (int i = 0; i < R_::N - 1; ++i) {
            if (i < mine) issue(i, row[i]);
            wm::cpa_commit();
        }
    }
    uint32_t next = R_::N - 1 < mine ? row_of(R_::N - 1) : NONE;
    for (int i = 0; i < mine; ++i) {
        wm::cpa_wait<R_::N - 2>();
        __syncwarp();  // every lane's copies of the tile are there, and its reads of the stage that is filled next are done
        if (i + R_::N - 1 < mine) issue(i + R_::N - 1, next);
        wm::cpa_commit();
        if (i + R_::N < mine) next = row_of(i + R_::N);
        const uint8_t* st = ring + (i % R_::N) * R_::BYTES;
        float sc[NG][4];
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[n][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk) {
            uint32_t kf[4];
            const int r = lane & 15, c = 2 * kk + (lane >> 4);
            wm::ldsm_x4(kf, st + r * DH * 2 + ((c ^ (r & 7)) * 16));
#pragma unroll
            for (int n = 0; n < NG; ++n) wm::mma16<T>(sc[n], kf, qf[n][kk][0], qf[n][kk][1]);
        }
        // keys lg and lg + 8 of the tile, heads 2 lq and 2 lq + 1
        const int left = k1 - (k0 + (warp + 4 * i) * TK);
        uint32_t ph[NG][2], pl[NG][2];
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            if (left < TK) {
                if (lg >= left) sc[n][0] = sc[n][1] = -INFINITY;
                if (lg + 8 >= left) sc[n][2] = sc[n][3] = -INFINITY;
            }
            float mx[2] = {fmaxf(sc[n][0], sc[n][2]), fmaxf(sc[n][1], sc[n][3])};
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], o));
                mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], o));
            }
            mx[0] *= a.scale_log2;
            mx[1] *= a.scale_log2;
            if (__any_sync(0xffffffffu, mx[0] > m[n][0] + Weights<T>::TOP || mx[1] > m[n][1] + Weights<T>::TOP)) {
                float f[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float to = fmaxf(m[n][e], mx[e] - Weights<T>::LOW);
                    f[e] = to == -INFINITY ? 1.f : fast_exp2(m[n][e] - to);
                    m[n][e] = to;
                    l[n][e] *= f[e];
                }
#pragma unroll
                for (int t = 0; t < DV / 16; ++t) {
                    ot[n][t][0] *= f[0];
                    ot[n][t][1] *= f[1];
                    ot[n][t][2] *= f[0];
                    ot[n][t][3] *= f[1];
                }
            }
            const float u0 = m[n][0] == -INFINITY ? 0.f : m[n][0], u1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
            const float p0 = fast_exp2(fmaf(sc[n][0], a.scale_log2, -u0)), p1 = fast_exp2(fmaf(sc[n][1], a.scale_log2, -u1));
            const float p2 = fast_exp2(fmaf(sc[n][2], a.scale_log2, -u0)), p3 = fast_exp2(fmaf(sc[n][3], a.scale_log2, -u1));
            l[n][0] += p0 + p2;
            l[n][1] += p1 + p3;
            uint32_t h01, l01, h23, l23;
            wm::split2<T>(p0, p1, &h01, &l01);
            wm::split2<T>(p2, p3, &h23, &l23);
            ph[n][0] = wm::transpose8(h01);
            ph[n][1] = wm::transpose8(h23);
            pl[n][0] = wm::transpose8(l01);
            pl[n][1] = wm::transpose8(l23);
        }
#pragma unroll
        for (int t = 0; t < DV / 16; ++t) {
            uint32_t vf[4];
            const int r = (lane & 7) + 8 * (lane >> 4), c = 2 * t + ((lane >> 3) & 1);
            wm::ldsm_x4_t(vf, st + R_::KB + r * DV * 2 + ((c ^ (r & 7)) * 16));
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                wm::mma16<T>(ot[n][t], vf, ph[n][0], ph[n][1]);
                wm::mma16<T>(ot[n][t], vf, pl[n][0], pl[n][1]);
            }
        }
    }
    wm::cpa_wait<0>();
    // join the warps: one max per head, each warp's sums brought to it
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], o);
            if (lg == 0) {
                ms[warp][n * 8 + 2 * lq + e] = m[n][e];
                ls[warp][n * 8 + 2 * lq + e] = l[n][e];
            }
        }
    bad = __syncthreads_or(bad);
    if (bad && tid == 0) set_status(status, HYMBA_ERR_DEVICE_RANGE);
    constexpr int LD = DV + 4;
    float* acc = reinterpret_cast<float*>(decode_raw);  // [4][8 NG][LD]
    static_assert(4 * 8 * NG * LD * 4 <= 4 * R_::SIZE, "the joined sums reuse the rings");
    float odd = 0.f;  // NaN once a sum of a head whose weights are finite is not
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float z = 0.f;
#pragma unroll
            for (int t = 0; t < DV / 16; ++t) z = fmaf(ot[n][t][e], 0.f, z);
            if (l[n][e & 1] - l[n][e & 1] == 0.f) odd += z;
        }
    const bool again = __any_sync(0xffffffffu, !(odd == 0.f));
    if (again)
        sums_again<T, DH, DV, 8 * NG, LD>(a, w, b, g, h0, nh, k0, k1, ms, ls, acc + warp * 8 * NG * LD);
#pragma unroll
    for (int n = 0; n < NG; ++n) {
        if (again) break;
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int h = n * 8 + 2 * lq + e;
            const float to = fmaxf(fmaxf(ms[0][h], ms[1][h]), fmaxf(ms[2][h], ms[3][h]));
            f[e] = m[n][e] == -INFINITY ? 0.f : fast_exp2(m[n][e] - to);
            // (a NaN or infinite max keeps a NaN sum)
            if (!(l[n][e] == l[n][e])) f[e] = l[n][e];
        }
#pragma unroll
        for (int t = 0; t < DV / 16; ++t) {
            float* p = acc + (warp * 8 * NG + n * 8 + 2 * lq) * LD + 16 * t + lg;
            p[0] = ot[n][t][0] * f[0];
            p[LD] = ot[n][t][1] * f[1];
            p[8] = ot[n][t][2] * f[0];
            p[LD + 8] = ot[n][t][3] * f[1];
        }
    }
    __syncthreads();
    auto joined = [&](int h, float* to, float* lt) {
        *to = fmaxf(fmaxf(ms[0][h], ms[1][h]), fmaxf(ms[2][h], ms[3][h]));
        *lt = 0.f;
#pragma unroll
        for (int v = 0; v < 4; ++v) *lt += ms[v][h] == -INFINITY ? ls[v][h] : ls[v][h] * fast_exp2(ms[v][h] - *to);
    };
    if constexpr (CL) {
        // the block's sums, max and sum of p per head, read by every block of the cluster, each
        // of which writes its share of the outputs
        for (int x = tid; x < nh * DV; x += 128) {
            float* p = acc + x / DV * LD + x % DV;
            *p = p[0] + p[8 * NG * LD] + p[16 * NG * LD] + p[24 * NG * LD];
        }
        if (tid < nh) {
            float to, lt;
            joined(tid, &to, &lt);
            acc[tid * LD + DV] = to;
            acc[tid * LD + DV + 1] = bad ? -1.f : lt;
        }
        cluster_arrive();
        cluster_wait();
        for (int x = split * 128 + tid; x < nh * DV; x += 128 * a.n_split) {
            const int h = x / DV, col = x % DV;
            float mm[MAX_CL], to = -INFINITY, lt = 0.f, sum = 0.f;
            bool any_bad = false;
#pragma unroll
            for (int r = 0; r < MAX_CL; ++r) {
                mm[r] = r < a.n_split ? ld_cluster_f32(acc + h * LD + DV, r) : -INFINITY;
                to = fmaxf(to, mm[r]);
            }
            const float mu = to == -INFINITY ? 0.f : to;
#pragma unroll
            for (int r = 0; r < MAX_CL; ++r)
                if (r < a.n_split) {
                    const float lr = ld_cluster_f32(acc + h * LD + DV + 1, r), f = fast_exp2(mm[r] - mu);
                    any_bad |= lr < 0.f;
                    lt = fmaf(lr, f, lt);
                    sum = fmaf(ld_cluster_f32(acc + h * LD + col, r), f, sum);
                }
            a.o[b * a.ldo + (long long)(h0 + h) * DV + col] = from_f<T>(any_bad || lt == 0.f ? 0.f : sum / lt);
        }
        cluster_arrive();
        cluster_wait();  // no block leaves while another reads its shared memory
    } else {
        for (int x = tid; x < nh * DV; x += 128) {
            const int h = x / DV, col = x % DV;
            float sum = 0.f, to, lt;
#pragma unroll
            for (int v = 0; v < 4; ++v) sum += acc[(v * 8 * NG + h) * LD + col];
            joined(h, &to, &lt);
            if (a.n_split == 1) {
                a.o[b * a.ldo + (long long)(h0 + h) * DV + col] = from_f<T>(bad || lt == 0.f ? 0.f : sum / lt);
            } else {
                float* p = a.part + (((long long)b * a.H + h0 + h) * a.n_split + split) * (DV + 4);
                p[col] = sum;
                if (col == 0) {
                    p[DV] = to;
                    p[DV + 1] = bad ? -1.f : lt;
                }
            }
        }
    }
}

// Join the key splits of one (query head, sequence): weights 2^(m_s - max m), then the
// splits' sums, 256 / DV of them at a time per column.
template <typename T, int DV>
__global__ void __launch_bounds__(256) decode_paged_join_kernel(const DecodeArgs<T> a) {
    griddep_sync();
    __shared__ float f[MAX_SPLITS], red[256], top[8], tot[8];
    __shared__ int any_bad;
    const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    View w;
    view_of(a, b, &w);
    const int n = min(a.n_split, max(1, (w.n + a.split_keys - 1) / a.split_keys));
    const float* p = a.part + ((long long)b * a.H + h) * a.n_split * (DV + 4);
    static_assert(MAX_SPLITS <= 256, "one split per thread");
    const float m = tid < n ? p[tid * (DV + 4) + DV] : -INFINITY, ls = tid < n ? p[tid * (DV + 4) + DV + 1] : 0.f;
    if (tid == 0) any_bad = 0;
    float to = m;
#pragma unroll
    for (int o = 16; o; o >>= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, o));
    if (lane == 0) top[warp] = to;
    __syncthreads();
#pragma unroll
    for (int x = 0; x < 8; ++x) to = fmaxf(to, top[x]);
    const float e = tid < n ? fast_exp2(m - (to == -INFINITY ? 0.f : to)) : 0.f;
    if (ls < 0.f) any_bad = 1;
    if (tid < n) f[tid] = e;
    float l = ls * e;
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) tot[warp] = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int x = 0; x < 8; ++x) l += tot[x];
    constexpr int NP = 256 / DV;
    const int col = tid % DV, part = tid / DV;
    float sum = 0.f;
#pragma unroll 4
    for (int s = part; s < n; s += NP) sum = fmaf(p[s * (DV + 4) + col], f[s], sum);
    red[tid] = sum;
    __syncthreads();
    if (tid < DV) {
#pragma unroll
        for (int x = 1; x < NP; ++x) sum += red[x * DV + tid];
        a.o[b * a.ldo + (long long)h * DV + tid] = from_f<T>(any_bad || l == 0.f ? 0.f : sum / l);
    }
}

// How the keys are split: a function of the call's host arguments alone, so that the
// workspace has one size. `units` (KV heads and groups of all sequences) are the blocks
// without splitting, `slots` what the GPU's 148 SMs hold at a time.
//   - Where all sequences see about equally many keys (a window that is full, or a short
//     cache): up to 8 splits that still fit one wave; all blocks then share the bandwidth and
//     finish together, and the splits join within a cluster. 64 sequences, window 1024: 25.7
//     us in 1 split, 33.0 in 2 (a wave and a half); 16 of them: 10.8 in 4 with a cluster, 11.5
//     with the join kernel; one sequence of 1153: 5.8 in 7 against 6.3 in 10 with the join.
//   - Where the lengths may differ much (a global layer's long cache): about 8 blocks per SM,
//     which spread over the SMs as they come free, joined by the kernel after. 64 sequences of
//     up to 4224: 63.1 us in 4 splits, 71.8 in 1 (clusters of 4: 72.0, they wait for room); 16
//     of up to 32896: 101 in 15, 150 in 4. More than 64 splits of one sequence cost more in
//     the join than they give (one of 32000: 18.7 us in 60, 25.5 in 118).
struct Split {
    int keys, n;
    bool cluster;
};
int heads_per_block(const hymba_attn_shape& s) {
    return s.dtype == HYMBA_F32 || s.n_q_heads / s.n_kv_heads <= 8 ? 8 : 16;
}
Split split_of(const hymba_attn_shape& s, int batch, int max_len) {
    const long long full = (long long)s.n_meta + s.window;
    const bool windowed = s.window > 0 && full <= max_len;
    const long long span = windowed ? full : max_len;
    const int R = s.n_q_heads / s.n_kv_heads, hb = heads_per_block(s);
    const long long units = (long long)batch * s.n_kv_heads * ((R + hb - 1) / hb);
    const int step = s.dtype == HYMBA_F32 ? SC : 4 * TK;
    const long long chunks = (span + step - 1) / step;
    const long long slots = 148 * blocks_per_sm(s.head_dim + s.v_head_dim, hb / 8);
    const bool even = s.dtype != HYMBA_F32 && (span <= 1536 || (windowed && (span <= 4096 || units > slots / MAX_CL)));
    const long long most = even ? std::min<long long>(MAX_CL, slots / units) : std::min<long long>(MAX_SPLITS, (148 * 8 + units - 1) / units);
    const long long want = std::max<long long>(1, std::min(chunks, most));
    Split r;
    r.keys = (int)((chunks + want - 1) / want) * step;
    r.n = (int)((span + r.keys - 1) / r.keys);
    r.cluster = even && r.n > 1;
    return r;
}

template <typename T, int DH, int DV, int NG>
int launch_decode_mma(const Ctx& ctx, const DecodeArgs<T>& a, int batch, bool cluster) {
    const int R = a.H / a.G;
    const size_t smem = 4 * Ring<DH, DV>::SIZE;
    const dim3 grid(a.n_split, a.G * ((R + 8 * NG - 1) / (8 * NG)), batch);
    static std::atomic<unsigned long long> smem_set[2];
    if (cluster) {
        auto kern = decode_paged_mma_kernel<T, DH, DV, NG, true>;
        if (!smem_opt_in_once(smem_set[1], kern, smem, ctx)) return HYMBA_ERR_CUDA;
        HYMBA_LAUNCH_CLUSTER(ctx, "attn_decode_paged", kern, grid, 128, smem, (unsigned)a.n_split, a, ctx.status);
    } else {
        auto kern = decode_paged_mma_kernel<T, DH, DV, NG, false>;
        if (!smem_opt_in_once(smem_set[0], kern, smem, ctx)) return HYMBA_ERR_CUDA;
        HYMBA_LAUNCH(ctx, "attn_decode_paged", kern, grid, 128, smem, a, ctx.status);
    }
    return HYMBA_OK;
}

template <typename T, int DH, int DV>
int launch_decode_dims(const Ctx& ctx, const DecodeArgs<T>& a, int batch, bool cluster) {
    const int R = a.H / a.G;
    if constexpr (sizeof(T) == 2) {
        const int rc = R <= 8 ? launch_decode_mma<T, DH, DV, 1>(ctx, a, batch, cluster)
                              : launch_decode_mma<T, DH, DV, 2>(ctx, a, batch, cluster);
        if (rc) return rc;
    } else {
        dim3 grid(a.n_split, a.G * ((R + SR - 1) / SR), batch);
        HYMBA_LAUNCH(ctx, "attn_decode_paged", (decode_paged_simt_kernel<T, DH, DV>), grid, 128, 0, a, ctx.status);
    }
    if (a.n_split > 1 && !cluster)
        HYMBA_LAUNCH(ctx, "attn_decode_paged_join", (decode_paged_join_kernel<T, DV>), dim3(a.H, batch), 256, 0, a);
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
    if (s.head_dim == 64 && s.v_head_dim == 64) return launch_decode_dims<T, 64, 64>(ctx, a, kv.batch, sp.cluster);
    if (s.head_dim == 64 && s.v_head_dim == 128) return launch_decode_dims<T, 64, 128>(ctx, a, kv.batch, sp.cluster);
    if (s.head_dim == 128 && s.v_head_dim == 64) return launch_decode_dims<T, 128, 64>(ctx, a, kv.batch, sp.cluster);
    if (s.head_dim == 128 && s.v_head_dim == 128) return launch_decode_dims<T, 128, 128>(ctx, a, kv.batch, sp.cluster);
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
    if (sp.n == 1 || sp.cluster) return 256;
    return (size_t)round_up((long long)batch * s.n_q_heads * sp.n * (s.v_head_dim + 4) * 4, 256);
}

int launch_decode_paged(const Ctx& ctx, const hymba_attn_shape& s, float scale, const void* q, long long ldq,
                        const hymba_paged_kv& kv, int max_len, void* o, long long ldo, void* ws) {
    if (s.dtype == HYMBA_F32) return launch_decode_type<float>(ctx, s, scale, q, ldq, kv, max_len, o, ldo, ws);
    if (s.dtype == HYMBA_F16) return launch_decode_type<f16>(ctx, s, scale, q, ldq, kv, max_len, o, ldo, ws);
    return launch_decode_type<bf16>(ctx, s, scale, q, ldq, kv, max_len, o, ldo, ws);
}

}  // namespace hymba
