// Linear attention with a decay per head, chunked form on the warp MMAs (16-bit rows, key dim 16 or 128):
// S_t = exp(g_t) S_{t-1} + v_t k_t^T, o_t = scale S_t q_t over packed prompts ("Lecture 04 -
// Beyond the Dense Transformer", section 3: with a scalar decay per head the recurrence is a
// masked product with a semiseparable matrix and can be computed as blocks of matmuls). Per
// chunk of 64 rows, with cs_i = g_1 + .. + g_i counted from the chunk's start:
//     o_i = scale (sum_{j<=i} exp(cs_i - cs_j) (q_i . k_j) v_j  +  exp(cs_i) S q_i)
//     S  <- exp(cs_64) S + sum_j exp(cs_64 - cs_j) v_j k_j^T
//
// One CTA of 4 warps per (64 value columns, head, sequence) walks the chunks; cp.async
// stages the next chunk's q, k, v meanwhile. The state lives in registers as the
// accumulators of its own update: warp w owns value columns 16 w .. 16 w + 15, S^T rows, and
// the m16n8 accumulator layout of (value, key) is the B operand layout of (key, value), so the
// product with q takes S straight from the registers. Per chunk: warp w forms rows 16 w ..
// 16 w + 15 of P = mask * exp(cs_i - cs_j) * scale q k^T into shared memory while all warps
// form exp(cs_i) S q; then each adds P V for its columns and updates its S. The V fragments
// serve as the B operand of P V and as the A operand of the update.
//
// Numbers: cs is summed in 64 bits. A decay between rows j <= i is 2^(a_i + b_j) with a_i and b_j
// the fp32 distances of cs_i and cs_j from the cs at the start of i's 16 rows, and never formed from two
// factors. A row that forgets everything (a decay that is 0 in fp32) is no term of cs but a border that
// nothing before it passes and at which cs starts again, so the distances stay small after any number of them (only decays of 2^-100
// and less that are not 0, row after row, leave the others of their 16 rows right to 2^-12, half a step of
// P). P and the copy of S that meets q are rounded to the rows' type, like any MMA operand;
// the scaled v of the state update enters as three parts (bf16: 24 bits) or two (fp16: 22 bits, or
// 2^-37 of the column's largest scaled v in the chunk where that is more). fp16 has little range: P's
// rows and each value column of S's copy and of the scaled v are brought to the middle of it by powers of
// two, which are taken out again from the fp32 sums.
// A row's values reach only what sees them: rows behind the sequence are zero-filled; in a
// chunk where a decay may underflow to 0, what it multiplies is dropped; a chunk whose V holds a
// value that is not finite forms P V, and one whose K or V does its state, row by row.
// Bound: HBM (q, k, v once per 64 value columns, o) and the warp MMAs (1024 multiply-adds per
// clock and SM measured) are close; what is left is instruction issue, hence the tables that
// one warp (the one with the fewest tiles of P) forms a chunk ahead for all. Eight prompts of 2000
// rows, bf16: 50 heads of 16 x 64 with shared keys 110 us (their 212 MB take 32), 25 of 128 x 128
// with 5 key heads 302 us (fp16 119 and 345).
#include "kernels.h"
#include "ragged.cuh"

namespace hymba {

namespace {

using ragged::fade;
using ragged::inverse;
using ragged::to_middle;

constexpr int CQ = 64;   // rows per chunk
constexpr int CV = 64;   // value columns per CTA
constexpr int NT = 128;  // 4 warps

// Per chunk, from its 64 log decays (log2 units; cs_i the inclusive sums):
struct Tables {
    alignas(16) float a[CQ];      // cs_i - cs at the start of i's 16 rows + log2 scale
    alignas(16) float b[4][CQ];   // cs at the start of 16-row block t - cs_j, for j < 16 (t + 1)
    alignas(16) float e[CQ];      // 2^cs_i scale
    alignas(16) float w[CQ];      // 2^(cs_63 - cs_j)
    alignas(8) int border[CQ];    // the last row at or before each that forgets everything (below 0: none)
    float dec;                    // 2^cs_63
    int resets;                   // a decay within the chunk may be 0; 2: some rows forget everything (border holds)
    // the row that row i may see first
    __device__ __forceinline__ int first(int i) const { return resets == 2 ? max(border[i], 0) : 0; }
};

// a decay below 2^-150 is 0 in fp32
__device__ __forceinline__ bool forgets(float g) { return g < -104.f; }

template <int DK>
struct ChunkSmem {
    // rows of DK or 64 16-bit elements, 16-byte pieces swizzled by the row
    alignas(128) uint8_t q[2][CQ * DK * 2];
    alignas(128) uint8_t k[2][CQ * DK * 2];
    alignas(128) uint8_t v[2][CQ * CV * 2];
    alignas(128) uint8_t p[CQ * CQ * 2];
    Tables tab[2];
    alignas(16) float ps[CQ];  // the power of two that P's rows carry
};

// byte offset of 16-byte piece c of row r of a tile of COLS 16-bit columns; 8 rows at one c
// cover all banks
template <int COLS>
__device__ __forceinline__ uint32_t at(int r, int c) {
    if constexpr (COLS == 16) return r * 32 + ((c ^ ((r >> 2) & 1)) * 16);
    else return r * COLS * 2 + ((c ^ (r & 7)) * 16);
}

// A thread's share of staging 64 rows of COLS columns: one 16-byte column piece of every
// STEP-th row, so that its swizzle is one constant.
template <typename T, int COLS>
struct Stager {
    static constexpr int PC = COLS / 8, STEP = NT / PC < CQ ? NT / PC : CQ, N = CQ / STEP;
    const char* src;  // the thread's first row of the next chunk
    long long step;   // bytes between its rows
    uint32_t dst;
    int row;
    bool on;
    __device__ void init(const T* base, long long ld) {
        row = threadIdx.x / PC;
        on = row < CQ;
        const int c = threadIdx.x % PC;
        src = reinterpret_cast<const char*>(base + row * ld + c * 8);
        step = ld * STEP * (long long)sizeof(T);
        dst = at<COLS>(row, c);
    }
    // rows t0 .. t0 + 63; rows past the sequence's end read as zero
    __device__ __forceinline__ void load(uint8_t* tile, int t0, int len, const void* safe) {
        if (on) {
            const char* x = src;
            if (t0 + CQ <= len) {
#pragma unroll
                for (int i = 0; i < N; ++i, x += step) wm::cpa16(tile + dst + i * STEP * COLS * 2, x);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i, x += step) {
                    const bool in = t0 + row + i * STEP < len;
                    wm::cpa16(tile + dst + i * STEP * COLS * 2, in ? x : safe, !in);
                }
            }
        }
        src += step * N;
    }
};

template <typename T> struct Pair;
template <> struct Pair<f16> { typedef __half2 type; };
template <> struct Pair<bf16> { typedef __nv_bfloat162 type; };
template <typename T>
__device__ __forceinline__ typename Pair<T>::type pair(uint32_t x) {
    return *reinterpret_cast<const typename Pair<T>::type*>(&x);
}
template <typename P2>
__device__ __forceinline__ uint32_t bits(P2 x) { return *reinterpret_cast<const uint32_t*>(&x); }

__device__ __forceinline__ void scale_rows(float (&x)[2][4], float a, float b) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        x[n][0] *= a;
        x[n][1] *= a;
        x[n][2] *= b;
        x[n][3] *= b;
    }
}

// the two value rows of the warp's share of the state
template <int N>
__device__ __forceinline__ void scale_state(float (&st)[N][4], float a, float b) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
        st[n][0] *= a;
        st[n][1] *= a;
        st[n][2] *= b;
        st[n][3] *= b;
    }
}

// sum_{j <= i} P_ij v_j of one value column, over the rows that i sees through a decay above 0
template <typename T>
__device__ __noinline__ float row_product(const Tables& tab, const uint8_t* p, const uint8_t* v, int i, int col) {
    float sum = 0.f;
    for (int j = tab.first(i); j <= i; ++j) {
        if (fast_exp2(tab.a[i] + tab.b[i >> 4][j]) == 0.f) continue;
        const T pj = *reinterpret_cast<const T*>(p + at<CQ>(i, j >> 3) + 2 * (j & 7));
        const T vj = *reinterpret_cast<const T*>(v + at<CV>(j, col >> 3) + 2 * (col & 7));
        sum = fmaf(to_f(pj), to_f(vj), sum);
    }
    return sum;
}

// The state after a chunk, row by row in fp32 over the rows it still sees: S is the warp's share, val its
// first value column of the tile.
template <typename T, int DK>
__device__ __forceinline__ void row_states(const Tables& tab, const uint8_t* k, const uint8_t* v, int val,
                                           float (&S)[DK / 8][4]) {
    const int lq = threadIdx.x & 3;
#pragma unroll
    for (int n = 0; n < DK / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[n][e] = fade(tab.dec, S[n][e]);
#pragma unroll 1
    for (int j = 0; j < CQ; ++j) {
        const float w = tab.w[j];
        if (w == 0.f) continue;
        const float x = w * to_f(*reinterpret_cast<const T*>(v + at<CV>(j, val >> 3) + 2 * (val & 7)));
        const float y = w * to_f(*reinterpret_cast<const T*>(v + at<CV>(j, (val >> 3) + 1) + 2 * (val & 7)));
#pragma unroll
        for (int n = 0; n < DK / 8; ++n) {
            const uint32_t kk = *reinterpret_cast<const uint32_t*>(k + at<DK>(j, n) + 4 * lq);
            const T* e = reinterpret_cast<const T*>(&kk);
            S[n][0] = fmaf(x, to_f(e[0]), S[n][0]);
            S[n][1] = fmaf(x, to_f(e[1]), S[n][1]);
            S[n][2] = fmaf(y, to_f(e[0]), S[n][2]);
            S[n][3] = fmaf(y, to_f(e[1]), S[n][3]);
        }
    }
}

// the tables of one chunk from the two log decays each lane holds (rows 2 lane, 2 lane + 1). BORDERS: some
// of them forget everything; the sums start again there, so that what lies before, a NaN among it, enters
// nothing behind
template <bool BORDERS>
__device__ __forceinline__ void fill_tables(Tables& t, float g0, float g1, float log2_scale) {
    constexpr double LOG2E = 1.4426950408889634;
    const int lane = threadIdx.x & 31;
    const bool r0 = BORDERS && forgets(g0), r1 = BORDERS && forgets(g1);
    const double d0 = (double)(r0 ? 0.f : g0) * LOG2E, d1 = (double)(r1 ? 0.f : g1) * LOG2E;
    double sum = r1 ? 0.0 : d0 + d1;
    // the last border at or before the lane's two rows and in the chunk; the first lane of its run of rows
    int f0 = -1, f1 = -1, border = -1, head = 0;
    if (BORDERS) {
        const unsigned m0 = __ballot_sync(0xffffffffu, r0), m1 = __ballot_sync(0xffffffffu, r1), below = (1u << lane) - 1;
        auto row = [](unsigned even, unsigned odd) { return max(62 - 2 * __clz(even), 63 - 2 * __clz(odd)); };
        f0 = row(m0 & (below | 1u << lane), m1 & below);
        f1 = r1 ? 2 * lane + 1 : f0;
        border = row(m0, m1);
        head = max(31 - __clz((m0 | m1) & (below | 1u << lane)), 0);
        *reinterpret_cast<int2*>(&t.border[2 * lane]) = make_int2(f0, f1);
    }
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, sum, w);
        if (lane - w >= head) sum += y;
    }
    // forward from the rows before, so that a NaN or an infinity reaches no earlier row
    const double last = __shfl_sync(0xffffffffu, sum, 31), before = __shfl_up_sync(0xffffffffu, sum, 1);
    const double x0 = r0 ? 0.0 : lane ? before + d0 : d0, x1 = r1 ? 0.0 : x0 + d1;
    double from = 0.0;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        double c = b == 0 ? 0.0 : __shfl_sync(0xffffffffu, sum, b == 0 ? 0 : 8 * b - 1);
        if (BORDERS && !(c - c == 0.0)) c = 0.0;  // (only a reference point: it cancels)
        if ((lane >> 3) == b) from = c;
        if ((lane >> 3) <= b)
            *reinterpret_cast<float2*>(&t.b[b][2 * lane]) = make_float2((float)(c - x0), (float)(c - x1));
    }
    *reinterpret_cast<float2*>(&t.a[2 * lane]) =
        make_float2((float)(x0 - from) + log2_scale, (float)(x1 - from) + log2_scale);
    *reinterpret_cast<float2*>(&t.e[2 * lane]) = make_float2(f0 >= 0 ? 0.f : fast_exp2((float)x0 + log2_scale),
                                                             f1 >= 0 ? 0.f : fast_exp2((float)x1 + log2_scale));
    *reinterpret_cast<float2*>(&t.w[2 * lane]) = make_float2(2 * lane < border ? 0.f : fast_exp2((float)(last - x0)),
                                                             2 * lane + 1 < border ? 0.f : fast_exp2((float)(last - x1)));
    float down = fminf((float)d0, 0.f) + fminf((float)d1, 0.f);
#pragma unroll
    for (int w = 16; w; w >>= 1) down += __shfl_xor_sync(0xffffffffu, down, w);
    if (lane == 0) {
        t.dec = BORDERS ? 0.f : fast_exp2((float)last);
        t.resets = BORDERS ? 2 : !(down + fminf(log2_scale, 0.f) > -120.f);
    }
}
// (its own function, so that the ordinary tables, on which every chunk waits, stay short)
__device__ __noinline__ void border_tables(Tables* t, float g0, float g1, float log2_scale) {
    fill_tables<true>(*t, g0, g1, log2_scale);
}
__device__ __forceinline__ void make_tables(Tables& t, float g0, float g1, float log2_scale) {
    if (__any_sync(0xffffffffu, forgets(g0) || forgets(g1))) border_tables(&t, g0, g1, log2_scale);
    else fill_tables<false>(t, g0, g1, log2_scale);
}

template <typename T, int DK>
__global__ void __launch_bounds__(NT, DK == 128 ? 2 : 3)
linattn_chunk_kernel(const T* __restrict__ q, long long ldq, const T* __restrict__ k, long long ldk,
                     const T* __restrict__ v, long long ldv, const float* __restrict__ g, long long ldg,
                     const int* __restrict__ cu, int total, const float* state_in, float* state_out,
                     T* __restrict__ o, long long ldo, int Hk, int H, int dv, float log2_scale, int* status) {
    constexpr bool F16 = std::is_same<T, f16>::value;
    constexpr int PARTS = std::is_same<T, f16>::value ? 2 : 3;  // of the state update's scaled v
    constexpr int NKT = DK / 8, KK = DK / 16;  // 8- and 16-wide key tiles
    griddep_sync();
    extern __shared__ __align__(128) uint8_t chunk_raw[];
    ChunkSmem<DK>& sm = *reinterpret_cast<ChunkSmem<DK>*>(chunk_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, lg = lane >> 2, lq = lane & 3;
    const int h = blockIdx.y, hk = h / (H / Hk), c0 = blockIdx.x * CV;
    const int s = ragged::longest_first(cu, gridDim.z, total, blockIdx.z);
    int start, len;
    if (!ragged::sequence(cu, s, total, &start, &len)) {
        if (tid == 0) set_status(status, HYMBA_ERR_DEVICE_RANGE);
        return;
    }
    const int nchunk = (len + CQ - 1) / CQ;
    Stager<T, DK> sq, sk;
    Stager<T, CV> sv;
    sq.init(q + start * ldq + (long long)hk * DK, ldq);
    sk.init(k + start * ldk + (long long)hk * DK, ldk);
    sv.init(v + start * ldv + (long long)h * dv + c0, ldv);
    auto load = [&](int c) {
        sq.load(sm.q[c & 1], c * CQ, len, q);
        sk.load(sm.k[c & 1], c * CQ, len, q);
        sv.load(sm.v[c & 1], c * CQ, len, q);
    };
    g += start * ldg + h;
    auto decay = [&](int t) { return t < len ? g[t * ldg] : 0.f; };
    if (nchunk > 0) load(0);
    wm::cpa_commit();
    float g0 = 0.f, g1 = 0.f;
    if (warp == 0) {
        if (nchunk > 0) make_tables(sm.tab[0], decay(2 * lane), decay(2 * lane + 1), log2_scale);
        g0 = decay(CQ + 2 * lane);
        g1 = decay(CQ + 2 * lane + 1);
    }
    // S[value c0 + 16 warp + lg (+8)][key 8 n + 2 lq (+1)]
    float st[NKT][4];
    const long long sbase = (((long long)s * H + h) * dv + c0 + 16 * warp + lg) * DK + 2 * lq;
#pragma unroll
    for (int n = 0; n < NKT; ++n) {
        float2 a = make_float2(0.f, 0.f), b = a;
        if (state_in) {
            a = *reinterpret_cast<const float2*>(state_in + sbase + 8 * n);
            b = *reinterpret_cast<const float2*>(state_in + sbase + 8 * DK + 8 * n);
        }
        st[n][0] = a.x; st[n][1] = a.y; st[n][2] = b.x; st[n][3] = b.y;
    }
    // per-lane offsets of the ldmatrix pieces: rows lane % 16 at column half lane / 16 (A operands,
    // transposed B operands), and rows of two 8-row tiles at column half (lane / 8) % 2 (B operands)
    uint32_t xa[KK], xb[KK], xp[4];
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
        xa[kk] = at<DK>(lane & 15, 2 * kk + (lane >> 4));
        xb[kk] = at<DK>((lane & 7) + 8 * (lane >> 4), 2 * kk + ((lane >> 3) & 1));
    }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) xp[kk] = at<CQ>(lane & 15, 2 * kk + (lane >> 4));
    const uint32_t xv = at<CV>(lane & 15, 2 * warp + (lane >> 4));
    T* orow = o + (start + (long long)lg) * ldo + (long long)h * dv + c0 + 16 * warp + 2 * lq;

    for (int c = 0; c < nchunk; ++c) {
        const int buf = c & 1, t0 = c * CQ;
        wm::cpa_wait0();
        __syncthreads();  // chunk c and its tables are there; chunk c - 1's stage, tables and P are free
        if (c + 1 < nchunk) load(c + 1);
        wm::cpa_commit();
        const uint8_t *qs = sm.q[buf], *ks = sm.k[buf], *vs = sm.v[buf];
        const Tables& tab = sm.tab[buf];
        const bool resets = tab.resets;
        if (warp == 0 && c + 1 < nchunk) {
            make_tables(sm.tab[buf ^ 1], g0, g1, log2_scale);
            g0 = decay(t0 + 2 * CQ + 2 * lane);
            g1 = decay(t0 + 2 * CQ + 2 * lane + 1);
        }
        // ---- P: rows 16 warp + lg (+8). A row of K that is not finite shows in every score with it,
        // so in the diagonal tiles ----
        bool odd_k;
        {
            const float a0 = tab.a[16 * warp + lg], a1 = tab.a[16 * warp + lg + 8];
            float pr[4][2][4];
            float mx0 = 0.f, mx1 = 0.f;
            float any = 0.f;  // NaN once a score of the diagonal tile is not finite
#pragma unroll
            for (int jt = 0; jt < 4; ++jt)
#pragma unroll
                for (int e = 0; e < 4; ++e) pr[jt][0][e] = pr[jt][1][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                uint32_t qf[4];
                wm::ldsm_x4(qf, qs + warp * 16 * DK * 2 + xa[kk]);
#pragma unroll
                for (int jt = 0; jt < 4; ++jt)
                    if (jt <= warp) {
                        uint32_t kf[4];
                        wm::ldsm_x4(kf, ks + jt * 16 * DK * 2 + xb[kk]);
                        wm::mma16<T>(pr[jt][0], qf, kf[0], kf[1]);
                        wm::mma16<T>(pr[jt][1], qf, kf[2], kf[3]);
                    }
            }
#pragma unroll
            for (int jt = 0; jt < 4; ++jt) {
                if (jt <= warp) {
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const float2 bj = *reinterpret_cast<const float2*>(&tab.b[warp][16 * jt + 8 * n + 2 * lq]);
                        float* p = pr[jt][n];
                        if (jt == warp)
#pragma unroll
                            for (int e = 0; e < 4; ++e) any = fmaf(p[e], 0.f, any);
                        const float w0 = fast_exp2(a0 + bj.x), w1 = fast_exp2(a0 + bj.y);
                        const float w2 = fast_exp2(a1 + bj.x), w3 = fast_exp2(a1 + bj.y);
                        if (!resets) {
                            p[0] *= w0;
                            p[1] *= w1;
                            p[2] *= w2;
                            p[3] *= w3;
                        } else {
                            const int j = 16 * jt + 8 * n + 2 * lq;
                            const int from0 = tab.first(16 * warp + lg), from1 = tab.first(16 * warp + lg + 8);
                            p[0] = j < from0 ? 0.f : fade(w0, p[0]);
                            p[1] = j + 1 < from0 ? 0.f : fade(w1, p[1]);
                            p[2] = j < from1 ? 0.f : fade(w2, p[2]);
                            p[3] = j + 1 < from1 ? 0.f : fade(w3, p[3]);
                        }
                        if (jt == warp) {
                            const int j = 8 * n + 2 * lq;
                            p[0] = j <= lg ? p[0] : 0.f;
                            p[1] = j + 1 <= lg ? p[1] : 0.f;
                            p[2] = j <= lg + 8 ? p[2] : 0.f;
                            p[3] = j + 1 <= lg + 8 ? p[3] : 0.f;
                        }
                        if (F16) {
                            mx0 = fmaxf(mx0, fmaxf(fabsf(p[0]), fabsf(p[1])));
                            mx1 = fmaxf(mx1, fmaxf(fabsf(p[2]), fabsf(p[3])));
                        }
                    }
                }
            }
            odd_k = !(any == 0.f);
            float f0 = 1.f, f1 = 1.f;
            if (F16) {
#pragma unroll
                for (int w = 1; w < 4; w <<= 1) {
                    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, w));
                    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, w));
                }
                f0 = to_middle(mx0, -100, 100);
                f1 = to_middle(mx1, -100, 100);
                if (lq == 0) {
                    sm.ps[16 * warp + lg] = f0;
                    sm.ps[16 * warp + lg + 8] = f1;
                }
            }
            uint8_t* pw = sm.p + (16 * warp + lg) * CQ * 2 + 4 * lq;
#pragma unroll
            for (int jt = 0; jt < 4; ++jt)
                if (jt <= warp)
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        uint8_t* x = pw + ((2 * jt + n) ^ lg) * 16;
                        const float* p = pr[jt][n];
                        *reinterpret_cast<uint32_t*>(x) = F16 ? pack2<T>(p[0] * f0, p[1] * f0) : pack2<T>(p[0], p[1]);
                        *reinterpret_cast<uint32_t*>(x + 8 * CQ * 2) =
                            F16 ? pack2<T>(p[2] * f1, p[3] * f1) : pack2<T>(p[2], p[3]);
                    }
        }
        // ---- 2^cs_i scale S q_i for this warp's value columns ----
        float out[4][2][4];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) out[mt][0][e] = out[mt][1][e] = 0.f;
        if (c > 0 || state_in) {
            // fp16: each value column's power of two
            float fs[2] = {1.f, 1.f};
            if (F16) {
                float mx[2] = {0.f, 0.f};
#pragma unroll
                for (int n = 0; n < NKT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx[e >> 1] = fmaxf(mx[e >> 1], fabsf(st[n][e]));
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    mx[y] = fmaxf(mx[y], __shfl_xor_sync(0xffffffffu, mx[y], 1));
                    mx[y] = fmaxf(mx[y], __shfl_xor_sync(0xffffffffu, mx[y], 2));
                    fs[y] = to_middle(mx[y], -100, 100);
                }
            }
            auto part = [&](float x, float y, int row) { return F16 ? pack2<T>(x * fs[row], y * fs[row]) : pack2<T>(x, y); };
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                const uint32_t b0 = part(st[2 * kk][0], st[2 * kk][1], 0), b1 = part(st[2 * kk + 1][0], st[2 * kk + 1][1], 0);
                const uint32_t b2 = part(st[2 * kk][2], st[2 * kk][3], 1), b3 = part(st[2 * kk + 1][2], st[2 * kk + 1][3], 1);
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) {
                    uint32_t qf[4];
                    wm::ldsm_x4(qf, qs + mt * 16 * DK * 2 + xa[kk]);
                    wm::mma16<T>(out[mt][0], qf, b0, b1);
                    wm::mma16<T>(out[mt][1], qf, b2, b3);
                }
            }
            if (F16) {
                // this lane's columns 2 lq and 2 lq + 1 of both halves lie in the lanes with that lg
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float back = inverse(fs[n]);
                    const float b0 = __shfl_sync(0xffffffffu, back, 8 * lq), b1 = __shfl_sync(0xffffffffu, back, 8 * lq + 4);
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt) {
                        out[mt][n][0] *= b0;
                        out[mt][n][1] *= b1;
                        out[mt][n][2] *= b0;
                        out[mt][n][3] *= b1;
                    }
                }
            }
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                const float ea = tab.e[16 * mt + lg], eb = tab.e[16 * mt + lg + 8];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    if (!resets) {
                        out[mt][n][0] *= ea;
                        out[mt][n][1] *= ea;
                        out[mt][n][2] *= eb;
                        out[mt][n][3] *= eb;
                    } else {
                        out[mt][n][0] = fade(ea, out[mt][n][0]);
                        out[mt][n][1] = fade(ea, out[mt][n][1]);
                        out[mt][n][2] = fade(eb, out[mt][n][2]);
                        out[mt][n][3] = fade(eb, out[mt][n][3]);
                    }
                }
            }
        }
        // ---- V fragments: B operand (rows j x 16 value columns), and V^T as the A operand ----
        uint32_t vf[4][4];
        bool odd;
        {
            auto zero = pair<T>(0u), any = zero;  // 0 x (not finite) is NaN
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                wm::ldsm_x4_t(vf[kk], vs + kk * 16 * CV * 2 + xv);
#pragma unroll
                for (int e = 0; e < 4; ++e) any = __hfma2(pair<T>(vf[kk][e]), zero, any);
            }
            odd = __any_sync(0xffffffffu, (bits(any) & 0x7fff7fffu) != 0);
        }
        odd_k = __syncthreads_or(odd_k);  // P is there; K of the whole chunk
        // ---- + P V ----
        if (!odd) {
            if (F16) {
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) {
                    const float fa = sm.ps[16 * mt + lg], fb = sm.ps[16 * mt + lg + 8];
                    scale_rows(out[mt], fa, fb);
                }
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                for (int mt = kk; mt < 4; ++mt) {
                    uint32_t pf[4];
                    wm::ldsm_x4(pf, sm.p + mt * 16 * CQ * 2 + xp[kk]);
                    wm::mma16<T>(out[mt][0], pf, vf[kk][0], vf[kk][1]);
                    wm::mma16<T>(out[mt][1], pf, vf[kk][2], vf[kk][3]);
                }
            if (F16) {
#pragma unroll
                for (int mt = 0; mt < 4; ++mt)
                    scale_rows(out[mt], inverse(sm.ps[16 * mt + lg]), inverse(sm.ps[16 * mt + lg + 8]));
            }
        } else {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int n = e >> 2, i = 16 * mt + lg + 8 * ((e >> 1) & 1), col = 16 * warp + 8 * n + 2 * lq + (e & 1);
                    const float x = row_product<T>(tab, sm.p, vs, i, col);
                    out[mt][n][e & 3] += F16 ? x / sm.ps[i] : x;
                }
        }
        // ---- o ----
        {
            T* x = orow;
#pragma unroll
            for (int r = 0; r < 8; ++r, x += 8 * ldo) {
                if (t0 + 8 * r + lg < len) {
                    const float* y = out[r >> 1][0] + 2 * (r & 1);
                    *reinterpret_cast<uint32_t*>(x) = pack2<T>(y[0], y[1]);
                    *reinterpret_cast<uint32_t*>(x + 8) = pack2<T>(y[4], y[5]);
                }
            }
            orow = x;
        }
        // ---- state ----
        if (odd || odd_k) {
            row_states<T, DK>(tab, ks, vs, 16 * warp + lg, st);
        } else {
            // fp16: each value column's power of two, from its largest weighted value
            float fv[2] = {1.f, 1.f};
            if (F16) {
                float m[2] = {0.f, 0.f};
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float2 w = *reinterpret_cast<const float2*>(&tab.w[16 * kk + 8 * x + 2 * lq]);
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const T* e = reinterpret_cast<const T*>(&vf[kk][2 * y + x]);
                            const float2 z = __fmul2_rn(make_float2(to_f(e[0]), to_f(e[1])), w);
                            m[y] = fmaxf(m[y], fmaxf(fabsf(z.x), fabsf(z.y)));
                        }
                    }
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    m[y] = fmaxf(m[y], __shfl_xor_sync(0xffffffffu, m[y], 1));
                    m[y] = fmaxf(m[y], __shfl_xor_sync(0xffffffffu, m[y], 2));
                    fv[y] = to_middle(m[y], -100, 40);
                }
            }
            const float dec0 = tab.dec * fv[0], dec1 = tab.dec * fv[1];
            if (!resets) {
                scale_state<NKT>(st, dec0, dec1);
            } else {
#pragma unroll
                for (int n = 0; n < NKT; ++n) {
                    st[n][0] = fade(dec0, st[n][0]);
                    st[n][1] = fade(dec0, st[n][1]);
                    st[n][2] = fade(dec1, st[n][2]);
                    st[n][3] = fade(dec1, st[n][3]);
                }
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                uint32_t kf[KK][4];
#pragma unroll
                for (int n = 0; n < KK; ++n) wm::ldsm_x4_t(kf[n], ks + kk * 16 * DK * 2 + xa[n]);
                uint32_t part[PARTS][4];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float2 w = *reinterpret_cast<const float2*>(&tab.w[16 * kk + 8 * x + 2 * lq]);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        // V fragment (values 8 y .., rows 8 x ..) is operand part 2 x + y
                        const T* e = reinterpret_cast<const T*>(&vf[kk][2 * y + x]);
                        const float2 wf = F16 ? make_float2(w.x * fv[y], w.y * fv[y]) : w;
                        const float2 z = __fmul2_rn(make_float2(to_f(e[0]), to_f(e[1])), wf);
                        part[0][2 * x + y] = pack2<T>(z.x, z.y);
                        float2 left = z;
#pragma unroll
                        for (int p = 1; p < PARTS; ++p) {
                            const T* of = reinterpret_cast<const T*>(&part[p - 1][2 * x + y]);
                            left = make_float2(left.x - to_f(of[0]), left.y - to_f(of[1]));  // exact
                            part[p][2 * x + y] = pack2<T>(left.x, left.y);
                        }
                    }
                }
#pragma unroll
                for (int p = 0; p < PARTS; ++p)
#pragma unroll
                    for (int n = 0; n < KK; ++n) {
                        wm::mma16<T>(st[2 * n], part[p], kf[n][0], kf[n][1]);
                        wm::mma16<T>(st[2 * n + 1], part[p], kf[n][2], kf[n][3]);
                    }
            }
            if (F16) scale_state<NKT>(st, inverse(fv[0]), inverse(fv[1]));
        }
    }
    wm::cpa_wait0();
    if (state_out) {
#pragma unroll
        for (int n = 0; n < NKT; ++n) {
            *reinterpret_cast<float2*>(state_out + sbase + 8 * n) = make_float2(st[n][0], st[n][1]);
            *reinterpret_cast<float2*>(state_out + sbase + 8 * DK + 8 * n) = make_float2(st[n][2], st[n][3]);
        }
    }
}

template <typename T, int DK>
int launch_dk(const Ctx& ctx, const LinAttn& a) {
    auto kern = linattn_chunk_kernel<T, DK>;
    const size_t smem = sizeof(ChunkSmem<DK>);
    static std::atomic<unsigned long long> smem_set{0};
    if (!smem_opt_in_once(smem_set, kern, smem, ctx)) return HYMBA_ERR_CUDA;
    // sequences on the grid's slowest dimension, in runs it can hold
    for (int s0 = 0; s0 < a.n_seqs; s0 += 65535) {
        const int n = a.n_seqs - s0 < 65535 ? a.n_seqs - s0 : 65535;
        const long long st0 = (long long)s0 * a.H * a.dv * DK;
        HYMBA_LAUNCH(ctx, "linattn_chunk", kern, dim3(a.dv / CV, a.H, n), NT, smem, static_cast<const T*>(a.q), a.ldq,
                     static_cast<const T*>(a.k), a.ldk, static_cast<const T*>(a.v), a.ldv, a.g, a.ldg, a.cu + s0,
                     a.total, a.state_in ? a.state_in + st0 : nullptr, a.state_out ? a.state_out + st0 : nullptr,
                     static_cast<T*>(a.o), a.ldo, a.Hk, a.H, a.dv, log2f(a.scale), ctx.status);
    }
    return HYMBA_OK;
}

}  // namespace

template <typename T>
int launch_linattn_chunk(const Ctx& ctx, const LinAttn& a) {
    if (a.dk == 16) return launch_dk<T, 16>(ctx, a);
    if (a.dk == 128) return launch_dk<T, 128>(ctx, a);
    return HYMBA_ERR_UNSUPPORTED;
}
template int launch_linattn_chunk<f16>(const Ctx&, const LinAttn&);
template int launch_linattn_chunk<bf16>(const Ctx&, const LinAttn&);

}  // namespace hymba
