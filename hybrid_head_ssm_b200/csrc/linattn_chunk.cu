// Linear attention with a decay per head, chunked form on the tensor cores (16-bit rows):
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
// Numbers: cs is summed in 64 bits and kept as hi + lo pairs, so a decay between two rows is
// right to fp32 after any other row (one that forgets everything included). P and the copy of
// S that meets q are rounded to the rows' type, like any MMA operand; the scaled v of the state
// update enters as two 16-bit parts, so the fp32 state keeps 16 bits or more of every term.
// fp16 has little range: P's rows, S's copy and the scaled v are brought to the middle of it by
// powers of two, which are taken out again from the fp32 sums.
// A row's values reach only what sees them: rows behind the sequence are zero-filled, a
// decay of 0 drops what it multiplies, and a chunk whose V holds a value that is not finite
// forms P V row by row.
// Bound: HBM (q, k, v once per 64 value columns, o) with the MMAs close behind.
#include "kernels.h"
#include "ragged.cuh"

namespace hymba {

namespace {

constexpr int CQ = 64;   // rows per chunk
constexpr int CV = 64;   // value columns per CTA
constexpr int NT = 128;  // 4 warps
constexpr double LOG2E = 1.4426950408889634;

template <int DK>
struct ChunkSmem {
    // rows of DK or 64 16-bit elements, 16-byte pieces swizzled by the row
    alignas(128) uint8_t q[2][CQ * DK * 2];
    alignas(128) uint8_t k[2][CQ * DK * 2];
    alignas(128) uint8_t v[2][CQ * CV * 2];
    alignas(128) uint8_t p[CQ * CQ * 2];
    alignas(16) float2 cs[4][CQ];  // each warp's copy: cs in log2 units, hi and lo
    alignas(16) float ps[CQ];      // 1 / power of two that P's rows carry
};

// byte offset of 16-byte piece c of row r of a tile of COLS 16-bit columns; 8 rows at one c
// cover all banks
template <int COLS>
__device__ __forceinline__ uint32_t at(int r, int c) {
    if constexpr (COLS == 16) return r * 32 + ((c ^ ((r >> 2) & 1)) * 16);
    else return r * COLS * 2 + ((c ^ (r & 7)) * 16);
}

// rows t0 .. t0 + 63 of the sequence; rows past its end read as zero
template <typename T, int COLS>
__device__ __forceinline__ void stage(uint8_t* dst, const T* src, long long ld, int t0, int len) {
    constexpr int PC = COLS / 8;
#pragma unroll
    for (int x = threadIdx.x; x < CQ * PC; x += NT) {
        const int r = x / PC, c = x % PC;
        const bool in = t0 + r < len;
        wm::cpa16(dst + at<COLS>(r, c), src + (in ? (long long)(t0 + r) * ld : 0) + c * 8, !in);
    }
}

// a power of two that brings x (> 0) near 2^12, at most 2^40 (the fp32 sums that carry it stay
// far from their limits); 1 for 0 and what is not finite
__device__ __forceinline__ float to_middle(float x) {
    const int e = (__float_as_int(x) >> 23) & 255;
    if (e == 0 || e == 255) return 1.f;
    return __int_as_float(min(max(254 - e + 12, 1), 127 + 40) << 23);
}

// a decay of 0 drops what it multiplies, also what is not finite
__device__ __forceinline__ float fade(float d, float x) { return d == 0.f ? 0.f : d * x; }

template <typename T>
__device__ __forceinline__ bool odd2(uint32_t w) {
    constexpr uint32_t E = std::is_same<T, bf16>::value ? 0x7f807f80u : 0x7c007c00u;
    return __vcmpeq2(w & E, E) != 0;
}

template <typename T, int DK>
__global__ void __launch_bounds__(NT, DK == 128 ? 2 : 3)
linattn_chunk_kernel(const T* __restrict__ q, long long ldq, const T* __restrict__ k, long long ldk,
                     const T* __restrict__ v, long long ldv, const float* __restrict__ g, long long ldg,
                     const int* __restrict__ cu, int total, const float* state_in, float* state_out,
                     T* __restrict__ o, long long ldo, int Hk, int H, int dv, float scale, int* status) {
    constexpr bool F16 = std::is_same<T, f16>::value;
    constexpr int NKT = DK / 8;  // 8-wide key tiles of the state
    griddep_sync();
    extern __shared__ __align__(128) uint8_t chunk_raw[];
    ChunkSmem<DK>& sm = *reinterpret_cast<ChunkSmem<DK>*>(chunk_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, lg = lane >> 2, lq = lane & 3;
    const int h = blockIdx.y, s = blockIdx.z, hk = h / (H / Hk), c0 = blockIdx.x * CV;
    int start, len;
    if (!ragged::sequence(cu, s, total, &start, &len)) {
        if (tid == 0) set_status(status, HYMBA_ERR_DEVICE_RANGE);
        return;
    }
    q += start * ldq + (long long)hk * DK;
    k += start * ldk + (long long)hk * DK;
    v += start * ldv + (long long)h * dv + c0;
    o += start * ldo + (long long)h * dv + c0;
    g += start * ldg + h;
    const int nchunk = (len + CQ - 1) / CQ;
    auto load = [&](int c) {
        stage<T, DK>(sm.q[c & 1], q, ldq, c * CQ, len);
        stage<T, DK>(sm.k[c & 1], k, ldk, c * CQ, len);
        stage<T, CV>(sm.v[c & 1], v, ldv, c * CQ, len);
    };
    auto decay = [&](int t) { return t < len ? g[t * ldg] : 0.f; };
    if (nchunk > 0) load(0);
    wm::cpa_commit();
    float g0 = decay(2 * lane), g1 = decay(2 * lane + 1);
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

    for (int c = 0; c < nchunk; ++c) {
        const int buf = c & 1, t0 = c * CQ;
        wm::cpa_wait0();
        __syncthreads();  // chunk c is staged; chunk c - 1's stage and P are free
        if (c + 1 < nchunk) load(c + 1);
        wm::cpa_commit();
        // ---- decays: inclusive sums of the chunk's rows, every warp for itself ----
        {
            // a decay below 2^-160 is 0 in fp32; the limit keeps -infinity out of the sums
            const double d0 = fmax((double)g0 * LOG2E, -160.0), d1 = fmax((double)g1 * LOG2E, -160.0);
            double x = (g0 != g0 ? (double)g0 : d0) + (g1 != g1 ? (double)g1 : d1);
            const double mine1 = g1 != g1 ? (double)g1 : d1;
#pragma unroll
            for (int w = 1; w < 32; w <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, x, w);
                if (lane >= w) x += y;
            }
            const double x0 = x - mine1;
            const float a = (float)x0, b = (float)x;
            *reinterpret_cast<float4*>(&sm.cs[warp][2 * lane]) = make_float4(a, (float)(x0 - a), b, (float)(x - b));
            if (c + 1 < nchunk) {
                g0 = decay(t0 + CQ + 2 * lane);
                g1 = decay(t0 + CQ + 2 * lane + 1);
            }
        }
        __syncwarp();
        const float2* cs = sm.cs[warp];
        // ---- P: rows 16 warp + lg (+8) ----
        {
            const int r0 = 16 * warp;
            const float2 ci0 = cs[r0 + lg], ci1 = cs[r0 + lg + 8];
            float pr[4][2][4];
            float mx0 = 0.f, mx1 = 0.f;
            uint32_t qf[DK / 16][4];
#pragma unroll
            for (int kk = 0; kk < DK / 16; ++kk)
                wm::ldsm_x4(qf[kk], sm.q[buf] + at<DK>(r0 + (lane & 15), 2 * kk + (lane >> 4)));
#pragma unroll
            for (int jt = 0; jt < 4; ++jt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) pr[jt][0][e] = pr[jt][1][e] = 0.f;
                if (jt <= warp) {
#pragma unroll
                    for (int kk = 0; kk < DK / 16; ++kk) {
                        uint32_t kf[4];
                        wm::ldsm_x4(kf, sm.k[buf] + at<DK>(16 * jt + (lane & 7) + 8 * (lane >> 4), 2 * kk + ((lane >> 3) & 1)));
                        wm::mma16<T>(pr[jt][0], qf[kk], kf[0], kf[1]);
                        wm::mma16<T>(pr[jt][1], qf[kk], kf[2], kf[3]);
                    }
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const int j = 16 * jt + 8 * n + 2 * lq;
                        const float4 cj = *reinterpret_cast<const float4*>(&cs[j]);
                        const int i = r0 + lg;
                        float* p = pr[jt][n];
                        p[0] = j <= i ? fade(fast_exp2((ci0.x - cj.x) + (ci0.y - cj.y)), p[0] * scale) : 0.f;
                        p[1] = j + 1 <= i ? fade(fast_exp2((ci0.x - cj.z) + (ci0.y - cj.w)), p[1] * scale) : 0.f;
                        p[2] = j <= i + 8 ? fade(fast_exp2((ci1.x - cj.x) + (ci1.y - cj.y)), p[2] * scale) : 0.f;
                        p[3] = j + 1 <= i + 8 ? fade(fast_exp2((ci1.x - cj.z) + (ci1.y - cj.w)), p[3] * scale) : 0.f;
                        if (F16) {
                            mx0 = fmaxf(mx0, fmaxf(fabsf(p[0]), fabsf(p[1])));
                            mx1 = fmaxf(mx1, fmaxf(fabsf(p[2]), fabsf(p[3])));
                        }
                    }
                }
            }
            float f0 = 1.f, f1 = 1.f;
            if (F16) {
#pragma unroll
                for (int w = 1; w < 4; w <<= 1) {
                    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, w));
                    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, w));
                }
                f0 = to_middle(mx0);
                f1 = to_middle(mx1);
                if (lq == 0) {
                    sm.ps[r0 + lg] = f0;
                    sm.ps[r0 + lg + 8] = f1;
                }
            }
#pragma unroll
            for (int jt = 0; jt < 4; ++jt)
                if (jt <= warp)
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        uint8_t* a = sm.p + at<CQ>(r0 + lg, 2 * jt + n) + 4 * lq;
                        uint8_t* b = sm.p + at<CQ>(r0 + lg + 8, 2 * jt + n) + 4 * lq;
                        *reinterpret_cast<uint32_t*>(a) = pack2<T>(pr[jt][n][0] * f0, pr[jt][n][1] * f0);
                        *reinterpret_cast<uint32_t*>(b) = pack2<T>(pr[jt][n][2] * f1, pr[jt][n][3] * f1);
                    }
        }
        // ---- exp(cs_i) scale S q_i for this warp's value columns ----
        float out[4][2][4];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) out[mt][0][e] = out[mt][1][e] = 0.f;
        if (c > 0 || state_in) {
            float fs = 1.f;
            if (F16) {
                float mx = 0.f;
#pragma unroll
                for (int n = 0; n < NKT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fabsf(st[n][e]));
#pragma unroll
                for (int w = 1; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
                fs = to_middle(mx);
            }
#pragma unroll
            for (int kk = 0; kk < DK / 16; ++kk) {
                const uint32_t b0 = pack2<T>(st[2 * kk][0] * fs, st[2 * kk][1] * fs);
                const uint32_t b1 = pack2<T>(st[2 * kk + 1][0] * fs, st[2 * kk + 1][1] * fs);
                const uint32_t b2 = pack2<T>(st[2 * kk][2] * fs, st[2 * kk][3] * fs);
                const uint32_t b3 = pack2<T>(st[2 * kk + 1][2] * fs, st[2 * kk + 1][3] * fs);
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) {
                    uint32_t qf[4];
                    wm::ldsm_x4(qf, sm.q[buf] + at<DK>(16 * mt + (lane & 15), 2 * kk + (lane >> 4)));
                    wm::mma16<T>(out[mt][0], qf, b0, b1);
                    wm::mma16<T>(out[mt][1], qf, b2, b3);
                }
            }
            const float back = scale / fs;
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                const float2 a = cs[16 * mt + lg], b = cs[16 * mt + lg + 8];
                const float ea = fast_exp2(a.x + a.y), eb = fast_exp2(b.x + b.y);
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    out[mt][n][0] = fade(ea, out[mt][n][0] * back);
                    out[mt][n][1] = fade(ea, out[mt][n][1] * back);
                    out[mt][n][2] = fade(eb, out[mt][n][2] * back);
                    out[mt][n][3] = fade(eb, out[mt][n][3] * back);
                }
            }
        }
        // ---- V fragments: B operand (rows j x 16 value columns), and V^T as the A operand ----
        uint32_t vf[4][4];
        bool odd = false;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            wm::ldsm_x4_t(vf[kk], sm.v[buf] + at<CV>(16 * kk + (lane & 7) + 8 * ((lane >> 3) & 1), 2 * warp + (lane >> 4)));
#pragma unroll
            for (int e = 0; e < 4; ++e) odd |= odd2<T>(vf[kk][e]);
        }
        odd = __any_sync(0xffffffffu, odd);
        __syncthreads();  // P is there
        // ---- + P V ----
        if (!odd) {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                float fa = 1.f, fb = 1.f;
                if (F16) {
                    fa = sm.ps[16 * mt + lg];
                    fb = sm.ps[16 * mt + lg + 8];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        out[mt][n][0] *= fa;
                        out[mt][n][1] *= fa;
                        out[mt][n][2] *= fb;
                        out[mt][n][3] *= fb;
                    }
                }
#pragma unroll
                for (int kk = 0; kk <= mt; ++kk) {
                    uint32_t pf[4];
                    wm::ldsm_x4(pf, sm.p + at<CQ>(16 * mt + (lane & 15), 2 * kk + (lane >> 4)));
                    wm::mma16<T>(out[mt][0], pf, vf[kk][0], vf[kk][1]);
                    wm::mma16<T>(out[mt][1], pf, vf[kk][2], vf[kk][3]);
                }
                if (F16) {
                    fa = 1.f / fa;
                    fb = 1.f / fb;
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        out[mt][n][0] *= fa;
                        out[mt][n][1] *= fa;
                        out[mt][n][2] *= fb;
                        out[mt][n][3] *= fb;
                    }
                }
            }
        } else {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int n = e >> 2, i = 16 * mt + lg + 8 * ((e >> 1) & 1), col = 16 * warp + 8 * n + 2 * lq + (e & 1);
                    const float2 ci = cs[i];
                    float sum = 0.f;
#pragma unroll 1
                    for (int j = 0; j <= i; ++j) {
                        const float2 cj = cs[j];
                        if (fast_exp2((ci.x - cj.x) + (ci.y - cj.y)) == 0.f) continue;
                        const T pj = *reinterpret_cast<const T*>(sm.p + at<CQ>(i, j >> 3) + 2 * (j & 7));
                        const T vj = *reinterpret_cast<const T*>(sm.v[buf] + at<CV>(j, col >> 3) + 2 * (col & 7));
                        sum = fmaf(to_f(pj), to_f(vj), sum);
                    }
                    out[mt][n][e & 3] += F16 ? sum / sm.ps[i] : sum;
                }
        }
        // ---- o ----
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int i = t0 + 16 * mt + lg + 8 * half;
                if (i < len)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
                        *reinterpret_cast<uint32_t*>(o + i * ldo + 16 * warp + 8 * n + 2 * lq) =
                            pack2<T>(out[mt][n][2 * half], out[mt][n][2 * half + 1]);
            }
        // ---- state ----
        {
            const float2 cl = cs[CQ - 1];
            const float dec = fast_exp2(cl.x + cl.y);
            float w[4][4];  // exp(cs_64 - cs_j) of rows 16 kk + 2 lq, + 1, + 8, + 9
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float4 cj = *reinterpret_cast<const float4*>(&cs[16 * kk + 2 * lq + 8 * x]);
                    w[kk][2 * x] = fast_exp2((cl.x - cj.x) + (cl.y - cj.y));
                    w[kk][2 * x + 1] = fast_exp2((cl.x - cj.z) + (cl.y - cj.w));
                }
            auto scaled = [&](int kk, int e, float* x0, float* x1) {
                // fragment e: rows + 8 for odd e (the second row half of the ldmatrix pair)
                const T* x = reinterpret_cast<const T*>(&vf[kk][e]);
                *x0 = fade(w[kk][2 * (e & 1)], to_f(x[0]));
                *x1 = fade(w[kk][2 * (e & 1) + 1], to_f(x[1]));
            };
            float fv = 1.f;
            if (F16) {
                float mx = 0.f;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x0, x1;
                        scaled(kk, e, &x0, &x1);
                        mx = fmaxf(mx, fmaxf(fabsf(x0), fabsf(x1)));
                    }
#pragma unroll
                for (int x = 1; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
                fv = to_middle(mx);
            }
#pragma unroll
            for (int n = 0; n < NKT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) st[n][e] = fade(dec, st[n][e]) * fv;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // A operand order: (values 0-7, rows 0-7), (8-15, 0-7), (0-7, 8-15), (8-15, 8-15)
                    const int from = ((e & 1) << 1) | (e >> 1);
                    float x0, x1;
                    scaled(kk, from, &x0, &x1);
                    wm::split2<T>(x0 * fv, x1 * fv, &hi[e], &lo[e]);
                }
#pragma unroll
                for (int n2 = 0; n2 < DK / 16; ++n2) {
                    uint32_t kf[4];
                    wm::ldsm_x4_t(kf, sm.k[buf] + at<DK>(16 * kk + (lane & 7) + 8 * ((lane >> 3) & 1), 2 * n2 + (lane >> 4)));
                    wm::mma16<T>(st[2 * n2], hi, kf[0], kf[1]);
                    wm::mma16<T>(st[2 * n2 + 1], hi, kf[2], kf[3]);
                    wm::mma16<T>(st[2 * n2], lo, kf[0], kf[1]);
                    wm::mma16<T>(st[2 * n2 + 1], lo, kf[2], kf[3]);
                }
            }
            if (F16) {
                const float back = 1.f / fv;
#pragma unroll
                for (int n = 0; n < NKT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) st[n][e] *= back;
            }
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
                     static_cast<T*>(a.o), a.ldo, a.Hk, a.H, a.dv, a.scale, ctx.status);
    }
    return HYMBA_OK;
}

}  // namespace

template <typename T>
int launch_linattn_chunk(const Ctx& ctx, const LinAttn& a) {
    if (a.dk == 16) return launch_dk<T, 16>(ctx, a);
    if (a.dk == 64) return launch_dk<T, 64>(ctx, a);
    if (a.dk == 128) return launch_dk<T, 128>(ctx, a);
    return HYMBA_ERR_UNSUPPORTED;
}
template int launch_linattn_chunk<f16>(const Ctx&, const LinAttn&);
template int launch_linattn_chunk<bf16>(const Ctx&, const LinAttn&);

}  // namespace hymba
