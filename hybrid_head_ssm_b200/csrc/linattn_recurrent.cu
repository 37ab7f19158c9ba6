// Linear attention with a decay per head, recurrent form: S_t = exp(g_t) S_{t-1} + v_t
// k_t^T, o_t = scale S_t q_t ("Lecture 04 - Beyond the Dense Transformer", sections 2 and
// 3: the SSM recurrence with a scalar decay per head). One token per sequence, and
// packed fp32 prompts.
//
// State S [v_head_dim, key_dim] fp32 per (sequence, head). A warp owns VR consecutive rows
// of S in registers: LPR lanes per row, each with every LPR-th float4 of the key
// dimension, so a warp's loads are whole 128-byte lines and a row's product with q is a
// shuffle over LPR lanes. Single tokens are bound by HBM: 8 bytes per state element; 256 of 25
// heads of 64 x 128 64.9 us called back to back (the copy rate), one 2.2 us. fp32 prompts are bound by the chain of rows (a
// round trip to memory, 64 multiply-adds and a shuffle each): 185 rows 104 us, eight of up to 4224
// rows 3864 us (their bytes take 118).
#include "kernels.h"
#include "ragged.cuh"

namespace hymba {

namespace {

constexpr int NT = 128;  // 4 warps

template <typename T, int DK, int VR, bool PACKED>
__global__ void __launch_bounds__(NT)
linattn_recurrent_kernel(const T* __restrict__ q, long long ldq, const T* __restrict__ k, long long ldk,
                         const T* __restrict__ v, long long ldv, const float* __restrict__ g, long long ldg,
                         const int* __restrict__ cu, int total, const float* state_in, float* state_out,
                         T* __restrict__ o, long long ldo, int Hk, int H, int dv, float scale, int* status) {
    griddep_sync();
    constexpr int LPR = DK >= 32 ? 8 : DK / 4;  // lanes per state row
    constexpr int RPI = 32 / LPR;               // rows a warp touches at a time
    constexpr int NR = VR / RPI;                // rows per lane
    constexpr int NC = DK / 4 / LPR;            // float4s per lane and row
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane % LPR, rsub = lane / LPR;
    const int h = blockIdx.y, hk = h / (H / Hk);
    const int s = PACKED ? ragged::longest_first(cu, gridDim.z, total, blockIdx.z) : blockIdx.z;
    const int r0 = (blockIdx.x * (NT / 32) + warp) * VR;  // the warp's first v row
    if (r0 >= dv) return;
    int start = s, len = 1;
    if (PACKED && !ragged::sequence(cu, s, total, &start, &len)) {
        if (threadIdx.x == 0) set_status(status, HYMBA_ERR_DEVICE_RANGE);
        return;
    }
    const long long sbase = (((long long)s * H + h) * dv + r0) * DK;
    float4 S[NR][NC];
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int c = 0; c < NC; ++c)
            S[r][c] = state_in ? *reinterpret_cast<const float4*>(state_in + sbase + (r * RPI + rsub) * DK +
                                                                  4 * (c * LPR + sub))
                               : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int t = 0; t < len; ++t) {
        const long long row = (long long)start + t;
        const float dec = expf(g[row * ldg + h]);
        float4 kq[NC], qq[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            kq[c] = ragged::load4(k + row * ldk + (long long)hk * DK + 4 * (c * LPR + sub));
            qq[c] = ragged::load4(q + row * ldq + (long long)hk * DK + 4 * (c * LPR + sub));
        }
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const float x = to_f(v[row * ldv + (long long)h * dv + r0 + r * RPI + rsub]);
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                float4& e = S[r][c];
                // a decay of exactly 0 forgets whatever the state held (also what is not finite)
                e.x = fmaf(x, kq[c].x, dec == 0.f ? 0.f : dec * e.x);
                e.y = fmaf(x, kq[c].y, dec == 0.f ? 0.f : dec * e.y);
                e.z = fmaf(x, kq[c].z, dec == 0.f ? 0.f : dec * e.z);
                e.w = fmaf(x, kq[c].w, dec == 0.f ? 0.f : dec * e.w);
                sum = fmaf(e.x, qq[c].x, fmaf(e.y, qq[c].y, fmaf(e.z, qq[c].z, fmaf(e.w, qq[c].w, sum))));
            }
#pragma unroll
            for (int w = 1; w < LPR; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            if (sub == 0) o[row * ldo + (long long)h * dv + r0 + r * RPI + rsub] = from_f<T>(sum * scale);
        }
    }
    if (state_out) {
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int c = 0; c < NC; ++c)
                *reinterpret_cast<float4*>(state_out + sbase + (r * RPI + rsub) * DK + 4 * (c * LPR + sub)) = S[r][c];
    }
}

template <typename T, int DK, bool PACKED>
int launch_form(const Ctx& ctx, const LinAttn& a) {
    constexpr int VR = 16;
    auto kern = linattn_recurrent_kernel<T, DK, VR, PACKED>;
    // sequences on the grid's slowest dimension, in runs it can hold
    for (int s0 = 0; s0 < a.n_seqs; s0 += 65535) {
        const int n = a.n_seqs - s0 < 65535 ? a.n_seqs - s0 : 65535;
        const long long row0 = PACKED ? 0 : s0;
        const long long st0 = (long long)s0 * a.H * a.dv * DK;
        HYMBA_LAUNCH(ctx, PACKED ? "linattn_recurrent" : "linattn_step", kern,
                     dim3(ceil_div(a.dv, VR * (NT / 32)), a.H, n), NT, 0, static_cast<const T*>(a.q) + row0 * a.ldq,
                     a.ldq, static_cast<const T*>(a.k) + row0 * a.ldk, a.ldk, static_cast<const T*>(a.v) + row0 * a.ldv,
                     a.ldv, a.g + row0 * a.ldg, a.ldg, PACKED ? a.cu + s0 : nullptr, a.total,
                     a.state_in ? a.state_in + st0 : nullptr, a.state_out ? a.state_out + st0 : nullptr,
                     static_cast<T*>(a.o) + row0 * a.ldo, a.ldo, a.Hk, a.H, a.dv, a.scale, ctx.status);
    }
    return HYMBA_OK;
}

template <typename T, int DK>
int launch_dk(const Ctx& ctx, const LinAttn& a) {
    if constexpr (sizeof(T) == 4) {
        if (a.cu) return launch_form<T, DK, true>(ctx, a);
    }
    return launch_form<T, DK, false>(ctx, a);
}

}  // namespace

template <typename T>
int launch_linattn_recurrent(const Ctx& ctx, const LinAttn& a) {
    if (a.dk == 16) return launch_dk<T, 16>(ctx, a);
    if (a.dk == 64) return launch_dk<T, 64>(ctx, a);
    if (a.dk == 128) return launch_dk<T, 128>(ctx, a);
    return HYMBA_ERR_UNSUPPORTED;
}
template int launch_linattn_recurrent<float>(const Ctx&, const LinAttn&);
template int launch_linattn_recurrent<f16>(const Ctx&, const LinAttn&);
template int launch_linattn_recurrent<bf16>(const Ctx&, const LinAttn&);

}  // namespace hymba
