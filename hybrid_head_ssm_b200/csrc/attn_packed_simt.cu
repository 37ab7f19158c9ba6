// Causal attention over packed prompts on CUDA cores (fp32 rows): softmax(scale q k^T) v
// with grouped heads, meta prefix + window or the whole history, counted from each
// sequence's first row ("Jamba: Hybrid SSM-Transformer", section 1; "Hymba Guide",
// Learnable Meta-Tokens; 51cto Hymba-1.5B article, section 2).
//
// One 256-thread block per (tile of 64, 32 or 16 query rows of a sequence, head), the heaviest
// rows of a sequence first. Key tiles of 64: S as rows / 16 x 4 per thread from transposed Q
// and K tiles, one running max and sum per row, P transposed through shared memory, O as
// rows / 16 x DV / 16 per thread, all on packed pairs (two FMAs per instruction). Bound by the FMA
// pipe for long prompts (2 (dh + dv) flops per visible pair, and the diagonal tiles' masked
// half on top), by the chain of key tiles for short ones.
#include "kernels.h"
#include "ragged.cuh"

namespace hymba {

namespace {

constexpr int KT = 64, NT = 256;

template <int DH, int DV, int QT>
struct PackedSimtSmem {
    alignas(16) float q[DH][QT + 4];  // transposed: [dim][row]
    alignas(16) float k[DH][KT + 4];  // transposed: [dim][key]
    alignas(16) float v[KT][DV];
    alignas(16) float p[KT][QT + 4];  // transposed: [key][row]
    ragged::FindSmem find;
};

// RT consecutive values of a transposed tile (one load)
template <int RT>
__device__ __forceinline__ void row_values(const float* p, float (&v)[RT]) {
    if constexpr (RT == 4) {
        const float4 a = *reinterpret_cast<const float4*>(p);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    } else if constexpr (RT == 2) {
        const float2 a = *reinterpret_cast<const float2*>(p);
        v[0] = a.x; v[1] = a.y;
    } else {
        v[0] = *p;
    }
}

template <typename T, int DH, int DV, int QT>
__global__ void __launch_bounds__(NT)
attn_packed_simt_kernel(const T* __restrict__ q, long long ldq, const T* __restrict__ k, long long ldk,
                        const T* __restrict__ v, long long ldv, const int* __restrict__ cu, int n_seqs, int total,
                        T* __restrict__ o, long long ldo, int H, int G, int n_meta, int window, float scale_log2,
                        int* status) {
    griddep_sync();
    extern __shared__ __align__(16) uint8_t packed_simt_raw[];
    PackedSimtSmem<DH, DV, QT>& sm = *reinterpret_cast<PackedSimtSmem<DH, DV, QT>*>(packed_simt_raw);
    constexpr int RT = QT / 16;  // rows per thread
    const int h = blockIdx.x % H, tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const ragged::Item it = ragged::find_item<NT>(sm.find, cu, n_seqs, total, QT, blockIdx.x / H, status);
    if (it.seq < 0) return;
    const int L = it.len;
    const int i0 = ((L + QT - 1) / QT - 1 - it.tile) * QT;
    const long long row0 = it.start;
    const int g = h / (H / G);
    q += row0 * ldq + (long long)h * DH;
    k += row0 * ldk + (long long)g * DH;
    v += row0 * ldv + (long long)g * DV;

    const int i_last = min(i0 + QT, L) - 1;
    const int lo = window > 0 ? max(n_meta, i0 - window + 1) : n_meta;
    // key tiles: the meta range, then the window's; first key j0 of the range's `end`
    int range = 0, j0 = 0, end = min(n_meta, i_last + 1);
    auto settle = [&] {  // to the window's range when the meta range is done; false: no tile is left
        if (range == 0 && j0 >= end) {
            range = 1;
            j0 = lo;
            end = i_last + 1;
        }
        return j0 < end;
    };
    for (int j = tid; j < QT * (DH / 8); j += NT) {
        const int r = j % QT, c = j / QT;
        float x[8];
        ragged::load8(q + (long long)min(i0 + r, L - 1) * ldq + 8 * c, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) sm.q[8 * c + e][r] = x[e] * scale_log2;
    }
    float2 acc[RT][DV / 32];
    float mrun[RT], l[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        mrun[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int c = 0; c < DV / 32; ++c) acc[r][c] = make_float2(0.f, 0.f);
    }
    // this thread's pieces of a tile's K (8 values of one row each) and V: all loads in flight at once
    // (a loop of load and store: 61 us against 54 for 4 prompts of up to 3000 rows)
    constexpr int NKP = KT * (DH / 8) / NT, NVP = KT * (DV / 8) / NT;
    while (settle()) {
        float kx[NKP][8], vx[NVP][8];
#pragma unroll
        for (int x = 0; x < NKP; ++x) {
            const int j = tid + x * NT, r = j % KT, c = j / KT;
#pragma unroll
            for (int e = 0; e < 8; ++e) kx[x][e] = 0.f;
            if (j0 + r < end) ragged::load8(k + (long long)(j0 + r) * ldk + 8 * c, kx[x]);
        }
#pragma unroll
        for (int x = 0; x < NVP; ++x) {
            const int j = tid + x * NT, c = j % (DV / 8), r = j / (DV / 8);
#pragma unroll
            for (int e = 0; e < 8; ++e) vx[x][e] = 0.f;
            if (j0 + r < end) ragged::load8(v + (long long)(j0 + r) * ldv + 8 * c, vx[x]);
        }
        __syncthreads();
        int odd = 0;  // a value of V that is not finite: the product may not meet it where it is masked
#pragma unroll
        for (int x = 0; x < NKP; ++x) {
            const int j = tid + x * NT, r = j % KT, c = j / KT;
#pragma unroll
            for (int e = 0; e < 8; ++e) sm.k[8 * c + e][r] = kx[x][e];
        }
#pragma unroll
        for (int x = 0; x < NVP; ++x) {
            const int j = tid + x * NT, c = j % (DV / 8), r = j / (DV / 8);
#pragma unroll
            for (int e = 0; e < 8; ++e) odd |= !isfinite(vx[x][e]);
            *reinterpret_cast<float4*>(&sm.v[r][8 * c]) = make_float4(vx[x][0], vx[x][1], vx[x][2], vx[x][3]);
            *reinterpret_cast<float4*>(&sm.v[r][8 * c + 4]) = make_float4(vx[x][4], vx[x][5], vx[x][6], vx[x][7]);
        }
        odd = __syncthreads_or(odd);
        const int at = j0, to = end;
        const bool meta = range == 0;
        j0 += KT;
        float2 s2[RT][2];
#pragma unroll
        for (int r = 0; r < RT; ++r) s2[r][0] = s2[r][1] = make_float2(0.f, 0.f);
#pragma unroll 16
        for (int d = 0; d < DH; ++d) {
            float av[RT];
            row_values<RT>(&sm.q[d][RT * ty], av);
            const float4 b = *reinterpret_cast<const float4*>(&sm.k[d][4 * tx]);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const float2 a2 = make_float2(av[r], av[r]);
                s2[r][0] = __ffma2_rn(a2, make_float2(b.x, b.y), s2[r][0]);
                s2[r][1] = __ffma2_rn(a2, make_float2(b.z, b.w), s2[r][1]);
            }
        }
        float s[RT][4];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            s[r][0] = s2[r][0].x;
            s[r][1] = s2[r][0].y;
            s[r][2] = s2[r][1].x;
            s[r][3] = s2[r][1].y;
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int i = i0 + RT * ty + r;
            float mx = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int j = at + 4 * tx + c;
                const bool see = j < to && j <= i && (meta || window <= 0 || i - j < window);
                s[r][c] = see ? s[r][c] : -INFINITY;
                mx = fmaxf(mx, s[r][c]);
            }
#pragma unroll
            for (int w = 1; w < 16; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            const float m = fmaxf(mrun[r], mx), mu = m == -INFINITY ? 0.f : m;
            const float f = exp2f(mrun[r] - mu);
            mrun[r] = m;
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                s[r][c] = exp2f(s[r][c] - mu);
                sum += s[r][c];
            }
            l[r] = l[r] * f + sum;  // this thread's columns; the 16 threads of the row are added at the end
#pragma unroll
            for (int c = 0; c < DV / 32; ++c) acc[r][c] = __fmul2_rn(acc[r][c], make_float2(f, f));
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int r = 0; r < RT; ++r) sm.p[4 * tx + c][RT * ty + r] = s[r][c];
        __syncthreads();
        const int nk = min(KT, to - at);
        auto add = [&](int j, bool all) {
            float av[RT];
            row_values<RT>(&sm.p[j][RT * ty], av);
#pragma unroll
            for (int u = 0; u < DV / 64; ++u) {
                const float4 b = *reinterpret_cast<const float4*>(&sm.v[j][4 * tx + 64 * u]);
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const int i = i0 + RT * ty + r, jj = at + j;
                    if (!all && !(jj <= i && (meta || window <= 0 || i - jj < window))) continue;
                    const float2 a2 = make_float2(av[r], av[r]);
                    acc[r][2 * u] = __ffma2_rn(a2, make_float2(b.x, b.y), acc[r][2 * u]);
                    acc[r][2 * u + 1] = __ffma2_rn(a2, make_float2(b.z, b.w), acc[r][2 * u + 1]);
                }
            }
        };
        if (odd) {
            for (int j = 0; j < nk; ++j) add(j, false);
        } else {
            // (rows of V behind the tile's last key are zero, and so are their weights)
            const int n8 = (nk + 7) & ~7;
#pragma unroll 1
            for (int j = 0; j < n8; j += 8)
#pragma unroll
                for (int x = 0; x < 8; ++x) add(j + x, true);
        }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int i = i0 + RT * ty + r;
        float sum = l[r];
#pragma unroll
        for (int w = 1; w < 16; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
        // (a NaN sum divides: a visible NaN reaches its row; without a score above -infinity the row is
        // zero, whatever V holds)
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        if (sum == 0.f)
#pragma unroll
            for (int c = 0; c < DV / 32; ++c) acc[r][c] = make_float2(0.f, 0.f);
        if (i < L) {
            T* dst = o + (row0 + i) * ldo + (long long)h * DV + 4 * tx;
#pragma unroll
            for (int u = 0; u < DV / 64; ++u)
                ragged::store4(dst + 64 * u, acc[r][2 * u].x * inv, acc[r][2 * u].y * inv, acc[r][2 * u + 1].x * inv,
                               acc[r][2 * u + 1].y * inv);
        }
    }
}

template <typename T, int DH, int DV, int QT>
int launch_tile(const Ctx& ctx, const PackedAttn& a) {
    auto kern = attn_packed_simt_kernel<T, DH, DV, QT>;
    const size_t smem = sizeof(PackedSimtSmem<DH, DV, QT>);
    static std::atomic<unsigned long long> smem_set{0};
    if (!smem_opt_in_once(smem_set, kern, smem, ctx)) return HYMBA_ERR_CUDA;
    const long long blocks = ((long long)ceil_div(a.total, QT) + a.n_seqs) * a.H;
    if (blocks > 0x7fffffffLL) return HYMBA_ERR_UNSUPPORTED;
    HYMBA_LAUNCH(ctx, "attn_packed", kern, (unsigned)blocks, NT, smem, static_cast<const T*>(a.q), a.ldq,
                 static_cast<const T*>(a.k), a.ldk, static_cast<const T*>(a.v), a.ldv, a.cu, a.n_seqs, a.total,
                 static_cast<T*>(a.o), a.ldo, a.H, a.G, a.n_meta, a.window, a.scale * 1.4426950408889634f, ctx.status);
    return HYMBA_OK;
}

// The smallest tile whose blocks still fit one wave of the 148 SMs (a block's time is a chain of
// key tiles, shorter with fewer rows), 64 rows where none does. 4 heads of 64 x 128: prompts of
// 272 and 141 rows 14.1 us in tiles of 16, 16.6 in 32, 20.5 in 64; one of 700 rows 23.8 in 16 (a
// second wave), 16.7 in 32, 20.6 in 64; two of up to 1000 38.4 in 32, 20.7 in 64.
template <typename T, int DH, int DV>
int launch_dims(const Ctx& ctx, const PackedAttn& a) {
    auto blocks = [&](int qt) { return ((long long)ceil_div(a.total, qt) + a.n_seqs) * a.H; };
    if (blocks(16) <= 148) return launch_tile<T, DH, DV, 16>(ctx, a);
    if (blocks(32) <= 148) return launch_tile<T, DH, DV, 32>(ctx, a);
    return launch_tile<T, DH, DV, 64>(ctx, a);
}

}  // namespace

template <typename T>
int launch_attn_packed_simt(const Ctx& ctx, const PackedAttn& a) {
    if (a.dh == 64 && a.dv == 64) return launch_dims<T, 64, 64>(ctx, a);
    if (a.dh == 64 && a.dv == 128) return launch_dims<T, 64, 128>(ctx, a);
    if (a.dh == 128 && a.dv == 64) return launch_dims<T, 128, 64>(ctx, a);
    if (a.dh == 128 && a.dv == 128) return launch_dims<T, 128, 128>(ctx, a);
    return HYMBA_ERR_UNSUPPORTED;
}

template int launch_attn_packed_simt<float>(const Ctx&, const PackedAttn&);

}  // namespace hymba
