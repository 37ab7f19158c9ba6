// Causal attention over packed prompts on the tcgen05 tensor cores (16-bit rows):
// softmax(scale q k^T) v with grouped heads, meta prefix + window or the whole history,
// counted from each sequence's first row ("Jamba: Hybrid SSM-Transformer", section 1;
// "Hymba Guide", Learnable Meta-Tokens; 51cto Hymba-1.5B article, section 2).
//
// One CTA per (256 query rows of a sequence, head): two 128-row tiles that share every K
// and V block of 128 keys and run as two pipelines, so that the tensor cores work on one
// tile while the other tile's softmax runs. 12 warps:
//   warp 0      one lane: TMA of the two Q tiles and of the K and V blocks (rings);
//   warps 1, 2  one thread each that issues the products of tile A, B in steps of 64 keys: O_t
//               += P_t V once the softmax stored P_t over its scores in TMEM, then, that product
//               done, the scores S_t = Q_t K^T two steps on into the same columns. The other half
//               of the tile's columns holds the step between, so that the softmax goes from
//               step to step without waiting for a product. (One thread for both tiles could
//               not issue as fast as the softmax went: 969 us for the three prompts below.)
//   warp 3      looks at the V blocks that hold keys some row does not see: rows behind
//               the sequence become zero (they belong to another sequence, and 0 x NaN
//               would reach the product), and a value that is not finite is replaced by 0
//               and noted;
//   warps 4-7   softmax of tile A, warps 8-11 of tile B: one thread per query row. P =
//               2^(s - m) as 16-bit pairs, the row sum of the fp32 values; O is rescaled in
//               TMEM only when the running max grows by more than 2^4 (fp16) or 2^8 (bf16).
// A CTA that noted a value that is not finite computes its rows once more from global
// memory, key by key over what each row sees. A row whose sums are not finite though its weights are
// looks through the V that it sees: an infinity times a weight that rounds to 0 in 16 bits was NaN.
// P is rounded to the rows' type, as an MMA operand has to be: half a step relative to each
// weight, the size of the output's own rounding. fp16 has little range: m is the running max less
// 11, so that P lies between 2^11 and 2^15 at the largest weight and keeps all its bits down to
// 2^-25 of it (below, half of fp16's smallest step: 2^-36 of it); the factor leaves with the row sum.
// Bound by the tensor cores (2 (dh + dv) flops per visible pair); what is left is the softmax's
// latency, about 1500 clocks per 64 keys and tile: two warps per scheduler do not cover their own
// waits (XU pipe 61 %, issue slots 43 %, tensor pipe 46 % busy), and in windows a block's start and
// end, about 10,000 clocks. 25 heads of 64 x 128:
// three prompts of up to 8320 rows, whole history (bf16), 840 us, 53% of the bf16 rate; eight of up
// to 4224, window 1024 and 128 meta tokens (f16), 282 us, 39%. Part of the exponentials as
// polynomials on the FMA pipe: 869 us for a quarter of them, 910 for half, 829 then for none.
#include "attn_tile.cuh"
#include "kernels.h"
#include "ragged.cuh"

namespace hymba {

namespace {

constexpr int QT = 128, KB = 128;
constexpr int KS = 64;  // keys per softmax step: half a block
constexpr int NT = 384;
constexpr int REG_SOFT = 216, REG_OTHER = 64;
// the launch allocates 168 registers per thread (65536 / 384, rounded down to 8): the
// split must fit that pool (the launcher also checks the compiled count)
static_assert(4 * 32 * REG_OTHER + 8 * 32 * REG_SOFT <= NT * 168, "register split exceeds the launch's pool");
// m is the running max (log2 units) less LOW; it moves when a score passes it by more than TOP.
// fp16: 2^15 is the largest power of two there is; bf16 has fp32's range
template <typename T>
struct Weights {
    static constexpr float LOW = std::is_same<T, bf16>::value ? 0.f : 11.f;
    static constexpr float TOP = std::is_same<T, bf16>::value ? 8.f : 15.f;
};
// TMEM columns: O_A [0,128), O_B [128,256), S_A [256,384), S_B [384,512). S_t holds two steps of
// 64 keys, 64 columns each; a step's P lies in the first 32 of its columns (two 16-bit keys each)
constexpr uint32_t TM_O = 0, TM_S = 256;

// Ring depth: three stages of K and V where the Q/K dim leaves room for them, else two.
constexpr int stages(int dh) { return dh == 64 ? 3 : 2; }

template <int DH, int DV>
struct PackedSmem {
    static constexpr int ST = stages(DH);
    alignas(1024) uint8_t q[2][DH / 64][QT * 128];
    alignas(1024) uint8_t k[ST][DH / 64][KB * 128];
    alignas(1024) uint8_t v[ST][DV / 64][KB * 128];
    uint64_t q_full;
    uint64_t k_full[ST], k_empty[ST];
    uint64_t v_full[ST], v_ok[ST], v_empty[ST];
    uint64_t s_full[2][2], p_full[2][2], pv_done[2], o_done[2];
    uint32_t tmem_base;
    int abort, dirty;
    ragged::FindSmem find;
};

// Key blocks of a tile pair (tile t: rows i0 + 128 t ..): nmb meta blocks of 128 keys from 0,
// then window blocks of 128 keys from the pair's lowest window key. Each tile uses the
// first mc meta blocks and the window blocks ws .. ws + wn - 1 (block indexes).
struct Use {
    int meta_end, lo, hi;  // visible to some row of the tile: [0, meta_end) and [lo, hi)
    int mc, ws, wn;
    __device__ void span(int i0, int L, int n_meta, int window) {
        const int last = min(i0 + QT, L) - 1;
        const bool valid = i0 < L;
        meta_end = valid ? min(n_meta, last + 1) : 0;
        lo = window > 0 ? max(n_meta, i0 - window + 1) : n_meta;
        hi = valid ? max(last + 1, lo) : lo;
    }
    __device__ void place(int nmb, int lo0) {
        mc = (meta_end + KB - 1) / KB;
        const int first = (lo - lo0) / KB;
        ws = nmb + first;
        wn = hi > lo ? (hi - lo0 + KB - 1) / KB - first : 0;
    }
    __device__ int count() const { return mc + wn; }
    // the u-th block of the tile
    __device__ int nth(int u) const { return u < mc ? u : ws + (u - mc); }
};
struct Blocks {
    int nmb, lo, n;
    Use A, B;
    __device__ void init(int i0, int L, int n_meta, int window) {
        A.span(i0, L, n_meta, window);
        B.span(i0 + QT, L, n_meta, window);
        nmb = (max(A.meta_end, B.meta_end) + KB - 1) / KB;
        lo = A.lo;
        const int hi = max(A.hi, B.hi);
        n = nmb + (hi > lo ? (hi - lo + KB - 1) / KB : 0);
        A.place(nmb, lo);
        B.place(nmb, lo);
    }
    __device__ int key0(int j) const { return j < nmb ? j * KB : lo + (j - nmb) * KB; }
};

__device__ __forceinline__ void fail(volatile int* abort, int* status, int role, int step, int bar) {
    *abort = 1;
    tc::record_timeout(status, role, step, bar);
}

template <bool BF16>
__device__ __forceinline__ uint32_t drop_odd(uint32_t w) {
    constexpr uint32_t E = BF16 ? 0x7f807f80u : 0x7c007c00u;
    return w & ~__vcmpeq2(w & E, E);
}

// One row from global memory over exactly the keys it sees, with the row's m and sum.
template <typename T, int DH, int DV>
__device__ __noinline__ void recompute_row(const T* q, const T* k, long long ldk, const T* v, long long ldv, T* o, int i,
                                           int n_meta, int window, float scale, float mu, float inv) {
    const int meta_e = min(n_meta, i + 1), wa = window > 0 ? max(n_meta, i - window + 1) : n_meta;
#pragma unroll 1
    for (int c0 = 0; c0 < DV; c0 += 16) {
        float acc[16] = {};
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
#pragma unroll 1
            for (int j = part ? wa : 0; j < (part ? i + 1 : meta_e); ++j) {
                float s = 0.f;
#pragma unroll 1
                for (int d = 0; d < DH; d += 8) {
                    float x[8], y[8];
                    ragged::load8(q + d, x);
                    ragged::load8(k + j * ldk + d, y);
#pragma unroll
                    for (int e = 0; e < 8; ++e) s = fmaf(x[e], y[e], s);
                }
                const float p = fast_exp2(fmaf(s, scale, -mu));
#pragma unroll
                for (int e = 0; e < 16; e += 8) {
                    float y[8];
                    ragged::load8(v + j * ldv + c0 + e, y);
#pragma unroll
                    for (int x = 0; x < 8; ++x) acc[e + x] = fmaf(p, y[x], acc[e + x]);
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) o[c0 + e] = from_f<T>(inv == 0.f ? 0.f : acc[e] * inv);
    }
}

// The columns of one row where V holds infinities that it sees: weights of finite scores are above 0, so
// their sum is what the infinities add up to. `none`: no score above -infinity, the row is zero.
template <typename T, int DV>
__device__ __noinline__ void infinite_columns(const T* v, long long ldv, T* o, int i, int n_meta, int window, bool none) {
    const int meta_e = min(n_meta, i + 1), wa = window > 0 ? max(n_meta, i - window + 1) : n_meta;
#pragma unroll 1
    for (int c0 = 0; c0 < DV; c0 += 8) {
        float acc[8] = {};
        bool numbers = !none;  // a column is not NaN yet
#pragma unroll 1
        for (int part = 0; part < 2; ++part)
#pragma unroll 1
            for (int j = part ? wa : 0; numbers && j < (part ? i + 1 : meta_e); ++j) {
                float y[8];
                ragged::load8(v + j * ldv + c0, y);
                numbers = false;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    acc[e] += isfinite(y[e]) ? 0.f : y[e];
                    numbers |= acc[e] == acc[e];
                }
            }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (none || acc[e] != 0.f) o[c0 + e] = from_f<T>(acc[e]);
    }
}

template <typename T, int DH, int DV>
__global__ void __launch_bounds__(NT, 1)
attn_packed_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const PackedAttn a, float scale, int* status) {
    constexpr bool BF16 = std::is_same<T, bf16>::value;
    constexpr int ST = stages(DH);
    extern __shared__ uint8_t smem_raw[];
    PackedSmem<DH, DV>& s = *reinterpret_cast<PackedSmem<DH, DV>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                                 ~static_cast<uintptr_t>(1023));
    constexpr uint32_t IDESC_S = tc::idesc_f16(BF16, QT, KS);
    constexpr uint32_t IDESC_PV = tc::idesc_f16(BF16, QT, DV, true);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        tc::mbar_init(&s.q_full, 1);
        for (int i = 0; i < ST; ++i) {
            tc::mbar_init(&s.k_full[i], 1);
            tc::mbar_init(&s.k_empty[i], 2);  // the two tiles
            tc::mbar_init(&s.v_full[i], 1);
            tc::mbar_init(&s.v_ok[i], 32);
            tc::mbar_init(&s.v_empty[i], 2);
        }
        for (int t = 0; t < 2; ++t) {
            for (int x = 0; x < 2; ++x) {
                tc::mbar_init(&s.s_full[t][x], 1);
                tc::mbar_init(&s.p_full[t][x], QT);
            }
            tc::mbar_init(&s.pv_done[t], 1);
            tc::mbar_init(&s.o_done[t], 1);
        }
        s.abort = 0;
        s.dirty = 0;
        tc::fence_mbar_init();
        tc::prefetch_tmap(&tmQ);
        tc::prefetch_tmap(&tmK);
        tc::prefetch_tmap(&tmV);
    }
    // setup above touches no global memory; everything below may read the previous
    // kernel's output
    griddep_sync();
    const ragged::Item it = ragged::find_item<NT>(s.find, a.cu, a.n_seqs, a.total, 2 * QT, blockIdx.x / a.H, status);
    if (it.seq < 0) return;
    const int L = it.len;
    const int i0 = ((L + 2 * QT - 1) / (2 * QT) - 1 - it.tile) * 2 * QT;  // the heaviest rows first
    const int h = blockIdx.x % a.H, g = h / (a.H / a.G);
    const int n_meta = a.n_meta, window = a.window;
    Blocks blk;
    blk.init(i0, L, n_meta, window);
    const int nblk = blk.n;
    if (threadIdx.x == 0 && nblk > 0) {
        // (the thread that initialised the barriers; Q and the first K are on their way while TMEM is
        // allocated)
        tc::mbar_arrive_expect_tx(&s.q_full, 2 * QT * DH * 2);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int p = 0; p < DH / 64; ++p)
                tc::tma_load_2d(s.q[t][p], &tmQ, &s.q_full, h * DH + p * 64, it.start + i0 + t * QT);
        tc::mbar_arrive_expect_tx(&s.k_full[0], KB * DH * 2);
#pragma unroll
        for (int p = 0; p < DH / 64; ++p) tc::tma_load_2d(s.k[0][p], &tmK, &s.k_full[0], g * DH + p * 64, it.start + blk.key0(0));
    }
    if (warp == 1) {
        tc::tmem_alloc(&s.tmem_base, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = s.tmem_base;
    volatile int* abort = &s.abort;
    const long long wlim = tc::wait_limit(status);
    int zero = 0;

    if (warp < 4) {
        setmaxnreg_dec<REG_OTHER>();
        if (warp == 0) {
            // ---------------- TMA ----------------
            if (lane == 0) {
                int k_issued = 0, v_issued = 0;
                for (int j = 0; j < nblk; ++j) {
                    const int st = j % ST, key = it.start + blk.key0(j);
                    if (!tc::mbar_wait(&s.k_empty[st], ((j / ST) & 1) ^ 1, abort, wlim)) { fail(abort, status, 0, j, 1); break; }
                    if (j > 0) {
                        tc::mbar_arrive_expect_tx(&s.k_full[st], KB * DH * 2);
#pragma unroll
                        for (int p = 0; p < DH / 64; ++p)
                            tc::tma_load_2d(s.k[st][p], &tmK, &s.k_full[st], g * DH + p * 64, key);
                    }
                    k_issued = j + 1;
                    if (!tc::mbar_wait(&s.v_empty[st], ((j / ST) & 1) ^ 1, abort, wlim)) { fail(abort, status, 0, j, 9); break; }
                    tc::mbar_arrive_expect_tx(&s.v_full[st], KB * DV * 2);
#pragma unroll
                    for (int p = 0; p < DV / 64; ++p)
                        tc::tma_load_2d(s.v[st][p], &tmV, &s.v_full[st], g * DV + p * 64, key);
                    v_issued = j + 1;
                }
                // every copy issued has landed before the block exits
                tc::mbar_wait(&s.q_full, 0, &zero);
                for (int j = max(0, k_issued - ST); j < k_issued; ++j) tc::mbar_wait(&s.k_full[j % ST], (j / ST) & 1, &zero);
                for (int j = max(0, v_issued - ST); j < v_issued; ++j) tc::mbar_wait(&s.v_full[j % ST], (j / ST) & 1, &zero);
            }
        } else if (warp < 3) {
            // ---------------- MMA issuer of tile t ----------------
            if (tc::elect_one()) {
                const int t = warp - 1;
                const Use use = t ? blk.B : blk.A;
                const int n = 2 * use.count();  // steps of 64 keys
                bool ok = true;
                auto wait = [&](uint64_t* bar, uint32_t ph, int k, int id) {
                    if (ok && !tc::mbar_wait(bar, ph, abort, wlim)) {
                        fail(abort, status, 1, k, id);
                        ok = false;
                    }
                };
                const uint64_t qd = tc::sdesc_k_sw128(tc::smem_u32(s.q[t][0])), kd = tc::sdesc_k_sw128(tc::smem_u32(s.k[0][0]));
                const uint64_t vd = tc::sdesc_mn_sw128(tc::smem_u32(s.v[0][0]), KB * 128);
                const uint32_t sd = tmem + TM_S + t * 128, od = tmem + TM_O + t * 128;
                // Both tiles take part in every phase of the rings, so that neither can be a phase
                // ahead or behind: a block that the tile does not use is waited for and released.
                int jk = 0, jv = 0;
                auto pass_k = [&](int to) {
                    for (; ok && jk < to; ++jk) {
                        wait(&s.k_full[jk % ST], (jk / ST) & 1, jk, 2);
                        tc::mbar_arrive(&s.k_empty[jk % ST]);
                    }
                };
                auto pass_v = [&](int to) {
                    for (; ok && jv < to; ++jv) {
                        wait(&s.v_ok[jv % ST], (jv / ST) & 1, jv, 10);
                        tc::mbar_arrive(&s.v_empty[jv % ST]);
                    }
                };
                // step k: half k % 2 of the tile's block k / 2; its scores, and P over them, in half k % 2
                // of the tile's S columns.
                // S_t(k) = Q_t K^T; the second half frees the K stage
                auto issue_s = [&](int k) {
                    const int j = use.nth(k >> 1), st = j % ST, x = k & 1;
                    if (x == 0) {
                        pass_k(j);
                        wait(&s.k_full[st], (j / ST) & 1, j, 2);
                        jk = j + 1;
                    }
                    if (!ok) return;
                    tc::tc_fence_after();
                    const uint64_t kx = kd + (uint64_t)(st * (DH / 64) * (KB * 128 / 16) + x * (KS * 128 / 16));
#pragma unroll
                    for (int p = 0; p < DH / 64; ++p)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc::mma_f16_ss(sd + x * KS, qd + p * (QT * 128 / 16) + kk * 2, kx + p * (KB * 128 / 16) + kk * 2,
                                           IDESC_S, p > 0 || kk > 0);
                    tc::mma_commit(&s.s_full[t][x]);
                    if (x) tc::mma_commit(&s.k_empty[st]);
                };
                wait(&s.q_full, 0, 0, 0);
                for (int k = 0; k < min(n, 2); ++k) issue_s(k);
                for (int k = 0; ok && k < n; ++k) {
                    // O_t += P_t V, P_t read from TMEM
                    const int j = use.nth(k >> 1), st = j % ST, x = k & 1;
                    if (x == 0) {
                        pass_v(j);
                        wait(&s.v_ok[st], (j / ST) & 1, j, 10);
                        jv = j + 1;
                    }
                    wait(&s.p_full[t][x], (k >> 1) & 1, j, 4);
                    if (!ok) break;
                    tc::tc_fence_after();
                    const uint64_t vx = vd + (uint64_t)(st * (DV / 64) * (KB * 128 / 16) + x * (KS * 128 / 16));
#pragma unroll
                    for (int kk = 0; kk < KS / 16; ++kk)
                        mma_f16_ts(od, sd + x * KS + kk * 8, vx + kk * (2048 / 16), IDESC_PV, k > 0 || kk > 0);
                    tc::mma_commit(&s.pv_done[t]);
                    if (x) tc::mma_commit(&s.v_empty[st]);
                    // the scores two steps on take the columns of this P
                    if (k + 2 < n) {
                        wait(&s.pv_done[t], k & 1, k, 11);
                        if (ok) issue_s(k + 2);
                    }
                }
                // (block by block: the loads of K and V take turns)
                for (int j = jv; ok && j < nblk; ++j) {
                    pass_k(j + 1);
                    pass_v(j + 1);
                }
                // every MMA issued has completed: the tile's O is whole, and the block may exit
                tc::mma_commit(&s.o_done[t]);
                tc::mbar_wait(&s.o_done[t], 0, &zero);
            }
        } else {
            // ---------------- V blocks with keys that some row does not see ----------------
            const int last = min(i0 + 2 * QT, L) - 1;
            for (int j = 0; j < nblk; ++j) {
                const int st = j % ST;
                if (!__all_sync(0xffffffffu, tc::mbar_wait(&s.v_full[st], (j / ST) & 1, abort, wlim))) {
                    if (lane == 0) fail(abort, status, 0, j, 12);
                    break;
                }
                const int k0 = blk.key0(j);
                // every row of the pair sees keys k0 .. k0 + 127
                const bool whole = j < blk.nmb ? k0 + KB <= min(n_meta, i0 + 1)
                                               : k0 + KB <= i0 + 1 && (window <= 0 || last - k0 < window);
                if (!whole) {
                    // 16-byte piece x of panel p: row x / 8 (the swizzle moves pieces within a row)
                    uint4* vb = reinterpret_cast<uint4*>(s.v[st][0]);
                    constexpr int PIECES = KB * 8 * (DV / 64);
                    if (k0 + KB > L)
                        for (int x = lane; x < PIECES; x += 32)
                            if (k0 + ((x >> 3) & (KB - 1)) >= L) vb[x] = make_uint4(0, 0, 0, 0);
                    if (__any_sync(0xffffffffu, ragged::any_odd<BF16, PIECES>(vb, lane))) {
                        for (int x = lane; x < PIECES; x += 32) {
                            uint4 w = vb[x];
                            w.x = drop_odd<BF16>(w.x);
                            w.y = drop_odd<BF16>(w.y);
                            w.z = drop_odd<BF16>(w.z);
                            w.w = drop_odd<BF16>(w.w);
                            vb[x] = w;
                        }
                        if (lane == 0) *reinterpret_cast<volatile int*>(&s.dirty) = 1;
                    }
                    tc::fence_proxy_async_smem();
                }
                tc::mbar_arrive(&s.v_ok[st]);
            }
        }
    } else {
        setmaxnreg_inc<REG_SOFT>();
        // ---------------- softmax + output: tile t, TMEM lane quadrant q ----------------
        const int t = (warp - 4) >> 2, q = warp & 3;
        const int i = i0 + t * QT + q * 32 + lane;
        const uint32_t lane_base = (uint32_t)(q * 32) << 16;
        const uint32_t s_cols = tmem + lane_base + TM_S + t * 128;
        const uint32_t o_cols = tmem + lane_base + TM_O + t * 128;
        const Use use = t ? blk.B : blk.A;
        const int nt = use.count();
        // the row's visible keys: meta [0, min(n_meta, i+1)), window [wa, i+1)
        const int meta_e = min(n_meta, i + 1);
        const int wa = window > 0 ? max(n_meta, i - window + 1) : n_meta;
        float m_used = -INFINITY, l = 0.f;
        bool ok = true;
        for (int k = 0; k < 2 * nt; ++k) {
            const int x = k & 1;
            // tcgen05.ld/st are warp-collective: every decision that guards them is taken
            // by the whole warp (__all_sync / __any_sync)
            if (!__all_sync(0xffffffffu, tc::mbar_wait(&s.s_full[t][x], (k >> 1) & 1, abort, wlim))) {
                if (lane == 0) fail(abort, status, 2, k, 5);
                ok = false;
                break;
            }
            tc::tc_fence_after();
            // the two 32-column loads in flight together, one wait
            uint32_t sr[2][32];
#pragma unroll
            for (int c = 0; c < 2; ++c) tc::tmem_ld32(s_cols + x * KS + c * 32, sr[c]);
            tc::tmem_wait_ld();
            float* sv = reinterpret_cast<float*>(&sr[0][0]);
            // mask: the keys row i sees in this step form one interval [ka, ke)
            const int j = use.nth(k >> 1), k0 = blk.key0(j) + x * KS;
            const bool meta_blk = j < blk.nmb;
            const int ka = meta_blk ? 0 : wa;
            const int ke = meta_blk ? meta_e : i + 1;
            if (ka > k0 || ke < k0 + KS) {
                const unsigned span = ke > ka ? (unsigned)(ke - ka) : 0u;
#pragma unroll
                for (int c = 0; c < KS; ++c) sv[c] = (unsigned)(k0 + c - ka) < span ? sv[c] : -INFINITY;
            }
            // row max with three-input max: 8 independent chains over the 64 scores
            float mx8[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) mx8[c] = fmax3(sv[c], sv[c + 8], sv[c + 16]);
#pragma unroll
            for (int c = 24; c + 16 <= KS; c += 16)
#pragma unroll
                for (int y = 0; y < 8; ++y) mx8[y] = fmax3(mx8[y], sv[c + y], sv[c + 8 + y]);
#pragma unroll
            for (int y = 0; y < 8; ++y) mx8[y] = fmaxf(mx8[y], sv[KS - 8 + y]);
            const float mx = fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]),
                                   fmaxf(mx8[6], mx8[7])) * scale;
            // a row whose running max has grown too far moves to the new max, and its O is
            // scaled in TMEM, between the products of the step before and of this one
            float f = 1.f;
            bool scale_o = false;
            if (mx > m_used + Weights<T>::TOP) {
                const float to = mx - Weights<T>::LOW;
                if (m_used != -INFINITY) {
                    f = exp2f(m_used - to);
                    l *= f;
                    scale_o = true;
                }
                m_used = to;
            }
            // P = 2^(s * scale - m) in fp32, summed in fp32, stored as 16-bit pairs
            const float mu = m_used == -INFINITY ? 0.f : m_used;
            const float2 sc2 = make_float2(scale, scale), nmu2 = make_float2(-mu, -mu);
            uint32_t pk[32];
            float2 l4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int c = 0; c < KS / 2; ++c) {
                const float2 y = __ffma2_rn(make_float2(sv[2 * c], sv[2 * c + 1]), sc2, nmu2);
                const float2 p = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                l4[c & 3] = __fadd2_rn(l4[c & 3], p);
                pk[c] = pack2<T>(p.x, p.y);
            }
            const float2 l2 = __fadd2_rn(__fadd2_rn(l4[0], l4[1]), __fadd2_rn(l4[2], l4[3]));
            l += l2.x + l2.y;
            tc::tmem_st32(s_cols + x * KS, pk);
            tc::tmem_wait_st();
            if (__any_sync(0xffffffffu, scale_o)) {
                // (the product of this step waits for this thread; that of the step before may still run)
                if (!__all_sync(0xffffffffu, tc::mbar_wait(&s.pv_done[t], (k - 1) & 1, abort, wlim))) {
                    if (lane == 0) fail(abort, status, 2, k, 6);
                    ok = false;
                    break;
                }
                tc::tc_fence_after();
#pragma unroll
                for (int c = 0; c < DV / 32; ++c) {
                    uint32_t rr[32];
                    tc::tmem_ld32(o_cols + c * 32, rr);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int y = 0; y < 32; ++y) rr[y] = __float_as_uint(__uint_as_float(rr[y]) * f);
                    tc::tmem_st32(o_cols + c * 32, rr);
                }
                tc::tmem_wait_st();
            }
            tc::tc_fence_before();
            tc::mbar_arrive(&s.p_full[t][x]);
        }
        if (ok && nt > 0 && __all_sync(0xffffffffu, tc::mbar_wait(&s.o_done[t], 0, abort, wlim))) {
            tc::tc_fence_after();
            // no visible score above -infinity: zeros, whatever V holds; a NaN sum divides, so that a
            // visible NaN reaches its row
            const float inv = l == 0.f ? 0.f : 1.f / l;
            T* orow = static_cast<T*>(a.o) + (it.start + (long long)i) * a.ldo + (long long)h * DV;
            // 64 columns at a time through the tile's Q (no longer needed): the warp's 32 rows there,
            // then whole 128-byte pieces of rows out
            uint8_t* mid = s.q[t][0] + q * 4096;
            T* out = orow - (long long)lane * a.ldo;  // the warp's first row
            const int n = L - i + lane;               // rows from there to the sequence's end
            float odd = 0.f;                          // NaN once a sum of the row is not finite
#pragma unroll 1
            for (int v0 = 0; v0 < DV; v0 += 64) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t rr[32];
                    tc::tmem_ld32(o_cols + v0 + c * 32, rr);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int x = 0; x < 32; ++x) odd = fmaf(__uint_as_float(rr[x]), 0.f, odd);
#pragma unroll
                    for (int x = 0; x < 32; x += 8) {
                        uint4 pk;
                        pk.x = pack2<T>(__uint_as_float(rr[x]) * inv, __uint_as_float(rr[x + 1]) * inv);
                        pk.y = pack2<T>(__uint_as_float(rr[x + 2]) * inv, __uint_as_float(rr[x + 3]) * inv);
                        pk.z = pack2<T>(__uint_as_float(rr[x + 4]) * inv, __uint_as_float(rr[x + 5]) * inv);
                        pk.w = pack2<T>(__uint_as_float(rr[x + 6]) * inv, __uint_as_float(rr[x + 7]) * inv);
                        *reinterpret_cast<uint4*>(mid + lane * 128 + (((4 * c + (x >> 3)) ^ (lane & 7)) * 16)) = pk;
                    }
                }
                __syncwarp();
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const int row = 4 * x + (lane >> 3), e = lane & 7;
                    const uint4 w = *reinterpret_cast<const uint4*>(mid + row * 128 + ((e ^ (row & 7)) * 16));
                    if (row < n) *reinterpret_cast<uint4*>(out + row * a.ldo + v0 + 8 * e) = w;
                }
                __syncwarp();
            }
            if (i < L && *reinterpret_cast<volatile int*>(&s.dirty))
                recompute_row<T, DH, DV>(static_cast<const T*>(a.q) + (it.start + (long long)i) * a.ldq + (long long)h * DH,
                                         static_cast<const T*>(a.k) + it.start * a.ldk + (long long)g * DH, a.ldk,
                                         static_cast<const T*>(a.v) + it.start * a.ldv + (long long)g * DV, a.ldv, orow, i,
                                         n_meta, window, scale, m_used == -INFINITY ? 0.f : m_used, inv);
            else if (i < L && !(odd == 0.f) && l - l == 0.f)
                infinite_columns<T, DV>(static_cast<const T*>(a.v) + it.start * a.ldv + (long long)g * DV, a.ldv, orow, i,
                                        n_meta, window, l == 0.f);
        } else if (ok && nt > 0) {
            if (lane == 0) fail(abort, status, 2, nt, 8);
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <typename T, int DH, int DV>
int launch_dims(const Ctx& ctx, const PackedAttn& a) {
    constexpr bool BF16 = std::is_same<T, bf16>::value;
    CUtensorMap tq, tk, tv;
    if (!tc::make_tmap_2d(&tq, a.q, BF16, a.total, (uint64_t)a.H * DH, a.ldq, QT) ||
        !tc::make_tmap_2d(&tk, a.k, BF16, a.total, (uint64_t)a.G * DH, a.ldk, KB) ||
        !tc::make_tmap_2d(&tv, a.v, BF16, a.total, (uint64_t)a.G * DV, a.ldv, KB))
        return HYMBA_ERR_UNSUPPORTED;
    auto kern = attn_packed_tc_kernel<T, DH, DV>;
    const size_t smem = sizeof(PackedSmem<DH, DV>) + 1024;
    static std::atomic<unsigned long long> smem_set{0};
    if (!smem_opt_in_once(smem_set, kern, smem, ctx)) return HYMBA_ERR_CUDA;
    // the warpgroups' register split (setmaxnreg) must fit the registers the block is
    // launched with, or the increase would wait forever: check the compiled count
    static std::atomic<int> regs{0};
    if (regs.load(std::memory_order_relaxed) == 0) {
        cudaFuncAttributes fa;
        if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return HYMBA_ERR_CUDA;
        regs.store(fa.numRegs, std::memory_order_relaxed);
    }
    if (4 * 32 * REG_OTHER + 8 * 32 * REG_SOFT > NT * regs.load(std::memory_order_relaxed)) return HYMBA_ERR_UNSUPPORTED;
    const long long blocks = ((long long)ceil_div(a.total, 2 * QT) + a.n_seqs) * a.H;
    if (blocks > 0x7fffffffLL) return HYMBA_ERR_UNSUPPORTED;
    HYMBA_LAUNCH(ctx, "attn_packed", kern, (unsigned)blocks, NT, smem, tq, tk, tv, a, a.scale * 1.4426950408889634f,
                 ctx.status);
    return HYMBA_OK;
}

}  // namespace

template <typename T>
int launch_attn_packed_tc(const Ctx& ctx, const PackedAttn& a) {
    if (a.dh == 64 && a.dv == 64) return launch_dims<T, 64, 64>(ctx, a);
    if (a.dh == 64 && a.dv == 128) return launch_dims<T, 64, 128>(ctx, a);
    if (a.dh == 128 && a.dv == 64) return launch_dims<T, 128, 64>(ctx, a);
    if (a.dh == 128 && a.dv == 128) return launch_dims<T, 128, 128>(ctx, a);
    return HYMBA_ERR_UNSUPPORTED;
}

template int launch_attn_packed_tc<f16>(const Ctx&, const PackedAttn&);
template int launch_attn_packed_tc<bf16>(const Ctx&, const PackedAttn&);

}  // namespace hymba
