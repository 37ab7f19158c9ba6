// Linear attention with a decay per head, chunked form on the tcgen05 tensor cores (16-bit
// rows, key dim 64): S_t = exp(g_t) S_{t-1} + v_t k_t^T, o_t = scale S_t q_t over packed
// prompts ("Lecture 04 - Beyond the Dense Transformer", section 3: with a scalar decay per
// head the recurrence is a masked product with a semiseparable matrix and can be computed as
// blocks of matmuls). Per chunk of 128 rows, with cs_i = g_1 + .. + g_i from the chunk's start:
//     o_i = scale (sum_{j<=i} exp(cs_i - cs_j) (q_i . k_j) v_j  +  exp(cs_i) S q_i)
//     S  <- exp(cs_128) S + sum_j exp(cs_128 - cs_j) v_j k_j^T
//
// One CTA per (64 or 128 value columns, head, sequence) walks the chunks. 16 warps:
//   warp 0      TMA of q, k, v, two chunks deep;
//   warp 1      TMEM, and one thread that issues the four products of a chunk:
//               S1 = q k^T (128 x 128 x 64), D += V^T K' (the state, values x keys, both
//               operands read across their rows), O2 = q S^T, O = P V (P from TMEM over S1);
//   warp 2      the decay tables of the next chunk from 64-bit sums;
//   warp 3      V: rows behind the sequence become zero, values that are not finite are noted;
//   warps 4-7   one thread per row i: P = mask * decay * scale * S1 as 16-bit pairs into TMEM;
//   warps 8-11  one thread per state row (value): the state from TMEM, its 16-bit copy for O2 to
//               shared memory, the decayed state back; then, one thread per row j, K' =
//               exp(cs_128 - cs_j) k_j as 16-bit parts in shared memory;
//   warps 12-15 one thread per row i: o_i = O + exp(cs_i) scale O2 to global memory.
// The longest chain is S1 -> P -> P V of one chunk after the other (S1 overwrites P); the state
// and K' of a chunk are formed under it. Loops over a row are kept rolled: the warps run
// different code, and what does not fit the instruction caches together is fetched again every
// chunk (unrolled, 3.8 of every 5 stalls were waits for instructions and a chunk took twice as long).
// Numbers: a decay between rows of different 32-row blocks is A_i B_j, both distances from
// the start of i's block and so at most 1 each (a chunk with a positive log decay forms
// 2^(a_i + b_j) instead), within a block 2^(a_i + b_j). A row that forgets everything (a decay that is 0
// in fp32) is no term of cs but a border that nothing before it passes and at which cs starts again, so
// the distances stay small after any number of them (only decays of 2^-100 and less that are not 0, row
// after row, leave the others of their block right to 2^-11, a step of P). K' enters as three parts (bf16: 24 bits) or two
// (fp16: 22 bits, or 2^-37 of the chunk's largest weighted key where that is more); P and the state's
// copy are rounded to the rows' type, like any MMA operand. fp16 has little range: P's rows, the copy's rows and
// K' are brought to the middle of it by powers of two that the fp32 values give back (the
// state in TMEM carries K's power, changed together with its decay).
// Few long sequences are cut into segments of whole chunks (`segment_rows`): the same kernel first
// forms what each segment adds to a state of zero, a small one turns these into the state before
// each segment, and the segments then run side by side.
// A CTA that noted a value of V that is not finite, or an infinity in a row of K that the state takes
// up, computes its rows once more by the recurrence, in which nothing reaches a row that does not see it
// and an infinity stays one (its parts would be infinity minus infinity).
// Bound: HBM (q, k, v read and o written once per 128 value columns); what is left is the chain of a
// chunk, about 6900 clocks, and the last sequences' chunks alone. Eight prompts of up to 4224 rows
// (19800 in all), 25 heads of 64 x 128, bf16: 124 us, 49% of the copy rate.
#include <algorithm>

#include "attn_tile.cuh"
#include "kernels.h"
#include "ragged.cuh"

namespace hymba {

namespace {

using ragged::fade;
using ragged::inverse;
using ragged::to_middle;

constexpr int CQ = 128;  // rows per chunk
constexpr int DK = 64;
constexpr int NT = 512;
constexpr int NTAB = 2;  // chunks whose tables are kept
constexpr int TILE = CQ * 128;  // bytes of 128 rows x 64 16-bit columns
// TMEM columns: S1 / P, O, O2, the state
constexpr uint32_t TM_S1 = 0, TM_O = 128, TM_O2 = 256, TM_D = 384;

// Per chunk, from its log decays (log2 units; cs_i the inclusive sums):
struct Tables {
    alignas(16) float a[CQ];       // cs_i - cs at the start of i's 32-row block + log2 scale
    alignas(16) float b[CQ];       // cs at the start of j's block - cs_j
    // 2^(cs at the start of block t + 1 - cs_j), j below that block; in a chunk that resets or grows, from
    // B[0][0] on, the last row at or before each that forgets everything (-1: none)
    alignas(16) float B[3][96];
    alignas(16) float e[CQ];       // 2^cs_i scale
    alignas(16) float w[CQ];       // 2^(cs_127 - cs_j); 0 behind the sequence
    float between[4][4];           // cs at the start of block t - cs at the start of block u
    float dec;                     // 2^cs_127
    int resets;                    // a decay within the chunk may be 0
    int grows;                     // a log decay is positive
};

template <int PARTS>
struct TcSmem {
    alignas(1024) uint8_t q[2][TILE];
    alignas(1024) uint8_t k[2][TILE];
    alignas(1024) uint8_t v[2][2][TILE];
    alignas(1024) uint8_t ks[PARTS][TILE];  // K' parts, rows j
    alignas(1024) uint8_t s16[2][TILE];     // the state's copy, rows = values
    alignas(128) uint8_t mid[4][32 * 64];   // o of each warp on its way out, 32 columns at a time
    Tables tab[NTAB];
    // fp16: 1 / power of two of the copy's rows. Three: chunk c's are read until o_free(c), and the
    // state of chunk c + 2 may be written before that, of c + 3 not
    float col[3][CQ];
    float ps[2][CQ];   // fp16: the power of two of P's rows
    float kmax[2][4];
    uint64_t full[2], empty[2], v_ok[2], tab_full[NTAB], tab_empty[NTAB];
    uint64_t s1_full, p_full, o_full, o_free, s_ready, k_ready, k_max, d_done, drain;
    uint32_t tmem_base;
    int abort, dirty;
};

static_assert(sizeof(TcSmem<3>) + 1024 <= 227 * 1024, "more than a block's shared memory");

struct Args {
    const void *q, *k, *v;
    void* o;
    long long ldq, ldk, ldv, ldo, ldg;
    const float *g, *state_in;
    float* state_out;
    const int* cu;
    int n_seqs, total, Hk, H, dv;
    float log2_scale;
    // sequences in segments of `seg` rows (0: whole): item t of all sequences' `items` segments starts
    // from starts[t] [H, dv, DK], if the sequence has more than one; decays [items, H] are the
    // segments' log2 decays
    int seg, items;
    float *starts, *decays;
};

__device__ __forceinline__ void fail(volatile int* abort, int* status, int role, int step, int bar) {
    *abort = 1;
    tc::record_timeout(status, role, step, bar);
}


template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    const T* x = reinterpret_cast<const T*>(&w);
    return make_float2(to_f(x[0]), to_f(x[1]));
}

// A lane's part of the tables of one chunk, from the log decays of rows 4 l .. 4 l + 3; n rows
// are real.
struct LaneTables {
    float a[4], b[4], e[4], w[4], B[3][4], border[4], between, dec;
    double total;  // the chunk's log2 decay
    int resets, grows;
    __device__ __forceinline__ void make(const float (&g)[4], int n, float lsc) {
        constexpr double LOG2E = 1.4426950408889634;
        const int lane = threadIdx.x & 31, blk = lane >> 3;
        double d[4];
        float down = 0.f;
        bool up = false;
        unsigned m[4];  // the lanes whose i-th row forgets everything: below 2^-150 a decay is 0 in fp32
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool r = g[i] < -104.f;
            m[i] = __ballot_sync(0xffffffffu, r);
            const float x = r ? 0.f : g[i];
            d[i] = (double)x * LOG2E;
            down += fminf(x, 0.f);
            up |= !(x <= 0.f);
        }
        // the sums start again at a border: what lies before it, a NaN among it, enters nothing behind it
        const unsigned any = m[0] | m[1] | m[2] | m[3], below = (1u << lane) - 1;
        double sum = (d[0] + d[1]) + (d[2] + d[3]);
        int head = 0;  // the first lane of the lane's run of rows without a border
        if (any) {
            if ((m[1] | m[2]) >> lane & 1) sum = d[2] + d[3];
            if (m[3] >> lane & 1) sum = 0.0;
            head = max(31 - __clz(any & (below | 1u << lane)), 0);
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane - o >= head) sum += y;
        }
        const double last = __shfl_sync(0xffffffffu, sum, 31);
        double c1 = __shfl_sync(0xffffffffu, sum, 7), c2 = __shfl_sync(0xffffffffu, sum, 15),
               c3 = __shfl_sync(0xffffffffu, sum, 23);
        if (any) {
            // (only reference points: they cancel)
            if (!(c1 - c1 == 0.0)) c1 = 0.0;
            if (!(c2 - c2 == 0.0)) c2 = 0.0;
            if (!(c3 - c3 == 0.0)) c3 = 0.0;
        }
        const double from = blk == 0 ? 0.0 : blk == 1 ? c1 : blk == 2 ? c2 : c3;
        double before = __shfl_up_sync(0xffffffffu, sum, 1);
        if (lane == 0) before = 0.0;
        grows = __any_sync(0xffffffffu, up);
#pragma unroll
        for (int o = 16; o; o >>= 1) down += __shfl_xor_sync(0xffffffffu, down, o);
        resets = !(down * 1.4426950f + fminf(lsc, 0.f) > -120.f);
        double x = before;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x = m[i] >> lane & 1 ? 0.0 : x + d[i];
            a[i] = (float)(x - from) + lsc;
            b[i] = (float)(from - x);
            e[i] = fast_exp2((float)x + lsc);
            w[i] = 4 * lane + i < n ? fast_exp2((float)(last - x)) : 0.f;
            B[0][i] = fast_exp2((float)(c1 - x));
            B[1][i] = fast_exp2((float)(c2 - x));
            B[2][i] = fast_exp2((float)(c3 - x));
        }
        const int r = (lane >> 2) & 3, u = lane & 3;
        const double cr = r == 0 ? 0.0 : r == 1 ? c1 : r == 2 ? c2 : c3;
        const double cu = u == 0 ? 0.0 : u == 1 ? c1 : u == 2 ? c2 : c3;
        between = (float)(cr - cu);
        total = last;
        dec = fast_exp2((float)last);
        border[0] = border[1] = border[2] = border[3] = -1.f;
        if (any) {
            int at = -1, end = -1;  // of the rows before the lane's, and of the chunk
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                at = max(at, 4 * (31 - __clz(m[i] & below)) + i);
                end = max(end, 4 * (31 - __clz(m[i])) + i);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (m[i] >> lane & 1) at = 4 * lane + i;
                border[i] = (float)at;
                if (at >= 0) e[i] = 0.f;
                if (4 * lane + i < end) w[i] = 0.f;
            }
            total = -INFINITY;
            dec = 0.f;
            resets = 1;
        }
    }
    __device__ __forceinline__ void store(Tables& t) const {
        const int lane = threadIdx.x & 31, blk = lane >> 3;
        auto put = [](float* to, const float (&x)[4]) { *reinterpret_cast<float4*>(to) = make_float4(x[0], x[1], x[2], x[3]); };
        put(&t.a[4 * lane], a);
        put(&t.b[4 * lane], b);
        put(&t.e[4 * lane], e);
        put(&t.w[4 * lane], w);
        if (grows || resets) {
            put(&t.B[0][0] + 4 * lane, border);
        } else {
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (blk <= i) put(&t.B[i][4 * lane], B[i]);
        }
        if (lane < 16) t.between[lane >> 2][lane & 3] = between;
        if (lane == 0) {
            t.dec = dec;
            t.resets = resets;
            t.grows = grows;
        }
    }
};

// One value column of `len` rows by the recurrence, from the state row `from` (NULL: zero) to
// `to` (NULL: not kept); o only where asked for.
template <typename T>
__device__ __noinline__ void recurrence(const Args& a, const float* from, float* to, bool with_o, int h, int start, int len,
                                        int col) {
    const int hk = h / (a.H / a.Hk);
    const T* q = static_cast<const T*>(a.q) + start * a.ldq + (long long)hk * DK;
    const T* k = static_cast<const T*>(a.k) + start * a.ldk + (long long)hk * DK;
    const T* v = static_cast<const T*>(a.v) + start * a.ldv + (long long)h * a.dv + col;
    T* o = static_cast<T*>(a.o) + start * a.ldo + (long long)h * a.dv + col;
    const float* g = a.g + start * a.ldg + h;
    const float scale = exp2f(a.log2_scale);
    float S[DK];
#pragma unroll
    for (int e = 0; e < DK; ++e) S[e] = from ? from[e] : 0.f;
#pragma unroll 1
    for (int t = 0; t < len; ++t) {
        const float dec = expf(g[t * a.ldg]), x = to_f(v[t * a.ldv]);
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < DK; ++e) {
            S[e] = fmaf(x, to_f(k[t * a.ldk + e]), fade(dec, S[e]));
            sum = fmaf(S[e], to_f(q[t * a.ldq + e]), sum);
        }
        if (with_o) o[t * a.ldo] = from_f<T>(sum * scale);
    }
    if (to)
#pragma unroll
        for (int e = 0; e < DK; ++e) to[e] = S[e];
}

// Row r of K' = w k as parts of T; w = 0 drops the row. The 16-byte pieces are swizzled by the row.
// Returns whether the row holds an infinity (bf16; of fp16's the largest is looked at).
template <typename T, int PARTS>
__device__ __forceinline__ bool scaled_keys(uint8_t (*ks)[TILE], const uint8_t* krow, int r, float w) {
    const float2 w2 = make_float2(w, w);
    const bool drop = w == 0.f;
    const __nv_bfloat162 nul = __floats2bfloat162_rn(0.f, 0.f);
    __nv_bfloat162 odd = nul;  // 0 x (not finite) is NaN
#pragma unroll 2
    for (int e = 0; e < 8; ++e) {
        const int at = (e ^ (r & 7)) * 16;
        const uint4 x4 = *reinterpret_cast<const uint4*>(krow + at);
        const uint32_t kw[4] = {x4.x, x4.y, x4.z, x4.w};
        uint32_t part[PARTS][4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            float2 y = drop ? make_float2(0.f, 0.f) : __fmul2_rn(unpack2<T>(kw[x]), w2);
            if constexpr (std::is_same<T, bf16>::value)
                odd = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&kw[x]), nul, odd);
#pragma unroll
            for (int p = 0; p < PARTS; ++p) {
                part[p][x] = pack2<T>(y.x, y.y);
                if (p + 1 < PARTS) {
                    const float2 z = unpack2<T>(part[p][x]);
                    y = __ffma2_rn(z, make_float2(-1.f, -1.f), y);  // exact
                }
            }
        }
#pragma unroll
        for (int p = 0; p < PARTS; ++p)
            *reinterpret_cast<uint4*>(ks[p] + r * 128 + at) = make_uint4(part[p][0], part[p][1], part[p][2], part[p][3]);
    }
    if (drop || (*reinterpret_cast<const uint32_t*>(&odd) & 0x7fff7fffu) == 0) return false;
    const uint32_t* kw = reinterpret_cast<const uint32_t*>(krow);
    bool inf = false;
#pragma unroll 1
    for (int x = 0; x < 32; ++x) inf |= __vcmpeq2(kw[x] & 0x7fff7fffu, 0x7f807f80u) != 0;
    return inf;
}

// the power of two of a chunk's K' from its four warps' largest values. Down as far as weights above 1
// may need it; up as far as a state that is much larger than the chunk's keys leaves room in fp32
__device__ __forceinline__ float k_power(const float* m) {
    return to_middle(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), -100, 24);
}

// 32 lanes x 32 columns of fp32, read
__device__ __forceinline__ void ld32(uint32_t addr, float (&x)[32]) {
    tc::tmem_ld32(addr, *reinterpret_cast<uint32_t(*)[32]>(&x));
}

// STATE: only the state that a segment adds to nothing, and its decay, for the next segment's start.
template <typename T, int DV, bool STATE>
__global__ void __launch_bounds__(NT, 1)
linattn_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const Args a, int* status) {
    constexpr bool F16 = std::is_same<T, f16>::value;
    constexpr int PARTS = F16 ? 2 : 3;
    extern __shared__ uint8_t smem_raw[];
    TcSmem<PARTS>& s = *reinterpret_cast<TcSmem<PARTS>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                       ~static_cast<uintptr_t>(1023));
    constexpr uint32_t ID_S1 = tc::idesc_f16(!F16, CQ, CQ), ID_O2 = tc::idesc_f16(!F16, CQ, DV);
    constexpr uint32_t ID_O = tc::idesc_f16(!F16, CQ, DV, true);
    // the state's product reads both operands across their rows (A's bit is 15)
    constexpr uint32_t ID_D = tc::idesc_f16(!F16, 128, DK, true) | (1u << 15);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c0 = blockIdx.x * DV, h = blockIdx.y, hk = h / (a.H / a.Hk);

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&s.full[i], 1);
            tc::mbar_init(&s.empty[i], 1);
            tc::mbar_init(&s.v_ok[i], 32);
        }
        for (int i = 0; i < NTAB; ++i) {
            tc::mbar_init(&s.tab_full[i], 32);
            tc::mbar_init(&s.tab_empty[i], STATE ? 4 : 12);
        }
        tc::mbar_init(&s.s1_full, 1);
        tc::mbar_init(&s.p_full, 128);
        tc::mbar_init(&s.o_full, 1);
        tc::mbar_init(&s.o_free, 128);
        tc::mbar_init(&s.s_ready, 128);
        tc::mbar_init(&s.k_ready, 128);
        tc::mbar_init(&s.k_max, 128);
        tc::mbar_init(&s.d_done, 1);
        tc::mbar_init(&s.drain, 1);
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
    int start, len, item = 0;
    const float* from;  // the state before the first row and after the last, of these columns
    float* to;
    const long long per = (long long)a.dv * DK;
    if (a.seg == 0) {
        const int sq = ragged::longest_first(a.cu, gridDim.z, a.total, blockIdx.z);
        if (!ragged::sequence(a.cu, sq, a.total, &start, &len)) {
            if (tid == 0) set_status(status, HYMBA_ERR_DEVICE_RANGE);
            return;
        }
        from = a.state_in ? a.state_in + ((long long)sq * a.H + h) * per + c0 * DK : nullptr;
        to = a.state_out ? a.state_out + ((long long)sq * a.H + h) * per + c0 * DK : nullptr;
    } else {
        item = blockIdx.z;
        const ragged::Item it = ragged::find_item32(a.cu, a.n_seqs, a.total, a.seg, true, item, item == 0, status);
        if (it.seq < 0) return;
        start = it.start + it.tile * a.seg;
        len = min(a.seg, it.len - it.tile * a.seg);
        const bool last = (it.tile + 1) * a.seg >= it.len;
        if (STATE && last) return;
        const long long at = ((long long)it.seq * a.H + h) * per + c0 * DK;
        // (state_out may be state_in: of a sequence that was cut only `starts` is read)
        from = it.len > a.seg ? a.starts + ((long long)item * a.H + h) * per + c0 * DK : a.state_in ? a.state_in + at : nullptr;
        to = last && a.state_out ? a.state_out + at : nullptr;
        if (STATE) {
            if (item + 1 >= a.items) return;  // (offsets out of order)
            from = nullptr;
            to = a.starts + ((long long)(item + 1) * a.H + h) * per + c0 * DK;
        }
    }
    if (len == 0) {
        if (to)
            for (int i = tid; i < DV * DK; i += NT) to[i] = from ? from[i] : 0.f;
        return;
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
    const int nc = (len + CQ - 1) / CQ;
    int zero = 0;

    if (warp == 0) {
        // ---------------- TMA ----------------
        if (lane == 0) {
            int issued = 0;
            for (int c = 0; c < nc; ++c) {
                const int b = c & 1;
                // the stage's chunk is done with its last product, which follows every read of it
                if (!tc::mbar_wait(&s.empty[b], ((c >> 1) & 1) ^ 1, abort, wlim)) { fail(abort, status, 0, c, 1); break; }
                tc::mbar_arrive_expect_tx(&s.full[b], (STATE ? 1 + DV / 64 : 2 + DV / 64) * TILE);
                if (!STATE) tc::tma_load_2d(s.q[b], &tmQ, &s.full[b], hk * DK, start + c * CQ);
                tc::tma_load_2d(s.k[b], &tmK, &s.full[b], hk * DK, start + c * CQ);
#pragma unroll
                for (int p = 0; p < DV / 64; ++p)
                    tc::tma_load_2d(s.v[b][p], &tmV, &s.full[b], h * a.dv + c0 + p * 64, start + c * CQ);
                issued = c + 1;
            }
            // every copy issued has landed before the block exits
            for (int c = max(0, issued - 2); c < issued; ++c) tc::mbar_wait(&s.full[c & 1], (c >> 1) & 1, &zero);
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        if (tc::elect_one()) {
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t ph, int c, int id) {
                if (ok && !tc::mbar_wait(bar, ph, abort, wlim)) {
                    fail(abort, status, 1, c, id);
                    ok = false;
                }
            };
            for (int c = 0; ok && c < nc; ++c) {
                const int b = c & 1;
                const uint32_t ph2 = (c >> 1) & 1, ph = c & 1;
                const uint32_t qa = tc::smem_u32(s.q[b]), ka = tc::smem_u32(s.k[b]), va = tc::smem_u32(s.v[b][0]);
                wait(&s.full[b], ph2, c, 1);
                if (!STATE) {
                    if (c > 0) wait(&s.o_full, ph ^ 1, c, 2);  // S1 overwrites P
                    if (!ok) break;
                    tc::tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < DK / 16; ++kk)
                        tc::mma_f16_ss(tmem + TM_S1, tc::sdesc_k_sw128(qa + kk * 32), tc::sdesc_k_sw128(ka + kk * 32), ID_S1,
                                       kk > 0);
                    tc::mma_commit(&s.s1_full);
                }
                // the state, once it is decayed and K' is there
                wait(&s.s_ready, ph, c, 3);
                wait(&s.v_ok[b], ph2, c, 4);
                wait(&s.k_ready, ph, c, 5);
                if (!ok) break;
                tc::tc_fence_after();
#pragma unroll
                for (int p = 0; p < PARTS; ++p) {
                    const uint32_t ks = tc::smem_u32(s.ks[p]);
#pragma unroll
                    for (int kk = 0; kk < CQ / 16; ++kk)
                        tc::mma_f16_ss(tmem + TM_D, tc::sdesc_mn_sw128(va + kk * 2048, TILE),
                                       tc::sdesc_mn_sw128(ks + kk * 2048, TILE), ID_D, 1);
                }
                tc::mma_commit(&s.d_done);
                if (STATE) {
                    tc::mma_commit(&s.empty[b]);
                    continue;
                }
                if (c > 0) wait(&s.o_free, ph ^ 1, c, 6);  // O and O2 of the chunk before are read
                if (!ok) break;
                tc::tc_fence_after();
                const uint32_t sa = tc::smem_u32(s.s16[b]);
#pragma unroll
                for (int kk = 0; kk < DK / 16; ++kk)
                    tc::mma_f16_ss(tmem + TM_O2, tc::sdesc_k_sw128(qa + kk * 32), tc::sdesc_k_sw128(sa + kk * 32), ID_O2, kk > 0);
                wait(&s.p_full, ph, c, 7);
                if (!ok) break;
                tc::tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < CQ / 16; ++kk)
                    mma_f16_ts(tmem + TM_O, tmem + TM_S1 + kk * 8, tc::sdesc_mn_sw128(va + kk * 2048, TILE), ID_O, kk > 0);
                tc::mma_commit(&s.o_full);
                tc::mma_commit(&s.empty[b]);
            }
            // every MMA issued has completed before the block exits
            tc::mma_commit(&s.drain);
            tc::mbar_wait(&s.drain, 0, &zero);
        }
    } else if (warp == 2) {
        // ---------------- decay tables ----------------
        const float* g = a.g + start * a.ldg + h;
        float x[4];
        auto fetch = [&](int c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = c * CQ + 4 * lane + i;
                x[i] = t < len ? g[t * a.ldg] : 0.f;
            }
        };
        fetch(0);
        double total = 0.0;
        for (int c = 0; c < nc; ++c) {
            LaneTables t;
            t.make(x, len - c * CQ, a.log2_scale);
            if (c + 1 < nc) fetch(c + 1);
            if (!__all_sync(0xffffffffu, tc::mbar_wait(&s.tab_empty[c % NTAB], ((c / NTAB) & 1) ^ 1, abort, wlim))) {
                if (lane == 0) fail(abort, status, 0, c, 13);
                break;
            }
            t.store(s.tab[c % NTAB]);
            tc::mbar_arrive(&s.tab_full[c % NTAB]);
            // (a segment with a border anywhere takes nothing over, whatever its other decays are)
            total = total == -INFINITY || t.total == -INFINITY ? -INFINITY : total + t.total;
        }
        if (STATE && blockIdx.x == 0 && lane == 0) a.decays[(long long)item * a.H + h] = (float)total;
    } else if (warp == 3) {
        // ---------------- V ----------------
        for (int c = 0; c < nc; ++c) {
            const int b = c & 1;
            if (!__all_sync(0xffffffffu, tc::mbar_wait(&s.full[b], (c >> 1) & 1, abort, wlim))) {
                if (lane == 0) fail(abort, status, 0, c, 12);
                break;
            }
            const int n = len - c * CQ;
            // 16-byte piece x of panel p: row x / 8
            uint4* vb = reinterpret_cast<uint4*>(s.v[b][0]);
            constexpr int PIECES = CQ * 8 * (DV / 64);
            if (n < CQ)
                for (int x = lane; x < PIECES; x += 32)
                    if (((x >> 3) & (CQ - 1)) >= n) vb[x] = make_uint4(0, 0, 0, 0);
            if (__any_sync(0xffffffffu, ragged::any_odd<!F16, PIECES>(vb, lane)) && lane == 0)
                *reinterpret_cast<volatile int*>(&s.dirty) = 1;
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(&s.v_ok[b]);
        }
    } else if (warp < 8) {
        if constexpr (!STATE) {
        // ---------------- P: row i of the chunk, TMEM lane i ----------------
        const int blk = warp & 3, i = blk * 32 + lane;
        const uint32_t lane_base = (uint32_t)(blk * 32) << 16;
        const uint32_t s1 = tmem + lane_base + TM_S1;
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t ph, int c, int id) {
            if (ok && !__all_sync(0xffffffffu, tc::mbar_wait(bar, ph, abort, wlim))) {
                if (lane == 0) fail(abort, status, 2, c, id);
                ok = false;
            }
        };
        for (int c = 0; ok && c < nc; ++c) {
            const int b = c & 1;
            const Tables& tab = s.tab[c % NTAB];
            wait(&s.tab_full[c % NTAB], (c / NTAB) & 1, c, 20);
            wait(&s.s1_full, c & 1, c, 21);
            if (!ok) break;
            tc::tc_fence_after();
            const bool grows = tab.grows, plain = !grows && !tab.resets;
            const float ai = tab.a[i], Ai = fast_exp2(ai);
            // columns 32 u .. 32 u + 31 of the scores, in place -> scale * decay * score, 0 above the
            // diagonal
            auto decayed = [&](int u, float (&x)[32]) {
                if (u < blk && plain) {
                    const float2 A2 = make_float2(Ai, Ai);
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 B = *reinterpret_cast<const float4*>(&tab.B[blk - 1][32 * u + j]);
                        const float2 y = __fmul2_rn(__fmul2_rn(make_float2(x[j], x[j + 1]), A2), make_float2(B.x, B.y));
                        const float2 z = __fmul2_rn(__fmul2_rn(make_float2(x[j + 2], x[j + 3]), A2), make_float2(B.z, B.w));
                        x[j] = y.x;
                        x[j + 1] = y.y;
                        x[j + 2] = z.x;
                        x[j + 3] = z.y;
                    }
                } else {
                    const float base = ai + tab.between[blk][u];
                    const float2 base2 = make_float2(base, base);
                    unsigned see = u < blk ? 0xffffffffu : 0xffffffffu >> (31 - lane);
                    if (!plain) {
                        // a decay of 0 drops what it multiplies, also what is not finite
                        const int first = (int)(&tab.B[0][0])[i] - 32 * u;
#pragma unroll 1
                        for (int j = 0; j < 32; ++j)
                            if (j < first || fast_exp2(base + tab.b[32 * u + j]) == 0.f) see &= ~(1u << j);
                    }
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 bj = *reinterpret_cast<const float4*>(&tab.b[32 * u + j]);
                        const float2 d = __fadd2_rn(base2, make_float2(bj.x, bj.y)), e = __fadd2_rn(base2, make_float2(bj.z, bj.w));
                        const float2 y = __fmul2_rn(make_float2(fast_exp2(d.x), fast_exp2(d.y)), make_float2(x[j], x[j + 1]));
                        const float2 z = __fmul2_rn(make_float2(fast_exp2(e.x), fast_exp2(e.y)), make_float2(x[j + 2], x[j + 3]));
                        x[j] = see >> j & 1 ? y.x : 0.f;
                        x[j + 1] = see >> (j + 1) & 1 ? y.y : 0.f;
                        x[j + 2] = see >> (j + 2) & 1 ? z.x : 0.f;
                        x[j + 3] = see >> (j + 3) & 1 ? z.y : 0.f;
                    }
                }
            };
            float f = 1.f;
            if (F16) {
                // the row's power of two, from its largest score, which bounds P; from P itself where a
                // decay may be above 1 or hide a score
                float mx = 0.f;
#pragma unroll 1
                for (int u = 0; u <= blk; ++u) {
                    float x[32];
                    ld32(s1 + 32 * u, x);
                    tc::tmem_wait_ld();
                    if (!plain) decayed(u, x);
                    const int last = u < blk ? 31 : lane;  // (behind the diagonal: keys the row does not see)
#pragma unroll
                    for (int j = 0; j < 32; j += 2)
                        mx = fmax3(mx, j <= last ? fabsf(x[j]) : 0.f, j + 1 <= last ? fabsf(x[j + 1]) : 0.f);
                }
                f = to_middle(!plain ? mx : mx * fast_exp2(a.log2_scale), -100, 100);
                s.ps[b][i] = f;
            }
            // P over the scores: block u goes to columns 16 u .. 16 u + 15, all read by then
#pragma unroll 1
            for (int u = 0; u < 4; ++u) {
                uint32_t pk[16];
                if (u <= blk) {
                    float x[32];
                    ld32(s1 + 32 * u, x);
                    tc::tmem_wait_ld();
                    decayed(u, x);
#pragma unroll
                    for (int j = 0; j < 32; j += 2)
                        pk[j / 2] = F16 ? pack2<T>(x[j] * f, x[j + 1] * f) : pack2<T>(x[j], x[j + 1]);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) pk[j] = 0u;
                }
                tc::tmem_st16(s1 + 16 * u, pk);
            }
            tc::tmem_wait_st();
            tc::tc_fence_before();
            tc::mbar_arrive(&s.p_full);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&s.tab_empty[c % NTAB]);
        }
        }
    } else if (warp < 12) {
        // ---------------- the state (row r a value), then K' (row r of the chunk) ----------------
        const int quad = warp & 3, r = quad * 32 + lane;
        const uint32_t dc = tmem + ((uint32_t)(quad * 32) << 16) + TM_D;
        const bool mine = quad * 32 < DV;  // the warp's rows are values of this block
        float power = 1.f;                 // the state in TMEM is S * power (fp16)
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t ph, int c, int id) {
            if (ok && !__all_sync(0xffffffffu, tc::mbar_wait(bar, ph, abort, wlim))) {
                if (lane == 0) fail(abort, status, 2, c, id);
                ok = false;
            }
        };
        if (mine) {
#pragma unroll 1
            for (int u = 0; u < DK; u += 32) {
                float y[32];
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (from) z = *reinterpret_cast<const float4*>(from + (long long)r * DK + u + e);
                    y[e] = z.x;
                    y[e + 1] = z.y;
                    y[e + 2] = z.z;
                    y[e + 3] = z.w;
                }
                tc::tmem_st32(dc + u, *reinterpret_cast<uint32_t(*)[32]>(&y));
            }
            tc::tmem_wait_st();
        }
        for (int c = 0; ok && c < nc; ++c) {
            const int b = c & 1;
            const Tables& tab = s.tab[c % NTAB];
            wait(&s.tab_full[c % NTAB], (c / NTAB) & 1, c, 30);
            wait(&s.full[b], (c >> 1) & 1, c, 31);
            if (!ok) break;
            const uint8_t* krow = s.k[b] + r * 128;  // its 16-byte pieces are swizzled by the row
            const float w = tab.w[r], dec0 = tab.dec;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&s.tab_empty[c % NTAB]);
            float fk = 1.f;
            if (F16) {
                // the chunk's power for K': from the largest |w k|
                float m = 0.f;
#pragma unroll 2
                for (int e = 0; e < 8; ++e) {
                    const uint4 x = *reinterpret_cast<const uint4*>(krow + (e ^ (r & 7)) * 16);
                    const uint32_t kw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 y = unpack2<T>(kw[i]);
                        m = fmax3(m, fabsf(y.x), fabsf(y.y));
                    }
                }
                m = fade(w, m);
                if (m == INFINITY) *reinterpret_cast<volatile int*>(&s.dirty) = 1;
#pragma unroll
                for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
                if (lane == 0) s.kmax[b][quad] = m;
                tc::mbar_arrive(&s.k_max);
                wait(&s.k_max, c & 1, c, 34);
                if (!ok) break;
                fk = k_power(s.kmax[b]);
            }
            if (c > 0) wait(&s.d_done, (c - 1) & 1, c, 32);  // the state is whole, K' buffers are free
            if (!ok) break;
            tc::tc_fence_after();
            if (mine) {
                float fs = 1.f, dec = dec0;
                if (F16 && !STATE) {
                    float m = 0.f;
#pragma unroll 1
                    for (int u = 0; u < DK; u += 32) {
                        float y[32];
                        ld32(dc + u, y);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; e += 2) m = fmax3(m, fabsf(y[e]), fabsf(y[e + 1]));
                    }
                    fs = to_middle(m, -100, 100);
                    s.col[c % 3][r] = inverse(fs) * inverse(power);
                }
                if (F16) {
                    dec = dec0 * (fk * inverse(power));
                }
                uint8_t* row = s.s16[b] + r * 128;
#pragma unroll 1
                for (int u = 0; u < DK; u += 32) {
                    float y[32];
                    ld32(dc + u, y);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; !STATE && e < 32; e += 8)
                        *reinterpret_cast<uint4*>(row + ((((u + e) >> 3) ^ (r & 7)) * 16)) =
                            make_uint4(pack2<T>(y[e] * fs, y[e + 1] * fs), pack2<T>(y[e + 2] * fs, y[e + 3] * fs),
                                       pack2<T>(y[e + 4] * fs, y[e + 5] * fs), pack2<T>(y[e + 6] * fs, y[e + 7] * fs));
                    const float2 d2 = make_float2(dec, dec);
                    if (dec0 == 0.f) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) y[e] = 0.f;
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 z = __fmul2_rn(make_float2(y[e], y[e + 1]), d2);
                        y[e] = z.x;
                        y[e + 1] = z.y;
                    }
                    tc::tmem_st32(dc + u, *reinterpret_cast<uint32_t(*)[32]>(&y));
                }
                tc::tmem_wait_st();
            }
            power = fk;
            tc::fence_proxy_async_smem();
            tc::tc_fence_before();
            tc::mbar_arrive(&s.s_ready);
            if (scaled_keys<T, PARTS>(s.ks, krow, r, w * fk)) *reinterpret_cast<volatile int*>(&s.dirty) = 1;
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(&s.k_ready);
        }
        wait(&s.d_done, (nc - 1) & 1, nc, 33);
        if (ok && mine && to && !*reinterpret_cast<volatile int*>(&s.dirty)) {
            tc::tc_fence_after();
            const float back = F16 ? inverse(power) : 1.f;
            float* row = to + (long long)r * DK;
#pragma unroll 1
            for (int u = 0; u < DK; u += 32) {
                float y[32];
                ld32(dc + u, y);
                tc::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<float4*>(row + u + e) =
                        make_float4(y[e] * back, y[e + 1] * back, y[e + 2] * back, y[e + 3] * back);
            }
        }
    } else if constexpr (!STATE) {
        // ---------------- o: row r of the chunk ----------------
        const int quad = warp & 3, r = quad * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        const uint32_t oc = tmem + lane_base + TM_O, o2c = tmem + lane_base + TM_O2;
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t ph, int c, int id) {
            if (ok && !__all_sync(0xffffffffu, tc::mbar_wait(bar, ph, abort, wlim))) {
                if (lane == 0) fail(abort, status, 2, c, id);
                ok = false;
            }
        };
        for (int c = 0; ok && c < nc; ++c) {
            const int b = c & 1;
            wait(&s.tab_full[c % NTAB], (c / NTAB) & 1, c, 35);
            if (!ok) break;
            const float ei = s.tab[c % NTAB].e[r];
            const bool resets = s.tab[c % NTAB].resets;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&s.tab_empty[c % NTAB]);
            wait(&s.o_full, c & 1, c, 38);
            if (!ok) break;
            tc::tc_fence_after();
            const float back = F16 ? inverse(s.ps[b][r]) : 1.f;
            const float2 e2 = make_float2(ei, ei), back2 = make_float2(back, back);
            // 32 columns at a time: the warp's 32 rows to shared memory, then 64-byte pieces of rows out
            uint8_t* mid = s.mid[quad];
            T* orow = static_cast<T*>(a.o) + (start + (long long)c * CQ + r - lane + (lane >> 2)) * a.ldo +
                      (long long)h * a.dv + c0 + 8 * (lane & 3);
            const int n = len - c * CQ - quad * 32 - (lane >> 2);  // rows from the lane's first to the sequence's end
            uint32_t y[2][16], z[2][16];
            tc::tmem_ld16(oc, y[0]);
            tc::tmem_ld16(o2c, z[0]);
#pragma unroll 1
            for (int u0 = 0; u0 < DV / 16; u0 += 2) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int u = u0 + e;
                    tc::tmem_wait_ld();
                    if (u + 1 < DV / 16) {
                        tc::tmem_ld16(oc + 16 * (u + 1), y[e ^ 1]);
                        tc::tmem_ld16(o2c + 16 * (u + 1), z[e ^ 1]);
                    }
                    if (resets && ei == 0.f) {
#pragma unroll
                        for (int x = 0; x < 16; ++x) z[e][x] = 0u;
                    }
                    uint32_t w8[8];
#pragma unroll
                    for (int x = 0; x < 16; x += 2) {
                        float2 p = make_float2(__uint_as_float(y[e][x]), __uint_as_float(y[e][x + 1]));
                        float2 t = make_float2(__uint_as_float(z[e][x]), __uint_as_float(z[e][x + 1]));
                        if (F16) {
                            p = __fmul2_rn(p, back2);
                            t = __fmul2_rn(t, *reinterpret_cast<const float2*>(&s.col[c % 3][16 * u + x]));
                        }
                        const float2 v = __ffma2_rn(t, e2, p);
                        w8[x / 2] = pack2<T>(v.x, v.y);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        *reinterpret_cast<uint4*>(mid + lane * 64 + (((2 * e + i) ^ ((lane >> 1) & 3)) * 16)) =
                            make_uint4(w8[4 * i], w8[4 * i + 1], w8[4 * i + 2], w8[4 * i + 3]);
                }
                if (u0 + 2 == DV / 16) {
                    tc::tc_fence_before();
                    tc::mbar_arrive(&s.o_free);
                }
                __syncwarp();
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int row = 8 * x + (lane >> 2);
                    const uint4 w = *reinterpret_cast<const uint4*>(mid + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) * 16));
                    if (8 * x < n) *reinterpret_cast<uint4*>(orow + 8 * x * a.ldo + 16 * u0) = w;
                }
                __syncwarp();
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
    if (s.dirty && !s.abort && tid >= 128 && tid < 128 + DV) {
        const long long row = (long long)(tid - 128) * DK;
        recurrence<T>(a, from ? from + row : nullptr, to ? to + row : nullptr, !STATE, h, start, len, c0 + tid - 128);
    }
}

// The state before every segment of a sequence that was cut: the state before the segment before,
// decayed, plus what that segment added (already in `starts`), one after the other. The decay in
// two halves: over a whole segment it may leave fp32's range where the product does not; below
// 2^-159 it drops what it multiplies, like one row's.
__global__ void __launch_bounds__(256) linattn_starts_kernel(const Args a) {
    griddep_sync();
    const int h = blockIdx.y, sq = blockIdx.z;
    const long long per = (long long)a.dv * DK, at = (long long)blockIdx.x * 1024 + threadIdx.x * 4;
    int start, len;
    if (at >= per || !ragged::sequence(a.cu, sq, a.total, &start, &len) || len <= a.seg) return;
    int first = 0;  // the sequence's first item
    for (int j = 0; j < sq; ++j) {
        int x, n;
        if (ragged::sequence(a.cu, j, a.total, &x, &n)) first += n ? (n + a.seg - 1) / a.seg : 1;
    }
    float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.state_in) S = *reinterpret_cast<const float4*>(a.state_in + ((long long)sq * a.H + h) * per + at);
    const int end = min(first + (len + a.seg - 1) / a.seg, a.items);  // (more only with offsets out of order)
    for (int i = first; i < end; ++i) {
        if (i > first) {
            const float d2 = a.decays[(long long)(i - 1) * a.H + h], d = exp2f(0.5f * d2);
            const float4 u = *reinterpret_cast<const float4*>(a.starts + ((long long)i * a.H + h) * per + at);
            auto next = [&](float x, float add) { return (d2 < -159.f ? 0.f : x * d * d) + add; };
            S = make_float4(next(S.x, u.x), next(S.y, u.y), next(S.z, u.z), next(S.w, u.w));
        }
        *reinterpret_cast<float4*>(a.starts + ((long long)i * a.H + h) * per + at) = S;
    }
}

// How sequences are cut where they and their heads leave SMs idle: 0 (whole), or rows per segment
// such that the segments' blocks fill the GPU once, three chunks at least. A chunk costs about two
// thirds as much again in the pass over states, the launches and the join as much as 400 rows: that
// has to pay also where all sequences are equally long, which the host does not know. bf16,
// heads of 64 x 128, cut and whole: one prompt of 8192 rows, 25 heads 90 and 194 us, 73 heads 191
// and 196; of 1100 rows, 8 heads 29 and 32 (1000 rows would be even); of 30,000 rows 102 and 677; 8
// heads, four prompts of 2000 rows 44 and 53, one of 9000 and three of 1000 59 and 214.
int segment_rows(int n_seqs, int total, int H, int dv) {
    const long long per = (long long)H * (dv % 128 ? dv / 64 : dv / 128);  // blocks of a segment
    const long long want = 148 / per - (n_seqs - 1);  // segments of n sequences: up to n - 1 more than of one
    if (n_seqs > 32 || want < 2) return 0;
    const long long rows = std::max<long long>(3 * CQ, round_up((total + want - 1) / want, CQ));
    return n_seqs * (rows + rows * 2 / 3 + 400) < total ? (int)rows : 0;
}
long long segment_items(int seg, int n_seqs, int total) { return (total + seg - 1) / seg + n_seqs - 1; }

template <typename T, int DV, bool STATE>
int launch_pass(const Ctx& ctx, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const Args& a, int z) {
    auto kern = linattn_tc_kernel<T, DV, STATE>;
    const size_t smem = sizeof(TcSmem<std::is_same<T, bf16>::value ? 3 : 2>) + 1024;
    static std::atomic<unsigned long long> smem_set{0};
    if (!smem_opt_in_once(smem_set, kern, smem, ctx)) return HYMBA_ERR_CUDA;
    HYMBA_LAUNCH(ctx, STATE ? "linattn_segment_states" : "linattn_chunk", kern, dim3(a.dv / DV, a.H, z), NT, smem, tq, tk, tv, a,
                 ctx.status);
    return HYMBA_OK;
}

template <typename T, int DV>
int launch_dv(const Ctx& ctx, const LinAttn& x) {
    constexpr bool BF16 = std::is_same<T, bf16>::value;
    CUtensorMap tq, tk, tv;
    if (!tc::make_tmap_2d(&tq, x.q, BF16, x.total, (uint64_t)x.Hk * DK, x.ldq, CQ) ||
        !tc::make_tmap_2d(&tk, x.k, BF16, x.total, (uint64_t)x.Hk * DK, x.ldk, CQ) ||
        !tc::make_tmap_2d(&tv, x.v, BF16, x.total, (uint64_t)x.H * x.dv, x.ldv, CQ))
        return HYMBA_ERR_UNSUPPORTED;
    Args a;
    a.q = x.q; a.k = x.k; a.v = x.v; a.o = x.o;
    a.ldq = x.ldq; a.ldk = x.ldk; a.ldv = x.ldv; a.ldo = x.ldo; a.ldg = x.ldg;
    a.g = x.g;
    a.state_in = x.state_in;
    a.state_out = x.state_out;
    a.cu = x.cu;
    a.n_seqs = x.n_seqs; a.total = x.total; a.Hk = x.Hk; a.H = x.H; a.dv = x.dv;
    a.log2_scale = log2f(x.scale);
    a.seg = segment_rows(x.n_seqs, x.total, x.H, x.dv);
    a.items = 0;
    a.starts = a.decays = nullptr;
    if (a.seg) {
        const int items = a.items = (int)segment_items(a.seg, x.n_seqs, x.total);
        a.decays = static_cast<float*>(x.ws);
        a.starts = a.decays + round_up((long long)items * x.H, 64);
        int rc = launch_pass<T, DV, true>(ctx, tq, tk, tv, a, items);
        if (rc) return rc;
        HYMBA_LAUNCH(ctx, "linattn_starts", linattn_starts_kernel, dim3(ceil_div((long long)x.dv * DK, 1024), x.H, x.n_seqs), 256,
                     0, a);
        return launch_pass<T, DV, false>(ctx, tq, tk, tv, a, items);
    }
    // sequences on the grid's slowest dimension, in runs it can hold
    for (int s0 = 0; s0 < x.n_seqs; s0 += 65535) {
        const int n = x.n_seqs - s0 < 65535 ? x.n_seqs - s0 : 65535;
        const long long st0 = (long long)s0 * x.H * x.dv * DK;
        a.state_in = x.state_in ? x.state_in + st0 : nullptr;
        a.state_out = x.state_out ? x.state_out + st0 : nullptr;
        a.cu = x.cu + s0;
        const int rc = launch_pass<T, DV, false>(ctx, tq, tk, tv, a, n);
        if (rc) return rc;
    }
    return HYMBA_OK;
}

}  // namespace

bool linattn_tc_applies(int dk) { return dk == DK; }

size_t linattn_tc_bytes(int n_seqs, int total, int H, int dv) {
    const int seg = segment_rows(n_seqs, total, H, dv);
    if (!seg) return 256;
    const long long items = segment_items(seg, n_seqs, total);
    return (size_t)(round_up(items * H, 64) + items * H * dv * DK) * 4;
}

template <typename T>
int launch_linattn_tc(const Ctx& ctx, const LinAttn& a) {
    return a.dv % 128 == 0 ? launch_dv<T, 128>(ctx, a) : launch_dv<T, 64>(ctx, a);
}
template int launch_linattn_tc<f16>(const Ctx&, const LinAttn&);
template int launch_linattn_tc<bf16>(const Ctx&, const LinAttn&);

}  // namespace hymba
