// Pieces shared by the kernels of ragged batches (packed prompts, paged K/V, linear
// attention): work items of packed sequences, powers of two for fp16's range, a look for values
// that are not finite, 16-byte row loads of any type.
#pragma once
#include "common.cuh"
#include "warp_mma.cuh"

namespace hymba {
namespace ragged {

// One work item of a packed batch: `tile`-th run of rows of sequence `seq`, whose rows
// are start .. start + len - 1. seq < 0: no such item.
struct Item {
    int seq, start, len, tile;
};

// Sequence s of the packed batch; false when its offsets are out of order or out of range.
__device__ __forceinline__ bool sequence(const int* cu, int s, int total, int* start, int* len) {
    const int a = cu[s], b = cu[s + 1];
    *start = a;
    *len = b - a;
    return a >= 0 && b >= a && b <= total;
}

// The z-th longest of up to 32 sequences (z itself when there are more): blocks that walk one
// sequence each start with the longest, so that the last ones to start are short. Every lane of
// the warp returns it; one round trip to memory.
__device__ __forceinline__ int longest_first(const int* cu, int n_seqs, int total, int z) {
    if (n_seqs > 32) return z;
    const int lane = threadIdx.x & 31;
    int a = 0, n = -1;
    if (lane < n_seqs && !sequence(cu, lane, total, &a, &n)) n = 0;
    int rank = 0;
    for (int j = 0; j < n_seqs; ++j) {
        const int m = __shfl_sync(0xffffffffu, n, j);
        rank += m > n || (m == n && j < lane);
    }
    const unsigned hit = __ballot_sync(0xffffffffu, lane < n_seqs && rank == z);
    return __ffs(hit) - 1;
}

struct FindSmem {
    long long warp_sum[32];
    Item item;
};

// The t-th work item of up to 32 sequences, each cut into ceil(len / rows) runs (min_one: at least
// one, so that empty sequences are items too): every warp for itself, one round trip, no
// barrier. `report`: whether this warp records offsets that are out of order.
__device__ __forceinline__ Item find_item32(const int* cu, int n_seqs, int total, int rows, bool min_one, long long t,
                                            bool report, int* status) {
    const int lane = threadIdx.x & 31;
    int a = 0, n = 0, c = 0;
    if (lane < n_seqs) {
        if (sequence(cu, lane, total, &a, &n)) {
            c = (n + rows - 1) / rows;
            if (min_one && c == 0) c = 1;
        } else if (report) {
            set_status(status, HYMBA_ERR_DEVICE_RANGE);
        }
    }
    long long incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, t >= incl - c && t < incl);
    const int at = hit ? __ffs(hit) - 1 : 0;
    Item it;
    it.seq = hit ? at : -1;
    it.start = __shfl_sync(0xffffffffu, a, at);
    it.len = __shfl_sync(0xffffffffu, n, at);
    it.tile = (int)(t - __shfl_sync(0xffffffffu, incl - c, at));
    return it;
}

// The t-th work item when every sequence is cut into ceil(len / rows) runs. Called by all NT threads of the
// block; each thread counts a run of consecutive sequences and one block scan finds the
// sequence, so the cost is a few memory round trips for any number of sequences.
template <int NT>
__device__ Item find_item(FindSmem& sm, const int* cu, int n_seqs, int total, int rows, long long t, int* status) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (n_seqs <= 32) return find_item32(cu, n_seqs, total, rows, false, t, blockIdx.x == 0 && warp == 0, status);
    const int per = (n_seqs + NT - 1) / NT;
    const int s0 = min(tid * per, n_seqs), s1 = min(s0 + per, n_seqs);
    if (tid == 0) sm.item.seq = -1;
    long long mine = 0;
    for (int s = s0; s < s1; ++s) {
        int a, n;
        if (sequence(cu, s, total, &a, &n)) {
            mine += (n + rows - 1) / rows;
        } else if (blockIdx.x == 0) {
            set_status(status, HYMBA_ERR_DEVICE_RANGE);
        }
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) sm.warp_sum[warp] = incl;
    __syncthreads();
    long long before = incl - mine;
    for (int w = 0; w < warp; ++w) before += sm.warp_sum[w];
    if (t >= before && t < before + mine) {
        for (int s = s0; s < s1; ++s) {
            int a, n;
            if (!sequence(cu, s, total, &a, &n)) continue;
            const int c = (n + rows - 1) / rows;
            if (t < before + c) {
                sm.item.seq = s;
                sm.item.start = a;
                sm.item.len = n;
                sm.item.tile = (int)(t - before);
                break;
            }
            before += c;
        }
    }
    __syncthreads();
    return sm.item;
}

// a power of two that brings x (> 0) near 2^12, within 2^low and 2^high; 1 for 0 and what is
// not finite
__device__ __forceinline__ float to_middle(float x, int low, int high) {
    const int e = (__float_as_int(x) >> 23) & 255;
    if (e == 0 || e == 255) return 1.f;
    return __int_as_float((127 + min(max(127 - e + 12, low), high)) << 23);
}
// the inverse of a power of two: its exponent mirrored
__device__ __forceinline__ float inverse(float p) { return __int_as_float(0x7f000000 - __float_as_int(p)); }
// a decay of 0 drops what it multiplies, also what is not finite
__device__ __forceinline__ float fade(float d, float x) { return d == 0.f ? 0.f : d * x; }

// Whether the lane's share of PIECES 16-byte pieces holds a value that is infinite or NaN: 0 x it
// is NaN, and a sum of such products stays NaN. Eight loads in flight: one at a time, a block
// of V took longer to look through than its softmax.
template <bool BF16, int PIECES>
__device__ __forceinline__ bool any_odd(const uint4* v, int lane) {
    typedef typename std::conditional<BF16, __nv_bfloat162, __half2>::type P2;
    const uint32_t nul = 0u;
    uint32_t acc[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
    for (int x = lane; x < PIECES; x += 32 * 8) {
        uint4 w[8];
#pragma unroll
        for (int y = 0; y < 8; ++y) w[y] = v[x + 32 * y];
#pragma unroll
        for (int y = 0; y < 8; ++y) {
            const uint32_t ww[4] = {w[y].x, w[y].y, w[y].z, w[y].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const P2 r = __hfma2(*reinterpret_cast<const P2*>(&ww[i]), *reinterpret_cast<const P2*>(&nul),
                                     *reinterpret_cast<const P2*>(&acc[i]));
                acc[i] = *reinterpret_cast<const uint32_t*>(&r);
            }
        }
    }
    return ((acc[0] | acc[1] | acc[2] | acc[3]) & 0x7fff7fffu) != 0;
}
// 8 consecutive elements as fp32 (one or two 16-byte loads)
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const T* h = reinterpret_cast<const T*>(&u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f(h[i]);
    } else {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
}

// 4 consecutive elements as fp32 (one 8- or 16-byte load), and their store
template <typename T>
__device__ __forceinline__ float4 load4(const T* p) {
    if constexpr (sizeof(T) == 2) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        const T* h = reinterpret_cast<const T*>(&u);
        return make_float4(to_f(h[0]), to_f(h[1]), to_f(h[2]), to_f(h[3]));
    } else {
        return *reinterpret_cast<const float4*>(p);
    }
}
template <typename T>
__device__ __forceinline__ void store4(T* p, float a, float b, float c, float d) {
    if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack2<T>(a, b), pack2<T>(c, d));
    } else {
        *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
    }
}

}  // namespace ragged
}  // namespace hymba
