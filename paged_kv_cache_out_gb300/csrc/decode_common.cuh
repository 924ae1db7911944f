// decode_common.cuh -- the balanced partition that the decode kernels share:
// all (sequence, KV head) segments laid end to end in tiles and cut into equal
// ranges, one per persistent block (see decode.cu).
#pragma once

#include "common.cuh"

namespace pkv {
namespace decode {

constexpr int kMaxBatch = 4096;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegBig = -1.0e30f;  // running-max start: finite, so 2^(m - m') never is NaN

// Geometry of the balanced partition, shared by the main and merge kernels.
struct Part {
    int64_t W;   // total tiles
    int grid;    // blocks of the main kernel
    // floor(k W / grid), as k q + floor(k r / grid) with W = q grid + r: exact,
    // and k r < grid^2 fits 32 bits
    __device__ __forceinline__ int64_t start(int k) const {
        const int64_t q = W / grid;
        const int r = static_cast<int>(W - q * grid);
        return (int64_t)k * q + static_cast<int>(static_cast<unsigned>(k * r) / static_cast<unsigned>(grid));
    }
    __device__ __forceinline__ int block_of(int64_t x) const {
        return static_cast<int>(((x + 1) * grid - 1) / W);
    }
};

// Floats of one partial state in the workspace: G x D weighted sums, then a
// (max, sum) pair per head, padded to a multiple of 4 so that every state
// starts on a 16-byte boundary (the merge kernel reads it as float4).
__host__ __device__ constexpr int part_stride(int G, int D) { return ((G * D + 2 * G + 3) / 4) * 4; }

__device__ __forceinline__ int ntiles_of(int L, int64_t cap, int T) {
    return (L > 0 && L <= cap) ? (L + T - 1) / T : 0;
}

// Work units of a segment in the balanced partition: its tiles plus kLead
// units standing for the fixed cost of a segment piece (the page-id read, the
// q copy, the reduction across row groups and the output write), so that a
// block whose range holds many short segments gets fewer tiles.  A segment
// occupies [kLead lead units][its tiles]; lead units load nothing.  Empty
// segments occupy no units.
constexpr int kLead = 2;
template <int LEAD = kLead>
__device__ __forceinline__ int units_of(int ntiles) {
    return ntiles > 0 ? ntiles + LEAD : 0;
}

// Largest b in [0, B) with prefix[b] <= x (x < prefix[B]).
__device__ __forceinline__ int owner_search(const int32_t *prefix, int B, int64_t x) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

struct Piece {
    int b, g;
    int t0, t1;         // tile range inside the segment (t1 <= t0: lead units only)
    int nt;             // tiles of the whole segment
    bool whole;         // covers all tiles of the segment
    bool block_first;   // first piece of this block
};

// The next piece of the block's unit range, with its units turned into tiles.
template <int LEAD = kLead>
__device__ __forceinline__ bool next_piece(int64_t &pos, int64_t end, int64_t block_start,
                                           const int32_t *prefix, int B, int Hkv, Piece &p) {
    if (pos >= end) return false;
    const int b = owner_search(prefix, B, pos);
    const int nu = (prefix[b + 1] - prefix[b]) / Hkv;  // units of each segment of b
    const int64_t rel = pos - prefix[b];
    p.b = b;
    p.g = static_cast<int>(rel / nu);
    const int u0 = static_cast<int>(rel % nu);
    const int64_t seg_end = prefix[b] + (int64_t)(p.g + 1) * nu;
    const int64_t pend = end < seg_end ? end : seg_end;
    const int u1 = u0 + static_cast<int>(pend - pos);
    p.t0 = u0 > LEAD ? u0 - LEAD : 0;
    p.t1 = u1 - LEAD;
    p.nt = nu - LEAD;
    p.whole = (u0 <= LEAD) && (pend == seg_end);
    p.block_first = (pos == block_start);
    pos = pend;
    return true;
}

// Block-wide exclusive scan: prefix[b] = Hkv * sum_{b' < b} units(b'); the
// lengths themselves are kept in lens[b].
template <int THREADS, int LEAD = kLead>
__device__ void build_prefix(int32_t *prefix, int32_t *lens, const int32_t *seq_lens, int B,
                             int Hkv, int64_t cap, int T,
                             int32_t *scratch /* THREADS/32 + 1 ints */) {
    const int tid = threadIdx.x;
    const int per = (B + THREADS - 1) / THREADS;
    const int lo = tid * per;
    const int hi = min(B, lo + per);
    int local = 0;
    for (int b = lo; b < hi; ++b) {
        const int L = seq_lens[b];
        lens[b] = L;
        local += units_of<LEAD>(ntiles_of(L, cap, T)) * Hkv;
    }
    // inclusive scan of `local` over the block
    const int lane = tid & 31, warp = tid >> 5;
    int v = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += n;
    }
    if (lane == 31) scratch[warp] = v;
    __syncthreads();
    if (tid == 0) {
        int acc = 0;
        for (int w = 0; w < THREADS / 32; ++w) {
            const int t = scratch[w];
            scratch[w] = acc;
            acc += t;
        }
        scratch[THREADS / 32] = acc;
    }
    __syncthreads();
    int run = scratch[warp] + v - local;  // exclusive prefix of this thread's chunk
    for (int b = lo; b < hi; ++b) {
        prefix[b] = run;
        run += units_of<LEAD>(ntiles_of(lens[b], cap, T)) * Hkv;
    }
    if (tid == 0) prefix[B] = scratch[THREADS / 32];
    __syncthreads();
}

}  // namespace decode
}  // namespace pkv
