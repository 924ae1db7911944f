// kv_evict.cu -- shorten cached sequences: per (sequence, KV head) keep the
// first, the last and the heaviest keys, and move them to the front.
//
// miniVLLM "Engine Architecture" (allocate_kv_cache: the pool; block_tables map
// a sequence's positions to pages).  The pages of the source describe no
// eviction; a sequence that must shrink keeps the keys whose accumulated
// softmax weight (pkv_paged_decode_attn_weights) is largest.
//
//  * select: one block per (sequence, KV head).  The n - first - recent heaviest
//    keys are found by a radix select on the sums' bits: histogram passes (11, 11
//    and 10 bits, high to low) narrow down the weight of the last key that stays,
//    until at most 256 keys are left, which are ranked against each other; a last
//    pass over the positions in order writes the kept ones and moves their sums.
//    Bound by its instructions (60 % of issue slots): 1024 rows of 512-4096 sums
//    20 us, 64 rows of 16-32 K sums 26 us.
//  * move: the K and V rows of the kept positions.  kept[i] >= i, so a cluster that
//    takes the kept rows in rising order and loads a round of them before it
//    stores any of the round never overwrites a row that is still to be read:
//    the rows stored so far lie below the round, the rows to come at or above it.
//    Memory-bound: 128 sequences of 512-4096 keys, 8 KV heads of 128, halved in
//    place (1.2 GB) 183 us, 6.6 TB/s against 6.8 TB/s of a plain copy.
// Two launches, or one where there is little to do.
// Threads, shared memory and the number of launches go by acc_stride, the only bound on
// the lengths that the host has: rows of sums cut to the batch are fastest.  On rows 32768
// wide the batch above takes 228 us instead of 209, four sequences of 37-513 keys 10.1
// instead of 7.0, eight of 16-32 K keys 62 as before.
#include <math.h>

#include <mutex>

#include "common.cuh"

namespace pkv {
namespace evict {

struct Args {
    const int32_t *page_table, *page_table_out;
    int64_t pt_stride, pt_out_stride;
    const int32_t *seq_lens, *keep_lens;
    int Hkv, ps_log2;
    int64_t num_pages;
    int num_first, num_recent;
    const float *acc;
    float *acc_out;
    const int32_t *rows;
    int64_t num_rows, acc_stride;
    int32_t *kept;
    int64_t max_keep;
    int32_t *new_lens;
    int32_t *dev_status;
};

// What is to be done for sequence b.  n < 0: nothing; *bits says why.
struct Plan {
    int L, n;
    int64_t row;
};
__device__ __forceinline__ Plan plan_of(const Args &a, int b, int *bits) {
    Plan p;
    p.L = a.seq_lens[b];
    const int keep = a.keep_lens[b];
    p.row = a.rows ? a.rows[b] : b;
    p.n = keep < p.L ? keep : p.L;
    *bits = 0;
    if (p.row < 0) {
        p.n = -1;
    } else if (p.row >= a.num_rows) {
        p.n = -1;
        *bits = PKV_DEV_BAD_ROW;
    } else if (p.L < 0 || keep < 0 || p.L > (a.pt_stride << a.ps_log2) || p.L > a.acc_stride ||
               p.n > a.max_keep || p.n > (a.pt_out_stride << a.ps_log2)) {
        p.n = -1;
        *bits = PKV_DEV_BAD_SEQLEN;
    }
    return p;
}

// ---------------------------------------------------------------- select
constexpr int kBins = 2048;
constexpr int kMaxCached = 48 * 1024;           // sums of a row kept in shared memory (192 KB)
static_assert(kMaxCached <= 32 * kBins, "a flag word per 32 positions in the histogram's place");
constexpr int kCandidates = 256;                // few enough to rank against each other

// Bits of a float such that unsigned order is the order of the values, with 0
// and -0 equal and NaN below everything.
__device__ __forceinline__ uint32_t order_key(float x) {
    const int u = __float_as_int(x + 0.0f);  // -0 + 0 = 0
    return isnan(x) ? 0u : static_cast<uint32_t>(u ^ ((u >> 31) | 0x80000000));
}

__device__ __forceinline__ int warp_scan(int v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += n;
    }
    return v;
}

// One (sequence, KV head), p.n > 0, by the THREADS threads of a block.  s_val: the
// row's sums, when it has at most `cached`.
template <int THREADS>
__device__ __forceinline__ void select_row(const Args &a, const Plan &p, int b, int g, int cached, float *s_val) {
    constexpr int WARPS = THREADS / 32;
    __shared__ __align__(16) int s_hist[kBins];
    __shared__ unsigned long long s_candidate[kCandidates];
    __shared__ int s_warp[WARPS];
    __shared__ int s_digit, s_above, s_count, s_candidates;
    __shared__ uint32_t s_threshold;
    __shared__ int s_cut;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < kBins / 4; i += THREADS) reinterpret_cast<int4 *>(s_hist)[i] = make_int4(0, 0, 0, 0);
    if (tid == 0) s_candidates = 0;
    const int L = p.L, n = p.n;
    const int first = min(a.num_first, n);
    const int recent = min(a.num_recent, n - first);
    const int want = n - first - recent;  // keys to choose from [first, end)
    const int end = L - recent;
    const float *src = a.acc + (p.row * a.Hkv + g) * a.acc_stride;
    float *dst = a.acc_out + (p.row * a.Hkv + g) * a.acc_stride;
    int32_t *kept = a.kept + ((int64_t)b * a.Hkv + g) * a.max_keep;
    const bool choose = want > 0 && want < end - first;
    __syncthreads();  // the histogram is clear

    // the row's sums to shared memory, and the histogram of the top bits of the
    // ones to choose from, in one pass
    auto count_top = [&](float x, int j) {
        if (choose && static_cast<unsigned>(j - first) < static_cast<unsigned>(end - first))
            atomicAdd(&s_hist[order_key(x) >> 21], 1);
    };
    const bool in_smem = L <= cached;
    if (in_smem && (reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
        constexpr int AHEAD = 2;
        for (int j0 = 4 * tid; j0 < L; j0 += AHEAD * 4 * THREADS) {
            float4 x[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int j = j0 + i * 4 * THREADS;
                if (j + 3 < L) {
                    x[i] = *reinterpret_cast<const float4 *>(src + j);
                } else {
                    x[i].x = j < L ? src[j] : 0.f;
                    x[i].y = j + 1 < L ? src[j + 1] : 0.f;
                    x[i].z = j + 2 < L ? src[j + 2] : 0.f;
                    x[i].w = 0.f;
                }
            }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int j = j0 + i * 4 * THREADS;
                const float v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (j + e < L) {
                        s_val[j + e] = v[e];
                        count_top(v[e], j + e);
                    }
            }
        }
        src = s_val;
    } else {
#pragma unroll 8
        for (int j = tid; j < L; j += THREADS) {
            const float x = src[j];
            if (in_smem) s_val[j] = x;
            count_top(x, j);
        }
        if (in_smem) src = s_val;
    }
    __syncthreads();

    // A key stays when it is above `threshold`, or equal to it and not past
    // position `cut`.
    uint32_t threshold = 0u;  // everything stays
    int cut = L;
    if (want == 0) {
        threshold = 0xffffffffu;  // no float has this key
    } else if (choose) {
        uint32_t prefix = 0u, mask = 0u;
        int left = want;  // how many of the keys with this prefix stay
        for (int pass = 0;; ++pass) {
            // bits of this pass: 31..21, 20..10, 9..0 (counted already in pass 0)
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const uint32_t dmask = pass < 2 ? 0x7ffu : 0x3ffu;
            if (pass > 0) {
                for (int i = tid; i < kBins / 4; i += THREADS)
                    reinterpret_cast<int4 *>(s_hist)[i] = make_int4(0, 0, 0, 0);
                __syncthreads();
                for (int j = first + tid; j < end; j += THREADS) {
                    const uint32_t key = order_key(src[j]);
                    if ((key & mask) == prefix) atomicAdd(&s_hist[(key >> shift) & dmask], 1);
                }
                __syncthreads();
            }
            // bins from the top: a thread sums a run of them and finds whether the
            // left-th key falls into it
            constexpr int RUN = kBins / THREADS;
            const int top = kBins - 1 - tid * RUN;
            int mine = 0;
#pragma unroll
            for (int i = 0; i < RUN; ++i) mine += s_hist[top - i];
            int before = warp_scan(mine, lane);
            if (lane == 31) s_warp[warp] = before;
            __syncthreads();
            const int total = lane < WARPS ? s_warp[lane] : 0;
            const int base = __shfl_sync(0xffffffffu, warp_scan(total, lane) - total, warp);
            before += base - mine;  // keys in the runs above
            if (before < left && before + mine >= left) {
                int sum = before, bin = top;
                while (sum + s_hist[bin] < left) sum += s_hist[bin--];
                s_digit = bin;
                s_above = sum;
                s_count = s_hist[bin];
            }
            __syncthreads();
            prefix |= static_cast<uint32_t>(s_digit) << shift;
            mask |= dmask << shift;
            left -= s_above;
            const int count = s_count;  // keys with the prefix
            if (count == left) {        // all of them stay
                if (prefix != 0u) threshold = prefix - 1u, cut = -1;
                break;
            }
            if (count <= kCandidates) {
                // few enough: rank them against each other, heavier and earlier first;
                // the left-th is the last that stays
                for (int j = first + tid; j < end; j += THREADS) {
                    const uint32_t key = order_key(src[j]);
                    if ((key & mask) == prefix) {
                        const int i = atomicAdd(&s_candidates, 1);
                        if (i < kCandidates)  // (always, unless the sums change meanwhile)
                            s_candidate[i] = (static_cast<unsigned long long>(key) << 32) | ~static_cast<uint32_t>(j);
                    }
                }
                __syncthreads();
                for (int i = tid; i < count; i += THREADS) {
                    const unsigned long long me = s_candidate[i];
                    int rank = 0;  // up to this one, itself included
#pragma unroll 4
                    for (int o = 0; o < count; ++o) rank += s_candidate[o] >= me;
                    if (rank == left) {  // one candidate
                        s_threshold = static_cast<uint32_t>(me >> 32);
                        s_cut = static_cast<int>(~static_cast<uint32_t>(me));
                    }
                }
                __syncthreads();
                threshold = s_threshold;
                cut = s_cut;
                break;
            }
            if (pass == 2) {
                // the prefix is the whole key, and more keys are equal to it than the
                // list holds: find the left-th in order
                threshold = prefix;
                int seen = 0;
                for (int j0 = first; seen < left && j0 < end; j0 += THREADS) {
                    const int j = j0 + tid;
                    const bool is = j < end && order_key(src[j]) == prefix;
                    const unsigned ballot = __ballot_sync(0xffffffffu, is);
                    if (lane == 0) s_warp[warp] = __popc(ballot);
                    __syncthreads();
                    int at = seen + __popc(ballot & (0xffffffffu >> (31 - lane)));
                    for (int w = 0; w < WARPS; ++w) {
                        if (w < warp) at += s_warp[w];
                        seen += s_warp[w];
                    }
                    if (is && at == left) s_cut = j;
                    __syncthreads();
                }
                cut = s_cut;
                break;
            }
        }
    }

    // Kept positions in order get the next place.
    auto stays = [&](float x, int j) {
        const uint32_t key = order_key(x);
        return (j < L && (j < first || j >= end)) || (j < end && (key > threshold || (key == threshold && j <= cut)));
    };
    const unsigned below = (1u << lane) - 1u;
    __syncthreads();
    if (in_smem) {
        // A warp takes a run of 32-position groups: it counts the kept ones and keeps
        // a word of flags per group, and writes them once the runs before are counted.
        const int groups = (L + 31) / 32, run = (groups + WARPS - 1) / WARPS;
        const int g0 = min(groups, warp * run), g1 = min(groups, g0 + run);
        unsigned *flags = reinterpret_cast<unsigned *>(s_hist);
        int count = 0;
#pragma unroll 4
        for (int i = g0; i < g1; ++i) {
            const int j = 32 * i + lane;
            const unsigned word = __ballot_sync(0xffffffffu, stays(j < L ? s_val[j] : 0.f, j));
            if (lane == 0) flags[i] = word;
            count += __popc(word);
        }
        if (lane == 0) s_warp[warp] = count;
        __syncthreads();
        const int warps = lane < WARPS ? s_warp[lane] : 0;
        int at = __shfl_sync(0xffffffffu, warp_scan(warps, lane) - warps, warp);
#pragma unroll 4
        for (int i = g0; i < g1; ++i) {
            const unsigned word = flags[i];
            if ((word >> lane) & 1u) {
                const int to = at + __popc(word & below);
                kept[to] = 32 * i + lane;
                dst[to] = s_val[32 * i + lane];
            }
            at += __popc(word);
        }
    } else {
        // from and possibly back to global memory: every value of a step is read
        // before any is written, and none is written past its old place.  (Sums that
        // another call changes meanwhile give any choice, but no place past n.)
        int base = 0;
        for (int j0 = 0; j0 < L; j0 += THREADS) {
            const int j = j0 + tid;
            const float x = j < L ? src[j] : 0.f;
            const unsigned word = __ballot_sync(0xffffffffu, stays(x, j));
            if (lane == 0) s_warp[warp] = __popc(word);
            __syncthreads();
            const int warps = lane < WARPS ? s_warp[lane] : 0;
            const int sums = warp_scan(warps, lane);
            const int to = base + __shfl_sync(0xffffffffu, sums - warps, warp) + __popc(word & below);
            if (((word >> lane) & 1u) && to < n) {
                kept[to] = j;
                dst[to] = x;
            }
            base += __shfl_sync(0xffffffffu, sums, WARPS - 1);
            __syncthreads();
        }
    }
}

// The plan of sequence b, its new length written and its errors reported by one
// thread of the grid.
__device__ __forceinline__ Plan announce(const Args &a, int b, bool mine) {
    int bits;
    const Plan p = plan_of(a, b, &bits);
    if (mine) {
        a.new_lens[b] = p.n < 0 ? p.L : p.n;
        if (bits && a.dev_status) atomicOr(a.dev_status, bits);
    }
    return p;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS, 2048 / THREADS) select_kernel(const Args a, int cached) {
    extern __shared__ float s_val[];
    grid_dependency_wait();  // the sums come from the kernel before
    allow_dependents();
    const int g = blockIdx.x, b = blockIdx.y;
    const Plan p = announce(a, b, g == 0 && threadIdx.x == 0);
    if (p.n > 0) select_row<THREADS>(a, p, b, g, cached, s_val);
}

// ---------------------------------------------------------------- move
// A cluster of blocks moves the K or the V rows of one (sequence, KV head), in
// rounds: every warp copies its rows of the next round to shared memory with
// cp.async, waits for those of the current one, the cluster meets, and every
// warp stores its current rows.  The meeting is what makes moving in place right
// (see the top of the file); the next round's rows, which nothing stored so far
// or in this round can hit, are in flight meanwhile.  One lane per row finds its
// slots, a round ahead, and the positions two rounds ahead; the lanes that copy
// the row's pieces get them by shuffle.
constexpr int kMoveWarps = 8;
constexpr int kMoveThreads = kMoveWarps * 32;
constexpr int kPortableCluster = 8, kLargeCluster = 16;
// 16-byte pieces per lane and round: 4 where many blocks share an SM, as many as a warp
// has lanes to look rows up where they do not (few rows: the rounds' latency counts).
constexpr int kSteps = 4;
constexpr int many_steps(int D) { return 32 / (32 / (D / 8)); }
constexpr int move_smem(int steps) { return 2 * kMoveThreads * steps * 16; }

// All threads of the cluster have come this far.  Relaxed: no data passes between the
// blocks, it only keeps the stores of a round behind its loads.  Those are complete
// before any thread arrives: cp.async.wait_group has returned, so their values lie in
// shared memory, and a store that is issued after the barrier cannot change them.  (A
// release would also wait until the stores of the round before are visible: 208.7 ->
// 223.2 us for the batch above, 61.8 -> 67.6 us for 8 sequences of 16-32 K keys.)
__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// The rows of one (sequence, KV head) and tensor, p.n > 0, by `ranks` blocks of a
// cluster (alone: the block is a cluster of its own).  s_rows: move_smem(STEPS) bytes.
template <int D, int STEPS>
__device__ __forceinline__ void move_rows(const Args &a, const Plan &p, int b, int g, uint4 *tensor, int rank, int ranks,
                                          bool alone, uint4 *s_rows) {
    constexpr int VEC = D / 8;                       // 16-byte pieces of a row
    constexpr int PER_STEP = 32 / VEC;               // rows a warp copies at once
    constexpr int WARP_ROWS = PER_STEP * STEPS; // rows of a warp per round
    static_assert(WARP_ROWS <= 32, "one lane per row");
    constexpr int BLOCK_ROWS = WARP_ROWS * kMoveWarps;
    // s_rows: [2 rounds][steps][threads], a lane stores what it loaded
    uint4 *cache = tensor + (int64_t)g * VEC;
    const int32_t *kept = a.kept + ((int64_t)b * a.Hkv + g) * a.max_keep;
    const int32_t *pt = a.page_table + (int64_t)b * a.pt_stride;
    const int32_t *pt_out = a.page_table_out + (int64_t)b * a.pt_out_stride;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int vec = lane % VEC, sub = lane / VEC;
    const int ps_mask = (1 << a.ps_log2) - 1;
    const int64_t row_vecs = (int64_t)a.Hkv * VEC;
    const int64_t step = (int64_t)ranks * BLOCK_ROWS;
    // the row that this lane looks up in the round that starts at i0
    const int mine = rank * BLOCK_ROWS + warp * WARP_ROWS + lane;
    bool bad = false;
    auto position = [&](int64_t i0) -> int {
        const int j = lane < WARP_ROWS && i0 + mine < p.n ? kept[i0 + mine] : -1;
        return j < p.L ? j : -1;  // (a position, unless two sequences share a row of sums)
    };
    // slots of position j, the kept key i0 + mine; to < 0: nothing to move
    auto find = [&](int64_t i0, int j, int &from, int &to) {
        from = 0;
        to = -1;
        if (j < 0) return;
        const int i = static_cast<int>(i0 + mine);
        const int64_t from_page = pt[j >> a.ps_log2], to_page = pt_out[i >> a.ps_log2];
        if (from_page < 0 || from_page >= a.num_pages || to_page < 0 || to_page >= a.num_pages) {
            bad = true;
            return;
        }
        from = static_cast<int>((from_page << a.ps_log2) + (j & ps_mask));
        const int slot = static_cast<int>((to_page << a.ps_log2) + (i & ps_mask));
        if (from != slot) to = slot;
    };
    auto load = [&](int buf, int from, int to) {
        uint4 *rows = s_rows + buf * STEPS * kMoveThreads + threadIdx.x;
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            const int f = __shfl_sync(0xffffffffu, from, k * PER_STEP + sub);
            const int t = __shfl_sync(0xffffffffu, to, k * PER_STEP + sub);
            if (t >= 0) cp_async16(smem_u32(rows + k * kMoveThreads), cache + f * row_vecs + vec, 16);
        }
        cp_async_commit();
    };
    int from, to, next_from, next_to;
    find(0, position(0), from, to);
    load(0, from, to);
    int j = position(step);
    find(step, j, next_from, next_to);
    j = position(2 * step);
    int buf = 0;
    for (int64_t i0 = 0; i0 < p.n; i0 += step, buf ^= 1) {
        load(buf ^ 1, next_from, next_to);
        const int to_now = to;
        to = next_to;
        find(i0 + 2 * step, j, next_from, next_to);
        j = position(i0 + 3 * step);
        cp_async_wait<1>();  // this round's rows
        if (alone)
            __syncthreads();
        else
            cluster_meet();
        const uint4 *rows = s_rows + buf * STEPS * kMoveThreads + threadIdx.x;
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            const int t = __shfl_sync(0xffffffffu, to_now, k * PER_STEP + sub);
            if (t >= 0) cache[t * row_vecs + vec] = rows[k * kMoveThreads];
        }
    }
    cp_async_wait<0>();
    if (bad && a.dev_status) atomicOr(a.dev_status, PKV_DEV_BAD_PAGE);
}

template <int D, int STEPS>
__global__ void __launch_bounds__(kMoveThreads)
    move_kernel(const Args a, uint4 *k_cache, uint4 *v_cache, int ranks) {
    extern __shared__ uint4 s_rows[];
    grid_dependency_wait();  // kept comes from select_kernel
    allow_dependents();
    const int b = blockIdx.y;
    int bits;
    const Plan p = plan_of(a, b, &bits);
    if (p.n > 0)  // the same for the whole cluster
        move_rows<D, STEPS>(a, p, b, blockIdx.x / ranks, blockIdx.z ? v_cache : k_cache, blockIdx.x % ranks, ranks, ranks == 1,
                     s_rows);
}

// ---------------------------------------------------------------- both
// Little to do: one launch, a cluster of 2 * ranks blocks per (sequence, KV head)
// whose first block selects, and which then moves K with one half and V with the
// other.
constexpr int kFusedRow = 2048;
static_assert(kFusedRow * 4 <= move_smem(kSteps), "the row's sums lie where rows are staged later");

template <int D>
__global__ void __launch_bounds__(kMoveThreads)
    evict_kernel(const Args a, uint4 *k_cache, uint4 *v_cache, int cached, int ranks) {
    extern __shared__ uint4 s_rows[];
    grid_dependency_wait();  // the sums come from the kernel before
    allow_dependents();
    const int me = blockIdx.x % (2 * ranks), g = blockIdx.x / (2 * ranks), b = blockIdx.y;
    const Plan p = announce(a, b, blockIdx.x == 0 && threadIdx.x == 0);
    if (p.n <= 0) return;  // the whole cluster
    if (me == 0) select_row<kMoveThreads>(a, p, b, g, cached, reinterpret_cast<float *>(s_rows));
    // the first block's kept positions are there for all
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    move_rows<D, kSteps>(a, p, b, g, me < ranks ? k_cache : v_cache, me % ranks, ranks, false, s_rows);
}

// Allow the kernels their shared memory and clusters, once per device; the largest cluster
// of move_kernel, 0: an error.
static int prepare(const pkv_host::DeviceInfo &dev) {
    static std::mutex mu;
    static int largest[64];
    std::lock_guard<std::mutex> lk(mu);
    int &n = largest[dev.device];
    if (n) return n;
    bool ok = true, large = true;
    auto allow = [&](auto *kernel, int smem) {
        ok &= cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess;
    };
    // clusters of 16 where the device has room for one
    auto allow_large = [&](auto *kernel, int smem) {
        allow(kernel, smem);
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = kLargeCluster;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kLargeCluster);
        cfg.blockDim = dim3(kMoveThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        large &= cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                 cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) == cudaSuccess && clusters > 0;
    };
    allow(select_kernel<256>, kMaxCached * 4);
    allow(select_kernel<512>, kMaxCached * 4);
    allow(select_kernel<1024>, kMaxCached * 4);
    allow_large(move_kernel<128, kSteps>, move_smem(kSteps));
    allow_large(move_kernel<64, kSteps>, move_smem(kSteps));
    allow_large(move_kernel<128, many_steps(128)>, move_smem(many_steps(128)));
    allow_large(move_kernel<64, many_steps(64)>, move_smem(many_steps(64)));
    if (ok) n = large ? kLargeCluster : kPortableCluster;
    return n;
}

static bool overlap(const void *p, size_t np, const void *q, size_t nq) {
    if (!p || !q) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + nq && b < a + np;
}

}  // namespace evict
}  // namespace pkv

extern "C" pkv_status pkv_kv_evict(pkv_bf16 *k_cache, pkv_bf16 *v_cache, const int32_t *page_table,
                                   int64_t page_table_stride, const int32_t *page_table_out,
                                   int64_t page_table_out_stride, const int32_t *seq_lens,
                                   const int32_t *keep_lens, int batch, int num_kv_heads,
                                   int head_dim, int page_size, int64_t num_pages, int num_first,
                                   int num_recent, const float *acc, float *acc_out,
                                   const int32_t *acc_rows, int64_t num_acc_rows,
                                   int64_t acc_stride, int32_t *kept, int64_t max_keep,
                                   int32_t *new_seq_lens, int32_t *dev_status, void *stream) {
    using namespace pkv::evict;
    if (batch < 0 || num_kv_heads <= 0 || num_pages <= 0 || page_size <= 0 || page_table_stride < 0 ||
        page_table_out_stride < 0 || num_first < 0 || num_recent < 0 || num_acc_rows < 0 ||
        acc_stride < 0 || max_keep < 0)
        return PKV_EINVAL;
    if (batch == 0) return PKV_OK;
    if (!k_cache || !v_cache || !page_table || !page_table_out || !seq_lens || !keep_lens || !acc ||
        !acc_out || !kept || !new_seq_lens || (!acc_rows && num_acc_rows < batch))
        return PKV_EINVAL;
    if (head_dim != 64 && head_dim != 128) return PKV_EUNSUPPORTED;
    if ((page_size & (page_size - 1)) != 0 || page_size > 256) return PKV_EUNSUPPORTED;
    if (batch > 4096 || num_kv_heads > 65535) return PKV_EUNSUPPORTED;
    if (num_pages * page_size > 0x7fffffffll || page_table_stride > 0x7fffffffll ||
        page_table_out_stride > 0x7fffffffll)
        return PKV_EUNSUPPORTED;
    if (!pkv_host::aligned16(k_cache) || !pkv_host::aligned16(v_cache) ||
        (reinterpret_cast<uintptr_t>(acc) & 3u) || (reinterpret_cast<uintptr_t>(acc_out) & 3u))
        return PKV_EINVAL;
    if (acc_out != acc) {  // in place, or somewhere else altogether
        const size_t bytes = static_cast<size_t>(num_acc_rows) * num_kv_heads * acc_stride * 4;
        if (overlap(acc, bytes, acc_out, bytes)) return PKV_EINVAL;
    }
    // the kernels read these while the new lengths are written
    const size_t ints = static_cast<size_t>(batch) * 4;
    if (overlap(new_seq_lens, ints, seq_lens, ints) || overlap(new_seq_lens, ints, keep_lens, ints) ||
        overlap(new_seq_lens, ints, acc_rows, ints))
        return PKV_EINVAL;
    pkv_host::DeviceInfo dev;
    if (!pkv_host::current_device(&dev)) return PKV_ECUDA;
    int ps_log2 = 0;
    while ((1 << ps_log2) < page_size) ++ps_log2;
    const Args a{page_table, page_table_out, page_table_stride, page_table_out_stride, seq_lens,
                 keep_lens, num_kv_heads, ps_log2, num_pages, num_first, num_recent, acc, acc_out,
                 acc_rows, num_acc_rows, acc_stride, kept, max_keep, new_seq_lens, dev_status};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int cached = static_cast<int>(acc_stride < kMaxCached ? acc_stride : kMaxCached);
    const int largest = prepare(dev);
    if (!largest) return PKV_ECUDA;
    const int64_t rows = (int64_t)batch * num_kv_heads;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kMoveThreads);
    cfg.dynamicSmemBytes = move_smem(kSteps);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    uint4 *k = reinterpret_cast<uint4 *>(k_cache), *v = reinterpret_cast<uint4 *>(v_cache);
    // One launch where the second would cost more than the blocks that wait for their
    // cluster's first.  Measured, one launch against two, 8 KV heads, half kept: rows of
    // 512 keys at most, 4 sequences 6.2 / 7.9 us, 32 sequences 19.4 / 20.1; rows of 2048,
    // 1 sequence 9.5 / 9.9, 4 sequences 12.2 / 12.7, 16 sequences 31.8 / 30.3; rows of
    // 4096, 32 sequences 92.8 / 86.0.
    if (acc_stride <= 512 || (acc_stride <= kFusedRow && rows <= 64)) {
        // blocks per tensor: enough for 8 on every SM
        int ranks = 1;
        while (2 * ranks < kPortableCluster && 2 * rows * ranks < 8ll * dev.sm_count) ranks *= 2;
        cfg.gridDim = dim3(static_cast<unsigned>(num_kv_heads * 2 * ranks), batch);
        attr[1].val.clusterDim.x = 2 * ranks;
        return cudaLaunchKernelEx(&cfg, head_dim == 128 ? evict_kernel<128> : evict_kernel<64>, a, k, v, cached,
                                  ranks) == cudaSuccess
                   ? PKV_OK
                   : PKV_ECUDA;
    }
    // a block's fixed work grows with its threads, its time per key falls
    const int threads = cached > 16384 ? 1024 : cached > 4096 ? 512 : 256;
    if (pkv_host::launch_dependent(threads == 256   ? select_kernel<256>
                                   : threads == 512 ? select_kernel<512>
                                                    : select_kernel<1024>,
                                   dim3(num_kv_heads, batch), dim3(threads),
                                   static_cast<size_t>(cached) * 4, st, a, cached) != cudaSuccess)
        return PKV_ECUDA;
    // blocks per (sequence, KV head, tensor): enough for 16 on every SM.  (One sequence of
    // 32000 keys, 8 KV heads, half kept: 75 us with clusters of 8 at most, 62 us with 16.)
    int ranks = 1;
    while (ranks < largest && 2 * rows * ranks < 16ll * dev.sm_count) ranks *= 2;
    cfg.gridDim = dim3(static_cast<unsigned>(num_kv_heads * ranks), batch, 2);
    attr[1].val.clusterDim.x = ranks;
    auto move = head_dim == 128 ? move_kernel<128, kSteps> : move_kernel<64, kSteps>;
    if (2 * rows * ranks <= dev.sm_count) {  // a block per SM at most
        move = head_dim == 128 ? move_kernel<128, many_steps(128)> : move_kernel<64, many_steps(64)>;
        cfg.dynamicSmemBytes = move_smem(many_steps(head_dim));
    }
    return cudaLaunchKernelEx(&cfg, move, a, k, v, ranks) == cudaSuccess ? PKV_OK : PKV_ECUDA;
}
