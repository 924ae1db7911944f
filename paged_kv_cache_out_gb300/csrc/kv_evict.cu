// kv_evict.cu -- shorten cached sequences: per (sequence, KV head) keep the
// first, the last and the heaviest keys, and move them to the front.
//
// miniVLLM "Engine Architecture" (allocate_kv_cache: the pool; block_tables map
// a sequence's positions to pages).  The pages of the source describe no
// eviction; a sequence that must shrink keeps the keys whose accumulated
// softmax weight (pkv_paged_decode_attn_weights) is largest.
//
// Two kernels:
//  * select: one block per (sequence, KV head).  The n - first - recent heaviest
//    keys are found by a radix select on the sums' bits: three histogram passes
//    (11, 11 and 10 bits, high to low) find the weight of the last key that
//    stays and how many of that weight stay; a last pass over the positions in
//    order writes the kept ones and moves their sums.
//  * move: the K and V rows of the kept positions.  kept[i] >= i, so a block that
//    takes the kept rows in rising order and loads a group of them before it
//    stores any of the group never overwrites a row that is still to be read:
//    the rows stored so far lie below the group, the rows to come at or above it.
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
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kItems = 8;                       // positions per thread and step of the last pass
constexpr int kBins = 2048;
constexpr int kMaxCached = 48 * 1024;           // sums of a row kept in shared memory (192 KB)

// Bits of a float such that unsigned order is the order of the values, with 0
// and -0 equal and NaN below everything.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (isnan(x)) return 0u;
    const uint32_t u = __float_as_uint(x + 0.0f);  // -0 + 0 = 0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int warp_scan(int v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += n;
    }
    return v;
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const Args a, int cached) {
    extern __shared__ float s_val[];  // the row's sums, when it has at most `cached`
    __shared__ int s_hist[kBins];
    __shared__ int s_warp[kSelWarps];
    __shared__ int s_digit, s_above;
    const int g = blockIdx.x, b = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependency_wait();  // the sums come from the kernel before
    allow_dependents();
    int bits;
    const Plan p = plan_of(a, b, &bits);
    if (g == 0 && tid == 0) {
        a.new_lens[b] = p.n < 0 ? a.seq_lens[b] : p.n;
        if (bits && a.dev_status) atomicOr(a.dev_status, bits);
    }
    if (p.n <= 0) return;
    const int L = p.L, n = p.n;
    const int first = min(a.num_first, n);
    const int recent = min(a.num_recent, n - first);
    const int want = n - first - recent;  // keys to choose from [first, end)
    const int end = L - recent;
    const float *src = a.acc + (p.row * a.Hkv + g) * a.acc_stride;
    float *dst = a.acc_out + (p.row * a.Hkv + g) * a.acc_stride;
    int32_t *kept = a.kept + ((int64_t)b * a.Hkv + g) * a.max_keep;
    const bool in_smem = L <= cached;
    if (in_smem) {
        for (int j = tid; j < L; j += kSelThreads) s_val[j] = src[j];
        src = s_val;
    }

    // the order key of the last key that stays, and how many keys with that
    // order key stay (the first ones)
    uint32_t threshold = 0u;  // want == end - first: every key is at or above it
    int equal = 0x7fffffff;
    if (want == 0) {
        threshold = 0xffffffffu;  // no float has this key
        equal = 0;
    } else if (want < end - first) {
        uint32_t prefix = 0u, mask = 0u;
        int left = want;  // how many of the keys with this prefix stay
        const int shifts[3] = {21, 10, 0}, widths[3] = {11, 11, 10};
#pragma unroll
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = shifts[pass];
            const uint32_t dmask = (1u << widths[pass]) - 1u;
            for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0;
            __syncthreads();
            for (int j = first + tid; j < end; j += kSelThreads) {
                const uint32_t key = order_key(src[j]);
                if ((key & mask) == prefix) atomicAdd(&s_hist[(key >> shift) & dmask], 1);
            }
            __syncthreads();
            // from the top: thread t sums bins of one run, and finds whether the
            // left-th key falls into it
            constexpr int RUN = kBins / kSelThreads;
            const int top = kBins - 1 - tid * RUN;
            int mine = 0;
#pragma unroll
            for (int i = 0; i < RUN; ++i) mine += s_hist[top - i];
            int before = warp_scan(mine, lane);
            if (lane == 31) s_warp[warp] = before;
            __syncthreads();
            int base = 0;
            for (int w = 0; w < warp; ++w) base += s_warp[w];
            before += base - mine;  // keys in the runs above
            if (before < left && before + mine >= left) {
                int sum = before, bin = top;
                while (sum + s_hist[bin] < left) sum += s_hist[bin--];
                s_digit = bin;
                s_above = sum;
            }
            __syncthreads();
            prefix |= static_cast<uint32_t>(s_digit) << shift;
            mask |= dmask << shift;
            left -= s_above;
        }
        threshold = prefix;
        equal = left;
    }

    // positions in order: kept ones get the next place.  A warp takes
    // kItems * 32 consecutive positions of a step.
    int base_more = 0, base_equal = 0;  // keys above the threshold / equal to it so far
    __syncthreads();
    for (int j0 = 0; j0 < L; j0 += kSelThreads * kItems) {
        float val[kItems];
        unsigned more[kItems], same[kItems];
        int nm = 0, ne = 0;
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int j = j0 + (warp * kItems + i) * 32 + lane;
            bool is_more = false, is_same = false;
            val[i] = 0.f;
            if (j < L) {
                val[i] = src[j];
                const bool safe = j < first || j >= end;
                const uint32_t key = order_key(val[i]);
                is_more = safe || key > threshold;
                is_same = !safe && key == threshold;
            }
            more[i] = __ballot_sync(0xffffffffu, is_more);
            same[i] = __ballot_sync(0xffffffffu, is_same);
            nm += __popc(more[i]);
            ne += __popc(same[i]);
        }
        if (lane == 0) s_hist[warp] = nm, s_hist[kSelWarps + warp] = ne;
        __syncthreads();  // also: every value of this step is in registers
        int before_more = base_more, before_same = base_equal;
#pragma unroll
        for (int w = 0; w < kSelWarps; ++w) {
            const int cm = s_hist[w], ce = s_hist[kSelWarps + w];
            if (w < warp) before_more += cm, before_same += ce;
            base_more += cm, base_equal += ce;
        }
        const unsigned below = (1u << lane) - 1u;
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int j = j0 + (warp * kItems + i) * 32 + lane;
            const int m = before_more + __popc(more[i] & below);
            const int e = before_same + __popc(same[i] & below);
            const bool is_more = (more[i] >> lane) & 1u, is_same = (same[i] >> lane) & 1u;
            if (is_more || (is_same && e < equal)) {
                const int at = m + min(e, equal);
                kept[at] = j;
                dst[at] = val[i];
            }
            before_more += __popc(more[i]);
            before_same += __popc(same[i]);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- move
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 8;  // 16-byte pieces per thread and group

template <int D>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const Args a, uint4 *k_cache, uint4 *v_cache) {
    constexpr int VEC = D / 8;                     // 16-byte pieces of a row
    constexpr int ROWS = kMoveThreads / VEC;       // rows a block touches at once
    grid_dependency_wait();  // kept comes from select_kernel
    allow_dependents();
    const int g = blockIdx.x, b = blockIdx.y;
    uint4 *cache = blockIdx.z ? v_cache : k_cache;
    int bits;
    const Plan p = plan_of(a, b, &bits);
    if (p.n <= 0) return;
    const int32_t *kept = a.kept + ((int64_t)b * a.Hkv + g) * a.max_keep;
    const int32_t *pt = a.page_table + (int64_t)b * a.pt_stride;
    const int32_t *pt_out = a.page_table_out + (int64_t)b * a.pt_out_stride;
    const int vec = threadIdx.x % VEC, r = threadIdx.x / VEC;
    const int ps_mask = (1 << a.ps_log2) - 1;
    bool bad = false;
    for (int i0 = 0; i0 < p.n; i0 += ROWS * kMoveRows) {
        uint4 buf[kMoveRows];
        int64_t to[kMoveRows];
#pragma unroll
        for (int u = 0; u < kMoveRows; ++u) {
            const int i = i0 + u * ROWS + r;
            to[u] = -1;
            if (i < p.n) {
                const int j = kept[i];
                const int64_t from_page = pt[j >> a.ps_log2], to_page = pt_out[i >> a.ps_log2];
                if (from_page < 0 || from_page >= a.num_pages || to_page < 0 || to_page >= a.num_pages) {
                    bad = true;
                } else {
                    const int64_t from = (from_page << a.ps_log2) + (j & ps_mask);
                    const int64_t slot = (to_page << a.ps_log2) + (i & ps_mask);
                    if (from != slot) {
                        to[u] = (slot * a.Hkv + g) * VEC + vec;
                        buf[u] = cache[(from * a.Hkv + g) * VEC + vec];
                    }
                }
            }
        }
        __syncthreads();  // the whole group is loaded
#pragma unroll
        for (int u = 0; u < kMoveRows; ++u)
            if (to[u] >= 0) cache[to[u]] = buf[u];
    }
    if (bad && a.dev_status) atomicOr(a.dev_status, PKV_DEV_BAD_PAGE);
}

// Allow select_kernel its shared memory, once per device.
static bool prepare(const pkv_host::DeviceInfo &dev) {
    static std::mutex mu;
    static bool ready[64];
    std::lock_guard<std::mutex> lk(mu);
    if (!ready[dev.device] &&
        cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMaxCached * 4) != cudaSuccess)
        return false;
    return ready[dev.device] = true;
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
    if (!prepare(dev)) return PKV_ECUDA;
    if (pkv_host::launch_dependent(select_kernel, dim3(num_kv_heads, batch), dim3(kSelThreads),
                                   static_cast<size_t>(cached) * 4, st, a, cached) != cudaSuccess)
        return PKV_ECUDA;
    auto move = head_dim == 128 ? move_kernel<128> : move_kernel<64>;
    if (pkv_host::launch_dependent(move, dim3(num_kv_heads, batch, 2), dim3(kMoveThreads), 0, st, a,
                                   reinterpret_cast<uint4 *>(k_cache),
                                   reinterpret_cast<uint4 *>(v_cache)) != cudaSuccess)
        return PKV_ECUDA;
    return PKV_OK;
}
