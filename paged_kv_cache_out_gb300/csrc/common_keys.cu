// common_keys.cu -- pkv_paged_decode_attn_shared and pkv_paged_cross_attn: the
// kernel that cuts the work into ranges, the kernels that join the partial
// states which common_keys_tiles.cu and common_keys_few.cu leave, and the entry
// points.  A call is four launches (three where no block can have more than 16
// rows), each started early behind the one before: plan (3 us, a chain of
// dependent reads and a sum over the entries), tiles, few rows, join (3-8 us:
// the states that the cut segments left, 28 MB in long cross attention).
//
// zero-to-sglang "Chapter 1 mini-sglang: What an Inference Engine Looks Like",
// the roadmap on prefix caching: requests that begin with the same tokens reuse
// one cached copy of that prefix's KV; miniVLLM "Engine Architecture":
// block_tables may list the same blocks for several sequences.
#include <math.h>

#include <mutex>

#include "common_keys.cuh"

namespace pkv {
namespace ck {

namespace {

// ---------------------------------------------------------------- the plan
// Both kernels' entries, ranges and borders.  Block 0 makes those of the tiles kernel and writes the
// entries, the others each a share of the few-rows kernel's borders; each finds the units of all
// entries for itself (they are few, and it takes no longer than to wait for another's).  Two blocks
// instead of eight: calls 3 us longer.
constexpr int kPlanBlocks = 8;
// ints of shared memory: per entry the units before it, its query tokens and its keys; per sequence
// its group's prefix and first sequence
constexpr int plan_smem(int entries, int batch) { return (3 * entries + 2 * batch) * 4; }

template <int D, int KERNEL, int THREADS>
__device__ __forceinline__ void plan(const Args &a, int part, int parts) {
    extern __shared__ int smem_ints[];
    __shared__ int warp_sum[32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int E = a.op == kCross ? a.batch : a.groups + a.batch;
    int *units_before = smem_ints, *tokens_of = units_before + E, *keys_of = tokens_of + E;
    int *prefix_of = keys_of + E, *first_of = prefix_of + a.batch;
    const bool small = a.ps_log2 < 3;
    const int per = (E + THREADS - 1) / THREADS;
    const int lo = min(E, tid * per), hi = min(E, lo + per);
    if (a.op == kShared && lo < hi && lo >= a.groups)  // on its way while the groups are read
        asm volatile("prefetch.global.L1 [%0];" ::"l"(a.lens + lo - a.groups));
    // groups that do not partition the batch, offsets that run backwards or out of the tokens: no work
    bool bad_parts = false;
    if (a.op == kCross) {
#pragma unroll 1
        for (int e = lo; e < hi; ++e) {
            const int t0 = a.cu[e], t1 = a.cu[e + 1];
            bad_parts |= t0 < 0 || t1 < t0 || t1 > a.tokens || (e == 0 && t0 != 0);
        }
        bad_parts = __syncthreads_or(bad_parts);
    }
    if (a.op == kShared && a.groups > 0) {
#pragma unroll 1
        for (int e = warp; e < a.groups; e += THREADS / 32) {
            const int r0 = a.gstart[e], r1 = a.gstart[e + 1], S = checked_prefix(a, a.glen[e]);
            if (r0 < 0 || r1 <= r0 || r1 > a.batch || (e == 0 && r0 != 0) || (e == a.groups - 1 && r1 != a.batch)) {
                bad_parts = true;
            } else {
#pragma unroll 1
                for (int b = r0 + lane; b < r1; b += 32) prefix_of[b] = S, first_of[b] = r0;
            }
        }
        bad_parts = __syncthreads_or(bad_parts);
    }
    auto entry_at = [&](int e) -> Entry {
        const int b = e - a.groups;
        const bool grouped = a.op == kShared && a.groups > 0 && b >= 0;
        return get_entry(a, e, grouped ? prefix_of[b] : 0, grouped ? first_of[b] : b);
    };
    int local = 0;
    if (!bad_parts)
#pragma unroll 1
        for (int e = lo; e < hi; ++e) {
            const Entry x = entry_at(e);
            if (part == 0 && (KERNEL == kTiles || !a.tiles_run)) {
                a.entries[e] = x;
                const int bits = x.flags >> 8;  // (a decode step's: where its sequences are told of)
                if (a.op == kCross && a.dev_status && bits && x.n > 0) atomicOr(a.dev_status, bits);
                if (a.op == kShared && e >= a.groups && a.dev_status && bits) atomicOr(a.dev_status, bits);
            }
            units_before[e] = local;  // within this thread's, for now
            tokens_of[e] = x.n;
            keys_of[e] = x.kend - x.klo;
            local += blocks_of<D, KERNEL>(a, x.n, x.kend - x.klo, small).per_head * a.Hkv;
        }
    int v = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += n;
    }
    if (lane == 31) warp_sum[warp] = v;
    __syncthreads();
    const int sum = lane < THREADS / 32 ? warp_sum[lane] : 0;
    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? sum : 0) + v - local;
    const int W = __reduce_add_sync(0xffffffffu, sum);
#pragma unroll 1
    for (int e = lo; e < hi; ++e) units_before[e] = bad_parts ? 0 : units_before[e] + before;
    __syncthreads();
    Ranges rg;
    const int n = max(1, min(a.blocks[KERNEL], W / min_units(KERNEL)));
    {  // part of the work in short ranges, so that blocks that fall behind take fewer
        const int rest = W / kShortShare;
        const int more = n < a.blocks[KERNEL] ? 0 : min(short_ranges(KERNEL) * n, rest / kShortUnits);
        if (more < n) rg.set(W, n, n, 0);
        else rg.set(W, n + more, n, max((W - rest) / n - rest / more, 0));
    }
    if (part == 0 && tid == 0) {
        a.counts[KERNEL] = W > 0 ? rg.n : 0;
        if (KERNEL == kFew) *a.next_range = 0;
    }
    if (part == 0 && KERNEL == kFew && bad_parts) {
        const OwnInfo bad = {{-1, 0}, 0, kBad};  // (every row of a decode step is NaN)
        if (a.op == kShared)
            for (int i = tid; i < a.batch * a.Hkv; i += THREADS) a.own[i] = bad;
        if (tid == 0 && a.dev_status)
            atomicOr(a.dev_status, a.op == kShared ? PKV_DEV_BAD_SHARED : PKV_DEV_BAD_CUSEQ);
    }
    if (W == 0) return;
#pragma unroll 1
    for (int k = part * THREADS + tid; k <= rg.n; k += parts * THREADS) {
        Border b = {E, 0, 0, 0, 0, 0, 0, 0};
        const int x = k < rg.n ? rg.start(k) : W - 1;  // (the end lies behind the last entry that has units)
        if (x < W) {
            int e = 0, end = E;  // the last entry that starts at or before x: entries without units come first
            while (end - e > 1) {
                const int mid = (e + end) >> 1;
                if (units_before[mid] <= x) e = mid; else end = mid;
            }
            b.e = e;
            const Blocks bl = blocks_of<D, KERNEL>(a, tokens_of[e], keys_of[e], small);
            const int rel = x - units_before[e], g = rel / bl.per_head, u0 = rel - g * bl.per_head;
            const int m = bl.nblk > 1 ? min(u0 / bl.pair_units, bl.nblk - 1) : 0, u = u0 - m * bl.pair_units;
            const int form = m < bl.nblk - 1 ? (KERNEL == kTiles ? kPair : kFewForm) : bl.last;
            const int w = tile_cost(form, small), lead = lead_cost(form), snap = snap_cost(form), all = w * bl.nk + lead;
            b.seg = g * bl.nblk + m;
            if (k == rg.n) {
                ++b.e;
                b.seg = 0;
            } else if (u > snap && all - u <= snap) {
                ++b.seg;
            } else if (u > snap) {
                b.t = (u - lead + w - 1) / w;
                b.k0 = rg.range_of(x - u + snap);
                b.k1 = rg.range_of(x - u + all - snap - 1);
            }
        }
        a.borders[KERNEL][k] = b;
    }
}

template <int D, int THREADS>
__global__ void __launch_bounds__(THREADS) plan_kernel(const __grid_constant__ Args a) {
    grid_dependency_wait();  // the lengths may come from the kernel before
    allow_dependents();
    if (a.tiles_run && blockIdx.x == 0) plan<D, kTiles, THREADS>(a, 0, 1);
    else plan<D, kFew, THREADS>(a, blockIdx.x - (a.tiles_run ? 1 : 0), gridDim.x - (a.tiles_run ? 1 : 0));
}

constexpr int kJoinThreads = 256;

// Four columns of a row, of the states added so far.
struct Join {
    float mx = kNoKey, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    bool bad = false;
    __device__ __forceinline__ void add(float2 ml, float4 o) {
        bad |= isnan(ml.x);
        const float m = fmaxf(mx, ml.x);
        const float a = ex2(mx - m), b = ex2(ml.x - m);
        mx = m;
        sum = sum * a + ml.y * b;
        acc.x = acc.x * a + o.x * b;
        acc.y = acc.y * a + o.y * b;
        acc.z = acc.z * a + o.z * b;
        acc.w = acc.w * a + o.w * b;
    }
    __device__ __forceinline__ void shuffle(int off) {
        const float2 ml = make_float2(__shfl_xor_sync(0xffffffffu, mx, off), __shfl_xor_sync(0xffffffffu, sum, off));
        const float4 o = make_float4(
            __shfl_xor_sync(0xffffffffu, acc.x, off), __shfl_xor_sync(0xffffffffu, acc.y, off),
            __shfl_xor_sync(0xffffffffu, acc.z, off), __shfl_xor_sync(0xffffffffu, acc.w, off));
        const bool other = __shfl_xor_sync(0xffffffffu, bad ? 1 : 0, off) != 0;
        add(ml, o);
        bad |= other;
    }
    __device__ __forceinline__ uint2 result() const {
        const float inv = 1.f / sum, nan = __int_as_float(0x7fc00000);
        return make_uint2(pack_bf16x2(bad ? nan : acc.x * inv, bad ? nan : acc.y * inv),
                          pack_bf16x2(bad ? nan : acc.z * inv, bad ? nan : acc.w * inv));
    }
};


// kShared: a block per (sequence, KV head): the states of its shared and its own keys.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_shared_kernel(const __grid_constant__ Args a) {
    grid_dependency_wait();
    const int G = 1 << a.g_log2, Hkv = a.Hkv, Hq = Hkv << a.g_log2;
    const int b = blockIdx.x / Hkv, g = blockIdx.x - b * Hkv;
    OwnInfo own = a.own[b * Hkv + g];
    if (own.flags & kDone) return;
    // (a call whose kernels gave up has left places that lie anywhere)
    auto place_ok = [&](const Place &p) {
        return p.k0 < 0 || (p.k0 <= (p.where >> 1) && (p.where >> 1) < a.ranges[p.where & 1]);
    };
    if (own.r0 < 0 || own.r0 > b || !place_ok(own.own)) own.flags = kBad;
    const int NV = G * D / 4;                 // float4 pieces of the output rows
    const int KL = kJoinThreads / NV;         // states read side by side
    const int v = threadIdx.x / KL, kl = threadIdx.x % KL;
    const int h = 4 * v / D, c = 4 * v % D;
    const int64_t row = static_cast<int64_t>(b) * Hq + g * G + h;
    uint2 *dst = reinterpret_cast<uint2 *>(a.out + row * D + c);
    if (own.flags & (kBad | kEmpty)) {
        const uint32_t two = own.flags & kBad ? 0x7fc07fc0u : 0u;
        if (kl == 0) *dst = make_uint2(two, two);
        return;
    }
    Join s;
    // states in the slots of ranges k0 .. k1 of a kernel, at row `at` of each
    auto add_slots = [&](const Place &p, int at) {
        const int kernel = p.where & 1, k1 = p.where >> 1;
#pragma unroll 2
        for (int k = p.k0 + kl; k <= k1; k += KL) {
            const int slot = slot_of(k, p.k0);
            s.add(a.slot_ml[kernel][static_cast<int64_t>(slot) * slot_rows(kernel) + at],
                  *reinterpret_cast<const float4 *>(a.slot_o[kernel] + state_at(kernel, D, slot, at, c)));
        }
    };
    if (own.flags & kHasShared) {
        const int two = kBlockRows >> a.g_log2;
        const int first = own.r0 + (b - own.r0) / two * two;  // of this sequence's block in its group
        const Place sh = a.shared[first * Hkv + g];
        const int at = ((b - first) << a.g_log2) + h, n = -sh.k0;
        if (!place_ok(sh) || (sh.k0 < 0 && (b - first >= n || n > a.batch - first)))
            s.bad = true;
        else if (sh.k0 >= 0)
            add_slots(sh, at);
        else if (kl == 0)
            s.add(a.row_ml[0][block_row(Hkv, a.g_log2, first, n, g, at)],
                  *reinterpret_cast<const float4 *>(
                      a.row_o[0] + block_state_at(sh.where & 1, D, Hkv, a.g_log2, first, n, g, at, c)));
    }
    if (!(own.flags & kNoOwn)) {
        if (own.own.k0 >= 0) add_slots(own.own, h);
        else if (kl == 0) s.add(a.row_ml[1][row], *reinterpret_cast<const float4 *>(a.row_o[1] + row * D + c));
    }
    for (int off = KL / 2; off >= 1; off >>= 1) s.shuffle(off);
    if (kl == 0) *dst = s.result();
}

// kCross: the slots of the two kernels (those of the tiles kernel kSplit times) dealt to warps.  The
// slots of a cut segment's pieces share its outputs.
//  * Few-rows kernel: outputs four columns at a time, each the sum of all the pieces' states, by one
//    lane where there are many outputs and by up to 32 where there are few.
//  * Tiles kernel: tasks of 32 rows, one per lane, and 32 columns, so that many loads are under way;
//    8 columns where there are many pieces.
constexpr int kSplit = 32;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_cross_kernel(const __grid_constant__ Args a) {
    grid_dependency_wait();
    const int G = 1 << a.g_log2, Hq = a.Hkv << a.g_log2, lane = threadIdx.x & 31;
    const int tiles = a.tiles_run ? 2 * a.counts[kTiles] * kSplit : 0, few = 2 * a.counts[kFew];
#pragma unroll 1
    for (int at = (blockIdx.x * kJoinThreads + threadIdx.x) >> 5; at < tiles + few; at += gridDim.x * (kJoinThreads / 32)) {
        const int kernel = at < tiles ? kTiles : kFew;
        const int slot = kernel == kTiles ? at / kSplit : at - tiles, k = slot >> 1;
        const Cut cut = a.cuts[kernel][slot];
        if (cut.k0 < 0 || cut.k0 > k || cut.k1 < k || cut.k1 >= a.ranges[kernel] || cut.n <= 0 ||
            cut.n > slot_rows(kernel) >> a.g_log2 || cut.tok0 < 0 || cut.tok0 > a.tokens - cut.n || cut.g < 0 ||
            cut.g >= a.Hkv)
            continue;  // none (or left by a kernel that gave up)
        const int np = cut.k1 - cut.k0 + 1, R = cut.n << a.g_log2;
        auto out_at = [&](int r, int c) {
            return a.out + (static_cast<int64_t>(cut.tok0 + (r >> a.g_log2)) * Hq + cut.g * G + (r & (G - 1))) * D + c;
        };
        auto ml_at = [&](int p, int r) {
            return a.slot_ml[kernel][static_cast<int64_t>(slot_of(cut.k0 + p, cut.k0)) * slot_rows(kernel) + r];
        };
        auto o_at = [&](int p, int r, int c) {
            return *reinterpret_cast<const float4 *>(a.slot_o[kernel] +
                                                     state_at(kernel, D, slot_of(cut.k0 + p, cut.k0), r, c));
        };
        if (kernel == kTiles) {
            const bool wide = np <= 4;
            const int RG = (R + 31) / 32, task = at % kSplit * np + k - cut.k0;
            // at most 8 x 4 tasks, or 8 x 16 where there are over 4 pieces: kSplit np suffices for both
            if (task >= RG * (wide ? D / 32 : D / 8)) continue;
            const int r = task % RG * 32 + lane, c = task / RG * (wide ? 32 : 8), rr = min(r, R - 1);
            if (wide) {
                float2 ml[4];
                float mx = kNoKey, sum = 0.f;
                bool bad = false;
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    ml[p] = p < np ? ml_at(p, rr) : make_float2(kNoKey, 0.f);
                    mx = fmaxf(mx, ml[p].x);
                    bad |= isnan(ml[p].x);
                }
                float4 acc[8];
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    if (p >= np) break;
                    const float f = ex2(ml[p].x - mx);
                    sum = fmaf(ml[p].y, f, sum);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 o = o_at(p, rr, c + 4 * i);
                        if (p == 0) {
                            acc[i] = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
                        } else {
                            acc[i].x = fmaf(o.x, f, acc[i].x);
                            acc[i].y = fmaf(o.y, f, acc[i].y);
                            acc[i].z = fmaf(o.z, f, acc[i].z);
                            acc[i].w = fmaf(o.w, f, acc[i].w);
                        }
                    }
                }
                const float inv = bad ? __int_as_float(0x7fc00000) : 1.f / sum;
                if (r < R)
#pragma unroll
                    for (int i = 0; i < 8; i += 2)
                        *reinterpret_cast<uint4 *>(out_at(r, c + 4 * i)) = make_uint4(
                            pack_bf16x2(acc[i].x * inv, acc[i].y * inv), pack_bf16x2(acc[i].z * inv, acc[i].w * inv),
                            pack_bf16x2(acc[i + 1].x * inv, acc[i + 1].y * inv),
                            pack_bf16x2(acc[i + 1].z * inv, acc[i + 1].w * inv));
            } else {
                Join s, t;
#pragma unroll 4
                for (int p = 0; p < np; ++p) {
                    const float2 ml = ml_at(p, rr);
                    s.add(ml, o_at(p, rr, c));
                    t.add(ml, o_at(p, rr, c + 4));
                }
                if (r < R) {
                    const uint2 x = s.result(), y = t.result();
                    *reinterpret_cast<uint4 *>(out_at(r, c)) = make_uint4(x.x, x.y, y.x, y.y);
                }
            }
            continue;
        }
        const int U = R * (D / 4), lo = U * (k - cut.k0) / np, hi = U * (k - cut.k0 + 1) / np;
        int KL = 1;  // lanes of an output
        while (KL < 32 && KL < np && KL * 2 * (hi - lo) <= 32) KL *= 2;
        const int kl = lane % KL;
#pragma unroll 1
        for (int u0 = lo; u0 < hi; u0 += 32 / KL) {
            const int u = u0 + lane / KL, r = u / (D / 4), c = u % (D / 4) * 4;
            Join s;
            if (u < hi) {
#pragma unroll 4
                for (int p = kl; p < np; p += KL) s.add(ml_at(p, r), o_at(p, r, c));
            }
            for (int off = KL / 2; off >= 1; off >>= 1) s.shuffle(off);
            if (u < hi && kl == 0) *reinterpret_cast<uint2 *>(out_at(r, c)) = s.result();
        }
    }
}

// ---------------------------------------------------------------- host side
struct Sizes {
    size_t slot_o[2], slot_ml[2], row_o, row_ml, cuts[2], own, shared, counts, entries, borders[2], total;
};
Sizes sizes_of(int op, int64_t batch, int Hq, int Hkv, int D, const int *ranges) {
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at = (at + n + 255) & ~size_t(255);
        return here;
    };
    Sizes s;
    const size_t rows = op == kShared ? static_cast<size_t>(batch) * Hq : 0;
    const size_t segs = op == kShared ? static_cast<size_t>(batch) * Hkv : 0;
    for (int k = 0; k < 2; ++k) {
        const size_t slots = 2 * static_cast<size_t>(ranges[k]);
        s.slot_o[k] = take(slots * slot_rows(k) * D * 4);
        s.slot_ml[k] = take(slots * slot_rows(k) * 8);
        s.cuts[k] = take(op == kCross ? slots * sizeof(Cut) : 0);
        s.borders[k] = take((static_cast<size_t>(ranges[k]) + 1) * sizeof(Border));
    }
    s.row_o = take(2 * rows * D * 4);
    s.row_ml = take(2 * rows * 8);
    s.own = take(segs * sizeof(OwnInfo));
    s.shared = take(segs * sizeof(Place));
    s.entries = take((op == kShared ? 2 : 1) * static_cast<size_t>(batch) * sizeof(Entry));
    s.counts = take(16);  // ranges of the two kernels, the next one of the few-rows kernel
    s.total = at;
    return s;
}

void blocks_on(const pkv_host::DeviceInfo &dev, int *blocks, int *ranges) {
    for (int k = 0; k < 2; ++k) {
        blocks[k] = (k == kTiles ? 1 : 2) * dev.sm_count;
        ranges[k] = (1 + short_ranges(k)) * blocks[k];
    }
}

template <int D>
pkv_status launch(const Args &a, int64_t num_pages, const pkv_host::DeviceInfo &dev, cudaStream_t stream) {
    const int G = 1 << a.g_log2, Hq = a.Hkv * G;
    const int64_t slots = num_pages << a.ps_log2;
    CUtensorMap qmap, kmap[2], vmap[2];
    if (!pkv_host::encode_q_map(&qmap, a.q, a.tokens, Hq, D, G, BM / G)) return PKV_EINVAL;
    for (int k = 0; k < 2; ++k) {
        if (a.box_log2[k] >= 3) {  // page boxes
            if (!pkv_host::encode_kv_map(&kmap[k], a.k_cache, slots, a.Hkv, D, 64, 1 << a.box_log2[k], true) ||
                !pkv_host::encode_kv_map(&vmap[k], a.v_cache, slots, a.Hkv, D, 64, 1 << a.box_log2[k], true))
                return PKV_EINVAL;
        } else {  // rows gathered four at a time
            if (!pkv_host::encode_rows_map_swizzled(&kmap[k], a.k_cache, slots * a.Hkv, D) ||
                !pkv_host::encode_rows_map_swizzled(&vmap[k], a.v_cache, slots * a.Hkv, D))
                return PKV_EINVAL;
        }
    }
    static std::mutex mu;
    static bool ready[64] = {};
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!ready[dev.device] &&
            cudaFuncSetAttribute(plan_kernel<D, 1024>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 plan_smem(2 * kMaxBatch, kMaxBatch)) != cudaSuccess)
            return PKV_ECUDA;
        ready[dev.device] = true;
    }
    // few entries: a thread for each of them, and smaller blocks start sooner
    const int entries = a.op == kCross ? a.batch : a.groups + a.batch;
    const bool many = entries > 256;
    if (pkv_host::launch_dependent(many ? plan_kernel<D, 1024> : plan_kernel<D, 256>, dim3(kPlanBlocks),
                                   dim3(many ? 1024 : 256), plan_smem(entries, a.batch), stream, a) != cudaSuccess)
        return PKV_ECUDA;
    const bool rows_long = (a.pt_stride << a.ps_log2) > kShortKeys;
    const auto tiles = rows_long ? launch_tiles<D, true> : launch_tiles<D, false>;
    const auto few = rows_long ? launch_few<D, true> : launch_few<D, false>;
    if ((a.tiles_run && !tiles(a, qmap, kmap[kTiles], vmap[kTiles], dev, stream)) ||
        !few(a, kmap[kFew], vmap[kFew], dev, stream))
        return PKV_ECUDA;
    const cudaError_t err =
        a.op == kCross
            ? pkv_host::launch_dependent(join_cross_kernel<D>, dim3(5 * a.blocks[kTiles]),
                                         dim3(kJoinThreads), 0, stream, a)
            : pkv_host::launch_dependent(join_shared_kernel<D>, dim3(a.batch * a.Hkv), dim3(kJoinThreads), 0, stream, a);
    return err == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

size_t workspace_size(int op, int batch, int num_q_heads, int num_kv_heads, int head_dim) {
    if (batch < 0 || batch > kMaxBatch || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads)
        return 0;
    if (head_dim != 64 && head_dim != 128) return 0;
    pkv_host::DeviceInfo dev;
    if (!pkv_host::current_device(&dev)) return 0;
    int blocks[2], ranges[2];
    blocks_on(dev, blocks, ranges);
    return sizes_of(op, batch, num_q_heads, num_kv_heads, head_dim, ranges).total;
}

// Checks of both entry points, the workspace's parts and the launches.
pkv_status entry(Args &a, int num_q_heads, int head_dim, int page_size, int64_t num_pages, float softmax_scale,
                 void *workspace, size_t workspace_bytes, void *stream) {
    if (a.batch < 0 || a.groups < 0 || a.tokens < 0 || num_q_heads <= 0 || a.Hkv <= 0 || num_pages <= 0 ||
        a.pt_stride < 0 || page_size <= 0 || num_q_heads % a.Hkv != 0 || !(softmax_scale == softmax_scale))
        return PKV_EINVAL;
    if (a.batch == 0 || a.tokens == 0) return PKV_OK;
    if (!a.q || !a.k_cache || !a.v_cache || !a.page_table || !a.lens || !a.out || !workspace) return PKV_EINVAL;
    if (a.op == kCross ? !a.cu : a.groups > 0 && (!a.gstart || !a.glen)) return PKV_EINVAL;
    const int G = num_q_heads / a.Hkv;
    if ((head_dim != 64 && head_dim != 128) || (G != 1 && G != 2 && G != 4 && G != 8)) return PKV_EUNSUPPORTED;
    if ((page_size & (page_size - 1)) != 0 || page_size > 256) return PKV_EUNSUPPORTED;
    if (a.groups > a.batch) return PKV_EINVAL;
    if (a.batch > kMaxBatch) return PKV_EUNSUPPORTED;
    if (!pkv_host::aligned16(a.q) || !pkv_host::aligned16(a.k_cache) || !pkv_host::aligned16(a.v_cache) ||
        !pkv_host::aligned16(a.out) || !pkv_host::aligned16(workspace))
        return PKV_EINVAL;
    if (num_pages > 0x7fffffffll / page_size || a.tokens > 0x7fffff00ll || a.pt_stride > 0x7fffffffll / page_size)
        return PKV_EUNSUPPORTED;
    // rows gathered four at a time have numbers of 31 bits
    if (page_size < 8 && num_pages * page_size > 0x7fffffffll / a.Hkv) return PKV_EUNSUPPORTED;
    // the units of all segments at most (the few-rows kernel's tiles may have half of the keys)
    const double tiles = static_cast<double>(a.pt_stride) * page_size / 64 + 1;
    const double blocks = static_cast<double>(a.tokens) * G / kBlockRows + a.batch + a.groups;
    if (blocks * a.Hkv * (tile_cost(kPair, false) * tiles + lead_cost(kPair)) >= kMostUnits)
        return PKV_EUNSUPPORTED;
    pkv_host::DeviceInfo dev;
    if (!pkv_host::current_device(&dev)) return PKV_ECUDA;
    blocks_on(dev, a.blocks, a.ranges);
    const Sizes s = sizes_of(a.op, a.batch, num_q_heads, a.Hkv, head_dim, a.ranges);
    if (workspace_bytes < s.total) return PKV_EINVAL;
    a.g_log2 = G == 1 ? 0 : G == 2 ? 1 : G == 4 ? 2 : 3;
    a.ps_log2 = 0;
    while ((1 << a.ps_log2) < page_size) ++a.ps_log2;
    a.num_pages = static_cast<int>(num_pages);
    // (not 0, so that a masked score, -infinity, stays it; the least number has the same weights)
    a.scale_log2 = fmaxf(fabsf(softmax_scale) * kLog2e, 0x1p-149f);
    a.negate = softmax_scale < 0.f ? 1u : 0u;
    uint8_t *w = static_cast<uint8_t *>(workspace);
    const size_t rows = a.op == kShared ? static_cast<size_t>(a.batch) * num_q_heads : 0;
    for (int k = 0; k < 2; ++k) {
        const int keys_log2 = head_dim == 64 || k == kTiles ? 7 : 6;
        a.box_log2[k] = a.ps_log2 < keys_log2 ? a.ps_log2 : keys_log2;
        a.slot_o[k] = reinterpret_cast<float *>(w + s.slot_o[k]);
        a.slot_ml[k] = reinterpret_cast<float2 *>(w + s.slot_ml[k]);
        a.cuts[k] = reinterpret_cast<Cut *>(w + s.cuts[k]);
        a.borders[k] = reinterpret_cast<Border *>(w + s.borders[k]);
        a.row_o[k] = reinterpret_cast<float *>(w + s.row_o) + k * rows * head_dim;
        a.row_ml[k] = reinterpret_cast<float2 *>(w + s.row_ml) + k * rows;
    }
    a.own = reinterpret_cast<OwnInfo *>(w + s.own);
    a.shared = reinterpret_cast<Place *>(w + s.shared);
    a.entries = reinterpret_cast<Entry *>(w + s.entries);
    a.counts = reinterpret_cast<int *>(w + s.counts);
    a.next_range = reinterpret_cast<unsigned int *>(a.counts + 2);
    // Blocks of 9 to 16 rows: the tiles kernel reads memory faster (heads of 128; two tokens of 8 query
    // heads: 38 requests of 1000-8000 states 85 -> 72 us, 20 of 100-1500 29 -> 30), but starts later and
    // needs longer for a segment, so not where there are few of them (10 of 100-1500 23 -> 28), nor for
    // heads of 64, whose rows cost half as much here (16 tokens of 30 requests 29 -> 32, long ones equal).
    // In a decode step the few-rows kernel has the own keys to read as well: 64 groups of two on 4 KV
    // heads 74 -> 66 us, but 24 groups of one to 30 65 -> 72.
    const int64_t segments = a.op == kCross ? int64_t{2} * a.batch * a.Hkv : int64_t{a.groups} * a.Hkv;
    a.few_rows = head_dim == 128 && segments >= dev.sm_count ? kFewRows / 2 : kFewRows;
    a.tiles_run = a.tokens * G > a.few_rows && (a.op == kCross || a.groups > 0);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return head_dim == 128 ? launch<128>(a, num_pages, dev, st) : launch<64>(a, num_pages, dev, st);
}

}  // namespace
}  // namespace ck
}  // namespace pkv

extern "C" size_t pkv_decode_shared_workspace_size(int batch, int num_q_heads, int num_kv_heads, int head_dim) {
    return pkv::ck::workspace_size(pkv::ck::kShared, batch, num_q_heads, num_kv_heads, head_dim);
}

extern "C" size_t pkv_cross_workspace_size(int batch, int num_q_heads, int num_kv_heads, int head_dim) {
    return pkv::ck::workspace_size(pkv::ck::kCross, batch, num_q_heads, num_kv_heads, head_dim);
}

extern "C" pkv_status pkv_paged_decode_attn_shared(
    const pkv_bf16 *q, const pkv_bf16 *k_cache, const pkv_bf16 *v_cache, const int32_t *page_table,
    int64_t page_table_stride, const int32_t *seq_lens, int batch, int num_q_heads, int num_kv_heads, int head_dim,
    int page_size, int64_t num_pages, float softmax_scale, const int32_t *prefix_group_start,
    const int32_t *prefix_len, int num_prefix_groups, void *workspace, size_t workspace_bytes, int32_t *dev_status,
    pkv_bf16 *out, void *stream) {
    pkv::ck::Args a = {};
    a.op = pkv::ck::kShared;
    a.q = reinterpret_cast<const __nv_bfloat16 *>(q);
    a.k_cache = reinterpret_cast<const __nv_bfloat16 *>(k_cache);
    a.v_cache = reinterpret_cast<const __nv_bfloat16 *>(v_cache);
    a.page_table = page_table;
    a.pt_stride = page_table_stride;
    a.lens = seq_lens;
    a.gstart = prefix_group_start;
    a.glen = prefix_len;
    a.batch = batch;
    a.groups = num_prefix_groups;
    a.tokens = batch;
    a.Hkv = num_kv_heads;
    a.dev_status = dev_status;
    a.out = reinterpret_cast<__nv_bfloat16 *>(out);
    return pkv::ck::entry(a, num_q_heads, head_dim, page_size, num_pages, softmax_scale, workspace,
                          workspace_bytes, stream);
}

extern "C" pkv_status pkv_paged_cross_attn(const pkv_bf16 *q, const int32_t *cu_seqlens_q, const pkv_bf16 *k_cache,
                                           const pkv_bf16 *v_cache, const int32_t *page_table,
                                           int64_t page_table_stride, const int32_t *kv_lens, int batch,
                                           int64_t total_q_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                           int page_size, int64_t num_pages, float softmax_scale, void *workspace,
                                           size_t workspace_bytes, int32_t *dev_status, pkv_bf16 *out, void *stream) {
    pkv::ck::Args a = {};
    a.op = pkv::ck::kCross;
    a.q = reinterpret_cast<const __nv_bfloat16 *>(q);
    a.k_cache = reinterpret_cast<const __nv_bfloat16 *>(k_cache);
    a.v_cache = reinterpret_cast<const __nv_bfloat16 *>(v_cache);
    a.page_table = page_table;
    a.pt_stride = page_table_stride;
    a.lens = kv_lens;
    a.cu = cu_seqlens_q;
    a.batch = batch;
    a.tokens = total_q_tokens;
    a.Hkv = num_kv_heads;
    a.dev_status = dev_status;
    a.out = reinterpret_cast<__nv_bfloat16 *>(out);
    return pkv::ck::entry(a, num_q_heads, head_dim, page_size, num_pages, softmax_scale, workspace,
                          workspace_bytes, stream);
}
