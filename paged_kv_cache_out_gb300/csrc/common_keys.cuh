// common_keys.cuh -- attention over paged keys that several query rows read
// without a causal mask: what the kernels of pkv_paged_decode_attn_shared and
// pkv_paged_cross_attn share.
//
// For a query row and its keys j, with s_j = scale * q.k_j:
//     m = max_j s_j,  l = sum_j e^(s_j - m),  o = sum_j e^(s_j - m) v_j,  out = o / l,
// and two disjoint sets of keys join as
//     m = max(m1, m2),  l = l1 e^(m1 - m) + l2 e^(m2 - m),  o likewise.
//
// An entry is a run of query tokens that read the same keys: a request's
// queries over its states, a group's sequences over the shared keys, or one
// sequence over its own.  An entry's tokens x the query heads of a KV head are
// packed into blocks of up to 256 rows.  Blocks of more than 16 rows (or 8, see
// few_rows) go to the tiles kernel (tcgen05), the others to the few-rows kernel
// (mma.sync), and
// each kernel cuts its own work the same way: all its (entry, KV head, block)
// segments are laid end to end, each as long as its cost (some units for the
// fixed work, then its key tiles), and cut into ranges of equal length: one
// per block of the tiles kernel; some long ones and many short ones for the
// few-rows kernel, whose blocks take one after the other.  So every SM gets
// its share whatever the mix of long and short; a segment that is cut leaves
// partial states (m, l, o), which the join kernel brings together in a fixed
// order.  A plan kernel finds the borders of the ranges first: the others
// would each spend longer on it, in code that they run once.
#pragma once

#include "umma_tiles.cuh"

namespace pkv {
namespace ck {

constexpr int kMaxBatch = 4096;
constexpr int BM = 128;               // rows of a query tile of the tiles kernel
constexpr int kBlockRows = 2 * BM;    // rows of a block, of a partial state of that kernel
constexpr int kFewRows = 16;          // most rows of the few-rows kernel
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNoKey = -3.0e38f;    // reference of a row whose scores are all -infinity
// A tensor-core sum cuts off where an FMA rounds: with V of one sign, an output whose products go to one
// accumulator (16 keys an instruction) is too small by 9e-5 of it after 16384 keys, 8e-4 after 131072,
// 7e-3 after 2^20, where a rounding to bf16 is off by 1.4e-3 (2-norm).  So rows that may be longer are
// taken by other forms of both kernels (LONG): the few-rows kernel adds the products of 16 keys in fp32,
// the tiles kernel moves its outputs to fp32 totals after this many keys.  (In the short forms' place
// these take 0.7 us more of 128 chats, 1 of prompts, 3 of long and of ragged cross attention.)
constexpr int kShortKeys = 16384;
constexpr float kRescaleLog2 = 8.0f;  // the reference moves when a score exceeds it by 2^8

enum Op : int { kCross = 0, kShared = 1 };
enum Kernel : int { kTiles = 0, kFew = 1 };

// Where the rows of a finished piece go.
enum Dest : int {
    kOut = 0,         // normalised, to out
    kSlot = 1,        // partial state, to one of this block's two slots
    kRowsShared = 2,  // partial state of a decode step's shared keys, in the rows of its block
    kRowsOwn = 3,     // partial state of its own keys, by row of out
};

// A segment that is cut has a piece in each of ranges k0 .. k1 of its kernel.  A range's slot 1 holds
// the state of the piece that goes on in the next range (so that of range k0), slot 0 that of a piece
// that began in an earlier one.
__host__ __device__ constexpr int slot_of(int k, int k0) { return 2 * k + (k == k0 ? 1 : 0); }
// What a partial state in a slot belongs to (kCross).  k0 < 0: none.
struct Cut {
    int k0, k1, tok0, n, g;
};
// Where the states of some keys lie: ranges k0 .. k1 of a kernel, or, k0 < 0, by row (of shared keys:
// in the rows of a block of -k0 sequences); `where` = 2 k1 + kernel.
struct Place {
    int k0, where;
};
// A sequence and KV head of a decode step: its own keys' states, the first
// sequence of its group, and what there is to join.
struct OwnInfo {
    Place own;
    int r0, flags;
};
enum : int { kHasShared = 1, kBad = 2, kDone = 4, kEmpty = 8, kNoOwn = 16 };

struct Args {
    const __nv_bfloat16 *q, *k_cache, *v_cache;
    const int32_t *page_table;
    int64_t pt_stride;
    const int32_t *lens;
    const int32_t *cu;               // kCross: [batch + 1]
    const int32_t *gstart, *glen;    // kShared: [groups + 1], [groups]
    int op, batch, groups;
    int64_t tokens;
    int Hkv, g_log2;
    int ps_log2, box_log2[2];        // log2 of the rows of a page box, by kernel
    int num_pages;
    int blocks[2], ranges[2];        // of the two kernels; most ranges
    unsigned int *next_range;        // claimed by blocks of the few-rows kernel (the plan kernel starts it at 0)
    int *counts;                     // [2]: ranges of the two kernels in this call
    struct Entry *entries;           // [groups + batch]
    struct Border *borders[2];       // by kernel: [ranges + 1]
    int few_rows;                    // most rows of a block of the few-rows kernel
    int tiles_run;                   // whether the tiles kernel is launched
    float scale_log2;                // of |scale|
    uint32_t negate;                 // scale < 0
    float *slot_o[2];                // by kernel: [2 x ranges][kBlockRows or kFewRows][D]
    float2 *slot_ml[2];
    float *row_o[2];                 // kShared: shared, own: [batch x Hq][D]
    float2 *row_ml[2];
    Cut *cuts[2];                    // kCross, by kernel: [2 x ranges]
    OwnInfo *own;                    // kShared: [batch x Hkv]
    Place *shared;                   // kShared: [batch x Hkv] by a block's first sequence
    int32_t *dev_status;
    __nv_bfloat16 *out;
};

__host__ __device__ constexpr int slot_rows(int kernel) { return kernel == kTiles ? kBlockRows : kFewRows; }
// Columns c .. c + 3 of row r of the state in a slot: by rows in the few-rows kernel's slots, by fours of
// columns in the tiles kernel's, whose threads write a row each.
__device__ __forceinline__ int64_t state_at(int kernel, int D, int slot, int r, int c) {
    return kernel == kTiles ? (static_cast<int64_t>(slot) * (D / 4) + c / 4) * (4 * kBlockRows) + 4 * r
                            : (static_cast<int64_t>(slot) * kFewRows + r) * D + c;
}
// Row r of a whole block of n sequences from tok0 on in the states of shared keys, and its columns
// c .. c + 3 (in the order of the slots).
__device__ __forceinline__ int64_t block_row(int Hkv, int g_log2, int tok0, int n, int g, int r) {
    return ((static_cast<int64_t>(tok0) * Hkv + static_cast<int64_t>(g) * n) << g_log2) + r;
}
__device__ __forceinline__ int64_t block_state_at(int kernel, int D, int Hkv, int g_log2, int tok0, int n, int g, int r,
                                                  int c) {
    const int64_t first = block_row(Hkv, g_log2, tok0, n, g, 0) * D;
    return first + (kernel == kTiles ? (c / 4) * (static_cast<int64_t>(n << g_log2) * 4) + 4 * r
                                     : static_cast<int64_t>(r) * D + c);
}
__device__ __forceinline__ uint64_t l2_normal_policy() {
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
    return pol;
}

// ---------------------------------------------------------------- waits
// A wait gives up after kTries suspensions of at most 20 us each (4 s at most).  Not mbar_wait's clock:
// with its reads prompts took 51.2 us instead of 48.6, ragged cross attention 118.0 instead of 114.8.
constexpr int kTries = 200000;
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// All lanes of a warp wait for the phase of that parity, with one outcome: false when the time is up
// or another warp of the block gave up, and the block winds down.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int *abort_flag, int32_t *dev_status) {
    bool ok = try_wait(bar, parity);
#pragma unroll 1
    for (int i = 0; !ok && i < kTries; ++i) {
        ok = try_wait(bar, parity);
        if (!ok && *abort_flag) break;
    }
    if (!__all_sync(0xffffffffu, ok)) {
        *abort_flag = 1;
        if (dev_status) atomicOr(dev_status, PKV_DEV_TIMEOUT);
        return false;
    }
    return true;
}

// ---------------------------------------------------------------- weights
// Two weights as bf16 pairs: the upper 16 bits, and the rest, rounded and never 0, so that the
// second product of a value that is infinite is the first's.
__device__ __forceinline__ void split_weights(float p0, float p1, uint32_t &high, uint32_t &low) {
    const uint32_t u0 = __float_as_uint(p0), u1 = __float_as_uint(p1);
    high = __byte_perm(u0, u1, 0x7632);
    float l0 = -__uint_as_float(u0 & 0xffff0000u), l1 = -__uint_as_float(u1 & 0xffff0000u);
    add2(l0, l1, p0, p1);
    low = pack_bf16x2(l0, l1) | 0x00010001u;
}

// ---------------------------------------------------------------- entries
struct __align__(16) Entry {
    int tok0, n, klo, kend;
    int row, r0, flags, pad;
};
// Where a range starts: tile t of segment `seg` (KV head * blocks + block) of an entry.  t > 0: the
// segment is cut, with pieces in ranges k0 .. k1.
struct __align__(16) Border {
    int e, seg, t, k0;
    int k1, pad0, pad1, pad2;
};

// kShared: a group's prefix length if it is a whole number of pages within a row, else -1.
__device__ __forceinline__ int checked_prefix(const Args &a, int S) {
    return S >= 0 && S <= (a.pt_stride << a.ps_log2) && (S & ((1 << a.ps_log2) - 1)) == 0 ? S : -1;
}
__device__ __forceinline__ Entry own_entry(const Args &a, int b, int L, int S, int r0) {
    Entry x;
    x.tok0 = x.row = b;
    x.n = 1;
    x.r0 = r0;
    x.klo = max(S, 0);
    x.kend = x.klo;
    if (L < 0 || L > (a.pt_stride << a.ps_log2))
        x.flags = kBad | (PKV_DEV_BAD_SEQLEN << 8);
    else if (S < 0 || (L > 0 && L < S))
        x.flags = kBad | (PKV_DEV_BAD_SHARED << 8);
    else if (L == 0)
        x.flags = kEmpty;
    else {
        x.kend = L;
        x.flags = (S > 0 ? kHasShared : 0) | (L == S ? kNoOwn : 0);
    }
    return x;
}
// Entry e; S and r0: a sequence's group's checked prefix and first sequence.
__device__ __forceinline__ Entry get_entry(const Args &a, int e, int S, int r0) {
    if (a.op == kShared && e >= a.groups) return own_entry(a, e - a.groups, a.lens[e - a.groups], S, r0);
    Entry x;
    if (a.op == kCross) {
        const int t0 = a.cu[e], t1 = a.cu[e + 1], L = a.lens[e];
        const bool bad = L < 0 || L > (a.pt_stride << a.ps_log2);
        x.tok0 = t0;
        x.n = t1 - t0;
        x.klo = 0;
        x.kend = bad ? 0 : L;
        x.row = e;
        x.r0 = 0;
        x.flags = bad ? kBad | (PKV_DEV_BAD_SEQLEN << 8) : 0;
    } else {
        x.tok0 = x.row = x.r0 = a.gstart[e];
        const int shared = checked_prefix(a, a.glen[e]);
        x.n = shared > 0 ? a.gstart[e + 1] - x.tok0 : 0;
        x.klo = 0;
        x.kend = max(shared, 0);
        x.flags = 0;
    }
    return x;
}

// ---------------------------------------------------------------- cost
// Forms of a block: few rows (up to 16 or 8), one query tile (up to 128), two that
// share each K/V tile (up to 256).
enum Form : int { kFewForm = 0, kSingle = 1, kPair = 2 };

// Keys of a tile, by kernel.
template <int D>
__host__ __device__ constexpr int tile_keys(int kernel) { return kernel == kTiles || D == 64 ? 128 : 64; }
// The cost of a segment in units of about 0.26 us of a block: a lead for its fixed work, then its
// tiles (the few-rows kernel's at the rate at which two blocks per SM read them from memory).  Fitted
// to the tiles kernel's blocks: a pair's tile 1.6 us, a single block's 0.95, or 1.3 where pages have
// fewer than 8 tokens (small) and its copies set the pace, a segment 2.0-2.8.
__host__ __device__ constexpr int lead_cost(int form) { return form == kFewForm ? 3 : form == kSingle ? 8 : 12; }
__host__ __device__ constexpr int tile_cost(int form, bool small) {
    return form == kFewForm ? 6 : form == kSingle ? (small ? 5 : 4) : 6;
}
// Least units of a range: shorter ones cost more states than they save time (24 units of the tiles
// kernel instead of 48: decode of 24 groups 68.1 us instead of 65.7, of 128 chats after one prompt
// 42.5 instead of 41.5).
__host__ __device__ constexpr int min_units(int kernel) { return kernel == kFew ? 9 : 48; }
// Short ranges beside the long one of each block, the part of the work in them, least units of one.
// For the few-rows kernel, some of whose blocks start when the tiles kernel leaves their SM (decode of
// 24 groups 89 us without them, 66 with; where no block waits, 96 chats, equal); not for the tiles
// kernel, whose blocks start together and whose tiles take equal times (long cross attention 240 us
// without, 266 with a short range per block): its ranges are no more than its blocks.
__host__ __device__ constexpr int short_ranges(int kernel) { return kernel == kFew ? 5 : 0; }
constexpr int kShortShare = 2, kShortUnits = 24;
// A cut costs a state written and read, so one that would fall this near an end of a segment (at least
// the lead: a piece has tiles) falls between segments instead.  (Pairs: 20 instead of 14 made the
// prompts' ranges uneven, 50 us instead of 48.5.)
__host__ __device__ constexpr int snap_cost(int form) { return form == kFewForm ? 9 : form == kSingle ? 10 : 14; }
// An entry's segments of one kernel, per KV head: nblk of them, all pairs but the last.
struct Blocks {
    int nblk, last, nk;
    int pair_units, per_head;
};
template <int D, int KERNEL>
__device__ __forceinline__ Blocks blocks_of(const Args &a, int n, int keys, bool small) {
    Blocks k;
    const int g_log2 = a.g_log2, two_log2 = 8 - g_log2;  // tokens of a pair block
    const int nblk = (n + (1 << two_log2) - 1) >> two_log2;
    const int rows = (n - ((nblk - 1) << two_log2)) << g_log2;
    const int last = rows <= a.few_rows ? kFewForm : rows <= BM ? kSingle : kPair;
    constexpr int BN = tile_keys<D>(KERNEL);
    k.nk = static_cast<int>((static_cast<unsigned>(keys) + BN - 1) / BN);
    k.nblk = 0;
    k.last = last;
    k.pair_units = k.per_head = 0;
    if (n <= 0) return k;
    if (KERNEL == kTiles) {
        if (k.nk == 0) return k;
        k.pair_units = tile_cost(kPair, small) * k.nk + lead_cost(kPair);
        k.nblk = nblk - (last == kFewForm ? 1 : 0);
        if (last == kFewForm) k.last = kPair;
        k.per_head = (nblk - 1) * k.pair_units + (last == kFewForm ? 0 : tile_cost(last, small) * k.nk + lead_cost(last));
    } else if (k.nk == 0) {  // no keys: rows to fill, whatever their number
        k.nblk = nblk;
        k.last = kFewForm;
        k.pair_units = lead_cost(kFewForm);
        k.per_head = nblk * k.pair_units;
    } else if (last == kFewForm) {
        k.nblk = 1;
        k.pair_units = k.per_head = tile_cost(kFewForm, small) * k.nk + lead_cost(kFewForm);
    }
    return k;
}

// The ranges of W units: `early` long ones, and others that are `delta` units shorter.
// (delta (n - early) is at most 2 W, and W under 2^32 / 3, so that 32 bits without sign hold it all.)
constexpr double kMostUnits = 4294967296.0 / 3;
struct Ranges {
    int W, n, early, delta;
    unsigned q;
    int r;           // W + delta (n - early) = q n + r
    float inv;       // 1 / n
    __device__ __forceinline__ void set(int w, int count, int n_early, int d) {
        W = w, n = count, early = n_early, delta = d;
        const unsigned all = static_cast<unsigned>(w) + static_cast<unsigned>(d) * static_cast<unsigned>(n - n_early);
        q = all / static_cast<unsigned>(n), r = static_cast<int>(all - q * static_cast<unsigned>(n));
        inv = 1.f / static_cast<float>(n);
    }
    // floor(k (q n + r) / n) = k q + floor(k r / n).  With n < 2048, k r < 2^22 and its half step are
    // exact, and the half keeps the quotient 0.5 / n from whole numbers, its rounding is under n 2^-23.
    __device__ __forceinline__ int start(int k) const {
        return static_cast<int>(static_cast<unsigned>(k) * q +
                                static_cast<unsigned>((static_cast<float>(k * r) + 0.5f) * inv) -
                                static_cast<unsigned>(max(k - early, 0)) * static_cast<unsigned>(delta));
    }
    // the last range that starts at or before x
    __device__ __forceinline__ int range_of(int x) const {
        const int turn = start(early);
        const float each = static_cast<float>(q) + static_cast<float>(r) * inv;
        int k = x < turn ? static_cast<int>(static_cast<float>(x) / each)
                         : early + static_cast<int>(static_cast<float>(x - turn) / (each - static_cast<float>(delta)));
        k = min(max(k, 0), n - 1);
        while (k > 0 && start(k) > x) --k;
        while (k + 1 < n && start(k + 1) <= x) ++k;
        return k;
    }
};
// ---------------------------------------------------------------- the pieces of a block
struct __align__(16) Item {
    int form, tok0, n, g;          // tokens tok0 .. tok0 + n - 1, KV head
    int row, key0, kend, nt;       // page-table row, first key, one past the entry's last, key tiles (-1: no more)
    int dest, slot, flags, again;  // its entry's flags, whether other blocks read the same keys
};

// The walk over a block's ranges, by one warp.
template <int D, int KERNEL>
struct Walk {
    bool own_first;
    Border from, to;
    int n, range;         // ranges of the kernel, this one
    int e, seg, t;        // where it goes on
    int win;              // 32 entries from there on, one per lane
    uint32_t busy;        // those of them that have blocks
    Entry we;
    bool cut_set[2];

    // A block's first range is the one of its own number, whose borders are on their way before the
    // number of ranges is known, where its blocks all start together: a block of the few-rows kernel
    // that starts when the tiles kernel leaves takes what is there then.
    __device__ __forceinline__ explicit Walk(const Args &a)
        : own_first(KERNEL == kTiles || !a.tiles_run),
          from(a.borders[KERNEL][own_first ? blockIdx.x : 0]), to(a.borders[KERNEL][own_first ? blockIdx.x + 1 : 0]),
          n(a.counts[KERNEL]), range(-1), e(0), seg(0), t(0), win(-64), busy(0), cut_set{false, false} {
        e = to.e, seg = to.seg, t = to.t;  // (nothing to do until a range is taken)
    }
    // The next range of this block; false when there is none.
    __device__ __forceinline__ bool next_range(const Args &a) {
        int k = blockIdx.x;
        if (!own_first || range >= 0) {
            if (KERNEL == kTiles) return false;  // (no more ranges than blocks)
            if ((threadIdx.x & 31) == 0) k = static_cast<int>(atomicAdd(a.next_range, 1u));
            k = __shfl_sync(0xffffffffu, k, 0) + (own_first ? static_cast<int>(gridDim.x) : 0);
        }
        if (k >= n) return false;
        if (!own_first || range >= 0) {
            from = a.borders[KERNEL][k];
            to = a.borders[KERNEL][k + 1];
        }
        finish(a);
        range = k;
        e = from.e, seg = from.seg, t = from.t;
        cut_set[0] = cut_set[1] = false;
        return true;
    }
    // The slots of the range that hold no piece of a cut segment.
    __device__ __forceinline__ void finish(const Args &a) const {
        const int lane = threadIdx.x & 31;
        if (a.op == kCross && range >= 0 && lane < 2 && !(lane ? cut_set[1] : cut_set[0]))
            a.cuts[KERNEL][2 * range + lane].k0 = -1;
    }
    // The next piece; false when there is none.  nt == 0: rows without keys, to be filled (kCross) or
    // told of (kShared).  Where the states of the pieces will lie is written down.  due() returns when
    // another range may be taken.
    template <typename Due>
    __device__ __forceinline__ bool next(const Args &a, Item &it, Due due) {
        constexpr int BN = tile_keys<D>(KERNEL);
        const int lane = threadIdx.x & 31;
#pragma unroll 1
        for (;;) {
            if (e > to.e || (e == to.e && (seg > to.seg || (seg == to.seg && t >= to.t)))) {
                if (due() && next_range(a)) continue;
                finish(a);
                return false;
            }
            if (e < win || e >= win + 32) {
                win = e;
                const bool there = win + lane < (a.op == kCross ? a.batch : a.groups + a.batch);
                if (there) we = a.entries[win + lane];
                busy = __ballot_sync(0xffffffffu, there && blocks_of<D, KERNEL>(a, we.n, we.kend - we.klo, false).nblk > 0);
            }
            // entries of the other kernel alone are stepped over together (one by one, 240 of them kept the
            // block with the last range for 20 us)
            const uint32_t ahead = busy >> (e - win);
            if (!(ahead & 1)) {
                e = ahead ? e + __ffs(static_cast<int>(ahead)) - 1 : win + 32;
                seg = t = 0;
                continue;
            }
            Entry x;
            const int src = e - win;
            x.tok0 = __shfl_sync(0xffffffffu, we.tok0, src);
            x.n = __shfl_sync(0xffffffffu, we.n, src);
            x.klo = __shfl_sync(0xffffffffu, we.klo, src);
            x.kend = __shfl_sync(0xffffffffu, we.kend, src);
            const Blocks bl = blocks_of<D, KERNEL>(a, x.n, x.kend - x.klo, false);
            if (seg >= bl.nblk * a.Hkv) {
                ++e;
                seg = t = 0;
                continue;
            }
            const int g = bl.nblk > 1 ? seg / bl.nblk : seg, m = seg - g * bl.nblk;
            const int t1 = e == to.e && seg == to.seg ? to.t : bl.nk;
            const bool whole = t == 0 && t1 == bl.nk;
            const int two = kBlockRows >> a.g_log2;
            // the few-rows block is an entry's last
            const int blk = KERNEL == kTiles || bl.nk == 0 ? m : (x.n - 1) / two;
            const int k0 = whole ? -1 : t > 0 ? from.k0 : to.k0, k1 = whole ? 0 : t > 0 ? from.k1 : to.k1;
            const int flags = __shfl_sync(0xffffffffu, we.flags, src);
            const bool is_own = a.op == kShared && e >= a.groups;
            it.form = m < bl.nblk - 1 ? (KERNEL == kTiles ? kPair : kFewForm) : bl.last;
            it.tok0 = x.tok0 + blk * two;
            it.n = min(x.n - blk * two, two);
            it.g = g;
            it.row = __shfl_sync(0xffffffffu, we.row, src);
            it.key0 = x.klo + t * BN;
            it.kend = x.kend;
            it.nt = t1 - t;
            it.slot = slot_of(range, k0);
            it.dest = !whole ? kSlot : a.op == kCross ? kOut : !is_own ? kRowsShared
                             : flags & kHasShared ? kRowsOwn : kOut;
            it.flags = flags;
            it.again = x.n > two;
            if (a.op == kCross) {
                if (!whole) {
                    cut_set[0] |= (it.slot & 1) == 0;
                    cut_set[1] |= (it.slot & 1) != 0;
                    if (lane == 0) a.cuts[KERNEL][it.slot] = Cut{k0, k1, it.tok0, it.n, g};
                }
            } else {
                const int r0 = __shfl_sync(0xffffffffu, we.r0, src);
                if (t == 0 && lane == 0) {
                    const Place place = {whole && !is_own ? -it.n : k0, k1 * 2 + KERNEL};
                    if (is_own)
                        a.own[it.tok0 * a.Hkv + g] =
                            OwnInfo{place, r0, flags | (bl.nk > 0 && it.dest == kOut ? kDone : 0)};
                    else
                        a.shared[it.tok0 * a.Hkv + g] = place;
                }
            }
            if (t1 == bl.nk) ++seg, t = 0;
            else t = t1;
            return true;
        }
    }
};

// ---------------------------------------------------------------- page copies
// What a loader warp needs to know of the cache.
struct Pages {
    const CUtensorMap *map;
    int ps_log2, ps_mask, num_pages, Hkv;
    int box_rows, box_log2, bpt;  // rows of a page box, boxes per tile
    bool small;                   // pages under 8 tokens: rows gathered four at a time
    __device__ __forceinline__ Pages(const Args &a, const CUtensorMap *m, int kernel, int BN)
        : map(m), ps_log2(a.ps_log2), ps_mask((1 << a.ps_log2) - 1), num_pages(a.num_pages), Hkv(a.Hkv),
          box_rows(1 << a.box_log2[kernel]), box_log2(a.box_log2[kernel]), bpt(BN >> a.box_log2[kernel]),
          small(a.box_log2[kernel] < 3) {}
};

// Copies one K or V tile after another of an item to a ring's stages, tiles of BN keys stored as
// 64-column blocks of BN x 128 bytes with the 128-byte swizzle: copies c0 .. c1 - 1 of each tile.
//  * Pages of 8 tokens and more: one TMA box per page (of up to BN rows) and 64 columns.  Page ids
//    come in warp-wide windows of 32 boxes, the next window loaded ahead.
//  * Smaller pages: tile::gather4 of four arbitrary rows of 64 columns (the pool seen as rows of one
//    head, slot * Hkv + head).  Page ids of the next tile are loaded ahead.
// A page id outside the pool is flagged and something else inside the pool (or zeros) copied.
// Keys have numbers up to 2^31 - 1, and those looked ahead for lie up to 8192 behind the last, so such
// sums are compared without sign.
template <int D, int BN>
struct Copier {
    static constexpr int NBLK = D / 64;
    int ids[4], box, pg_cur, pg_nxt;
    const int32_t *prow;
    int key0, kend, nt, g;

    __device__ __forceinline__ int window(const Pages &p, int w) const {
        const unsigned key = key0 + ((32u * w + (threadIdx.x & 31u)) << p.box_log2);
        return key < static_cast<unsigned>(kend) ? prow[key >> p.ps_log2] : 0;
    }
    __device__ __forceinline__ void load_ids(const Pages &p, int j) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const unsigned key = static_cast<unsigned>(key0 + j * BN) + 4u * lane + r;
            ids[r] = 4 * lane < BN && key < static_cast<unsigned>(kend) ? prow[key >> p.ps_log2] : -1;
        }
    }
    __device__ __forceinline__ void begin(const Args &a, const Pages &p, const Item &it) {
        prow = a.page_table + static_cast<int64_t>(it.row) * a.pt_stride;
        key0 = it.key0;
        kend = it.kend;
        nt = it.nt;
        g = it.g;
        box = 0;
        if (p.small) {
            load_ids(p, 0);
        } else {
            pg_cur = window(p, 0);
            pg_nxt = window(p, 1);
        }
    }
    // Tile j: what to copy is worked out before `ready` waits for the stage.
    template <typename Ready>
    __device__ __forceinline__ bool tile(const Pages &p, int j, uint32_t dst, uint32_t full, uint64_t policy, int c0,
                                         int c1, volatile int *bad_flag, Ready ready) {
        const int lane = threadIdx.x & 31;
        const int k0 = key0 + j * BN, nkeys = min(BN, kend - k0);
        if (!p.small) {
            const int i = c0 + lane, blk = i % NBLK, unit = i / NBLK;  // this lane's box
            const int end = min(c1, ((nkeys + p.box_rows - 1) >> p.box_log2) * NBLK);  // at most 32 boxes
            const int pg = __shfl_sync(0xffffffffu, pg_cur, (box & 31) + min(unit, p.bpt - 1));
            const bool bad = i < end && (pg < 0 || pg >= p.num_pages);
            const bool any_bad = __any_sync(0xffffffffu, bad);
            // (a box before the pool, which the copy engine fills with zeros)
            const int in_page = static_cast<int>((static_cast<unsigned>(k0) + unit * p.box_rows) & p.ps_mask);
            const int row = bad ? -p.box_rows : (pg << p.ps_log2) + in_page;
            box += p.bpt;
            if ((box & 31) == 0) {  // the next window
                pg_cur = pg_nxt;
                pg_nxt = window(p, (box >> 5) + 1);
            }
            if (!ready()) return false;
            if (lane == 0) {
                if (any_bad) *bad_flag = 1;
                mbar_arrive_expect_tx(full, static_cast<uint32_t>(max(end - c0, 0) * p.box_rows * 128));
            }
            __syncwarp();
            if (i < end)
                tma_load_3d(dst + blk * (BN * 128) + unit * p.box_rows * 128, p.map, full, blk * 64, g, row, policy);
        } else {
            bool bad = false;
            int rows[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const unsigned key = static_cast<unsigned>(k0) + 4u * lane + r;
                const bool there = 4 * lane < BN && key < static_cast<unsigned>(kend);
                const bool fine = there && ids[r] >= 0 && ids[r] < p.num_pages;
                bad |= there && !fine;
                rows[r] = (fine ? (ids[r] << p.ps_log2) + static_cast<int>(key & p.ps_mask) : 0) * p.Hkv + g;
            }
            const bool any_bad = __any_sync(0xffffffffu, bad);
            if (j + 1 < nt) load_ids(p, j + 1);
            const int end = min(c1, (nkeys + 3) / 4 * NBLK);
            if (!ready()) return false;
            if (lane == 0) {
                if (any_bad) *bad_flag = 1;
                mbar_arrive_expect_tx(full, static_cast<uint32_t>(max(end - c0, 0) * 512));
            }
            __syncwarp();
#pragma unroll 1
            for (int i0 = c0; i0 < end; i0 += 32) {
                const int i = i0 + lane, blk = i % NBLK, unit = i / NBLK;
                int r[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) r[q] = __shfl_sync(0xffffffffu, rows[q], unit & 31);
                if (i < end)
                    tma_gather4(dst + blk * (BN * 128) + unit * 512, p.map, full, blk * 64, r[0], r[1], r[2], r[3], policy);
            }
        }
        __syncwarp();
        return true;
    }
};

// ---------------------------------------------------------------- host side
// Launch one of the two kernels for head size D (defined in common_keys_tiles.cu and
// common_keys_few.cu); false when a CUDA call failed.
template <int D, bool LONG>
bool launch_tiles(const Args &a, const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap,
                  const pkv_host::DeviceInfo &dev, cudaStream_t stream);
template <int D, bool LONG>
bool launch_few(const Args &a, const CUtensorMap &kmap, const CUtensorMap &vmap, const pkv_host::DeviceInfo &dev,
                cudaStream_t stream);

}  // namespace ck
}  // namespace pkv
