// decode_weights.cu -- paged decode attention that also adds up how much softmax
// weight every cached key receives.
//
// miniVLLM "Engine Architecture", prepare_decode: one query token per sequence,
// block_tables map its keys to pages.  For query head h of KV head g,
//     p[h][j] = exp(scale q[h].k[j]) / sum_j' exp(scale q[h].k[j'])
//     out[h] = sum_j p[h][j] v[j],     acc[g][j] += sum_{h of g} p[h][j].
//
// Memory-bound on K and V, each read once.  A key's weight needs the maximum and
// the sum over all keys, which exist only at the end, so every score is written
// to a scratch row (4 bytes per key and query head, against 4 * head_dim bytes
// of K and V per key and KV head) and turned into weights from there by a second
// kernel, out of L2.  Reading K a second time would cost half of the first pass
// again.
//
//  * The work is cut as in decode.cu: segments (sequence, KV head) end to end,
//    equal ranges of units per persistent block; pieces of cut segments leave
//    partial states that the second kernel joins.
//  * Producer warps stage 16 KB tiles of K and V rows with TMA (page boxes, or
//    four rows per copy for pages under 8 tokens), two blocks per SM, four tiles
//    in flight each.
//  * Each of four consumer warps takes 8 keys (16 at head size 64) of a tile and
//    multiplies with mma.sync, heads in the rows: any number of query heads up to
//    8 costs the same, where an FMA loop costs 4 * heads flops per byte and is no
//    longer memory-bound from 4 heads on (256 sequences of 1-8192 keys, 32 query /
//    4 KV heads, page size 1: 237 us with FMA loops and no scores, 118 us here, the
//    second kernel included).
//    tcgen05 needs 128 rows; the 8 used here would leave it 94 % idle, and its
//    operands must lie in shared-memory layouts that row-by-row gathers do not
//    write.  The tensor pipe is 18-26 % busy as it is.
//    Both products contract in an order of their own: the head elements are dealt
//    to lanes in 16-byte pieces, the output columns in runs of 8, so that every
//    shared-memory read is 16 bytes wide and no operand is transposed.
//  * The softmax weights enter the second product with all of their 24 bits, as three
//    bf16 terms p = 2 half + mid + low: a key stands twice in the contraction, times
//    half and half in rows 0-7 and times mid and low in rows 8-15, which the 8 heads
//    do not use.  (half twice, and not p and 0: 0 times an infinite V would be NaN.)
//    The tensor core cuts off what its fp32 accumulators cannot hold where an FMA
//    rounds, so a long sum drifts towards zero; after every 32 instructions the
//    accumulators are added to a total in shared memory and start again.  Error of
//    the output before it is rounded to bf16, 10^6 keys: 3e-7, or 4e-7 where V has
//    one sign; without totals 1e-6 and 3e-6, growing with the length; with weights of
//    two terms 2.7e-6 (the FMA kernel, on V of either sign, 2.6e-7).
//    Against two terms and no totals, same GPU: batch below 201.5 -> 202.2 us, long
//    contexts 83.1 -> 84.2, 8 heads per KV head 113.3 -> 118.2, small 10.4 -> 10.6.
//
// Measured on several GPUs (copy peak 6.8 TB/s): 128 sequences of 512-4096 keys, 16 / 8
// heads of 128, 1.23 GB: 198-202 us, 6.1-6.2 TB/s; 8 sequences of 16-32 K keys, 32 / 8
// heads of 64, 415 MB: 76-84 us, 4.9-5.4 TB/s.  Without scores and second kernel the main
// kernel (its form with weights of two terms) read the batch's K and V, 1.21 GB, at the
// copy peak, in 177 us, and the long contexts', 403 MB, in 64 us, 0.93 of it.
#include <math.h>

#include <mutex>

#include "decode_common.cuh"

namespace pkv {
namespace decode_weights {

using decode::kLog2e;
using decode::kMaxBatch;
using decode::kNegBig;
using decode::Part;
using decode::Piece;

constexpr int kConsumerWarps = 4;
constexpr int kProducerWarps = 4;
constexpr int kConsumers = kConsumerWarps * 32;
constexpr int kThreads = (kConsumerWarps + kProducerWarps) * 32;
constexpr int kMaxHeads = 8;  // query heads per KV head
constexpr int kStages = 4;
// Units for a segment's fixed work.  Ragged batch above, with weights of two terms: 3 / 4 /
// 5 / 6 units 125 / 114 / 114 / 116 us; the others do not care.
constexpr int kLead = 4;
// A block takes at least so many units, since the pieces of a segment have to be joined
// again.  1 / 4 / 8 / 16 units: 5 sequences of 150-14062 keys, 8 query heads on one KV
// head 16.9 / 15.4 / 15.6 / 19.7 us; one of 500 keys 9.1 / 10.3 / 13.6 / 17.3 us.
constexpr int kMinUnits = 4;
// Blocks that get work; each of them gets a unit.
__device__ __forceinline__ int blocks_of(int W, int grid) { return min(grid, max(1, W / kMinUnits)); }

constexpr int kCtasPerSm = 2;
// A block launches with 128 registers per thread; the producers give up all but
// 80 and the consumers take 176 (128 x (176 + 80) = 256 x 128).
constexpr int kConsumerRegs = 176;
constexpr int kProducerRegs = 80;
static_assert(kConsumers * kConsumerRegs + kProducerWarps * 32 * kProducerRegs <= kThreads * (65536 / (2 * kThreads)),
              "register split exceeds the registers of a block at two blocks per SM");

template <int D>
struct Shape {
    static constexpr int T = 4096 / D;               // keys of a tile: 8 KB of K, 8 KB of V
    static constexpr int N = T / (kConsumerWarps * 8);  // 8-key groups per warp: 1 or 2
    static constexpr int CH = D / 32;                // 16-byte pieces of a K row per lane
    static constexpr int VC = D / 64;                // 16-byte pieces of a V row per lane
    static constexpr int TILE_BYTES = T * D * 2;
    static constexpr int FLUSH = 32 / N;             // tiles that one accumulator sums up
};

template <int D>
struct Smem {
    static constexpr int Q_BYTES = kMaxHeads * D * 2;
    static constexpr int STAGE_BYTES = 2 * Shape<D>::TILE_BYTES + Q_BYTES;
    static constexpr int RING = kStages * STAGE_BYTES;
    static constexpr int RED_O = kConsumerWarps * kMaxHeads * D * 4;
    static constexpr int RED_ML = kConsumerWarps * kMaxHeads * 2 * 4;
    static constexpr int BARS = 2 * kStages * 8;
    static constexpr int FLAGS = (kStages * kProducerWarps + 4) * 4;
    static constexpr int FIXED = RING + RED_O + RED_ML + BARS + FLAGS;
    // + tile offsets [batch + 1] and sequence lengths [batch], int32
    static size_t bytes(int batch) { return 1024 + FIXED + static_cast<size_t>(2 * batch + 1) * 4; }
};

// The running sums, one row per request, and the scratch rows of scores
// [b][query head][row_len], each on a 128-byte boundary.
struct Sums {
    float *acc;
    const int32_t *rows;
    int64_t num_rows, stride;
    float *scores;
    int64_t row_len;
};

// Forget a 128-byte line of global memory: what it holds becomes undefined and is not
// written back from L2.  (The scores, once read, with weights of two terms: 203.5 ->
// 197.5 us for the batch above, 81.6 -> 77.0 us for the long contexts.)
__device__ __forceinline__ void discard_line(const float *line) {
    asm volatile("discard.global.L2 [%0], 128;" ::"l"(line) : "memory");
}

// decode::next_piece in 32 bits (units do not pass them, and a 64-bit division is a
// call of a hundred instructions).
__device__ __forceinline__ bool next_piece(int &pos, int end, int start, const int32_t *prefix, int B, int Hkv,
                                           Piece &p) {
    if (pos >= end) return false;
    const int b = decode::owner_search(prefix, B, pos);
    const unsigned nu = static_cast<unsigned>(prefix[b + 1] - prefix[b]) / static_cast<unsigned>(Hkv);
    const unsigned rel = pos - prefix[b];
    const unsigned g = rel / nu, u0 = rel - g * nu;
    const int seg_end = prefix[b] + static_cast<int>((g + 1) * nu);
    const int pend = min(end, seg_end);
    p.b = b;
    p.g = g;
    p.t0 = max(static_cast<int>(u0) - kLead, 0);
    p.t1 = static_cast<int>(u0) + (pend - pos) - kLead;
    p.nt = static_cast<int>(nu) - kLead;
    p.whole = u0 <= kLead && pend == seg_end;
    p.block_first = pos == start;
    pos = pend;
    return true;
}

__device__ __forceinline__ void mma_k16(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    decode_weights_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                          const __nv_bfloat16 *__restrict__ q, const int32_t *__restrict__ page_table,
                          int64_t pt_stride, const int32_t *__restrict__ seq_lens, int B, int Hkv, int G, int ps_log2,
                          int box_rows, int64_t num_pages, float scale_log2, int64_t max_len,
                          float *__restrict__ ws_part, float2 *__restrict__ ws_state, int32_t *__restrict__ ws_prefix,
                          int32_t *dev_status,
                          __nv_bfloat16 *__restrict__ out, const Sums sums) {
    using S = Shape<D>;
    using M = Smem<D>;
    constexpr int T = S::T, N = S::N, CH = S::CH, VC = S::VC;
    const int Hq = Hkv * G;
    const int64_t row_cap = pt_stride << ps_log2;
    const int64_t cap = max_len < row_cap ? max_len : row_cap;
    const int part_floats = decode::part_stride(G, D);

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *ring = smem;
    float *red_o = reinterpret_cast<float *>(smem + M::RING);
    float *red_ml = reinterpret_cast<float *>(smem + M::RING + M::RED_O);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + M::RING + M::RED_O + M::RED_ML);
    int *flags = reinterpret_cast<int *>(smem + M::FIXED - M::FLAGS);  // [stage][producer warp]: a bad page
    volatile int *abort_flag = flags + kStages * kProducerWarps;
    int32_t *prefix = reinterpret_cast<int32_t *>(smem + M::FIXED);
    int32_t *lens = prefix + (B + 1);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool small = box_rows < 8;  // pages too short for boxes: rows gathered four at a time
    grid_dependency_wait();
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&bars[s]), small ? static_cast<uint32_t>(kProducerWarps) : 1u);  // full
            mbar_init(smem_u32(&bars[kStages + s]), kConsumerWarps);                            // empty
        }
        for (int i = 0; i < kStages * kProducerWarps; ++i) flags[i] = 0;
        *abort_flag = 0;
        fence_mbar_init();
    }
    // red_ml doubles as the scan scratch before any piece is reduced
    decode::build_prefix<kThreads, kLead>(prefix, lens, seq_lens, B, Hkv, cap, T, reinterpret_cast<int32_t *>(red_ml));
    if (blockIdx.x == 0)
        for (int b = tid; b <= B; b += kThreads) ws_prefix[b] = prefix[b];
    // sequences without keys: zeros, or NaN for a bad length
    for (int b = blockIdx.x; b < B; b += gridDim.x) {
        if (tid == 0 && sums.rows && sums.rows[b] >= sums.num_rows && dev_status)
            atomicOr(dev_status, PKV_DEV_BAD_ROW);
        if (prefix[b + 1] != prefix[b]) continue;
        const bool bad = lens[b] < 0 || lens[b] > cap;
        if (bad && tid == 0 && dev_status) atomicOr(dev_status, PKV_DEV_BAD_SEQLEN);
        for (int i = tid; i < Hq * D; i += kThreads)
            out[(int64_t)b * Hq * D + i] = __float2bfloat16_rn(bad ? __int_as_float(0x7fc00000) : 0.f);
    }

    const Part part{prefix[B], blocks_of(prefix[B], gridDim.x)};
    if (part.W == 0 || static_cast<int>(blockIdx.x) >= part.grid) return;
    const int my_start = static_cast<int>(part.start(blockIdx.x));
    const int my_end = static_cast<int>(part.start(blockIdx.x + 1));

    if (warp >= kConsumerWarps) {
        // ------------------------------------------------------------ producers
        // Page boxes are issued by warp 4; gathers of K by warps 4 and 5, of V by
        // warps 6 and 7 (a warp's TMA issue rate limits four-row copies).
        const int pw = warp - kConsumerWarps;
        regs_decrease<kProducerRegs>();
        if (pw > 0 && !small) return;
        const uint64_t policy = l2_evict_first_policy();
        if (lane == 0) {
            prefetch_tmap(&kmap);
            prefetch_tmap(&vmap);
        }
        const int ps_mask = (1 << ps_log2) - 1;
        const uint32_t box_bytes = static_cast<uint32_t>(box_rows) * D * 2;
        constexpr int NH = T / 8;         // gathers per producer warp and tile
        static_assert(NH <= 32, "one gather per lane");
        const int gi = (pw & 1) * NH + lane % NH;
        int pos = my_start;
        Piece p;
        uint32_t it = 0;
        bool ok = true;
        const int bpt = T / box_rows;     // boxes per tile
        while (ok && next_piece(pos, my_end, my_start, prefix, B, Hkv, p)) {
            if (p.t1 <= p.t0) continue;  // lead units only: nothing to load
            const int L = lens[p.b];
            const int32_t *prow = page_table + (int64_t)p.b * pt_stride;
            // page ids: for boxes in warp-wide windows of 32, the next window a
            // window ahead; for gathers this lane's four keys, a tile ahead
            auto load_window = [&](int w) -> int {
                const int key = (32 * w + lane) * box_rows;
                return key < L ? prow[key >> ps_log2] : 0;
            };
            int w_cur = 0, pg_cur = 0, pg_nxt = 0;
            int ids[4] = {0, 0, 0, 0};
            auto load_ids = [&](int tile) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int key = tile * T + 4 * gi + r;
                    ids[r] = key < L ? prow[key >> ps_log2] : 0;
                }
            };
            if (small) {
                load_ids(p.t0);
            } else {
                w_cur = (p.t0 * bpt) >> 5;
                pg_cur = load_window(w_cur);
                pg_nxt = load_window(w_cur + 1);
            }
            for (int tile = p.t0; tile < p.t1; ++tile, ++it) {
                const int s = it % kStages;
                const uint32_t ph = (it / kStages) & 1;
                const int tok0 = tile * T;
                const int ntok = min(T, L - tok0);
                const bool first = tile == p.t0;
                uint8_t *st = ring + s * M::STAGE_BYTES;
                const uint32_t full = smem_u32(&bars[s]);
                const uint32_t q_bytes = first && pw == 0 ? static_cast<uint32_t>(G * D * 2) : 0u;
                int rows[4] = {0, 0, 0, 0};
                bool bad = false;
                if (small) {
                    // keys past the end take the row of this tile's first key, which
                    // exists (the consumers never use them)
                    const int id0 = __shfl_sync(0xffffffffu, ids[0], 0);
                    const int key0 = (pw & 1) * NH * 4;  // first key of this warp's half
                    const int64_t slot0 = ((int64_t)id0 << ps_log2) + ((tok0 + key0) & ps_mask);
                    if (key0 < ntok && (id0 < 0 || id0 >= num_pages)) bad = true;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int key = 4 * gi + r;
                        int64_t slot = slot0;
                        if (key < ntok) {
                            if (ids[r] < 0 || ids[r] >= num_pages) bad = true;
                            slot = ((int64_t)ids[r] << ps_log2) + ((tok0 + key) & ps_mask);
                        }
                        rows[r] = static_cast<int>(slot * Hkv + p.g);
                    }
                    if (tile + 1 < p.t1) load_ids(tile + 1);
                }
                if (it >= kStages &&
                    !mbar_wait_warp(smem_u32(&bars[kStages + s]), ph ^ 1, abort_flag, dev_status)) {
                    ok = false;
                    break;
                }
                if (!small) {
                    const int nbox = (ntok + box_rows - 1) / box_rows;
                    const int b0 = tile * bpt;
                    if ((b0 >> 5) != w_cur) {
                        w_cur = b0 >> 5;
                        pg_cur = pg_nxt;
                        pg_nxt = load_window(w_cur + 1);
                    }
                    const int pg = __shfl_sync(0xffffffffu, pg_cur, (b0 + (lane % bpt)) & 31);
                    bad = __any_sync(0xffffffffu, lane < nbox && (pg < 0 || pg >= num_pages));
                    if (lane == 0) {
                        flags[s * kProducerWarps] = bad;
                        mbar_arrive_expect_tx(full, (bad ? 0u : 2u * box_bytes * nbox) + q_bytes);
                    }
                    __syncwarp();
                    if (!bad && lane < nbox) {
                        const int row = (pg << ps_log2) + ((tok0 + lane * box_rows) & ps_mask);
                        tma_load_3d(smem_u32(st + lane * box_bytes), &kmap, full, 0, p.g, row, policy);
                        tma_load_3d(smem_u32(st + S::TILE_BYTES + lane * box_bytes), &vmap, full, 0, p.g, row, policy);
                    }
                } else {
                    // a warp whose half of the tile lies past the end copies nothing
                    const bool any = (pw & 1) * NH * 4 < ntok;
                    bad = __any_sync(0xffffffffu, bad);
                    const bool copy = any && !bad;
                    if (lane == 0) {
                        flags[s * kProducerWarps + pw] = bad;
                        mbar_arrive_expect_tx(full, (copy ? static_cast<uint32_t>(S::TILE_BYTES / 2) : 0u) + q_bytes);
                    }
                    __syncwarp();
                    if (copy && lane < NH)
                        tma_gather4(smem_u32(st) + (pw < 2 ? 0u : S::TILE_BYTES) + gi * 4 * D * 2,
                                    pw < 2 ? &kmap : &vmap, full, 0, rows[0], rows[1], rows[2], rows[3], policy);
                }
                if (first && pw == 0 && lane == 0)
                    bulk_load(smem_u32(st + 2 * S::TILE_BYTES), q + ((int64_t)p.b * Hq + (int64_t)p.g * G) * D,
                              G * D * 2, full);
            }
        }
        return;
    }

    // ---------------------------------------------------------------- consumers
    regs_increase<kConsumerRegs>();
    // lane (r, c): row r of the products' heads, keys or output columns, c the
    // quarter of the contraction
    const int r = lane >> 2, c = lane & 3;
    const bool odd = c & 1;
    uint32_t qf[CH][4];   // pieces c, c + 4, .. of query head r
    float o[VC][8][4];    // (piece, column): rows r and r + 8, output columns of pieces VC * (2c), VC * (2c + 1)
    float m, l;           // of head r: reference, and this lane's share of the sum
    float m_total;        // the reference that `total` goes by
    // rows r of o of all tiles but the last FLUSH, in a piece of so many: a lane's own
    float4 *total = reinterpret_cast<float4 *>(red_o + warp * kMaxHeads * D) + lane;
    static_assert(32 * 4 * VC * sizeof(float4) == kMaxHeads * D * sizeof(float), "where the warp's rows are joined later");
    int pos = my_start;
    Piece p;
    uint32_t it = 0;
    bool ok = true;
    while (ok && next_piece(pos, my_end, my_start, prefix, B, Hkv, p)) {
        if (p.t1 <= p.t0) continue;  // lead units only: nothing to do
        const int L = lens[p.b];
        const int64_t head0 = (int64_t)p.b * Hq + (int64_t)p.g * G;  // the segment's first query head
        float *srow = sums.scores + (head0 + r) * sums.row_len;
        m = m_total = kNegBig;
        l = 0.f;
#pragma unroll
        for (int v = 0; v < VC; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e) o[v][e][0] = o[v][e][1] = o[v][e][2] = o[v][e][3] = 0.f;
        bool bad_piece = false;
        for (int tile = p.t0; tile < p.t1; ++tile, ++it) {
            const int s = it % kStages;
            const uint32_t ph = (it / kStages) & 1;
            if (!mbar_wait_warp(smem_u32(&bars[s]), ph, abort_flag, dev_status)) {
                ok = false;
                break;
            }
            const uint32_t kbase = smem_u32(ring + s * M::STAGE_BYTES);
            const uint32_t vbase = kbase + S::TILE_BYTES;
            if (small) {
                const int4 f = *reinterpret_cast<const int4 *>(flags + s * kProducerWarps);
                if (f.x | f.y | f.z | f.w) bad_piece = true;
            } else if (flags[s * kProducerWarps]) {
                bad_piece = true;
            }
            if (tile == p.t0) {
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    uint4 w = make_uint4(0u, 0u, 0u, 0u);
                    if (r < G) w = lds128(vbase + S::TILE_BYTES + (r * D + (c + 4 * i) * 8) * 2);
                    qf[i][0] = w.x, qf[i][1] = w.y, qf[i][2] = w.z, qf[i][3] = w.w;
                }
            }
            const int tok0 = tile * T;
            const bool full_tile = tok0 + T <= L;
            // scores of head r, keys 8 (warp N + n) + 2 c and the next
            float sc[N][4];
#pragma unroll
            for (int n = 0; n < N; ++n) {
                uint4 kf[CH];
#pragma unroll
                for (int i = 0; i < CH; ++i)
                    kf[i] = lds128(kbase + (((warp * N + n) * 8 + r) * D + (c + 4 * i) * 8) * 2);
                // two chains of half the length
                float a[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    mma_k16(a, qf[i][0], 0u, qf[i][1], 0u, kf[i].x, kf[i].y);
                    mma_k16(b, qf[i][2], 0u, qf[i][3], 0u, kf[i].z, kf[i].w);
                }
                sc[n][0] = a[0] + b[0];
                sc[n][1] = a[1] + b[1];
            }
            // V rows of this lane's keys 2c, 2c + 1 of each group: pieces VC r ..; with
            // two of them odd quarters read the second first, so that the lanes of a
            // quarter warp spread over twice the banks
            uint4 vf[2 * N][VC];
#pragma unroll
            for (int x = 0; x < 2 * N; ++x) {
                const int key = (warp * N + x / 2) * 8 + 2 * c + (x & 1);
#pragma unroll
                for (int v = 0; v < VC; ++v) {
                    const int piece = VC * r + (VC == 2 && odd ? 1 - v : v);
                    vf[x][v] = lds128(vbase + (key * D + piece * 8) * 2);
                }
                if (!full_tile && tok0 + key >= L) {
                    // stale data, maybe NaN: 0 * NaN would poison the sum
#pragma unroll
                    for (int v = 0; v < VC; ++v) vf[x][v] = make_uint4(0u, 0u, 0u, 0u);
                }
                if (VC == 2) {
                    const uint4 t0 = vf[x][0], t1 = vf[x][VC - 1];
                    vf[x][0] = odd ? t1 : t0;
                    vf[x][VC - 1] = odd ? t0 : t1;
                }
            }
            __syncwarp();  // the tile is in registers
            if (lane == 0) mbar_arrive(smem_u32(&bars[kStages + s]));
            float mt = kNegBig;
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int j = tok0 + (warp * N + n) * 8 + 2 * c;
                float s0 = sc[n][0] * scale_log2, s1 = sc[n][1] * scale_log2;
                if (!full_tile) {  // past the sequence end: score -inf, so p = 0
                    if (j >= L) s0 = -INFINITY;
                    if (j + 1 >= L) s1 = -INFINITY;
                }
                // (the score row has room for a pair's second key past the end)
                if (r < G && j < L) *reinterpret_cast<float2 *>(srow + j) = make_float2(s0, s1);
                sc[n][0] = s0;
                sc[n][1] = s1;
                mt = fmax3(mt, s0, s1);
            }
            // online softmax with a lazy reference: m only moves when a score exceeds
            // it by more than 8 (a factor of 2^8), so rescaling is rare
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
            if (__any_sync(0xffffffffu, mt > m + 8.0f)) {
                const float m_new = mt > m + 8.0f ? mt : m;
                const float alpha = ex2(m - m_new);
                m = m_new;
                l *= alpha;
#pragma unroll
                for (int v = 0; v < VC; ++v)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
#pragma unroll
                        for (int x = 0; x < 4; ++x) o[v][e][x] *= alpha;
            }
            // p = 2 half + mid + low, each difference exact
            uint32_t half[N], mid[N], low[N];
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const float2 p = make_float2(ex2(sc[n][0] - m), ex2(sc[n][1] - m));
                l += p.x + p.y;
                const float2 h = fmul2(p, make_float2(0.5f, 0.5f));
                half[n] = pack_bf16x2(h.x, h.y);
                const float2 rest = ffma2(bf16x2_to_f2(half[n]), make_float2(-2.f, -2.f), p);
                mid[n] = pack_bf16x2(rest.x, rest.y);
                const float2 last = ffma2(bf16x2_to_f2(mid[n]), make_float2(-1.f, -1.f), rest);
                low[n] = pack_bf16x2(last.x, last.y);
            }
#pragma unroll
            for (int v = 0; v < VC; ++v) {
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const uint32_t *x0 = reinterpret_cast<const uint32_t *>(&vf[2 * n][v]);
                    const uint32_t *x1 = reinterpret_cast<const uint32_t *>(&vf[2 * n + 1][v]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t vv = __byte_perm(x0[e / 2], x1[e / 2], (e & 1) ? 0x7632u : 0x5410u);
                        mma_k16(o[v][e], half[n], mid[n], half[n], low[n], vv, vv);
                    }
                }
            }
            if ((tile - p.t0) % S::FLUSH == S::FLUSH - 1) {
                const bool more = tile - p.t0 >= S::FLUSH;
                const float f = ex2(m_total - m);
                m_total = m;
#pragma unroll
                for (int v = 0; v < VC; ++v)
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        float4 *at = total + 32 * (4 * v + e / 2);
                        float4 t = make_float4(o[v][e][0], o[v][e][1], o[v][e + 1][0], o[v][e + 1][1]);
                        if (more) {
                            const float4 u = *at;
                            t = make_float4(fmaf(u.x, f, t.x), fmaf(u.y, f, t.y), fmaf(u.z, f, t.z), fmaf(u.w, f, t.w));
                        }
                        *at = t;
                        o[v][e][0] = o[v][e][1] = o[v][e + 1][0] = o[v][e + 1][1] = 0.f;
                    }
            }
        }
        if (!ok) break;

        // ---- join the warps' states of this piece
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (p.t1 - p.t0 >= S::FLUSH) {
            const float f = ex2(m_total - m);
#pragma unroll
            for (int v = 0; v < VC; ++v)
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float4 t = total[32 * (4 * v + e / 2)];
                    o[v][e][0] = fmaf(t.x, f, o[v][e][0]), o[v][e][1] = fmaf(t.y, f, o[v][e][1]);
                    o[v][e + 1][0] = fmaf(t.z, f, o[v][e + 1][0]), o[v][e + 1][1] = fmaf(t.w, f, o[v][e + 1][1]);
                }
            __syncwarp();  // the same memory takes the rows in order
        }
        if (r < G) {
            float *ro = red_o + (warp * kMaxHeads + r) * D;
#pragma unroll
            for (int v = 0; v < VC; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        // the halves' part alone is right where V is not finite
                        const float a = o[v][e][x], b = o[v][e][x + 2];
                        ro[(VC * (2 * c + x) + v) * 8 + e] = isfinite(a) ? a + b : a;
                    }
            if (c == 0) {
                red_ml[(warp * G + r) * 2 + 0] = m;
                red_ml[(warp * G + r) * 2 + 1] = l;
            }
        }
        named_bar_sync(1, kConsumers);
        const int slot = static_cast<int>(blockIdx.x) * 2 + (p.block_first ? 0 : 1);
        for (int idx = tid; idx < G * D; idx += kConsumers) {
            const int h = idx / D;
            float mx = kNegBig;
#pragma unroll
            for (int w = 0; w < kConsumerWarps; ++w) mx = fmaxf(mx, red_ml[(w * G + h) * 2]);
            float sum = 0.f, acc = 0.f;
#pragma unroll
            for (int w = 0; w < kConsumerWarps; ++w) {
                const float f = ex2(red_ml[(w * G + h) * 2] - mx);
                sum = fmaf(red_ml[(w * G + h) * 2 + 1], f, sum);
                acc = fmaf(red_o[(w * kMaxHeads + h) * D + (idx % D)], f, acc);
            }
            if (p.whole) {
                out[head0 * D + idx] = __float2bfloat16_rn(bad_piece ? __int_as_float(0x7fc00000) : acc / sum);
                if (idx % D == 0) ws_state[head0 + h] = make_float2(bad_piece ? __int_as_float(0x7fc00000) : mx, sum);
            } else {
                float *state = ws_part + (int64_t)slot * part_floats;
                state[idx] = acc;
                if (idx % D == 0) {
                    state[G * D + 2 * h] = bad_piece ? __int_as_float(0x7fc00000) : mx;
                    state[G * D + 2 * h + 1] = sum;
                }
            }
        }
        if (bad_piece && tid == 0 && dev_status) atomicOr(dev_status, PKV_DEV_BAD_PAGE);
        named_bar_sync(1, kConsumers);
    }
}

// After the main kernel, in one launch: the first main_grid blocks join the
// outputs of cut segments (block k the share of the cut at the start of the main
// kernel's block k, so that a segment in many pieces has many blocks), the others
// turn all scores into weights,
//     w[j] = sum_h 2^(score[h][j] - max_h) / sum_h,
// added to the running sums.  Both are bound by latency (a few MB, mostly in L2:
// about 12 us after the main kernel).  The weights' units are dealt to warps, so that
// all of it is short chains (prefix sums, softmax state, scores) that no other warp
// waits for.
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kJoinPerSm = 3;

// The balanced partition with its division done once and 32-bit (the prefix sums
// are).
struct Cuts {
    uint32_t q, r, n;
    __device__ __forceinline__ Cuts(uint32_t W, uint32_t parts) : q(W / parts), r(W % parts), n(parts) {}
    __device__ __forceinline__ int start(uint32_t k) const { return static_cast<int>(k * q + k * r / n); }
    // the part that holds unit x: a guess in fp32, at most a few parts off, put right
    __device__ __forceinline__ int of(int x, float parts_per_unit) const {
        int k = min(static_cast<int>(n) - 1, static_cast<int>(static_cast<float>(x) * parts_per_unit));
        while (start(k) > x) --k;
        while (start(k + 1) <= x) ++k;
        return k;
    }
};

// The partial states of a segment's pieces, its tiles in blocks k0 to k1 of the main
// kernel: the state of its first piece, and of block k's later on.
struct States {
    const float *part;
    int stride, k0, k1, slot0;
    __device__ __forceinline__ const float *of(int k) const {
        return part + (int64_t)(k == k0 ? slot0 : 2 * k) * stride;
    }
};

// (max, sum) of two disjoint sets of scores as one: returns the factors by which
// what belongs to each is to be scaled.
__device__ __forceinline__ float2 join_two(float &mx, float &sum, float mx2, float sum2) {
    const float up = fmaxf(mx, mx2);
    const float2 f = make_float2(ex2(mx - up), ex2(mx2 - up));
    sum = sum * f.x + sum2 * f.y;
    mx = up;
    return f;
}

// Maximum and sum of head h over the states k0 + first, k0 + first + step, ..; bad: one
// of them holds keys on a bad page.
__device__ __forceinline__ float2 join_states(const States &st, int E, int h, int first, int step, bool &bad) {
    constexpr int AHEAD = 4;
    float mx = kNegBig, sum = 0.f;
    for (int k = st.k0 + first; k <= st.k1; k += AHEAD * step) {
        float2 ml[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            ml[i] = k + i * step <= st.k1 ? *reinterpret_cast<const float2 *>(st.of(k + i * step) + E + 2 * h)
                                          : make_float2(kNegBig, 0.f);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            bad |= isnan(ml[i].x);
            join_two(mx, sum, ml[i].x, ml[i].y);
        }
    }
    return make_float2(mx, sum);
}

// Float4s v0 to v1 - 1 of a cut segment's output (out: the segment's), by a block:
// threads over the float4s and, as far as they go, over the states.  A state of keys on
// a bad page (maximum NaN) makes everything NaN.
template <int D>
__device__ __forceinline__ void join_outputs(const States &st, int v0, int v1, int G, __nv_bfloat16 *out) {
    __shared__ float4 s_acc[kJoinThreads];
    __shared__ float2 s_ml[kJoinThreads];
    static_assert(kJoinThreads * 4 >= kMaxHeads * D, "a thread for each float4");
    constexpr int AHEAD = 4;
    const int E = G * D;
    int span = 1;  // threads over the float4s: a power of two
    while (span < v1 - v0) span *= 2;
    const int step = kJoinThreads / span;
    const int i = threadIdx.x % span, v = min(v0 + i, v1 - 1), h = 4 * v / D;
    float mx = kNegBig, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float2 ml, float4 o) {
        const float2 f = join_two(mx, sum, ml.x, ml.y);
        acc.x = fmaf(o.x, f.y, acc.x * f.x), acc.y = fmaf(o.y, f.y, acc.y * f.x);
        acc.z = fmaf(o.z, f.y, acc.z * f.x), acc.w = fmaf(o.w, f.y, acc.w * f.x);
    };
    for (int k = st.k0 + threadIdx.x / span; k <= st.k1; k += AHEAD * step) {
        float2 ml[AHEAD];
        float4 o[AHEAD];
#pragma unroll
        for (int x = 0; x < AHEAD; ++x) {
            ml[x] = make_float2(kNegBig, 0.f);
            o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k + x * step <= st.k1) {
                const float *state = st.of(k + x * step);
                ml[x] = *reinterpret_cast<const float2 *>(state + E + 2 * h);
                o[x] = *reinterpret_cast<const float4 *>(state + 4 * v);
            }
        }
#pragma unroll
        for (int x = 0; x < AHEAD; ++x) add(ml[x], o[x]);
    }
    // the lanes of a warp with the same float4, then the warps
    for (int d = 16; d >= span; d >>= 1) {
        const float2 ml = make_float2(__shfl_xor_sync(0xffffffffu, mx, d), __shfl_xor_sync(0xffffffffu, sum, d));
        const float4 o = make_float4(__shfl_xor_sync(0xffffffffu, acc.x, d), __shfl_xor_sync(0xffffffffu, acc.y, d),
                                     __shfl_xor_sync(0xffffffffu, acc.z, d), __shfl_xor_sync(0xffffffffu, acc.w, d));
        add(ml, o);
    }
    s_acc[threadIdx.x] = acc;
    s_ml[threadIdx.x] = make_float2(mx, sum);
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < span && v0 + i < v1) {
        const int apart = max(span, 32);
        for (int x = threadIdx.x + apart; x < kJoinThreads; x += apart) add(s_ml[x], s_acc[x]);
        const float f = 1.f / sum;
        *reinterpret_cast<uint2 *>(out + 4 * v) =
            make_uint2(pack_bf16x2(acc.x * f, acc.y * f), pack_bf16x2(acc.z * f, acc.w * f));
    }
}

template <int D, int G>
__global__ void __launch_bounds__(kJoinThreads, kJoinPerSm)
    decode_weights_join_kernel(const float *__restrict__ ws_part, const float2 *__restrict__ ws_state,
                               const int32_t *__restrict__ ws_prefix, const int32_t *__restrict__ seq_lens, int B, int Hkv,
                               int main_grid, __nv_bfloat16 *__restrict__ out, const Sums sums) {
    constexpr int T = Shape<D>::T, E = G * D;
    constexpr int U = G == 1 ? 4 : G <= 4 ? 8 / G : 1;  // groups of four keys per lane and step
    extern __shared__ int32_t prefix[];  // [B + 1]
    grid_dependency_wait();  // states and scores come from the main kernel
    for (int b = threadIdx.x; b <= B; b += kJoinThreads) prefix[b] = ws_prefix[b];
    __syncthreads();
    const int W = prefix[B];
    if (W == 0) return;
    const int blocks = blocks_of(W, main_grid);
    const float per_unit = static_cast<float>(blocks) / static_cast<float>(W);
    const Cuts cuts(W, blocks);
    // the states of the segment with units s0 .. s0 + nu - 1
    auto states_of = [&](int s0, int nu) {
        States st{ws_part, decode::part_stride(G, D), cuts.of(s0 + kLead, per_unit), cuts.of(s0 + nu - 1, per_unit), 0};
        st.slot0 = 2 * st.k0 + (s0 > cuts.start(st.k0) ? 1 : 0);
        return st;
    };
    if (static_cast<int>(blockIdx.x) < main_grid) {
        // The main kernel's block begins in a segment whose tiles began before: one of
        // the cuts of that segment, with that share of its output to join.
        if (static_cast<int>(blockIdx.x) >= blocks) return;
        const int a = cuts.start(blockIdx.x);
        const int b = decode::owner_search(prefix, B, a);
        const int nu = (prefix[b + 1] - prefix[b]) / Hkv;
        const int g = (a - prefix[b]) / nu;
        const int s0 = prefix[b] + g * nu;
        if (a - s0 <= kLead) return;
        const States st = states_of(s0, nu);
        const int cut = blockIdx.x - st.k0 - 1, all = st.k1 - st.k0;
        const int v0 = E / 4 * cut / all, v1 = E / 4 * (cut + 1) / all;
        if (v0 < v1) join_outputs<D>(st, v0, v1, G, out + ((int64_t)b * Hkv + g) * E);
        return;
    }
    const int lane = threadIdx.x & 31;
    const int me = (blockIdx.x - main_grid) * kJoinWarps + (threadIdx.x >> 5);
    const Cuts mine(W, (gridDim.x - main_grid) * kJoinWarps);
    int pos = mine.start(me);
    const int start = pos, end = mine.start(me + 1);
    Piece p;
    while (next_piece(pos, end, start, prefix, B, Hkv, p)) {
        if (p.t1 <= p.t0) continue;
        const int row = sums.rows ? sums.rows[p.b] : p.b;
        const int64_t head0 = ((int64_t)p.b * Hkv + p.g) * G;
        const int L = seq_lens[p.b];
        const States st = states_of(prefix[p.b] + p.g * (p.nt + kLead), p.nt + kLead);
        // lane % G = head: its maximum and 1 / sum (maximum NaN: keys on a bad page)
        const int h = lane % G;
        float2 ml;
        bool bad = false;
        if (st.k0 == st.k1) {
            ml = ws_state[head0 + h];
            bad = isnan(ml.x);
        } else {
            ml = join_states(st, E, h, lane / G, 32 / G, bad);
#pragma unroll
            for (int o = 16; o >= G; o >>= 1)
                join_two(ml.x, ml.y, __shfl_xor_sync(0xffffffffu, ml.x, o), __shfl_xor_sync(0xffffffffu, ml.y, o));
        }
        if (__any_sync(0xffffffffu, bad) || row < 0 || row >= sums.num_rows) continue;
        const float inv = 1.f / ml.y;
        const float *scores = sums.scores + head0 * sums.row_len;
        float *acc = sums.acc + ((int64_t)row * Hkv + p.g) * sums.stride;
        const bool vec = (reinterpret_cast<uintptr_t>(acc) & 15u) == 0;
        const int stop = min(L, p.t1 * T);
        float mx[G], iv[G];
#pragma unroll
        for (int hh = 0; hh < G; ++hh) {
            mx[hh] = __shfl_sync(0xffffffffu, ml.x, hh);
            iv[hh] = __shfl_sync(0xffffffffu, inv, hh);
        }
        // U groups of four keys per lane and step, all their loads in flight together
        for (int jb = p.t0 * T; jb < stop; jb += 128 * U) {
            const int j0 = jb + 4 * lane;
            float4 w[U], x[U][G];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j = j0 + 128 * u;
                const int at = j < stop ? j : jb;  // a group that exists
#pragma unroll
                for (int hh = 0; hh < G; ++hh)
                    x[u][hh] = *reinterpret_cast<const float4 *>(scores + hh * sums.row_len + at);
                w[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (vec && j + 4 < L) {
                    if (j < stop) w[u] = *reinterpret_cast<const float4 *>(acc + j);
                } else if (j < stop) {  // the newest key's old sum is not read
                    if (j + 0 < L - 1) w[u].x = acc[j];
                    if (j + 1 < L - 1) w[u].y = acc[j + 1];
                    if (j + 2 < L - 1) w[u].z = acc[j + 2];
                    if (j + 3 < L - 1) w[u].w = acc[j + 3];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j = j0 + 128 * u;
                float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int hh = 0; hh < G; ++hh) {
                    t.x = fmaf(ex2(x[u][hh].x - mx[hh]), iv[hh], t.x);
                    t.y = fmaf(ex2(x[u][hh].y - mx[hh]), iv[hh], t.y);
                    t.z = fmaf(ex2(x[u][hh].z - mx[hh]), iv[hh], t.z);
                    t.w = fmaf(ex2(x[u][hh].w - mx[hh]), iv[hh], t.w);
                }
                t.x += w[u].x, t.y += w[u].y, t.z += w[u].z, t.w += w[u].w;
                if (j >= stop) break;
                if (vec && j + 4 <= L) {
                    *reinterpret_cast<float4 *>(acc + j) = t;
                } else {
                    acc[j] = t.x;
                    if (j + 1 < L) acc[j + 1] = t.y;
                    if (j + 2 < L) acc[j + 2] = t.z;
                    if (j + 3 < L) acc[j + 3] = t.w;
                }
            }
            // the scores are used up: their lines need not go to memory.  (A line is
            // 32 keys of one head, all of them this warp's: a tile is 32 or 64 keys.)
            __syncwarp();
#pragma unroll
            for (int u = 0; u < U; ++u)
                if ((lane & 7) == 0 && j0 + 128 * u < stop)
#pragma unroll
                    for (int hh = 0; hh < G; ++hh) discard_line(scores + hh * sums.row_len + j0 + 128 * u);
        }
    }
}

// ---------------------------------------------------------------- host side
// Workspace: prefix sums, two partial states per block, a softmax state per query
// head, the score rows.
struct Layout {
    size_t part, state, scores, bytes;
    int64_t row_len;
};
static Layout layout_of(int grid, int batch, int Hq, int Hkv, int D, int max_len) {
    auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
    Layout w;
    const int G = Hq / Hkv;
    w.row_len = ((int64_t)max_len + 31) / 32 * 32;
    w.part = up((static_cast<size_t>(batch) + 1) * sizeof(int32_t));
    w.state = w.part + up(static_cast<size_t>(grid) * 2 * decode::part_stride(G, D) * sizeof(float));
    w.scores = w.state + up(static_cast<size_t>(batch) * Hq * sizeof(float2));
    w.bytes = w.scores + static_cast<size_t>(batch) * Hq * w.row_len * sizeof(float) + 128;  // (rows start on 128)
    return w;
}

template <int D>
static bool prepare(const pkv_host::DeviceInfo &dev) {
    static std::mutex mu;
    static bool ready[64];
    std::lock_guard<std::mutex> lk(mu);
    if (!ready[dev.device]) {
        const size_t most = Smem<D>::bytes(kMaxBatch);
        if (most > static_cast<size_t>(dev.max_smem_optin) ||
            cudaFuncSetAttribute(decode_weights_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(most)) != cudaSuccess)
            return false;
        ready[dev.device] = true;
    }
    return true;
}

template <int D>
static pkv_status launch(const pkv_bf16 *q, const pkv_bf16 *k_cache, const pkv_bf16 *v_cache,
                         const int32_t *page_table, int64_t pt_stride, const int32_t *seq_lens, int B, int Hq, int Hkv,
                         int page_size, int64_t num_pages, float scale, Sums sums, int max_len, void *workspace,
                         int32_t *dev_status, pkv_bf16 *out, const pkv_host::DeviceInfo &dev, cudaStream_t stream) {
    if (!prepare<D>(dev)) return PKV_ECUDA;
    const int T = Shape<D>::T;
    const int box_rows = page_size < T ? page_size : T;
    CUtensorMap kmap, vmap;
    const int64_t slots = num_pages * page_size;
    if (box_rows >= 8) {  // page boxes
        if (!pkv_host::encode_kv_map(&kmap, k_cache, slots, Hkv, D, D, box_rows, false) ||
            !pkv_host::encode_kv_map(&vmap, v_cache, slots, Hkv, D, D, box_rows, false))
            return PKV_EINVAL;
    } else {  // rows gathered four at a time
        if (slots * Hkv > 0x7fffffffll) return PKV_EUNSUPPORTED;
        if (!pkv_host::encode_rows_map(&kmap, k_cache, slots * Hkv, D) ||
            !pkv_host::encode_rows_map(&vmap, v_cache, slots * Hkv, D))
            return PKV_EINVAL;
    }
    int ps_log2 = 0;
    while ((1 << ps_log2) < page_size) ++ps_log2;
    const int grid = dev.sm_count * kCtasPerSm, G = Hq / Hkv;
    const Layout w = layout_of(grid, B, Hq, Hkv, D, max_len);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    int32_t *prefix = reinterpret_cast<int32_t *>(ws);
    float *states = reinterpret_cast<float *>(ws + w.part);
    float2 *finals = reinterpret_cast<float2 *>(ws + w.state);
    sums.scores = reinterpret_cast<float *>((reinterpret_cast<uintptr_t>(ws + w.scores) + 127) & ~uintptr_t(127));
    sums.row_len = w.row_len;
    if (pkv_host::launch_dependent(decode_weights_kernel<D>, dim3(grid), dim3(kThreads), Smem<D>::bytes(B), stream,
                                   kmap, vmap, reinterpret_cast<const __nv_bfloat16 *>(q), page_table, pt_stride,
                                   seq_lens, B, Hkv, G, ps_log2, box_rows, num_pages, scale * kLog2e,
                                   static_cast<int64_t>(max_len), states, finals, prefix, dev_status,
                                   reinterpret_cast<__nv_bfloat16 *>(out), sums) != cudaSuccess)
        return PKV_ECUDA;
    auto join = G == 1   ? decode_weights_join_kernel<D, 1>
                : G == 2 ? decode_weights_join_kernel<D, 2>
                : G == 4 ? decode_weights_join_kernel<D, 4>
                         : decode_weights_join_kernel<D, 8>;
    if (pkv_host::launch_dependent(join, dim3(grid + dev.sm_count * kJoinPerSm), dim3(kJoinThreads),
                                   static_cast<size_t>(B + 1) * sizeof(int32_t), stream,
                                   static_cast<const float *>(states), static_cast<const float2 *>(finals),
                                   static_cast<const int32_t *>(prefix), seq_lens, B, Hkv, grid,
                                   reinterpret_cast<__nv_bfloat16 *>(out), sums) != cudaSuccess)
        return PKV_ECUDA;
    return PKV_OK;
}

static bool supported(int Hq, int Hkv, int D) {
    const int G = Hq / Hkv;
    return (D == 64 || D == 128) && (G == 1 || G == 2 || G == 4 || G == 8);
}

}  // namespace decode_weights
}  // namespace pkv

extern "C" size_t pkv_decode_weights_workspace_size(int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                                    int max_seq_len) {
    using namespace pkv::decode_weights;
    if (batch < 0 || max_seq_len < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads ||
        !supported(num_q_heads, num_kv_heads, head_dim))
        return 0;
    pkv_host::DeviceInfo dev;
    if (!pkv_host::current_device(&dev)) return 0;
    return layout_of(dev.sm_count * kCtasPerSm, batch, num_q_heads, num_kv_heads, head_dim, max_seq_len).bytes;
}

extern "C" pkv_status pkv_paged_decode_attn_weights(
    const pkv_bf16 *q, const pkv_bf16 *k_cache, const pkv_bf16 *v_cache, const int32_t *page_table,
    int64_t page_table_stride, const int32_t *seq_lens, int batch, int num_q_heads, int num_kv_heads, int head_dim,
    int page_size, int64_t num_pages, float softmax_scale, float *acc, const int32_t *acc_rows, int64_t num_acc_rows,
    int64_t acc_stride, int max_seq_len, void *workspace, size_t workspace_bytes, int32_t *dev_status, pkv_bf16 *out,
    void *stream) {
    using namespace pkv::decode_weights;
    if (batch < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_pages <= 0 || page_table_stride < 0 ||
        page_size <= 0 || num_q_heads % num_kv_heads != 0 || !(softmax_scale == softmax_scale) || max_seq_len < 0 ||
        num_acc_rows < 0 || acc_stride < max_seq_len)
        return PKV_EINVAL;
    if (batch == 0) return PKV_OK;
    if (!q || !k_cache || !v_cache || !page_table || !seq_lens || !out || !workspace || !acc ||
        (!acc_rows && num_acc_rows < batch))
        return PKV_EINVAL;
    if (!supported(num_q_heads, num_kv_heads, head_dim)) return PKV_EUNSUPPORTED;
    if ((page_size & (page_size - 1)) != 0 || page_size > 256 || batch > kMaxBatch) return PKV_EUNSUPPORTED;
    if (!pkv_host::aligned16(q) || !pkv_host::aligned16(k_cache) || !pkv_host::aligned16(v_cache) ||
        !pkv_host::aligned16(out) || !pkv_host::aligned16(workspace) || (reinterpret_cast<uintptr_t>(acc) & 3u))
        return PKV_EINVAL;
    // pool slots and rows of sums are 32-bit, and so are the prefix sums of the tiles
    if (num_pages > 0x7fffffffll / page_size || page_table_stride > 0x7fffffffll || num_acc_rows > 0x7fffffffll)
        return PKV_EUNSUPPORTED;
    const int T = head_dim == 128 ? Shape<128>::T : Shape<64>::T;
    const int64_t table_keys = page_table_stride * page_size;
    const int64_t most = (table_keys < max_seq_len ? table_keys : max_seq_len) / T + 1 + kLead;
    if (static_cast<double>(batch) * num_kv_heads * most >= 2147483647.0) return PKV_EUNSUPPORTED;
    pkv_host::DeviceInfo dev;
    if (!pkv_host::current_device(&dev)) return PKV_ECUDA;
    if (workspace_bytes < layout_of(dev.sm_count * kCtasPerSm, batch, num_q_heads, num_kv_heads, head_dim, max_seq_len).bytes)
        return PKV_EINVAL;
    const Sums sums{acc, acc_rows, num_acc_rows, acc_stride, nullptr, 0};
    return (head_dim == 128 ? launch<128> : launch<64>)(
        q, k_cache, v_cache, page_table, page_table_stride, seq_lens, batch, num_q_heads, num_kv_heads, page_size,
        num_pages, softmax_scale, sums, max_seq_len, workspace, dev_status, out, dev, static_cast<cudaStream_t>(stream));
}
