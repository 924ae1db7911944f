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
// of K and V per key and KV head) and turned into weights from there, mostly out
// of L2.  Reading K a second time would cost half of the first pass again.
//
//  * The work is cut as in decode.cu: segments (sequence, KV head) end to end,
//    equal ranges of tiles per persistent block; pieces of cut segments leave
//    partial states that a second kernel joins.
//  * Producer warps stage 32 KB tiles of K and V rows with TMA (page boxes, or
//    four rows per copy for pages under 8 tokens).  One block per SM, 5 tiles in
//    flight.
//  * Each of four consumer warps takes 16 keys of a tile at a time and multiplies
//    with mma.sync m16n8k16, heads in the rows: any number of query heads up to 8
//    costs the same, where an FMA loop costs 4 * heads flops per byte and is no
//    longer memory-bound from 4 heads on.  (tcgen05 needs 128 rows; the 8 used
//    here would leave it 94 % idle, and its operands must lie in shared-memory
//    layouts that row-by-row gathers do not write.)
//    Both products contract in an order of their own: the head elements are dealt
//    to lanes in 16-byte pieces, the output columns in runs of 8, so that every
//    shared-memory read is 16 bytes wide and no operand is transposed.
//  * The softmax weights enter the second product as two bf16 terms, the rounded
//    weight in rows 0-7 and what the rounding left in rows 8-15, which the 8 heads
//    do not use: 16 bits of weight for nothing.
#include <math.h>

#include <mutex>

#include "decode_common.cuh"

namespace pkv {
namespace decode_weights {

using decode::kLead;
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
constexpr int kStages = 5;

template <int D>
struct Shape {
    static constexpr int T = 8192 / D;               // keys of a tile: 16 KB of K, 16 KB of V
    static constexpr int KG = T / (kConsumerWarps * 16);  // 16-key groups per warp
    static constexpr int CH = D / 32;                // 16-byte pieces of a K row per lane
    static constexpr int VC = D / 64;                // 16-byte pieces of a V row per lane
    static constexpr int TILE_BYTES = T * D * 2;
};

template <int D>
struct Smem {
    static constexpr int Q_BYTES = kMaxHeads * D * 2;
    static constexpr int STAGE_BYTES = 2 * Shape<D>::TILE_BYTES + Q_BYTES;
    static constexpr int RING = kStages * STAGE_BYTES;
    static constexpr int RED_O = kConsumerWarps * kMaxHeads * D * 4;
    static constexpr int RED_ML = kConsumerWarps * kMaxHeads * 2 * 4;
    static constexpr int FINAL = kMaxHeads * 2 * 4;
    static constexpr int BARS = 2 * kStages * 8;
    static constexpr int FLAGS = (kStages * kProducerWarps + 4) * 4;
    static constexpr int FIXED = RING + RED_O + RED_ML + FINAL + BARS + FLAGS;
    // + tile offsets [batch + 1] and sequence lengths [batch], int32
    static size_t bytes(int batch) { return 1024 + FIXED + static_cast<size_t>(2 * batch + 1) * 4; }
};

// The running sums, one row per request, and the scratch rows of scores
// [b][query head][len4].
struct Sums {
    float *acc;
    const int32_t *rows;
    int64_t num_rows, stride;
    float *scores;
    int64_t len4;
};

// A segment cut across blocks, written by the block that holds its last tile:
// slot0 is the partial state of its first piece (block k0), the others are slots
// 2k of blocks k up to k1.
struct __align__(16) Cut {
    int32_t segment;  // b * Hkv + g, -1: none
    int32_t k0, k1, slot0;
    int32_t W, L;
    int32_t row;  // of the running sums, -1: none
    int32_t pad;
};

__device__ __forceinline__ void mma_bf16(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Add the weights of keys j0, j0 + step, .. (groups of four) below L to the sums:
// w[j] = sum_h 2^(score[h][j] - ml[h].x) * ml[h].y, ml = (maximum, 1 / sum).
__device__ __forceinline__ void add_weights(const float *scores, int64_t len4, const float2 *ml, int G, float *row,
                                            int L, int j0, int step) {
    const bool vec = (reinterpret_cast<uintptr_t>(row) & 15u) == 0;
    for (int j = j0; j < L; j += step) {
        float4 old = make_float4(0.f, 0.f, 0.f, 0.f);
        if (vec && j + 4 < L) {
            old = *reinterpret_cast<const float4 *>(row + j);
        } else {  // the newest key's old sum is not read
            if (j + 0 < L - 1) old.x = row[j];
            if (j + 1 < L - 1) old.y = row[j + 1];
            if (j + 2 < L - 1) old.z = row[j + 2];
            if (j + 3 < L - 1) old.w = row[j + 3];
        }
        float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int h = 0; h < G; ++h) {
            const float4 s = *reinterpret_cast<const float4 *>(scores + h * len4 + j);
            const float mx = ml[h].x, inv = ml[h].y;
            w.x = fmaf(ex2(s.x - mx), inv, w.x);
            w.y = fmaf(ex2(s.y - mx), inv, w.y);
            w.z = fmaf(ex2(s.z - mx), inv, w.z);
            w.w = fmaf(ex2(s.w - mx), inv, w.w);
        }
        old.x += w.x, old.y += w.y, old.z += w.z, old.w += w.w;
        if (vec && j + 4 <= L) {
            *reinterpret_cast<float4 *>(row + j) = old;
        } else {
            row[j] = old.x;
            if (j + 1 < L) row[j + 1] = old.y;
            if (j + 2 < L) row[j + 2] = old.z;
            if (j + 3 < L) row[j + 3] = old.w;
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    decode_weights_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                          const __nv_bfloat16 *__restrict__ q, const int32_t *__restrict__ page_table,
                          int64_t pt_stride, const int32_t *__restrict__ seq_lens, int B, int Hkv, int G, int ps_log2,
                          int box_rows, int64_t num_pages, float scale_log2, int64_t max_len,
                          float *__restrict__ ws_part, Cut *__restrict__ cuts, int32_t *dev_status,
                          __nv_bfloat16 *__restrict__ out, const Sums sums) {
    using S = Shape<D>;
    using M = Smem<D>;
    constexpr int T = S::T, KG = S::KG, CH = S::CH, VC = S::VC;
    const int Hq = Hkv * G;
    const int64_t row_cap = pt_stride << ps_log2;
    const int64_t cap = max_len < row_cap ? max_len : row_cap;
    const int part_floats = ((G * D + 2 * G + 3) / 4) * 4;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *ring = smem;
    float *red_o = reinterpret_cast<float *>(smem + M::RING);
    float *red_ml = reinterpret_cast<float *>(smem + M::RING + M::RED_O);
    float2 *final_ml = reinterpret_cast<float2 *>(smem + M::RING + M::RED_O + M::RED_ML);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + M::RING + M::RED_O + M::RED_ML + M::FINAL);
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
        cuts[blockIdx.x].segment = -1;
    }
    // red_ml doubles as the scan scratch before any piece is reduced
    decode::build_prefix<kThreads>(prefix, lens, seq_lens, B, Hkv, cap, T, reinterpret_cast<int32_t *>(red_ml));
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

    const Part part{prefix[B], static_cast<int>(gridDim.x)};
    if (part.W == 0) return;
    const int64_t my_start = part.start(blockIdx.x);
    const int64_t my_end = part.start(blockIdx.x + 1);
    if (my_start >= my_end) return;

    if (warp >= kConsumerWarps) {
        // ------------------------------------------------------------ producers
        // Page boxes are issued by warp 4; gathers of K by warps 4 and 5, of V by
        // warps 6 and 7 (a warp's TMA issue rate limits four-row copies).
        const int pw = warp - kConsumerWarps;
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
        int64_t pos = my_start;
        Piece p;
        uint32_t it = 0;
        bool ok = true;
        const int bpt = T / box_rows;     // boxes per tile
        while (ok && decode::next_piece(pos, my_end, my_start, prefix, B, Hkv, p)) {
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
    // lane (r, c): row r of the products' heads, keys or output columns, c the
    // quarter of the contraction
    const int r = lane >> 2, c = lane & 3;
    const bool odd = c & 1;
    uint32_t qf[CH][4];   // pieces c, c + 4, .. of query head r
    float o[VC][8][4];    // (piece, column): rows r and r + 8, output columns of pieces VC * (2c), VC * (2c + 1)
    float m, l;           // of head r: reference, and this lane's share of the sum
    int64_t pos = my_start;
    Piece p;
    uint32_t it = 0;
    bool ok = true;
    while (ok && decode::next_piece(pos, my_end, my_start, prefix, B, Hkv, p)) {
        if (p.t1 <= p.t0) continue;  // lead units only: nothing to do
        const int L = lens[p.b];
        const int64_t head0 = (int64_t)p.b * Hq + (int64_t)p.g * G;  // the segment's first query head
        float *srow = sums.scores + (head0 + r) * sums.len4;
        m = kNegBig;
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
            // scores of head r, keys 16 (warp KG + k) + 8 n + 2 c and the next
            float sc[KG][2][4];
#pragma unroll
            for (int k = 0; k < KG; ++k) {
                const int key0 = (warp * KG + k) * 16;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    uint4 kf[CH];
#pragma unroll
                    for (int i = 0; i < CH; ++i)
                        kf[i] = lds128(kbase + ((key0 + 8 * n + r) * D + (c + 4 * i) * 8) * 2);
                    float *a = sc[k][n];
                    a[0] = a[1] = a[2] = a[3] = 0.f;
#pragma unroll
                    for (int i = 0; i < CH; ++i) {
                        mma_bf16(a, qf[i][0], 0u, qf[i][1], 0u, kf[i].x, kf[i].y);
                        mma_bf16(a, qf[i][2], 0u, qf[i][3], 0u, kf[i].z, kf[i].w);
                    }
                }
            }
            float mt = kNegBig;
#pragma unroll
            for (int k = 0; k < KG; ++k)
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int j = tok0 + (warp * KG + k) * 16 + 8 * n + 2 * c;
                    float s0 = sc[k][n][0] * scale_log2, s1 = sc[k][n][1] * scale_log2;
                    if (!full_tile) {  // past the sequence end: score -inf, so p = 0
                        if (j >= L) s0 = -INFINITY;
                        if (j + 1 >= L) s1 = -INFINITY;
                    }
                    // (the score row has room for a pair's second key past the end)
                    if (r < G && j < L) *reinterpret_cast<float2 *>(srow + j) = make_float2(s0, s1);
                    sc[k][n][0] = s0;
                    sc[k][n][1] = s1;
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
#pragma unroll
            for (int k = 0; k < KG; ++k) {
                const int key0 = (warp * KG + k) * 16;
                // V rows of this lane's keys 2c, 2c + 1, 2c + 8, 2c + 9: pieces VC r ..;
                // with two of them odd quarters read the second first, so that the
                // lanes of a quarter warp spread over twice the banks
                uint4 vf[4][VC];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int key = key0 + 2 * c + (x & 1) + 8 * (x >> 1);
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
                if (k == KG - 1) {  // the tile is in registers
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bars[kStages + s]));
                }
                uint32_t hi[2], lo[2];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float p0 = ex2(sc[k][n][0] - m), p1 = ex2(sc[k][n][1] - m);
                    l += p0 + p1;
                    hi[n] = pack_bf16x2(p0, p1);
                    lo[n] = pack_bf16x2(p0 - bf16lo(hi[n]), p1 - bf16hi(hi[n]));
                }
#pragma unroll
                for (int v = 0; v < VC; ++v) {
                    const uint32_t *x0 = reinterpret_cast<const uint32_t *>(&vf[0][v]);
                    const uint32_t *x1 = reinterpret_cast<const uint32_t *>(&vf[1][v]);
                    const uint32_t *x2 = reinterpret_cast<const uint32_t *>(&vf[2][v]);
                    const uint32_t *x3 = reinterpret_cast<const uint32_t *>(&vf[3][v]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t sel = (e & 1) ? 0x7632u : 0x5410u;
                        mma_bf16(o[v][e], hi[0], lo[0], hi[1], lo[1], __byte_perm(x0[e / 2], x1[e / 2], sel),
                                 __byte_perm(x2[e / 2], x3[e / 2], sel));
                    }
                }
            }
        }
        if (!ok) break;

        // ---- join the warps' states of this piece
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (r < G) {
            float *ro = red_o + (warp * G + r) * D;
#pragma unroll
            for (int v = 0; v < VC; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        // the rounded weights' part alone is right where V is not finite
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
                acc = fmaf(red_o[(w * G + h) * D + (idx % D)], f, acc);
            }
            if (p.whole) {
                out[head0 * D + idx] = __float2bfloat16_rn(bad_piece ? __int_as_float(0x7fc00000) : acc / sum);
                if (idx % D == 0) final_ml[h] = make_float2(mx, 1.f / sum);
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
        const int64_t row = sums.rows ? sums.rows[p.b] : p.b;
        const bool summed = row >= 0 && row < sums.num_rows;
        if (!p.whole && p.t1 == p.nt && tid == 0) {  // the last piece of a cut segment
            const int64_t s0 = prefix[p.b] + (int64_t)p.g * (p.nt + kLead);
            const int k0 = part.block_of(s0 + kLead);  // blocks before hold lead units only
            Cut cut;
            cut.segment = p.b * Hkv + p.g;
            cut.k0 = k0;
            cut.k1 = blockIdx.x;
            cut.slot0 = 2 * k0 + (s0 > part.start(k0) ? 1 : 0);
            cut.W = static_cast<int32_t>(part.W);
            cut.L = L;
            cut.row = summed ? static_cast<int32_t>(row) : -1;
            cut.pad = 0;
            cuts[blockIdx.x] = cut;
        }
        named_bar_sync(1, kConsumers);
        if (p.whole && summed && !bad_piece)
            add_weights(sums.scores + head0 * sums.len4, sums.len4, final_ml, G,
                        sums.acc + (row * Hkv + p.g) * sums.stride, L, 4 * tid, 4 * kConsumers);
    }
}

// The segments that were cut across blocks, one per blockIdx.x: blockIdx.y == 0
// joins the pieces' outputs, the others add the weights of a share of the keys.
constexpr int kJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kJoinThreads)
    decode_weights_join_kernel(const float *__restrict__ ws_part, const Cut *__restrict__ cuts, int Hkv, int G, int grid,
                               __nv_bfloat16 *__restrict__ out, const Sums sums) {
    __shared__ float2 s_ml[kMaxHeads];  // (maximum, 1 / sum), NaN maximum: keys on a bad page
    grid_dependency_wait();  // states and scores come from the main kernel
    const Cut cut = cuts[blockIdx.x];
    if (cut.segment < 0) return;
    const int part0 = (blockIdx.y - 1) * kJoinThreads * 4;  // first key of this block (y > 0)
    if (blockIdx.y > 0 && (cut.row < 0 || part0 >= cut.L)) return;
    const int E = G * D;
    const int stride = ((E + 2 * G + 3) / 4) * 4;
    const Part part{cut.W, grid};
    // partial state of block k, -1: its range is empty (fewer units than blocks)
    auto slot_of = [&](int k) -> int {
        if (k == cut.k0) return cut.slot0;
        return part.start(k + 1) > part.start(k) ? 2 * k : -1;
    };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int h = warp; h < G; h += kJoinThreads / 32) {
        float mx = kNegBig, sum = 0.f;
        bool bad = false;
        for (int k = cut.k0 + lane; k <= cut.k1; k += 32) {
            const int s = slot_of(k);
            if (s < 0) continue;
            const float2 ml = *reinterpret_cast<const float2 *>(ws_part + (int64_t)s * stride + E + 2 * h);
            bad |= isnan(ml.x);
            const float up = fmaxf(mx, ml.x);
            sum = sum * ex2(mx - up) + ml.y * ex2(ml.x - up);
            mx = up;
        }
        float all = mx;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, o));
        sum *= ex2(mx - all);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        bad = __any_sync(0xffffffffu, bad);
        if (lane == 0) s_ml[h] = make_float2(bad ? __int_as_float(0x7fc00000) : all, 1.f / sum);
    }
    __syncthreads();
    const bool bad = isnan(s_ml[0].x);
    const int64_t head0 = (int64_t)cut.segment * G;
    if (blockIdx.y > 0) {
        if (bad) return;
        const int g = cut.segment % Hkv;
        add_weights(sums.scores + head0 * sums.len4, sums.len4, s_ml, G,
                    sums.acc + ((int64_t)cut.row * Hkv + g) * sums.stride, cut.L, part0 + 4 * threadIdx.x,
                    4 * kJoinThreads * (gridDim.y - 1));
        return;
    }
    for (int idx = threadIdx.x; idx < E; idx += kJoinThreads) {
        const float mx = s_ml[idx / D].x, inv = s_ml[idx / D].y;
        float acc = 0.f;
        for (int k = cut.k0; k <= cut.k1; ++k) {
            const int s = slot_of(k);
            if (s < 0) continue;
            const float *state = ws_part + (int64_t)s * stride;
            acc = fmaf(state[idx], ex2(state[E + 2 * (idx / D)] - mx), acc);
        }
        out[head0 * D + idx] = __float2bfloat16_rn(bad ? __int_as_float(0x7fc00000) : acc * inv);
    }
}

// ---------------------------------------------------------------- host side
// Workspace: a Cut per block, two partial states per block, the score rows.
struct Layout {
    size_t states, scores, bytes;
    int64_t len4;
};
static Layout layout_of(int grid, int batch, int Hq, int Hkv, int D, int max_len) {
    Layout w;
    const int G = Hq / Hkv;
    w.len4 = ((int64_t)max_len + 3) / 4 * 4;
    w.states = static_cast<size_t>(grid) * sizeof(Cut);
    w.scores = w.states + static_cast<size_t>(grid) * 2 * (((G * D + 2 * G + 3) / 4) * 4) * sizeof(float);
    w.bytes = w.scores + static_cast<size_t>(batch) * Hq * w.len4 * sizeof(float);
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
    const int grid = dev.sm_count, G = Hq / Hkv;
    const Layout w = layout_of(grid, B, Hq, Hkv, D, max_len);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    Cut *cuts = reinterpret_cast<Cut *>(ws);
    float *states = reinterpret_cast<float *>(ws + w.states);
    sums.scores = reinterpret_cast<float *>(ws + w.scores);
    sums.len4 = w.len4;
    if (pkv_host::launch_dependent(decode_weights_kernel<D>, dim3(grid), dim3(kThreads), Smem<D>::bytes(B), stream,
                                   kmap, vmap, reinterpret_cast<const __nv_bfloat16 *>(q), page_table, pt_stride,
                                   seq_lens, B, Hkv, G, ps_log2, box_rows, num_pages, scale * kLog2e,
                                   static_cast<int64_t>(max_len), states, cuts, dev_status,
                                   reinterpret_cast<__nv_bfloat16 *>(out), sums) != cudaSuccess)
        return PKV_ECUDA;
    // a block per 1024 keys of a cut segment, up to 16, which then take several
    int split = (max_len + 4 * kJoinThreads - 1) / (4 * kJoinThreads);
    if (split > 16) split = 16;
    if (pkv_host::launch_dependent(decode_weights_join_kernel<D>, dim3(grid, 1 + split), dim3(kJoinThreads), 0, stream,
                                   static_cast<const float *>(states), static_cast<const Cut *>(cuts), Hkv, G, grid,
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
    return layout_of(dev.sm_count, batch, num_q_heads, num_kv_heads, head_dim, max_seq_len).bytes;
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
    if (workspace_bytes < layout_of(dev.sm_count, batch, num_q_heads, num_kv_heads, head_dim, max_seq_len).bytes)
        return PKV_EINVAL;
    const Sums sums{acc, acc_rows, num_acc_rows, acc_stride, nullptr, 0};
    return (head_dim == 128 ? launch<128> : launch<64>)(
        q, k_cache, v_cache, page_table, page_table_stride, seq_lens, batch, num_q_heads, num_kv_heads, page_size,
        num_pages, softmax_scale, sums, max_seq_len, workspace, dev_status, out, dev, static_cast<cudaStream_t>(stream));
}
