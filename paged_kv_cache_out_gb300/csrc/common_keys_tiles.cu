// common_keys_tiles.cu -- blocks of more than 16 (or 8) query rows over paged keys
// (see common_keys.cuh) on the tcgen05 tensor cores: the shared keys of a
// decode step's groups, the prompts of a cross attention.
//
// One persistent block of 512 threads per SM.  A block of up to 256 rows runs
// in one of two forms:
//   pair    two query tiles of 128 rows, each with a half of the softmax warps
//           and of tensor memory, share every K/V tile of 128 keys: the tensor
//           core works on one half's products while the other half's softmax runs
//   single  up to 128 rows: the two halves take the key tiles of the one query
//           tile in turn and join their states at the end
// Roles:
//   warp 8      takes the pieces of the block's range and loads their queries
//   warps 10-12, 13-15  copy the K and the V tiles (TMA, 128-byte swizzle), a third of
//               each tile each: a warp starts a copy every 80 cycles whatever its size, so
//               that rows gathered four at a time (pages under 8 tokens) keep one warp busy
//               for 5000 cycles a tile
//   warp 9      allocates all 512 TMEM columns (per half 128 of fp32 scores, in
//               whose place the bf16 weights come, and 128 of fp32 outputs) and
//               issues every MMA, in the order in which the tensor core then
//               runs them: O += P(j) V(j), S(j+1) = Q K(j+1)^T of one half, then
//               of the other
//   warps 0-3, 4-7  the halves' softmax: thread i owns row i; running maximum
//               and sum in the log2 domain, the output row rescaled in place
//               when the maximum grew by more than 2^8 (exact: every term shares
//               the reference)
// A softmax weight enters the product with V as one bf16 term (with two, which
// add half of a product's time, long cross attention took 380 us instead of
// 260); sums of weights, outputs and states are fp32.
//
// Bound by the chain of a tile: the scores of a half (0.27 us of the tensor
// core), its softmax (0.7), two hand-offs, its product with V (0.27); the other
// half's products fill in, so a pair's tile takes 1.6 us and the tensor core is
// 64 % busy (ncu, four requests of 1024-2048 tokens over 4096-8192 states: 243-247
// us, 1280-1305 TFLOP/s, 0.67-0.69 of the measured peak).  At page size 1 (61
// requests of 1-300 tokens, 32/4 heads) 114-116 us, with 49 % of the tensor core.
#include <mutex>

#include "common_keys.cuh"

namespace pkv {
namespace ck {

namespace {

constexpr int kThreads = 512;
constexpr int kProducerWarp = 8, kMmaWarp = 9, kLoaderWarp = 10, kLoaders = 3;
constexpr int kItemSlots = 4;
constexpr int kItemConsumers = 1 + 8 + 2 * kLoaders;  // MMA, softmax and loader warps
constexpr uint32_t kTmemCols = 512;
constexpr int kRegsLaunch = 128;
constexpr int kRegsSoftmax = 184, kRegsOther = 72;
static_assert(8 * 32 * kRegsSoftmax + 8 * 32 * kRegsOther <= kThreads * kRegsLaunch,
              "register split exceeds the block's registers");

template <int D>
struct Layout {
    static constexpr int NBLK = D / 64;           // 64-column blocks of a row
    static constexpr int BLK = 128 * 128;         // bytes of such a block of 128 rows
    static constexpr int TILE = NBLK * BLK;       // a query, key or value tile
    static constexpr int KS = D == 128 ? 2 : 6, VS = D == 128 ? 3 : 6;  // ring stages
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + 2 * TILE;
    static constexpr int OFF_V = OFF_K + KS * TILE;
    static constexpr int OFF_EX = OFF_V + VS * TILE;          // float2 [2][BM]: the halves' (max, sum)
    static constexpr int OFF_ITEMS = OFF_EX + 2 * BM * 8;
    static constexpr int OFF_BAR = OFF_ITEMS + kItemSlots * static_cast<int>(sizeof(Item));
    static constexpr int NBARS = 2 + 2 * KS + 2 * VS + 10 + 2 * kItemSlots + 1;
    static constexpr int OFF_MISC = OFF_BAR + NBARS * 8;      // abort flag, bad pages of the items, TMEM address
    static constexpr int TOTAL = OFF_MISC + 32;
    static_assert(TOTAL <= 232448, "shared memory of a block");
};

// LONG: rows of the page table may hold more than kShortKeys keys.
template <int D, bool LONG>
__global__ void __launch_bounds__(kThreads, 1)
    tiles_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Args a) {
    using Lo = Layout<D>;
    constexpr int KS = Lo::KS, VS = Lo::VS, NBLK = Lo::NBLK;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = 1 << a.g_log2, Hkv = a.Hkv, Hq = Hkv << a.g_log2;
    const int TOK = BM >> a.g_log2;  // tokens of a query tile
    constexpr int BN = 128;
    // LONG: a half's outputs move to fp32 totals after every so many of its key tiles
    constexpr int kWindow = LONG ? kShortKeys / BN : 1 << 30;
    static_assert((kWindow & (kWindow - 1)) == 0, "a power of two");

    extern __shared__ __align__(1024) uint8_t smem[];
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + Lo::OFF_MISC);
    volatile int *bad_flag = abort_flag + 1;  // [kItemSlots]: a page id of that item was invalid
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Lo::OFF_MISC + 24);
    float2 *ex = reinterpret_cast<float2 *>(smem + Lo::OFF_EX);
    Item *items = reinterpret_cast<Item *>(smem + Lo::OFF_ITEMS);

    const uint32_t bar0 = smem_u32(smem + Lo::OFF_BAR);
    auto BAR = [&](int i) -> uint32_t { return bar0 + 8u * i; };
    constexpr int B_QFULL = 0, B_QEMPTY = 1, B_KFULL = 2, B_KEMPTY = B_KFULL + KS, B_VFULL = B_KEMPTY + KS,
                  B_VEMPTY = B_VFULL + VS, B_SFULL = B_VEMPTY + VS, B_PFULL = B_SFULL + 2, B_ODONE = B_PFULL + 2,
                  B_OFREE = B_ODONE + 2, B_HW = B_OFREE + 2, B_HR = B_HW + 1, B_IFULL = B_HR + 1, B_IEMPTY = B_IFULL + kItemSlots,
                  B_END = B_IEMPTY + kItemSlots;
    static_assert(B_END + 1 == Lo::NBARS, "barriers");

    if (smem_u32(smem) & 1023u) {  // the 128-byte swizzle needs 1024-byte aligned tiles
        if (tid == 0 && a.dev_status) atomicOr(a.dev_status, PKV_DEV_TIMEOUT);
        return;  // uniform for the whole block, before any barrier (the join kernel checks what it reads)
    }
    if (tid == 0) {
        mbar_init(BAR(B_QFULL), 1);
        mbar_init(BAR(B_QEMPTY), 1);
        for (int s = 0; s < KS; ++s) {
            mbar_init(BAR(B_KFULL + s), kLoaders);
            mbar_init(BAR(B_KEMPTY + s), 1);
        }
        for (int s = 0; s < VS; ++s) {
            mbar_init(BAR(B_VFULL + s), kLoaders);
            mbar_init(BAR(B_VEMPTY + s), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(BAR(B_SFULL + t), 1);
            mbar_init(BAR(B_PFULL + t), 4);
            mbar_init(BAR(B_ODONE + t), 1);
            mbar_init(BAR(B_OFREE + t), 8);
        }
        mbar_init(BAR(B_END), 1);
        mbar_init(BAR(B_HW), 8);  // single blocks: the halves' (max, sum) are written, are read
        mbar_init(BAR(B_HR), 8);
        for (int s = 0; s < kItemSlots; ++s) {
            mbar_init(BAR(B_IFULL + s), 1);
            mbar_init(BAR(B_IEMPTY + s), kItemConsumers);
        }
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&qmap);
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
    }
    grid_dependency_wait();  // the plan; queries and pool rows may come from the kernels before
    allow_dependents();      // the few-rows kernel may start where this one leaves room
    if (static_cast<int>(blockIdx.x) >= a.counts[kTiles]) return;  // uniform: makes room at once (no range is left for it)
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // TMEM columns: S (then the weights over it) of half t at 128 t, O of half t at 256 + 128 t
    auto tm_s = [&](int t) -> uint32_t { return tmem + t * BN; };
    auto tm_o = [&](int t) -> uint32_t { return tmem + 2 * BN + t * 128; };

    const uint32_t sQ = smem_u32(smem + Lo::OFF_Q);
    const uint32_t sK = smem_u32(smem + Lo::OFF_K);
    const uint32_t sV = smem_u32(smem + Lo::OFF_V);

    if (warp >= kProducerWarp) {
    regs_decrease<kRegsOther>();
    // Where the block winds down after a wait that gave up, its copies and products in flight end first.
    auto drain = [&](int bar, uint32_t parity) {
        for (int i = 0; i < 50 && !try_wait(BAR(bar), parity); ++i) {
        }
    };
    const uint64_t pol_normal = l2_normal_policy(), pol_once = l2_evict_first_policy();
    if (warp == kProducerWarp) {
        // ================================================================ producer
        // takes the pieces and loads their queries
        Walk<D, kTiles> walk(a);
        uint32_t loads = 0;
#pragma unroll 1
        for (uint32_t ii = 0;; ++ii) {
            const int slot = ii % kItemSlots;
            Item it;
            if (!walk.next(a, it, [] { return true; })) it.nt = -1;  // (there is no other range to wait for)
            if (ii >= kItemSlots &&
                !wait_warp(BAR(B_IEMPTY + slot), ((ii / kItemSlots) & 1) ^ 1, abort_flag, a.dev_status))
                break;
            if (lane == 0) {
                bad_flag[slot] = 0;
                items[slot] = it;
                mbar_arrive(BAR(B_IFULL + slot));
            }
            __syncwarp();
            if (it.nt < 0) break;
            // the products with the query tiles before are done
            if (ii > 0 && !wait_warp(BAR(B_QEMPTY), (ii - 1) & 1, abort_flag, a.dev_status)) break;
            if (lane == 0) {
                const int tiles = it.form == kPair ? 2 : 1;
                mbar_arrive_expect_tx(BAR(B_QFULL), static_cast<uint32_t>(tiles * Lo::TILE));
                for (int t = 0; t < tiles; ++t)
#pragma unroll
                    for (int blk = 0; blk < NBLK; ++blk)
                        tma_load_3d(sQ + t * Lo::TILE + blk * Lo::BLK, &qmap, BAR(B_QFULL), blk * 64, it.g * G,
                                    it.tok0 + t * TOK, pol_once);
            }
            __syncwarp();
            ++loads;
        }
        if (*abort_flag && loads > 0) drain(B_QFULL, (loads - 1) & 1);
    } else if (warp != kMmaWarp) {
        // ================================================================ K and V loaders
        // three warps for each: a third of every tile's copies each
        const bool first = warp < kLoaderWarp + kLoaders;
        const uint32_t ring = first ? sK : sV;
        const int full = first ? B_KFULL : B_VFULL, empty = first ? B_KEMPTY : B_VEMPTY, stages = first ? KS : VS;
        const Pages pages(a, first ? &kmap : &vmap, kTiles, BN);
        const int copies = (pages.small ? BN / 4 : pages.bpt) * NBLK;
        const int c0 = (warp - kLoaderWarp) % kLoaders * copies / kLoaders,
                  c1 = ((warp - kLoaderWarp) % kLoaders + 1) * copies / kLoaders;
        int st = 0;
        uint32_t ph = 0;
        bool ok = true;
#pragma unroll 1
        for (uint32_t ii = 0; ok; ++ii) {
            const int slot = ii % kItemSlots;
            if (!wait_warp(BAR(B_IFULL + slot), (ii / kItemSlots) & 1, abort_flag, a.dev_status)) break;
            const Item &it = items[slot];
            const int nt = it.nt;
            if (nt < 0) break;
            const uint64_t policy = it.again ? pol_normal : pol_once;
            Copier<D, BN> copy;
            copy.begin(a, pages, it);
#pragma unroll 1
            for (int j = 0; ok && j < nt; ++j) {
                ok = copy.tile(pages, j, ring + st * Lo::TILE, BAR(full + st), policy, c0, c1, bad_flag + slot,
                               [&]() { return wait_warp(BAR(empty + st), ph ^ 1, abort_flag, a.dev_status); });
                if (++st == stages) st = 0, ph ^= 1;
            }
            if (ok && lane == 0) mbar_arrive(BAR(B_IEMPTY + slot));
        }
        if (*abort_flag)
            for (int i = 0; i < stages; ++i) drain(full + i, ph ^ (i < st ? 0u : 1u));
    } else {
        // ================================================================ MMA issuer
        // One elected lane issues every MMA, in the order the tensor core runs them.
        const uint32_t idesc_s = instr_desc(BM, BN, false) | (a.negate << 13);  // bit 13: A negated
        constexpr uint32_t idesc_o = instr_desc(BM, D, true);
        auto issue_s = [&](int t, int qt, uint32_t pos) {  // S(t) = Q(qt) K^T; K tile at ring position pos
            const uint32_t kb = sK + (pos % KS) * Lo::TILE, qb = sQ + qt * Lo::TILE;
            const uint32_t leader = elect_one();
            uint64_t qd = smem_desc(qb, 16, 1024), kd = smem_desc(kb, 16, 1024);
#pragma unroll 1
            for (int blk = 0; blk < NBLK; ++blk, qd += Lo::BLK >> 4, kd += Lo::BLK >> 4)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)  // 16 columns, 32 bytes, each
                    umma_bf16_ss_if(tm_s(t), qd + 2 * kk, kd + 2 * kk, idesc_s, blk + kk > 0 ? 1u : 0u, leader);
            umma_commit_if(BAR(B_SFULL + t), leader);
        };
        auto issue_pv = [&](int t, uint32_t pos, bool acc) {  // O(t) += P(t) V; V tile at ring position pos
            const uint32_t vb = sV + (pos % VS) * Lo::TILE;
            const uint32_t leader = elect_one();
            const uint64_t vd = smem_desc(vb, Lo::BLK, 1024);
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {  // 64 keys each
                const uint32_t pt = tm_s(t) + i * 32;
                const uint64_t v = vd + i * (4 * 16 * 128 >> 4);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    umma_bf16_ts_if(tm_o(t), pt + kk * 8, v + kk * (16 * 128 >> 4), idesc_o,
                                    (acc || i + kk > 0) ? 1u : 0u, leader);
            }
        };
        auto commit = [&](int bar) { umma_commit_if(BAR(bar), elect_one()); };

        uint32_t kt = 0, vt = 0;        // ring positions of the current item's K(0) and V(0)
        uint32_t pc[2] = {0u, 0u};      // weight tiles consumed per half
        uint32_t nq = 0;                // items of these forms so far
        auto wait = [&](int bar, uint32_t parity) -> bool {
            return wait_warp(BAR(bar), parity & 1, abort_flag, a.dev_status);
        };
        bool ok = true;
        for (uint32_t ii = 0; ok; ++ii) {
            const int slot = ii % kItemSlots;
            if (!wait(B_IFULL + slot, ii / kItemSlots)) break;
            const Item &itm = items[slot];
            const int nt = itm.nt, kend = itm.kend, key0 = itm.key0;
            const int form = itm.form;
            if (nt < 0) break;
            // V rows past the last key hold stale data (maybe NaN): zeros, so that weight 0 adds 0
            auto clear_dead = [&](int j) {
                const int first_dead = kend - (key0 + j * BN);
                if (first_dead >= BN) return;
                const uint32_t off = Lo::OFF_V + ((vt + j) % VS) * Lo::TILE;
                for (int idx = lane; idx < (BN - first_dead) * (D / 8); idx += 32) {
                    const int key = first_dead + idx / (D / 8), ch = idx % (D / 8);
                    *reinterpret_cast<uint4 *>(smem + off + swz_offset(key, ch, BN)) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                __syncwarp();
            };
            auto wait_k = [&](int j) { return wait(B_KFULL + (kt + j) % KS, (kt + j) / KS); };
            auto wait_v = [&](int j) { return wait(B_VFULL + (vt + j) % VS, (vt + j) / VS); };
            // the weights of half t are there and, before its first product of the
            // item, the output of the item before has been read out
            auto wait_p = [&](int t, bool first) -> bool {
                if (!wait(B_PFULL + t, pc[t])) return false;
                ++pc[t];
                return !first || nq == 0 || wait(B_OFREE + t, nq - 1);
            };
            ok = wait(B_QFULL, nq) && wait_k(0);
            if (!ok) break;
            tc_fence_after();
            if (form == kPair) {
                issue_s(0, 0, kt);
                issue_s(1, 1, kt);
                if (nt == 1) commit(B_QEMPTY);  // every product with Q is issued
                commit(B_KEMPTY + kt % KS);
                for (int j = 0; ok && j < nt; ++j) {
                    ok = wait_v(j);
                    if (!ok) break;
                    clear_dead(j);
                    bool k_ready = false;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        ok = ok && wait_p(t, j == 0);
                        if (!ok) break;
                        tc_fence_after();
                        issue_pv(t, vt + j, (j & (kWindow - 1)) > 0);
                        if (j == nt - 1) {
                            commit(B_ODONE + t);
                        } else {
                            if (!k_ready) {
                                ok = wait_k(j + 1);
                                if (!ok) break;
                                k_ready = true;
                                tc_fence_after();
                            }
                            issue_s(t, t, kt + j + 1);
                        }
                    }
                    if (!ok) break;
                    commit(B_VEMPTY + (vt + j) % VS);
                    if (j + 1 < nt) {
                        if (j + 2 == nt) commit(B_QEMPTY);
                        commit(B_KEMPTY + (kt + j + 1) % KS);
                    }
                }
            } else {
                issue_s(0, 0, kt);
                if (nt == 1) commit(B_QEMPTY);
                commit(B_KEMPTY + kt % KS);
                if (nt > 1) {
                    ok = wait_k(1);
                    if (!ok) break;
                    tc_fence_after();
                    issue_s(1, 0, kt + 1);
                    if (nt == 2) commit(B_QEMPTY);
                    commit(B_KEMPTY + (kt + 1) % KS);
                }
                for (int j = 0; ok && j < nt; ++j) {
                    const int t = j & 1;
                    ok = wait_v(j);
                    if (!ok) break;
                    clear_dead(j);
                    ok = wait_p(t, j < 2);
                    if (!ok) break;
                    tc_fence_after();
                    issue_pv(t, vt + j, ((j >> 1) & (kWindow - 1)) > 0);
                    commit(B_VEMPTY + (vt + j) % VS);
                    if (j + 2 < nt) {
                        ok = wait_k(j + 2);
                        if (!ok) break;
                        tc_fence_after();
                        issue_s(t, 0, kt + j + 2);
                        if (j + 3 == nt) commit(B_QEMPTY);
                        commit(B_KEMPTY + (kt + j + 2) % KS);
                    }
                }
                if (!ok) break;
                commit(B_ODONE + 0);
                // Half 1 has nothing to do in a single tile, so nothing of this item has told that it is
                // past the phase of the item before: a second phase over a warp that still waits for
                // the first would leave it waiting.
                if (nt == 1 && nq > 0) ok = wait(B_OFREE + 1, nq - 1);
                if (!ok) break;
                commit(B_ODONE + 1);
            }
            ++nq;
            kt += nt;
            vt += nt;
            if (ok) {
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(B_IEMPTY + slot));
            }
        }
        if (*abort_flag) {
            commit(B_END);
            drain(B_END, 0);
        }
    }
    } else {
        // ================================================================ softmax
        regs_increase<kRegsSoftmax>();
        const int t = warp >> 2;                   // half: query tile of a pair, or every other key tile
        const int row = tid & 127;                 // TMEM lane == tile row
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        uint32_t sc = 0;                           // S tiles consumed by this half (all items)
        uint32_t nh = 0, nq = 0;                   // single blocks, items so far
        const bool sectors = whole_sectors(a.out);
        bool ok = true;
        for (uint32_t ii = 0; ok; ++ii) {
            const int slot = ii % kItemSlots;
            if (!wait_warp(BAR(B_IFULL + slot), (ii / kItemSlots) & 1, abort_flag, a.dev_status)) break;
            const Item &itm = items[slot];
            const int nt = itm.nt;
            if (nt < 0) break;
            const bool pair = itm.form == kPair;
            const int tok = (row >> a.g_log2) + (pair ? t * TOK : 0);
            const bool row_valid = tok < itm.n;
            const bool warp_live = __any_sync(0xffffffffu, row_valid);
            const int my_nt = pair ? nt : (nt + 1 - t) >> 1;
            int left = itm.kend - itm.key0 - (pair ? 0 : t * BN);  // keys from this half's tile on
            const int stride = pair ? BN : 2 * BN;
            float m_ref = kNoKey, l_sum = 0.f;
            float m_tot = kNoKey;  // the totals' reference
            // this thread's row of them: in the slot that the piece's state will take, or, for a whole
            // segment, in that of the range's last piece, which comes later
            auto totals = [&]() -> float * {
                const int at = itm.dest == kSlot ? itm.slot : 2 * static_cast<int>(blockIdx.x) + 1;
                return a.slot_o[kTiles] + state_at(kTiles, D, at, t * BM + row, 0);
            };
            for (int j = 0; j < my_nt; ++j, left -= stride) {
                // S(j) complete implies that the product before it is: O is stable, the weights are free
                ok = wait_warp(BAR(B_SFULL + t), (sc + j) & 1, abort_flag, a.dev_status);
                if (!ok) break;
                if (warp_live) {
                    tc_fence_after();
                    if (LONG && j > 0 && (j & (kWindow - 1)) == 0) {  // totals = totals 2^(m_tot - m_ref) + O
                        float *tot = totals();
                        const float f = ex2(m_tot - m_ref);
#pragma unroll 1
                        for (int cc = 0; cc < D / 32; ++cc) {
                            uint32_t ov[32];
                            tmem_ld_32cols(tm_o(t) + lane_off + cc * 32, ov);
                            tmem_wait_ld();
                            const float *o = reinterpret_cast<const float *>(ov);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                float4 *p = reinterpret_cast<float4 *>(tot + (cc * 8 + i) * (4 * kBlockRows));
                                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                                if (j > kWindow) x = *p;
                                *p = make_float4(fmaf(x.x, f, o[4 * i]), fmaf(x.y, f, o[4 * i + 1]),
                                                 fmaf(x.z, f, o[4 * i + 2]), fmaf(x.w, f, o[4 * i + 3]));
                            }
                        }
                        m_tot = m_ref;
                    }
                    uint32_t sv[BN];
#pragma unroll
                    for (int cc = 0; cc < BN / 32; ++cc) tmem_ld_32cols(tm_s(t) + lane_off + cc * 32, sv + cc * 32);
                    tmem_wait_ld();
                    if (left < BN) {  // the last tile of the entry: keys past the end
#pragma unroll
                        for (int i = 0; i < BN; ++i)
                            if (i >= left) sv[i] = __float_as_uint(-INFINITY);
                    }
                    float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < BN; i += 2)
                        mx4[(i >> 1) & 3] =
                            fmax3(mx4[(i >> 1) & 3], __uint_as_float(sv[i]), __uint_as_float(sv[i + 1]));
                    const float mt_max = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * a.scale_log2;
                    const bool need = (j > 0) && row_valid && (mt_max > m_ref + kRescaleLog2);
                    const bool warp_need = __any_sync(0xffffffffu, need);
                    float alpha = 1.f;
                    if (j == 0) {
                        m_ref = fmaxf(mt_max, kNoKey);
                    } else if (warp_need) {
                        const float mn = fmaxf(m_ref, mt_max);
                        alpha = ex2(m_ref - mn);
                        m_ref = mn;
                    }
                    const float neg_m = -m_ref;
                    float rs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int cc = 0; cc < BN / 32; ++cc) {
                        uint32_t pk[16];
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            const int i = cc * 32 + 2 * q;
                            float x0, x1;
                            fma2(x0, x1, __uint_as_float(sv[i]), __uint_as_float(sv[i + 1]), a.scale_log2,
                                 a.scale_log2, neg_m, neg_m);
                            const float p0 = ex2(x0), p1 = ex2(x1);
                            add2(rs[2 * (q & 1)], rs[2 * (q & 1) + 1], p0, p1);
                            pk[q] = pack_bf16x2(p0, p1);
                        }
                        tmem_st_16cols(tm_s(t) + lane_off + cc * 16, pk);
                    }
                    l_sum = l_sum * alpha + ((rs[0] + rs[1]) + (rs[2] + rs[3]));
                    if (warp_need) {  // the output row to the new reference
#pragma unroll 1
                        for (int cc = 0; cc < D / 32; ++cc) {
                            uint32_t ov[32];
                            tmem_ld_32cols(tm_o(t) + lane_off + cc * 32, ov);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                            tmem_st_32cols(tm_o(t) + lane_off + cc * 32, ov);
                        }
                    }
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(B_PFULL + t));
            }
            if (!ok) break;
            sc += my_nt;
            ok = wait_warp(BAR(B_ODONE + t), nq & 1, abort_flag, a.dev_status);
            ++nq;
            if (!ok) break;
            tc_fence_after();
            if (LONG && my_nt > kWindow && warp_live) {  // O = O + totals 2^(m_tot - m_ref)
                const float *tot = totals();
                const float f = ex2(m_tot - m_ref);
#pragma unroll 1
                for (int cc = 0; cc < D / 32; ++cc) {
                    uint32_t ov[32];
                    tmem_ld_32cols(tm_o(t) + lane_off + cc * 32, ov);
                    tmem_wait_ld();
                    float *o = reinterpret_cast<float *>(ov);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 x = *reinterpret_cast<const float4 *>(tot + (cc * 8 + i) * (4 * kBlockRows));
                        o[4 * i] = fmaf(x.x, f, o[4 * i]);
                        o[4 * i + 1] = fmaf(x.y, f, o[4 * i + 1]);
                        o[4 * i + 2] = fmaf(x.z, f, o[4 * i + 2]);
                        o[4 * i + 3] = fmaf(x.w, f, o[4 * i + 3]);
                    }
                    tmem_st_32cols(tm_o(t) + lane_off + cc * 32, ov);
                }
                tmem_wait_st();
                tc_fence_before();  // (the other half reads them, in a single block)
            }
            const bool poison = bad_flag[slot] != 0;
            const int dest = itm.dest;
            // (own keys of a decode step go to the other kernel)
            const int64_t out_row = static_cast<int64_t>(itm.tok0 + tok) * Hq + itm.g * G + (row & (G - 1));
            const int block_at = (pair ? t * BM : 0) + row;
            // (states lie four columns at a time, so that a warp's 32 rows are 512 bytes: a pair's 256 rows
            // of 128 columns take 0.9 us, and 4.5 us where each row lies by itself)
            float *o_dst = dest == kSlot ? a.slot_o[kTiles] + state_at(kTiles, D, itm.slot, block_at, 0)
                           : dest == kOut
                               ? nullptr
                               : a.row_o[0] + block_state_at(kTiles, D, Hkv, a.g_log2, itm.tok0, itm.n, itm.g, block_at, 0);
            const int o_step = 4 * (dest == kSlot ? kBlockRows : itm.n << a.g_log2);  // from four columns to the next
            float2 *ml_dst = dest == kSlot ? a.slot_ml[kTiles] + static_cast<int64_t>(itm.slot) * kBlockRows + block_at
                             : dest == kOut
                                 ? nullptr
                                 : a.row_ml[0] + block_row(Hkv, a.g_log2, itm.tok0, itm.n, itm.g, block_at);
            // 32 columns of a row, normalised to bf16 or as they are
            auto put = [&](int cc, const float *o, float inv) {
                if (dest == kOut) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        pk[i] = poison ? 0x7fc07fc0u : pack_bf16x2(o[2 * i] * inv, o[2 * i + 1] * inv);
                    st_global_32B(a.out + out_row * D + cc * 32, pk, sectors);
                    st_global_32B(a.out + out_row * D + cc * 32 + 16, pk + 8, sectors);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<float4 *>(o_dst + (cc * 8 + i) * o_step) =
                            make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                }
            };
            if (pair) {
                if (warp_live) {
                    const float inv = 1.f / l_sum;
#pragma unroll 1
                    for (int cc = 0; cc < D / 32; ++cc) {
                        uint32_t ov[32];
                        tmem_ld_32cols(tm_o(t) + lane_off + cc * 32, ov);
                        tmem_wait_ld();
                        if (row_valid) put(cc, reinterpret_cast<const float *>(ov), inv);
                    }
                    if (row_valid && dest != kOut) *ml_dst = make_float2(poison ? __int_as_float(0x7fc00000) : m_ref, l_sum);
                }
            } else {
                // the halves' states of the same rows meet; each half writes half of the columns
                const bool two = nt > 1;
                ok = nh < 1 || wait_warp(BAR(B_HR), (nh - 1) & 1, abort_flag, a.dev_status);
                if (!ok) break;
                ex[t * BM + row] = make_float2(m_ref, l_sum);
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(B_HW));
                ok = wait_warp(BAR(B_HW), nh & 1, abort_flag, a.dev_status);
                ++nh;
                if (!ok) break;
                if (LONG) tc_fence_after();
                if (warp_live) {
                    const float2 s0 = ex[row], s1 = ex[BM + row];
                    const float mm = two ? fmaxf(s0.x, s1.x) : s0.x;
                    const float w0 = ex2(s0.x - mm), w1 = two ? ex2(s1.x - mm) : 0.f;
                    const float l = two ? s0.y * w0 + s1.y * w1 : s0.y;
                    const float inv = 1.f / l;
#pragma unroll 1
                    for (int c = 0; c < D / 64; ++c) {
                        const int cc = t * (D / 64) + c;
                        uint32_t ov[32];
                        tmem_ld_32cols(tm_o(0) + lane_off + cc * 32, ov);
                        tmem_wait_ld();
                        float o[32];
                        if (two) {
                            uint32_t ow[32];
                            tmem_ld_32cols(tm_o(1) + lane_off + cc * 32, ow);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[i] = fmaf(__uint_as_float(ow[i]), w1, __uint_as_float(ov[i]) * w0);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(ov[i]);
                        }
                        if (row_valid) put(cc, o, inv);
                    }
                    if (row_valid && dest != kOut && t == 0)
                        *ml_dst = make_float2(poison ? __int_as_float(0x7fc00000) : mm, l);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(B_HR));
            }
            if (poison && tid == 0 && a.dev_status) atomicOr(a.dev_status, PKV_DEV_BAD_PAGE);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                // both halves of a single block read both outputs: each is free after
                // eight warps; a pair's warps count twice for their own
                mbar_arrive(BAR(B_OFREE + t));
                mbar_arrive(BAR(B_OFREE + (pair ? t : 1 - t)));
                mbar_arrive(BAR(B_IEMPTY + slot));
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}


}  // namespace

template <int D, bool LONG>
bool launch_tiles(const Args &a, const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap,
                  const pkv_host::DeviceInfo &dev, cudaStream_t stream) {
    static std::mutex mu;
    static bool ready[64] = {};
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!ready[dev.device]) {
            if (Layout<D>::TOTAL > dev.max_smem_optin ||
                cudaFuncSetAttribute(tiles_kernel<D, LONG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     Layout<D>::TOTAL) != cudaSuccess)
                return false;
            ready[dev.device] = true;
        }
    }
    return pkv_host::launch_dependent(tiles_kernel<D, LONG>, dim3(a.blocks[kTiles]), dim3(kThreads), Layout<D>::TOTAL,
                                      stream, qmap, kmap, vmap, a) == cudaSuccess;
}

template bool launch_tiles<64, false>(const Args &, const CUtensorMap &, const CUtensorMap &, const CUtensorMap &,
                                      const pkv_host::DeviceInfo &, cudaStream_t);
template bool launch_tiles<64, true>(const Args &, const CUtensorMap &, const CUtensorMap &, const CUtensorMap &,
                                     const pkv_host::DeviceInfo &, cudaStream_t);
template bool launch_tiles<128, false>(const Args &, const CUtensorMap &, const CUtensorMap &, const CUtensorMap &,
                                       const pkv_host::DeviceInfo &, cudaStream_t);
template bool launch_tiles<128, true>(const Args &, const CUtensorMap &, const CUtensorMap &, const CUtensorMap &,
                                      const pkv_host::DeviceInfo &, cudaStream_t);

}  // namespace ck
}  // namespace pkv
