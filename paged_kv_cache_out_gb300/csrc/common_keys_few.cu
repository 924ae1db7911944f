// common_keys_few.cu -- blocks of up to 16 query rows over paged keys (see
// common_keys.cuh): a decode step's own keys, the beams or the next tokens of
// a cross attention.  Bound by reading K and V once.
//
// Two persistent blocks of 256 threads per SM, so that the fixed work of one
// block's short segments hides behind the other's copies:
//   warps 0-3  each takes 16 keys of every 64 (head size 64: 32 of every 128)
//              and keeps a softmax state of its own over them; the warps meet
//              at the end of a segment only.  Both products are mma.sync
//              m16n8k16 with the rows as N, so 8 rows cost half of what 16 do:
//                  S^T (16 keys x 8 NT) = K Q^T,   O^T (D x 8 NT) += V^T P^T,
//              K and V fragments by ldmatrix from the swizzled tiles (V
//              transposed on the way), P^T from S^T's registers by 8 x 8
//              transpositions.  (Why not tcgen05: its M is 128, and a tile's
//              chain of two hand-offs would be longer than the copies.)
//   warp 4     takes ranges and publishes their pieces
//   warps 5, 6 copy the K and the V tiles through rings of three stages; warp
//              7 takes a quarter of both where pages have fewer than 8 tokens
//              (a warp issues a TMA copy in about 80 cycles whatever its size)
// The weights enter the second product with 16 bits, as two bf16 terms, and
// all sums are fp32.
//
// Measured (page size 16 unless said): 96 chats of 500-5000 keys after four
// prompts, 910 MB in 144 us under ncu, 6.3 TB/s (0.93 of the copy bandwidth);
// whole calls: 64 next tokens over 1024-8192 states (page size 256) 109-117 us,
// 0.76-0.82; five beams of 96 requests over 100-1500 states 41-43 us, 0.54-0.57,
// where the plan, the join and the first copies are 12 us.
#include <mutex>

#include "common_keys.cuh"

namespace pkv {
namespace ck {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = 4;  // consumers
constexpr int kProducerWarp = 4;
constexpr int kItemSlots = 4;
constexpr int kStages = 3;
constexpr int kRegsConsumer = 176, kRegsOther = 80;
static_assert(128 * kRegsConsumer + 128 * kRegsOther <= kThreads * 128, "register split exceeds the block's registers");

template <int D>
struct Layout {
    static constexpr int BN = tile_keys<D>(kFew);
    static constexpr int NBLK = D / 64;
    static constexpr int BLK = BN * 128;        // bytes of 64 columns of a tile
    static constexpr int TILE = NBLK * BLK;     // 16 KB
    static constexpr int OFF_K = 0;
    static constexpr int OFF_V = OFF_K + kStages * TILE;
    static constexpr int OFF_EO = OFF_V + kStages * TILE;      // float [kWarps][8][D]: the warps' outputs
    static constexpr int OFF_EX = OFF_EO + kWarps * 8 * D * 4; // float2 [kWarps][8]: their (max, sum)
    static constexpr int OFF_ITEMS = OFF_EX + kWarps * 8 * 8;
    static constexpr int OFF_BAR = OFF_ITEMS + kItemSlots * static_cast<int>(sizeof(Item));
    // ring full and empty, exchange written and read, items full and empty
    static constexpr int NBARS = 4 * kStages + 2 + 2 * kItemSlots;
    static constexpr int OFF_MISC = OFF_BAR + NBARS * 8;       // abort flag, bad pages of the items
    static constexpr int TOTAL = OFF_MISC + 32;
    static_assert(TOTAL <= (233472 - 2 * 1024) / 2, "two blocks per SM");
};

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma_bf16(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The 8 x 8 matrix of bf16 whose row lane / 4 this lane holds two columns of, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Where value d of row r lies in the exchange: rows two apart, which the lanes of a warp write at
// the same time, on other banks.
__device__ __forceinline__ int exchange_at(int r, int d) { return d ^ (((r >> 1) & 3) << 3); }

__device__ __forceinline__ void acquire(const int *p) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
}

struct Ring {
    uint32_t k, v;            // shared memory of the first stages
    uint32_t kfull, kempty, vfull, vempty;  // barriers
    uint32_t s, ph;           // position: K and V tiles are consumed together
};

// A piece: NT x 8 rows, by the consumer warps.  LONG: rows of the page table may hold more than
// kShortKeys keys, and the products with 16 keys each are added in fp32.
template <int D, int NT, bool LONG>
__device__ __forceinline__ bool piece(const Args &a, const Item &it, Ring &ring, float *eo, float2 *ex,
                                      uint32_t written_bar, uint32_t read_bar, uint32_t &nx, volatile int *bad_flag,
                                      volatile int *abort_flag) {
    using Lo = Layout<D>;
    constexpr int NS = D / 16, KG = Lo::BN / (16 * kWarps);  // 16-key groups of a warp per tile
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = 1 << a.g_log2, Hq = a.Hkv << a.g_log2;
    const int tok0 = it.tok0, g = it.g, nt = it.nt, R = it.n << a.g_log2;
    int left = it.kend - it.key0 - 16 * KG * warp;  // keys from this warp's first of the tile on
    // Q^T fragments: row lane / 4 of each eight, columns 2 (lane % 4) .. + 1 and 8 more of every 16
    uint32_t q[NT][NS][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int r = 8 * i + lane / 4;
        const bool live = r < R;
        const __nv_bfloat16 *src =
            a.q + (static_cast<int64_t>(tok0 + (live ? r >> a.g_log2 : 0)) * Hq + g * G + (r & (G - 1))) * D +
            (lane % 4) * 2;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            q[i][s][0] = live ? __ldg(reinterpret_cast<const uint32_t *>(src + 16 * s)) : 0u;
            q[i][s][1] = live ? __ldg(reinterpret_cast<const uint32_t *>(src + 16 * s + 8)) : 0u;
        }
    }
    const float scale = a.negate ? -a.scale_log2 : a.scale_log2;
    float o[NT][NS][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        m[i][0] = m[i][1] = kNoKey;
        l[i][0] = l[i][1] = 0.f;
#pragma unroll
        for (int s = 0; s < NS; ++s) o[i][s][0] = o[i][s][1] = o[i][s][2] = o[i][s][3] = 0.f;
    }
    // ldmatrix: this lane's row and 16-byte piece.  K: (keys 0-7, piece), (8-15, piece), (0-7,
    // piece + 1), (8-15, piece + 1); V: (0-7, piece), (0-7, piece + 1), (8-15, piece), (8-15, piece + 1)
    const int kkey = 16 * KG * warp + ((lane >> 3) & 1) * 8 + (lane & 7), kpiece = lane >> 4;
    const int vkey = 16 * KG * warp + (lane >> 4) * 8 + (lane & 7), vpiece = (lane >> 3) & 1;
#pragma unroll 1
    for (int j = 0; j < nt; ++j, left -= Lo::BN) {
        if (!wait_warp(ring.kfull + 8u * ring.s, ring.ph, abort_flag, a.dev_status)) return false;
        float c[KG][NT][2][4] = {};
        if (left > 0) {
            const uint32_t base = ring.k + ring.s * Lo::TILE + kkey * 128;
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
                for (int kg = 0; kg < KG; ++kg) {
                    uint32_t k[4];
                    ldmatrix4(base + kg * 16 * 128 + (s >> 2) * Lo::BLK + ((((2 * s + kpiece) ^ kkey) & 7) << 4), k);
#pragma unroll
                    for (int i = 0; i < NT; ++i) mma_bf16(c[kg][i][s & 1], k, q[i][s][0], q[i][s][1]);
                }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(ring.kempty + 8u * ring.s);
        uint32_t bh[KG][NT][2], bl[KG][NT][2];
        if (left > 0) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                float x[KG][4];
                float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
                for (int kg = 0; kg < KG; ++kg) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)  // this lane's keys: lane / 4 and 8 more
                        x[kg][e] = 16 * kg + lane / 4 + (e < 2 ? 0 : 8) < left ? (c[kg][i][0][e] + c[kg][i][1][e]) * scale
                                                                               : -INFINITY;
                    top0 = fmaxf(top0, fmaxf(x[kg][0], x[kg][2]));
                    top1 = fmaxf(top1, fmaxf(x[kg][1], x[kg][3]));
                }
                if (__any_sync(0xffffffffu, top0 > m[i][0] + kRescaleLog2 || top1 > m[i][1] + kRescaleLog2)) {
                    float mx0 = top0, mx1 = top1;
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) {
                        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
                        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
                    }
                    mx0 = fmaxf(mx0, m[i][0]);
                    mx1 = fmaxf(mx1, m[i][1]);
                    const float f0 = ex2(m[i][0] - mx0), f1 = ex2(m[i][1] - mx1);
                    m[i][0] = mx0, m[i][1] = mx1;
                    l[i][0] *= f0, l[i][1] *= f1;
#pragma unroll
                    for (int s = 0; s < NS; ++s) {
                        o[i][s][0] *= f0, o[i][s][1] *= f1;
                        o[i][s][2] *= f0, o[i][s][3] *= f1;
                    }
                }
#pragma unroll
                for (int kg = 0; kg < KG; ++kg) {
                    const float p0 = ex2(x[kg][0] - m[i][0]), p1 = ex2(x[kg][1] - m[i][1]);
                    const float p2 = ex2(x[kg][2] - m[i][0]), p3 = ex2(x[kg][3] - m[i][1]);
                    l[i][0] += p0 + p2;
                    l[i][1] += p1 + p3;
                    uint32_t h0, h1, l0, l1;
                    split_weights(p0, p1, h0, l0);
                    split_weights(p2, p3, h1, l1);
                    bh[kg][i][0] = transpose8(h0), bh[kg][i][1] = transpose8(h1);
                    bl[kg][i][0] = transpose8(l0), bl[kg][i][1] = transpose8(l1);
                }
            }
        }
        if (!wait_warp(ring.vfull + 8u * ring.s, ring.ph, abort_flag, a.dev_status)) return false;
        if (left > 0) {
            const uint32_t base = ring.v + ring.s * Lo::TILE + vkey * 128;
#pragma unroll
            for (int kg = 0; kg < KG; ++kg) {
                // V rows past the last key hold stale data (maybe NaN): zeros
                const int mine = left - 16 * kg - 2 * (lane % 4);
                const uint32_t m0 = (mine > 0 ? 0xffffu : 0u) | (mine > 1 ? 0xffff0000u : 0u);
                const uint32_t m1 = (mine > 8 ? 0xffffu : 0u) | (mine > 9 ? 0xffff0000u : 0u);
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    uint32_t v[4];
                    ldmatrix4_trans(base + kg * 16 * 128 + (s >> 2) * Lo::BLK + ((((2 * s + vpiece) ^ vkey) & 7) << 4), v);
                    v[0] &= m0, v[1] &= m0, v[2] &= m1, v[3] &= m1;
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        if constexpr (LONG) {
                            float t[4] = {};
                            mma_bf16(t, v, bh[kg][i][0], bh[kg][i][1]);
                            mma_bf16(t, v, bl[kg][i][0], bl[kg][i][1]);
                            add2(o[i][s][0], o[i][s][1], t[0], t[1]);
                            add2(o[i][s][2], o[i][s][3], t[2], t[3]);
                        } else {
                            mma_bf16(o[i][s], v, bh[kg][i][0], bh[kg][i][1]);
                            mma_bf16(o[i][s], v, bl[kg][i][0], bl[kg][i][1]);
                        }
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(ring.vempty + 8u * ring.s);
        if (++ring.s == kStages) ring.s = 0, ring.ph ^= 1;
    }
    // ---- the warps' states meet, eight rows at a time
    const bool poison = *bad_flag != 0;
    const int dest = it.dest, slot = it.slot;
#pragma unroll
    for (int i = 0; i < NT; ++i, ++nx) {
        if (nx > 0 && !wait_warp(read_bar, (nx - 1) & 1, abort_flag, a.dev_status)) return false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], off);
            const int r = 2 * (lane % 4) + e;
            if (8 * i + r < R) {
                if (lane < 4) ex[warp * 8 + r] = make_float2(m[i][e], l[i][e]);
                float *dst = eo + (warp * 8 + r) * D;
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    dst[exchange_at(r, 16 * s + lane / 4)] = o[i][s][e];
                    dst[exchange_at(r, 16 * s + 8 + lane / 4)] = o[i][s][e + 2];
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(written_bar);
        if (!wait_warp(written_bar, nx & 1, abort_flag, a.dev_status)) return false;
        const int rows = min(R - 8 * i, 8);
#pragma unroll 1
        for (int at = threadIdx.x; at < rows * (D / 4); at += kWarps * 32) {
            const int r = at / (D / 4), col = at % (D / 4) * 4, row = 8 * i + r;
            float2 ml[kWarps];
            float4 v[kWarps];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                ml[w] = ex[w * 8 + r];
                v[w] = *reinterpret_cast<const float4 *>(eo + (w * 8 + r) * D + exchange_at(r, col));
            }
            float mx = kNoKey, sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, ml[w].x);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2(ml[w].x - mx);
                sum = fmaf(ml[w].y, f, sum);
                acc.x = fmaf(v[w].x, f, acc.x);
                acc.y = fmaf(v[w].y, f, acc.y);
                acc.z = fmaf(v[w].z, f, acc.z);
                acc.w = fmaf(v[w].w, f, acc.w);
            }
            const float nan = __int_as_float(0x7fc00000);
            const int64_t out_row = static_cast<int64_t>(tok0 + (row >> a.g_log2)) * Hq + g * G + (row & (G - 1));
            if (dest == kOut) {
                const float inv = poison ? nan : 1.f / sum;
                *reinterpret_cast<uint2 *>(a.out + out_row * D + col) =
                    make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
            } else {
                const int64_t to = dest == kSlot         ? static_cast<int64_t>(slot) * kFewRows + row
                                   : dest == kRowsShared ? block_row(a.Hkv, a.g_log2, tok0, it.n, g, row)
                                                         : out_row;
                float *o_dst = dest == kSlot ? a.slot_o[kFew] : dest == kRowsShared ? a.row_o[0] : a.row_o[1];
                float2 *ml_dst = dest == kSlot ? a.slot_ml[kFew] : dest == kRowsShared ? a.row_ml[0] : a.row_ml[1];
                *reinterpret_cast<float4 *>(o_dst + to * D + col) = acc;
                if (col == 0) ml_dst[to] = make_float2(poison ? nan : mx, sum);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(read_bar);
    }
    if (poison && threadIdx.x == 0 && a.dev_status) atomicOr(a.dev_status, PKV_DEV_BAD_PAGE);
    return true;
}

// Rows without keys, by one warp.
template <int D>
__device__ __forceinline__ void fill_rows(const Args &a, const Item &it) {
    const int G = 1 << a.g_log2, Hq = a.Hkv << a.g_log2;
    const uint32_t pair = it.flags & kBad ? 0x7fc07fc0u : 0u;
    constexpr int VPR = D / 8;  // 16-byte pieces of a row
#pragma unroll 1
    for (int i = threadIdx.x & 31; i < it.n * G * VPR; i += 32) {
        const int t = i / (G * VPR), r = i - t * (G * VPR);
        uint4 *dst = reinterpret_cast<uint4 *>(a.out + (static_cast<int64_t>(it.tok0 + t) * Hq + it.g * G) * D);
        dst[r] = make_uint4(pair, pair, pair, pair);
    }
}

template <int D, bool LONG>
__global__ void __launch_bounds__(kThreads, 2)
    few_rows_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                    const __grid_constant__ Args a) {
    using Lo = Layout<D>;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    extern __shared__ __align__(1024) uint8_t smem[];
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + Lo::OFF_MISC);
    volatile int *bad_flag = abort_flag + 1;  // [kItemSlots]
    Item *items = reinterpret_cast<Item *>(smem + Lo::OFF_ITEMS);
    const uint32_t bar0 = smem_u32(smem + Lo::OFF_BAR);
    auto BAR = [&](int i) -> uint32_t { return bar0 + 8u * i; };
    constexpr int B_KFULL = 0, B_KEMPTY = kStages, B_VFULL = 2 * kStages, B_VEMPTY = 3 * kStages, B_XW = 4 * kStages,
                  B_XR = B_XW + 1, B_IFULL = B_XR + 1, B_IEMPTY = B_IFULL + kItemSlots;
    static_assert(B_IEMPTY + kItemSlots == Lo::NBARS, "barriers");
    const bool small = a.box_log2[kFew] < 3;
    if (smem_u32(smem) & 1023u) {  // the 128-byte swizzle needs 1024-byte aligned tiles
        if (tid == 0 && a.dev_status) atomicOr(a.dev_status, PKV_DEV_TIMEOUT);
        return;  // uniform for the whole block (the join kernel checks what it reads)
    }
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(BAR(B_KFULL + s), small ? 2 : 1);
            mbar_init(BAR(B_VFULL + s), small ? 2 : 1);
            mbar_init(BAR(B_KEMPTY + s), kWarps);
            mbar_init(BAR(B_VEMPTY + s), kWarps);
        }
        mbar_init(BAR(B_XW), kWarps);
        mbar_init(BAR(B_XR), kWarps);
        for (int s = 0; s < kItemSlots; ++s) {
            mbar_init(BAR(B_IFULL + s), 1);
            mbar_init(BAR(B_IEMPTY + s), kWarps + (small ? 3 : 2));
        }
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
    }
    // With the tiles kernel running, no wait for its end: nothing of it is read here.  What is read was
    // written by the plan kernel and by kernels before it.  They are complete and their writes performed:
    // every block of the tiles kernel has waited for that before it lets this grid start.  But the wait's
    // promise is to who waits, so this relies on the order of the two starts, with an acquire (of a word
    // of the plan) that keeps the block from anything read earlier, and a fence for the copies, which read
    // by the other proxy: 0.1 us.  (Releases of words in front of it, beside that order: at the plan
    // kernel's end 0.5 us of each call, at the tiles kernel's beginning 0.6-0.9.)
    if (!a.tiles_run) {
        grid_dependency_wait();
    } else if (tid == kThreads - 1) {  // (thread 0 makes the barriers)
        acquire(a.counts + kFew);
        fence_proxy_async_global();
    }
    __syncthreads();
    if (warp < kWarps) {
        // ================================================================ consumers
        regs_increase<kRegsConsumer>();
        Ring ring{smem_u32(smem + Lo::OFF_K), smem_u32(smem + Lo::OFF_V), BAR(B_KFULL), BAR(B_KEMPTY), BAR(B_VFULL),
                  BAR(B_VEMPTY), 0u, 0u};
        float *eo = reinterpret_cast<float *>(smem + Lo::OFF_EO);
        float2 *ex = reinterpret_cast<float2 *>(smem + Lo::OFF_EX);
        uint32_t nx = 0;  // exchanges so far
#pragma unroll 1
        for (uint32_t ii = 0;; ++ii) {
            const int slot = ii % kItemSlots;
            if (!wait_warp(BAR(B_IFULL + slot), (ii / kItemSlots) & 1, abort_flag, a.dev_status)) break;
            const Item it = items[slot];
            if (it.nt < 0) break;
            const bool ok = it.n << a.g_log2 <= 8
                                ? piece<D, 1, LONG>(a, it, ring, eo, ex, BAR(B_XW), BAR(B_XR), nx, bad_flag + slot, abort_flag)
                                : piece<D, 2, LONG>(a, it, ring, eo, ex, BAR(B_XW), BAR(B_XR), nx, bad_flag + slot, abort_flag);
            if (!ok) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(B_IEMPTY + slot));
        }
        return;
    }
    regs_decrease<kRegsOther>();
    if (warp == kProducerWarp) {
        // ================================================================ producer
        Walk<D, kFew> walk(a);
        Item it;
#pragma unroll 1
        for (uint32_t ii = 0;; ++ii) {
            const int slot = ii % kItemSlots;
            // (a range is taken when one piece is left to do, so that slow blocks take fewer)
            auto due = [&]() {
                return ii < 2 || wait_warp(BAR(B_IEMPTY + (ii - 2) % kItemSlots), ((ii - 2) / kItemSlots) & 1, abort_flag,
                                           a.dev_status);
            };
            bool more = walk.next(a, it, due);
            while (more && it.nt == 0) {  // rows without keys: zeros, or NaN for a bad length
                if (a.op == kCross) fill_rows<D>(a, it);
                more = walk.next(a, it, due);
            }
            if (!more) it.nt = -1;
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
        }
        if (a.tiles_run) grid_dependency_wait();  // the join kernel waits for this one, and needs both
        return;
    }
    // ==================================================================== K and V copies
    if (warp == kProducerWarp + 3 && !small) return;
    constexpr int kCopies = Lo::BN / 4 * Lo::NBLK, kShare = kCopies * 3 / 4;  // gathers of a tile, of warps 5 and 6
    const bool helper = warp == kProducerWarp + 3;
    const uint64_t policy = l2_evict_first_policy();  // read once
    uint32_t s = 0, ph = 0;
#pragma unroll 1
    for (uint32_t ii = 0;; ++ii) {
        const int slot = ii % kItemSlots;
        if (!wait_warp(BAR(B_IFULL + slot), (ii / kItemSlots) & 1, abort_flag, a.dev_status)) break;
        const Item it = items[slot];
        if (it.nt < 0) break;
        const int first = helper || warp == kProducerWarp + 1 ? 0 : 1, last = helper || warp == kProducerWarp + 2 ? 1 : 0;
        Copier<D, Lo::BN> copy;
        Pages pages(a, first ? &vmap : &kmap, kFew, Lo::BN);
        copy.begin(a, pages, it);
        bool ok = true;
#pragma unroll 1
        for (int j = 0; ok && j < it.nt; ++j) {
            const Copier<D, Lo::BN> before = copy;
#pragma unroll 1
            for (int kv = first; ok && kv <= last; ++kv) {
                if (kv > first) copy = before;  // the helper's second tile: the same pages
                pages.map = kv ? &vmap : &kmap;
                const uint32_t full = BAR((kv ? B_VFULL : B_KFULL) + s), empty = BAR((kv ? B_VEMPTY : B_KEMPTY) + s);
                const uint32_t dst = smem_u32(smem + (kv ? Lo::OFF_V : Lo::OFF_K)) + s * Lo::TILE;
                ok = copy.tile(pages, j, dst, full, policy, helper ? kShare : 0, helper || !small ? kCopies : kShare,
                               bad_flag + slot, [&]() { return wait_warp(empty, ph ^ 1, abort_flag, a.dev_status); });
            }
            if (++s == kStages) s = 0, ph ^= 1;
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(BAR(B_IEMPTY + slot));
    }
    if (*abort_flag) {  // the block winds down: its copies in flight end first
        for (int i = 0; i < 2 * kStages; ++i) {
            const uint32_t full = BAR((i < kStages ? B_KFULL : B_VFULL) + i % kStages);
            for (int t = 0; t < 50 && !try_wait(full, ph ^ (static_cast<uint32_t>(i % kStages) < s ? 0u : 1u)); ++t) {
            }
        }
    }
}

}  // namespace

template <int D, bool LONG>
bool launch_few(const Args &a, const CUtensorMap &kmap, const CUtensorMap &vmap, const pkv_host::DeviceInfo &dev,
                cudaStream_t stream) {
    static std::mutex mu;
    static bool ready[64] = {};
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!ready[dev.device]) {
            if (Layout<D>::TOTAL > dev.max_smem_optin ||
                cudaFuncSetAttribute(few_rows_kernel<D, LONG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     Layout<D>::TOTAL) != cudaSuccess)
                return false;
            ready[dev.device] = true;
        }
    }
    return pkv_host::launch_dependent(few_rows_kernel<D, LONG>, dim3(a.blocks[kFew]), dim3(kThreads), Layout<D>::TOTAL, stream,
                                      kmap, vmap, a) == cudaSuccess;
}
template bool launch_few<64, false>(const Args &, const CUtensorMap &, const CUtensorMap &,
                                    const pkv_host::DeviceInfo &, cudaStream_t);
template bool launch_few<64, true>(const Args &, const CUtensorMap &, const CUtensorMap &, const pkv_host::DeviceInfo &,
                                   cudaStream_t);
template bool launch_few<128, false>(const Args &, const CUtensorMap &, const CUtensorMap &,
                                     const pkv_host::DeviceInfo &, cudaStream_t);
template bool launch_few<128, true>(const Args &, const CUtensorMap &, const CUtensorMap &,
                                    const pkv_host::DeviceInfo &, cudaStream_t);

}  // namespace ck
}  // namespace pkv
