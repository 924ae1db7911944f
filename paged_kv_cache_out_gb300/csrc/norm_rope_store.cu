// norm_rope_store.cu -- per-head RMS norm and rotation of a step's new queries
// and keys, with the K/V rows scattered to their pool slots.
//
// miniVLLM "LLMEngine" (model shapes: Qwen3-0.6B norms each query and key head
// before the rotation, Llama-3.2-1B only rotates) and mini-sglang "Engine
// Class" (out_loc: the pool slot of every new token).
//
// Memory-bound: every q, k and v element is read once and written once, with
// about 8 flops for an element of q and k.  head_dim / 16 lanes hold one head
// row, 16 elements (two 16-byte pieces) each; the pieces are chosen so that a
// lane holds both elements of each of its pairs: the rotation is then
// lane-local, and the mean of squares is the only exchange (3 or 2 shuffles).
// The rotation factors of a token are the same for all its heads: a warp keeps
// its lanes' 8 cosines and 8 sines in registers and runs over the token's
// heads.
//
// Two kernels: heads in registers, for few tokens, and whole tokens streamed
// through shared memory, for many.  Measured: one token 2.6 us a call (the launch),
// 256 tokens of 16 + 8 + 8 heads of 128 3.0 us, 16384 tokens (277 MB) 47.8 us, 5.8 TB/s
// against 6.8 TB/s of a plain copy.
#include <math.h>

#include <mutex>

#include "common.cuh"

namespace pkv {
namespace nrs {

constexpr int kThreads = 128;

struct Args {
    const __nv_bfloat16 *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const __nv_bfloat16 *q_weight, *k_weight;
    float eps;
    const int32_t *positions;
    const float *cos_sin;
    int64_t max_positions;
    int rot_dim;
    const int32_t *out_loc;
    int64_t num_tokens;
    int Hq, Hkv;
    __nv_bfloat16 *k_cache, *v_cache;
    int64_t num_slots;
    __nv_bfloat16 *q_out;
    int32_t *dev_status;
    int split;  // warps that share a token's heads
};

// Eight bf16 as four fp32 pairs, and back.
__device__ __forceinline__ void unpack8(const uint4 &w, float2 *f) {
    f[0] = bf16x2_to_f2(w.x), f[1] = bf16x2_to_f2(w.y), f[2] = bf16x2_to_f2(w.z), f[3] = bf16x2_to_f2(w.w);
}
__device__ __forceinline__ uint4 pack8(const float2 *f) {
    return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                      pack_bf16x2(f[3].x, f[3].y));
}

// (a, b) turned by (c, s), pair by pair: (a c - b s, a s + b c)
__device__ __forceinline__ void turn(float2 &a, float2 &b, float2 c, float2 s) {
    const float2 ns = make_float2(-s.x, -s.y);
    const float2 x = ffma2(b, ns, fmul2(a, c));
    b = ffma2(b, c, fmul2(a, s));
    a = x;
}

// Norm and rotation of a lane's two pieces of a head row: packed bf16 in and out.
// w0, w1: the weights when `norm`; cs, sn: factors of the lane's pairs when `rot`.
template <int D, bool INTERLEAVED>
__device__ __forceinline__ void norm_rope(uint4 &y0, uint4 &y1, bool norm, const float2 *w0, const float2 *w1,
                                          float eps, bool rot, const float2 *cs, const float2 *sn, bool bad_pos) {
    constexpr int LPH = D / 16;
    float2 f0[4], f1[4];
    unpack8(y0, f0);
    unpack8(y1, f1);
    if (norm) {
        float2 sq = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) sq = ffma2(f0[e], f0[e], ffma2(f1[e], f1[e], sq));
        float ss = sq.x + sq.y;
#pragma unroll
        for (int o = LPH / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(ss * (1.0f / D) + eps);
        const float2 r2 = make_float2(r, r);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f0[e] = fmul2(f0[e], fmul2(w0[e], r2));
            f1[e] = fmul2(f1[e], fmul2(w1[e], r2));
        }
    }
    if (rot) {
        if constexpr (INTERLEAVED) {
            // f[e] is the pair (2i, 2i + 1)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float c0 = (e & 1) ? cs[e / 2].y : cs[e / 2].x;
                const float s0 = (e & 1) ? sn[e / 2].y : sn[e / 2].x;
                const float c1 = (e & 1) ? cs[2 + e / 2].y : cs[2 + e / 2].x;
                const float s1 = (e & 1) ? sn[2 + e / 2].y : sn[2 + e / 2].x;
                f0[e] = make_float2(f0[e].x * c0 - f0[e].y * s0, f0[e].x * s0 + f0[e].y * c0);
                f1[e] = make_float2(f1[e].x * c1 - f1[e].y * s1, f1[e].x * s1 + f1[e].y * c1);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) turn(f0[e], f1[e], cs[e], sn[e]);
        }
    }
    if (bad_pos) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            f0[e] = f1[e] = make_float2(__int_as_float(0x7fc00000), __int_as_float(0x7fc00000));
    }
    if (norm || rot || bad_pos) y0 = pack8(f0), y1 = pack8(f1);
}

// This lane's rotation factors at a table row.
__device__ __forceinline__ void load_factors(const float *row, int rot_dim, int l, float2 *cs, float2 *sn) {
    const float4 *c = reinterpret_cast<const float4 *>(row) + 2 * l, *s = c + rot_dim / 8;
    const float4 c0 = __ldg(c), c1 = __ldg(c + 1), s0 = __ldg(s), s1 = __ldg(s + 1);
    cs[0] = make_float2(c0.x, c0.y), cs[1] = make_float2(c0.z, c0.w);
    cs[2] = make_float2(c1.x, c1.y), cs[3] = make_float2(c1.z, c1.w);
    sn[0] = make_float2(s0.x, s0.y), sn[1] = make_float2(s0.z, s0.w);
    sn[2] = make_float2(s1.x, s1.y), sn[3] = make_float2(s1.z, s1.w);
}

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) norm_rope_store_kernel(const Args a) {
    constexpr int LPH = D / 16;   // lanes per head row
    constexpr int HPW = 32 / LPH; // heads per warp step
    constexpr int UNROLL = 4;     // warp steps whose loads are in flight together
    grid_dependency_wait();  // inputs come from the kernel before
    allow_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t warp = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
    const int64_t nwarps = ((int64_t)gridDim.x * kThreads) >> 5;
    const int l = lane % LPH, sub = lane / LPH;
    // this lane's two pieces of 8 elements.  Interleaved pairs lie in one
    // piece; otherwise element i's partner is i + rot_dim / 2, in the piece
    // rot_dim / 16 further on.  The pieces past rot_dim go to the lanes past
    // rot_dim / 16, two in a row.
    const int nrot = a.rot_dim / 16;  // lanes with a rotation to do
    const bool rot = l < nrot;
    const int p0 = INTERLEAVED || !rot ? 2 * l : l;
    const int p1 = INTERLEAVED || !rot ? 2 * l + 1 : l + nrot;
    // a token's warp steps: HPW query heads each, then key heads, then value heads
    const int q_steps = (a.Hq + HPW - 1) / HPW, kv_steps = (a.Hkv + HPW - 1) / HPW;
    const int steps = q_steps + 2 * kv_steps;

    for (int64_t unit = warp; unit < a.num_tokens * a.split; unit += nwarps) {
        const int64_t t = unit / a.split;
        const int part = static_cast<int>(unit - t * a.split);
        const int64_t slot = a.out_loc[t];
        bool bad_pos = false;
        const float *table = nullptr;
        if (nrot > 0) {
            const int64_t pos = a.positions[t];
            bad_pos = pos < 0 || pos >= a.max_positions;
            if (rot && !bad_pos) table = a.cos_sin + pos * a.rot_dim;
        }
        const bool store = slot >= 0 && slot < a.num_slots && !bad_pos;
        if (lane == 0 && part == 0 && a.dev_status) {
            const int bits = (slot >= a.num_slots ? PKV_DEV_BAD_SLOT : 0) | (bad_pos ? PKV_DEV_BAD_POS : 0);
            if (bits) atomicOr(a.dev_status, bits);
        }
        // cosines and sines of this lane's eight pairs
        float2 cs[4], sn[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) cs[e] = make_float2(1.f, 1.f), sn[e] = make_float2(0.f, 0.f);
        if (table) load_factors(table, a.rot_dim, l, cs, sn);
        float2 w0[4], w1[4];  // the weights of the kind of head in hand
        int kind = -1;        // 0: query, 1: key, 2: value
        const __nv_bfloat16 *weight = nullptr;
        for (int step0 = part; step0 < steps; step0 += UNROLL * a.split) {
            uint4 x0[UNROLL], x1[UNROLL];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int step = step0 + u * a.split;
                const int first = step < q_steps ? 0 : step < q_steps + kv_steps ? q_steps : q_steps + kv_steps;
                const int h = (step - first) * HPW + sub;
                const __nv_bfloat16 *src = first == 0         ? a.q + t * a.q_stride
                                           : first == q_steps ? a.k + t * a.k_stride
                                                              : a.v + t * a.v_stride;
                x0[u] = x1[u] = make_uint4(0u, 0u, 0u, 0u);
                if (step < steps && h < (first == 0 ? a.Hq : a.Hkv)) {
                    x0[u] = reinterpret_cast<const uint4 *>(src + h * D)[p0];
                    x1[u] = reinterpret_cast<const uint4 *>(src + h * D)[p1];
                }
            }
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int step = step0 + u * a.split;
                if (step >= steps) break;  // the same for the whole warp
                const int first = step < q_steps ? 0 : step < q_steps + kv_steps ? q_steps : q_steps + kv_steps;
                const int h = (step - first) * HPW + sub;
                const int now = first == 0 ? 0 : first == q_steps ? 1 : 2;
                uint4 y0 = x0[u], y1 = x1[u];
                if (now < 2) {
                    if (now != kind) {
                        kind = now;
                        weight = now ? a.k_weight : a.q_weight;
                        if (weight) {
                            unpack8(__ldg(reinterpret_cast<const uint4 *>(weight) + p0), w0);
                            unpack8(__ldg(reinterpret_cast<const uint4 *>(weight) + p1), w1);
                        }
                    }
                    norm_rope<D, INTERLEAVED>(y0, y1, weight != nullptr, w0, w1, a.eps, rot, cs, sn, bad_pos);
                }
                if (h < (now ? a.Hkv : a.Hq) && (now == 0 || store)) {
                    __nv_bfloat16 *dst = now == 0 ? a.q_out + (t * a.Hq + h) * D
                                                  : (now == 1 ? a.k_cache : a.v_cache) + (slot * a.Hkv + h) * D;
                    reinterpret_cast<uint4 *>(dst)[p0] = y0;
                    reinterpret_cast<uint4 *>(dst)[p1] = y1;
                }
            }
        }
    }
}

// The same for many tokens.  Here the loads that a warp has in flight limit the
// rate, and registers limit those; so every warp is a block of its own that keeps a
// ring of whole tokens in shared memory: the q, k and v rows of a token come by
// three bulk copies two tokens ahead, are normed and rotated in place, and leave by
// bulk copies; the values never pass through registers.  The rotation factors are
// loaded a token ahead.
constexpr int kRing = 3;
static size_t stream_smem(int heads, int D) { return static_cast<size_t>(kRing) * heads * D * 2 + 64; }

__device__ __forceinline__ void bulk_store(void *dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// at most N of this thread's groups of bulk stores still read shared memory
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(32) norm_rope_store_stream_kernel(const Args a) {
    constexpr int LPH = D / 16;
    constexpr int HPW = 32 / LPH;
    extern __shared__ __align__(128) uint8_t smem[];
    const int H = a.Hq + 2 * a.Hkv;
    const uint32_t tb = H * D * 2, qb = a.Hq * D * 2, kb = a.Hkv * D * 2;  // of a token, its q and its k
    const uint32_t ring = smem_u32(smem);
    const uint32_t bars = ring + kRing * tb;  // [kRing]
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kRing * tb + 8 * kRing);
    const int lane = threadIdx.x;
    const int l = lane % LPH, sub = lane / LPH;
    const int nrot = a.rot_dim / 16;
    const bool rot = l < nrot;
    const int p0 = INTERLEAVED || !rot ? 2 * l : l;
    const int p1 = INTERLEAVED || !rot ? 2 * l + 1 : l + nrot;
    if (lane == 0) {
        for (int s = 0; s < kRing; ++s) mbar_init(bars + 8 * s, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    __syncwarp();
    grid_dependency_wait();  // inputs come from the kernel before
    allow_dependents();

    const int64_t step = gridDim.x;
    auto fetch = [&](int64_t t, int s) {  // lane 0
        if (t >= a.num_tokens) return;
        const uint32_t dst = ring + s * tb, bar = bars + 8 * s;
        mbar_arrive_expect_tx(bar, tb);
        bulk_load(dst, a.q + t * a.q_stride, qb, bar);
        bulk_load(dst + qb, a.k + t * a.k_stride, kb, bar);
        bulk_load(dst + qb + kb, a.v + t * a.v_stride, kb, bar);
    };
    // slot, and position (-1: out of range), of a token
    auto place = [&](int64_t t, int &slot, int64_t &pos) {
        slot = -1;
        pos = 0;
        if (t >= a.num_tokens) return;
        slot = a.out_loc[t];
        if (nrot > 0) {
            pos = a.positions[t];
            if (pos < 0 || pos >= a.max_positions) pos = -1;
        }
    };
    float2 w[2][2][4];  // query and key weights of this lane's two pieces
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const __nv_bfloat16 *src = k ? a.k_weight : a.q_weight;
        if (src) {
            unpack8(__ldg(reinterpret_cast<const uint4 *>(src) + p0), w[k][0]);
            unpack8(__ldg(reinterpret_cast<const uint4 *>(src) + p1), w[k][1]);
        }
    }
    int64_t t = blockIdx.x;
    int slot, next_slot;
    int64_t pos, next_pos;
    if (lane == 0) {
        fetch(t, 0);
        fetch(t + step, 1);
    }
    place(t, slot, pos);
    place(t + step, next_slot, next_pos);
    float2 cs[4], sn[4];
    if (rot && pos >= 0) load_factors(a.cos_sin + pos * a.rot_dim, a.rot_dim, l, cs, sn);
    uint32_t it = 0;
    for (; t < a.num_tokens; t += step, ++it) {
        const int s = it % kRing;
        float2 next_cs[4], next_sn[4];
        const bool more = t + step < a.num_tokens;
        if (rot && more && next_pos >= 0)
            load_factors(a.cos_sin + next_pos * a.rot_dim, a.rot_dim, l, next_cs, next_sn);
        int slot2;
        int64_t pos2;
        place(t + 2 * step, slot2, pos2);
        if (!mbar_wait_warp(bars + 8 * s, (it / kRing) & 1, abort_flag, a.dev_status)) break;
        const uint32_t row = ring + s * tb;
        const bool bad_pos = pos < 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const bool norm = (k ? a.k_weight : a.q_weight) != nullptr;
            if (!norm && nrot == 0) continue;
            const int heads = k ? a.Hkv : a.Hq;
#pragma unroll 2
            for (int h0 = 0; h0 < heads; h0 += HPW) {
                const int h = h0 + sub;
                const uint32_t at = row + (k ? qb : 0u) + (h < heads ? h : heads - 1) * (D * 2);
                uint4 y0 = lds128(at + 16 * p0), y1 = lds128(at + 16 * p1);
                norm_rope<D, INTERLEAVED>(y0, y1, norm, w[k][0], w[k][1], a.eps, rot, cs, sn, bad_pos);
                if (h < heads) {
                    sts128(at + 16 * p0, y0);
                    sts128(at + 16 * p1, y1);
                }
            }
        }
        fence_proxy_async_smem();  // the copies that follow read what the lanes wrote
        __syncwarp();
        if (lane == 0) {
            bulk_store(a.q_out + t * a.Hq * D, row, qb);
            if (slot >= 0 && slot < a.num_slots && !bad_pos) {
                bulk_store(a.k_cache + (int64_t)slot * a.Hkv * D, row + qb, kb);
                bulk_store(a.v_cache + (int64_t)slot * a.Hkv * D, row + qb + kb, kb);
            }
            bulk_commit();
            const int bits = (slot >= a.num_slots ? PKV_DEV_BAD_SLOT : 0) | (bad_pos ? PKV_DEV_BAD_POS : 0);
            if (bits && a.dev_status) atomicOr(a.dev_status, bits);
            bulk_wait_read<1>();  // the token before has left its place, which is taken next
            fetch(t + 2 * step, (it + 2) % kRing);
        }
        slot = next_slot, pos = next_pos;
        next_slot = slot2, next_pos = pos2;
#pragma unroll
        for (int e = 0; e < 4; ++e) cs[e] = next_cs[e], sn[e] = next_sn[e];
    }
    if (t < a.num_tokens && lane == 0) {
        // gave up on a copy: the others may still write to the ring
        for (int k = 1; k < kRing && t + k * step < a.num_tokens; ++k) {
            const uint32_t n = it + k;
            *abort_flag = 0;
            if (k < kRing - 1) mbar_wait(bars + 8 * (n % kRing), (n / kRing) & 1, abort_flag, a.dev_status);
        }
    }
    if (lane == 0) bulk_wait_all();
}

// ---------------------------------------------------------------- host side
constexpr int kMinWarps = 4;

// Allow the stream kernels their shared memory, once per device.
static bool prepare(const pkv_host::DeviceInfo &dev) {
    static std::mutex mu;
    static bool ready[64];
    std::lock_guard<std::mutex> lk(mu);
    if (!ready[dev.device]) {
        auto allow = [&](void (*kernel)(Args)) {
            return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        dev.max_smem_optin / kMinWarps) == cudaSuccess;
        };
        ready[dev.device] = allow(norm_rope_store_stream_kernel<128, true>) &&
                            allow(norm_rope_store_stream_kernel<128, false>) &&
                            allow(norm_rope_store_stream_kernel<64, true>) &&
                            allow(norm_rope_store_stream_kernel<64, false>);
    }
    return ready[dev.device];
}

}  // namespace nrs
}  // namespace pkv

extern "C" pkv_status pkv_qk_norm_rope_store(
    const pkv_bf16 *q, int64_t q_stride, const pkv_bf16 *k, int64_t k_stride, const pkv_bf16 *v,
    int64_t v_stride, const pkv_bf16 *q_weight, const pkv_bf16 *k_weight, float eps,
    const int32_t *positions, const float *cos_sin, int64_t max_positions, int rot_dim,
    int interleaved, const int32_t *out_loc, int64_t num_tokens, int num_q_heads, int num_kv_heads,
    int head_dim, pkv_bf16 *k_cache, pkv_bf16 *v_cache, int64_t num_pages, int page_size,
    pkv_bf16 *q_out, int32_t *dev_status, void *stream) {
    using namespace pkv::nrs;
    if (num_tokens < 0 || num_pages < 0 || page_size <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
        head_dim <= 0 || max_positions < 0 || rot_dim < 0 || rot_dim > head_dim || !(eps >= 0.f) ||
        isinf(eps))
        return PKV_EINVAL;
    if (num_tokens == 0) return PKV_OK;
    if (!q || !k || !v || !out_loc || !k_cache || !v_cache || !q_out) return PKV_EINVAL;
    if (rot_dim > 0 && (!positions || !cos_sin)) return PKV_EINVAL;
    if ((head_dim != 64 && head_dim != 128) || rot_dim % 16 != 0) return PKV_EUNSUPPORTED;
    const int64_t q_row = (int64_t)num_q_heads * head_dim, kv_row = (int64_t)num_kv_heads * head_dim;
    if (q_stride < q_row || k_stride < kv_row || v_stride < kv_row || q_stride % 8 || k_stride % 8 ||
        v_stride % 8)
        return PKV_EINVAL;
    if (q_out == q && q_stride != q_row) return PKV_EINVAL;
    // head indexes and pool slots are 32-bit
    if (q_row + 2 * kv_row > 0x7fffffffll || num_pages > 0x7fffffffll / page_size) return PKV_EUNSUPPORTED;
    const void *const aligned[] = {q, k, v, q_weight, k_weight, k_cache, v_cache, q_out,
                                   rot_dim > 0 ? cos_sin : nullptr};
    for (const void *p : aligned)
        if (!pkv_host::aligned16(p)) return PKV_EINVAL;
    pkv_host::DeviceInfo dev;
    if (!pkv_host::current_device(&dev)) return PKV_ECUDA;
    auto bf = [](const pkv_bf16 *p) { return reinterpret_cast<const __nv_bfloat16 *>(p); };
    auto bfw = [](pkv_bf16 *p) { return reinterpret_cast<__nv_bfloat16 *>(p); };
    const int heads_per_step = 32 / (head_dim / 16);
    const int steps = (num_q_heads + heads_per_step - 1) / heads_per_step +
                      2 * ((num_kv_heads + heads_per_step - 1) / heads_per_step);
    Args a{bf(q), bf(k), bf(v), q_stride, k_stride, v_stride, bf(q_weight), bf(k_weight), eps,
           positions, cos_sin, max_positions, rot_dim, out_loc, num_tokens, num_q_heads,
           num_kv_heads, bfw(k_cache), bfw(v_cache), num_pages * page_size, bfw(q_out),
           dev_status, 1};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // Many tokens are streamed through rings of shared memory, where the rings of
    // at least kMinWarps warps fit an SM and every other warp gets a token.  Below
    // that the ring's start-up costs more than it saves.  Measured, heads in
    // registers against streamed: 16 + 8 + 8 heads of 128, 300 tokens 3.0 / 4.1 us,
    // 700 tokens 5.5 / 5.1, 2000 tokens 10.2 / 9.5, 16384 tokens 54.1 / 47.9;
    // 8 + 1 + 1 heads, 1021 tokens 4.6 / 4.8, 2900 tokens 7.2 / 6.5.
    const size_t smem = stream_smem(num_q_heads + 2 * num_kv_heads, head_dim);
    int64_t per_sm = dev.max_smem_optin / (static_cast<int64_t>(smem) + 1024);
    if (per_sm > 32) per_sm = 32;  // blocks that an SM holds
    const int64_t warps = dev.sm_count * per_sm;
    if (per_sm >= kMinWarps && 2 * num_tokens >= warps) {
        if (!prepare(dev)) return PKV_ECUDA;
        auto kernel = head_dim == 128 ? (interleaved ? norm_rope_store_stream_kernel<128, true>
                                                     : norm_rope_store_stream_kernel<128, false>)
                                      : (interleaved ? norm_rope_store_stream_kernel<64, true>
                                                     : norm_rope_store_stream_kernel<64, false>);
        return pkv_host::launch_dependent(kernel, dim3(static_cast<unsigned>(warps < num_tokens ? warps : num_tokens)), dim3(32), smem,
                                          st, a) == cudaSuccess
                   ? PKV_OK
                   : PKV_ECUDA;
    }
    // few tokens: their heads are shared between warps until the machine has
    // 16 warps per SM
    const int64_t want = (int64_t)dev.sm_count * 16;
    int64_t split = (want + num_tokens - 1) / num_tokens;
    if (split > steps) split = steps;
    a.split = static_cast<int>(split);
    const int64_t blocks_needed = (num_tokens * split + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t max_blocks = (int64_t)dev.sm_count * 4;
    const dim3 grid(static_cast<unsigned>(blocks_needed < max_blocks ? blocks_needed : max_blocks));
    auto kernel = head_dim == 128
                      ? (interleaved ? norm_rope_store_kernel<128, true> : norm_rope_store_kernel<128, false>)
                      : (interleaved ? norm_rope_store_kernel<64, true> : norm_rope_store_kernel<64, false>);
    return pkv_host::launch_dependent(kernel, grid, dim3(kThreads), 0, st, a) == cudaSuccess ? PKV_OK : PKV_ECUDA;
}
