// Append to a block-scaled pool (PA_FP8E4M3_BLOCK), and the read-back of
// cached rows by slot (every pool type).  16-token blocks of 128-wide heads take
// pa_append_tile.cu instead.
//
// The mathematics.  K and V of each (block, KV head) carry one scale 2^(b-127)
// each.  For the finite values x that a call writes into a block, e(x) is the
// smallest power of two with max|x| / e <= 448 (b >= 1); from the fp32 bits of
// the maximum m this is b = (bits(m) + 0x1fffff >> 23) - 8: the addition
// carries into the exponent exactly when the significand is above 1.75.  A
// block whose offset 0 is written starts anew (b from the new rows alone, every
// other code zero); otherwise b = max(b, b_new), and if it rose, the codes that
// stay are re-rounded, code' = e4m3(value(code) 2^(b_old - b)): exact but for
// values that become subnormal.  code = e4m3(x 2^(127-b)), nearest even,
// saturating; powers of two make the division exact.
//
// Which thread does it.  A block's scale depends on all rows of the call that
// land in it, and they may come in any order.  A first kernel notes, per block,
// which offsets the call writes and by which token; in the second, the CTA of
// the token with a block's lowest written offset is the block's leader, builds
// the block's tiles in shared memory and writes them whole (16 bytes a thread,
// V^T rows too, instead of one byte per token), and clears the note.
//
// Bound: instructions and shared memory, an element at a time.  On the shapes of
// pa_append_tile.cu it took 74 us where that takes 27 (5378 tokens, appended and read
// back), 30 against 17 for 64 tokens.
#include <algorithm>
#include <cstdint>

#include "pa_rope.cuh"

namespace {

using pa_detail::RopeParams;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

__global__ void __launch_bounds__(256) append_note_kernel(const int64_t* __restrict__ slots, int T, int B,
                                                          int64_t num_slots, unsigned long long* mask,
                                                          int32_t* token, int* err) {
    pa_dev::wait_prior_grid();
    pa_dev::allow_next_grid();
    const int t = blockIdx.x * 256 + threadIdx.x;
    if (t >= T) return;
    const int64_t slot = slots[t];
    if (slot < 0) return;
    if (slot >= num_slots) {
        pa_dev::record_error(err, PA_ERR_BAD_SLOT);
        return;
    }
    token[slot] = t;
    atomicOr(mask + slot / B, 1ull << (slot % B));
}

__device__ __forceinline__ int scale_exponent(float amax) {
    return max(1, static_cast<int>((__float_as_uint(amax) + 0x1fffffu) >> 23) - 8);
}
__device__ __forceinline__ float pow2(int biased) {                 // 2^(biased - 127), 0 for 0
    return __uint_as_float(static_cast<uint32_t>(biased) << 23);
}
__device__ __forceinline__ float code_value(uint32_t code) {
    return pa_dev::f16_lo(pa_dev::e4m3x2_to_f16x2(code & 0xffu));
}

// One CTA per token of the call: its angles and its query rows, and, if the
// token leads a block, that block's tiles (one warp per KV head).
__global__ void __launch_bounds__(kThreads) append_scaled_kernel(
    uint8_t* __restrict__ kpool, uint8_t* __restrict__ vpool, uint8_t* __restrict__ scales,
    const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, const int64_t* __restrict__ slots, int T,
    int Hkv, int D, int B, int64_t num_slots, unsigned long long* mask, const int32_t* __restrict__ token,
    const RopeParams r, int tile_warps, int* err) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float2 cs[128];
    pa_dev::wait_prior_grid();
    pa_dev::allow_next_grid();
    const int t = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int half = r.half;
    if (r.q) {
        for (int f = tid; f < half; f += kThreads) cs[f] = pa_rope::angle(r, t, T, f, err);
        __syncthreads();
        pa_rope::rotate_queries<uint16_t>(r, t, D, cs, tid, kThreads);
    }
    const int64_t slot = slots[t];
    if (slot < 0 || slot >= num_slots) return;
    const int64_t blk = slot / B;
    const int off0 = static_cast<int>(slot - blk * B);
    // the leader alone clears the mask, so any other CTA sees it whole or zero
    const unsigned long long m = *reinterpret_cast<volatile unsigned long long*>(mask + blk);
    if (m == 0 || __ffsll(static_cast<long long>(m)) - 1 != off0 || token[slot] != t) return;

    const int32_t* tok = token + blk * B;
    // angles of the block's new tokens: [B][half] behind the warps' tiles
    float2* bcs = reinterpret_cast<float2*>(smem + (tile_warps * B * D + 15) / 16 * 16);
    if (half > 0) {
        for (int i = tid; i < B * half; i += kThreads) {
            const int o = i / half;
            if ((m >> o) & 1) bcs[i] = pa_rope::angle(r, tok[o], T, i - o * half, err);
        }
        __syncthreads();
    }
    const bool fresh = m & 1;
    const int units = D / 2, tile_bytes = B * D;
    unsigned char* tile = smem + warp * tile_bytes;
    // work: (KV head, K or V), one warp each
    for (int w = warp; w < 2 * Hkv && warp < tile_warps; w += tile_warps) {
        const int h = w >> 1, is_v = w & 1;
        const uint16_t* src = is_v ? v : k;
        const int64_t stride = is_v ? r.v_stride : r.k_stride;
        const int hrot = is_v ? 0 : half;                        // values are not rotated
        auto load = [&](int o, int u, int2 e) {
            const uint16_t* row = src + static_cast<int64_t>(tok[o]) * stride + h * D;
            const float2 x = make_float2(pa_rope::to_f32(__ldg(row + e.x)), pa_rope::to_f32(__ldg(row + e.y)));
            return u < hrot ? pa_rope::rotate(x, bcs[o * half + u]) : x;
        };
        // largest finite magnitude of the new rows
        float amax = 0.f;
        for (unsigned long long left = m; left; left &= left - 1) {
            const int o = __ffsll(static_cast<long long>(left)) - 1;
            for (int u = lane; u < units; u += 32) {
                const float2 x = load(o, u, pa_rope::unit(u, hrot, r.interleaved));
                const float a = fabsf(x.x), b = fabsf(x.y);
                if (a < INFINITY) amax = fmaxf(amax, a);         // false for NaN too
                if (b < INFINITY) amax = fmaxf(amax, b);
            }
        }
        for (int s = 16; s > 0; s >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, s));
        const int64_t si = (blk * Hkv + h) * 2 + is_v;
        const int b_old = fresh ? 0 : scales[si];
        const int b = max(b_old, scale_exponent(amax));
        // the tile as it stays: copied, re-rounded, or zero
        uint8_t* dst = (is_v ? vpool : kpool) + (blk * Hkv + h) * static_cast<int64_t>(tile_bytes);
        const float shrink = b_old > 0 ? pow2(b_old - b + 127 > 0 ? b_old - b + 127 : 0) : 0.f;
        for (int i = lane; i < tile_bytes / 4; i += 32) {
            uint32_t c = 0;
            if (b_old > 0) {
                c = reinterpret_cast<const uint32_t*>(dst)[i];
                if (b != b_old)
                    c = pa_dev::e4m3x2_from_f32(code_value(c) * shrink, code_value(c >> 8) * shrink) |
                        pa_dev::e4m3x2_from_f32(code_value(c >> 16) * shrink, code_value(c >> 24) * shrink) << 16;
            }
            reinterpret_cast<uint32_t*>(tile)[i] = c;
        }
        __syncwarp();
        // the new rows over it
        const float inv = pa_dev::inverse_scale(b);
        for (unsigned long long left = m; left; left &= left - 1) {
            const int o = __ffsll(static_cast<long long>(left)) - 1;
            for (int u = lane; u < units; u += 32) {
                const int2 e = pa_rope::unit(u, hrot, r.interleaved);
                const float2 x = load(o, u, e);
                const uint32_t c = pa_dev::e4m3x2_from_f32(x.x * inv, x.y * inv);
                tile[is_v ? e.x * B + o : o * D + e.x] = static_cast<uint8_t>(c);
                tile[is_v ? e.y * B + o : o * D + e.y] = static_cast<uint8_t>(c >> 8);
            }
        }
        __syncwarp();
        if (tile_bytes % 16 == 0)
            for (int i = lane; i < tile_bytes / 16; i += 32)
                reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(tile)[i];
        else
            for (int i = lane; i < tile_bytes / 4; i += 32)
                reinterpret_cast<uint32_t*>(dst)[i] = reinterpret_cast<const uint32_t*>(tile)[i];
        if (lane == 0) scales[si] = static_cast<uint8_t>(b);
        __syncwarp();
    }
    __syncthreads();
    if (tid == 0) mask[blk] = 0;
}

// One warp per (entry, KV head): the slot's key row and value column.
template <typename E, typename O>
__global__ void __launch_bounds__(256) read_kv_kernel(const E* __restrict__ kpool, const E* __restrict__ vpool,
                                                      const uint8_t* __restrict__ scales,
                                                      const int64_t* __restrict__ slots, O* __restrict__ k,
                                                      O* __restrict__ v, int T, int Hkv, int D, int B,
                                                      int64_t num_slots, float k_scale, float v_scale, int* err) {
    pa_dev::wait_prior_grid();
    pa_dev::allow_next_grid();
    const int64_t wi = (blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (wi >= static_cast<int64_t>(T) * Hkv) return;
    const int t = static_cast<int>(wi / Hkv), h = static_cast<int>(wi - static_cast<int64_t>(t) * Hkv);
    const int64_t slot = slots[t];
    const int64_t out = wi * D;
    if (slot < 0 || slot >= num_slots) {
        if (slot >= 0 && lane == 0) pa_dev::record_error(err, PA_ERR_BAD_SLOT);
        for (int d = lane; d < D; d += 32) k[out + d] = v[out + d] = O(0);
        return;
    }
    const int64_t blk = slot / B;
    const int off = static_cast<int>(slot - blk * B);
    const int64_t tile = (blk * Hkv + h) * static_cast<int64_t>(B) * D;
    if constexpr (sizeof(E) == 1) {
        float ks = k_scale, vs = v_scale;
        if (scales) {
            ks = pow2(scales[(blk * Hkv + h) * 2]);
            vs = pow2(scales[(blk * Hkv + h) * 2 + 1]);
        }
        for (int d = lane; d < D; d += 32) {
            pa_rope::from_f32(k[out + d], code_value(kpool[tile + static_cast<int64_t>(off) * D + d]) * ks);
            pa_rope::from_f32(v[out + d], code_value(vpool[tile + static_cast<int64_t>(d) * B + off]) * vs);
        }
    } else {
        for (int d = lane; d < D; d += 32) {
            k[out + d] = kpool[tile + static_cast<int64_t>(off) * D + d];
            v[out + d] = vpool[tile + static_cast<int64_t>(d) * B + off];
        }
    }
}

}  // namespace

namespace pa_detail {

int launch_append_notes(pa_pool* p, const int64_t* slots, int T, cudaStream_t st) {
    const cudaError_t e = launch_pdl(append_note_kernel, dim3((T + 255) / 256), dim3(256), 0, st, slots, T,
                                     p->block_size, static_cast<int64_t>(p->num_blocks) * p->block_size, p->app_mask,
                                     p->app_token, p->err);
    count_launch();
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int launch_append_scaled(pa_pool* p, const void* k, const void* v, const int64_t* slots, int T,
                         const RopeParams& rope, cudaStream_t st) {
    if (append_tile_eligible(p, k, v, rope)) return launch_append_tile(p, k, v, slots, T, rope, st);
    const int64_t num_slots = static_cast<int64_t>(p->num_blocks) * p->block_size;
    // as many warps with a tile each as 96 KB hold
    const size_t tile = static_cast<size_t>(p->block_size) * p->head_dim;
    const int warps = static_cast<int>(std::min<size_t>(kWarps, std::max<size_t>(1, (96u << 10) / tile)));
    const size_t smem = (warps * tile + 15) / 16 * 16 + static_cast<size_t>(p->block_size) * rope.half * sizeof(float2);
    // (the most that any pool asks for: 96 KB, and the angles of 64 tokens)
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(append_scaled_kernel, p->device, (96u << 10) + 64 * 128 * sizeof(float2) + 16, done)) return PA_ERR_CUDA;
    const int rc = launch_append_notes(p, slots, T, st);
    if (rc != PA_OK) return rc;
    const cudaError_t e = launch_pdl(append_scaled_kernel, dim3(T), dim3(kThreads), smem, st, static_cast<uint8_t*>(p->k),
                   static_cast<uint8_t*>(p->v), p->scales, static_cast<const uint16_t*>(k),
                   static_cast<const uint16_t*>(v), slots, T, p->kv_heads, p->head_dim, p->block_size, num_slots,
                   p->app_mask, static_cast<const int32_t*>(p->app_token), rope, warps, p->err);
    count_launch();
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa_detail

extern "C" int pa_read_kv(pa_pool* pool, const int64_t* slots, int num_slots, void* k, void* v, void* stream) {
    if (!pool || num_slots < 0) return PA_ERR_INVALID_ARG;
    if (num_slots == 0) return PA_OK;
    const size_t es = pool->dtype == PA_F32 ? 4 : 2;
    if (!slots || !k || !v || reinterpret_cast<uintptr_t>(slots) % 8 != 0 ||
        reinterpret_cast<uintptr_t>(k) % es != 0 || reinterpret_cast<uintptr_t>(v) % es != 0)
        return PA_ERR_INVALID_ARG;
    const int64_t grid = (static_cast<int64_t>(num_slots) * pool->kv_heads + 7) / 8;
    if (grid > 0x7fffffff) return PA_ERR_UNSUPPORTED;
    pa_detail::DeviceGuard g(pool->device);
    if (!g.ok) return PA_ERR_CUDA;
    if (pa_detail::read_tile_eligible(pool, k, v))
        return pa_detail::launch_read_tile(pool, slots, num_slots, k, v, static_cast<cudaStream_t>(stream));
    const int64_t total = static_cast<int64_t>(pool->num_blocks) * pool->block_size;
    auto launch = [&](auto kernel, auto elem, auto outv) {
        typedef decltype(elem) E;
        typedef decltype(outv) O;
        return pa_detail::launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(256), 0,
                                     static_cast<cudaStream_t>(stream), static_cast<const E*>(pool->k),
                                     static_cast<const E*>(pool->v), static_cast<const uint8_t*>(pool->scales), slots,
                                     static_cast<O*>(k), static_cast<O*>(v), num_slots, pool->kv_heads,
                                     pool->head_dim, pool->block_size, total, pool->k_scale, pool->v_scale, pool->err);
    };
    cudaError_t e;
    if (pa_detail::is_code(pool->dtype)) e = launch(read_kv_kernel<uint8_t, uint16_t>, uint8_t{}, uint16_t{});
    else if (pool->dtype == PA_BF16) e = launch(read_kv_kernel<uint16_t, uint16_t>, uint16_t{}, uint16_t{});
    else e = launch(read_kv_kernel<float, float>, float{}, float{});
    pa_detail::count_launch();
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
