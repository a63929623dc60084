// Rotary positions fused with the append (pa_append_rope), f32, bf16 and
// per-pool-scaled fp8 pools; block-scaled pools rotate inside their own append
// (pa_kv_scaled.cu), and 16-token blocks of 128-wide heads take pa_append_tile.cu.
//
// Bound: bytes.  Rotating in the append saves writing the rotated keys and
// reading them back (a third of the keys' and values' traffic), and rounds
// them once, from the fp32 rotation to the pool's type.  A thread takes a pair at a
// time: 60 us for 64 tokens where pa_append_tile.cu takes 30, append and read-back.
#include <cstdint>

#include "pa_rope.cuh"

namespace {

using pa_detail::RopeParams;

constexpr int kThreads = 256;

template <typename E>
struct Store;                       // how an element of the pool is written
template <>
struct Store<uint16_t> {
    typedef uint16_t In;
    static __device__ __forceinline__ uint16_t conv(float x, float) { uint16_t y; pa_rope::from_f32(y, x); return y; }
};
template <>
struct Store<float> {
    typedef float In;
    static __device__ __forceinline__ float conv(float x, float) { return x; }
};
template <>
struct Store<uint8_t> {
    typedef uint16_t In;
    static __device__ __forceinline__ uint8_t conv(float x, float scale) {
        return static_cast<uint8_t>(pa_dev::e4m3x2_from_f32(__fdiv_rn(x, scale), 0.f));
    }
};

// One CTA per token: its angles once in shared memory, then its query rows and
// its key and value rows.
template <typename E>
__global__ void __launch_bounds__(kThreads) append_rope_kernel(
    E* __restrict__ kpool, E* __restrict__ vpool, const void* __restrict__ k, const void* __restrict__ v,
    const int64_t* __restrict__ slots, int T, int Hkv, int D, int B, int64_t num_slots, float k_scale,
    float v_scale, const RopeParams r, int* err) {
    typedef typename Store<E>::In In;
    __shared__ float2 cs[128];
    pa_dev::wait_prior_grid();
    pa_dev::allow_next_grid();
    const int t = blockIdx.x, tid = threadIdx.x;
    for (int f = tid; f < r.half; f += kThreads) cs[f] = pa_rope::angle(r, t, T, f, err);
    __syncthreads();
    if (r.q) pa_rope::rotate_queries<In>(r, t, D, cs, tid, kThreads);
    const int64_t slot = slots[t];
    if (slot < 0) return;
    if (slot >= num_slots) {
        if (tid == 0) pa_dev::record_error(err, PA_ERR_BAD_SLOT);
        return;
    }
    const int64_t blk = slot / B;
    const int off = static_cast<int>(slot - blk * B);
    const In* ks = static_cast<const In*>(k) + static_cast<int64_t>(t) * r.k_stride;
    const In* vs = static_cast<const In*>(v) + static_cast<int64_t>(t) * r.v_stride;
    const int units = D / 2;
    for (int i = tid; i < Hkv * units; i += kThreads) {
        const int h = i / units, u = i - h * units;
        const int2 e = pa_rope::unit(u, r.half, r.interleaved);
        const int64_t tile = (blk * Hkv + h) * static_cast<int64_t>(B) * D;
        float2 x = make_float2(pa_rope::to_f32(ks[h * D + e.x]), pa_rope::to_f32(ks[h * D + e.y]));
        if (u < r.half) x = pa_rope::rotate(x, cs[u]);
        E* kd = kpool + tile + static_cast<int64_t>(off) * D;
        kd[e.x] = Store<E>::conv(x.x, k_scale);
        kd[e.y] = Store<E>::conv(x.y, k_scale);
        E* vd = vpool + tile + off;
        vd[static_cast<int64_t>(2 * u) * B] = Store<E>::conv(pa_rope::to_f32(vs[h * D + 2 * u]), v_scale);
        vd[static_cast<int64_t>(2 * u + 1) * B] = Store<E>::conv(pa_rope::to_f32(vs[h * D + 2 * u + 1]), v_scale);
    }
}

}  // namespace

extern "C" int pa_append_rope(pa_pool* pool, const void* q, int64_t q_stride, int num_q_heads, const void* k,
                              int64_t k_stride, const void* v, int64_t v_stride, const int64_t* slot_mapping,
                              int num_tokens, const int32_t* positions, int num_axes, const float* inv_freq,
                              const int32_t* axis, int rotary_dim, int interleaved, void* q_out, void* stream) {
    if (!pool || num_tokens < 0 || num_q_heads < 0) return PA_ERR_INVALID_ARG;
    const int D = pool->head_dim;
    const int64_t row = static_cast<int64_t>(pool->kv_heads) * D;
    if (rotary_dim < 2 || rotary_dim > D || rotary_dim % 2 != 0 || num_axes < 1 || num_axes > 4)
        return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    const size_t es = pool->dtype == PA_F32 ? 4 : 2;                 // q, k and v elements
    auto aligned = [](const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; };
    if (!k || !v || !slot_mapping || !positions || !inv_freq || k_stride < row || v_stride < row ||
        !aligned(slot_mapping, 8) || !aligned(k, es) || !aligned(v, es) || !aligned(positions, 4) ||
        !aligned(inv_freq, 4) || !aligned(axis, 4))
        return PA_ERR_INVALID_ARG;
    if (num_q_heads > 0 && (!q || !q_out || q_stride < static_cast<int64_t>(num_q_heads) * D ||
                            !aligned(q, es) || !aligned(q_out, es)))
        return PA_ERR_INVALID_ARG;
    pa_detail::DeviceGuard g(pool->device);
    if (!g.ok) return PA_ERR_CUDA;
    RopeParams r{};
    r.q = num_q_heads > 0 ? q : nullptr;
    r.q_out = q_out;
    r.positions = positions;
    r.inv_freq = inv_freq;
    r.axis = axis;
    r.q_stride = q_stride;
    r.k_stride = k_stride;
    r.v_stride = v_stride;
    r.Hq = num_q_heads;
    r.num_axes = num_axes;
    r.half = rotary_dim / 2;
    r.interleaved = interleaved != 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (pool->scales) return pa_detail::launch_append_scaled(pool, k, v, slot_mapping, num_tokens, r, st);
    if (pa_detail::append_tile_eligible(pool, k, v, r) && pa_detail::append_notes_ready(pool, num_tokens))
        return pa_detail::launch_append_tile(pool, k, v, slot_mapping, num_tokens, r, st);
    const int64_t num_slots = static_cast<int64_t>(pool->num_blocks) * pool->block_size;
    auto launch = [&](auto* kp, auto* vp, auto kernel) {
        return pa_detail::launch_pdl(kernel, dim3(num_tokens), dim3(kThreads), 0, st, kp, vp, k, v, slot_mapping,
                                     num_tokens, pool->kv_heads, D, pool->block_size, num_slots, pool->k_scale,
                                     pool->v_scale, r, pool->err);
    };
    cudaError_t e;
    if (pool->dtype == PA_FP8E4M3)
        e = launch(static_cast<uint8_t*>(pool->k), static_cast<uint8_t*>(pool->v), append_rope_kernel<uint8_t>);
    else if (pool->dtype == PA_BF16)
        e = launch(static_cast<uint16_t*>(pool->k), static_cast<uint16_t*>(pool->v), append_rope_kernel<uint16_t>);
    else
        e = launch(static_cast<float*>(pool->k), static_cast<float*>(pool->v), append_rope_kernel<float>);
    pa_detail::count_launch();
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
