// Attention with a sliding window and sinks over the paged cache, every pool
// type and shape: the entry points and the CUDA-core kernel.
//
// A query at position p sees key j iff j <= p and (j < sinks or p - j < window):
//   out = sum_j softmax_j(scale <q, K_j>) V_j  over those keys.
// They form one or two runs of positions, [0, ns) and [w0, p], which the kernel
// walks as one list of nv = ns + p + 1 - w0 keys; blocks between the runs are
// never read, so their table entries may hold anything.  The kernel is the form
// for shapes the tensor-core kernels do not take (f32 pools, block sizes other
// than 16, head widths other than 128): one CTA per (query, KV head), or per
// key range of it when a decode batch has few rows; 128 keys at a time, a
// thread per key for the scores, a thread per output column for the values.
// Bound: its own instructions, and for prefill the reads of each key once per row:
// 683 us where the tcgen05 decode takes 47 (64 sequences of 128 .. 2048 tokens,
// block-scaled), 62 ms where the prefill takes 0.22 (a prompt of 8191 tokens).
#include <algorithm>
#include <climits>
#include <cstdint>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace {

constexpr int kThreads = 128;
constexpr int kKeys = 128;           // keys per chunk
bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
constexpr int kMaxG = 16;

__device__ __forceinline__ float elem(const float* p) { return __ldg(p); }
__device__ __forceinline__ float elem(const uint16_t* p) {
    return __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16);
}
__device__ __forceinline__ float elem(const uint8_t* p) {
    return pa_dev::f16_lo(pa_dev::e4m3x2_to_f16x2(__ldg(p)));
}
// four consecutive elements (rows are multiples of four, at least 4-byte aligned)
__device__ __forceinline__ float4 elem4(const float* p) {
    const float4 x = __ldg(reinterpret_cast<const float4*>(p));
    return x;
}
__device__ __forceinline__ float4 elem4(const uint16_t* p) {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
    return make_float4(pa_dev::bf16_lo(x.x), pa_dev::bf16_hi(x.x), pa_dev::bf16_lo(x.y), pa_dev::bf16_hi(x.y));
}
__device__ __forceinline__ float4 elem4(const uint8_t* p) {
    const uint32_t x = __ldg(reinterpret_cast<const uint32_t*>(p));
    const uint32_t a = pa_dev::e4m3x2_to_f16x2(x & 0xffffu), b = pa_dev::e4m3x2_to_f16x2(x >> 16);
    return make_float4(pa_dev::f16_lo(a), pa_dev::f16_hi(a), pa_dev::f16_lo(b), pa_dev::f16_hi(b));
}
__device__ __forceinline__ float pow2(int biased) { return __uint_as_float(static_cast<uint32_t>(biased) << 23); }

__device__ __forceinline__ void store_out(const WindowParams& p, size_t i, float x) {
    if (p.out_bf16) reinterpret_cast<__nv_bfloat16*>(p.out)[i] = __float2bfloat16_rn(x);
    else reinterpret_cast<float*>(p.out)[i] = x;
}

// Decode: grid (S * nsplit, Hkv), row s.  Prefill: grid (max_q, Hkv, S), row
// blockIdx.x of sequence blockIdx.z.
template <typename QE, typename E>
__global__ void __launch_bounds__(kThreads) window_kernel(const WindowParams p) {
    extern __shared__ __align__(16) float sm[];
    float* qs = sm;                                        // [G][D]
    float* sc = qs + p.G * p.D;                            // [G][kKeys]
    __shared__ int64_t s_base[kKeys];                      // tile (elements) of each key's block, -1: none
    __shared__ int s_off[kKeys];
    __shared__ float s_vs[kKeys], s_m[kMaxG], s_l[kMaxG], s_cr[kMaxG];
    pa_dev::wait_prior_grid();
    pa_dev::allow_next_grid();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, h = blockIdx.y;
    const int G = p.G, D = p.D, B = p.B;
    int s, pos, split = 0;
    int64_t row;
    bool empty = false;
    if (p.cu_q) {
        s = blockIdx.z;
        const int q0 = __ldg(p.cu_q + s), n = __ldg(p.cu_q + s + 1) - q0, L = __ldg(p.lens + s);
        const bool reporter = tid == 0 && blockIdx.x == 0 && h == 0;
        if (q0 < 0 || n < 0 || q0 + static_cast<int64_t>(n) > p.T || L < n || n > p.max_q) {
            if (reporter) pa_dev::record_error(p.err, PA_ERR_INVALID_ARG);
            return;
        }
        if (L > static_cast<int64_t>(p.max_blocks) * B) {
            if (reporter) pa_dev::record_error(p.err, PA_ERR_BAD_LENGTH);
            return;
        }
        const int i = blockIdx.x;
        if (i >= n) return;
        pos = L - n + i;
        row = q0 + static_cast<int64_t>(i);
    } else {
        s = blockIdx.x / p.nsplit;
        split = blockIdx.x - s * p.nsplit;
        int L = __ldg(p.lens + s);
        const int cap = p.max_blocks * B;
        if (L < 0 || L > cap) {
            if (tid == 0 && h == 0 && split == 0) pa_dev::record_error(p.err, PA_ERR_BAD_LENGTH);
            L = L < 0 ? 0 : cap;
        }
        pos = max(0, L - 1);
        row = s;
        empty = L == 0;
    }
    const int w0 = max(0, pos - (p.window - 1)), ns = min(p.sinks, w0);
    const int nv = empty ? 0 : ns + pos + 1 - w0;
    int v0 = 0, v1 = nv;
    if (p.nsplit > 1) {                                    // this CTA's part of the keys
        const int per = (nv + p.nsplit - 1) / p.nsplit;
        v0 = min(nv, split * per);
        v1 = min(nv, v0 + per);
    }
    const QE* q = static_cast<const QE*>(p.q) + (row * p.Hq + static_cast<int64_t>(h) * G) * D;
    for (int i = tid; i < G * D; i += kThreads) qs[i] = elem(q + i);
    if (tid < G) {
        s_m[tid] = -INFINITY;
        s_l[tid] = 0.f;
    }
    float acc[2][kMaxG];
#pragma unroll
    for (int g = 0; g < kMaxG; ++g) acc[0][g] = acc[1][g] = 0.f;
    const int32_t* table = p.tables + static_cast<size_t>(s) * p.max_blocks;
    const E* kp = static_cast<const E*>(p.k);
    const E* vp = static_cast<const E*>(p.v);
    for (int c0 = v0; c0 < v1; c0 += kKeys) {
        const int nk = min(kKeys, v1 - c0);
        __syncthreads();                                   // qs written; the last chunk's sc, s_base read
        if (tid < nk) {
            const int v = c0 + tid, j = v < ns ? v : v - ns + w0;
            const int lb = j / B, off = j - lb * B, phys = __ldg(table + lb);
            const bool ok = phys >= 0 && phys < p.num_blocks;
            float x[kMaxG];
#pragma unroll
            for (int g = 0; g < kMaxG; ++g) x[g] = 0.f;
            const int64_t tile = (static_cast<int64_t>(phys) * p.Hkv + h) * B * D;
            float ks = p.scale_log2, vs = 1.f;
            if (ok) {
                if (p.scales) {
                    const uint8_t* e = p.scales + (static_cast<int64_t>(phys) * p.Hkv + h) * 2;
                    ks *= pow2(__ldg(e));
                    vs = pow2(__ldg(e + 1));
                }
                const E* kr = kp + tile + static_cast<int64_t>(off) * D;
                for (int d = 0; d < D; d += 4) {
                    const float4 k4 = elem4(kr + d);
#pragma unroll
                    for (int g = 0; g < kMaxG; ++g)
                        if (g < G) {
                            const float4 q4 = *reinterpret_cast<const float4*>(qs + g * D + d);
                            x[g] = fmaf(k4.x, q4.x, fmaf(k4.y, q4.y, fmaf(k4.z, q4.z, fmaf(k4.w, q4.w, x[g]))));
                        }
                }
            } else if (h == 0) {
                pa_dev::record_error(p.err, PA_ERR_BAD_BLOCK_ID);
            }
#pragma unroll
            for (int g = 0; g < kMaxG; ++g)
                if (g < G) sc[g * kKeys + tid] = ok ? x[g] * ks : -INFINITY;
            s_base[tid] = ok ? tile : -1;
            s_off[tid] = off;
            s_vs[tid] = vs;
        }
        __syncthreads();
        for (int g = warp; g < G; g += kThreads / 32) {    // a warp per head: reference, weights, sum
            float mx = -INFINITY;
            for (int j = lane; j < nk; j += 32) mx = fmaxf(mx, sc[g * kKeys + j]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float mo = s_m[g], mn = fmaxf(mo, mx), ms = mn == -INFINITY ? 0.f : mn;
            float l = 0.f;
            for (int j = lane; j < nk; j += 32) {
                const float w = pa_dev::ex2(sc[g * kKeys + j] - ms);
                l += w;
                sc[g * kKeys + j] = w * s_vs[j];           // the block's value scale rides on the weight
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            __syncwarp();
            if (lane == 0) {
                const float cr = mo == -INFINITY ? 0.f : pa_dev::ex2(mo - ms);
                s_cr[g] = cr;
                s_l[g] = s_l[g] * cr + l;
                s_m[g] = mn;
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int d = tid + r * kThreads;
            if (d >= D) break;
#pragma unroll
            for (int g = 0; g < kMaxG; ++g)
                if (g < G) acc[r][g] *= s_cr[g];
            for (int j = 0; j < nk; ++j) {
                if (s_base[j] < 0) continue;
                const float x = elem(vp + s_base[j] + static_cast<int64_t>(d) * B + s_off[j]);
#pragma unroll
                for (int g = 0; g < kMaxG; ++g)
                    if (g < G) acc[r][g] = fmaf(sc[g * kKeys + j], x, acc[r][g]);
            }
        }
    }
    __syncthreads();
    const size_t item = (static_cast<size_t>(s) * p.Hkv + h) * p.nsplit + split;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int d = tid + r * kThreads;
        if (d >= D) break;
#pragma unroll
        for (int g = 0; g < kMaxG; ++g) {
            if (g >= G) break;
            if (p.nsplit > 1) {
                p.part[(item * G + g) * (D + 2) + d] = acc[r][g];
            } else {
                const float l = s_l[g];
                store_out(p, (row * p.Hq + static_cast<int64_t>(h) * G + g) * D + d,
                          l == 0.f ? 0.f : acc[r][g] * p.v_scale / l);   // (a NaN stays one)
            }
        }
    }
    if (p.nsplit > 1 && tid < G) {
        p.part[(item * G + tid) * (D + 2) + D] = s_m[tid];
        p.part[(item * G + tid) * (D + 2) + D + 1] = s_l[tid];
    }
}

// One CTA per (sequence, KV head): the splits' partials, by log-sum-exp.
__global__ void __launch_bounds__(kThreads) window_merge_kernel(const WindowParams p) {
    pa_dev::wait_prior_grid();
    pa_dev::allow_next_grid();
    const int s = blockIdx.x / p.Hkv, h = blockIdx.x - s * p.Hkv, G = p.G, D = p.D;
    const size_t item = static_cast<size_t>(blockIdx.x) * p.nsplit;
    for (int i = threadIdx.x; i < G * D; i += kThreads) {
        const int g = i / D, d = i - g * D;
        float M = -INFINITY;
        for (int k = 0; k < p.nsplit; ++k) M = fmaxf(M, p.part[((item + k) * G + g) * (D + 2) + D]);
        const float Ms = M == -INFINITY ? 0.f : M;               // (sums without a reference are 0 or NaN)
        float l = 0.f, a = 0.f;
        for (int k = 0; k < p.nsplit; ++k) {
            const float* e = p.part + ((item + k) * G + g) * (D + 2);
            const float f = e[D] == -INFINITY ? 1.f : pa_dev::ex2(e[D] - Ms);
            l = fmaf(e[D + 1], f, l);
            a = fmaf(e[d], f, a);
        }
        store_out(p, (static_cast<int64_t>(s) * p.Hq + static_cast<int64_t>(h) * G) * D + i,
                  l == 0.f ? 0.f : a * p.v_scale / l);
    }
}

template <typename QE, typename E>
cudaError_t launch_generic(const WindowParams& p, dim3 grid, size_t smem, cudaStream_t st) {
    return pa_detail::launch_pdl(window_kernel<QE, E>, grid, dim3(kThreads), smem, st, p);
}

cudaError_t launch_any(const pa_pool* pool, const WindowParams& p, dim3 grid, cudaStream_t st) {
    const size_t smem = static_cast<size_t>(p.G) * (p.D + kKeys) * sizeof(float);      // at most 24 KB
    const cudaError_t e = pool->dtype == PA_F32 ? launch_generic<float, float>(p, grid, smem, st)
                        : pool->dtype == PA_BF16 ? launch_generic<uint16_t, uint16_t>(p, grid, smem, st)
                                                 : launch_generic<uint16_t, uint8_t>(p, grid, smem, st);
    pa_detail::count_launch();
    return e;
}

// Key ranges per (sequence, KV head) of a decode batch: four CTAs per SM, at
// least 256 keys a range.
int splits(const pa_pool* pool, int S, int64_t max_keys) {
    const int64_t items = static_cast<int64_t>(S) * pool->kv_heads;
    const int64_t want = std::max<int64_t>(1, 4LL * pool->num_sms / items);
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, (max_keys + 255) / 256)));
}

// Grow a workspace to at least `bytes`, zeroed.  An outgrown one is kept until
// the pool goes: a captured graph may still write to it.
int grow(pa_pool* pool, void** ws, size_t* have, size_t bytes) {
    if (*have >= bytes) return PA_OK;
    void* w = nullptr;
    if (cudaMalloc(&w, bytes) != cudaSuccess) {
        cudaGetLastError();
        return PA_ERR_OUT_OF_MEMORY;
    }
    // (not ordered with the caller's stream: waited for)
    if (cudaMemset(w, 0, bytes) != cudaSuccess || cudaStreamSynchronize(cudaStreamLegacy) != cudaSuccess) {
        cudaFree(w);
        return PA_ERR_CUDA;
    }
    if (*ws) pool->wws_old.push_back(*ws);
    *ws = w;
    *have = bytes;
    return PA_OK;
}

int ensure_partials(pa_pool* pool, size_t bytes) { return grow(pool, &pool->wws, &pool->wws_bytes, bytes); }
int ensure_tc(pa_pool* pool, int S) {
    return grow(pool, &pool->wtc, &pool->wtc_bytes,
                pa_detail::window_decode_tc_partials(pool) + pa_detail::window_decode_tc_counters(pool, S));
}

// The plain decode's partials, whatever the batch: a batch is split into no more than four
// ranges per SM (splits), and one that is not split has none.
size_t generic_partials(const pa_pool* pool, int G) {
    return 4 * static_cast<size_t>(pool->num_sms) * G * (pool->head_dim + 2) * sizeof(float);
}

void fill(const pa_pool* pool, int Hq, float scale, WindowParams* p) {
    const bool f8 = pool->dtype == PA_FP8E4M3;
    p->k = pool->k;
    p->v = pool->v;
    p->scales = pool->scales;
    p->err = pool->err;
    p->scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634 *
                                       (f8 ? static_cast<double>(pool->k_scale) : 1.0));
    p->v_scale = f8 ? pool->v_scale : 1.f;
    p->Hq = Hq;
    p->Hkv = pool->kv_heads;
    p->G = Hq / pool->kv_heads;
    p->D = pool->head_dim;
    p->B = pool->block_size;
    p->num_blocks = pool->num_blocks;
    p->nsplit = 1;
}

}  // namespace

namespace pa_detail {

int window_reserve(pa_pool* pool, int max_seqs, int max_q_heads) {
    if (max_q_heads / pool->kv_heads > kMaxG) return PA_ERR_UNSUPPORTED;
    const int rc = ensure_partials(pool, generic_partials(pool, max_q_heads / pool->kv_heads));
    return rc == PA_OK ? ensure_tc(pool, max_seqs) : rc;
}

// Everything of a windowed decode that can fail before a launch: its arguments, its workspace.
static int plan_decode_window(pa_pool* pool, const void* q, int num_seqs, int num_q_heads, const int32_t* block_tables,
                              int max_blocks_per_seq, const int32_t* context_lens, int window, int sinks, float scale,
                              void* out, pa_dtype out_dtype, WindowParams* params, bool* tc) {
    WindowParams& p = *params;
    fill(pool, num_q_heads, scale, &p);
    p.q = q;
    p.tables = block_tables;
    p.lens = context_lens;
    p.out = out;
    p.S = p.T = num_seqs;
    p.max_blocks = max_blocks_per_seq;
    // positions stay below 2^30: clamped here, differences of positions fit an int
    p.window = std::min(window, 1 << 30);
    p.sinks = std::min(sinks, 1 << 30);
    p.out_bf16 = out_dtype == PA_BF16;
    *tc = window_decode_tc_eligible(pool, p);
    if (*tc) {
        const int rc = ensure_tc(pool, num_seqs);
        p.part = static_cast<float*>(pool->wtc);
        return rc;
    }
    const int64_t cap = static_cast<int64_t>(max_blocks_per_seq) * pool->block_size;
    p.nsplit = splits(pool, num_seqs, std::min<int64_t>(cap, static_cast<int64_t>(window) + sinks));
    if (p.nsplit > 1) {
        const int rc = ensure_partials(pool, generic_partials(pool, p.G));
        if (rc != PA_OK) return rc;
        p.part = static_cast<float*>(pool->wws);
    }
    return PA_OK;
}

int check_decode_window(pa_pool* pool, const void* q, int num_seqs, int num_q_heads, const int32_t* block_tables,
                        int max_blocks_per_seq, const int32_t* context_lens, int window, int sinks, void* out,
                        pa_dtype out_dtype) {
    WindowParams p{};
    bool tc;
    return plan_decode_window(pool, q, num_seqs, num_q_heads, block_tables, max_blocks_per_seq, context_lens, window,
                              sinks, 1.f, out, out_dtype, &p, &tc);
}

int decode_window(pa_pool* pool, const void* q, int num_seqs, int num_q_heads, const int32_t* block_tables,
                  int max_blocks_per_seq, const int32_t* context_lens, int window, int sinks, float scale, void* out,
                  pa_dtype out_dtype, cudaStream_t st) {
    WindowParams p{};
    bool tc;
    const int rc = plan_decode_window(pool, q, num_seqs, num_q_heads, block_tables, max_blocks_per_seq, context_lens,
                                      window, sinks, scale, out, out_dtype, &p, &tc);
    if (rc != PA_OK) return rc;
    if (tc)
        return launch_window_decode_tc(
            pool, p, reinterpret_cast<int*>(static_cast<char*>(pool->wtc) + window_decode_tc_partials(pool)), st);
    cudaError_t e = launch_any(pool, p, dim3(num_seqs * p.nsplit, p.Hkv), st);
    if (e == cudaSuccess && p.nsplit > 1) {
        e = launch_pdl(window_merge_kernel, dim3(num_seqs * p.Hkv), dim3(kThreads), 0, st, p);
        count_launch();
    }
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int prefill_window(pa_pool* pool, const void* q, int num_tokens, int num_q_heads, const int32_t* cu_seqlens_q,
                   int num_seqs, int max_q_len, const int32_t* block_tables, int max_blocks_per_seq,
                   const int32_t* context_lens, int window, int sinks, float scale, void* out, pa_dtype out_dtype,
                   cudaStream_t st) {
    WindowParams p{};
    fill(pool, num_q_heads, scale, &p);
    p.q = q;
    p.cu_q = cu_seqlens_q;
    p.tables = block_tables;
    p.lens = context_lens;
    p.out = out;
    p.T = num_tokens;
    p.S = num_seqs;
    p.max_blocks = max_blocks_per_seq;
    p.max_q = max_q_len;
    // positions stay below 2^30: clamped here, differences of positions fit an int
    p.window = std::min(window, 1 << 30);
    p.sinks = std::min(sinks, 1 << 30);
    p.out_bf16 = out_dtype == PA_BF16;
    if (pool->opt_prefill_kernel == 0 && window_prefill_tc_eligible(pool, p))
        return launch_window_prefill_tc(pool, p, st);
    return launch_any(pool, p, dim3(max_q_len, p.Hkv, num_seqs), st) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa_detail

extern "C" int pa_prefill_window(pa_pool* pool, const void* q, int num_tokens, int num_q_heads,
                                 const int32_t* cu_seqlens_q, int num_seqs, int max_q_len,
                                 const int32_t* block_tables, int max_blocks_per_seq, const int32_t* context_lens,
                                 int window, int sinks, float scale, void* out, pa_dtype out_dtype, void* stream) {
    if (!pool || num_tokens < 0 || num_seqs < 0 || max_q_len < 0 || num_q_heads <= 0 || max_blocks_per_seq < 0 ||
        window < 1 || sinks < 0)
        return PA_ERR_INVALID_ARG;
    if (out_dtype != PA_F32 && out_dtype != PA_BF16) return PA_ERR_DTYPE;
    if (num_q_heads % pool->kv_heads != 0 || num_q_heads / pool->kv_heads > kMaxG || num_seqs > 65535 ||
        pool->kv_heads > 65535)
        return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || num_tokens == 0 || max_q_len == 0) return PA_OK;
    const size_t osz = out_dtype == PA_BF16 ? 2 : 4;
    if (!q || !cu_seqlens_q || !block_tables || !context_lens || !out || max_blocks_per_seq == 0 ||
        !aligned(q, 16) || !aligned(out, osz) || !aligned(cu_seqlens_q, 4) || !aligned(block_tables, 4) ||
        !aligned(context_lens, 4))
        return PA_ERR_INVALID_ARG;
    if (static_cast<int64_t>(max_blocks_per_seq) * pool->block_size > (int64_t{1} << 30)) return PA_ERR_UNSUPPORTED;
    pa_detail::DeviceGuard g(pool->device);
    if (!g.ok) return PA_ERR_CUDA;
    return pa_detail::prefill_window(pool, q, num_tokens, num_q_heads, cu_seqlens_q, num_seqs, max_q_len,
                                     block_tables, max_blocks_per_seq, context_lens, window, sinks, scale, out,
                                     out_dtype, static_cast<cudaStream_t>(stream));
}
