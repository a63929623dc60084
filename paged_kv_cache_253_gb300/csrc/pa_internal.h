// Internal interface between the C-ABI front end (pa_api.cu) and the kernel
// translation units (pa_kv.cu, pa_decode.cu).  Not installed, not part of the ABI.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <utility>
#include <vector>

#include <cuda.h>
#include <cuda_runtime.h>

#include "pa.h"

struct pa_pool {
    int device = 0;
    int num_blocks = 0, block_size = 0, kv_heads = 0, head_dim = 0;
    pa_dtype dtype = PA_BF16;
    float k_scale = 1.f, v_scale = 1.f;   // fp8 pools: a code stands for e4m3(code) * scale
    void* k = nullptr;          // K [num_blocks][kv_heads][block_size][head_dim]
    void* v = nullptr;          // V [num_blocks][kv_heads][head_dim][block_size]
    int* err = nullptr;         // device error word (first recorded PA_ERR_*)
    void* ws = nullptr;         // decode workspace: header, then partials
    size_t ws_bytes = 0;
    // block-scaled pools (PA_FP8E4M3_BLOCK): biased exponents [num_blocks][kv_heads][2] (K, V)
    uint8_t* scales = nullptr;
    // scratch of appends by block: which offsets of a block the call writes (all zero
    // between calls) and the token that writes each: 72 bytes per block of 16.  Block-scaled
    // pools have it from the start, others from their first rotary append that needs it
    unsigned long long* app_mask = nullptr;     // [num_blocks]
    int32_t* app_token = nullptr;               // [num_blocks][block_size]
    // windowed attention's partials; outgrown buffers live until the pool is
    // destroyed (a captured graph may still name them)
    void* wws = nullptr;
    size_t wws_bytes = 0;
    std::vector<void*> wws_old;
    // the same of its tensor-core decode: partials, then a counter per item
    // (zero between calls)
    void* wtc = nullptr;
    size_t wtc_bytes = 0;
    int num_sms = 0;
    int smem_optin = 0;         // largest dynamic shared memory a CTA may opt in to
    // TMA descriptors of K (boxes 64 d x 16 tokens, 128-byte swizzle) and of V^T
    // (boxes 16 tokens x 128 d, 32-byte swizzle), made on first use
    CUtensorMap kmap;
    CUtensorMap vmap;
    bool tmaps_ready = false;
    // kernel-choice options (pa_pool_set_option)
    int opt_partition_cap = -1;     // decode partition cap, tokens; -1 automatic, 0 none
    int opt_shared_kernel = 0;      // 0 tcgen05 where eligible, 1 mma.sync
    int opt_prefill_kernel = 0;     // 0 tcgen05 where eligible, 1 mma.sync
    // shared-prefix descriptor last uploaded by pa_decode_shared (host copy + device copy)
    std::vector<int> desc_host;
    int* desc_dev = nullptr;
    size_t desc_cap = 0;        // ints
};

// Everything one decode launch needs, passed by value to the kernels.
struct DecodeParams {
    const void* q;              // [S][Hq][D]
    const void* k;              // pool K
    const void* v;              // pool V (transposed tiles)
    const int32_t* tables;      // [S][max_blocks]
    const int32_t* lens;        // [S]
    void* out;                  // [S][Hq][D]
    float* part_acc;            // [max_items][G][D]  un-normalised partial sums
    float* part_ml;             // [max_items][G][2]  (running max, sum) in log2 units
    int* ticket;                // [2] work ticket and retired-CTA count, zero between launches
    int* sched;                 // [S + 3] PT, item count, first item of each sequence
    int* err;
    float scale_log2;           // scale * log2(e) (* k_scale for an fp8 pool)
    float v_scale;              // factor on the value sums (fp8 pool's v_scale, else 1)
    float k_scale;              // fp8 pool's k_scale (quantizing a fused append), else 1
    int S, Hq, Hkv, G, D, B, num_blocks, max_blocks;
    int out_bf16;
    int items_target;           // wanted number of work items (fast path)
    int pt_min;                 // smallest partition, tokens (multiple of B)
    int pt_soft;                // > pt_min: the smallest partition grows towards this many
                                // tokens (multiple of B) while at least items_floor items remain
    int items_floor;            // (both zero: pt_min alone)
    int wave_items;             // > 0: the item target is whole waves of this many items,
    int wave_tokens;            // one wave per wave_tokens token-heads per item, at most
                                // items_target
    int pt_max;                 // largest partition, tokens (multiple of B; 0: no cap)
    int max_items;              // partial slots the workspace holds (fast path)
    int pt_fixed;               // > 0: use exactly this partition size
    // Shared-prefix description (pa_decode_shared); all zero / null otherwise.
    int n_shared_items;         // shared work items, heads included (K * Hkv)
    int chunk_tokens;           // shared tokens per item (multiple of B)
    int members_per_tile;       // group members per item (16-row tiles of members x G)
    const int* sh_items;        // [K][4] (group, member tile, chunk, 0)
    const int* seq_group;       // [S] group of each sequence, -1 if none
    const int* seq_member;      // [S] index of the sequence inside its group
    const int* seq_start;       // [S] first private token (the shared span precedes it)
    const int* g_members_off;   // [Ng + 1]
    const int* g_members;       // batch indices, grouped
    const int* g_nchunks;       // [Ng] shared chunks of each group
    const int* g_spart_base;    // [Ng] first shared-partial slot of each group
    const int* g_shared_tokens; // [Ng] shared tokens of each group
    float* spart_acc;           // [slots][Hkv][G][D] shared-span partial sums
    float* spart_ml;            // [slots][Hkv][G][2]
    // Fused append (pa_append_decode): each sequence's new token, written by
    // the warp that reads the sequence's last block; null otherwise.
    const void* new_k;          // [S][Hkv][D]
    const void* new_v;          // [S][Hkv][D]
    const int64_t* new_slots;   // [S] slot of position L-1 of each sequence, or < 0
    // 1: the preceding kernel is the tcgen05 shared-prefix kernel, which already
    // waited for the work before it; the split kernel then runs alongside it and
    // waits for it only before exiting (so the merge after it sees both).
    int defer_wait;
};

// Everything one prefill launch needs (pa_prefill), passed by value.
struct PrefillParams {
    const uint16_t* q;          // [T][Hq][D] bf16
    const void* k;              // pool K (bf16 values or e4m3 codes)
    const void* v;              // pool V^T tiles
    const int32_t* cu_q;        // [S + 1] first query row of each sequence
    const int32_t* tables;      // [S][max_blocks]
    const int32_t* lens;        // [S] context length after the chunk's append
    void* out;                  // [T][Hq][D]
    int* err;
    float scale_log2;           // scale * log2(e) (* k_scale for an fp8 pool)
    float v_scale;              // factor on the outputs (fp8 pool's v_scale, else 1)
    int T, S, Hq, Hkv, G, B, num_blocks, max_blocks;
    int max_q;                  // longest chunk the launch was sized for
    int out_bf16;
};

// Bytes of one K or V element of the pool.
inline size_t pool_elem_size(pa_dtype t) {
    return t == PA_FP8E4M3 || t == PA_FP8E4M3_BLOCK ? 1 : t == PA_BF16 ? 2 : 4;
}

// Score factor of a decode in log2 units (an fp8 pool's k_scale folded in)
// and the factor on the value sums.
inline void decode_scales(const pa_pool* pool, float scale, DecodeParams* p) {
    const bool f8 = pool->dtype == PA_FP8E4M3;
    p->scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634 *
                                       (f8 ? static_cast<double>(pool->k_scale) : 1.0));
    p->v_scale = f8 ? pool->v_scale : 1.f;
    p->k_scale = f8 ? pool->k_scale : 1.f;
}

// Decode workspace header: ticket[2], 2 spare ints, the published schedule
// (S + 3 ints used of S + 4); zeroed before first use (the kernels reset the
// tickets they count).
inline size_t decode_header_bytes(int S) {
    return ((static_cast<size_t>(S) + 8) * sizeof(int) + 255) / 256 * 256;
}

// Everything one windowed attention launch needs (decode: one query per
// sequence at position lens[s] - 1; prefill: chunks), passed by value.
struct WindowParams {
    const void* q;              // decode [S][Hq][D], prefill [T][Hq][D]
    const void* k;              // pool K
    const void* v;              // pool V (transposed tiles)
    const uint8_t* scales;      // block-scaled pool: biased exponents, else null
    const int32_t* cu_q;        // prefill: [S + 1] first query row of each sequence, else null
    const int32_t* tables;      // [S][max_blocks]
    const int32_t* lens;        // [S]
    void* out;
    int* err;
    float* part;                // partials of split decode rows
    float scale_log2;           // scale * log2(e) (* k_scale for an fp8 pool)
    float v_scale;              // factor on the outputs (fp8 pool's v_scale, else 1)
    int T, S, Hq, Hkv, G, D, B, num_blocks, max_blocks;
    int max_q;                  // longest chunk the launch was sized for
    int window, sinks;          // key j of query p: j <= p and (j < sinks or p - j < window)
    int out_bf16;
    int nsplit;                 // decode: key ranges per (sequence, KV head)
    int by_length;              // tcgen05 prefill: start long contexts first
};

// Pools whose elements are e4m3 codes.
namespace pa_detail {
inline bool is_code(pa_dtype t) { return t == PA_FP8E4M3 || t == PA_FP8E4M3_BLOCK; }

// Makes the pool's device current for a call and restores the caller's after it.
struct DeviceGuard {
    int prev = -1, own;
    bool ok = true;
    explicit DeviceGuard(int dev) : own(dev) {
        if (cudaGetDevice(&prev) != cudaSuccess) { ok = false; return; }
        if (prev != dev && cudaSetDevice(dev) != cudaSuccess) ok = false;
    }
    ~DeviceGuard() {
        if (prev >= 0 && prev != own) cudaSetDevice(prev);
    }
};

// Raise a kernel's dynamic shared memory limit, once per device (done: one bit each,
// a variable of the kernel's own).
template <typename K>
inline bool allow_smem(K kernel, int device, size_t bytes, std::atomic<uint64_t>& done) {
    const uint64_t bit = device < 64 ? uint64_t{1} << device : 0;
    if (bit && (done.load(std::memory_order_acquire) & bit)) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) != cudaSuccess)
        return false;
    done.fetch_or(bit, std::memory_order_release);
    return true;
}
}  // namespace pa_detail

// A window no context reaches: plain causal attention.
constexpr int kNoWindow = 0x7fffffff;

namespace pa_detail {

void count_launch();

// Launch `kernel` on `st` allowing programmatic dependent launch (the kernel
// must call pa_dev::wait_prior_grid() before reading any input).
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t st, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Launchers; each returns PA_OK or PA_ERR_CUDA (launch failure).
int launch_append(const pa_pool* p, const void* k, const void* v, const int64_t* slots,
                  int T, cudaStream_t st);
int launch_copy(const pa_pool* p, const int64_t* pairs, int P, cudaStream_t st);

// Rotary positions applied while appending (pa_append_rope); null q: no queries.
struct RopeParams {
    const void* q;
    void* q_out;                // [T][Hq][D]
    const int32_t* positions;   // [num_axes][T]
    const float* inv_freq;      // [half]
    const int32_t* axis;        // [half] or null: axis 0
    int64_t q_stride, k_stride, v_stride;   // elements between tokens
    int Hq, num_axes, half, interleaved;    // half 0: nothing is rotated
};
// Append to a block-scaled pool, rotating k (and q) on the way if rope->half > 0.
int launch_append_scaled(pa_pool* p, const void* k, const void* v, const int64_t* slots, int T,
                         const RopeParams& rope, cudaStream_t st);

// Its note of which offsets of each block the call writes, and by which token.
int launch_append_notes(pa_pool* p, const int64_t* slots, int T, cudaStream_t st);
// Appends by whole block tiles (16-token blocks, head width 128), every pool type
// but f32, and the read-back of such pools (pa_append_tile.cu).
bool append_tile_eligible(const pa_pool* p, const void* k, const void* v, const RopeParams& r);
bool append_notes_ready(pa_pool* p, int T);     // its scratch for T tokens is there (made if need be)
int launch_append_tile(pa_pool* p, const void* k, const void* v, const int64_t* slots, int T,
                       const RopeParams& rope, cudaStream_t st);
bool read_tile_eligible(const pa_pool* p, const void* k, const void* v);
int launch_read_tile(pa_pool* p, const int64_t* slots, int n, void* k, void* v, cudaStream_t st);

// Windowed attention: generic kernel for every shape and pool type.  check_decode_window
// is what decode_window checks and allocates before it launches.
int check_decode_window(pa_pool* pool, const void* q, int num_seqs, int num_q_heads,
                        const int32_t* block_tables, int max_blocks_per_seq,
                        const int32_t* context_lens, int window, int sinks, void* out,
                        pa_dtype out_dtype);
int decode_window(pa_pool* pool, const void* q, int num_seqs, int num_q_heads,
                  const int32_t* block_tables, int max_blocks_per_seq,
                  const int32_t* context_lens, int window, int sinks, float scale, void* out,
                  pa_dtype out_dtype, cudaStream_t st);
int prefill_window(pa_pool* pool, const void* q, int num_tokens, int num_q_heads,
                   const int32_t* cu_seqlens_q, int num_seqs, int max_q_len,
                   const int32_t* block_tables, int max_blocks_per_seq,
                   const int32_t* context_lens, int window, int sinks, float scale, void* out,
                   pa_dtype out_dtype, cudaStream_t st);
int window_reserve(pa_pool* pool, int max_seqs, int max_q_heads);
// Its tcgen05 prefill form (pa_window_tc.cu).
bool window_prefill_tc_eligible(const pa_pool* pool, const WindowParams& p);
int launch_window_prefill_tc(pa_pool* pool, const WindowParams& p, cudaStream_t st);
// Its tcgen05 decode form (pa_window_decode.cu).
bool window_decode_tc_eligible(const pa_pool* pool, const WindowParams& p);
size_t window_decode_tc_counters(const pa_pool* pool, int S);
size_t window_decode_tc_partials(const pa_pool* pool);
int launch_window_decode_tc(pa_pool* pool, const WindowParams& p, int* counters, cudaStream_t st);

// Decode: how the launch is shaped for a pool and batch.
struct DecodePlan {
    bool shared = false;        // shared-prefix items present (fast path only)
    bool fuse = false;          // the decode kernel also appends each sequence's new token
    bool tc = false;            // shared items run in the tcgen05 kernel before the split pass
    pa_pool* pool = nullptr;
    bool fast;                  // tensor-core path (bf16 pool, or fp8 codes widened to f16)
    bool bf16;                  // pool element type is bf16
    bool fp8;                   // pool element type is e4m3
    int grid, threads;
    size_t smem;
    int items_target, pt_min, pt_max = 0, pt_fixed;
    int pt_soft = 0, items_floor = 0;
    int wave_items = 0, wave_tokens = 0;
    size_t max_items;
    size_t min_items;           // fewest partial slots the kernel can work with (fast path)
};
int plan_decode(pa_pool* p, int S, int Hq, int max_blocks, DecodePlan* plan);
// Host checks of pa_decode's arguments (shared by every decode entry point).
int check_decode_args(const pa_pool* pool, const void* q, int S, int Hq, const int32_t* tables,
                      int max_blocks, const int32_t* lens, const void* out, pa_dtype out_dtype);
int launch_decode(const DecodePlan& plan, const DecodeParams& prm, cudaStream_t st);

// TMA descriptors of the pool's K and V^T (16-token blocks), made once per pool.
int ensure_tensor_maps(pa_pool* pool);

// tcgen05 shared-prefix items (pa_shared_tc.cu).
bool shared_tc_eligible(const pa_pool* pool, int G);
int shared_tc_rows();
int shared_tc_chunk_tokens();     // shared tokens per item (a multiple of 16)
int launch_shared_tc(pa_pool* pool, const DecodeParams& p, cudaStream_t st);

// tcgen05 prefill (pa_shared_tc.cu): one CTA per (128 query rows, KV head,
// sequence); bf16 pools of 16-token blocks, head_dim 128.
bool prefill_tc_eligible(const pa_pool* pool);
int prefill_tc_rows();
int launch_prefill_tc(pa_pool* pool, const PrefillParams& p, dim3 grid, cudaStream_t st);

}  // namespace pa_detail
