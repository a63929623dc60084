// Appends by block tile: 16-token blocks, head width 128, bf16 and code pools,
// with rotary positions or without; and the read-back of such pools by slot.
// Other shapes: pa_kv.cu, pa_rope.cu and pa_kv_scaled.cu, which also states the
// scale rule of block-scaled pools.
//
// Bound: bytes.  Values are stored transposed, so one token's value is 128
// scattered elements, but a block's 16 tokens fill whole 16-byte rows.  The CTA
// of the token with the lowest written offset of a block leads the block: a warp
// takes one KV head's keys or values of all 16 positions into registers (16-byte
// loads, two rows at a time), rotates, quantises and transposes them there, and
// writes 16 bytes a thread.
//
// Which tokens of the call share a block: every CTA looks for them among the
// call's slots itself while there are at most kDirect of them (one launch, and
// one memory latency; a note's kernel takes 4 us by itself); more tokens are noted per
// block by a kernel in front (pa_kv_scaled.cu).
//
// Measured (8 KV heads, block-scaled): 64 tokens of 64 sequences appended and read back
// 16 us, both calls' launches (the kernels alone, one by one: 6 and 5); 5378 tokens 27 us
// (notes 3, tiles 18, read-back 10); four images' 9896 tokens with 32 query heads rotated
// 80 us (notes 3, queries 29 at 5.6 TB/s, tiles 37, read-back 13).  The tiles are bound by their instructions, 700 to 1200
// for a lane's 64 elements, and by four dependent loads in a row before them.
//
// Angles: positions times frequencies in turns, as 64-bit fixed-point fractions
// of a turn, where the multiplication wraps as angles do.  Frequencies are
// converted once per CTA in 64-bit floating point, whose rate on this GPU is 2
// operations per cycle and SM.  A frequency below 1 is off by up to 2^-55.6 of a turn, its
// product with 1 / 2 pi being rounded to 53 bits, so an angle by that times the position:
// 2^-35.6 of a turn at 2^20, 2^-24.6 at 2^31.
#include <algorithm>
#include <cstdint>

#include "pa_rope.cuh"

namespace {

using pa_detail::RopeParams;

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kD = 128, kB = 16, kTile = kD * kB;
constexpr int kDirect = 512;
enum Kind { kBf16, kFp8, kScaled };

__device__ __forceinline__ int scale_exponent(float amax) {         // see pa_kv_scaled.cu
    return max(1, static_cast<int>((__float_as_uint(amax) + 0x1fffffu) >> 23) - 8);
}
__device__ __forceinline__ float pow2(int biased) { return __uint_as_float(static_cast<uint32_t>(biased) << 23); }
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    return (pa_dev::e4m3x2_from_f32(a, b) & 0xffffu) | pa_dev::e4m3x2_from_f32(c, d) << 16;
}
__device__ __forceinline__ uint32_t shrink4(uint32_t c, float f) {  // four codes times f, re-rounded
    const uint32_t a = pa_dev::e4m3x2_to_f16x2(c & 0xffffu), b = pa_dev::e4m3x2_to_f16x2(c >> 16);
    return codes4(pa_dev::f16_lo(a) * f, pa_dev::f16_hi(a) * f, pa_dev::f16_lo(b) * f, pa_dev::f16_hi(b) * f);
}
__device__ __forceinline__ uint32_t byte_mask(uint32_t four) {      // bit i -> byte i
    return ((four & 1) | (four & 2) << 7 | (four & 4) << 14 | (four & 8) << 21) * 255u;
}

// Eight bf16 as floats.
__device__ __forceinline__ void widen(uint4 x, float (&f)[8]) {
    f[0] = pa_dev::bf16_lo(x.x); f[1] = pa_dev::bf16_hi(x.x);
    f[2] = pa_dev::bf16_lo(x.y); f[3] = pa_dev::bf16_hi(x.y);
    f[4] = pa_dev::bf16_lo(x.z); f[5] = pa_dev::bf16_hi(x.z);
    f[6] = pa_dev::bf16_lo(x.w); f[7] = pa_dev::bf16_hi(x.w);
}

// What a lane needs of a token's angles to rotate elements 8c .. 8c + 7 of its
// rows: eight cosines and sines (four of each when the pairs are neighbours).
struct Angles { float co[8], si[8]; };
__device__ __forceinline__ void load_angles(Angles& a, const float* cs, int half, bool interleaved, int lane) {
    const int c = lane & 15, hc = half / 8;                          // hc: chunks of half the rotated part
    const int f0 = interleaved ? 4 * c : 8 * (c < hc ? c : c - hc);
    if (interleaved ? 8 * c < 2 * half : c < 2 * hc) {
        const float4* co = reinterpret_cast<const float4*>(cs + f0);
        const float4* si = reinterpret_cast<const float4*>(cs + kD / 2 + f0);
        *reinterpret_cast<float4*>(a.co) = co[0];
        *reinterpret_cast<float4*>(a.si) = si[0];
        if (!interleaved) {
            *reinterpret_cast<float4*>(a.co + 4) = co[1];
            *reinterpret_cast<float4*>(a.si + 4) = si[1];
        }
    }
}

// Rotate this lane's elements of a row held by 16 lanes.  rotary_dim is a multiple
// of 16 (of 8 when interleaved).
__device__ __forceinline__ void rotate8(uint4 x, float (&y)[8], const Angles& a, int half, bool interleaved, int lane) {
    const int c = lane & 15;
    widen(x, y);
    if (half == 0) return;
    if (interleaved) {
        if (8 * c < 2 * half) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float co = a.co[i / 2], si = a.si[i / 2], u = y[i], v = y[i + 1];
                y[i] = u * co - v * si;
                y[i + 1] = u * si + v * co;
            }
        }
        return;
    }
    const int hc = half / 8;
    const int pc = c < hc ? c + hc : c < 2 * hc ? c - hc : c;
    uint4 z;
    const int src = (lane & 16) | pc;
    z.x = __shfl_sync(0xffffffffu, x.x, src);
    z.y = __shfl_sync(0xffffffffu, x.y, src);
    z.z = __shfl_sync(0xffffffffu, x.z, src);
    z.w = __shfl_sync(0xffffffffu, x.w, src);
    if (c < 2 * hc) {
        float o[8];
        widen(z, o);
        const float sign = c < hc ? -1.f : 1.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = y[i] * a.co[i] + sign * o[i] * a.si[i];
    }
}

// The pairs' frequencies in turns per position, as fractions of 2^64, and their axes.
struct Table {
    unsigned long long freq[kD / 2];
    float bad[kD / 2];                                               // 0, or NaN for a frequency that is not finite
    int axis[kD / 2];                                                // -1: unknown, not rotated
    __device__ __forceinline__ void fill(const RopeParams& r, int f, int* err) {
        const float x = __ldg(r.inv_freq + f);
        double turns = static_cast<double>(x) * 0.15915494309189533577;
        turns -= floor(turns);                                       // [0, 1]; whole turns do not count
        freq[f] = __double2ull_rn(turns * 4294967296.0 * 2147483648.0) << 1;          // (2^63 at most, then 0)
        bad[f] = x * 0.f;
        const int ax = r.axis ? __ldg(r.axis + f) : 0;
        const bool known = ax >= 0 && ax < r.num_axes;
        if (!known) pa_dev::record_error(err, PA_ERR_INVALID_ARG);
        axis[f] = known ? ax : -1;
    }
    // pair f of a token: cosine to cs[f], sine to cs[kD / 2 + f]
    __device__ __forceinline__ void angle(const RopeParams& r, int T, float* cs, int token, int f) const {
        float si = 0.f, co = 1.f;
        if (axis[f] >= 0) {
            const long long pos = __ldg(r.positions + static_cast<int64_t>(axis[f]) * T + token);
            const unsigned long long frac = static_cast<unsigned long long>(pos) * freq[f];
            // quarter turns, and the rest, at most half of one: its float has 2^-27 of a half-turn
            const int quarter = static_cast<int>((frac + (1ull << 61)) >> 62);
            const long long rest = static_cast<long long>(frac - (static_cast<unsigned long long>(quarter) << 62));
            const float2 cs2 = pa_rope::turned(static_cast<float>(static_cast<int>(rest >> 30)) * (1.f / 8589934592.f), quarter);
            co = cs2.x;
            si = cs2.y;
            si += bad[f];
            co += bad[f];
        }
        cs[f] = co;
        cs[kD / 2 + f] = si;
    }
};

// Query rows `sub`, `sub` + `subs`, ... (in pairs) of a token, by one warp: two rows at
// a time, four such pairs in flight.
__device__ __forceinline__ void rotate_queries(const RopeParams& r, int t, const float* cs, int sub, int subs, int lane) {
    const int hi = lane >> 4, c8 = 8 * (lane & 15);
    const uint16_t* src = static_cast<const uint16_t*>(r.q) + static_cast<int64_t>(t) * r.q_stride + c8;
    uint16_t* dst = static_cast<uint16_t*>(r.q_out) + static_cast<int64_t>(t) * r.Hq * kD + c8;
    Angles a;
    load_angles(a, cs, r.half, r.interleaved, lane);
    for (int h0 = 2 * sub; h0 < r.Hq; h0 += 8 * subs) {
        uint4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int h = h0 + 2 * k * subs + hi;
            x[k] = h < r.Hq ? __ldg(reinterpret_cast<const uint4*>(src + h * kD)) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int h = h0 + 2 * k * subs + hi;
            float y[8];
            rotate8(x[k], y, a, r.half, r.interleaved, lane);
            if (h < r.Hq)
                *reinterpret_cast<uint4*>(dst + h * kD) =
                    make_uint4(pa_dev::pack_bf16(y[0], y[1]), pa_dev::pack_bf16(y[2], y[3]),
                               pa_dev::pack_bf16(y[4], y[5]), pa_dev::pack_bf16(y[6], y[7]));
        }
    }
}

// The queries of many tokens, a warp each: apart from the tiles, whose registers
// would leave too few warps to keep these copies going.
__global__ void __launch_bounds__(kThreads, 4) rotate_queries_kernel(const RopeParams r, int T, int* err) {
    __shared__ Table table;
    __shared__ __align__(16) float s_cs[kWarps][kD];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = blockIdx.x * kWarps + warp;
    pa_dev::wait_prior_grid();
    pa_dev::allow_next_grid();
    if (static_cast<int>(threadIdx.x) < r.half) table.fill(r, threadIdx.x, err);
    __syncthreads();
    if (t >= T) return;
    for (int f = lane; f < r.half; f += 32) table.angle(r, T, s_cs[warp], t, f);
    __syncwarp();
    rotate_queries(r, t, s_cs[warp], 0, 1, lane);
}

struct TileParams {
    uint8_t* kpool;
    uint8_t* vpool;
    uint8_t* scales;
    const void* k;
    const void* v;
    const int64_t* slots;
    unsigned long long* mask;       // notes of the kernel in front, null: look yourself
    const int32_t* token;
    int* err;
    int64_t num_slots;
    int T, Hkv;
    float k_scale, v_scale;
};

// A CTA takes `per` tokens of the list: one while it searches the slots itself, else
// 16, of which about one leads a block; gridDim.y CTAs share their rows and tiles.  (A CTA per token, 15 of 16 with nothing to store, spent 34 us on a
// prefill step's 5378 tokens, most of it starting CTAs.)
template <int KIND, bool ROPE>
__global__ void __launch_bounds__(kThreads, ROPE ? 2 : 3) append_tile_kernel(const TileParams p, const RopeParams r, int per) {
    __shared__ __align__(16) float s_cs[kB][kD];                                   // of a block's new tokens: cosines, sines
    __shared__ __align__(16) float s_own[kD];                        // of this CTA's token (queries)
    __shared__ Table table;
    __shared__ int s_tok[kB];
    __shared__ unsigned s_m[kB];                                     // offsets of the block that token i leads, or 0
    const int t0 = blockIdx.x * per, cnt = min(per, p.T - t0), tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int half = ROPE ? r.half : 0;
    if (tid < kB) {
        s_m[tid] = 0;
        s_tok[tid] = -1;
    }
    pa_dev::wait_prior_grid();
    pa_dev::allow_next_grid();
    auto block_of = [&](int t) {                                     // -1: nothing to store
        const int64_t slot = p.slots[t];
        return slot >= 0 && slot < p.num_slots ? slot / kB : int64_t{-1};
    };
    if (ROPE && tid < half) table.fill(r, tid, p.err);
    __syncthreads();
    if (p.mask) {
        if (tid < cnt) {
            const int64_t b = block_of(t0 + tid);
            if (b >= 0) {
                // leaders alone clear their block's note, so any other CTA sees it whole or zero
                const unsigned m = static_cast<unsigned>(*reinterpret_cast<volatile unsigned long long*>(p.mask + b));
                const int off = static_cast<int>(p.slots[t0 + tid] - b * kB);
                if (m && __ffs(m) - 1 == off && p.token[b * kB + off] == t0 + tid) s_m[tid] = m;
            }
        }
    } else {
        const int64_t b = block_of(t0);
        if (p.slots[t0] >= p.num_slots && tid == 0 && blockIdx.y == 0) pa_dev::record_error(p.err, PA_ERR_BAD_SLOT);
        if (b >= 0) {
            for (int i = tid; i < p.T; i += kThreads) {
                const int64_t x = p.slots[i];
                if (x >= 0 && x / kB == b) {
                    atomicOr(&s_m[0], 1u << (x % kB));
                    atomicMax(&s_tok[x % kB], i);                    // one slot twice: the later token, for every CTA
                }
            }
            __syncthreads();
            const int off = static_cast<int>(p.slots[t0] - b * kB);
            const bool leads = __ffs(s_m[0]) - 1 == off && s_tok[off] == t0;
            __syncthreads();
            if (!leads && tid == 0) s_m[0] = 0;
        }
    }
    if (ROPE && r.q) {                                               // (then cnt is 1)
        if (tid < half) table.angle(r, p.T, s_own, t0, tid);
        __syncthreads();
        rotate_queries(r, t0, s_own, blockIdx.y * kWarps + warp, kWarps * gridDim.y, lane);
    }
    __syncthreads();
    for (int lead = 0; lead < cnt; ++lead) {
    const unsigned m = s_m[lead];
    if (m == 0) continue;                                            // uniform
    const int64_t blk = block_of(t0 + lead);
    if (p.mask) {
        if (tid < kB) s_tok[tid] = p.token[blk * kB + tid];
        __syncthreads();
    }
    if constexpr (ROPE) {
        for (int i = tid; i < kB * half; i += kThreads)
            if ((m >> (i / half)) & 1) table.angle(r, p.T, s_cs[i / half], s_tok[i / half], i % half);
        __syncthreads();
    }
    const bool fresh = m & 1, whole = m == 0xffffu;
    const int hi = lane >> 4, c = lane & 15;
    // keys and values in turn for each warp: rotated keys take longer
    for (int w = blockIdx.y * kWarps + warp, turn = 0; w < 2 * p.Hkv; w += kWarps * gridDim.y, turn ^= 1) {
        const int h = w >> 1, is_v = (w ^ turn) & 1;
        const uint16_t* src = static_cast<const uint16_t*>(is_v ? p.v : p.k) + h * kD + 8 * c;
        const int64_t stride = is_v ? r.v_stride : r.k_stride;
        const int64_t tile = (blk * p.Hkv + h) * kTile;
        // row 2i + hi of the block, elements 8c .. 8c + 7
        uint4 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int o = 2 * i + hi;
            x[i] = (m >> o) & 1 ? __ldg(reinterpret_cast<const uint4*>(src + static_cast<int64_t>(s_tok[o]) * stride))
                                : make_uint4(0u, 0u, 0u, 0u);
        }
        if constexpr (KIND == kBf16) {
            if (!is_v) {
                uint16_t* dst = reinterpret_cast<uint16_t*>(p.kpool) + tile + 8 * c;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int o = 2 * i + hi;
                    float y[8];
                    Angles a;
                    load_angles(a, s_cs[o], half, r.interleaved, lane);
                    rotate8(x[i], y, a, half, r.interleaved, lane);
                    if ((m >> o) & 1)
                        *reinterpret_cast<uint4*>(dst + o * kD) =
                            make_uint4(pa_dev::pack_bf16(y[0], y[1]), pa_dev::pack_bf16(y[2], y[3]),
                                       pa_dev::pack_bf16(y[4], y[5]), pa_dev::pack_bf16(y[6], y[7]));
                }
            } else {
                // this lane's four columns d of all 16 tokens: the two half-warps trade
                uint16_t* dst = reinterpret_cast<uint16_t*>(p.vpool) + tile + (8 * c + 4 * hi) * kB;
                uint32_t a[16][2];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t r0 = __shfl_xor_sync(0xffffffffu, hi ? x[i].x : x[i].z, 16);
                    const uint32_t r1 = __shfl_xor_sync(0xffffffffu, hi ? x[i].y : x[i].w, 16);
                    const uint32_t o0 = hi ? x[i].z : x[i].x, o1 = hi ? x[i].w : x[i].y;
                    a[2 * i][0] = hi ? r0 : o0;
                    a[2 * i][1] = hi ? r1 : o1;
                    a[2 * i + 1][0] = hi ? o0 : r0;
                    a[2 * i + 1][1] = hi ? o1 : r1;
                }
                if (whole) {
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        uint32_t y[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            y[j] = __byte_perm(a[2 * j][d >> 1], a[2 * j + 1][d >> 1], d & 1 ? 0x7632 : 0x5410);
                        uint4* q = reinterpret_cast<uint4*>(dst + d * kB);
                        q[0] = make_uint4(y[0], y[1], y[2], y[3]);
                        q[1] = make_uint4(y[4], y[5], y[6], y[7]);
                    }
                } else {
#pragma unroll
                    for (int o = 0; o < 16; ++o)
                        if ((m >> o) & 1)
#pragma unroll
                            for (int d = 0; d < 4; ++d)
                                dst[d * kB + o] = static_cast<uint16_t>(a[o][d >> 1] >> (16 * (d & 1)));
                }
            }
        } else {
            uint8_t* const pool = (is_v ? p.vpool : p.kpool) + tile;
            // what stays of a partly written block (8 codes of each of this lane's K rows,
            // 16 of each of its V columns), and its scale, while the rows are on their way
            const bool keeps = KIND == kScaled && !fresh && !whole;
            int b_old = 0;
            uint4 old[4];
            const int64_t si = (blk * p.Hkv + h) * 2 + is_v;
            if (keeps) {
                b_old = p.scales[si];
                if (is_v) {
#pragma unroll
                    for (int d = 0; d < 4; ++d) old[d] = reinterpret_cast<const uint4*>(pool)[8 * c + 4 * hi + d];
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint2 y = reinterpret_cast<const uint2*>(pool)[(2 * i + hi) * 16 + c];
                        if (i & 1) { old[i / 2].z = y.x; old[i / 2].w = y.y; }
                        else { old[i / 2].x = y.x; old[i / 2].y = y.y; }
                    }
                }
            }
            // rotated rows are kept as floats (64 a lane, two CTAs an SM); of rows as they came
            // the maximum is taken of the bf16 bits (three CTAs)
            float y[ROPE ? 8 : 1][8];
            float amax = 0.f;
            if constexpr (ROPE) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    Angles a;
                    if (!is_v) load_angles(a, s_cs[2 * i + hi], half, r.interleaved, lane);
                    rotate8(x[i], y[i], a, is_v ? 0 : half, r.interleaved, lane);
                    if (KIND == kScaled)
#pragma unroll
                        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(y[i][e]));
                }
                if (KIND == kScaled && amax == INFINITY) {           // finite values only (a NaN is not a maximum)
                    amax = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(y[i][e]) < INFINITY ? fabsf(y[i][e]) : 0.f);
                }
            } else {
                // magnitudes of two bf16 at a time, as integers
                auto top = [&](uint32_t w, uint32_t mx) { return __vmaxu2(mx, w & 0x7fff7fffu); };
                uint32_t mx = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) mx = top(x[i].w, top(x[i].z, top(x[i].y, top(x[i].x, mx))));
                mx = max(mx & 0xffffu, mx >> 16);
                if (mx >= 0x7f80u) {                                 // finite values only
                    auto fin = [](uint32_t w, uint32_t m) {
                        const uint32_t a = w & 0x7fffu, b = (w >> 16) & 0x7fffu;
                        return max(m, max(a < 0x7f80u ? a : 0u, b < 0x7f80u ? b : 0u));
                    };
                    mx = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) mx = fin(x[i].w, fin(x[i].z, fin(x[i].y, fin(x[i].x, mx))));
                }
                amax = __uint_as_float(mx << 16);
            }
            float inv = 1.f, shrink = 1.f;
            bool rises = false;
            if constexpr (KIND == kScaled) {
                asm volatile("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(amax));
                const int b = max(b_old, scale_exponent(amax));
                inv = pa_dev::inverse_scale(b);
                rises = b != b_old;
                shrink = b_old > 0 ? pow2(max(0, b_old - b + 127)) : 0.f;
                if (lane == 0) p.scales[si] = static_cast<uint8_t>(b);
            }
            const float div = is_v ? p.v_scale : p.k_scale;
            uint2 cw[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float (&z)[8] = y[ROPE ? i : 0];
                if (!ROPE) widen(x[i], z);
#pragma unroll
                for (int e = 0; e < 8; ++e) z[e] = KIND == kScaled ? z[e] * inv : __fdiv_rn(z[e], div);
                cw[i] = make_uint2(codes4(z[0], z[1], z[2], z[3]), codes4(z[4], z[5], z[6], z[7]));
            }
            if (!is_v) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int o = 2 * i + hi;
                    const bool is_new = (m >> o) & 1;
                    uint2 z = cw[i];
                    if (KIND == kScaled && !is_new) {                // stays: zero, or re-rounded
                        z = make_uint2(0u, 0u);
                        if (keeps && b_old > 0) {
                            const uint4 q = old[i / 2];
                            z = i & 1 ? make_uint2(q.z, q.w) : make_uint2(q.x, q.y);
                            if (rises) z = make_uint2(shrink4(z.x, shrink), shrink4(z.y, shrink));
                        }
                    }
                    if (is_new || (KIND == kScaled && (fresh || rises)))
                        reinterpret_cast<uint2*>(pool)[o * 16 + c] = z;
                }
            } else {
                uint32_t a[16];                                      // four codes (columns) of each token
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, hi ? cw[i].x : cw[i].y, 16);
                    const uint32_t own = hi ? cw[i].y : cw[i].x;
                    a[2 * i] = hi ? got : own;
                    a[2 * i + 1] = hi ? own : got;
                }
                if (KIND == kScaled || whole) {
                    uint32_t z[4][4];                                // [column][four tokens]: 4 x 4 byte transposes
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t t0 = __byte_perm(a[4 * q], a[4 * q + 1], 0x5140), t1 = __byte_perm(a[4 * q + 2], a[4 * q + 3], 0x5140);
                        const uint32_t t2 = __byte_perm(a[4 * q], a[4 * q + 1], 0x7362), t3 = __byte_perm(a[4 * q + 2], a[4 * q + 3], 0x7362);
                        z[0][q] = __byte_perm(t0, t1, 0x5410);
                        z[1][q] = __byte_perm(t0, t1, 0x7632);
                        z[2][q] = __byte_perm(t2, t3, 0x5410);
                        z[3][q] = __byte_perm(t2, t3, 0x7632);
                    }
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        if (KIND == kScaled && !whole) {
                            uint32_t w4[4] = {0u, 0u, 0u, 0u};
                            if (keeps && b_old > 0) {
                                w4[0] = old[d].x; w4[1] = old[d].y; w4[2] = old[d].z; w4[3] = old[d].w;
                                if (rises)
#pragma unroll
                                    for (int q = 0; q < 4; ++q) w4[q] = shrink4(w4[q], shrink);
                            }
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const uint32_t mk = byte_mask(m >> (4 * q));
                                z[d][q] = (z[d][q] & mk) | (w4[q] & ~mk);
                            }
                        }
                        reinterpret_cast<uint4*>(pool)[8 * c + 4 * hi + d] = make_uint4(z[d][0], z[d][1], z[d][2], z[d][3]);
                    }
                } else {
#pragma unroll
                    for (int o = 0; o < 16; ++o)
                        if ((m >> o) & 1)
#pragma unroll
                            for (int d = 0; d < 4; ++d) pool[(8 * c + 4 * hi + d) * kB + o] = static_cast<uint8_t>(a[o] >> (8 * d));
                }
            }
        }
    }
    __syncthreads();
    if (p.mask && tid == 0) {
        // the last of the block's CTAs (marked in the note's upper half) clears it
        const unsigned long long me = 1ull << (32 + blockIdx.y), all = ((1ull << gridDim.y) - 1) << 32;
        if (((atomicOr(p.mask + blk, me) | me) & all) == all) p.mask[blk] = 0;
    }
    }
}

// One warp per (per_warp <= 16 list entries, KV head).  Keys: a row per entry.  Values: the
// entries' blocks are walked in runs; a run's tile comes in once (64 codes, or 64
// bf16, a lane: four columns of 16 tokens) and each entry takes its token.
template <int KIND>
__global__ void __launch_bounds__(256) read_tile_kernel(const uint8_t* __restrict__ kpool, const uint8_t* __restrict__ vpool,
                                                        const uint8_t* __restrict__ scales,
                                                        const int64_t* __restrict__ slots, uint16_t* __restrict__ k,
                                                        uint16_t* __restrict__ v, int T, int Hkv, int64_t num_slots,
                                                        float k_scale, float v_scale, int per_warp, int* err) {
    pa_dev::wait_prior_grid();
    pa_dev::allow_next_grid();
    const int64_t wi = (blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    const int64_t grp = wi / Hkv;
    const int h = static_cast<int>(wi - grp * Hkv);
    if (grp * per_warp >= T) return;
    const int e0 = static_cast<int>(grp * per_warp), cnt = min(per_warp, T - e0);
    int64_t slot = -1;
    if (lane < cnt) {
        slot = slots[e0 + lane];
        if (slot >= num_slots) {
            if (h == 0) pa_dev::record_error(err, PA_ERR_BAD_SLOT);
            slot = -1;
        }
    }
    const int blk = slot < 0 ? -1 : static_cast<int>(slot / kB), off = static_cast<int>(slot & (kB - 1));
    auto put = [&](uint16_t* out, int e, uint32_t lo, uint32_t hi) { // columns 4 lane .. 4 lane + 3 of entry e
        *reinterpret_cast<uint2*>(out + ((e0 + e) * static_cast<int64_t>(Hkv) + h) * kD + 4 * lane) = make_uint2(lo, hi);
    };
    auto values4 = [](uint32_t c, float s, uint32_t& lo, uint32_t& hi) {
        const uint32_t a = pa_dev::e4m3x2_to_f16x2(c & 0xffffu), b = pa_dev::e4m3x2_to_f16x2(c >> 16);
        lo = pa_dev::pack_bf16(pa_dev::f16_lo(a) * s, pa_dev::f16_hi(a) * s);
        hi = pa_dev::pack_bf16(pa_dev::f16_lo(b) * s, pa_dev::f16_hi(b) * s);
    };
    uint32_t left = (1u << cnt) - 1u;                                // entries still to serve (uniform)
    const uint32_t none = __ballot_sync(0xffffffffu, blk < 0) & left;
    for (uint32_t z = none; z; z &= z - 1) {
        put(k, __ffs(z) - 1, 0u, 0u);
        put(v, __ffs(z) - 1, 0u, 0u);
    }
    left &= ~none;
    while (left) {
        const int b = __shfl_sync(0xffffffffu, blk, __ffs(left) - 1);
        const uint32_t run = __ballot_sync(0xffffffffu, blk == b) & left;
        left &= ~run;
        const int64_t tile = (static_cast<int64_t>(b) * Hkv + h) * kTile;
        float ks = k_scale, vs = v_scale;
        if (KIND == kScaled) {
            const uint32_t e = *reinterpret_cast<const uint16_t*>(scales + (static_cast<int64_t>(b) * Hkv + h) * 2);
            ks = pow2(e & 0xff);
            vs = pow2(e >> 8);
        }
        // the run's tokens; their key rows and the value tile are loaded at once
        const uint32_t tokens = __reduce_or_sync(0xffffffffu, (run >> lane) & 1 ? 1u << off : 0u);
        uint2 tk[kB];                                                // (codes: .x alone)
        uint4 tv[KIND == kBf16 ? 8 : 4];
        if constexpr (KIND == kBf16) {
#pragma unroll
            for (int i = 0; i < 8; ++i) tv[i] = __ldg(reinterpret_cast<const uint4*>(vpool + tile * 2) + 8 * lane + i);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) tv[i] = __ldg(reinterpret_cast<const uint4*>(vpool + tile) + 4 * lane + i);
        }
#pragma unroll
        for (int o = 0; o < kB; ++o)
            if ((tokens >> o) & 1) {
                if constexpr (KIND == kBf16) tk[o] = __ldg(reinterpret_cast<const uint2*>(kpool + (tile + o * kD) * 2) + lane);
                else tk[o].x = __ldg(reinterpret_cast<const uint32_t*>(kpool + tile + o * kD) + lane);
            }
#pragma unroll
        for (int o = 0; o < kB; ++o) {
            // the run's entries of token o (usually one, perhaps several)
            for (uint32_t es = __ballot_sync(0xffffffffu, off == o) & run; es; es &= es - 1) {
                const int e = __ffs(es) - 1;
                uint32_t lo, hi;
                if constexpr (KIND == kBf16) {
                    put(k, e, tk[o].x, tk[o].y);
                    auto pick = [&](int d) {                         // column d's token o
                        const uint4 q = tv[2 * d + (o >> 3)];
                        const int j = (o & 7) >> 1;
                        const uint32_t wd = j == 0 ? q.x : j == 1 ? q.y : j == 2 ? q.z : q.w;
                        return (wd >> (16 * (o & 1))) & 0xffffu;
                    };
                    lo = pick(0) | pick(1) << 16;
                    hi = pick(2) | pick(3) << 16;
                } else {
                    values4(tk[o].x, ks, lo, hi);
                    put(k, e, lo, hi);
                    auto pick = [&](int d) {
                        const uint4 q = tv[d];
                        const uint32_t wd = o < 4 ? q.x : o < 8 ? q.y : o < 12 ? q.z : q.w;
                        return (wd >> (8 * (o & 3))) & 0xffu;
                    };
                    values4(pick(0) | pick(1) << 8 | pick(2) << 16 | pick(3) << 24, vs, lo, hi);
                }
                put(v, e, lo, hi);
            }
        }
    }
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

namespace pa_detail {

bool append_tile_eligible(const pa_pool* p, const void* k, const void* v, const RopeParams& r) {
    const bool rotary = r.half == 0 || (r.interleaved ? r.half % 4 == 0 : r.half % 8 == 0);
    return p->head_dim == kD && p->block_size == kB && p->dtype != PA_F32 && rotary && aligned16(k) && aligned16(v) &&
           r.k_stride % 8 == 0 && r.v_stride % 8 == 0 &&
           (!r.q || (aligned16(r.q) && aligned16(r.q_out) && r.q_stride % 8 == 0));
}

// False without memory for it; the plain kernels need none.  A first call inside a capture
// makes it too: allocated and cleared beside the capture, on a stream of its own, which a
// thread in relaxed mode may do.
bool append_notes_ready(pa_pool* p, int T) {
    if (T <= kDirect || p->app_mask) return true;
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return false;
    const size_t nb = static_cast<size_t>(p->num_blocks);
    void *mask = nullptr, *token = nullptr;
    cudaStream_t own = nullptr;
    const bool ok = cudaMalloc(&mask, nb * sizeof(unsigned long long)) == cudaSuccess &&
                    cudaMalloc(&token, nb * kB * sizeof(int32_t)) == cudaSuccess &&
                    cudaStreamCreateWithFlags(&own, cudaStreamNonBlocking) == cudaSuccess &&
                    cudaMemsetAsync(mask, 0, nb * sizeof(unsigned long long), own) == cudaSuccess &&
                    cudaStreamSynchronize(own) == cudaSuccess;
    if (own) cudaStreamDestroy(own);
    if (!ok) {
        cudaGetLastError();
        cudaFree(mask);
        cudaFree(token);
    } else {
        p->app_mask = static_cast<unsigned long long*>(mask);
        p->app_token = static_cast<int32_t*>(token);
    }
    cudaThreadExchangeStreamCaptureMode(&mode);
    return ok;
}

int launch_append_tile(pa_pool* p, const void* k, const void* v, const int64_t* slots, int T, const RopeParams& rope,
                       cudaStream_t st) {
    RopeParams r = rope;
    TileParams t{};
    t.kpool = static_cast<uint8_t*>(p->k);
    t.vpool = static_cast<uint8_t*>(p->v);
    t.scales = p->scales;
    t.k = k;
    t.v = v;
    t.slots = slots;
    t.err = p->err;
    t.num_slots = static_cast<int64_t>(p->num_blocks) * kB;
    t.T = T;
    t.Hkv = p->kv_heads;
    t.k_scale = p->k_scale;
    t.v_scale = p->v_scale;
    if (T > kDirect) {
        const int rc = launch_append_notes(p, slots, T, st);
        if (rc != PA_OK) return rc;
        t.mask = p->app_mask;
        t.token = p->app_token;
        if (r.q) {
            const cudaError_t e = launch_pdl(rotate_queries_kernel, dim3((T + kWarps - 1) / kWarps), dim3(kThreads), 0, st, r, T, p->err);
            count_launch();
            if (e != cudaSuccess) return PA_ERR_CUDA;
            r.q = nullptr;
        }
    }
    // few tokens: a warp per (KV head, keys or values).  Many, rotated: two per warp, which
    // forms a block's angles half as often (9896 tokens: 619 CTAs, two waves of the 304 that
    // fit and eleven CTAs more; 5378 without rotation: 674, one and a half waves of 456).  A
    // note's upper half has room for 32 CTAs
    const int per = T > kDirect ? kB : 1, items = T > kDirect && rope.half > 0 ? 2 : 1;
    const dim3 grid((T + per - 1) / per, std::min(32, (2 * p->kv_heads + kWarps * items - 1) / (kWarps * items)));
    // (bf16 pools and pools with one scale come here for pa_append_rope alone)
    auto kernel = p->dtype == PA_BF16 ? append_tile_kernel<kBf16, true>
                : p->dtype == PA_FP8E4M3 ? append_tile_kernel<kFp8, true>
                : rope.half > 0 ? append_tile_kernel<kScaled, true> : append_tile_kernel<kScaled, false>;
    const cudaError_t e = launch_pdl(kernel, grid, dim3(kThreads), 0, st, t, r, per);
    count_launch();
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

bool read_tile_eligible(const pa_pool* p, const void* k, const void* v) {
    return p->head_dim == kD && p->block_size == kB && p->dtype != PA_F32 && aligned16(k) && aligned16(v);
}

int launch_read_tile(pa_pool* p, const int64_t* slots, int n, void* k, void* v, cudaStream_t st) {
    // 16 entries a warp read a block's value tile once for all its tokens; few entries
    // are a warp each, for latency (64 entries in 64 blocks: a warp that took 16 of
    // them waited 16 times, 16 us in all)
    const int per_warp = n > 1024 ? 16 : 1;
    const int64_t warps = (static_cast<int64_t>(n) + per_warp - 1) / per_warp * p->kv_heads;
    auto kernel = p->dtype == PA_BF16 ? read_tile_kernel<kBf16>
                : p->dtype == PA_FP8E4M3 ? read_tile_kernel<kFp8> : read_tile_kernel<kScaled>;
    const cudaError_t e = launch_pdl(kernel, dim3(static_cast<unsigned>((warps + 7) / 8)), dim3(256), 0, st,
                                     static_cast<const uint8_t*>(p->k), static_cast<const uint8_t*>(p->v),
                                     static_cast<const uint8_t*>(p->scales), slots, static_cast<uint16_t*>(k),
                                     static_cast<uint16_t*>(v), n, p->kv_heads,
                                     static_cast<int64_t>(p->num_blocks) * kB, p->k_scale, p->v_scale, per_warp, p->err);
    count_launch();
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa_detail
