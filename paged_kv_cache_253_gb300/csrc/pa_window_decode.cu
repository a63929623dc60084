// Windowed and block-scaled decode attention on the 5th-generation tensor
// cores: 16-token blocks, head width 128, at most 16 query heads per KV head;
// bf16 pools and e4m3-code pools.
//
// Bound: the visible keys' and values' bytes.  Decode has few query rows, so
// keys and values are the M side of the MMAs and the queries the N side:
//   S^T[128 tokens x N] = K[128 x 128] . Q^T        thread t = token t = TMEM lane t
//   O^T[128 dims x N]  += V^T[128 x 128] . P^T
// and nothing is done to a key or value after its copy into shared memory.
// Code pools feed the e4m3 codes to the tensor cores as they are
// (kind::f8f6f4), which wants 8 bits on the N side too: a query is the sum of
// three e4m3 parts, each the remainder of the last one times 16.  The parts are
// extra columns, which are free: the MMAs' time goes by the M side's reads of
// shared memory.  Error of n parts: 2^-4n of the number, or 2^(-6-4n) of the unit;
// queries are first scaled by a power of two that puts the row's largest
// element into [2^7, 2^8).
// Weights span more binary orders than a query's elements: many small ones
// together may count as much as the largest, or be all of the result where the
// largest one's value is zero, so the smallest part's last place matters, not
// only the largest weight's error.  For a bf16 result they are four e5m2 parts,
// each the remainder of the last one times 8 (error 2^-12 of the weight, or 2^-26
// of the unit), with the largest at 2^12 .. 2^15: what is cut off is under 2^-38
// of the largest weight per key.  (Three e4m3 parts with the largest at 2^4 ..
// 2^8, 2^-22, lost half of 131072 weights of e^-15.5.)  For fp32 they are five e4m3
// parts (2^-20 of the weight, or 2^-26 of the unit), the largest at 2^6 .. 2^8.5:
// 2^-32 of the largest per key.  (2^7 .. 2^8.5 raises references more often: 256
// sequences on a window, 147 -> 156 us.)  bf16 pools take the weights as two or three
// bf16 parts, which have a float's range.
//
// A block's key scale multiplies its tokens' scores.  Its value scale goes into
// the weights, w = 2^(x + log2 ev - r_o), with a reference r_o of their own (a
// running maximum of x + log2 ev): one that is far below another's drops out of
// the value sums as it should, and the normaliser's l = sum 2^(x - r) is not
// touched by it.
//
// Work is split evenly: all (sequence, KV head, 128-token step)s in one list,
// cut into one contiguous range per weight group, two groups per CTA.  A range
// begins and ends inside items; those write partials, and the group that
// finishes an item last (a counter per item) merges them in a fixed order, so
// nothing waits and results do not depend on timing.
//
// Warps: 0-3 and 4-7 weights of group 0 and 1, 8 copies of keys (TMA), 9 and 10
// MMA issue of each group, 11 copies of values, and queries.  A group's step is a chain of waits (scores,
// one vote on the references, the value product before) of about 1000 cycles;
// two groups that share nothing but the copies' ring cover it (one group: 90 against 73 us, 64 sequences).  Every mbarrier
// wait is bounded (see pa_window_tc.cu).
//
// Measured (32 query, 8 KV heads): 8 sequences of 32768 .. 131072 tokens,
// block-scaled, 195 us, 6.0 TB/s; 64 of 128 .. 2048, 47 us, 3.0 TB/s; 64 on a window of
// 1024, bf16, 55 us, 4.9 TB/s; 256 on a window of 512, 64 query heads, fp32 out, 143 us,
// 2.0 TB/s.  Long ranges run at the memory's rate; where items are a few steps long
// the weights' chain of waits (about 4500 cycles a step, two under way) and the ends of
// items set the pace.  Three groups, a warp that plans the copies for the others and
// two buffers for the weights of a step were each no faster: the first for want of
// registers, the others because the chain stayed.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include <cuda.h>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_tc.cuh"

namespace {

constexpr int kD = 128;
constexpr int kStep = 128;                   // tokens per step (M)
constexpr int kBlk = 16;
constexpr int kStepBlks = kStep / kBlk;
constexpr int kThreads = 384;
constexpr int kMaxG = 16;
constexpr uint32_t kWaitLimit = 1u << 20;

// Barriers; of two kinds per group or per (group, parity), and per ring slot.
enum Bar { kQFull0, kQEmpty0 = kQFull0 + 4, kSFull0 = kQEmpty0 + 4, kSEmpty0 = kSFull0 + 4, kPFull0 = kSEmpty0 + 4,
           kPEmpty0 = kPFull0 + 2, kOFull0 = kPEmpty0 + 2, kOEmpty0 = kOFull0 + 4, kDone0 = kOEmpty0 + 4,
           kKEmpty0 = kDone0 + 2, kVEmpty0 = kKEmpty0 + 6, kKFull0 = kVEmpty0 + 6, kVFull0 = kKFull0 + 12,
           kNumBars = kVFull0 + 12 };
// A ring slot has a "full" barrier for each group (kKFull0 + 6 grp + slot): a parity
// wait tells only a phase from its neighbours, so whoever waits must have seen every
// phase before.  Slots pass between the groups and copies may land out of order; with
// one barrier for both, a group could ask for its own copy while the other's, in the
// phase before, is still under way, and be told that it has landed.

constexpr int kSlot = kMaxG * (kD + 4);       // floats of a partial: sums, then (reference, sum of weights, weights' reference)
constexpr int kChunk = 64;                   // steps of a chunk (see Cfg)
constexpr int kInfo = 16;                    // steps whose description is kept

// The small things behind the operands.
template <bool CODE, int GM>
struct Misc {
    static constexpr int kMax = CODE ? 2 : 1;
    uint64_t bars[kNumBars];
    alignas(16) float red[2][2][4][kMax][GM];   // [group][step parity][warp][x, x + ev][head]: maxima
    alignas(16) int flags[2][2][4];          // [group][vote parity][warp]: a reference has to rise
    union {
        float lsum[2][2][4][GM];             // [group][item parity][warp][head]: sums of weights
        long long scan[kThreads / 32];       // before the ranges are known
    };
    float ref[2][2][kMax][GM];               // [group][item parity][score, weight][head]: references
    // score factor of each head, a group's item it at it % 4: the weight warps read it
    // before they release a step's scores, and item it + 4 is written after the
    // scores of item it + 2, which take the place of item it's, are complete
    alignas(16) float qscale[CODE ? 2 : 1][CODE ? 4 : 1][CODE ? GM : 4];   // (bf16: the pool's alone)
    // the step in place i, at i % 16: block b's exponents (K in the low byte, V in the
    // next) and which blocks were loaded.  Written for i + 16 when the keys of i + 10
    // are free, that is after the scores of i + 6 were read
    uint16_t exps[CODE ? kInfo : 1][kStepBlks];
    uint8_t have[kInfo];
    long long start_base[2];                 // per group: steps before the range's first sequence
    int start_s[2];
    int merge[2];
    uint32_t tmem;
    int abort_flag;
};

// Everything that follows from the template arguments.  GM: 4, 8 or 16, at
// least the query heads per KV head.  Column part * GM + g of an N side holds
// part `part` of head g.
template <bool CODE, bool WIDE, int GM, bool CHUNKS = false>      // WIDE: fp32 output
struct Cfg {
    static constexpr int kQParts = CODE ? 3 : 1;
    static constexpr int kPParts = CODE ? (WIDE ? 5 : 4) : (WIDE ? 3 : 2);
    // code pools' weights (see above): the factor between two parts; the largest weight
    // is 2^kLift when a reference is set, 2^(kLift + kLag) when it is raised (e5m2 holds
    // up to 2^15.8, e4m3 up to 2^8.8)
    static constexpr bool kE5 = CODE && !WIDE;
    static constexpr float kPart = kE5 ? 8.f : 16.f;
    static constexpr float kLift = !CODE ? 0.f : WIDE ? 6.f : 12.f, kLag = !CODE ? 8.f : WIDE ? 2.5f : 3.f;
    // The tensor cores cut a sum to fp32 after each 16 keys (32 of codes), always towards
    // zero: over 30000 bf16 keys that made a result 1e-5 smaller than it is, over 131072 of
    // codes in one range up to 3e-4.  For fp32 results of bf16 pools each step's product
    // starts from zero and the steps are added in registers, rounded to nearest.  For fp32
    // results of code pools, whose products have fewer bits, an item of many steps is walked
    // in chunks of kChunk, which are joined like the parts of an item that several groups
    // share.  That is a kernel of its own: whatever makes the code longer costs the others
    // (8 sequences of 32768 .. 131072, fp32: 213 us without chunks, 225 with; sums in
    // registers or added to memory step by step cost all of them 12 to 38 % from eight
    // heads a group on).
    static constexpr bool kAddSteps = WIDE && !CODE;
    static constexpr int kNQ = (kQParts * GM + 15) / 16 * 16;
    static constexpr int kNP = (kPParts * GM + 15) / 16 * 16;
    static constexpr int kHalf = CODE ? 16384 : 32768;           // bytes of K (and of V) per step
    static constexpr int kStages = CODE ? (GM == 16 ? 5 : 6) : (GM == 16 ? 2 : 3);
    static constexpr int kQBytes = (CODE ? 128 : 256) * ((kNQ + 7) / 8 * 8);
    // P^T without swizzle: token groups of 16 bytes, 16 bytes apart from a multiple of
    // 128, so that a warp's stores fall into different banks (where that fits)
    static constexpr int kLbo = kNP / 8 * 128 + (CODE || kNP < 32 ? 16 : 0);
    static constexpr int kPBytes = kStep * (CODE ? 1 : 2) / 16 * kLbo;
    // TMEM columns: S of (group, step parity), then O of (group, item parity)
    static constexpr int kOCol = 4 * kNQ;
    static constexpr int kTmemCols = kOCol + 4 * kNP <= 256 ? 256 : 512;
    static_assert(kOCol + 4 * kNP <= 512, "TMEM");
    // shared memory: a ring of K and one of V, Q of (group, item parity), P of each
    // group, small things
    static constexpr int kVOff = kStages * kHalf;
    static constexpr int kQOff = kStages * 2 * kHalf;
    static constexpr int kQStride = (kQBytes + 1023) / 1024 * 1024;
    static constexpr int kPOff = kQOff + 4 * kQStride;
    static constexpr int kMisc = kPOff + 2 * kPBytes;
    static constexpr int kSmem = kMisc + static_cast<int>(sizeof(Misc<CODE, GM>)) + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    const uint32_t a = pa_tc::smem_u32(bar);
    uint32_t done = 0;
    for (uint32_t i = 0; i < kWaitLimit; ++i) {
        asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
                     " selp.u32 %0, 1, 0, p;\n}\n" : "=r"(done) : "r"(a), "r"(parity) : "memory");
        if (done || ((i & 31) == 31 && *abort_flag)) break;
    }
    if (__all_sync(0xffffffffu, done)) return true;
    *abort_flag = 1;
    return false;
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(pa_tc::smem_u32(bar)) : "memory");
}
// Barrier of a group's four weight warps.  They take the same barriers in the same
// order whatever happens: after an abort they run on, their waits return at once.
__device__ __forceinline__ void sync_group(int grp) {
    if (grp) asm volatile("bar.sync 2, 128;" ::: "memory");
    else asm volatile("bar.sync 1, 128;" ::: "memory");
}
__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

// K-major operand without swizzle: core matrices of 8 rows x 16 bytes, 128
// contiguous bytes each; lbo: bytes between core matrices along K, sbo: along rows.
__device__ __forceinline__ uint64_t plain_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(lbo >> 4) << 16 |
           static_cast<uint64_t>(sbo >> 4) << 32 | static_cast<uint64_t>(1) << 46;
}
// e4m3 A, e4m3 or e5m2 B (both K-major), fp32 D, M x N.
__host__ __device__ constexpr uint32_t idesc_8bit(int M, int N, bool e5m2_b) {
    return (1u << 4) | (e5m2_b ? 1u << 10 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void mma_8bit(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b),
                 "r"(idesc), "r"(acc ? 1u : 0u) : "memory");
}
// Two fp32 values rounded to e5m2 codes (nearest, ties to even; NaN stays), `lo` in the
// low byte; and such codes as an f16 pair: an e5m2 code is the upper half of an f16.
__device__ __forceinline__ uint32_t e5m2x2_from_f32(float lo, float hi) {
    uint16_t y;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(y) : "f"(hi), "f"(lo));
    return y;
}
__device__ __forceinline__ uint32_t e5m2x2_to_f16x2(uint32_t two_codes) { return __byte_perm(two_codes, 0u, 0x1404); }
// Four consecutive columns of this warp's lanes (the caller waits).
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, float (&v)[4]) {
    uint32_t r[4];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(taddr) : "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const float (&v)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(__float_as_uint(v[0])),
                 "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])) : "memory");
}
// The first four to the end, the others forward.
template <int N>
__device__ __forceinline__ void next_four(float (&v)[N]) {
    if constexpr (N == 4) return;
    const float a[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int i = 0; i + 4 < N; ++i) v[i] = v[i + 4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[N - 4 + i] = a[i];
}

__device__ __forceinline__ float pow2f(int biased) { return __uint_as_float(static_cast<uint32_t>(biased) << 23); }
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 16 ? 0xffffu : n <= 0 ? 0u : (1u << n) - 1u; }
__device__ __forceinline__ uint32_t seen_bits(int p, int j0, int window, int sinks) {
    return low_bits(p + 1 - j0) & (low_bits(sinks - j0) | ~low_bits(p - (window - 1) - j0));
}
__device__ __forceinline__ int seq_len(const WindowParams& p, int s) {
    const int L = __ldg(p.lens + s);
    return L < 0 ? 0 : min(L, p.max_blocks * kBlk);
}

// Blocks of a step that the value product reads, of the `left` blocks that remain:
// it takes 32 tokens of codes at a time, 16 of bf16.
template <bool CODE>
__device__ __forceinline__ int read_blocks(int left) {
    return left >= kStepBlks ? kStepBlks : CODE ? (left + 1) / 2 * 2 : left;
}

// A position in the list of steps: step `tile` of the nt steps of (s, h).
struct Walk {
    int s, h, tile, nt, L, sb, wb, nv;
    __device__ __forceinline__ void load(const WindowParams& p) {      // the lengths of sequence s
        L = seq_len(p, s);
        const int w0 = max(0, L - 1 - (p.window - 1));
        wb = w0 / kBlk;
        sb = (min(p.sinks, w0) + kBlk - 1) / kBlk;
        if (sb >= wb) sb = wb = 0;
        nv = L > 0 ? sb + (L - 1) / kBlk + 1 - wb : 0;
        nt = (nv + kStepBlks - 1) / kStepBlks;
    }
    __device__ __forceinline__ int block(int i) const { return i < sb ? i : i - sb + wb; }
    __device__ __forceinline__ void next(const WindowParams& p) {
        if (++tile < nt) return;
        tile = 0;
        if (++h < p.Hkv) return;
        h = 0;
        do {
            if (++s >= p.S) { nt = 1 << 30; return; }          // behind the last step: nobody looks
            load(p);
        } while (nt == 0);
    }
};

// An item's partials, of ranges c_first .. c_first + parts - 1, by log-sum-exp: 128
// threads, four columns of a head each, one 16-byte load per partial.  (bf16 pools
// write the same reference twice, so the factor between the two is 1.)
template <bool WIDE>
__device__ __forceinline__ void merge_item(const WindowParams& p, long long c_first, int parts, size_t row0, int gt) {
    for (int qd = gt; qd < p.G * (kD / 4); qd += 128) {
        const int g = qd / (kD / 4), d = qd % (kD / 4) * 4;
        auto part = [&](int i) {
            return p.part + (2 * static_cast<size_t>(c_first + i) + (i == 0 ? 1 : 0)) * kSlot;
        };
        float M = -INFINITY, R = -INFINITY, ls = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kBatch = 8;                                  // partials in flight
        for (int i0 = 0; i0 < parts; i0 += kBatch) {
            float4 e[kBatch], y[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (i0 + i < parts) {
                    e[i] = __ldcg(reinterpret_cast<const float4*>(part(i0 + i) + kMaxG * kD + g * 4));
                    y[i] = __ldcg(reinterpret_cast<const float4*>(part(i0 + i) + g * kD + d));
                }
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (i0 + i < parts) {
                    const float nM = fmaxf(M, e[i].x), nR = fmaxf(R, e[i].z);
                    if (nM != -INFINITY) {
                        ls = ls * pa_dev::ex2(M - nM) + e[i].y * pa_dev::ex2(e[i].x - nM);
                        M = nM;
                    } else {
                        ls += e[i].y;                              // 0, or NaN: without a reference
                    }
                    if (nR != -INFINITY) {
                        const float fa = pa_dev::ex2(R - nR), fy = pa_dev::ex2(e[i].z - nR);
                        a.x = a.x * fa + y[i].x * fy;
                        a.y = a.y * fa + y[i].y * fy;
                        a.z = a.z * fa + y[i].z * fy;
                        a.w = a.w * fa + y[i].w * fy;
                        R = nR;
                    } else {
                        a.x += y[i].x;
                        a.y += y[i].y;
                        a.z += y[i].z;
                        a.w += y[i].w;
                    }
                }
        }
        const float f = ls > 0.f && R != -INFINITY ? p.v_scale / ls * pa_dev::ex2(R - M) : 0.f;
        const size_t i = (row0 + g) * kD + d;
        if (WIDE)
            *reinterpret_cast<float4*>(static_cast<float*>(p.out) + i) = make_float4(a.x * f, a.y * f, a.z * f, a.w * f);
        else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + i) =
                make_uint2(pa_dev::pack_bf16(a.x * f, a.y * f), pa_dev::pack_bf16(a.z * f, a.w * f));
    }
}

// A chunk's partial into the sum of those before it, by log-sum-exp: a group's 128 threads,
// thread gt column gt of every head.  (Every partial was written behind a barrier.)
__device__ __noinline__ void add_chunk(float* sum, const float* part, int G, int gt, int grp) {
    auto ex = [](float x, float ref) { return x == -INFINITY ? 1.f : pa_dev::ex2(x - ref); };   // (sums without a reference are 0 or NaN)
    sync_group(grp);
#pragma unroll 1
    for (int g = 0; g < G; ++g) {
        const float ra = sum[kMaxG * kD + g * 4 + 2], rb = part[kMaxG * kD + g * 4 + 2], r = fmaxf(ra, rb);
        sum[g * kD + gt] = sum[g * kD + gt] * ex(ra, r) + part[g * kD + gt] * ex(rb, r);
    }
    sync_group(grp);                                               // the references are read
    if (gt < G) {
        float4* const at = reinterpret_cast<float4*>(sum + kMaxG * kD) + gt;
        const float4 a = *at, b = reinterpret_cast<const float4*>(part + kMaxG * kD)[gt];
        const float m = fmaxf(a.x, b.x);
        *at = make_float4(m, a.y * ex(a.x, m) + b.y * ex(b.x, m), fmaxf(a.z, b.z), 0.f);
    }
}

// One warp: the query rows of (s, h) into an N-side operand, and each head's score factor.
template <bool CODE, bool WIDE, int GM>
__device__ __forceinline__ void queries(const WindowParams& p, unsigned char* qt, float* qscale, int s, int h, int lane) {
    using C = Cfg<CODE, WIDE, GM>;
    const uint2* src = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.q) +
                                                      (static_cast<size_t>(s) * p.Hq + static_cast<size_t>(h) * p.G) * kD) + lane;
    uint2 q[GM];
#pragma unroll
    for (int g = 0; g < GM; ++g)
        if (g < p.G) q[g] = __ldg(src + g * 32);                   // elements 4 lane .. 4 lane + 3
#pragma unroll
    for (int g = 0; g < GM; ++g) {
        if (g >= p.G) break;
        if constexpr (CODE) {
            const uint32_t mag = __vmaxu2(q[g].x & 0x7fff7fffu, q[g].y & 0x7fff7fffu);
            const uint32_t top = __reduce_max_sync(0xffffffffu, max(mag & 0xffffu, mag >> 16));
            const int e = static_cast<int>(top >> 7);
            // 2^k, the largest element into [2^7, 2^8); zero and non-finite rows stay
            const int k = e == 0 || e == 255 ? 0 : min(126, max(-126, e - 134));
            const float mul = pow2f(127 - k);
            float f[4] = {pa_dev::bf16_lo(q[g].x) * mul, pa_dev::bf16_hi(q[g].x) * mul, pa_dev::bf16_lo(q[g].y) * mul,
                          pa_dev::bf16_hi(q[g].y) * mul};
#pragma unroll 1
            for (int r = 0; r < C::kQParts; ++r) {
                const uint32_t a = pa_dev::e4m3x2_from_f32(f[0], f[1]), b = pa_dev::e4m3x2_from_f32(f[2], f[3]);
                *reinterpret_cast<uint32_t*>(qt + pa_tc::sw128_off(r * GM + g, lane >> 2) + (lane & 3) * 4) = (a & 0xffffu) | b << 16;
                const uint32_t fa = pa_dev::e4m3x2_to_f16x2(a), fb = pa_dev::e4m3x2_to_f16x2(b);
                f[0] = (f[0] - pa_dev::f16_lo(fa)) * 16.f;
                f[1] = (f[1] - pa_dev::f16_hi(fa)) * 16.f;
                f[2] = (f[2] - pa_dev::f16_lo(fb)) * 16.f;
                f[3] = (f[3] - pa_dev::f16_hi(fb)) * 16.f;
            }
            // a row with an infinity (which e4m3 does not have) or a NaN gives NaN
            if (lane == 0) qscale[g] = e == 255 ? __int_as_float(0x7fffffff) : p.scale_log2 * pow2f(127 + k);
        } else {
            *reinterpret_cast<uint2*>(qt + (lane >> 4) * (C::kNQ * 128) + pa_tc::sw128_off(g, (lane & 15) >> 1) + (lane & 1) * 8) = q[g];
        }
    }
}

template <bool CODE, bool WIDE, int GM, bool CHUNKS>
__global__ void __launch_bounds__(kThreads, 1)
window_decode_kernel(const WindowParams p, int* counters, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap) {
    using C = Cfg<CODE, WIDE, GM>;
    extern __shared__ unsigned char raw[];
    const uint32_t raw_s = pa_tc::smem_u32(raw);
    unsigned char* base = raw + ((1024u - (raw_s & 1023u)) & 1023u);
    const uint32_t sbase = pa_tc::smem_u32(base);
    Misc<CODE, GM>& m = *reinterpret_cast<Misc<CODE, GM>*>(base + C::kMisc);
    volatile int* abort_flag = &m.abort_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            pa_tc::mbar_init(&m.bars[kQFull0 + i], 1);
            pa_tc::mbar_init(&m.bars[kQEmpty0 + i], 1);
            pa_tc::mbar_init(&m.bars[kSFull0 + i], 1);
            pa_tc::mbar_init(&m.bars[kSEmpty0 + i], 4);
            pa_tc::mbar_init(&m.bars[kOFull0 + i], 1);
            pa_tc::mbar_init(&m.bars[kOEmpty0 + i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            pa_tc::mbar_init(&m.bars[kPFull0 + i], 4);
            pa_tc::mbar_init(&m.bars[kPEmpty0 + i], 1);
            pa_tc::mbar_init(&m.bars[kDone0 + i], 1);
        }
        for (int i = 0; i < C::kStages; ++i) {
            for (int q = 0; q < 2; ++q) {
                pa_tc::mbar_init(&m.bars[kKFull0 + 6 * q + i], 33);    // + each lane: the step's description is written
                pa_tc::mbar_init(&m.bars[kVFull0 + 6 * q + i], 1);
            }
            pa_tc::mbar_init(&m.bars[kKEmpty0 + i], 1);
            pa_tc::mbar_init(&m.bars[kVEmpty0 + i], 1);
        }
        m.abort_flag = 0;
        pa_tc::mbar_init_fence();
    }
    // N-side rows and columns that no head uses stay zero
    for (int i = tid * 16; i < 4 * C::kQStride + 2 * C::kPBytes; i += kThreads * 16)
        *reinterpret_cast<uint4*>(base + C::kQOff + i) = make_uint4(0u, 0u, 0u, 0u);
    pa_tc::fence_smem_to_async();
    pa_dev::wait_prior_grid();
    pa_dev::allow_next_grid();

    // the groups' ranges of steps [u0, u0 + n) and the sequences they start in; the
    // first groups of all CTAs come first in the list, so little work spreads out
    const int seg = (p.S + kThreads - 1) / kThreads;
    const int s_lo = min(p.S, tid * seg), s_hi = min(p.S, s_lo + seg);
    long long mine = 0;
    for (int s = s_lo; s < s_hi; ++s) {
        Walk w;
        w.s = s;
        w.load(p);
        mine += w.nt;
        if (blockIdx.x == 0) {
            const int L = __ldg(p.lens + s);
            if (L < 0 || L > p.max_blocks * kBlk) pa_dev::record_error(p.err, PA_ERR_BAD_LENGTH);
        }
    }
    long long inc = mine;
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) m.scan[warp] = inc;
    __syncthreads();
    long long before = inc - mine, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += m.scan[w];
        total += m.scan[w];
    }
    total *= p.Hkv;
    const long long per = (total + 2 * gridDim.x - 1) / (2 * gridDim.x);
    int n[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const long long u0 = min(total, per * (blockIdx.x + q * static_cast<long long>(gridDim.x)));
        n[q] = static_cast<int>(min(total, u0 + per) - u0);
        if (n[q] > 0 && before * p.Hkv <= u0 && u0 < (before + mine) * p.Hkv) {
            long long b = before * p.Hkv;
            for (int s = s_lo; s < s_hi; ++s) {
                Walk w;
                w.s = s;
                w.load(p);
                if (u0 < b + static_cast<long long>(w.nt) * p.Hkv) {
                    m.start_s[q] = s;
                    m.start_base[q] = b;
                    break;
                }
                b += static_cast<long long>(w.nt) * p.Hkv;
            }
        }
    }
    // rows of empty contexts, spread over the CTAs
    for (int s = blockIdx.x; s < p.S; s += gridDim.x)
        if (seq_len(p, s) == 0)
            for (int i = tid; i < p.Hq * kD; i += kThreads) {
                const size_t o = static_cast<size_t>(s) * p.Hq * kD + i;
                if (WIDE) static_cast<float*>(p.out)[o] = 0.f;
                else static_cast<uint16_t*>(p.out)[o] = 0;
            }
    if (n[0] == 0) return;                                         // uniform; no TMEM held yet (n[1] <= n[0])
    if (warp == 9) pa_tc::tmem_alloc<C::kTmemCols>(&m.tmem);
    pa_tc::fence_before_sync();
    __syncthreads();
    pa_tc::fence_after_sync();
    const uint32_t tmem = m.tmem;
    const int G = p.G, Hkv = p.Hkv;
    auto starts = [](int tile) { return (CHUNKS ? tile % kChunk : tile) == 0; };      // an item, or a chunk of one
    auto begin = [&](int q) {                                      // group q's first step
        Walk w;
        w.s = m.start_s[q];
        w.load(p);
        const long long u = per * (blockIdx.x + q * static_cast<long long>(gridDim.x)) - m.start_base[q];
        w.h = static_cast<int>(u / w.nt);
        w.tile = static_cast<int>(u - static_cast<long long>(w.h) * w.nt);
        return w;
    };
    // copies alternate between the groups while both have steps: the place of group
    // q's step t in the ring
    auto place = [&](int q, int t) { return t < n[1] ? 2 * t + q : n[1] + t; };
    bool ok = true;

    if (warp < 8) {
        // ------------------------------------------------------ weights
        const int grp = warp >> 2, wq = warp & 3, gt = tid & 127;  // thread gt: token gt of the group's steps
        const uint32_t lane_sel = static_cast<uint32_t>(wq * 32) << 16;
        const int blk = gt / kBlk, bit = gt % kBlk;
        // Heads are taken four at a time, by code that is not unrolled: with eight heads
        // written out, a step's code did not fit the instruction cache and a third of the
        // warps' time went into fetching it.  A thread's references and sums of each
        // four move along, so that the four at work are always the first ones.
        float r_m[GM], r_o[GM], l[GM];
#pragma unroll
        for (int g = 0; g < GM; ++g) {
            r_m[g] = r_o[g] = -INFINITY;
            l[g] = 0.f;
        }
        int votes = 0;
        float acc[C::kAddSteps ? GM : 4] = {};                     // kAddSteps: the item's steps before the last one
        auto add_parts = [&](const float (&o)[C::kPParts][4], int k) {
            // (bf16 remainders have their own exponents; 8-bit ones were scaled)
            float y = 0.f;
#pragma unroll
            for (int i = C::kPParts - 1; i >= 0; --i) y = CODE ? fmaf(y, 1.f / C::kPart, o[i][k]) : y + o[i][k];
            return y;
        };
        const int steps = n[grp];
        const long long range = blockIdx.x + grp * static_cast<long long>(gridDim.x), u0 = per * range;
        // An item's (or chunk's) result is written while the next one's first step is under
        // way (its last value product is done by then).  cont, more: the range holds chunks
        // of the item before, after this one
        struct Pending { int it, s, h, nt, begins, ends, cont, more; long long u_first; } pend = {-1, 0, 0, 0, 0, 0, 0, 0, 0};
        auto finish = [&]() {
            const int ip = pend.it & 1;
            ok &= wait(&m.bars[kOFull0 + grp * 2 + ip], (pend.it >> 1) & 1, abort_flag);
            pa_tc::fence_after_sync();
            const size_t row0 = static_cast<size_t>(pend.s) * p.Hq + static_cast<size_t>(pend.h) * G;
            const bool whole = pend.begins && pend.ends && !(CHUNKS && pend.cont);
            float* const sum = p.part + (2 * static_cast<size_t>(range) + pend.begins) * kSlot;
            float* const slot = CHUNKS && pend.cont ? p.part + (4 * static_cast<size_t>(gridDim.x) + range) * kSlot : sum;
            const uint32_t od = tmem + C::kOCol + (grp * 2 + ip) * C::kNP + lane_sel;
#pragma unroll 1
            for (int g0 = 0; g0 < GM; g0 += 4) {                   // four heads at a time: their columns of every part
                float o[C::kPParts][4];
#pragma unroll
                for (int i = 0; i < C::kPParts; ++i) tmem_ld4(od + i * GM + g0, o[i]);
                pa_tc::tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int g = g0 + k;
                    if (g >= G) break;
                    const float y = add_parts(o, k) + (C::kAddSteps ? acc[k] : 0.f);
                    const float* q = &m.lsum[grp][ip][0][g];
                    const float ls = (q[0] + q[GM]) + (q[2 * GM] + q[3 * GM]);
                    const float rm = m.ref[grp][ip][0][g], ro = m.ref[grp][ip][CODE ? 1 : 0][g];
                    if (whole) {
                        const float f = ls > 0.f && ro != -INFINITY ? p.v_scale / ls * (CODE ? pa_dev::ex2(ro - rm) : 1.f) : 0.f;
                        const size_t i = (row0 + g) * kD + gt;
                        if (WIDE) static_cast<float*>(p.out)[i] = y * f;
                        else static_cast<__nv_bfloat16*>(p.out)[i] = __float2bfloat16_rn(y * f);
                    } else {
                        slot[g * kD + gt] = y;
                        if (gt == 0) *reinterpret_cast<float4*>(slot + kMaxG * kD + g * 4) = make_float4(rm, ls, ro, 0.f);
                    }
                }
                if constexpr (C::kAddSteps) {
                    acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
                    next_four(acc);
                }
                __syncwarp();
            }
            pa_tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) arrive(&m.bars[kOEmpty0 + grp * 2 + ip]);
            if (CHUNKS && pend.cont) add_chunk(sum, slot, G, gt, grp);
            if (!whole && !(CHUNKS && pend.more)) {
                // the last of the item's groups to get here merges them, in their order
                const long long c_first = pend.u_first / per, c_last = (pend.u_first + pend.nt - 1) / per;
                const int item = pend.s * Hkv + pend.h, parts = static_cast<int>(c_last - c_first) + 1;
                __threadfence();
                sync_group(grp);
                if (gt == 0) m.merge[grp] = atomicAdd(counters + item, 1) == parts - 1;
                sync_group(grp);
                if (m.merge[grp]) {
                    __threadfence();
                    merge_item<WIDE>(p, c_first, parts, row0, gt);
                    if (gt == 0) counters[item] = 0;               // for the next call
                }
            }
        };
        long long u_first = u0;                                    // the item's first step in the list
        int it = -1, cont = 0;                                     // items (chunks) begun
        uint32_t v_ph = 0;                                         // bit st: parity of slot st's next phase
        Walk w = {};
        if (steps > 0) w = begin(grp);
        for (int j = 0; j < steps; ++j) {
            const bool first = j == 0 || starts(w.tile);
            const bool last = j == steps - 1 || w.tile == w.nt - 1 || (CHUNKS && (w.tile + 1) % kChunk == 0);
            if (first) {
                ++it;
                if constexpr (CHUNKS) cont = j > 0 && w.tile > 0;
                u_first = u0 + j - w.tile;
            }
            const int par = j & 1;
            const int pl = place(grp, j), st = pl % C::kStages;
            ok &= wait(&m.bars[kSFull0 + grp * 2 + par], (j >> 1) & 1, abort_flag);
            pa_tc::fence_after_sync();
            const int have = *const_cast<volatile uint8_t*>(&m.have[pl % kInfo]);
            float kf = 1.f, ev = 0.f;
            if (CODE && p.scales) {
                const uint32_t e = *const_cast<volatile uint16_t*>(&m.exps[pl % kInfo][blk]);
                kf = pow2f(e & 0xff);
                ev = (e >> 8) ? static_cast<float>(static_cast<int>(e >> 8) - 127) : -INFINITY;
            }
            // which keys the query sees: all of the step's, or, lane by lane, each block's bits
            const int pos = w.L - 1, i0 = w.tile * kStepBlks, first_key = w.block(i0) * kBlk;
            const bool full = have == 0xff && i0 >= w.sb && first_key + kStep - 1 <= pos &&
                              first_key >= pos - (p.window - 1);
            uint32_t my_bits = 0xffffu;                            // lane b < 8: block b's
            if (!full)
                my_bits = (have >> (lane & 7)) & 1 ? seen_bits(pos, w.block(i0 + (lane & 7)) * kBlk, p.window, p.sinks) : 0u;
            const bool seen = full || ((__shfl_sync(0xffffffffu, my_bits, blk) >> bit) & 1);
            // P^T element (column n, token gt); column n of a token group's 8-row tiles starts at 16 n
            unsigned char* const prow = base + C::kPOff + grp * C::kPBytes +
                                        (CODE ? (gt >> 4) * C::kLbo + (gt & 15) : (gt >> 3) * C::kLbo + (gt & 7) * 2);
#pragma unroll 1
            for (int g0 = 0; g0 < GM; g0 += 4) {
                float x[C::kQParts][4], qs[4];
#pragma unroll
                for (int i = 0; i < C::kQParts; ++i) tmem_ld4(tmem + (grp * 2 + par) * C::kNQ + lane_sel + i * GM + g0, x[i]);
                if constexpr (CODE) {
                    const float4 y = *reinterpret_cast<const float4*>(&m.qscale[grp][it & 3][g0]);
                    qs[0] = y.x;
                    qs[1] = y.y;
                    qs[2] = y.z;
                    qs[3] = y.w;
                } else {
                    qs[0] = qs[1] = qs[2] = qs[3] = p.scale_log2;
                }
                pa_tc::tmem_wait_ld();
                if (g0 == GM - 4) {                                // the scores are taken out
                    pa_tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) arrive(&m.bars[kSEmpty0 + grp * 2 + par]);
                }
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    if constexpr (CODE) x[0][g] = fmaf(x[2][g], 1.f / 256, fmaf(x[1][g], 1.f / 16, x[0][g])) * (qs[g] * kf);
                    else x[0][g] = x[0][g] * qs[g];
                    x[0][g] = seen ? x[0][g] : -INFINITY;          // (after the scaling: -inf times 0 is NaN)
                }
                // References, the same for the group's 128 tokens: raised when unset or
                // passed by 2^8, of codes' weights by 2^kLag.  Usually none rises, which one
                // vote and four flags tell; the maxima are formed only when one does.
                if (first) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        r_m[g] = r_o[g] = -INFINITY;
                        l[g] = 0.f;
                    }
                }
                bool rises = first;
                if (!first) {
                    bool need = false;
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        if (g0 + g < G) need |= x[0][g] > r_m[g] + 8.f || (CODE && x[0][g] + ev > r_o[g] + (C::kLift + C::kLag));
                    const bool any = __any_sync(0xffffffffu, need);
                    // (a vote's flags are written again two votes on, past another barrier)
                    if (lane == 0) m.flags[grp][votes & 1][wq] = any;
                    sync_group(grp);
                    const int4 f = *reinterpret_cast<const int4*>(m.flags[grp][votes & 1]);
                    rises = f.x | f.y | f.z | f.w;
                    ++votes;
                }
                if (rises) {
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        if (g0 + g < G) {
                            const float a = warp_max(x[0][g]);
                            const float b = CODE ? warp_max(x[0][g] + ev) : a;
                            if (lane == 0) {
                                m.red[grp][par][wq][0][g0 + g] = a;
                                if constexpr (CODE) m.red[grp][par][wq][1][g0 + g] = b;
                            }
                        }
                    sync_group(grp);
                }
                // the P buffer and O were last touched by this group's value product before
                if (g0 == 0 && j >= 1) ok &= wait(&m.bars[kPEmpty0 + grp], (j - 1) & 1, abort_flag);
                if constexpr (C::kAddSteps) {
                    if (!first) {                                  // the step before
                        float o[C::kPParts][4];
                        pa_tc::fence_after_sync();
#pragma unroll
                        for (int i = 0; i < C::kPParts; ++i)
                            tmem_ld4(tmem + C::kOCol + (grp * 2 + (it & 1)) * C::kNP + lane_sel + i * GM + g0, o[i]);
                        pa_tc::tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 4; ++k) acc[k] += add_parts(o, k);
                    }
                }
                if (rises) {
                    // (these maxima's place is written again two steps on, past another barrier)
                    float top[2][4];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int e = 0; e < (CODE ? 2 : 1); ++e) {
                            const float4 y = *reinterpret_cast<const float4*>(&m.red[grp][par][q][e][g0]);
                            top[e][0] = q ? fmaxf(top[e][0], y.x) : y.x;
                            top[e][1] = q ? fmaxf(top[e][1], y.y) : y.y;
                            top[e][2] = q ? fmaxf(top[e][2], y.z) : y.z;
                            top[e][3] = q ? fmaxf(top[e][3], y.w) : y.w;
                        }
                    float corr[4];
                    bool scale_o = false;
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        corr[g] = 1.f;
                        if (g0 + g < G) {
                            const float mx = top[0][g], mo = top[CODE ? 1 : 0][g];
                            const float old_m = r_m[g], old_o = r_o[g];
                            if (mx > old_m + 8.f) {
                                r_m[g] = mx;
                                l[g] *= old_m == -INFINITY ? 0.f : pa_dev::ex2(old_m - mx);
                            }
                            if (mo - C::kLift > old_o + C::kLag) {
                                r_o[g] = mo - C::kLift;
                                if (old_o != -INFINITY) {
                                    corr[g] = pa_dev::ex2(old_o - r_o[g]);
                                    scale_o = true;
                                }
                            }
                        }
                    }
                    if constexpr (C::kAddSteps) {
#pragma unroll
                        for (int g = 0; g < 4; ++g) acc[g] *= corr[g];
                    } else if (scale_o) {
                        const uint32_t od = tmem + C::kOCol + (grp * 2 + (it & 1)) * C::kNP + lane_sel + g0;
                        pa_tc::fence_after_sync();
#pragma unroll 1
                        for (int i = 0; i < C::kPParts; ++i) {
                            float o[4];
                            tmem_ld4(od + i * GM, o);
                            pa_tc::tmem_wait_ld();
#pragma unroll
                            for (int g = 0; g < 4; ++g) o[g] *= corr[g];
                            tmem_st4(od + i * GM, o);
                        }
                        pa_tc::tmem_wait_st();
                    }
                }
                float v[4];
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    v[g] = 0.f;
                    if (g0 + g < G) {
                        const float r = r_m[g] == -INFINITY ? 0.f : r_m[g];
                        const float ro = r_o[g] == -INFINITY ? 0.f : r_o[g];
                        const float e = pa_dev::ex2(x[0][g] - r);
                        l[g] += e;
                        v[g] = CODE ? pa_dev::ex2(x[0][g] + ev - ro) : e;
                    }
                }
                unsigned char* pcol = prow + g0 * 16;
#pragma unroll 1
                for (int i = 0; i < C::kPParts; ++i, pcol += GM * 16) {
#pragma unroll
                    for (int g = 0; g < 4; g += 2) {
                        if constexpr (CODE) {
                            const uint32_t c = C::kE5 ? e5m2x2_from_f32(v[g], v[g + 1]) : pa_dev::e4m3x2_from_f32(v[g], v[g + 1]);
                            pcol[g * 16] = static_cast<unsigned char>(c);
                            pcol[g * 16 + 16] = static_cast<unsigned char>(c >> 8);
                            const uint32_t f = C::kE5 ? e5m2x2_to_f16x2(c) : pa_dev::e4m3x2_to_f16x2(c);
                            v[g] = (v[g] - pa_dev::f16_lo(f)) * C::kPart;
                            v[g + 1] = (v[g + 1] - pa_dev::f16_hi(f)) * C::kPart;
                        } else {
                            const uint32_t c = pa_dev::pack_bf16(v[g], v[g + 1]);
                            *reinterpret_cast<uint16_t*>(pcol + g * 16) = static_cast<uint16_t>(c);
                            *reinterpret_cast<uint16_t*>(pcol + g * 16 + 16) = static_cast<uint16_t>(c >> 16);
                            v[g] -= pa_dev::bf16_lo(c);
                            v[g + 1] -= pa_dev::bf16_hi(c);
                        }
                    }
                }
                next_four(r_m);
                next_four(r_o);
                next_four(l);
                if constexpr (C::kAddSteps) next_four(acc);
            }
            // values of keys that the query does not see become zero (0 * Inf is NaN, and a
            // block that was not loaded leaves what an earlier step left): thread d clears
            // its row of each such block, of those that the value product reads
            if (!full) {
                // (this group's earlier copies into the slot have landed: their products are done)
                ok &= wait(&m.bars[kVFull0 + 6 * grp + st], (v_ph >> st) & 1, abort_flag);
                unsigned char* vt = base + C::kVOff + st * C::kHalf;
                uint32_t todo = __ballot_sync(0xffffffffu, lane < read_blocks<CODE>(w.nv - i0) && (my_bits & 0xffffu) != 0xffffu);
                while (todo) {
                    const int b = __ffs(todo) - 1;
                    todo &= todo - 1;
                    const uint32_t bits = __shfl_sync(0xffffffffu, my_bits, b);
                    if constexpr (CODE) {
                        uint4* row = reinterpret_cast<uint4*>(vt + b * 2048 + gt * 16);
                        auto keep = [](uint32_t four) {            // bit i -> byte i
                            return (((four & 1) | (four & 2) << 7 | (four & 4) << 14 | (four & 8) << 21)) * 255u;
                        };
                        uint4 y = *row;
                        y.x &= keep(bits);
                        y.y &= keep(bits >> 4);
                        y.z &= keep(bits >> 8);
                        y.w &= keep(bits >> 12);
                        *row = y;
                    } else {
                        unsigned char* row = vt + b * 4096 + gt * 32;
                        const int flip = (gt >> 2) & 1;            // the halves trade places (32-byte swizzle)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            uint4* q = reinterpret_cast<uint4*>(row + ((hf ^ flip) << 4));
                            const uint32_t e = bits >> (8 * hf);
                            auto keep = [](uint32_t two) { return (two & 1 ? 0xffffu : 0u) | (two & 2 ? 0xffff0000u : 0u); };
                            uint4 y = *q;
                            y.x &= keep(e);
                            y.y &= keep(e >> 2);
                            y.z &= keep(e >> 4);
                            y.w &= keep(e >> 6);
                            *q = y;
                        }
                    }
                }
            }
            v_ph ^= 1u << st;
            pa_tc::fence_smem_to_async();
            pa_tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) arrive(&m.bars[kPFull0 + grp]);
            // the item before, if it ended with the last step: its sums are visible, this
            // step's `first` has taken a barrier since
            if (pend.it >= 0) {
                finish();
                pend.it = -1;
            }
            if (last) {
                // Sums over the warp's lanes, halving the heads with the lanes: lane i ends
                // with head (i >> 3) of the four
#pragma unroll 1
                for (int g0 = 0; g0 < GM; g0 += 4) {
                    float y[4] = {l[0], l[1], l[2], l[3]};
#pragma unroll
                    for (int cnt = 2, off = 16; cnt >= 1; cnt >>= 1, off >>= 1)
#pragma unroll
                        for (int i = 0; i < cnt; ++i) {
                            const bool up = lane & off;
                            const float give = up ? y[i] : y[i + cnt], keep = up ? y[i + cnt] : y[i];
                            y[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
                        }
#pragma unroll
                    for (int off = 4; off >= 1; off >>= 1) y[0] += __shfl_xor_sync(0xffffffffu, y[0], off);
                    if ((lane & 7) == 0) m.lsum[grp][it & 1][wq][g0 + (lane >> 3)] = y[0];
                    if (gt == 0)
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            m.ref[grp][it & 1][0][g0 + g] = r_m[g];
                            if constexpr (CODE) m.ref[grp][it & 1][1][g0 + g] = r_o[g];
                        }
                    next_four(r_m);
                    next_four(r_o);
                    next_four(l);
                }
                pend = {it, w.s, w.h, w.nt, u_first >= u0, w.tile == w.nt - 1, cont, CHUNKS && j < steps - 1 && w.tile < w.nt - 1, u_first};
            }
            w.next(p);
        }
        if (steps > 0) {
            sync_group(grp);
            finish();
        }
    } else if (warp == 8 || warp == 11) {
        // ------------------------------------------------------- copies
        // Warp 8 copies keys (and describes the steps), warp 11 values; it also prepares
        // the queries.  Three steps are under way at once: one's copies go out, the next
        // one's exponents and table entries after that are on their way.
        const bool values = warp == 11;
        Walk w[2] = {begin(0), {}};
        if (n[1] > 0) w[1] = begin(1);
        const int all = n[0] + n[1];
        struct Next { int x, s, h, first; };                       // a step's table entry (lane b < 8: block b), item
        auto entry = [&](int i) {                                  // of the step in place i; -2: no block there
            Next e = {-2, 0, 0, 0};
            if (i >= all) return e;
            const int q = i < 2 * n[1] ? i & 1 : 0;
            Walk v = q ? w[1] : w[0];
            const int b = v.tile * kStepBlks + lane;
            if (lane < kStepBlks && b < v.nv) e.x = __ldg(p.tables + static_cast<size_t>(v.s) * p.max_blocks + v.block(b));
            e.s = v.s;
            e.h = v.h;
            e.first = starts(v.tile);
            v.next(p);
            if (q) w[1] = v;
            else w[0] = v;
            return e;
        };
        auto tile_of = [&](const Next& e) {                        // (block, head) index, below 2^31 / 16; -1: none
            if (e.x >= 0 && e.x < p.num_blocks) return e.x * Hkv + e.h;
            if (e.x != -2 && !values) pa_dev::record_error(p.err, PA_ERR_BAD_BLOCK_ID);
            return -1;
        };
        auto exponents = [&](int tile) {
            return CODE && !values && p.scales && tile >= 0 ? static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(
                       p.scales + static_cast<size_t>(tile) * 2))) : 0u;
        };
        int its[2] = {-1, -1};
        uint32_t used[2] = {0, 0}, ph[2] = {0, 0};                 // bit st: slot st was filled; parity of its next phase
        Next n0 = entry(0);
        int t0 = tile_of(n0);
        uint32_t e0 = exponents(t0);
        Next n1 = entry(1);
        for (int i = 0; i < all; ++i) {
            const int st = i % C::kStages;
            const int t1 = tile_of(n1);
            const uint32_t e1 = exponents(t1);
            const Next n2 = entry(i + 2);
            const int q = i < 2 * n[1] ? i & 1 : 0, j = i < 2 * n[1] ? i >> 1 : i - n[1];
            if (values && (j == 0 || n0.first)) {
                const int it = q ? ++its[1] : ++its[0];
                if (it >= 2 && !wait(&m.bars[kQEmpty0 + q * 2 + (it & 1)], ((it >> 1) - 1) & 1, abort_flag)) { ok = false; break; }
                queries<CODE, WIDE, GM>(p, base + C::kQOff + (q * 2 + (it & 1)) * C::kQStride, CODE ? m.qscale[CODE ? q : 0][CODE ? it & 3 : 0] : nullptr, n0.s, n0.h, lane);
                pa_tc::fence_smem_to_async();
                __syncwarp();
                if (lane == 0) arrive(&m.bars[kQFull0 + q * 2 + (it & 1)]);
            }
            uint64_t* full = &m.bars[(values ? kVFull0 : kKFull0) + 6 * q + st];
            if (i >= C::kStages && !wait(&m.bars[(values ? kVEmpty0 : kKEmpty0) + st], (i / C::kStages - 1) & 1, abort_flag)) {
                ok = false;
                break;
            }
            const uint32_t have = __ballot_sync(0xffffffffu, t0 >= 0);
            const uint32_t dst = sbase + (values ? C::kVOff : 0) + st * C::kHalf;
            if (CODE && !values && lane < kStepBlks) m.exps[i % kInfo][lane] = static_cast<uint16_t>(e0);
            if (!values && lane == 0) m.have[i % kInfo] = static_cast<uint8_t>(have);
            int tiles[kStepBlks];
#pragma unroll
            for (int b = 0; b < kStepBlks; ++b) tiles[b] = __shfl_sync(0xffffffffu, t0, b);
            if (pa_tc::elect_one()) {
                pa_tc::mbar_expect_tx(full, __popc(have) * (CODE ? 2048 : 4096));
                if (values) {
#pragma unroll
                    for (int b = 0; b < kStepBlks; ++b) {
                        if (tiles[b] < 0) continue;
                        if constexpr (CODE)
                            pa_tc::bulk_load(dst + b * 2048, static_cast<const unsigned char*>(p.v) + static_cast<size_t>(tiles[b]) * 2048,
                                             2048, full);
                        else
                            pa_tc::tma_load_2d(dst + b * 4096, &vmap, 0, tiles[b] * kD, full);
                    }
                } else {
#pragma unroll
                    for (int b = 0; b < kStepBlks; ++b) {
                        if (tiles[b] < 0) continue;
                        pa_tc::tma_load_2d(dst + b * 2048, &kmap, 0, tiles[b] * kBlk, full);
                        if (!CODE) pa_tc::tma_load_2d(dst + 16384 + b * 2048, &kmap, 64, tiles[b] * kBlk, full);
                    }
                }
            }
            __syncwarp();
            if (!values) arrive(full);                             // every lane: its part of the description is written
            if (q) {
                used[1] |= 1u << st;
                ph[1] ^= 1u << st;
            } else {
                used[0] |= 1u << st;
                ph[0] ^= 1u << st;
            }
            n0 = n1;
            n1 = n2;
            t0 = t1;
            e0 = e1;
        }
        // copies in flight land before the shared memory goes: each slot's last one of
        // each group
#pragma unroll
        for (int q = 0; q < 2; ++q)
            for (int st = 0; st < C::kStages; ++st)
                if ((used[q] >> st) & 1) pa_tc::mbar_wait(&m.bars[(values ? kVFull0 : kKFull0) + 6 * q + st], ((ph[q] >> st) & 1) ^ 1, kWaitLimit);
    } else if (warp < 11) {
        // --------------------------------------------------- MMA issue
        // QK(j) goes out before PV(j - 1), so the next scores are ready when the
        // weight warps come back
        const int grp = warp - 9, steps = n[grp];
        Walk w = {};
        if (steps > 0) w = begin(grp);
        int it = -1, pv_it = -1;
        uint32_t k_ph = 0, v_ph = 0;                               // bit st: parity of slot st's next phase
        auto value_product = [&](int j, bool first, bool last, int blocks) {
            const int pl = place(grp, j), st = pl % C::kStages;
            if (first) ++pv_it;
            const int ob = grp * 2 + (pv_it & 1);
            if (first && pv_it >= 2 && !wait(&m.bars[kOEmpty0 + ob], ((pv_it >> 1) - 1) & 1, abort_flag)) return false;
            if (!wait(&m.bars[kPFull0 + grp], j & 1, abort_flag) ||
                !wait(&m.bars[kVFull0 + 6 * grp + st], (v_ph >> st) & 1, abort_flag))
                return false;
            v_ph ^= 1u << st;
            pa_tc::fence_after_sync();
            if (pa_tc::elect_one()) {
                const uint32_t v = sbase + C::kVOff + st * C::kHalf, pt = sbase + C::kPOff + grp * C::kPBytes;
                const uint32_t o = tmem + C::kOCol + ob * C::kNP;
                constexpr uint32_t kLbo = C::kLbo;
                if constexpr (CODE) {
#pragma unroll
                    for (int i = 0; i < kStep / 32; ++i)
                        if (2 * i < blocks) mma_8bit(o, plain_desc(v + i * 4096, 2048, 128), plain_desc(pt + i * 2 * kLbo, kLbo, 128),
                                 idesc_8bit(kD, C::kNP, C::kE5), !(first && i == 0));
                } else {
#pragma unroll
                    for (int i = 0; i < kStep / 16; ++i)
                        if (i < blocks) pa_tc::mma_bf16(o, pa_tc::sw32_desc(v + i * 4096), plain_desc(pt + i * 2 * kLbo, kLbo, 128),
                                        pa_tc::idesc_bf16_f32(kD, C::kNP), i > 0 || !(first || C::kAddSteps));
                }
                pa_tc::commit(&m.bars[kPEmpty0 + grp]);
                pa_tc::commit(&m.bars[kVEmpty0 + st]);
                if (last) pa_tc::commit(&m.bars[kOFull0 + ob]);
            }
            __syncwarp();
            return true;
        };
        bool first_prev = false, last_prev = false;
        int blocks_prev = 0;
        for (int j = 0; j < steps; ++j) {
            const int pl = place(grp, j), st = pl % C::kStages, sb = grp * 2 + (j & 1);
            const bool first = j == 0 || starts(w.tile);
            const bool last = j == steps - 1 || w.tile == w.nt - 1 || (CHUNKS && (w.tile + 1) % kChunk == 0);
            if (first) {
                ++it;
                if (!wait(&m.bars[kQFull0 + grp * 2 + (it & 1)], (it >> 1) & 1, abort_flag)) { ok = false; break; }
            }
            if (!wait(&m.bars[kKFull0 + 6 * grp + st], (k_ph >> st) & 1, abort_flag) ||
                (j >= 2 && !wait(&m.bars[kSEmpty0 + sb], ((j >> 1) - 1) & 1, abort_flag))) {
                ok = false;
                break;
            }
            k_ph ^= 1u << st;
            pa_tc::fence_after_sync();
            if (pa_tc::elect_one()) {
                const uint32_t k = sbase + st * C::kHalf, q = sbase + C::kQOff + (grp * 2 + (it & 1)) * C::kQStride;
                if constexpr (CODE) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mma_8bit(tmem + sb * C::kNQ, pa_tc::sw128_desc(k + i * 32), pa_tc::sw128_desc(q + i * 32),
                                 idesc_8bit(kStep, C::kNQ, false), i > 0);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        pa_tc::mma_bf16(tmem + sb * C::kNQ, pa_tc::sw128_desc(k + (i >> 2) * 16384 + (i & 3) * 32),
                                        pa_tc::sw128_desc(q + (i >> 2) * (C::kNQ * 128) + (i & 3) * 32),
                                        pa_tc::idesc_bf16_f32(kStep, C::kNQ), i > 0);
                }
                pa_tc::commit(&m.bars[kSFull0 + sb]);
                pa_tc::commit(&m.bars[kKEmpty0 + st]);
                if (last) pa_tc::commit(&m.bars[kQEmpty0 + grp * 2 + (it & 1)]);
            }
            __syncwarp();
            if (j > 0 && !value_product(j - 1, first_prev, last_prev, blocks_prev)) { ok = false; break; }
            first_prev = first;
            last_prev = last;
            blocks_prev = w.nv - w.tile * kStepBlks;
            w.next(p);
        }
        if (ok && steps > 0) ok = value_product(steps - 1, first_prev, last_prev, blocks_prev);
        if (pa_tc::elect_one()) pa_tc::commit(&m.bars[kDone0 + grp]);
        __syncwarp();
        pa_tc::mbar_wait(&m.bars[kDone0 + grp], 0, kWaitLimit);    // MMAs are done before TMEM is freed
    }
    if (!ok) {
        *abort_flag = 1;
        if (lane == 0) pa_dev::record_error(p.err, PA_ERR_CUDA);
    }
    pa_tc::fence_before_sync();
    __syncthreads();
    pa_tc::fence_after_sync();
    if (warp == 9) pa_tc::tmem_free<C::kTmemCols>(tmem);
}

template <bool CODE, bool WIDE, int GM, bool CHUNKS = false>
int launch(pa_pool* pool, const WindowParams& p, int* counters, cudaStream_t st) {
    using C = Cfg<CODE, WIDE, GM>;
    auto kernel = window_decode_kernel<CODE, WIDE, GM, CHUNKS>;
    static std::atomic<uint64_t> done{0};
    if (!pa_detail::allow_smem(kernel, pool->device, C::kSmem, done)) return PA_ERR_CUDA;
    const cudaError_t e = pa_detail::launch_pdl(kernel, dim3(pool->num_sms), dim3(kThreads), C::kSmem, st, p, counters,
                                                pool->kmap, pool->vmap);
    pa_detail::count_launch();
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

namespace pa_detail {

// 32-bit TMA coordinates: key rows num_blocks * Hkv * 16, and for bf16 pools
// value rows num_blocks * Hkv * 128
bool window_decode_tc_eligible(const pa_pool* pool, const WindowParams& p) {
    const long long tiles = static_cast<long long>(pool->num_blocks) * pool->kv_heads;
    return pool->head_dim == kD && pool->block_size == kBlk && pool->dtype != PA_F32 && p.G <= kMaxG &&
           pool->smem_optin >= 227 * 1024 && reinterpret_cast<uintptr_t>(p.out) % 16 == 0 &&
           tiles * (pool->dtype == PA_BF16 ? kD : kBlk) < (1LL << 31);
}

// Bytes of the counters (one per item) and of the partials (two per range and one for a
// chunk, two ranges per CTA).
size_t window_decode_tc_counters(const pa_pool* pool, int S) {
    return (static_cast<size_t>(S) * pool->kv_heads * sizeof(int) + 255) / 256 * 256;
}
size_t window_decode_tc_partials(const pa_pool* pool) {
    return static_cast<size_t>(pool->num_sms) * 6 * kSlot * sizeof(float);
}

int launch_window_decode_tc(pa_pool* pool, const WindowParams& p, int* counters, cudaStream_t st) {
    const int rc = ensure_tensor_maps(pool);
    if (rc != PA_OK) return rc;
    const bool code = is_code(pool->dtype), wide = !p.out_bf16;
    // whether an item's steps in one range can be more than a chunk: by the table's width and
    // the window, which the host knows
    const int64_t blocks = std::min<int64_t>(p.max_blocks, (static_cast<int64_t>(p.window) + p.sinks) / kBlk + 3);
    const int64_t steps = (blocks + kStepBlks - 1) / kStepBlks, ranges = 2 * pool->num_sms;
    const bool chunks = code && wide && std::min(steps, (steps * p.S * p.Hkv + ranges - 1) / ranges) > kChunk;
    auto pick = [&](auto gm) {
        constexpr int GM = decltype(gm)::value;
        return chunks ? launch<true, true, GM, true>(pool, p, counters, st)
             : code ? (wide ? launch<true, true, GM>(pool, p, counters, st) : launch<true, false, GM>(pool, p, counters, st))
                    : (wide ? launch<false, true, GM>(pool, p, counters, st) : launch<false, false, GM>(pool, p, counters, st));
    };
    if (p.G <= 4) return pick(std::integral_constant<int, 4>{});
    if (p.G <= 8) return pick(std::integral_constant<int, 8>{});
    return pick(std::integral_constant<int, 16>{});
}

}  // namespace pa_detail
