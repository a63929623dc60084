// Windowed and block-scaled prefill attention on the 5th-generation tensor
// cores: 16-token blocks, head width 128; bf16 pools and e4m3-code pools.
//
// The mathematics.  A row is one (chunk token, query head of the group) pair; a
// CTA takes 256 consecutive rows of one (sequence, KV head) as two tiles of
// 128, and walks the keys that any of them sees in steps of 128 keys (8
// blocks): the blocks that hold sinks, then those of the windows' union.
//   S[128 x 128] = Q . K^T             tcgen05.mma, fp32 in TMEM
//   weights      one thread per row (TMEM lane); 2^(x - m) with a reference m
//                that is raised only when a row's maximum passes it by 2^8
//   O[128 x 128] += P . V              tcgen05.mma, P read from TMEM
// P takes the place of S (its columns are read before they are overwritten).
// For an fp32 output the weights enter the value product as a rounded part and a
// remainder; a bf16 output, rounded to 8 bits anyway, takes the rounded part alone.
//
// The tensor cores cut O to fp32 towards zero with every product of 16 keys, so a long
// sum shrinks.  For fp32 outputs O starts anew every kFlush steps, and what it held is
// added, rounded to nearest, to a total that is kept in the rows' own place in the
// output until they are done.
//
// Code pools: the codes are widened to f16 (exact) into the layouts the MMAs
// read, f16 MMAs.  Each query row is scaled by a power of two that puts its
// largest element into [2^7, 2^8), so bf16 queries of any size are exact in f16
// down to 2^-24 of the row's largest.  A block's key scale multiplies its
// scores.  Its value scale multiplies the weights: w = 2^(x - m) * 2^ev, f16
// relative to a reference of its own, because blocks may differ by more than f16
// holds.  The reference keeps the largest w at 2^9 .. 2^15, the upper end of f16:
// small weights are what its range is needed for, since many of them may count as
// much as the largest, or be all of the result where the largest one's value is
// zero.  What f16 cuts off is then under 2^-34 of the largest per key (2^-25 with
// the largest at 1 .. 2^8: of 131072 keys, weights of e^-17.6 all vanished).  A
// reference that is raised sooner gives more, and more sums to scale: 16 chunks,
// cold L2, 215 us with 1 .. 2^8, 219 now, 227 with 2^12 .. 2^15.
//
// Why this shape: one tile's QK^T and PV take the tensor cores while the other
// tile's threads compute weights; four MMA-sized TMEM buffers (two S/P, two O)
// fill TMEM, and two K and two V stages beside both Q tiles fill 192 KB.
//
// Measured (32 query, 8 KV heads): a prompt of 8191 tokens, window 2048, bf16, 221 us,
// 1.09 PFLOP/s of the visible scores' and values' products, 0.59 of the matrix rate
// (steps also compute what their masks hide, 6 % more); 16 chunks on up to 4096
// cached tokens, block-scaled, 216 us, 0.84 PFLOP/s.  A step of two tiles takes about 3000
// (bf16) to 3800 (codes) cycles, of which the MMAs need 2600; a CTA spends another
// 14000 or so, a third of a 10-step one, on its queries, its first keys, its results
// and the change to the next CTA.  A form whose CTAs stay and take tiles by ticket
// was a tenth to a quarter slower (its softmax warps spilled), and code for queries and results
// that is unrolled further costs more in fetching than it saves.
// Every mbarrier wait is bounded; on a timeout the CTA records PA_ERR_CUDA,
// drains its own copies and MMAs, frees TMEM and returns.
#include <cstdint>

#include <cuda.h>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_tc.cuh"

namespace {

constexpr int kD = 128;
constexpr int kTile = 128;               // rows per tile (M)
constexpr int kRows = 2 * kTile;         // rows per CTA
constexpr int kStep = 128;               // keys per step
constexpr int kBlk = 16;                 // tokens per block
constexpr int kStepBlks = kStep / kBlk;
constexpr int kStages = 2;
constexpr int kMaxSort = 128;            // sequences that are put in order of length
constexpr uint32_t kWaitLimit = 1u << 20;
constexpr uint32_t kTileBytes = 32768;   // one Q tile, K step or V step (16-bit elements)
constexpr uint32_t kQOff = 0;
constexpr uint32_t kKOff = 2 * kTileBytes;
constexpr uint32_t kVOff = kKOff + kStages * kTileBytes;
constexpr uint32_t kBarOff = kVOff + kStages * kTileBytes;
constexpr uint32_t kInfoOff = kBarOff + 256;             // descriptions of the last kInfo steps
constexpr int kInfo = 8;
constexpr uint32_t kCodeOff = kInfoOff + 256;             // code pools: a step's codes, K then V
constexpr uint32_t kCodeBytes = 16384;
constexpr uint32_t smem_bytes(bool code) { return kCodeOff + (code ? 2 * kCodeBytes : 0) + 1024; }   // + alignment slack
constexpr int kTmemCols = 512;           // S/P of tile t at 128 t, O of tile t at 256 + 128 t
constexpr int kFlush = 32;                // steps between flushes of fp32 outputs
// Code pools: the largest weight is 2^kLift when a reference is set, 2^(kLift + kLag)
// when it is raised (f16 holds up to 2^16)
constexpr float kLift = 9.f, kLag = 6.f;
enum Bar { kQFull, kSFull0, kSFull1, kPFull0, kPFull1, kOFull, kDone, kPartFull0, kPartFull1, kCodeFull0, kCodeFull1, kCodeEmpty0, kCodeEmpty1, kKFull0, kKEmpty0 = kKFull0 + kStages,
           kVFull0 = kKEmpty0 + kStages, kVEmpty0 = kVFull0 + kStages, kNumBars = kVEmpty0 + kStages };
// warps: 0-3 and 4-7 weights of tile 0 and 1, 8 copies, 9 MMA issue, 12-15 widening
// (codes); 10 unseen values (bf16), 11 idle (register allocation is by warpgroup)
constexpr int kThreadsBf16 = 384, kThreadsCode = 512;

// Bounded wait of a whole warp on an mbarrier phase; gives up, for every lane
// alike, when another role has raised the abort flag, and raises it on a timeout.
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

// What the copying warps tell the weight warps of step j, at j % kInfo: which blocks
// were loaded, and their exponents (K in the low byte, V in the next).  Written when
// the keys of step j - 2 are free, so long after anyone read step j - 8.
struct Info {
    uint16_t exps[kInfo][kStepBlks];
    int have[kInfo];
    int part[kInfo];                         // bf16: blocks whose values have positions that no row sees
};
static_assert(sizeof(Info) <= 256, "info area");

// The blocks a CTA walks: [0, sb) and [wb, eb), as one list of nv.
struct Keys {
    int sb, wb, nv, nsteps;
    __device__ __forceinline__ int block(int i) const { return i < sb ? i : i - sb + wb; }
};

__device__ __forceinline__ Keys key_list(int pa, int pb, int window, int sinks) {
    Keys k;
    const int wa = max(0, pa - (window - 1)), wz = max(0, pb - (window - 1));     // first window positions
    k.wb = wa / kBlk;
    k.sb = (min(sinks, wz) + kBlk - 1) / kBlk;       // blocks with a sink that some window has left behind
    if (k.sb >= k.wb) k.sb = k.wb = 0;               // one run
    k.nv = k.sb + pb / kBlk + 1 - k.wb;
    k.nsteps = (k.nv + kStepBlks - 1) / kStepBlks;
    return k;
}

// A row of a chunk, as (token, head of the group); rows are walked two by two
// without a division.
struct Row {
    int r, tok, head;
    __device__ __forceinline__ Row(int row, int G) : r(row), tok(row / G), head(row - tok * G) {}
    __device__ __forceinline__ void skip2(int G) {
        r += 2;
        head += 2;
        if (head >= G) { head -= G; ++tok; }
        if (head >= G) { head -= G; ++tok; }                         // one head a group
    }
};

// Bits of a block's 16 keys that a row at position p sees; the block starts at key j0.
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 16 ? 0xffffu : n <= 0 ? 0u : (1u << n) - 1u; }
__device__ __forceinline__ uint32_t seen_bits(int p, int j0, int window, int sinks) {
    return low_bits(p + 1 - j0) & (low_bits(sinks - j0) | ~low_bits(p - (window - 1) - j0));
}

// The keys that some row of the CTA sees: those from w_lo (the first row's window) to
// `end` (behind the last row's position), and the sinks.
struct Seen {
    int w_lo, end, sinks;
    __device__ __forceinline__ Seen(int pa, int pb, int window, int sinks_)
        : w_lo(max(0, pa - (window - 1))), end(pb + 1), sinks(sinks_) {}
    __device__ __forceinline__ uint32_t bits(int j0) const {         // of a block's 16 keys
        return low_bits(end - j0) & (low_bits(sinks - j0) | ~low_bits(w_lo - j0)) & 0xffffu;
    }
    __device__ __forceinline__ bool all(const Keys& k, int j) const { // every key of step j
        const int first = (j * kStepBlks - k.sb + k.wb) * kBlk;
        return j * kStepBlks >= k.sb && first >= w_lo && first + kStep <= end;
    }
};

__device__ __forceinline__ uint4 widen8(uint2 c) {
    return make_uint4(pa_dev::e4m3x2_to_f16x2(c.x), pa_dev::e4m3x2_to_f16x2(c.x >> 16),
                      pa_dev::e4m3x2_to_f16x2(c.y), pa_dev::e4m3x2_to_f16x2(c.y >> 16));
}
// 32, or 16, consecutive columns of this warp's lanes (the caller waits).
__device__ __forceinline__ void tmem_ld32_at(uint32_t taddr, float* v) {
    float y[32];
    pa_tc::tmem_ld32(taddr, y);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = y[i];
}
__device__ __forceinline__ void tmem_ld16_at(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr) : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ float pow2f(int biased) { return __uint_as_float(static_cast<uint32_t>(biased) << 23); }

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t y;
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ void unpack2(uint64_t y, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(y));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t y;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(a), "l"(b), "l"(c));
    return y;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t y;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
    return y;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t y;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
    return y;
}
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
// The weight warps hold 128 scores a thread, the widening ones 32 registers of codes.
// The block starts with 168 registers a thread (bf16, 384 threads) or 128 (codes, 512)
// and is split by warpgroup, within that total:
__host__ __device__ constexpr int regs_weights(bool code) { return code ? 192 : 200; }
__host__ __device__ constexpr int regs_rest(bool code) { return code ? 56 : 104; }
constexpr int kRegsWiden = 72;
static_assert(2 * regs_weights(true) + regs_rest(true) + kRegsWiden <= 4 * 128, "registers of the block");
static_assert(2 * regs_weights(false) + regs_rest(false) <= 3 * 168, "registers of the block");

template <bool CODE, bool PAIR>
__global__ void __launch_bounds__(CODE ? kThreadsCode : kThreadsBf16, 1)
window_prefill_kernel(const WindowParams p, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ unsigned char raw[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // Tiles start longest first, so that no long one is left running alone at the end: a
    // chunk's last rows see the most keys, and (p.by_length) long contexts go before
    // short ones.  KV heads are next to each other.
    const int G = p.G, Hkv = p.Hkv;
    const int from_last = blockIdx.y, h = blockIdx.x;
    int s = blockIdx.z;
    pa_dev::wait_prior_grid();
    pa_dev::allow_next_grid();
    const uint32_t raw_s = pa_tc::smem_u32(raw);
    unsigned char* base = raw + ((1024u - (raw_s & 1023u)) & 1023u);
    if (p.by_length) {
        int* s_len = reinterpret_cast<int*>(base + kQOff);           // (no query is there yet)
        const int mine = tid < p.S ? __ldg(p.lens + tid) : 0;
        if (tid < p.S) s_len[tid] = mine;
        __syncthreads();
        if (tid < p.S) {
            int rank = 0;
            for (int u = 0; u < p.S; ++u) rank += s_len[u] > mine || (s_len[u] == mine && u < tid);
            if (rank == s) s_len[kMaxSort] = tid;
        }
        __syncthreads();
        s = s_len[kMaxSort];
    }
    // the item; early returns are uniform and come before any barrier or TMEM
    const int q0 = __ldg(p.cu_q + s), q1 = __ldg(p.cu_q + s + 1), n = q1 - q0, L = __ldg(p.lens + s);
    const bool reporter = tid == 0 && from_last == 0 && h == 0;
    if (q0 < 0 || q1 < q0 || q1 > p.T || L < n || n > p.max_q) {
        if (reporter) pa_dev::record_error(p.err, PA_ERR_INVALID_ARG);
        return;
    }
    if (L > p.max_blocks * kBlk) {
        if (reporter) pa_dev::record_error(p.err, PA_ERR_BAD_LENGTH);
        return;
    }
    const int r_lo = ((n * G + kRows - 1) / kRows - 1 - from_last) * kRows;
    if (r_lo < 0) return;
    const int rows_end = min(n * G, r_lo + kRows), P0 = L - n;
    const int tiles = rows_end - r_lo > kTile ? 2 : 1;
    const Keys keys = key_list(P0 + r_lo / G, P0 + (rows_end - 1) / G, p.window, p.sinks);
    const int32_t* table = p.tables + static_cast<size_t>(s) * p.max_blocks;

    const uint32_t sbase = pa_tc::smem_u32(base);
    uint64_t* bars = reinterpret_cast<uint64_t*>(base + kBarOff);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(base + kBarOff + 8 * kNumBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
    static_assert(8 * kNumBars + 8 <= 256, "barrier area");
    Info& info = *reinterpret_cast<Info*>(base + kInfoOff);
    if (tid == 0) {
        pa_tc::mbar_init(&bars[kQFull], 8);
        pa_tc::mbar_init(&bars[kSFull0], 1);
        pa_tc::mbar_init(&bars[kSFull1], 1);
        pa_tc::mbar_init(&bars[kPFull0], 4);
        pa_tc::mbar_init(&bars[kPFull1], 4);
        pa_tc::mbar_init(&bars[kOFull], 1);
        pa_tc::mbar_init(&bars[kDone], 1);
        for (int i = 0; i < 2; ++i) {
            pa_tc::mbar_init(&bars[kCodeFull0 + i], 1);
            pa_tc::mbar_init(&bars[kCodeEmpty0 + i], 4);
        }
        for (int i = 0; i < kStages; ++i) {
            pa_tc::mbar_init(&bars[kKFull0 + i], CODE ? 4 : 1);
            pa_tc::mbar_init(&bars[kVFull0 + i], CODE ? 4 : 2);
            pa_tc::mbar_init(&bars[kPartFull0 + i], 1);
            pa_tc::mbar_init(&bars[kKEmpty0 + i], 1);
            pa_tc::mbar_init(&bars[kVEmpty0 + i], 1);
        }
        *abort_flag = 0;
        pa_tc::mbar_init_fence();
    }
    if (warp == 9) pa_tc::tmem_alloc<kTmemCols>(tslot);
    pa_tc::fence_before_sync();
    __syncthreads();
    pa_tc::fence_after_sync();
    const uint32_t tmem = *tslot;
    bool ok = true;
    constexpr uint32_t kIdesc = CODE ? pa_tc::idesc_f16_f32(kTile, kStep) : pa_tc::idesc_bf16_f32(kTile, kStep);

    if (warp >= 8 && warp < 12) fewer_registers<regs_rest(CODE)>();
    if (warp < 8) {
        // ------------------------------------------------------ weights
        more_registers<regs_weights(CODE)>();
        const int t = warp >> 2, row = tid, r = r_lo + row;          // row = 128 t + TMEM lane
        const bool row_ok = r < rows_end;
        const int qi = r / G, pos = row_ok ? P0 + qi : -1;
        float sl = p.scale_log2;
        {
            // the warp's 32 query rows into their tile (128-byte swizzle), two rows at a
            // time, 16 bytes a lane
            unsigned char* qt = base + kQOff + t * kTileBytes;
            const int hi = lane >> 4, c = lane & 15, w0 = (warp & 3) * 32;
            const uint16_t* qh = static_cast<const uint16_t*>(p.q) + static_cast<size_t>(h) * G * kD + 8 * c;
            Row at(r_lo + t * kTile + w0 + hi, G);
#pragma unroll
            for (int i0 = 0; i0 < 16; i0 += 8) {
                uint4 x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i, at.skip2(G)) {
                    x[i] = at.r < rows_end ? __ldg(reinterpret_cast<const uint4*>(qh + (static_cast<size_t>(q0 + at.tok) * p.Hq + at.head) * kD))
                                           : make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint4 y = x[i];
                    if constexpr (CODE) {
                        // largest magnitude of the row as bf16 bits (packed maxima of halves)
                        uint32_t mag = __vmaxu2(__vmaxu2(y.x & 0x7fff7fffu, y.y & 0x7fff7fffu),
                                                __vmaxu2(y.z & 0x7fff7fffu, y.w & 0x7fff7fffu));
#pragma unroll
                        for (int o = 8; o > 0; o >>= 1) mag = __vmaxu2(mag, __shfl_xor_sync(0xffffffffu, mag, o));
                        const int e = static_cast<int>(max(mag & 0xffffu, mag >> 16) >> 7);  // biased exponent of the largest
                        // 2^k with k = e - 134 (largest into [2^7, 2^8)); rows of zeros and
                        // of non-finite elements stay as they are
                        const int k = e == 0 || e == 255 ? 0 : min(126, max(-126, e - 134));
                        const float mul = pow2f(127 - k);
                        auto cv = [mul](uint32_t w) { return pa_dev::pack_f16(pa_dev::bf16_lo(w) * mul, pa_dev::bf16_hi(w) * mul); };
                        y = make_uint4(cv(y.x), cv(y.y), cv(y.z), cv(y.w));
                        // to the thread that owns the row
                        const int mine = __shfl_sync(0xffffffffu, k, (lane & 1) << 4);
                        if ((lane >> 1) == i0 + i) sl *= pow2f(127 + mine);
                    }
                    *reinterpret_cast<uint4*>(qt + (c >> 3) * 16384 + pa_tc::sw128_off(w0 + 2 * (i0 + i) + hi, c & 7)) = y;
                }
            }
            pa_tc::fence_smem_to_async();
            __syncwarp();
            if (lane == 0) arrive(&bars[kQFull]);
        }
        const uint32_t e_min = max(1, 128 - static_cast<int>((__float_as_uint(sl) >> 23) & 0xff));   // sl 2^(e_min - 127) >= 2^-126
        // the tile's first and last positions, for steps that need no mask
        const int pa = P0 + (r_lo + t * kTile) / G, pb = P0 + (min(rows_end, r_lo + (t + 1) * kTile) - 1) / G;
        const uint32_t lane_sel = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + t * 128 + lane_sel, tO = tmem + 256 + t * 128 + lane_sel;
        float m_ref = -INFINITY, o_ref = -INFINITY, l = 0.f;         // o_ref: code pools' weight reference
        // fp32 outputs: the rows' totals are kept in the warp's rows of p.out, relative to t_ref
        // (nothing there before the first flush).  Sixteen bytes of every row side by side,
        // not row by row: the rows there are (32, or a chunk's last few) make 32 times as many
        // places of 16 bytes, filled in the order (part of the row, lane), so that a warp's
        // access is 512 bytes in a row.  A prompt of 8191 on a bf16 pool, no window: 553 us; with
        // a flush every 16 steps 577, and row by row 653.
        float t_ref = -INFINITY;
        int fr = r;                                                  // (places are formed where they are used, not kept in registers)
        auto own_place = [&]() {
            asm volatile("" : "+r"(fr));
            const int tok = fr / G;
            return fr < rows_end ? reinterpret_cast<unsigned long long>(
                static_cast<float*>(p.out) + (static_cast<size_t>(q0 + tok) * p.Hq + static_cast<size_t>(h) * G + (fr - tok * G)) * kD) : 0ull;
        };
        auto total_at = [&](unsigned long long place, int i) {       // sixteen-byte part i of this lane's row
            const int at = i * min(32, rows_end - (fr - lane)) + lane;
            return reinterpret_cast<float4*>(__shfl_sync(0xffffffffu, place, (at >> 5) & 31)) + (at & 31);
        };
        auto add_totals = [&](unsigned long long place, int c, float ref, float (&o)[32]) {   // columns c .. c + 31
            const float f = t_ref == -INFINITY ? 1.f : pa_dev::ex2(t_ref - ref);
            float4 y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4* const at = total_at(place, c / 4 + i);
                y[i] = row_ok ? *at : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                o[4 * i] = fmaf(y[i].x, f, o[4 * i]);
                o[4 * i + 1] = fmaf(y[i].y, f, o[4 * i + 1]);
                o[4 * i + 2] = fmaf(y[i].z, f, o[4 * i + 2]);
                o[4 * i + 3] = fmaf(y[i].w, f, o[4 * i + 3]);
            }
        };
        const int steps = t < tiles ? keys.nsteps : 0;
        int j = 0;
        auto step = [&]() {                                          // step j's weights
            if (!wait(&bars[kSFull0 + t], j & 1, abort_flag)) return false;
            pa_tc::fence_after_sync();
            const uint32_t have = *const_cast<volatile int*>(&info.have[j % kInfo]);
            uint4 exps = make_uint4(0u, 0u, 0u, 0u);
            if constexpr (CODE) exps = *reinterpret_cast<const uint4*>(info.exps[j % kInfo]);
            // whether every row of the tile sees every key of the step (uniform)
            const int i0 = j * kStepBlks;
            const int f = keys.block(i0) * kBlk;
            const bool full = have == 0xffu && i0 >= keys.sb && f + kStep - 1 <= pa && f >= pb - (p.window - 1);
            float x[kStep];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32_at(tS + 32 * c, x + 32 * c);
            pa_tc::tmem_wait_ld();
            float kf[kStepBlks] = {}, ev[kStepBlks] = {};            // per-block score factor, value exponent
            if constexpr (CODE) {
#pragma unroll
                for (int b = 0; b < kStepBlks; ++b) {
                    const uint32_t w = b < 2 ? exps.x : b < 4 ? exps.y : b < 6 ? exps.z : exps.w, e = (w >> (16 * (b & 1))) & 0xffffu;
                    // (no smaller than 2^-126, so that masked scores of -inf stay that)
                    kf[b] = sl * pow2f(max(e_min, e & 0xff));
                    ev[b] = (e >> 8) ? static_cast<float>(static_cast<int>(e >> 8) - 127) : -INFINITY;
                }
            }
            if (!(sl > 0.f)) {                                       // fold a factor that is not positive in
#pragma unroll
                for (int i = 0; i < kStep; ++i) x[i] *= CODE ? kf[i / kBlk] : sl;
#pragma unroll
                for (int b = 0; b < kStepBlks; ++b) kf[b] = 1.f;
            }
            const float plain = sl > 0.f ? sl : 1.f;
            auto factor = [&](int b) { return CODE ? kf[b] : plain; };
            if (!full) {
#pragma unroll
                for (int b = 0; b < kStepBlks; ++b) {
                    const uint32_t bits = (have >> b) & 1 ? seen_bits(pos, keys.block(i0 + b) * kBlk, p.window, p.sinks) : 0u;
#pragma unroll
                    for (int i = 0; i < kBlk; ++i) x[kBlk * b + i] = (bits >> i) & 1 ? x[kBlk * b + i] : -INFINITY;
                }
            }
            float mx = -INFINITY, mo = -INFINITY;
#pragma unroll
            for (int b = 0; b < kStepBlks; ++b) {
                float bm = x[kBlk * b];
#pragma unroll
                for (int i = 1; i < kBlk; ++i) bm = fmaxf(bm, x[kBlk * b + i]);
                if constexpr (CODE) {
                    bm *= factor(b);
                    mo = fmaxf(mo, bm + ev[b]);
                }
                mx = fmaxf(mx, bm);
            }
            if constexpr (!CODE) mx *= plain;
            // raise the references when they are unset or far behind
            const bool up = mx > m_ref + 8.f;
            const float old_m = m_ref;
            if (up) {
                m_ref = mx;
                if (old_m != -INFINITY) l *= pa_dev::ex2(old_m - mx);
            }
            const float oref_old = CODE ? o_ref : old_m;
            const bool up_o = CODE ? mo - kLift > o_ref + kLag : up;
            if (CODE && up_o) o_ref = mo - kLift;
            const float oref_new = CODE ? o_ref : m_ref;
            if (__any_sync(0xffffffffu, up_o && oref_old != -INFINITY)) {
                // O holds the sums of all earlier steps, or since the last flush (S(j) is full: their MMAs are done)
                const float corr = up_o && oref_old != -INFINITY ? pa_dev::ex2(oref_old - oref_new) : 1.f;
#pragma unroll 1
                for (int cc = 0; cc < kD / 16; ++cc) {
                    float o[16];
                    tmem_ld16_at(tO + cc * 16, o);
                    pa_tc::tmem_wait_ld();
                    uint32_t y[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(o[i] * corr);
                    pa_tc::tmem_st16u(tO + cc * 16, y);
                }
            }
            const float ref = m_ref == -INFINITY ? 0.f : m_ref;
            const float oref = oref_new == -INFINITY ? 0.f : oref_new;
            // weights, 32 keys at a time: P over S, rounded parts in columns 0..63,
            // remainders in 64..127
            const uint64_t nref = pack2(-ref, -ref);
            uint64_t sum2 = 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int hb = 0; hb < 2; ++hb) {
                    const int b = 2 * c + hb;
                    const uint64_t fb = pack2(factor(b), factor(b));
                    // a weight's value factor; a power of two up to rounding of the references
                    const float vf = CODE ? pa_dev::ex2(fminf(ev[b] + ref - oref, 126.f)) : 1.f;
#pragma unroll
                    for (int i = 0; i < kBlk; i += 2) {
                        float w0, w1;
                        unpack2(fma2(pack2(x[kBlk * b + i], x[kBlk * b + i + 1]), fb, nref), w0, w1);
                        w0 = pa_dev::ex2(w0);
                        w1 = pa_dev::ex2(w1);
                        uint64_t w2 = pack2(w0, w1);
                        sum2 = add2(sum2, w2);
                        if constexpr (CODE) unpack2(mul2(w2, pack2(vf, vf)), w0, w1);
                        const int e = 8 * hb + i / 2;
                        hi[e] = CODE ? pa_dev::pack_f16(w0, w1) : pa_dev::pack_bf16(w0, w1);
                        if constexpr (PAIR)
                            lo[e] = CODE ? pa_dev::pack_f16(w0 - pa_dev::f16_lo(hi[e]), w1 - pa_dev::f16_hi(hi[e]))
                                         : pa_dev::pack_bf16(w0 - pa_dev::bf16_lo(hi[e]), w1 - pa_dev::bf16_hi(hi[e]));
                    }
                }
                pa_tc::tmem_st16u(tS + 16 * c, hi);
                if constexpr (PAIR) pa_tc::tmem_st16u(tS + 64 + 16 * c, lo);
            }
            float sum, sum1;
            unpack2(sum2, sum, sum1);
            sum += sum1;
            l += sum;
            pa_tc::tmem_wait_st();
            pa_tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) arrive(&bars[kPFull0 + t]);
            return true;
        };
        auto flush = [&]() {                                         // O, once S(j) is full: the sums of the steps since the last flush
            if (!wait(&bars[kSFull0 + t], j & 1, abort_flag)) return false;
            pa_tc::fence_after_sync();
            const float ref = CODE ? o_ref : m_ref;
            const unsigned long long place = own_place();
#pragma unroll 1
            for (int c = 0; c < kD; c += 32) {
                float o[32];
                tmem_ld32_at(tO + c, o);
                pa_tc::tmem_wait_ld();
                if (j > kFlush) add_totals(place, c, ref, o);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float4* const at = total_at(place, c / 4 + i);
                    if (row_ok) *at = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                }
                __syncwarp();                                        // (TMEM is read by whole warps)
            }
            t_ref = ref;
            return true;
        };
        while (ok && j < steps) {
            for (const int stop = PAIR ? min(steps, j + kFlush) : steps; ok && j < stop; j += ok) ok = step();
            if (PAIR && ok && j < steps) ok = flush();
        }
        if (ok && t < tiles && wait(&bars[kOFull], 0, abort_flag)) {
            pa_tc::fence_after_sync();
            if (PAIR && keys.nsteps > kFlush) {                      // the totals into O
                const unsigned long long place = own_place();
#pragma unroll 1
                for (int c = 0; c < kD; c += 32) {
                    float o[32];
                    tmem_ld32_at(tO + c, o);
                    pa_tc::tmem_wait_ld();
                    add_totals(place, c, CODE ? o_ref : m_ref, o);
                    __syncwarp();
                    pa_tc::tmem_st32(tO + c, o);
                }
                pa_tc::tmem_wait_st();
                __syncwarp();                                        // every total is read before results go there
            }
            float inv = l > 0.f ? p.v_scale / l : 0.f;
            if (CODE && l > 0.f) inv *= o_ref == -INFINITY ? 0.f : pa_dev::ex2(o_ref - m_ref);
            // each thread's row into the warp's part of the query tile (every QK^T is done), 16
            // bytes at a time and swizzled, then out two (bf16) or one row a warp, coalesced
            unsigned char* mine = base + kQOff + t * kTileBytes + (warp & 3) * 8192;
            const int rows0 = r_lo + t * kTile + (warp & 3) * 32;
            constexpr int kRowBytes = 256;                           // staged at a time: 128 bf16 or 64 fp32
            const int passes = p.out_bf16 ? 1 : 2;
#pragma unroll 1
            for (int ps = 0; ps < passes; ++ps) {
#pragma unroll 1
                for (int cc = 0; cc < (p.out_bf16 ? 8 : 4); ++cc) {
                    float o[16];
                    tmem_ld16_at(tO + ps * 64 + cc * 16, o);
                    pa_tc::tmem_wait_ld();
                    if (p.out_bf16) {
#pragma unroll
                        for (int i = 0; i < 16; i += 8)
                            *reinterpret_cast<uint4*>(mine + lane * kRowBytes + (((2 * cc + i / 8) ^ (lane & 15)) << 4)) =
                                make_uint4(pa_dev::pack_bf16(o[i] * inv, o[i + 1] * inv), pa_dev::pack_bf16(o[i + 2] * inv, o[i + 3] * inv),
                                           pa_dev::pack_bf16(o[i + 4] * inv, o[i + 5] * inv), pa_dev::pack_bf16(o[i + 6] * inv, o[i + 7] * inv));
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; i += 4)
                            *reinterpret_cast<float4*>(mine + lane * kRowBytes + (((4 * cc + i / 4) ^ (lane & 15)) << 4)) =
                                make_float4(o[i] * inv, o[i + 1] * inv, o[i + 2] * inv, o[i + 3] * inv);
                    }
                }
                __syncwarp();
                const int hi = lane >> 4, c = lane & 15;
                Row at(rows0 + hi, G);
#pragma unroll 8
                for (int i = 0; i < 16; ++i, at.skip2(G)) {
                    const int lr = 2 * i + hi;
                    const uint4 y = *reinterpret_cast<const uint4*>(mine + lr * kRowBytes + ((c ^ (lr & 15)) << 4));
                    if (at.r < rows_end) {
                        const size_t e = (static_cast<size_t>(q0 + at.tok) * p.Hq + static_cast<size_t>(h) * G + at.head) * kD;
                        if (p.out_bf16) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + e + 8 * c) = y;
                        else *reinterpret_cast<uint4*>(static_cast<float*>(p.out) + e + ps * 64 + 4 * c) = y;
                    }
                }
                __syncwarp();
            }
        } else if (t < tiles) {
            ok = false;
        }
    } else if (warp == 9) {
        // -------------------------------------------------- MMA issue
        // S(j) of a tile overwrites its P(j-1): the tensor core runs what one
        // thread issues in order, so issuing it behind that PV is enough
        ok = wait(&bars[kQFull], 0, abort_flag);
        auto qk = [&](int t, int j) {
            if (!pa_tc::elect_one()) return;
            const uint32_t q = sbase + kQOff + t * kTileBytes, k = sbase + kKOff + (j % kStages) * kTileBytes;
#pragma unroll
            for (int i = 0; i < kD / 16; ++i)
                pa_tc::mma_bf16(tmem + t * 128, pa_tc::sw128_desc(q + (i >> 2) * 16384 + (i & 3) * 32),
                                pa_tc::sw128_desc(k + (i >> 2) * 16384 + (i & 3) * 32), kIdesc, i > 0);
            pa_tc::commit(&bars[kSFull0 + t]);
            if (t == tiles - 1) pa_tc::commit(&bars[kKEmpty0 + j % kStages]);
        };
        auto k_ready = [&](int j) {
            return wait(&bars[kKFull0 + j % kStages], (j / kStages) & 1, abort_flag);
        };
        if (ok) ok = k_ready(0);
        pa_tc::fence_after_sync();
        if (ok)
            for (int t = 0; t < tiles; ++t) qk(t, 0);
        for (int j = 0; ok && j < keys.nsteps; ++j) {
            for (int t = 0; t < tiles; ++t) {
                if (!wait(&bars[kPFull0 + t], j & 1, abort_flag) ||
                    (t == 0 && !wait(&bars[kVFull0 + j % kStages], (j / kStages) & 1, abort_flag))) {
                    ok = false;
                    break;
                }
                pa_tc::fence_after_sync();
                if (pa_tc::elect_one()) {
                    const uint32_t v = sbase + kVOff + (j % kStages) * kTileBytes, o = tmem + 256 + t * 128;
#pragma unroll
                    for (int i = 0; i < kStepBlks; ++i) {
                        const uint64_t b = pa_tc::sw32_desc(v + i * 4096);           // block i's V^T
                        pa_tc::mma_bf16_ta(o, tmem + t * 128 + i * 8, b, kIdesc, (PAIR ? j % kFlush > 0 : j > 0) || i > 0);
                        if (PAIR) pa_tc::mma_bf16_ta(o, tmem + t * 128 + 64 + i * 8, b, kIdesc, true);
                    }
                    if (t == tiles - 1) pa_tc::commit(&bars[kVEmpty0 + j % kStages]);
                }
                __syncwarp();
                if (j + 1 < keys.nsteps) {
                    if (t == 0 && !k_ready(j + 1)) { ok = false; break; }
                    pa_tc::fence_after_sync();
                    qk(t, j + 1);
                }
            }
        }
        // the last commits: outputs are ready, and every MMA issued is complete
        // before TMEM is freed
        if (pa_tc::elect_one()) {
            if (ok) pa_tc::commit(&bars[kOFull]);
            pa_tc::commit(&bars[kDone]);
        }
        __syncwarp();
        pa_tc::mbar_wait(&bars[kDone], 0, kWaitLimit);
    } else if (!CODE && warp == 8) {
        // ------------------------------------------- loads, bf16 pools
        uint32_t k_fills = 0, v_fills = 0;
        const Seen seen(P0 + r_lo / G, P0 + (rows_end - 1) / G, p.window, p.sinks);
        uint32_t part_used = 0, part_ph = 0;                          // bit st: slot st had a step in part; parity of its next phase
        int ids = -1;
        for (int j = 0; ok && j < keys.nsteps; ++j) {
            if ((j & 3) == 0) {                                       // block ids of four steps
                const int i = j * kStepBlks + lane;
                ids = -1;
                if (i < keys.nv) {
                    const int x = __ldg(table + keys.block(i));
                    if (x >= 0 && x < p.num_blocks) ids = x;
                    else pa_dev::record_error(p.err, PA_ERR_BAD_BLOCK_ID);
                }
            }
            const int st = j % kStages;
            const uint32_t use = j / kStages;
            const int mine = __shfl_sync(0xffffffffu, ids, (j & 3) * kStepBlks + (lane & 7));
            const uint32_t have = __ballot_sync(0xffffffffu, mine >= 0) & 0xffu;
            if (use > 0 && !wait(&bars[kKEmpty0 + st], (use - 1) & 1, abort_flag)) { ok = false; break; }
            if (lane == 0) {
                *const_cast<volatile int*>(&info.have[j % kInfo]) = static_cast<int>(have);
                pa_tc::mbar_expect_tx(&bars[kKFull0 + st], __popc(have) * 4096);
            }
            __syncwarp();
            if (lane < kStepBlks && mine >= 0) {
                const uint32_t k = sbase + kKOff + st * kTileBytes + lane * 2048;
                const int y = (mine * Hkv + h) * kBlk;
                pa_tc::tma_load_2d(k, &kmap, 0, y, &bars[kKFull0 + st]);
                pa_tc::tma_load_2d(k + 16384, &kmap, 64, y, &bars[kKFull0 + st]);
            }
            ++k_fills;
            if (use > 0 && !wait(&bars[kVEmpty0 + st], (use - 1) & 1, abort_flag)) { ok = false; break; }
            unsigned char* vt = base + kVOff + st * kTileBytes;
            for (int b = 0; b < kStepBlks; ++b)
                if (!((have >> b) & 1))
                    for (int o = lane * 16; o < 4096; o += 512)
                        *reinterpret_cast<uint4*>(vt + b * 4096 + o) = make_uint4(0u, 0u, 0u, 0u);
            const bool some = !seen.all(keys, j);                     // (warp 10 finishes the step's values)
            const bool in_part = some && lane < kStepBlks && mine >= 0 &&
                                 seen.bits(keys.block(j * kStepBlks + lane) * kBlk) != 0xffffu;
            const uint32_t part = __ballot_sync(0xffffffffu, in_part);
            pa_tc::fence_smem_to_async();
            __syncwarp();
            if (lane == 0) {
                pa_tc::mbar_expect_tx(&bars[kVFull0 + st], __popc(have & ~part) * 4096);
                if (some) {
                    *const_cast<volatile int*>(&info.part[j % kInfo]) = static_cast<int>(part);
                    pa_tc::mbar_expect_tx(&bars[kPartFull0 + st], __popc(part) * 4096);
                }
            }
            __syncwarp();
            if (lane < kStepBlks && mine >= 0)
                pa_tc::tma_load_2d(sbase + kVOff + st * kTileBytes + lane * 4096, &vmap, 0, (mine * Hkv + h) * kD,
                                   in_part ? &bars[kPartFull0 + st] : &bars[kVFull0 + st]);
            if (some) {
                part_used |= 1u << st;
                part_ph ^= 1u << st;
            } else if (lane == 0) {
                arrive(&bars[kVFull0 + st]);
            }
            ++v_fills;
        }
        // copies in flight land before the shared memory goes
        for (int st = 0; st < kStages; ++st) {
            const uint32_t kn = (k_fills + kStages - 1 - st) / kStages, vn = (v_fills + kStages - 1 - st) / kStages;
            if (kn > 0) pa_tc::mbar_wait(&bars[kKFull0 + st], (kn - 1) & 1, kWaitLimit);
            if (vn > 0) pa_tc::mbar_wait(&bars[kVFull0 + st], (vn - 1) & 1, kWaitLimit);
            if ((part_used >> st) & 1) pa_tc::mbar_wait(&bars[kPartFull0 + st], ((part_ph >> st) & 1) ^ 1, kWaitLimit);
        }
    } else if (!CODE && warp == 10) {
        // ------------------------------- values that no row sees, bf16 pools
        // They must be finite (0 * Inf is NaN): of blocks that some row sees in part, the
        // positions that none sees become zero once the copies have landed.  (In the
        // copying warp, which then sends the next step's values later, it cost 2 % of a
        // prompt's time.)
        const Seen seen(P0 + r_lo / G, P0 + (rows_end - 1) / G, p.window, p.sinks);
        uint32_t ph = 0;                                              // bit st: parity of slot st's next phase
        for (int j = 0; j < keys.nsteps; ++j) {
            if (seen.all(keys, j)) continue;
            const int st = j % kStages;
            if (!wait(&bars[kPartFull0 + st], (ph >> st) & 1, abort_flag)) { ok = false; break; }
            ph ^= 1u << st;
            unsigned char* vt = base + kVOff + st * kTileBytes;
            for (uint32_t left = *const_cast<volatile int*>(&info.part[j % kInfo]); left; left &= left - 1) {
                const int b = __ffs(left) - 1;
                const uint32_t bits = seen.bits(keys.block(j * kStepBlks + b) * kBlk);
                for (int d = lane; d < kD; d += 32) {
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {                  // (the halves trade places: 32-byte swizzle)
                        uint4* q = reinterpret_cast<uint4*>(vt + b * 4096 + d * 32 + ((hf ^ ((d >> 2) & 1)) << 4));
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
            pa_tc::fence_smem_to_async();
            __syncwarp();
            if (lane == 0) arrive(&bars[kVFull0 + st]);
        }
    } else if (CODE && warp == 8) {
        // ------------------------------------------- copies, code pools
        // A step's codes by bulk copy (2 KB per block, K and V), K(j+1) as soon as K(j) has
        // been taken out, V likewise.  (Loads into the widening threads' registers, 32 KB
        // under way, were more than the L1 beside 193 KB of shared memory takes: issuing
        // them stalled for 3000 cycles a step.)
        // Blocks are looked up four steps at a time, one a lane, in stages that do not wait:
        // the next four's table entries at the first of four steps, their exponents at the
        // third.
        auto entry = [&](int j) {                                     // -2: no block there
            const int i = j * kStepBlks + lane;
            return i < keys.nv ? __ldg(table + keys.block(i)) : -2;
        };
        auto checked = [&](int x) {
            if (x >= 0 && x < p.num_blocks) return x;
            if (x != -2) pa_dev::record_error(p.err, PA_ERR_BAD_BLOCK_ID);
            return -1;
        };
        auto exponents = [&](int id) -> uint32_t {                    // (pools without scales: factors 1)
            return p.scales && id >= 0 ? __ldg(reinterpret_cast<const uint16_t*>(p.scales + (static_cast<size_t>(id) * Hkv + h) * 2)) : 0x7f7fu;
        };
        int raw_next = -2, ids = checked(entry(0)), ids_next = -1, fills_k = 0, fills_v = 0;
        uint32_t exps = exponents(ids), exps_next = 0x7f7fu;
        for (int j = 0; j < keys.nsteps; ++j) {
            int id[kStepBlks];
#pragma unroll
            for (int b = 0; b < kStepBlks; ++b) id[b] = __shfl_sync(0xffffffffu, ids, (j & 3) * kStepBlks + b);
            const uint32_t have = __ballot_sync(0xffffffffu, ids >= 0) >> (8 * (j & 3)) & 0xffu;
            auto copy = [&](const void* pool, int which) {
                if (pa_tc::elect_one()) {
                    pa_tc::mbar_expect_tx(&bars[kCodeFull0 + which], __popc(have) * 2048);
#pragma unroll
                    for (int b = 0; b < kStepBlks; ++b)
                        if (id[b] >= 0)
                            pa_tc::bulk_load(sbase + kCodeOff + which * kCodeBytes + b * 2048,
                                             static_cast<const unsigned char*>(pool) + (static_cast<size_t>(id[b]) * Hkv + h) * 2048,
                                             2048, &bars[kCodeFull0 + which]);
                }
                __syncwarp();
            };
            if (j > 0 && !wait(&bars[kCodeEmpty0], (j - 1) & 1, abort_flag)) { ok = false; break; }
            if (lane == 0) *const_cast<volatile int*>(&info.have[j % kInfo]) = static_cast<int>(have);
            if ((lane >> 3) == (j & 3)) info.exps[j % kInfo][lane & 7] = static_cast<uint16_t>(exps);
            __syncwarp();
            copy(p.k, 0);
            ++fills_k;
            if (j > 0 && !wait(&bars[kCodeEmpty1], (j - 1) & 1, abort_flag)) { ok = false; break; }
            copy(p.v, 1);
            ++fills_v;
            if ((j & 3) == 0) raw_next = entry(j + 4);
            if ((j & 3) == 2) {
                ids_next = checked(raw_next);
                exps_next = exponents(ids_next);
            }
            if ((j & 3) == 3) {
                ids = ids_next;
                exps = exps_next;
            }
        }
        // copies in flight land before the shared memory goes
        if (fills_k > 0) pa_tc::mbar_wait(&bars[kCodeFull0], (fills_k - 1) & 1, kWaitLimit);
        if (fills_v > 0) pa_tc::mbar_wait(&bars[kCodeFull1], (fills_v - 1) & 1, kWaitLimit);
    } else if (CODE && warp >= 12) {
        // -------------------------------------------- widening, code pools
        // thread ct takes 16 codes of each block: 16 of a key's 128, a value row's 16
        // tokens; once every warp has them in registers the copies go on
        fewer_registers<kRegsWiden>();
        const int ct = tid - 12 * 32;
        const Seen seen(P0 + r_lo / G, P0 + (rows_end - 1) / G, p.window, p.sinks);
        for (int j = 0; j < keys.nsteps; ++j) {
            const int st = j % kStages;
            const uint32_t use = j / kStages;
            uint4 c[kStepBlks];
            uint32_t have = 0;
            auto take = [&](int which) {
                if (!wait(&bars[kCodeFull0 + which], j & 1, abort_flag)) return false;
                have = *const_cast<volatile int*>(&info.have[j % kInfo]);
#pragma unroll
                for (int b = 0; b < kStepBlks; ++b)
                    c[b] = (have >> b) & 1 ? *reinterpret_cast<const uint4*>(base + kCodeOff + which * kCodeBytes + b * 2048 + ct * 16)
                                           : make_uint4(0u, 0u, 0u, 0u);     // code 0 is +0
                // the loads are done before the next copy, of another proxy, may write there: an
                // arrival alone does not order them (beside slow loads and stores of the weight
                // warps, some lanes then read the codes of the step after)
                pa_tc::fence_smem_to_async();
                __syncwarp();
                if (lane == 0) arrive(&bars[kCodeEmpty0 + which]);
                return true;
            };
            if (!take(0) || (use > 0 && !wait(&bars[kKEmpty0 + st], (use - 1) & 1, abort_flag))) { ok = false; break; }
            unsigned char* kt = base + kKOff + st * kTileBytes;
#pragma unroll
            for (int b = 0; b < kStepBlks; ++b) {
                const int key = b * kBlk + (ct >> 3), cc = 2 * (ct & 7);
                unsigned char* half = kt + (cc >> 3) * 16384;
                *reinterpret_cast<uint4*>(half + pa_tc::sw128_off(key, cc & 7)) = widen8(make_uint2(c[b].x, c[b].y));
                *reinterpret_cast<uint4*>(half + pa_tc::sw128_off(key, (cc & 7) + 1)) = widen8(make_uint2(c[b].z, c[b].w));
            }
            pa_tc::fence_smem_to_async();
            __syncwarp();
            if (lane == 0) arrive(&bars[kKFull0 + st]);
            if (!take(1) || (use > 0 && !wait(&bars[kVEmpty0 + st], (use - 1) & 1, abort_flag))) { ok = false; break; }
            unsigned char* vt = base + kVOff + st * kTileBytes;
            // positions that no row sees: zero codes (0 * NaN is NaN).  A step inside the
            // windows' union has none
            if (!seen.all(keys, j)) {
#pragma unroll
                for (int b = 0; b < kStepBlks; ++b) {
                    const uint32_t bits = seen.bits(keys.block(j * kStepBlks + b) * kBlk);
                    auto keep = [](uint32_t four) {                  // bit i -> byte i
                        return ((four & 1) | (four & 2) << 7 | (four & 4) << 14 | (four & 8) << 21) * 255u;
                    };
                    c[b] = make_uint4(c[b].x & keep(bits), c[b].y & keep(bits >> 4), c[b].z & keep(bits >> 8),
                                      c[b].w & keep(bits >> 12));
                }
            }
#pragma unroll
            for (int b = 0; b < kStepBlks; ++b) {
                unsigned char* rowp = vt + b * 4096 + ct * 32;
                const int flip = (ct >> 2) & 1;
                *reinterpret_cast<uint4*>(rowp + (flip << 4)) = widen8(make_uint2(c[b].x, c[b].y));
                *reinterpret_cast<uint4*>(rowp + ((flip ^ 1) << 4)) = widen8(make_uint2(c[b].z, c[b].w));
            }
            pa_tc::fence_smem_to_async();
            __syncwarp();
            if (lane == 0) arrive(&bars[kVFull0 + st]);
        }
    }
    if (!ok) {
        *abort_flag = 1;
        if (lane == 0) pa_dev::record_error(p.err, PA_ERR_CUDA);
    }
    pa_tc::fence_before_sync();
    __syncthreads();
    pa_tc::fence_after_sync();
    if (warp == 9) pa_tc::tmem_free<kTmemCols>(tmem);
}

}  // namespace

namespace pa_detail {

// bf16: 32-bit TMA coordinates (value rows num_blocks * Hkv * D); at most 65535 tiles
// a chunk (16.7 million rows), the grid's second dimension
bool window_prefill_tc_eligible(const pa_pool* pool, const WindowParams& p) {
    return pool->head_dim == kD && pool->block_size == kBlk && pool->dtype != PA_F32 &&
           (static_cast<int64_t>(p.max_q) * p.G + kRows - 1) / kRows <= 65535 &&
           static_cast<uint32_t>(pool->smem_optin) >= smem_bytes(true) && reinterpret_cast<uintptr_t>(p.out) % 16 == 0 &&
           (pool->dtype != PA_BF16 || static_cast<long long>(pool->num_blocks) * pool->kv_heads * kD < (1LL << 31));
}

int launch_window_prefill_tc(pa_pool* pool, const WindowParams& p, cudaStream_t st) {
    const bool code = is_code(pool->dtype);
    if (!code) {
        const int rc = ensure_tensor_maps(pool);
        if (rc != PA_OK) return rc;
    }
    auto kernel = code ? (p.out_bf16 ? window_prefill_kernel<true, false> : window_prefill_kernel<true, true>)
                       : (p.out_bf16 ? window_prefill_kernel<false, false> : window_prefill_kernel<false, true>);
    static std::atomic<uint64_t> done[4];
    if (!done[2 * code + (p.out_bf16 != 0)].load(std::memory_order_acquire)) {
        // the split of registers draws on what the block starts with: fewer, and the
        // warps that ask for more would wait for ever
        cudaFuncAttributes a;
        if (cudaFuncGetAttributes(&a, kernel) != cudaSuccess || a.numRegs < (code ? 128 : 168)) return PA_ERR_CUDA;
    }
    if (!allow_smem(kernel, pool->device, smem_bytes(code), done[2 * code + (p.out_bf16 != 0)])) return PA_ERR_CUDA;
    const dim3 grid(p.Hkv, static_cast<unsigned>((static_cast<int64_t>(p.max_q) * p.G + kRows - 1) / kRows), p.S);
    WindowParams q = p;
    // with windows much shorter than the contexts may be, tiles are about equally long and
    // the order is not worth its look-up (16 chunks, block-scaled, no window: 240 -> 217 us;
    // window 1024: 121 us either way)
    q.by_length = p.S > 1 && p.S <= kMaxSort && p.window > p.max_blocks * kBlk / 2;
    const cudaError_t e = launch_pdl(kernel, grid, dim3(code ? kThreadsCode : kThreadsBf16), smem_bytes(code), st, q,
                                     pool->kmap, pool->vmap);
    count_launch();
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa_detail
