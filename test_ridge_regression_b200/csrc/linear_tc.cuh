// Gated linear recurrence on the tensor cores: bf16 inputs, D = 32, 64 or 128.
//
// The same passes, with the same operands x, y, z, weights and dbeta terms, as on
// CUDA cores (linear_simt.cuh, which has the formulas); here a chunk is 128
// tokens and every product is tcgen05 with fp32 accumulators in TMEM:
//   P  [128 t][128 i] = X Y^T                      scores (both operands as loaded)
//   OI [128 t][64 z]  = (w . P)_hi,mid,lo Z        inside the chunk; w . P in TMEM
//   OS [128 t][64 z]  = X (S_hi + S_mid + S_lo)    against the state before the chunk
//   DS [128 y][64 z]  = Y^T (u Z)_hi,mid,lo        the chunk's increment
//   S' = b S + DS                                  fp32, in registers for the whole sequence
// A CTA owns 64 of z's columns for one head and one segment (a whole sequence where
// the heads alone fill the SMs); with D = 128 the two CTAs of a head read the same x
// and y, the second time from L2.  Heads of 32 and 64 columns take the same tiles:
// their boxes' missing columns read as zeros, the K steps and column halves beyond D
// are not issued.  (B8 H8 T2048 D64 took 345 us on CUDA cores, here 52.)
//
// Roundings.  bf16 inputs enter the products exactly.  The increments' weighted
// rows u z are split into three bf16 parts (24 bits: the state is an fp32 one, and
// final_state is an output).  The state read by OS is split into three too: an error of two
// parts, 2^-17 of the state, is more than the output's own rounding where a query reads
// something 2^9 times smaller than the rest of the state, and shows in dbeta and dgate, fp32
// outputs (1e-6 to 3e-6 off with two parts, 2e-7 to 8e-7 with three).  The weighted scores
// enter in three for the same reason: a write that the next token takes back leaves a
// difference of weights, which two parts hold to 2^-17 of either (one part is a rounding as large
// as the output's own).  What is left of the difference from fp32 arithmetic is the hardware's
// exponential (2^-22).  B8 H8 T2048 D128, kernel: state and scores in two parts 50 us, the
// state in three 54, both in three 56.  Rounded parts, not cut ones: cut, three hold an fp32
// number to the bit, but the aggregates took 152 us, not 136, and the passes as long.
//
// Roles (640 threads, one CTA an SM).  What follows at -> is a barrier and who waits:
//   warp 18      loads x (one stage), y (two) -> 17;  z (two) -> 17, 8-15;  decay tables (three)
//                -> 0-15
//   warp 17      x from shared memory to TMEM, P -> 0-7;  OI -> 0-7
//   warp 16      OS -> 0-7, 17;  DS -> 8-15
//   warps 0-7    P -> weighted scores in TMEM (thread: a token, 64 columns) -> 17;
//                a OS + OI -> rows staged where z was -> 19
//   warps 8-15   S as OS's operand -> 16;  two parts of u z -> 16;  once OS is done, the third,
//                which lies where the state's third was -> 16;  S' = b S + DS
//   warp 19      rows out by TMA, z's stage free again -> 18
// An operand's load is waited for by the issuer that reads it, or by a role whose arrival that
// issuer waits for: y by 17, whose copies of x 16 waits for; z by 17 itself, since the state's
// warps hand S over (and so let OS run) before they look at z.
// A barrier that some waiter could be two phases behind on has two copies.  Every wait
// is bounded and gives up once another role has; the issuers and the loader then drain
// what they have in flight, TMEM is freed and the device flag set.
//
// What decided the layout (cycles a chunk, B8 H8 T2048 D128, 1.9 GHz).
// - An MMA with both operands in shared memory and N = 128 leaves the warps no bandwidth
//   there: P took 1222.  X as a TMEM operand (copied once, used by P and OS) frees it.
// - Two parts of an operand are columns of one product (N = 128 for DS: y is read once); the
//   third, which comes later, is added to the second's columns.  All three parts of u z held
//   back until OS is done, in one product: 62 us, not 54.
// - Issuing an MMA costs 33 from a converged warp under elect_one, 70 to 200 otherwise,
//   hence a warp per queue and operand addresses that are constants.
// - Rows leave through shared memory and TMA: a thread's 32 bytes of a row, stored from
//   registers, are a pass of the memory pipe per row.
// - Loops stay rolled: unrolled, the roles' code no longer fits the instruction caches
//   together (no variant of it was faster).
// - With scores in two parts, sixteen warps for the outputs (registers split by role) were 7 %
//   slower, and rows formed one chunk late, under the next chunk's OI and P, 6 %.
// - OI begun on the first half of the scores while the second is formed: 5 % slower.
// What bounds it: several chains from chunk to chunk of one length, 4800 against 3500 of tensor
// work.  The outputs' warps: P (300 left to wait), scores (2200), OI (1500 with its hand-offs and
// the products queued before it), rows (650); the state's: its operand (650), OS with its
// hand-offs (2250, u z's first parts formed under it), the third part and DS (1700), sum (240).
// Loads, stores and hand-offs alone: 29 us of the kernel's 56 (the bytes 21.5 at the copy rate).
// No unit is full: tensor pipe 53 % active, issue slots 52 %, the warps' shared memory accesses
// 27 %, its banks 18 % reading and 12 % writing.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "linear_simt.cuh"
#include "ptx.cuh"
#include "state_tc.cuh"
#include "tcgen05.cuh"

namespace gka {

constexpr int kLtC = 128;                       // tokens per chunk
constexpr int kLtZN = 64;                       // columns of z a CTA owns
constexpr int kLtGroup = 256;                   // threads of an arithmetic group (two)
constexpr int kLtThreads = 2 * kLtGroup + 128;  // + two issuers, the loader, the rows' store
constexpr int kLtTabs = 3;                      // stages of decay tables
constexpr int kLtTabB = 10 * kLtC;              // a table's b
constexpr int kLtTabF = kLtTabB + 4;            // floats of a table
constexpr int kLtDots = 2, kLtFdots = 8;        // planes of dot and fdot partials per column split
constexpr uint32_t kLtProbes = 1u << 20;
constexpr uint32_t kLtHintNs = 2000;            // a probe suspends its warp for up to this long

struct LtSmem {
    static constexpr uint32_t TILE = kLtC * 256;          // [128][128] bf16, two column halves
    static constexpr uint32_t HALF = kLtC * 128;          // [128][64] bf16
    static constexpr uint32_t X = 0;
    static constexpr uint32_t Y = X + TILE;               // 2 stages
    static constexpr uint32_t Z = Y + 2 * TILE;           // 2 stages
    static constexpr uint32_t PARTS = Z + 2 * HALF;       // hi, mid, lo of u z
    static constexpr uint32_t SOP = PARTS + 3 * HALF;     // hi, mid of the state
    static constexpr uint32_t TAB = SOP + 2 * HALF;       // decay tables of the chunks in flight
    // table floats, 128 tokens each: a, u, l (of the row), ta, c[3], and g (backward) or m (l
    // less log2 of the gate, of the column; forward), what l and (forward) m are short of as
    // one float; then b
    static constexpr uint32_t BARS = TAB + kLtTabs * 4 * kLtTabF;
    static constexpr uint32_t TBASE = BARS + 8 * (21 + 2 * kLtTabs);      // TMEM base, abort flag
    static constexpr uint32_t END = TBASE + 16;
    static constexpr size_t bytes = END + 1024;
};

struct LinTcPass {
    // [B*H][T][D] bf16, boxes of 64 columns x 128 tokens of a head, 128B swizzle; tokens
    // past T and columns past D read as zeros and are not written
    CUtensorMap x, y, z, out;
    LinPass p;
    const float *tab;             // decay tables of the pass's direction
};
// Column splits of z, and the bytes of a tile of x or y: a head of 32 or 64 columns has one
// column half (32: the rest of its box reads as zeros).
__host__ __device__ __forceinline__ int lt_splits(int D) { return D > kLtZN ? D / kLtZN : 1; }
__device__ __forceinline__ uint32_t lt_tile_bytes(int D) { return D > 64 ? LtSmem::TILE : LtSmem::HALF; }
struct LinTcArgs {
    LinTcPass pass[2];
};

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int c0, int c1, int c2,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, int c0, int c1, int c2,
                                             const void *src) {
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
            reinterpret_cast<uint64_t>(map)),
        "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(src))
        : "memory");
}

// 128 rows x 32 bytes of a K-major operand (one K step) from shared memory to 8 TMEM columns.
__device__ __forceinline__ void cp_128x256b(uint32_t dst_tmem, uint64_t sdesc) {
    asm volatile("tcgen05.cp.cta_group::1.128x256b [%0], %1;" ::"r"(dst_tmem), "l"(sdesc) : "memory");
}
// One lane of the warp, always the same.  Issuing under it from a warp that runs the loop as
// a whole costs 33 cycles an MMA; under `lane == 0`, 70 to 200 (operands go through
// per-thread registers and a loop that makes them uniform).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(p));
    return p != 0;
}

// D[tmem] (+)= A[tmem] * B[smem]: A is bf16, two K elements to a 32-bit column.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                            uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}

// One probe of a barrier's phase (barriers are shared addresses here).
__device__ __forceinline__ bool lt_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(kLtHintNs)
        : "memory");
    return ok != 0;
}
// The rest of a bounded wait, which also gives up once another role has (the word at
// shared address `abort` set).
__device__ __noinline__ bool lt_wait_more(uint32_t bar, uint32_t parity, uint32_t abort) {
    for (uint32_t i = 0; i < kLtProbes; ++i) {
        if (lt_try(bar, parity)) return true;
        uint32_t a;
        asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(a) : "r"(abort) : "memory");
        if (a) break;
    }
    asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(abort), "r"(1u) : "memory");
    return false;
}
__device__ __forceinline__ bool lt_wait(uint32_t bar, uint32_t parity, uint32_t abort) {
    return lt_try(bar, parity) || lt_wait_more(bar, parity, abort);
}
// By a whole warp, with one outcome.
__device__ __forceinline__ bool lt_wait_warp(uint32_t bar, uint32_t parity, uint32_t abort) {
    if (__all_sync(0xffffffffu, lt_try(bar, parity))) return true;
    return __all_sync(0xffffffffu, lt_wait_more(bar, parity, abort)) != 0;
}
__device__ __forceinline__ void lt_bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}
// After a time-out: a bounded wait for work in flight.
__device__ __noinline__ void lt_drain(uint32_t bar, uint32_t parity) {
    for (uint32_t i = 0; i < kLtProbes; ++i)
        if (lt_try(bar, parity)) return;
}
__device__ __forceinline__ void lt_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void lt_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void lt_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void lt_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}

// Two bf16 as a pair of floats, a pair as two bf16, and what the rounding left.
__device__ __forceinline__ float2 bf16x2_f2(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }
__device__ __forceinline__ uint32_t f2_bf16x2(float2 y) { return bf16x2_bits(y.x, y.y); }
__device__ __forceinline__ float2 f2_rest(float2 y, uint32_t w) {
    return __ffma2_rn(bf16x2_f2(w), make_float2(-1.f, -1.f), y);
}
// Decay tables of every chunk, a warp each, into tab [B*H][N][kLtTabF] (LtSmem lists a table's
// parts).  A kernel of its own: formed by a warp of the passes, chunk by chunk, they took 4500
// to 6300 cycles a chunk (600 instructions that no cache held) and bounded those; this one is
// 3.5 us (B8 H8 T2048; 5 KB a chunk, latency), most of it under the set-up of the pass.
// Differences of logs within a block of 32 tokens are of pairs: as single floats they were up to
// 2^-17 off behind a reset in the block, 2^-12 behind thirty.
// grid B*H*N, block 32 (a small block fits beside a pass that is still running: 8 chunks a block
// were 1.3 to 2 us slower a call, all of them on the few SMs that the pass leaves free).  Lane l
// holds tokens 32 j + l.
template <bool REV>
__global__ void __launch_bounds__(32)
k_linear_tables(const float *__restrict__ beta, const float *__restrict__ gate, float *__restrict__ tab,
                int N, int T, float scale, float log2_min) {
    // once what came before is done, the pass after this one may begin: it reads that at once
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x;
    const unsigned c = blockIdx.x;
    const int bh = (int)(c / (unsigned)N), n = (int)(c - (unsigned)bh * (unsigned)N), t0 = n * kLtC + lane;
    const Log2Sum zero = {0.f, 0.f};
    float g[4];
    Log2Sum l[4], e[4], end = zero;   // e[b]: cumulative log at the end of block b
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const bool in = t0 + 32 * j < T;   // past the sequence's end: no decay, no write
        const size_t at = (size_t)bh * T + t0 + 32 * j;
        const float b = in ? beta[at] : 1.f;
        g[j] = in ? (gate ? gate[at] : 1.f) : 0.f;
        l[j] = {log2_decay(b, log2_min), 0.f};
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const Log2Sum y = {__shfl_up_sync(0xffffffffu, l[j].hi, o), __shfl_up_sync(0xffffffffu, l[j].lo, o)};
            if (lane >= o) l[j] = l[j] + y;
        }
    }
    Log2Sum lb[4];   // from the block's start
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const Log2Sum c2 = end + l[j];
        lb[j] = l[j];
        end = end + shfl(l[j], 31);
        l[j] = c2;
        e[j] = end;
    }
    float *ta = tab + (size_t)c * kLtTabF + lane;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float to = exp2_diff(l[j], zero), from = exp2_diff(end, l[j]);
        Log2Sum m = lb[j];
        if (!REV && gate)   // a closed gate's m, +inf, weighs 0
            m = g[j] == 0.f ? Log2Sum{INFINITY, 0.f} : m + Log2Sum{-log2f(g[j]), 0.f};
        const float v[10] = {
            REV ? from : scale * to,                       // a
            REV ? scale * to : g[j] * from,                // u
            lb[j].hi,                                      // l
            REV ? exp2_diff(e[j], l[j]) : exp2_diff(lb[j], zero),   // ta
            // c: forward, c[b] serves block row b + 1, the blocks before it; backward, block row
            // b, the blocks after it (0 elsewhere, where it is not read)
            (REV ? j > 0 : j <= 0) ? (REV ? exp2_diff(l[j], e[0]) : g[j] * exp2_diff(e[0], l[j])) : 0.f,
            (REV ? j > 1 : j <= 1) ? (REV ? exp2_diff(l[j], e[1]) : g[j] * exp2_diff(e[1], l[j])) : 0.f,
            (REV ? j > 2 : j <= 2) ? (REV ? exp2_diff(l[j], e[2]) : g[j] * exp2_diff(e[2], l[j])) : 0.f,
            REV ? g[j] : m.hi,                             // g, or m
            lb[j].lo, m.lo};
#pragma unroll
        for (int i = 0; i < (REV ? 9 : 10); ++i) ta[i * kLtC + 32 * j] = v[i];
    }
    if (lane < 4) ta[kLtTabB] = lane ? 0.f : ex2(end.hi + end.lo);   // b
}

// (u z) of item i (16 bytes of a row) in three bf16 parts: the first two stored 16 KB apart, the
// third returned.
__device__ __forceinline__ uint4 lt_parts(const uint8_t *z, uint8_t *dst, float u) {
    const uint4 w4 = *reinterpret_cast<const uint4 *>(z);
    const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
    uint32_t a[4], b[4], c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float2 y = __fmul2_rn(bf16x2_f2(w[e]), make_float2(u, u));
        a[e] = f2_bf16x2(y);
        y = f2_rest(y, a[e]);
        b[e] = f2_bf16x2(y);
        c[e] = f2_bf16x2(f2_rest(y, b[e]));
    }
    *reinterpret_cast<uint4 *>(dst) = make_uint4(a[0], a[1], a[2], a[3]);
    *reinterpret_cast<uint4 *>(dst + LtSmem::HALF) = make_uint4(b[0], b[1], b[2], b[3]);
    return make_uint4(c[0], c[1], c[2], c[3]);
}

// GRAD: the passes of the backward, which also keep the states and form dbeta's dots.
// B8 H8 T2048 D128: dq's pass 68 us, dv's and dk's 139 (256 CTAs, two waves on 148 SMs).
// grid (lt_splits(D) * passes, B*H, S), block kLtThreads.
template <bool REV, bool GRAD>
__global__ void __launch_bounds__(kLtThreads, 1)
k_linear_tc(const __grid_constant__ LinTcArgs args, int *__restrict__ timeout_flag) {
    using L = LtSmem;
    constexpr int C = kLtC;
    // the swizzled tiles start at the array's own 1024-byte boundary: operand addresses are
    // constants, which an MMA takes without a register (checked below)
    extern __shared__ __align__(1024) uint8_t lt_smem[];
    uint8_t *sm = lt_smem;
    const uint32_t sb = smem_u32(sm);
    const uint32_t bars = sb + L::BARS;
    const uint32_t b_p = bars, b_parts = bars + 8, b_s = bars + 16, b_pb = bars + 24, b_ds = bars + 32,
                   b_os = bars + 40, b_xfree = bars + 48, b_oi = bars + 56;
    const uint32_t b_xy = bars + 64, b_z = bars + 80, b_o = bars + 96, b_out = bars + 112,
                   b_fin = bars + 128;                                                        // [2]
    const uint32_t b_zfree = bars + 144;                                                      // [2]
    const uint32_t b_lo = bars + 160;
    const uint32_t b_w = bars + 168, b_tfree = b_w + 8 * kLtTabs;                             // [kLtTabs]
    uint32_t *tbase = reinterpret_cast<uint32_t *>(sm + L::TBASE);
    const uint32_t abort = sb + L::TBASE + 4;
    float *s_tab = reinterpret_cast<float *>(sm + L::TAB);
    const int ZS = lt_splits(args.pass[0].p.D);
    const LinTcPass &A = args.pass[blockIdx.x / ZS];
    const LinPass &p = A.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int zh = blockIdx.x % ZS, bh = blockIdx.y, seg = blockIdx.z, D = p.D;
    const uint32_t tile = lt_tile_bytes(D);   // of a tile of x or y in memory
    const int n0 = lin_seg(seg, p.S, p.N), n1 = lin_seg(seg + 1, p.S, p.N), NL = n1 - n0;
    auto chunk = [&](int it) { return REV ? n1 - 1 - it : n0 + it; };

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            lt_init(b_xy + 8 * i, 2);   // x's load and y's
            lt_init(b_z + 8 * i, 1);
            lt_init(b_o + 8 * i, 2);    // both issuers': every product of the chunk is done
            lt_init(b_out + 8 * i, 8);
            lt_init(b_zfree + 8 * i, 1);
            lt_init(b_fin + 8 * i, 1);
        }
        for (int i = 0; i < kLtTabs; ++i) {
            lt_init(b_w + 8 * i, 1);
            lt_init(b_tfree + 8 * i, 16);
        }
        lt_init(b_p, 1);
        lt_init(b_parts, 8);
        lt_init(b_lo, 8);
        lt_init(b_s, 16);   // S staged, and the last chunk's OS read
        lt_init(b_pb, 8);
        lt_init(b_ds, 1);
        lt_init(b_os, 1);
        lt_init(b_xfree, 1);
        lt_init(b_oi, 1);
        asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(abort), "r"(0u) : "memory");
        fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(tbase, 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    // all 512 columns: they begin at 0
    constexpr uint32_t tmem = 0;
    if (*tbase != tmem || (sb & 1023u)) {   // what the constants rest on; nothing is in flight yet
        if (tid == 0) atomicExch(timeout_flag, 1);
        __syncthreads();
        if (warp == 1) tc::tmem_dealloc(*tbase, 512);
        return;
    }
    // Launched as the tables' programmatic dependent, this kernel may read what was there before
    // those (x, y, z, beta) at once; the tables, the start states and the other direction's states
    // only after the wait (loader, state warps).
    griddep_launch_dependents();
    // TMEM columns; of the three bf16 parts of 16 weighted scores, two lie over those scores
    constexpr uint32_t kP = 0, kOI = 128, kOS = 192, kDS = 256, kPL = 384, kX = 448;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;              // TMEM lane: token of P, OI, OS; y row of S
    const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
    auto arrive = [&](uint32_t bar) {
        __syncwarp();
        if (lane == 0) lt_arrive(bar);
    };
    auto wait = [&](uint32_t bar, uint32_t parity) { return lt_wait_warp(bar, parity, abort); };
    constexpr uint32_t ID_P = tc::idesc_bf16(128, 128, false, false);
    constexpr uint32_t ID_O = tc::idesc_bf16(128, 64, false, true);
    constexpr uint32_t ID_D = tc::idesc_bf16(128, 128, true, true), ID_DL = tc::idesc_bf16(128, 64, true, true);
    // steps (in 16 bytes) from an operand's descriptor to its kk-th K step
    auto kmaj = [](int kk) { return (uint64_t)((kk >> 2) * (L::HALF / 16) + (kk & 3) * 2); };
    auto mnmaj = [](int kk) { return (uint64_t)(kk * 128); };

    if (warp == 16) {
        // ---- issuer of the state's products, OS and DS ----
        const uint64_t d_y = tc::sdesc(sb + L::Y, L::HALF, 1024), d_s = tc::sdesc(sb + L::SOP, L::HALF, 1024),
                       d_u = tc::sdesc(sb + L::PARTS, L::HALF, 1024);
        bool ok = true;
#pragma unroll 1
        for (int it = 0; it < NL; ++it) {
            const int st = it & 1, ph = it & 1;
            // x is in TMEM (and y in shared memory); the state operand is there and the last
            // chunk's OS has been read
            ok = wait(b_xfree, ph) && wait(b_s, ph);
            if (!ok) break;
            tc::fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < 16; ++kk)   // K steps against S_hi, then S_mid, 16 KB on
                    if ((kk & 7) * 16 < D)
                        mma_bf16_ta(tmem + kOS, tmem + kX + (kk & 7) * 8, d_s + mnmaj(kk), ID_O, kk > 0);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)   // and S_lo
                    if (kk * 16 < D)
                        mma_bf16_ta(tmem + kOS, tmem + kX + kk * 8, d_u + 2 * (L::HALF / 16) + mnmaj(kk), ID_O, true);
                lt_commit(b_os);
            }
            ok = wait(b_parts, ph);
            if (!ok) break;
            tc::fence_after_sync();
            if (elect_one()) {
                const uint64_t y = d_y + st * (L::TILE / 16);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    tc::mma_f16(tmem + kDS, y + mnmaj(kk), d_u + mnmaj(kk), ID_D, kk > 0);
            }
            ok = wait(b_lo, ph);
            if (!ok) break;
            tc::fence_after_sync();
            if (elect_one()) {   // the third part, onto the second's columns
                const uint64_t y = d_y + st * (L::TILE / 16);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    tc::mma_f16(tmem + kDS + 64, y + mnmaj(kk), d_u + 2 * (L::HALF / 16) + mnmaj(kk), ID_DL, true);
                lt_commit(b_ds);
                lt_commit(b_o + 8 * st);
            }
        }
        if (!ok && elect_one()) {   // a wait gave up: flag it, then drain this thread's products
            atomicExch(timeout_flag, 1);
            lt_commit(b_fin);
            lt_drain(b_fin, 0);
        }
        __syncwarp();
    } else if (warp == 17) {
        // ---- issuer of x's copies to TMEM, of the scores P and of OI ----
        const uint64_t d_x = tc::sdesc(sb + L::X, 16, 1024), d_y = tc::sdesc(sb + L::Y, 16, 1024),
                       d_z = tc::sdesc(sb + L::Z, L::HALF, 1024);
        // x(it) to TMEM, which frees its stage
        auto copy_x = [&](int it) {
            if (!wait(b_xy + 8 * (it & 1), (it >> 1) & 1)) return false;
            tc::fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    if (kk * 16 < D) cp_128x256b(tmem + kX + kk * 8, d_x + kmaj(kk));
                lt_commit(b_xfree);
            }
            return true;
        };
        auto issue_p = [&](int it) {
            if (elect_one()) {
                const uint64_t y = d_y + (it & 1) * (L::TILE / 16);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    if (kk * 16 < D) mma_bf16_ta(tmem + kP, tmem + kX + kk * 8, y + kmaj(kk), ID_P, kk > 0);
                lt_commit(b_p);
            }
        };
        bool ok = copy_x(0);
        if (ok) issue_p(0);
#pragma unroll 1
        for (int it = 0; ok && it < NL; ++it) {
            const int st = it & 1, ph = it & 1;
            // x of the next chunk once this one's OS and P have read it in TMEM, while the
            // weighted scores are formed
            if (it + 1 < NL) ok = wait(b_p, ph) && wait(b_os, ph) && copy_x(it + 1);
            ok = ok && wait(b_z + 8 * st, (it >> 1) & 1) && wait(b_pb, ph);
            if (!ok) break;
            tc::fence_after_sync();
            if (elect_one()) {
                const uint64_t z = d_z + st * (L::HALF / 16);
#pragma unroll
                for (int kk = 0; kk < 16; ++kk)   // the parts that lie over the scores, two for every 16
                    mma_bf16_ta(tmem + kOI, tmem + kP + kk * 8, z + mnmaj(kk >> 1), ID_O, kk > 0);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)    // and the third
                    mma_bf16_ta(tmem + kOI, tmem + kPL + kk * 8, z + mnmaj(kk), ID_O, true);
                lt_commit(b_oi);
                lt_commit(b_o + 8 * st);
            }
            // the next chunk's scores once OI has read the weighted ones, whose columns they take
            if (it + 1 < NL) {
                ok = wait(b_oi, ph);
                if (!ok) break;
                tc::fence_after_sync();
                issue_p(it + 1);
            }
        }
        if (!ok && elect_one()) {
            atomicExch(timeout_flag, 1);
            lt_commit(b_fin + 8);
            lt_drain(b_fin + 8, 0);
        }
        __syncwarp();
    } else if (warp == 18) {
        // ---- loads into freed stages ----
        if (lane == 0) {
            int loads_x = 0, loads_y = 0, loads_z = 0, loads_t = 0;   // begun
            auto load_x = [&](int it) {
                const int t0 = chunk(it) * C;
                lt_expect(b_xy + 8 * (it & 1), tile);
                tma_load_3d(sm + L::X, &A.x, 0, t0, bh, b_xy + 8 * (it & 1));
                if (D > 64) tma_load_3d(sm + L::X + L::HALF, &A.x, 64, t0, bh, b_xy + 8 * (it & 1));
                ++loads_x;
            };
            auto load_y = [&](int it) {
                const int st = it & 1, t0 = chunk(it) * C;
                lt_expect(b_xy + 8 * st, tile);
                tma_load_3d(sm + L::Y + st * L::TILE, &A.y, 0, t0, bh, b_xy + 8 * st);
                if (D > 64) tma_load_3d(sm + L::Y + st * L::TILE + L::HALF, &A.y, 64, t0, bh, b_xy + 8 * st);
                ++loads_y;
            };
            auto load_z = [&](int it) {
                const int st = it & 1;
                lt_expect(b_z + 8 * st, L::HALF);
                tma_load_3d(sm + L::Z + st * L::HALF, &A.z, zh * kLtZN, chunk(it) * C, bh, b_z + 8 * st);
                ++loads_z;
            };
            auto load_tab = [&](int it) {
                const int ts = it % kLtTabs;
                lt_expect(b_w + 8 * ts, 4 * kLtTabF);
                lt_bulk_load(sb + L::TAB + ts * 4 * kLtTabF, A.tab + ((size_t)bh * p.N + chunk(it)) * kLtTabF,
                             4 * kLtTabF, b_w + 8 * ts);
                ++loads_t;
            };
            load_x(0);
            load_y(0);
            load_z(0);
            if (NL > 1) {
                load_y(1);
                load_z(1);
            }
            griddep_wait();   // the tables' kernel is done
            for (int it = 0; it < kLtTabs && it < NL; ++it) load_tab(it);
            bool ok = true;
            if (NL > 1) {
                ok = lt_wait(b_xfree, 0, abort);
                if (ok) load_x(1);
            }
#pragma unroll 1
            for (int it = 0; ok && it + 2 < NL; ++it) {
                const int st = it & 1, ph2 = (it >> 1) & 1, ts = it % kLtTabs;
                ok = lt_wait(b_xfree, (it + 1) & 1, abort);   // x(it + 1) is in TMEM
                if (!ok) break;
                load_x(it + 2);
                ok = lt_wait(b_o + 8 * st, ph2, abort);       // y's readers are done
                if (!ok) break;
                load_y(it + 2);
                ok = lt_wait(b_zfree + 8 * st, ph2, abort);   // the rows that lay in z's place are out
                if (!ok) break;
                load_z(it + 2);
                if (it + kLtTabs < NL) {
                    ok = lt_wait(b_tfree + 8 * ts, (it / kLtTabs) & 1, abort);
                    if (!ok) break;
                    load_tab(it + kLtTabs);
                }
            }
            if (!ok) {   // a wait gave up: drain this thread's copies (chunk i's loads on barrier i & 1)
                for (int i = 0; i < 2; ++i) {
                    const int n = (min(loads_x, loads_y) + 1 - i) / 2, m = (loads_z + 1 - i) / 2;
                    if (n) lt_drain(b_xy + 8 * i, (n - 1) & 1);
                    if (m) lt_drain(b_z + 8 * i, (m - 1) & 1);
                }
                for (int i = 0; i < kLtTabs; ++i) {
                    const int n = (loads_t + kLtTabs - 1 - i) / kLtTabs;
                    if (n) lt_drain(b_w + 8 * i, (n - 1) & 1);
                }
                // a load whose barrier's other half was never begun: time for it to land
                if (loads_x != loads_y) __nanosleep(1000000);
            }
        }
        __syncwarp();
    } else if (warp == 19) {
        // ---- rows out ----
        if (lane == 0) {
#pragma unroll 1
            for (int it = 0; it < NL; ++it) {
                const int st = it & 1;
                if (!lt_wait(b_out + 8 * st, (it >> 1) & 1, abort)) break;
                tma_store_3d(&A.out, zh * kLtZN, chunk(it) * C, bh, sm + L::Z + st * L::HALF);
                tc::bulk_commit();
                tc::bulk_wait_read0();
                lt_arrive(b_zfree + 8 * st);
            }
            tc::bulk_wait0();
        }
        __syncwarp();
    } else if (warp < 8) {
        // ---- scores and outputs: thread has token `row`, 64 score columns, 32 of z ----
        {
            const int half = warp >> 2, z0 = zh * kLtZN + half * 32;
            arrive(b_s);   // no OS to read before the first
#pragma unroll 1
            for (int it = 0; it < NL; ++it) {
                const int sg = it & 1, ph = it & 1, ts = it % kLtTabs;
                const float *tab = s_tab + ts * kLtTabF;
                if (!wait(b_w + 8 * ts, (it / kLtTabs) & 1) || !wait(b_p, ph)) break;
                tc::fence_after_sync();
                // 16 columns at a time, in a loop: straight-line code for all of them would not
                // stay in the instruction caches.  Two of their parts take the columns that they were in.
#pragma unroll 1
                for (int h = 0; h < 4; ++h) {
                    const int c0 = half * 64 + h * 16, cb = c0 >> 5;
                    float pk[24];   // pairs of bf16 as 32-bit columns, then what their rounding left, twice
                    auto put = [&](int j, float2 x) {
#pragma unroll
                        for (int e = 0; e < 3; ++e) {
                            const uint32_t w = f2_bf16x2(x);
                            pk[8 * e + j] = __uint_as_float(w);
                            x = f2_rest(x, w);
                        }
                    };
                    if (REV ? cb < quarter : cb > quarter) {   // beyond the diagonal
#pragma unroll
                        for (int j = 0; j < 24; ++j) pk[j] = 0.f;
                    } else {
                        float v[16];
                        tc::tmem_ld16(tl + kP + c0, v);
                        if (cb == quarter) {
                            const float4 *w4 = reinterpret_cast<const float4 *>(tab + (REV ? 2 : 7) * C + c0);
                            const float4 *x4 = reinterpret_cast<const float4 *>(tab + (REV ? 8 : 9) * C + c0);
                            // 2^(l_t - l_i) (backward: its inverse) up to and including the token
                            // itself; l and what it is short of apart, so that differences keep their bits
                            const float sgn = REV ? 1.f : -1.f;
                            const float lt = -sgn * tab[2 * C + row], xt = -sgn * tab[8 * C + row];
                            const int first = lane - (h & 1) * 16;   // column of the token itself
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; j += 4) {
                                const float4 c4 = w4[j / 4], d4 = x4[j / 4];
#pragma unroll
                                for (int e = 0; e < 4; e += 2) {
                                    const float2 c = e ? make_float2(c4.z, c4.w) : make_float2(c4.x, c4.y);
                                    const float2 d = e ? make_float2(d4.z, d4.w) : make_float2(d4.x, d4.y);
                                    const float2 s2 = make_float2(sgn, sgn);
                                    const float2 l2 = __fadd2_rn(__ffma2_rn(c, s2, make_float2(lt, lt)),
                                                                 __ffma2_rn(d, s2, make_float2(xt, xt)));
                                    float2 w = __fmul2_rn(make_float2(ex2(l2.x), ex2(l2.y)),
                                                          make_float2(v[j + e], v[j + e + 1]));
                                    w.x = (REV ? j + e >= first : j + e <= first) ? w.x : 0.f;
                                    w.y = (REV ? j + e + 1 >= first : j + e + 1 <= first) ? w.y : 0.f;
                                    put((j + e) / 2, w);
                                }
                            }
                        } else {
                            const float4 *w4 = reinterpret_cast<const float4 *>(
                                tab + (4 + (REV ? quarter : quarter - 1)) * C + c0);
                            float2 rf;
                            rf.x = rf.y = tab[3 * C + row];
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; j += 4) {
                                const float4 c4 = w4[j / 4];
                                const float2 x = __fmul2_rn(__fmul2_rn(make_float2(c4.x, c4.y), rf),
                                                            make_float2(v[j], v[j + 1]));
                                const float2 y = __fmul2_rn(__fmul2_rn(make_float2(c4.z, c4.w), rf),
                                                            make_float2(v[j + 2], v[j + 3]));
                                put(j / 2, x);
                                put(j / 2 + 1, y);
                            }
                        }
                    }
                    tc::tmem_st16(tl + kP + c0, pk);
                    tc::tmem_st8(tl + kPL + c0 / 2, pk + 16);
                }
                tc::tmem_wait_st();
                tc::fence_before_sync();
                arrive(b_pb);

                const int t = chunk(it) * C + row;
                const size_t grow = (size_t)bh * p.T + t;
                const bool in = t < p.T;
                const bool dots = GRAD && p.dot && in;
                uint4 xd[4] = {};   // (in flight while the products run)
                if (dots && z0 < D) {
                    const uint4 *src = reinterpret_cast<const uint4 *>(
                        static_cast<const __nv_bfloat16 *>(p.xd) + grow * D + z0);
#pragma unroll
                    for (int j = 0; j < 4; ++j) xd[j] = __ldg(src + j);
                }
                const float a = tab[row], g = REV ? tab[7 * C + row] : 1.f;
                float d = 0.f;
                if (!wait(b_o + 8 * sg, (it >> 1) & 1)) break;
                tc::fence_after_sync();
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    float vs[16], vi[16];
                    tc::tmem_ld16(tl + kOS + half * 32 + h * 16, vs);
                    tc::tmem_ld16(tl + kOI + half * 32 + h * 16, vi);
                    tc::tmem_wait_ld();
                    if (h == 1) {
                        tc::fence_before_sync();
                        arrive(b_s);
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) vs[j] *= a;
                    if (dots) {
                        const uint4 x0 = h ? xd[2] : xd[0], x1 = h ? xd[3] : xd[1];
                        const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            d = fmaf(vs[2 * j], bf16_lo(w[j]), fmaf(vs[2 * j + 1], bf16_hi(w[j]), d));
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        vi[j] = fmaf(p.scale, vi[j], vs[j]) * g;
                    // staged where the chunk's z was (its last reader, OI, has completed)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        Vec16<__nv_bfloat16>::store(
                            reinterpret_cast<__nv_bfloat16 *>(
                                sm + L::Z + sg * L::HALF + row * 128 +
                                (((half * 4 + h * 2 + e) ^ (row & 7)) << 4)),
                            vi + 8 * e);
                }
                if (dots) p.dot[(size_t)(zh * 2 + half) * p.BH * p.T + grow] = d;
                fence_proxy_async_smem();
                arrive(b_out + 8 * sg);
                arrive(b_tfree + 8 * ts);
            }
        }
    } else {
        // ---- state: thread has y row `row`, 32 columns of z ----
        const int half = (warp >> 2) & 1, z0 = zh * kLtZN + half * 32, gt = tid - kLtGroup;
        const bool owns = row < D && z0 < D;   // else: nothing of the state in memory
        float st[32];
        // a state in memory: [y][z], or [z][y] (then lanes are neighbours)
        const int first = p.zy ? z0 * D + row : row * D + z0, step = p.zy ? D : 1;
#pragma unroll
        for (int j = 0; j < 32; ++j) st[j] = 0.f;
        griddep_wait();
        if (p.start && owns) {
            const float *src = p.start + ((size_t)bh * p.S + seg) * D * D + first;
#pragma unroll
            for (int j = 0; j < 32; ++j, src += step) st[j] = *src;
        }
        bool ok = true;
        for (int it = 0; it < NL; ++it) {
            const int sg = it & 1, ph = it & 1, ts = it % kLtTabs, n = chunk(it);
            const float *tab = s_tab + ts * kLtTabF;
            {
                // the state before the chunk as the B operand, rows of y, three bf16 parts
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t a[4], b[4], c[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float2 y = make_float2(st[h * 8 + 2 * e], st[h * 8 + 2 * e + 1]);
                        a[e] = f2_bf16x2(y);
                        y = f2_rest(y, a[e]);
                        b[e] = f2_bf16x2(y);
                        c[e] = f2_bf16x2(f2_rest(y, b[e]));
                    }
                    const uint32_t at = row * 128 + (((half * 4 + h) ^ (row & 7)) << 4);
                    *reinterpret_cast<uint4 *>(sm + L::SOP + at) = make_uint4(a[0], a[1], a[2], a[3]);
                    *reinterpret_cast<uint4 *>(sm + L::SOP + L::HALF + at) = make_uint4(b[0], b[1], b[2], b[3]);
                    // in the place of the third part of u z, which waits for OS
                    *reinterpret_cast<uint4 *>(sm + L::PARTS + 2 * L::HALF + at) = make_uint4(c[0], c[1], c[2], c[3]);
                }
                fence_proxy_async_smem();
                arrive(b_s);
            }
            ok = wait(b_w + 8 * ts, (it / kLtTabs) & 1) && wait(b_z + 8 * sg, (it >> 1) & 1);
            if (!ok) break;
            {
                uint4 lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int item = gt + i * kLtGroup;   // row item / 8
                    lo[i] = lt_parts(sm + L::Z + sg * L::HALF + item * 16, sm + L::PARTS + item * 16, tab[C + (item >> 3)]);
                }
                fence_proxy_async_smem();
                arrive(b_parts);
                ok = wait(b_os, ph);
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<uint4 *>(sm + L::PARTS + 2 * L::HALF + (gt + i * kLtGroup) * 16) = lo[i];
                fence_proxy_async_smem();
                arrive(b_lo);
            }
            const float b = tab[kLtTabB];
            if (GRAD && p.states && owns) {
                float *dst = p.states + ((size_t)bh * p.N + n) * D * D + (size_t)z0 * D + row;
#pragma unroll
                for (int j = 0; j < 32; ++j, dst += D) *dst = st[j];
            }
            if (GRAD && p.states_in) {
                float f = 0.f;
                if (owns) {
                    const float *src = p.states_in + ((size_t)bh * p.N + n) * D * D + (size_t)z0 * D + row;
#pragma unroll
                    for (int j = 0; j < 32; ++j, src += D) f = fmaf(st[j], __ldcs(src), f);
                }
                f = warp_sum(f);
                if (lane == 0) p.fdot[((size_t)(zh * 8 + warp - 8) * p.BH + bh) * p.N + n] = b * f;
            }
            // S' = b S + DS
            ok = wait(b_ds, ph);
            if (!ok) break;
            tc::fence_after_sync();
#pragma unroll
            for (int h = 0; h < 32; h += 16) {
                float v[16], w[16];
                tc::tmem_ld16(tl + kDS + 64 + half * 32 + h, v);
                tc::tmem_ld16(tl + kDS + half * 32 + h, w);
                tc::tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) st[h + j] = fmaf(b, st[h + j], w[j] + v[j]);
            }
            tc::fence_before_sync();
            arrive(b_tfree + 8 * ts);
        }
        if (ok && p.last && owns && seg == (REV ? 0 : p.S - 1)) {
            float *dst = p.last + (size_t)bh * D * D + first;
#pragma unroll
            for (int j = 0; j < 32; ++j, dst += step) *dst = st[j];
        }
    }
    // every product and copy has completed (the arithmetic warps waited for the last
    // chunk's; after a time-out their issuers drained them)
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

// Segment aggregates: a segment's increment from a zero state, its chunks taken from the end
// the state leaves by (the last chunk first, or in a backward pass the first), so that every
// weight is a product of decays down from one, A = sum u_i y_i z_i^T with
//   u_i = g_i prod_{m > i} beta_m   (backward: c prod_{m <= i} beta_m)
// over the segment (a chunk's u times the decay of the chunks between it and that end): one
// product per chunk into the same accumulators, with nothing of the state in between.  Warps
// 0-15 form the weighted rows (as in k_linear_tc), warp 16 issues, warp 18 loads.  B1 H8
// T131072 D128: 136 us for 538 MB (61 % of the copy rate); the parts (48 KB of shared
// memory written a chunk) and the product follow one another, 2400 cycles a chunk.
struct LaSmem {
    static constexpr int ST = 3;                                 // stages of loads
    static constexpr uint32_t Y = 0;
    static constexpr uint32_t Z = Y + ST * LtSmem::TILE;
    static constexpr uint32_t PARTS = Z + ST * LtSmem::HALF;     // hi, mid, lo
    static constexpr uint32_t U = PARTS + 3 * LtSmem::HALF;      // u, b
    static constexpr uint32_t BARS = U + ST * (4 * kLtC + 16);
    static constexpr uint32_t TBASE = BARS + 8 * (2 * ST + 2);
    static constexpr uint32_t END = TBASE + 16;
    static constexpr size_t bytes = END + 1024;
};

// grid (lt_splits(D), B*H, S), block kLtThreads.
template <bool REV>
__global__ void __launch_bounds__(kLtThreads, 1)
k_linear_agg_tc(const __grid_constant__ LinTcPass A, int *__restrict__ timeout_flag) {
    using L = LaSmem;
    constexpr int C = kLtC, ST = L::ST;
    extern __shared__ uint8_t smraw[];
    uint8_t *sm = smem_align1024(smraw);
    const uint32_t sb = smem_u32(sm), bars = sb + L::BARS;
    const uint32_t b_yz = bars, b_ds = bars + 8 * ST, b_parts = b_ds + 8 * ST, b_fin = b_parts + 8;   // [ST], [ST]
    uint32_t *tbase = reinterpret_cast<uint32_t *>(sm + L::TBASE);
    const uint32_t abort = sb + L::TBASE + 4;
    float *s_u = reinterpret_cast<float *>(sm + L::U);
    const LinPass &p = A.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int zh = blockIdx.x, bh = blockIdx.y, seg = blockIdx.z, D = p.D;
    if (seg == (REV ? 0 : p.S - 1)) return;   // never carried on
    const int n0 = lin_seg(seg, p.S, p.N), n1 = lin_seg(seg + 1, p.S, p.N), NL = n1 - n0;
    auto chunk = [&](int it) { return REV ? n0 + it : n1 - 1 - it; };
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            lt_init(b_yz + 8 * i, 1);
            lt_init(b_ds + 8 * i, 1);
        }
        lt_init(b_parts, 16);
        lt_init(b_fin, 1);
        asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(abort), "r"(0u) : "memory");
        fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(tbase, 256);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tbase;
    auto wait = [&](uint32_t bar, uint32_t parity) { return lt_wait_warp(bar, parity, abort); };
    // phase of chunk it on a barrier of ST: (it / ST) & 1; done(it): its product has completed
    auto done = [&](int it) { return wait(b_ds + 8 * (it % ST), (it / ST) & 1); };
    bool ok = true;

    if (warp == 16) {
        constexpr uint32_t ID_D = tc::idesc_bf16(128, 192, true, true);
        const uint64_t d_y = tc::sdesc(sb + L::Y, LtSmem::HALF, 1024),
                       d_u = tc::sdesc(sb + L::PARTS, LtSmem::HALF, 1024);
#pragma unroll 1
        for (int it = 0; it < NL; ++it) {
            const int st = it % ST;
            ok = wait(b_parts, it & 1);
            if (!ok) break;
            tc::fence_after_sync();
            if (elect_one()) {
                const uint64_t y = d_y + st * (LtSmem::TILE / 16);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    tc::mma_f16(tmem, y + kk * 128, d_u + kk * 128, ID_D, (it | kk) != 0);
                lt_commit(b_ds + 8 * st);
            }
        }
        if (!ok && elect_one()) {
            atomicExch(timeout_flag, 1);
            lt_commit(b_fin);
            lt_drain(b_fin, 0);
        }
        __syncwarp();
    } else if (warp == 18) {
        if (lane == 0) {
            int loads = 0;
#pragma unroll 1
            for (int it = 0; it < NL; ++it) {
                const int st = it % ST, t0 = chunk(it) * C;
                if (it >= ST) ok = lt_wait(b_ds + 8 * st, (it / ST - 1) & 1, abort);
                if (!ok) break;
                lt_expect(b_yz + 8 * st, lt_tile_bytes(D) + LtSmem::HALF + 4 * kLtC + 16);
                tma_load_3d(sm + L::Z + st * LtSmem::HALF, &A.z, zh * kLtZN, t0, bh, b_yz + 8 * st);
                tma_load_3d(sm + L::Y + st * LtSmem::TILE, &A.y, 0, t0, bh, b_yz + 8 * st);
                if (D > 64)
                    tma_load_3d(sm + L::Y + st * LtSmem::TILE + LtSmem::HALF, &A.y, 64, t0, bh, b_yz + 8 * st);
                if (it == 0) griddep_wait();   // the tables' kernel is done
                const float *tab = A.tab + ((size_t)bh * p.N + chunk(it)) * kLtTabF;
                lt_bulk_load(sb + L::U + st * (4 * kLtC + 16), tab + kLtC, 4 * kLtC, b_yz + 8 * st);
                lt_bulk_load(sb + L::U + st * (4 * kLtC + 16) + 4 * kLtC, tab + kLtTabB, 16, b_yz + 8 * st);
                ++loads;
            }
            if (!ok)
                for (int i = 0; i < ST; ++i)
                    if (loads > i) lt_drain(b_yz + 8 * i, ((loads - 1 - i) / ST) & 1);
        }
        __syncwarp();
    } else if (warp < 16) {
        float far = 1.f;   // decay of the chunks between this one and the segment's end
#pragma unroll 1
        for (int it = 0; it < NL; ++it) {
            const int st = it % ST;
            const float *u = s_u + st * (kLtC + 4);
            ok = wait(b_yz + 8 * st, (it / ST) & 1) && (it < 1 || done(it - 1));
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int item = tid + i * 512;   // row item / 8
                const uint4 lo = lt_parts(sm + L::Z + st * LtSmem::HALF + item * 16, sm + L::PARTS + item * 16,
                                          u[item >> 3] * far);
                *reinterpret_cast<uint4 *>(sm + L::PARTS + 2 * LtSmem::HALF + item * 16) = lo;
            }
            far *= u[kLtC];
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) lt_arrive(b_parts);
        }
        if (ok) ok = done(NL - 1);
        if (ok && tid == 0 && zh == 0) p.segdec[(size_t)bh * p.S + seg] = far;
        if (ok) {
            tc::fence_after_sync();
            const int quarter = warp & 3, cg = warp >> 2, row = quarter * 32 + lane, z0 = zh * kLtZN + cg * 16;
            const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16) + cg * 16;
            float v[16], w[16];
            tc::tmem_ld16(tl + 64, v);
            tc::tmem_ld16(tl + 128, w);
            tc::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] += w[j];
            tc::tmem_ld16(tl, w);
            tc::tmem_wait_ld();
            const size_t base = ((size_t)bh * p.S + seg) * D * D;
            if (row < D && z0 < D)
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    p.agg[base + (p.zy ? (size_t)(z0 + j) * D + row : (size_t)row * D + z0 + j)] = w[j] + v[j];
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 256);
    }
}

// ---------------------------------------------------------------------------
// dbeta and dgate of one 128-token chunk (k_linear_pairs on the tensor cores).
//
// The two score matrices are tcgen05 products of bf16 inputs (exact operands);
// weights, pairs and sums are fp32, with the cumulative logs as a sum of two
// floats so that differences after a reset keep fp32 precision.  q and k, then
// dout and v, go through the same 64 KB, which leaves room for two CTAs an SM (TMEM's
// limit too): one loads while the other computes.  B8 H8 T2048 D128: 38 us for 140 MB,
// bounded by a CTA's sequence of load, product and column sums (issue slots 33 %).
// grid (N, B*H), block 256: thread (quarter, lane, half) has row s = 32 quarter +
// lane and the 32-column blocks 2 half, 2 half + 1.
// ---------------------------------------------------------------------------
constexpr int kLpThreads = 256;

struct LpSmem {
    static constexpr uint32_t A = 0, B = LtSmem::TILE;       // q / dout, k / v
    static constexpr uint32_t LH = B + LtSmem::TILE;         // [128] high and low of l (log2)
    static constexpr uint32_t G = LH + 2 * 4 * kLtC;         // [128] gate
    static constexpr uint32_t RS = G + 4 * kLtC;             // [4][128] row sums of gated pairs
    static constexpr uint32_t CG = RS + 4 * 4 * kLtC;        // [4][128] column sums of pairs
    static constexpr uint32_t CX = CG + 4 * 4 * kLtC;        // [4][128] column sums of prefixes
    static constexpr uint32_t SC = CX + 4 * 4 * kLtC;        // scan scratch
    static constexpr uint32_t BARS = SC + 64;
    static constexpr uint32_t TBASE = BARS + 5 * 8;
    static constexpr uint32_t END = TBASE + 24;
    static constexpr size_t bytes = END + 1024;
};

struct LinPairsTc {
    CUtensorMap q, k, v, d_o;
    LinPairs p;
    int D;
};

// x[j] over the 32 lanes of a warp: lane j returns the sum of every lane's x[j].
__device__ __forceinline__ float column_sums(float *x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float send = up ? x[i] : x[i + o], keep = up ? x[i + o] : x[i];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    return x[0];
}

__global__ void __launch_bounds__(kLpThreads, 2)
k_linear_pairs_tc(const __grid_constant__ LinPairsTc args, int *__restrict__ timeout_flag) {
    using L = LpSmem;
    constexpr int C = kLtC;
    extern __shared__ uint8_t smraw[];
    uint8_t *sm = smem_align1024(smraw);
    const uint32_t sb = smem_u32(sm);
    const uint32_t bars = sb + L::BARS;   // load[2], mma[2], fin
    uint32_t *tbase = reinterpret_cast<uint32_t *>(sm + L::TBASE);
    const uint32_t abort = sb + L::TBASE + 4;
    float *s_lh = reinterpret_cast<float *>(sm + L::LH), *s_ll = s_lh + C;
    float *s_g = reinterpret_cast<float *>(sm + L::G), *s_rs = reinterpret_cast<float *>(sm + L::RS);
    float *s_cg = reinterpret_cast<float *>(sm + L::CG), *s_cx = reinterpret_cast<float *>(sm + L::CX);
    double *s_wl = reinterpret_cast<double *>(sm + L::SC);
    float *s_wz = reinterpret_cast<float *>(sm + L::SC + 32), *s_we = s_wz + 4;
    const LinPairs &p = args.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n = blockIdx.x, bh = blockIdx.y, t0 = n * C;
    const size_t head = (size_t)bh * p.T, all = (size_t)p.BH * p.T;

    if (tid == 0) {
        for (int i = 0; i < 5; ++i) lt_init(bars + 8 * i, 1);
        asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(abort), "r"(0u) : "memory");
        fence_mbar_init();
    }
    if (warp == 0) {
        tc::tmem_alloc(tbase, 256);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tbase;
    bool ok = true;
    if (tid == kLpThreads - 32) {   // warps 0-3 prepare the tokens meanwhile
        auto load = [&](const CUtensorMap *a, const CUtensorMap *b, uint32_t bar) {
            lt_expect(bar, 2 * lt_tile_bytes(args.D));
            for (int h = 0; h * 64 < args.D; ++h) {
                tma_load_3d(sm + L::A + h * LtSmem::HALF, a, h * 64, t0, bh, bar);
                tma_load_3d(sm + L::B + h * LtSmem::HALF, b, h * 64, t0, bh, bar);
            }
        };
        auto kmaj = [&](uint32_t base, int kk) {
            return tc::sdesc(sb + base + (kk >> 2) * LtSmem::HALF + (kk & 3) * 32, 16, 1024);
        };
        auto mma = [&](uint32_t col, uint32_t bar) {
            constexpr uint32_t ID = tc::idesc_bf16(128, 128, false, false);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                if (kk * 16 < args.D) tc::mma_f16(tmem + col, kmaj(L::A, kk), kmaj(L::B, kk), ID, kk > 0);
            lt_commit(bar);
        };
        load(&args.q, &args.k, bars + 8 * 0);
        ok = lt_wait(bars + 8 * 0, 0, abort);
        if (ok) {
            mma(0, bars + 8 * 2);
            ok = lt_wait(bars + 8 * 2, 0, abort);
        }
        if (ok) {
            load(&args.d_o, &args.v, bars + 8 * 1);
            ok = lt_wait(bars + 8 * 1, 0, abort);
            if (ok) mma(128, bars + 8 * 3);
        }
        if (!ok) {
            atomicExch(timeout_flag, 1);
            lt_commit(bars + 8 * 4);
            lt_drain(bars + 8 * 4, 0);
            lt_drain(bars + 8 * 1, 0);
            lt_drain(bars + 8 * 0, 0);
        }
    }
    __syncwarp();
    // tokens by threads 0..127: logs, gates, and the sums of zeta from and g eta before a token
    float eta = 0.f, zeta = 0.f, ge = 0.f, through = 0.f;
    if (tid < C) {
        griddep_wait();   // the passes are done (what came before them was, before the first began)
        if (lane < p.FS) through = p.fdot[((size_t)lane * p.BH + bh) * p.N + n];   // FS <= 32
        through = warp_sum(through);
        const int t = t0 + tid;
        float g = 0.f;
        double l = 0.0;
        if (t < p.T) {
            l = (double)log2_decay(p.beta[head + t], kLinLog2MinBwd);
            g = p.gate ? p.gate[head + t] : 1.f;
            for (int z = 0; z < p.ZS; ++z) {
                zeta += p.zeta[z * all + head + t];
                eta += p.eta[z * all + head + t];
            }
        }
        s_g[tid] = g;
        ge = g * eta;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, l, o);
            const float d = __shfl_up_sync(0xffffffffu, ge, o), u = __shfl_down_sync(0xffffffffu, zeta, o);
            if (lane >= o) {
                l += y;
                ge += d;
            }
            if (lane + o < 32) zeta += u;
        }
        if (lane == 31) {
            s_wl[warp] = l;
            s_we[warp] = ge;
        }
        if (lane == 0) s_wz[warp] = zeta;
        // exclusive: before this token
        ge = __shfl_up_sync(0xffffffffu, ge, 1);
        if (lane == 0) ge = 0.f;
        named_barrier_sync(1, C);
        for (int w = 0; w < 4; ++w) {
            if (w < warp) {
                l += s_wl[w];
                ge += s_we[w];
            }
            if (w > warp) zeta += s_wz[w];
        }
        s_lh[tid] = (float)l;
        s_ll[tid] = (float)(l - (double)(float)l);
    }
    __syncthreads();
    ok = lt_wait(bars + 8 * 3, 0, abort);
    ok = __syncthreads_and(ok);
    tc::fence_after_sync();
    const int quarter = warp & 3, half = warp >> 2, s = quarter * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
    if (ok) {
        const float lh = s_lh[s], ll = s_ll[s];
#pragma unroll 1
        for (int b = 0; b < 2; ++b) {
            const int cb = 2 * half + b;
            float rs = 0.f, cs = 0.f;
            if (cb <= quarter) {
                float a[32], v[16];
                tc::tmem_ld16(tl + cb * 32, a);
                tc::tmem_ld16(tl + cb * 32 + 16, a + 16);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    tc::tmem_ld16(tl + 128 + cb * 32 + h * 16, v);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int c = cb * 32 + h * 16 + j;
                        const float w = ex2((lh - s_lh[c]) + (ll - s_ll[c]));
                        float &x = a[h * 16 + j];
                        x = c <= s ? p.scale * w * x * v[j] : 0.f;
                        rs = fmaf(x, s_g[c], rs);
                    }
                }
                tc::tmem_st16(tl + cb * 32, a);
                tc::tmem_st16(tl + cb * 32 + 16, a + 16);
                tc::tmem_wait_st();
                cs = column_sums(a);
            }
            s_rs[cb * C + s] = rs;
            s_cg[quarter * C + cb * 32 + lane] = cs;
        }
    }
    __syncthreads();
    if (ok) {
#pragma unroll 1
        for (int b = 0; b < 2; ++b) {
            const int cb = 2 * half + b;
            float cs = 0.f;
            if (cb <= quarter) {
                float a[32], run = 0.f;
                tc::tmem_ld16(tl + cb * 32, a);
                tc::tmem_ld16(tl + cb * 32 + 16, a + 16);
                for (int e = 0; e < cb; ++e) run += s_rs[e * C + s];   // the blocks before
                tc::tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const int c = cb * 32 + j;   // column t: the gated pairs before it, if s >= t
                    const float x = a[j] * s_g[c];
                    a[j] = c <= s ? run : 0.f;
                    run += x;
                }
                cs = column_sums(a);
            }
            s_cx[quarter * C + cb * 32 + lane] = cs;
        }
    }
    __syncthreads();
    if (ok && tid < C && t0 + tid < p.T) {
        float d = zeta + ge + through, dg = eta;
        for (int q = 0; q < 4; ++q) {
            d += s_cx[q * C + tid];
            dg += s_cg[q * C + tid];
        }
        const float bt = fmaxf(p.beta[head + t0 + tid], 8.6736174e-19f);   // 2^-60
        p.dbeta[head + t0 + tid] = d / bt;
        if (p.dgate) p.dgate[head + t0 + tid] = dg;
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 256);
    }
}

}  // namespace gka
