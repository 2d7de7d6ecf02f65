// Gated linear recurrence on the tensor cores: bf16 inputs, D = 128.
//
// The same passes, with the same operands x, y, z, weights and dbeta terms, as on
// CUDA cores (linear_simt.cuh, which has the formulas); here a chunk is 128
// tokens and every product is tcgen05 with fp32 accumulators in TMEM:
//   P  [128 t][128 i] = X Y^T                      scores (both operands as loaded)
//   OI [128 t][64 z]  = (w . P) Z                  inside the chunk; w . P bf16 in TMEM
//   OS [128 t][64 z]  = X (S_hi + S_lo)            against the state before the chunk
//   DS [128 y][64 z]  = Y^T (u Z)_hi,mid,lo        the chunk's increment
//   S' = b S + DS                                  fp32, in registers for the whole sequence
// A CTA owns 64 of z's 128 columns for one head and one segment (a whole sequence
// where the heads alone fill the SMs), so that 64 heads make 128 CTAs for 148 SMs
// and the state takes 16 registers a thread; the two CTAs of a head read the same
// x and y, the second time from L2.
//
// Roundings.  bf16 inputs enter the products exactly.  The increments' weighted
// rows u z are split into three bf16 parts (24 bits: the state is an fp32 one, and
// final_state is an output), the state read by OS into two (16 bits, relative
// 2^-17), the weighted scores are rounded once to bf16 (as
// large as the output's own rounding and independent of it).
//
// Warps 0-15 (arithmetic): thread (quarter q, lane, group cg) owns TMEM lane
// 32 q + lane and a 16- or 32-column group cg.  Warp 16 issues TMA loads and MMAs;
// warp 17 forms each chunk's decay tables one chunk ahead.
//
// Decay weights.  exp(l_t - l_i) of a 32 x 32 block below the diagonal is the
// product of two factors at most 1, ta_t (from the block row's edge to t) and
// c_b,i (from i to that edge), both from differences in double: two vectors
// instead of 1024 exponentials, no overflow however strong the decay.  Only
// diagonal blocks evaluate exponentials, blocks beyond the diagonal are zero.
//
// Chunk n's steps, by role (-> barrier -> waiting role):
//   math: S operand(n) -> MMA OS(n);  parts(n) -> MMA DS(n);  P(n) -> weights ->
//         MMA OI(n);  S += DS(n);  OS, OI -> rows staged in shared memory -> TMA store
//   issuer: between them loads x(n + 1) once P(n) and OS(n) are done, y and z of
//         n + 2 once chunk n is, and issues P(n + 1) while OI(n) runs
// Shared memory's bandwidth is what the products compete for with the warps, so the
// parts of one operand are columns of one product (N = 192 for DS, 128 for OS: the
// other operand is read once) and their sums are taken in registers; rows leave
// through shared memory and TMA, since a thread's 32 bytes of a row, stored from
// registers, cost a pass of the memory pipe per row.
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
constexpr int kLtMath = 512;                    // arithmetic threads
constexpr int kLtThreads = kLtMath + 64;        // + issuer, decay warp
constexpr int kLtDots = 8, kLtFdots = 32;       // planes of dot and fdot partials per pass
constexpr uint32_t kLtProbes = 1u << 20;

struct LtSmem {
    static constexpr uint32_t TILE = kLtC * 256;          // [128][128] bf16, two column halves
    static constexpr uint32_t HALF = kLtC * 128;          // [128][64] bf16
    static constexpr uint32_t X = 0;
    static constexpr uint32_t Y = X + TILE;               // 2 stages
    static constexpr uint32_t Z = Y + 2 * TILE;           // 2 stages
    static constexpr uint32_t PARTS = Z + 2 * HALF;       // hi, mid, lo of u z
    static constexpr uint32_t SOP = PARTS + 3 * HALF;     // hi, lo of the state
    static constexpr uint32_t TAB = SOP + 2 * HALF;       // 2 x decay tables
    // table floats: a, u, g, lrel, ta, c[3] of 128 tokens each, then b
    static constexpr uint32_t TABF = 8 * kLtC + 4;
    static constexpr uint32_t BARS = TAB + 2 * 4 * TABF;
    static constexpr uint32_t TBASE = BARS + 8 * 22;      // TMEM base, abort flag
    static constexpr uint32_t END = TBASE + 16;
    static constexpr size_t bytes = END + 1024;
};

struct LinTcPass {
    // [B*H][T][128] bf16, boxes of 64 columns x 128 tokens of a head, 128B swizzle; tokens
    // past T read as zeros and are not written
    CUtensorMap x, y, z, out;
    LinPass p;
};
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

// Bounded wait that also gives up once another role has (the word at shared address
// `abort` set).  Barriers here are shared addresses: a register each, made where used.
__device__ __forceinline__ bool lt_wait(uint32_t bar, uint32_t parity, uint32_t abort) {
#pragma unroll 1
    for (uint32_t i = 0; i < kLtProbes; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((i & 255) == 255) {
            uint32_t a;
            asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(a) : "r"(abort) : "memory");
            if (a) break;
        }
    }
    asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(abort), "r"(1u) : "memory");
    return false;
}
// After a time-out: a bounded wait for work in flight.
__device__ __noinline__ void lt_drain(uint32_t bar, uint32_t parity) {
    for (uint32_t i = 0; i < kLtProbes; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return;
    }
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

// A sum of log decays as an unevaluated pair of floats (about 45 bits): differences of
// cumulative logs keep fp32 precision after a reset, at a fraction of the latency that
// doubles have on the one warp that forms the tables (1200 against 5400 cycles a chunk).
struct Log2Sum {
    float hi, lo;
};
__device__ __forceinline__ Log2Sum operator+(Log2Sum a, Log2Sum b) {
    const float s = a.hi + b.hi, t = s - a.hi;
    const float e = (a.hi - (s - t)) + (b.hi - t) + (a.lo + b.lo);
    const float h = s + e;
    return {h, e - (h - s)};
}
// 2^(a - b)
__device__ __forceinline__ float exp2_diff(Log2Sum a, Log2Sum b) {
    return exp2f((a.hi - b.hi) + (a.lo - b.lo));
}
__device__ __forceinline__ Log2Sum shfl(Log2Sum x, int src) {
    return {__shfl_sync(0xffffffffu, x.hi, src), __shfl_sync(0xffffffffu, x.lo, src)};
}

// Decay tables of one chunk by one warp; lane l holds tokens 4l..4l+3, whose beta and
// gate are bv and gv (1 and 0 past the sequence's end).  Returns the chunk's log2 decay.
template <bool REV>
__device__ __forceinline__ float lt_tables(float *tab, const float *bv, const float *gv, float scale,
                                           float log2_min) {
    const int lane = threadIdx.x & 31, blk = lane >> 3;
    float *ta_a = tab, *ta_u = tab + kLtC, *ta_g = tab + 2 * kLtC, *ta_l = tab + 3 * kLtC,
          *ta_t = tab + 4 * kLtC, *ta_c = tab + 5 * kLtC;
    const Log2Sum zero = {0.f, 0.f};
    Log2Sum l[4], run = zero;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        run = run + Log2Sum{fmaxf(log2f(bv[p]), log2_min), 0.f};
        l[p] = run;
    }
    Log2Sum incl = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Log2Sum y = {__shfl_up_sync(0xffffffffu, incl.hi, o), __shfl_up_sync(0xffffffffu, incl.lo, o)};
        if (lane >= o) incl = incl + y;
    }
    Log2Sum excl = {__shfl_up_sync(0xffffffffu, incl.hi, 1), __shfl_up_sync(0xffffffffu, incl.lo, 1)};
    if (lane == 0) excl = zero;
    Log2Sum edge[4];   // cumulative log at the end of block 0..3
#pragma unroll
    for (int b = 0; b < 4; ++b) edge[b] = shfl(incl, 8 * b + 7);
    const Log2Sum start = blk == 0 ? zero : blk == 1 ? edge[0] : blk == 2 ? edge[1] : edge[2];
    const Log2Sum stop = blk == 0 ? edge[0] : blk == 1 ? edge[1] : blk == 2 ? edge[2] : edge[3];
    float va[4], vu[4], vl[4], vt[4], vc[3][4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const Log2Sum lt = excl + l[p];
        va[p] = REV ? exp2_diff(edge[3], lt) : scale * exp2_diff(lt, zero);
        vu[p] = REV ? scale * exp2_diff(lt, zero) : gv[p] * exp2_diff(edge[3], lt);
        vl[p] = (lt.hi - start.hi) + (lt.lo - start.lo);
        vt[p] = REV ? scale * exp2_diff(stop, lt) : exp2f(vl[p]);
        // forward: c[b] serves block row b + 1, the blocks before it; backward: block row
        // b, the blocks after it (other entries are not read)
#pragma unroll
        for (int b = 0; b < 3; ++b)
            vc[b][p] = REV ? exp2_diff(lt, edge[b]) : gv[p] * exp2_diff(edge[b], lt);
    }
    auto put = [&](float *dst, const float *v) {
        *reinterpret_cast<float4 *>(dst + 4 * lane) = make_float4(v[0], v[1], v[2], v[3]);
    };
    put(ta_a, va);
    put(ta_u, vu);
    put(ta_g, gv);
    put(ta_l, vl);
    put(ta_t, vt);
#pragma unroll
    for (int b = 0; b < 3; ++b)
        if (REV ? blk > b : blk <= b) put(ta_c + b * kLtC, vc[b]);
    const float lC = edge[3].hi + edge[3].lo;
    if (lane == 0) tab[8 * kLtC] = exp2f(lC);
    return lC;
}

// grid (2 * passes, B*H, S), block kLtThreads.  OUT = false: segment aggregates.
template <bool REV, bool OUT>
__global__ void __launch_bounds__(256,1)
k_linear_tc(const __grid_constant__ LinTcArgs args, int *__restrict__ timeout_flag) {
    using L = LtSmem;
    constexpr int C = kLtC, D = 128;
    extern __shared__ uint8_t smraw[];
    uint8_t *sm = smem_align1024(smraw);
    const uint32_t sb = smem_u32(sm);
    const uint32_t bars = sb + L::BARS;
    const uint32_t b_x = bars, b_p = bars + 8, b_parts = bars + 16, b_s = bars + 24, b_pb = bars + 32,
                   b_ds = bars + 40, b_o = bars + 48, b_xfree = bars + 56, b_out = bars + 64,
                   b_ofree = bars + 72, b_fin = bars + 80;
    const uint32_t b_yz = bars + 88, b_w = bars + 104, b_tfree = bars + 120, b_quart = bars + 136;
    const uint32_t abort = sb + L::TBASE + 4;
    uint32_t *tbase = reinterpret_cast<uint32_t *>(sm + L::TBASE);
    float *s_tab = reinterpret_cast<float *>(sm + L::TAB);
    const LinTcPass &A = args.pass[blockIdx.x >> 1];
    const LinPass &p = A.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int zh = blockIdx.x & 1, bh = blockIdx.y, seg = blockIdx.z;
    const int n0 = lin_seg(seg, p.S, p.N), n1 = lin_seg(seg + 1, p.S, p.N), NL = n1 - n0;
    // the last segment's aggregate is never carried on
    if (!OUT && seg == (REV ? 0 : p.S - 1)) return;
    auto chunk = [&](int it) { return REV ? n1 - 1 - it : n0 + it; };

    if (tid == kLtMath) {
        for (int i = 0; i < 2; ++i) {
            lt_init(b_yz + 8 * i, 1);
            lt_init(b_w + 8 * i, 32);
            lt_init(b_tfree + 8 * i, 16);
        }
        lt_init(b_x, 1);
        lt_init(b_p, 1);
        lt_init(b_parts, 16);
        lt_init(b_s, 16);
        lt_init(b_pb, 16);
        lt_init(b_ds, 1);
        lt_init(b_o, 1);
        lt_init(b_xfree, 1);
        lt_init(b_out, 16);
        lt_init(b_ofree, 1);
        for (int i = 0; i < 4; ++i) lt_init(b_quart + 8 * i, 4);
        lt_init(b_fin, 1);
        asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(abort), "r"(0u) : "memory");
        fence_mbar_init();
    }
    __syncthreads();
    int loads_x = 0, loads_yz[2] = {0, 0};   // issuer: loads begun per barrier
    auto load_yz = [&](int it) {
        const int st = it & 1, t0 = chunk(it) * C;
        lt_expect(b_yz + 8 * st, L::TILE + L::HALF);
        tma_load_3d(sm + L::Y + st * L::TILE, &A.y, 0, t0, bh, b_yz + 8 * st);
        tma_load_3d(sm + L::Y + st * L::TILE + L::HALF, &A.y, 64, t0, bh, b_yz + 8 * st);
        tma_load_3d(sm + L::Z + st * L::HALF, &A.z, zh * kLtZN, t0, bh, b_yz + 8 * st);
        ++loads_yz[st];
    };
    auto load_x = [&](int it) {
        const int t0 = chunk(it) * C;
        lt_expect(b_x, L::TILE);
        tma_load_3d(sm + L::X, &A.x, 0, t0, bh, b_x);
        tma_load_3d(sm + L::X + L::HALF, &A.x, 64, t0, bh, b_x);
        ++loads_x;
    };
    if (tid == kLtMath) {
        load_yz(0);
        if (OUT) load_x(0);
        if (NL > 1) load_yz(1);
    }
    if (warp == 0) {
        tc::tmem_alloc(tbase, 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tbase;
    // TMEM columns; the bf16 weighted scores take the place of the scores
    constexpr uint32_t kP = 0, kPB = 0, kOI = 128, kOS = 192, kDS = 320;

    if (warp == 16) {
        if (lane == 0) {
            constexpr uint32_t ID_P = tc::idesc_bf16(128, 128, false, false);
            constexpr uint32_t ID_O = tc::idesc_bf16(128, 64, false, true);
            constexpr uint32_t ID_S = tc::idesc_bf16(128, 128, false, true);
            constexpr uint32_t ID_D = tc::idesc_bf16(128, 192, true, true);
            // first descriptors of an operand, opaque so that the eight K steps' are not kept
            // in registers across the loop, and the step to the kk-th
            auto first = [&](uint32_t base, uint32_t lbo) {
                uint64_t d = tc::sdesc(sb + base, lbo, 1024);
                asm volatile("" : "+l"(d));
                return d;
            };
            auto kmaj = [](int kk) { return (uint64_t)(((kk >> 2) * L::HALF + (kk & 3) * 32) >> 4); };
            auto mnmaj = [](int kk) { return (uint64_t)((kk * 2048) >> 4); };
            auto issue_p = [&](int it) {
                if (!lt_wait(b_x, it & 1, abort) || !lt_wait(b_yz + 8 * (it & 1), (it >> 1) & 1, abort))
                    return false;
                const uint64_t x = first(L::X, 16), y = first(L::Y + (it & 1) * L::TILE, 16);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    tc::mma_f16(tmem + kP, x + kmaj(kk), y + kmaj(kk), ID_P, kk > 0);
                lt_commit(b_p);
                return true;
            };
            bool ok = !OUT || issue_p(0);
            for (int it = 0; ok && it < NL; ++it) {
                const int st = it & 1, ph = it & 1;
                if (OUT) {
                    ok = lt_wait(b_s, ph, abort);
                    if (!ok) break;
                    tc::fence_after_sync();
                    const uint64_t x = first(L::X, 16), s = first(L::SOP, L::HALF);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        tc::mma_f16(tmem + kOS, x + kmaj(kk), s + mnmaj(kk), ID_S, kk > 0);
                    lt_commit(b_xfree);
                }
                ok = lt_wait(b_parts, ph, abort);
                if (!ok) break;
                tc::fence_after_sync();
                {
                    const uint64_t y = first(L::Y + st * L::TILE, L::HALF), u = first(L::PARTS, L::HALF);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        tc::mma_f16(tmem + kDS, y + mnmaj(kk), u + mnmaj(kk), ID_D, kk > 0);
                }
                lt_commit(b_ds);
                if (OUT) {
                    if (it + 1 < NL) {
                        ok = lt_wait(b_xfree, ph, abort);
                        if (!ok) break;
                        load_x(it + 1);
                    }
                    ok = lt_wait(b_pb, ph, abort);
                    if (!ok) break;
                    tc::fence_after_sync();
                    const uint64_t z = first(L::Z + st * L::HALF, L::HALF);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_bf16_ta(tmem + kOI, tmem + kPB + kk * 8, z + mnmaj(kk), ID_O, kk > 0);
                    lt_commit(b_o);
                    if (it + 1 < NL) ok = issue_p(it + 1);
                    if (ok && it + 2 < NL) {
                        ok = lt_wait(b_o, ph, abort);
                        if (ok) load_yz(it + 2);
                    }
                } else if (it + 2 < NL) {
                    ok = lt_wait(b_ds, ph, abort);
                    if (ok) load_yz(it + 2);
                }
            }
            if (!ok) {
                // a wait gave up: flag it, then drain this thread's products and copies
                atomicExch(timeout_flag, 1);
                lt_commit(b_fin);
                lt_drain(b_fin, 0);
                if (loads_x) lt_drain(b_x, (loads_x - 1) & 1);
                for (int i = 0; i < 2; ++i)
                    if (loads_yz[i]) lt_drain(b_yz + 8 * i, (loads_yz[i] - 1) & 1);
            }
        }
        __syncwarp();
    } else if (warp == 17) {
        const float *beta = p.beta + (size_t)bh * p.T;
        const float *gate = p.gate ? p.gate + (size_t)bh * p.T : nullptr;
        const float log2_min = (float)(p.log_min * 1.4426950408889634);
        float bv[4], gv[4];
        auto fetch = [&](int it) {
            const int t0 = chunk(it) * C + 4 * lane;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool in = t0 + j < p.T;
                bv[j] = in ? beta[t0 + j] : 1.f;
                gv[j] = in ? (gate ? gate[t0 + j] : 1.f) : 0.f;
            }
        };
        fetch(0);
        float seglog = 0.f;
        bool ok = true;
        // chunk it's output rows, staged by the arithmetic warps, on their way
        auto store_out = [&](int it) {
            bool done = lt_wait(b_out, it & 1, abort);
            if (lane == 0 && done) {
                tma_store_3d(&A.out, zh * kLtZN, chunk(it) * C, bh, sm + L::PARTS);
                tc::bulk_commit();
                tc::bulk_wait_read0();
                lt_arrive(b_ofree);
            }
            return __all_sync(0xffffffffu, done);
        };
        for (int it = 0; it < NL; ++it) {
            if (it >= 2) ok = __all_sync(0xffffffffu, lt_wait(b_tfree + 8 * (it & 1), ((it - 2) >> 1) & 1, abort));
            if (!ok) break;
            float cb[4], cg[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                cb[j] = bv[j];
                cg[j] = gv[j];
            }
            if (it + 1 < NL) fetch(it + 1);
            
            lt_arrive(b_w + 8 * (it & 1));
            if (OUT && it >= 1) ok = store_out(it - 1);
            if (!ok) break;
        }
        if (OUT && ok) store_out(NL - 1);
        if (lane == 0) tc::bulk_wait0();
        if (!OUT && ok && lane == 0 && blockIdx.x == 0)
            p.segdec[(size_t)bh * p.S + seg] = exp2f(seglog);
    } else {
        const int quarter = warp & 3, cg = warp >> 2;
        const int row = quarter * 32 + lane;              // TMEM lane: token of P, OI, OS; y row of S
        const int z0 = zh * kLtZN + cg * 16;              // this thread's columns of z
        const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
        float st[16];
        // a state in memory: [y][z], or [z][y] (then lanes are neighbours)
        auto at = [&](size_t base, int j) {
            return base + (p.zy ? (size_t)(z0 + j) * D + row : (size_t)row * D + z0 + j);
        };
#pragma unroll
        for (int j = 0; j < 16; ++j) st[j] = 0.f;
        if (OUT && p.start) {
            const size_t base = ((size_t)bh * p.S + seg) * D * D;
#pragma unroll
            for (int j = 0; j < 16; ++j) st[j] = p.start[at(base, j)];
        }
        auto arrive = [&](uint32_t bar) {
            __syncwarp();
            if (lane == 0) lt_arrive(bar);
        };
        bool ok = true;
        for (int it = 0; it < NL; ++it) {
            const int sg = it & 1, ph = it & 1, ph2 = (it >> 1) & 1, n = chunk(it);
            const float *tab = s_tab + sg * L::TABF;
            if (OUT) {
                // the state before the chunk as the B operand, rows of y, two bf16 parts
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t a[4], b[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float y0 = st[h * 8 + 2 * e], y1 = st[h * 8 + 2 * e + 1];
                        a[e] = bf16x2_bits(y0, y1);
                        b[e] = bf16x2_bits(y0 - bf16_lo(a[e]), y1 - bf16_hi(a[e]));
                    }
                    uint8_t *dst = sm + L::SOP + row * 128 + (((cg * 2 + h) ^ (row & 7)) << 4);
                    *reinterpret_cast<uint4 *>(dst) = make_uint4(a[0], a[1], a[2], a[3]);
                    *reinterpret_cast<uint4 *>(dst + L::HALF) = make_uint4(b[0], b[1], b[2], b[3]);
                }
                fence_proxy_async_smem();
                arrive(b_s);
            }
            ok = __all_sync(0xffffffffu,
                            lt_wait(b_w + 8 * sg, ph2, abort) && lt_wait(b_yz + 8 * sg, ph2, abort));
            if (!ok) break;
            // (u z) in three bf16 parts, at the places of z (and of the last chunk's staged rows)
            if (OUT && it >= 1) ok = __all_sync(0xffffffffu, lt_wait(b_ofree, (it - 1) & 1, abort));
            if (!ok) break;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t item = tid + j * kLtMath, off = item * 16;   // row item / 8
                const uint4 w4 = *reinterpret_cast<const uint4 *>(sm + L::Z + sg * L::HALF + off);
                const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
                const float u = tab[C + (item >> 3)];
                uint32_t a[4], b[4], c[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float y0 = u * bf16_lo(w[e]), y1 = u * bf16_hi(w[e]);
                    a[e] = bf16x2_bits(y0, y1);
                    y0 -= bf16_lo(a[e]);
                    y1 -= bf16_hi(a[e]);
                    b[e] = bf16x2_bits(y0, y1);
                    c[e] = bf16x2_bits(y0 - bf16_lo(b[e]), y1 - bf16_hi(b[e]));
                }
                uint8_t *dst = sm + L::PARTS + off;
                *reinterpret_cast<uint4 *>(dst) = make_uint4(a[0], a[1], a[2], a[3]);
                *reinterpret_cast<uint4 *>(dst + L::HALF) = make_uint4(b[0], b[1], b[2], b[3]);
                *reinterpret_cast<uint4 *>(dst + 2 * L::HALF) = make_uint4(c[0], c[1], c[2], c[3]);
            }
            fence_proxy_async_smem();
            arrive(b_parts);
            if (OUT) {
                if (p.states) {
                    float *dst = p.states + ((size_t)bh * p.N + n) * D * D + (size_t)z0 * D + row;
#pragma unroll
                    for (int j = 0; j < 16; ++j) dst[j * D] = st[j];
                }
                if (p.states_in) {
                    const float *src = p.states_in + ((size_t)bh * p.N + n) * D * D + (size_t)z0 * D + row;
                    float f = 0.f;
#pragma unroll
                    for (int j = 0; j < 16; ++j) f = fmaf(st[j], __ldcs(src + j * D), f);
                    f = warp_sum(f);
                    if (lane == 0)
                        p.fdot[((size_t)(zh * 16 + warp) * p.BH + bh) * p.N + n] = tab[8 * C] * f;
                }
                // weighted scores: columns 32 cg .. of token `row`
                const bool zero = REV ? cg < quarter : cg > quarter;
                float pk[16];   // pairs of bf16 as 32-bit columns
                ok = __all_sync(0xffffffffu, lt_wait(b_p, ph, abort));
                if (!ok) break;
                tc::fence_after_sync();
#pragma unroll
                for (int j = 0; j < 16; ++j) pk[j] = 0.f;
                if (!zero) {
                    // 16 columns at a time, so that the state's registers need not be spilled
#pragma unroll
                    for (int h = 0; h < 32; h += 16) {
                        const int c0 = cg * 32 + h;
                        float v[16];
                        tc::tmem_ld16(tl + kP + c0, v);
                        tc::tmem_wait_ld();
                        if (cg == quarter) {
                            const float lt = tab[3 * C + row];
#pragma unroll
                            for (int j = 0; j < 16; j += 4) {
                                const float4 l4 = *reinterpret_cast<const float4 *>(tab + 3 * C + c0 + j);
                                const float4 g4 = *reinterpret_cast<const float4 *>(tab + 2 * C + c0 + j);
                                const float li[4] = {l4.x, l4.y, l4.z, l4.w};
                                const float gi[4] = {g4.x, g4.y, g4.z, g4.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float d = lt - li[e], w = REV ? p.scale : gi[e];
                                    const bool in = REV ? h + j + e >= lane : h + j + e <= lane;
                                    v[j + e] = in ? v[j + e] * (w * exp2f(REV ? -d : d)) : 0.f;
                                }
                            }
                        } else {
                            const float ta = tab[4 * C + row];
                            const float *c = tab + (5 + (REV ? quarter : quarter - 1)) * C + c0;
#pragma unroll
                            for (int j = 0; j < 16; j += 4) {
                                const float4 c4 = *reinterpret_cast<const float4 *>(c + j);
                                v[j] *= ta * c4.x;
                                v[j + 1] *= ta * c4.y;
                                v[j + 2] *= ta * c4.z;
                                v[j + 3] *= ta * c4.w;
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            pk[h / 2 + j] = __uint_as_float(bf16x2_bits(v[2 * j], v[2 * j + 1]));
                    }
                }
                // the four warps of these lanes have their scores: the columns are free
                tc::fence_before_sync();
                arrive(b_quart + 8 * quarter);
                ok = __all_sync(0xffffffffu, lt_wait(b_quart + 8 * quarter, ph, abort));
                if (!ok) break;
                tc::fence_after_sync();
                tc::tmem_st16(tl + kPB + cg * 16, pk);
                tc::tmem_wait_st();
                tc::fence_before_sync();
                arrive(b_pb);
            }
            // S' = b S + DS
            ok = __all_sync(0xffffffffu, lt_wait(b_ds, ph, abort));
            if (!ok) break;
            tc::fence_after_sync();
            {
                float v[16], w[16];
                tc::tmem_ld16(tl + kDS + 64 + cg * 16, v);
                tc::tmem_ld16(tl + kDS + 128 + cg * 16, w);
                tc::tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] += w[j];
                tc::tmem_ld16(tl + kDS + cg * 16, w);
                tc::tmem_wait_ld();
                const float b = tab[8 * C];
#pragma unroll
                for (int j = 0; j < 16; ++j) st[j] = fmaf(b, st[j], w[j] + v[j]);
            }
            if (OUT) {
                const int t = n * C + row;
                const size_t grow = (size_t)bh * p.T + t;
                const bool in = t < p.T;
                uint4 xd[2] = {};
                if (p.dot && in) {
                    const uint4 *src = reinterpret_cast<const uint4 *>(
                        static_cast<const __nv_bfloat16 *>(p.xd) + grow * D + z0);
                    xd[0] = __ldg(src);
                    xd[1] = __ldg(src + 1);
                }
                const float a = tab[row], g = tab[2 * C + row];
                ok = __all_sync(0xffffffffu, lt_wait(b_o, ph, abort));
                if (!ok) break;
                tc::fence_after_sync();
                float vs[16], vi[16];
                tc::tmem_ld16(tl + kOS + cg * 16, vs);
                tc::tmem_ld16(tl + kOS + 64 + cg * 16, vi);
                tc::tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) vs[j] = a * (vs[j] + vi[j]);
                tc::tmem_ld16(tl + kOI + cg * 16, vi);
                float d = 0.f;
                if (p.dot) {
                    const uint32_t w[8] = {xd[0].x, xd[0].y, xd[0].z, xd[0].w,
                                           xd[1].x, xd[1].y, xd[1].z, xd[1].w};
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        d = fmaf(vs[2 * j], bf16_lo(w[j]), fmaf(vs[2 * j + 1], bf16_hi(w[j]), d));
                }
                tc::tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    vi[j] = REV ? g * (vs[j] + vi[j]) : fmaf(p.scale, vi[j], vs[j]);
                if (p.dot && in) p.dot[(size_t)(zh * 4 + cg) * p.BH * p.T + grow] = d;
                // staged where the increments' parts were (their product has completed)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    Vec16<__nv_bfloat16>::store(
                        reinterpret_cast<__nv_bfloat16 *>(sm + L::PARTS + row * 128 +
                                                          (((cg * 2 + h) ^ (row & 7)) << 4)),
                        vi + 8 * h);
                fence_proxy_async_smem();
                tc::fence_before_sync();
                arrive(b_out);
            }
            tc::fence_before_sync();
            arrive(b_tfree + 8 * sg);
        }
        float *dst = OUT ? (seg == (REV ? 0 : p.S - 1) ? p.last : nullptr) : p.agg;
        if (ok && dst) {
            const size_t base = OUT ? (size_t)bh * D * D : ((size_t)bh * p.S + seg) * D * D;
#pragma unroll
            for (int j = 0; j < 16; ++j) dst[at(base, j)] = st[j];
        }
    }
    // every product and copy has completed (the arithmetic warps waited for the last
    // chunk's; after a time-out the issuer drained them)
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// dbeta and dgate of one 128-token chunk (k_linear_pairs on the tensor cores).
//
// The two score matrices are tcgen05 products of bf16 inputs (exact operands);
// weights, pairs and sums are fp32, with the cumulative logs as a sum of two
// floats so that differences after a reset keep fp32 precision.  q and k, then
// dout and v, go through the same 64 KB, which leaves room for two CTAs an SM:
// one loads while the other computes.
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
    int FS;          // planes of fdot
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
            lt_expect(bar, 2 * LtSmem::TILE);
            for (int h = 0; h < 2; ++h) {
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
                tc::mma_f16(tmem + col, kmaj(L::A, kk), kmaj(L::B, kk), ID, kk > 0);
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
    float eta = 0.f, zeta = 0.f, ge = 0.f;
    if (tid < C) {
        const int t = t0 + tid;
        float g = 0.f;
        double l = 0.0;
        if (t < p.T) {
            l = (double)fmaxf(log2f(p.beta[head + t]), -60.f);
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
                        const float w = exp2f((lh - s_lh[c]) + (ll - s_ll[c]));
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
        float d = zeta + ge, dg = eta;
        for (int f = 0; f < args.FS; ++f) d += p.fdot[((size_t)f * p.BH + bh) * p.N + n];
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
