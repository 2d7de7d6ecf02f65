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
//   math: parts(n) -> MMA DS(n);  S operand(n) -> MMA OS(n);  P(n) -> weights ->
//         MMA OI(n);  S += DS(n);  OS, OI -> out rows
//   issuer: between them loads x(n + 1) once P(n) and OS(n) are done, y and z of
//         n + 2 once chunk n is, and issues P(n + 1) while OI(n) runs
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
    static constexpr uint32_t TBASE = BARS + 8 * 16;      // TMEM base, abort flag
    static constexpr uint32_t END = TBASE + 16;
    static constexpr size_t bytes = END + 1024;
};

struct LinTcPass {
    CUtensorMap x, y, z;          // [B*H][T][128] bf16, box 64 x 128 x 1, 128B swizzle, zero fill
    LinPass p;
};
struct LinTcArgs {
    LinTcPass pass[2];
};

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int c0, int c1, int c2,
                                            uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
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

// Bounded wait that also gives up once another role has (`abort` set).
__device__ __forceinline__ bool lt_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    for (uint32_t i = 0; i < kLtProbes; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 255) == 255 && *abort) break;
    }
    *abort = 1;
    return false;
}

// Decay tables of one chunk by one warp; lane l holds tokens 4l..4l+3, whose beta and
// gate are bv and gv (1 and 0 past the sequence's end).  Returns the chunk's log2 decay.
template <bool REV>
__device__ __forceinline__ double lt_tables(float *tab, const float *bv, const float *gv, float scale,
                                            float log2_min) {
    const int lane = threadIdx.x & 31, blk = lane >> 3;
    float *ta_a = tab, *ta_u = tab + kLtC, *ta_g = tab + 2 * kLtC, *ta_l = tab + 3 * kLtC,
          *ta_t = tab + 4 * kLtC, *ta_c = tab + 5 * kLtC;
    double l[4], run = 0.0;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        run += (double)fmaxf(log2f(bv[p]), log2_min);
        l[p] = run;
    }
    double incl = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    const double excl = incl - run, lC = __shfl_sync(0xffffffffu, incl, 31);
    double edge[5];   // cumulative log at the start of block 0..3 and at the end
    edge[0] = 0.0;
#pragma unroll
    for (int b = 1; b < 5; ++b) edge[b] = __shfl_sync(0xffffffffu, incl, 8 * b - 1);
    const double start = blk == 0 ? 0.0 : blk == 1 ? edge[1] : blk == 2 ? edge[2] : edge[3];
    const double stop = blk == 0 ? edge[1] : blk == 1 ? edge[2] : blk == 2 ? edge[3] : edge[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int t = 4 * lane + p;
        const double lt = excl + l[p];
        ta_a[t] = REV ? exp2f((float)(lC - lt)) : scale * exp2f((float)lt);
        ta_u[t] = REV ? scale * exp2f((float)lt) : gv[p] * exp2f((float)(lC - lt));
        ta_g[t] = gv[p];
        ta_l[t] = (float)(lt - start);
        ta_t[t] = REV ? scale * exp2f((float)(stop - lt)) : exp2f((float)(lt - start));
#pragma unroll
        for (int b = 0; b < 3; ++b) {
            // forward: c[b] serves block row b + 1, the blocks before it; backward: block
            // row b, the blocks after it
            if (REV ? blk > b : blk <= b)
                ta_c[b * kLtC + t] = REV ? exp2f((float)(lt - edge[b + 1]))
                                         : gv[p] * exp2f((float)(edge[b + 1] - lt));
        }
    }
    if (lane == 0) tab[8 * kLtC] = exp2f((float)lC);
    return lC;
}

// grid (2 * passes, B*H, S), block kLtThreads.  OUT = false: segment aggregates.
template <bool REV, bool OUT>
__global__ void __launch_bounds__(kLtThreads, 1)
k_linear_tc(const __grid_constant__ LinTcArgs args, int *__restrict__ timeout_flag) {
    using L = LtSmem;
    constexpr int C = kLtC, D = 128;
    extern __shared__ uint8_t smraw[];
    uint8_t *sm = smem_align1024(smraw);
    const uint32_t sb = smem_u32(sm);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BARS);
    uint64_t *b_yz = bars, *b_w = bars + 2, *b_tfree = bars + 4, *b_x = bars + 6, *b_p = bars + 7,
             *b_parts = bars + 8, *b_s = bars + 9, *b_pb = bars + 10, *b_ds = bars + 11, *b_o = bars + 12,
             *b_xfree = bars + 13, *b_fin = bars + 14;
    uint32_t *tbase = reinterpret_cast<uint32_t *>(sm + L::TBASE);
    volatile int *abort = reinterpret_cast<volatile int *>(sm + L::TBASE + 4);
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
            mbar_init(&b_yz[i], 1);
            mbar_init(&b_w[i], 32);
            mbar_init(&b_tfree[i], 16);
        }
        mbar_init(b_x, 1);
        mbar_init(b_p, 1);
        mbar_init(b_parts, 16);
        mbar_init(b_s, 16);
        mbar_init(b_pb, 16);
        mbar_init(b_ds, 1);
        mbar_init(b_o, 1);
        mbar_init(b_xfree, 1);
        mbar_init(b_fin, 1);
        *abort = 0;
        fence_mbar_init();
    }
    __syncthreads();
    int loads_x = 0, loads_yz[2] = {0, 0};   // issuer: loads begun per barrier
    auto load_yz = [&](int it) {
        const int st = it & 1, t0 = chunk(it) * C;
        mbar_arrive_expect_tx(&b_yz[st], L::TILE + L::HALF);
        tma_load_3d(sm + L::Y + st * L::TILE, &A.y, 0, t0, bh, &b_yz[st]);
        tma_load_3d(sm + L::Y + st * L::TILE + L::HALF, &A.y, 64, t0, bh, &b_yz[st]);
        tma_load_3d(sm + L::Z + st * L::HALF, &A.z, zh * kLtZN, t0, bh, &b_yz[st]);
        ++loads_yz[st];
    };
    auto load_x = [&](int it) {
        const int t0 = chunk(it) * C;
        mbar_arrive_expect_tx(b_x, L::TILE);
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
    constexpr uint32_t kP = 0, kOI = 128, kOS = 192, kDS = 256, kPB = 320;   // TMEM columns

    if (warp == 16) {
        if (lane == 0) {
            constexpr uint32_t ID_P = tc::idesc_bf16(128, 128, false, false);
            constexpr uint32_t ID_O = tc::idesc_bf16(128, 64, false, true);
            constexpr uint32_t ID_D = tc::idesc_bf16(128, 64, true, true);
            auto kmaj = [&](uint32_t base, int kk) {
                return tc::sdesc(sb + base + (kk >> 2) * L::HALF + (kk & 3) * 32, 16, 1024);
            };
            auto mnmaj = [&](uint32_t base, int kk) {
                return tc::sdesc(sb + base + kk * 2048, L::HALF, 1024);
            };
            auto issue_p = [&](int it) {
                if (!lt_wait(b_x, it & 1, abort) || !lt_wait(&b_yz[it & 1], (it >> 1) & 1, abort))
                    return false;
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    tc::mma_f16(tmem + kP, kmaj(L::X, kk), kmaj(L::Y + (it & 1) * L::TILE, kk), ID_P,
                                kk > 0);
                tc::commit(b_p);
                return true;
            };
            bool ok = !OUT || issue_p(0);
            for (int it = 0; ok && it < NL; ++it) {
                const int st = it & 1, ph = it & 1;
                ok = lt_wait(b_parts, ph, abort);
                if (!ok) break;
                tc::fence_after_sync();
#pragma unroll
                for (int q = 0; q < 3; ++q)
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        tc::mma_f16(tmem + kDS, mnmaj(L::Y + st * L::TILE, kk),
                                    mnmaj(L::PARTS + q * L::HALF, kk), ID_D, (q | kk) != 0);
                tc::commit(b_ds);
                if (OUT) {
                    ok = lt_wait(b_s, ph, abort);
                    if (!ok) break;
                    tc::fence_after_sync();
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            tc::mma_f16(tmem + kOS, kmaj(L::X, kk), mnmaj(L::SOP + q * L::HALF, kk), ID_O,
                                        (q | kk) != 0);
                    tc::commit(b_xfree);
                    if (it + 1 < NL) {
                        ok = lt_wait(b_xfree, ph, abort);
                        if (!ok) break;
                        load_x(it + 1);
                    }
                    ok = lt_wait(b_pb, ph, abort);
                    if (!ok) break;
                    tc::fence_after_sync();
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_bf16_ta(tmem + kOI, tmem + kPB + kk * 8, mnmaj(L::Z + st * L::HALF, kk), ID_O,
                                    kk > 0);
                    tc::commit(b_o);
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
                tc::commit(b_fin);
                mbar_wait_bounded(b_fin, 0, kLtProbes);
                if (loads_x) mbar_wait_bounded(b_x, (loads_x - 1) & 1, kLtProbes);
                for (int i = 0; i < 2; ++i)
                    if (loads_yz[i]) mbar_wait_bounded(&b_yz[i], (loads_yz[i] - 1) & 1, kLtProbes);
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
        double seglog = 0.0;
        bool ok = true;
        for (int it = 0; it < NL; ++it) {
            if (it >= 2) ok = __all_sync(0xffffffffu, lt_wait(&b_tfree[it & 1], ((it - 2) >> 1) & 1, abort));
            if (!ok) break;
            float cb[4], cg[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                cb[j] = bv[j];
                cg[j] = gv[j];
            }
            if (it + 1 < NL) fetch(it + 1);
            seglog += lt_tables<REV>(s_tab + (it & 1) * L::TABF, cb, cg, p.scale, log2_min);
            mbar_arrive(&b_w[it & 1]);
        }
        if (!OUT && ok && lane == 0 && blockIdx.x == 0)
            p.segdec[(size_t)bh * p.S + seg] = exp2f((float)seglog);
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
        bool ok = true;
        for (int it = 0; it < NL; ++it) {
            const int sg = it & 1, ph = it & 1, ph2 = (it >> 1) & 1, n = chunk(it);
            const float *tab = s_tab + sg * L::TABF;
            auto arrive = [&](uint64_t *bar) {
                __syncwarp();
                if (lane == 0) mbar_arrive(bar);
            };
            ok = __all_sync(0xffffffffu,
                            lt_wait(&b_w[sg], ph2, abort) && lt_wait(&b_yz[sg], ph2, abort));
            if (!ok) break;
            // (u z) in three bf16 parts, at the places of z
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
                if (p.states) {
                    float *dst = p.states + ((size_t)bh * p.N + n) * D * D;
#pragma unroll
                    for (int j = 0; j < 16; ++j) dst[at(0, j)] = st[j];
                }
                if (p.states_in) {
                    const float *src = p.states_in + ((size_t)bh * p.N + n) * D * D;
                    float f = 0.f;
#pragma unroll
                    for (int j = 0; j < 16; ++j) f = fmaf(st[j], src[at(0, j)], f);
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
                if (zero) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) pk[j] = 0.f;
                } else {
                    float v[32];
                    tc::tmem_ld16(tl + kP + cg * 32, v);
                    tc::tmem_ld16(tl + kP + cg * 32 + 16, v + 16);
                    tc::tmem_wait_ld();
                    if (cg == quarter) {
                        const float lt = tab[3 * C + row];
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const float d = lt - tab[3 * C + cg * 32 + j];
                            const float w = REV ? p.scale : tab[2 * C + cg * 32 + j];
                            const bool in = REV ? j >= lane : j <= lane;
                            v[j] = in ? v[j] * (w * exp2f(REV ? -d : d)) : 0.f;
                        }
                    } else {
                        const float ta = tab[4 * C + row];
                        const float *c = tab + (5 + (REV ? quarter : quarter - 1)) * C + cg * 32;
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] *= ta * c[j];
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        pk[j] = __uint_as_float(bf16x2_bits(v[2 * j], v[2 * j + 1]));
                }
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
                float v[16];
                tc::tmem_ld16(tl + kDS + cg * 16, v);
                tc::tmem_wait_ld();
                const float b = tab[8 * C];
#pragma unroll
                for (int j = 0; j < 16; ++j) st[j] = fmaf(b, st[j], v[j]);
            }
            if (OUT) {
                const int t = n * C + row;
                const size_t grow = (size_t)bh * p.T + t;
                const bool in = t < p.T;
                float xd[16];
                if (p.dot && in) {
                    const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(p.xd) + grow * D + z0;
                    Vec16<__nv_bfloat16>::load(src, xd);
                    Vec16<__nv_bfloat16>::load(src + 8, xd + 8);
                }
                const float a = tab[row], g = tab[2 * C + row];
                ok = __all_sync(0xffffffffu, lt_wait(b_o, ph, abort));
                if (!ok) break;
                tc::fence_after_sync();
                float vs[16], vi[16];
                tc::tmem_ld16(tl + kOS + cg * 16, vs);
                tc::tmem_ld16(tl + kOI + cg * 16, vi);
                tc::tmem_wait_ld();
                float d = 0.f;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    vs[j] *= a;
                    if (p.dot && in) d = fmaf(vs[j], xd[j], d);
                    vi[j] = REV ? g * (vs[j] + vi[j]) : fmaf(p.scale, vi[j], vs[j]);
                }
                if (in) {
                    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + grow * D + z0;
                    Vec16<__nv_bfloat16>::store(o, vi);
                    Vec16<__nv_bfloat16>::store(o + 8, vi + 8);
                    if (p.dot) p.dot[(size_t)(zh * 4 + cg) * p.BH * p.T + grow] = d;
                }
            }
            tc::fence_before_sync();
            arrive(&b_tfree[sg]);
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
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BARS);   // load[2], mma[2], fin
    uint32_t *tbase = reinterpret_cast<uint32_t *>(sm + L::TBASE);
    volatile int *abort = reinterpret_cast<volatile int *>(sm + L::TBASE + 4);
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
        for (int i = 0; i < 5; ++i) mbar_init(&bars[i], 1);
        *abort = 0;
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
        auto load = [&](const CUtensorMap *a, const CUtensorMap *b, uint64_t *bar) {
            mbar_arrive_expect_tx(bar, 2 * LtSmem::TILE);
            for (int h = 0; h < 2; ++h) {
                tma_load_3d(sm + L::A + h * LtSmem::HALF, a, h * 64, t0, bh, bar);
                tma_load_3d(sm + L::B + h * LtSmem::HALF, b, h * 64, t0, bh, bar);
            }
        };
        auto kmaj = [&](uint32_t base, int kk) {
            return tc::sdesc(sb + base + (kk >> 2) * LtSmem::HALF + (kk & 3) * 32, 16, 1024);
        };
        auto mma = [&](uint32_t col, uint64_t *bar) {
            constexpr uint32_t ID = tc::idesc_bf16(128, 128, false, false);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                tc::mma_f16(tmem + col, kmaj(L::A, kk), kmaj(L::B, kk), ID, kk > 0);
            tc::commit(bar);
        };
        load(&args.q, &args.k, &bars[0]);
        ok = lt_wait(&bars[0], 0, abort);
        if (ok) {
            mma(0, &bars[2]);
            ok = lt_wait(&bars[2], 0, abort);
        }
        if (ok) {
            load(&args.d_o, &args.v, &bars[1]);
            ok = lt_wait(&bars[1], 0, abort);
            if (ok) mma(128, &bars[3]);
        }
        if (!ok) {
            atomicExch(timeout_flag, 1);
            tc::commit(&bars[4]);
            mbar_wait_bounded(&bars[4], 0, kLtProbes);
            mbar_wait_bounded(&bars[1], 0, kLtProbes);
            mbar_wait_bounded(&bars[0], 0, kLtProbes);
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
    ok = lt_wait(&bars[3], 0, abort);
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
