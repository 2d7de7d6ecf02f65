// Gated linear recurrence on CUDA cores (fp32 inputs), and its single step (every type).
//
// Per (batch, head), with decay beta_t, write gate g_t and scale c:
//   M_t = beta_t M_{t-1} + g_t v_t k_t^T,   o_t = c M_t q_t
// (the layer's value state read without its ridge solve; "Gated KalmaNet",
// arXiv 2511.21016, ai.info page, Methodology, gives the recurrence and its
// chunk-wise form).  With R_t the gradient of M_t,
//   R_t = beta_{t+1} R_{t+1} + c do_t q_t^T,
//   dq_t = c M_t^T do_t,   dk_t = g_t R_t^T v_t,   dv_t = g_t R_t k_t,
//   dg_t = v_t^T R_t k_t,  dbeta_t = <R_t, M_{t-1}>,  dM_{-1} = beta_0 R_0.
//
// One pass.  o, dq, dk and dv are four instances of the same pass over rows
// x, y, z, forwards or backwards in time:
//   out_t = a_t S x_t + sum_i P_ti z_i,   P_ti = w_ti (x_t . y_i),
//   S' = b S + sum_i u_i y_i z_i^T        (S here is [D of y][D of z])
//             x   y   z   time      a_t              w_ti                 u_i
//     o       q   k   v   forward   e^{l_t}          e^{l_t - l_i} g_i    e^{l_C - l_i} g_i
//     dq      do  v   k   forward   e^{l_t}          e^{l_t - l_i} g_i    e^{l_C - l_i} g_i
//     dv      k   q   do  backward  e^{l_C - l_t}    e^{l_i - l_t} c      e^{l_i} c
//     dk      v   do  q   backward  e^{l_C - l_t}    e^{l_i - l_t} c      e^{l_i} c
// with l the cumulative log decay inside the chunk (a sum of two floats, so that a
// difference keeps fp32 precision after a reset) and the sum over i <= t
// (forward) or i >= t (backward).  o and dq are scaled by c at the end, dk and dv
// by g_t.  S runs along the sequence in fp32; a CTA owns ZN columns of z for one
// head and one segment of the sequence (segments: see k_linear_scan).
//
// dbeta.  beta_t scales every product of a write before t with a read at or
// after t, so with the pair terms A_si = c g_i w_si (q_s . k_i)(do_s . v_i),
//   beta_t dbeta_t = F + sum_{s >= t} zeta_s + sum_{i < t} g_i eta_i + sum_{i < t <= s} A_si
// over the chunk of t, where F = e^{l_C} <E, M_s> (write before, read behind the
// chunk), zeta_s = q_s . (state part of dq_s) and eta_i = v_i . (state part of
// dv_i / g_i).  No term cancels another, and every one holds the factor beta_t, so
// the quotient is as exact as the terms; log beta is clamped at 2^-60 in
// the backward for that quotient to exist at beta = 0 (a reset), where what the
// clamp lets through is below 2^-60 of what was written.  dg_i = eta_i plus the
// pair terms' column sums.  The passes leave zeta, eta and F in the workspace and
// k_linear_pairs forms the pairs, all chunks in parallel.
#pragma once

#include <cuda_bf16.h>

#include "block_rows.cuh"
#include "common.cuh"
#include "ptx.cuh"

namespace gka {

constexpr int kLinC = 32;         // tokens per chunk of the CUDA-core pass
constexpr int kLinThreads = 256;
// Clamps of log2 beta: in the forward, below every fp32 product (a reset passes exactly
// nothing); 2^-60 is the smallest decay the backward tells from zero.
constexpr float kLinLog2Min = -216.f, kLinLog2MinBwd = -60.f;

// A sum of log decays as an unevaluated pair of floats (about 45 bits): differences of
// cumulative logs keep fp32 precision after a reset, at a fraction of doubles' latency.
struct Log2Sum {
    float hi, lo;
};
__device__ __forceinline__ Log2Sum operator+(Log2Sum a, Log2Sum b) {
    const float s = a.hi + b.hi, t = s - a.hi;
    const float e = (a.hi - (s - t)) + (b.hi - t) + (a.lo + b.lo);
    const float h = s + e;
    return {h, e - (h - s)};
}
// log2 beta, not below `least` (a NaN stays one)
__device__ __forceinline__ float log2_decay(float beta, float least) {
    const float l = log2f(beta);
    return l < least ? least : l;
}
// 2^x, results below 2^-126 as zero (relative error 2^-22: the hardware's function)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 2^(a - b)
__device__ __forceinline__ float exp2_diff(Log2Sum a, Log2Sum b) {
    return ex2((a.hi - b.hi) + (a.lo - b.lo));
}
__device__ __forceinline__ Log2Sum shfl(Log2Sum x, int src) {
    return {__shfl_sync(0xffffffffu, x.hi, src), __shfl_sync(0xffffffffu, x.lo, src)};
}

struct LinPass {
    const void *x, *y, *z;        // [B*H, T, D]
    const void *xd;               // nullable: rows whose dot with the state part goes to `dot`
    void *out;                    // [B*H, T, D]
    const float *beta, *gate;     // [B*H, T]; gate nullable
    const float *start;           // nullable fp32 states [B*H][S][D][D] in force at each segment
    float *last;                  // nullable fp32 [B*H][D][D]: state past the last token
    float *agg, *segdec;          // aggregates (k_linear_pass without output): [B*H][S][D][D], [B*H][S]
    float *states;                // nullable fp32 [B*H][N][D][D]: state in force at each chunk
    const float *states_in;       // nullable: the same, of the other direction, for `fdot`
    float *dot;                   // [ZS][B*H*T]
    float *fdot;                  // [ZS][B*H*N]
    float scale;
    float log2_min;               // clamp of log2 beta
    int BH, T, N, S, D;
    int zy;                       // a state's memory is [z][y] (else [y][z])
};

// Segments [n0, n1) of chunks in time order; the backward passes run them, and the
// chunks in them, from the end.
__host__ __device__ __forceinline__ int lin_seg(int s, int S, int N) {
    return (int)(((long long)s * N) / S);
}

// Columns of z a CTA owns, and the floats that lie before the tiles (two tables of 4 x kLinC,
// cumulative logs among them as pairs, and a warp's worth of sums).
template <int D>
struct LinSmem {
    static constexpr int ZN = D < 64 ? D : 64;
    static constexpr int LD = D + 4;
    static constexpr int TAB = 5 * kLinC, HEAD = 2 * TAB + 8;
    static constexpr int floats = HEAD + 2 * kLinC * LD + 2 * kLinC * ZN + D * ZN + kLinC * (kLinC + 1);
    static constexpr size_t bytes = sizeof(float) * floats;
};

// A chunk's tile of rows [kLinC][COLS] (from [T][D] at column c0; rows past T: zeros) into
// registers, and from there into shared memory: every load of a chunk goes out before the
// first store.
template <int COLS>
struct LinTile {
    static constexpr int PER = COLS / 4, N = kLinC * PER / kLinThreads;
    float4 v[N];
    __device__ __forceinline__ void load(const float *src, int t0, int Ttot, int D, int c0) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = threadIdx.x + k * kLinThreads, r = i / PER;
            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (t0 + r < Ttot)
                v[k] = __ldg(reinterpret_cast<const float4 *>(src + (size_t)(t0 + r) * D + c0 + (i - r * PER) * 4));
        }
    }
    __device__ __forceinline__ void store(float *dst, int ld) const {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = threadIdx.x + k * kLinThreads, r = i / PER;
            *reinterpret_cast<float4 *>(dst + r * ld + (i - r * PER) * 4) = v[k];
        }
    }
    // row r times u[r]
    __device__ __forceinline__ void store(float *dst, int ld, const float *u) const {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = threadIdx.x + k * kLinThreads, r = i / PER;
            const float w = u[r];
            *reinterpret_cast<float4 *>(dst + r * ld + (i - r * PER) * 4) =
                make_float4(w * v[k].x, w * v[k].y, w * v[k].z, w * v[k].w);
        }
    }
};

// Inclusive prefix of a chunk's clamped log2 decays by one warp (lane = token).
__device__ __forceinline__ Log2Sum lin_log_prefix(float log2_beta) {
    const int lane = threadIdx.x & 31;
    Log2Sum x = {log2_beta, 0.f};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Log2Sum y = {__shfl_up_sync(0xffffffffu, x.hi, o), __shfl_up_sync(0xffffffffu, x.lo, o)};
        if (lane >= o) x = x + y;
    }
    return x;
}
// the same from memory; past T: no decay
__device__ __forceinline__ Log2Sum lin_log_prefix(const float *beta, int t0, int T, float log2_min) {
    const int t = t0 + (threadIdx.x & 31);
    return lin_log_prefix(t < T ? log2_decay(beta[t], log2_min) : 0.f);
}

// A 4 x 4 tile's sums over lanes 8 (STEPS = 1) or 8 and 16 (2) apart, the rows shared out among
// those lanes: lane group k = (lane >> 3) % (2 STEPS) is left with rows 2 k, 2 k + 1 (1) or k (2)
// as its first.
template <int STEPS>
__device__ __forceinline__ void quarter_sums(float (&a)[4][4]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int s = STEPS; s > 0; --s) {
        const int rows = STEPS == 2 && s == 1 ? 1 : 2;   // left after this exchange
        const bool up = lane & (8 * s);
#pragma unroll
        for (int i = 0; i < rows; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float send = up ? a[i][j] : a[i + rows][j], keep = up ? a[i + rows][j] : a[i][j];
                a[i][j] = keep + __shfl_xor_sync(0xffffffffu, send, 8 * s);
            }
    }
}

struct LinPasses {
    LinPass pass[2];
};

// CTAs of k_linear_pass an SM holds.  With these D = 128 spills 20 bytes (forward), 64 88 to 100, 32
// 20 to 28, and all are faster than the smaller tiles that spilled less (B8 H8 T2048 624 -> 546,
// 203 -> 176, 110 -> 98 us).  Without spills, three CTAs of D = 32 take 105 us, two of 64 171.
__host__ __device__ constexpr int lin_per_sm(int D) { return D > 64 ? 2 : D > 32 ? 3 : 4; }

// grid (passes * D / ZN, B*H, S), block kLinThreads.  OUT = false: the segments' aggregates
// (states from zero) and decays only.
//
// Warp (token group, column half) and lane (four tokens or state rows) x (eight groups of four
// columns): a thread has SR x 4 of the state and, for the scores and the state's part of the
// outputs, a 4 x 4 tile over a part of the sum, which shuffles join, since a 16-byte load is four
// passes of shared memory whatever its lanes share.  Chunk n + 1's tiles and decays come from
// memory, and its decay table is formed, while chunk n is worked on.  What bounds it (D = 128):
// shared memory 68 % of the cycles, issue slots 63 %, the fp32 pipe 47 %.  B2 H1 T88769 D128:
// 635 us with the aggregates (whole sums a thread, 2 x 2 and 2 x 4: 730; 32 columns a CTA and
// tables between the chunks: 1276), of which the recurrence's own 4 D^2 a token would be 194 at
// 60 TFLOP/s; the aggregates and the chunks' scores are as much again.
// Where few chunks are left a launch (T of some hundreds), the launches' latency.
template <int D, bool REV, bool OUT>
__global__ void __launch_bounds__(kLinThreads, lin_per_sm(D))
k_linear_pass(const __grid_constant__ LinPasses args) {
    using L = LinSmem<D>;
    constexpr int C = kLinC, ZN = L::ZN, LD = L::LD;
    constexpr int HC = ZN / 32, TG = 8 / HC, R = C / (4 * TG), SR = D * ZN / 1024;
    extern __shared__ float4 lin_smem[];
    float *s_tab = reinterpret_cast<float *>(lin_smem);       // [2][TAB]: l (pairs), a, u, g
    float *s_red = s_tab + 2 * L::TAB;                        // [8]
    float *xs = s_tab + L::HEAD;                              // [C][LD]
    float *ys = xs + C * LD;                                  // [C][LD]
    float *zs = ys + C * LD;                                  // [C][ZN]
    float *wz = zs + C * ZN;                                  // [C][ZN] u_i z_i
    float *St = wz + C * ZN;                                  // [D][ZN]
    float *Ps = St + D * ZN;                                  // [C][C + 1]
    // in this order: the pair terms' kernel, further on in the call, reads the call's inputs
    // before its own wait, and may only exist once what wrote them is done
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const LinPass &p = args.pass[blockIdx.x / (D / ZN)];
    const int zsp = blockIdx.x % (D / ZN), z0 = zsp * ZN, bh = blockIdx.y, seg = blockIdx.z;
    const int n0 = lin_seg(seg, p.S, p.N), n1 = lin_seg(seg + 1, p.S, p.N);
    if (!OUT && seg == (REV ? 0 : p.S - 1)) return;   // never carried on
    const float *X = static_cast<const float *>(p.x) + (size_t)bh * p.T * D;
    const float *Y = static_cast<const float *>(p.y) + (size_t)bh * p.T * D;
    const float *Z = static_cast<const float *>(p.z) + (size_t)bh * p.T * D;
    const float *beta = p.beta + (size_t)bh * p.T;
    const float *gate = p.gate ? p.gate + (size_t)bh * p.T : nullptr;

    const int ch = warp % HC, tg = warp / HC, zc = ch * 32 + (lane & 7) * 4;   // columns zc..zc + 3
    constexpr int KG = 4 / R;                                                  // parts of a sum over d
    const int kg = (lane >> 3) % KG, tile = tg * 4 * R + (lane >> 3) / KG * 4;  // its tile's first token
    const int tok = tile + kg * R;                                             // tokens tok + i
    const int yr = (tg * 4 + (lane >> 3)) * SR;                                // state rows yr + i
    float st[SR][4];
    auto state_at = [&](size_t base, int i, int j) {
        return base + (p.zy ? (size_t)(z0 + zc + j) * D + yr + i : (size_t)(yr + i) * D + z0 + zc + j);
    };
#pragma unroll
    for (int i = 0; i < SR; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) st[i][j] = 0.f;
    if (OUT && p.start) {
        const size_t base = ((size_t)bh * p.S + seg) * D * D;
#pragma unroll
        for (int i = 0; i < SR; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) st[i][j] = p.start[state_at(base, i, j)];
    }
    const Log2Sum zero = {0.f, 0.f};
    Log2Sum seglog = zero;

    auto first = [&](int it) { return (REV ? n1 - 1 - it : n0 + it) * C; };
    LinTile<D> tx, ty;
    LinTile<ZN> tz;
    float nl = 0.f, ng = 0.f;   // warp 0: the token's log decay and gate
    auto fetch = [&](int it) {
        const int t0 = first(it);
        if (warp == 0) {
            const bool in = t0 + lane < p.T;
            nl = in ? log2_decay(beta[t0 + lane], p.log2_min) : 0.f;
            ng = in ? (gate ? gate[t0 + lane] : 1.f) : 0.f;
        }
        if (OUT) tx.load(X, t0, p.T, D, 0);
        ty.load(Y, t0, p.T, D, 0);
        tz.load(Z, t0, p.T, D, z0);
    };
    auto table = [&](int it) {
        if (warp) return;
        float *t = s_tab + (it & 1) * L::TAB;
        const Log2Sum l = lin_log_prefix(nl), lC = shfl(l, 31);
        const float to = exp2_diff(l, zero), from = exp2_diff(lC, l);
        reinterpret_cast<Log2Sum *>(t)[lane] = l;
        t[2 * C + lane] = REV ? from : to;
        t[3 * C + lane] = REV ? p.scale * to : ng * from;
        t[4 * C + lane] = ng;
    };
    fetch(0);
    table(0);
    for (int it = 0; it < n1 - n0; ++it) {
        const int t0 = first(it), n = t0 / C;
        const float *tab = s_tab + (it & 1) * L::TAB;
        const Log2Sum *s_l = reinterpret_cast<const Log2Sum *>(tab);
        const float *s_a = tab + 2 * C, *s_u = tab + 3 * C, *s_g = tab + 4 * C;
        __syncthreads();
        if (OUT) {
#pragma unroll
            for (int i = 0; i < SR; ++i)
                *reinterpret_cast<float4 *>(St + (yr + i) * ZN + zc) =
                    make_float4(st[i][0], st[i][1], st[i][2], st[i][3]);
            tx.store(xs, LD);
            tz.store(zs, ZN);
        }
        ty.store(ys, LD);
        tz.store(wz, ZN, s_u);
        __syncthreads();
        if (it + 1 < n1 - n0) fetch(it + 1);
        const Log2Sum lC = s_l[C - 1];
        const float b = exp2_diff(lC, zero);
        seglog = seglog + lC;
        float4 si[R];
        if (OUT) {
            if (p.states) {
                const size_t base = ((size_t)bh * p.N + n) * D * D;
#pragma unroll
                for (int i = 0; i < SR; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) p.states[state_at(base, i, j)] = st[i][j];
            }
            // F: the state of the other direction against this one's, before the chunk
            if (p.states_in) {
                float f = 0.f;
                const size_t base = ((size_t)bh * p.N + n) * D * D;
#pragma unroll
                for (int i = 0; i < SR; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) f = fmaf(st[i][j], p.states_in[state_at(base, i, j)], f);
                f = warp_sum(f);
                if (lane == 0) s_red[warp] = f;
            }
            // P: a lane's 4 x 4 tile, rows 4 warp + i and columns (lane & 7) + 8 j, over a quarter
            // of d (16 bytes of every 64); columns beyond the warp's diagonal are left out
            {
                const int p4 = lane & 7, k4 = lane >> 3;
                float acc[4][4] = {};
#pragma unroll 2
                for (int d = 4 * k4; d < D; d += 16) {
                    float4 xv[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) xv[i] = *reinterpret_cast<const float4 *>(xs + (4 * warp + i) * LD + d);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (REV ? j < (warp >> 1) : j > (warp >> 1)) continue;
                        const float4 yv = *reinterpret_cast<const float4 *>(ys + (p4 + 8 * j) * LD + d);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            acc[i][j] = fmaf(xv[i].x, yv.x, acc[i][j]);
                            acc[i][j] = fmaf(xv[i].y, yv.y, acc[i][j]);
                            acc[i][j] = fmaf(xv[i].z, yv.z, acc[i][j]);
                            acc[i][j] = fmaf(xv[i].w, yv.w, acc[i][j]);
                        }
                    }
                }
                quarter_sums<2>(acc);   // row k4 of the tile is left
                const int t = 4 * warp + k4;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = p4 + 8 * j;
                    const bool in = REV ? c >= t : c <= t;
                    const float w = REV ? p.scale : s_g[c];
                    Ps[t * (C + 1) + c] =
                        in ? acc[0][j] * w * (REV ? exp2_diff(s_l[c], s_l[t]) : exp2_diff(s_l[t], s_l[c])) : 0.f;
                }
            }
            // the state's part of the outputs: 4 tokens x 4 columns, over a part of d
            float acc[4][4] = {};
#pragma unroll 2
            for (int d = 4 * kg; d < D; d += 4 * KG) {
                float xa[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 xv = *reinterpret_cast<const float4 *>(xs + (tile + i) * LD + d);
                    xa[i][0] = xv.x; xa[i][1] = xv.y; xa[i][2] = xv.z; xa[i][3] = xv.w;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 s = *reinterpret_cast<const float4 *>(St + (d + e) * ZN + zc);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        acc[i][0] = fmaf(xa[i][e], s.x, acc[i][0]);
                        acc[i][1] = fmaf(xa[i][e], s.y, acc[i][1]);
                        acc[i][2] = fmaf(xa[i][e], s.z, acc[i][2]);
                        acc[i][3] = fmaf(xa[i][e], s.w, acc[i][3]);
                    }
                }
            }
            quarter_sums<KG / 2>(acc);
#pragma unroll
            for (int i = 0; i < R; ++i) si[i] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        }
        if (it + 1 < n1 - n0) table(it + 1);
        if (OUT) {
            __syncthreads();
            if (p.states_in && tid == 0) {
                float f = 0.f;
                for (int w = 0; w < kLinThreads / 32; ++w) f += s_red[w];
                p.fdot[((size_t)zsp * p.BH + bh) * p.N + n] = b * f;
            }
            // the chunk's own part, over the tokens of the thread's warp or before (after) them
            float4 in[R];
#pragma unroll
            for (int i = 0; i < R; ++i) in[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            const int i0 = REV ? tg * 4 * R : 0, i1 = REV ? C : (tg + 1) * 4 * R;
#pragma unroll 4
            for (int c = i0; c < i1; ++c) {
                const float4 z = *reinterpret_cast<const float4 *>(zs + c * ZN + zc);
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float pv = Ps[(tok + i) * (C + 1) + c];
                    in[i].x = fmaf(pv, z.x, in[i].x);
                    in[i].y = fmaf(pv, z.y, in[i].y);
                    in[i].z = fmaf(pv, z.z, in[i].z);
                    in[i].w = fmaf(pv, z.w, in[i].w);
                }
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int t = tok + i;
                const bool inside = t0 + t < p.T;
                const float a = s_a[t] * (REV ? 1.f : p.scale), c = REV ? s_g[t] : p.scale;
                const float4 r = make_float4(a * si[i].x, a * si[i].y, a * si[i].z, a * si[i].w);   // (without g)
                const size_t row = (size_t)bh * p.T + t0 + t;
                if (p.dot) {
                    float d = 0.f;
                    if (inside) {
                        const float4 xd = __ldg(reinterpret_cast<const float4 *>(
                            static_cast<const float *>(p.xd) + row * D + z0 + zc));
                        d = fmaf(r.x, xd.x, fmaf(r.y, xd.y, fmaf(r.z, xd.z, r.w * xd.w)));
                    }
#pragma unroll
                    for (int o = 4; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
                    if ((lane & 7) == 0 && inside) p.dot[(size_t)(zsp * HC + ch) * p.BH * p.T + row] = d;
                }
                if (inside)
                    *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + row * D + z0 + zc) =
                        REV ? make_float4(c * (r.x + in[i].x), c * (r.y + in[i].y), c * (r.z + in[i].z),
                                          c * (r.w + in[i].w))
                            : make_float4(fmaf(c, in[i].x, r.x), fmaf(c, in[i].y, r.y), fmaf(c, in[i].z, r.z),
                                          fmaf(c, in[i].w, r.w));
            }
        }
        // S' = b S + sum_i y_i (u_i z_i)^T
#pragma unroll
        for (int i = 0; i < SR; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) st[i][j] *= b;
#pragma unroll 4
        for (int c = 0; c < C; ++c) {
            const float4 zv = *reinterpret_cast<const float4 *>(wz + c * ZN + zc);
            float ya[SR];
            if constexpr (SR >= 4) {
#pragma unroll
                for (int i = 0; i < SR; i += 4) {
                    const float4 yv = *reinterpret_cast<const float4 *>(ys + c * LD + yr + i);
                    ya[i] = yv.x; ya[i + 1] = yv.y; ya[i + 2] = yv.z; ya[i + 3] = yv.w;
                }
            } else {
                ya[0] = ys[c * LD + yr];
            }
#pragma unroll
            for (int i = 0; i < SR; ++i) {
                st[i][0] = fmaf(ya[i], zv.x, st[i][0]);
                st[i][1] = fmaf(ya[i], zv.y, st[i][1]);
                st[i][2] = fmaf(ya[i], zv.z, st[i][2]);
                st[i][3] = fmaf(ya[i], zv.w, st[i][3]);
            }
        }
    }
    float *dst = OUT ? (seg == (REV ? 0 : p.S - 1) ? p.last : nullptr) : p.agg;
    if (dst) {
        const size_t base = OUT ? (size_t)bh * D * D : ((size_t)bh * p.S + seg) * D * D;
#pragma unroll
        for (int i = 0; i < SR; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) dst[state_at(base, i, j)] = st[i][j];
    }
    if (!OUT && tid == 0 && zsp == 0) p.segdec[(size_t)bh * p.S + seg] = exp2_diff(seglog, zero);
}

// Segment starts in place of the segments' aggregates: the carry over a segment is
// linear, S(end) = dec S(start) + A, so with few heads the sequences are cut into S
// segments whose aggregates A (states from zero) are formed in parallel, and this
// kernel, element-wise and in order, leaves in each entry the state in force where
// the segment begins (rev: behind its end).  init nullable [B*H][D2].  Latency bounds it (a
// chain over S): 32 segments' loads at a time, not 8, took the fp32 gradient of B1 H1 T16000
// D128 from 381 to 313 us.
// grid (D2 / 1024, B*H), block 256.
__global__ void __launch_bounds__(256)
k_linear_scan(float *__restrict__ agg, const float *__restrict__ segdec,
              const float *__restrict__ init, int S, int D2, int rev) {
    griddep_launch_dependents();
    griddep_wait();
    const int bh = blockIdx.y, e = (blockIdx.x * 256 + threadIdx.x) * 4;
    if (e >= D2) return;
    float4 run = make_float4(0.f, 0.f, 0.f, 0.f);
    if (init) run = *reinterpret_cast<const float4 *>(init + (size_t)bh * D2 + e);
    float *base = agg + (size_t)bh * S * D2 + e;
    constexpr int kB = 32;   // loads of so many segments go out before the first store
    for (int s0 = 0; s0 < S; s0 += kB) {
        float4 av[kB];
        float bv[kB];
#pragma unroll
        for (int j = 0; j < kB; ++j)
            if (s0 + j < S - 1) {   // the last one's aggregate is not carried on
                const int s = rev ? S - 1 - s0 - j : s0 + j;
                av[j] = *reinterpret_cast<const float4 *>(base + (size_t)s * D2);
                bv[j] = segdec[(size_t)bh * S + s];
            }
#pragma unroll
        for (int j = 0; j < kB; ++j)
            if (s0 + j < S) {
                const int s = rev ? S - 1 - s0 - j : s0 + j;
                *reinterpret_cast<float4 *>(base + (size_t)s * D2) = run;
                if (s0 + j < S - 1)
                    run = make_float4(fmaf(bv[j], run.x, av[j].x), fmaf(bv[j], run.y, av[j].y),
                                  fmaf(bv[j], run.z, av[j].z), fmaf(bv[j], run.w, av[j].w));
            }
    }
}

struct LinPairs {
    const void *q, *k, *v, *d_o;   // [B*H, T, D]
    const float *beta, *gate;      // [B*H, T]; gate nullable
    const float *zeta, *eta;       // [ZS][B*H*T]
    const float *fdot;             // [ZS][B*H*N]
    float *dbeta, *dgate;          // [B*H, T]; dgate nullable
    float scale;
    int BH, T, N, ZS, FS;          // ZS planes of zeta and eta, FS of fdot
};

// dbeta and dgate of one chunk from its pair terms (top of this file).
// grid (N, B*H), block kLinThreads.
template <int D>
__global__ void __launch_bounds__(kLinThreads) k_linear_pairs(const LinPairs p) {
    constexpr int C = kLinC, LD = D + 4;
    extern __shared__ float4 lin_smem[];
    Log2Sum *s_l = reinterpret_cast<Log2Sum *>(lin_smem);
    float *qs = reinterpret_cast<float *>(s_l + C), *ks = qs + C * LD, *vs = ks + C * LD,
          *os = vs + C * LD;
    float *As = os + C * LD;                       // [C][C + 1]
    float *s_g = As + C * (C + 1), *s_ze = s_g + C, *s_ge = s_ze + C;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = blockIdx.x, bh = blockIdx.y, t0 = n * C;
    const size_t head = (size_t)bh * p.T, rowsall = (size_t)p.BH * p.T;
    {
        LinTile<D> tq, tk, tv, to;
        tq.load(static_cast<const float *>(p.q) + head * D, t0, p.T, D, 0);
        tk.load(static_cast<const float *>(p.k) + head * D, t0, p.T, D, 0);
        tv.load(static_cast<const float *>(p.v) + head * D, t0, p.T, D, 0);
        to.load(static_cast<const float *>(p.d_o) + head * D, t0, p.T, D, 0);
        tq.store(qs, LD);
        tk.store(ks, LD);
        tv.store(vs, LD);
        to.store(os, LD);
    }
    float eta = 0.f;
    if (warp == 0) {
        s_l[lane] = lin_log_prefix(p.beta + head, t0, p.T, kLinLog2MinBwd);
        float zeta = 0.f, g = 0.f;
        griddep_wait();   // the passes are done (what came before them was, before the first began)
        if (t0 + lane < p.T) {
            g = p.gate ? p.gate[head + t0 + lane] : 1.f;
            for (int z = 0; z < p.ZS; ++z) {
                zeta += p.zeta[z * rowsall + head + t0 + lane];
                eta += p.eta[z * rowsall + head + t0 + lane];
            }
        }
        s_g[lane] = g;
        // sum of zeta from this token on; sum of g eta before it
        float ge = g * eta, z = zeta;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float u = __shfl_down_sync(0xffffffffu, z, o), d = __shfl_up_sync(0xffffffffu, ge, o);
            if (lane + o < 32) z += u;
            if (lane >= o) ge += d;
        }
        const float before = __shfl_up_sync(0xffffffffu, ge, 1);
        s_ze[lane] = z;
        s_ge[lane] = lane ? before : 0.f;
    }
    __syncthreads();
    {
        const int tr = tid >> 4, tc = tid & 15;   // rows s = tr, tr + 16; columns i = tc, tc + 16
        float aq[2][2] = {}, av[2][2] = {};
#pragma unroll 2
        for (int d = 0; d < D; d += 4) {
            float4 qv[2], kv[2], ov[2], vv[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                qv[i] = *reinterpret_cast<const float4 *>(qs + (tr + 16 * i) * LD + d);
                ov[i] = *reinterpret_cast<const float4 *>(os + (tr + 16 * i) * LD + d);
                kv[i] = *reinterpret_cast<const float4 *>(ks + (tc + 16 * i) * LD + d);
                vv[i] = *reinterpret_cast<const float4 *>(vs + (tc + 16 * i) * LD + d);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    aq[i][j] = fmaf(qv[i].x, kv[j].x, aq[i][j]);
                    aq[i][j] = fmaf(qv[i].y, kv[j].y, aq[i][j]);
                    aq[i][j] = fmaf(qv[i].z, kv[j].z, aq[i][j]);
                    aq[i][j] = fmaf(qv[i].w, kv[j].w, aq[i][j]);
                    av[i][j] = fmaf(ov[i].x, vv[j].x, av[i][j]);
                    av[i][j] = fmaf(ov[i].y, vv[j].y, av[i][j]);
                    av[i][j] = fmaf(ov[i].z, vv[j].z, av[i][j]);
                    av[i][j] = fmaf(ov[i].w, vv[j].w, av[i][j]);
                }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int s = tr + 16 * i, c = tc + 16 * j;
                As[s * (C + 1) + c] =
                    c <= s ? p.scale * exp2_diff(s_l[s], s_l[c]) * aq[i][j] * av[i][j] : 0.f;
            }
    }
    __syncthreads();
    float dg = eta;
    if (warp == 0)
        for (int s = lane; s < C; ++s) dg += As[s * (C + 1) + lane];   // column sums, s >= i
    __syncthreads();
    // row s: sum of its gated pairs before t, for every t <= s
    for (int s = warp; s < C; s += kLinThreads / 32) {
        float x = As[s * (C + 1) + lane] * s_g[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        x = __shfl_up_sync(0xffffffffu, x, 1);
        As[s * (C + 1) + lane] = lane ? x : 0.f;
    }
    __syncthreads();
    if (warp == 0 && t0 + lane < p.T) {
        float d = s_ze[lane] + s_ge[lane];
        for (int z = 0; z < p.FS; ++z) d += p.fdot[((size_t)z * p.BH + bh) * p.N + n];
        float pairs = 0.f;
        for (int s = lane; s < C; ++s) pairs += As[s * (C + 1) + lane];
        const float bt = fmaxf(p.beta[head + t0 + lane], 8.6736174e-19f);   // 2^-60
        p.dbeta[head + t0 + lane] = (d + pairs) / bt;
        if (p.dgate) p.dgate[head + t0 + lane] = dg;
    }
}

template <int D>
constexpr size_t lin_pairs_smem() {
    return sizeof(Log2Sum) * kLinC +
           sizeof(float) * (4 * kLinC * (D + 4) + kLinC * (kLinC + 1) + 3 * kLinC);
}

// ---------------------------------------------------------------------------
// One token: M <- beta M + g v k^T, o = c M q, in place on the fp32 state.
//
// The state's read and write is all the traffic (8 D^2 bytes a head against 8 to
// 16 D of everything else) and bounds it.  A row of M is D / 4 neighbouring lanes
// of 16 bytes; a thread carries kStepRows rows, whose loads all go out before the
// first use.  256 x 32 heads of D = 128, bf16: 157 us for 1083 MB, the copy rate; one
// sequence of 8 heads: 2 us, a launch.
// ---------------------------------------------------------------------------
constexpr int kStepRows = 4;
constexpr int kStepThreads = 128;

// grid (D * (D / 4) / (kStepThreads * kStepRows) rounded up, B*H)
template <typename T, int D>
__global__ void __launch_bounds__(kStepThreads)
k_linear_step(float *__restrict__ state, const T *__restrict__ q, const T *__restrict__ k,
              const T *__restrict__ v, const float *__restrict__ beta,
              const float *__restrict__ gate, T *__restrict__ o, float scale, int parts) {
    constexpr int LPR = D / 4, GROUPS = kStepThreads / LPR;
    const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR;
    const size_t bh = blockIdx.x / (unsigned)parts;
    const int row0 = (int)(blockIdx.x % (unsigned)parts) * (GROUPS * kStepRows) + grp;
    float4 m[kStepRows];
    float4 *M = reinterpret_cast<float4 *>(state + bh * D * D) + lane;
#pragma unroll
    for (int j = 0; j < kStepRows; ++j)
        if (row0 + j * GROUPS < D) m[j] = __ldcs(M + (size_t)(row0 + j * GROUPS) * LPR);
    const float b = beta[bh], g = gate ? gate[bh] : 1.f;
    float kk[4], qq[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        kk[e] = load_f(k + bh * D + lane * 4 + e);
        qq[e] = load_f(q + bh * D + lane * 4 + e);
    }
#pragma unroll
    for (int j = 0; j < kStepRows; ++j) {
        const int r = row0 + j * GROUPS;
        const bool in = r < D;
        const float gv = in ? g * load_f(v + bh * D + r) : 0.f;
        float4 &x = m[j];
        if (!in) x = make_float4(0.f, 0.f, 0.f, 0.f);
        x.x = fmaf(b, x.x, gv * kk[0]);
        x.y = fmaf(b, x.y, gv * kk[1]);
        x.z = fmaf(b, x.z, gv * kk[2]);
        x.w = fmaf(b, x.w, gv * kk[3]);
        if (in) __stcs(M + (size_t)r * LPR, x);
        float s = fmaf(x.x, qq[0], fmaf(x.y, qq[1], fmaf(x.z, qq[2], x.w * qq[3])));
        s = row_sum<LPR>(s);
        if (in && lane == 0) store_f(o + bh * D + r, scale * s);
    }
}

}  // namespace gka
