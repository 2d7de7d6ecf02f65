// Gated linear recurrence on CUDA cores: every type, head size and length.
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
constexpr int kLinZN = 32;        // columns of z a CTA owns
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
    int BH, T, N, S;
    int zy;                       // a state's memory is [z][y] (else [y][z])
};

// Segments [n0, n1) of chunks in time order; the backward passes run them, and the
// chunks in them, from the end.
__host__ __device__ __forceinline__ int lin_seg(int s, int S, int N) {
    return (int)(((long long)s * N) / S);
}

template <int D>
struct LinSmem {
    static constexpr int LD = D + 4;
    static constexpr int floats = 2 * kLinC * LD + 2 * kLinC * kLinZN + D * kLinZN +
                                  kLinC * (kLinC + 1) + 3 * kLinC + 8;
    static constexpr size_t bytes = sizeof(Log2Sum) * kLinC + sizeof(float) * floats;
};

// A chunk's tile of rows [kLinC][COLS] (from [T][D] at column c0; rows past T: zeros) into
// registers, and from there as floats into shared memory: every load of a chunk goes out
// before the first store.
template <typename T, int COLS>
struct LinTile {
    using V = Vec16<T>;
    static constexpr int PER = COLS / V::N, ITEMS = kLinC * PER, N = (ITEMS + kLinThreads - 1) / kLinThreads;
    uint4 v[N];
    __device__ __forceinline__ void load(const T *src, int t0, int Ttot, int D, int c0) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = threadIdx.x + k * kLinThreads, r = i / PER;
            v[k] = make_uint4(0u, 0u, 0u, 0u);
            if (i < ITEMS && t0 + r < Ttot)
                v[k] = V::raw(src + (size_t)(t0 + r) * D + c0 + (i - r * PER) * V::N);
        }
    }
    __device__ __forceinline__ void store(float *dst, int ld) const {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = threadIdx.x + k * kLinThreads, r = i / PER;
            if (i >= ITEMS) continue;
            float f[V::N];
            V::unpack(v[k], f);
#pragma unroll
            for (int e = 0; e < V::N; e += 4)
                *reinterpret_cast<float4 *>(dst + r * ld + (i - r * PER) * V::N + e) =
                    make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
        }
    }
};

// Inclusive prefix of the clamped log2 decays of one chunk by one warp (lane =
// token; past T: no decay).
__device__ __forceinline__ Log2Sum lin_log_prefix(const float *beta, int t0, int T, float log2_min) {
    const int lane = threadIdx.x & 31;
    Log2Sum x = {0.f, 0.f};
    if (t0 + lane < T) x.hi = log2_decay(beta[t0 + lane], log2_min);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Log2Sum y = {__shfl_up_sync(0xffffffffu, x.hi, o), __shfl_up_sync(0xffffffffu, x.lo, o)};
        if (lane >= o) x = x + y;
    }
    return x;
}

// grid (D / kLinZN, B*H, S), block kLinThreads.  OUT = false: the segments'
// aggregates (states from zero) and decays only.
template <typename T, int D, bool REV, bool OUT>
__global__ void __launch_bounds__(kLinThreads) k_linear_pass(const LinPass p) {
    using L = LinSmem<D>;
    constexpr int C = kLinC, ZN = kLinZN, LD = L::LD;
    extern __shared__ float4 lin_smem[];
    Log2Sum *s_l = reinterpret_cast<Log2Sum *>(lin_smem);     // [C]
    float *xs = reinterpret_cast<float *>(s_l + C);           // [C][LD]
    float *ys = xs + C * LD;                                  // [C][LD]
    float *zs = ys + C * LD;                                  // [C][ZN]
    float *wz = zs + C * ZN;                                  // [C][ZN] u_i z_i
    float *St = wz + C * ZN;                                  // [D][ZN]
    float *Ps = St + D * ZN;                                  // [C][C + 1]
    float *s_a = Ps + C * (C + 1), *s_u = s_a + C, *s_g = s_u + C, *s_red = s_g + C;   // s_red [8]
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int zsp = blockIdx.x, z0 = zsp * ZN, bh = blockIdx.y, seg = blockIdx.z;
    const int n0 = lin_seg(seg, p.S, p.N), n1 = lin_seg(seg + 1, p.S, p.N);
    if (!OUT && seg == (REV ? 0 : p.S - 1)) return;   // never carried on
    const T *X = static_cast<const T *>(p.x) + (size_t)bh * p.T * D;
    const T *Y = static_cast<const T *>(p.y) + (size_t)bh * p.T * D;
    const T *Z = static_cast<const T *>(p.z) + (size_t)bh * p.T * D;
    const float *beta = p.beta + (size_t)bh * p.T;
    const float *gate = p.gate ? p.gate + (size_t)bh * p.T : nullptr;

    // state: thread (yg, zg) owns rows 4 yg.. and columns 4 zg..
    const int yg = tid / (ZN / 4), zg = tid % (ZN / 4);
    const bool has_state = yg < D / 4;
    float st[4][4];
    auto state_at = [&](size_t base, int i, int j) {
        const int y = 4 * yg + i, z = z0 + 4 * zg + j;
        return base + (p.zy ? (size_t)z * D + y : (size_t)y * D + z);
    };
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) st[i][j] = 0.f;
    if (OUT && p.start && has_state) {
        const size_t base = ((size_t)bh * p.S + seg) * D * D;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) st[i][j] = p.start[state_at(base, i, j)];
    }
    const Log2Sum zero = {0.f, 0.f};
    Log2Sum seglog = zero;

    // a chunk's tiles are on their way while the one before is worked on
    LinTile<T, D> tx, ty;
    LinTile<T, ZN> tz;
    auto fetch = [&](int it) {
        const int t0 = (REV ? n1 - 1 - it : n0 + it) * C;
        if (OUT) tx.load(X, t0, p.T, D, 0);
        ty.load(Y, t0, p.T, D, 0);
        tz.load(Z, t0, p.T, D, z0);
    };
    fetch(0);
    for (int it = 0; it < n1 - n0; ++it) {
        const int n = REV ? n1 - 1 - it : n0 + it, t0 = n * C;
        __syncthreads();
        if (has_state) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<float4 *>(St + (4 * yg + i) * ZN + 4 * zg) =
                    make_float4(st[i][0], st[i][1], st[i][2], st[i][3]);
            if (OUT && p.states) {
                const size_t base = ((size_t)bh * p.N + n) * D * D;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) p.states[state_at(base, i, j)] = st[i][j];
            }
        }
        if (OUT) tx.store(xs, LD);
        ty.store(ys, LD);
        tz.store(zs, ZN);
        if (warp == 0) {
            const Log2Sum l = lin_log_prefix(beta, t0, p.T, p.log2_min), lC = shfl(l, 31);
            const float g = t0 + lane < p.T ? (gate ? gate[t0 + lane] : 1.f) : 0.f;
            s_l[lane] = l;
            s_g[lane] = g;
            const float to = exp2_diff(l, zero), from = exp2_diff(lC, l);
            s_a[lane] = REV ? from : to;
            s_u[lane] = REV ? p.scale * to : g * from;
        }
        __syncthreads();
        if (it + 1 < n1 - n0) fetch(it + 1);
        const Log2Sum lC = s_l[C - 1];
        const float b = exp2_diff(lC, zero);
        seglog = seglog + lC;
        // F: the state of the other direction against this one's, before the chunk
        if (OUT && p.states_in) {
            float f = 0.f;
            if (has_state) {
                const size_t base = ((size_t)bh * p.N + n) * D * D;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        f = fmaf(st[i][j], p.states_in[state_at(base, i, j)], f);
            }
            f = warp_sum(f);
            if (lane == 0) s_red[warp] = f;
        }
        for (int i = tid; i < C * ZN; i += kLinThreads) wz[i] = s_u[i / ZN] * zs[i];
        if (OUT) {
            // P: thread (tr, tc) holds rows tr, tr + 16 and columns tc, tc + 16
            const int tr = tid >> 4, tc = tid & 15;
            float acc[2][2] = {};
#pragma unroll 4
            for (int d = 0; d < D; d += 4) {
                float4 xv[2], yv[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    xv[i] = *reinterpret_cast<const float4 *>(xs + (tr + 16 * i) * LD + d);
                    yv[i] = *reinterpret_cast<const float4 *>(ys + (tc + 16 * i) * LD + d);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        acc[i][j] = fmaf(xv[i].x, yv[j].x, acc[i][j]);
                        acc[i][j] = fmaf(xv[i].y, yv[j].y, acc[i][j]);
                        acc[i][j] = fmaf(xv[i].z, yv[j].z, acc[i][j]);
                        acc[i][j] = fmaf(xv[i].w, yv[j].w, acc[i][j]);
                    }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int t = tr + 16 * i, c = tc + 16 * j;
                    const bool in = REV ? c >= t : c <= t;
                    const float w = REV ? p.scale : s_g[c];
                    Ps[t * (C + 1) + c] =
                        in ? acc[i][j] * w * (REV ? exp2_diff(s_l[c], s_l[t]) : exp2_diff(s_l[t], s_l[c])) : 0.f;
                }
        }
        __syncthreads();
        if (OUT) {
            if (p.states_in && tid == 0) {
                float f = 0.f;
                for (int w = 0; w < kLinThreads / 32; ++w) f += s_red[w];
                p.fdot[((size_t)zsp * p.BH + bh) * p.N + n] = b * f;
            }
            // out: thread (t, zc) holds 4 columns of one token
            const int t = tid >> 3, zc = (tid & 7) * 4;
            float4 si = make_float4(0.f, 0.f, 0.f, 0.f), in = si;
#pragma unroll 4
            for (int d = 0; d < D; d += 4) {
                const float4 xv = *reinterpret_cast<const float4 *>(xs + t * LD + d);
                const float xa[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 s = *reinterpret_cast<const float4 *>(St + (d + e) * ZN + zc);
                    si.x = fmaf(xa[e], s.x, si.x);
                    si.y = fmaf(xa[e], s.y, si.y);
                    si.z = fmaf(xa[e], s.z, si.z);
                    si.w = fmaf(xa[e], s.w, si.w);
                }
            }
            const int i0 = REV ? t : 0, i1 = REV ? C : t + 1;
            for (int i = i0; i < i1; ++i) {
                const float pv = Ps[t * (C + 1) + i];
                const float4 z = *reinterpret_cast<const float4 *>(zs + i * ZN + zc);
                in.x = fmaf(pv, z.x, in.x);
                in.y = fmaf(pv, z.y, in.y);
                in.z = fmaf(pv, z.z, in.z);
                in.w = fmaf(pv, z.w, in.w);
            }
            const float a = s_a[t] * (REV ? 1.f : p.scale), c = REV ? s_g[t] : p.scale;
            float r[4] = {a * si.x, a * si.y, a * si.z, a * si.w};   // state part (without g)
            const size_t row = (size_t)bh * p.T + t0 + t;
            if (p.dot) {
                float d = 0.f;
                if (t0 + t < p.T) {
                    const T *xd = static_cast<const T *>(p.xd) + row * D + z0 + zc;
#pragma unroll
                    for (int e = 0; e < 4; ++e) d = fmaf(r[e], load_f(xd + e), d);
                }
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
                if ((tid & 7) == 0 && t0 + t < p.T) p.dot[(size_t)zsp * p.BH * p.T + row] = d;
            }
            if (t0 + t < p.T) {
                const float pin[4] = {in.x, in.y, in.z, in.w};
                T *o = static_cast<T *>(p.out) + row * D + z0 + zc;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    store_f(o + e, REV ? c * (r[e] + pin[e]) : fmaf(c, pin[e], r[e]));
            }
        }
        // S' = b S + sum_i y_i (u_i z_i)^T
        if (has_state) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) st[i][j] *= b;
#pragma unroll 4
            for (int i = 0; i < C; ++i) {
                const float4 yv = *reinterpret_cast<const float4 *>(ys + i * LD + 4 * yg);
                const float4 zv = *reinterpret_cast<const float4 *>(wz + i * ZN + 4 * zg);
                const float ya[4] = {yv.x, yv.y, yv.z, yv.w}, za[4] = {zv.x, zv.y, zv.z, zv.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int j = 0; j < 4; ++j) st[e][j] = fmaf(ya[e], za[j], st[e][j]);
            }
        }
    }
    float *dst = OUT ? (seg == (REV ? 0 : p.S - 1) ? p.last : nullptr) : p.agg;
    if (dst && has_state) {
        const size_t base = OUT ? (size_t)bh * D * D : ((size_t)bh * p.S + seg) * D * D;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) dst[state_at(base, i, j)] = st[i][j];
    }
    if (!OUT && tid == 0 && zsp == 0) p.segdec[(size_t)bh * p.S + seg] = exp2_diff(seglog, zero);
}

// Segment starts in place of the segments' aggregates: the carry over a segment is
// linear, S(end) = dec S(start) + A, so with few heads the sequences are cut into S
// segments whose aggregates A (states from zero) are formed in parallel, and this
// kernel, element-wise and in order, leaves in each entry the state in force where
// the segment begins (rev: behind its end).  init nullable [B*H][D2].
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
    constexpr int kB = 8;   // loads of eight segments go out before the first store
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
    int BH, T, N, ZS;
};

// dbeta and dgate of one chunk from its pair terms (top of this file).
// grid (N, B*H), block kLinThreads.
template <typename T, int D>
__global__ void __launch_bounds__(kLinThreads) k_linear_pairs(const LinPairs p) {
    constexpr int C = kLinC, LD = D + 4;
    extern __shared__ float4 lin_smem[];
    Log2Sum *s_l = reinterpret_cast<Log2Sum *>(lin_smem);
    float *qs = reinterpret_cast<float *>(s_l + C), *ks = qs + C * LD, *vs = ks + C * LD,
          *os = vs + C * LD;
    float *As = os + C * LD;                       // [C][C + 1]
    float *s_g = As + C * (C + 1), *s_ze = s_g + C, *s_ge = s_ze + C;
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = blockIdx.x, bh = blockIdx.y, t0 = n * C;
    const size_t head = (size_t)bh * p.T, rowsall = (size_t)p.BH * p.T;
    {
        LinTile<T, D> tq, tk, tv, to;
        tq.load(static_cast<const T *>(p.q) + head * D, t0, p.T, D, 0);
        tk.load(static_cast<const T *>(p.k) + head * D, t0, p.T, D, 0);
        tv.load(static_cast<const T *>(p.v) + head * D, t0, p.T, D, 0);
        to.load(static_cast<const T *>(p.d_o) + head * D, t0, p.T, D, 0);
        tq.store(qs, LD);
        tk.store(ks, LD);
        tv.store(vs, LD);
        to.store(os, LD);
    }
    float eta = 0.f;
    if (warp == 0) {
        s_l[lane] = lin_log_prefix(p.beta + head, t0, p.T, kLinLog2MinBwd);
        float zeta = 0.f, g = 0.f;
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
        for (int z = 0; z < p.ZS; ++z) d += p.fdot[((size_t)z * p.BH + bh) * p.N + n];
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
// first use.
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
