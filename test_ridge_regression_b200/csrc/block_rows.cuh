// The row operations on either side of the layer inside its block: unit rows of
// q and k, sigmoid gates and the head-major layout before it; residual, RMS
// norm, SiLU gate and the token-major layout after it; and their gradients.
//
// Method: "Gated KalmaNet" (arXiv 2511.21016), pith.science page, Fig. 2 (the
// block normalises q and k by their l2 norm before the layer).  Per row x of D
// elements, with r = (|x|^2 + eps)^-1/2:
//   y = r x,              dx = r (dy - y (y . dy))
// and per row u = o + skip_h v of the output, r = (|u|^2 / D + eps)^-1/2, n = r u:
//   y = n w silu(z),      dn = dy w silu(z),  du = r (dn - n (n . dn) / D),
//   dz = dy n w silu'(z), dw = sum dy n silu(z),  dskip_h = sum du . v,  dv = skip_h du.
//
// Every kernel reads each row once and writes each result once: memory traffic
// bounds them.  A row is spread over D * sizeof(T) / 16 neighbouring lanes, 16
// bytes a lane, so a warp's loads and stores are whole rows (64 to 512 bytes
// each) whichever of the two layouts a side has, and a row's sum is a few
// shuffles.  A block takes a tile of tokens x heads (8 heads where there are as
// many), so that it touches kilobytes in a run on either side, and finds the tile with
// one division.  A lane group's rows (RPT) are all loaded before the first is used; more
// of them, or fewer, were slower (block_out and block_in's gradient: 1, 2, 4 rows 27, 25,
// 30 us and 70, 55, 68).  bf16 B8 T2048 H8 D128, with gate, z and skip (fp32: 62, 90, 44, 84 us,
// 87 % of the copy rate and more):
//   block_in       32 us, 203 MB, 98 % of the copy rate (a division a row: 88)
//   its gradient   54 us, 271 MB, 77 %: issue slots 75 % used
//   block_out      25 us, 134 MB, 84 % (row by row: 43)
//   its gradient   51 us, 235 MB, 71 %: 115 registers for dw and the next rows, two CTAs an SM
// All sums are fp32; the gradients of what is shared by many rows (biases, w, skip) are
// summed per block and then over the blocks in a fixed order, so results do not
// depend on scheduling.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace gka {

constexpr int kRowThreads = 256;

// [B, T, heads, D] rows (or [B, T, heads] scalars) with element strides.
struct StridedRows {
    const void *ptr;
    long long sb, st, sh;
};

// 16 bytes of a row as floats and back, rounded once to nearest.
template <typename T>
struct Vec16;
template <>
struct Vec16<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(uint4 v, float *x) {
        x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ void load(const float *p, float *x) { unpack(raw(p), x); }
    static __device__ __forceinline__ uint4 raw(const float *p) {
        return __ldg(reinterpret_cast<const uint4 *>(p));
    }
    static __device__ __forceinline__ uint4 pack(const float *x) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
    }
    static __device__ __forceinline__ void store(float *p, const float *x) {
        *reinterpret_cast<uint4 *>(p) = pack(x);
    }
};
template <>
struct Vec16<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ uint4 raw(const __nv_bfloat16 *p) {
        return __ldg(reinterpret_cast<const uint4 *>(p));
    }
    static __device__ __forceinline__ void unpack(uint4 v, float *x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void load(const __nv_bfloat16 *p, float *x) { unpack(raw(p), x); }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float *x) {
        *reinterpret_cast<uint4 *>(p) = pack(x);
    }
    static __device__ __forceinline__ uint4 pack(const float *x) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Sum over the LPR neighbouring lanes of a row.
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ float sigmoid_f(float x) { return 1.f / (1.f + expf(-x)); }
// For rows that are rounded to bf16 in the end the hardware's exponential and quotient do: a
// relative error of (4 + 1.2 |x|) 2^-23, 2^-16 at the far end (x = -90, where x sigmoid(x) is near
// bf16's smallest normal) against the rounding's 2^-8.  From e^-|x|, so that neither the sum nor
// the quotient leaves the range where the hardware's quotient is one.
template <typename T>
__device__ __forceinline__ float sigmoid_row(float x) {
    if constexpr (sizeof(T) == 2) {
        const float e = __expf(-fabsf(x));
        return __fdividef(x < 0.f ? e : 1.f, 1.f + e);
    }
    return sigmoid_f(x);
}

// Tile of a block of R rows: 2^tb tokens x R / 2^tb slots; tiles count tokens first.
struct RowTile {
    int tb;             // log2 of the tile's tokens
    unsigned tcount;    // tiles along t
    unsigned scount;    // tiles along the slots
};
// Row i of the block's tile; false past the end.
struct SlotRow {
    int b, slot, t;
    bool in;
};
struct TileAt {
    int b, s0, t0;
};
template <int R>
__device__ __forceinline__ TileAt tile_at(const RowTile &g, unsigned blk) {
    const unsigned q = blk / g.tcount, b = q / g.scount;
    return {(int)b, (int)((q - b * g.scount) * (R >> g.tb)), (int)((blk - q * g.tcount) << g.tb)};
}
__device__ __forceinline__ SlotRow tile_row(const RowTile &g, const TileAt &a, int i, int T, int slots) {
    SlotRow s;
    s.b = a.b;
    s.t = a.t0 + (i & ((1 << g.tb) - 1));
    s.slot = a.s0 + (i >> g.tb);
    s.in = s.t < T && s.slot < slots;
    return s;
}

// ---------------------------------------------------------------------------
// Before the layer
// ---------------------------------------------------------------------------
struct BlockInArgs {
    StridedRows q, k, v, beta_logit, gate_logit;   // gate_logit.ptr nullable
    const float *beta_bias, *gate_bias;            // [H], nullable
    const int *lengths;                            // [B], nullable
    int B, T, H, Hk;
    float eps;
    unsigned row_blocks;   // blocks of the row part; the rest do the gates
    RowTile qtile, ktile;
};

// The block's rows are of one kind, queries, keys or values, each with its own tiles.
struct KindAt {
    int kind, heads;   // 0 q, 1 k, 2 v
    TileAt at;
};
template <int R>
__device__ __forceinline__ KindAt kind_at(const BlockInArgs &a) {
    KindAt k;
    unsigned blk = blockIdx.x;
    const unsigned nq = a.qtile.tcount * a.qtile.scount * a.B, nk = a.ktile.tcount * a.ktile.scount * a.B;
    k.kind = blk < nq ? 0 : blk < nq + nk ? 1 : 2;
    blk -= k.kind == 0 ? 0 : k.kind == 1 ? nq : nq + nk;
    k.heads = k.kind ? a.Hk : a.H;
    k.at = tile_at<R>(k.kind ? a.ktile : a.qtile, blk);
    return k;
}

// grid: row_blocks blocks of rows (RPT rows a lane group), then ceil(B*H*T / 256)
// blocks of gates.
template <typename T, int D, int RPT>
__global__ void __launch_bounds__(kRowThreads)
k_block_in(const BlockInArgs a, T *__restrict__ qo, T *__restrict__ ko, T *__restrict__ vo,
           float *__restrict__ beta, float *__restrict__ gate) {
    using V = Vec16<T>;
    constexpr int LPR = D / V::N, GROUPS = kRowThreads / LPR;
    if (blockIdx.x >= a.row_blocks) {
        // gates: beta = sigmoid(logit + bias), padding keeps the state (beta 1, gate 0)
        const size_t n = (size_t)a.B * a.H * a.T;
        const size_t i = (size_t)(blockIdx.x - a.row_blocks) * kRowThreads + threadIdx.x;
        if (i >= n) return;
        const size_t bh = i / (unsigned)a.T;
        const int t = (int)(i - bh * (unsigned)a.T), b = (int)(bh / (unsigned)a.H);
        const int h = (int)(bh - (size_t)b * (unsigned)a.H);
        const bool ok = !a.lengths || t < a.lengths[b];
        const T *bl = static_cast<const T *>(a.beta_logit.ptr) + b * a.beta_logit.sb +
                      t * a.beta_logit.st + h * a.beta_logit.sh;
        beta[i] = ok ? sigmoid_f(load_f(bl) + (a.beta_bias ? a.beta_bias[h] : 0.f)) : 1.f;
        if (gate) {
            float g = 1.f;
            if (a.gate_logit.ptr) {
                const T *gl = static_cast<const T *>(a.gate_logit.ptr) + b * a.gate_logit.sb +
                              t * a.gate_logit.st + h * a.gate_logit.sh;
                g = sigmoid_f(load_f(gl) + (a.gate_bias ? a.gate_bias[h] : 0.f));
            }
            gate[i] = ok ? g : 0.f;
        }
        return;
    }
    const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR;
    const KindAt k = kind_at<GROUPS * RPT>(a);
    const RowTile &tile = k.kind ? a.ktile : a.qtile;
    const StridedRows &in = k.kind == 0 ? a.q : k.kind == 1 ? a.k : a.v;
    T *out = k.kind == 0 ? qo : k.kind == 1 ? ko : vo;
    const T *src = static_cast<const T *>(in.ptr) + k.at.b * in.sb + lane * V::N;
    const int rep = k.kind ? a.H / a.Hk : 1;
    const int len = a.lengths ? min(a.lengths[k.at.b], a.T) : a.T;
    uint4 x[RPT];
    // every load of the group's rows goes out before the first sum
#pragma unroll
    for (int j = 0; j < RPT; ++j) {
        const SlotRow s = tile_row(tile, k.at, grp + j * GROUPS, len, k.heads);
        x[j] = make_uint4(0u, 0u, 0u, 0u);
        if (s.in) x[j] = V::raw(src + s.t * in.st + s.slot * in.sh);
    }
#pragma unroll
    for (int j = 0; j < RPT; ++j) {
        const SlotRow s = tile_row(tile, k.at, grp + j * GROUPS, a.T, k.heads);
        uint4 y = x[j];
        if (k.kind < 2) {   // values pass as they are
            float f[V::N], ss = 0.f;
            V::unpack(y, f);
#pragma unroll
            for (int i = 0; i < V::N; ++i) ss = fmaf(f[i], f[i], ss);
            ss = row_sum<LPR>(ss);
            const float rn = s.t < len ? rsqrtf(ss + a.eps) : 0.f;   // padding stays zero, with eps = 0 too
#pragma unroll
            for (int i = 0; i < V::N; ++i) f[i] *= rn;
            y = V::pack(f);
        }
        if (!s.in) continue;
        T *dst = out + (((size_t)k.at.b * a.H + s.slot * rep) * a.T + s.t) * D + lane * V::N;
        for (int h = 0; h < rep; ++h, dst += (size_t)a.T * D) *reinterpret_cast<uint4 *>(dst) = y;
    }
}

struct BlockInGrad {
    const void *dq, *dk, *dv;        // [B, H, T, D]
    const float *dbeta, *dgate;      // [B, H, T]; dgate nullable
    void *xq, *xk, *xv;              // gradients of the raw rows, dense [B, T, heads, D]
    void *xbeta, *xgate;             // gradients of the logits, dense [B, T, H]
    float *part;                     // [2][H][gblk] sums of the logits' gradients
    int gblk;                        // gate blocks per head
};

// grid: row_blocks blocks of rows, then H * gblk blocks of gates (each a run of
// the B*T tokens of one head).
template <typename T, int D, int RPT>
__global__ void __launch_bounds__(kRowThreads)
k_block_in_grad(const BlockInArgs a, const BlockInGrad g) {
    griddep_launch_dependents();
    using V = Vec16<T>;
    constexpr int LPR = D / V::N, GROUPS = kRowThreads / LPR;
    const int lane = threadIdx.x % LPR;
    if (blockIdx.x >= a.row_blocks) {
        const unsigned id = blockIdx.x - a.row_blocks;
        const int h = (int)(id / (unsigned)g.gblk), part = (int)(id % (unsigned)g.gblk);
        const size_t n = (size_t)a.B * a.T;
        const size_t e0 = n * part / g.gblk, e1 = n * (part + 1) / g.gblk;
        const float bb = a.beta_bias ? a.beta_bias[h] : 0.f;
        const float gb = a.gate_bias ? a.gate_bias[h] : 0.f;
        float sb = 0.f, sg = 0.f;
        // token e of the head's run, its (b, t) carried along
        const size_t eb = (e0 + threadIdx.x) / (unsigned)a.T;
        unsigned t = (unsigned)(e0 + threadIdx.x - eb * (unsigned)a.T);
        size_t b = eb;
        for (size_t e = e0 + threadIdx.x; e < e1; e += kRowThreads, t += kRowThreads) {
            if (t >= (unsigned)a.T) {
                const unsigned q = t / (unsigned)a.T;
                b += q;
                t -= q * (unsigned)a.T;
            }
            const bool ok = !a.lengths || (int)t < a.lengths[b];
            const size_t src = (b * a.H + h) * a.T + t, dst = e * a.H + h;
            float d = 0.f, dg = 0.f;
            if (ok) {
                // sigma'(x) = sigma(x) sigma(-x): no difference from 1 is formed
                const float x = bb + load_f(static_cast<const T *>(a.beta_logit.ptr) +
                                            b * a.beta_logit.sb + t * a.beta_logit.st +
                                            h * a.beta_logit.sh);
                d = g.dbeta[src] * sigmoid_f(x) * sigmoid_f(-x);
                if (g.xgate) {
                    const float y = gb + load_f(static_cast<const T *>(a.gate_logit.ptr) +
                                                b * a.gate_logit.sb + t * a.gate_logit.st +
                                                h * a.gate_logit.sh);
                    dg = g.dgate[src] * sigmoid_f(y) * sigmoid_f(-y);
                }
            }
            store_f(static_cast<T *>(g.xbeta) + dst, d);
            if (g.xgate) store_f(static_cast<T *>(g.xgate) + dst, dg);
            sb += d;
            sg += dg;
        }
        __shared__ float red[2][kRowThreads / 32];
        sb = warp_sum(sb);
        sg = warp_sum(sg);
        if ((threadIdx.x & 31) == 0) {
            red[0][threadIdx.x >> 5] = sb;
            red[1][threadIdx.x >> 5] = sg;
        }
        __syncthreads();
        if (threadIdx.x < 2) {
            float s = 0.f;
            for (int w = 0; w < kRowThreads / 32; ++w) s += red[threadIdx.x][w];
            g.part[((size_t)threadIdx.x * a.H + h) * g.gblk + part] = s;
        }
        return;
    }
    const int grp = threadIdx.x / LPR;
    const KindAt k = kind_at<GROUPS * RPT>(a);
    const RowTile &tile = k.kind ? a.ktile : a.qtile;
    const StridedRows &in = k.kind ? a.k : a.q;
    const T *src = static_cast<const T *>(in.ptr) + k.at.b * in.sb + lane * V::N;
    const T *up = static_cast<const T *>(k.kind == 0 ? g.dq : k.kind == 1 ? g.dk : g.dv) + lane * V::N;
    T *out = static_cast<T *>(k.kind == 0 ? g.xq : k.kind == 1 ? g.xk : g.xv) + lane * V::N;
    const int rep = k.kind ? a.H / a.Hk : 1;
    const int len = a.lengths ? min(a.lengths[k.at.b], a.T) : a.T;
    uint4 x[RPT], d[RPT];
    float dy[RPT][V::N];
    // the loads of all the group's rows go out together
    auto grads = [&](int h) {
#pragma unroll
        for (int j = 0; j < RPT; ++j) {
            const SlotRow s = tile_row(tile, k.at, grp + j * GROUPS, len, k.heads);
            d[j] = make_uint4(0u, 0u, 0u, 0u);
            if (s.in) d[j] = V::raw(up + (((size_t)k.at.b * a.H + s.slot * rep + h) * a.T + s.t) * D);
        }
    };
#pragma unroll
    for (int j = 0; j < RPT; ++j) {
        const SlotRow s = tile_row(tile, k.at, grp + j * GROUPS, len, k.heads);
        x[j] = make_uint4(0u, 0u, 0u, 0u);
        if (s.in && k.kind < 2) x[j] = V::raw(src + s.t * in.st + s.slot * in.sh);
    }
    grads(0);
#pragma unroll
    for (int j = 0; j < RPT; ++j) V::unpack(d[j], dy[j]);
    // a shared key or value head collects the gradients of its group
    for (int h = 1; h < rep; ++h) {
        grads(h);
#pragma unroll
        for (int j = 0; j < RPT; ++j) {
            float y[V::N];
            V::unpack(d[j], y);
#pragma unroll
            for (int i = 0; i < V::N; ++i) dy[j][i] += y[i];
        }
    }
#pragma unroll
    for (int j = 0; j < RPT; ++j) {
        const SlotRow s = tile_row(tile, k.at, grp + j * GROUPS, a.T, k.heads);
        if (k.kind < 2) {
            float f[V::N], ss = 0.f, xd = 0.f;
            V::unpack(x[j], f);
#pragma unroll
            for (int i = 0; i < V::N; ++i) {
                ss = fmaf(f[i], f[i], ss);
                xd = fmaf(f[i], dy[j][i], xd);
            }
            ss = row_sum<LPR>(ss);
            xd = row_sum<LPR>(xd);
            const float rn = s.t < len ? rsqrtf(ss + a.eps) : 0.f;   // (as in k_block_in)
            const float c = rn * rn * xd;                            // r (dy - r x (r x . dy))
#pragma unroll
            for (int i = 0; i < V::N; ++i) dy[j][i] = rn * (dy[j][i] - c * f[i]);
        }
        if (s.in) V::store(out + (((size_t)k.at.b * a.T + s.t) * k.heads + s.slot) * D, dy[j]);
    }
}

// out[i] = sum of part[i][0..n), i < count, one block per output, in a fixed order; two such
// arrays (the second's count may be 0, either's out NULL).  grid count0 + count1, launched as
// the programmatic dependent of the kernel that writes the parts.
struct SumsOf {
    const float *part;
    int count, n;
    float *out;
};
__global__ void __launch_bounds__(128) k_block_sums(const SumsOf a, const SumsOf b) {
    __shared__ float red[4];
    griddep_wait();
    const bool first = (int)blockIdx.x < a.count;
    const SumsOf &s = first ? a : b;
    const int i = (int)blockIdx.x - (first ? 0 : a.count);
    if (!s.out) return;
    float x = 0.f;
    for (int e = threadIdx.x; e < s.n; e += 128) x += s.part[(size_t)i * s.n + e];
    x = warp_sum(x);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    if (threadIdx.x == 0) s.out[i] = red[0] + red[1] + red[2] + red[3];
}

// ---------------------------------------------------------------------------
// After the layer
// ---------------------------------------------------------------------------
struct BlockOutArgs {
    const void *o, *v;         // [B, H, T, D]; v nullable
    StridedRows z;             // [B, T, H, D], ptr nullable
    const float *w, *skip;     // [D]; [H], non-null exactly when v is
    int B, T, H;
    float eps;
    RowTile tile;              // (forward)
};

template <typename T, int D, int RPT>
__global__ void __launch_bounds__(kRowThreads)
k_block_out(const BlockOutArgs a, T *__restrict__ y) {
    using V = Vec16<T>;
    constexpr int LPR = D / V::N, GROUPS = kRowThreads / LPR;
    const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR;
    const TileAt at = tile_at<GROUPS * RPT>(a.tile, blockIdx.x);
    float w[V::N];
#pragma unroll
    for (int i = 0; i < V::N; i += 4) Vec16<float>::load(a.w + lane * V::N + i, w + i);
    uint4 o[RPT], v[RPT], z[RPT];   // the loads of all the group's rows go out together
    float sk[RPT];
#pragma unroll
    for (int j = 0; j < RPT; ++j) {
        const SlotRow s = tile_row(a.tile, at, grp + j * GROUPS, a.T, a.H);
        o[j] = v[j] = z[j] = make_uint4(0u, 0u, 0u, 0u);
        sk[j] = 0.f;
        if (!s.in) continue;
        const size_t r = (((size_t)s.b * a.H + s.slot) * a.T + s.t) * D + lane * V::N;
        o[j] = V::raw(static_cast<const T *>(a.o) + r);
        if (a.z.ptr)
            z[j] = V::raw(static_cast<const T *>(a.z.ptr) + s.b * a.z.sb + s.t * a.z.st + s.slot * a.z.sh +
                          lane * V::N);
        if (a.v) {
            v[j] = V::raw(static_cast<const T *>(a.v) + r);
            sk[j] = a.skip[s.slot];
        }
    }
#pragma unroll
    for (int j = 0; j < RPT; ++j) {
        const SlotRow s = tile_row(a.tile, at, grp + j * GROUPS, a.T, a.H);
        float u[V::N], g[V::N], ss = 0.f;
        V::unpack(o[j], u);
        if (a.v) {
            V::unpack(v[j], g);
#pragma unroll
            for (int i = 0; i < V::N; ++i) u[i] = fmaf(sk[j], g[i], u[i]);
        }
#pragma unroll
        for (int i = 0; i < V::N; ++i) ss = fmaf(u[i], u[i], ss);
        ss = row_sum<LPR>(ss);
        if (!s.in) continue;
        const float rn = rsqrtf(ss * (1.f / D) + a.eps);
        V::unpack(z[j], g);
#pragma unroll
        for (int i = 0; i < V::N; ++i) {
            u[i] *= rn * w[i];
            if (a.z.ptr) u[i] *= g[i] * sigmoid_row<T>(g[i]);
        }
        V::store(y + (((size_t)s.b * a.T + s.t) * a.H + s.slot) * D + lane * V::N, u);
    }
}

struct BlockOutGrad {
    const void *dy;            // [B, T, H, D]
    void *d_o, *dv;            // [B, H, T, D]; dv with a.v
    void *dz;                  // [B, T, H, D], with a.z
    float *wpart;              // [D][H * blk] sums of dw
    float *spart;              // [H][blk] sums of dskip (with a.v)
    int blk;                   // blocks per head
};

// grid (blk, H): block (i, h) walks a run of head h's B*T rows, so that dw and
// dskip_h stay in registers to its end.
template <typename T, int D>
__global__ void __launch_bounds__(kRowThreads)
k_block_out_grad(const BlockOutArgs a, const BlockOutGrad g) {
    griddep_launch_dependents();
    using V = Vec16<T>;
    constexpr int LPR = D / V::N, GROUPS = kRowThreads / LPR;
    const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR, h = blockIdx.y;
    const size_t n = (size_t)a.B * a.T;
    const size_t e0 = n * blockIdx.x / g.blk, e1 = n * (blockIdx.x + 1) / g.blk;
    const float sk = a.v ? a.skip[h] : 0.f;
    float w[V::N], dw[V::N], ds = 0.f;
#pragma unroll
    for (int i = 0; i < V::N; ++i) {
        w[i] = a.w[lane * V::N + i];
        dw[i] = 0.f;
    }
    // every lane of a warp runs the same number of rounds: the row sums are shuffles
    // over the whole warp
    const int rounds = (int)((e1 - e0 + GROUPS - 1) / GROUPS);
    size_t b = (e0 + grp) / (unsigned)a.T;
    unsigned t = (unsigned)(e0 + grp - b * (unsigned)a.T);
    // the next round's rows are on their way while this one's are worked on
    struct Rows {
        uint4 o, v, z, dy;
    } nx;
    size_t hm, tm;
    bool in;
    auto fetch = [&](int k) {
        if (t >= (unsigned)a.T) {
            const unsigned q = t / (unsigned)a.T;
            b += q;
            t -= q * (unsigned)a.T;
        }
        in = e0 + (size_t)k * GROUPS + grp < e1;
        hm = ((b * a.H + h) * a.T + t) * D + lane * V::N;
        tm = ((b * (unsigned)a.T + t) * a.H + h) * D + lane * V::N;
        nx.o = nx.v = nx.z = nx.dy = make_uint4(0u, 0u, 0u, 0u);
        if (in) {
            nx.o = V::raw(static_cast<const T *>(a.o) + hm);
            nx.dy = V::raw(static_cast<const T *>(g.dy) + tm);
            if (a.v) nx.v = V::raw(static_cast<const T *>(a.v) + hm);
            if (a.z.ptr)
                nx.z = V::raw(static_cast<const T *>(a.z.ptr) + b * a.z.sb + t * a.z.st + h * a.z.sh +
                              lane * V::N);
        }
        t += GROUPS;
    };
    if (rounds > 0) fetch(0);
    for (int k = 0; k < rounds; ++k) {
        float u[V::N], v[V::N], z[V::N], dy[V::N];
        V::unpack(nx.o, u);
        V::unpack(nx.v, v);
        V::unpack(nx.z, z);
        V::unpack(nx.dy, dy);
        const size_t hm0 = hm, tm0 = tm;
        const bool in0 = in;
        if (k + 1 < rounds) fetch(k + 1);
        if (a.v) {
#pragma unroll
            for (int i = 0; i < V::N; ++i) u[i] = fmaf(sk, v[i], u[i]);
        }
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < V::N; ++i) ss = fmaf(u[i], u[i], ss);
        ss = row_sum<LPR>(ss);
        const float rn = in0 ? rsqrtf(ss * (1.f / D) + a.eps) : 0.f;   // past the end zeros, with eps = 0 too
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < V::N; ++i) {
            u[i] *= rn;   // n
            if (a.z.ptr) {
                const float sg = sigmoid_row<T>(z[i]);
                // d silu(z) / dz = s (1 + z (1 - s)); where 1 - s cancels, it is added to 1
                const float dsil = sg * fmaf(z[i], 1.f - sg, 1.f);
                const float dyi = dy[i];
                dy[i] = dyi * (z[i] * sg);
                z[i] = dyi * u[i] * w[i] * dsil;
            }
            dw[i] = fmaf(dy[i], u[i], dw[i]);   // (zeros past the end)
            dy[i] *= w[i];   // dn
            dot = fmaf(dy[i], u[i], dot);
        }
        dot = row_sum<LPR>(dot) * (1.f / D);
#pragma unroll
        for (int i = 0; i < V::N; ++i) dy[i] = rn * (dy[i] - u[i] * dot);   // du
        if (!in0) continue;
        V::store(static_cast<T *>(g.d_o) + hm0, dy);
        if (a.z.ptr) V::store(static_cast<T *>(g.dz) + tm0, z);
        if (a.v) {
#pragma unroll
            for (int i = 0; i < V::N; ++i) {
                ds = fmaf(dy[i], v[i], ds);
                dy[i] *= sk;
            }
            V::store(static_cast<T *>(g.dv) + hm0, dy);
        }
    }
    __shared__ float red[GROUPS][D];
    __shared__ float reds[kRowThreads / 32];
#pragma unroll
    for (int i = 0; i < V::N; ++i) red[grp][lane * V::N + i] = dw[i];
    ds = warp_sum(ds);
    if ((threadIdx.x & 31) == 0) reds[threadIdx.x >> 5] = ds;
    __syncthreads();
    if (threadIdx.x < D) {
        float s = 0.f;
        for (int i = 0; i < GROUPS; ++i) s += red[i][threadIdx.x];
        g.wpart[((size_t)threadIdx.x * a.H + h) * g.blk + blockIdx.x] = s;
    }
    if (threadIdx.x == 0 && a.v) {
        float s = 0.f;
        for (int i = 0; i < kRowThreads / 32; ++i) s += reds[i];
        g.spart[(size_t)h * g.blk + blockIdx.x] = s;
    }
}

}  // namespace gka
