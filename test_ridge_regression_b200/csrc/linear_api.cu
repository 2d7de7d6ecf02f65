// C ABI of the gated linear recurrence and of the block's row operations:
// argument checks, workspace layout, launches.  The contract of every entry
// point is in include/gka.h.
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "../../include/gka.h"
#include "block_rows.cuh"
#include "host.cuh"
#include "linear_simt.cuh"
#include "linear_tc.cuh"

namespace gka {

constexpr int kSms = 148;   // SMs of the one GPU this library is built for

static bool valid_dtype(gka_dtype dt) { return dt == GKA_F32 || dt == GKA_BF16; }

// Launches `kern` as the programmatic dependent of the kernel before it (`pdl`): it may set
// itself up while that one ends, and waits for it on the device.
template <typename K, typename... Args>
static int launch_after(K kern, dim3 grid, int threads, size_t smem, bool pdl, cudaStream_t s, Args... args) {
    cudaError_t e;
    if (smem && (e = set_smem(kern, smem)) != cudaSuccess) return cuda_fail(e);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    if ((e = cudaLaunchKernelEx(&cfg, kern, args...)) != cudaSuccess) return cuda_fail(e);
    return GKA_OK;
}

// ---------------------------------------------------------------------------
// Gated linear recurrence
// ---------------------------------------------------------------------------
struct LinLayout {
    bool tc;                                   // tensor-core path
    int N, S, ZS;                              // chunks, segments, column splits
    int dots, fdots;                           // planes of the dbeta terms' partial sums
    size_t agg, segdec;                        // segment aggregates, decays (S > 1)
    size_t tab;                                // decay tables (tensor cores), forward's then backward's
    size_t states, zeta, eta, fdot;            // backward
    size_t total;
};

// Segments per sequence: enough CTAs for every SM, whole chunks each.  A few chunks in a row are
// faster than the two launches more: 4 heads of D = 128, device time without and with segments, on
// the tensor cores 5 chunks 18.2 and 17.2 us (gradients 49 and 54), 6 chunks 20.9 and 17.3 (56
// and 54); on CUDA cores 2 chunks 21.2 and 24.4 (47 and 48), 3 chunks 29 and 24.5 (66 and 49).
static int lin_segments(int ctas, int N, int D, bool tc) {
    const int S = ctas > 0 ? kSms * (tc ? 1 : lin_per_sm(D)) / ctas : 1;
    return N <= (tc ? 5 : 2) ? 1 : std::max(1, std::min(S, N));
}

static int lin_layout(int B, int H, int T, int D, gka_dtype dt, bool bwd, LinLayout *L) {
    if (B < 0 || H < 0 || T < 0 || !valid_dtype(dt)) return GKA_ERR_INVALID_ARG;
    if (!supported_d(D)) return GKA_ERR_UNSUPPORTED;
    if ((size_t)B * H > 65535) return GKA_ERR_UNSUPPORTED;   // grid limit
    const size_t BH = (size_t)B * H, st = sizeof(float) * (size_t)D * D;
    L->tc = dt == GKA_BF16;
    const int C = L->tc ? kLtC : kLinC;
    L->ZS = lt_splits(D);   // of 64 columns, in both forms
    L->N = (int)(((long long)T + C - 1) / C);
    L->S = lin_segments((int)BH * L->ZS, L->N, D, L->tc);
    L->dots = L->tc ? kLtDots * L->ZS : D / 32;
    L->fdots = L->tc ? kLtFdots * L->ZS : L->ZS;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = round256(off + bytes);
        return at;
    };
    L->agg = take(L->S > 1 ? BH * L->S * st : 0);
    L->segdec = take(L->S > 1 ? BH * L->S * sizeof(float) : 0);
    L->tab = take(L->tc ? (bwd ? 2 : 1) * BH * L->N * kLtTabF * sizeof(float) : 0);
    L->states = L->zeta = L->eta = L->fdot = off;
    if (bwd) {
        L->states = take(BH * L->N * st);
        L->zeta = take(L->dots * BH * T * sizeof(float));
        L->eta = take(L->dots * BH * T * sizeof(float));
        L->fdot = take(L->fdots * BH * L->N * sizeof(float));
    }
    L->total = off;
    return GKA_OK;
}

template <int D, bool REV, bool OUT>
static int lin_launch(const LinPasses &a, int passes, int prof, cudaStream_t s) {
    const LinPass &p = a.pass[0];
    ProfScope ps(prof, s);
    return launch_after(k_linear_pass<D, REV, OUT>, dim3(passes * (D / LinSmem<D>::ZN), p.BH, p.S), kLinThreads,
                        LinSmem<D>::bytes, true, s, a);
}

// Segment starts for the first pass (S > 1): aggregates, then their scan from `init`.
template <int D, bool REV>
static int lin_starts(LinPasses &a, const LinLayout &L, char *ws, const float *init, int prof,
                      cudaStream_t s) {
    LinPass &p = a.pass[0];
    if (L.S == 1) {
        p.start = init;
        return GKA_OK;
    }
    p.agg = reinterpret_cast<float *>(ws + L.agg);
    p.segdec = reinterpret_cast<float *>(ws + L.segdec);
    if (int rc = lin_launch<D, REV, false>(a, 1, prof, s)) return rc;
    ProfScope ps(prof, s);
    p.start = p.agg;
    return launch_after(k_linear_scan, dim3((D * D + 1023) / 1024, p.BH), 256, 0, true, s, p.agg,
                        (const float *)p.segdec, init, L.S, D * D, (int)REV);
}

struct LinCall {
    const void *q, *k, *v, *d_o;
    const float *beta, *gate, *init, *dlast;
    void *o, *dq, *dk, *dv;
    float *last, *dbeta, *dgate, *dinit;
    int BH, T, D;
    float scale;
    char *ws;
    cudaStream_t s;
};

template <int D>
static int lin_forward(const LinCall &c, const LinLayout &L) {
    LinPasses a = {};
    LinPass &p = a.pass[0];
    p.x = c.q; p.y = c.k; p.z = c.v;
    p.out = c.o;
    p.beta = c.beta; p.gate = c.gate;
    p.scale = c.scale;
    p.log2_min = kLinLog2Min;
    p.BH = c.BH; p.T = c.T; p.N = L.N; p.S = L.S; p.D = c.D;
    p.zy = 1;
    if (int rc = lin_starts<D, false>(a, L, c.ws, c.init, GKA_KERNEL_LINEAR, c.s)) return rc;
    p.last = c.last;
    return lin_launch<D, false, true>(a, 1, GKA_KERNEL_LINEAR, c.s);
}

template <int D>
static int lin_backward(const LinCall &c, const LinLayout &L) {
    constexpr int kProf = GKA_KERNEL_LINEAR_GRAD;
    float *states = reinterpret_cast<float *>(c.ws + L.states);
    float *zeta = reinterpret_cast<float *>(c.ws + L.zeta);
    float *eta = reinterpret_cast<float *>(c.ws + L.eta);
    float *fdot = reinterpret_cast<float *>(c.ws + L.fdot);
    LinPass p = {};
    p.beta = c.beta; p.gate = c.gate;
    p.scale = c.scale;
    p.log2_min = kLinLog2MinBwd;
    p.BH = c.BH; p.T = c.T; p.N = L.N; p.S = L.S; p.D = c.D;
    // dq, forwards in time; M before every chunk stays for F
    LinPasses a = {};
    LinPass &f = a.pass[0];
    f = p;
    f.x = c.d_o; f.y = c.v; f.z = c.k;
    if (int rc = lin_starts<D, false>(a, L, c.ws, c.init, kProf, c.s)) return rc;
    f.out = c.dq;
    f.xd = c.q;
    f.dot = zeta;
    f.states = states;
    if (int rc = lin_launch<D, false, true>(a, 1, kProf, c.s)) return rc;
    // dv and dk, backwards in time, in one launch
    a = {};
    LinPass &r = a.pass[0], &d = a.pass[1];
    r = p;
    r.x = c.k; r.y = c.q; r.z = c.d_o;
    r.zy = 1;
    if (int rc = lin_starts<D, true>(a, L, c.ws, c.dlast, kProf, c.s)) return rc;
    r.out = c.dv;
    r.xd = c.v;
    r.dot = eta;
    r.last = c.dinit;
    d = p;
    d.x = c.v; d.y = c.d_o; d.z = c.q;
    d.start = r.start;
    d.out = c.dk;
    // dk's state has dq's orientation: F there reads what dq's pass wrote, as it wrote it
    d.states_in = states;
    d.fdot = fdot;
    if (int rc = lin_launch<D, true, true>(a, 2, kProf, c.s)) return rc;
    LinPairs w = {};
    w.q = c.q; w.k = c.k; w.v = c.v; w.d_o = c.d_o;
    w.beta = c.beta; w.gate = c.gate;
    w.zeta = zeta; w.eta = eta; w.fdot = fdot;
    w.dbeta = c.dbeta; w.dgate = c.dgate;
    w.scale = c.scale;
    w.BH = c.BH; w.T = c.T; w.N = L.N; w.ZS = L.dots; w.FS = L.fdots;
    ProfScope ps(kProf, c.s);
    return launch_after(k_linear_pairs<D>, dim3(L.N, c.BH), kLinThreads, lin_pairs_smem<D>(), true, c.s, w);
}

// ---------------------------------------------------------------------------
// The same calls on the tensor cores
// ---------------------------------------------------------------------------
// [B*H][T][D] bf16 in boxes of 64 columns x 128 tokens of one head, 128-byte
// swizzle; tokens past T and columns past D read as zeros and are not written.
static int head_map(CUtensorMap *m, const void *base, int T, int BH, int D) {
    auto enc = tensor_map_encoder();
    if (!enc) return cuda_fail(cudaErrorNotSupported);
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)T, (cuuint64_t)BH};
    cuuint64_t strides[2] = {2 * (cuuint64_t)D, 2 * (cuuint64_t)D * T};
    cuuint32_t box[3] = {64, kLtC, 1}, es[3] = {1, 1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims,
                           strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? GKA_OK : cuda_fail(cudaErrorInvalidValue);
}

// Every chunk's decay tables for one direction, into the workspace.
template <bool REV>
static int lin_tc_tables(LinTcArgs &a, int passes, const LinLayout &L, char *ws, int prof, cudaStream_t s) {
    const LinPass &p = a.pass[0].p;
    float *tab = reinterpret_cast<float *>(ws + L.tab) + (REV ? (size_t)p.BH * L.N * kLtTabF : 0);
    for (int i = 0; i < passes; ++i) a.pass[i].tab = tab;
    ProfScope ps(prof, s);
    return launch_after(k_linear_tables<REV>, dim3((unsigned)p.BH * (unsigned)L.N), 32, 0, true, s, p.beta, p.gate, tab,
                        L.N, p.T, p.scale, p.log2_min);
}

// `pdl`: the kernel before is the tables'.
template <bool REV, bool GRAD>
static int lin_tc_launch(const LinTcArgs &a, int passes, bool pdl, int prof, cudaStream_t s) {
    int *flag = nullptr;
    if (int rc = timeout_flag_ptr(&flag)) return rc;
    const LinPass &p = a.pass[0].p;
    ProfScope ps(prof, s);
    return launch_after(k_linear_tc<REV, GRAD>, dim3(lt_splits(p.D) * passes, p.BH, p.S), kLtThreads, LtSmem::bytes, pdl, s, a, flag);
}

template <bool REV>
static int lin_tc_starts(LinTcArgs &a, const LinLayout &L, char *ws, const float *init, int prof,
                         cudaStream_t s) {
    LinPass &p = a.pass[0].p;
    if (L.S == 1) {
        p.start = init;
        return GKA_OK;
    }
    p.agg = reinterpret_cast<float *>(ws + L.agg);
    p.segdec = reinterpret_cast<float *>(ws + L.segdec);
    int *flag = nullptr;
    if (int rc = timeout_flag_ptr(&flag)) return rc;
    {
        ProfScope ps(prof, s);
        if (int rc = launch_after(k_linear_agg_tc<REV>, dim3(L.ZS, p.BH, L.S), kLtThreads, LaSmem::bytes, true, s,
                                  a.pass[0], flag))
            return rc;
    }
    ProfScope ps(prof, s);
    p.start = p.agg;
    return launch_after(k_linear_scan, dim3((p.D * p.D + 1023) / 1024, p.BH), 256, 0, false, s, p.agg,
                        (const float *)p.segdec, init, L.S, p.D * p.D, (int)REV);
}

static int lin_tc_forward(const LinCall &c, const LinLayout &L) {
    LinTcArgs a = {};
    if (int rc = head_map(&a.pass[0].x, c.q, c.T, c.BH, c.D)) return rc;
    if (int rc = head_map(&a.pass[0].y, c.k, c.T, c.BH, c.D)) return rc;
    if (int rc = head_map(&a.pass[0].z, c.v, c.T, c.BH, c.D)) return rc;
    if (int rc = head_map(&a.pass[0].out, c.o, c.T, c.BH, c.D)) return rc;
    LinPass &p = a.pass[0].p;
    p.beta = c.beta; p.gate = c.gate;
    p.scale = c.scale;
    p.log2_min = kLinLog2Min;
    p.BH = c.BH; p.T = c.T; p.N = L.N; p.S = L.S; p.D = c.D;
    p.zy = 1;
    if (int rc = lin_tc_tables<false>(a, 1, L, c.ws, GKA_KERNEL_LINEAR, c.s)) return rc;
    if (int rc = lin_tc_starts<false>(a, L, c.ws, c.init, GKA_KERNEL_LINEAR, c.s)) return rc;
    p.last = c.last;
    return lin_tc_launch<false, false>(a, 1, L.S == 1, GKA_KERNEL_LINEAR, c.s);
}

static int lin_tc_backward(const LinCall &c, const LinLayout &L) {
    constexpr int kProf = GKA_KERNEL_LINEAR_GRAD;
    CUtensorMap q, k, v, d_o;
    if (int rc = head_map(&q, c.q, c.T, c.BH, c.D)) return rc;
    if (int rc = head_map(&k, c.k, c.T, c.BH, c.D)) return rc;
    if (int rc = head_map(&v, c.v, c.T, c.BH, c.D)) return rc;
    if (int rc = head_map(&d_o, c.d_o, c.T, c.BH, c.D)) return rc;
    LinPass p = {};
    p.beta = c.beta; p.gate = c.gate;
    p.scale = c.scale;
    p.log2_min = kLinLog2MinBwd;
    p.BH = c.BH; p.T = c.T; p.N = L.N; p.S = L.S; p.D = c.D;
    LinPairsTc w = {};
    w.p.zeta = reinterpret_cast<float *>(c.ws + L.zeta);
    w.p.eta = reinterpret_cast<float *>(c.ws + L.eta);
    w.p.fdot = reinterpret_cast<float *>(c.ws + L.fdot);
    // dq, forwards in time; M before every chunk stays for F
    LinTcArgs f = {};
    f.pass[0].x = d_o; f.pass[0].y = v; f.pass[0].z = k;
    f.pass[0].p = p;
    if (int rc = lin_tc_tables<false>(f, 1, L, c.ws, kProf, c.s)) return rc;
    if (int rc = lin_tc_starts<false>(f, L, c.ws, c.init, kProf, c.s)) return rc;
    LinPass &pf = f.pass[0].p;
    if (int rc = head_map(&f.pass[0].out, c.dq, c.T, c.BH, c.D)) return rc;
    pf.xd = c.q;
    pf.dot = const_cast<float *>(w.p.zeta);
    pf.states = reinterpret_cast<float *>(c.ws + L.states);
    if (int rc = lin_tc_launch<false, true>(f, 1, L.S == 1, kProf, c.s)) return rc;
    // dv and dk, backwards in time, in one launch
    LinTcArgs r = {};
    r.pass[0].x = k; r.pass[0].y = q; r.pass[0].z = d_o;
    r.pass[0].p = p;
    r.pass[0].p.zy = 1;
    if (int rc = lin_tc_tables<true>(r, 2, L, c.ws, kProf, c.s)) return rc;
    if (int rc = lin_tc_starts<true>(r, L, c.ws, c.dlast, kProf, c.s)) return rc;
    LinPass &pv = r.pass[0].p, &pk = r.pass[1].p;
    r.pass[1].x = v; r.pass[1].y = d_o; r.pass[1].z = q;
    if (int rc = head_map(&r.pass[0].out, c.dv, c.T, c.BH, c.D)) return rc;
    if (int rc = head_map(&r.pass[1].out, c.dk, c.T, c.BH, c.D)) return rc;
    pk = p;
    pk.start = pv.start;
    // dk's state has dq's orientation: F there reads what dq's pass wrote, as it wrote it
    pk.states_in = pf.states;
    pk.fdot = const_cast<float *>(w.p.fdot);
    pv.xd = c.v;
    pv.dot = const_cast<float *>(w.p.eta);
    pv.last = c.dinit;
    if (int rc = lin_tc_launch<true, true>(r, 2, L.S == 1, kProf, c.s)) return rc;
    w.q = q; w.k = k; w.v = v; w.d_o = d_o;
    w.p.beta = c.beta; w.p.gate = c.gate;
    w.p.dbeta = c.dbeta; w.p.dgate = c.dgate;
    w.p.scale = c.scale;
    w.p.BH = c.BH; w.p.T = c.T; w.p.N = L.N; w.p.ZS = L.dots; w.p.FS = L.fdots;
    w.D = c.D;
    int *flag = nullptr;
    if (int rc = timeout_flag_ptr(&flag)) return rc;
    ProfScope ps(kProf, c.s);
    return launch_after(k_linear_pairs_tc, dim3(L.N, c.BH), kLpThreads, LpSmem::bytes, true, c.s, w, flag);
}

// f(size tag) for the call's head size, f(type tag, size tag) for its type too.
template <typename F>
static int by_size(int D, F f) {
    switch (D) {
        case 32: return f(std::integral_constant<int, 32>());
        case 64: return f(std::integral_constant<int, 64>());
        default: return f(std::integral_constant<int, 128>());
    }
}
template <typename F>
static int by_type(gka_dtype dt, int D, F f) {
    return by_size(D, [&](auto d) { return dt == GKA_BF16 ? f(__nv_bfloat16(), d) : f(float(), d); });
}

// ---------------------------------------------------------------------------
// Block rows
// ---------------------------------------------------------------------------
static int strided(const gka_strided *r, bool rows, int es, StridedRows *out) {
    *out = StridedRows{r->ptr, r->stride_b, r->stride_t, r->stride_h};
    if (!r->ptr) return GKA_ERR_INVALID_ARG;
    if (rows) {
        if (!aligned16(r->ptr)) return GKA_ERR_MISALIGNED;
        if ((r->stride_b * es) % 16 || (r->stride_t * es) % 16 || (r->stride_h * es) % 16)
            return GKA_ERR_MISALIGNED;
    }
    return GKA_OK;
}

static int rows_ok(int B, int T, int H, int Hk, int D, gka_dtype dt, float eps) {
    if (B < 0 || T < 0 || H < 0 || Hk < 0 || !valid_dtype(dt)) return GKA_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || !isfinite(eps)) return GKA_ERR_INVALID_ARG;
    if (H > 0 && (Hk == 0 || H % Hk)) return GKA_ERR_INVALID_ARG;
    if (!supported_d(D)) return GKA_ERR_UNSUPPORTED;
    if (H > 65535) return GKA_ERR_UNSUPPORTED;
    // blocks in one grid dimension
    if ((double)B * T * ((double)H + 2.0 * Hk) > 2e9) return GKA_ERR_UNSUPPORTED;
    return GKA_OK;
}

static int gate_blocks(int B, int T) {
    return (int)std::max<size_t>(1, std::min<size_t>(64, ((size_t)B * T + 1023) / 1024));
}

// Blocks per head of the output norm's gradient: at most eight a SM in all, at
// least four rounds of rows each.
static int out_blocks(int B, int T, int H, int D, gka_dtype dt) {
    const size_t groups = kRowThreads / (D * (dt == GKA_BF16 ? 2 : 4) / 16);
    const size_t rounds = ((size_t)B * T + groups * 4 - 1) / (groups * 4);
    const size_t most = std::max(1, kSms * 8 / std::max(1, H));
    return (int)std::max<size_t>(1, std::min(rounds, most));
}

// Tiles of R rows over B x slots x T: 8 slots by R / 8 tokens, with fewer slots where there
// are not as many, and fewer tokens where the sequences are short.  Returns their number.
static size_t row_tiles(int R, int B, int T, int slots, RowTile *g) {
    int tb = 0;
    while ((1 << tb) < T && (1 << tb) < R && ((1 << tb) < R / 8 || (R >> tb) >= 2 * slots)) ++tb;
    g->tb = tb;
    g->tcount = (unsigned)(((size_t)T + (1u << tb) - 1) >> tb);
    g->scount = (unsigned)((slots + (R >> tb) - 1) / (R >> tb));
    return (size_t)B * g->scount * g->tcount;
}
// Blocks of the block_in rows: queries, then keys, then values.
static unsigned in_blocks(int R, int B, int T, int H, int Hk, BlockInArgs *a) {
    return (unsigned)(row_tiles(R, B, T, H, &a->qtile) + 2 * row_tiles(R, B, T, Hk, &a->ktile));
}
template <typename T, int D>
constexpr int rows_per_block(int rpt) {
    return kRowThreads / (D / Vec16<T>::N) * rpt;
}

}  // namespace gka

using namespace gka;

extern "C" {

size_t gka_linear_forward_workspace_bytes(int B, int H, int T, int D, gka_dtype dt) {
    LinLayout L;
    return lin_layout(B, H, T, D, dt, false, &L) == GKA_OK ? L.total : 0;
}

size_t gka_linear_backward_workspace_bytes(int B, int H, int T, int D, gka_dtype dt) {
    LinLayout L;
    return lin_layout(B, H, T, D, dt, true, &L) == GKA_OK ? L.total : 0;
}

// A state that no token touches: dst = src, or zero.
static int pass_state(float *dst, const float *src, size_t floats, cudaStream_t s) {
    if (!dst || dst == src) return GKA_OK;
    const cudaError_t e =
        src ? cudaMemcpyAsync(dst, src, floats * sizeof(float), cudaMemcpyDeviceToDevice, s)
            : cudaMemsetAsync(dst, 0, floats * sizeof(float), s);
    return e == cudaSuccess ? GKA_OK : cuda_fail(e);
}

int gka_linear_forward(const void *q, const void *k, const void *v, const float *beta,
                       const float *gate, void *o, int B, int H, int T, int D, gka_dtype dt,
                       float scale, const float *initial_state, float *final_state,
                       void *workspace, size_t workspace_bytes, void *stream) {
    LinLayout L;
    if (int rc = lin_layout(B, H, T, D, dt, false, &L)) return rc;
    if (!isfinite(scale)) return GKA_ERR_INVALID_ARG;
    const size_t BH = (size_t)B * H;
    if (BH == 0) return GKA_OK;
    const void *ptrs[] = {q, k, v, beta, gate, o, initial_state, final_state};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GKA_ERR_MISALIGNED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) return pass_state(final_state, initial_state, BH * D * D, s);
    if (!q || !k || !v || !beta || !o) return GKA_ERR_INVALID_ARG;
    if (L.total > 0 && !workspace) return GKA_ERR_INVALID_ARG;
    if ((uintptr_t)workspace & 255u) return GKA_ERR_MISALIGNED;
    if (workspace_bytes < L.total) return GKA_ERR_WORKSPACE_TOO_SMALL;
    LinCall c = {};
    c.q = q; c.k = k; c.v = v; c.beta = beta; c.gate = gate; c.o = o;
    c.init = initial_state; c.last = final_state;
    c.BH = (int)BH; c.T = T; c.D = D; c.scale = scale;
    c.ws = static_cast<char *>(workspace);
    c.s = s;
    if (L.tc) return lin_tc_forward(c, L);
    return by_size(D, [&](auto d) { return lin_forward<decltype(d)::value>(c, L); });
}

int gka_linear_backward(const void *q, const void *k, const void *v, const float *beta,
                        const float *gate, const void *dout, const float *initial_state,
                        const float *dfinal_state, void *dq, void *dk, void *dv, float *dbeta,
                        float *dgate, float *dinitial_state, int B, int H, int T, int D,
                        gka_dtype dt, float scale, void *workspace, size_t workspace_bytes,
                        void *stream) {
    LinLayout L;
    if (int rc = lin_layout(B, H, T, D, dt, true, &L)) return rc;
    if (!isfinite(scale)) return GKA_ERR_INVALID_ARG;
    if ((dgate != nullptr) != (gate != nullptr)) return GKA_ERR_INVALID_ARG;
    const size_t BH = (size_t)B * H;
    if (BH == 0) return GKA_OK;
    const void *ptrs[] = {q, k, v, beta, gate, dout, initial_state, dfinal_state, dq, dk, dv, dbeta,
                          dgate, dinitial_state};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GKA_ERR_MISALIGNED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) return pass_state(dinitial_state, dfinal_state, BH * D * D, s);
    // dk's pass still reads the one while dv's writes the other
    if (dinitial_state && dinitial_state == dfinal_state) return GKA_ERR_INVALID_ARG;
    if (!q || !k || !v || !beta || !dout || !dq || !dk || !dv || !dbeta || !workspace)
        return GKA_ERR_INVALID_ARG;
    if ((uintptr_t)workspace & 255u) return GKA_ERR_MISALIGNED;
    if (workspace_bytes < L.total) return GKA_ERR_WORKSPACE_TOO_SMALL;
    LinCall c = {};
    c.q = q; c.k = k; c.v = v; c.beta = beta; c.gate = gate; c.d_o = dout;
    c.init = initial_state; c.dlast = dfinal_state;
    c.dq = dq; c.dk = dk; c.dv = dv; c.dbeta = dbeta; c.dgate = dgate; c.dinit = dinitial_state;
    c.BH = (int)BH; c.T = T; c.D = D; c.scale = scale;
    c.ws = static_cast<char *>(workspace);
    c.s = s;
    if (L.tc) return lin_tc_backward(c, L);
    return by_size(D, [&](auto d) { return lin_backward<decltype(d)::value>(c, L); });
}

int gka_linear_decode_step(float *state, const void *q, const void *k, const void *v,
                           const float *beta, const float *gate, void *o, int B, int H, int D,
                           gka_dtype dt, float scale, void *stream) {
    if (B < 0 || H < 0 || !valid_dtype(dt) || !isfinite(scale)) return GKA_ERR_INVALID_ARG;
    if (!supported_d(D)) return GKA_ERR_UNSUPPORTED;
    const size_t BH = (size_t)B * H;
    if (BH == 0) return GKA_OK;
    if (BH > 0x7fffffffu / 8) return GKA_ERR_UNSUPPORTED;   // eight parts a head in one grid dimension
    if (!state || !q || !k || !v || !beta || !o) return GKA_ERR_INVALID_ARG;
    const void *ptrs[] = {state, q, k, v, beta, gate, o};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GKA_ERR_MISALIGNED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return by_type(dt, D, [&](auto tag, auto d) {
        using T = decltype(tag);
        constexpr int DD = decltype(d)::value;
        constexpr int rows = kStepThreads / (DD / 4) * kStepRows;
        constexpr int parts = (DD + rows - 1) / rows;
        ProfScope ps(GKA_KERNEL_LINEAR, s);
        k_linear_step<T, DD><<<(unsigned)(BH * parts), kStepThreads, 0, s>>>(
            state, static_cast<const T *>(q), static_cast<const T *>(k), static_cast<const T *>(v),
            beta, gate, static_cast<T *>(o), scale, parts);
        return check_launch();
    });
}

int gka_block_in_forward(const gka_strided *q, const gka_strided *k, const gka_strided *v,
                         const gka_strided *beta_logit, const gka_strided *gate_logit,
                         const float *beta_bias, const float *gate_bias, const int *lengths,
                         void *q_out, void *k_out, void *v_out, float *beta, float *gate, int B,
                         int T, int H, int Hk, int D, gka_dtype dt, float eps, void *stream) {
    if (int rc = rows_ok(B, T, H, Hk, D, dt, eps)) return rc;
    const size_t n = (size_t)B * H * T;
    if (n == 0) return GKA_OK;   // before any pointer is looked at: empty buffers may be NULL
    if (!gate && (gate_logit || lengths)) return GKA_ERR_INVALID_ARG;
    if (gate && !gate_logit && !lengths) return GKA_ERR_INVALID_ARG;
    if (!q || !k || !v || !beta_logit || !q_out || !k_out || !v_out || !beta)
        return GKA_ERR_INVALID_ARG;
    const int es = dt == GKA_BF16 ? 2 : 4;
    BlockInArgs a = {};
    if (int rc = strided(q, true, es, &a.q)) return rc;
    if (int rc = strided(k, true, es, &a.k)) return rc;
    if (int rc = strided(v, true, es, &a.v)) return rc;
    if (int rc = strided(beta_logit, false, es, &a.beta_logit)) return rc;
    if (gate_logit)
        if (int rc = strided(gate_logit, false, es, &a.gate_logit)) return rc;
    const void *ptrs[] = {q_out, k_out, v_out, beta, gate};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GKA_ERR_MISALIGNED;
    a.beta_bias = beta_bias; a.gate_bias = gate_bias; a.lengths = lengths;
    a.B = B; a.T = T; a.H = H; a.Hk = Hk; a.eps = eps;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return by_type(dt, D, [&](auto tag, auto d) {
        using Tin = decltype(tag);
        constexpr int DD = decltype(d)::value, RPT = 4;
        a.row_blocks = in_blocks(rows_per_block<Tin, DD>(RPT), B, T, H, Hk, &a);
        const size_t gates = (n + kRowThreads - 1) / kRowThreads;
        ProfScope ps(GKA_KERNEL_BLOCK_ROWS, s);
        k_block_in<Tin, DD, RPT><<<(unsigned)(a.row_blocks + gates), kRowThreads, 0, s>>>(
            a, static_cast<Tin *>(q_out), static_cast<Tin *>(k_out), static_cast<Tin *>(v_out), beta,
            gate);
        return check_launch();
    });
}

size_t gka_block_in_backward_workspace_bytes(int B, int T, int H, int Hk, int D, gka_dtype dt) {
    if (rows_ok(B, T, H, Hk, D, dt, 0.f)) return 0;
    return round256(sizeof(float) * 2 * (size_t)H * gate_blocks(B, T));
}

int gka_block_in_backward(const gka_strided *q, const gka_strided *k,
                          const gka_strided *beta_logit, const gka_strided *gate_logit,
                          const float *beta_bias, const float *gate_bias, const int *lengths,
                          const void *dq_out, const void *dk_out, const void *dv_out,
                          const float *dbeta, const float *dgate, void *dq, void *dk, void *dv,
                          void *dbeta_logit, void *dgate_logit, float *dbeta_bias,
                          float *dgate_bias, int B, int T, int H, int Hk, int D, gka_dtype dt,
                          float eps, void *workspace, size_t workspace_bytes, void *stream) {
    if (int rc = rows_ok(B, T, H, Hk, D, dt, eps)) return rc;
    if (dgate_bias && !gate_logit) return GKA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t n = (size_t)B * H * T;
    if (n == 0) {
        // no token: the shared gradients are empty sums; no query heads: those of k and v too
        const size_t kv = (size_t)B * T * Hk * D * (dt == GKA_BF16 ? 2 : 4) / sizeof(float);
        if (kv > 0) {
            if (!dk || !dv) return GKA_ERR_INVALID_ARG;
            if (int rc = pass_state(static_cast<float *>(dk), nullptr, kv, s)) return rc;
            if (int rc = pass_state(static_cast<float *>(dv), nullptr, kv, s)) return rc;
        }
        if (int rc = pass_state(dbeta_bias, nullptr, H, s)) return rc;
        return pass_state(dgate_bias, nullptr, H, s);
    }
    if ((gate_logit != nullptr) != (dgate != nullptr) ||
        (gate_logit != nullptr) != (dgate_logit != nullptr))
        return GKA_ERR_INVALID_ARG;
    if (!q || !k || !beta_logit || !dq_out || !dk_out || !dv_out || !dbeta || !dq || !dk || !dv ||
        !dbeta_logit || !workspace)
        return GKA_ERR_INVALID_ARG;
    const int es = dt == GKA_BF16 ? 2 : 4;
    BlockInArgs a = {};
    if (int rc = strided(q, true, es, &a.q)) return rc;
    if (int rc = strided(k, true, es, &a.k)) return rc;
    if (int rc = strided(beta_logit, false, es, &a.beta_logit)) return rc;
    if (gate_logit)
        if (int rc = strided(gate_logit, false, es, &a.gate_logit)) return rc;
    const void *ptrs[] = {dq_out, dk_out, dv_out, dbeta, dgate, dq, dk, dv, dbeta_logit, dgate_logit};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GKA_ERR_MISALIGNED;
    if ((uintptr_t)workspace & 255u) return GKA_ERR_MISALIGNED;
    BlockInGrad g = {};
    g.gblk = gate_blocks(B, T);
    if (workspace_bytes < round256(sizeof(float) * 2 * (size_t)H * g.gblk))
        return GKA_ERR_WORKSPACE_TOO_SMALL;
    g.dq = dq_out; g.dk = dk_out; g.dv = dv_out; g.dbeta = dbeta; g.dgate = dgate;
    g.xq = dq; g.xk = dk; g.xv = dv; g.xbeta = dbeta_logit; g.xgate = dgate_logit;
    g.part = static_cast<float *>(workspace);
    a.beta_bias = beta_bias; a.gate_bias = gate_bias; a.lengths = lengths;
    a.B = B; a.T = T; a.H = H; a.Hk = Hk; a.eps = eps;
    return by_type(dt, D, [&](auto tag, auto d) {
        using Tin = decltype(tag);
        constexpr int DD = decltype(d)::value, RPT = 2;
        a.row_blocks = in_blocks(rows_per_block<Tin, DD>(RPT), B, T, H, Hk, &a);
        {
            ProfScope ps(GKA_KERNEL_BLOCK_ROWS, s);
            k_block_in_grad<Tin, DD, RPT>
                <<<a.row_blocks + (unsigned)H * g.gblk, kRowThreads, 0, s>>>(a, g);
        }
        if (int rc = check_launch()) return rc;
        if (!dbeta_bias && !dgate_bias) return (int)GKA_OK;
        ProfScope ps(GKA_KERNEL_BLOCK_ROWS, s);
        const SumsOf db = {g.part, H, g.gblk, dbeta_bias};
        const SumsOf dg = {g.part + (size_t)H * g.gblk, dgate_bias ? H : 0, g.gblk, dgate_bias};
        return launch_after(k_block_sums, dim3(db.count + dg.count), 128, 0, true, s, db, dg);
    });
}

int gka_block_out_forward(const void *o, const void *v, const gka_strided *z, const float *w,
                          const float *skip, void *y, int B, int T, int H, int D, gka_dtype dt,
                          float eps, void *stream) {
    if (int rc = rows_ok(B, T, H, H, D, dt, eps)) return rc;
    const size_t n = (size_t)B * H * T;
    if (n == 0) return GKA_OK;
    if ((v != nullptr) != (skip != nullptr)) return GKA_ERR_INVALID_ARG;
    if (!o || !w || !y) return GKA_ERR_INVALID_ARG;
    BlockOutArgs a = {};
    if (z)
        if (int rc = strided(z, true, dt == GKA_BF16 ? 2 : 4, &a.z)) return rc;
    const void *ptrs[] = {o, v, w, y};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GKA_ERR_MISALIGNED;
    a.o = o; a.v = v; a.w = w; a.skip = skip;
    a.B = B; a.T = T; a.H = H; a.eps = eps;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return by_type(dt, D, [&](auto tag, auto d) {
        using Tin = decltype(tag);
        constexpr int DD = decltype(d)::value, RPT = 2;
        ProfScope ps(GKA_KERNEL_BLOCK_ROWS, s);
        const size_t blocks = row_tiles(rows_per_block<Tin, DD>(RPT), B, T, H, &a.tile);
        k_block_out<Tin, DD, RPT><<<(unsigned)blocks, kRowThreads, 0, s>>>(
            a, static_cast<Tin *>(y));
        return check_launch();
    });
}

size_t gka_block_out_backward_workspace_bytes(int B, int T, int H, int D, gka_dtype dt) {
    if (rows_ok(B, T, H, H, D, dt, 0.f)) return 0;
    const size_t blk = out_blocks(B, T, H, D, dt);
    return round256(sizeof(float) * D * H * blk) + round256(sizeof(float) * H * blk);
}

int gka_block_out_backward(const void *o, const void *v, const gka_strided *z, const float *w,
                           const float *skip, const void *dy, void *d_o, void *dv, void *dz,
                           float *dw, float *dskip, int B, int T, int H, int D, gka_dtype dt,
                           float eps, void *workspace, size_t workspace_bytes, void *stream) {
    if (int rc = rows_ok(B, T, H, H, D, dt, eps)) return rc;
    if (!dw) return GKA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t n = (size_t)B * H * T;
    if (n == 0) {
        if (int rc = pass_state(dw, nullptr, D, s)) return rc;
        return pass_state(dskip, nullptr, H, s);
    }
    if ((v != nullptr) != (skip != nullptr) || (v != nullptr) != (dv != nullptr) ||
        (v != nullptr) != (dskip != nullptr) || (z != nullptr) != (dz != nullptr))
        return GKA_ERR_INVALID_ARG;
    if (!o || !w || !dy || !d_o || !workspace) return GKA_ERR_INVALID_ARG;
    BlockOutArgs a = {};
    if (z)
        if (int rc = strided(z, true, dt == GKA_BF16 ? 2 : 4, &a.z)) return rc;
    const void *ptrs[] = {o, v, w, dy, d_o, dv, dz};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GKA_ERR_MISALIGNED;
    if ((uintptr_t)workspace & 255u) return GKA_ERR_MISALIGNED;
    if (workspace_bytes < gka_block_out_backward_workspace_bytes(B, T, H, D, dt))
        return GKA_ERR_WORKSPACE_TOO_SMALL;
    a.o = o; a.v = v; a.w = w; a.skip = skip;
    a.B = B; a.T = T; a.H = H; a.eps = eps;
    BlockOutGrad g = {};
    g.blk = out_blocks(B, T, H, D, dt);
    g.dy = dy; g.d_o = d_o; g.dv = dv; g.dz = dz;
    g.wpart = static_cast<float *>(workspace);
    g.spart = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                        round256(sizeof(float) * (size_t)D * H * g.blk));
    return by_type(dt, D, [&](auto tag, auto d) {
        using Tin = decltype(tag);
        {
            ProfScope ps(GKA_KERNEL_BLOCK_ROWS, s);
            k_block_out_grad<Tin, decltype(d)::value>
                <<<dim3(g.blk, H), kRowThreads, 0, s>>>(a, g);
        }
        if (int rc = check_launch()) return rc;
        ProfScope ps(GKA_KERNEL_BLOCK_ROWS, s);
        const SumsOf sw = {g.wpart, D, H * g.blk, dw}, ss = {g.spart, v ? H : 0, g.blk, dskip};
        return launch_after(k_block_sums, dim3(sw.count + ss.count), 128, 0, true, s, sw, ss);
    });
}

}  // extern "C"
