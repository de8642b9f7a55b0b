// qlora_nf4.cu -- C ABI of the library: validation, launch planning and kernel launches.
// Every kernel lives in a header of this directory; this file is the only translation unit.

#include <algorithm>
#include <cstddef>
#include <cstdint>
#include <cstdlib>
#include <mutex>
#include <utility>

#include "host_common.cuh"
#include "ptx.cuh"
#include "quant_kernels.cuh"
#include "skinny_mma.cuh"
#include "fused_fwd.cuh"
#include "fused_fwd_pair.cuh"
#include "fused_bwd_pair.cuh"
#include "decode_mma.cuh"
#include "optimizer.cuh"
#include "embedding.cuh"

using namespace qlora;

// Scratch of qlora_lora_linear_fwd_static_ws: part of this module's global
// memory on every device where the module is loaded; zero-filled at load, and
// each call clears the parts it accumulates into.
static __device__ __align__(256) uint8_t g_static_scratch[QLORA_STATIC_SCRATCH_BYTES];

// Self-test of the bounded-wait path: one thread waits on a barrier that nothing
// arrives on, with the same wait every pipeline uses; it gives up after the
// current limit, raises the device error word and returns.
__global__ void wait_probe_kernel() {
    __shared__ uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    if (threadIdx.x == 0) mbar_wait(&bar, 0, &abort_flag);
}

namespace {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

static_assert(sizeof(qlora_nf4_weight) == 48 && offsetof(qlora_nf4_weight, quant_type) == 40 &&
                  offsetof(qlora_nf4_weight, format) == 44,
              "the weight descriptor layout is part of the ABI");

// Where the kernels find a weight's first-level scales (see scale_src.cuh).
ScaleSrc scale_src(const qlora_nf4_weight *w) {
    ScaleSrc sc;
    sc.scales = w->scales;
    sc.scales2 = w->scales2;
    sc.blk_shift = fmt_block(w->format) == 128 ? 1 : 0;
    sc.dq = fmt_dq(w->format) ? 1 : 0;
    return sc;
}

CodebookArg codebook_arg(int32_t quant_type) {
    CodebookArg a;
    const Codebook &cb = codebook_for(quant_type);
    for (int i = 0; i < 16; ++i) {
        a.level[i] = cb.level[i];
        a.thresh[i] = cb.thresh[i];
    }
    return a;
}

// Token-tile width: the MMA N dimension (multiple of 16, at most 256), chosen
// to split M into equal tiles with little padding.
int token_tile(int64_t M) {
    const int64_t tiles = ceil_div(M, 256);
    const int64_t bn = ceil_div(ceil_div(M, tiles), 16) * 16;
    return static_cast<int>(std::max<int64_t>(16, std::min<int64_t>(256, bn)));
}

struct GemmPlan {
    int BN;
    int64_t tiles_rows, tiles_tok;
    int splits;
    int stages_per_split;
};

// rows = output rows of the MMA M dimension (N for forward, K for dX),
// stages = 64-wide contraction stages.  Split the contraction across CTAs only
// when the output tiles leave most SMs idle (small-M decode shapes).
GemmPlan plan_gemm(int64_t M, int64_t rows, int64_t stages) {
    GemmPlan g;
    g.BN = token_tile(M);
    g.tiles_rows = ceil_div(rows, 128);
    g.tiles_tok = ceil_div(M, g.BN);
    const int64_t tiles = g.tiles_rows * g.tiles_tok;
    const int sms = sm_count();
    int splits = 1;
    if (tiles * 2 <= sms) {
        const int64_t want = ceil_div(2 * sms, tiles);
        const int64_t maxs = std::max<int64_t>(1, stages / 4);
        splits = static_cast<int>(std::min(want, maxs));
    }
    // whole four-stage code chunks per split
    g.stages_per_split = static_cast<int>(ceil_div(ceil_div(stages, splits), 4) * 4);
    g.splits = static_cast<int>(ceil_div(stages, g.stages_per_split));
    return g;
}

// Raises a kernel's dynamic shared-memory limit to at least `bytes` on the current
// device; the attribute is set once per (kernel, device, size increase), so calls
// after the first make no CUDA call here.
struct SmemSetting {
    const void *kernel;
    int dev, bytes;
};
template <typename K>
qlora_status set_smem(K kernel, int bytes) {
    static std::mutex mu;
    static SmemSetting done[256];
    static int ndone = 0;
    const void *key = reinterpret_cast<const void *>(kernel);
    int dev = 0;
    QL_TRY(cuda_check(cudaGetDevice(&dev), "cudaGetDevice"));
    std::lock_guard<std::mutex> lock(mu);
    int slot = -1;
    for (int i = 0; i < ndone; ++i)
        if (done[i].kernel == key && done[i].dev == dev) slot = i;
    if (slot >= 0 && done[slot].bytes >= bytes) return QLORA_OK;
    QL_TRY(cuda_check(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes),
                      "cudaFuncSetAttribute(max dynamic smem)"));
    if (slot < 0 && ndone < 256) slot = ndone++;
    if (slot >= 0) done[slot] = SmemSetting{key, dev, bytes};
    return QLORA_OK;
}

// Launch with programmatic stream serialization: the kernel may start while the preceding one still
// runs, and calls pdl_wait() before it touches memory that others write.
template <typename... P, typename... A>
qlora_status launch_pdl(const char *what, void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t st,
                        A &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cuda_check(cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...), what);
}

qlora_status launch_check(const char *what) { return cuda_check(cudaGetLastError(), what); }

// Workspace layout of the forward / dX calls:
//   [0, a)      bf16 [M, r]   scaling * (X A^T) or scaling * (dY B): the adapter chunk operand
//   [a, a+b)    fp32 [M, r]   accumulator of that rank-r product
//   [a+b, ...)  fp32 [M, N] or [M, K]  split-K accumulator (small-M shapes only)
struct WsLayout {
    size_t rank_bf16, rank_acc, split_acc, total;
};
WsLayout ws_layout(int64_t M, int64_t rows, int r, bool split) {
    WsLayout w;
    w.rank_bf16 = round256(size_t(M) * size_t(std::max(r, 0)) * 2);
    w.rank_acc = round256(size_t(M) * size_t(std::max(r, 0)) * 4);
    w.split_acc = split ? round256(size_t(M) * size_t(rows) * 4) : 0;
    w.total = w.rank_bf16 + w.rank_acc + w.split_acc;
    return w;
}
// Forward kernel choice: CTA pairs (cta_group::2, 256 W rows per tile) from 64
// tokens up; the single-CTA kernel with split-K below that (decode shapes).
bool use_pair_fwd(int64_t M) { return M >= 64; }
int pair_token_tile(int64_t M) {
    const int64_t tiles = ceil_div(M, 256);
    const int64_t bn = ceil_div(ceil_div(M, tiles), 32) * 32;
    return static_cast<int>(std::max<int64_t>(32, std::min<int64_t>(256, bn)));
}
// Shared-memory plan of the small-M kernel (decode_mma.cuh): table, code ring,
// activation ring, two scale buffers, partial sums, barriers.  The rings are as deep
// as the 227 KB allow; a shape whose shallowest rings do not fit is not planned.
struct DecodePlan {
    dec::Params p;
    int smem;
    bool fits;
};
DecodePlan plan_decode(int64_t M, int64_t K, int r) {
    DecodePlan d{};
    dec::Params &p = d.p;
    const int KB = static_cast<int>(K / 64);
    const int sc_q = (dec::kRows * KB + 16 + 15) & ~15;
    const int s2_floats = ((dec::kRows * KB) / 256 + 2 + 3) & ~3;
    p.sc_q = sc_q;
    p.sc_stage = (sc_q + 4 * s2_floats + 127) & ~127;
    p.xa_stage = static_cast<int>((M + r) * dec::kStageBlocks * 128);
    p.c3d = (K % 256 == 0) ? 1 : 0;
    auto total = [&](int dc, int dx) {
        p.dc = dc;
        p.dx = dx;
        p.off_code = dec::kLutBytes;
        p.off_xa = p.off_code + dc * dec::kCodeStage;
        p.off_sc = p.off_xa + dx * p.xa_stage;
        p.off_part = p.off_sc + 2 * p.sc_stage;
        p.off_upart = p.off_part + dec::kPartFloats * 4;
        p.off_ufin = p.off_upart + 4 * 256 * 4;
        p.off_bars = p.off_ufin + 256 * 4;
        const int bars = (2 * dec::kMaxCodeStages + 2 * dec::kMaxXaStages + 4) * 8 + 16;
        return 1024 + p.off_bars + bars;   // + alignment slack of the dynamic base
    };
    int dc = dec::kMaxCodeStages, dx = dec::kMaxXaStages;
    while (total(dc, dx) > dec::kSmemLimit && (dx > 2 || dc > 3)) {
        if (dx > 2) --dx;
        else --dc;
    }
    d.smem = total(dc, dx);
    d.fits = d.smem <= dec::kSmemLimit;
    return d;
}
// Small-M forward: the weight-streaming warp-MMA kernel, which needs no workspace,
// for up to 16 tokens, adapter ranks up to 16 and n_in up to 32768 (when its rings fit).
// (Default storage format only: other formats take the tensor-core path.)
bool use_decode(int64_t M, int64_t K, int r, int32_t format) {
    return format == 0 && M <= 16 && r <= dec::kMaxRank && K / 64 <= dec::kMaxKB && plan_decode(M, K, r).fits;
}
// format < 0: the largest need over every storage format
size_t fwd_ws_bytes(int64_t M, int64_t N, int64_t K, int r, int32_t format) {
    if (format >= 0 && use_decode(M, K, r, format)) return 0;
    const bool split = !use_pair_fwd(M) && plan_gemm(M, N, K / 64).splits > 1;
    return ws_layout(M, N, r, split).total;
}
// dX plan: CTA pairs (256 k columns x BN tokens per pair) at every M.  When the pair
// tiles would fill less than half of the SM pairs (small M), the contraction over n
// is split along blockIdx.z into whole four-stage code chunks, and the splits add
// into an fp32 accumulator.
struct DxPlan {
    int BN;
    int64_t pairs, tiles_tok;
    int splits, nb_per_split;
};
// Tiles of the dX kernel.  wide: 512-token tiles (two accumulators) are allowed.  They are taken
// when the estimated time of the whole grid is lower: per pair tile about 0.73 us per
// 64-n stage at 256 tokens and 0.97 us at 512 (measured on the 70B shapes), plus about
// 10 us of set-up and epilogue, times the number of waves of the pair tiles over the SM pairs.
DxPlan plan_dx(int64_t M, int64_t N, int64_t K, bool wide) {
    DxPlan d;
    d.BN = pair_token_tile(M);
    d.pairs = ceil_div(K, 2 * bwdp::BM);
    d.tiles_tok = ceil_div(M, d.BN);
    const int64_t nb = ceil_div(N, 64);
    const int64_t tiles = d.pairs * d.tiles_tok;
    const int64_t pair_slots = std::max(1, sm_count() / 2);
    int64_t splits = 1;
    if (tiles * 2 <= pair_slots) splits = std::min(ceil_div(pair_slots, tiles), std::max<int64_t>(1, nb / 4));
    d.nb_per_split = static_cast<int>(ceil_div(ceil_div(nb, splits), 4) * 4);
    d.splits = static_cast<int>(ceil_div(nb, d.nb_per_split));
    if (wide && d.splits == 1 && M > 256) {
        const int64_t t512 = ceil_div(M, 512);
        const double w256 = double(ceil_div(tiles, pair_slots)), w512 = double(ceil_div(d.pairs * t512, pair_slots));
        if (w512 * (double(nb) * 0.97 + 10.0) < w256 * (double(nb) * 0.73 + 10.0)) {
            d.BN = 512;
            d.tiles_tok = t512;
        }
    }
    return d;
}
size_t bwd_ws_bytes(int64_t M, int64_t N, int64_t K, int r) {
    return ws_layout(M, K, r, plan_dx(M, N, K, false).splits > 1).total;
}

// Launches the rank-r tensor-core product out[i*ld_i + j*ld_j] += scaling *
// sum_t P(i, t) Q(j, t) (see skinny_mma.cuh) over bf16 operands:
//   P: p_mn = 0 -> [I, T] row-major (t contiguous); p_mn = 1 -> [T, I] row-major
//   Q: q_mn = 0 -> [r, T] row-major;                q_mn = 1 -> [T, r] row-major
// The output must already hold zeros or the values to accumulate into.
qlora_status launch_skinny(const void *P, int p_mn, const void *Q, int q_mn, int64_t T, int64_t I, int r,
                           float scaling, float *out, int64_t ld_i, int64_t ld_j, cudaStream_t st) {
    using namespace skinny;
    Params p;
    p.T = static_cast<int>(T);
    p.I = static_cast<int>(I);
    p.r = r;
    p.p_mn = p_mn;
    p.q_mn = q_mn;
    CUtensorMap tmP, tmQ;
    // P: one 3-D box per stage when the t (K-major) or i (MN-major) extent is whole 64-element chunks
    const int64_t p_rows = p_mn ? T : I, p_cols = p_mn ? I : T;
    p.p_3d = p_cols % 64 == 0;
    if (p.p_3d)
        QL_TRY(make_tmap_chunks(&tmP, P, p_rows, p_cols, BT, 2));
    else
        QL_TRY(make_tmap_2d(&tmP, P, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p_rows, p_cols, p_cols, BT, 64,
                            CU_TENSOR_MAP_SWIZZLE_128B));
    if (!q_mn) {
        // [r, T]: Nq rows per 64-t chunk, rows past r zero-filled
        p.Nq = static_cast<int>(ceil_div(r, 16) * 16);
        p.q_3d = T % 64 == 0;
        p.q_atoms = 0;
        p.q_span = 128;
        p.q_bytes = 2 * p.Nq * 128;
        if (p.q_3d)
            QL_TRY(make_tmap_chunks(&tmQ, Q, r, T, p.Nq, 2));
        else
            QL_TRY(make_tmap_2d(&tmQ, Q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, r, T, T, p.Nq, 64,
                                CU_TENSOR_MAP_SWIZZLE_128B));
    } else {
        // [T, r]: j contiguous; the narrowest swizzle atom that covers r (16, 32 or 64 elements)
        p.Nq = r <= 16 ? 16 : (r <= 32 ? 32 : (r <= 64 ? 64 : 128));
        p.q_span = p.Nq >= 64 ? 128 : p.Nq * 2;
        p.q_atoms = p.Nq >= 64 ? p.Nq / 64 : 1;
        p.q_3d = 0;
        p.q_bytes = p.q_atoms * BT * p.q_span;
        const CUtensorMapSwizzle swz = p.q_span == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                       : p.q_span == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                        : CU_TENSOR_MAP_SWIZZLE_32B;
        QL_TRY(make_tmap_2d(&tmQ, Q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, T, r, r, BT, p.q_span / 2, swz));
    }
    p.stages = std::min(kMaxStages, kRingBudget / stage_bytes(p.q_bytes));
    p.units = ceil_div(I, BI) * ceil_div(T, BT);
    p.scaling = scaling;
    p.out = out;
    p.ld_i = ld_i;
    p.ld_j = ld_j;
    const int smem = smem_bytes(p.stages, p.q_bytes);
    QL_TRY(set_smem(skinny_mma_kernel, smem));
    // stream-K: two CTAs per SM, each a contiguous run of (tile, stage) units
    const int64_t grid = std::min<int64_t>(p.units, 2 * sm_count());
    skinny_mma_kernel<<<static_cast<unsigned>(grid), kThreads, smem, st>>>(tmP, tmQ, p);
    return launch_check("skinny_mma_kernel launch");
}

qlora_status launch_finalize(const float *acc, int64_t n, float scaling, uint16_t *save, uint16_t *scaled,
                             cudaStream_t st) {
    skinny::finalize_rank_kernel<<<static_cast<unsigned>(std::min<int64_t>(ceil_div(n, 256), 2048)), 256, 0, st>>>(
        acc, n, scaling, save, scaled);
    return launch_check("finalize_rank_kernel launch");
}

qlora_status check_rank(int r, float scaling, const void *A, const void *B) {
    if (r == 0) return QLORA_OK;
    if (r < 8 || r > 128 || r % 8) return fail(QLORA_ERR_SHAPE, "r (%d) must be 0 or a multiple of 8 in [8, 128]", r);
    if (!A || !B) return fail(QLORA_ERR_ARG, "A and B must be non-NULL when r > 0");
    if (!aligned16(A) || !aligned16(B)) return fail(QLORA_ERR_ALIGN, "A and B must be 16-byte aligned");
    if (!std::isfinite(scaling)) return fail(QLORA_ERR_ARG, "scaling must be finite");
    return QLORA_OK;
}

// Device address of g_static_scratch on the current device, looked up by the
// first call on that device and cached (one lookup per device, under a lock).
qlora_status static_scratch(void **out) {
    constexpr int kMaxDevices = 64;
    static void *ptrs[kMaxDevices] = {};
    static std::mutex mu;
    int dev = 0;
    QL_TRY(cuda_check(cudaGetDevice(&dev), "cudaGetDevice"));
    if (dev < 0 || dev >= kMaxDevices)
        return fail(QLORA_ERR_UNSUPPORTED, "device %d: the static scratch serves devices 0..%d", dev, kMaxDevices - 1);
    std::lock_guard<std::mutex> lock(mu);
    if (!ptrs[dev]) {
        void *p = nullptr;
        QL_TRY(cuda_check(cudaGetSymbolAddress(&p, g_static_scratch), "cudaGetSymbolAddress(static scratch)"));
        if (!p) return fail(QLORA_ERR_CUDA, "cudaGetSymbolAddress returned NULL for the static scratch");
        ptrs[dev] = p;
    }
    *out = ptrs[dev];
    return QLORA_OK;
}

// The packed base weight as the CTA-pair GEMM kernels see it: 4-bit codes with the
// scales of their storage format and the levels of their quant type, or Q8_0 int8
// codes with an fp16 scale per 32 weights.
struct BaseW {
    const uint8_t *codes;     // [N, K/2] (4-bit) or [N, K] (int8) bytes
    bool q8;
    ScaleSrc sc;              // 4-bit only
    const uint16_t *d8;       // Q8_0 only
    const float *level;       // 4-bit only: the 16 levels
};

// Tile order of a pair kernel (raster_tile in ptx.cuh): nw weight tiles of w_bytes each
// and nt token tiles of t_bytes each.  A band of tiles that fits the L2 budget is read
// from DRAM once; the other operand streams once per band.  Mode 0 keeps a band of
// weight tiles (DRAM bytes: all weight + all tokens x bands), mode 1 a band of token
// tiles (all tokens + all weight x bands); the smaller total wins.
struct Raster {
    int mode, group;
};
Raster pair_raster(int64_t nw, int64_t nt, double w_bytes, double t_bytes) {
    const double budget = 64e6;   // half of the 126 MB L2: the rest holds the stream and the output
    const int64_t g0 = std::max<int64_t>(1, std::min<int64_t>(nw, static_cast<int64_t>(budget / w_bytes)));
    const int64_t g1 = std::max<int64_t>(1, std::min<int64_t>(nt, static_cast<int64_t>(budget / t_bytes)));
    const double wt = double(nw) * w_bytes, tt = double(nt) * t_bytes;
    const double c0 = wt + tt * double(ceil_div(nw, g0));
    const double c1 = tt + wt * double(ceil_div(nt, g1));
    return c0 <= c1 ? Raster{0, static_cast<int>(g0)} : Raster{1, static_cast<int>(g1)};
}

// Forward base GEMM plus the adapter stage on CTA pairs: Y = X W'^T + us B^T, with
// us = bf16(scaling * U) [M, r] already in the workspace (r > 0).
qlora_status launch_fwd_pair(const BaseW &bw, const qlora_bf16 *X, int64_t M, int64_t N, int64_t K,
                             const qlora_bf16 *B, int r, const uint16_t *us, qlora_bf16 *Y, cudaStream_t st) {
    const int BN = pair_token_tile(M);
    CUtensorMap tmX, tmC, tmU;
    QL_TRY(make_tmap_chunks(&tmX, X, M, K, BN / 2, 2));
    const uint64_t row_bytes = bw.q8 ? uint64_t(K) : uint64_t(K / 2);
    QL_TRY(make_tmap_2d(&tmC, bw.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, N, row_bytes, row_bytes, 128, 128,
                        CU_TENSOR_MAP_SWIZZLE_128B));
    if (r > 0)
        QL_TRY(make_tmap_2d(&tmU, us, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, M, r, r, BN / 2, 64,
                            CU_TENSOR_MAP_SWIZZLE_128B));
    else
        tmU = tmX;
    // the Y tile store of each CTA: [BN tokens, 128 rows of W] boxes, unswizzled
    CUtensorMap tmY;
    QL_TRY(make_tmap_2d(&tmY, Y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, M, N, N, BN, fwdp::BM,
                        CU_TENSOR_MAP_SWIZZLE_NONE));
    fwdp::Params p;
    p.sc = bw.sc;
    p.d8 = bw.d8;
    p.Blora = B;
    p.Y = Y;
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.r = r;
    p.BN = BN;
    const int64_t nw = ceil_div(N, 256), nt = ceil_div(M, BN);
    // launch order (weight tile fastest): measured as fast as any banded order here, where
    // the re-read weight tiles come at well under the DRAM bandwidth
    p.raster_mode = 0;
    p.raster_group = static_cast<int>(nw);
    for (int i = 0; i < 16; ++i) p.level[i] = bw.q8 ? 0.f : bw.level[i];
    dim3 grid(static_cast<unsigned>(2 * nw), static_cast<unsigned>(nt), 1);
    if (bw.q8) {
        QL_TRY(set_smem(fwdp::fused_fwd_pair_kernel<true>, fwdp::smem_bytes(256, true)));
        fwdp::fused_fwd_pair_kernel<true><<<grid, fwdp::kThreads, fwdp::smem_bytes(BN, true), st>>>(tmX, tmC, tmU, tmY, p);
    } else {
        QL_TRY(set_smem(fwdp::fused_fwd_pair_kernel<false>, fwdp::smem_bytes(256)));
        fwdp::fused_fwd_pair_kernel<false><<<grid, fwdp::kThreads, fwdp::smem_bytes(BN), st>>>(tmX, tmC, tmU, tmY, p);
    }
    return launch_check("fused_fwd_pair_kernel launch");
}

// dX kernel forms (stage slots = dequant groups kS, stages per code chunk kCS): 4-bit
// codes take kS = kCS = 4 at every tile (165 KB of shared memory at 256 tokens, 226 KB at
// 512); 8-bit codes take kS = kCS = 4 up to 256 tokens (198 KB) and kS = kCS = 3 at 512
// (194 KB: four-stage 8-bit chunks do not fit beside the 512-token rings).
template <bool kQ8, int kS, int kCS>
qlora_status launch_dx_variant(dim3 grid, int BN, int most, const CUtensorMap &tmY, const CUtensorMap &tmC,
                               const CUtensorMap &tmG, const CUtensorMap &tmD, const bwdp::Params &p,
                               cudaStream_t st) {
    // most: the largest tile this form runs, which sets its shared-memory limit
    QL_TRY(set_smem(bwdp::fused_bwd_pair_kernel<kQ8, kS, kCS>, bwdp::smem_bytes(most, kQ8, kS, kCS)));
    bwdp::fused_bwd_pair_kernel<kQ8, kS, kCS>
        <<<grid, bwdp::threads_for(kS), bwdp::smem_bytes(BN, kQ8, kS, kCS), st>>>(tmY, tmC, tmG, tmD, p);
    return QLORA_OK;
}

// dX = dY W' + gs A on CTA pairs (gs = bf16(scaling * G) [M, r] in the workspace when
// r > 0), split over n into dxacc (zeroed by the caller) when the plan says so.
qlora_status launch_dx_pair(const BaseW &bw, const DxPlan &g, const qlora_bf16 *dY, int64_t M, int64_t N, int64_t K,
                            const qlora_bf16 *A, int r, const uint16_t *gs, qlora_bf16 *dX, float *dxacc,
                            cudaStream_t st) {
    const int BN = g.BN;
    const int box = std::min(BN, 256) / 2;        // dY rows per TMA box: one CTA's share of an accumulator
    CUtensorMap tmY, tmC, tmG;
    QL_TRY(make_tmap_2d(&tmY, dY, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, M, N, N, box, 64,
                        CU_TENSOR_MAP_SWIZZLE_128B));
    const int crow = bwdp::chunk_rows(bw.q8 && BN > 256 ? 3 : 4);   // code rows per TMA box
    if (bw.q8)
        QL_TRY(make_tmap_2d(&tmC, bw.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, N, K, K, crow, 128,
                            CU_TENSOR_MAP_SWIZZLE_128B));
    else
        QL_TRY(make_tmap_2d(&tmC, bw.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, N, K / 2, K / 2, crow, 64,
                            CU_TENSOR_MAP_SWIZZLE_64B));
    if (r > 0)
        QL_TRY(make_tmap_2d(&tmG, gs, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, M, r, r, box, 64,
                            CU_TENSOR_MAP_SWIZZLE_128B));
    else
        tmG = tmY;
    // the dX tile store: [tokens, 128 k] boxes, unswizzled (with splits the epilogue adds into dxacc instead)
    CUtensorMap tmD;
    if (!dxacc)
        QL_TRY(make_tmap_2d(&tmD, dX, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, M, K, K, std::min(BN, 256),
                            bwdp::BM, CU_TENSOR_MAP_SWIZZLE_NONE));
    else
        tmD = tmY;
    bwdp::Params p;
    p.sc = bw.sc;
    p.d8 = bw.d8;
    p.Alora = A;
    p.dX = dX;
    p.dXacc = dxacc;
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.r = r;
    p.BN = BN;
    p.nb_per_split = g.nb_per_split;
    // a weight tile: 256 columns of codes over the split's n rows; a token tile: BN rows of dY
    const double n_split = double(std::min<int64_t>(N, int64_t(g.nb_per_split) * 64));
    const Raster ras = pair_raster(g.pairs, g.tiles_tok, 256.0 * n_split * (bw.q8 ? 1.0 : 0.5),
                                   double(BN) * n_split * 2.0);
    p.raster_mode = ras.mode;
    p.raster_group = ras.group;
    for (int i = 0; i < 16; ++i) p.level[i] = bw.q8 ? 0.f : bw.level[i];
    dim3 grid(static_cast<unsigned>(2 * g.pairs), static_cast<unsigned>(g.tiles_tok), static_cast<unsigned>(g.splits));
    if (bw.q8 && BN > 256)
        QL_TRY((launch_dx_variant<true, 3, 3>(grid, BN, 512, tmY, tmC, tmG, tmD, p, st)));
    else if (bw.q8)
        QL_TRY((launch_dx_variant<true, 4, 4>(grid, BN, 256, tmY, tmC, tmG, tmD, p, st)));
    else
        QL_TRY((launch_dx_variant<false, 4, 4>(grid, BN, 512, tmY, tmC, tmG, tmD, p, st)));
    QL_TRY(launch_check("fused_bwd_pair_kernel launch"));
    if (dxacc) QL_TRY(launch_finalize(dxacc, M * K, 1.0f, dX, nullptr, st));
    return QLORA_OK;
}

// The rank-r side product of the forward (U = X A^T: us = bf16(scaling U), U_save = bf16(U))
// or of dX (G = dY B), into the workspace.
qlora_status rank_side_product(bool fwd, const qlora_bf16 *act, int64_t M, int64_t width, const qlora_bf16 *factor,
                               int r, float scaling, uint16_t *scaled, float *acc, qlora_bf16 *save, cudaStream_t st) {
    QL_TRY(cuda_check(cudaMemsetAsync(acc, 0, size_t(M) * r * 4, st), "zero rank accumulator"));
    if (fwd) QL_TRY(launch_skinny(act, 0, factor, 0, width, M, r, 1.0f, acc, r, 1, st));
    else QL_TRY(launch_skinny(act, 0, factor, 1, width, M, r, 1.0f, acc, r, 1, st));
    return launch_finalize(acc, M * r, scaling, save, scaled, st);
}

BaseW base_of(const qlora_nf4_weight *w, const Codebook &cb) {
    BaseW b;
    b.codes = w->codes;
    b.q8 = false;
    b.sc = scale_src(w);
    b.d8 = nullptr;
    b.level = cb.level;
    return b;
}

qlora_status check_ws(void *ws, size_t ws_bytes, size_t need) {
    if (need == 0) return QLORA_OK;
    if (!ws) return fail(QLORA_ERR_WORKSPACE, "workspace is NULL but %zu bytes are needed", need);
    if (!aligned16(ws)) return fail(QLORA_ERR_ALIGN, "workspace must be 16-byte aligned");
    if (ws_bytes < need) return fail(QLORA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
    return QLORA_OK;
}


}  // namespace

extern "C" {

size_t qlora_packed_bytes(int64_t numel) { return qlora_packed_bytes_fmt(numel, 0); }

size_t qlora_packed_bytes_fmt(int64_t numel, int32_t format) {
    if (!fmt_valid(format)) return 0;
    const int64_t blk = fmt_block(format);
    if (numel <= 0 || numel % blk) return 0;
    const int64_t nb = numel / blk;
    if (!fmt_dq(format)) return size_t(numel / 2) + 4 * size_t(nb);
    return size_t(numel / 2) + size_t(nb) + 4 * size_t(ceil_div(nb, 256));
}

qlora_status qlora_nf4_codebook(float out[16]) {
    if (!out) return fail(QLORA_ERR_ARG, "out is NULL");
    const Codebook &cb = codebook();
    for (int i = 0; i < 16; ++i) out[i] = cb.level[i];
    return QLORA_OK;
}

qlora_status qlora_codebook(int quant_type, float *out) {
    if (!out) return fail(QLORA_ERR_ARG, "out is NULL");
    if (quant_type != QLORA_QT_NF4 && quant_type != QLORA_QT_FP4)
        return fail(QLORA_ERR_ARG, "quant_type (%d) must be QLORA_QT_NF4 (0) or QLORA_QT_FP4 (1)", quant_type);
    const Codebook &cb = codebook_for(quant_type);
    for (int i = 0; i < 16; ++i) out[i] = cb.level[i];
    return QLORA_OK;
}

const char *qlora_last_error(void) { return t_last_error; }

qlora_status qlora_set_wait_limit_ns(uint64_t ns) {
    if (ns < 1000000ull || ns > 60000000000ull)
        return fail(QLORA_ERR_ARG, "wait limit %llu ns outside [1e6, 6e10]", (unsigned long long)ns);
    QL_TRY(require_sm100());
    const unsigned long long v = ns;
    return cuda_check(cudaMemcpyToSymbol(g_wait_limit_ns, &v, sizeof(v)), "set the wait limit");
}

qlora_status qlora_probe_wait_timeout(void *stream) {
    QL_TRY(require_sm100());
    wait_probe_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>();
    return launch_check("wait_probe_kernel launch");
}

size_t qlora_workspace_bytes(int64_t M, int64_t N, int64_t K, int r) {
    if (M <= 0 || N <= 0 || K <= 0) return 0;
    return std::max<size_t>(256, std::max(fwd_ws_bytes(M, N, K, r, -1), bwd_ws_bytes(M, N, K, r)));
}

qlora_status qlora_sync_status(void *stream) {
    QL_TRY(cuda_check(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)), "cudaStreamSynchronize"));
    int v = 0;
    QL_TRY(cuda_check(cudaMemcpyFromSymbol(&v, g_device_error, sizeof(int)), "read device error word"));
    if (v) {
        const int zero = 0;
        cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int));
        if (v == kDeviceErrTmemStore)
            return fail(QLORA_ERR_CUDA, "a tensor-memory store did not read back as written (device error %d)", v);
        if (v == kDeviceErrIndex)
            return fail(QLORA_ERR_ARG, "a token id lies outside its embedding table (device error %d)", v);
        return fail(QLORA_ERR_TIMEOUT, "a kernel pipeline wait timed out (device error %d)", v);
    }
    return QLORA_OK;
}

qlora_status qlora_quantize_nf4_dq(const float *W, const qlora_nf4_weight *w, void *stream) {
    QL_TRY(check_weight(w));
    if (!W) return fail(QLORA_ERR_ARG, "W is NULL");
    if (!aligned16(W)) return fail(QLORA_ERR_ALIGN, "W must be 16-byte aligned");
    QL_TRY(require_sm100());
    const int64_t numel = w->n_out * w->n_in;
    const int blk = fmt_block(w->format);
    const int64_t nblocks = numel / blk;
    const int64_t ngroups = ceil_div(nblocks, 256);
    if (ngroups > INT32_MAX) return fail(QLORA_ERR_SHAPE, "weight too large");
    const dim3 grid(static_cast<unsigned>(ngroups));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const CodebookArg cb = codebook_arg(w->quant_type);
    const bool dq = fmt_dq(w->format), after = (w->format & QLORA_FMT_CODES_AFTER_DQ) != 0;
#define QL_ENC(B, D, A) nf4_encode_kernel<B, D, A><<<grid, kEncThreads, 0, st>>>(W, w->codes, w->scales, w->scales2, nblocks, cb)
    if (blk == 64) {
        if (!dq) QL_ENC(64, false, false);
        else if (after) QL_ENC(64, true, true);
        else QL_ENC(64, true, false);
    } else {
        if (!dq) QL_ENC(128, false, false);
        else if (after) QL_ENC(128, true, true);
        else QL_ENC(128, true, false);
    }
#undef QL_ENC
    return launch_check("nf4_encode_kernel launch");
}

qlora_status qlora_dequant(const qlora_nf4_weight *w, void *out, int out_is_bf16, void *stream) {
    QL_TRY(check_weight(w));
    if (!out) return fail(QLORA_ERR_ARG, "out is NULL");
    if (!aligned16(out)) return fail(QLORA_ERR_ALIGN, "out must be 16-byte aligned");
    if (out_is_bf16 != 0 && out_is_bf16 != 1) return fail(QLORA_ERR_ARG, "out_is_bf16 must be 0 or 1");
    QL_TRY(require_sm100());
    const int64_t n16 = w->n_out * w->n_in / 16;
    const int64_t grid = std::min<int64_t>(ceil_div(n16, 256), int64_t(sm_count()) * 8);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (out_is_bf16)
        nf4_dequant_kernel<true><<<static_cast<unsigned>(grid), 256, 0, st>>>(w->codes, scale_src(w), out, n16,
                                                                               codebook_arg(w->quant_type));
    else
        nf4_dequant_kernel<false><<<static_cast<unsigned>(grid), 256, 0, st>>>(w->codes, scale_src(w), out, n16,
                                                                                codebook_arg(w->quant_type));
    return launch_check("nf4_dequant_kernel launch");
}

qlora_status qlora_lora_merge_requant(const qlora_nf4_weight *w_in, const qlora_bf16 *A, const qlora_bf16 *B, int r,
                                      float scaling, float *W_scratch, const qlora_nf4_weight *w_out, void *stream) {
    QL_TRY(check_weight(w_in));
    QL_TRY(check_weight(w_out));
    if (w_out->n_out != w_in->n_out || w_out->n_in != w_in->n_in)
        return fail(QLORA_ERR_SHAPE, "w_out must have the shape of w_in");
    QL_TRY(check_rank(r, scaling, A, B));
    if (!W_scratch) return fail(QLORA_ERR_ARG, "W_scratch is NULL");
    if (!aligned16(W_scratch)) return fail(QLORA_ERR_ALIGN, "W_scratch must be 16-byte aligned");
    QL_TRY(require_sm100());
    // x: a row's groups of kMergeCols weights; y: groups of kMergeRows rows, about 8 CTAs per SM in all
    const int64_t gx = std::min<int64_t>(ceil_div(w_in->n_in / kMergeCols, kMergeThreads), 32);
    const int64_t gy = std::min<int64_t>(ceil_div(w_in->n_out, kMergeRows),
                                         std::max<int64_t>(1, int64_t(sm_count()) * 8 / gx));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    nf4_lora_merge_kernel<<<dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), kMergeThreads, 0, st>>>(
        w_in->codes, scale_src(w_in), r > 0 ? reinterpret_cast<const uint16_t *>(A) : nullptr,
        r > 0 ? reinterpret_cast<const uint16_t *>(B) : nullptr, r, r > 0 ? scaling : 0.f, w_in->n_out, w_in->n_in,
        W_scratch, codebook_arg(w_in->quant_type));
    QL_TRY(launch_check("nf4_lora_merge_kernel launch"));
    return qlora_quantize_nf4_dq(W_scratch, w_out, stream);
}

qlora_status qlora_lora_linear_fwd(const qlora_nf4_weight *w, const qlora_bf16 *X, int64_t M, const qlora_bf16 *A,
                                   const qlora_bf16 *B, int r, float scaling, qlora_bf16 *Y, qlora_bf16 *U_save,
                                   void *ws, size_t ws_bytes, void *stream) {
    QL_TRY(check_weight(w));
    if (!X || !Y) return fail(QLORA_ERR_ARG, "X and Y must be non-NULL");
    if (!aligned16(X) || !aligned16(Y)) return fail(QLORA_ERR_ALIGN, "X and Y must be 16-byte aligned");
    if (U_save && !aligned16(U_save)) return fail(QLORA_ERR_ALIGN, "U_save must be 16-byte aligned");
    if (M <= 0 || M > INT32_MAX) return fail(QLORA_ERR_SHAPE, "M (%lld) must be in [1, 2^31)", (long long)M);
    QL_TRY(check_rank(r, scaling, A, B));
    const int64_t N = w->n_out, K = w->n_in;
    const size_t need = fwd_ws_bytes(M, N, K, r, w->format);
    QL_TRY(check_ws(ws, ws_bytes, need));
    QL_TRY(require_sm100());
    cudaStream_t st = static_cast<cudaStream_t>(stream);

    if (use_decode(M, K, r, w->format)) {
        DecodePlan d = plan_decode(M, K, r);
        dec::Params &p = d.p;
        p.codes = w->codes;
        p.scales = w->scales;
        p.scales2 = w->scales2;
        p.Blora = r > 0 ? B : nullptr;
        p.Y = Y;
        p.U_save = r > 0 ? U_save : nullptr;
        p.M = static_cast<int>(M);
        p.N = static_cast<int>(N);
        p.K = static_cast<int>(K);
        p.r = r;
        p.units = static_cast<int>(ceil_div(N, dec::kRows));
        p.scaling = scaling;
        const Codebook &cbd = codebook_for(w->quant_type);
        for (int i = 0; i < 16; ++i) p.level[i] = cbd.level[i];
        // codes as u8 [N, K/2] in [32 rows x 128 B] boxes (3-D: four 256-k chunks per box);
        // X and A as [K/64][rows][64] bf16 chunks, sixteen chunks per box
        CUtensorMap tmC, tmX, tmA;
        if (p.c3d) QL_TRY(make_tmap_code_chunks(&tmC, w->codes, N, K, dec::kRows, dec::kStageK / 256));
        else QL_TRY(make_tmap_2d(&tmC, w->codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, N, K / 2, K / 2, dec::kRows, 128,
                                 CU_TENSOR_MAP_SWIZZLE_128B));
        QL_TRY(make_tmap_chunks(&tmX, X, M, K, static_cast<uint32_t>(M), dec::kStageBlocks));
        if (r > 0) QL_TRY(make_tmap_chunks(&tmA, A, r, K, static_cast<uint32_t>(r), dec::kStageBlocks));
        else tmA = tmX;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(p.units, sm_count())));
        cfg.blockDim = dim3(dec::kThreads);
        cfg.dynamicSmemBytes = d.smem;
        cfg.stream = st;
        // programmatic dependent launch: the kernel builds its table and initialises its
        // barriers before waiting for the preceding grid
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        if (M <= 8) {
            QL_TRY(set_smem(dec::decode_kernel<1>, d.smem));
            QL_TRY(cuda_check(cudaLaunchKernelEx(&cfg, dec::decode_kernel<1>, tmC, tmX, tmA, p), "decode_kernel launch"));
        } else {
            QL_TRY(set_smem(dec::decode_kernel<2>, d.smem));
            QL_TRY(cuda_check(cudaLaunchKernelEx(&cfg, dec::decode_kernel<2>, tmC, tmX, tmA, p), "decode_kernel launch"));
        }
        return QLORA_OK;
    }

    const bool pair = use_pair_fwd(M);
    const GemmPlan g = plan_gemm(M, N, K / 64);
    const bool split = !pair && g.splits > 1;
    const WsLayout L = ws_layout(M, N, r, split);
    uint8_t *wsb = static_cast<uint8_t *>(ws);
    uint16_t *us = reinterpret_cast<uint16_t *>(wsb);
    float *uacc = reinterpret_cast<float *>(wsb + L.rank_bf16);
    float *yacc = split ? reinterpret_cast<float *>(wsb + L.rank_bf16 + L.rank_acc) : nullptr;
    // U = X A^T on tensor cores, then bf16 copies: U (saved) and scaling * U (adapter chunk)
    if (r > 0) QL_TRY(rank_side_product(true, X, M, K, A, r, scaling, us, uacc, U_save, st));
    const Codebook &cb = codebook_for(w->quant_type);

    if (pair) return launch_fwd_pair(base_of(w, cb), X, M, N, K, B, r, us, Y, st);

    if (yacc) QL_TRY(cuda_check(cudaMemsetAsync(yacc, 0, size_t(M) * N * 4, st), "zero split accumulator"));
    CUtensorMap tmX, tmC, tmU;
    QL_TRY(make_tmap_2d(&tmX, X, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, M, K, K, g.BN, 64,
                        CU_TENSOR_MAP_SWIZZLE_128B));
    QL_TRY(make_tmap_2d(&tmC, w->codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, N, K / 2, K / 2, 128, 128,
                        CU_TENSOR_MAP_SWIZZLE_128B));
    if (r > 0)
        QL_TRY(make_tmap_2d(&tmU, us, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, M, r, r, g.BN, 64,
                            CU_TENSOR_MAP_SWIZZLE_128B));
    else
        tmU = tmX;

    fwd::Params p;
    p.sc = scale_src(w);
    p.Blora = B;
    p.Y = Y;
    p.Yacc = yacc;
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.r = r;
    p.BN = g.BN;
    p.kb_per_split = g.stages_per_split;
    for (int i = 0; i < 16; ++i) p.level[i] = cb.level[i];

    const int smem = fwd::smem_bytes(g.BN);
    QL_TRY(set_smem(fwd::fused_fwd_kernel, fwd::smem_bytes(256)));
    dim3 grid(static_cast<unsigned>(g.tiles_rows), static_cast<unsigned>(g.tiles_tok), static_cast<unsigned>(g.splits));
    fwd::fused_fwd_kernel<<<grid, fwd::kThreads, smem, st>>>(tmX, tmC, tmU, p);
    QL_TRY(launch_check("fused_fwd_kernel launch"));
    if (yacc) QL_TRY(launch_finalize(yacc, M * N, 1.0f, Y, nullptr, st));
    return QLORA_OK;
}

qlora_status qlora_lora_linear_fwd_static_ws(const qlora_nf4_weight *w, const qlora_bf16 *X, int64_t M,
                                             const qlora_bf16 *A, const qlora_bf16 *B, int r, float scaling,
                                             qlora_bf16 *Y, qlora_bf16 *U_save, void *stream) {
    // the size check needs only host arithmetic: reject before any CUDA call
    QL_TRY(check_weight(w));
    if (M <= 0 || M > INT32_MAX) return fail(QLORA_ERR_SHAPE, "M (%lld) must be in [1, 2^31)", (long long)M);
    QL_TRY(check_rank(r, scaling, A, B));
    const size_t need = fwd_ws_bytes(M, w->n_out, w->n_in, r, w->format);
    if (need > QLORA_STATIC_SCRATCH_BYTES)
        return fail(QLORA_ERR_WORKSPACE,
                    "M=%lld N=%lld K=%lld r=%d needs %zu bytes of scratch; the static scratch holds %zu "
                    "(use qlora_lora_linear_fwd with a caller workspace)",
                    (long long)M, (long long)w->n_out, (long long)w->n_in, r, need,
                    size_t(QLORA_STATIC_SCRATCH_BYTES));
    QL_TRY(require_sm100());
    void *scratch = nullptr;
    QL_TRY(static_scratch(&scratch));
    return qlora_lora_linear_fwd(w, X, M, A, B, r, scaling, Y, U_save, scratch, QLORA_STATIC_SCRATCH_BYTES, stream);
}

qlora_status qlora_lora_linear_bwd_dx(const qlora_nf4_weight *w, const qlora_bf16 *dY, int64_t M, const qlora_bf16 *A,
                                      const qlora_bf16 *B, int r, float scaling, qlora_bf16 *dX, qlora_bf16 *G_save,
                                      void *ws, size_t ws_bytes, void *stream) {
    QL_TRY(check_weight(w));
    if (!dY || !dX) return fail(QLORA_ERR_ARG, "dY and dX must be non-NULL");
    if (!aligned16(dY) || !aligned16(dX)) return fail(QLORA_ERR_ALIGN, "dY and dX must be 16-byte aligned");
    if (G_save && !aligned16(G_save)) return fail(QLORA_ERR_ALIGN, "G_save must be 16-byte aligned");
    if (M <= 0 || M > INT32_MAX) return fail(QLORA_ERR_SHAPE, "M (%lld) must be in [1, 2^31)", (long long)M);
    QL_TRY(check_rank(r, scaling, A, B));
    const int64_t N = w->n_out, K = w->n_in;
    if (N % 8) return fail(QLORA_ERR_SHAPE, "n_out (%lld) must be a multiple of 8 for the dX pass", (long long)N);
    const size_t need = bwd_ws_bytes(M, N, K, r);
    QL_TRY(check_ws(ws, ws_bytes, need));
    QL_TRY(require_sm100());
    cudaStream_t st = static_cast<cudaStream_t>(stream);

    // CTA pairs at every M; split-K over n when the output tiles are few
    const DxPlan g = plan_dx(M, N, K, true);
    const bool split = g.splits > 1;
    const WsLayout L = ws_layout(M, K, r, split);
    uint8_t *wsb = static_cast<uint8_t *>(ws);
    uint16_t *gs = reinterpret_cast<uint16_t *>(wsb);
    float *gacc = reinterpret_cast<float *>(wsb + L.rank_bf16);
    float *dxacc = split ? reinterpret_cast<float *>(wsb + L.rank_bf16 + L.rank_acc) : nullptr;
    // G = dY B on tensor cores (B read MN-major), then bf16 copies G and scaling * G
    if (r > 0) QL_TRY(rank_side_product(false, dY, M, N, B, r, scaling, gs, gacc, G_save, st));
    if (dxacc) QL_TRY(cuda_check(cudaMemsetAsync(dxacc, 0, size_t(M) * K * 4, st), "zero split accumulator"));
    return launch_dx_pair(base_of(w, codebook_for(w->quant_type)), g, dY, M, N, K, A, r, gs, dX, dxacc, st);
}

// ------------------------------------------------------------------ Q8_0 route

static qlora_status check_q8(const qlora_q8_0_weight *w) {
    if (!w) return fail(QLORA_ERR_ARG, "weight descriptor is NULL");
    if (w->n_out <= 0 || w->n_in <= 0) return fail(QLORA_ERR_SHAPE, "n_out and n_in must be positive");
    if (w->n_in % 64) return fail(QLORA_ERR_SHAPE, "n_in (%lld) must be a multiple of 64", (long long)w->n_in);
    if (w->n_out > (int64_t(1) << 31) || w->n_in > (int64_t(1) << 31))
        return fail(QLORA_ERR_SHAPE, "n_out and n_in must be below 2^31");
    if (!w->q || !w->d) return fail(QLORA_ERR_ARG, "weight buffers must be non-NULL");
    if (!aligned16(w->q) || !aligned16(w->d)) return fail(QLORA_ERR_ALIGN, "weight buffers must be 16-byte aligned");
    return QLORA_OK;
}

static BaseW base_of_q8(const qlora_q8_0_weight *w) {
    BaseW b;
    b.codes = reinterpret_cast<const uint8_t *>(w->q);
    b.q8 = true;
    b.sc = ScaleSrc{nullptr, nullptr, 0, 1};
    b.d8 = w->d;
    b.level = nullptr;
    return b;
}

size_t qlora_q8_0_packed_bytes(int64_t numel) {
    if (numel <= 0 || numel % 32) return 0;
    return size_t(numel) + 2 * size_t(numel / 32);
}

qlora_status qlora_quantize_q8_0(const float *W, const qlora_q8_0_weight *w, void *stream) {
    QL_TRY(check_q8(w));
    if (!W) return fail(QLORA_ERR_ARG, "W is NULL");
    if (!aligned16(W)) return fail(QLORA_ERR_ALIGN, "W must be 16-byte aligned");
    QL_TRY(require_sm100());
    const int64_t numel = w->n_out * w->n_in;
    const int64_t grid = std::min<int64_t>(ceil_div(ceil_div(numel, 128), 8), int64_t(sm_count()) * 16);
    q8_0_encode_kernel<<<static_cast<unsigned>(grid), 256, 0, static_cast<cudaStream_t>(stream)>>>(W, w->q, w->d,
                                                                                                 numel);
    return launch_check("q8_0_encode_kernel launch");
}

qlora_status qlora_dequant_q8_0(const qlora_q8_0_weight *w, void *out, int out_is_bf16, void *stream) {
    QL_TRY(check_q8(w));
    if (!out) return fail(QLORA_ERR_ARG, "out is NULL");
    if (!aligned16(out)) return fail(QLORA_ERR_ALIGN, "out must be 16-byte aligned");
    if (out_is_bf16 != 0 && out_is_bf16 != 1) return fail(QLORA_ERR_ARG, "out_is_bf16 must be 0 or 1");
    QL_TRY(require_sm100());
    const int64_t n16 = w->n_out * w->n_in / 16;
    const int64_t grid = std::min<int64_t>(ceil_div(n16, 256), int64_t(sm_count()) * 8);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (out_is_bf16) q8_0_dequant_kernel<true><<<static_cast<unsigned>(grid), 256, 0, st>>>(w->q, w->d, out, n16);
    else q8_0_dequant_kernel<false><<<static_cast<unsigned>(grid), 256, 0, st>>>(w->q, w->d, out, n16);
    return launch_check("q8_0_dequant_kernel launch");
}

qlora_status qlora_q8_0_lora_linear_fwd(const qlora_q8_0_weight *w, const qlora_bf16 *X, int64_t M,
                                        const qlora_bf16 *A, const qlora_bf16 *B, int r, float scaling,
                                        qlora_bf16 *Y, qlora_bf16 *U_save, void *ws, size_t ws_bytes, void *stream) {
    QL_TRY(check_q8(w));
    if (!X || !Y) return fail(QLORA_ERR_ARG, "X and Y must be non-NULL");
    if (!aligned16(X) || !aligned16(Y)) return fail(QLORA_ERR_ALIGN, "X and Y must be 16-byte aligned");
    if (U_save && !aligned16(U_save)) return fail(QLORA_ERR_ALIGN, "U_save must be 16-byte aligned");
    if (M <= 0 || M > INT32_MAX) return fail(QLORA_ERR_SHAPE, "M (%lld) must be in [1, 2^31)", (long long)M);
    QL_TRY(check_rank(r, scaling, A, B));
    const int64_t N = w->n_out, K = w->n_in;
    const WsLayout L = ws_layout(M, N, r, false);
    QL_TRY(check_ws(ws, ws_bytes, L.total));
    QL_TRY(require_sm100());
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint8_t *wsb = static_cast<uint8_t *>(ws);
    uint16_t *us = reinterpret_cast<uint16_t *>(wsb);
    if (r > 0)
        QL_TRY(rank_side_product(true, X, M, K, A, r, scaling, us, reinterpret_cast<float *>(wsb + L.rank_bf16),
                                 U_save, st));
    // every M on CTA pairs (a small M pads the token tile)
    return launch_fwd_pair(base_of_q8(w), X, M, N, K, B, r, us, Y, st);
}

qlora_status qlora_q8_0_lora_linear_bwd_dx(const qlora_q8_0_weight *w, const qlora_bf16 *dY, int64_t M,
                                           const qlora_bf16 *A, const qlora_bf16 *B, int r, float scaling,
                                           qlora_bf16 *dX, qlora_bf16 *G_save, void *ws, size_t ws_bytes,
                                           void *stream) {
    QL_TRY(check_q8(w));
    if (!dY || !dX) return fail(QLORA_ERR_ARG, "dY and dX must be non-NULL");
    if (!aligned16(dY) || !aligned16(dX)) return fail(QLORA_ERR_ALIGN, "dY and dX must be 16-byte aligned");
    if (G_save && !aligned16(G_save)) return fail(QLORA_ERR_ALIGN, "G_save must be 16-byte aligned");
    if (M <= 0 || M > INT32_MAX) return fail(QLORA_ERR_SHAPE, "M (%lld) must be in [1, 2^31)", (long long)M);
    QL_TRY(check_rank(r, scaling, A, B));
    const int64_t N = w->n_out, K = w->n_in;
    if (N % 8) return fail(QLORA_ERR_SHAPE, "n_out (%lld) must be a multiple of 8 for the dX pass", (long long)N);
    const DxPlan g = plan_dx(M, N, K, true);
    const bool split = g.splits > 1;
    const WsLayout L = ws_layout(M, K, r, split);
    QL_TRY(check_ws(ws, ws_bytes, L.total));
    QL_TRY(require_sm100());
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint8_t *wsb = static_cast<uint8_t *>(ws);
    uint16_t *gs = reinterpret_cast<uint16_t *>(wsb);
    float *dxacc = split ? reinterpret_cast<float *>(wsb + L.rank_bf16 + L.rank_acc) : nullptr;
    if (r > 0)
        QL_TRY(rank_side_product(false, dY, M, N, B, r, scaling, gs, reinterpret_cast<float *>(wsb + L.rank_bf16),
                                 G_save, st));
    if (dxacc) QL_TRY(cuda_check(cudaMemsetAsync(dxacc, 0, size_t(M) * K * 4, st), "zero split accumulator"));
    return launch_dx_pair(base_of_q8(w), g, dY, M, N, K, A, r, gs, dX, dxacc, st);
}

qlora_status qlora_lora_grad_AB(const qlora_bf16 *X, const qlora_bf16 *dY, const qlora_bf16 *U, const qlora_bf16 *G,
                                int64_t M, int64_t N, int64_t K, int r, float scaling, float *dA, float *dB,
                                int accumulate, void *stream) {
    if (!X || !dY || !U || !G || !dA || !dB) return fail(QLORA_ERR_ARG, "all tensors must be non-NULL");
    if (!aligned16(X) || !aligned16(dY) || !aligned16(U) || !aligned16(G) || !aligned16(dA) || !aligned16(dB))
        return fail(QLORA_ERR_ALIGN, "all tensors must be 16-byte aligned");
    if (M <= 0 || N <= 0 || K <= 0 || M > INT32_MAX || N > INT32_MAX || K > INT32_MAX)
        return fail(QLORA_ERR_SHAPE, "M, N and K must be in [1, 2^31)");
    if (r < 8 || r > 128 || r % 8) return fail(QLORA_ERR_SHAPE, "r (%d) must be a multiple of 8 in [8, 128]", r);
    if (K % 64 || N % 8) return fail(QLORA_ERR_SHAPE, "K must be a multiple of 64 and N a multiple of 8");
    if (accumulate != 0 && accumulate != 1) return fail(QLORA_ERR_ARG, "accumulate must be 0 or 1");
    if (!std::isfinite(scaling)) return fail(QLORA_ERR_ARG, "scaling must be finite");
    QL_TRY(require_sm100());
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!accumulate) {
        QL_TRY(cuda_check(cudaMemsetAsync(dA, 0, size_t(r) * K * 4, st), "zero dA"));
        QL_TRY(cuda_check(cudaMemsetAsync(dB, 0, size_t(N) * r * 4, st), "zero dB"));
    }
    // dA^T [K, r] = s X^T G  and  dB [N, r] = s dY^T U, contraction over the M tokens
    QL_TRY(launch_skinny(X, 1, G, 1, M, K, r, scaling, dA, 1, K, st));
    QL_TRY(launch_skinny(dY, 1, U, 1, M, N, r, scaling, dB, r, 1, st));
    return QLORA_OK;
}

// ------------------------------------------------------------------ embedding

static qlora_status check_ids(const void *ids, int ids_bytes, int64_t T, int64_t V, int64_t H) {
    if (V <= 0 || H <= 0 || V > INT32_MAX || H > INT32_MAX) return fail(QLORA_ERR_SHAPE, "V and H must be in [1, 2^31)");
    if (H % 8) return fail(QLORA_ERR_SHAPE, "the row length (%lld) must be a multiple of 8", (long long)H);
    if (T < 0 || T > INT32_MAX) return fail(QLORA_ERR_SHAPE, "T (%lld) must be in [0, 2^31)", (long long)T);
    if (ids_bytes != 4 && ids_bytes != 8) return fail(QLORA_ERR_ARG, "ids_bytes must be 4 (int32) or 8 (int64)");
    if (T > 0 && !ids) return fail(QLORA_ERR_ARG, "ids is NULL");
    if (reinterpret_cast<uintptr_t>(ids) % ids_bytes)
        return fail(QLORA_ERR_ALIGN, "ids must be aligned to its elements (%d bytes)", ids_bytes);
    return QLORA_OK;
}

}  // extern "C" (a template has no C linkage)

template <int kTable, bool kDq>
static qlora_status launch_embed_fwd(emb::FwdArgs &a, const void *ids, int ids_bytes, int64_t T, int64_t V, int64_t H,
                                     float scale, void *Y, int y_is_bf16, void *stream) {
    QL_TRY(check_ids(ids, ids_bytes, T, V, H));
    if (y_is_bf16 != 0 && y_is_bf16 != 1) return fail(QLORA_ERR_ARG, "y_is_bf16 must be 0 or 1");
    if (!std::isfinite(scale)) return fail(QLORA_ERR_ARG, "scale must be finite");
    if (T == 0) return QLORA_OK;
    if (!Y) return fail(QLORA_ERR_ARG, "Y is NULL");
    if (!aligned16(Y)) return fail(QLORA_ERR_ALIGN, "Y must be 16-byte aligned");
    const int64_t segs = ceil_div(H, emb::kRun);
    a.seg_shift = 0;
    while ((1 << a.seg_shift) < segs && (2 << a.seg_shift) <= emb::kFwdWarps) ++a.seg_shift;
    const int64_t gy = ceil_div(segs, int64_t(1) << a.seg_shift), per_pass = emb::kFwdWarps >> a.seg_shift;
    if (gy > 65535) return fail(QLORA_ERR_SHAPE, "the row length (%lld) is too large", (long long)H);
    QL_TRY(require_sm100());
    // Tokens a warp takes one after the other: table set-up and id loads are shared, but a small batch then
    // leaves SMs idle.  1 / 2 / 4 tokens, 4-bit table: 4.3 / 5.3 / 7.7 us at 2048 x 4096 (1024 CTAs of one token a
    // warp), 16.7 / 15.8 / 16.6 at 4096 x 8192 (4096 CTAs), 58.5 / 53.2 / 52.1 at 16384 x 8192.
    const int64_t ctas = ceil_div(T, per_pass) * gy, full = int64_t(sm_count()) * 8;
    a.passes = ctas >= 8 * full ? emb::kFwdPasses : ctas >= 2 * full ? 2 : 1;
    a.ids = emb::Ids{ids, ids_bytes == 8};
    a.out = Y;
    a.T = T;
    a.V = V;
    a.H = static_cast<int>(H);
    a.scale = scale;
    return launch_pdl("embed_fwd_kernel launch",
                      y_is_bf16 ? emb::embed_fwd_kernel<kTable, kDq, true> : emb::embed_fwd_kernel<kTable, kDq, false>,
                      dim3(static_cast<unsigned>(ceil_div(T, per_pass * a.passes)), static_cast<unsigned>(gy)), emb::kFwdThreads, 0,
                      static_cast<cudaStream_t>(stream), a);
}

extern "C" {

qlora_status qlora_embed_nf4_fwd(const qlora_nf4_weight *w, const void *ids, int ids_bytes, int64_t T, float scale,
                                 void *Y, int y_is_bf16, void *stream) {
    QL_TRY(check_weight(w));
    emb::FwdArgs a = {};
    a.table = w->codes;
    a.sc = scale_src(w);
    const Codebook &cb = codebook_for(w->quant_type);
    for (int i = 0; i < 16; ++i) a.level[i] = cb.level[i];
    if (fmt_dq(w->format))
        return launch_embed_fwd<emb::kTableNf4, true>(a, ids, ids_bytes, T, w->n_out, w->n_in, scale, Y, y_is_bf16, stream);
    return launch_embed_fwd<emb::kTableNf4, false>(a, ids, ids_bytes, T, w->n_out, w->n_in, scale, Y, y_is_bf16, stream);
}

qlora_status qlora_embed_q8_0_fwd(const qlora_q8_0_weight *w, const void *ids, int ids_bytes, int64_t T, float scale,
                                  void *Y, int y_is_bf16, void *stream) {
    QL_TRY(check_q8(w));
    emb::FwdArgs a = {};
    a.table = w->q;
    a.d8 = w->d;
    return launch_embed_fwd<emb::kTableQ8, false>(a, ids, ids_bytes, T, w->n_out, w->n_in, scale, Y, y_is_bf16, stream);
}

qlora_status qlora_embed_fwd(const void *E, int e_is_bf16, int64_t V, int64_t H, const void *ids, int ids_bytes,
                             int64_t T, float scale, void *Y, int y_is_bf16, void *stream) {
    if (!E) return fail(QLORA_ERR_ARG, "E is NULL");
    if (!aligned16(E)) return fail(QLORA_ERR_ALIGN, "E must be 16-byte aligned");
    if (e_is_bf16 != 0 && e_is_bf16 != 1) return fail(QLORA_ERR_ARG, "e_is_bf16 must be 0 or 1");
    emb::FwdArgs a = {};
    a.table = E;
    if (e_is_bf16) return launch_embed_fwd<emb::kTableBf16, false>(a, ids, ids_bytes, T, V, H, scale, Y, y_is_bf16, stream);
    return launch_embed_fwd<emb::kTableF32, false>(a, ids, ids_bytes, T, V, H, scale, Y, y_is_bf16, stream);
}

// Sorted tokens per chunk of the gradient's reduction: a power of two in [8, 128], about eight blocks per
// SM (148) where T allows it; longer chunks leave fewer partial sums, shorter ones more blocks.  Added, bf16 to
// fp32, chunks of 8 / 16 / 32 / 64 / 128: 24 / 29 / 29 / 30 / 41 us at 2047 x 4096, 52 / 51 / 52 / 61 / 69 at 8192 x 4096,
// 285 / 235 / 212 / 202 / 200 at 32768 x 8192; the rule takes 8, 16 and 128.
static int embed_chunk(int64_t T, int64_t H) {
    const int64_t want = T * ceil_div(H, emb::kRedCols) / (8 * 148);
    int c = 8;
    while (c < emb::kMaxChunk && 2 * c <= want) c *= 2;
    return c;
}

size_t qlora_embed_grad_workspace_bytes(int64_t T, int64_t V, int64_t H) {
    if (T < 0 || V <= 0 || H <= 0 || T > INT32_MAX || V > INT32_MAX || H > INT32_MAX || H % 8) return 0;
    return 4 * round256(size_t(T) * 4) + round256(size_t(ceil_div(V, 32)) * 4) +
           size_t(ceil_div(T, embed_chunk(T, H))) * 2 * size_t(H) * 4;
}

qlora_status qlora_embed_grad(const void *ids, int ids_bytes, int64_t T, const void *dY, int dy_is_bf16, int64_t V,
                              int64_t H, float scale, int64_t padding_id, void *dE, int de_is_bf16, int accumulate,
                              void *ws, size_t ws_bytes, void *stream) {
    QL_TRY(check_ids(ids, ids_bytes, T, V, H));
    if (!dE || (T > 0 && !dY)) return fail(QLORA_ERR_ARG, "dY and dE must be non-NULL");
    if (!aligned16(dY) || !aligned16(dE)) return fail(QLORA_ERR_ALIGN, "dY and dE must be 16-byte aligned");
    if ((dy_is_bf16 | 1) != 1 || (de_is_bf16 | 1) != 1) return fail(QLORA_ERR_ARG, "dy_is_bf16 and de_is_bf16 must be 0 or 1");
    if (accumulate != 0 && accumulate != 1) return fail(QLORA_ERR_ARG, "accumulate must be 0 or 1");
    if (!std::isfinite(scale)) return fail(QLORA_ERR_ARG, "scale must be finite");
    if (padding_id < -1 || padding_id >= V) return fail(QLORA_ERR_ARG, "padding_id (%lld) must be -1 or a row", (long long)padding_id);
    QL_TRY(check_ws(ws, ws_bytes, T > 0 ? qlora_embed_grad_workspace_bytes(T, V, H) : 0));
    if (T == 0 && accumulate) return QLORA_OK;
    emb::GradArgs a = {};
    a.ids = emb::Ids{ids, ids_bytes == 8};
    a.T = T;
    a.V = V;
    a.H = H;
    a.pad = padding_id;
    uint8_t *wsb = static_cast<uint8_t *>(ws);
    const size_t list = round256(size_t(T) * 4), mask = round256(size_t(ceil_div(V, 32)) * 4);
    for (int i = 0; i < 2; ++i) {
        a.key[i] = reinterpret_cast<uint32_t *>(wsb + list * i);
        a.pos[i] = reinterpret_cast<uint32_t *>(wsb + list * (2 + i));
    }
    a.named = reinterpret_cast<uint32_t *>(wsb + 4 * list);
    a.part = reinterpret_cast<float *>(wsb + 4 * list + mask);
    int nbits = 1;                                   // of the largest key, V
    while ((V >> nbits) != 0) ++nbits;
    a.passes = static_cast<int>(ceil_div(nbits, emb::kMaxBits));
    a.bits = static_cast<int>(ceil_div(nbits, a.passes));
    a.dY = dY;
    a.dy_bf16 = dy_is_bf16;
    a.dE = dE;
    a.de_bf16 = de_is_bf16;
    a.accumulate = accumulate;
    a.scale = scale;
    a.chunk = embed_chunk(T, H);
    a.nchunks = ceil_div(T, a.chunk);
    const int64_t tiles = ceil_div(H, emb::kRedCols), jtiles = ceil_div(H, emb::kJoinCols);
    if (jtiles > 65535) return fail(QLORA_ERR_SHAPE, "H (%lld) must be at most %d", (long long)H, 65535 * emb::kJoinCols);
    QL_TRY(require_sm100());
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int variant = 4 * dy_is_bf16 + 2 * de_is_bf16 + accumulate;
    const bool few = T > 0 && T <= emb::kFewTokens;
    if (few) {
        void (*const sum[8])(emb::GradArgs) = {
            emb::embed_few_kernel<false, false, false>, emb::embed_few_kernel<false, false, true>,
            emb::embed_few_kernel<false, true, false>,  emb::embed_few_kernel<false, true, true>,
            emb::embed_few_kernel<true, false, false>,  emb::embed_few_kernel<true, false, true>,
            emb::embed_few_kernel<true, true, false>,   emb::embed_few_kernel<true, true, true>};
        QL_TRY(launch_pdl("embed_few_kernel launch", sum[variant],
                          dim3(static_cast<unsigned>(ceil_div(T, emb::kFewRun)), static_cast<unsigned>(tiles)), emb::kRedThreads, 0, st, a));
    } else if (T > 0) {
        if (!accumulate)
            QL_TRY(launch_pdl("embed_mark_kernel launch", emb::embed_mark_kernel, dim3(emb::kSortCtas), emb::kSortThreads, 0, st, a));
        if (T <= emb::kHeldTokens) {
            const bool one = T <= emb::kOneTokens;
            const int rounds = static_cast<int>(ceil_div(T, int64_t(one ? 1 : emb::kSortCtas) * emb::kSortThreads));
            void (*sort)(emb::GradArgs, int);
            if (one) sort = rounds == 1 ? emb::embed_sort_one_kernel<1> : emb::embed_sort_one_kernel<2>;
            else if (rounds <= 2) sort = emb::embed_sort_held_kernel<2>;
            else sort = rounds <= 4 ? emb::embed_sort_held_kernel<4> : emb::embed_sort_held_kernel<emb::kCtaRounds>;
            QL_TRY(set_smem(sort, emb::held_smem(rounds)));
            QL_TRY(launch_pdl("embed_sort kernel launch", sort, dim3(one ? 1 : emb::kSortCtas), emb::kSortThreads,
                              emb::held_smem(rounds), st, a, rounds));
        } else {
            QL_TRY(set_smem(emb::embed_sort_swept_kernel, emb::kSortSmem));
            QL_TRY(launch_pdl("embed_sort_swept_kernel launch", emb::embed_sort_swept_kernel, dim3(emb::kSortCtas),
                              emb::kSortThreads, emb::kSortSmem, st, a));
        }
        void (*const reduce[8])(emb::GradArgs) = {
            emb::embed_reduce_kernel<false, false, false>, emb::embed_reduce_kernel<false, false, true>,
            emb::embed_reduce_kernel<false, true, false>,  emb::embed_reduce_kernel<false, true, true>,
            emb::embed_reduce_kernel<true, false, false>,  emb::embed_reduce_kernel<true, false, true>,
            emb::embed_reduce_kernel<true, true, false>,   emb::embed_reduce_kernel<true, true, true>};
        QL_TRY(launch_pdl("embed_reduce_kernel launch", reduce[variant],
                          dim3(static_cast<unsigned>(a.nchunks), static_cast<unsigned>(tiles)), emb::kRedThreads, 0, st, a));
        // (more than kFewTokens tokens are more than one chunk)
        QL_TRY(launch_pdl("embed_join_kernel launch", de_is_bf16 ? emb::embed_join_kernel<true> : emb::embed_join_kernel<false>,
                          dim3(static_cast<unsigned>(ceil_div(a.nchunks - 1, emb::kJoinWarps)), static_cast<unsigned>(jtiles)),
                          emb::kJoinWarps * 32, 0, st, a));
    }
    if (!accumulate) {
        a.zero_rows = static_cast<int>(std::min<int64_t>(V, std::max<int64_t>(1, emb::kZeroBytes / (H * (de_is_bf16 ? 2 : 4)))));
        QL_TRY(launch_pdl("embed_zero_kernel launch", few ? emb::embed_zero_kernel<true> : emb::embed_zero_kernel<false>,
                          dim3(static_cast<unsigned>(ceil_div(V, a.zero_rows))), emb::kZeroThreads, 0, st, a));
    }
    return QLORA_OK;
}

// ------------------------------------------------------------------ optimizer

static_assert(sizeof(qlora_adamw_tensor) == 80 && offsetof(qlora_adamw_tensor, flags) == 72, "ABI layout");
static_assert(sizeof(qlora_adamw_plan) == 48, "ABI layout");
constexpr int32_t kOptFlags = QLORA_OPT_PARAM_BF16 | QLORA_OPT_GRAD_BF16 | QLORA_OPT_STATE_8BIT | QLORA_OPT_GRAD_ONLY;
constexpr int32_t kPlanMagic = 0x51504c4e;

// Elements of a plan's chunk for `numel` in all: the largest of 256, 512 and 1024 that still gives every warp of
// the device (64 per SM) a chunk.  256 / 512 / 1024 / 2048: 2.9 / 3.1 / 4.6 / 7.1 us for a 32-bit step on 262 K parameters,
// 36.8 / 31.1 / 33.1 / 37.4 for an 8-bit one (and its state read back) on 5.8 M, 144 / 147 / 149 / 153 and
// 184 / 152 / 154 / 158 on 32 M, and 92 / 83 / 81 / 80 for the norm of 129 M gradients.
static int64_t plan_chunk(int64_t numel) {
    int64_t c = 1024;
    while (c > 256 && numel / c < 64 * 148) c /= 2;
    return c;
}

static qlora_status check_opt_tensors(const qlora_adamw_tensor *ts, int64_t count, int64_t *numel) {
    if (!ts) return fail(QLORA_ERR_ARG, "tensors is NULL");
    if (count < 1 || count > INT32_MAX) return fail(QLORA_ERR_SHAPE, "count (%lld) must be in [1, 2^31)", (long long)count);
    *numel = 0;
    for (int64_t i = 0; i < count; ++i) {
        const qlora_adamw_tensor &t = ts[i];
        const long long k = (long long)i;
        if (t.numel < 0 || t.numel > (int64_t(1) << 40)) return fail(QLORA_ERR_SHAPE, "tensor %lld: numel out of range", k);
        if (t.flags & ~kOptFlags) return fail(QLORA_ERR_ARG, "tensor %lld: unknown flags (%d)", k, t.flags);
        if (t.numel == 0) continue;
        *numel += t.numel;
        if (!t.grad) return fail(QLORA_ERR_ARG, "tensor %lld: grad is NULL", k);
        if (!aligned16(t.grad)) return fail(QLORA_ERR_ALIGN, "tensor %lld: grad must be 16-byte aligned", k);
        if (t.flags & QLORA_OPT_GRAD_ONLY) continue;
        if (!t.param || !t.exp_avg || !t.exp_avg_sq) return fail(QLORA_ERR_ARG, "tensor %lld: param, exp_avg and exp_avg_sq must be non-NULL", k);
        if (!aligned16(t.param) || !aligned16(t.exp_avg) || !aligned16(t.exp_avg_sq) || !aligned16(t.param_bf16))
            return fail(QLORA_ERR_ALIGN, "tensor %lld: buffers must be 16-byte aligned", k);
        if (t.param_bf16 && (t.flags & QLORA_OPT_PARAM_BF16))
            return fail(QLORA_ERR_ARG, "tensor %lld: a bf16 copy goes with a float32 parameter only", k);
        if (t.flags & QLORA_OPT_STATE_8BIT) {
            if (!t.exp_avg_step || !t.exp_avg_sq_step) return fail(QLORA_ERR_ARG, "tensor %lld: 8-bit states need their block steps", k);
            if (((reinterpret_cast<uintptr_t>(t.exp_avg_step) | reinterpret_cast<uintptr_t>(t.exp_avg_sq_step)) & 3) != 0)
                return fail(QLORA_ERR_ALIGN, "tensor %lld: block steps must be 4-byte aligned", k);
        }
        if (!std::isfinite(t.lr_scale) || !std::isfinite(t.weight_decay) || t.lr_scale < 0 || t.weight_decay < 0)
            return fail(QLORA_ERR_ARG, "tensor %lld: lr_scale and weight_decay must be finite and not negative", k);
    }
    return QLORA_OK;
}

// A run of device memory that a step reads or writes.
struct MemRange {
    uintptr_t lo, hi;
    bool written;
    int64_t tensor;
};
// Refuses a list whose written buffers overlap one another or a gradient: its elements would be updated
// twice, or in an order that nothing fixes.  Gradients may share memory.
static qlora_status check_opt_overlap(const qlora_adamw_tensor *ts, int64_t count) {
    MemRange *r = static_cast<MemRange *>(std::malloc(size_t(count) * 7 * sizeof(MemRange)));
    if (!r) return fail(QLORA_ERR_ARG, "no host memory for the plan");
    int64_t n = 0;
    for (int64_t i = 0; i < count; ++i) {
        const qlora_adamw_tensor &t = ts[i];
        if (t.numel == 0) continue;
        const int64_t state = (t.flags & QLORA_OPT_STATE_8BIT) ? t.numel : 4 * t.numel, steps = 4 * ceil_div(t.numel, optim::kBlock);
        auto add = [&](const void *p, int64_t bytes, bool written) {
            const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
            if (p) r[n++] = MemRange{lo, lo + uintptr_t(bytes), written, i};
        };
        add(t.grad, t.numel * ((t.flags & QLORA_OPT_GRAD_BF16) ? 2 : 4), false);
        if (t.flags & QLORA_OPT_GRAD_ONLY) continue;
        add(t.param, t.numel * ((t.flags & QLORA_OPT_PARAM_BF16) ? 2 : 4), true);
        add(t.param_bf16, t.numel * 2, true);
        add(t.exp_avg, state, true);
        add(t.exp_avg_sq, state, true);
        if (t.flags & QLORA_OPT_STATE_8BIT) {
            add(t.exp_avg_step, steps, true);
            add(t.exp_avg_sq_step, steps, true);
        }
    }
    std::sort(r, r + n, [](const MemRange &a, const MemRange &b) { return a.lo < b.lo; });
    uintptr_t end_read = 0, end_written = 0;
    int64_t bad = -1;
    for (int64_t i = 0; i < n && bad < 0; ++i) {
        if (r[i].lo < end_written || (r[i].written && r[i].lo < end_read)) bad = r[i].tensor;
        uintptr_t &end = r[i].written ? end_written : end_read;
        end = std::max(end, r[i].hi);
    }
    std::free(r);
    if (bad >= 0) return fail(QLORA_ERR_ARG, "tensor %lld: a buffer overlaps one that the step writes", (long long)bad);
    return QLORA_OK;
}

static int64_t plan_chunks(const qlora_adamw_tensor *ts, int64_t count, int64_t chunk) {
    int64_t n = 0;
    for (int64_t i = 0; i < count; ++i) n += ceil_div(ts[i].numel, chunk);
    return n;
}

// head, chunk list, tensors
static size_t plan_need(int64_t count, int64_t nchunks) {
    return sizeof(optim::PlanHead) + size_t(nchunks) * sizeof(optim::Chunk) + size_t(count) * sizeof(optim::TensorDesc);
}

size_t qlora_adamw_plan_bytes(const qlora_adamw_tensor *tensors, int64_t count) {
    int64_t numel = 0;
    if (check_opt_tensors(tensors, count, &numel) != QLORA_OK) return 0;
    return plan_need(count, plan_chunks(tensors, count, plan_chunk(numel)));
}

qlora_status qlora_adamw_plan_init(const qlora_adamw_tensor *tensors, int64_t count, void *buffer, size_t bytes,
                                   qlora_adamw_plan *plan, void *stream) {
    if (!plan) return fail(QLORA_ERR_ARG, "plan is NULL");
    *plan = qlora_adamw_plan{};
    int64_t numel = 0;
    QL_TRY(check_opt_tensors(tensors, count, &numel));
    QL_TRY(check_opt_overlap(tensors, count));
    const int64_t chunk = plan_chunk(numel), nchunks = plan_chunks(tensors, count, chunk);
    if (nchunks > (1 << 30)) return fail(QLORA_ERR_SHAPE, "the tensors have too many elements for one plan");
    const size_t need = plan_need(count, nchunks);
    if (!buffer || bytes < need) return fail(QLORA_ERR_WORKSPACE, "the plan buffer holds %zu bytes, %zu needed", buffer ? bytes : size_t(0), need);
    if (reinterpret_cast<uintptr_t>(buffer) % 256) return fail(QLORA_ERR_ALIGN, "the plan buffer must be 256-byte aligned");
    QL_TRY(require_sm100());
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    QL_TRY(cuda_check(cudaStreamIsCapturing(st, &cap), "cudaStreamIsCapturing"));
    if (cap != cudaStreamCaptureStatusNone) return fail(QLORA_ERR_ARG, "a plan cannot be made during stream capture");
    optim::TensorDesc *const host = static_cast<optim::TensorDesc *>(std::calloc(size_t(count), sizeof(optim::TensorDesc)));
    if (!host) return fail(QLORA_ERR_ARG, "no host memory for the plan");
    // tensors with 32-bit states first, then those with 8-bit states: a kernel for each
    int64_t n = 0, first = 0, chunks32 = 0;
    int32_t grad_only = 0, elem8 = 0;
    for (int pass = 0; pass < 2; ++pass) {
        for (int64_t i = 0; i < count; ++i) {
            const qlora_adamw_tensor &t = tensors[i];
            const bool only = (t.flags & QLORA_OPT_GRAD_ONLY) != 0, eight = !only && (t.flags & QLORA_OPT_STATE_8BIT) != 0;
            if (t.numel == 0 || eight != (pass == 1)) continue;
            auto at = [](const void *p) { return uint64_t(reinterpret_cast<uintptr_t>(p)); };
            optim::TensorDesc &d = host[n++];
            d.numel = t.numel;
            d.first = first;
            first += ceil_div(t.numel, chunk);
            d.pb = (t.flags & QLORA_OPT_PARAM_BF16) ? 2 : 4;
            d.gb = (t.flags & QLORA_OPT_GRAD_BF16) ? 2 : 4;
            d.sb = eight ? 1 : 4;
            d.base.g = at(t.grad);
            d.base.flags = uint32_t(t.flags) & (optim::kParamBf16 | optim::kGradBf16);
            if (only) {
                grad_only = 1;
                continue;
            }
            d.base.p = at(t.param);
            d.base.copy = at(t.param_bf16);
            d.base.m = at(t.exp_avg);
            d.base.v = at(t.exp_avg_sq);
            d.base.dm = eight ? at(t.exp_avg_step) : 0;
            d.base.dv = eight ? at(t.exp_avg_sq_step) : 0;
            d.base.lr_scale = t.lr_scale;
            d.base.decay = t.weight_decay;
            if (eight) elem8 = std::max(elem8, d.gb + d.pb + 2);
        }
        if (pass == 0) chunks32 = first;
    }
    optim::Chunk *const list = reinterpret_cast<optim::Chunk *>(static_cast<optim::PlanHead *>(buffer) + 1);
    optim::TensorDesc *const descs = reinterpret_cast<optim::TensorDesc *>(list + nchunks);
    cudaError_t e = cudaMemsetAsync(buffer, 0, sizeof(optim::PlanHead), st);
    if (e == cudaSuccess && n > 0) e = cudaMemcpyAsync(descs, host, size_t(n) * sizeof(optim::TensorDesc), cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess && n > 0) {
        optim::expand_plan_kernel<<<static_cast<unsigned>(ceil_div(nchunks, optim::kThreads)), optim::kThreads, 0, st>>>(
            descs, static_cast<int>(n), static_cast<int>(chunk), nchunks, list);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    std::free(host);
    QL_TRY(cuda_check(e, "making of the plan"));
    plan->buffer = buffer;
    plan->chunks = nchunks;
    plan->chunks32 = chunks32;
    plan->numel = numel;
    plan->grad_only = grad_only;
    plan->elem8 = elem8;
    plan->magic = kPlanMagic;
    return QLORA_OK;
}

static qlora_status check_plan(const qlora_adamw_plan *plan) {
    if (!plan) return fail(QLORA_ERR_ARG, "plan is NULL");
    if (plan->magic != kPlanMagic || !plan->buffer) return fail(QLORA_ERR_ARG, "plan was not made by qlora_adamw_plan_init");
    return QLORA_OK;
}
static optim::PlanHead *plan_head(const qlora_adamw_plan *plan) { return static_cast<optim::PlanHead *>(plan->buffer); }
static const optim::Chunk *plan_list(const qlora_adamw_plan *plan) {
    return reinterpret_cast<const optim::Chunk *>(plan_head(plan) + 1);
}
// CTAs for `chunks` chunks: a warp each, at most `per_sm` CTAs per SM
static dim3 plan_grid(int64_t chunks, int per_sm) {
    return dim3(static_cast<unsigned>(std::max<int64_t>(
        1, std::min<int64_t>(ceil_div(chunks, optim::kWarps), int64_t(per_sm) * sm_count()))));
}

qlora_status qlora_adamw_step(const qlora_adamw_plan *plan, double lr, double beta1, double beta2, double eps,
                              int64_t step, const float *grad_scale, const float *lr_dev, int64_t *step_dev,
                              void *stream) {
    QL_TRY(check_plan(plan));
    if (plan->grad_only) return fail(QLORA_ERR_ARG, "the plan holds QLORA_OPT_GRAD_ONLY tensors");
    if (!(beta1 >= 0 && beta1 < 1 && beta2 >= 0 && beta2 < 1)) return fail(QLORA_ERR_ARG, "betas must be in [0, 1)");
    if (!(eps >= 0) || !std::isfinite(eps)) return fail(QLORA_ERR_ARG, "eps must be finite and not negative");
    if (!lr_dev && !(lr >= 0 && std::isfinite(lr))) return fail(QLORA_ERR_ARG, "lr must be finite and not negative");
    if (step_dev ? step != 0 : step < 1)
        return fail(QLORA_ERR_ARG, "step (%lld) must be at least 1, or 0 with a step counter on the device", (long long)step);
    if ((reinterpret_cast<uintptr_t>(grad_scale) | reinterpret_cast<uintptr_t>(lr_dev)) & 3 || reinterpret_cast<uintptr_t>(step_dev) & 7)
        return fail(QLORA_ERR_ALIGN, "grad_scale, lr_dev and step_dev must be aligned to their types");
    QL_TRY(require_sm100());
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    optim::StepArgs a = {};
    a.head = plan_head(plan);
    a.coef = grad_scale;
    a.lr_dev = lr_dev;
    a.lr = lr_dev ? 0.f : static_cast<float>(lr);
    auto pair = [](double x) {
        const float f = static_cast<float>(x);
        uint32_t u;
        std::memcpy(&u, &f, 4);
        return uint64_t(u) << 32 | u;
    };
    a.one = pair(1.0);
    a.b1 = pair(beta1);
    a.w1 = pair(1.0 - beta1);
    a.b2 = pair(beta2);
    a.w2 = pair(1.0 - beta2);
    if (step_dev) {
        a.counted = 1;
        QL_TRY(launch_pdl("step_scalars_kernel launch", optim::step_scalars_kernel, dim3(1), 1, 0, st, plan_head(plan), step_dev,
                          grad_scale, beta1, beta2, eps));
    } else {
        const double bc1 = 1.0 - std::pow(beta1, double(step));
        a.ds = static_cast<float>(bc1 / std::sqrt(1.0 - std::pow(beta2, double(step))));
        a.de = static_cast<float>(bc1 * eps);
    }
    if (plan->chunks32 > 0) {
        a.chunks = plan_list(plan);
        a.nchunks = static_cast<int>(plan->chunks32);
        QL_TRY(launch_pdl("adamw32_kernel launch", optim::adamw32_kernel,
                          dim3(static_cast<unsigned>(ceil_div(a.nchunks, optim::kWarps))), optim::kThreads, 0, st, a));
    }
    if (plan->chunks > plan->chunks32) {
        a.chunks = plan_list(plan) + plan->chunks32;
        a.nchunks = static_cast<int>(plan->chunks - plan->chunks32);
        // The stages of three CTAs fit an SM's shared memory up to 8 bytes an element, of two at 10.  One / two / three
        // CTAs, 32 M parameters, state read back: 232 / 169 / 136 us at 6 bytes, 228 / 181 / 148 at 8, 225 / 153 at 10.
        const int smem = optim::step8_smem(plan->elem8);
        QL_TRY(set_smem(optim::adamw8_kernel, optim::step8_smem(10)));
        QL_TRY(launch_pdl("adamw8_kernel launch", optim::adamw8_kernel, plan_grid(a.nchunks, plan->elem8 > 8 ? 2 : optim::kCtas8),
                          optim::kThreads, smem, st, a, int(plan->elem8)));
    }
    return QLORA_OK;
}

qlora_status qlora_grad_norm(const qlora_adamw_plan *plan, float max_norm, float *out, void *stream) {
    QL_TRY(check_plan(plan));
    if (!(max_norm > 0)) return fail(QLORA_ERR_ARG, "max_norm must be positive (infinity for no limit)");
    if (!out) return fail(QLORA_ERR_ARG, "out is NULL");
    if (reinterpret_cast<uintptr_t>(out) & 3) return fail(QLORA_ERR_ALIGN, "out must be 4-byte aligned");
    QL_TRY(require_sm100());
    const int64_t per_warp = std::max<int64_t>(1, ceil_div(plan->chunks, int64_t(optim::kWarps) * optim::kPartials));
    if (per_warp > INT32_MAX) return fail(QLORA_ERR_SHAPE, "the plan is too large");
    const int64_t grid = std::max<int64_t>(1, ceil_div(plan->chunks, optim::kWarps * per_warp));
    return launch_pdl("grad_norm_kernel launch", optim::grad_norm_kernel, dim3(static_cast<unsigned>(grid)), optim::kThreads, 0,
                      static_cast<cudaStream_t>(stream), plan_list(plan), plan_head(plan), plan->chunks, static_cast<int>(per_warp),
                      max_norm, out);
}

static qlora_status check_adam8(const void *codes, int kind, const float *steps, const float *x, int64_t numel) {
    if (kind != QLORA_ADAM8_FIRST && kind != QLORA_ADAM8_SECOND) return fail(QLORA_ERR_ARG, "kind (%d) must be a QLORA_ADAM8_* value", kind);
    if (numel < 0 || numel > (int64_t(1) << 40)) return fail(QLORA_ERR_SHAPE, "numel out of range");
    if (numel == 0) return QLORA_OK;
    if (!codes || !steps || !x) return fail(QLORA_ERR_ARG, "codes, steps and x must be non-NULL");
    if (!aligned16(codes) || !aligned16(x)) return fail(QLORA_ERR_ALIGN, "codes and x must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(steps) & 3) return fail(QLORA_ERR_ALIGN, "steps must be 4-byte aligned");
    return QLORA_OK;
}
static dim3 adam8_grid(int64_t numel) {
    return dim3(static_cast<unsigned>(std::min<int64_t>(ceil_div(numel, optim::kBlock * optim::kWarps), int64_t(sm_count()) * 32)));
}

qlora_status qlora_adam8_encode(const float *x, int kind, void *codes, float *steps, int64_t numel, void *stream) {
    QL_TRY(check_adam8(codes, kind, steps, x, numel));
    if (numel == 0) return QLORA_OK;
    QL_TRY(require_sm100());
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint8_t *c = static_cast<uint8_t *>(codes);
    return launch_pdl("adam8_encode_kernel launch",
                      kind == QLORA_ADAM8_SECOND ? optim::adam8_encode_kernel<true> : optim::adam8_encode_kernel<false>,
                      adam8_grid(numel), optim::kThreads, 0, st, x, c, steps, numel);
}

qlora_status qlora_adam8_decode(const void *codes, int kind, const float *steps, float *x, int64_t numel, void *stream) {
    QL_TRY(check_adam8(codes, kind, steps, x, numel));
    if (numel == 0) return QLORA_OK;
    QL_TRY(require_sm100());
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const uint8_t *c = static_cast<const uint8_t *>(codes);
    return launch_pdl("adam8_decode_kernel launch",
                      kind == QLORA_ADAM8_SECOND ? optim::adam8_decode_kernel<true> : optim::adam8_decode_kernel<false>,
                      adam8_grid(numel), optim::kThreads, 0, st, c, steps, x, numel);
}

}  // extern "C"
