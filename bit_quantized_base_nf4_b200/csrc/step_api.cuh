// step_api.cuh -- the C ABI of the calls around the layer in a training step: embedding lookup and gradient,
// gradient norm, AdamW.  Part of the library's one translation unit: qlora_nf4.cu includes it last.
#pragma once

#include <cstdlib>
#include <utility>

#include "embedding.cuh"
#include "optimizer.cuh"

namespace {

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

}  // namespace

extern "C" {

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
    const bool few = T <= emb::kFewTokens;
    // what is zeroed beside the sort and beside the sums (the rules stand at zero_rows)
    const int64_t row_bytes = H * (de_is_bf16 ? 2 : 4), table = accumulate ? 0 : V * row_bytes;
    const bool one = T <= (table >= emb::kOneTable ? emb::kOneWritten : emb::kOneTokens);
    a.sort_ctas = one ? 1 : emb::kSortCtas;
    a.sum_ctas = static_cast<int>(few ? ceil_div(T, emb::kFewRun) : a.nchunks);
    int64_t early_ctas = 0, zero_columns = 0;
    if (!accumulate) {
        const auto rows_of = [&](int64_t bytes) { return std::min(V, std::max<int64_t>(1, bytes / row_bytes)); };
        if (!few && (one || table >= emb::kEarlyTable)) {
            const int64_t beside = emb::kEarlyClusters * emb::kSortCtas;
            const int64_t rows = one ? rows_of(emb::kOneZeroBytes) : std::min(rows_of(emb::kEarlyBytes), ceil_div(V, 2 * beside));
            a.early = one ? V : std::min(V, rows * beside);
            a.sort_rows = static_cast<int>(rows);
            early_ctas = ceil_div(ceil_div(a.early, rows), a.sort_ctas) * a.sort_ctas;      // whole clusters
        }
        a.sum_rows = static_cast<int>(rows_of(emb::kZeroBytes));
        zero_columns = ceil_div(ceil_div(V - a.early, a.sum_rows), tiles);
    }
    const dim3 sort_grid(static_cast<unsigned>(a.sort_ctas + early_ctas));
    const dim3 sum_grid(static_cast<unsigned>(a.sum_ctas + zero_columns), static_cast<unsigned>(tiles));
    if (few) {
        void (*const sum[8])(emb::GradArgs) = {
            emb::embed_few_kernel<false, false, false>, emb::embed_few_kernel<false, false, true>,
            emb::embed_few_kernel<false, true, false>,  emb::embed_few_kernel<false, true, true>,
            emb::embed_few_kernel<true, false, false>,  emb::embed_few_kernel<true, false, true>,
            emb::embed_few_kernel<true, true, false>,   emb::embed_few_kernel<true, true, true>};
        QL_TRY(launch_pdl("embed_few_kernel launch", sum[variant], sum_grid, emb::kRedThreads, 0, st, a));
    } else {
        if (!accumulate && !one)
            QL_TRY(launch_pdl("embed_mark_kernel launch", emb::embed_mark_kernel, dim3(emb::kSortCtas), emb::kSortThreads, 0, st, a));
        if (T <= emb::kHeldTokens) {
            const int rounds = static_cast<int>(ceil_div(T, int64_t(one ? 1 : emb::kSortCtas) * emb::kSortThreads));
            void (*sort)(emb::GradArgs, int);
            if (one) sort = rounds == 1 ? emb::embed_sort_one_kernel<1> : rounds == 2 ? emb::embed_sort_one_kernel<2> : emb::embed_sort_one_kernel<4>;
            else if (rounds <= 2) sort = emb::embed_sort_held_kernel<2>;
            else sort = rounds <= 4 ? emb::embed_sort_held_kernel<4> : emb::embed_sort_held_kernel<emb::kCtaRounds>;
            QL_TRY(set_smem(sort, emb::held_smem(rounds)));
            QL_TRY(launch_pdl("embed_sort kernel launch", sort, sort_grid, emb::kSortThreads,
                              emb::held_smem(rounds), st, a, rounds));
        } else {
            QL_TRY(set_smem(emb::embed_sort_swept_kernel, emb::kSortSmem));
            QL_TRY(launch_pdl("embed_sort_swept_kernel launch", emb::embed_sort_swept_kernel, sort_grid,
                              emb::kSortThreads, emb::kSortSmem, st, a));
        }
        void (*const reduce[8])(emb::GradArgs) = {
            emb::embed_reduce_kernel<false, false, false>, emb::embed_reduce_kernel<false, false, true>,
            emb::embed_reduce_kernel<false, true, false>,  emb::embed_reduce_kernel<false, true, true>,
            emb::embed_reduce_kernel<true, false, false>,  emb::embed_reduce_kernel<true, false, true>,
            emb::embed_reduce_kernel<true, true, false>,   emb::embed_reduce_kernel<true, true, true>};
        QL_TRY(launch_pdl("embed_reduce_kernel launch", reduce[variant], sum_grid, emb::kRedThreads, 0, st, a));
        // (more than kFewTokens tokens are more than one chunk)
        QL_TRY(launch_pdl("embed_join_kernel launch", de_is_bf16 ? emb::embed_join_kernel<true> : emb::embed_join_kernel<false>,
                          dim3(static_cast<unsigned>(ceil_div(a.nchunks - 1, emb::kJoinWarps)), static_cast<unsigned>(jtiles)),
                          emb::kJoinWarps * 32, 0, st, a));
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
        if (*numel > (int64_t(1) << 40)) return fail(QLORA_ERR_SHAPE, "the tensors have too many elements for one plan (tensor %lld)", k);
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
    // a smaller eps (1 - beta1^t), the denominator of an element that never had a gradient, would count as zero
    if (eps > 0 && eps * (1.0 - beta1) < 1.17549435082228751e-38)
        return fail(QLORA_ERR_ARG, "eps must be 0, or eps (1 - beta1) at least 2^-126");
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
