// embedding.cuh -- rows of a packed or plain embedding table for a batch of token ids, and
// the gradient of a plain table from the tokens sorted by id.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"
#include "quant_kernels.cuh"
#include "scale_src.cuh"

namespace qlora {
namespace emb {

// Token ids: int32 or int64 on the device.
struct Ids {
    const void *ptr;
    int is64;
};
// (Kernels here start before the preceding one has ended, so what that one may have written is read
// through L2, not through the read-only path.)
__device__ __forceinline__ int64_t id_at(const Ids &ids, int64_t t) {
    return ids.is64 ? __ldcg(reinterpret_cast<const long long *>(ids.ptr) + t)
                    : int64_t(__ldcg(reinterpret_cast<const int *>(ids.ptr) + t));
}
__device__ __forceinline__ void report_bad_id() { atomicExch(&g_device_error, kDeviceErrIndex); }

// ------------------------------------------------------------------ lookup
// y[t, :] = round(scale * w'[id_t, :]), w' the table's float32 values (4-bit: fp32(c[code] s_b);
// Q8_0: q d; plain: the element), the product rounded to float32 and then to the output type.
enum { kTableNf4 = 0, kTableQ8 = 1, kTableBf16 = 2, kTableF32 = 3 };

struct FwdArgs {
    const void *table;     // codes, int8 codes or elements
    ScaleSrc sc;           // 4-bit
    const uint16_t *d8;    // Q8_0
    Ids ids;
    void *out;
    int64_t T, V, H;
    float scale;
    int seg_shift;         // log2 of the row segments of kRun elements that a CTA takes (at most its warps)
    float level[16];
};
constexpr int kFwdThreads = 256;
constexpr int kFwdWarps = kFwdThreads / 32;
constexpr int kUnroll = 4;
constexpr int kRun = 256 * kUnroll;   // elements of a row a warp takes: 8 per lane and step

// scale words of the 64-weight run b64, as scale_load reads them
__device__ __forceinline__ void scale_words(const ScaleSrc &s, int64_t b64, uint32_t &a, float &d) {
    const int64_t b = b64 >> s.blk_shift;
    if (s.dq) {
        a = __ldcg(s.scales + b);
        d = __ldcg(s.scales2 + (b >> 8));
    } else {
        a = __ldcg(reinterpret_cast<const uint32_t *>(s.scales) + b);
        d = 1.f;
    }
}

// 32-bit words of 8 elements of a table
template <int kTable>
constexpr int kWordsOf = kTable == kTableNf4 ? 1 : kTable == kTableQ8 ? 2 : kTable == kTableBf16 ? 4 : 8;
__device__ __forceinline__ float level_at(const float *levels, uint32_t byte_offset) {
    return *reinterpret_cast<const float *>(reinterpret_cast<const char *>(levels) + byte_offset);
}

// A warp takes one segment of one token's row: its id, then every code and scale load of the
// segment at once, 8 elements per lane and step, so that a bf16 output is one 16-byte store.
// CTAs: x over tokens, y over groups of 2^seg_shift segments.
template <int kTable, bool kOutBf16>
__global__ void __launch_bounds__(kFwdThreads) embed_fwd_kernel(const FwdArgs a) {
    __shared__ float s_lv[16];
    if (kTable == kTableNf4) {
        float lv = 0.f;
#pragma unroll
        for (int l = 0; l < 16; ++l)
            if ((threadIdx.x & 15) == l) lv = a.level[l];
        if (threadIdx.x < 16) s_lv[threadIdx.x] = lv;
        __syncthreads();
    }
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = int64_t(blockIdx.x) * (kFwdWarps >> a.seg_shift) + (warp >> a.seg_shift);
    const int64_t e0 = ((int64_t(blockIdx.y) << a.seg_shift) + (warp & ((1 << a.seg_shift) - 1))) * kRun + lane * 8;
    if (t >= a.T) return;
    const int64_t id = id_at(a.ids, t);
    const bool ok = id >= 0 && id < a.V;
    if (!ok && lane == 0) report_bad_id();
    const int64_t row = ok ? id * a.H : 0;

    uint32_t raw[kUnroll][kWordsOf<kTable>];
    uint32_t sa[kUnroll];
    float sd[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t e = e0 + u * 256;
        if (e >= a.H || !ok) continue;
        const int64_t at = row + e;
        if (kTable == kTableNf4) {
            raw[u][0] = __ldcg(reinterpret_cast<const uint32_t *>(a.table) + (at >> 3));
            scale_words(a.sc, at >> 6, sa[u], sd[u]);
        } else if (kTable == kTableQ8) {
            const uint2 q = __ldcg(reinterpret_cast<const uint2 *>(a.table) + (at >> 3));
            raw[u][0] = q.x;
            raw[u][1 % kWordsOf<kTable>] = q.y;
            sa[u] = __ldcg(a.d8 + (at >> 5));
        } else {
#pragma unroll
            for (int h = 0; h < kWordsOf<kTable> / 4; ++h) {
                const uint4 x = __ldcg(reinterpret_cast<const uint4 *>(static_cast<const char *>(a.table) + at * (kTable == kTableBf16 ? 2 : 4)) + h);
                raw[u][(4 * h) % kWordsOf<kTable>] = x.x, raw[u][(4 * h + 1) % kWordsOf<kTable>] = x.y;
                raw[u][(4 * h + 2) % kWordsOf<kTable>] = x.z, raw[u][(4 * h + 3) % kWordsOf<kTable>] = x.w;
            }
        }
    }
    const uint64_t scale = pack2(a.scale, a.scale);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t e = e0 + u * 256;
        if (e >= a.H) break;
        uint64_t w[4] = {0, 0, 0, 0};              // pairs of elements
        if (ok) {
            if (kTable == kTableNf4) {
                // byte offsets 4 c into the level table, four codes at a time; level(c) of two neighbours
                const float f = scale_of(a.sc, sa[u], sd[u]);
                const uint32_t lo = (raw[u][0] << 2) & 0x3C3C3C3Cu, hi = (raw[u][0] >> 2) & 0x3C3C3C3Cu;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = mul2(pack2(level_at(s_lv, __byte_perm(lo, 0u, 0x4440u + j)), level_at(s_lv, __byte_perm(hi, 0u, 0x4440u + j))),
                                pack2(f, f));
            } else if (kTable == kTableQ8) {
                const float f = __half2float(__ushort_as_half(static_cast<unsigned short>(sa[u])));
                const uint64_t magic = pack2(-8388736.f, -8388736.f);   // -(2^23 + 128)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t b = raw[u][(j / 2) % kWordsOf<kTable>] ^ 0x80808080u;
                    w[j] = mul2(add2(pack2(__uint_as_float(__byte_perm(b, 0x4B000000u, 0x7650 + 2 * (j & 1))),
                                           __uint_as_float(__byte_perm(b, 0x4B000000u, 0x7651 + 2 * (j & 1)))), magic), pack2(f, f));
                }
            } else if (kTable == kTableBf16) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t x = raw[u][j % kWordsOf<kTable>];
                    w[j] = pack2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = pack2(__uint_as_float(raw[u][(2 * j) % kWordsOf<kTable>]), __uint_as_float(raw[u][(2 * j + 1) % kWordsOf<kTable>]));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = mul2(w[j], scale);
        }
        float y[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) unpack2(w[j], y[2 * j], y[2 * j + 1]);
        const int64_t o = t * a.H + e;
        if (kOutBf16) {
            uint32_t b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 p = __floats2bfloat162_rn(y[2 * j], y[2 * j + 1]);
                b[j] = *reinterpret_cast<const uint32_t *>(&p);
            }
            reinterpret_cast<uint4 *>(a.out)[o >> 3] = make_uint4(b[0], b[1], b[2], b[3]);
        } else {
            float4 *dst = reinterpret_cast<float4 *>(a.out) + (o >> 2);
            dst[0] = make_float4(y[0], y[1], y[2], y[3]);
            dst[1] = make_float4(y[4], y[5], y[6], y[7]);
        }
    }
}

// ------------------------------------------------------------------ gradient
// dE[v, :] (+)= scale * sum over the tokens t with id_t = v of dY[t, :], in up to four launches:
//   sort    the tokens by id (stable);
//   reduce  equal runs of `chunk` sorted tokens each: an id that lies wholly in a chunk is summed
//           and written, one that crosses a border leaves a partial sum per chunk;
//   join    adds the partial sums of each such id in order and writes its row;
//   zero    (unless the gradient is added) zeroes the rows that no token names.
// Every sum is float32, in an order fixed by the ids alone: results repeat bit for bit.
// The last three overlap: each starts once the one before it has started (programmatic dependent
// launch).  `zero` needs the sort only, so its writes, nearly all of the time when the table is large, run
// beside the reduction; its last CTA waits for the join, so that its completion means the whole call's.
constexpr int kSortCtas = 8;            // one cluster sorts: bins and counts meet in shared memory
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxBits = 9;             // bits of a digit: 512 bins
constexpr int kMaxBins = 1 << kMaxBits;
constexpr int kSortBatch = 4;           // rounds of 32 tokens whose loads a warp has in flight
constexpr int kSortSmem = (kSortWarps * kMaxBins + 2 * kMaxBins + 64) * 4;

struct GradArgs {
    Ids ids;
    int64_t T, V, H, pad;
    uint32_t *key[2], *pos[2];   // ping-pong buffers of T each; the sorted list ends in [passes & 1]
    int bits, passes;            // bits of a digit, digits
    const void *dY;
    int dy_bf16;
    void *dE;
    int de_bf16, accumulate;
    float scale;
    int chunk;                   // sorted tokens per chunk of the reduction
    int64_t nchunks;
    uint32_t *named;             // bit v: a token names row v (when the gradient is written, not added)
    int zero_rows;               // rows a CTA zeroes
    float *part;                 // [nchunks][2][H] partial sums: of the run at a chunk's first token, of its last run
};

// key of token t: its id, or V (sorted last, in no row) for the padding id and ids outside the table
__device__ __forceinline__ uint32_t key_of(const GradArgs &a, int64_t t) {
    const int64_t id = id_at(a.ids, t);
    if (id < 0 || id >= a.V) {
        report_bad_id();
        return static_cast<uint32_t>(a.V);
    }
    return static_cast<uint32_t>(id == a.pad ? a.V : id);
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// barrier of the cluster's CTAs; also orders their global and shared memory
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t ld_cluster(const uint32_t *p, uint32_t rank) {
    uint32_t addr, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// Radix sort by the cluster of blocks 0 .. kSortCtas - 1, least significant digit first.  Tokens are
// dealt in order to CTAs, warps and rounds of 32, so a token's place among equal digits is the count
// in lower CTAs, in lower warps, in its warp's earlier rounds and in its lower lanes: stable without
// atomics.
__device__ void sort_tokens(const GradArgs &a, uint32_t *smem) {
    uint32_t *hist = smem;                               // [warp][bin]
    uint32_t *total = hist + kSortWarps * kMaxBins;      // [bin] of this CTA
    uint32_t *first = total + kMaxBins;                  // [bin] first place of this CTA's tokens
    uint32_t *wsum = first + kMaxBins;                   // [warp] sums of the scan
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const int bins = 1 << a.bits;
    const int64_t per_warp = (a.T + int64_t(kSortCtas) * kSortThreads - 1) / (int64_t(kSortCtas) * kSortThreads) * 32;
    const int64_t i_lo = min((int64_t(rank) * kSortWarps + warp) * per_warp, a.T);
    const int64_t i_hi = min(i_lo + per_warp, a.T);
    uint32_t *my = hist + warp * kMaxBins;
    for (int pass = 0; pass < a.passes; ++pass) {
        const uint32_t *src_k = a.key[pass & 1], *src_p = a.pos[pass & 1];
        uint32_t *dst_k = a.key[(pass + 1) & 1], *dst_p = a.pos[(pass + 1) & 1];
        const int shift = pass * a.bits;
        for (int b = lane; b < bins; b += 32) my[b] = 0;
        __syncwarp();
        for (int64_t i = i_lo; i < i_hi; i += 32 * kSortBatch) {
            uint32_t k[kSortBatch];
#pragma unroll
            for (int u = 0; u < kSortBatch; ++u) {
                const int64_t t = i + 32 * u + lane;
                k[u] = t < i_hi ? (pass ? __ldcg(src_k + t) : key_of(a, t)) : 0u;
            }
#pragma unroll
            for (int u = 0; u < kSortBatch; ++u) {
                if (i + 32 * u >= i_hi) break;
                const bool in = i + 32 * u + lane < i_hi;
                if (pass == 0 && !a.accumulate && in && k[u] < a.V) atomicOr(a.named + (k[u] >> 5), 1u << (k[u] & 31));
                const uint32_t d = in ? (k[u] >> shift) & (bins - 1) : uint32_t(kMaxBins);   // idle lanes match none
                const uint32_t same = __match_any_sync(0xffffffffu, d);
                if (in && (same & ((1u << lane) - 1u)) == 0) my[d] += __popc(same);
                __syncwarp();
            }
        }
        __syncthreads();
        // per bin: counts of lower warps, and this CTA's total
        if (tid < bins) {
            uint32_t sum = 0, n[kSortWarps];
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) n[w] = hist[w * kMaxBins + tid];
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) {
                hist[w * kMaxBins + tid] = sum;
                sum += n[w];
            }
            total[tid] = sum;
        }
        cluster_barrier();
        uint32_t below = 0, all = 0;
        if (tid < bins) {
#pragma unroll
            for (uint32_t r = 0; r < kSortCtas; ++r) {
                const uint32_t n = ld_cluster(total + tid, r);
                all += n;
                if (r < rank) below += n;
            }
        }
        // exclusive scan of `all` over the bins (the first bins / 32 warps hold them)
        uint32_t incl = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t n = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += n;
        }
        if (lane == 31) wsum[warp] = incl;
        __syncthreads();
        if (tid < bins) {
            uint32_t base = incl - all + below;
            for (int w = 0; w < warp; ++w) base += wsum[w];
            first[tid] = base;
        }
        __syncthreads();
        for (int64_t i = i_lo; i < i_hi; i += 32 * kSortBatch) {
            uint32_t k[kSortBatch], p[kSortBatch];
#pragma unroll
            for (int u = 0; u < kSortBatch; ++u) {
                const int64_t t = i + 32 * u + lane;
                k[u] = t < i_hi ? (pass ? __ldcg(src_k + t) : key_of(a, t)) : 0u;
                p[u] = t < i_hi && pass ? __ldcg(src_p + t) : static_cast<uint32_t>(t);
            }
#pragma unroll
            for (int u = 0; u < kSortBatch; ++u) {
                if (i + 32 * u >= i_hi) break;
                const bool in = i + 32 * u + lane < i_hi;
                const uint32_t d = in ? (k[u] >> shift) & (bins - 1) : uint32_t(kMaxBins);
                const uint32_t same = __match_any_sync(0xffffffffu, d);
                const uint32_t lower = same & ((1u << lane) - 1u);
                uint32_t at = 0;
                if (in) at = first[d] + my[d] + __popc(lower);
                __syncwarp();
                if (in && lower == 0) my[d] += __popc(same);
                __syncwarp();
                if (in) {
                    __stcg(dst_k + at, k[u]);
                    __stcg(dst_p + at, p[u]);
                }
            }
        }
        cluster_barrier();   // the next pass reads what every CTA wrote; total is free again
    }
}

__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads) embed_sort_kernel(const GradArgs a) {
    extern __shared__ uint32_t sort_smem[];
    pdl_launch_dependents();
    pdl_wait();
    if (!a.accumulate) {        // which rows are named; the marks are set by the sort's first pass
        for (int64_t i = int64_t(cluster_rank()) * kSortThreads + threadIdx.x; i < (a.V + 31) / 32; i += kSortCtas * kSortThreads)
            __stcg(a.named + i, 0u);
        cluster_barrier();
    }
    sort_tokens(a, sort_smem);
}

// Zero: a CTA of 256 threads for about 16 KB of rows, in the order of the table.  (A grid of two CTAs per SM
// that strides over the rows wrote 6.0 TB/s, this order 7.2: what is written at any time lies close together.)
constexpr int kZeroThreads = 256;
__global__ void __launch_bounds__(kZeroThreads) embed_zero_kernel(const GradArgs a) {
    pdl_launch_dependents();
    if (a.T == 0) pdl_wait();   // otherwise the reduction has let this kernel start, after its own wait for the sort
    const int64_t row_words = a.H * (a.de_bf16 ? 2 : 4) / 16;
    const int64_t end = min((blockIdx.x + int64_t(1)) * a.zero_rows, a.V);
    if (row_words >= kZeroThreads) {
        for (int64_t r = blockIdx.x * int64_t(a.zero_rows); r < end; ++r) {
            if (a.T > 0 && ((__ldcg(a.named + (r >> 5)) >> (r & 31)) & 1u)) continue;
            uint4 *dst = static_cast<uint4 *>(a.dE) + r * row_words;
#pragma unroll 4
            for (int64_t i = threadIdx.x; i < row_words; i += kZeroThreads) dst[i] = make_uint4(0, 0, 0, 0);
        }
    } else {
        // short rows: the CTA's words as one run (at most 1024 + 255 rows' words, 32-bit)
        const int64_t r0 = blockIdx.x * int64_t(a.zero_rows);
        const uint32_t words = static_cast<uint32_t>((end - r0) * row_words), rw = static_cast<uint32_t>(row_words);
        uint4 *dst = static_cast<uint4 *>(a.dE) + r0 * row_words;
        for (uint32_t i = threadIdx.x; i < words; i += kZeroThreads) {
            const int64_t r = r0 + i / rw;
            if (a.T > 0 && ((__ldcg(a.named + (r >> 5)) >> (r & 31)) & 1u)) continue;
            dst[i] = make_uint4(0, 0, 0, 0);
        }
    }
    if (blockIdx.x == gridDim.x - 1) pdl_wait();
}

// kN (4 or 8) elements of a row of dY or dE as loaded, and as floats
template <bool kBf16, int kN>
struct Raw {
    static constexpr int kWords = kN / (kBf16 ? 2 : 1);
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const void *base, int64_t o) {
        const char *p = static_cast<const char *>(base) + o * (kBf16 ? 2 : 4);
        if (kWords == 2) {
            const uint2 x = __ldcg(reinterpret_cast<const uint2 *>(p));
            w[0] = x.x, w[1] = x.y;
        } else {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 x = __ldcg(reinterpret_cast<const uint4 *>(p) + i);
                w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
            }
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ float at(int i) const {
        if (!kBf16) return __uint_as_float(w[i % kWords]);
        return __uint_as_float((i & 1) ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
};
// dE[row, c .. c + kN) = old + scale * s, one rounding (old: zeros when the gradient is written)
template <bool kDeBf16, int kN>
__device__ __forceinline__ void write_row(const GradArgs &a, uint32_t row, int64_t c, const float *s, const Raw<kDeBf16, kN> &old) {
    const int64_t o = int64_t(row) * a.H + c;
    float v[kN];
#pragma unroll
    for (int j = 0; j < kN; ++j) v[j] = fmaf(a.scale, s[j], old.at(j));
    if (kDeBf16) {
        uint2 *dst = reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.dE) + o);
#pragma unroll
        for (int h = 0; h < kN / 4; ++h) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(v[4 * h], v[4 * h + 1]);
            const __nv_bfloat162 hi = __floats2bfloat162_rn(v[4 * h + 2], v[4 * h + 3]);
            dst[h] = make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
        }
    } else {
        float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(a.dE) + o);
#pragma unroll
        for (int h = 0; h < kN / 4; ++h) dst[h] = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
    }
}

// Reduce: block (chunk, column tile); a thread owns 8 columns and walks the chunk's tokens in order,
// kBatch rows of dY in flight, with the old rows of dE that they will be added to.
constexpr int kRedThreads = 128;
constexpr int kRedCols = kRedThreads * 8;
constexpr int kMaxChunk = 64;
constexpr int kBatch = 4;
template <bool kDyBf16, bool kDeBf16, bool kAdd>
__global__ void __launch_bounds__(kRedThreads) embed_reduce_kernel(const GradArgs a) {
    __shared__ uint32_t s_id[kMaxChunk + 2], s_pos[kMaxChunk];   // s_id[0]: the token before the chunk; last + 1: after it
    pdl_wait();                 // before the release: `zero` may rely on the sort
    pdl_launch_dependents();
    const uint32_t *ids = a.key[a.passes & 1], *pos = a.pos[a.passes & 1];
    const int64_t ch = blockIdx.x;
    const int64_t i0 = ch * a.chunk;
    const int n = static_cast<int>(min(int64_t(a.chunk), a.T - i0));
    constexpr uint32_t kNone = 0xFFFFFFFFu;
    for (int i = threadIdx.x; i < n + 2; i += kRedThreads) {
        const int64_t t = i0 + i - 1;
        s_id[i] = t >= 0 && t < a.T ? __ldcg(ids + t) : kNone;
        if (i >= 1 && i <= n) s_pos[i - 1] = __ldcg(pos + t);
    }
    __syncthreads();
    const int64_t c = int64_t(blockIdx.y) * kRedCols + threadIdx.x * 8;
    const uint32_t V = static_cast<uint32_t>(a.V), first = s_id[1], before = s_id[0];
    if (c >= a.H || first >= V) return;              // keys ascend: V at the first token means V throughout
    float acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    for (int i = 0; i < n; i += kBatch) {
        Raw<kDyBf16, 8> r[kBatch];
        Raw<kDeBf16, 8> old[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            old[u].zero();
            if (i + u >= n) continue;
            const uint32_t id = s_id[i + u + 1];
            if (id >= V) continue;
            r[u].load(a.dY, int64_t(s_pos[i + u]) * a.H + c);
            if (kAdd && s_id[i + u + 2] != id && !(id == first && before == id)) old[u].load(a.dE, int64_t(id) * a.H + c);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (i + u >= n) break;
            const uint32_t id = s_id[i + u + 1], next = s_id[i + u + 2];
            if (id >= V) break;
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += r[u].at(j);
            if (next == id && i + u + 1 < n) continue;
            // the run ends in this chunk, or the chunk ends in it
            if (next == id || (id == first && before == id)) {
                float4 *dst = reinterpret_cast<float4 *>(a.part + (2 * ch + (id == first ? 0 : 1)) * a.H + c);
                dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
                dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
            } else {
                write_row<kDeBf16, 8>(a, id, c, acc, old[u]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] = 0.f;
        }
    }
}

// Join: an id whose tokens cross a chunk border belongs to the chunk where it starts; its row is that
// chunk's partial sum and those of the next chunks' first runs, as far as they have the same id.  A warp
// takes one chunk and 512 columns; an id with more than kLongJoin partial sums is added by all eight warps,
// each over an equal part of the list, and the eight sums in order.
constexpr int kJoinWarps = 8;
constexpr int kJoinCols = 512;         // four runs of 128
constexpr int kLongJoin = 32;
__device__ __forceinline__ void add4(float4 &s, const float4 x) {
    s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
}
__device__ __forceinline__ float4 load_part(const GradArgs &a, int64_t slot, int64_t c) {
    return __ldcg(reinterpret_cast<const float4 *>(a.part + slot * a.H + c));
}
// sum of the first-run partials of chunks [lo, hi), columns c .. c + 3, on top of s
__device__ __forceinline__ float4 sum_firsts(const GradArgs &a, float4 s, int64_t lo, int64_t hi, int64_t c) {
    for (; lo + 8 <= hi; lo += 8) {
        float4 x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) x[u] = load_part(a, 2 * (lo + u), c);
#pragma unroll
        for (int u = 0; u < 8; ++u) add4(s, x[u]);
    }
    for (; lo < hi; ++lo) add4(s, load_part(a, 2 * lo, c));
    return s;
}
// one past the last chunk that starts with id, given that chunk lo does: 32 chunks at a time over the
// whole warp, the next 32 first (few ids go further), then 32 places spread over what is left
__device__ __forceinline__ int64_t end_of_id(const GradArgs &a, const uint32_t *ids, uint32_t id, int64_t lo, int lane) {
    int64_t hi = a.nchunks, stride = 1;
    while (lo + 1 < hi) {                      // chunk lo starts with id, chunk hi does not (or is the end)
        const int64_t k = lo + (lane + 1) * stride;
        const bool same = k < hi && __ldcg(ids + k * a.chunk) == id;
        const int n = __popc(__ballot_sync(0xffffffffu, same));      // sorted: the first n places hold id
        lo += n * stride;
        hi = min(hi, n < 32 ? lo + stride : hi);
        stride = max(int64_t(1), (hi - lo + 31) / 32);
    }
    return lo + 1;
}
template <bool kDeBf16>
__global__ void __launch_bounds__(kJoinWarps * 32) embed_join_kernel(const GradArgs a) {
    __shared__ int64_t s_end[kJoinWarps];
    __shared__ uint32_t s_id[kJoinWarps], s_slot[kJoinWarps];
    __shared__ float4 s_part[kJoinWarps][32];
    pdl_launch_dependents();
    pdl_wait();
    const uint32_t *ids = a.key[a.passes & 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c = int64_t(blockIdx.y) * kJoinCols + lane * 4;
    const int64_t ch = int64_t(blockIdx.x) * kJoinWarps + warp;
    int64_t end = 0;                     // one past the last chunk of this warp's id; 0: none
    uint32_t id = 0, slot = 0;
    if (ch + 1 < a.nchunks) {
        const int64_t i0 = ch * a.chunk;
        id = __ldcg(ids + i0 + a.chunk - 1);
        const uint32_t after = __ldcg(ids + i0 + a.chunk), first = __ldcg(ids + i0);
        const uint32_t before = ch > 0 ? __ldcg(ids + i0 - 1) : 0xFFFFFFFFu;
        // first == id: one id throughout the chunk; if it also ends the chunk before, that one (or one before) owns it
        if (id < a.V && after == id && !(first == id && before == id)) {
            slot = first == id ? 0 : 1;
            end = end_of_id(a, ids, id, ch + 1, lane);
        }
    }
    if (end && end - ch <= kLongJoin) {
#pragma unroll
        for (int q = 0; q < kJoinCols / 128; ++q) {
            const int64_t cq = c + 128 * q;
            if (cq >= a.H) break;
            Raw<kDeBf16, 4> old;
            old.zero();
            if (a.accumulate) old.load(a.dE, int64_t(id) * a.H + cq);
            const float4 s = sum_firsts(a, load_part(a, 2 * ch + slot, cq), ch + 1, end, cq);
            write_row<kDeBf16, 4>(a, id, cq, reinterpret_cast<const float *>(&s), old);
        }
    }
    if (lane == 0) {
        s_end[warp] = end && end - ch > kLongJoin ? end : 0;
        s_id[warp] = id;
        s_slot[warp] = slot;
    }
    __syncthreads();
    for (int w = 0; w < kJoinWarps; ++w) {
        if (!s_end[w]) continue;                                  // the same for the whole block
        const int64_t lo = ch - warp + w + 1, n = s_end[w] - lo;  // first-run partials of chunks [lo, lo + n)
        for (int64_t cq = c; cq < c - lane * 4 + kJoinCols && cq - lane * 4 < a.H; cq += 128) {
            Raw<kDeBf16, 4> old;
            old.zero();
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            if (cq < a.H) {
                if (warp == 0) s = load_part(a, 2 * (lo - 1) + s_slot[w], cq);
                if (warp == 0 && a.accumulate) old.load(a.dE, int64_t(s_id[w]) * a.H + cq);
                s = sum_firsts(a, s, lo + n * warp / kJoinWarps, lo + n * (warp + 1) / kJoinWarps, cq);
            }
            s_part[warp][lane] = s;
            __syncthreads();
            if (warp == 0 && cq < a.H) {
#pragma unroll
                for (int i = 1; i < kJoinWarps; ++i) add4(s, s_part[i][lane]);
                write_row<kDeBf16, 4>(a, s_id[w], cq, reinterpret_cast<const float *>(&s), old);
            }
            __syncthreads();
        }
    }
}

}  // namespace emb
}  // namespace qlora
