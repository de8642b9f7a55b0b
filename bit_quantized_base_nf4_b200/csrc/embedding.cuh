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
__device__ __forceinline__ int64_t id_at(const Ids &ids, int64_t t) {
    return ids.is64 ? __ldg(reinterpret_cast<const long long *>(ids.ptr) + t)
                    : int64_t(__ldg(reinterpret_cast<const int *>(ids.ptr) + t));
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
    int segs;              // row segments of kRun elements
    float level[16];
};
constexpr int kFwdThreads = 256;
constexpr int kUnroll = 4;
constexpr int kRun = 256 * kUnroll;   // elements of a row a warp takes: 8 per lane and step

// A warp takes one segment of one token's row: its id, then every code and scale load of the
// segment at once, 8 elements per lane and step, so that a bf16 output is one 16-byte store.
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
    const int lane = threadIdx.x & 31;
    const int64_t task = int64_t(blockIdx.x) * (kFwdThreads / 32) + (threadIdx.x >> 5);
    if (task >= a.T * a.segs) return;
    const int64_t t = task / a.segs;
    const int64_t e0 = (task - t * a.segs) * kRun + lane * 8;
    const int64_t id = id_at(a.ids, t);
    const bool ok = id >= 0 && id < a.V;
    if (!ok && lane == 0) report_bad_id();
    const int64_t row = ok ? id * a.H : 0;

    uint4 raw[kUnroll], raw2[kTable == kTableF32 ? kUnroll : 1];
    uint32_t sa[kUnroll];
    float sd[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t e = e0 + u * 256;
        raw[u] = make_uint4(0, 0, 0, 0);
        sa[u] = 0;
        sd[u] = 0.f;
        if (kTable == kTableF32) raw2[u] = make_uint4(0, 0, 0, 0);
        if (e < a.H && ok) {
            if (kTable == kTableNf4) {
                raw[u].x = __ldg(reinterpret_cast<const uint32_t *>(a.table) + ((row + e) >> 3));
                scale_load(a.sc, (row + e) >> 6, sa[u], sd[u]);
            } else if (kTable == kTableQ8) {
                const uint2 q = __ldg(reinterpret_cast<const uint2 *>(a.table) + ((row + e) >> 3));
                raw[u].x = q.x;
                raw[u].y = q.y;
                sa[u] = __ldg(a.d8 + ((row + e) >> 5));
            } else if (kTable == kTableBf16) {
                raw[u] = __ldg(reinterpret_cast<const uint4 *>(a.table) + ((row + e) >> 3));
            } else {
                raw[u] = __ldg(reinterpret_cast<const uint4 *>(a.table) + ((row + e) >> 2));
                raw2[u] = __ldg(reinterpret_cast<const uint4 *>(a.table) + ((row + e) >> 2) + 1);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t e = e0 + u * 256;
        if (e >= a.H) break;
        float w[8];
        if (kTable == kTableNf4) {
            const float s = scale_of(a.sc, sa[u], sd[u]);
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = __fmul_rn(s_lv[(raw[u].x >> (4 * j)) & 15u], s);
        } else if (kTable == kTableQ8) {
            const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(sa[u])));
            const float magic = 8388736.f;   // 2^23 + 128
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t b = (j < 4 ? raw[u].x : raw[u].y) ^ 0x80808080u;
                w[j] = __fmul_rn(__uint_as_float(__byte_perm(b, 0x4B000000u, 0x7650 + (j & 3))) - magic, s);
            }
        } else if (kTable == kTableBf16) {
            const uint32_t x[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[2 * j] = __uint_as_float(x[j] << 16);
                w[2 * j + 1] = __uint_as_float(x[j] & 0xFFFF0000u);
            }
        } else {
            const uint32_t x[8] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w, raw2[u].x, raw2[u].y, raw2[u].z, raw2[u].w};
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = __uint_as_float(x[j]);
        }
        if (ok) {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = __fmul_rn(w[j], a.scale);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 0.f;
        }
        const int64_t o = t * a.H + e;
        if (kOutBf16) {
            uint32_t b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 p = __floats2bfloat162_rn(w[2 * j], w[2 * j + 1]);
                b[j] = *reinterpret_cast<const uint32_t *>(&p);
            }
            reinterpret_cast<uint4 *>(a.out)[o >> 3] = make_uint4(b[0], b[1], b[2], b[3]);
        } else {
            float4 *dst = reinterpret_cast<float4 *>(a.out) + (o >> 2);
            dst[0] = make_float4(w[0], w[1], w[2], w[3]);
            dst[1] = make_float4(w[4], w[5], w[6], w[7]);
        }
    }
}

// ------------------------------------------------------------------ gradient
// dE[v, :] (+)= scale * sum over the tokens t with id_t = v of dY[t, :], in three launches:
//   sort    the tokens by id (stable), and zero the rows that no token names;
//   reduce  equal runs of `chunk` sorted tokens each: an id that lies wholly in a chunk is summed
//           and written, one that crosses a border leaves a partial sum per chunk;
//   join    adds the partial sums of each such id in order and writes its row.
// Every sum is float32, in an order fixed by the ids alone: results repeat bit for bit.
constexpr int kSortCtas = 8;            // one cluster sorts: bins and counts meet in shared memory
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxBits = 9;             // bits of a digit: 512 bins
constexpr int kMaxBins = 1 << kMaxBits;
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
        for (int64_t i = i_lo; i < i_hi; i += 32) {
            const bool in = i + lane < i_hi;
            const uint32_t k = in ? (pass ? __ldcg(src_k + i + lane) : key_of(a, i + lane)) : 0u;
            const uint32_t d = in ? (k >> shift) & (bins - 1) : uint32_t(kMaxBins);   // idle lanes match none
            const uint32_t same = __match_any_sync(0xffffffffu, d);
            if (in && (same & ((1u << lane) - 1u)) == 0) my[d] += __popc(same);
            __syncwarp();
        }
        __syncthreads();
        // per bin: counts of lower warps, and this CTA's total
        if (tid < bins) {
            uint32_t sum = 0;
#pragma unroll 8
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t n = hist[w * kMaxBins + tid];
                hist[w * kMaxBins + tid] = sum;
                sum += n;
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
        for (int64_t i = i_lo; i < i_hi; i += 32) {
            const bool in = i + lane < i_hi;
            uint32_t k = 0, p = 0;
            if (in) {
                k = pass ? __ldcg(src_k + i + lane) : key_of(a, i + lane);
                p = pass ? __ldcg(src_p + i + lane) : static_cast<uint32_t>(i + lane);
            }
            const uint32_t d = in ? (k >> shift) & (bins - 1) : uint32_t(kMaxBins);
            const uint32_t same = __match_any_sync(0xffffffffu, d);
            const uint32_t lower = same & ((1u << lane) - 1u);
            uint32_t at = 0;
            if (in) at = first[d] + my[d] + __popc(lower);
            __syncwarp();
            if (in && lower == 0) my[d] += __popc(same);
            __syncwarp();
            if (in) {
                __stcg(dst_k + at, k);
                __stcg(dst_p + at, p);
            }
        }
        cluster_barrier();   // the next pass reads what every CTA wrote; total is free again
    }
}

// Zeroes the rows of [lo, hi) that no token names: the CTA marks the named ones in a bitmap of at
// most kMaskRows rows at a time, reading every id (from L2) for itself, so that it need not wait for the sort.
constexpr int kMaskRows = kSortWarps * kMaxBins * 32;
__device__ void zero_rows(const GradArgs &a, uint32_t *mask, int64_t lo, int64_t hi) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t row_bytes = a.H * (a.de_bf16 ? 2 : 4);
    for (; lo < hi; lo += kMaskRows) {
        const int64_t end = min(lo + int64_t(kMaskRows), hi);
        const int words = static_cast<int>((end - lo + 31) / 32);
        __syncthreads();
        for (int i = tid; i < words; i += kSortThreads) mask[i] = 0;
        __syncthreads();
        for (int64_t t = tid; t < a.T; t += kSortThreads) {
            const int64_t id = id_at(a.ids, t);
            if (id >= lo && id < end && id != a.pad) atomicOr(mask + ((id - lo) >> 5), 1u << ((id - lo) & 31));
        }
        __syncthreads();
        for (int64_t r = lo + warp; r < end; r += kSortWarps) {
            if ((mask[(r - lo) >> 5] >> ((r - lo) & 31)) & 1u) continue;
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<char *>(a.dE) + r * row_bytes);
            for (int64_t i = lane; i < row_bytes / 16; i += 32) dst[i] = make_uint4(0, 0, 0, 0);
        }
    }
}

// Block roles: the first cluster sorts, the others zero.
__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads) embed_sort_kernel(const GradArgs a) {
    extern __shared__ uint32_t sort_smem[];
    if (blockIdx.x < kSortCtas) {
        if (a.T > 0) sort_tokens(a, sort_smem);
    } else {
        const int64_t n = gridDim.x - kSortCtas, i = blockIdx.x - kSortCtas;
        zero_rows(a, sort_smem, a.V * i / n, a.V * (i + 1) / n);
    }
}

// 8 columns of dY row p from column c on, added to acc
__device__ __forceinline__ void load_dy(const GradArgs &a, uint32_t p, int64_t c, uint4 *r) {
    const int64_t o = int64_t(p) * a.H + c;
    if (a.dy_bf16) {
        r[0] = __ldg(reinterpret_cast<const uint4 *>(a.dY) + (o >> 3));
    } else {
        r[0] = __ldg(reinterpret_cast<const uint4 *>(a.dY) + (o >> 2));
        r[1] = __ldg(reinterpret_cast<const uint4 *>(a.dY) + (o >> 2) + 1);
    }
}
__device__ __forceinline__ void add_dy(const GradArgs &a, const uint4 *r, float *acc) {
    const uint32_t x[4] = {r[0].x, r[0].y, r[0].z, r[0].w};
    if (a.dy_bf16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            acc[2 * j] += __uint_as_float(x[j] << 16);
            acc[2 * j + 1] += __uint_as_float(x[j] & 0xFFFF0000u);
        }
    } else {
        const uint32_t y[4] = {r[1].x, r[1].y, r[1].z, r[1].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            acc[j] += __uint_as_float(x[j]);
            acc[4 + j] += __uint_as_float(y[j]);
        }
    }
}
// dE[row, c .. c + kN) = (the old values +) scale * s, one rounding; kN = 4 or 8
template <int kN>
__device__ __forceinline__ void write_row(const GradArgs &a, uint32_t row, int64_t c, const float *s) {
    const int64_t o = int64_t(row) * a.H + c;
    float v[kN];
    if (a.de_bf16) {
        uint2 *dst = reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.dE) + o);
#pragma unroll
        for (int h = 0; h < kN / 4; ++h) {
            uint2 old = make_uint2(0, 0);
            if (a.accumulate) old = dst[h];
            v[4 * h] = fmaf(a.scale, s[4 * h], __uint_as_float(old.x << 16));
            v[4 * h + 1] = fmaf(a.scale, s[4 * h + 1], __uint_as_float(old.x & 0xFFFF0000u));
            v[4 * h + 2] = fmaf(a.scale, s[4 * h + 2], __uint_as_float(old.y << 16));
            v[4 * h + 3] = fmaf(a.scale, s[4 * h + 3], __uint_as_float(old.y & 0xFFFF0000u));
            const __nv_bfloat162 lo = __floats2bfloat162_rn(v[4 * h], v[4 * h + 1]);
            const __nv_bfloat162 hi = __floats2bfloat162_rn(v[4 * h + 2], v[4 * h + 3]);
            dst[h] = make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
        }
    } else {
        float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(a.dE) + o);
#pragma unroll
        for (int h = 0; h < kN / 4; ++h) {
            float4 old = make_float4(0.f, 0.f, 0.f, 0.f);
            if (a.accumulate) old = dst[h];
            dst[h] = make_float4(fmaf(a.scale, s[4 * h], old.x), fmaf(a.scale, s[4 * h + 1], old.y),
                                 fmaf(a.scale, s[4 * h + 2], old.z), fmaf(a.scale, s[4 * h + 3], old.w));
        }
    }
}

// Reduce: block (chunk, column tile); a thread owns 8 columns and walks the chunk's tokens in order,
// eight rows in flight.
constexpr int kRedThreads = 128;
constexpr int kRedCols = kRedThreads * 8;
constexpr int kMaxChunk = 64;
__global__ void __launch_bounds__(kRedThreads) embed_reduce_kernel(const GradArgs a) {
    __shared__ uint32_t s_id[kMaxChunk + 2], s_pos[kMaxChunk];   // s_id[0]: the token before the chunk; last + 1: after it
    const uint32_t *ids = a.key[a.passes & 1], *pos = a.pos[a.passes & 1];
    const int64_t ch = blockIdx.x;
    const int64_t i0 = ch * a.chunk;
    const int n = static_cast<int>(min(int64_t(a.chunk), a.T - i0));
    constexpr uint32_t kNone = 0xFFFFFFFFu;
    for (int i = threadIdx.x; i < n + 2; i += kRedThreads) {
        const int64_t t = i0 + i - 1;
        s_id[i] = t >= 0 && t < a.T ? __ldg(ids + t) : kNone;
        if (i >= 1 && i <= n) s_pos[i - 1] = __ldg(pos + t);
    }
    __syncthreads();
    const int64_t c = int64_t(blockIdx.y) * kRedCols + threadIdx.x * 8;
    if (c >= a.H || s_id[1] >= a.V) return;         // keys ascend: V at the first token means V throughout
    float acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    bool from_first = true;                          // the current run starts at the chunk's first token
    for (int i = 0; i < n; i += 8) {
        uint4 r[8][2];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (i + u < n && s_id[i + u + 1] < a.V) load_dy(a, s_pos[i + u], c, r[u]);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (i + u >= n || s_id[i + u + 1] >= a.V) break;
            add_dy(a, r[u], acc);
            const uint32_t id = s_id[i + u + 1], next = s_id[i + u + 2];
            if (next == id && i + u + 1 < n) continue;
            // the run ends in this chunk, or the chunk ends in it
            if (next == id || (from_first && s_id[0] == id)) {
                float4 *dst = reinterpret_cast<float4 *>(a.part + (2 * ch + (from_first ? 0 : 1)) * a.H + c);
                dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
                dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
            } else {
                write_row<8>(a, id, c, acc);
            }
            from_first = false;
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] = 0.f;
        }
    }
}

// Join: an id whose tokens cross a chunk border belongs to the chunk where it starts; its row is that
// chunk's partial sum and those of the next chunks' first runs, as far as they have the same id.  A warp
// takes one chunk and 128 columns; an id with more than kLongJoin partial sums is added by all eight warps,
// each over an equal part of the list, and the eight sums in order.
constexpr int kJoinWarps = 8;
constexpr int kJoinCols = 128;
constexpr int kLongJoin = 32;
__device__ __forceinline__ void add4(float4 &s, const float4 x) {
    s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
}
// sum of the first-run partials of chunks [lo, hi), columns c .. c + 3, on top of s
__device__ __forceinline__ float4 sum_firsts(const GradArgs &a, float4 s, int64_t lo, int64_t hi, int64_t c) {
    for (; lo + 8 <= hi; lo += 8) {
        float4 x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) x[u] = __ldcg(reinterpret_cast<const float4 *>(a.part + 2 * (lo + u) * a.H + c));
#pragma unroll
        for (int u = 0; u < 8; ++u) add4(s, x[u]);
    }
    for (; lo < hi; ++lo) add4(s, __ldcg(reinterpret_cast<const float4 *>(a.part + 2 * lo * a.H + c)));
    return s;
}
__global__ void __launch_bounds__(kJoinWarps * 32) embed_join_kernel(const GradArgs a) {
    __shared__ int64_t s_end[kJoinWarps];
    __shared__ uint32_t s_id[kJoinWarps], s_slot[kJoinWarps];
    __shared__ float4 s_part[kJoinWarps][32];
    const uint32_t *ids = a.key[a.passes & 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c = int64_t(blockIdx.y) * kJoinCols + lane * 4;
    const int64_t ch = int64_t(blockIdx.x) * kJoinWarps + warp;
    int64_t end = 0;                     // one past the last chunk of this warp's id; 0: none
    uint32_t id = 0, slot = 0;
    if (ch + 1 < a.nchunks) {
        const int64_t i0 = ch * a.chunk;
        id = __ldg(ids + i0 + a.chunk - 1);
        if (id < a.V && __ldg(ids + i0 + a.chunk) == id) {
            const bool whole = __ldg(ids + i0) == id;             // one id throughout the chunk
            if (!(whole && ch > 0 && __ldg(ids + i0 - 1) == id)) {
                slot = whole ? 0 : 1;
                int64_t lo = ch + 1, hi = a.nchunks;              // chunk lo starts with id; find the first that does not
                while (hi - lo > 1) {
                    const int64_t mid = (lo + hi) / 2;
                    if (__ldg(ids + mid * a.chunk) == id) lo = mid;
                    else hi = mid;
                }
                end = lo + 1;
            }
        }
    }
    if (end && end - ch <= kLongJoin && c < a.H) {
        float4 s = __ldcg(reinterpret_cast<const float4 *>(a.part + (2 * ch + slot) * a.H + c));
        s = sum_firsts(a, s, ch + 1, end, c);
        write_row<4>(a, id, c, reinterpret_cast<const float *>(&s));
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
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < a.H) {
            if (warp == 0) s = __ldcg(reinterpret_cast<const float4 *>(a.part + (2 * (lo - 1) + s_slot[w]) * a.H + c));
            s = sum_firsts(a, s, lo + n * warp / kJoinWarps, lo + n * (warp + 1) / kJoinWarps, c);
        }
        s_part[warp][lane] = s;
        __syncthreads();
        if (warp == 0 && c < a.H) {
#pragma unroll
            for (int i = 1; i < kJoinWarps; ++i) add4(s, s_part[i][lane]);
            write_row<4>(a, s_id[w], c, reinterpret_cast<const float *>(&s));
        }
        __syncthreads();
    }
}

}  // namespace emb
}  // namespace qlora
