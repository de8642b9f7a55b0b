// embedding.cuh -- rows of a packed or plain embedding table for a batch of token ids, and
// the gradient of a plain table from the tokens sorted by id.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"
#include "quant_kernels.cuh"
#include "scale_src.cuh"
#include "step_common.cuh"

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
// (only where nothing is recorded yet: a timeout or a failed tensor-memory store of an earlier kernel is the graver error)
__device__ __forceinline__ void report_bad_id() { atomicCAS(&g_device_error, 0, kDeviceErrIndex); }

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
    int64_t T, V;
    int H;
    float scale;
    int seg_shift;         // log2 of the row segments of kRun elements that a CTA takes (at most its warps)
    int passes;            // tokens a warp takes, one after the other
    float level[16];
};
constexpr int kFwdThreads = 256;
constexpr int kFwdWarps = kFwdThreads / 32;
constexpr int kUnroll = 4;
constexpr int kRun = 256 * kUnroll;   // elements of a row a warp takes: 8 per lane and step
constexpr int kFwdPasses = 4;         // most tokens a warp takes

// 32-bit words of 8 elements of a table
template <int kTable>
constexpr int kWordsOf = kTable == kTableNf4 ? 1 : kTable == kTableQ8 ? 2 : kTable == kTableBf16 ? 4 : 8;
__device__ __forceinline__ float level_at(const float *levels, uint32_t byte_offset) {
    return *reinterpret_cast<const float *>(reinterpret_cast<const char *>(levels) + byte_offset);
}

// 8 elements from column e of a row on: as loaded (with the words of their scale), and as pairs of floats
template <int kTable, bool kDq>
struct Fetch {
    uint32_t w[kWordsOf<kTable>];
    uint32_t sa;
    float sd;
    // at: the place of the 8 elements in the table; off: 0, 256, 512 ... elements behind it
    __device__ __forceinline__ void load(const FwdArgs &a, int64_t at, int off) {
        if (kTable == kTableNf4) {
            w[0] = __ldcg(reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(a.table) + (at >> 1)) + off / 8);
            const int64_t b = (at >> 6 >> a.sc.blk_shift) + (off / 64 >> a.sc.blk_shift);
            if (kDq) {
                sa = __ldcg(a.sc.scales + b);
                sd = __ldcg(a.sc.scales2 + (b >> 8));
            } else {
                sa = __ldcg(reinterpret_cast<const uint32_t *>(a.sc.scales) + b);
            }
        } else if (kTable == kTableQ8) {
            const uint2 q = __ldcg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.table) + at) + off / 8);
            w[0] = q.x;
            w[1 % kWordsOf<kTable>] = q.y;
            sa = __ldcg(a.d8 + (at >> 5) + off / 32);
        } else {
            const char *p = static_cast<const char *>(a.table) + at * (kTable == kTableBf16 ? 2 : 4);
#pragma unroll
            for (int h = 0; h < kWordsOf<kTable> / 4; ++h) {
                const uint4 x = __ldcg(reinterpret_cast<const uint4 *>(p) + off / (kTable == kTableBf16 ? 8 : 4) + h);
                w[(4 * h) % kWordsOf<kTable>] = x.x, w[(4 * h + 1) % kWordsOf<kTable>] = x.y;
                w[(4 * h + 2) % kWordsOf<kTable>] = x.z, w[(4 * h + 3) % kWordsOf<kTable>] = x.w;
            }
        }
    }
    __device__ __forceinline__ void values(const float *levels, uint64_t scale, uint64_t *y) const {
        if (kTable == kTableNf4) {
            // byte offsets 4 c into the level table, four codes at a time
            const float f = kDq ? __fmul_rn(static_cast<float>(sa), sd) : __uint_as_float(sa);
            const uint32_t lo = (w[0] << 2) & 0x3C3C3C3Cu, hi = (w[0] >> 2) & 0x3C3C3C3Cu;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                y[j] = mul2(pack2(level_at(levels, __byte_perm(lo, 0u, 0x4440u + j)), level_at(levels, __byte_perm(hi, 0u, 0x4440u + j))),
                            pack2(f, f));
        } else if (kTable == kTableQ8) {
            const float f = __half2float(__ushort_as_half(static_cast<unsigned short>(sa)));
            const uint64_t magic = pack2(-8388736.f, -8388736.f);   // -(2^23 + 128)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t b = w[(j / 2) % kWordsOf<kTable>] ^ 0x80808080u;
                y[j] = mul2(add2(pack2(__uint_as_float(__byte_perm(b, 0x4B000000u, 0x7650 + 2 * (j & 1))),
                                       __uint_as_float(__byte_perm(b, 0x4B000000u, 0x7651 + 2 * (j & 1)))), magic), pack2(f, f));
            }
        } else if (kTable == kTableBf16) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t x = w[j % kWordsOf<kTable>];
                y[j] = pack2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                y[j] = pack2(__uint_as_float(w[(2 * j) % kWordsOf<kTable>]), __uint_as_float(w[(2 * j + 1) % kWordsOf<kTable>]));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = mul2(y[j], scale);
    }
};
// 8 elements to a row of the output
template <bool kOutBf16>
__device__ __forceinline__ void put8(char *row, int e, const uint64_t *w) {
    float y[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) unpack2(w[j], y[2 * j], y[2 * j + 1]);
    if (kOutBf16) {
        uint32_t b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(y[2 * j], y[2 * j + 1]);
            b[j] = *reinterpret_cast<const uint32_t *>(&p);
        }
        reinterpret_cast<uint4 *>(row)[e >> 3] = make_uint4(b[0], b[1], b[2], b[3]);
    } else {
        float4 *dst = reinterpret_cast<float4 *>(row) + (e >> 2);
        dst[0] = make_float4(y[0], y[1], y[2], y[3]);
        dst[1] = make_float4(y[4], y[5], y[6], y[7]);
    }
}

// A warp takes one segment of a token's row: every code and scale load of the segment at once, 8 elements
// per lane and step, so that a bf16 output is one 16-byte store.  Then the same segment of the CTA's next token.
// CTAs: x over groups of tokens, in the order of the output; y over groups of 2^seg_shift segments.
template <int kTable, bool kDq, bool kOutBf16>
__global__ void __launch_bounds__(kFwdThreads) embed_fwd_kernel(const __grid_constant__ FwdArgs a) {
    __shared__ float s_lv[16];
    if (kTable == kTableNf4) {
        if (threadIdx.x < 16) s_lv[threadIdx.x] = a.level[threadIdx.x];
        __syncthreads();
    }
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per_pass = kFwdWarps >> a.seg_shift;           // tokens of the CTA in one pass
    const int64_t t0 = int64_t(blockIdx.x) * (per_pass * a.passes) + (warp >> a.seg_shift);
    const int e0 = static_cast<int>((blockIdx.y << a.seg_shift) + (warp & ((1 << a.seg_shift) - 1))) * kRun + lane * 8;
    if (e0 - lane * 8 >= a.H) return;
    int64_t ids[kFwdPasses];
#pragma unroll
    for (int p = 0; p < kFwdPasses; ++p)
        ids[p] = p < a.passes && t0 + p * per_pass < a.T ? id_at(a.ids, t0 + p * per_pass) : 0;
    const uint64_t scale = pack2(a.scale, a.scale);
#pragma unroll 1
    for (int p = 0; p < a.passes; ++p) {
        const int64_t t = t0 + p * per_pass;
        if (t >= a.T) return;
        int64_t id = ids[0];
#pragma unroll
        for (int j = 1; j < kFwdPasses; ++j) id = p == j ? ids[j] : id;
        char *row = static_cast<char *>(a.out) + t * a.H * (kOutBf16 ? 2 : 4);
        if (id < 0 || id >= a.V) {
            if (lane == 0) report_bad_id();
            const uint64_t zero[4] = {0, 0, 0, 0};
            for (int e = e0; e < a.H && e < e0 + kRun; e += 256) put8<kOutBf16>(row, e, zero);
            continue;
        }
        const int64_t at = id * a.H + e0;
        Fetch<kTable, kDq> x[kUnroll];
        uint64_t y[4];
        if (e0 - lane * 8 + kRun <= a.H) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) x[u].load(a, at, u * 256);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                x[u].values(s_lv, scale, y);
                put8<kOutBf16>(row, e0 + u * 256, y);
            }
        } else {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (e0 + u * 256 < a.H) x[u].load(a, at, u * 256);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (e0 + u * 256 >= a.H) break;
                x[u].values(s_lv, scale, y);
                put8<kOutBf16>(row, e0 + u * 256, y);
            }
        }
    }
}

// ------------------------------------------------------------------ gradient
// dE[v, :] (+)= scale * sum over the tokens t with id_t = v of dY[t, :], in three or four launches:
//   mark    (where the cluster sorts, and unless the gradient is added) sets a bit for every row that a token names;
//   sort    the tokens by id (stable);
//   reduce  equal runs of `chunk` sorted tokens each: an id that lies wholly in a chunk is summed
//           and written, one that crosses a border leaves a partial sum per chunk;
//   join    adds the partial sums of each such id in order and writes its row.
// Unless the gradient is added, further CTAs of these launches zero the table: the whole of it beside the sort where that
// takes one CTA, else the rows without a bit.
// Up to kFewTokens tokens take one launch, whose zeroing CTAs look at the ids themselves.
// Every sum is float32, in an order fixed by the ids alone: results repeat bit for bit.
// Programmatic dependent launch: a kernel may start while the one before it still runs, and every thread waits for
// that one to end before it reads or writes global memory: the trigger of a launch promises no visibility, not even of
// what was complete before it.  (So no launch of zeros runs beside the whole chain: 8192 x 4096 into 32000 rows takes
// 114 us where one that relied on the trigger took 107, 2047 x 4096 takes 88 as it did.)
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
    // CTAs (along x) that sort and that sum.  Those behind them zero rows of the table, sort_rows or sum_rows each: the
    // first `early` beside the sort, the others beside the sums.
    int sort_ctas, sum_ctas;
    int sort_rows, sum_rows;
    int64_t early;
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

// The place of a token among the equal digits that its warp has met so far, counted in my[].
__device__ __forceinline__ uint32_t rank_digit(uint32_t *my, uint32_t d, bool in, int lane) {
    const uint32_t same = __match_any_sync(0xffffffffu, in ? d : uint32_t(kMaxBins));   // idle lanes match none
    const uint32_t lower = same & ((1u << lane) - 1u);
    uint32_t r = 0;
    if (in) r = my[d] + __popc(lower);
    __syncwarp();
    if (in && lower == 0) my[d] += __popc(same);
    __syncwarp();
    return r;
}
// Per bin: counts of lower warps in hist, the CTA's total as the result (threads below `bins`).
__device__ __forceinline__ uint32_t scan_warps(uint32_t *hist, int bin) {
    uint32_t sum = 0, n[kSortWarps];
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) n[w] = hist[w * kMaxBins + bin];
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
        hist[w * kMaxBins + bin] = sum;
        sum += n[w];
    }
    return sum;
}
// Exclusive scan over the CTA's threads of n; wsum holds kSortWarps words.
__device__ __forceinline__ uint32_t scan_threads(uint32_t n, uint32_t *wsum, int warp, int lane) {
    uint32_t incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    uint32_t base = lane < warp ? wsum[lane] : 0u;
    base = __reduce_add_sync(0xffffffffu, base);
    return base + incl - n;
}

// Radix sort, least significant digit first, by one CTA (up to 2048 tokens; 4096 where a large table is written) or by the
// cluster of kSortCtas (up to 131072), with a CTA's tokens in registers (16 a thread, from 32769 tokens on, spill 176 bytes
// under the 64 registers that 1024 threads leave).  Whole gradient of rows of 64, one CTA / cluster: 11.4 / 14.4 us at 1024
// tokens, 15.0 / 15.9 at 2048, 20.2 / 17.5 at 4096; held in registers / swept from memory (below): 34.9 / 40.4 us
// at 32768, 89.7 / 96.5 at 131072.  Tokens are dealt in order to CTAs, warps and rounds of 32, so a
// token's place among equal digits is the count in lower CTAs, in lower warps, in its warp's earlier rounds and
// in its lower lanes: stable without atomics.  A CTA reorders its tokens in shared memory first, so that what it
// writes to global memory comes in runs (scattered 4-byte stores kept one SM busy for 25 us per 16384 tokens).
constexpr int kCtaRounds = 16;                       // most rounds of 1024 tokens a CTA holds
constexpr int kOneTokens = 2 * kSortThreads;
constexpr int kOneWritten = 4 * kSortThreads;         // of a large table that is written, see zero_rows
constexpr int kHeldTokens = kCtaRounds * kSortThreads * kSortCtas;
constexpr int kHeldWords = kSortWarps * kMaxBins + 4 * kMaxBins + 64;
constexpr int held_smem(int rounds) { return 4 * kHeldWords + 8 * kSortThreads * rounds; }
template <bool kCluster, int kRounds>
__device__ void sort_held(const GradArgs &a, uint32_t *smem, int rounds) {
    uint32_t *hist = smem;                           // [warp][bin]
    uint32_t *total = hist + kSortWarps * kMaxBins;  // [bin] of this CTA
    uint32_t *local = total + kMaxBins;              // [bin] first place of the bin among this CTA's tokens
    uint32_t *delta = local + kMaxBins;              // [bin] from there to its first place in the whole list
    uint32_t *wsum = delta + kMaxBins;               // [warp] sums of a scan, twice
    uint32_t *keys = smem + kHeldWords, *places = keys + rounds * kSortThreads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, bins = 1 << a.bits;
    const uint32_t rank = kCluster ? cluster_rank() : 0u;
    const int64_t lo = min(int64_t(rank) * rounds * kSortThreads, a.T);
    const int n = static_cast<int>(min(int64_t(rounds) * kSortThreads, a.T - lo));    // this CTA's tokens
    const int i0 = warp * rounds * 32 + lane;
    uint32_t *my = hist + warp * kMaxBins;
    uint32_t k[kRounds], p[kRounds], r[kRounds];
#pragma unroll
    for (int u = 0; u < kRounds; ++u) {
        if (u >= rounds) break;
        const int t = i0 + 32 * u;
        k[u] = t < n ? key_of(a, lo + t) : 0u;
        p[u] = static_cast<uint32_t>(lo + t);
    }
    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = pass * a.bits;
        for (int b = lane; b < bins; b += 32) my[b] = 0;
        __syncwarp();
#pragma unroll
        for (int u = 0; u < kRounds; ++u) {
            if (u >= rounds) break;
            r[u] = rank_digit(my, (k[u] >> shift) & (bins - 1), i0 + 32 * u < n, lane);
        }
        __syncthreads();
        const uint32_t mine = tid < bins ? scan_warps(hist, tid) : 0u;
        uint32_t below = 0, all = mine;
        if constexpr (kCluster) {
            if (tid < bins) total[tid] = mine;
            cluster_barrier();
            all = 0;
            if (tid < bins) {
#pragma unroll
                for (uint32_t c = 0; c < kSortCtas; ++c) {
                    const uint32_t x = ld_cluster(total + tid, c);
                    all += x;
                    if (c < rank) below += x;
                }
            }
        }
        const uint32_t in_cta = scan_threads(mine, wsum, warp, lane);
        const uint32_t in_list = kCluster ? scan_threads(all, wsum + kSortWarps, warp, lane) + below : in_cta;
        if (tid < bins) {
            local[tid] = in_cta;
            delta[tid] = in_list - in_cta;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kRounds; ++u) {
            if (u >= rounds || i0 + 32 * u >= n) break;          // a lane's places ascend
            const uint32_t d = (k[u] >> shift) & (bins - 1), at = local[d] + my[d] + r[u];
            keys[at] = k[u];
            places[at] = p[u];
        }
        __syncthreads();
        const bool last = pass + 1 == a.passes;
        if (kCluster || last) {
            uint32_t *dst_k = a.key[(pass + 1) & 1], *dst_p = a.pos[(pass + 1) & 1];
            for (int j = tid; j < n; j += kSortThreads) {
                const uint32_t key = keys[j], at = j + delta[(key >> shift) & (bins - 1)];
                __stcg(dst_k + at, key);
                __stcg(dst_p + at, places[j]);
            }
            if (last) break;
            cluster_barrier();   // the next pass reads what every CTA wrote; total is free again
        }
#pragma unroll
        for (int u = 0; u < kRounds; ++u) {
            const int t = i0 + 32 * u;
            if (u >= rounds || t >= n) break;
            k[u] = kCluster ? __ldcg(a.key[(pass + 1) & 1] + lo + t) : keys[t];
            p[u] = kCluster ? __ldcg(a.pos[(pass + 1) & 1] + lo + t) : places[t];
        }
    }
    if (kCluster) cluster_barrier();   // no CTA leaves while another may read its totals
}

// More tokens than the cluster holds: the same dealing, with two sweeps over the tokens in global memory per
// digit, to count and to place them.
__device__ void sort_swept(const GradArgs &a, uint32_t *smem) {
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
        // two sweeps over the warp's tokens: count the digits, then place the tokens
        auto sweep = [&](auto &&use) {
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
                    const uint32_t d = (k[u] >> shift) & (bins - 1);
                    use(k[u], p[u], d, rank_digit(my, d, in, lane), in);
                }
            }
        };
        sweep([](uint32_t, uint32_t, uint32_t, uint32_t, bool) {});
        __syncthreads();
        if (tid < bins) total[tid] = scan_warps(hist, tid);
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
        const uint32_t base = scan_threads(all, wsum, warp, lane);
        if (tid < bins) first[tid] = base + below;
        __syncthreads();
        // hist now counts on from the lower warps' numbers
        sweep([&](uint32_t k, uint32_t p, uint32_t d, uint32_t r, bool in) {
            if (in) {
                const uint32_t at = first[d] + r;
                __stcg(dst_k + at, k);
                __stcg(dst_p + at, p);
            }
        });
        cluster_barrier();   // the next pass reads what every CTA wrote; total is free again
    }
}

__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads) embed_mark_kernel(const GradArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t first = int64_t(cluster_rank()) * kSortThreads + threadIdx.x, step = kSortCtas * kSortThreads;
    for (int64_t i = first; i < (a.V + 31) / 32; i += step) __stcg(a.named + i, 0u);
    cluster_barrier();
#pragma unroll 4
    for (int64_t t = first; t < a.T; t += step) {
        const int64_t id = id_at(a.ids, t);
        if (id >= 0 && id < a.V && id != a.pad) atomicOr(a.named + (id >> 5), 1u << (id & 31));
    }
}
// Zero: CTAs come in the order of the table.  (A grid of two CTAs per SM that strides over the rows wrote 6.0 TB/s, this
// order 7.2: what is written at any time lies close together.)  What is zeroed where, us a call from bf16 rows of 1024 into
// fp32 tables:
// - up to 2048 tokens the whole table beside the sort of one CTA, where marking and zeroing beside the sums took 25.8 for
//   20.2 (2047 into 16000 rows) and 14.2 for 11.9 (300 into 1000).  With 16 / 32 / 64 KB a CTA there: 20.1 / 18.7 / 20.8 at
//   2047 into 4000 rows, 36.3 / 32.0 / 29.7 into 32000.
// - so too up to 4096 tokens from 40 MB of table on: the slower sort is hidden then (4096 tokens, by one CTA / by the
//   cluster: 26.1 / 24.6 into 16 MB, 28.6 / 30.7 into 65 MB, 35.6 / 36.9 into 131 MB).
// - else beside the sums, but from 56 MB of table on for a share beside the cluster that sorts (6000 tokens, with the
//   share / without: 31.6 / 29.5 into 49 MB, 38.1 / 45.3 into 131 MB).  Clusters of zeroing CTAs 2 / 6 / 9 / 14, with as much
//   in all: 140 / 123 / 118 / 114 at 8192 x 4096 into 32000 rows.
constexpr int kRedThreads = 128;                          // of the kernels that sum
constexpr int kZeroBytes = 16384;                         // of a CTA beside the sums
constexpr int kZeroWords = kZeroBytes / 16 / 32 + 1;      // words of bits of its rows, at 16 bytes a row
constexpr int kOneZeroBytes = 32768;                      // of a CTA beside the sort of one CTA
constexpr int64_t kOneTable = 40 << 20;                   // bytes of a table from which up to kOneWritten tokens are sorted by one
constexpr int kEarlyBytes = 524288;                       // of a CTA beside the cluster that sorts
constexpr int64_t kEarlyTable = 56 << 20;                 // bytes of a table from which there are such CTAs
constexpr int kEarlyClusters = 14;                        // clusters of them: 15 of 8 SMs fit at once
enum { kZeroAll = 0, kZeroMarked = 1, kZeroFew = 2 };     // every row; those without a mark; those not among the few ids
// Zeroes rows [r0, end) of dE.  bits: room for a bit a row.
template <int kThreads, int kWhich>
__device__ __forceinline__ void zero_rows(const GradArgs &a, int64_t r0, int64_t end, uint32_t *bits) {
    if (r0 >= end) return;      // the last CTAs may go past what there is
    const int64_t row_words = a.H * (a.de_bf16 ? 2 : 4) / 16, b0 = r0 >> 5;
    uint4 *dst = static_cast<uint4 *>(a.dE) + r0 * row_words;
    if (kWhich == kZeroAll) {
        const int64_t all = (end - r0) * row_words;
#pragma unroll 4
        for (int64_t i = threadIdx.x; i < all; i += kThreads) dst[i] = make_uint4(0, 0, 0, 0);
        return;
    }
    const int words = static_cast<int>(((end - 1) >> 5) - b0) + 1;
    for (int i = threadIdx.x; i < words; i += kThreads) bits[i] = kWhich == kZeroFew ? 0u : __ldcg(a.named + b0 + i);
    __syncthreads();
    if (kWhich == kZeroFew) {   // the CTA looks for its own rows among the ids
        for (int t = threadIdx.x; t < a.T; t += kThreads) {
            const int64_t id = id_at(a.ids, t);
            if (id >= r0 && id < end && id != a.pad) atomicOr(bits + ((id >> 5) - b0), 1u << (id & 31));
        }
        __syncthreads();
    }
    auto named = [&](int64_t r) { return (bits[(r >> 5) - b0] >> (r & 31)) & 1u; };
    if (row_words >= kThreads) {
        for (int64_t r = r0; r < end; ++r, dst += row_words) {
            if (named(r)) continue;
#pragma unroll 4
            for (int64_t i = threadIdx.x; i < row_words; i += kThreads) dst[i] = make_uint4(0, 0, 0, 0);
        }
    } else {
        // short rows: the CTA's words (at most kEarlyBytes / 16) as one run
        const uint32_t all = static_cast<uint32_t>((end - r0) * row_words), rw = static_cast<uint32_t>(row_words);
#pragma unroll 4
        for (uint32_t i = threadIdx.x; i < all; i += kThreads)
            if (!named(r0 + i / rw)) dst[i] = make_uint4(0, 0, 0, 0);
    }
}
// what a CTA behind those that sort, or behind those that sum, zeroes
template <int kWhich>
__device__ __forceinline__ void zero_beside_sort(const GradArgs &a, uint32_t *smem) {
    const int64_t r0 = int64_t(blockIdx.x - a.sort_ctas) * a.sort_rows;
    zero_rows<kSortThreads, kWhich>(a, r0, min(r0 + a.sort_rows, a.early), smem);
}
template <int kWhich>
__device__ __forceinline__ void zero_beside_sums(const GradArgs &a) {
    __shared__ uint32_t s_named[kZeroWords];
    const int64_t r0 = a.early + (int64_t(blockIdx.y) * (gridDim.x - a.sum_ctas) + (blockIdx.x - a.sum_ctas)) * a.sum_rows;
    zero_rows<kRedThreads, kWhich>(a, r0, min(r0 + a.sum_rows, a.V), s_named);
}

template <int kRounds>
__global__ void __launch_bounds__(kSortThreads, 2) embed_sort_one_kernel(const GradArgs a, int rounds) {
    extern __shared__ uint32_t sort_smem[];
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x >= a.sort_ctas) {
        zero_beside_sort<kZeroAll>(a, sort_smem);
        return;
    }
    sort_held<false, kRounds>(a, sort_smem, rounds);
}
template <int kRounds>
__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads, 1) embed_sort_held_kernel(const GradArgs a, int rounds) {
    extern __shared__ uint32_t sort_smem[];
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x >= a.sort_ctas) {
        zero_beside_sort<kZeroMarked>(a, sort_smem);
        return;
    }
    sort_held<true, kRounds>(a, sort_smem, rounds);
}
__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads, 1) embed_sort_swept_kernel(const GradArgs a) {
    extern __shared__ uint32_t sort_smem[];
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x >= a.sort_ctas) {
        zero_beside_sort<kZeroMarked>(a, sort_smem);
        return;
    }
    sort_swept(a, sort_smem);
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
constexpr int kRedCols = kRedThreads * 8;
constexpr int kMaxChunk = 128;
constexpr int kBatch = 4;
template <bool kDyBf16, bool kDeBf16, bool kAdd>
__global__ void __launch_bounds__(kRedThreads) embed_reduce_kernel(const GradArgs a) {
    __shared__ uint32_t s_id[kMaxChunk + 2], s_pos[kMaxChunk];   // s_id[0]: the token before the chunk; last + 1: after it
    pdl_launch_dependents();
    pdl_wait();
    if (!kAdd && blockIdx.x >= a.sum_ctas) {
        zero_beside_sums<kZeroMarked>(a);
        return;
    }
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

// A few tokens (up to kFewTokens): one launch instead of sort, reduce and join.  Every block ranks the ids for
// itself (a thread counts the smaller ones), and a group of blocks takes the ids that start in kFewRun
// places of the sorted list, each to its end.  Sorted / in one launch, rows of 4096 added: 9.2 / 3.4 us at 64
// tokens, 9.3 / 4.3 at 128, 9.6 / 7.9 at 192, 9.9 / 9.8 at 256, 11.9 / 20.5 at 384 (the ranks grow with T^2).
constexpr int kFewTokens = 192;
constexpr int kFewRun = 4;
template <bool kDyBf16, bool kDeBf16, bool kAdd>
__global__ void __launch_bounds__(kRedThreads) embed_few_kernel(const GradArgs a) {
    __shared__ uint32_t s_key[kFewTokens], s_id[kFewTokens + 2], s_pos[kFewTokens];   // s_id as in embed_reduce_kernel
    pdl_wait();
    pdl_launch_dependents();
    if (!kAdd && blockIdx.x >= a.sum_ctas) {
        zero_beside_sums<kZeroFew>(a);
        return;
    }
    const int tid = threadIdx.x, T = static_cast<int>(a.T);
    const uint32_t V = static_cast<uint32_t>(a.V);
    for (int t = tid; t < T; t += kRedThreads) s_key[t] = key_of(a, t);
    if (tid == 0) s_id[0] = s_id[T + 1] = 0xFFFFFFFFu;
    __syncthreads();
    for (int t = tid; t < T; t += kRedThreads) {
        const uint32_t key = s_key[t];
        int place = 0;
#pragma unroll 8
        for (int s = 0; s < T; ++s) place += s_key[s] < key || (s_key[s] == key && s < t);
        s_id[place + 1] = key;
        s_pos[place] = t;
    }
    __syncthreads();
    int lo = blockIdx.x * kFewRun, hi = min(lo + kFewRun, T);
    while (lo < hi && s_id[lo + 1] == s_id[lo]) ++lo;        // an id that starts before belongs to the block before
    if (lo >= hi || s_id[lo + 1] >= V) return;
    while (s_id[hi + 1] == s_id[hi]) ++hi;
    const int64_t c = int64_t(blockIdx.y) * kRedCols + tid * 8;
    if (c >= a.H) return;
    float acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    for (int i = lo; i < hi; i += kBatch) {
        Raw<kDyBf16, 8> r[kBatch];
        Raw<kDeBf16, 8> old[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            old[u].zero();
            if (i + u >= hi) continue;
            const uint32_t id = s_id[i + u + 1];
            if (id >= V) continue;
            r[u].load(a.dY, int64_t(s_pos[i + u]) * a.H + c);
            if (kAdd && s_id[i + u + 2] != id) old[u].load(a.dE, int64_t(id) * a.H + c);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (i + u >= hi) break;
            const uint32_t id = s_id[i + u + 1];
            if (id >= V) break;
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += r[u].at(j);
            if (s_id[i + u + 2] == id) continue;
            write_row<kDeBf16, 8>(a, id, c, acc, old[u]);
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
constexpr int kLongJoin = 8;
__device__ __forceinline__ void add4(float4 &s, const float4 x) {
    s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
}
__device__ __forceinline__ float4 load_part(const GradArgs &a, int64_t slot, int64_t c) {
    return __ldcg(reinterpret_cast<const float4 *>(a.part + slot * a.H + c));
}
constexpr int kJoinRuns = kJoinCols / 128;
// adds the first-run partials of chunks [lo, hi), columns c + 128 q .. + 3, to s[q]; two chunks in flight
__device__ __forceinline__ void sum_firsts(const GradArgs &a, float4 *s, int64_t lo, int64_t hi, int64_t c) {
    for (; lo < hi; lo += 2) {
        float4 x[2][kJoinRuns];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int q = 0; q < kJoinRuns; ++q) {
                x[u][q] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (lo + u < hi && c + 128 * q < a.H) x[u][q] = load_part(a, 2 * (lo + u), c + 128 * q);
            }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int q = 0; q < kJoinRuns; ++q) add4(s[q], x[u][q]);
    }
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
    __shared__ float4 s_part[kJoinWarps][kJoinRuns][32];
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
    // the id's row from the sums s of the columns c + 128 q, on top of its old values
    auto finish = [&](uint32_t row, const float4 *s) {
        Raw<kDeBf16, 4> old[kJoinRuns];
#pragma unroll
        for (int q = 0; q < kJoinRuns; ++q) {
            old[q].zero();
            if (a.accumulate && c + 128 * q < a.H) old[q].load(a.dE, int64_t(row) * a.H + c + 128 * q);
        }
#pragma unroll
        for (int q = 0; q < kJoinRuns; ++q)
            if (c + 128 * q < a.H) write_row<kDeBf16, 4>(a, row, c + 128 * q, reinterpret_cast<const float *>(s + q), old[q]);
    };
    auto start = [&](float4 *s, int64_t chunk, uint32_t which) {
#pragma unroll
        for (int q = 0; q < kJoinRuns; ++q) {
            s[q] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (chunk >= 0 && c + 128 * q < a.H) s[q] = load_part(a, 2 * chunk + which, c + 128 * q);
        }
    };
    float4 s[kJoinRuns];
    if (end && end - ch <= kLongJoin) {
        start(s, ch, slot);
        sum_firsts(a, s, ch + 1, end, c);
        finish(id, s);
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
        start(s, warp == 0 ? lo - 1 : -1, s_slot[w]);
        sum_firsts(a, s, lo + n * warp / kJoinWarps, lo + n * (warp + 1) / kJoinWarps, c);
#pragma unroll
        for (int q = 0; q < kJoinRuns; ++q) s_part[warp][q][lane] = s[q];
        __syncthreads();
        if (warp == 0) {
#pragma unroll
            for (int i = 1; i < kJoinWarps; ++i)
#pragma unroll
                for (int q = 0; q < kJoinRuns; ++q) add4(s[q], s_part[i][q][lane]);
            finish(s_id[w], s);
        }
        __syncthreads();
    }
}

}  // namespace emb
}  // namespace qlora
