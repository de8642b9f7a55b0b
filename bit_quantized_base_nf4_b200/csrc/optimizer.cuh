// optimizer.cuh -- AdamW over many tensors in one launch (states in 32 bits or in 8 bits),
// the global gradient norm with its clip coefficient, and the 8-bit state code.
//
// One step, per element, every operation rounded to float32:
//   g = grad (* clip coefficient)
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2
//   p = p - lr (decay p + (m / (1 - b1^t)) / (sqrt(v) / sqrt(1 - b2^t) + eps))
//
// 8-bit states: blocks of 256 values with one fp32 step d each, value = k |k| d, where x is
// m (k in -127 .. 127) or sqrt(v) (k in 0 .. 255; the second moment is the value's square).
//   d = RN(max |x| / K^2), K = 127 or 255;  y = RN(|x| RN(1 / d));
//   |k| = #{j : y > j^2 + j + 1/2}, the square nearest to y, ties to the lower k.
// Evenly spaced roots resolve a block's small values (smallest 1/16129 and 1/65025 of the
// block's largest) at a bounded cost for its large ones (half a step is 0.8 % and 0.4 % at
// the top).  sqrt(v) is stored, not v, so that m and the denominator keep the same range.
// All roundings up to the code are fixed (no fused multiply-add), so codes are bit-exact.
// A block with a non-finite value stores d = NaN and k = 0: every later step on it is NaN.
// d below 2^-126, where 1 / d could overflow, is stored as 0 with k = 0.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "ptx.cuh"

namespace qlora {
namespace optim {

constexpr int kBlock = 256;          // values per 8-bit block: one warp step, 8 per lane
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPartials = 2048;      // slots for per-CTA partial sums of the norm
constexpr int kTopM = 127, kTopW = 255;

enum : uint32_t { kParamBf16 = 1, kGradBf16 = 2, kState8 = 4 };

// A run of at most `chunk` elements of one tensor, starting at a multiple of kBlock: the
// addresses of its first element in every buffer.  80 bytes; a warp loads it with one
// coalesced read (20 words) and broadcasts the fields.
struct alignas(16) Chunk {
    uint64_t p, copy, g, m, v, dm, dv;
    int32_t n;
    uint32_t flags;
    float lr_scale, decay;
    uint64_t unused;
};
static_assert(sizeof(Chunk) == 80, "a chunk is 20 words");

// Head of the plan buffer: the CTA ticket of the norm and of the device step counter, then the
// partial sums.  Every kernel leaves the ticket at zero.
struct alignas(256) PlanHead {
    unsigned int ticket;
    unsigned int unused[63];
    double partial[kPartials];
};

__device__ __forceinline__ uint32_t chunk_word(const Chunk *chunks, int64_t c, int lane) {
    return lane < 20 ? __ldg(reinterpret_cast<const uint32_t *>(chunks + c) + lane) : 0u;
}
__device__ __forceinline__ uint32_t word32(uint32_t w, int i) { return __shfl_sync(0xffffffffu, w, i); }
__device__ __forceinline__ uint64_t word64(uint32_t w, int i) {
    return uint64_t(word32(w, i)) | (uint64_t(word32(w, i + 1)) << 32);
}

// Element of half h (0, 1) and place j (0..3) of a lane's 8 in a block: h * 128 + lane * 4 + j.
__device__ __forceinline__ void unpack4(uint2 u, float *x) {
    x[0] = __uint_as_float(u.x << 16);
    x[1] = __uint_as_float(u.x & 0xFFFF0000u);
    x[2] = __uint_as_float(u.y << 16);
    x[3] = __uint_as_float(u.y & 0xFFFF0000u);
}
// rem: elements of the chunk from the block's first on.  kFull: rem >= 256.
template <bool kFull>
__device__ __forceinline__ void load8(uint64_t base, bool bf16, int64_t i0, int rem, int lane, float *x) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int e = h * 128 + lane * 4;
        if (kFull) {
            if (bf16) {
                unpack4(*reinterpret_cast<const uint2 *>(base + 2 * (i0 + e)), x + 4 * h);
            } else {
                const float4 f = *reinterpret_cast<const float4 *>(base + 4 * (i0 + e));
                x[4 * h] = f.x, x[4 * h + 1] = f.y, x[4 * h + 2] = f.z, x[4 * h + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float f = 0.f;
                if (e + j < rem)
                    f = bf16 ? __uint_as_float(uint32_t(reinterpret_cast<const uint16_t *>(base)[i0 + e + j]) << 16)
                             : reinterpret_cast<const float *>(base)[i0 + e + j];
                x[4 * h + j] = f;
            }
        }
    }
}
template <bool kFull>
__device__ __forceinline__ void store8(uint64_t base, bool bf16, int64_t i0, int rem, int lane, const float *x) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int e = h * 128 + lane * 4;
        const float *y = x + 4 * h;
        if (kFull) {
            if (bf16) {
                const __nv_bfloat162 a = __floats2bfloat162_rn(y[0], y[1]), b = __floats2bfloat162_rn(y[2], y[3]);
                *reinterpret_cast<uint2 *>(base + 2 * (i0 + e)) =
                    make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
            } else {
                *reinterpret_cast<float4 *>(base + 4 * (i0 + e)) = make_float4(y[0], y[1], y[2], y[3]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (e + j < rem) {
                    if (bf16) reinterpret_cast<__nv_bfloat16 *>(base)[i0 + e + j] = __float2bfloat16_rn(y[j]);
                    else reinterpret_cast<float *>(base)[i0 + e + j] = y[j];
                }
        }
    }
}
// the two code words (4 codes each) of a lane
template <bool kFull>
__device__ __forceinline__ void load_codes(uint64_t base, int64_t i0, int rem, int lane, uint32_t *c) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int e = h * 128 + lane * 4;
        if (kFull) {
            c[h] = *reinterpret_cast<const uint32_t *>(base + i0 + e);
        } else {
            c[h] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (e + j < rem) c[h] |= uint32_t(reinterpret_cast<const uint8_t *>(base)[i0 + e + j]) << (8 * j);
        }
    }
}
template <bool kFull>
__device__ __forceinline__ void store_codes(uint64_t base, int64_t i0, int rem, int lane, const uint32_t *c) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int e = h * 128 + lane * 4;
        if (kFull) {
            *reinterpret_cast<uint32_t *>(base + i0 + e) = c[h];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (e + j < rem) reinterpret_cast<uint8_t *>(base)[i0 + e + j] = uint8_t(c[h] >> (8 * j));
        }
    }
}

// k of byte j as a float: the byte becomes the low mantissa byte of 2^23 (one permute and one
// exact subtraction; no integer conversion, whose pipe is eight times narrower)
template <bool kSigned>
__device__ __forceinline__ float code_value(uint32_t w, int j) {
    const uint32_t u = kSigned ? w ^ 0x80808080u : w;
    const float magic = kSigned ? 8388736.f : 8388608.f;   // 2^23 (+ 128)
    return __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7650 + j)) - magic;
}
// x[0..7] = k |k| d of a lane's codes
template <bool kSigned>
__device__ __forceinline__ void decode8(const uint32_t *c, float d, float *x) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float k = code_value<kSigned>(c[i >> 2], i & 3);
        x[i] = __fmul_rn(__fmul_rn(k, fabsf(k)), d);
    }
}
// roots to 2^-23: kFtz takes inputs below 2^-126 as 0
template <bool kFtz>
__device__ __forceinline__ float sqrt_approx(float x) {
    float r;
    if (kFtz) asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    else asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// the larger magnitude as bits: an infinity is above every finite value, a NaN above that
__device__ __forceinline__ uint32_t max_bits(uint32_t a, float x) { return max(a, __float_as_uint(x) & 0x7FFFFFFFu); }

// A block's step d = RN(a / top^2) from the bits of its largest magnitude a, and RN(1 / d)
__device__ __forceinline__ void block_step(uint32_t a_bits, float top2, float &d, float &inv) {
    d = __fdiv_rn(__uint_as_float(a_bits), top2);
    inv = __frcp_rn(d);
    if (d < 1.17549435e-38f) d = 0.f, inv = 0.f;
    if (a_bits >= 0x7F800000u) d = __uint_as_float(0x7FC00000u), inv = 0.f;
}

// Codes of a lane's 8 values given inv = RN(1 / d).  kSigned: x holds m.  Otherwise x holds v, of
// which y = RN(RN(sqrt(v)) inv) is coded, and w its approximate root.  The candidate is the
// nearest integer to an approximate sqrt(y - 1/4), good to 1e-4 for k up to 255 (relative errors of
// 2^-22 each in root and product); only where that root lies within 2e-4 of a half is y formed
// exactly and the candidate checked against the borders.
constexpr float kMagic = 12582912.f;   // 1.5 * 2^23: adding it rounds to an integer in the low mantissa bits
template <bool kSigned>
__device__ __forceinline__ void encode8(const float *x, const float *w, float inv, uint32_t *c) {
    float t[8], off = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float r = sqrt_approx<true>(fmaxf(fmaf(kSigned ? fabsf(x[i]) : w[i], inv, -0.25f), 0.f));
        t[i] = __fadd_rn(r, kMagic);
        off = fmaxf(off, fabsf(r - __fsub_rn(t[i], kMagic)));
    }
    if (off > 0.4998f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float y = __fmul_rn(kSigned ? fabsf(x[i]) : __fsqrt_rn(x[i]), inv), k = __fsub_rn(t[i], kMagic);
            // k^2 + k + 1/2 is exact: at most 17 significant bits
            if (y > __fmaf_rn(k, k, k) + 0.5f) t[i] += 1.f;
            else if (k > 0.f && y <= __fmaf_rn(k, k, -k) + 0.5f) t[i] -= 1.f;
        }
    }
    if (kSigned) {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = __fadd_rn(copysignf(__fsub_rn(t[i], kMagic), x[i]), kMagic);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t lo = __byte_perm(__float_as_uint(t[4 * h]), __float_as_uint(t[4 * h + 1]), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(t[4 * h + 2]), __float_as_uint(t[4 * h + 3]), 0x0040);
        c[h] = __byte_perm(lo, hi, 0x5410);
    }
}

struct StepArgs {
    const Chunk *chunks;
    PlanHead *head;
    const float *coef;         // clip coefficient on the device, or NULL
    const float *lr_dev;       // learning rate on the device, or NULL
    int64_t *step_dev;         // number of steps taken, or NULL
    double beta1, beta2, eps;
    int64_t nchunks;
    float lr, b1, w1, b2, w2;  // w = 1 - b
    float ds, de;              // (1 - b1^t) / sqrt(1 - b2^t) and (1 - b1^t) eps
};

// b^t by squaring (t >= 1): at most 2 log2(t) products, each rounded in double
__device__ __forceinline__ double pow_int(double b, int64_t t) {
    double r = 1.0;
    for (; t > 0; t >>= 1, b *= b)
        if (t & 1) r *= b;
    return r;
}

// A chunk's addresses and settings, the same in every lane.
struct View {
    uint64_t p, copy, g, m, v, dm, dv;
    int n;
    uint32_t flags;
    float lr, decay;
};
__device__ __forceinline__ View view_of(uint32_t word, float lr) {
    View c;
    c.p = word64(word, 0), c.copy = word64(word, 2), c.g = word64(word, 4), c.m = word64(word, 6);
    c.v = word64(word, 8), c.dm = word64(word, 10), c.dv = word64(word, 12);
    c.n = static_cast<int>(word32(word, 14));
    c.flags = word32(word, 15);
    c.lr = lr * __uint_as_float(word32(word, 16));
    c.decay = __uint_as_float(word32(word, 17));
    return c;
}
// The step's scalars: denominators are (sqrt(v) ibc2 + eps) bc1 = sqrt(v) ds + de.
struct Scalars {
    float coef, ds, de;
};

// One block of 256 (kFull) or the rem < 256 last elements of a tensor.
template <bool kState8, bool kPBf16, bool kGBf16, bool kFull>
__device__ __forceinline__ void step_block(const StepArgs &a, const View &c, const Scalars &s, int64_t i0, int rem, int lane) {
    float g[8], p[8], m[8], v[8], w[8];
    uint32_t cm[2], cv[2];
    float dm = 0.f, dv = 0.f;
    if (kState8) {
        load_codes<kFull>(c.m, i0, rem, lane, cm);
        load_codes<kFull>(c.v, i0, rem, lane, cv);
        dm = reinterpret_cast<const float *>(c.dm)[i0 / kBlock];
        dv = reinterpret_cast<const float *>(c.dv)[i0 / kBlock];
    } else {
        load8<kFull>(c.m, false, i0, rem, lane, m);
        load8<kFull>(c.v, false, i0, rem, lane, v);
    }
    load8<kFull>(c.g, kGBf16, i0, rem, lane, g);
    load8<kFull>(c.p, kPBf16, i0, rem, lane, p);
    if (kState8) {
        decode8<true>(cm, dm, m);
        decode8<false>(cv, dv, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], v[i]);
    }
    uint32_t am = 0, av = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float gi = __fmul_rn(g[i], s.coef);
        m[i] = __fadd_rn(__fmul_rn(a.b1, m[i]), __fmul_rn(a.w1, gi));
        v[i] = __fadd_rn(__fmul_rn(a.b2, v[i]), __fmul_rn(a.w2, __fmul_rn(gi, gi)));
        w[i] = sqrt_approx<false>(v[i]);
        p[i] = fmaf(-c.lr, fmaf(c.decay, p[i], m[i] * rcp_approx(fmaf(w[i], s.ds, s.de))), p[i]);
        if (kState8 && (kFull || (i >> 2) * 128 + lane * 4 + (i & 3) < rem)) {
            am = max_bits(am, m[i]);
            av = max_bits(av, v[i]);
        }
    }
    store8<kFull>(c.p, kPBf16, i0, rem, lane, p);
    if (!kPBf16 && c.copy) store8<kFull>(c.copy, true, i0, rem, lane, p);
    if (kState8) {
        am = __reduce_max_sync(0xffffffffu, am);
        av = __reduce_max_sync(0xffffffffu, av);
        // the root is monotonic, so the largest root is the root of the largest v; even lanes work out m's
        // step and odd lanes sqrt(v)'s
        const bool odd = lane & 1;
        if (av < 0x7F800000u) av = __float_as_uint(__fsqrt_rn(__uint_as_float(av)));
        float d, inv;
        block_step(odd ? av : am, odd ? float(kTopW * kTopW) : float(kTopM * kTopM), d, inv);
        dm = __shfl_sync(0xffffffffu, d, 0);
        dv = __shfl_sync(0xffffffffu, d, 1);
        encode8<true>(m, nullptr, __shfl_sync(0xffffffffu, inv, 0), cm);
        encode8<false>(v, w, __shfl_sync(0xffffffffu, inv, 1), cv);
        store_codes<kFull>(c.m, i0, rem, lane, cm);
        store_codes<kFull>(c.v, i0, rem, lane, cv);
        if (lane == 0) {
            reinterpret_cast<float *>(c.dm)[i0 / kBlock] = dm;
            reinterpret_cast<float *>(c.dv)[i0 / kBlock] = dv;
        }
    } else {
        store8<kFull>(c.m, false, i0, rem, lane, m);
        store8<kFull>(c.v, false, i0, rem, lane, v);
    }
}
template <bool kState8, bool kPBf16, bool kGBf16>
__device__ __forceinline__ void step_chunk(const StepArgs &a, const View &c, const Scalars &s, int lane) {
    int i0 = 0;
    for (; i0 + kBlock <= c.n; i0 += kBlock) step_block<kState8, kPBf16, kGBf16, true>(a, c, s, i0, kBlock, lane);
    if (i0 < c.n) step_block<kState8, kPBf16, kGBf16, false>(a, c, s, i0, c.n - i0, lane);
}
template <bool kState8>
__device__ __forceinline__ void step_types(const StepArgs &a, const View &c, const Scalars &s, int lane) {
    switch (c.flags & (kParamBf16 | kGradBf16)) {
        case 0: step_chunk<kState8, false, false>(a, c, s, lane); break;
        case kParamBf16: step_chunk<kState8, true, false>(a, c, s, lane); break;
        case kGradBf16: step_chunk<kState8, false, true>(a, c, s, lane); break;
        default: step_chunk<kState8, true, true>(a, c, s, lane);
    }
}

// A warp takes every (warps of the grid)-th chunk, with the next chunk's 80 bytes already on
// their way; no barrier and no shared memory in the loop.  kKinds: the states the plan holds,
// kKind32 | kKind8.
enum { kKind32 = 1, kKind8 = 2 };
constexpr int kCtas32 = 4, kCtas8 = 3;      // CTAs per SM that the registers are capped for
template <int kKinds>
__global__ void __launch_bounds__(kThreads, kKinds == kKind32 ? kCtas32 : kCtas8) adamw_kernel(const StepArgs a) {
    __shared__ float s_bc[2];
    const int lane = threadIdx.x & 31;
    const int64_t nw = int64_t(gridDim.x) * kWarps;
    int64_t i = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    // the chunk list was complete when the plan's call returned: it may be read before the wait
    uint32_t word = i < a.nchunks ? chunk_word(a.chunks, i, lane) : 0u;
    pdl_launch_dependents();
    pdl_wait();
    Scalars s;
    s.coef = a.coef ? __ldcg(a.coef) : 1.f;          // a product with 1 changes nothing
    if (!isfinite(s.coef)) return;                   // the gradients held an infinity or a NaN: nothing changes
    const float lr = a.lr_dev ? __ldcg(a.lr_dev) : a.lr;
    s.ds = a.ds;
    s.de = a.de;
    if (a.step_dev) {
        if (threadIdx.x == 0) {
            const int64_t t = *a.step_dev + 1;
            const double bc1 = 1.0 - pow_int(a.beta1, t);
            s_bc[0] = static_cast<float>(bc1 / sqrt(1.0 - pow_int(a.beta2, t)));
            s_bc[1] = static_cast<float>(bc1 * a.eps);
        }
        __syncthreads();
        s.ds = s_bc[0];
        s.de = s_bc[1];
    }
    for (; i < a.nchunks; i += nw) {
        const View c = view_of(word, lr);
        if (i + nw < a.nchunks) word = chunk_word(a.chunks, i + nw, lane);
        if (kKinds == kKind32 || (kKinds != kKind8 && !(c.flags & kState8))) step_types<false>(a, c, s, lane);
        else step_types<true>(a, c, s, lane);
    }
    if (a.step_dev) {
        // the last CTA to get here counts the step: every CTA has read the counter by then
        __syncthreads();
        if (threadIdx.x == 0) {
            __threadfence();
            if (atomicAdd(&a.head->ticket, 1u) == gridDim.x - 1) {
                a.head->ticket = 0;
                *a.step_dev += 1;
            }
        }
    }
}

// Sum of squares of every gradient: each lane sums in double (a float32 square overflows at
// 1.8e19 and loses what lies below 1e-19), each CTA leaves one partial sum, and the last CTA
// adds the partials in a fixed order.  Chunks are dealt to warps by index, so the result
// depends on the plan and the number of SMs only.
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const Chunk *chunks, PlanHead *head, int64_t nchunks,
                                                             float max_norm, float *out) {
    __shared__ double s_sum[kWarps];
    __shared__ bool s_last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t nw = int64_t(gridDim.x) * kWarps;
    int64_t c = int64_t(blockIdx.x) * kWarps + warp;
    uint32_t word = c < nchunks ? chunk_word(chunks, c, lane) : 0u;
    pdl_launch_dependents();
    pdl_wait();
    double sum = 0.0;
    for (; c < nchunks; c += nw) {
        const uint64_t G = word64(word, 4);
        const int n = static_cast<int>(word32(word, 14));
        const bool bf16 = (word32(word, 15) & kGradBf16) != 0;
        if (c + nw < nchunks) word = chunk_word(chunks, c + nw, lane);
        for (int i0 = 0; i0 < n; i0 += kBlock) {
            float g[8];
            if (n - i0 >= kBlock) load8<true>(G, bf16, i0, n - i0, lane, g);
            else load8<false>(G, bf16, i0, n - i0, lane, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fma(double(g[i]), double(g[i]), sum);
        }
    }
    auto block_sum = [&](double x) {   // the sum of all threads' x, in thread 0
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        __syncthreads();
        if (lane == 0) s_sum[warp] = x;
        __syncthreads();
        double t = 0.0;
        if (threadIdx.x == 0)
            for (int i = 0; i < kWarps; ++i) t += s_sum[i];
        return t;
    };
    const double mine = block_sum(sum);
    if (threadIdx.x == 0) {
        head->partial[blockIdx.x] = mine;
        __threadfence();
        s_last = atomicAdd(&head->ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    double x = 0.0;
    for (int i = threadIdx.x; i < int(gridDim.x); i += kThreads) x += __ldcg(&head->partial[i]);
    const double total = block_sum(x);
    if (threadIdx.x == 0) {
        head->ticket = 0;
        const double norm = sqrt(total);
        const double coef = double(max_norm) / (norm + 1e-6);
        out[0] = static_cast<float>(norm);
        // a norm that is not finite gives NaN, which the step takes as "change nothing"
        out[1] = isfinite(norm) ? static_cast<float>(coef < 1.0 ? coef : 1.0) : __uint_as_float(0x7FC00000u);
    }
}

// 8-bit state from float32 moments, and back.  kSecond: x is the second moment v, coded by
// its root, and comes back as the square of the decoded root.
template <bool kSecond>
__global__ void __launch_bounds__(kThreads) adam8_encode_kernel(const float *x, uint8_t *codes, float *steps, int64_t n) {
    const int lane = threadIdx.x & 31;
    const int64_t nblk = (n + kBlock - 1) / kBlock;
    pdl_launch_dependents();
    pdl_wait();
    for (int64_t b = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); b < nblk; b += int64_t(gridDim.x) * kWarps) {
        const int rem = static_cast<int>(n - b * kBlock < kBlock ? n - b * kBlock : kBlock);
        const uint64_t src = reinterpret_cast<uint64_t>(x), dst = reinterpret_cast<uint64_t>(codes);
        float f[8];
        if (rem == kBlock) load8<true>(src, false, b * kBlock, rem, lane, f);
        else load8<false>(src, false, b * kBlock, rem, lane, f);
        uint32_t c[2], top = 0;
        float w[8], d, inv;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (kSecond) f[i] += 0.f;                       // -0 becomes 0
            // a negative v has no root: its sign bit puts it above infinity here, with the NaNs
            top = max(top, __float_as_uint(f[i]) & (kSecond ? 0xFFFFFFFFu : 0x7FFFFFFFu));
            w[i] = sqrt_approx<false>(f[i]);
        }
        top = __reduce_max_sync(0xffffffffu, top);
        if (kSecond && top < 0x7F800000u) top = __float_as_uint(__fsqrt_rn(__uint_as_float(top)));
        block_step(top, kSecond ? float(kTopW * kTopW) : float(kTopM * kTopM), d, inv);
        encode8<!kSecond>(f, w, inv, c);
        if (rem == kBlock) store_codes<true>(dst, b * kBlock, rem, lane, c);
        else store_codes<false>(dst, b * kBlock, rem, lane, c);
        if (lane == 0) steps[b] = d;
    }
}
template <bool kSecond>
__global__ void __launch_bounds__(kThreads) adam8_decode_kernel(const uint8_t *codes, const float *steps, float *x, int64_t n) {
    const int lane = threadIdx.x & 31;
    const int64_t nblk = (n + kBlock - 1) / kBlock;
    pdl_launch_dependents();
    pdl_wait();
    for (int64_t b = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); b < nblk; b += int64_t(gridDim.x) * kWarps) {
        const int rem = static_cast<int>(n - b * kBlock < kBlock ? n - b * kBlock : kBlock);
        const uint64_t src = reinterpret_cast<uint64_t>(codes), dst = reinterpret_cast<uint64_t>(x);
        uint32_t c[2];
        if (rem == kBlock) load_codes<true>(src, b * kBlock, rem, lane, c);
        else load_codes<false>(src, b * kBlock, rem, lane, c);
        float f[8];
        decode8<!kSecond>(c, __ldcg(steps + b), f);
        if (kSecond) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __fmul_rn(f[i], f[i]);
        }
        if (rem == kBlock) store8<true>(dst, false, b * kBlock, rem, lane, f);
        else store8<false>(dst, false, b * kBlock, rem, lane, f);
    }
}

}  // namespace optim
}  // namespace qlora
