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
// Codes of a lane's 8 values x (signed m, or sqrt(v) >= 0) and the block's step d.  The
// candidate is the square root's nearest integer; only where the root lies within 2e-4 of a
// half (the approximate root is good to 4e-5 there) is it checked against the exact border.
template <bool kSigned>
__device__ __forceinline__ float encode8(const float *x, uint32_t *c) {
    constexpr float kTop2 = kSigned ? float(kTopM * kTopM) : float(kTopW * kTopW);
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    a = __reduce_max_sync(0xffffffffu, a);
    float d = 0.f, inv = 0.f;
    if (a >= 0x7F800000u) {
        d = __uint_as_float(0x7FC00000u);
    } else {
        d = __fdiv_rn(__uint_as_float(a), kTop2);
        if (d < 1.17549435e-38f) d = 0.f;
        else inv = __frcp_rn(d);
    }
    constexpr float kMagic = 12582912.f;   // 1.5 * 2^23: adding it rounds to an integer in the low bits
    float y[8], k[8], off = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = __fmul_rn(fabsf(x[i]), inv);
        float r;
        asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(fmaxf(__fsub_rn(y[i], 0.25f), 0.f)));
        k[i] = __fsub_rn(__fadd_rn(r, kMagic), kMagic);
        off = fmaxf(off, fabsf(r - k[i]));
    }
    if (off > 0.4998f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // k^2 + k + 1/2 is exact: at most 17 significant bits
            if (y[i] > __fmaf_rn(k[i], k[i], k[i]) + 0.5f) k[i] += 1.f;
            else if (k[i] > 0.f && y[i] <= __fmaf_rn(k[i], k[i], -k[i]) + 0.5f) k[i] -= 1.f;
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float s = kSigned ? copysignf(k[4 * h + j], x[4 * h + j]) : k[4 * h + j];
            b[j] = __float_as_uint(__fadd_rn(s, kMagic));
        }
        c[h] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    }
    return d;
}

struct StepArgs {
    const Chunk *chunks;
    PlanHead *head;
    const float *coef;         // clip coefficient on the device, or NULL
    const float *lr_dev;       // learning rate on the device, or NULL
    int64_t *step_dev;         // number of steps taken, or NULL
    double beta1, beta2;
    int64_t nchunks;
    float lr, b1, w1, b2, w2, eps, ibc1, ibc2;   // w = 1 - b; ibc1 = 1/(1 - b1^t), ibc2 = 1/sqrt(1 - b2^t)
};

// b^t by squaring (t >= 1): at most 2 log2(t) products, each rounded in double
__device__ __forceinline__ double pow_int(double b, int64_t t) {
    double r = 1.0;
    for (; t > 0; t >>= 1, b *= b)
        if (t & 1) r *= b;
    return r;
}

template <bool kState8, bool kFull>
__device__ __forceinline__ void step_block(const StepArgs &a, uint64_t P, uint64_t copy, uint64_t G, uint64_t Mo,
                                           uint64_t Vo, uint64_t DM, uint64_t DV, uint32_t flags, float lr, float decay,
                                           float coef, float ibc1, float ibc2, int64_t i0, int rem, int lane) {
    float g[8], p[8], m[8], v[8];
    uint32_t cm[2], cv[2];
    float dm = 0.f, dv = 0.f;
    load8<kFull>(G, (flags & kGradBf16) != 0, i0, rem, lane, g);
    load8<kFull>(P, (flags & kParamBf16) != 0, i0, rem, lane, p);
    if (kState8) {
        load_codes<kFull>(Mo, i0, rem, lane, cm);
        load_codes<kFull>(Vo, i0, rem, lane, cv);
        dm = reinterpret_cast<const float *>(DM)[i0 / kBlock];
        dv = reinterpret_cast<const float *>(DV)[i0 / kBlock];
        decode8<true>(cm, dm, m);
        decode8<false>(cv, dv, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], v[i]);
    } else {
        load8<kFull>(Mo, false, i0, rem, lane, m);
        load8<kFull>(Vo, false, i0, rem, lane, v);
    }
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float gi = a.coef ? __fmul_rn(g[i], coef) : g[i];
        m[i] = __fadd_rn(__fmul_rn(a.b1, m[i]), __fmul_rn(a.w1, gi));
        v[i] = __fadd_rn(__fmul_rn(a.b2, v[i]), __fmul_rn(a.w2, __fmul_rn(gi, gi)));
        w[i] = __fsqrt_rn(v[i]);
        const float u = __fdividef(m[i] * ibc1, fmaf(w[i], ibc2, a.eps));
        p[i] = fmaf(-lr, fmaf(decay, p[i], u), p[i]);
    }
    store8<kFull>(P, (flags & kParamBf16) != 0, i0, rem, lane, p);
    if (copy) store8<kFull>(copy, true, i0, rem, lane, p);
    if (kState8) {
        if (!kFull) {   // places past the tensor's end take no part in the block's largest value
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if ((i >> 2) * 128 + lane * 4 + (i & 3) >= rem) m[i] = w[i] = 0.f;
        }
        dm = encode8<true>(m, cm);
        dv = encode8<false>(w, cv);
        store_codes<kFull>(Mo, i0, rem, lane, cm);
        store_codes<kFull>(Vo, i0, rem, lane, cv);
        if (lane == 0) {
            reinterpret_cast<float *>(DM)[i0 / kBlock] = dm;
            reinterpret_cast<float *>(DV)[i0 / kBlock] = dv;
        }
    } else {
        store8<kFull>(Mo, false, i0, rem, lane, m);
        store8<kFull>(Vo, false, i0, rem, lane, v);
    }
}

// A warp takes every (warps of the grid)-th chunk, with the next chunk's 80 bytes already on
// their way; no barrier and no shared memory in the loop.
__global__ void __launch_bounds__(kThreads) adamw_kernel(const StepArgs a) {
    __shared__ float s_bc[2];
    const int lane = threadIdx.x & 31;
    const int64_t nw = int64_t(gridDim.x) * kWarps;
    int64_t c = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    uint32_t word = c < a.nchunks ? chunk_word(a.chunks, c, lane) : 0u;
    const float coef = a.coef ? __ldg(a.coef) : 1.f;
    if (!isfinite(coef)) return;          // the gradients held an infinity or a NaN: nothing changes
    const float lr = a.lr_dev ? __ldg(a.lr_dev) : a.lr;
    float ibc1 = a.ibc1, ibc2 = a.ibc2;
    if (a.step_dev) {
        if (threadIdx.x == 0) {
            const int64_t t = *a.step_dev + 1;
            s_bc[0] = static_cast<float>(1.0 / (1.0 - pow_int(a.beta1, t)));
            s_bc[1] = static_cast<float>(1.0 / sqrt(1.0 - pow_int(a.beta2, t)));
        }
        __syncthreads();
        ibc1 = s_bc[0];
        ibc2 = s_bc[1];
    }
    for (; c < a.nchunks; c += nw) {
        const uint64_t P = word64(word, 0), copy = word64(word, 2), G = word64(word, 4), Mo = word64(word, 6),
                       Vo = word64(word, 8), DM = word64(word, 10), DV = word64(word, 12);
        const int n = static_cast<int>(word32(word, 14));
        const uint32_t flags = word32(word, 15);
        const float lrc = lr * __uint_as_float(word32(word, 16)), decay = __uint_as_float(word32(word, 17));
        if (c + nw < a.nchunks) word = chunk_word(a.chunks, c + nw, lane);
        for (int i0 = 0; i0 < n; i0 += kBlock) {
            const int rem = n - i0;
            if (flags & kState8) {
                if (rem >= kBlock)
                    step_block<true, true>(a, P, copy, G, Mo, Vo, DM, DV, flags, lrc, decay, coef, ibc1, ibc2, i0, rem, lane);
                else
                    step_block<true, false>(a, P, copy, G, Mo, Vo, DM, DV, flags, lrc, decay, coef, ibc1, ibc2, i0, rem, lane);
            } else {
                if (rem >= kBlock)
                    step_block<false, true>(a, P, copy, G, Mo, Vo, DM, DV, flags, lrc, decay, coef, ibc1, ibc2, i0, rem, lane);
                else
                    step_block<false, false>(a, P, copy, G, Mo, Vo, DM, DV, flags, lrc, decay, coef, ibc1, ibc2, i0, rem, lane);
            }
        }
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
__global__ void __launch_bounds__(kThreads) adam8_encode_kernel(const float *__restrict__ x, uint8_t *__restrict__ codes,
                                                                float *__restrict__ steps, int64_t n) {
    const int lane = threadIdx.x & 31;
    const int64_t nblk = (n + kBlock - 1) / kBlock;
    for (int64_t b = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); b < nblk; b += int64_t(gridDim.x) * kWarps) {
        const int rem = static_cast<int>(n - b * kBlock < kBlock ? n - b * kBlock : kBlock);
        const uint64_t src = reinterpret_cast<uint64_t>(x), dst = reinterpret_cast<uint64_t>(codes);
        float f[8];
        if (rem == kBlock) load8<true>(src, false, b * kBlock, rem, lane, f);
        else load8<false>(src, false, b * kBlock, rem, lane, f);
        if (kSecond) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __fsqrt_rn(f[i]);
        }
        uint32_t c[2];
        const float d = encode8<!kSecond>(f, c);
        if (rem == kBlock) store_codes<true>(dst, b * kBlock, rem, lane, c);
        else store_codes<false>(dst, b * kBlock, rem, lane, c);
        if (lane == 0) steps[b] = d;
    }
}
template <bool kSecond>
__global__ void __launch_bounds__(kThreads) adam8_decode_kernel(const uint8_t *__restrict__ codes,
                                                                const float *__restrict__ steps, float *__restrict__ x,
                                                                int64_t n) {
    const int lane = threadIdx.x & 31;
    const int64_t nblk = (n + kBlock - 1) / kBlock;
    for (int64_t b = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); b < nblk; b += int64_t(gridDim.x) * kWarps) {
        const int rem = static_cast<int>(n - b * kBlock < kBlock ? n - b * kBlock : kBlock);
        const uint64_t src = reinterpret_cast<uint64_t>(codes), dst = reinterpret_cast<uint64_t>(x);
        uint32_t c[2];
        if (rem == kBlock) load_codes<true>(src, b * kBlock, rem, lane, c);
        else load_codes<false>(src, b * kBlock, rem, lane, c);
        float f[8];
        decode8<!kSecond>(c, __ldg(steps + b), f);
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
