// optimizer.cuh -- AdamW over many tensors in one launch (states in 32 bits or in 8 bits),
// the global gradient norm with its clip coefficient, and the 8-bit state code.
//
// One step, per element:
//   g = grad (* clip coefficient)
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2
//   p = p - lr (decay p + (m / (1 - b1^t)) / (sqrt(v) / sqrt(1 - b2^t) + eps))
// g, m and v are rounded to float32 operation by operation.  p takes an approximate root and reciprocal (2^-23 each),
// denominators sqrt(v) ds + de with the corrections worked out beforehand, and fused multiply-adds: at most 11 half steps
// of float32 relative to lr (|decay p| + |u|) before its own rounding, 16 in the interface.
//
// 8-bit states: blocks of 256 values with one fp32 step d each, value = k |k| d, where x is
// m (k in -127 .. 127) or sqrt(v) (k in 0 .. 255; the second moment is the value's square).
//   d = RN(max |x| / K^2), K = 127 or 255;  y = RN(|x| RN(1 / d));
//   |k| = #{j : y > j^2 + j + 1/2}, the square nearest to y, ties to the lower k.
// Evenly spaced roots resolve a block's small values (smallest 1/16129 and 1/65025 of the
// block's largest) at a bounded cost for its large ones (half a step is 0.8 % and 0.4 % at
// the top).  sqrt(v) is stored, not v, so that m and the denominator keep the same range.
// All roundings up to the code are fixed (no fused multiply-add), so codes are bit-exact.
// A block with a non-finite value (or a negative v) stores d = NaN and k = 0: every later step on it is NaN.
// d below 2^-126, where 1 / d could overflow, is stored as 0 with k = 0.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "step_common.cuh"

namespace qlora {
namespace optim {

constexpr int kBlock = 256;          // values per 8-bit block: one warp step, 8 per lane
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPartials = 4096;      // most CTAs of the norm: slots for their partial sums
constexpr int kTopM = 127, kTopW = 255;

enum : uint32_t { kParamBf16 = 1, kGradBf16 = 2 };

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

// Head of the plan buffer: the CTA ticket of the norm (left at zero), the scalars of a step counted on
// the device, and the norm's partial sums.
struct alignas(256) PlanHead {
    unsigned int ticket;
    float ds, de;
    unsigned int unused[61];
    double partial[kPartials];
};

// A tensor of a plan as the host hands it over: its first chunk (n not set), where its chunks begin in the list,
// and the bytes of an element of p, g and the states.
struct TensorDesc {
    Chunk base;
    int64_t numel, first;
    int32_t pb, gb, sb, unused;
};
// Writes the chunk list: a thread a chunk, which finds its tensor by the first chunk of each (ascending).
__global__ void __launch_bounds__(kThreads) expand_plan_kernel(const TensorDesc *ts, int count, int chunk, int64_t nchunks, Chunk *out) {
    const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= nchunks) return;
    int lo = 0, hi = count;                       // ts[lo].first <= i < ts[hi].first
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (ts[mid].first <= i) lo = mid;
        else hi = mid;
    }
    const TensorDesc &t = ts[lo];
    const int64_t e = (i - t.first) * chunk;
    Chunk c = t.base;
    c.n = static_cast<int32_t>(min(int64_t(chunk), t.numel - e));
    c.g += uint64_t(e) * t.gb;
    if (c.p) c.p += uint64_t(e) * t.pb;
    if (c.copy) c.copy += uint64_t(e) * 2;
    if (c.m) c.m += uint64_t(e) * t.sb;
    if (c.v) c.v += uint64_t(e) * t.sb;
    if (c.dm) c.dm += uint64_t(e / kBlock) * 4;
    if (c.dv) c.dv += uint64_t(e / kBlock) * 4;
    out[i] = c;
}

__device__ __forceinline__ uint32_t chunk_word(const Chunk *chunks, int64_t c, int lane) {
    return lane < 20 ? __ldg(reinterpret_cast<const uint32_t *>(chunks + c) + lane) : 0u;
}
__device__ __forceinline__ uint32_t word32(uint32_t w, int i) { return __shfl_sync(0xffffffffu, w, i); }
__device__ __forceinline__ uint64_t word64(uint32_t w, int i) {
    return uint64_t(word32(w, i)) | (uint64_t(word32(w, i + 1)) << 32);
}

// Element of half h (0, 1) and place j (0..3) of a lane's 8 in a block: h * 128 + lane * 4 + j.
// rem: elements of the chunk from the block's first on.  kFull: rem >= 256.
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

// Bytes j and j + 1 of w as floats k: a byte becomes the low mantissa byte of 2^23 (one permute each and
// one exact subtraction; no integer conversion, whose pipe is eight times narrower)
template <bool kSigned>
__device__ __forceinline__ uint64_t code_pair(uint32_t w, int j) {
    const uint32_t u = kSigned ? w ^ 0x80808080u : w;
    const float magic = kSigned ? -8388736.f : -8388608.f;   // -(2^23 (+ 128))
    return add2(pack2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7650 + j)),
                      __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7651 + j))), pack2(magic, magic));
}
// A lane's 8 values as 4 pairs: k |k| d, or the square of k^2 d
template <bool kSecond>
__device__ __forceinline__ void decode8(const uint32_t *c, float d, uint64_t *x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t k = code_pair<!kSecond>(c[i >> 1], 2 * (i & 1));
        if (kSecond) {
            const uint64_t w = mul2(mul2(k, k), pack2(d, d));
            x[i] = mul2(w, w);
        } else {
            float a, b;
            unpack2(k, a, b);
            x[i] = mul2(pack2(__fmul_rn(a, fabsf(a)), __fmul_rn(b, fabsf(b))), pack2(d, d));
        }
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
// the larger of a and |x|; a NaN once seen stays
__device__ __forceinline__ float max_nan(float a, float x) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(x)));
    return r;
}

// A block's step d = RN(a / top^2) from its largest magnitude a, and RN(1 / d)
__device__ __forceinline__ void block_step(float a, float top2, float &d, float &inv) {
    d = __fdiv_rn(a, top2);
    inv = __frcp_rn(d);
    if (d < 1.17549435e-38f) d = 0.f, inv = 0.f;
    if (!(a < INFINITY)) d = __uint_as_float(0x7FC00000u), inv = 0.f;
}

// Codes of a lane's 8 values given inv = RN(1 / d).  kSecond = false: x holds m.  Otherwise x holds v, of
// which y = RN(RN(sqrt(v)) inv) is coded, and w its approximate root.  The candidate is the
// nearest integer to an approximate sqrt(y - 1/4): relative errors of 2^-23 for w and for the root and 2^-24 for
// the product put it within 255 * 1.75 * 2^-23 = 5.4e-5 (m: 127 * 1.25 * 2^-23 = 1.9e-5).  Only where that root lies
// closer to a half is y formed exactly and the candidate checked against the borders: in 3 % (m: 1 %) of
// the blocks, for the elements concerned.  (y - 1/4) / 4^8 (m: / 4^7) is in [0, 1), so one saturating
// multiply-add clamps what is below 1/4, and a NaN, to zero.
constexpr float kMagic = 12582912.f;   // 1.5 * 2^23: adding it rounds to an integer in the low mantissa bits
__device__ __forceinline__ float fma_sat(float a, float b, float c) {
    float r;
    asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
template <bool kSecond>
__device__ __forceinline__ void encode8(const float *x, const float *w, float inv, bool exact, uint32_t *c) {
    constexpr float kNear = kSecond ? 0.49994f : 0.499975f, kRoot = kSecond ? 256.f : 128.f;
    uint32_t t[8];
    float e[8];
    // below 2^-100 the scaled reciprocal could lose bits
    exact = exact || inv < 7.8886091e-31f;
    float off = exact && inv > 0.f ? 1.f : 0.f;
    const float scaled = inv * (1.f / (kRoot * kRoot));
    const uint64_t root = pack2(kRoot, kRoot), magic = pack2(kMagic, kMagic), minus = pack2(-1.f, -1.f);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        float z0 = sqrt_approx<true>(fma_sat(kSecond ? w[i] : fabsf(x[i]), scaled, -0.25f / (kRoot * kRoot)));
        float z1 = sqrt_approx<true>(fma_sat(kSecond ? w[i + 1] : fabsf(x[i + 1]), scaled, -0.25f / (kRoot * kRoot)));
        if (!kSecond) {
            z0 = copysignf(z0, x[i]);
            z1 = copysignf(z1, x[i + 1]);
        }
        const uint64_t z = pack2(z0, z1), r = fma2(z, root, magic);
        float r0, r1;
        unpack2(r, r0, r1);
        unpack2(fma2(z, root, fma2(r, minus, magic)), e[i], e[i + 1]);    // root z - (r - magic)
        off = fmaxf(off, fmaxf(fabsf(e[i]), fabsf(e[i + 1])));
        t[i] = __float_as_uint(r0);
        t[i + 1] = __float_as_uint(r1);
    }
    if (__any_sync(0xffffffffu, off > kNear)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (!__any_sync(0xffffffffu, exact || fabsf(e[i]) > kNear)) continue;
            const float y = __fmul_rn(kSecond ? __fsqrt_rn(x[i]) : fabsf(x[i]), inv);
            float k = rintf(sqrt_approx<true>(fmaxf(__fsub_rn(y, 0.25f), 0.f)));
            // k^2 + k + 1/2 is exact: at most 17 significant bits
            if (y > __fmaf_rn(k, k, k) + 0.5f) k += 1.f;
            else if (k > 0.f && y <= __fmaf_rn(k, k, -k) + 0.5f) k -= 1.f;
            t[i] = __float_as_uint(__fadd_rn(kSecond ? k : copysignf(k, x[i]), kMagic));
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
        c[h] = __byte_perm(__byte_perm(t[4 * h], t[4 * h + 1], 0x0040), __byte_perm(t[4 * h + 2], t[4 * h + 3], 0x0040), 0x5410);
}

struct StepArgs {
    const Chunk *chunks;
    const PlanHead *head;
    const float *coef;         // clip coefficient on the device, or NULL
    const float *lr_dev;       // learning rate on the device, or NULL
    int counted;               // 1: ds and de are in the head (step_scalars_kernel)
    int nchunks;
    uint64_t b1, w1, b2, w2;   // pairs of b and w = 1 - b
    uint64_t one;              // a pair of 1, as a value that the compiler does not know
    float lr;
    float ds, de;              // (1 - b1^t) / sqrt(1 - b2^t) and (1 - b1^t) eps
};

// b^t by squaring (t >= 1): at most 2 log2(t) products, each rounded in double
__device__ __forceinline__ double pow_int(double b, int64_t t) {
    double r = 1.0;
    for (; t > 0; t >>= 1, b *= b)
        if (t & 1) r *= b;
    return r;
}
// The scalars of a step whose number is kept on the device, and the count of it (one thread): a launch of
// its own, because worked out by every CTA it cost each of them about 0.5 us of double-precision latency.
__global__ void step_scalars_kernel(PlanHead *head, int64_t *step_dev, const float *coef, double beta1, double beta2, double eps) {
    pdl_launch_dependents();
    pdl_wait();
    if (coef && !isfinite(__ldcg(coef))) return;
    const int64_t t = *step_dev + 1;
    *step_dev = t;
    const double bc1 = 1.0 - pow_int(beta1, t);
    head->ds = static_cast<float>(bc1 / sqrt(1.0 - pow_int(beta2, t)));
    head->de = static_cast<float>(bc1 * eps);
}

// The step's scalars: denominators are (sqrt(v) ibc2 + eps) bc1 = sqrt(v) ds + de.  flush: the root may take
// a v below 2^-126 as zero (its root, at most 1.1e-19, is then under 2^-24 of the denominator).
struct Scalars {
    float coef, lr, ds, de;
    bool flush;
};
// false: the gradients held an infinity or a NaN, and nothing changes
__device__ __forceinline__ bool read_scalars(const StepArgs &a, Scalars &s) {
    s.coef = a.coef ? __ldcg(a.coef) : 1.f;          // a product with 1 changes nothing
    s.lr = a.lr_dev ? __ldcg(a.lr_dev) : a.lr;
    s.ds = a.counted ? __ldcg(&a.head->ds) : a.ds;
    s.de = a.counted ? __ldcg(&a.head->de) : a.de;
    s.flush = s.de >= 2e-12f * s.ds;
    return isfinite(s.coef);
}

// A lane's 8 elements of a block of a parameter or gradient as loaded: what is not used yet takes no
// conversion, so that a block's loads are all issued before the first of them is waited for.
template <bool kBf16>
struct Raw8 {
    uint32_t w[kBf16 ? 4 : 8];
    template <bool kFull>
    __device__ __forceinline__ void load(uint64_t base, int64_t i0, int rem, int lane) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int e = h * 128 + lane * 4;
            if (kFull && kBf16) {
                const uint2 x = *reinterpret_cast<const uint2 *>(base + 2 * (i0 + e));
                w[2 * h] = x.x, w[2 * h + 1] = x.y;
            } else if (kFull) {
                const uint4 x = *reinterpret_cast<const uint4 *>(base + 4 * (i0 + e));
                w[4 * h] = x.x, w[4 * h + 1] = x.y, w[(4 * h + 2) % (kBf16 ? 4 : 8)] = x.z, w[(4 * h + 3) % (kBf16 ? 4 : 8)] = x.w;
            } else {
                uint32_t x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[j] = 0;
                    if (e + j < rem)
                        x[j] = kBf16 ? uint32_t(reinterpret_cast<const uint16_t *>(base)[i0 + e + j])
                                     : reinterpret_cast<const uint32_t *>(base)[i0 + e + j];
                }
                if (kBf16) {
                    w[2 * h] = x[0] | (x[1] << 16), w[2 * h + 1] = x[2] | (x[3] << 16);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[(4 * h + j) % (kBf16 ? 4 : 8)] = x[j];
                }
            }
        }
    }
    // elements 2 i and 2 i + 1
    __device__ __forceinline__ uint64_t pair(int i) const {
        if (kBf16) return pack2(__uint_as_float(w[i % 4] << 16), __uint_as_float(w[i % 4] & 0xFFFF0000u));
        return pack2(__uint_as_float(w[(2 * i) % (kBf16 ? 4 : 8)]), __uint_as_float(w[(2 * i + 1) % (kBf16 ? 4 : 8)]));
    }
};

// The moments of pair i and the parameters, from g and the old moments.  Products and sums of the moments are
// rounded one by one: the sum is a product with the argument `one`, because a plain paired product and
// sum were merged into one rounding by the assembler (codes then differed).
__device__ __forceinline__ void moments(const StepArgs &a, const Scalars &s, uint64_t g, uint64_t &m, uint64_t &v) {
    g = mul2(g, pack2(s.coef, s.coef));
    m = fma2(mul2(a.b1, m), a.one, mul2(a.w1, g));
    v = fma2(mul2(a.b2, v), a.one, mul2(a.w2, mul2(g, g)));
}
// the approximate roots w of a lane's 8 second moments
__device__ __forceinline__ void roots(const Scalars &s, const float *v, float *w) {
    if (s.flush) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = sqrt_approx<true>(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = sqrt_approx<false>(v[i]);
    }
}
// minus_lr, decay: pairs
__device__ __forceinline__ uint64_t update(const Scalars &s, uint64_t minus_lr, uint64_t decay, uint64_t p, uint64_t m, float w0, float w1) {
    float d0, d1;
    unpack2(fma2(pack2(w0, w1), pack2(s.ds, s.ds), pack2(s.de, s.de)), d0, d1);
    const uint64_t u = mul2(m, pack2(rcp_approx(d0), rcp_approx(d1)));
    return fma2(minus_lr, fma2(decay, p, u), p);
}

// ---- 32-bit states: 30 bytes per fp32 parameter, bound by HBM.
template <bool kPBf16, bool kGBf16, bool kFull>
__device__ __forceinline__ void step32_block(const StepArgs &a, const Scalars &s, const Chunk &c, int i0, int rem, int lane) {
    Raw8<kGBf16> g;
    Raw8<kPBf16> p;
    Raw8<false> m, v;
    m.template load<kFull>(c.m, i0, rem, lane);
    v.template load<kFull>(c.v, i0, rem, lane);
    g.template load<kFull>(c.g, i0, rem, lane);
    p.template load<kFull>(c.p, i0, rem, lane);
    float mf[8], vf[8], w[8], pf[8];
    uint64_t mp[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint64_t vp = v.pair(i);
        mp[i] = m.pair(i);
        moments(a, s, g.pair(i), mp[i], vp);
        unpack2(mp[i], mf[2 * i], mf[2 * i + 1]);
        unpack2(vp, vf[2 * i], vf[2 * i + 1]);
    }
    roots(s, vf, w);
    const float lr = -(s.lr * c.lr_scale);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        unpack2(update(s, pack2(lr, lr), pack2(c.decay, c.decay), p.pair(i), mp[i], w[2 * i], w[2 * i + 1]), pf[2 * i], pf[2 * i + 1]);
    store8<kFull>(c.p, kPBf16, i0, rem, lane, pf);
    if (!kPBf16 && c.copy) store8<kFull>(c.copy, true, i0, rem, lane, pf);
    store8<kFull>(c.m, false, i0, rem, lane, mf);
    store8<kFull>(c.v, false, i0, rem, lane, vf);
}
template <bool kPBf16, bool kGBf16>
__device__ __forceinline__ void step32_chunk(const StepArgs &a, const Scalars &s, const Chunk &c, int lane) {
    int i0 = 0;
    for (; i0 + kBlock <= c.n; i0 += kBlock) step32_block<kPBf16, kGBf16, true>(a, s, c, i0, kBlock, lane);
    if (i0 < c.n) step32_block<kPBf16, kGBf16, false>(a, s, c, i0, c.n - i0, lane);
}
// A warp takes one chunk, and the CTAs come in the order of the list: what is read and written at any time
// lies close together, which HBM rewards (a grid of four CTAs per SM that strides over the list took 631 us
// where this takes 583, on 129 M fp32 parameters with bf16 copies).
__global__ void __launch_bounds__(kThreads, 4) adamw32_kernel(const StepArgs a) {
    const int lane = threadIdx.x & 31;
    const int i = blockIdx.x * kWarps + (threadIdx.x >> 5);
    // the chunk list was complete when the plan's call returned: it may be read before the wait
    const uint32_t word = i < a.nchunks ? chunk_word(a.chunks, i, lane) : 0u;
    pdl_launch_dependents();
    pdl_wait();
    Scalars s;
    if (!read_scalars(a, s) || i >= a.nchunks) return;
    Chunk c;
    c.p = word64(word, 0), c.copy = word64(word, 2), c.g = word64(word, 4), c.m = word64(word, 6), c.v = word64(word, 8);
    c.n = static_cast<int>(word32(word, 14)), c.flags = word32(word, 15);
    c.lr_scale = __uint_as_float(word32(word, 16)), c.decay = __uint_as_float(word32(word, 17));
    switch (c.flags & (kParamBf16 | kGradBf16)) {
        case 0: step32_chunk<false, false>(a, s, c, lane); break;
        case kParamBf16: step32_chunk<true, false>(a, s, c, lane); break;
        case kGradBf16: step32_chunk<false, true>(a, s, c, lane); break;
        default: step32_chunk<true, true>(a, s, c, lane);
    }
}

// ---- 8-bit states: 10 to 18 bytes per parameter.  A step takes 62 instructions per parameter, which take longer than HBM
// (69 % of the issue slots used at 24 warps an SM), and a block's dependent chain (absmax, division, root, code) is as
// long as a load.  So each warp streams its elements through two stages of 512 in shared memory by
// asynchronous copies, one stage ahead of the two blocks it works on.  A lane copies exactly what it reads
// back itself, so the ring needs no barrier; copies past a tensor's end are zero-filled.
constexpr int kUnit = 2 * kBlock;
constexpr int kSlots = 4;                                  // chunks between the unit worked on and the one copied
// A chunk at hand, in the warp's shared memory: the list's 80 bytes, and its rate and decay as pairs.
struct alignas(16) Slot {
    Chunk c;
    uint64_t minus_lr, decay;
};
// elem: bytes of g, p, m and v of the plan's widest element (6, 8 or 10)
constexpr int step8_smem(int elem) { return kWarps * (2 * kUnit * elem + kSlots * int(sizeof(Slot))); }

template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t dst, uint64_t src) {
    if (kBytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else if (kBytes == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
template <int kBytes>
__device__ __forceinline__ void copy_async_part(uint32_t dst, uint64_t src, int bytes) {
    if (kBytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
    else if (kBytes == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// a lane's four runs of four elements (kSize bytes each) of the unit at i0, of which rem elements are there
template <int kSize>
__device__ __forceinline__ void copy_runs(uint32_t dst, uint64_t base, int i0, int rem, int lane) {
    const uint64_t src = base + static_cast<uint32_t>((i0 + lane * 4) * kSize);
    dst += lane * 4 * kSize;
    if (rem >= kUnit) {
#pragma unroll
        for (int h = 0; h < 4; ++h) copy_async<4 * kSize>(dst + h * 128 * kSize, src + h * 128 * kSize);
    } else {
        // a run past the end reads nothing, so its address may lie anywhere
#pragma unroll
        for (int h = 0; h < 4; ++h)
            copy_async_part<4 * kSize>(dst + h * 128 * kSize, src + h * 128 * kSize, kSize * min(max(rem - lane * 4 - h * 128, 0), 4));
    }
}
__device__ __forceinline__ void copy_unit(const Chunk &c, uint32_t stage, int i0, int lane) {
    const int rem = c.n - i0;
    const uint32_t flags = c.flags;
    if (flags & kGradBf16) copy_runs<2>(stage, c.g, i0, rem, lane);
    else copy_runs<4>(stage, c.g, i0, rem, lane);
    stage += (flags & kGradBf16) ? 2 * kUnit : 4 * kUnit;
    if (flags & kParamBf16) copy_runs<2>(stage, c.p, i0, rem, lane);
    else copy_runs<4>(stage, c.p, i0, rem, lane);
    stage += (flags & kParamBf16) ? 2 * kUnit : 4 * kUnit;
    copy_runs<1>(stage, c.m, i0, rem, lane);
    copy_runs<1>(stage + kUnit, c.v, i0, rem, lane);
}
// pairs 2 h and 2 h + 1 of a lane's elements of a parameter or gradient in a stage
template <bool kBf16>
__device__ __forceinline__ void stage_pairs(const uint8_t *base, int h, int lane, uint64_t *x) {
    const int e = h * 128 + lane * 4;
    if (kBf16) {
        const uint2 w = *reinterpret_cast<const uint2 *>(base + 2 * e);
        x[0] = pack2(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u));
        x[1] = pack2(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
    } else {
        const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(base + 4 * e);
        x[0] = w.x;
        x[1] = w.y;
    }
}

// One block: i0 its place in the chunk, g / p / mc / vc its parts of the stage, d its steps before (even lanes: m's,
// odd lanes: sqrt(v)'s; replaced by the new ones).
template <bool kPBf16, bool kGBf16, bool kFull>
__device__ __forceinline__ void step8_block(const StepArgs &a, const Scalars &s, const Slot &c, const uint8_t *g, const uint8_t *p,
                                            const uint8_t *mc, const uint8_t *vc, float dm, float dv, float &d, int i0, int lane) {
    const int rem = c.c.n - i0;
    float mf[8], vf[8], w[8], pf[8];
    uint64_t m[4], v[4], x[2];
    uint32_t cm[2], cv[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        cm[h] = *reinterpret_cast<const uint32_t *>(mc + h * 128 + lane * 4);
        cv[h] = *reinterpret_cast<const uint32_t *>(vc + h * 128 + lane * 4);
    }
    decode8<false>(cm, dm, m);
    decode8<true>(cv, dv, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i % 2 == 0) stage_pairs<kGBf16>(g, i / 2, lane, x);
        moments(a, s, x[i % 2], m[i], v[i]);
        unpack2(m[i], mf[2 * i], mf[2 * i + 1]);
        unpack2(v[i], vf[2 * i], vf[2 * i + 1]);
    }
    roots(s, vf, w);
    const uint64_t minus_lr = c.minus_lr, decay = c.decay;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i % 2 == 0) stage_pairs<kPBf16>(p, i / 2, lane, x);
        unpack2(update(s, minus_lr, decay, x[i % 2], m[i], w[2 * i], w[2 * i + 1]), pf[2 * i], pf[2 * i + 1]);
    }
    store8<kFull>(c.c.p, kPBf16, i0, rem, lane, pf);
    if (!kPBf16 && c.c.copy) store8<kFull>(c.c.copy, true, i0, rem, lane, pf);
    float am = 0.f, av = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // places past a tensor's end take no part in its last block's largest value
        if (!kFull && (i >> 2) * 128 + lane * 4 + (i & 3) >= rem) mf[i] = vf[i] = w[i] = 0.f;
        am = max_nan(am, mf[i]);
        av = max_nan(av, vf[i]);
    }
    am = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(am)));
    av = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(av)));
    // the root is monotonic, so the largest root is the root of the largest v; even lanes work out m's
    // step and odd lanes sqrt(v)'s
    const bool odd = lane & 1;
    float inv;
    block_step(odd ? __fsqrt_rn(av) : am, odd ? float(kTopW * kTopW) : float(kTopM * kTopM), d, inv);
    encode8<false>(mf, nullptr, __shfl_sync(0xffffffffu, inv, 0), false, cm);
    // below 2^-92 a flushed root could have had a code above 0
    encode8<true>(vf, w, __shfl_sync(0xffffffffu, inv, 1), s.flush && av < 2.0194839e-28f, cv);
    store_codes<kFull>(c.c.m, i0, rem, lane, cm);
    store_codes<kFull>(c.c.v, i0, rem, lane, cv);
}
// The unit at i0 of a chunk; steps: in lanes 0 .. 3 the steps before of (m, sqrt(v)) of its two blocks.
template <bool kPBf16, bool kGBf16>
__device__ __forceinline__ void step8_unit(const StepArgs &a, const Scalars &s, const Slot &c, const uint8_t *stage, float steps,
                                           int i0, int lane) {
    constexpr int kG = kGBf16 ? 2 : 4, kP = kPBf16 ? 2 : 4;
    const int blocks = min((c.c.n - i0 + kBlock - 1) / kBlock, 2);
    float out = 0.f;
#pragma unroll 1
    for (int b = 0; b < blocks; ++b) {
        const float dm = __shfl_sync(0xffffffffu, steps, 2 * b), dv = __shfl_sync(0xffffffffu, steps, 2 * b + 1);
        const uint8_t *g = stage + b * (kBlock * kG), *p = stage + kUnit * kG + b * (kBlock * kP),
                      *mc = stage + kUnit * (kG + kP) + b * kBlock, *vc = mc + kUnit;
        float d;
        if (c.c.n - i0 - b * kBlock >= kBlock)
            step8_block<kPBf16, kGBf16, true>(a, s, c, g, p, mc, vc, dm, dv, d, i0 + b * kBlock, lane);
        else
            step8_block<kPBf16, kGBf16, false>(a, s, c, g, p, mc, vc, dm, dv, d, i0 + b * kBlock, lane);
        if ((lane >> 1) == b) out = d;
    }
    if (lane < 2 * blocks) reinterpret_cast<float *>((lane & 1) ? c.c.dv : c.c.dm)[i0 / kBlock + (lane >> 1)] = out;
}

constexpr int kCtas8 = 3;      // CTAs per SM that the registers are capped for
__global__ void __launch_bounds__(kThreads, kCtas8) adamw8_kernel(const __grid_constant__ StepArgs a, int elem) {
    extern __shared__ __align__(16) uint8_t step8_smem_base[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int stage_bytes = kUnit * elem;
    uint8_t *ring = step8_smem_base + warp * (2 * stage_bytes);
    Slot *slots = reinterpret_cast<Slot *>(step8_smem_base + kWarps * 2 * stage_bytes) + warp * kSlots;
    const uint32_t ring_at = smem_u32(ring);
    const int stride = gridDim.x * kWarps;
    int done = blockIdx.x * kWarps + warp;                    // the chunk worked on
    if (done >= a.nchunks) return;
    // the chunk list was complete when the plan's call returned: it may be read before the wait
    int ahead = done;                                         // the chunk copied from
    uint32_t word = chunk_word(a.chunks, ahead, lane);
    pdl_launch_dependents();
    pdl_wait();
    Scalars s;
    if (!read_scalars(a, s)) return;
    int to_slot = 0, to_i0 = 0, to_stage = 0;
    float next_steps = 0.f;
    // the chunk `ahead`, whose words are here, into slot to_slot; the words of the one after it are sent for
    auto open_slot = [&]() {
        const float lr = -(s.lr * __uint_as_float(word32(word, 16))), decay = __uint_as_float(word32(word, 17));
        __syncwarp();
        if (lane < 20) reinterpret_cast<uint32_t *>(slots + to_slot)[lane] = word;
        if (lane == 20) slots[to_slot].minus_lr = pack2(lr, lr);
        if (lane == 21) slots[to_slot].decay = pack2(decay, decay);
        __syncwarp();
        if (ahead + stride < a.nchunks) word = chunk_word(a.chunks, ahead + stride, lane);
    };
    open_slot();
    // starts the copies of the next unit of the list, if there is one, and loads its steps
    auto copy_next = [&]() {
        if (ahead < a.nchunks) {
            const Chunk &c = slots[to_slot].c;
            copy_unit(c, ring_at + to_stage * stage_bytes, to_i0, lane);
            if (lane < 4 && to_i0 + (lane >> 1) * kBlock < c.n)
                next_steps = reinterpret_cast<const float *>((lane & 1) ? c.dv : c.dm)[to_i0 / kBlock + (lane >> 1)];
            to_i0 += kUnit;
            if (to_i0 >= c.n) {
                to_i0 = 0;
                ahead += stride;
                to_slot = (to_slot + 1) % kSlots;
                open_slot();
            }
        }
        to_stage ^= 1;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    copy_next();
    int slot = 0, stage = 0, i0 = 0;
    while (true) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        const float steps = next_steps;
        copy_next();
        const Slot &c = slots[slot];
        const uint8_t *at = ring + stage * stage_bytes;
        switch (c.c.flags & (kParamBf16 | kGradBf16)) {
            case 0: step8_unit<false, false>(a, s, c, at, steps, i0, lane); break;
            case kParamBf16: step8_unit<true, false>(a, s, c, at, steps, i0, lane); break;
            case kGradBf16: step8_unit<false, true>(a, s, c, at, steps, i0, lane); break;
            default: step8_unit<true, true>(a, s, c, at, steps, i0, lane);
        }
        stage ^= 1;
        i0 += kUnit;
        if (i0 >= c.c.n) {
            i0 = 0;
            slot = (slot + 1) % kSlots;
            done += stride;
            if (done >= a.nchunks) return;
        }
    }
}

// Sum of squares of every gradient: each lane sums in double (a float32 square overflows at
// 1.8e19 and loses what lies below 1e-19), each CTA leaves one partial sum, and the last CTA
// adds the partials in a fixed order.  CTA b takes the chunks [8 per_warp b, 8 per_warp (b + 1)), warp by
// warp in turn: the result depends on the plan only, and the CTAs read in the order of the list (as in
// adamw32_kernel).
template <bool kBf16>
__device__ __forceinline__ double sum_squares(const uint32_t *w, double sum) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float g = kBf16 ? __uint_as_float((i & 1) ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16) : __uint_as_float(w[i]);
        sum = fma(double(g), double(g), sum);
    }
    return sum;
}
template <bool kBf16>
__device__ __forceinline__ double norm_chunk(uint64_t g, int n, int lane, double sum) {
    int i0 = 0;
    for (; i0 + 2 * kBlock <= n; i0 += 2 * kBlock) {
        Raw8<kBf16> x, y;
        x.template load<true>(g, i0, kBlock, lane);
        y.template load<true>(g, i0 + kBlock, kBlock, lane);
        sum = sum_squares<kBf16>(x.w, sum);
        sum = sum_squares<kBf16>(y.w, sum);
    }
    for (; i0 < n; i0 += kBlock) {
        Raw8<kBf16> x;
        if (n - i0 >= kBlock) x.template load<true>(g, i0, kBlock, lane);
        else x.template load<false>(g, i0, n - i0, lane);
        sum = sum_squares<kBf16>(x.w, sum);
    }
    return sum;
}
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const Chunk *chunks, PlanHead *head, int64_t nchunks, int per_warp,
                                                             float max_norm, float *out) {
    __shared__ double s_sum[kWarps];
    __shared__ bool s_last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t first = int64_t(blockIdx.x) * kWarps * per_warp + warp;
    uint32_t word = first < nchunks ? chunk_word(chunks, first, lane) : 0u;
    pdl_launch_dependents();
    pdl_wait();
    double sum = 0.0;
    for (int j = 0; j < per_warp && first + j * kWarps < nchunks; ++j) {
        const uint64_t g = word64(word, 4);
        const int n = static_cast<int>(word32(word, 14));
        const bool bf16 = (word32(word, 15) & kGradBf16) != 0;
        if (j + 1 < per_warp && first + (j + 1) * kWarps < nchunks) word = chunk_word(chunks, first + (j + 1) * kWarps, lane);
        sum = bf16 ? norm_chunk<true>(g, n, lane, sum) : norm_chunk<false>(g, n, lane, sum);
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
        Raw8<false> raw;
        if (rem == kBlock) raw.template load<true>(src, b * kBlock, rem, lane);
        else raw.template load<false>(src, b * kBlock, rem, lane);
        uint32_t c[2];
        float f[8], w[8], top = 0.f, d, inv;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[i] = __uint_as_float(raw.w[i]);
            w[i] = 0.f;
            if (kSecond) {
                w[i] = sqrt_approx<false>(f[i]);
                if (!(f[i] >= 0.f)) top = __uint_as_float(0x7FC00000u);   // a negative v has no root, like a NaN
            }
            top = max_nan(top, f[i]);
        }
        top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
        block_step(kSecond ? __fsqrt_rn(top) : top, kSecond ? float(kTopW * kTopW) : float(kTopM * kTopM), d, inv);
        encode8<kSecond>(f, w, inv, false, c);
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
        uint64_t y[4];
        float f[8];
        decode8<kSecond>(c, __ldcg(steps + b), y);
#pragma unroll
        for (int i = 0; i < 4; ++i) unpack2(y[i], f[2 * i], f[2 * i + 1]);
        if (rem == kBlock) store8<true>(dst, false, b * kBlock, rem, lane, f);
        else store8<false>(dst, false, b * kBlock, rem, lane, f);
    }
}

}  // namespace optim
}  // namespace qlora
