// bs_adamw.cu -- one AdamW step over many tensors in one launch, moments in 32 bits or in 8 bits
// with a scale for each 256 elements, and the norm of all gradients before it.
//
//   g = clip * grad;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g g
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Each kernel is one pass over its bytes. A warp takes 256 consecutive elements at a time, 8 a lane:
// 16 bytes of BF16 or 32 of FP32 per lane and tensor, all loads of a group issued before its
// arithmetic. 256 elements are also one block of the 8-bit moments, so a block's largest magnitude is
// one warp reduction and nothing is exchanged between warps.
//
// Measured on one B200, whose plain copy runs at 6.56 TB/s, BF16 parameters and gradients:
//   step, 32-bit moments    198M elements    660 us   6.6 TB/s   memory
//   step, 8-bit moments     198M elements    504 us   3.9 TB/s   instructions: 10 bytes an element, and
//                                                                about 70 instructions for each
//   norm of the gradients   208M elements     80 us   5.2 TB/s   memory latency: reads alone
//   8-bit moments as FP32   208M elements    367 us   5.7 TB/s   memory, 4 bytes of 5 written
//
// The 8-bit moments. m is held as e4m3 (sign, 4 exponent and 3 fraction bits), v, which is never
// negative, as 5 exponent and 3 fraction bits: the upper half of a half-precision number. Each
// block's largest magnitude is scaled to the format's largest value. Values are rounded up or down
// at random in proportion to the distance, so that the moment is right on average: v moves by
// 1 - b2 = 0.001 of itself a step, far below half of its spacing (1/16 .. 1/8), and rounding to
// nearest would leave it where it is. 5 exponent bits span 2^30 inside a block, that is 2^15
// between gradients; a v above zero never becomes zero (it would leave m / eps as the step), it
// stops at the smallest code. The random bits are splitmix64 outputs for (seed, step, tensor,
// element), so a step can be repeated bit for bit.
//
// The moments' updates round after every product and sum (no fused multiply-add), so that the
// codes, which depend on the last bit now and then, are those of the formula in plain FP32
// operations. They are kept in FP32 until the step has been taken from them; only then are they
// rounded to 8 bits. A BF16 parameter without a FP32 master copy is rounded to nearest.
#include <cuda_runtime.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdint>
#include <cstring>
#include <memory>
#include <new>

#include "bs_host.h"
#include "bs_internal.h"

namespace bs {
namespace {

constexpr uint32_t kBlock = BS_ADAMW_BLOCK; // elements of a warp's group and of an 8-bit block
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr float kTopM = 448.f, kTopV = 61440.f; // the formats' largest values
constexpr float kMost = 3.40282346638528860e38f; // FLT_MAX
constexpr float kDead = 7.8886090522101181e-31f; // 2^-100: a block below this counts as zero
constexpr int kFewItems = 16, kManyItems = 250;

struct OptOut { // where a step goes
    uint8_t *p, *m, *v;
    float *master, *ms, *vs;
};
struct OptItem {
    const uint8_t *p, *m, *v, *g;
    const float *master, *ms, *vs;
    OptOut to;
    uint64_t n;
    uint32_t group_begin; // first 256-element group of this tensor in the launch
    float decay;
    uint32_t tensor;      // its number in the call
    uint32_t flags;       // kP16, kG16, kVec
};
static_assert(sizeof(OptItem) == 128, "OptItem layout");
constexpr uint32_t kP16 = 1, kG16 = 2, kVec = 4; // BF16 parameters, BF16 gradients, all pointers aligned for vectors

struct NormItem {
    const uint8_t* g;
    uint64_t n;
    uint32_t group_begin, flags;
};
constexpr int kFewNorm = 64, kManyNorm = 1300;
template <int CAP>
struct NormParams {
    uint32_t n_items, groups, last, partial_at;
    float max_norm;
    bs_adamw_ctl* ctl;
    double* partial; // one sum a CTA, those of earlier launches before it
    NormItem item[CAP];
};
static_assert(sizeof(NormParams<kManyNorm>) < 32764, "kernel parameters");

template <int CAP>
struct OptParams {
    uint32_t n_items, groups, per_cta; // groups of the launch, groups a CTA takes
    uint32_t last;                     // the call's last launch
    uint32_t step;                     // the step's number, 0: one more than ctl->step
    uint32_t into;                     // results go into other buffers than those that are read
    float b1, b2, c1, c2, eps;         // c = 1 - b, rounded from 64 bits
    double log_b1, log_b2;
    uint64_t seed;
    bs_adamw_ctl* ctl;
    OptItem item[CAP];
};
static_assert(sizeof(OptParams<kManyItems>) < 32764, "kernel parameters");

__device__ __forceinline__ uint64_t mix64(uint64_t z) { // splitmix64's output function
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}
__device__ __forceinline__ uint32_t to_bf16x2(float lo, float hi) { // to nearest, ties to even; NaN stays NaN
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// sqrt and 1 / x within 2^-23, numbers below the normal range as 0: a v below 2^-126 is a root below
// 2^-63, which eps (at least 1e-12) hides.
__device__ __forceinline__ float sqrt_fast(float x) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) { // NaN if either is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// 8 elements of a lane as they stand in memory, from `at` on (4 words of BF16 pairs, or 8 of FP32);
// with `full` false only the first `cnt` exist (0 for the others).
__device__ __forceinline__ void load_raw(uint32_t (&r)[8], const uint8_t* base, uint64_t at, bool b16, bool full, uint32_t cnt) {
    if (b16) {
        const uint16_t* s = reinterpret_cast<const uint16_t*>(base) + at;
        if (full) {
            const uint4 w = *reinterpret_cast<const uint4*>(s);
            r[0] = w.x; r[1] = w.y; r[2] = w.z; r[3] = w.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; i += 2)
                r[i >> 1] = (i < cnt ? uint32_t(s[i]) : 0u) | (i + 1 < cnt ? uint32_t(s[i + 1]) << 16 : 0u);
        }
    } else {
        const float* s = reinterpret_cast<const float*>(base) + at;
        if (full) {
            const uint4 a = *reinterpret_cast<const uint4*>(s), b = *reinterpret_cast<const uint4*>(s + 4);
            r[0] = a.x; r[1] = a.y; r[2] = a.z; r[3] = a.w; r[4] = b.x; r[5] = b.y; r[6] = b.z; r[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i] = i < cnt ? __float_as_uint(s[i]) : 0u;
        }
    }
}
__device__ __forceinline__ void unpack(float (&f)[8], const uint32_t (&r)[8], bool b16) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        f[i] = b16 ? __uint_as_float(r[i >> 1] << 16) : __uint_as_float(r[i]);
        f[i + 1] = b16 ? __uint_as_float(r[i >> 1] & 0xFFFF0000u) : __uint_as_float(r[i + 1]);
    }
}
__device__ __forceinline__ void load8(float (&f)[8], const uint8_t* base, uint64_t at, bool b16, bool full, uint32_t cnt) {
    uint32_t r[8];
    load_raw(r, base, at, b16, full, cnt);
    unpack(f, r, b16);
}
__device__ __forceinline__ void store8(const float (&f)[8], uint8_t* base, uint64_t at, bool b16, bool full, uint32_t cnt) {
    if (b16) {
        uint16_t* d = reinterpret_cast<uint16_t*>(base) + at;
        if (full) {
            uint4 w;
            w.x = to_bf16x2(f[0], f[1]); w.y = to_bf16x2(f[2], f[3]);
            w.z = to_bf16x2(f[4], f[5]); w.w = to_bf16x2(f[6], f[7]);
            *reinterpret_cast<uint4*>(d) = w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) if (i < cnt) d[i] = static_cast<uint16_t>(to_bf16x2(f[i], 0.f));
        }
    } else {
        float* d = reinterpret_cast<float*>(base) + at;
        if (full) {
            *reinterpret_cast<float4*>(d) = make_float4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<float4*>(d + 4) = make_float4(f[4], f[5], f[6], f[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) if (i < cnt) d[i] = f[i];
        }
    }
}
__device__ __forceinline__ uint2 load_codes(const uint8_t* base, uint64_t at, bool full, uint32_t cnt) {
    if (full) return *reinterpret_cast<const uint2*>(base + at);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) if (i < cnt) w[i >> 2] |= uint32_t(base[at + i]) << (8 * (i & 3));
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes(uint2 w, uint8_t* base, uint64_t at, bool full, uint32_t cnt) {
    if (full) { *reinterpret_cast<uint2*>(base + at) = w; return; }
    const uint32_t q[2] = {w.x, w.y};
#pragma unroll
    for (int i = 0; i < 8; ++i) if (i < cnt) base[at + i] = static_cast<uint8_t>(q[i >> 2] >> (8 * (i & 3)));
}
__device__ __forceinline__ void decode_m(float (&f)[8], uint2 w, float scale) {
    const uint32_t q[2] = {w.x, w.y};
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(q[i >> 2] >> (8 * (i & 3))), __NV_E4M3);
        const float2 d = __half22float2(__half2(h));
        f[i] = __fmul_rn(d.x, scale);
        f[i + 1] = __fmul_rn(d.y, scale);
    }
}
__device__ __forceinline__ void decode_v(float (&f)[8], uint2 w, float scale) {
    const uint32_t q[2] = {w.x, w.y};
#pragma unroll
    for (int i = 0; i < 8; i += 2) { // two codes to the upper bytes of two halves, then down by one bit
        const uint32_t h = (__byte_perm(q[i >> 2], 0, (i & 2) ? 0x3424 : 0x1404) >> 1) & 0x7F807F80u;
        __half2 hh;
        std::memcpy(&hh, &h, 4);
        const float2 d = __half22float2(hh);
        f[i] = __fmul_rn(d.x, scale);
        f[i + 1] = __fmul_rn(d.y, scale);
    }
}
// The code of |y|, rounded up where its 16 random bits u reach what is left of it below. Scaled by
// 2^(BIAS - 127), the format's exponent range becomes FP32's lowest, so bits 20 and up of the number
// are the code, and adding the random bits 16 times carries into it. The block's largest, at most two
// steps of FP32 above the format's largest value, cannot carry beyond it. Below the format's normal
// range the scaled number is subnormal; there the sum is taken as the definition has it, in FP32,
// where the last bit could differ (code_slow). Such values are few, and their code is at most 8: a
// lane that has one such code does its 16 anew.
template <int BIAS>
__device__ __forceinline__ float down() { return __uint_as_float(static_cast<uint32_t>(BIAS) << 23); } // 2^(BIAS - 127)
template <int BIAS>
constexpr uint32_t kSmall = (static_cast<uint32_t>(128 - BIAS) << 23) - 1u; // the bits of 2^(1 - BIAS), less one
template <int BIAS>
__device__ __forceinline__ bool is_small(float y) { return __float_as_uint(y) - 1u < kSmall<BIAS>; } // 0 is not small
template <int BIAS, uint32_t MOST>
__device__ __forceinline__ uint32_t code_slow(float y, uint32_t u) { // y >= 0 or NaN, which gives the largest code
    if (!is_small<BIAS>(y)) return min(__float_as_uint(__fmul_rn(y, down<BIAS>())) + u * 16u, (MOST << 20) | 0xFFFFFu) >> 20;
    return static_cast<uint32_t>(static_cast<int>(
        __fadd_rn(__fmul_rn(y, static_cast<float>(1 << (BIAS + 2))), __fmul_rn(static_cast<float>(u), 1.f / 65536.f))));
}
// 4 codes from bits 20 .. 27 of 4 words
__device__ __forceinline__ uint32_t pack_v(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x7632) >> 4, __byte_perm(c, d, 0x7632) >> 4, 0x6420);
}
// 4 codes from bits 20 .. 26 of 4 words and their signs from bit 31
__device__ __forceinline__ uint32_t pack_m(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t x = __byte_perm(a, b, 0x7632), y = __byte_perm(c, d, 0x7632);
    return __byte_perm((x >> 4 & 0x007F007Fu) | (x >> 8 & 0x00800080u), (y >> 4 & 0x007F007Fu) | (y >> 8 & 0x00800080u), 0x6420);
}
// Whether one of 4 codes is at most 8, its upper bit left out (m) or not (v).
__device__ __forceinline__ bool low_m(uint32_t q) { return (~((q & 0x7F7F7F7Fu) + 0x77777777u) & 0x80808080u) != 0; }
__device__ __forceinline__ bool low_v(uint32_t q) { return (~(((q & 0x7F7F7F7Fu) + 0x77777777u) | q) & 0x80808080u) != 0; }
// The largest magnitude of the block, NaN when any is NaN.
__device__ __forceinline__ float block_max(const float (&f)[8]) {
    float b = fabsf(f[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) b = max_nan(b, fabsf(f[i]));
    return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(b))); // as integers every NaN is above infinity
}

template <typename Params>
__device__ __forceinline__ int item_of(const Params& p, uint32_t group, int lo) {
    int hi = static_cast<int>(p.n_items) - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.item[mid].group_begin <= group) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// What a lane has loaded of one group: 8 elements of everything the step reads.
template <int BITS>
struct Held {
    uint32_t w[8], g[8];
    float m[8], v[8];
};
template <>
struct Held<8> {
    uint32_t w[8], g[8];
    uint2 cm, cv;
    float sm, sv;
};
// The constants of a step.
struct StepConst {
    float b1, b2, c1, c2, eps, clip, lr, step, r2;
};

template <int BITS>
__device__ __forceinline__ void load_group(Held<BITS>& h, const OptItem& it, uint64_t block, uint64_t at, bool p16, bool g16, bool master,
                                           bool full, uint32_t cnt) {
    if (master) load_raw(h.w, reinterpret_cast<const uint8_t*>(it.master), at, false, full, cnt);
    else load_raw(h.w, it.p, at, p16, full, cnt);
    load_raw(h.g, it.g, at, g16, full, cnt);
    if constexpr (BITS == 32) {
        load8(h.m, it.m, at, false, full, cnt);
        load8(h.v, it.v, at, false, full, cnt);
    } else {
        h.cm = load_codes(it.m, at, full, cnt);
        h.cv = load_codes(it.v, at, full, cnt);
        h.sm = it.ms[block];
        h.sv = it.vs[block];
    }
}

template <int BITS>
__device__ __forceinline__ void step_group(const Held<BITS>& h, const OptItem& it, const StepConst& c, float decay, float keep, uint64_t key, uint32_t lane,
                                           uint64_t block, uint64_t at, bool p16, bool g16, bool master, bool full, uint32_t cnt) {
    float w[8], g[8], m[8], v[8];
    unpack(w, h.w, p16 && !master);
    unpack(g, h.g, g16);
    if constexpr (BITS == 32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) { m[i] = h.m[i]; v[i] = h.v[i]; }
    } else {
        decode_m(m, h.cm, h.sm);
        decode_v(v, h.cv, h.sv);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float gi = __fmul_rn(g[i], c.clip);
        m[i] = __fadd_rn(__fmul_rn(m[i], c.b1), __fmul_rn(gi, c.c1));
        v[i] = __fadd_rn(__fmul_rn(v[i], c.b2), __fmul_rn(__fmul_rn(gi, c.c2), gi));
        // FP32 weights: decay and step are added up before they meet the weight. 1 - lr decay alone would be rounded
        // to a multiple of 2^-24 for every weight and step: at lr 1e-5 and decay 0.01 a fifth too much. A weight that
        // is kept in BF16 rounds by 2^-9 itself, and this is an instruction more. (An infinite weight stays one.)
        if (p16 && !master) w[i] = w[i] * keep - c.step * m[i] * rcp_fast(sqrt_fast(v[i]) * c.r2 + c.eps);
        else w[i] -= fmaf(decay, fminf(fmaxf(w[i], -kMost), kMost), c.step * m[i] * rcp_fast(sqrt_fast(v[i]) * c.r2 + c.eps));
    }
    store8(w, it.to.p, at, p16, full, cnt);
    if (master) store8(w, reinterpret_cast<uint8_t*>(it.to.master), at, false, full, cnt);
    if constexpr (BITS == 32) {
        store8(m, it.to.m, at, false, full, cnt);
        store8(v, it.to.v, at, false, full, cnt);
    } else {
        const float bm = block_max(m), bv = block_max(v);
        // One division serves the warp: lanes 0 and 1 take what the values are multiplied by, lanes 2
        // and 3 the scales that are stored. A NaN is not below kDead, so the scale carries it.
        const float top = lane & 1 ? kTopV : kTopM, big = lane & 1 ? bv : bm;
        const float quot = big < kDead ? 0.f : __fdiv_rn(lane & 2 ? big : top, lane & 2 ? top : big);
        float im = __shfl_sync(0xFFFFFFFFu, quot, 0), iv = __shfl_sync(0xFFFFFFFFu, quot, 1);
        if ((lane >> 1) == 1) (lane & 1 ? it.to.vs : it.to.ms)[block] = quot;
        uint64_t pair0 = key + 0x9E3779B97F4A7C15ull * ((at >> 1) + 1), pair = pair0;
        const float fm = im * down<7>(), fv = iv * down<15>();
        uint32_t qm[2], qv[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            uint32_t cm[4], cv[4];
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                const uint64_t z = mix64(pair);
                pair += 0x9E3779B97F4A7C15ull;
#pragma unroll
                for (int k = j; k < j + 2; ++k) {
                    const uint32_t u = k & 1 ? static_cast<uint32_t>(z >> 32) : static_cast<uint32_t>(z);
                    cm[k] = __float_as_uint(__fmul_rn(m[4 * q + k], fm)) + __byte_perm(u, 0, 0x4410) * 16u;
                    cv[k] = __float_as_uint(__fmul_rn(v[4 * q + k], fv)) + __byte_perm(u, 0, 0x4432) * 16u;
                }
            }
            qm[q] = pack_m(cm[0], cm[1], cm[2], cm[3]);
            qv[q] = pack_v(cv[0], cv[1], cv[2], cv[3]);
        }
        // fm and fv are exact while they are normal: not for a block with infinity or NaN, or with an
        // m above 28672 or a v above 10^9
        constexpr float kNormal = 1.17549435082228751e-38f;
        const bool exact = (fm >= kNormal || bm < kDead) && (fv >= kNormal || bv < kDead);
        if (!exact || low_m(qm[0]) || low_m(qm[1]) || low_v(qv[0]) || low_v(qv[1])) {
            asm volatile("" : "+l"(pair0), "+f"(im), "+f"(iv)); // nothing of the usual way is kept in registers for this one
            bool anew = !exact;
#pragma unroll
            for (int e = 0; e < 8; ++e) anew |= is_small<7>(__fmul_rn(fabsf(m[e]), im)) || is_small<15>(__fmul_rn(v[e], iv));
            if (anew) {
                qm[0] = qm[1] = qv[0] = qv[1] = 0;
                uint64_t z = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (!(e & 1)) {
                        z = mix64(pair0);
                        pair0 += 0x9E3779B97F4A7C15ull;
                    }
                    const uint32_t u = e & 1 ? static_cast<uint32_t>(z >> 32) : static_cast<uint32_t>(z);
                    const uint32_t sign = __float_as_uint(m[e]) >> 24 & 0x80u;
                    qm[e >> 2] |= (code_slow<7, 0x7E>(__fmul_rn(fabsf(m[e]), im), u & 0xFFFFu) | sign) << (8 * (e & 3));
                    qv[e >> 2] |= code_slow<15, 0xF7>(__fmul_rn(v[e], iv), u >> 16) << (8 * (e & 3));
                }
            }
            if (!(bv < kDead)) {
#pragma unroll
                for (int e = 0; e < 8; ++e) // what is above zero stays above it
                    if (v[e] > 0.f && ((qv[e >> 2] >> (8 * (e & 3))) & 0xFFu) == 0) qv[e >> 2] |= 1u << (8 * (e & 3));
            }
        }
        store_codes(make_uint2(qm[0], qm[1]), it.to.m, at, full, cnt);
        store_codes(make_uint2(qv[0], qv[1]), it.to.v, at, full, cnt);
    }
}

// Groups begin, begin + kWarps, .. below end of one tensor, all of them whole and aligned. With BF16
// parameters and gradients and 32-bit moments the next group's loads are under way during a group's
// arithmetic; with 8-bit moments two groups are loaded at once. The wider ones do not fit into the
// registers beside each other.
template <int BITS, bool P16, bool G16, bool MASTER>
__device__ __forceinline__ void whole_groups(const OptItem& it, const StepConst& c, float decay, float keep, uint64_t key, uint32_t lane, uint32_t begin,
                                             uint32_t end) {
    if (begin >= end) return;
    constexpr bool kNarrow = P16 && G16 && !MASTER, kAhead = BITS == 32 && kNarrow, kTwo = BITS == 8 && kNarrow;
    auto load = [&](Held<BITS>& h, uint32_t b) {
        load_group<BITS>(h, it, b, uint64_t(b) * kBlock + 8u * lane, P16, G16, MASTER, true, 8);
    };
    auto step = [&](const Held<BITS>& h, uint32_t b) {
        step_group<BITS>(h, it, c, decay, keep, key, lane, b, uint64_t(b) * kBlock + 8u * lane, P16, G16, MASTER, true, 8);
    };
    Held<BITS> h;
    if constexpr (kAhead) load(h, begin);
    for (uint32_t b = begin; b < end; b += kWarps) {
        if constexpr (kAhead) {
            Held<BITS> next;
            if (b + kWarps < end) load(next, b + kWarps);
            step(h, b);
            h = next;
        } else {
            load(h, b);
            if (kTwo && b + kWarps < end) {
                Held<BITS> second;
                load(second, b + kWarps);
                step(h, b);
                b += kWarps;
                step(second, b);
            } else {
                step(h, b);
            }
        }
    }
}

// With 32-bit moments each kind of tensor is a function of its own, so that its loop gets registers and an order of
// its own whatever the others need: 198M BF16 weights 660 us, 665 to 670 us inlined, 588 tensors with
// master copies 279 us against 290. With 8-bit ones the call's registers cost more than that gives (559 against 504 us).
template <bool P16, bool G16, bool MASTER>
__device__ __noinline__ void whole_groups_32(const OptItem& it, const StepConst c, float decay, float keep, uint64_t key, uint32_t lane,
                                             uint32_t begin, uint32_t end) {
    whole_groups<32, P16, G16, MASTER>(it, c, decay, keep, key, lane, begin, end);
}
template <int BITS, bool P16, bool G16, bool MASTER>
__device__ __forceinline__ void groups_of_kind(const OptItem& it, const StepConst& c, float decay, float keep, uint64_t key, uint32_t lane,
                                               uint32_t begin, uint32_t end) {
    if constexpr (BITS == 32) whole_groups_32<P16, G16, MASTER>(it, c, decay, keep, key, lane, begin, end);
    else whole_groups<BITS, P16, G16, MASTER>(it, c, decay, keep, key, lane, begin, end);
}

// 8 elements of a lane, of es bytes each, as they are.
__device__ __forceinline__ void copy8(uint8_t* to, const uint8_t* from, uint64_t at, uint32_t es, bool full, uint32_t cnt) {
    to += at * es;
    from += at * es;
    if (full) {
        if (es == 1) *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(from);
        else
            for (uint32_t i = 0; i < es / 2; ++i) reinterpret_cast<uint4*>(to)[i] = reinterpret_cast<const uint4*>(from)[i];
    } else {
        for (uint32_t i = 0; i < cnt; ++i)
            if (es == 1) to[i] = from[i];
            else if (es == 2) reinterpret_cast<uint16_t*>(to)[i] = reinterpret_cast<const uint16_t*>(from)[i];
            else reinterpret_cast<uint32_t*>(to)[i] = reinterpret_cast<const uint32_t*>(from)[i];
    }
}
// A step that is left out but has buffers of its own for its results: they receive everything as it was,
// so that the caller may go on from them. Not inlined: the step's registers are not these.
template <int CAP, int BITS>
__device__ __noinline__ void copy_all(const OptParams<CAP>& p) {
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    for (uint32_t g0 = blockIdx.x * p.per_cta; g0 < p.groups; g0 += gridDim.x * p.per_cta) {
        const uint32_t g1 = min(g0 + p.per_cta, p.groups);
        int k = item_of(p, g0, 0);
        for (uint32_t g = g0 + warp; g < g1; g += kWarps) {
            if (k + 1 < static_cast<int>(p.n_items) && p.item[k + 1].group_begin <= g) k = item_of(p, g, k);
            const OptItem& it = p.item[k];
            const uint64_t block = g - it.group_begin, at = block * kBlock + 8u * lane;
            const uint32_t cnt = at < it.n ? static_cast<uint32_t>(it.n - at < 8 ? it.n - at : 8) : 0u;
            const bool full = cnt == 8 && (it.flags & kVec);
            copy8(it.to.p, it.p, at, it.flags & kP16 ? 2 : 4, full, cnt);
            if (it.master) copy8(reinterpret_cast<uint8_t*>(it.to.master), reinterpret_cast<const uint8_t*>(it.master), at, 4, full, cnt);
            copy8(it.to.m, it.m, at, BITS / 8, full, cnt);
            copy8(it.to.v, it.v, at, BITS / 8, full, cnt);
            if (BITS == 8 && lane < 2) (lane ? it.to.vs : it.to.ms)[block] = (lane ? it.vs : it.ms)[block];
        }
    }
}

// CTAs of a pass that an SM holds: with 32-bit moments 2 of up to 128 registers, which hold the next
// group, with 8-bit ones 4 of up to 64 (208M BF16 weights: 520 us, with 3 of up to 80 535 us). The
// moments' read-out takes the same time with 2, 4 and 6.
constexpr int ctas_per_sm(int bits) { return bits == 8 ? 4 : 2; }
constexpr int kReadCtas = 4;
// With 32-bit moments the CTAs go through the groups together, 32 (4 a warp) at a time, so that the
// memory being read and written at any time is a few contiguous stretches: 198M BF16 weights take 655
// us, against 740 us with one equal run a CTA. With 8-bit ones the search for each run's tensor costs
// more than that gives (574 us with one run, 607 us with these, before the pairs of groups).
constexpr uint32_t kRun = 32;

template <int CAP, int BITS>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(BITS)) adamw_kernel(const __grid_constant__ OptParams<CAP> p) {
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    // Read before this CTA arrives below: ctl changes only after every CTA has arrived.
    const volatile bs_adamw_ctl* ctl = p.ctl;
    const bool skip = ctl->skip != 0;
    if (!skip) {
        const uint32_t t = p.step ? p.step : static_cast<uint32_t>(ctl->step) + 1u;
        // once: 0: clip is for every step; 1: no norm since the last step; 3: this is a norm's step
        const float shared_clip = ctl->clip, own_clip = ctl->own_clip, clip = ctl->once == 1 ? own_clip : shared_clip;
        // 1 - b^t = -expm1(t log b): relative error of a few 2^-24 for every t
        const float bc1 = -expm1f(static_cast<float>(t * p.log_b1)), bc2 = -expm1f(static_cast<float>(t * p.log_b2));
        StepConst c{p.b1, p.b2, p.c1, p.c2, p.eps, clip, ctl->lr, 0.f, rsqrtf(bc2)};
        c.step = c.lr / bc1;
        const uint64_t key0 = mix64(p.seed + t * 2654435769ull);
        // A CTA's runs of per_cta groups; a run may cross tensors, and warp w takes the groups at w,
        // w + 8, .. of it.
        for (uint32_t g0 = blockIdx.x * p.per_cta; g0 < p.groups; g0 += gridDim.x * p.per_cta) {
        const uint32_t g1 = min(g0 + p.per_cta, p.groups);
        for (uint32_t k = static_cast<uint32_t>(item_of(p, g0, 0)); k < p.n_items; ++k) {
            const OptItem& it = p.item[k];
            const uint32_t base = it.group_begin, lo = max(g0, base);
            if (lo >= g1) break;
            const uint32_t last = k + 1 < p.n_items ? p.item[k + 1].group_begin : p.groups;
            const uint32_t begin = lo + ((warp - (lo - g0)) & (kWarps - 1u)) - base, end = min(g1, last) - base;
            const float decay = c.lr * it.decay, keep = 1.f - c.lr * it.decay;
            const uint64_t key = BITS == 8 ? mix64(key0 + it.tensor) : 0;
            const uint32_t whole = it.flags & kVec ? min(end, static_cast<uint32_t>(it.n / kBlock)) : 0u;
            switch ((it.flags & (kP16 | kG16)) | (it.master ? 4u : 0u)) {
            case 0: groups_of_kind<BITS, false, false, false>(it, c, decay, keep, key, lane, begin, whole); break;
            case kP16: groups_of_kind<BITS, true, false, false>(it, c, decay, keep, key, lane, begin, whole); break;
            case kG16: groups_of_kind<BITS, false, true, false>(it, c, decay, keep, key, lane, begin, whole); break;
            case kP16 | kG16: groups_of_kind<BITS, true, true, false>(it, c, decay, keep, key, lane, begin, whole); break;
            case 4: groups_of_kind<BITS, false, false, true>(it, c, decay, keep, key, lane, begin, whole); break;
            case kP16 | 4: groups_of_kind<BITS, true, false, true>(it, c, decay, keep, key, lane, begin, whole); break;
            case kG16 | 4: groups_of_kind<BITS, false, true, true>(it, c, decay, keep, key, lane, begin, whole); break;
            default: groups_of_kind<BITS, true, true, true>(it, c, decay, keep, key, lane, begin, whole); break;
            }
            // the tensor's last group where it is part-filled, and every group of unaligned tensors
            uint32_t b = begin;
            if (whole > begin) b += (whole - begin + kWarps - 1) / kWarps * kWarps;
            for (; b < end; b += kWarps) {
                const uint64_t at = uint64_t(b) * kBlock + 8u * lane;
                const uint32_t cnt = at < it.n ? static_cast<uint32_t>(it.n - at < 8 ? it.n - at : 8) : 0u;
                const bool p16 = it.flags & kP16, g16 = it.flags & kG16, master = it.master != nullptr;
                Held<BITS> h;
                load_group<BITS>(h, it, b, at, p16, g16, master, false, cnt);
                step_group<BITS>(h, it, c, decay, keep, key, lane, b, at, p16, g16, master, false, cnt);
            }
        }
        }
    } else if (p.into) {
        copy_all<CAP, BITS>(p);
    }
    if (!p.last) return;
    __syncthreads();
    if (threadIdx.x != 0) return;
    // again, beside the arrival: kept from above they would take registers all the way
    const uint32_t once = __ldcg(&p.ctl->once);
    const float own_clip = __ldcg(&p.ctl->own_clip);
    if (atomicInc(&p.ctl->arrived, gridDim.x - 1) != gridDim.x - 1) return;
    if (!skip) p.ctl->step = p.step ? static_cast<int32_t>(p.step) : p.ctl->step + 1;
    if (once == 1) p.ctl->clip = own_clip;
    if (once == 3) { // this was the norm's step
        p.ctl->skip = 0;
        p.ctl->once = 1;
    }
}

// The squares of 4 groups of a warp, kWarps groups apart, all loads before the sums.
template <bool B16>
__device__ __forceinline__ double run_squares(const uint8_t* g, uint64_t at) {
    uint32_t r[4][8];
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) load_raw(r[j], g, at + j * kWarps * kBlock, B16, true, 8);
    double sum = 0;
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) {
        float f[8], part = 0;
        unpack(f, r[j], B16);
#pragma unroll
        for (int i = 0; i < 8; ++i) part = fmaf(f[i], f[i], part);
        sum += part;
    }
    return sum;
}

// Sum of squares: FP32 over a lane's 8 elements of a group, 64 bits from there on. Every
// CTA's sum goes to its place; the last CTA to arrive adds them in the order of their places.
template <int CAP>
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ NormParams<CAP> p) {
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    __shared__ double s_sum[kWarps];
    __shared__ bool s_last;
    double sum = 0;
    int k0 = 0; // the runs go up, so the search for a run's tensor starts at the last one's
    for (uint32_t g0 = blockIdx.x * kRun; g0 < p.groups; g0 += gridDim.x * kRun) { // 4 groups' loads at once
        if (k0 + 1 < static_cast<int>(p.n_items) && p.item[k0 + 1].group_begin <= g0) k0 = item_of(p, g0, k0);
        const NormItem& first = p.item[k0];
        const uint32_t in = g0 - first.group_begin;
        if ((first.flags & kVec) && (uint64_t(in) + kRun) * kBlock <= first.n) { // whole groups of one tensor
            const uint64_t at = uint64_t(in + warp) * kBlock + 8u * lane;
            if (first.flags & kG16) sum += run_squares<true>(first.g, at);
            else sum += run_squares<false>(first.g, at);
            continue;
        }
        int k = k0;
        uint32_t r[4][8];
        bool b16[4];
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {
            const uint32_t gr = g0 + warp + j * kWarps;
            b16[j] = false;
#pragma unroll
            for (int i = 0; i < 8; ++i) r[j][i] = 0;
            if (gr < p.groups) {
                if (k + 1 < static_cast<int>(p.n_items) && p.item[k + 1].group_begin <= gr) k = item_of(p, gr, k);
                const NormItem& it = p.item[k];
                const uint64_t at = uint64_t(gr - it.group_begin) * kBlock + 8u * lane;
                const uint32_t cnt = at < it.n ? static_cast<uint32_t>(it.n - at < 8 ? it.n - at : 8) : 0u;
                b16[j] = it.flags & kG16;
                load_raw(r[j], it.g, at, b16[j], cnt == 8 && (it.flags & kVec), cnt);
            }
        }
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {
            float part = 0;
            if (b16[j]) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float lo = __uint_as_float(r[j][i] << 16), hi = __uint_as_float(r[j][i] & 0xFFFF0000u);
                    part = fmaf(lo, lo, part);
                    part = fmaf(hi, hi, part);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) part = fmaf(__uint_as_float(r[j][i]), __uint_as_float(r[j][i]), part);
            }
            sum += part;
        }
    }
    auto cta_sum = [&](double x) { // every thread's x, added in a fixed order; valid in thread 0
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
        if (lane == 0) s_sum[warp] = x;
        __syncthreads();
        double r = 0;
        if (threadIdx.x == 0)
            for (int i = 0; i < kWarps; ++i) r += s_sum[i];
        __syncthreads();
        return r;
    };
    const double mine = cta_sum(sum);
    if (threadIdx.x == 0) {
        __stcg(p.partial + p.partial_at + blockIdx.x, mine);
        __threadfence();
        s_last = p.last && atomicInc(&p.ctl->arrived, gridDim.x - 1) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    const uint32_t once = threadIdx.x == 0 ? __ldcg(&p.ctl->once) : 0;
    double x = 0;
    for (uint32_t i = threadIdx.x; i < p.partial_at + gridDim.x; i += kThreads) x += __ldcg(p.partial + i);
    x = cta_sum(x);
    if (threadIdx.x == 0) {
        const float norm = static_cast<float>(sqrt(x));
        const bool finite = norm < __uint_as_float(0x7F800000u);
        p.ctl->norm = norm;
        if (once) p.ctl->once = 3;
        p.ctl->skip = finite ? 0u : 1u;
        p.ctl->clip = finite ? static_cast<float>(fmin(1.0, static_cast<double>(p.max_norm) / (sqrt(x) + 1e-6))) : 0.f;
    }
}

// The 8-bit moments as FP32 values.
template <int CAP>
__global__ void __launch_bounds__(kThreads) read_states_kernel(const __grid_constant__ OptParams<CAP> p) {
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    int k0 = 0; // the runs go up, so the search for a run's tensor starts at the last one's
    for (uint32_t g0 = blockIdx.x * kRun; g0 < p.groups; g0 += gridDim.x * kRun) {
        if (k0 + 1 < static_cast<int>(p.n_items) && p.item[k0 + 1].group_begin <= g0) k0 = item_of(p, g0, k0);
        const OptItem& first = p.item[k0]; // to.m, to.v: FP32
        const uint32_t in = g0 - first.group_begin;
        if ((first.flags & kVec) && (uint64_t(in) + kRun) * kBlock <= first.n) { // whole groups of one tensor: 4 groups' loads at once
            uint2 m[4], v[4];
            float sm[4], sv[4];
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) { // 4 elements of each half a lane, so that a warp's store is one stretch: 367 us, 501 us with 8 in a row
                const uint64_t block = in + warp + j * kWarps, at = block * kBlock + 4u * lane;
                m[j] = make_uint2(*reinterpret_cast<const uint32_t*>(first.m + at), *reinterpret_cast<const uint32_t*>(first.m + at + 128));
                v[j] = make_uint2(*reinterpret_cast<const uint32_t*>(first.v + at), *reinterpret_cast<const uint32_t*>(first.v + at + 128));
                sm[j] = first.ms[block];
                sv[j] = first.vs[block];
            }
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) {
                const uint64_t at = uint64_t(in + warp + j * kWarps) * kBlock + 4u * lane;
                float f[8];
                decode_m(f, m[j], sm[j]);
                float* d = reinterpret_cast<float*>(first.to.m) + at;
                *reinterpret_cast<float4*>(d) = make_float4(f[0], f[1], f[2], f[3]);
                *reinterpret_cast<float4*>(d + 128) = make_float4(f[4], f[5], f[6], f[7]);
                decode_v(f, v[j], sv[j]);
                d = reinterpret_cast<float*>(first.to.v) + at;
                *reinterpret_cast<float4*>(d) = make_float4(f[0], f[1], f[2], f[3]);
                *reinterpret_cast<float4*>(d + 128) = make_float4(f[4], f[5], f[6], f[7]);
            }
            continue;
        }
        const uint32_t g1 = min(g0 + kRun, p.groups);
        int k = k0;
        for (uint32_t gr = g0 + warp; gr < g1; gr += kWarps) {
            if (k + 1 < static_cast<int>(p.n_items) && p.item[k + 1].group_begin <= gr) k = item_of(p, gr, k);
            const OptItem& it = p.item[k];
            const uint64_t block = gr - it.group_begin, at = block * kBlock + 8u * lane;
            const uint32_t cnt = at < it.n ? static_cast<uint32_t>(it.n - at < 8 ? it.n - at : 8) : 0u;
            const bool full = cnt == 8 && (it.flags & kVec);
            float f[8];
            decode_m(f, load_codes(it.m, at, full, cnt), it.ms[block]);
            store8(f, it.to.m, at, false, full, cnt);
            decode_v(f, load_codes(it.v, at, full, cnt), it.vs[block]);
            store8(f, it.to.v, at, false, full, cnt);
        }
    }
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

enum class Pass { Step, To, Norm, Read };

// What the three entry points check of an item alike; the pointers that the pass uses must be set
// and naturally aligned.
bs_status check_items(int32_t n, const bs_adamw_item* items, uint32_t bits, Pass pass) {
    if (n < 0 || (n > 0 && !items)) return BS_E_ARG;
    for (int32_t k = 0; k < n; ++k) {
        const bs_adamw_item& t = items[k];
        if (t.n > (1ull << 34)) return BS_E_SIZE; // 2^26 groups
        if (t.param_type > BS_TYPE_BF16 || t.grad_type > BS_TYPE_BF16) return BS_E_ARG;
        if (t.n == 0) continue;
        const uint32_t ga = t.grad_type == BS_TYPE_BF16 ? 2 : 4, pa = t.param_type == BS_TYPE_BF16 ? 2 : 4;
        if ((pass == Pass::Step || pass == Pass::Norm) && (!t.d_grad || !aligned(t.d_grad, ga))) return BS_E_ARG;
        if (pass == Pass::Norm) continue;
        if (pass != Pass::Read) {
            if (!t.d_param || !aligned(t.d_param, pa) || !aligned(t.d_master, 4)) return BS_E_ARG;
            if (pass == Pass::Step && !(t.weight_decay >= 0.f && t.weight_decay < INFINITY)) return BS_E_ARG;
        }
        if (!t.d_m || !t.d_v) return BS_E_ARG;
        if (bits == 32 && (!aligned(t.d_m, 4) || !aligned(t.d_v, 4))) return BS_E_ARG;
        if (bits == 8 && (!t.d_m_scale || !t.d_v_scale || !aligned(t.d_m_scale, 4) || !aligned(t.d_v_scale, 4))) return BS_E_ARG;
    }
    return BS_OK;
}

uint64_t groups_of(uint64_t n) { return (n + kBlock - 1) / kBlock; }

// The CTAs of a pass are one wave: more of them would pay their set-up (the step's constants, the
// search for the first tensor) for every few groups.
constexpr uint32_t kNormCtas = 148 * 5; // of the norm; not the device's own number, so that the order of the sums is one

template <int CAP>
bs_status launch_all(Pass pass, int32_t n, const bs_adamw_item* items, const bs_adamw_item* to, uint32_t bits, float* const* rm,
                     float* const* rv, OptParams<CAP>& p, int sms, cudaStream_t s) {
    int32_t k = 0, left = 0;
    for (int32_t i = 0; i < n; ++i) left += items[i].n != 0;
    do {
        p.n_items = 0;
        uint64_t groups = 0;
        for (; k < n && p.n_items < static_cast<uint32_t>(CAP); ++k) {
            const bs_adamw_item &t = items[k], &d = to[k];
            if (t.n == 0) continue;
            if (groups + groups_of(t.n) > (1ull << 31)) break;
            OptItem& it = p.item[p.n_items++];
            it.p = static_cast<const uint8_t*>(t.d_param);
            it.g = static_cast<const uint8_t*>(t.d_grad);
            it.m = static_cast<const uint8_t*>(t.d_m);
            it.v = static_cast<const uint8_t*>(t.d_v);
            it.master = t.d_master;
            it.ms = t.d_m_scale;
            it.vs = t.d_v_scale;
            it.to = OptOut{static_cast<uint8_t*>(d.d_param), static_cast<uint8_t*>(d.d_m), static_cast<uint8_t*>(d.d_v),
                           d.d_master, d.d_m_scale, d.d_v_scale};
            it.n = t.n;
            it.group_begin = static_cast<uint32_t>(groups);
            it.decay = t.weight_decay;
            it.tensor = static_cast<uint32_t>(k);
            bool vec;
            if (pass == Pass::Read) {
                it.to.m = reinterpret_cast<uint8_t*>(rm[k]);
                it.to.v = reinterpret_cast<uint8_t*>(rv[k]);
                vec = aligned(it.m, 8) && aligned(it.v, 8) && aligned(it.to.m, 16) && aligned(it.to.v, 16);
            } else {
                const uintptr_t a = bits == 8 ? 8 : 16;
                vec = aligned(it.p, 16) && aligned(it.g, 16) && aligned(it.master, 16) && aligned(it.m, a) && aligned(it.v, a) &&
                      aligned(it.to.p, 16) && aligned(it.to.master, 16) && aligned(it.to.m, a) && aligned(it.to.v, a);
            }
            it.flags = (t.param_type == BS_TYPE_BF16 ? kP16 : 0u) | (t.grad_type == BS_TYPE_BF16 ? kG16 : 0u) | (vec ? kVec : 0u);
            groups += groups_of(t.n);
            --left;
        }
        p.groups = static_cast<uint32_t>(groups);
        p.last = left == 0;
        const uint64_t wave = uint64_t(sms) * (pass == Pass::Read ? kReadCtas : ctas_per_sm(bits));
        p.per_cta = pass == Pass::Read ? kRun : static_cast<uint32_t>(std::max<uint64_t>(kWarps, std::min<uint64_t>(bits == 32 ? kRun : ~0u, (groups + wave - 1) / wave)));
        const uint32_t ctas = static_cast<uint32_t>(std::max<uint64_t>(1, std::min<uint64_t>(wave, (groups + p.per_cta - 1) / p.per_cta)));
        if (pass == Pass::Read) read_states_kernel<CAP><<<ctas, kThreads, 0, s>>>(p);
        else if (bits == 8) adamw_kernel<CAP, 8><<<ctas, kThreads, 0, s>>>(p);
        else adamw_kernel<CAP, 32><<<ctas, kThreads, 0, s>>>(p);
        count_launch();
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_status(e);
    } while (left > 0);
    return BS_OK;
}

template <int CAP>
bs_status launch_norm(int32_t n, const bs_adamw_item* items, NormParams<CAP>& p, cudaStream_t s) {
    int32_t k = 0, left = 0;
    for (int32_t i = 0; i < n; ++i) left += items[i].n != 0;
    do {
        p.n_items = 0;
        uint64_t groups = 0;
        for (; k < n && p.n_items < static_cast<uint32_t>(CAP); ++k) {
            const bs_adamw_item& t = items[k];
            if (t.n == 0) continue;
            if (groups + groups_of(t.n) > (1ull << 31)) break;
            p.item[p.n_items++] = NormItem{static_cast<const uint8_t*>(t.d_grad), t.n, static_cast<uint32_t>(groups),
                                           (t.grad_type == BS_TYPE_BF16 ? kG16 : 0u) | (aligned(t.d_grad, 16) ? kVec : 0u)};
            groups += groups_of(t.n);
            --left;
        }
        p.groups = static_cast<uint32_t>(groups);
        p.last = left == 0;
        const uint32_t ctas = static_cast<uint32_t>(std::max<uint64_t>(1, std::min<uint64_t>(kNormCtas, (groups + kRun - 1) / kRun)));
        grad_norm_kernel<CAP><<<ctas, kThreads, 0, s>>>(p);
        count_launch();
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_status(e);
        p.partial_at += ctas;
    } while (left > 0);
    return BS_OK;
}

// The parameter block of a launch takes the room of its items: calls of few tensors use a small one.
template <typename Fill>
bs_status launch_sized(Pass pass, int32_t n, const bs_adamw_item* items, const bs_adamw_item* to, uint32_t bits,
                       float* const* rm, float* const* rv, int sms, cudaStream_t s, Fill fill) {
    if (n <= kFewItems) {
        OptParams<kFewItems> p;
        std::memset(&p, 0, offsetof(OptParams<kFewItems>, item));
        fill(p);
        return launch_all(pass, n, items, to, bits, rm, rv, p, sms, s);
    }
    std::unique_ptr<OptParams<kManyItems>> p(new (std::nothrow) OptParams<kManyItems>);
    if (!p) return BS_E_NOMEM;
    std::memset(p.get(), 0, offsetof(OptParams<kManyItems>, item));
    fill(*p);
    return launch_all(pass, n, items, to, bits, rm, rv, *p, sms, s);
}

} // namespace
} // namespace bs

using namespace bs;

extern "C" size_t bs_grad_norm_scratch_bytes(int32_t n, const bs_adamw_item* items) {
    if (check_items(n, items, 32, Pass::Norm) != BS_OK) return 0;
    // a launch takes 32 tensors at least, or all: that many of 2^26 groups stay within 2^31
    return sizeof(double) * kNormCtas * (2 + static_cast<size_t>(n) / 32);
}

extern "C" bs_status bs_grad_norm(int32_t n, const bs_adamw_item* items, float max_norm, bs_adamw_ctl* d_ctl, void* d_scratch,
                                  size_t scratch_bytes, void* stream) {
    bs_status st = check_items(n, items, 32, Pass::Norm);
    if (st != BS_OK) return st;
    if (!d_ctl || !aligned(d_ctl, 16) || !d_scratch || !aligned(d_scratch, 8) || !(max_norm > 0.f)) return BS_E_ARG;
    if (scratch_bytes < bs_grad_norm_scratch_bytes(n, items)) return BS_E_SIZE;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms)) != BS_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto go = [&](auto& p) {
        p.partial_at = 0;
        p.max_norm = max_norm;
        p.ctl = d_ctl;
        p.partial = static_cast<double*>(d_scratch);
        return launch_norm(n, items, p, s);
    };
    if (n <= kFewNorm) {
        NormParams<kFewNorm> p;
        return go(p);
    }
    std::unique_ptr<NormParams<kManyNorm>> p(new (std::nothrow) NormParams<kManyNorm>);
    return p ? go(*p) : BS_E_NOMEM;
}

extern "C" bs_status bs_adamw(int32_t n, const bs_adamw_item* items, const bs_adamw_item* to, const bs_adamw_params* prm,
                              bs_adamw_ctl* d_ctl, void* stream) {
    if (!prm || !d_ctl || !aligned(d_ctl, 16) || (prm->bits != 8 && prm->bits != 32) || prm->step > 0x7FFFFFFFu) return BS_E_ARG;
    if (!(prm->beta1 >= 0 && prm->beta1 < 1) || !(prm->beta2 >= 0 && prm->beta2 < 1) || !(prm->eps >= 1e-12 && prm->eps < INFINITY))
        return BS_E_ARG;
    bs_status st = check_items(n, items, prm->bits, Pass::Step);
    if (st != BS_OK) return st;
    if (!to) {
        to = items;
    } else {
        if ((st = check_items(n, to, prm->bits, Pass::To)) != BS_OK) return st;
        for (int32_t k = 0; k < n; ++k)
            if (to[k].n != items[k].n || to[k].param_type != items[k].param_type || !to[k].d_master != !items[k].d_master) return BS_E_ARG;
    }
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms)) != BS_OK) return st;
    return launch_sized(Pass::Step, n, items, to, prm->bits, nullptr, nullptr, sms, static_cast<cudaStream_t>(stream), [&](auto& p) {
        p.b1 = static_cast<float>(prm->beta1);
        p.b2 = static_cast<float>(prm->beta2);
        p.c1 = static_cast<float>(1.0 - prm->beta1);
        p.c2 = static_cast<float>(1.0 - prm->beta2);
        p.eps = static_cast<float>(prm->eps);
        p.log_b1 = prm->beta1 > 0 ? std::log(prm->beta1) : -1e9; // beta 0: 1 - 0^t = 1
        p.log_b2 = prm->beta2 > 0 ? std::log(prm->beta2) : -1e9;
        p.seed = prm->seed;
        p.step = prm->step;
        p.into = to != items;
        p.ctl = d_ctl;
    });
}

extern "C" bs_status bs_adamw_read_states(int32_t n, const bs_adamw_item* items, float* const* d_m, float* const* d_v, void* stream) {
    bs_status st = check_items(n, items, 8, Pass::Read);
    if (st != BS_OK) return st;
    if (n > 0 && (!d_m || !d_v)) return BS_E_ARG;
    bool any = false;
    for (int32_t k = 0; k < n; ++k) {
        if (items[k].n == 0) continue;
        any = true;
        if (!d_m[k] || !d_v[k] || !aligned(d_m[k], 4) || !aligned(d_v[k], 4)) return BS_E_ARG;
    }
    if (!any) return BS_OK;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms)) != BS_OK) return st;
    return launch_sized(Pass::Read, n, items, items, 8, d_m, d_v, sms, static_cast<cudaStream_t>(stream), [](auto&) {});
}
