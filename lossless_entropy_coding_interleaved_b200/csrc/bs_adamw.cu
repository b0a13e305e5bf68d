// bs_adamw.cu -- one AdamW step over many tensors in one launch, moments in 32 bits or in 8 bits
// with a scale for each 256 elements, and the norm of all gradients before it.
//
//   g = clip * grad;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g g
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Both kernels are one pass over their bytes and bound by them. A warp takes 256 consecutive
// elements at a time, 8 a lane: 16 bytes of BF16 or 32 of FP32 per lane and tensor, all loads of a
// group issued before its arithmetic. 256 elements are also one block of the 8-bit moments, so a
// block's largest magnitude is one warp reduction and nothing is exchanged between warps.
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

template <int CAP>
struct OptParams {
    uint32_t n_items, groups, per_cta; // groups of the launch, groups a CTA takes
    uint32_t last;                     // the call's last launch
    uint32_t step;                     // the step's number, 0: one more than ctl->step
    float b1, b2, c1, c2, eps;         // c = 1 - b, rounded from 64 bits
    float max_norm;
    double log_b1, log_b2;
    uint64_t seed;
    bs_adamw_ctl* ctl;
    double* partial;                   // norm: one sum a CTA, those of earlier launches before it
    uint32_t partial_at;
    OptItem item[CAP];
};
static_assert(sizeof(OptParams<kManyItems>) < 32764, "kernel parameters");

__device__ __forceinline__ uint64_t mix64(uint64_t z) { // splitmix64's output function
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}
__device__ __forceinline__ float bf16_bits(uint32_t lo16) { return __uint_as_float(lo16 << 16); }
__device__ __forceinline__ uint32_t to_bf16(float f) { // to nearest, ties to even; NaN stays NaN
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (u >> 16) | 0x40u;
    return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

// 8 elements of a lane, from `at` on; with `full` false only the first `cnt` exist (0 for the others).
__device__ __forceinline__ void load8(float (&f)[8], const uint8_t* base, uint64_t at, bool b16, bool full, uint32_t cnt) {
    if (b16) {
        const uint16_t* s = reinterpret_cast<const uint16_t*>(base) + at;
        if (full) {
            const uint4 w = *reinterpret_cast<const uint4*>(s);
            const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) { f[2 * i] = bf16_bits(q[i] & 0xFFFFu); f[2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u); }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = i < cnt ? bf16_bits(s[i]) : 0.f;
        }
    } else {
        const float* s = reinterpret_cast<const float*>(base) + at;
        if (full) {
            const float4 a = *reinterpret_cast<const float4*>(s), b = *reinterpret_cast<const float4*>(s + 4);
            f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = i < cnt ? s[i] : 0.f;
        }
    }
}
__device__ __forceinline__ void store8(const float (&f)[8], uint8_t* base, uint64_t at, bool b16, bool full, uint32_t cnt) {
    if (b16) {
        uint16_t* d = reinterpret_cast<uint16_t*>(base) + at;
        if (full) {
            uint4 w;
            w.x = to_bf16(f[0]) | (to_bf16(f[1]) << 16); w.y = to_bf16(f[2]) | (to_bf16(f[3]) << 16);
            w.z = to_bf16(f[4]) | (to_bf16(f[5]) << 16); w.w = to_bf16(f[6]) | (to_bf16(f[7]) << 16);
            *reinterpret_cast<uint4*>(d) = w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) if (i < cnt) d[i] = static_cast<uint16_t>(to_bf16(f[i]));
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
    for (int i = 0; i < 8; ++i) {
        const uint32_t c = (q[i >> 2] >> (8 * (i & 3))) & 0xFFu;
        f[i] = __fmul_rn(__half2float(__ushort_as_half(static_cast<unsigned short>(c << 7))), scale);
    }
}
// The code of y >= 0, rounded up where the 16 random bits u reach what is left of y below it.
template <int BIAS, uint32_t MOST>
__device__ __forceinline__ uint32_t encode(float y, uint32_t u) {
    const uint32_t normal = ((__float_as_uint(y) + (u << 4)) >> 20) - ((127 - BIAS) << 3);
    const uint32_t small = static_cast<uint32_t>(static_cast<int>(
        __fadd_rn(__fmul_rn(y, static_cast<float>(1 << (BIAS + 2))), __fmul_rn(static_cast<float>(u), 1.f / 65536.f))));
    return min(y < 1.f / static_cast<float>(1 << (BIAS - 1)) ? small : normal, MOST);
}
// The largest magnitude of the block; NaN when any is NaN (as integers, every NaN is above infinity).
__device__ __forceinline__ float block_max(const float (&f)[8]) {
    uint32_t b = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) b = max(b, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, b));
}

template <int CAP>
__device__ __forceinline__ int item_of(const OptParams<CAP>& p, uint32_t group, int lo) {
    int hi = static_cast<int>(p.n_items) - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.item[mid].group_begin <= group) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <int CAP, int BITS>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ OptParams<CAP> p) {
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    // Read before this CTA arrives below: the step count moves only after every CTA has arrived.
    const volatile bs_adamw_ctl* ctl = p.ctl;
    const bool skip = ctl->skip != 0;
    if (!skip) {
        const float lr = ctl->lr, clip = ctl->clip;
        const uint32_t t = p.step ? p.step : static_cast<uint32_t>(ctl->step) + 1u;
        // 1 - b^t = -expm1(t log b): relative error of a few 2^-24 for every t
        const float bc1 = -expm1f(static_cast<float>(t * p.log_b1)), bc2 = -expm1f(static_cast<float>(t * p.log_b2));
        const float step = lr / bc1, r2 = rsqrtf(bc2);
        const uint64_t key0 = mix64(p.seed + t * 2654435769ull);
        const uint32_t g0 = blockIdx.x * p.per_cta, g1 = min(g0 + p.per_cta, p.groups);
        int k = item_of(p, g0, 0);
        for (uint32_t gr = g0 + warp; gr < g1; gr += kWarps) {
            if (k + 1 < static_cast<int>(p.n_items) && p.item[k + 1].group_begin <= gr) k = item_of(p, gr, k);
            const OptItem& it = p.item[k];
            const uint64_t block = gr - it.group_begin, at = block * kBlock + 8u * lane;
            const uint32_t cnt = at < it.n ? static_cast<uint32_t>(it.n - at < 8 ? it.n - at : 8) : 0u;
            const bool full = cnt == 8 && (it.flags & kVec);
            const bool p16 = it.flags & kP16, g16 = it.flags & kG16;
            float g[8], m[8], v[8], w[8];
            load8(g, it.g, at, g16, full, cnt);
            if (it.master) load8(w, reinterpret_cast<const uint8_t*>(it.master), at, false, full, cnt);
            else load8(w, it.p, at, p16, full, cnt);
            if (BITS == 32) {
                load8(m, it.m, at, false, full, cnt);
                load8(v, it.v, at, false, full, cnt);
            } else {
                const uint2 cm = load_codes(it.m, at, full, cnt), cv = load_codes(it.v, at, full, cnt);
                decode_m(m, cm, it.ms[block]);
                decode_v(v, cv, it.vs[block]);
            }
            const float keep = 1.f - lr * it.decay;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float gi = __fmul_rn(g[i], clip);
                m[i] = __fadd_rn(__fmul_rn(m[i], p.b1), __fmul_rn(gi, p.c1));
                v[i] = __fadd_rn(__fmul_rn(v[i], p.b2), __fmul_rn(__fmul_rn(gi, p.c2), gi));
                w[i] = w[i] * keep - step * __fdividef(m[i], sqrtf(v[i]) * r2 + p.eps);
            }
            store8(w, it.to.p, at, p16, full, cnt);
            if (it.master) store8(w, reinterpret_cast<uint8_t*>(it.to.master), at, false, full, cnt);
            if (BITS == 32) {
                store8(m, it.to.m, at, false, full, cnt);
                store8(v, it.to.v, at, false, full, cnt);
            } else {
                const float bm = block_max(m), bv = block_max(v);
                const bool dm = bm < kDead, dv = bv < kDead; // false for NaN, which the scale then carries
                const float im = dm ? 0.f : __fdiv_rn(kTopM, bm), iv = dv ? 0.f : __fdiv_rn(kTopV, bv);
                const uint64_t key = mix64(key0 + it.tensor);
                uint32_t qm[2] = {0, 0}, qv[2] = {0, 0};
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const uint64_t z = mix64(key + 0x9E3779B97F4A7C15ull * (((at + i) >> 1) + 1));
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t u = static_cast<uint32_t>(z >> (32 * h)), e = i + h, sh = 8 * (e & 3);
                        const uint32_t cm = encode<7, 0x7E>(__fmul_rn(fabsf(m[e]), im), u & 0xFFFFu);
                        uint32_t cv = encode<15, 0xF7>(__fmul_rn(v[e], iv), u >> 16);
                        if (v[e] > 0.f && !dv) cv = max(cv, 1u);
                        qm[e >> 2] |= (cm | ((__float_as_uint(m[e]) >> 24) & 0x80u)) << sh;
                        qv[e >> 2] |= cv << sh;
                    }
                }
                store_codes(make_uint2(qm[0], qm[1]), it.to.m, at, full, cnt);
                store_codes(make_uint2(qv[0], qv[1]), it.to.v, at, full, cnt);
                if (lane == 0) {
                    it.to.ms[block] = dm ? 0.f : __fdiv_rn(bm, kTopM);
                    it.to.vs[block] = dv ? 0.f : __fdiv_rn(bv, kTopV);
                }
            }
        }
    }
    if (!p.last) return;
    __syncthreads();
    if (threadIdx.x == 0 && atomicInc(&p.ctl->arrived, gridDim.x - 1) == gridDim.x - 1 && !skip)
        p.ctl->step = p.step ? static_cast<int32_t>(p.step) : p.ctl->step + 1;
}

// Sum of squares: FP32 over a lane's elements of 8 groups at most, 64 bits from there on. Every
// CTA's sum goes to its place; the last CTA to arrive adds them in the order of their places.
template <int CAP>
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ OptParams<CAP> p) {
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    __shared__ double s_sum[kWarps];
    __shared__ bool s_last;
    double sum = 0;
    const uint32_t g0 = blockIdx.x * p.per_cta, g1 = min(g0 + p.per_cta, p.groups);
    if (g0 < g1) {
        int k = item_of(p, g0, 0);
        float part = 0;
        uint32_t held = 0;
        for (uint32_t gr = g0 + warp; gr < g1; gr += kWarps) {
            if (k + 1 < static_cast<int>(p.n_items) && p.item[k + 1].group_begin <= gr) k = item_of(p, gr, k);
            const OptItem& it = p.item[k];
            const uint64_t at = uint64_t(gr - it.group_begin) * kBlock + 8u * lane;
            const uint32_t cnt = at < it.n ? static_cast<uint32_t>(it.n - at < 8 ? it.n - at : 8) : 0u;
            float g[8];
            load8(g, it.g, at, it.flags & kG16, cnt == 8 && (it.flags & kVec), cnt);
#pragma unroll
            for (int i = 0; i < 8; ++i) part = fmaf(g[i], g[i], part);
            if (++held == 8) { sum += part; part = 0; held = 0; }
        }
        sum += part;
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
    double x = 0;
    for (uint32_t i = threadIdx.x; i < p.partial_at + gridDim.x; i += kThreads) x += __ldcg(p.partial + i);
    x = cta_sum(x);
    if (threadIdx.x == 0) {
        const float norm = static_cast<float>(sqrt(x));
        const bool finite = norm < __uint_as_float(0x7F800000u);
        p.ctl->norm = norm;
        p.ctl->skip = finite ? 0u : 1u;
        p.ctl->clip = finite ? static_cast<float>(fmin(1.0, static_cast<double>(p.max_norm) / (sqrt(x) + 1e-6))) : 0.f;
    }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) read_states_kernel(const __grid_constant__ OptParams<CAP> p) {
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    const uint32_t g0 = blockIdx.x * p.per_cta, g1 = min(g0 + p.per_cta, p.groups);
    int k = item_of(p, g0, 0);
    for (uint32_t gr = g0 + warp; gr < g1; gr += kWarps) {
        if (k + 1 < static_cast<int>(p.n_items) && p.item[k + 1].group_begin <= gr) k = item_of(p, gr, k);
        const OptItem& it = p.item[k]; // to.m, to.v: FP32
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

bs_status device_ok(int* sms) {
    int dev = 0, major = 0, minor = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_status(e);
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    return major == 10 && minor == 0 ? BS_OK : BS_E_UNSUPPORTED;
}

uint64_t groups_of(uint64_t n) { return (n + kBlock - 1) / kBlock; }

// The CTAs of a pass: one wave of them (4 an SM, the most that fit), each with an equal run of
// groups and at least one group a warp. More CTAs than that pay their set-up (the step's
// constants, the search for the first tensor) for every few groups.
constexpr uint32_t kNormCtas = 148 * 4;

template <int CAP>
bs_status launch_all(Pass pass, int32_t n, const bs_adamw_item* items, const bs_adamw_item* to, uint32_t bits, float* const* rm,
                     float* const* rv, OptParams<CAP>& p, int sms, cudaStream_t s) {
    int32_t k = 0, left = 0;
    for (int32_t i = 0; i < n; ++i) left += items[i].n != 0;
    p.partial_at = 0;
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
            } else if (pass == Pass::Norm) {
                vec = aligned(it.g, 16);
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
        const uint64_t wave = pass == Pass::Norm ? kNormCtas : uint64_t(sms) * 4;
        p.per_cta = static_cast<uint32_t>(std::max<uint64_t>(kWarps, (groups + wave - 1) / wave));
        const uint32_t ctas = static_cast<uint32_t>(std::max<uint64_t>(1, (groups + p.per_cta - 1) / p.per_cta));
        if (pass == Pass::Norm) grad_norm_kernel<CAP><<<ctas, kThreads, 0, s>>>(p);
        else if (pass == Pass::Read) read_states_kernel<CAP><<<ctas, kThreads, 0, s>>>(p);
        else if (bits == 8) adamw_kernel<CAP, 8><<<ctas, kThreads, 0, s>>>(p);
        else adamw_kernel<CAP, 32><<<ctas, kThreads, 0, s>>>(p);
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
    // a launch takes kFewItems tensors at least, or all: that many of 2^26 groups stay below 2^31
    return sizeof(double) * kNormCtas * (2 + static_cast<size_t>(n) / kFewItems);
}

extern "C" bs_status bs_grad_norm(int32_t n, const bs_adamw_item* items, float max_norm, bs_adamw_ctl* d_ctl, void* d_scratch,
                                  size_t scratch_bytes, void* stream) {
    bs_status st = check_items(n, items, 32, Pass::Norm);
    if (st != BS_OK) return st;
    if (!d_ctl || !aligned(d_ctl, 16) || !d_scratch || !aligned(d_scratch, 8) || !(max_norm > 0.f)) return BS_E_ARG;
    if (scratch_bytes < bs_grad_norm_scratch_bytes(n, items)) return BS_E_SIZE;
    int sms = 148;
    if ((st = device_ok(&sms)) != BS_OK) return st;
    return launch_sized(Pass::Norm, n, items, items, 32, nullptr, nullptr, sms, static_cast<cudaStream_t>(stream), [&](auto& p) {
        p.max_norm = max_norm;
        p.ctl = d_ctl;
        p.partial = static_cast<double*>(d_scratch);
    });
}

extern "C" bs_status bs_adamw(int32_t n, const bs_adamw_item* items, const bs_adamw_item* to, const bs_adamw_params* prm,
                              bs_adamw_ctl* d_ctl, void* stream) {
    if (!prm || !d_ctl || !aligned(d_ctl, 16) || (prm->bits != 8 && prm->bits != 32) || prm->step > 0x7FFFFFFFu) return BS_E_ARG;
    if (!(prm->beta1 >= 0 && prm->beta1 < 1) || !(prm->beta2 >= 0 && prm->beta2 < 1) || !(prm->eps >= 0) || std::isinf(prm->eps))
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
    int sms = 148;
    if ((st = device_ok(&sms)) != BS_OK) return st;
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
    int sms = 148;
    if ((st = device_ok(&sms)) != BS_OK) return st;
    return launch_sized(Pass::Read, n, items, items, 8, d_m, d_v, sms, static_cast<cudaStream_t>(stream), [](auto&) {});
}
