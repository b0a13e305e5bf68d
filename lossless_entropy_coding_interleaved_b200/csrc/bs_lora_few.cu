// bs_lora_few.cu -- the adapters' forward product for batches of few tokens, as in decoding.
//
//   h[t] = s_a A_a x[t],  y[t] = base[t] + B_a h[t]
//
// With a token or a few per adapter the product is bound by the bytes of A and B, and at the
// smallest sizes by latency: two kernels with a trip of h through memory between them would cost
// more than the bytes. So one cluster of 8 CTAs takes up to 8 tokens of one adapter through both
// products: its 64 warps share the K range of A x, the CTAs exchange their sums of h (rank x 8
// numbers each) through distributed shared memory, and the warps share the rows of B h. The
// first rows of B are on their way to registers during that exchange.
//
// Weights are the matrix instructions' 16-row operand and the tokens the 8 columns of the other, so
// weights go from global memory to registers in the order that they lie in: a sum does not depend on
// the order of its terms, so each lane takes 16 (A) or 8 (B) contiguous bytes of a row and the tokens' side
// is indexed to match. Nothing is staged in shared memory but h. h enters the second product as three
// BF16 numbers (24 bits).
//
// On one B200: one token, q, k and v at rank 16: 9.5 us with the plan's launch, all of it latency. 37
// tokens of 24 adapters of rank up to 64, gate and up (14336 x 3584 each): 32 us with the plan's, 88 MB
// at 2.7 TB/s; with h through memory between two kernels 53 us.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "bs_lora.cuh"

namespace bs {
namespace lora {
namespace {
namespace cg = cooperative_groups;

constexpr uint32_t kWarps = kFewThreads / 32, kSlices = kFewCluster * kWarps;

__device__ __forceinline__ uint4 ld16(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }

// WORDS words from p, where `on`; what stands in d is undefined where not.
template <int WORDS>
__device__ __forceinline__ void load_if(uint32_t* d, const uint16_t* p, uint32_t on) {
    if constexpr (WORDS == 2)
        asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %3, 0;\n @p ld.global.v2.u32 {%0, %1}, [%2];\n}"
                     : "=r"(d[0]), "=r"(d[1]) : "l"(p), "r"(on));
    else
        asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %5, 0;\n @p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
                     : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]) : "l"(p), "r"(on));
}

// What a lane has of a block of 128 rows of B: words of its rows g and g + 8 of the warp's 16 (for
// R = 16, 4 ranks of each; else 8 ranks of each 32).
template <int R>
struct BRows {
    static constexpr int W = R == 16 ? 2 : R / 8; // words of a row
    uint32_t lo[W], hi[W];
};

// Blocks of rows whose loads a warp has under way while it works on one. At rank 64, 3 CTAs an SM with
// one block ahead take 41 us for 37 tokens over 24 adapters (14336 rows, twice); 2 CTAs with 4 ahead
// take 46, since clusters of 8 then leave slots of their group of SMs empty.
template <int R>
constexpr uint32_t kAhead = R > 32 ? 1 : 4;

// B h of a CTA gathers in shared memory, up to 16 blocks of 128 rows at a time, and goes from there to
// y with base added, token by token in whole lines: from the matrix instructions' registers it would
// be 4 scattered numbers a lane, most of them of tokens that the tile does not have.
constexpr uint32_t kHold = 16, kHoldRows = kHold * 128 + 4; // 4: another bank for each token
template <int R>
constexpr uint32_t few_smem() { return std::max<uint32_t>(kFew * kHoldRows * 4, kWarps * R * 8 * 4); }

template <int R>
__global__ void __launch_bounds__(kFewThreads, R == 16 ? 4 : R <= 64 ? 3 : 2) lora_few_kernel(const __grid_constant__ FewParams p) {
    constexpr int MT = R / 16;
    extern __shared__ __align__(16) float s_dyn[];
    __shared__ __align__(16) float s_part[R * 8], s_h[R * 8]; // [rank][token]
    float(*s_red)[R * 8] = reinterpret_cast<float(*)[R * 8]>(s_dyn); // [warps]
    float* s_y = s_dyn;                                              // [token][kHoldRows]
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5, g = lane >> 2, q = lane & 3u;
    const uint32_t cta = blockIdx.x % kFewCluster, part = blockIdx.x / kFewCluster % p.split, tile = blockIdx.x / kFewCluster / p.split;
    const FewJob& job = p.job[blockIdx.y];
    const uint32_t N = job.rows, K = job.cols, rm = p.b.rank_max;
    next_kernel_may_start();
    kernels_before_done();
    const PlanAt o = plan_at(p.b.tokens, p.b.n);
    const FewTile* entry = reinterpret_cast<const FewTile*>(p.b.plan + o.few) + tile;
    const uint32_t a = entry->bucket, first = entry->first, count = entry->count, tok_g = entry->token[g];
    if (tile >= plan_head(p.b).w) return; // the whole cluster
    if (a >= p.b.n) { // tokens without an adapter: base as it is
        if (!job.out || (job.base == job.out && job.base_stride == job.out_stride)) return;
        const uint32_t es = job.bf16 ? 2 : 4, pieces = N * es / 16;
        for (uint32_t t = 0; t < count; ++t) {
            const uint4* src = reinterpret_cast<const uint4*>(job.base + uint64_t(entry->token[t]) * job.base_stride * es);
            uint4* dst = reinterpret_cast<uint4*>(job.out + uint64_t(entry->token[t]) * job.out_stride * es);
            for (uint32_t i = (part * kFewCluster + cta) * kFewThreads + tid; i < pieces; i += p.split * kFewCluster * kFewThreads)
                dst[i] = job.base ? src[i] : make_uint4(0, 0, 0, 0);
        }
        return;
    }
    const uint32_t rank = rank_of(p.b, a);
    const float scale = p.b.scales ? p.b.scales[a] : 1.f;
    const uint16_t* A = job.a + uint64_t(a) * rm * K;
    const uint16_t* B = job.b + uint64_t(a) * rm * N;
    // ---- A x: the warp's columns, 64 at a time; lane (g, q) has row g (and g + 8) of each 16 ranks,
    // token g, and columns 8 q .. 8 q + 7 of each half of the 64. A warp's chain of sums is K / 1024
    // matrix instructions long.
    const uint16_t* x = g < count ? job.x + uint64_t(tok_g) * job.x_stride : nullptr;
    float acc[MT][4] = {};
    for (uint32_t k0 = (cta * kWarps + warp) * 64; k0 < K; k0 += kSlices * 64) {
#pragma unroll
        for (uint32_t half = 0; half < 2; ++half) {
            const uint32_t k = k0 + 32 * half + 8 * q;
            const bool on = k < K;
            uint4 xv = make_uint4(0, 0, 0, 0);
            if (on && x) xv = ld16(x + k);
            uint4 lo[MT], hi[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                lo[m] = hi[m] = make_uint4(0, 0, 0, 0);
                if (on && 16 * m + g < rank) lo[m] = ld16(A + uint64_t(16 * m + g) * K + k);
                if (on && 16 * m + g + 8 < rank) hi[m] = ld16(A + uint64_t(16 * m + g + 8) * K + k);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const uint32_t a0[4] = {lo[m].x, hi[m].x, lo[m].y, hi[m].y}, a1[4] = {lo[m].z, hi[m].z, lo[m].w, hi[m].w};
                mma16816(acc[m], a0, xv.x, xv.y);
                mma16816(acc[m], a1, xv.z, xv.w);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        *reinterpret_cast<float2*>(&s_red[warp][(16 * m + g) * 8 + 2 * q]) = make_float2(acc[m][0], acc[m][1]);
        *reinterpret_cast<float2*>(&s_red[warp][(16 * m + g + 8) * 8 + 2 * q]) = make_float2(acc[m][2], acc[m][3]);
    }
    __syncthreads();
    for (uint32_t i = tid; i < R * 8; i += kFewThreads) {
        float v = 0.f;
#pragma unroll
        for (uint32_t w = 0; w < kWarps; ++w) v += s_red[w][i];
        s_part[i] = v;
    }
    cg::cluster_group cluster = cg::this_cluster();
    cluster.barrier_arrive();
    // ranks past the adapter's are cut off: bits of this lane's pairs of the last 16 or 32
    constexpr uint32_t kStep = R == 16 ? 16 : 32, kLane = kStep / 4; // ranks of a lane in each step
    constexpr int W = BRows<R>::W, WS = kLane / 2;                   // words of a row, and in each step
    const uint32_t steps = (rank + kStep - 1) / kStep;
    uint32_t mask[WS];
#pragma unroll
    for (int i = 0; i < WS; ++i) {
        const uint32_t k = (steps - 1) * kStep + kLane * q + 2 * i; // not used where there are no steps
        mask[i] = k + 1 < rank ? ~0u : k < rank ? 0xFFFFu : 0u;
    }
    const uint16_t* rows_g = B + uint64_t(g) * rm + kLane * q;
    // The warp's 16 rows from n0 on (n0 < N; N is a multiple of 8, so the upper 8 are all there or not,
    // and stand for nothing where not). A lane whose ranks are all past the adapter's loads nothing:
    // its mask is 0.
    auto load = [&](BRows<R>& r, uint32_t n0) {
        const uint16_t* p0 = rows_g + uint64_t(n0) * rm;
        const uint16_t* p1 = n0 + 8 < N ? p0 + 8 * rm : p0;
#pragma unroll
        for (int m = 0; m < W / WS; ++m) {
            if (static_cast<uint32_t>(m) >= steps) break;
            const uint32_t on = kStep * m + kLane * q < rank;
            load_if<WS>(&r.lo[WS * m], p0 + kStep * m, on);
            load_if<WS>(&r.hi[WS * m], p1 + kStep * m, on);
        }
    };
    // the rows of B h in blocks of 128, dealt out to the CTAs of the tile's clusters, 16 rows a warp
    BRows<R> ring[kAhead<R>];
    const uint32_t first_row = (part * kFewCluster + cta) * 128 + warp * 16, row_deal = p.split * kFewCluster * 128;
    const uint32_t rows_end = job.out ? N : 0;
#pragma unroll
    for (uint32_t d = 0; d < kAhead<R>; ++d) // under way while the sums of h are exchanged
        if (first_row + d * row_deal < rows_end) load(ring[d], first_row + d * row_deal);
    cluster.barrier_wait();
    for (uint32_t i = tid; i < R * 8; i += kFewThreads) {
        float peer[kFewCluster], v = 0.f;
#pragma unroll
        for (uint32_t c = 0; c < kFewCluster; ++c) peer[c] = cluster.map_shared_rank(s_part, c)[i];
#pragma unroll
        for (uint32_t c = 0; c < kFewCluster; ++c) v += peer[c];
        s_h[i] = (i >> 3) < rank && (i & 7u) < count ? v * scale : 0.f;
    }
    cluster.barrier_arrive(); // the peers' sums have been read
    __syncthreads();
    if (part == 0 && cta < count && tid < R / 2) { // CTA c writes token c's h
        uint32_t lo[3], hi[3];
        split3(s_h[2 * tid * 8 + cta], lo);
        split3(s_h[(2 * tid + 1) * 8 + cta], hi);
        uint32_t* dst = reinterpret_cast<uint32_t*>(job.h) + (uint64_t(first + cta) * R) / 2 + tid;
#pragma unroll
        for (int t = 0; t < 3; ++t) dst[uint64_t(t) * (p.b.part_stride / 2)] = lo[t] | (hi[t] << 16);
    }
    // ---- B h: the token's side of each step, in the order of the lane's words
    uint32_t hf[W][3];
#pragma unroll
    for (int w = 0; w < W; ++w) {
        uint32_t lo[3], hi[3];
        const uint32_t k = w / WS * kStep + kLane * q + 2 * (w % WS);
        split3(s_h[k * 8 + g], lo);
        split3(s_h[(k + 1) * 8 + g], hi);
#pragma unroll
        for (int t = 0; t < 3; ++t) hf[w][t] = lo[t] | (hi[t] << 16);
    }
    for (uint32_t hold = first_row - warp * 16; hold < rows_end; hold += kHold * row_deal) { // the same for every warp
        for (uint32_t held = 0; held < kHold; held += kAhead<R>)
#pragma unroll
            for (uint32_t r = 0; r < kAhead<R>; ++r) {
                const uint32_t n0 = hold + warp * 16 + (held + r) * row_deal;
                if (n0 >= rows_end) break;
                BRows<R>& cur = ring[r];
                float d[4] = {};
#pragma unroll
                for (int m = 0; m < W / WS; ++m)
                    if (static_cast<uint32_t>(m) + 1 == steps) {
#pragma unroll
                        for (int i = 0; i < WS; ++i) {
                            cur.lo[m * WS + i] &= mask[i];
                            cur.hi[m * WS + i] &= mask[i];
                        }
                    }
#pragma unroll
                for (int t = 2; t >= 0; --t) // small parts first: the sum is rounded at its size R / 16 times, not three times as often
#pragma unroll
                    for (int m = 0; m < W / WS; ++m) {
                        if (static_cast<uint32_t>(m) >= steps) break;
#pragma unroll
                        for (int w = m * WS; w < (m + 1) * WS; w += 2) {
                            const uint32_t af[4] = {cur.lo[w], cur.hi[w], cur.lo[w + 1], cur.hi[w + 1]};
                            mma16816(d, af, hf[w][t], hf[w + 1][t]);
                        }
                    }
                if (n0 + kAhead<R> * row_deal < rows_end) load(cur, n0 + kAhead<R> * row_deal);
                float* y = s_y + 2 * q * kHoldRows + (held + r) * 128 + warp * 16 + g;
                if (2 * q < count) { y[0] = d[0]; y[8] = d[2]; }
                if (2 * q + 1 < count) { y[kHoldRows] = d[1]; y[kHoldRows + 8] = d[3]; }
            }
        __syncthreads();
        // 4 columns a thread: a block of 128 by a warp
        const uint32_t left = (rows_end - hold + row_deal - 1) / row_deal, n_held = min(left, kHold);
        for (uint32_t i = warp; i < n_held * count; i += kWarps) {
            const uint32_t t = i / n_held, block = i % n_held, n = hold + block * row_deal + 4 * lane;
            if (n >= N) continue;
            const uint32_t tok = entry->token[t];
            const float4 d = *reinterpret_cast<const float4*>(s_y + t * kHoldRows + block * 128 + 4 * lane);
            const uint64_t from = uint64_t(tok) * job.base_stride + n, to = uint64_t(tok) * job.out_stride + n;
            if (job.bf16) {
                uint2 v = make_uint2(0, 0);
                if (job.base) v = *reinterpret_cast<const uint2*>(job.base + 2 * from);
                v.x = bf16_of(__uint_as_float(v.x << 16) + d.x) | (bf16_of(__uint_as_float(v.x & 0xFFFF0000u) + d.y) << 16);
                v.y = bf16_of(__uint_as_float(v.y << 16) + d.z) | (bf16_of(__uint_as_float(v.y & 0xFFFF0000u) + d.w) << 16);
                *reinterpret_cast<uint2*>(job.out + 2 * to) = v;
            } else {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (job.base) v = *reinterpret_cast<const float4*>(job.base + 4 * from);
                *reinterpret_cast<float4*>(job.out + 4 * to) = make_float4(v.x + d.x, v.y + d.y, v.z + d.z, v.w + d.w);
            }
        }
        __syncthreads();
    }
    cluster.barrier_wait();
}

template <int R>
bs_status launch(FewParams& p, uint32_t jobs, int dev, int sms, cudaStream_t s) {
    // Where few tiles leave SMs idle, several clusters share a tile's rows of B h, and each works out
    // the whole of h, which costs them the same time.
    const uint32_t tiles = tile_cap(p.b.tokens, p.b.n, kFew);
    p.split = 1;
    while (p.split < 4 && tiles * jobs * kFewCluster * p.split * 2 <= static_cast<uint32_t>(sms)) p.split *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(tiles * p.split * kFewCluster, jobs);
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = few_smem<R>();
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kFewCluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization; // see the kernel's wait
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = allow_smem<lora_few_kernel<R>>(dev, few_smem<R>());
    if (e != cudaSuccess) return cuda_status(e);
    e = cudaLaunchKernelEx(&cfg, lora_few_kernel<R>, p);
    count_launch();
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? BS_OK : cuda_status(e);
}

} // namespace

bs_status launch_few(FewParams& p, uint32_t jobs, uint32_t R, int dev, int sms, cudaStream_t s) {
    switch (R) {
    case 16: return launch<16>(p, jobs, dev, sms, s);
    case 32: return launch<32>(p, jobs, dev, sms, s);
    case 64: return launch<64>(p, jobs, dev, sms, s);
    default: return launch<128>(p, jobs, dev, sms, s);
    }
}

} // namespace lora
} // namespace bs
