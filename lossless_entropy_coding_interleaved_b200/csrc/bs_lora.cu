// bs_lora.cu -- low-rank adapters of many requests at once beside a shared projection, and their
// gradients.
//
//   forward:  h[t] = s_a A_a x[t],  y[t] = base[t] + B_a h[t]           with a = idx[t]
//   backward: g[t] = s_a B_a^T dy[t],  dx[t] = A_a^T g[t],
//             dA_a = sum_t g[t] x[t]^T,  dB_a = sum_t dy[t] h[t]^T
//
// Every product has one side of the adapter's rank (8 to 128) and is bound by the bytes of its wide
// side (x, y, dy, dx). lora_plan_kernel groups the tokens by adapter once a batch; the kernels
// below take tiles of up to 128 tokens of one adapter, gathered through the plan:
//   shrink: [128 tokens x K] times [K x rank] -> h or g. The K range is split over a cluster of
//           CTAs, whose parts are added through distributed shared memory in a fixed order.
//   expand: [128 tokens x rank] times [rank x 64 or 128 columns], added to base on the way to y or dx.
//   outer:  [rank x tokens of an adapter] times [tokens x 128 or 256 columns] -> dA or dB; the tokens
//           are split over a cluster in the same way.
// (Batches of few tokens per adapter go forward through bs_lora_few.cu.) All three are tcgen05 matrix
// instructions on operands in shared memory: loading warps gather rows by cp.async into the 128-byte
// swizzle, one thread issues, other warps read tensor memory. An operand that lies the other way round
// (B for g, A for dx, both for dA and dB) is used as it lies, MN-major.
// x, dy and the weights are BF16, so their products are exact in FP32. h and g, FP32 sums, enter
// the next product as three BF16 numbers each (24 bits, see split3): three small matrix
// instructions in place of one lossy one, on a side where the tensor cores wait for memory.
// The tensor cores' accumulation rounds towards zero, so chains of matrix instructions are kept
// to 16 (shrink, outer) or 28 (expand: links at the size of the sum; 56 at rank 128) and their sums added in
// FP32 outside.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <iterator>

#include "bs_lora.cuh"
#include "bs_lora_tc.cuh"

namespace bs {
namespace {
using namespace lora;
namespace cg = cooperative_groups;

// ---------------------------------------------------------------- plan
// A stable counting sort by one CTA: W warps each take a contiguous run of tokens, count them per
// bucket, and after a scan over buckets and warps put them in their places, 32 at a time; lanes of
// the same bucket are ranked by their lane. No order depends on timing.
// 7 us for up to 333 tokens, 12 us for 8192, alone on the GPU: latency, and the steps of one CTA. The
// next kernel's start is beside its end.
__global__ void __launch_bounds__(1024) lora_plan_kernel(const int32_t* idx, uint32_t tokens, uint32_t n,
                                                         uint32_t* plan, uint32_t warps, uint32_t* err) {
    extern __shared__ uint32_t sm[];
    __shared__ uint32_t s_scan[3][32], s_carry[3];
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5, nb = n + 1; // buckets
    next_kernel_may_start();
    kernels_before_done();
    uint32_t* hist = sm;                    // [warps][nb]
    uint32_t* first = hist + warps * nb;    // [nb + 1] first place of each bucket
    uint32_t* t128 = first + nb + 1;        // [nb + 1] first tile of each bucket
    uint32_t* t8 = t128 + nb + 1;           // [nb + 1]
    for (uint32_t i = tid; i < warps * nb; i += blockDim.x) hist[i] = 0;
    if (tid < 3) s_carry[tid] = 0;
    __syncthreads();
    const uint32_t per = ((tokens + warps - 1) / warps + 31u) & ~31u;
    const uint32_t b0 = min(warp * per, tokens), b1 = min(b0 + per, tokens);
    bool bad = false;
    auto bucket = [&](uint32_t t) {
        const int32_t a = idx[t];
        bad |= a >= static_cast<int32_t>(n);
        return a < 0 || a >= static_cast<int32_t>(n) ? n : static_cast<uint32_t>(a);
    };
    constexpr int kAhead = 8; // rows of 32 tokens whose loads are under way together
    if (warp < warps)
        for (uint32_t t0 = b0; t0 < b1; t0 += 32 * kAhead) {
            uint32_t a[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) a[i] = t0 + 32 * i + lane < b1 ? bucket(t0 + 32 * i + lane) : nb;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (t0 + 32 * i >= b1) break;
                const uint32_t same = __match_any_sync(0xFFFFFFFFu, a[i]);
                if (a[i] < nb && (same & lanemask_lt()) == 0) hist[warp * nb + a[i]] += __popc(same);
                __syncwarp();
            }
        }
    if (bad && err) atomicOr(err, 4u);
    __syncthreads();
    for (uint32_t a0 = 0; a0 < nb; a0 += blockDim.x) { // scan over buckets, a chunk at a time
        const uint32_t a = a0 + tid;
        uint32_t v[3] = {0, 0, 0};
        if (a < nb) {
            for (uint32_t w = 0; w < warps; ++w) {
                const uint32_t c = hist[w * nb + a];
                hist[w * nb + a] = v[0];
                v[0] += c;
            }
            v[1] = (v[0] + kTile - 1) / kTile;
            v[2] = (v[0] + kFew - 1) / kFew;
        }
        uint32_t own[3] = {v[0], v[1], v[2]};
#pragma unroll
        for (int q = 0; q < 3; ++q) {
#pragma unroll
            for (uint32_t d = 1; d < 32; d <<= 1) {
                const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, v[q], d);
                if (lane >= d) v[q] += u;
            }
            if (lane == 31) s_scan[q][warp] = v[q];
        }
        __syncthreads();
        if (warp < 3) {
            uint32_t u = lane < blockDim.x / 32 ? s_scan[warp][lane] : 0;
#pragma unroll
            for (uint32_t d = 1; d < 32; d <<= 1) {
                const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, u, d);
                if (lane >= d) u += up;
            }
            s_scan[warp][lane] = u; // inclusive over warps
        }
        __syncthreads();
        if (a < nb) {
            uint32_t* dst[3] = {first, t128, t8};
#pragma unroll
            for (int q = 0; q < 3; ++q)
                dst[q][a] = s_carry[q] + (warp ? s_scan[q][warp - 1] : 0) + v[q] - own[q];
        }
        __syncthreads();
        if (tid < 3) s_carry[tid] += s_scan[tid][blockDim.x / 32 - 1];
        __syncthreads();
    }
    const PlanAt o = plan_at(tokens, n);
    // the adapters by falling number of tokens, in classes of its upper three bits (order inside a class
    // is as it comes: it only decides which CTAs start first)
    constexpr uint32_t kClasses = 8 * 21;
    __shared__ uint32_t s_class[kClasses];
    auto class_of = [&](uint32_t a) {
        const uint32_t c = (a + 1 < nb ? first[a + 1] : s_carry[0]) - first[a], lg = c ? 31u - __clz(c) : 0u;
        return kClasses - 1 - (c ? lg * 8 + ((lg >= 3 ? c >> (lg - 3) : c << (3 - lg)) & 7u) : 0u);
    };
    for (uint32_t i = tid; i < kClasses; i += blockDim.x) s_class[i] = 0;
    __syncthreads();
    for (uint32_t a = tid; a < n; a += blockDim.x) atomicAdd(&s_class[class_of(a)], 1u);
    __syncthreads();
    if (warp == 0) { // classes to first places
        uint32_t before = 0;
        for (uint32_t i = 0; i < kClasses; i += 32) {
            const uint32_t c = i + lane < kClasses ? s_class[i + lane] : 0;
            uint32_t u = c;
#pragma unroll
            for (uint32_t d = 1; d < 32; d <<= 1) {
                const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, u, d);
                if (lane >= d) u += up;
            }
            if (i + lane < kClasses) s_class[i + lane] = before + u - c;
            before += __shfl_sync(0xFFFFFFFFu, u, 31);
        }
    }
    __syncthreads();
    for (uint32_t a = tid; a < n; a += blockDim.x)
        reinterpret_cast<uint4*>(plan + o.order)[atomicAdd(&s_class[class_of(a)], 1u)] = make_uint4(a, first[a], a + 1 < nb ? first[a + 1] : s_carry[0], 0);
    if (tid == 0) {
        first[nb] = s_carry[0];
        t128[nb] = s_carry[1];
        t8[nb] = s_carry[2];
        const bool few = tokens <= kFewTokens;
        plan[0] = t128[n];
        plan[1] = t128[nb];
        plan[2] = few ? t8[n] : 0;
        plan[3] = few ? t8[nb] : 0;
        plan[4] = tokens;
        plan[5] = n;
    }
    __syncthreads();
    for (uint32_t a = tid; a <= nb; a += blockDim.x) plan[o.begin + a] = first[a];
    if (warp < warps)
        for (uint32_t t0 = b0; t0 < b1; t0 += 32 * kAhead) {
            uint32_t a[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) a[i] = t0 + 32 * i + lane < b1 ? bucket(t0 + 32 * i + lane) : nb;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (t0 + 32 * i >= b1) break;
                const uint32_t same = __match_any_sync(0xFFFFFFFFu, a[i]);
                uint32_t at = 0;
                if (a[i] < nb) at = first[a[i]] + hist[warp * nb + a[i]] + __popc(same & lanemask_lt());
                __syncwarp();
                if (a[i] < nb && (same & lanemask_lt()) == 0) hist[warp * nb + a[i]] += __popc(same);
                __syncwarp();
                if (a[i] < nb) plan[o.perm + at] = t0 + 32 * i + lane;
            }
        }
    auto tile_at = [&](const uint32_t* tb, uint32_t size, uint32_t i) {
        uint32_t lo = 0, hi = nb - 1; // the last bucket whose first tile is at or before i
        while (lo < hi) {
            const uint32_t mid = (lo + hi + 1) >> 1;
            if (tb[mid] <= i) lo = mid;
            else hi = mid - 1;
        }
        const uint32_t f = first[lo] + (i - tb[lo]) * size;
        return make_uint4(lo, f, min(size, first[lo + 1] - f), 0);
    };
    for (uint32_t i = tid; i < t128[nb]; i += blockDim.x) reinterpret_cast<uint4*>(plan + o.tiles)[i] = tile_at(t128, kTile, i);
    if (tokens > kFewTokens) return;
    __syncthreads(); // perm is complete
    for (uint32_t i = tid; i < t8[nb] * kFew; i += blockDim.x) { // a thread for each token of a tile
        const uint4 t = tile_at(t8, kFew, i / kFew);
        FewTile& e = reinterpret_cast<FewTile*>(plan + o.few)[i / kFew];
        const uint32_t j = i % kFew;
        e.token[j] = j < t.z ? plan[o.perm + t.y + j] : ~0u;
        if (j == 0) *reinterpret_cast<uint4*>(&e) = t;
    }
}

constexpr uint32_t kPlanSmem = 220 * 1024;

// ---------------------------------------------------------------- what the tiled kernels share
template <int R>
constexpr uint32_t atoms_of = R > 64 ? 2 : 1; // 64 ranks each

struct ShrinkJob {
    const uint16_t* src; // [tokens][stride]: x or dy
    const uint16_t* w;   // A [n][rank_max][width], or B [n][width][rank_max]
    uint16_t* out;       // three parts of [tokens][R], in the plan's order
    uint64_t stride;
    uint32_t width, pad;
};
struct ShrinkParams {
    Batch b;
    uint32_t split; // CTAs of a cluster
    uint32_t pad;
    ShrinkJob job[kMaxItems];
};

// 8192 tokens at rank 64: h from 3584 columns 23 us, g from 14336 53 us, that is 5.9 TB/s for the
// difference of the two: what is left is the start, the exchange and the end of a cluster. By mma.sync
// they took 39 and 80 us. 8 loading warps, or 256 bytes of a row at a time, change nothing.
// Threads that add up, that load; a warp more issues. 4 stages of 64 of the summed index: x (128 tokens
// x 64, K-major) and the weights (R x 64 K-major, or 64 x R MN-major).
constexpr uint32_t kShrinkLoad = 128, kShrinkStages = 4;
template <int R>
constexpr uint32_t shrink_out = R > 64 ? 256 : 128; // rank 128: two threads a token, 64 ranks each
template <int R>
constexpr uint32_t shrink_threads = shrink_out<R> + kShrinkLoad + 32;
template <int R, bool WT>
__host__ __device__ constexpr uint32_t shrink_stage() { return 16384 + (WT ? 8192 * atoms_of<R> : R * 128); }
template <int R, bool WT>
constexpr uint32_t shrink_smem() {
    return 1024 + std::max<uint32_t>(kShrinkStages * shrink_stage<R, WT>(), kTile * (R + 4) * 4);
}
template <int R>
constexpr uint32_t shrink_tmem = R <= 16 ? 32 : 2 * R; // columns
constexpr uint32_t kFlush = 4; // stages whose sums stay in tensor memory: chains of 16 matrix instructions

// WT: the weights' rank index is the contiguous one (B), else the summed index is (A).
template <int R, bool WT>
__global__ void __launch_bounds__(shrink_threads<R>, R <= 64 ? 2 : 1) lora_shrink_kernel(const __grid_constant__ ShrinkParams p) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_bar[2 * kShrinkStages + 4];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    constexpr uint32_t kTmem = shrink_tmem<R>, S = kShrinkStages, kShrinkOut = shrink_out<R>, kRanks = R > 64 ? 64 : R;
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    const uint32_t tile = blockIdx.x / p.split, part = blockIdx.x % p.split;
    const uint32_t s0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
    constexpr uint32_t kStage = shrink_stage<R, WT>();
    // barriers: full[S] (a stage has landed), empty[S] (its matrix instructions are done), d[2] (a
    // chain's sums are complete), free[2] (they have been added up)
    const uint32_t bar_full = smem_u32(s_bar), bar_empty = bar_full + 8 * S, bar_d = bar_empty + 8 * S, bar_free = bar_d + 16;
    if (tid == 0) {
        s_abort = 0;
        for (uint32_t i = 0; i < S; ++i) {
            bar_init(bar_full + 8 * i, kShrinkLoad);
            bar_init(bar_empty + 8 * i, 1);
        }
        for (uint32_t i = 0; i < 2; ++i) {
            bar_init(bar_d + 8 * i, 1);
            bar_init(bar_free + 8 * i, kShrinkOut);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    constexpr uint32_t kIssueWarp = (kShrinkOut + kShrinkLoad) / 32;
    if (warp == kIssueWarp) tmem_alloc(smem_u32(&s_tmem), kTmem);
    kernels_before_done(); // the above goes on beside the end of the kernel before
    const PlanAt o = plan_at(p.b.tokens, p.b.n);
    const uint32_t tiles = plan_head(p.b).x;
    const uint4 tl = reinterpret_cast<const uint4*>(p.b.plan + o.tiles)[tile];
    const ShrinkJob& job = p.job[blockIdx.y];
    const uint32_t a = tl.x, first = tl.y, count = tl.z, K = job.width;
    const uint32_t steps = (K + 63) / 64, per = (steps + p.split - 1) / p.split;
    const uint32_t k_begin = min(part * per, steps), n_steps = min(k_begin + per, steps) - k_begin;
    const uint16_t* row[8] = {}; // of the loading threads: piece t0 % 8 of the rows t0 / 8 + 16 i of x
    if (tile < tiles && warp >= kShrinkOut / 32 && warp < kIssueWarp) {
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) {
            const uint32_t r = ((tid - kShrinkOut) >> 3) + 16 * i;
            row[i] = r < count ? job.src + p.b.plan[o.perm + first + r] * job.stride : nullptr;
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = s_tmem;
    next_kernel_may_start();
    if (tile >= tiles) { // the whole cluster
        if (warp == kIssueWarp) tmem_free(tmem, kTmem);
        return;
    }
    const uint32_t rank = rank_of(p.b, a);
    volatile int* abort_flag = &s_abort;
    float* red = reinterpret_cast<float*>(smem_raw + (s0 - smem_u32(smem_raw))); // [128][R + 4], over the stages at the end

    if (warp >= kShrinkOut / 32 && warp < kIssueWarp) {
        const uint32_t t0 = tid - kShrinkOut, chunk = t0 & 7u; // rows past the tokens stand for nothing
        const uint16_t* w = job.w + uint64_t(a) * p.b.rank_max * K;
        for (uint32_t s = 0; s < n_steps; ++s) {
            if (s >= S && !bar_wait(bar_empty + 8 * (s % S), (s / S - 1) & 1u, abort_flag)) break;
            const uint32_t k = (k_begin + s) * 64, sb = s0 + s % S * kStage, sw = sb + 16384, kx = k + 8 * chunk;
            // rows t0 / 8 + 16 i of x and of A (their swizzle is the same for every i)
            const uint32_t in = kx < K ? 16u : 0u, dst = sb + sw128(t0 >> 3, chunk);
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) cp_async16_if(row[i] != nullptr, dst + 2048 * i, in ? row[i] + kx : job.src, in);
            if (!WT) {
#pragma unroll
                for (uint32_t i = 0; i < (R + 15) / 16; ++i) {
                    const uint32_t j = (t0 >> 3) + 16 * i;
                    const uint32_t on = j < rank ? in : 0u;
                    cp_async16(sw + sw128(t0 >> 3, chunk) + 2048 * i, on ? w + uint64_t(j) * K + kx : job.w, on);
                }
            } else {
                constexpr uint32_t kC = R / 8, kEvery = kShrinkLoad / kC; // pieces of a row; piece j of every kEvery-th row
                const uint32_t j = t0 % kC, take = 8 * j < rank ? min(rank - 8 * j, 8u) * 2u : 0u;
                const uint16_t* from = w + uint64_t(k + t0 / kC) * p.b.rank_max + 8 * j;
#pragma unroll
                for (uint32_t i = 0; i < 64 / kEvery; ++i) {
                    const uint32_t on = k + t0 / kC + kEvery * i < K ? take : 0u;
                    cp_async16(sw + (j >> 3) * 8192 + sw128(t0 / kC + kEvery * i, j & 7u), on ? from + uint64_t(kEvery * i) * p.b.rank_max : job.w, on);
                }
            }
            bar_arrive_copies(bar_full + 8 * (s % S));
        }
        cp_async_wait<0>();
    } else if (tid == kIssueWarp * 32) {
        const uint32_t idesc = idesc_of(R, false, WT);
        for (uint32_t s = 0; s < n_steps; ++s) {
            const uint32_t chain = s / kFlush, db = chain & 1u;
            if (s % kFlush == 0 && chain >= 2 && !bar_wait(bar_free + 8 * db, (chain / 2 - 1) & 1u, abort_flag)) break;
            if (!bar_wait(bar_full + 8 * (s % S), (s / S) & 1u, abort_flag)) break;
            fence_operands(); // the copies, before the tensor cores read them
            fence_after();
            const uint32_t x = s0 + s % S * kStage, w = x + 16384;
#pragma unroll
            for (uint32_t kk = 0; kk < 4; ++kk)
                mma_tc(tmem + db * R, k_major(x + kk * 32), WT ? mn_major(w + kk * 2048, 8192) : k_major(w + kk * 32), idesc, !(s % kFlush == 0 && kk == 0));
            commit_tc(bar_empty + 8 * (s % S));
            if (s % kFlush == kFlush - 1 || s + 1 == n_steps) commit_tc(bar_d + 8 * db);
        }
    } else if (warp < kShrinkOut / 32) {
        const uint32_t chains = (n_steps + kFlush - 1) / kFlush, j0 = (warp >> 2) * kRanks;
        float sum[kRanks] = {}; // of token 32 (warp % 4) + lane
        for (uint32_t c = 0; c < chains; ++c) {
            if (!bar_wait(bar_d + 8 * (c & 1u), (c / 2) & 1u, abort_flag)) break;
            fence_after();
#pragma unroll
            for (uint32_t j = 0; j < kRanks; j += 16) {
                uint32_t d[16];
                tmem_ld16(d, tmem + ((warp & 3u) * 32 << 16) + (c & 1u) * R + j0 + j);
#pragma unroll
                for (uint32_t i = 0; i < 16; ++i) sum[j + i] += __uint_as_float(d[i]);
            }
            fence_before();
            bar_arrive(bar_free + 8 * (c & 1u));
        }
        // every stage has been read: their place holds the sums from here on
#pragma unroll
        for (uint32_t j = 0; j < kRanks; j += 4)
            *reinterpret_cast<float4*>(red + ((warp & 3u) * 32 + lane) * (R + 4) + j0 + j) = make_float4(sum[j], sum[j + 1], sum[j + 2], sum[j + 3]);
    }
    fence_before();
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    const float scale = p.b.scales ? p.b.scales[a] : 1.f;
    const uint32_t rows = kTile / p.split; // rows that this CTA adds up and writes
    for (uint32_t i = tid; i < rows * (R / 8); i += shrink_threads<R>) {
        const uint32_t r = part * rows + i / (R / 8), c = 8 * (i % (R / 8));
        if (r >= count) continue;
        float v[8] = {};
        for (uint32_t q = 0; q < p.split; ++q) {
            const float* src = cluster.map_shared_rank(red, q) + r * (R + 4) + c;
            const float4 lo = *reinterpret_cast<const float4*>(src), hi = *reinterpret_cast<const float4*>(src + 4);
            v[0] += lo.x; v[1] += lo.y; v[2] += lo.z; v[3] += lo.w;
            v[4] += hi.x; v[5] += hi.y; v[6] += hi.z; v[7] += hi.w;
        }
        uint32_t w3[3][4] = {};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t q[3];
            split3(c + j < rank ? v[j] * scale : 0.f, q);
#pragma unroll
            for (int t = 0; t < 3; ++t) w3[t][j >> 1] |= q[t] << (16 * (j & 1));
        }
        uint16_t* dst = job.out + uint64_t(first + r) * R + c;
#pragma unroll
        for (int t = 0; t < 3; ++t)
            *reinterpret_cast<uint4*>(dst + uint64_t(t) * p.b.part_stride) = make_uint4(w3[t][0], w3[t][1], w3[t][2], w3[t][3]);
    }
    cluster.sync(); // the peers may still read this CTA's sums
    if (tid == 0 && s_abort && p.b.err) atomicOr(p.b.err, 2u);
    if (warp == kIssueWarp) {
        __syncwarp();
        tmem_free(tmem, kTmem);
    }
}

// ---------------------------------------------------------------- expand
struct ExpandSrc {
    const uint16_t* parts; // three parts of [tokens][R]
    const uint16_t* w;     // B [n][width][rank_max], or A [n][rank_max][width]
};
struct ExpandJob {
    const uint8_t* base; // nullptr: 0
    uint8_t* out;
    uint64_t base_stride, out_stride; // elements
    uint32_t width;
    uint32_t src, n_src; // sources whose products are added up
    uint32_t bf16;       // type of base and out
};
struct ExpandParams {
    Batch b;
    uint32_t n_jobs, pad;
    ExpandJob job[kMaxItems];
    ExpandSrc src[kMaxItems];
};
// threads that write and that load; a warp more issues
constexpr uint32_t kExpandOut = 256, kExpandLoad = 128, kExpandThreads = kExpandOut + kExpandLoad + 32;
// A block's rows of base, which become those of out. The 16-byte piece c of row r stands at piece
// (c & 8) | ((c ^ r) & 7): 8 lanes that take one piece of 8 rows, or 8 pieces of one, meet no bank twice.
constexpr uint32_t kRowBytes = 256;
__device__ __forceinline__ uint32_t row_piece(uint32_t r, uint32_t c) { return ((c & 8u) | ((c ^ r) & 7u)) << 4; }
template <bool BF16>
constexpr uint32_t expand_cols = kRowBytes / (BF16 ? 2 : 4); // columns of a block
// Buffers of base and of sums: as many as fit beside the operands, of which rank 128 has twice the bytes.
template <int R>
constexpr uint32_t expand_bufs = R > 64 ? 2 : 4;
// Sources that stand beside each other in an operand's 64 (or 128) ranks.
template <int R>
constexpr uint32_t group_of = R >= 64 ? 1 : 64 / R;
// Groups whose products are one chain of matrix instructions. The links of the lower parts come first in a group, so
// in the first one only those of the upper part (4, at rank 128 8) are rounded at the size of the sum; each group
// behind it has 12 (24). So a chain has 28 such links at most (rank 128: 56), and q, k and v are one. A dx of more
// sources is several chains, each a turn of the buffers, added up in tensor memory by the warps that write
// (MANY). q, k and v at rank 128, 8192 tokens, in BF16: 333 us in one chain, 366 us in two.
template <int R>
constexpr uint32_t chain_of = 3 * group_of<R>; // its sources
// Shared memory: h's parts (tokens x ranks, K-major), two buffers of weights, then those of base.
template <int R, bool BF16>
__host__ __device__ constexpr uint32_t expand_w() { return expand_cols<BF16> * 128 * atoms_of<R>; }
template <int R, bool BF16>
constexpr uint32_t expand_smem() {
    return 1024 + 3 * 16384 * atoms_of<R> + 2 * expand_w<R, BF16>() + expand_bufs<R> * kTile * kRowBytes;
}

// A place in the sequence of (job, tile, block) that the CTAs share out.
struct ExpandAt {
    uint32_t job, tile, block;
};

// One wave of CTAs shares the blocks (128 tokens of a tile x 256 bytes of their rows) of all jobs
// evenly, in the order job, tile, block, so that a CTA keeps a tile's h for its run of blocks. base's
// rows are copied to shared memory some blocks ahead, the matrix instructions' sums (128 tokens x the
// block's columns, in tensor memory) are added to them there, and they leave in lines of 128 bytes.
// 8192 tokens x 14336 columns, BF16, rank 64: 94 us (91 with two parts of h). Before: 209 us by mma.sync with the sums
// going to memory from its registers, 243 us from tensor memory number by number (20 to 33
// instructions for each 32 of them), 143 us with a bulk copy for each row's 256 or 128 bytes, which
// the copy engine takes 14 cycles each for.
// WT: the weights' column index is the contiguous one (A), else the rank index is (B).
// BF16: base and out are BF16. h enters as all of its three parts (24 bits) here too: with the upper two
// an output could be off by 2^-17 of the products' magnitudes, which is more than its own rounding
// where the products cancel.
// MANY: some dx has more sources than a chain holds.
template <int R, bool WT, bool BF16, bool MANY>
__global__ void __launch_bounds__(kExpandThreads, 1) lora_expand_kernel(const __grid_constant__ ExpandParams p) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_bar[4 + 3 * expand_bufs<R>];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    constexpr uint32_t kParts = 3, kCols = expand_cols<BF16>, es = BF16 ? 2 : 4, kPart = 16384 * atoms_of<R>;
    constexpr uint32_t kBufs = expand_bufs<R>, kGroup = group_of<R>, kChain = chain_of<R>, kTmem = kBufs * kCols;
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    const uint32_t s0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t sH = s0, sW = sH + kParts * kPart, sRow = sW + 2 * expand_w<R, BF16>();
    uint8_t* const rows = smem_raw + (sRow - smem_u32(smem_raw));
    // barriers: full[2] (weights, and parts before them, have landed), empty[2] (the matrix instructions
    // that read them are done); for each buffer d (a block's sums are complete), base (its base has
    // landed), free (its sums and its rows have been read out)
    const uint32_t bar_full = smem_u32(s_bar), bar_empty = bar_full + 16, bar_d = bar_full + 32, bar_base = bar_d + 8 * kBufs,
                   bar_free = bar_base + 8 * kBufs;
    if (tid == 0) {
        s_abort = 0;
        for (uint32_t i = 0; i < 2; ++i) {
            bar_init(bar_full + 8 * i, kExpandLoad);
            bar_init(bar_empty + 8 * i, 1);
        }
        for (uint32_t i = 0; i < kBufs; ++i) {
            bar_init(bar_d + 8 * i, 1);
            bar_init(bar_base + 8 * i, kExpandLoad);
            bar_init(bar_free + 8 * i, kExpandOut);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    constexpr uint32_t kIssueWarp = (kExpandOut + kExpandLoad) / 32;
    if (warp == kIssueWarp) tmem_alloc(smem_u32(&s_tmem), kTmem);
    kernels_before_done(); // the above goes on beside the end of the kernel before
    const PlanAt o = plan_at(p.b.tokens, p.b.n);
    const uint32_t tiles = plan_head(p.b).y;
    const uint4* tile_of = reinterpret_cast<const uint4*>(p.b.plan + o.tiles);
    auto blocks_of = [&](uint32_t job) { return (p.job[job].width + kCols - 1) / kCols; };
    uint64_t total = 0;
    for (uint32_t k = 0; k < p.n_jobs; ++k) total += uint64_t(tiles) * blocks_of(k);
    const uint64_t u0 = total * blockIdx.x / gridDim.x, u1 = total * (blockIdx.x + 1) / gridDim.x;
    const uint32_t n_units = static_cast<uint32_t>(u1 - u0);
    ExpandAt start{0, 0, 0};
    if (n_units) {
        uint64_t u = u0;
        while (u >= uint64_t(tiles) * blocks_of(start.job)) u -= uint64_t(tiles) * blocks_of(start.job++);
        start.tile = static_cast<uint32_t>(u / blocks_of(start.job));
        start.block = static_cast<uint32_t>(u % blocks_of(start.job));
    }
    // steps to the next unit; true where the tile (or job) is another one
    auto next = [&](ExpandAt& at) {
        if (++at.block < blocks_of(at.job)) return false;
        at.block = 0;
        if (++at.tile == tiles) {
            at.tile = 0;
            ++at.job;
        }
        return true;
    };
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = s_tmem;
    next_kernel_may_start(); // outer, of the same call, relies on every CTA of this one having waited above
    volatile int* abort_flag = &s_abort;
    // What a role needs of a tile: its adapter's rank (0: base as it is), and whether nothing at all is
    // to be done for it. Units left out take no turn of the buffers: every role counts the same ones.
    auto rank_at = [&](const uint4& tl) { return tl.x < p.b.n ? rank_of(p.b, tl.x) : 0u; };
    auto left_out = [&](const ExpandJob& j, uint32_t rank) { return rank == 0 && j.base == j.out && j.base_stride == j.out_stride; };

    if (warp >= kExpandOut / 32 && warp < kIssueWarp) {
        // base: piece t0 % 16 of the rows t0 / 16 + 8 i; weights and parts likewise by pieces of 16 bytes
        const uint32_t t0 = tid - kExpandOut, piece = t0 & 15u;
        constexpr uint32_t kC = R / 8;
        uint4 tl = make_uint4(0, 0, 0, 0);
        uint32_t rank = 0, turn = 0, step = 0;
        uint64_t row[16] = {};
        bool fresh = true, parts_in = false, ok = true; // another tile; the parts in place are those of all sources
        ExpandAt at = start;
        for (uint32_t u = 0; u < n_units && ok; ++u) {
            const ExpandJob& job = p.job[at.job];
            if (fresh) {
                tl = tile_of[at.tile];
                rank = rank_at(tl);
                parts_in = false;
#pragma unroll
                for (uint32_t i = 0; i < 16; ++i) {
                    const uint32_t r = (t0 >> 4) + 8 * i;
                    row[i] = r < tl.z ? p.b.plan[o.perm + tl.y + r] * job.base_stride : ~0ull;
                }
            }
            const uint32_t n0 = at.block * kCols, N = job.width, count = tl.z, sources = rank ? job.n_src : 0u;
            auto take_turn = [&](bool last) { // base goes with a unit's last chain
                const uint32_t buf = turn % kBufs, n = n0 + piece * (16 / es);
                if (turn >= kBufs && !bar_wait(bar_free + 8 * buf, (turn / kBufs - 1) & 1u, abort_flag)) return false;
                if (last && job.base && n < N) {
                    const uint32_t dst = sRow + (buf * kTile + (t0 >> 4)) * kRowBytes + row_piece(t0 >> 4, piece);
#pragma unroll
                    for (uint32_t i = 0; i < 16; ++i)
                        cp_async16_if(row[i] != ~0ull, dst + 8 * i * kRowBytes, job.base + (row[i] + n) * es, 16u);
                }
                bar_arrive_copies(bar_base + 8 * buf);
                ++turn;
                return true;
            };
            if (!left_out(job, rank) && !take_turn(!MANY || sources <= kChain)) break;
            for (uint32_t g0 = 0; g0 < sources; g0 += kGroup, ++step) { // a group of sources at a time
                if (MANY && g0 > 0 && g0 % kChain == 0 && !take_turn(g0 + kChain >= sources)) { ok = false; break; }
                const uint32_t wb = step & 1u, sb = sW + wb * expand_w<R, BF16>(), g1 = min(g0 + kGroup, sources);
                if (step >= 2 && !bar_wait(bar_empty + 8 * wb, (step / 2 - 1) & 1u, abort_flag)) { ok = false; break; }
                if (!parts_in) { // once what stood there has been read
                    if (step > 0 && !bar_wait(bar_empty + 8 * (wb ^ 1u), ((step - 1) / 2) & 1u, abort_flag)) { ok = false; break; }
                    for (uint32_t g = g0; g < g1; ++g)
#pragma unroll
                        for (uint32_t t = 0; t < kParts; ++t)
                            for (uint32_t c = t0; c < count * kC; c += kExpandLoad) {
                                const uint32_t r = c / kC, j = c % kC, at_j = (g - g0) * kC + j;
                                cp_async16(sH + t * kPart + (at_j >> 3) * 16384 + sw128(r, at_j & 7u),
                                           p.src[job.src + g].parts + uint64_t(t) * p.b.part_stride + uint64_t(tl.y + r) * R + 8 * j, 16u);
                            }
                    parts_in = sources <= kGroup;
                }
                for (uint32_t g = g0; g < g1; ++g) {
                    const ExpandSrc& src = p.src[job.src + g];
                    const uint16_t* w = src.w + uint64_t(tl.x) * p.b.rank_max * N;
                    if (!WT) { // piece j of the ranks, every kExpandLoad / kC-th column
                        const uint32_t j = t0 % kC, n = n0 + t0 / kC, at_j = (g - g0) * kC + j;
                        const uint32_t take = 8 * j < rank ? min(rank - 8 * j, 8u) * 2u : 0u, dst = sb + (at_j >> 3) * (kCols * 128);
                        const uint16_t* from = take ? w + uint64_t(n) * p.b.rank_max + 8 * j : src.w;
                        const uint64_t hop = take ? uint64_t(kExpandLoad / kC) * p.b.rank_max : 0;
#pragma unroll 4
                        for (uint32_t i = 0; i < kCols * kC / kExpandLoad; ++i, from += hop) {
                            const bool in = n + i * (kExpandLoad / kC) < N;
                            cp_async16(dst + sw128(t0 / kC + i * (kExpandLoad / kC), at_j & 7u), in ? from : src.w, in ? take : 0u);
                        }
                    } else {
                        constexpr uint32_t kRow = kCols / 8; // pieces of a rank's columns
#pragma unroll 4
                        for (uint32_t c = t0; c < R * kRow; c += kExpandLoad) {
                            const uint32_t j = c / kRow, q = c % kRow, n = n0 + 8 * q;
                            const bool on = j < rank && n < N;
                            cp_async16(sb + (q >> 3) * (kGroup * R * 128) + sw128((g - g0) * R + j, q & 7u), on ? w + uint64_t(j) * N + n : src.w, on ? 16u : 0u);
                        }
                    }
                }
                bar_arrive_copies(bar_full + 8 * wb);
            }
            fresh = next(at);
        }
        cp_async_wait<0>();
    } else if (tid == kIssueWarp * 32) {
        const uint32_t idesc = idesc_of(kCols, false, WT);
        uint32_t rank = 0, turn = 0, step = 0;
        bool fresh = true, ok = true;
        ExpandAt at = start;
        for (uint32_t u = 0; u < n_units && ok; ++u) {
            const ExpandJob& job = p.job[at.job];
            if (fresh) rank = rank_at(tile_of[at.tile]);
            if (!left_out(job, rank)) {
                const uint32_t kn = (rank + 15) / 16, sources = rank ? job.n_src : 0u;
                uint32_t db = turn % kBufs;
                if (turn >= kBufs && !bar_wait(bar_free + 8 * db, (turn / kBufs - 1) & 1u, abort_flag)) break;
                for (uint32_t g0 = 0; g0 < sources; g0 += kGroup, ++step) {
                    const bool begins = g0 == 0 || (MANY && g0 % kChain == 0);
                    if (MANY && begins && g0 > 0) { // the next chain
                        commit_tc(bar_d + 8 * db);
                        db = ++turn % kBufs;
                        if (turn >= kBufs && !bar_wait(bar_free + 8 * db, (turn / kBufs - 1) & 1u, abort_flag)) { ok = false; break; }
                    }
                    const uint32_t wb = step & 1u, w = sW + wb * expand_w<R, BF16>();
                    if (!bar_wait(bar_full + 8 * wb, (step / 2) & 1u, abort_flag)) { ok = false; break; }
                    fence_operands(); // the copies, before the tensor cores read them
                    fence_after();
                    // the descriptors' address field counts 16 bytes, and no sum carries out of it
                    const uint64_t wd = WT ? mn_major(w, kGroup * R * 128) : k_major(w), hd = k_major(sH);
                    const uint32_t in_group = min(sources - g0, kGroup);
                    uint32_t more = !begins;
#pragma unroll
                    for (int t = kParts - 1; t >= 0; --t) // small parts first
                        for (uint32_t g = 0; g < in_group; ++g)
#pragma unroll
                            for (uint32_t k1 = 0; k1 < R / 16; ++k1) {
                                if (k1 >= kn) break;
                                const uint32_t kk = g * (R / 16) + k1;
                                mma_tc(tmem + db * kCols, hd + ((t * kPart + (kk >> 2) * 16384 + (kk & 3u) * 32) >> 4),
                                       wd + ((WT ? kk * 2048 : (kk >> 2) * (kCols * 128) + (kk & 3u) * 32) >> 4), idesc, more);
                                more = 1;
                            }
                    commit_tc(bar_empty + 8 * wb);
                }
                if (!ok) break;
                if (rank) commit_tc(bar_d + 8 * db);
                else bar_arrive(bar_d + 8 * db);
                ++turn;
            }
            fresh = next(at);
        }
    } else if (warp < kExpandOut / 32) {
        // warps w and w + 4: tokens 32 (w % 4) .. of the tile, w the first half of a block's rows, w + 4
        // the second. A lane adds a token's sums to its row; then 8 lanes write 128 bytes of a row. (16
        // such warps, 8 for every other block, take as long.)
        const uint32_t r0 = (warp & 3u) * 32, half = warp >> 2;
        constexpr uint32_t kHalf = kCols / 2;
        uint4 tl = make_uint4(0, 0, 0, 0);
        uint32_t rank = 0, turn = 0;
        uint64_t row[8] = {}; // of the rows r0 + lane / 8 + 4 i
        bool fresh = true;
        ExpandAt at = start;
        auto chain_done = [&](uint32_t t) { // of turn t, and its base has landed
            const uint32_t buf = t % kBufs, parity = (t / kBufs) & 1u;
            if (!bar_wait(bar_base + 8 * buf, parity, abort_flag) || !bar_wait(bar_d + 8 * buf, parity, abort_flag)) return false;
            fence_after();
            return true;
        };
        auto join = [&](uint32_t t) { // the sum of turn t - 1 joins that of turn t
            const uint32_t mine = tmem + (r0 << 16) + half * kHalf, to = mine + t % kBufs * kCols, from = mine + (t - 1) % kBufs * kCols;
#pragma unroll 1
            for (uint32_t k = 0; k < kHalf; k += 16) {
                uint32_t d[16], e[16];
                tmem_ld16(d, to + k);
                tmem_ld16(e, from + k);
#pragma unroll
                for (uint32_t i = 0; i < 16; ++i) d[i] = __float_as_uint(__uint_as_float(d[i]) + __uint_as_float(e[i]));
                tmem_st16(to + k, d);
            }
            fence_before();
            bar_arrive(bar_free + 8 * ((t - 1) % kBufs));
            return true;
        };
        for (uint32_t u = 0; u < n_units; ++u) {
            const ExpandJob& job = p.job[at.job];
            if (fresh) {
                tl = tile_of[at.tile];
                rank = rank_at(tl);
#pragma unroll
                for (uint32_t i = 0; i < 8; ++i) {
                    const uint32_t r = r0 + (lane >> 3) + 4 * i;
                    row[i] = r < tl.z ? p.b.plan[o.perm + tl.y + r] * job.out_stride : ~0ull;
                }
            }
            if (!left_out(job, rank)) {
                if (MANY) { // the chains before the last: each joins the sum of those before it, in its own buffer
                    bool ok = true;
                    const uint32_t sources = rank ? job.n_src : 0u;
                    for (uint32_t g = kChain; g < sources; g += kChain, ++turn) {
                        ok = chain_done(turn) && (g == kChain || join(turn));
                        if (!ok) break;
                    }
                    if (!ok || (sources > kChain && !(chain_done(turn) && join(turn)))) break;
                }
                const uint32_t buf = turn % kBufs, n = at.block * kCols + half * kHalf + (lane & 7u) * (16 / es);
                uint8_t* mine = rows + (buf * kTile + r0) * kRowBytes; // the warp's rows
                if (!chain_done(turn)) break;
                if (rank || !job.base)
#pragma unroll
                    for (uint32_t c = 0; c < kHalf; c += 16) {
                        uint32_t d[16] = {};
                        if (rank) tmem_ld16(d, tmem + (r0 << 16) + buf * kCols + half * kHalf + c);
#pragma unroll
                        for (uint32_t q = 0; q < es; ++q) { // 16 bytes: 8 BF16 or 4 FP32
                            uint4* at16 = reinterpret_cast<uint4*>(mine + lane * kRowBytes + row_piece(lane, 8 * half + c * es / 16 + q));
                            uint4 v = job.base ? *at16 : make_uint4(0, 0, 0, 0);
                            uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (uint32_t i = 0; i < 4; ++i) {
                                if (BF16)
                                    w[i] = bf16x2_of(__uint_as_float(w[i] << 16) + __uint_as_float(d[8 * (q & 1u) + 2 * i]),
                                                     __uint_as_float(w[i] & 0xFFFF0000u) + __uint_as_float(d[8 * (q & 1u) + 2 * i + 1]));
                                else
                                    w[i] = __float_as_uint(__uint_as_float(w[i]) + __uint_as_float(d[4 * q + i]));
                            }
                            *at16 = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                fence_before();
                __syncwarp();
                if (n < job.width) {
                    uint8_t* to = job.out + uint64_t(n) * es;
#pragma unroll
                    for (uint32_t i = 0; i < 8; ++i) {
                        const uint32_t r = (lane >> 3) + 4 * i;
                        if (row[i] != ~0ull) *reinterpret_cast<uint4*>(to + row[i] * es) = *reinterpret_cast<const uint4*>(mine + r * kRowBytes + row_piece(r, 8 * half + (lane & 7u)));
                    }
                }
                __syncwarp();
                bar_arrive(bar_free + 8 * buf);
                ++turn;
            }
            fresh = next(at);
        }
    }
    fence_before();
    __syncthreads();
    if (tid == 0 && s_abort && p.b.err) atomicOr(p.b.err, 2u);
    if (warp == kIssueWarp) {
        __syncwarp();
        tmem_free(tmem, kTmem);
    }
}

// ---------------------------------------------------------------- outer
struct OuterJob {
    const uint16_t* src;   // [tokens][stride]: x or dy
    const uint16_t* parts; // three parts of [tokens][R]: g or h
    float* out;            // dA [n][rank_max][width], or dB [n][width][rank_max]
    uint64_t stride;
    uint32_t width, transposed;
};
struct OuterParams {
    Batch b;
    uint32_t split;
    uint32_t accumulate; // add to out, adapters without tokens left as they are
    // The kernel before this one is the expand product of the same call. It lets this one start when all
    // of its CTAs have seen the kernel before it (shrink, whose g is needed here) complete, so nothing
    // has to be waited for; its own completion is, at the end.
    uint32_t beside_expand, pad;
    OuterJob job[2 * kMaxItems];
};
// Threads that add up, that load; a warp more issues. A stage holds 64 tokens: their columns (MN-major)
// and the three parts of their ranks side by side (MN-major). Up to rank 32: 128 columns a CTA, a
// thread each; rank 64: 256 columns; rank 128: 128 columns, two threads each, 64 ranks a thread.
template <int R>
constexpr uint32_t outer_out = R > 32 ? 256 : 128;
template <int R>
constexpr uint32_t outer_cols = R == 64 ? 256 : 128;
template <int R>
constexpr uint32_t outer_load = R > 32 ? 256 : 128;
constexpr uint32_t kOuterTok = 64;
// Up to rank 32 a CTA is small and an adapter's tokens are often few, so that its start and end are what
// it costs: 4 CTAs of 2 stages an SM (3 at rank 32, with one sum in tensor memory). 1003 tokens of 36
// adapters, gate and up projections: 131 us at rank 16, 205 at rank 32; with 2 CTAs of 3 stages 182
// and 283. 8192 tokens of 2 adapters, gate: 56 and 68 us, against 59 and 78.
template <int R>
constexpr uint32_t outer_stages = R <= 32 ? 2 : 3;
constexpr uint32_t outer_ctas(uint32_t R) { return R <= 16 ? 4 : R <= 32 ? 3 : 1; }
template <int R>
constexpr uint32_t outer_threads = outer_out<R> + outer_load<R> + 32;
template <int R>
__host__ __device__ constexpr uint32_t outer_stage() { return outer_cols<R> * 128 + 8192 * ((3 * R + 63) / 64); }
template <int R>
constexpr uint32_t outer_smem() {
    // rank 64: 9 KB more than it uses, so that no CTA of rank 16 fits beside one (see kClustered)
    return std::max<uint32_t>(R == 64 ? 178 * 1024 : 0, 1024 + std::max<uint32_t>(outer_stages<R> * outer_stage<R>(), outer_cols<R> * (R + 4) * 4));
}
constexpr uint32_t kOuterFlush = 4; // stages whose sums stay in tensor memory: chains of 16 matrix instructions
// Sums in tensor memory: 128 columns x the 3 parts' ranks, beside each other (one matrix instruction
// reads the columns once for all parts; one for each part read them three times, and 8192 tokens at
// rank 64 took 135 us, bound by shared memory, against 94). At rank 16 two of them take turns;
// rank 64 has one for each 128 of its 256 columns, which are added up two stages apart, so that one
// half's matrix instructions go on meanwhile; ranks 32 and 128 have one.
template <int R>
constexpr uint32_t outer_accs = R == 16 || R == 64 ? 2 : 1;
template <int R>
constexpr uint32_t outer_tmem = R <= 32 ? 128 : 512; // columns, a power of two

// Two of these kernels may run at a time, on two streams. The CTAs of a cluster wait for each other, so if tensor
// memory ran out, a CTA could wait for that of another kernel's cluster, which waits for a peer that waits
// for this cluster's, for good. Shared memory has to keep CTAs apart that take more than the SM's 512
// columns together: whatever of them it holds at a time must find its columns.
struct Takes {
    uint32_t tmem, smem;
};
constexpr uint32_t kSmShared = 228 * 1024, kCtaShared = 1024; // of an SM, and what a CTA takes of it besides its own
constexpr Takes kClustered[] = {
    {shrink_tmem<16>, shrink_smem<16, false>()}, {shrink_tmem<16>, shrink_smem<16, true>()}, {shrink_tmem<32>, shrink_smem<32, false>()},
    {shrink_tmem<32>, shrink_smem<32, true>()}, {shrink_tmem<64>, shrink_smem<64, false>()}, {shrink_tmem<64>, shrink_smem<64, true>()},
    {shrink_tmem<128>, shrink_smem<128, false>()}, {shrink_tmem<128>, shrink_smem<128, true>()}, {outer_tmem<16>, outer_smem<16>()},
    {outer_tmem<32>, outer_smem<32>()}, {outer_tmem<64>, outer_smem<64>()}, {outer_tmem<128>, outer_smem<128>()}};
constexpr uint32_t most_columns(uint32_t from, uint32_t smem_left) { // of kinds `from` and later, that fit
    uint32_t most = 0;
    for (uint32_t k = from; k < std::size(kClustered); ++k) {
        const uint32_t need = kClustered[k].smem + kCtaShared;
        if (need > smem_left) continue;
        const uint32_t all = kClustered[k].tmem + most_columns(k, smem_left - need);
        most = all > most ? all : most;
    }
    return most;
}
static_assert(most_columns(0, kSmShared) <= 512, "CTAs that fit beside each other take more tensor memory than there is");

template <int R>
__global__ void __launch_bounds__(outer_threads<R>, outer_ctas(R)) lora_outer_kernel(const __grid_constant__ OuterParams p) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    constexpr uint32_t S = outer_stages<R>, kOuterCols = outer_cols<R>, kHalves = kOuterCols / 128, kAccs = outer_accs<R>, kWide = 3 * R;
    constexpr uint32_t kTmem = outer_tmem<R>;
    static_assert(kTmem >= kAccs * kWide);
    constexpr uint32_t kStage = outer_stage<R>(), kRanks = R > 64 ? 64 : R, kOuterOut = outer_out<R>, kOuterThreads = outer_threads<R>;
    constexpr uint32_t kOuterLoad = outer_load<R>;
    __shared__ __align__(8) uint64_t s_bar[2 * S + 4];
    __shared__ uint32_t s_tmem, s_rank;
    __shared__ int s_abort;
    const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
    const uint32_t s0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t bar_full = smem_u32(s_bar), bar_empty = bar_full + 8 * S, bar_d = bar_empty + 8 * S, bar_free = bar_d + 16; // as in shrink
    if (tid == 0) {
        s_abort = 0;
        for (uint32_t i = 0; i < S; ++i) {
            bar_init(bar_full + 8 * i, kOuterLoad);
            bar_init(bar_empty + 8 * i, 1);
        }
        for (uint32_t i = 0; i < 2; ++i) {
            bar_init(bar_d + 8 * i, 1);
            bar_init(bar_free + 8 * i, R > 64 ? 256 : 128);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    constexpr uint32_t kIssueWarp = (kOuterOut + kOuterLoad) / 32;
    if (warp == kIssueWarp) tmem_alloc(smem_u32(&s_tmem), kTmem);
    if (!p.beside_expand) kernels_before_done(); // the above goes on beside the end of the kernel before
    const PlanAt o = plan_at(p.b.tokens, p.b.n);
    bool planned;
    plan_head(p.b, &planned);
    const uint4 entry = planned ? reinterpret_cast<const uint4*>(p.b.plan + o.order)[blockIdx.y] : make_uint4(0, 0, 0, 0);
    // all jobs' blocks of columns for the adapter with the most tokens first, then the next: the last
    // CTAs to start are the shortest
    const uint32_t part = blockIdx.x % p.split, a = entry.x;
    uint32_t block = blockIdx.x / p.split, k = 0;
    while (block >= (p.job[k].width + kOuterCols - 1) / kOuterCols) block -= (p.job[k++].width + kOuterCols - 1) / kOuterCols;
    const OuterJob& job = p.job[k];
    const uint32_t c0 = block * kOuterCols;
    const uint32_t t_begin = entry.y, t_end = entry.z;
    const uint32_t rm = p.b.rank_max, cols = min(kOuterCols, job.width - c0);
    float* out = job.out + uint64_t(a) * rm * job.width;
    const uint32_t steps = (t_end - t_begin + kOuterTok - 1) / kOuterTok, per = (steps + p.split - 1) / p.split;
    const uint32_t s_begin = min(part * per, steps), n_steps = min(s_begin + per, steps) - s_begin;
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = s_tmem;
    if (!p.beside_expand) next_kernel_may_start();
    if (t_begin == t_end) { // no tokens: zero, or as it is
        if (warp == kIssueWarp) tmem_free(tmem, kTmem);
        if (!planned || p.accumulate) {
            if (p.beside_expand) kernels_before_done();
            return;
        }
        if (!job.transposed) {
            for (uint32_t i = part * kOuterThreads + tid; i < rm * (cols / 4); i += p.split * kOuterThreads)
                *reinterpret_cast<float4*>(out + uint64_t(i / (cols / 4)) * job.width + c0 + 4 * (i % (cols / 4))) = make_float4(0.f, 0.f, 0.f, 0.f);
        } else {
            float4* d = reinterpret_cast<float4*>(out + uint64_t(c0) * rm);
            for (uint32_t i = part * kOuterThreads + tid; i < cols * rm / 4; i += p.split * kOuterThreads) d[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (p.beside_expand) kernels_before_done();
        return;
    }
    volatile int* abort_flag = &s_abort;
    float* red = reinterpret_cast<float*>(smem_raw + (s0 - smem_u32(smem_raw))); // [256][R + 4], over the stages at the end

    if (warp >= kOuterOut / 32 && warp < kIssueWarp) {
        // columns: 16-byte pieces, of every 4th (8th) token; pieces past the width stand for nothing, tokens
        // past the last are 0 on both sides
        constexpr uint32_t kPieces = kOuterCols / 8, kEvery = kOuterLoad / kPieces, kRows = kOuterTok / kEvery;
        const uint32_t t0 = tid - kOuterOut, piece = t0 % kPieces, r0 = t0 / kPieces;
        const bool in = 8 * piece < cols;
        const uint16_t* from = job.src + c0 + 8 * piece;
        constexpr uint32_t kC = R / 8;
        uint32_t tok[kRows]; // of the step's tokens; the next step's are fetched a step ahead
        auto fetch = [&](uint32_t step) {
            const uint32_t first = t_begin + (s_begin + step) * kOuterTok;
#pragma unroll
            for (uint32_t i = 0; i < kRows; ++i) {
                const uint32_t at = first + r0 + kEvery * i;
                tok[i] = step < n_steps && at < t_end ? p.b.plan[o.perm + at] : ~0u;
            }
        };
        fetch(0);
        for (uint32_t s = 0; s < n_steps; ++s) {
            const uint32_t first = t_begin + (s_begin + s) * kOuterTok, left = t_end - first;
            uint32_t now[kRows];
#pragma unroll
            for (uint32_t i = 0; i < kRows; ++i) now[i] = tok[i];
            fetch(s + 1);
            if (s >= S && !bar_wait(bar_empty + 8 * (s % S), (s / S - 1) & 1u, abort_flag)) break;
            const uint32_t sb = s0 + s % S * kStage, sg = sb + kOuterCols * 128, dst = sb + (piece >> 3) * 8192;
            if (in) {
#pragma unroll
                for (uint32_t i = 0; i < kRows; ++i) {
                    const uint32_t on = now[i] != ~0u ? 16u : 0u;
                    cp_async16(dst + sw128(r0 + kEvery * i, piece & 7u), on ? from + now[i] * job.stride : job.src, on);
                }
            }
            // the parts: 16-byte piece t0 % kC of every kPart-th token
            constexpr uint32_t kPartRows = kOuterLoad / kC;
            const uint32_t j = t0 % kC, pr = t0 / kC;
            const uint16_t* part0 = job.parts + uint64_t(first + pr) * R + 8 * j;
#pragma unroll
            for (uint32_t t = 0; t < 3; ++t) {
                const uint32_t q = t * kC + j;
#pragma unroll
                for (uint32_t i = 0; i < kOuterTok / kPartRows; ++i) {
                    const uint32_t on = pr + kPartRows * i < left ? 16u : 0u;
                    cp_async16(sg + (q >> 3) * 8192 + sw128(pr + kPartRows * i, q & 7u), on ? part0 + kPartRows * i * R : job.parts, on);
                }
                part0 += p.b.part_stride;
            }
            bar_arrive_copies(bar_full + 8 * (s % S));
        }
        cp_async_wait<0>();
    } else if (tid == kIssueWarp * 32) {
        constexpr uint32_t kN = kWide > 192 ? 192 : kWide;
        const uint32_t idesc = idesc_of(kN, true, true);
        for (uint32_t s = 0; s < n_steps; ++s) {
            if (!bar_wait(bar_full + 8 * (s % S), (s / S) & 1u, abort_flag)) break;
            fence_operands(); // the copies, before the tensor cores read them
            fence_after();
            const uint32_t x = s0 + s % S * kStage, g = x + kOuterCols * 128;
            bool ok = true;
#pragma unroll
            for (uint32_t i = 0; i < kHalves; ++i) {
                // the half that begins a chain goes second: its sums may still be being added up
                const uint32_t h = kHalves == 2 && s % kOuterFlush == 0 ? 1 - i : i, at = s + 2 * h;
                const uint32_t chain = at / kOuterFlush, acc = kHalves == 2 ? h : chain % kAccs, use = kHalves == 2 ? chain : chain / kAccs;
                const bool begins = s == 0 || at % kOuterFlush == 0;
                if (begins && use >= 1 && !bar_wait(bar_free + 8 * acc, (use - 1) & 1u, abort_flag)) { ok = false; break; }
#pragma unroll
                for (uint32_t kk = 0; kk < kOuterTok / 16; ++kk)
#pragma unroll
                    for (uint32_t n = 0; n < kWide / kN; ++n)
                        mma_tc(tmem + acc * kWide + n * kN, mn_major(x + h * 16384 + kk * 2048, 8192), mn_major(g + n * (kN / 64) * 8192 + kk * 2048, 8192),
                               idesc, !(begins && kk == 0));
                if (at % kOuterFlush == kOuterFlush - 1 || s + 1 == n_steps) commit_tc(bar_d + 8 * acc);
            }
            if (!ok) break;
            commit_tc(bar_empty + 8 * (s % S));
        }
    } else if (warp < kOuterOut / 32) {
        // column 32 (warp % 4) + lane of a half; warps 4 to 7: the other half, or the other ranks
        if (tid == 0) s_rank = rank_of(p.b, a); // for the end, while nothing is there to be added up
        const uint32_t up = warp >> 2, h = kHalves == 2 ? up : 0, j0 = R > 64 ? up * kRanks : 0; // up: 0 with 128 threads
        const uint32_t chains = n_steps ? (n_steps - 1 + 2 * h) / kOuterFlush + 1 : 0;
        float sum[kRanks] = {};
        // Where x or dy has an infinity or NaN, the upper part's sum is what the product is: the lower parts may be 0
        // or of the other sign there, and give NaN for an infinity. From the first such sum of the warp on,
        // the upper part goes first, and what it has made infinite takes no more. (Columns past the width are
        // whatever shared memory held.)
        const bool within = h * 128 + (warp & 3u) * 32 + lane < cols;
        constexpr float kInf = __builtin_huge_valf();
        bool special = false;
        for (uint32_t c = 0; c < chains; ++c) {
            const uint32_t acc = kHalves == 2 ? h : c % kAccs, use = kHalves == 2 ? c : c / kAccs;
            if (!bar_wait(bar_d + 8 * acc, use & 1u, abort_flag)) break;
            fence_after();
            const uint32_t at = tmem + ((warp & 3u) * 32 << 16) + acc * kWide + j0;
            float odd[2] = {};
#pragma unroll
            for (uint32_t j = 0; j < kRanks; j += 16) {
                uint32_t d[16];
                if (!special) {
#pragma unroll
                    for (int part = 2; part >= 0; --part) { // small parts first
                        tmem_ld16(d, at + part * R + j);
#pragma unroll
                        for (uint32_t i = 0; i < 16; ++i) sum[j + i] += __uint_as_float(d[i]);
                    }
#pragma unroll
                    for (uint32_t i = 0; i < 16; ++i) odd[i & 1u] = fmaf(__uint_as_float(d[i]), 0.f, odd[i & 1u]); // NaN from the first such number on
                } else {
#pragma unroll
                    for (int part = 0; part < 3; ++part) {
                        tmem_ld16(d, at + part * R + j);
#pragma unroll
                        for (uint32_t i = 0; i < 16; ++i)
                            if (part == 0 || fabsf(sum[j + i]) < kInf) sum[j + i] += __uint_as_float(d[i]);
                    }
                }
            }
            if (__any_sync(0xFFFFFFFFu, within && odd[0] + odd[1] != 0.f)) { // what such a sum was before is finite
                special = true;
#pragma unroll
                for (uint32_t j = 0; j < kRanks; j += 16) {
                    uint32_t d[16];
                    tmem_ld16(d, at + j);
#pragma unroll
                    for (uint32_t i = 0; i < 16; ++i)
                        if (!(fabsf(__uint_as_float(d[i])) < kInf)) sum[j + i] = __uint_as_float(d[i]);
                }
            }
            fence_before();
            bar_arrive(bar_free + 8 * acc);
        }
        // once all of their matrix instructions are done, the stages' place holds the sums
        asm volatile("bar.sync 1, %0;" ::"n"(kOuterOut) : "memory");
#pragma unroll
        for (uint32_t j = 0; j < kRanks; j += 4)
            *reinterpret_cast<float4*>(red + (h * 128 + (warp & 3u) * 32 + lane) * (R + 4) + j0 + j) = make_float4(sum[j], sum[j + 1], sum[j + 2], sum[j + 3]);
    }
    fence_before();
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    // columns part * cols / split ..: the parts of all CTAs added up, 4 ranks of a column at a time
    const uint32_t each = kOuterCols / p.split, quads = rm / 4, rank = s_rank;
    for (uint32_t i = tid; i < each * quads; i += kOuterThreads) {
        // neighbouring threads have neighbouring columns (dA), or neighbouring ranks of a column (dB)
        const uint32_t c = part * each + (job.transposed ? i / quads : i % each), j = 4 * (job.transposed ? i % quads : i / each);
        if (c >= cols) continue;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (uint32_t q = 0; q < p.split; ++q) {
            const float4 u = *reinterpret_cast<const float4*>(cluster.map_shared_rank(red, q) + c * (R + 4) + j);
            v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
        }
        // past the adapter's rank 0, whatever stood in x and dy (the parts are 0 there, but 0 times infinity is not)
        v = make_float4(j < rank ? v.x : 0.f, j + 1 < rank ? v.y : 0.f, j + 2 < rank ? v.z : 0.f, j + 3 < rank ? v.w : 0.f);
        if (job.transposed) {
            float4* d = reinterpret_cast<float4*>(out + uint64_t(c0 + c) * rm + j);
            if (p.accumulate) { const float4 u = *d; v = make_float4(u.x + v.x, u.y + v.y, u.z + v.z, u.w + v.w); }
            *d = v;
        } else {
            float* d = out + uint64_t(j) * job.width + c0 + c;
            const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (uint32_t q = 0; q < 4; ++q, d += job.width) *d = p.accumulate ? *d + w[q] : w[q];
        }
    }
    cluster.sync(); // the peers may still read this CTA's sums
    if (tid == 0 && s_abort && p.b.err) atomicOr(p.b.err, 2u);
    if (warp == kIssueWarp) {
        __syncwarp();
        tmem_free(tmem, kTmem);
    }
    if (p.beside_expand) kernels_before_done();
}

// ---------------------------------------------------------------- host
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bs_status check_batch(const bs_lora_batch* b) {
    if (!b || b->tokens > kMaxTokens || b->n_adapters < 1 || b->n_adapters > kMaxAdapters || b->reserved) return BS_E_ARG;
    if (b->rank_max < 8 || b->rank_max > kMaxRank || b->rank_max % 8) return BS_E_ARG;
    if (!b->d_plan || !aligned(b->d_plan, 16) || b->plan_bytes < bs_lora_plan_bytes(b->tokens, b->n_adapters) || !aligned(b->d_ranks, 4) || !aligned(b->d_scales, 4) || !aligned(b->d_err, 4)) return BS_E_ARG;
    return BS_OK;
}
bs_status check_item(const bs_lora_item& t) {
    if (t.rows < 8 || t.cols < 8 || t.rows % 8 || t.cols % 8 || t.rows > (1u << 24) || t.cols > (1u << 24)) return BS_E_ARG;
    if (!t.d_a || !t.d_b || !aligned(t.d_a, 16) || !aligned(t.d_b, 16)) return BS_E_ARG;
    if (t.type > BS_TYPE_BF16 || t.reserved) return BS_E_ARG;
    return BS_OK;
}
bool row_ok(const void* p, uint64_t stride, uint32_t width) { // BF16 rows read 16 bytes at a time
    return p && aligned(p, 16) && stride >= width && stride % 8 == 0 && stride <= (1ull << 32);
}
bool out_ok(const void* p, uint64_t stride, uint32_t width, uint32_t type) {
    return p && aligned(p, 16) && stride >= width && stride % (type == BS_TYPE_BF16 ? 8 : 4) == 0 && stride <= (1ull << 32);
}
Batch batch_of(const bs_lora_batch& b) {
    Batch o;
    o.tokens = b.tokens;
    o.n = b.n_adapters;
    o.rank_max = b.rank_max;
    o.part_stride = b.tokens * padded_rank(b.rank_max); // below 2^27
    o.plan = static_cast<const uint32_t*>(b.d_plan);
    o.ranks = b.d_ranks;
    o.scales = b.d_scales;
    o.err = b.d_err;
    return o;
}
struct Gpu {
    int dev = 0, sms = 148;
    cudaStream_t s = nullptr;
};
template <auto FN, uint32_t THREADS, typename Params>
bs_status launch(dim3 grid, uint32_t smem, uint32_t cluster, const Gpu& gpu, const Params& p) {
    cudaError_t e = allow_smem<FN>(gpu.dev, smem);
    if (e != cudaSuccess) return cuda_status(e);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = gpu.s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization; // see kernels_before_done
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, FN, p);
    count_launch();
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? BS_OK : cuda_status(e);
}
// Whether a batch goes through the decoding kernel. It reads an adapter's weights for every 8 of its
// tokens (0.4 to 0.8 us a tile of 8 at 3584 x 14336, ranks 16 and 64), the tiled kernels for every
// 128, but they pass through tiles that are mostly empty (2 to 2.4 us an adapter). 64 tokens of one
// adapter: 27 and 33 us here, 22 and 25 us tiled (18 and 22 us at 3584 x 4096, rank 64); 256 tokens of 8:
// 31 and 39 us, tiled 35 and 41; 512 of 32: 55 and 82, tiled 78 and 92; 1024 of 256: 121 and 223,
// tiled 514 and 618. n is the pool's size, all that the host knows: where few adapters of a large pool are in use
// the rule is off (1000 tokens of one adapter: 32 us tiled, in a pool of up to 8, and 48 us here, in one of 64).
bool few_tokens(uint32_t tokens, uint32_t n) { return tokens <= kFewTokens && tokens <= 16 * n + 48; }

// CTAs of a cluster that share a sum: the most of 1, 2, 4, 8 that leave each CTA 4 steps and fit into
// `slots` CTAs at a time.
uint32_t split_for(uint64_t ctas, uint32_t steps, uint64_t slots) {
    uint32_t c = 1;
    while (c < 8 && ctas * c * 2 <= slots && steps >= 8 * c) c *= 2;
    return c;
}

template <bool WT>
bs_status launch_shrink(ShrinkParams& p, uint32_t jobs, uint32_t R, const Gpu& gpu) {
    uint32_t steps = ~0u;
    for (uint32_t k = 0; k < jobs; ++k) steps = std::min(steps, (p.job[k].width + 63) / 64);
    const uint32_t cap = tile_cap(p.b.tokens, p.b.n, kTile);
    p.split = split_for(uint64_t(std::min(cap, (p.b.tokens + kTile - 1) / kTile)) * jobs, steps, uint64_t(gpu.sms) * (R <= 64 ? 2 : 1));
    const dim3 grid(cap * p.split, jobs);
    switch (R) {
    case 16: return launch<lora_shrink_kernel<16, WT>, shrink_threads<16>>(grid, shrink_smem<16, WT>(), p.split, gpu, p);
    case 32: return launch<lora_shrink_kernel<32, WT>, shrink_threads<32>>(grid, shrink_smem<32, WT>(), p.split, gpu, p);
    case 64: return launch<lora_shrink_kernel<64, WT>, shrink_threads<64>>(grid, shrink_smem<64, WT>(), p.split, gpu, p);
    default: return launch<lora_shrink_kernel<128, WT>, shrink_threads<128>>(grid, shrink_smem<128, WT>(), p.split, gpu, p);
    }
}
template <int R, bool WT, bool BF16>
bs_status launch_expand_rank(const ExpandParams& p, dim3 grid, const Gpu& gpu) {
    constexpr uint32_t smem = expand_smem<R, BF16>();
    if constexpr (WT) // forward has one source
        for (uint32_t k = 0; k < p.n_jobs; ++k)
            if (p.job[k].n_src > chain_of<R>) return launch<lora_expand_kernel<R, WT, BF16, true>, kExpandThreads>(grid, smem, 1, gpu, p);
    return launch<lora_expand_kernel<R, WT, BF16, false>, kExpandThreads>(grid, smem, 1, gpu, p);
}
template <bool WT, bool BF16>
bs_status launch_expand_of(ExpandParams& p, uint32_t jobs, uint32_t R, const Gpu& gpu) {
    p.n_jobs = jobs;
    uint64_t units = 0; // at most: the plan, on the device, knows the tiles
    for (uint32_t k = 0; k < jobs; ++k)
        units += uint64_t(tile_cap(p.b.tokens, p.b.n, kTile)) * ((p.job[k].width + expand_cols<BF16> - 1) / expand_cols<BF16>);
    const dim3 grid(static_cast<uint32_t>(std::min<uint64_t>(units, gpu.sms)));
    switch (R) {
    case 16: return launch_expand_rank<16, WT, BF16>(p, grid, gpu);
    case 32: return launch_expand_rank<32, WT, BF16>(p, grid, gpu);
    case 64: return launch_expand_rank<64, WT, BF16>(p, grid, gpu);
    default: return launch_expand_rank<128, WT, BF16>(p, grid, gpu);
    }
}
// The jobs of a call may be of both types: those of each go together.
template <bool WT>
bs_status launch_expand(const ExpandParams& all, uint32_t jobs, uint32_t R, const Gpu& gpu) {
    ExpandParams p = all;
    for (uint32_t type : {BS_TYPE_F32, BS_TYPE_BF16}) {
        uint32_t n = 0;
        for (uint32_t k = 0; k < jobs; ++k)
            if (all.job[k].bf16 == type) p.job[n++] = all.job[k];
        if (n == 0) continue;
        const bs_status st = type == BS_TYPE_BF16 ? launch_expand_of<WT, true>(p, n, R, gpu) : launch_expand_of<WT, false>(p, n, R, gpu);
        if (st != BS_OK) return st;
    }
    return BS_OK;
}
// An adapter's tokens are taken to be tokens / n, the pool's share: the plan alone knows better (4096 tokens of one
// adapter, gradients: 83 us in a pool of 1, 120 us in one of 64).
bs_status launch_outer(OuterParams& p, uint32_t jobs, uint32_t R, const Gpu& gpu) {
    const uint32_t cols = R == 64 ? outer_cols<64> : outer_cols<128>;
    uint32_t ctas = 0;
    for (uint32_t k = 0; k < jobs; ++k) ctas += (p.job[k].width + cols - 1) / cols;
    p.split = split_for(uint64_t(ctas) * p.b.n, p.b.tokens / p.b.n / kOuterTok, uint64_t(std::max(2u, outer_ctas(R))) * gpu.sms);
    const dim3 grid(ctas * p.split, p.b.n);
    switch (R) {
    case 16: return launch<lora_outer_kernel<16>, outer_threads<16>>(grid, outer_smem<16>(), p.split, gpu, p);
    case 32: return launch<lora_outer_kernel<32>, outer_threads<32>>(grid, outer_smem<32>(), p.split, gpu, p);
    case 64: return launch<lora_outer_kernel<64>, outer_threads<64>>(grid, outer_smem<64>(), p.split, gpu, p);
    default: return launch<lora_outer_kernel<128>, outer_threads<128>>(grid, outer_smem<128>(), p.split, gpu, p);
    }
}

} // namespace
} // namespace bs

using namespace bs;
using namespace bs::lora;

extern "C" size_t bs_lora_plan_bytes(uint32_t tokens, uint32_t n_adapters) {
    if (tokens > kMaxTokens || n_adapters < 1 || n_adapters > kMaxAdapters) return 0;
    return 4 * plan_at(tokens, n_adapters).words;
}

extern "C" size_t bs_lora_state_bytes(uint32_t tokens, uint32_t rank_max) {
    if (tokens > kMaxTokens || rank_max < 8 || rank_max > kMaxRank || rank_max % 8) return 0;
    return std::max<size_t>(16, size_t(6) * tokens * padded_rank(rank_max));
}

extern "C" bs_status bs_lora_plan(const int32_t* d_idx, uint32_t tokens, uint32_t n_adapters, void* d_plan, size_t plan_bytes,
                                  uint32_t* d_err, void* stream) {
    const size_t need = bs_lora_plan_bytes(tokens, n_adapters);
    if (need == 0) return BS_E_ARG;
    if ((tokens && !d_idx) || !aligned(d_idx, 4) || !d_plan || !aligned(d_plan, 16) || !aligned(d_err, 4)) return BS_E_ARG;
    if (plan_bytes < need) return BS_E_SIZE;
    int dev = 0, sms = 0;
    const bs_status st = current_device(&dev, &sms);
    if (st != BS_OK) return st;
    // as many counting warps as their tables fit into shared memory, and as have tokens
    const uint32_t nb = n_adapters + 1;
    const uint32_t fit = kPlanSmem / 4 / nb - 4;
    const uint32_t warps = std::max(1u, std::min({32u, fit, (tokens + 31) / 32})); // at most threads / 32 below
    const uint32_t smem = 4 * (warps * nb + 3 * (nb + 1));
    cudaError_t e = allow_smem<lora_plan_kernel>(dev, kPlanSmem);
    if (e != cudaSuccess) return cuda_status(e);
    // a thread for each token or bucket; a small block passes its barriers sooner (the scan needs 3 warps)
    const uint32_t threads = std::min(1024u, std::max(128u, (std::max(tokens, nb) + 31) & ~31u));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization; // see kernels_before_done
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, lora_plan_kernel, d_idx, tokens, n_adapters, static_cast<uint32_t*>(d_plan), warps, d_err);
    count_launch();
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? BS_OK : cuda_status(e);
}

extern "C" bs_status bs_lora_forward_check(int32_t n, const bs_lora_item* items, const bs_lora_batch* batch) {
    bs_status st = check_batch(batch);
    if (st != BS_OK) return st;
    if (n < 0 || (n > 0 && !items)) return BS_E_ARG;
    for (int32_t k = 0; k < n; ++k) {
        const bs_lora_item& t = items[k];
        if ((st = check_item(t)) != BS_OK) return st;
        if (batch->tokens == 0) continue;
        if (!row_ok(t.d_x, t.x_stride, t.cols) || !t.d_h || !aligned(t.d_h, 16)) return BS_E_ARG;
        if (t.d_y && !out_ok(t.d_y, t.y_stride, t.rows, t.type)) return BS_E_ARG;
        for (int32_t q = 0; q < k; ++q) // two items that write the same memory
            if (items[q].d_h == t.d_h || (t.d_y && items[q].d_y == t.d_y)) return BS_E_ARG;
        if (t.d_base && (!t.d_y || !out_ok(t.d_base, t.base_stride, t.rows, t.type))) return BS_E_ARG;
        if (t.d_base && t.d_base == t.d_y && t.base_stride != t.y_stride && batch->tokens > 1) return BS_E_ARG;
        for (int32_t q = 0; t.d_y && q < n; ++q) // a y is not also read
            if (items[q].d_x == t.d_y || (q != k && items[q].d_base == t.d_y)) return BS_E_ARG;
    }
    return BS_OK;
}

extern "C" bs_status bs_lora_forward(int32_t n, const bs_lora_item* items, const bs_lora_batch* batch, void* stream) {
    bs_status st = bs_lora_forward_check(n, items, batch);
    if (st != BS_OK) return st;
    Gpu gpu;
    gpu.s = static_cast<cudaStream_t>(stream);
    if ((st = current_device(&gpu.dev, &gpu.sms)) != BS_OK) return st;
    if (n == 0 || batch->tokens == 0) return BS_OK;
    const uint32_t R = padded_rank(batch->rank_max);
    if (few_tokens(batch->tokens, batch->n_adapters)) {
        FewParams fp;
        fp.b = batch_of(*batch);
        for (int32_t k0 = 0; k0 < n; k0 += kMaxItems) {
            const uint32_t m = static_cast<uint32_t>(std::min(n - k0, kMaxItems));
            for (uint32_t k = 0; k < m; ++k) {
                const bs_lora_item& t = items[k0 + k];
                fp.job[k] = FewJob{static_cast<const uint16_t*>(t.d_x), static_cast<const uint16_t*>(t.d_a), static_cast<const uint16_t*>(t.d_b),
                                   static_cast<const uint8_t*>(t.d_base), static_cast<uint8_t*>(t.d_y), static_cast<uint16_t*>(t.d_h),
                                   t.x_stride, t.base_stride, t.y_stride, t.rows, t.cols, t.type, 0};
            }
            if ((st = launch_few(fp, m, R, gpu.dev, gpu.sms, gpu.s)) != BS_OK) return st;
        }
        return BS_OK;
    }
    ShrinkParams sp;
    ExpandParams ep;
    sp.b = ep.b = batch_of(*batch);
    for (int32_t k0 = 0; k0 < n; k0 += kMaxItems) {
        const uint32_t m = static_cast<uint32_t>(std::min(n - k0, kMaxItems));
        uint32_t outs = 0;
        for (uint32_t k = 0; k < m; ++k) {
            const bs_lora_item& t = items[k0 + k];
            sp.job[k] = ShrinkJob{static_cast<const uint16_t*>(t.d_x), static_cast<const uint16_t*>(t.d_a),
                                  static_cast<uint16_t*>(t.d_h), t.x_stride, t.cols, 0};
            if (!t.d_y) continue;
            ep.src[outs] = ExpandSrc{static_cast<const uint16_t*>(t.d_h), static_cast<const uint16_t*>(t.d_b)};
            ep.job[outs] = ExpandJob{static_cast<const uint8_t*>(t.d_base), static_cast<uint8_t*>(t.d_y), t.base_stride, t.y_stride,
                                     t.rows, outs, 1, t.type};
            ++outs;
        }
        if ((st = launch_shrink<false>(sp, m, R, gpu)) != BS_OK) return st;
        if (outs && (st = launch_expand<false>(ep, outs, R, gpu)) != BS_OK) return st;
    }
    return BS_OK;
}

extern "C" bs_status bs_lora_backward(int32_t n, const bs_lora_item* items, const bs_lora_batch* batch, uint32_t flags, void* stream) {
    bs_status st = check_batch(batch);
    if (st != BS_OK) return st;
    if (n < 0 || (n > 0 && !items) || (flags & ~BS_LORA_ACCUMULATE)) return BS_E_ARG;
    for (int32_t k = 0; k < n; ++k) {
        const bs_lora_item& t = items[k];
        if ((st = check_item(t)) != BS_OK) return st;
        if (!t.d_da || !t.d_db || !aligned(t.d_da, 16) || !aligned(t.d_db, 16)) return BS_E_ARG;
        if (batch->tokens == 0) continue;
        if (!row_ok(t.d_x, t.x_stride, t.cols) || !row_ok(t.d_dy, t.dy_stride, t.rows)) return BS_E_ARG;
        if (!t.d_h || !t.d_g || !aligned(t.d_h, 16) || !aligned(t.d_g, 16)) return BS_E_ARG;
        if (t.d_dx && !out_ok(t.d_dx, t.dx_stride, t.cols, t.type)) return BS_E_ARG;
        if (t.d_dx_base && (!t.d_dx || !out_ok(t.d_dx_base, t.dx_base_stride, t.cols, t.type))) return BS_E_ARG;
        for (int32_t q = 0; q < k; ++q) // two items that write the same memory
            if (items[q].d_g == t.d_g || items[q].d_da == t.d_da || items[q].d_db == t.d_db) return BS_E_ARG;
        if (t.d_dx_base && t.d_dx_base == t.d_dx && t.dx_base_stride != t.dx_stride && batch->tokens > 1) return BS_E_ARG;
        for (int32_t q = 0; q < n; ++q) // what is written is not also read
            if (items[q].d_h == t.d_g || (t.d_dx && (items[q].d_x == t.d_dx || items[q].d_dy == t.d_dx ||
                                                     (items[q].d_dx_base == t.d_dx && items[q].d_dx != t.d_dx))))
                return BS_E_ARG;
        // items that share dx share its base, strides and type too
        for (int32_t q = 0; q < k; ++q)
            if (t.d_dx && items[q].d_dx == t.d_dx &&
                (items[q].d_dx_base != t.d_dx_base || items[q].dx_stride != t.dx_stride || items[q].dx_base_stride != t.dx_base_stride ||
                 items[q].type != t.type || items[q].cols != t.cols || q / kMaxItems != k / kMaxItems))
                return BS_E_ARG;
    }
    Gpu gpu;
    gpu.s = static_cast<cudaStream_t>(stream);
    if ((st = current_device(&gpu.dev, &gpu.sms)) != BS_OK) return st;
    if (n == 0) return BS_OK;
    const uint32_t R = padded_rank(batch->rank_max);
    ShrinkParams sp;
    ExpandParams ep;
    OuterParams op;
    sp.b = ep.b = op.b = batch_of(*batch);
    op.accumulate = flags & BS_LORA_ACCUMULATE;
    for (int32_t k0 = 0; k0 < n; k0 += kMaxItems) {
        const uint32_t m = static_cast<uint32_t>(std::min(n - k0, kMaxItems));
        uint32_t outs = 0, srcs = 0;
        bool done[kMaxItems] = {};
        for (uint32_t k = 0; k < m; ++k) {
            const bs_lora_item& t = items[k0 + k];
            sp.job[k] = ShrinkJob{static_cast<const uint16_t*>(t.d_dy), static_cast<const uint16_t*>(t.d_b),
                                  static_cast<uint16_t*>(t.d_g), t.dy_stride, t.rows, 0};
            op.job[2 * k] = OuterJob{static_cast<const uint16_t*>(t.d_x), static_cast<const uint16_t*>(t.d_g), t.d_da, t.x_stride, t.cols, 0};
            op.job[2 * k + 1] = OuterJob{static_cast<const uint16_t*>(t.d_dy), static_cast<const uint16_t*>(t.d_h), t.d_db, t.dy_stride, t.rows, 1};
            if (!t.d_dx || done[k]) continue;
            ExpandJob& e = ep.job[outs++];
            e = ExpandJob{static_cast<const uint8_t*>(t.d_dx_base), static_cast<uint8_t*>(t.d_dx), t.dx_base_stride, t.dx_stride,
                          t.cols, srcs, 0, t.type};
            for (uint32_t q = k; q < m; ++q) // every item with this dx is a source of it
                if (items[k0 + q].d_dx == t.d_dx) {
                    done[q] = true;
                    ep.src[srcs++] = ExpandSrc{static_cast<const uint16_t*>(items[k0 + q].d_g), static_cast<const uint16_t*>(items[k0 + q].d_a)};
                    ++e.n_src;
                }
        }
        if (batch->tokens) {
            if ((st = launch_shrink<true>(sp, m, R, gpu)) != BS_OK) return st;
            if (outs && (st = launch_expand<true>(ep, outs, R, gpu)) != BS_OK) return st;
        }
        op.beside_expand = batch->tokens && outs;
        if ((st = launch_outer(op, 2 * m, R, gpu)) != BS_OK) return st;
    }
    return BS_OK;
}
