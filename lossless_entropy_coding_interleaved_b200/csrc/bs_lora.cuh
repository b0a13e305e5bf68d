// bs_lora.cuh -- definitions shared by the kernels of the low-rank adapters (bs_lora*.cu).
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "bs_device.cuh"
#include "bs_host.h"
#include "bs_internal.h"

namespace bs {
namespace lora {

constexpr uint32_t kMaxTokens = 1u << 20, kMaxAdapters = 8192, kMaxRank = 128;
constexpr uint32_t kTile = 128;   // tokens of one adapter that a CTA of the tiled kernels takes
constexpr uint32_t kFew = 8;      // the same for the decoding kernel
constexpr uint32_t kFewTokens = 1024; // the largest batch whose plan lists tiles of kFew tokens
constexpr int kMaxItems = 16;     // projections of one launch

// The plan of a batch, in 32-bit words: the tokens sorted by adapter, those without one last
// (bucket n_adapters), each adapter's tokens in their own order.
//   [0] tiles of kTile tokens that have an adapter, [1] all tiles of kTile (those without an
//   adapter follow), [2] and [3] the same for kFew (0 above kFewTokens), [4] tokens, [5] adapters
//   begin[n_adapters + 2]: the first place of each bucket, then the end
//   order: (adapter, first place, end, 0) of each adapter, those with the most tokens first (about)
//   perm[tokens]: the token at each place
//   tiles: (bucket, first place, tokens, 0) each
//   tiles of kFew: the same, and the tokens themselves
struct FewTile {
    uint32_t bucket, first, count, pad, token[kFew]; // token: ~0 past the count
};
struct PlanAt {
    uint64_t begin, order, perm, tiles, few, words;
};
__host__ __device__ inline uint32_t tile_cap(uint32_t tokens, uint32_t n, uint32_t size) {
    const uint32_t most = tokens / size + n + 1; // every bucket ends in a part-filled tile
    return most < tokens ? most : tokens;
}
__host__ __device__ inline PlanAt plan_at(uint32_t tokens, uint32_t n) {
    PlanAt o;
    auto up4 = [](uint64_t v) { return (v + 3) & ~uint64_t(3); };
    o.begin = 16;
    o.order = o.begin + up4(n + 2);
    o.perm = o.order + 4ull * n;
    o.tiles = o.perm + up4(tokens);
    o.few = o.tiles + 4ull * tile_cap(tokens, n, kTile);
    o.words = o.few + (tokens <= kFewTokens ? sizeof(FewTile) / 4 * tile_cap(tokens, n, kFew) : 0);
    return o;
}
// Rank rows of the kernels: 16, 32, 64 or 128, the least that holds rank_max.
inline uint32_t padded_rank(uint32_t rank_max) { return rank_max <= 16 ? 16 : rank_max <= 32 ? 32 : rank_max <= 64 ? 64 : 128; }

// What every kernel knows of the batch.
struct Batch {
    uint32_t tokens, n, rank_max, part_stride; // part_stride: elements of one of the three parts
    const uint32_t* plan;
    const int32_t* ranks;  // nullptr: every adapter has rank_max
    const float* scales;   // nullptr: 1
    uint32_t* err;         // nullptr, or a word for what kernels report (bits 1 and 3)
};
// The plan's first four words: tiles with an adapter, all tiles, the same of kFew. All 0, and bit 3 of
// the error word, where the plan is of another batch (its buffer is as large as this batch's at least,
// so whatever is read of it besides is in its bounds).
__device__ __forceinline__ uint4 plan_head(const Batch& b, bool* good = nullptr) {
    const uint4 head = *reinterpret_cast<const uint4*>(b.plan), of = *reinterpret_cast<const uint4*>(b.plan + 4);
    const bool ok = of.x == b.tokens && of.y == b.n;
    if (!ok && b.err && threadIdx.x == 0) atomicOr(b.err, 8u);
    if (good) *good = ok;
    return ok ? head : make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ uint32_t rank_of(const Batch& b, uint32_t a) {
    if (!b.ranks) return b.rank_max;
    const int32_t r = b.ranks[a];
    return r < 0 ? 0u : min(static_cast<uint32_t>(r), b.rank_max);
}

// Programmatic dependent launch: the next kernel of the stream may be scheduled once every CTA of this
// one has started, and takes over the SMs that it leaves; this one goes on when the kernels before it
// have completed and what they wrote is visible. Nothing global is read or written before, and nothing by
// ld.global.nc (or __ldg), which is for data that stays as it is from the kernel's start to its end: the kernel
// before, which may still run then, can be the one that writes it (x may be the y of the call before).
// A kernel that takes tensor memory lets the next one go only once all of its CTA has seen tcgen05.alloc
// return (next_kernel_may_start behind that barrier). The next kernel's CTAs take tensor memory too, and hold it
// while they wait for this kernel to complete: if a CTA of this one still had to wait for its own share then, both
// could wait for good. So whenever a kernel's CTA is resident, those of the kernels before it have
// what they need.
__device__ __forceinline__ void kernels_before_done() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void next_kernel_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// The decoding kernel (bs_lora_few.cu): a cluster takes up to kFew tokens of one adapter through
// both products.
constexpr uint32_t kFewCluster = 8, kFewThreads = 256;
struct FewJob {
    const uint16_t *x, *a, *b;
    const uint8_t* base; // nullptr: 0
    uint8_t* out;        // nullptr: h only
    uint16_t* h;         // three parts of [tokens][R], in the plan's order
    uint64_t x_stride, base_stride, out_stride;
    uint32_t rows, cols, bf16, pad;
};
struct FewParams {
    Batch b;
    uint32_t split, pad; // clusters of a tile
    FewJob job[kMaxItems];
};
bs_status launch_few(FewParams& p, uint32_t jobs, uint32_t R, int dev, int sms, cudaStream_t s);

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t bf16_of(float f) { // to nearest, ties to even
    uint32_t r;
    asm("{\n .reg .b16 h;\n cvt.rn.bf16.f32 h, %1;\n mov.b32 %0, {h, 0};\n}" : "=r"(r) : "f"(f));
    return r;
}
__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// The three BF16 numbers whose sum is f: each takes 8 bits of what the ones before it left, 24 in
// all, so a rank-wide FP32 intermediate goes through the BF16 tensor cores without loss. What an
// infinity or NaN leaves is taken as 0, not as the NaN of inf - inf.
__device__ __forceinline__ void split3(float f, uint32_t (&q)[3]) {
    q[0] = bf16_of(f);
    const float h = __uint_as_float(q[0] << 16);
    const float r1 = (q[0] & 0x7F80u) == 0x7F80u ? 0.f : f - h;
    q[1] = bf16_of(r1);
    const float r2 = r1 - __uint_as_float(q[1] << 16);
    q[2] = bf16_of(r2);
}

// Raises a kernel's limit of dynamic shared memory, once per device (the limit stays).
template <auto FN>
inline cudaError_t allow_smem(int dev, uint32_t smem) {
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(FN, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

} // namespace lora
} // namespace bs
