// kv.cuh -- what the paged key-value cache kernels share: the cache and its
// page tables as the kernels see them, checked look-ups, and element types.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "lookback.cuh"

namespace ss {

// Every kernel of this family is launched so that it may start before the
// kernel ahead of it on the stream has ended (programmatic dependent launch),
// and waits for that end here, first of all: only its launch overlaps.  What
// the kernel ahead may have written is therefore written while this one runs,
// so none of it is read as constant (no non-coherent loads, no const
// __restrict__ parameters).
__device__ __forceinline__ void begin_dependent() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename... P, typename... A>
inline cudaError_t launch_dependent(void (*kern)(P...), size_t grid, int threads, size_t smem, int cluster, cudaStream_t s, const A&... args) {
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

// Division of numbers below 2^31 by a fixed one, by a multiplication: with
// 2^l >= d and m = floor(2^32 (2^l - d) / d) + 1, n / d = (n m / 2^32 + n) / 2^l
// (Granlund and Montgomery, "Division by invariant integers using multiplication").
struct FastDiv {
    uint32_t mul;
    int shift;
    FastDiv() = default;
    explicit FastDiv(uint32_t d) : shift(0) {
        while ((1ull << shift) < d) ++shift;
        mul = (uint32_t)((((1ull << shift) - d) << 32) / d + 1);
    }
    __device__ __forceinline__ int div(int n) const { return (int)((__umulhi((uint32_t)n, mul) + (uint32_t)n) >> shift); }
};

// Rows of a CTA that first looks up its rows' places, a thread a row, and then
// moves their vectors, `round` rows at a time: more rounds share the look-up,
// as long as every SM still has 8 CTAs of them, up to `most` rows.
inline int kv_rows_per_cta(int round, int most, int64_t rows, int sms) {
    round = round < 1 ? 1 : round > most ? most : round;
    int64_t rounds = rows / ((int64_t)round * sms * 8);
    rounds = rounds < 1 ? 1 : rounds > most / round ? most / round : rounds;
    return round * (int)rounds;
}

// The length of sequence b as every kernel reads it: clamped to what the
// table can hold, and reported where it had to be.
__device__ __forceinline__ int kv_len(const KvTable& t, int b, uint32_t* status) {
    const int n = t.lens[b];
    const int m = min(max(n, 0), t.max_len);
    if (m != n) record_error(status, kErrKvTable, (uint32_t)(t.first + b));
    return m;
}

// The page of position `pos` of sequence b, or -1 (reported) if the table
// names a page outside the pool.
__device__ __forceinline__ int kv_page(const KvTable& t, int64_t num_pages, int b, int index, uint32_t* status) {
    const int p = t.pages[(int64_t)b * t.row_stride + index];
    if (p >= 0 && p < num_pages) return p;
    record_error(status, kErrKvTable, (uint32_t)(t.first + b));
    return -1;
}

// A 16-byte vector from L2, and one stored.
__device__ __forceinline__ uint4 ldg_vec(const void* p) { return __ldcg(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ void stg_vec(void* p, uint4 v) { *reinterpret_cast<uint4*>(p) = v; }

template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// Weights in the order of eviction as 32-bit keys, best first: a larger
// weight has the smaller key, -0 and +0 the same one, NaN the last.  Key 0 is
// no number's: it stands for the positions that stay whatever their weight.
__device__ __forceinline__ uint32_t evict_key(float w) {
    const int u = __float_as_int(w + 0.0f);  // -0 + 0 = +0
    const uint32_t k = (uint32_t)u ^ ((uint32_t)(~u >> 31) & 0x7fffffffu);
    return w != w ? 0xffffffffu : k;
}

}  // namespace ss
