// kv_append.cu -- new tokens' keys and values into their pages (streamscan.h,
// ss_kv_append): a row copy, or a quantisation to e4m3 with one scale per
// head.  Bound by memory: each row is read once and written once.
#include "kv.cuh"

namespace ss {

namespace {

constexpr int kAppendThreads = 256;

// One thread per element: simple, and right for every size.
template <typename T, bool QUANT>
__global__ void __launch_bounds__(kAppendThreads) k_kv_append(KvPages c, KvTable t, const T* __restrict__ k_new,
                                                             const T* __restrict__ v_new, int64_t token_stride,
                                                             int64_t head_stride, const int32_t* __restrict__ offsets,
                                                             int64_t rows, uint32_t* status) {
    const int64_t i = (int64_t)blockIdx.x * kAppendThreads + threadIdx.x;
    if (i >= rows * c.head_dim) return;
    const int64_t row = i / c.head_dim;
    const int d = (int)(i % c.head_dim);
    const int64_t tok = row / c.kv_heads;
    const int h = (int)(row % c.kv_heads);
    int b = (int)tok;
    int64_t back = 1;  // positions before the end
    if (offsets) {
        int lo = 0, hi = t.batch;  // the sequence with offsets[b] <= tok < offsets[b + 1]
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (offsets[mid] <= tok) lo = mid; else hi = mid;
        }
        b = lo;
        back = offsets[b + 1] - tok;
    }
    const int len = kv_len(t, b, status);
    const int64_t pos = len - back;
    if (back < 1 || pos < 0) {
        record_error(status, kErrKvTable, (uint32_t)b);
        return;
    }
    const int page = kv_page(t, c.num_pages, b, (int)(pos / c.page_size), status);
    if (page < 0) return;
    const int slot = (int)(pos % c.page_size);
    const int64_t src = tok * token_stride + h * head_stride + d;
    const int64_t dst = page * c.page_stride + h * c.head_stride + slot * c.slot_stride + d;
    if (QUANT) {
        const float ks = c.k_scale ? c.k_scale[h] : 1.0f, vs = c.v_scale ? c.v_scale[h] : 1.0f;
        reinterpret_cast<__nv_fp8_e4m3*>(c.k)[dst] = __nv_fp8_e4m3(__fdiv_rn(to_f32(k_new[src]), ks));
        reinterpret_cast<__nv_fp8_e4m3*>(c.v)[dst] = __nv_fp8_e4m3(__fdiv_rn(to_f32(v_new[src]), vs));
    } else {
        reinterpret_cast<T*>(c.k)[dst] = k_new[src];
        reinterpret_cast<T*>(c.v)[dst] = v_new[src];
    }
    if (d == 0 && c.weight) c.weight[((int64_t)page * c.kv_heads + h) * c.page_size + slot] = 0.0f;
}

}  // namespace

cudaError_t launch_kv_append(const KvPages& c, const KvTable& t, KvElem type, const void* k_new, const void* v_new,
                             int64_t token_stride, int64_t head_stride, const int32_t* offsets, int64_t tokens,
                             uint32_t* status, cudaStream_t s) {
    const int64_t rows = tokens * c.kv_heads;
    const unsigned grid = (unsigned)((rows * c.head_dim + kAppendThreads - 1) / kAppendThreads);
    const bool quant = c.type == KvElem::E4M3;
    if (type == KvElem::BF16) {
        const auto *k = static_cast<const __nv_bfloat16*>(k_new), *v = static_cast<const __nv_bfloat16*>(v_new);
        if (quant) k_kv_append<__nv_bfloat16, true><<<grid, kAppendThreads, 0, s>>>(c, t, k, v, token_stride, head_stride, offsets, rows, status);
        else k_kv_append<__nv_bfloat16, false><<<grid, kAppendThreads, 0, s>>>(c, t, k, v, token_stride, head_stride, offsets, rows, status);
    } else {
        const auto *k = static_cast<const __half*>(k_new), *v = static_cast<const __half*>(v_new);
        if (quant) k_kv_append<__half, true><<<grid, kAppendThreads, 0, s>>>(c, t, k, v, token_stride, head_stride, offsets, rows, status);
        else k_kv_append<__half, false><<<grid, kAppendThreads, 0, s>>>(c, t, k, v, token_stride, head_stride, offsets, rows, status);
    }
    return cudaGetLastError();
}

}  // namespace ss
