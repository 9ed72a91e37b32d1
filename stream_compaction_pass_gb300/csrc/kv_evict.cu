// kv_evict.cu -- eviction from a paged key-value cache by gathered attention
// weight (streamscan.h, ss_kv_evict).  Two launches: the selection finds, for
// every (sequence, head), the m-th best weight and writes the kept positions
// in order (a compaction whose predicate is a rank); the move copies the rows.
#include "kv.cuh"

namespace ss {

namespace {

constexpr int kSelectThreads = 256;
constexpr int kSelectWarps = kSelectThreads / 32;

__device__ __forceinline__ uint32_t key_at(const KvPages& c, const KvTable& t, int b, int h, int pos, int len,
                                           int sinks, int recent, uint32_t* status) {
    if (pos < sinks || pos >= len - recent) return 0u;
    const int page = kv_page(t, c.num_pages, b, pos / c.page_size, status);
    if (page < 0) return 0xffffffffu;
    return evict_key(c.weight[((int64_t)page * c.kv_heads + h) * c.page_size + pos % c.page_size]);
}

// One CTA per (sequence, head).  A radix selection, 8 bits of the key at a
// time from the top: a histogram of the keys that share the digits found so
// far, and the digit whose bin holds the m-th best.  Then one ordered pass
// writes the positions of the better keys and of the first ties.
__global__ void __launch_bounds__(kSelectThreads) k_kv_select(KvPages c, KvTable t, int keep, int sinks, int recent,
                                                             int32_t* __restrict__ kept, int32_t* __restrict__ new_lens,
                                                             uint32_t* status) {
    __shared__ uint32_t hist[256];
    __shared__ uint32_t s_digit, s_before;
    __shared__ uint32_t s_lt[kSelectWarps], s_eq[kSelectWarps];
    const int row = blockIdx.x, b = row / c.kv_heads, h = row % c.kv_heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int len = kv_len(t, b, status);
    const int m = min(len, keep);
    int32_t* out = kept + (int64_t)row * keep;
    if (h == 0 && tid == 0) new_lens[b] = m;
    for (int j = m + tid; j < keep; j += kSelectThreads) out[j] = -1;
    if (len <= keep) {
        for (int j = tid; j < m; j += kSelectThreads) out[j] = j;
        return;
    }
    uint32_t prefix = 0, mask = 0, want = (uint32_t)m;
    for (int shift = 24; shift >= 0; shift -= 8) {
        hist[tid] = 0;
        __syncthreads();
        for (int p = tid; p < len; p += kSelectThreads) {
            const uint32_t k = key_at(c, t, b, h, p, len, sinks, recent, status);
            if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (tid == 0) {
            uint32_t before = 0, d = 0;
            while (before + hist[d] < want) before += hist[d++];
            s_digit = d;
            s_before = before;
        }
        __syncthreads();
        want -= s_before;
        prefix |= s_digit << shift;
        mask |= 255u << shift;
        __syncthreads();
    }
    // `prefix` is the m-th best key; `want` of the positions that hold it stay.
    uint32_t lt_base = 0, eq_base = 0;
    for (int p0 = 0; p0 < len; p0 += kSelectThreads) {
        const int p = p0 + tid;
        const uint32_t k = p < len ? key_at(c, t, b, h, p, len, sinks, recent, status) : 0xffffffffu;
        const uint32_t lt = __ballot_sync(kFullMask, p < len && k < prefix);
        const uint32_t eq = __ballot_sync(kFullMask, p < len && k == prefix);
        if (lane == 0) {
            s_lt[warp] = __popc(lt);
            s_eq[warp] = __popc(eq);
        }
        __syncthreads();
        uint32_t my_lt = lt_base, my_eq = eq_base;
        for (int w = 0; w < kSelectWarps; ++w) {
            if (w < warp) {
                my_lt += s_lt[w];
                my_eq += s_eq[w];
            }
            lt_base += s_lt[w];
            eq_base += s_eq[w];
        }
        const uint32_t below = (1u << lane) - 1u;
        my_lt += __popc(lt & below);
        my_eq += __popc(eq & below);
        const bool is_lt = (lt >> lane) & 1u, is_eq = (eq >> lane) & 1u;
        if (is_lt || (is_eq && my_eq < want)) out[my_lt + min(my_eq, want)] = p;
        __syncthreads();
    }
}

// One CTA per kept row: its key, value and weight.
__global__ void __launch_bounds__(64) k_kv_move(KvPages c, KvTable t, KvPages d, KvTable dt, int keep,
                                                const int32_t* __restrict__ kept, int elem_bytes, uint32_t* status) {
    const int j = blockIdx.x % keep;
    const int row = blockIdx.x / keep;
    const int b = row / c.kv_heads, h = row % c.kv_heads;
    const int p = kept[(int64_t)row * keep + j];
    if (p < 0) return;
    if (j >= dt.max_pages * (int64_t)d.page_size) {
        if (threadIdx.x == 0) record_error(status, kErrKvTable, (uint32_t)b);
        return;
    }
    const int from = kv_page(t, c.num_pages, b, p / c.page_size, status);
    const int to = kv_page(dt, d.num_pages, b, j / d.page_size, status);
    if (from < 0 || to < 0) return;
    const int64_t src = (from * c.page_stride + h * c.head_stride + (p % c.page_size) * c.slot_stride) * elem_bytes;
    const int64_t dst = (to * d.page_stride + h * d.head_stride + (j % d.page_size) * d.slot_stride) * elem_bytes;
    const int vecs = c.head_dim * elem_bytes / 16;
    for (int i = threadIdx.x; i < vecs; i += 64) {
        stg_vec(d.k + dst + i * 16, ldg_vec(c.k + src + i * 16));
        stg_vec(d.v + dst + i * 16, ldg_vec(c.v + src + i * 16));
    }
    if (threadIdx.x == 0 && d.weight)
        d.weight[((int64_t)to * d.kv_heads + h) * d.page_size + j % d.page_size] =
            c.weight[((int64_t)from * c.kv_heads + h) * c.page_size + p % c.page_size];
}

}  // namespace

cudaError_t launch_kv_evict(const KvPages& c, const KvTable& t, const KvPages& d, const KvTable& dt, int keep,
                            int sinks, int recent, int32_t* kept, uint32_t* status, cudaStream_t s) {
    const unsigned rows = (unsigned)t.batch * (unsigned)c.kv_heads;
    k_kv_select<<<rows, kSelectThreads, 0, s>>>(c, t, keep, sinks, recent, kept, dt.lens, status);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    k_kv_move<<<rows * (unsigned)keep, 64, 0, s>>>(c, t, d, dt, keep, kept, kv_elem_bytes(c.type), status);
    return cudaGetLastError();
}

}  // namespace ss
