// kv_attend.cu -- attention of one new token per sequence over a paged
// key-value cache (streamscan.h, ss_kv_attend).
#include "kv.cuh"

namespace ss {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPerLane = 8;  // head_dim 256

// The visible positions of a sequence: p < len, and p < sinks or p >= start.
struct Visible {
    int len, sinks, start;
    __device__ Visible(int len_, int window, int sinks_) : len(len_) {
        start = window > 0 && window < len ? len - window : 0;
        sinks = sinks_;
    }
    __device__ bool operator()(int p) const { return p < sinks || p >= start; }
};

// One CTA per (sequence, key-value head); one warp per position, with the
// running maximum and sum of each warp's softmax, merged at the end.
template <typename QT, typename CT>
__global__ void __launch_bounds__(kThreads) k_kv_attend(KvPages c, KvTable t, KvAttention a, uint32_t* status) {
    extern __shared__ float s_q[];  // group x head_dim
    __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][32 * kMaxPerLane];
    const int b = blockIdx.x / c.kv_heads, h = blockIdx.x % c.kv_heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int D = c.head_dim, G = a.q_heads / c.kv_heads;
    float* s_lse = s_q + G * D;
    const QT* q = static_cast<const QT*>(a.q) + b * a.q_seq_stride;
    for (int i = tid; i < G * D; i += kThreads) s_q[i] = to_f32(q[(int64_t)(h * G + i / D) * a.q_head_stride + i % D]);
    __syncthreads();
    const int len = kv_len(t, b, status);
    const Visible seen(len, a.window, a.sinks);
    const float ks = (c.k_scale ? c.k_scale[h] : 1.0f) * a.scale;
    const float vs = c.v_scale ? c.v_scale[h] : 1.0f;
    const CT* kbase = reinterpret_cast<const CT*>(c.k) + h * c.head_stride;
    const CT* vbase = reinterpret_cast<const CT*>(c.v) + h * c.head_stride;
    auto score = [&](const CT* row, int g) {
        float x = 0.0f;
        for (int d = lane; d < D; d += 32) x += s_q[g * D + d] * to_f32(row[d]);
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFullMask, x, o);
        return x * ks;
    };
    for (int g = 0; g < G; ++g) {
        float m = -INFINITY, l = 0.0f, acc[kMaxPerLane] = {};
        for (int p = warp; p < len; p += kWarps) {
            if (!seen(p)) continue;
            const int page = kv_page(t, c.num_pages, b, p / c.page_size, status);
            if (page < 0) continue;
            const int64_t off = page * c.page_stride + (p % c.page_size) * c.slot_stride;
            const float x = score(kbase + off, g);
            const float top = fmaxf(m, x), ref = top == -INFINITY ? 0.0f : top;
            const float keep = __expf(m - ref), w = __expf(x - ref);
            m = top;
            l = l * keep + w;
            for (int i = 0; i < kMaxPerLane; ++i) {
                const int d = lane + 32 * i;
                if (d < D) acc[i] = acc[i] * keep + w * to_f32(vbase[off + d]);
            }
        }
        if (lane == 0) {
            s_m[warp] = m;
            s_l[warp] = l;
        }
        for (int i = 0; i < kMaxPerLane; ++i) s_o[warp][lane + 32 * i] = acc[i];
        __syncthreads();
        float top = -INFINITY, total = 0.0f;
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
        const float ref = top == -INFINITY ? 0.0f : top;
        for (int w = 0; w < kWarps; ++w) total += s_l[w] * expf(s_m[w] - ref);
        for (int d = tid; d < D; d += kThreads) {
            float o = 0.0f;
            for (int w = 0; w < kWarps; ++w) o += s_o[w][d] * expf(s_m[w] - ref);
            static_cast<QT*>(a.out)[b * a.out_seq_stride + (int64_t)(h * G + g) * a.out_head_stride + d] =
                from_f32<QT>(total == 0.0f ? 0.0f : o / total * vs);
        }
        const float lse = total == 0.0f ? -INFINITY : ref + logf(total);
        if (tid == 0) {
            s_lse[g] = lse;
            if (a.lse) a.lse[(int64_t)b * a.q_heads + h * G + g] = lse;
        }
        __syncthreads();
    }
    if (a.weight_out == nullptr) return;
    for (int p = warp; p < len; p += kWarps) {
        const int page = kv_page(t, c.num_pages, b, p / c.page_size, status);
        if (page < 0) continue;
        const int slot = p % c.page_size;
        const int64_t off = page * c.page_stride + slot * c.slot_stride;
        float w = 0.0f;
        if (seen(p))
            for (int g = 0; g < G; ++g) {
                const float x = score(kbase + off, g);
                w += s_lse[g] == -INFINITY ? 0.0f : expf(x - s_lse[g]);
            }
        const int64_t at = ((int64_t)page * c.kv_heads + h) * c.page_size + slot;
        if (lane == 0) a.weight_out[at] = (a.weight_in ? a.weight_in[at] : 0.0f) + w;
    }
}

template <typename QT, typename CT>
cudaError_t launch(const KvPages& c, const KvTable& t, const KvAttention& a, uint32_t* status, cudaStream_t s) {
    const int G = a.q_heads / c.kv_heads;
    const size_t smem = (size_t)G * (c.head_dim + 1) * 4;
    KernelSetup su;
    cudaError_t e = kernel_setup(reinterpret_cast<const void*>(k_kv_attend<QT, CT>), kThreads, (size_t)200 << 10, &su);
    if (e != cudaSuccess) return e;
    k_kv_attend<QT, CT><<<(unsigned)t.batch * (unsigned)c.kv_heads, kThreads, smem, s>>>(c, t, a, status);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_attend(const KvPages& c, const KvTable& t, const KvAttention& a, uint32_t* status, cudaStream_t s) {
    const bool bf = a.type == KvElem::BF16;
    if (c.type == KvElem::E4M3)
        return bf ? launch<__nv_bfloat16, __nv_fp8_e4m3>(c, t, a, status, s) : launch<__half, __nv_fp8_e4m3>(c, t, a, status, s);
    return bf ? launch<__nv_bfloat16, __nv_bfloat16>(c, t, a, status, s) : launch<__half, __half>(c, t, a, status, s);
}

}  // namespace ss
