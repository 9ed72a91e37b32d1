// kv_append.cu -- new tokens' keys and values into their pages (streamscan.h,
// ss_kv_append): a row copy, a quantisation to e4m3 with one scale per head, or
// one to e2m1 with a scale of every 16 elements beside it.  Bound by memory: each
// row is read once and written once.  A CTA takes a few (token, head) rows: one
// thread a row finds its page and slot, then all threads move 16-byte vectors of
// the result, every load issued before the first store.  57,382 tokens of 8 heads
// of 128, bf16 to e4m3: 62 us, 0.84 of the copy rate (96 with a look-up for every 64
// rows, 102 with IEEE divisions, which made it instruction-bound); to e2m1, 15 % fewer
// bytes and more instructions (issued in 71 % of the cycles, with 28 warps an SM
// waiting for loads), 63.2 us, 0.71; 64 tokens 2.5 us.
#include "kv_quant.cuh"

namespace ss {

namespace {

constexpr int kAppendThreads = 256;
// 16-byte vectors read for one written, and result vectors of a thread: 64 bytes
// of input in flight.
template <int BITS> constexpr int kAppendIn = 16 / BITS;
template <int BITS> constexpr int kAppendVecs = 4 / kAppendIn<BITS>;

// 32 elements, times the inverse of the head's scale, as e2m1 codes of two blocks
// and the blocks' scales.
template <typename T> __device__ __forceinline__ uint4 quant32(const uint4 (&x)[4], float inverse, uint32_t& scales) {
    uint32_t codes[4];
    scales = 0;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const uint32_t w[8] = {x[2 * b].x, x[2 * b].y, x[2 * b].z, x[2 * b].w, x[2 * b + 1].x, x[2 * b + 1].y, x[2 * b + 1].z, x[2 * b + 1].w};
        float y[16], most = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 a = open_pair<T>(w[i]);
            y[2 * i] = a.x * inverse;
            y[2 * i + 1] = a.y * inverse;
            most = abs_max(abs_max(most, y[2 * i]), y[2 * i + 1]);
        }
        const BlockScale s(most);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float z[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = s.over(y[half * 8 + i]);
            codes[2 * b + half] = e2m1x8(z);
        }
        scales |= s.code << (8 * b);
    }
    return make_uint4(codes[0], codes[1], codes[2], codes[3]);
}

template <typename T, int BITS>
__global__ void __launch_bounds__(kAppendThreads, BITS < 16 ? 4 : 6) k_kv_append(KvPages c, KvTable t, const T* k_new,
                                                             const T* v_new, int64_t token_stride,
                                                             int64_t head_stride, const int32_t* offsets,
                                                             int64_t rows, int per, int vecs, FastDiv by_vecs, FastDiv page,
                                                             uint32_t* status) {
    constexpr int kVecs = kAppendVecs<BITS>;
    constexpr int kIn = kAppendIn<BITS>;
    constexpr int kUnit = BITS == 16 ? 2 : 1;  // bytes that strides count in
    __shared__ int64_t s_src[kAppendThreads], s_dst[kAppendThreads];  // byte offsets, dst -1: not written
    __shared__ int64_t s_block[BITS == 4 ? kAppendThreads : 1];  // where the row's scales go
    __shared__ float2 s_scale[2][kAppendThreads];  // k's and v's scale and its inverse
    begin_dependent();
    const int tid = threadIdx.x;
    const int64_t row0 = (int64_t)blockIdx.x * per;
    if (tid < per && row0 + tid < rows) {
        const int64_t tok = (row0 + tid) / c.kv_heads;
        const int h = (int)((row0 + tid) % c.kv_heads);
        int b = (int)tok;
        int64_t back = 1;  // positions before the end
        if (offsets) {
            int lo = 0, hi = t.batch;  // the last b with offsets[b] <= tok
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (offsets[mid] <= tok) lo = mid; else hi = mid;
            }
            b = lo;
            back = offsets[b + 1] - tok;
        }
        const int64_t pos = kv_len(t, b, status) - back;
        int64_t dst = -1;
        if (back < 1 || pos < 0) {
            record_error(status, kErrKvTable, (uint32_t)(t.first + b));
        } else {
            const int index = page.div((int)pos), slot = (int)pos - index * c.page_size;
            const int at = kv_page(t, c.num_pages, b, index, status);
            if (at >= 0) {
                dst = ((int64_t)at * c.page_stride + (int64_t)h * c.head_stride + (int64_t)slot * c.slot_stride) * kUnit;
                const int64_t row = ((int64_t)at * c.kv_heads + h) * c.page_size + slot;
                if (c.weight) c.weight[row] = 0.0f;
                if constexpr (BITS == 4) s_block[tid] = row * (c.head_dim / 16);
            }
        }
        s_src[tid] = (tok * token_stride + h * head_stride) * 2;
        s_dst[tid] = dst;
        if (BITS < 16) {
            const float ks = c.k_scale ? c.k_scale[h] : 1.0f, vs = c.v_scale ? c.v_scale[h] : 1.0f;
            s_scale[0][tid] = make_float2(ks, BITS == 4 ? __frcp_rn(ks) : inverse_of(ks));
            s_scale[1][tid] = make_float2(vs, BITS == 4 ? __frcp_rn(vs) : inverse_of(vs));
        }
    }
    __syncthreads();
    const int here = (int)min((int64_t)per, rows - row0);
    const int half = here * vecs;  // k's vectors, then v's
    for (int i0 = tid; i0 < 2 * half; i0 += kAppendThreads * kVecs) {
        uint4 x[kVecs][kIn];
        int64_t to[kVecs];
        int at[kVecs];
#pragma unroll
        for (int l = 0; l < kVecs; ++l) {
            const int i = i0 + l * kAppendThreads;
            to[l] = -1;
            if (i >= 2 * half) continue;
            const bool is_v = i >= half;
            const int k = is_v ? i - half : i, r = by_vecs.div(k), v = k - r * vecs;
            if (s_dst[r] < 0) continue;
            const char* from = reinterpret_cast<const char*>(is_v ? v_new : k_new) + s_src[r] + v * (16 * kIn);
#pragma unroll
            for (int e = 0; e < kIn; ++e) x[l][e] = ldg_vec(from + 16 * e);
            to[l] = s_dst[r] + v * 16;
            at[l] = is_v ? r + kAppendThreads : r;
        }
#pragma unroll
        for (int l = 0; l < kVecs; ++l) {
            if (to[l] < 0) continue;
            uint4 y = x[l][0];
            if constexpr (BITS == 8) {
                const float2 s = (&s_scale[0][0])[at[l]];
                y = quant16<T>(x[l], s.x, s.y);
            }
            if constexpr (BITS == 4) {
                const bool is_v = at[l] >= kAppendThreads;
                const int r = at[l] & (kAppendThreads - 1), i = i0 + l * kAppendThreads, k = is_v ? i - half : i;
                uint32_t scales;
                y = quant32<T>(x[l], (&s_scale[0][0])[at[l]].y, scales);
                *reinterpret_cast<uint16_t*>((is_v ? c.v_block : c.k_block) + s_block[r] + 2 * (k - r * vecs)) = (uint16_t)scales;
            }
            stg_vec((at[l] >= kAppendThreads ? c.v : c.k) + to[l], y);
        }
    }
}

template <typename T, int BITS>
cudaError_t run(const KvPages& c, const KvTable& t, const void* k_new, const void* v_new, int64_t token_stride,
                int64_t head_stride, const int32_t* offsets, int64_t tokens, int sms, uint32_t* status, cudaStream_t s) {
    const int64_t rows = tokens * c.kv_heads;
    const int vecs = c.head_dim * BITS / 128;
    const int per = kv_rows_per_cta(kAppendThreads * kAppendVecs<BITS> / (2 * vecs), kAppendThreads, rows, sms);
    return launch_dependent(k_kv_append<T, BITS>, (rows + per - 1) / per, kAppendThreads, 0, 1, s, c, t, static_cast<const T*>(k_new),
                            static_cast<const T*>(v_new), token_stride, head_stride, offsets, rows, per, vecs, FastDiv(vecs),
                            FastDiv(c.page_size), status);
}

}  // namespace

cudaError_t launch_kv_append(const KvPages& c, const KvTable& t, KvElem type, const void* k_new, const void* v_new,
                             int64_t token_stride, int64_t head_stride, const int32_t* offsets, int64_t tokens, int sms,
                             uint32_t* status, cudaStream_t s) {
    auto go = [&](auto bits) {
        constexpr int kBits = decltype(bits)::value;
        return type == KvElem::BF16 ? run<__nv_bfloat16, kBits>(c, t, k_new, v_new, token_stride, head_stride, offsets, tokens, sms, status, s)
                                    : run<__half, kBits>(c, t, k_new, v_new, token_stride, head_stride, offsets, tokens, sms, status, s);
    };
    if (c.type == KvElem::E2M1) return go(std::integral_constant<int, 4>());
    if (c.type == KvElem::E4M3) return go(std::integral_constant<int, 8>());
    return go(std::integral_constant<int, 16>());
}

}  // namespace ss
