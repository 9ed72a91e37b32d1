// kv_append.cu -- new tokens' keys and values into their pages (streamscan.h,
// ss_kv_append): a row copy, or a quantisation to e4m3 with one scale per
// head.  Bound by memory: each row is read once and written once.  A CTA takes
// a few (token, head) rows: one thread a row finds its page and slot, then all
// threads move 16-byte vectors of the result, every load issued before the
// first store.  108 thousand tokens of 8 heads of 128, bf16 to e4m3: 62 us, 0.84
// of the copy rate (96 with a look-up for every 64 rows, 102 with IEEE
// divisions, which made it instruction-bound); 64 tokens 2.5 us.
#include "kv.cuh"

namespace ss {

namespace {

constexpr int kAppendThreads = 256;
// Result vectors of a thread: 64 bytes of input in flight.
template <bool QUANT> constexpr int kAppendVecs = QUANT ? 2 : 4;

__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

template <typename T> __device__ __forceinline__ float2 open_pair(uint32_t u);
template <> __device__ __forceinline__ float2 open_pair<__nv_bfloat16>(uint32_t u) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
}
template <> __device__ __forceinline__ float2 open_pair<__half>(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// 16 elements over the scale, as e4m3, by a reciprocal and one correction: q =
// x r, then q - (q s - x) r, with r = 1 / s rounded.  That is the rounded
// quotient unless x / s lies within 2^-22 of a unit in the last place of the
// middle of two floats, which could matter only next to a tie of two e4m3
// values.  There, with X (11 bits), S (24) and T (5, of the tie) the integer
// significands, it takes |X 2^k - S (T 2^20 + 1)| < 8 with k >= 37, hence S =
// S1 2^20 + e with |e| < 8, 8 <= S1 <= 16 and T e + S1 = 0: only S = 2^24 - 1
// with T = 16, whose corrected quotient is (1 + 2^-24 + 2^-70) times the tie,
// on the same side of the middle as x / s.  (On the lower side, T e = S1 has no
// solution.)  So the e4m3 result is that of the division, and a zero keeps its
// sign: q s - x is then +0, and the correction -0, which changes no q, where
// r > 0.  Other scales, those for which a step could leave fp32's normal range,
// and non-finite elements are divided.
template <typename T> __device__ __forceinline__ uint4 quant16(const uint4 (&x)[2], float scale, float inverse) {
    const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    float y[16], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 a = open_pair<T>(w[i]);
        const float q0 = a.x * inverse, q1 = a.y * inverse;
        y[2 * i] = fmaf(-fmaf(q0, scale, -a.x), inverse, q0);
        y[2 * i + 1] = fmaf(-fmaf(q1, scale, -a.y), inverse, q1);
        sum += fabsf(y[2 * i]) + fabsf(y[2 * i + 1]);
    }
    if (!(sum < INFINITY)) {  // an infinity or NaN among them, or no inverse
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 a = open_pair<T>(w[i]);
            y[2 * i] = __fdiv_rn(a.x, scale);
            y[2 * i + 1] = __fdiv_rn(a.y, scale);
        }
    }
    return make_uint4(quant4(y[0], y[1], y[2], y[3]), quant4(y[4], y[5], y[6], y[7]), quant4(y[8], y[9], y[10], y[11]),
                      quant4(y[12], y[13], y[14], y[15]));
}

// The reciprocal of a scale, NaN for those outside [2^-60, 2^60] and negative ones.
__device__ __forceinline__ float inverse_of(float s) {
    return s >= 0x1p-60f && s <= 0x1p60f ? __frcp_rn(s) : NAN;
}

template <typename T, bool QUANT>
__global__ void __launch_bounds__(kAppendThreads, QUANT ? 4 : 6) k_kv_append(KvPages c, KvTable t, const T* k_new,
                                                             const T* v_new, int64_t token_stride,
                                                             int64_t head_stride, const int32_t* offsets,
                                                             int64_t rows, int per, int vecs, FastDiv by_vecs, FastDiv page,
                                                             uint32_t* status) {
    constexpr int kVecs = kAppendVecs<QUANT>;
    constexpr int kIn = QUANT ? 2 : 1;  // 16-byte vectors read for one written
    constexpr int kBytes = QUANT ? 1 : 2;
    __shared__ int64_t s_src[kAppendThreads], s_dst[kAppendThreads];  // byte offsets, dst -1: not written
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
                dst = ((int64_t)at * c.page_stride + (int64_t)h * c.head_stride + (int64_t)slot * c.slot_stride) * kBytes;
                if (c.weight) c.weight[((int64_t)at * c.kv_heads + h) * c.page_size + slot] = 0.0f;
            }
        }
        s_src[tid] = (tok * token_stride + h * head_stride) * 2;
        s_dst[tid] = dst;
        if (QUANT) {
            const float ks = c.k_scale ? c.k_scale[h] : 1.0f, vs = c.v_scale ? c.v_scale[h] : 1.0f;
            s_scale[0][tid] = make_float2(ks, inverse_of(ks));
            s_scale[1][tid] = make_float2(vs, inverse_of(vs));
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
            if constexpr (QUANT) {
                const float2 s = (&s_scale[0][0])[at[l]];
                y = quant16<T>(x[l], s.x, s.y);
            }
            stg_vec((at[l] >= kAppendThreads ? c.v : c.k) + to[l], y);
        }
    }
}

template <typename T, bool QUANT>
cudaError_t run(const KvPages& c, const KvTable& t, const void* k_new, const void* v_new, int64_t token_stride,
                int64_t head_stride, const int32_t* offsets, int64_t tokens, int sms, uint32_t* status, cudaStream_t s) {
    const int64_t rows = tokens * c.kv_heads;
    const int vecs = c.head_dim * (QUANT ? 1 : 2) / 16;
    const int per = kv_rows_per_cta(kAppendThreads * kAppendVecs<QUANT> / (2 * vecs), kAppendThreads, rows, sms);
    return launch_dependent(k_kv_append<T, QUANT>, (rows + per - 1) / per, kAppendThreads, 0, 1, s, c, t, static_cast<const T*>(k_new),
                            static_cast<const T*>(v_new), token_stride, head_stride, offsets, rows, per, vecs, FastDiv(vecs),
                            FastDiv(c.page_size), status);
}

}  // namespace

cudaError_t launch_kv_append(const KvPages& c, const KvTable& t, KvElem type, const void* k_new, const void* v_new,
                             int64_t token_stride, int64_t head_stride, const int32_t* offsets, int64_t tokens, int sms,
                             uint32_t* status, cudaStream_t s) {
    const bool quant = c.type == KvElem::E4M3;
    if (type == KvElem::BF16)
        return quant ? run<__nv_bfloat16, true>(c, t, k_new, v_new, token_stride, head_stride, offsets, tokens, sms, status, s)
                     : run<__nv_bfloat16, false>(c, t, k_new, v_new, token_stride, head_stride, offsets, tokens, sms, status, s);
    return quant ? run<__half, true>(c, t, k_new, v_new, token_stride, head_stride, offsets, tokens, sms, status, s)
                 : run<__half, false>(c, t, k_new, v_new, token_stride, head_stride, offsets, tokens, sms, status, s);
}

}  // namespace ss
