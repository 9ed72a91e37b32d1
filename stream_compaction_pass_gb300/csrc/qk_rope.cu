// qk_rope.cu -- norms of query and key rows with the rotation by their positions
// (streamscan.h, ss_qk_norm_rope), the gradients (ss_qk_norm_rope_backward), and
// the form that writes keys and values into a paged cache (ss_kv_append_rope).
//
// Mathematics.  Of a head's row x, r = 1 / sqrt(mean x^2 + eps), u = r w x, and y =
// R u, where R turns pairs of u by the position's angles.  Backward, with h = R^T
// g: dw = sum r x h over all rows, and dx = r (w h - x r^2 mean(w h x)).  An angle
// is a fraction of a turn: position times frequency modulo 1, which 64-bit integers
// multiply exactly with the frequency in units of 2^-64 turns, however far the
// position.  Of what is left, fp32 rows and those for narrow caches (where a value
// beside a tie of two codes moves by a whole step) take CUDA's sincospif, with what
// the angle's rounding to fp32 leaves out added by the derivatives (of 164 million
// e4m3 codes 233 differ from those of 64 bits, 358 without), and the rounded
// reciprocal root; 16-bit ones the approximations, whose errors (2^-21 of 1,
// 2 units in the last place) are a thousandth of the outputs' rounding and whose
// instructions are fewer (57.5 us without, 55.4 with them, of 16384 x 40 rows, in
// CTAs of 256).
//
// What bounds it.  Memory: every row is read once and written once (backward:
// two and one), for about 10 operations an element, so that instructions come
// close.  L lanes share a row, each with two 16-byte vectors whose elements are
// each other's partners in the rotation, so that it needs no exchange, and the norm
// log2 L shuffles.  A CTA takes consecutive rows of one of the tensors, which
// leaves it one set of strides and weights, and computes their tokens' sines and
// cosines once, in shared memory; its threads copy the rows to come, each its own
// vectors, two steps ahead (three into a cache).  bf16 rows of 128, 16384 x 40: 53.7
// us, 0.92 of the copy rate, issuing in 82 % of the cycles; the gradients 83.8, 0.88,
// with the 16 warps an SM that 109 registers leave; 20000 x 48 into an 8-bit cache
// 82.3, 0.80, by quantisation's instructions, into 4 bits 91.8, 0.69, by the same (both
// issue in 78 % of the cycles), into bf16 79, 0.91.  fp32 rows, 16384 x 40: 148 us,
// 0.67, waiting for shared memory with the 16 warps that 100 registers leave.
#include <algorithm>

#include "kv_quant.cuh"

namespace ss {

namespace {

// Small CTAs: as many warps wait at a barrier as share its tables, and a rotation by
// all 256 elements has a thread for each of its 128 angles.  Threads of 128 / 256, as
// many warps an SM: backward 84.6 / 90.1 us, forward 55.3 / 56.1, into an 8-bit cache
// 84.4 / 88.4 (64: 85.2, 55.7, 86.0).  20 warps an SM backward, for 16, leave 96
// registers, which are too few: 117.
constexpr int kThreads = 128;
// Rows of a ring: those on their way, and the one at hand.  Of tensors 3 (backward
// 83.8 us, 4 86.5; forward 55.8, 55.9), into a cache 4 (84.4, 3 91.1, 5 86.6).
template <int BITS> constexpr int kStages = BITS > 0 ? 4 : 3;

__device__ __forceinline__ uint32_t pack_pair(__nv_bfloat16, float x, float y) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_pair(__half, float x, float y) {
    const __half2 v = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Two fp32 numbers side by side, which one instruction works on.
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float x, float y) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 open_f2(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ float sum_f2(F2 a) {
    const float2 x = open_f2(a);
    return x.x + x.y;
}
// a - b c, rounded once.
__device__ __forceinline__ F2 less2(F2 a, F2 b, F2 c) { return fma2(b * f2(-1.0f, -1.0f), c, a); }

// Eight elements as they lie in memory, and as fp32.
template <typename T> struct Eight {
    uint4 v[sizeof(T) / 2];
    static constexpr int kVecs = sizeof(T) / 2;
    // The copies of eight elements to vectors v and on of a ring's stage (zeros where
    // bytes is 0), and they from there.
    template <typename R> static __device__ __forceinline__ void copy(const R& ring, uint32_t stage, int v, const T* p, int bytes) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) ring.copy(stage, v + i, reinterpret_cast<const uint4*>(p) + i, bytes);
    }
    template <typename R> __device__ __forceinline__ Eight(const R& ring, uint32_t stage, int at) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i] = ring.get(stage, at + i);
    }
    __device__ __forceinline__ void open(F2 (&x)[4]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x[2 * i] = f2(__uint_as_float(v[i].x), __uint_as_float(v[i].y));
                x[2 * i + 1] = f2(__uint_as_float(v[i].z), __uint_as_float(v[i].w));
            }
        } else {
            const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 a = open_pair<T>(w[i]);
                x[i] = f2(a.x, a.y);
            }
        }
    }
    static __device__ __forceinline__ void store(T* p, const F2 (&x)[4]) {
        float2 f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = open_f2(x[i]);
        if constexpr (sizeof(T) == 4) {
            stg_vec(p, make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y)));
            stg_vec(p + 4, make_uint4(__float_as_uint(f[2].x), __float_as_uint(f[2].y), __float_as_uint(f[3].x), __float_as_uint(f[3].y)));
        } else {
            stg_vec(p, make_uint4(pack_pair(T(), f[0].x, f[0].y), pack_pair(T(), f[1].x, f[1].y), pack_pair(T(), f[2].x, f[2].y), pack_pair(T(), f[3].x, f[3].y)));
        }
    }
};
__device__ __forceinline__ void floats(const F2 (&x)[4], float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = open_f2(x[i]);
        f[2 * i] = a.x;
        f[2 * i + 1] = a.y;
    }
}

// A lane's own vectors of the rows to come, in shared memory: only the thread that
// copied them reads them, so nothing but its own copies is waited for.  NV vectors
// of 16 bytes a row, S rows; a row's stage is given by its offset.
template <int NV, int S> struct Ring {
    uint32_t base;
    __device__ __forceinline__ Ring(void* smem)
        : base((uint32_t)__cvta_generic_to_shared(smem) + (threadIdx.x / 32) * (S * NV * 512) + threadIdx.x % 32 * 16) {}
    static size_t bytes(int threads) { return (size_t)NV * S * threads * 16; }
    static constexpr uint32_t kStage = NV * 512;
    static __device__ __forceinline__ uint32_t after(uint32_t stage) { return stage == (S - 1) * kStage ? 0 : stage + kStage; }
    __device__ __forceinline__ void copy(uint32_t stage, int v, const void* from, int bytes) const {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(base + stage + v * 512), "l"(from), "r"(bytes) : "memory");
    }
    static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    static __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory"); }
    static __device__ __forceinline__ void wait_all() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
    __device__ __forceinline__ uint4 get(uint32_t stage, int v) const {
        uint4 x;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(base + stage + v * 512) : "memory");
        return x;
    }
};

// How a row of head_dim = 8 vecs elements lies over its lanes: lane p < pairs
// has the vectors p and p + pairs, which are turned with each other (or each in
// itself, where pairs are adjacent), the lanes after them 2 p and 2 p + 1.
struct Layout {
    int vecs, pairs;
    __device__ __forceinline__ int first(int p) const { return p < pairs ? p : 2 * p; }
    __device__ __forceinline__ int second(int p) const { return p < pairs ? p + pairs : 2 * p + 1; }
};

// A lane's part of a group's rows, every `groups`th one: where its first vector is.
struct Walk {
    const char* at;
    int head;
    int64_t step, wrap;  // to the next row; more, where that is another token's
    __device__ __forceinline__ Walk(const char* base, int64_t token_stride, int64_t head_stride, int size, int64_t token, int head_, int heads, int step_tokens, int step_heads,
                                    int first)
        : at(base + (token * token_stride + head_ * head_stride + first) * size), head(head_),
          step((step_tokens * token_stride + step_heads * head_stride) * size), wrap((token_stride - heads * head_stride) * size) {}
    // Whether the next row is another token's (beside step_tokens).
    __device__ __forceinline__ bool next(int heads, int step_heads) {
        head += step_heads;
        const bool over = head >= heads;
        at += over ? step + wrap : step;
        head -= over ? heads : 0;
        return over;
    }
};

// Shared memory: the weights, and cosines and sines of the tokens at hand, each in
// four planes of L float4: plane j of lane p has a lane's numbers 4 j and on.
template <int L> struct Tables {
    float4 *weight, *turn;
    int pairs, lanes;
    __device__ __forceinline__ Tables(void* smem, const Layout& l) : pairs(l.pairs), lanes((l.vecs + 1) / 2) {
        weight = static_cast<float4*>(smem);
        turn = weight + 4 * L;
    }
    __device__ __forceinline__ void* end(int tokens) const { return turn + tokens * 4 * L; }
    static size_t bytes(int tokens) { return ((size_t)tokens + 1) * 4 * L * 16; }
    static __device__ __forceinline__ void get(const float4* plane, F2 (&x)[4], F2 (&y)[4]) {
        const float4 v[4] = {plane[0], plane[L], plane[2 * L], plane[3 * L]};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            x[2 * i] = f2(v[i].x, v[i].y);
            x[2 * i + 1] = f2(v[i].z, v[i].w);
            y[2 * i] = f2(v[2 + i].x, v[2 + i].y);
            y[2 * i + 1] = f2(v[2 + i].z, v[2 + i].w);
        }
    }
    __device__ __forceinline__ void turns_of(int token, int p, F2 (&c)[4], F2 (&s)[4]) const { get(turn + token * 4 * L + p, c, s); }
    __device__ __forceinline__ void weights_of(int p, F2 (&a)[4], F2 (&b)[4]) const { get(weight + p, a, b); }

    // A thread has one of the frequencies, and every few tokens.
    template <bool FINE> __device__ __forceinline__ void fill_turns(const QkRope& a, int64_t t0, int tokens) const {
        const int per = pairs * 8, side = blockDim.x / per, m = threadIdx.x % per, p = m >> 3, j = m & 7;
        if ((int)threadIdx.x >= side * per) return;
        const unsigned long long f = a.turns[!a.interleaved ? m : j < 4 ? 4 * p + j : 4 * (p + pairs) + j - 4];
        float* to = reinterpret_cast<float*>(turn + (j >> 2) * L + p) + (j & 3);
        for (int t = threadIdx.x / per; t < tokens; t += side) {
            const int at = a.positions[t0 + t];
            float s, c;
            if (FINE) {
                // and what rounding the angle to fp32 leaves out, by the derivatives
                const long long turns = (long long)(f * (unsigned long long)(long long)at);
                const float near = __ll2float_rn(turns), rest = __ll2float_rn(turns - __float2ll_rn(near)) * (0x1p-63f * 3.14159265358979f);
                float s0, c0;
                sincospif(near * 0x1p-63f, &s0, &c0);
                s = fmaf(c0, rest, s0);
                c = fmaf(-s0, rest, c0);
            } else {  // the product's high half
                const uint32_t low = (uint32_t)f, high = (uint32_t)(f >> 32) * (uint32_t)at + __umulhi(low, (uint32_t)at) - (at < 0 ? low : 0u);
                __sincosf((float)(int)high * (0x1p-31f * 3.14159265358979f), &s, &c);
            }
            to[t * 16 * L] = c;
            to[t * 16 * L + 8 * L] = s;
        }
    }
    __device__ __forceinline__ void fill_weights(const char* w, KvElem type, const Layout& l) const {
        for (int i = threadIdx.x; i < 16 * lanes; i += blockDim.x) {
            const int p = i >> 4, j = i & 15, vec = j < 8 ? l.first(p) : l.second(p), d = vec * 8 + (j & 7);
            float x = 1.0f;
            if (w && vec < l.vecs) {
                x = type == KvElem::F32    ? reinterpret_cast<const float*>(w)[d]
                    : type == KvElem::BF16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(w)[d])
                                           : __half2float(reinterpret_cast<const __half*>(w)[d]);
            }
            reinterpret_cast<float*>(weight + (j >> 2) * L + p)[j & 3] = x;
        }
    }
};

// Turns a lane's 16 elements by their angles, or back.
template <bool BACK> __device__ __forceinline__ void turn16(F2 (&a)[4], F2 (&b)[4], const F2 (&c)[4], const F2 (&s)[4], bool interleaved) {
    if (!interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const F2 x = a[i], y = b[i];
            a[i] = BACK ? fma2(y, s[i], x * c[i]) : less2(x * c[i], y, s[i]);
            b[i] = BACK ? less2(y * c[i], x, s[i]) : fma2(x, s[i], y * c[i]);
        }
    } else {
        auto turn = [](F2& z, float co, float si) {
            const float2 x = open_f2(z);
            const float w = BACK ? -si : si;
            z = f2(x.x * co - x.y * w, x.y * co + x.x * w);
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 ca = open_f2(c[i / 2]), sa = open_f2(s[i / 2]), cb = open_f2(c[2 + i / 2]), sb = open_f2(s[2 + i / 2]);
            turn(a[i], i % 2 ? ca.y : ca.x, i % 2 ? sa.y : sa.x);
            turn(b[i], i % 2 ? cb.y : cb.x, i % 2 ? sb.y : sb.x);
        }
    }
}

template <bool FINE> __device__ __forceinline__ float inverse_root(float x) { return FINE ? __frsqrt_rn(x) : rsqrtf(x); }

template <int L> __device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int i = 1; i < L; i <<= 1) x += __shfl_xor_sync(kFullMask, x, i);
    return x;
}

// ---- forward ----

// Where a token's rows go in a cache: offsets in what strides count in, and
// the number of head 0's row among [page][head][slot]; -1: nowhere.
struct Place {
    int64_t at, row;
};

template <int BITS, typename T>
__device__ __forceinline__ void store_cached(const KvPages& c, const Place& to, bool is_v, int h, const Layout& l, int p, bool in, const F2 (&a2)[4], const F2 (&b2)[4]) {
    char* pool = is_v ? c.v : c.k;
    const int64_t at = to.at + (int64_t)h * c.head_stride;
    const float* scales = is_v ? c.v_scale : c.k_scale;
    const int first = l.first(p), second = l.second(p);
    if constexpr (BITS == 16) {
        if (!in) return;
        Eight<T>::store(reinterpret_cast<T*>(pool) + at + first * 8, a2);
        if (second < l.vecs) Eight<T>::store(reinterpret_cast<T*>(pool) + at + second * 8, b2);
    } else if constexpr (BITS == 8) {
        if (!in) return;
        const float s = scales ? scales[h] : 1.0f, inverse = inverse_of(s);
        auto put = [&](int vec, const F2 (&x2)[4]) {
            float x[8], y[8];
            floats(x2, x);
            quotients(x, s, inverse, y);
            *reinterpret_cast<uint2*>(pool + at + vec * 8) = make_uint2(quant4(y[0], y[1], y[2], y[3]), quant4(y[4], y[5], y[6], y[7]));
        };
        put(first, a2);
        if (second < l.vecs) put(second, b2);
    } else {
        const float inverse = scales && in ? __frcp_rn(scales[h]) : 1.0f;
        float a[8], b[8], y[16], ma = 0.0f, mb = 0.0f;
        floats(a2, a);
        floats(b2, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            y[i] = a[i] * inverse;
            y[8 + i] = b[i] * inverse;
            ma = abs_max(ma, y[i]);
            mb = abs_max(mb, y[8 + i]);
        }
        // a block of 16 lies in a lane and its neighbour (pairs is even), or in one lane
        const float na = __shfl_xor_sync(kFullMask, ma, 1), nb = __shfl_xor_sync(kFullMask, mb, 1);
        const bool turned = p < l.pairs;
        const BlockScale sa(abs_max(ma, turned ? na : mb)), sb(abs_max(mb, turned ? nb : ma));
        if (!in) return;
        uint8_t* block = (is_v ? c.v_block : c.k_block) + (to.row + (int64_t)h * c.page_size) * (c.head_dim / 16);
        float za[8], zb[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            za[i] = sa.over(y[i]);
            zb[i] = sb.over(y[8 + i]);
        }
        *reinterpret_cast<uint32_t*>(pool + at + first * 4) = e2m1x8(za);
        *reinterpret_cast<uint32_t*>(pool + at + second * 4) = e2m1x8(zb);
        if (!turned || (p & 1) == 0) {
            block[first / 2] = (uint8_t)sa.code;
            if (turned) block[second / 2] = (uint8_t)sb.code;
        }
    }
}

// The CTAs of each tensor.  A row's number is token * heads + head.
struct Jobs {
    int ctas[3];   // of q, k and v
    int steps[3];  // of a CTA: a row for every group
    int chunk[3];  // steps between two fillings of the tables
    FastDiv by_heads[3];
};
// Selected, not indexed: parameters that are would be copied to local memory.
template <typename X> __device__ __forceinline__ X pick(const X (&x)[3], int i) { return i == 0 ? x[0] : i == 1 ? x[1] : x[2]; }

// What a CTA does: `kind` 0, 1 or 2 for q, k or v, and consecutive rows of it, of
// which a thread's group has every `groups`th.
struct Share {
    int kind, heads, steps, chunk, token, head, step_tokens, step_heads;
    int64_t t0;
    bool last;  // whether the last step has a row for this group
    __device__ __forceinline__ Share(const QkRope& a, const Jobs& jobs, int group, int groups) {
        const int c = blockIdx.x;
        kind = c < jobs.ctas[0] ? 0 : c < jobs.ctas[0] + jobs.ctas[1] ? 1 : 2;
        heads = kind == 0 ? a.q.heads : kind == 1 ? a.k.heads : a.v.heads;
        const FastDiv by_heads = pick(jobs.by_heads, kind);
        const int most = pick(jobs.steps, kind) * groups;
        const int64_t begin = (int64_t)(c - (kind == 0 ? 0 : kind == 1 ? jobs.ctas[0] : jobs.ctas[0] + jobs.ctas[1])) * most;
        chunk = pick(jobs.chunk, kind);
        t0 = begin < 0x7fffffff ? by_heads.div((int)begin) : begin / heads;
        head0 = (int)(begin - t0 * heads);
        rows = (int)min((int64_t)most, a.tokens * heads - begin);
        steps = (rows + groups - 1) / groups;
        last = (steps - 1) * groups + group < rows;
        step_tokens = by_heads.div(groups);
        step_heads = groups - step_tokens * heads;
        token = by_heads.div(head0 + group);
        head = head0 + group - token * heads;
    }
    int head0, rows;
    // The tokens, from t0 on, of the rows of steps [k, k + chunk).
    __device__ __forceinline__ int2 tokens(const Jobs& jobs, int k, int groups) const {
        const FastDiv by_heads = pick(jobs.by_heads, kind);
        const int from = by_heads.div(head0 + k * groups);
        return make_int2(from, by_heads.div(head0 + min((k + chunk) * groups, rows) - 1) - from + 1);
    }
};

// BITS 0: rows go to tensors; else k's and v's go to a cache of so many bits.
template <typename T, int L, int BITS>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 4 : BITS ? 6 : 8) k_qk_rope(QkRope a, Layout l, Jobs jobs, int most_tokens, float inv_dim, KvPages c, const int64_t* slots, FastDiv page,
                                                          uint32_t* status) {
    constexpr bool CACHE = BITS > 0, kFine = sizeof(T) == 4 || BITS == 8 || BITS == 4;
    constexpr int kVecs = Eight<T>::kVecs, S = kStages<BITS>;
    extern __shared__ float4 s_tables[];
    __shared__ Place s_place[CACHE ? kThreads / L + 2 : 1];
    const Tables<L> tables(s_tables, l);
    using Rows = Ring<2 * kVecs, S>;
    const Rows ring(tables.end(most_tokens));
    const int tid = threadIdx.x, p = tid % L, groups = blockDim.x / L, lanes = (l.vecs + 1) / 2, first = l.first(p), second = l.second(p);
    const Share me(a, jobs, tid / L, groups);
    const bool is_q = me.kind == 0, is_v = CACHE && me.kind == 2;
    const QkRows& of = is_q ? a.q : is_v ? a.v : a.k;
    const bool one = p < lanes, two = one && second < l.vecs;
    // Lanes without a vector take zeros, and rows behind the last what is there.
    const int one_bytes = one ? 16 : 0, two_bytes = two ? 16 : 0, apart = two ? (second - first) * 8 : 0;
    auto walk = [&](const char* base, int64_t token_stride, int64_t head_stride) {
        return Walk(base, token_stride, head_stride, sizeof(T), me.t0 + me.token, me.head, me.heads, me.step_tokens, me.step_heads, one ? first * 8 : 0);
    };
    Walk from = walk(of.x, of.token_stride, of.head_stride), to = walk(of.y, of.y_token_stride, of.y_head_stride);
    const int mine = me.last ? me.steps : me.steps - 1;  // rows of this group
    auto issue = [&](int k, uint32_t stage) {
        if (k < mine) {
            const T* x = reinterpret_cast<const T*>(from.at);
            Eight<T>::copy(ring, stage, 0, x, one_bytes);
            Eight<T>::copy(ring, stage, kVecs, x + apart, two_bytes);
        }
        from.next(me.heads, me.step_heads);
    };
    begin_dependent();
    // the first rows are on their way while the tables are filled
#pragma unroll
    for (int k = 0; k < S - 1; ++k) {
        issue(k, k * Rows::kStage);
        ring.commit();
    }
    F2 wa[4] = {}, wb[4] = {};
    if (!is_v) tables.fill_weights(of.weight, a.weight_type, l);

    // The row's token among those of the tables, the first of which is `done`, and the next filling.
    uint32_t stage = 0, refilled = (S - 1) * Rows::kStage;  // at hand, and read in the last step
    int token = 0, done = 0, fill = 0;
    for (int k = 0; k < me.steps; ++k) {
        if (k == fill) {
            const int2 range = me.tokens(jobs, k, groups);
            if (k > 0) __syncthreads();
            if (kFine && sizeof(T) < 4 && is_q) tables.template fill_turns<false>(a, me.t0 + range.x, range.y);
            else if (!is_v) tables.template fill_turns<kFine>(a, me.t0 + range.x, range.y);
            if constexpr (CACHE) {
                for (int i = tid; !is_q && i < range.y; i += blockDim.x) {
                    const int64_t t = me.t0 + range.x + i, slot = slots[t], all = c.num_pages * c.page_size;
                    Place at{-1, -1};
                    if (slot >= 0 && slot < all) {
                        const int64_t index = slot < 0x7fffffff ? page.div((int)slot) : slot / c.page_size, s = slot - index * c.page_size;
                        at.at = index * c.page_stride + s * c.slot_stride;
                        at.row = index * c.kv_heads * c.page_size + s;
                    } else if (slot >= all) {
                        record_error(status, kErrKvTable, (uint32_t)t);
                    }
                    s_place[i] = at;
                }
            }
            __syncthreads();
            if (k == 0) {
                token = me.token;
                if (one && !is_v) tables.weights_of(p, wa, wb);
            } else {
                token -= range.x - done;
            }
            done = range.x;
            fill += me.chunk;
        }
        // A step: a row of every group.
        const bool in = k < mine && one;
        ring.wait();
        F2 x[4], y[4];
        Eight<T>(ring, stage, 0).open(x);
        Eight<T>(ring, stage, kVecs).open(y);
        issue(k + S - 1, refilled);
        ring.commit();
        refilled = stage;
        stage = Rows::after(stage);
        if (!is_v) {
            F2 sum = x[0] * x[0];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i) sum = fma2(x[i], x[i], sum);
                sum = fma2(y[i], y[i], sum);
            }
            const float inv = inverse_root<kFine>(row_sum<L>(sum_f2(sum)) * inv_dim + a.eps);
            const F2 both = f2(inv, inv);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = x[i] * (wa[i] * both);
                y[i] = y[i] * (wb[i] * both);
            }
            if (p < l.pairs && in) {
                F2 co[4], si[4];
                tables.turns_of(token, p, co, si);
                turn16<false>(x, y, co, si, a.interleaved);
            }
        }
        if (is_q || !CACHE) {
            if (in) {
                T* y_row = reinterpret_cast<T*>(const_cast<char*>(to.at));
                Eight<T>::store(y_row, x);
                if (two) Eight<T>::store(y_row + apart, y);
            }
        } else if constexpr (CACHE) {
            const Place at = s_place[in ? token : 0];
            const bool put = in && at.at >= 0;
            store_cached<BITS, T>(c, at, is_v, put ? to.head : 0, l, p, put, x, y);
            if (put && !is_v && p == 0 && c.weight) c.weight[at.row + (int64_t)to.head * c.page_size] = 0.0f;
        }
        token += me.step_tokens + (to.next(me.heads, me.step_heads) ? 1 : 0);
    }
    ring.wait_all();
}

// ---- backward ----

// A CTA has consecutive rows of q or of k, and leaves its share of the weight's
// gradient in `parts`, head_dim numbers: which rows are whose, and so the order of
// all sums, is fixed.
template <typename T, int L>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 2 : 4) k_qk_rope_back(QkRope a, Layout l, Jobs jobs, int most_tokens, float inv_dim, float* parts) {
    extern __shared__ float4 s_tables[];
    constexpr int kVecs = Eight<T>::kVecs, S = kStages<0>;
    const Tables<L> tables(s_tables, l);
    using Rows = Ring<4 * kVecs, S>;
    const Rows ring(tables.end(most_tokens));
    const int tid = threadIdx.x, p = tid % L, groups = blockDim.x / L, lanes = (l.vecs + 1) / 2, first = l.first(p), second = l.second(p);
    const Share me(a, jobs, tid / L, groups);
    const QkRows& of = me.kind == 0 ? a.q : a.k;
    const bool one = p < lanes, two = one && second < l.vecs;
    const int one_bytes = one ? 16 : 0, two_bytes = two ? 16 : 0, apart = two ? (second - first) * 8 : 0;
    auto walk = [&](const char* base, int64_t token_stride, int64_t head_stride) {
        return Walk(base, token_stride, head_stride, sizeof(T), me.t0 + me.token, me.head, me.heads, me.step_tokens, me.step_heads, one ? first * 8 : 0);
    };
    Walk from = walk(of.x, of.token_stride, of.head_stride), grad = walk(of.g, of.g_token_stride, of.g_head_stride), to = walk(of.y, of.y_token_stride, of.y_head_stride);
    const int mine = me.last ? me.steps : me.steps - 1;  // rows of this group
    auto issue = [&](int k, uint32_t stage) {
        if (k < mine) {
            const T *x = reinterpret_cast<const T*>(from.at), *g = reinterpret_cast<const T*>(grad.at);
            Eight<T>::copy(ring, stage, 0, x, one_bytes);
            Eight<T>::copy(ring, stage, kVecs, x + apart, two_bytes);
            Eight<T>::copy(ring, stage, 2 * kVecs, g, one_bytes);
            Eight<T>::copy(ring, stage, 3 * kVecs, g + apart, two_bytes);
        }
        from.next(me.heads, me.step_heads);
        grad.next(me.heads, me.step_heads);
    };
    begin_dependent();
#pragma unroll
    for (int k = 0; k < S - 1; ++k) {
        issue(k, k * Rows::kStage);
        ring.commit();
    }
    tables.fill_weights(of.weight, a.weight_type, l);
    F2 wa[4] = {}, wb[4] = {}, da[4] = {}, db[4] = {};
    uint32_t stage = 0, refilled = (S - 1) * Rows::kStage;  // at hand, and read in the last step
    int token = 0, done = 0, fill = 0;
    for (int k = 0; k < me.steps; ++k) {
        if (k == fill) {
            const int2 range = me.tokens(jobs, k, groups);
            if (k > 0) __syncthreads();
            tables.template fill_turns<sizeof(T) == 4>(a, me.t0 + range.x, range.y);
            __syncthreads();
            if (k == 0) {
                token = me.token;
                if (one) tables.weights_of(p, wa, wb);
            } else {
                token -= range.x - done;
            }
            done = range.x;
            fill += me.chunk;
        }
        const bool in = k < mine && one;
        ring.wait();
        F2 x[4], y[4], g[4], h[4];
        Eight<T>(ring, stage, 0).open(x);
        Eight<T>(ring, stage, kVecs).open(y);
        Eight<T>(ring, stage, 2 * kVecs).open(g);
        Eight<T>(ring, stage, 3 * kVecs).open(h);
        issue(k + S - 1, refilled);
        ring.commit();
        refilled = stage;
        stage = Rows::after(stage);
        if (p < l.pairs && in) {
            F2 co[4], si[4];
            tables.turns_of(token, p, co, si);
            turn16<true>(g, h, co, si, a.interleaved);
        }
        F2 sum = x[0] * x[0], dot = f2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i) sum = fma2(x[i], x[i], sum);
            sum = fma2(y[i], y[i], sum);
            dot = fma2(g[i] * wa[i], x[i], dot);
            dot = fma2(h[i] * wb[i], y[i], dot);
        }
        const float squares = row_sum<L>(sum_f2(sum)), dots = row_sum<L>(sum_f2(dot));
        if (in) {
            const float inv = inverse_root<sizeof(T) == 4>(squares * inv_dim + a.eps), mean = -inv * inv * dots * inv_dim;
            const F2 both = f2(inv, inv), means = f2(mean, mean);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = x[i] * both;
                y[i] = y[i] * both;
                da[i] = fma2(g[i], x[i], da[i]);
                db[i] = fma2(h[i], y[i], db[i]);
                x[i] = fma2(x[i], means, (g[i] * wa[i]) * both);
                y[i] = fma2(y[i], means, (h[i] * wb[i]) * both);
            }
            T* y_row = reinterpret_cast<T*>(const_cast<char*>(to.at));
            Eight<T>::store(y_row, x);
            if (two) Eight<T>::store(y_row + apart, y);
        }
        token += me.step_tokens + (to.next(me.heads, me.step_heads) ? 1 : 0);
    }
    ring.wait_all();
    // the CTA's groups, added up in their order
    float* s_sums = reinterpret_cast<float*>(s_tables);  // groups x lanes x 16
    __syncthreads();
    if (one) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = open_f2(da[i]), y = open_f2(db[i]);
            float* at = s_sums + (tid / L * lanes + p) * 16 + 2 * i;
            at[0] = x.x;
            at[1] = x.y;
            at[8] = y.x;
            at[9] = y.y;
        }
    }
    __syncthreads();
    for (int i = tid; i < lanes * 16; i += blockDim.x) {
        const int lane = i / 16, vec = i % 16 < 8 ? l.first(lane) : l.second(lane);
        float x = 0.0f;
        for (int g = 0; g < groups; ++g) x += s_sums[g * lanes * 16 + i];
        if (vec < l.vecs) parts[(int64_t)blockIdx.x * l.vecs * 8 + vec * 8 + i % 8] = x;
    }
}

// The CTAs' parts of 32 columns of (dq_weight, dk_weight), 32 threads a column.
__global__ void __launch_bounds__(1024) k_qk_rope_weights(const float* parts, int q_ctas, int ctas, int dim, float* dq_weight, float* dk_weight) {
    __shared__ float s_sum[32][33];
    begin_dependent();
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5, d = col < dim ? col : col - dim;
    const int from = col < dim ? 0 : q_ctas, to = col < dim ? q_ctas : ctas;
    float x = 0.0f;
    if (col < 2 * dim)
#pragma unroll 4
        for (int i = from + part; i < to; i += 32) x += parts[(int64_t)i * dim + d];
    s_sum[part][threadIdx.x & 31] = x;
    __syncthreads();
    x = warp_sum<float>(s_sum[threadIdx.x & 31][part]);
    const int at = blockIdx.x * 32 + part;
    if ((threadIdx.x & 31) == 0 && at < 2 * dim) {
        float* out = at < dim ? dq_weight : dk_weight;
        if (out) out[at < dim ? at : at - dim] = x;
    }
}

Layout layout_of(const QkRope& a) { return Layout{a.head_dim / 8, a.rotary_dim / 16}; }

// Most rows of a group between two fillings of the tables (into an 8-bit cache 83.3 us,
// 84.4 with 16, 85.3 with 8; backward 84.6 with 16, 86.2 with 32).
constexpr int kSteps = 32, kBackSteps = 16;
// CTAs for each that fits the GPU at a time: some tensors' rows take longer than
// others', and waves even that out (16384 x 40 rows 59.2 us with one, 55.8 with two,
// 53.7 four; 20000 x 48 into an 8-bit cache 84.4 with three, 85.9 four, 86.6 six).
constexpr int waves_of(int bits) { return bits ? 3 : 4; }
constexpr int kBackMostPerSm = 4;

// Rows over about `most` CTAs, whole steps each, and the tokens that a filling of the
// tables has at most: groups and two.
Jobs jobs_of(const QkRope& a, int groups, int most_steps, int64_t most, int* grid, int* tokens) {
    const int heads[3] = {a.q.heads, a.k.heads, a.v.heads};
    Jobs jobs;
    *grid = *tokens = 0;
    for (int i = 0; i < 3; ++i) {
        const int64_t all = a.tokens * heads[i], share = std::max<int64_t>(1, most * heads[i] / (heads[0] + heads[1] + heads[2]));
        const int64_t steps = std::min<int64_t>(std::max<int64_t>(1, (all + share * groups - 1) / (share * groups)), 1 << 20), rows = steps * groups;
        jobs.steps[i] = (int)steps;
        jobs.chunk[i] = (int)std::min<int64_t>(steps, std::max(1, std::min(most_steps, heads[i])));
        jobs.ctas[i] = (int)((all + rows - 1) / rows);
        jobs.by_heads[i] = FastDiv(std::max(1, heads[i]));
        *grid += jobs.ctas[i];
        if (all > 0) *tokens = std::max(*tokens, (jobs.chunk[i] * groups + heads[i] - 2) / heads[i] + 1);
    }
    return jobs;
}

template <typename F> cudaError_t for_lanes(int lanes, F&& f) {
    if (lanes <= 2) return f(std::integral_constant<int, 2>());
    if (lanes <= 4) return f(std::integral_constant<int, 4>());
    if (lanes <= 8) return f(std::integral_constant<int, 8>());
    return f(std::integral_constant<int, 16>());
}
template <typename F> cudaError_t for_type(KvElem type, F&& f) {
    if (type == KvElem::F32) return f(float());
    if (type == KvElem::BF16) return f(__nv_bfloat16());
    return f(__half());
}

template <typename T, int L, int BITS>
cudaError_t run(const QkRope& a, const KvPages& c, const int64_t* slots, int sms, uint32_t* status, cudaStream_t s) {
    const Layout l = layout_of(a);
    auto* kern = k_qk_rope<T, L, BITS>;
    using Rows = Ring<2 * Eight<T>::kVecs, kStages<BITS>>;
    KernelSetup su;
    constexpr int groups = kThreads / L;
    const cudaError_t e = kernel_setup(reinterpret_cast<const void*>(kern), kThreads, Tables<L>::bytes(groups + 2) + Rows::bytes(kThreads), &su);
    if (e != cudaSuccess) return e;
    int grid = 0, tokens = 0;
    const Jobs jobs = jobs_of(a, groups, kSteps, (int64_t)sms * su.blocks_per_sm * waves_of(BITS), &grid, &tokens);
    return launch_dependent(kern, (size_t)grid, kThreads, Tables<L>::bytes(tokens) + Rows::bytes(kThreads), 1, s, a, l, jobs, tokens, 1.0f / a.head_dim, c, slots,
                            FastDiv(BITS ? c.page_size : 1), status);
}

template <typename T, int L> cudaError_t run_back(const QkRope& a, float* dq_weight, float* dk_weight, float* parts, int sms, cudaStream_t s) {
    const Layout l = layout_of(a);
    auto* kern = k_qk_rope_back<T, L>;
    const int lanes = (l.vecs + 1) / 2, groups = kThreads / L;
    using Rows = Ring<4 * Eight<T>::kVecs, kStages<0>>;
    KernelSetup su;
    cudaError_t e = kernel_setup(reinterpret_cast<const void*>(kern), kThreads, Tables<L>::bytes(kThreads / L + 2) + Rows::bytes(kThreads), &su);
    if (e != cudaSuccess) return e;
    int grid = 0, tokens = 0;
    const Jobs jobs = jobs_of(a, groups, kBackSteps, (int64_t)sms * std::min(su.blocks_per_sm, kBackMostPerSm), &grid, &tokens);
    if (grid > sms * kBackMostPerSm + 2) return cudaErrorInvalidValue;  // more rows than memory can hold
    const size_t smem = std::max(Tables<L>::bytes(tokens) + Rows::bytes(kThreads), (size_t)groups * lanes * 16 * 4);
    e = launch_dependent(kern, grid, kThreads, smem, 1, s, a, l, jobs, tokens, 1.0f / a.head_dim, parts);
    if (e != cudaSuccess) return e;
    return launch_dependent(k_qk_rope_weights, (2 * a.head_dim + 31) / 32, 1024, 0, 1, s, static_cast<const float*>(parts), jobs.ctas[0], grid, a.head_dim, dq_weight, dk_weight);
}

}  // namespace

cudaError_t launch_qk_rope(const QkRope& a, int sms, cudaStream_t s) {
    return for_type(a.type, [&](auto t) {
        return for_lanes((a.head_dim / 8 + 1) / 2, [&](auto lanes) { return run<decltype(t), decltype(lanes)::value, 0>(a, KvPages{}, nullptr, sms, nullptr, s); });
    });
}

cudaError_t launch_kv_append_rope(const KvPages& c, const int64_t* slots, const QkRope& a, int sms, uint32_t* status, cudaStream_t s) {
    auto go = [&](auto t) {
        return for_lanes((a.head_dim / 8 + 1) / 2, [&](auto lanes) {
            constexpr int L = decltype(lanes)::value;
            using T = decltype(t);
            if (c.type == KvElem::E2M1) return run<T, L, 4>(a, c, slots, sms, status, s);
            if (c.type == KvElem::E4M3) return run<T, L, 8>(a, c, slots, sms, status, s);
            return run<T, L, 16>(a, c, slots, sms, status, s);
        });
    };
    return a.type == KvElem::BF16 ? go(__nv_bfloat16()) : go(__half());
}

size_t qk_rope_scratch(const QkRope& a, int sms) { return ((size_t)sms * kBackMostPerSm + 2) * a.head_dim * 4; }

cudaError_t launch_qk_rope_backward(const QkRope& a, float* dq_weight, float* dk_weight, float* scratch, int sms, cudaStream_t s) {
    return for_type(a.type, [&](auto t) {
        return for_lanes((a.head_dim / 8 + 1) / 2, [&](auto lanes) { return run_back<decltype(t), decltype(lanes)::value>(a, dq_weight, dk_weight, scratch, sms, s); });
    });
}

}  // namespace ss
