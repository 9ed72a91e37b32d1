// qk_rope.cu -- norms of query and key rows with the rotation by their positions
// (streamscan.h, ss_qk_norm_rope), the gradients (ss_qk_norm_rope_backward), and
// the form that writes keys and values into a paged cache (ss_kv_append_rope).
//
// Mathematics.  Of a head's row x, r = 1 / sqrt(mean x^2 + eps), u = r w x, and y =
// R u, where R turns pairs of u by the position's angles.  Backward, with h = R^T
// g: dw = sum r x h over all rows, and dx = r (w h - x r^2 mean(w h x)).  An angle
// is a fraction of a turn: position times frequency modulo 1, which 64-bit integers
// multiply exactly with the frequency in units of 2^-64 turns, however far the
// position; sine and cosine of what is left are those of CUDA's sincospi.
//
// What bounds it.  Memory: every row is read once and written once (backward:
// two and one), for about 10 operations an element.  So rows stay in registers:
// L lanes share a row, each with two 16-byte vectors whose elements are each
// other's partners in the rotation, so that it needs no exchange, and the norm
// log2 L shuffles.  A CTA takes all heads of a few tokens, whose sines and cosines
// it computes once, in shared memory, or a part of the heads where tokens are few.
#include <algorithm>

#include "kv_quant.cuh"

namespace ss {

namespace {

constexpr int kMostThreads = 256;
// Rows of a ring: those on their way, and the one at hand.
template <typename T> constexpr int kStages = sizeof(T) == 4 ? 3 : 4;

__device__ __forceinline__ uint32_t pack_pair(__nv_bfloat16, float x, float y) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_pair(__half, float x, float y) {
    const __half2 v = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Eight elements as they lie in memory, and as fp32.
template <typename T> struct Eight {
    uint4 v[sizeof(T) / 2];
    static constexpr int kVecs = sizeof(T) / 2;
    // The copies of eight elements to vectors v and on of a ring's stage (zeros where
    // there are none), and they from there.
    template <typename R> static __device__ __forceinline__ void copy(const R& ring, int stage, int v, const T* p, bool in) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) ring.copy(stage, v + i, reinterpret_cast<const uint4*>(p) + i, in);
    }
    template <typename R> __device__ __forceinline__ Eight(const R& ring, int stage, int at) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i] = ring.get(stage, at + i);
    }
    __device__ __forceinline__ void open(float (&x)[8]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x[4 * i] = __uint_as_float(v[i].x);
                x[4 * i + 1] = __uint_as_float(v[i].y);
                x[4 * i + 2] = __uint_as_float(v[i].z);
                x[4 * i + 3] = __uint_as_float(v[i].w);
            }
        } else {
            const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 a = open_pair<T>(w[i]);
                x[2 * i] = a.x;
                x[2 * i + 1] = a.y;
            }
        }
    }
    static __device__ __forceinline__ void store(T* p, const float (&x)[8]) {
        if constexpr (sizeof(T) == 4) {
            stg_vec(p, make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])));
            stg_vec(p + 4, make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7])));
        } else {
            stg_vec(p, make_uint4(pack_pair(T(), x[0], x[1]), pack_pair(T(), x[2], x[3]), pack_pair(T(), x[4], x[5]), pack_pair(T(), x[6], x[7])));
        }
    }
};

// A lane's own vectors of the rows to come, in shared memory: only the thread that
// copied them reads them, so nothing but its own copies is waited for.  NV vectors
// of 16 bytes a row, S rows.
template <int NV, int S> struct Ring {
    uint32_t base, step;
    __device__ __forceinline__ Ring(void* smem) : base((uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * 16), step(blockDim.x * 16) {}
    static size_t bytes(int threads) { return (size_t)NV * S * threads * 16; }
    __device__ __forceinline__ void copy(int stage, int v, const void* from, bool in) const {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(base + (stage * NV + v) * step), "l"(from), "r"(in ? 16 : 0) : "memory");
    }
    static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    static __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory"); }
    static __device__ __forceinline__ void wait_all() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
    __device__ __forceinline__ uint4 get(int stage, int v) const {
        uint4 x;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(base + (stage * NV + v) * step) : "memory");
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

// How the work is cut: a CTA has `tokens` tokens and `heads` heads of them.
struct Cut {
    int tokens, heads, splits;
    FastDiv by_heads;
};

// Shared memory: cosines and sines of the CTA's tokens, and the weights of q and k,
// each in four planes of float4: plane j of lane p has a lane's numbers 4 j and on.
struct Tables {
    float4 *turn, *weight;
    int pairs, lanes;
    __device__ __forceinline__ Tables(void* smem, const Layout& l, int tokens) : pairs(l.pairs), lanes((l.vecs + 1) / 2) {
        turn = static_cast<float4*>(smem);
        weight = turn + (size_t)tokens * 4 * pairs;
    }
    __device__ __forceinline__ void* end() const { return weight + 8 * lanes; }
    static size_t bytes(int vecs, int pairs, int tokens) { return ((size_t)tokens * 4 * pairs + 8 * ((vecs + 1) / 2)) * 16; }
    __device__ __forceinline__ void get(const float4* plane, int stride, int p, float (&x)[8], float (&y)[8]) const {
        const float4 v[4] = {plane[p], plane[stride + p], plane[2 * stride + p], plane[3 * stride + p]};
        x[0] = v[0].x; x[1] = v[0].y; x[2] = v[0].z; x[3] = v[0].w; x[4] = v[1].x; x[5] = v[1].y; x[6] = v[1].z; x[7] = v[1].w;
        y[0] = v[2].x; y[1] = v[2].y; y[2] = v[2].z; y[3] = v[2].w; y[4] = v[3].x; y[5] = v[3].y; y[6] = v[3].z; y[7] = v[3].w;
    }
    __device__ __forceinline__ void turns_of(int token, int p, float (&c)[8], float (&s)[8]) const { get(turn + (size_t)token * 4 * pairs, pairs, p, c, s); }
    __device__ __forceinline__ void weights_of(int k, int p, float (&a)[8], float (&b)[8]) const { get(weight + k * 4 * lanes, lanes, p, a, b); }

    __device__ __forceinline__ void fill_turns(const QkRope& a, int64_t t0, int tokens) const {
        const int per = pairs * 8;
        for (int i = threadIdx.x; i < tokens * per; i += blockDim.x) {
            const int t = i / per, m = i - t * per, p = m >> 3, j = m & 7;
            const int f = !a.interleaved ? m : j < 4 ? 4 * p + j : 4 * (p + pairs) + j - 4;
            const long long x = (long long)(a.turns[f] * (unsigned long long)(long long)a.positions[t0 + t]);
            float s, c;
            sincospif((float)x * 0x1p-63f, &s, &c);
            float* to = reinterpret_cast<float*>(turn + (size_t)t * 4 * pairs + (j >> 2) * pairs + p) + (j & 3);
            to[0] = c;
            to[8 * pairs] = s;
        }
    }
    __device__ __forceinline__ void fill_weights(const QkRope& a, const Layout& l) const {
        for (int i = threadIdx.x; i < 32 * lanes; i += blockDim.x) {
            const int k = i / (16 * lanes), m = i - k * 16 * lanes, p = m >> 4, j = m & 15;
            const int vec = j < 8 ? l.first(p) : l.second(p), d = vec * 8 + (j & 7);
            const char* w = k ? a.k.weight : a.q.weight;
            float x = 1.0f;
            if (w && vec < l.vecs) {
                x = a.weight_type == KvElem::F32    ? reinterpret_cast<const float*>(w)[d]
                    : a.weight_type == KvElem::BF16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(w)[d])
                                                    : __half2float(reinterpret_cast<const __half*>(w)[d]);
            }
            reinterpret_cast<float*>(weight + k * 4 * lanes + (j >> 2) * lanes + p)[j & 3] = x;
        }
    }
};

// Turns a lane's 16 elements by their angles, or back (SIGN -1).
template <int SIGN> __device__ __forceinline__ void turn16(float (&a)[8], float (&b)[8], const float (&c)[8], const float (&s)[8], bool interleaved) {
    if (!interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = a[i], y = b[i], z = SIGN * s[i];
            a[i] = x * c[i] - y * z;
            b[i] = y * c[i] + x * z;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = a[2 * i], y = a[2 * i + 1], z = SIGN * s[i];
            a[2 * i] = x * c[i] - y * z;
            a[2 * i + 1] = y * c[i] + x * z;
            const float u = b[2 * i], v = b[2 * i + 1], w = SIGN * s[4 + i];
            b[2 * i] = u * c[4 + i] - v * w;
            b[2 * i + 1] = v * c[4 + i] + u * w;
        }
    }
}

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
__device__ __forceinline__ void store_cached(const KvPages& c, const Place& to, bool is_v, int h, const Layout& l, int p, bool in, const float (&a)[8], const float (&b)[8]) {
    char* pool = is_v ? c.v : c.k;
    const int64_t at = to.at + (int64_t)h * c.head_stride;
    const float* scales = is_v ? c.v_scale : c.k_scale;
    const int first = l.first(p), second = l.second(p);
    if constexpr (BITS == 16) {
        if (!in) return;
        Eight<T>::store(reinterpret_cast<T*>(pool) + at + first * 8, a);
        if (second < l.vecs) Eight<T>::store(reinterpret_cast<T*>(pool) + at + second * 8, b);
    } else if constexpr (BITS == 8) {
        if (!in) return;
        const float s = scales ? scales[h] : 1.0f, inverse = inverse_of(s);
        auto put = [&](int vec, const float (&x)[8]) {
            float y[8];
            quotients(x, s, inverse, y);
            *reinterpret_cast<uint2*>(pool + at + vec * 8) = make_uint2(quant4(y[0], y[1], y[2], y[3]), quant4(y[4], y[5], y[6], y[7]));
        };
        put(first, a);
        if (second < l.vecs) put(second, b);
    } else {
        const float inverse = scales && in ? __frcp_rn(scales[h]) : 1.0f;
        float y[16], ma = 0.0f, mb = 0.0f;
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

// BITS 0: rows go to tensors; else k's and v's go to a cache of so many bits.
template <typename T, int L, int BITS>
__global__ void __launch_bounds__(kMostThreads) k_qk_rope(QkRope a, Layout l, Cut cut, float inv_dim, KvPages c, const int64_t* slots, FastDiv page, uint32_t* status) {
    constexpr bool CACHE = BITS > 0;
    extern __shared__ float4 s_tables[];
    __shared__ Place s_place[CACHE ? kMostThreads : 1];
    const Tables tables(s_tables, l, cut.tokens);
    const int tid = threadIdx.x, p = tid % L, groups = blockDim.x / L;
    const int64_t t0 = (int64_t)(blockIdx.x / cut.splits) * cut.tokens;
    const int h0 = (int)(blockIdx.x % cut.splits) * cut.heads;
    const int tokens = (int)min((int64_t)cut.tokens, a.tokens - t0);
    const int heads = min(cut.heads, a.q.heads + a.k.heads + a.v.heads - h0);
    const int rows = tokens * heads, lanes = (l.vecs + 1) / 2, first = l.first(p), second = l.second(p);
    const int mine = tid / L;  // this lane's rows: mine, mine + groups, ...
    constexpr int kVecs = Eight<T>::kVecs;
    const Ring<2 * kVecs, kStages<T>> ring(tables.end());
    struct Row {
        const QkRows* of;
        int token, head;
        bool in;
    };
    auto row_at = [&](int r) {
        Row x{&a.q, 0, h0, r < rows && p < lanes};
        if (r < rows) {
            x.token = cut.by_heads.div(r);
            x.head = h0 + r - x.token * heads;
        }
        if (x.head >= a.q.heads) {
            x.head -= a.q.heads;
            x.of = &a.k;
            if (CACHE && x.head >= a.k.heads) {
                x.head -= a.k.heads;
                x.of = &a.v;
            }
        }
        return x;
    };
    auto issue = [&](int r, int stage) {
        const Row x = row_at(r);
        const T* from = reinterpret_cast<const T*>(x.of->x) + (t0 + x.token) * x.of->token_stride + x.head * x.of->head_stride;
        Eight<T>::copy(ring, stage, 0, x.in ? from + first * 8 : reinterpret_cast<const T*>(a.positions), x.in);
        const bool both = x.in && second < l.vecs;
        Eight<T>::copy(ring, stage, kVecs, both ? from + second * 8 : reinterpret_cast<const T*>(a.positions), both);
    };
    begin_dependent();
    // the first rows are on their way while the tables are filled
#pragma unroll
    for (int k = 0; k < kStages<T> - 1; ++k) {
        if (mine / (32 / L) * (32 / L) + k * groups < rows) issue(mine + k * groups, k);
        ring.commit();
    }
    tables.fill_turns(a, t0, tokens);
    tables.fill_weights(a, l);
    if constexpr (CACHE) {
        if (tid < tokens) {
            const int64_t slot = slots[t0 + tid], all = c.num_pages * c.page_size;
            Place to{-1, -1};
            if (slot >= 0 && slot < all) {
                const int64_t at = slot < 0x7fffffff ? page.div((int)slot) : slot / c.page_size, s = slot - at * c.page_size;
                to.at = at * c.page_stride + s * c.slot_stride;
                to.row = at * c.kv_heads * c.page_size + s;
            } else if (slot >= all) {
                record_error(status, kErrKvTable, (uint32_t)(t0 + tid));
            }
            s_place[tid] = to;
        }
    }
    __syncthreads();

    int stage = 0;
    for (int r0 = tid / 32 * (32 / L); r0 < rows; r0 += groups) {  // the same for a warp
        const Row row = row_at(r0 + tid % 32 / L);
        ring.wait();
        float x[8], y[8];
        Eight<T>(ring, stage, 0).open(x);
        Eight<T>(ring, stage, kVecs).open(y);
        // the stage read in the last step is filled again
        const int next = r0 + (kStages<T> - 1) * groups;
        if (next < rows) issue(next + tid % 32 / L, stage == 0 ? kStages<T> - 1 : stage - 1);
        ring.commit();
        stage = stage + 1 == kStages<T> ? 0 : stage + 1;

        const bool is_q = row.of == &a.q, is_k = row.of == &a.k, is_v = CACHE && row.of == &a.v;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += x[i] * x[i] + y[i] * y[i];
        sum = row_sum<L>(sum);
        if (row.in && !is_v) {
            const float inv = __frsqrt_rn(sum * inv_dim + a.eps);
            float wa[8], wb[8];
            tables.weights_of(is_k ? 1 : 0, p, wa, wb);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] *= inv * wa[i];
                y[i] *= inv * wb[i];
            }
            if (p < l.pairs) {
                float co[8], si[8];
                tables.turns_of(row.token, p, co, si);
                turn16<1>(x, y, co, si, a.interleaved);
            }
        }
        if constexpr (CACHE) {
            const Place to = s_place[row.token];
            const bool put = row.in && !is_q && to.at >= 0;
            if (!is_q || BITS == 4) store_cached<BITS, T>(c, to, is_v, put ? row.head : 0, l, p, put, x, y);  // 4 bits: lanes exchange largest elements
            if (put && is_k && p == 0 && c.weight) c.weight[to.row + (int64_t)row.head * c.page_size] = 0.0f;
            if (!is_q) continue;
        }
        if (row.in) {
            T* to = reinterpret_cast<T*>(row.of->y) + (t0 + row.token) * row.of->y_token_stride + row.head * row.of->y_head_stride;
            Eight<T>::store(to + first * 8, x);
            if (second < l.vecs) Eight<T>::store(to + second * 8, y);
        }
    }
    ring.wait_all();
}

// ---- backward ----

// A CTA has rows of q or of k alone, tiles of `per` tokens of them, and leaves its
// share of the weight's gradient in `parts`, head_dim numbers; which tiles are
// whose, and so the order of all sums, is fixed.  The first q_ctas CTAs have q's.
template <typename T, int L>
__global__ void __launch_bounds__(kMostThreads) k_qk_rope_back(QkRope a, Layout l, int q_ctas, int per_q, int per_k, FastDiv by_q, FastDiv by_k, float inv_dim, float* parts) {
    extern __shared__ float4 s_tables[];
    const bool is_k = blockIdx.x >= q_ctas;
    const QkRows& of = is_k ? a.k : a.q;
    const FastDiv by_heads = is_k ? by_k : by_q;
    const int per = is_k ? per_k : per_q, cta = is_k ? blockIdx.x - q_ctas : blockIdx.x, ctas = is_k ? gridDim.x - q_ctas : q_ctas;
    const Tables tables(s_tables, l, max(per_q, per_k));
    constexpr int kVecs = Eight<T>::kVecs;
    const Ring<4 * kVecs, kStages<T>> ring(tables.end());
    const int tid = threadIdx.x, p = tid % L, groups = blockDim.x / L, lanes = (l.vecs + 1) / 2, first = l.first(p), second = l.second(p);
    const int64_t tiles = (a.tokens + per - 1) / per;
    begin_dependent();
    // A step is one row of every group; the steps of all tiles are one sequence, so
    // that the ring does not run empty between them.
    struct At {
        int64_t tile;
        int r0;  // of the warp's first row
    };
    auto rows_in = [&](int64_t tile) { return (int)min((int64_t)per, a.tokens - tile * per) * of.heads; };
    const int warp_row = tid / 32 * (32 / L);
    auto settle = [&](At& x) {  // on to the next tile that has rows for this warp
        while (x.tile < tiles && x.r0 >= rows_in(x.tile)) {
            x.tile += ctas;
            x.r0 = warp_row;
        }
    };
    auto issue = [&](const At& at, int stage) {
        const int r = at.r0 + tid % 32 / L;
        const bool in = r < rows_in(at.tile) && p < lanes, both = in && second < l.vecs;
        const int token = in ? by_heads.div(r) : 0, head = in ? r - token * of.heads : 0;
        const int64_t t = at.tile * per + token;
        const T* x = reinterpret_cast<const T*>(of.x) + t * of.token_stride + head * of.head_stride;
        const T* g = reinterpret_cast<const T*>(of.g) + t * of.g_token_stride + head * of.g_head_stride;
        const T* any = reinterpret_cast<const T*>(a.positions);
        Eight<T>::copy(ring, stage, 0, in ? x + first * 8 : any, in);
        Eight<T>::copy(ring, stage, kVecs, both ? x + second * 8 : any, both);
        Eight<T>::copy(ring, stage, 2 * kVecs, in ? g + first * 8 : any, in);
        Eight<T>::copy(ring, stage, 3 * kVecs, both ? g + second * 8 : any, both);
    };
    At ld{cta, warp_row};
#pragma unroll
    for (int k = 0; k < kStages<T> - 1; ++k) {
        settle(ld);
        if (ld.tile < tiles) {
            issue(ld, k);
            ld.r0 += groups;
        }
        ring.commit();
    }
    tables.fill_weights(a, l);
    __syncthreads();
    float wa[8] = {}, wb[8] = {}, da[8] = {}, db[8] = {};
    if (p < lanes) tables.weights_of(is_k ? 1 : 0, p, wa, wb);
    int stage = 0;
    for (int64_t tile = cta; tile < tiles; tile += ctas) {
        const int64_t t0 = tile * per;
        const int tokens = (int)min((int64_t)per, a.tokens - t0), rows = tokens * of.heads;
        __syncthreads();
        tables.fill_turns(a, t0, tokens);
        __syncthreads();
        for (int r0 = warp_row; r0 < rows; r0 += groups) {
            const int r = r0 + tid % 32 / L;
            const bool in = r < rows && p < lanes;
            const int token = in ? by_heads.div(r) : 0, head = in ? r - token * of.heads : 0;
            ring.wait();
            float x[8], y[8], g[8], h[8];
            Eight<T>(ring, stage, 0).open(x);
            Eight<T>(ring, stage, kVecs).open(y);
            Eight<T>(ring, stage, 2 * kVecs).open(g);
            Eight<T>(ring, stage, 3 * kVecs).open(h);
            settle(ld);
            if (ld.tile < tiles) {
                issue(ld, stage == 0 ? kStages<T> - 1 : stage - 1);
                ld.r0 += groups;
            }
            ring.commit();
            stage = stage + 1 == kStages<T> ? 0 : stage + 1;
            if (p < l.pairs) {
                float co[8], si[8];
                tables.turns_of(token, p, co, si);
                turn16<-1>(g, h, co, si, a.interleaved);
            }
            float sum = 0.0f, dot = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sum += x[i] * x[i] + y[i] * y[i];
                dot += g[i] * wa[i] * x[i] + h[i] * wb[i] * y[i];
            }
            sum = row_sum<L>(sum);
            dot = row_sum<L>(dot);
            if (!in) continue;
            const float inv = __frsqrt_rn(sum * inv_dim + a.eps), mean = inv * inv * dot * inv_dim;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                da[i] += g[i] * (x[i] * inv);
                db[i] += h[i] * (y[i] * inv);
                x[i] = inv * (g[i] * wa[i] - x[i] * mean);
                y[i] = inv * (h[i] * wb[i] - y[i] * mean);
            }
            T* to = reinterpret_cast<T*>(of.y) + (t0 + token) * of.y_token_stride + head * of.y_head_stride;
            Eight<T>::store(to + first * 8, x);
            if (second < l.vecs) Eight<T>::store(to + second * 8, y);
        }
    }
    ring.wait_all();
    // the CTA's groups, added up in their order
    float* s_sums = reinterpret_cast<float*>(s_tables);  // groups x lanes x 16
    __syncthreads();
    if (p < lanes) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s_sums[(tid / L * lanes + p) * 16 + i] = da[i];
            s_sums[(tid / L * lanes + p) * 16 + 8 + i] = db[i];
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

constexpr int kBackThreads = 256;
constexpr int kBackMostPerSm = 4;

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
    const int heads = a.q.heads + a.k.heads + a.v.heads;
    Cut cut;
    int threads = 256;
    cut.tokens = std::max(1, std::min(16, 256 / heads));
    cut.splits = 1;
    while (cut.tokens > 1 && (a.tokens + cut.tokens - 1) / cut.tokens < 4 * (int64_t)sms) cut.tokens /= 2;
    if (a.tokens < 2 * (int64_t)sms) {  // few tokens: a part of the heads each
        threads = 128;
        cut.splits = (int)std::min<int64_t>((heads + threads / L - 1) / (threads / L), std::max<int64_t>(1, 2 * sms / a.tokens));
    }
    cut.heads = (heads + cut.splits - 1) / cut.splits;
    cut.splits = (heads + cut.heads - 1) / cut.heads;
    cut.by_heads = FastDiv(cut.heads);
    auto* kern = k_qk_rope<T, L, BITS>;
    const size_t smem = Tables::bytes(l.vecs, l.pairs, cut.tokens) + Ring<2 * Eight<T>::kVecs, kStages<T>>::bytes(threads);
    KernelSetup su;
    const cudaError_t e = kernel_setup(reinterpret_cast<const void*>(kern), kMostThreads, Tables::bytes(32, 16, 16) + Ring<2 * Eight<T>::kVecs, kStages<T>>::bytes(kMostThreads), &su);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, (size_t)((a.tokens + cut.tokens - 1) / cut.tokens) * cut.splits, threads, smem, 1, s, a, l, cut, 1.0f / a.head_dim, c, slots,
                            FastDiv(BITS ? c.page_size : 1), status);
}

template <typename T, int L> cudaError_t run_back(const QkRope& a, float* dq_weight, float* dk_weight, float* parts, int sms, cudaStream_t s) {
    const Layout l = layout_of(a);
    auto* kern = k_qk_rope_back<T, L>;
    const int lanes = (l.vecs + 1) / 2, most_tokens = 16;
    // tiles of about 8 rows a group
    auto tokens_of = [&](int heads) { return std::max(1, std::min(most_tokens, 8 * kBackThreads / L / std::max(1, heads))); };
    const int per_q = tokens_of(a.q.heads), per_k = tokens_of(a.k.heads);
    const size_t ring = Ring<4 * Eight<T>::kVecs, kStages<T>>::bytes(kBackThreads);
    const size_t smem = std::max(Tables::bytes(l.vecs, l.pairs, std::max(per_q, per_k)) + ring, (size_t)kBackThreads / L * lanes * 16 * 4);
    KernelSetup su;
    cudaError_t e = kernel_setup(reinterpret_cast<const void*>(kern), kBackThreads, std::max(Tables::bytes(32, 16, most_tokens) + ring, (size_t)kBackThreads * 64), &su);
    if (e != cudaSuccess) return e;
    // CTAs for q and for k by their rows
    const int64_t most = (int64_t)sms * std::min(su.blocks_per_sm, kBackMostPerSm), heads = a.q.heads + a.k.heads;
    auto ctas_of = [&](int h, int per) { return h == 0 ? 0 : (int)std::max<int64_t>(1, std::min<int64_t>((a.tokens + per - 1) / per, most * h / heads)); };
    const int q_ctas = ctas_of(a.q.heads, per_q), ctas = q_ctas + ctas_of(a.k.heads, per_k);
    e = launch_dependent(kern, ctas, kBackThreads, smem, 1, s, a, l, q_ctas, per_q, per_k, FastDiv(std::max(1, a.q.heads)), FastDiv(std::max(1, a.k.heads)), 1.0f / a.head_dim,
                         parts);
    if (e != cudaSuccess) return e;
    return launch_dependent(k_qk_rope_weights, (2 * a.head_dim + 31) / 32, 1024, 0, 1, s, static_cast<const float*>(parts), q_ctas, ctas, a.head_dim, dq_weight, dk_weight);
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
