// kv_rows.cuh -- one unit of query heads against tiles of 16 or 32 positions:
// the products, the running softmax and the outputs of the attention kernel
// (kv_attend.cu), in two forms.
//
//   Rows16  query heads are the rows of the products: X = Q K^T is two m16n8
//           products per 16 of head_dim and 16 positions, O += P V.  For groups
//           of more than 8 query heads.
//   Rows8   query heads are the columns: X^T = K Q^T is one product for the
//           same, and O^T += V^T P^T, with half the products and half the
//           registers.  P^T changes its lane layout between the two by an 8 x 8
//           transposition in registers.  For groups of up to 8.
//
// Both keep, per query head, the largest X so far, l = sum 2^(X - R) and O,
// with R that maximum less 15 where products are fp16, so that small weights
// stay normal numbers, or plus 24 where they are bf16, so that O stays below
// the largest number whatever the values are.
#pragma once

#include "kv.cuh"

namespace ss {

// Which positions of a sequence are visible, and in which tiles they lie: the
// tiles (of 2^shift positions; a page may end inside one) of the first
// tokens, then those of the window.
struct Tiles {
    int len, start, sinks, nsink, first, count;
    __device__ __forceinline__ Tiles(int len_, int window, int sinks_, int shift) : len(len_), start(0), sinks(sinks_), nsink(0), first(0) {
        const int up = (1 << shift) - 1;
        if (window > 0 && window < len) {
            start = len - window;
            first = start >> shift;
            nsink = min((min(sinks, start) + up) >> shift, first);
        }
        count = nsink + ((len + up) >> shift) - first;
    }
    __device__ __forceinline__ int tile(int j) const { return j < nsink ? j : first + j - nsink; }
    __device__ __forceinline__ bool visible(int p) const { return p < len && (p < sinks || p >= start); }
    // Whether all of p .. p + n - 1 are visible.
    __device__ __forceinline__ bool whole(int p, int n) const { return p + n <= len && (p + n <= sinks || p >= start); }
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What sums shrink by when their largest X grows.  Not below 2^-126: an infinite
// sum stays infinite, however far its scores lie below the others.  (A sum whose
// largest X is -inf is 0, or NaN where it met an infinite value, whatever it is
// multiplied by.)
__device__ __forceinline__ float shrink(float from, float to) { return fmaxf(exp2_fast(from - to), 0x1p-126f); }

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// An 8 x 8 matrix of 16-bit values held two to a lane (lane 4 i + j: row i,
// columns 2 j and 2 j + 1), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <typename T> __device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <> __device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <> __device__ __forceinline__ void mma16816<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename T> struct Pair;
template <> struct Pair<__nv_bfloat16> {
    using type = __nv_bfloat162;
    static __device__ __forceinline__ type pack(float x, float y) { return __floats2bfloat162_rn(x, y); }
    static __device__ __forceinline__ float2 open(type v) { return __bfloat1622float2(v); }
};
template <> struct Pair<__half> {
    using type = __half2;
    static __device__ __forceinline__ type pack(float x, float y) { return __floats2half2_rn(x, y); }
    static __device__ __forceinline__ float2 open(type v) { return __half22float2(v); }
};
template <typename T> __device__ __forceinline__ uint32_t pack2(float x, float y) {
    const typename Pair<T>::type v = Pair<T>::pack(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename T> __device__ __forceinline__ float2 open2(uint32_t u) {
    return Pair<T>::open(*reinterpret_cast<const typename Pair<T>::type*>(&u));
}

// The larger ones of two pairs of 16-bit numbers; NaN stays.
template <typename T> __device__ __forceinline__ uint32_t max2(uint32_t x, uint32_t y) {
    uint32_t z;
    if constexpr (std::is_same<T, __half>::value)
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(z) : "r"(x), "r"(y));
    else
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(z) : "r"(x), "r"(y));
    return z;
}
// Two numbers as 16-bit ones, rounded toward zero.
template <typename T> __device__ __forceinline__ uint32_t trunc2(float x, float y) {
    uint32_t r;
    if constexpr (std::is_same<T, __half>::value)
        asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
    else
        asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
    return r;
}

// Weights (x, y) >= 0 as two 16-bit terms, of which the second has what the
// first leaves out.  POSITIVE: the first is truncated, so that the second is not
// negative, and both are kept at 2^-24 (fp16) or 2^-126 (bf16) and above: an
// infinite value that they multiply stays infinite instead of becoming inf - inf
// or 0 inf (0.2 % of the long ragged batch's time, 0.2 us of a call of 517
// positions).  That adds at most 2^-38 of the row's largest weight in fp16, 2^-101
// in bf16; scores of -inf get their 0 back (drop2).
template <typename T, bool POSITIVE> __device__ __forceinline__ void split2(float x, float y, uint32_t& high, uint32_t& rest) {
    constexpr uint32_t kLeast = std::is_same<T, __half>::value ? 0x00010001u : 0x00800080u;
    high = POSITIVE ? max2<T>(trunc2<T>(x, y), kLeast) : pack2<T>(x, y);
    const float2 h = open2<T>(high);
    rest = pack2<T>(x - h.x, y - h.y);
    if constexpr (POSITIVE) rest = max2<T>(rest, kLeast);
}
// Makes 0 of both terms of the weights whose scores x and y are -inf.
__device__ __forceinline__ void drop2(float x, float y, uint32_t& high, uint32_t& rest) {
    const uint32_t stay = (x == -INFINITY ? 0u : 0xffffu) | (y == -INFINITY ? 0u : 0xffff0000u);
    high &= stay;
    rest &= stay;
}

// Two e4m3 bytes as two fp16 (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t lo16) {
    uint32_t r;
    asm("{.reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t;}" : "=r"(r) : "r"(lo16));
    return r;
}

// A word of 8-bit values of each of two positions as four pairs of fp16, a pair
// per dimension.
__device__ __forceinline__ void pairs4(uint32_t w0, uint32_t w1, uint32_t (&f)[4]) {
    const uint32_t a = __byte_perm(w0, w1, 0x5140), b = __byte_perm(w0, w1, 0x7362);
    f[0] = e4m3x2_f16x2(a);
    f[1] = e4m3x2_f16x2(a >> 16);
    f[2] = e4m3x2_f16x2(b);
    f[3] = e4m3x2_f16x2(b >> 16);
}

// Where 16-byte vector `v` of row `row` of a tile lies within that row.  The
// exclusive-ors spread the addresses that one shared-memory access of a
// quarter warp touches over all banks: 16-bit tiles are read by ldmatrix (8
// rows of one vector), 8-bit keys by lanes (row g, vector t * DP / 64 + i) and
// 8-bit values by lanes (rows 2 t and on, vector g * DP / 128 + i).
template <bool FP8, int DP> __device__ __forceinline__ int k_vec(int row, int v) {
    if (!FP8) return v ^ (row & 7);
    if (DP == 64) return v;
    if (DP == 128) return v ^ (row & 1);
    return v ^ ((v >> 3) & 1) ^ ((row & 1) << 1);
}
template <bool FP8, int DP> __device__ __forceinline__ int v_vec(int row, int v) {
    if (!FP8) return v ^ (row & 7);
    if (DP == 64) return v ^ ((row >> 1) & 3);
    if (DP == 128) return v ^ (((row >> 1) & 3) << 1);
    return v ^ ((row >> 1) & 1) ^ (((row >> 2) & 1) << 2);
}


// What a unit's outputs need to know: which sequence and heads it is.
struct Unit {
    int b, head, row0, group;  // sequence, key-value head, first query head within the group of `group`
};

// The largest finite |q| of a row as a power of two that brings it to [2^7,
// 2^8), and the scale that undoes it: bf16 queries enter fp16 products this
// way (what falls below 2^-24 of the row's largest element is lost against
// sums that are rounded at 2^-24 themselves).
__device__ __forceinline__ void fit_f16(float most, float& factor, float& undo) {
    const int e = max((int)(__float_as_uint(most) >> 23) - 127, -118);
    factor = __uint_as_float((uint32_t)(127 + 7 - e) << 23);
    undo = __uint_as_float((uint32_t)(127 - 7 + e) << 23);
}
template <typename QT> __device__ __forceinline__ float finite_abs2(uint32_t w) {
    const float2 u = open2<QT>(w);
    return fmaxf(isfinite(u.x) ? fabsf(u.x) : 0.0f, isfinite(u.y) ? fabsf(u.y) : 0.0f);
}
template <typename QT> __device__ __forceinline__ uint32_t scaled_f16x2(uint32_t w, float factor) {
    const float2 u = open2<QT>(w);
    return pack2<__half>(u.x * factor, u.y * factor);
}

// What both forms share.  8-bit caches multiply in fp16, which holds every
// e4m3 value.  P enters the product with V as two 16-bit terms (kTwo), good to
// 2^-16 of itself in bf16 and 2^-22 in fp16, below the rounding of out (2^-8,
// 2^-11): 0.28 % of the ragged bf16 batch's outputs round to the other neighbour,
// 0.13 % of an 8-bit cache's, against 0.07 and 0.12 % with fp32 weights.  One fp16
// term, 2^-11, is left to bf16 outputs of 8-bit caches where two cost much (16
// query heads a key-value head 84 / 95 us, head_dim 64 71 / 77): 7 % of them
// round to the other neighbour, with the same error against the formula,
// 1.65e-3.  (At head_dim 128 two terms cost nothing of 100 us, at 256 123 / 124.5,
// at 80 60.7 / 64.4.)
//
// O is added up in the products' accumulators, which cut what falls below 24
// bits instead of rounding it: an error of one sign, up to 2^-24 a product.  So
// after kChain tiles, 128 products in a row (2^-17), O is set aside in memory, where
// fp32 additions go on (put_aside): rows of 131,072 equal values in fp16 came
// out 0.06 % low without that.  It takes 0 to 1 % of the time, 715 against 710 us
// of a 4.4 GB batch, 211 against 199 where 128 query heads share one key-value
// head; fp32 additions of every tile take more, 106.9 against 100.5 us over an
// 8-bit cache.
template <typename QT, bool FP8, int DP, int T, int HEADS> struct RowsBase {
    using MT = typename std::conditional<FP8, __half, QT>::type;
    static constexpr float kShift = std::is_same<MT, __half>::value ? 15.0f : -24.0f;
    static constexpr int kHeads = HEADS;
    static constexpr bool kTwo = !FP8 || std::is_same<QT, __half>::value || (HEADS == 8 && DP > 64);
    static constexpr bool kFit = FP8 && !std::is_same<QT, __half>::value;
    static constexpr int kChain = 128 / (T / 16 * (kTwo ? 2 : 1));
    static constexpr int kBytes = FP8 ? 1 : 2, kRowBytes = DP * kBytes, kKS = DP / 16;

    // Four elements of a query row for an 8-bit cache.  The products' index runs
    // over head_dim in another order there: step ks of lane q4 holds the four
    // dimensions q4 * DP / 4 + 4 ks and on, so that a lane's keys are
    // consecutive bytes.
    static __device__ __forceinline__ uint2 query4(const QT* p, bool in, int dim, int q4, int ks) {
        const int d = q4 * (DP / 4) + 4 * ks;
        return in && d < dim ? *reinterpret_cast<const uint2*>(p + d) : make_uint2(0u, 0u);
    }
    static __device__ __forceinline__ uint32_t query2(const QT* p, bool in, int dim, int d) {
        return in && d < dim ? *reinterpret_cast<const uint32_t*>(p + d) : 0u;
    }
    static __device__ __forceinline__ float row_scale(const KvPages& c, const KvAttention& a, int head) {
        return a.scale * 1.4426950408889634f * (FP8 && c.k_scale ? c.k_scale[head] : 1.0f);
    }
    // The values of 8-bit row `row` that this lane needs from vector v on: DP /
    // 8 bytes a row, in vectors of 16 (8 at DP = 64).
    static __device__ __forceinline__ uint4 values(uint32_t vt, int row, int g, int v) {
        if constexpr (DP == 64) {
            const uint2 w = lds64(vt + row * kRowBytes + v_vec<FP8, DP>(row, g >> 1) * 16 + (g & 1) * 8);
            return make_uint4(w.x, w.y, 0u, 0u);
        } else {
            return lds128(vt + row * kRowBytes + v_vec<FP8, DP>(row, g * (DP / 128) + v) * 16);
        }
    }
    static constexpr int kValueVecs = DP == 64 ? 1 : DP / 128, kValueWords = DP == 64 ? 2 : 4;
};

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

template <typename QT, bool FP8, int DP, int T> struct Rows16 : RowsBase<QT, FP8, DP, T, 16> {
    using Base = RowsBase<QT, FP8, DP, T, 16>;
    using MT = typename Base::MT;
    using Base::kKS; using Base::kRowBytes; using Base::kShift; using Base::kTwo;
    using Query = QT;
    static constexpr int kNT = DP / 8, kPT = T / 8, kVectors = kNT;  // of four O's a lane
    static constexpr bool kQShared = DP == 256;  // Q's fragments in shared memory: registers are short
    static constexpr int kQBytes = kQShared ? kKS * 32 * 16 : 0;

    uint32_t qf[kQShared ? 1 : kKS][4];
    float o[kNT][4];
    float m0, m1, l0, l1;  // largest X of heads g and g + 8, and this lane's share of l
    float sl0, sl1;        // X per unit of q . k

    __device__ __forceinline__ void open(const KvPages& c, const KvAttention& a, const Unit& u, uint32_t qs, int lane) {
        const int g = lane >> 2, q4 = lane & 3, ra = u.row0 + g, rb = ra + 8;
        const bool ina = ra < u.group, inb = rb < u.group;
        const QT* q = static_cast<const QT*>(a.q) + (int64_t)u.b * a.q_seq_stride;
        const QT* pa = q + (int64_t)(u.head * u.group + ra) * a.q_head_stride;
        const QT* pb = q + (int64_t)(u.head * u.group + rb) * a.q_head_stride;
        sl0 = sl1 = Base::row_scale(c, a, u.head);
        float fa = 1.0f, fb = 1.0f;
        if constexpr (Base::kFit) {
            float ma = 0.0f, mb = 0.0f, ua, ub;
            for (int ks = 0; ks < kKS; ++ks) {
                const uint2 x = Base::query4(pa, ina, c.head_dim, q4, ks), y = Base::query4(pb, inb, c.head_dim, q4, ks);
                ma = fmaxf(ma, fmaxf(finite_abs2<QT>(x.x), finite_abs2<QT>(x.y)));
                mb = fmaxf(mb, fmaxf(finite_abs2<QT>(y.x), finite_abs2<QT>(y.y)));
            }
            for (int i = 1; i < 4; i <<= 1) {
                ma = fmaxf(ma, __shfl_xor_sync(kFullMask, ma, i));
                mb = fmaxf(mb, __shfl_xor_sync(kFullMask, mb, i));
            }
            fit_f16(ma, fa, ua);
            fit_f16(mb, fb, ub);
            sl0 *= ua;
            sl1 *= ub;
        }
#pragma unroll
        for (int ks = 0; ks < kKS; ++ks) {
            uint32_t f[4];
            if constexpr (FP8) {
                const uint2 x = Base::query4(pa, ina, c.head_dim, q4, ks), y = Base::query4(pb, inb, c.head_dim, q4, ks);
                f[0] = x.x; f[1] = y.x; f[2] = x.y; f[3] = y.y;
                if constexpr (Base::kFit) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[i] = scaled_f16x2<QT>(f[i], i & 1 ? fb : fa);
                }
            } else {
                const int d = ks * 16 + 2 * q4;
                f[0] = Base::query2(pa, ina, c.head_dim, d);
                f[1] = Base::query2(pb, inb, c.head_dim, d);
                f[2] = Base::query2(pa, ina, c.head_dim, d + 8);
                f[3] = Base::query2(pb, inb, c.head_dim, d + 8);
            }
            if constexpr (kQShared) {
                sts128(qs + (ks * 32 + lane) * 16, make_uint4(f[0], f[1], f[2], f[3]));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) qf[ks][i] = f[i];
            }
        }
        m0 = m1 = -INFINITY;
        l0 = l1 = 0.0f;
#pragma unroll
        for (int i = 0; i < kNT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;
    }

    __device__ __forceinline__ void query(uint32_t qs, int ks, int lane, uint32_t (&f)[4]) const {
        if constexpr (kQShared) {
            const uint4 x = lds128(qs + (ks * 32 + lane) * 16);
            f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = qf[ks][i];
        }
    }

    // One tile of keys at kt and values at vt, positions p0 and on; `scores`
    // (or null) receives X, a row of T for each of the unit's heads.
    __device__ __forceinline__ void tile(uint32_t kt, uint32_t vt, uint32_t qs, const Tiles& t, int p0, float* scores, const Unit& u, int lane) {
        const int g = lane >> 2, q4 = lane & 3;
        float x[kPT][4] = {};
        if constexpr (!FP8) {
            const int row = (lane >> 4) * 8 + (lane & 7);
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks) {
                uint32_t f[4];
                query(qs, ks, lane, f);
#pragma unroll
                for (int h = 0; h < kPT / 2; ++h) {
                    uint32_t kf[4];
                    ldmatrix4(kf, kt + (row + 16 * h) * kRowBytes + k_vec<FP8, DP>(row, 2 * ks + ((lane >> 3) & 1)) * 16);
                    mma16816<MT>(x[2 * h], f, kf[0], kf[1]);
                    mma16816<MT>(x[2 * h + 1], f, kf[2], kf[3]);
                }
            }
        } else {
#pragma unroll
            for (int v = 0; v < DP / 64; ++v) {
                uint4 kw[kPT];
#pragma unroll
                for (int pt = 0; pt < kPT; ++pt) kw[pt] = lds128(kt + (g + 8 * pt) * kRowBytes + k_vec<FP8, DP>(g, q4 * (DP / 64) + v) * 16);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t f[4];
                    query(qs, v * 4 + i, lane, f);
#pragma unroll
                    for (int pt = 0; pt < kPT; ++pt) {
                        const uint32_t w = word(kw[pt], i);
                        mma16816<MT>(x[pt], f, e4m3x2_f16x2(w), e4m3x2_f16x2(w >> 16));
                    }
                }
            }
        }
        const bool whole = t.whole(p0, T);
#pragma unroll
        for (int pt = 0; pt < kPT; ++pt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const bool see = whole || t.visible(p0 + 2 * q4 + pt * 8 + e);
                x[pt][e] = see ? x[pt][e] * sl0 : -INFINITY;
                x[pt][2 + e] = see ? x[pt][2 + e] * sl1 : -INFINITY;
            }
        if (scores) {
#pragma unroll
            for (int pt = 0; pt < kPT; ++pt) {
                if (u.row0 + g < u.group) *reinterpret_cast<float2*>(scores + g * T + 2 * q4 + pt * 8) = make_float2(x[pt][0], x[pt][1]);
                if (u.row0 + g + 8 < u.group) *reinterpret_cast<float2*>(scores + (g + 8) * T + 2 * q4 + pt * 8) = make_float2(x[pt][2], x[pt][3]);
            }
        }
        float top0 = m0, top1 = m1, low = INFINITY;
#pragma unroll
        for (int pt = 0; pt < kPT; ++pt) {
            top0 = fmaxf(top0, fmaxf(x[pt][0], x[pt][1]));
            top1 = fmaxf(top1, fmaxf(x[pt][2], x[pt][3]));
            low = fminf(low, fminf(fminf(x[pt][0], x[pt][1]), fminf(x[pt][2], x[pt][3])));
        }
        const bool some_inf = !FP8 && __any_sync(kFullMask, low == -INFINITY);
#pragma unroll
        for (int s = 1; s < 4; s <<= 1) {
            top0 = fmaxf(top0, __shfl_xor_sync(kFullMask, top0, s));
            top1 = fmaxf(top1, __shfl_xor_sync(kFullMask, top1, s));
        }
        if (__any_sync(kFullMask, top0 != m0 || top1 != m1)) {
            const float f0 = shrink(m0, top0), f1 = shrink(m1, top1);
            m0 = top0;
            m1 = top1;
            l0 *= f0;
            l1 *= f1;
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
                o[nt][0] *= f0;
                o[nt][1] *= f0;
                o[nt][2] *= f1;
                o[nt][3] *= f1;
            }
        }
        // a row that has seen nothing but -inf keeps reference 0, and P = 0
        const float ref0 = m0 == -INFINITY ? 0.0f : m0 - kShift, ref1 = m1 == -INFINITY ? 0.0f : m1 - kShift;
#pragma unroll
        for (int h = 0; h < kPT / 2; ++h) {  // 16 positions
            uint32_t ph[4], pl[4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float* y = x[2 * h + k];
                const float a0 = exp2_fast(y[0] - ref0), a1 = exp2_fast(y[1] - ref0);
                const float b0 = exp2_fast(y[2] - ref1), b1 = exp2_fast(y[3] - ref1);
                l0 += a0 + a1;
                l1 += b0 + b1;
                if constexpr (kTwo) {
                    split2<MT, !FP8>(a0, a1, ph[k * 2], pl[k * 2]);
                    split2<MT, !FP8>(b0, b1, ph[k * 2 + 1], pl[k * 2 + 1]);
                } else {
                    ph[k * 2] = pack2<MT>(a0, a1);
                    ph[k * 2 + 1] = pack2<MT>(b0, b1);
                }
            }
            if constexpr (!FP8) {
                if (some_inf) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        drop2(x[2 * h + k][0], x[2 * h + k][1], ph[k * 2], pl[k * 2]);
                        drop2(x[2 * h + k][2], x[2 * h + k][3], ph[k * 2 + 1], pl[k * 2 + 1]);
                    }
                }
            }
            const uint32_t vh = vt + 16 * h * kRowBytes;
            if constexpr (!FP8) {
                const int row = ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
                for (int nt = 0; nt < kNT; nt += 2) {
                    uint32_t vf[4];
                    ldmatrix4_t(vf, vh + row * kRowBytes + v_vec<FP8, DP>(row, nt + (lane >> 4)) * 16);
                    mma16816<MT>(o[nt], ph, vf[0], vf[1]);
                    mma16816<MT>(o[nt + 1], ph, vf[2], vf[3]);
                    if constexpr (kTwo) {
                        mma16816<MT>(o[nt], pl, vf[0], vf[1]);
                        mma16816<MT>(o[nt + 1], pl, vf[2], vf[3]);
                    }
                }
            } else {
#pragma unroll
                for (int v = 0; v < Base::kValueVecs; ++v) {
                    uint4 w[4];  // positions 2 q4, 2 q4 + 1, and 8 later
#pragma unroll
                    for (int k = 0; k < 4; ++k) w[k] = Base::values(vh, 2 * q4 + (k & 1) + (k >> 1) * 8, g, v);
#pragma unroll
                    for (int i = 0; i < Base::kValueWords; ++i) {
                        uint32_t lo[4], hi[4];  // column n of product j is dimension n * DP / 8 + j
                        pairs4(word(w[0], i), word(w[1], i), lo);
                        pairs4(word(w[2], i), word(w[3], i), hi);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            mma16816<MT>(o[v * 16 + i * 4 + k], ph, lo[k], hi[k]);
                            if constexpr (kTwo) mma16816<MT>(o[v * 16 + i * 4 + k], pl, lo[k], hi[k]);
                        }
                    }
                }
            }
        }
    }

    // Visits this lane's outputs as (row half, first dimension, two values).
    template <typename F> __device__ __forceinline__ void each_pair(int q4, F&& f) const {
        if constexpr (!FP8) {
#pragma unroll
            for (int i = 0; i < kNT; ++i) {
                f(0, i * 8 + 2 * q4, o[i][0], o[i][1]);
                f(1, i * 8 + 2 * q4, o[i][2], o[i][3]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kNT; i += 2)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    f(0, (2 * q4 + e) * (DP / 8) + i, o[i][e], o[i + 1][e]);
                    f(1, (2 * q4 + e) * (DP / 8) + i, o[i][2 + e], o[i + 1][2 + e]);
                }
        }
    }
    static __device__ __forceinline__ float4 factors(float f0, float f1) { return make_float4(f0, f0, f1, f1); }
    // Adds l up over the lanes that share a head: to be called before store_*.
    __device__ __forceinline__ void gather() {
#pragma unroll
        for (int i = 1; i < 4; i <<= 1) {
            l0 += __shfl_xor_sync(kFullMask, l0, i);
            l1 += __shfl_xor_sync(kFullMask, l1, i);
        }
    }
    // Calls f(head of the unit, reference, l) in one lane for each head.
    template <typename F> __device__ __forceinline__ void each_sum(const Unit& u, int lane, F&& f) const {
        const int g = lane >> 2;
        if ((lane & 3) != 0) return;
        if (u.row0 + g < u.group) f(g, m0 - kShift, l0);
        if (u.row0 + g + 8 < u.group) f(g + 8, m1 - kShift, l1);
    }
    __device__ __forceinline__ void store_out(const KvAttention& a, const Unit& u, float vs, int dim, int lane) const {
        const int g = lane >> 2, q4 = lane & 3;
        const float f[2] = {vs / l0, vs / l1};
        const bool in[2] = {u.row0 + g < u.group, u.row0 + g + 8 < u.group}, some[2] = {l0 != 0.0f, l1 != 0.0f};
        QT* out = static_cast<QT*>(a.out) + (int64_t)u.b * a.out_seq_stride + (int64_t)(u.head * u.group + u.row0 + g) * a.out_head_stride;
        each_pair(q4, [&](int half, int d, float x, float y) {
            if (in[half] && d < dim) *reinterpret_cast<uint32_t*>(out + half * 8 * a.out_head_stride + d) = some[half] ? pack2<QT>(x * f[half], y * f[half]) : 0u;
        });
    }
    __device__ __forceinline__ void store_part(float* part, const Unit& u, int lane) const {
        const int g = lane >> 2, q4 = lane & 3;
        const bool in[2] = {u.row0 + g < u.group, u.row0 + g + 8 < u.group};
        each_pair(q4, [&](int half, int d, float x, float y) {
            if (in[half]) *reinterpret_cast<float2*>(part + (g + 8 * half) * DP + d) = make_float2(x, y);
        });
    }
};

template <typename QT, bool FP8, int DP, int T> struct Rows8 : RowsBase<QT, FP8, DP, T, 8> {
    using Base = RowsBase<QT, FP8, DP, T, 8>;
    using MT = typename Base::MT;
    using Base::kKS; using Base::kRowBytes; using Base::kShift; using Base::kTwo;
    using Query = QT;
    static constexpr int kMT = DP / 16, kHB = T / 16, kVectors = kMT;  // of four O's a lane
    static constexpr int kQBytes = 0;

    uint32_t qf[kKS][2];
    float o[kMT][4];       // 16-bit: dimensions 16 i + g and 8 later; 8-bit: g * DP / 8 + 2 i and 1 later; heads 2 q4, 2 q4 + 1
    float m0, m1, l0, l1;  // of heads 2 q4 and 2 q4 + 1
    float sl0, sl1;

    __device__ __forceinline__ void open(const KvPages& c, const KvAttention& a, const Unit& u, uint32_t, int lane) {
        const int g = lane >> 2, q4 = lane & 3, r = u.row0 + g;
        const bool in = r < u.group;
        const QT* p = static_cast<const QT*>(a.q) + (int64_t)u.b * a.q_seq_stride + (int64_t)(u.head * u.group + r) * a.q_head_stride;
        float sl = Base::row_scale(c, a, u.head), factor = 1.0f;
        if constexpr (Base::kFit) {
            float most = 0.0f, undo;
            for (int ks = 0; ks < kKS; ++ks) {
                const uint2 x = Base::query4(p, in, c.head_dim, q4, ks);
                most = fmaxf(most, fmaxf(finite_abs2<QT>(x.x), finite_abs2<QT>(x.y)));
            }
            for (int i = 1; i < 4; i <<= 1) most = fmaxf(most, __shfl_xor_sync(kFullMask, most, i));
            fit_f16(most, factor, undo);
            sl *= undo;
        }
        sl0 = __shfl_sync(kFullMask, sl, q4 * 8);  // lane 4 h holds head h's
        sl1 = __shfl_sync(kFullMask, sl, q4 * 8 + 4);
#pragma unroll
        for (int ks = 0; ks < kKS; ++ks) {
            if constexpr (FP8) {
                const uint2 x = Base::query4(p, in, c.head_dim, q4, ks);
                qf[ks][0] = Base::kFit ? scaled_f16x2<QT>(x.x, factor) : x.x;
                qf[ks][1] = Base::kFit ? scaled_f16x2<QT>(x.y, factor) : x.y;
            } else {
                qf[ks][0] = Base::query2(p, in, c.head_dim, ks * 16 + 2 * q4);
                qf[ks][1] = Base::query2(p, in, c.head_dim, ks * 16 + 2 * q4 + 8);
            }
        }
        m0 = m1 = -INFINITY;
        l0 = l1 = 0.0f;
#pragma unroll
        for (int i = 0; i < kMT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;
    }

    __device__ __forceinline__ void tile(uint32_t kt, uint32_t vt, uint32_t, const Tiles& t, int p0, float* scores, const Unit& u, int lane) {
        const int g = lane >> 2, q4 = lane & 3;
        float x[kHB][4] = {}, z[kHB][4] = {};  // positions 16 h + g and 8 later; two sums, so that products wait less for each other
        if constexpr (!FP8) {
            const int row = ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
                for (int h = 0; h < kHB; ++h) {
                    uint32_t kf[4];
                    ldmatrix4(kf, kt + (row + 16 * h) * kRowBytes + k_vec<FP8, DP>(row, 2 * ks + (lane >> 4)) * 16);
                    mma16816<MT>(ks & 1 ? z[h] : x[h], kf, qf[ks][0], qf[ks][1]);
                }
        } else {
#pragma unroll
            for (int v = 0; v < DP / 64; ++v) {
                const int vec = k_vec<FP8, DP>(g, q4 * (DP / 64) + v) * 16;
                uint4 ka[kHB], kb[kHB];
#pragma unroll
                for (int h = 0; h < kHB; ++h) {
                    ka[h] = lds128(kt + (16 * h + g) * kRowBytes + vec);
                    kb[h] = lds128(kt + (16 * h + g + 8) * kRowBytes + vec);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int h = 0; h < kHB; ++h) {
                        const uint32_t wa = word(ka[h], i), wb = word(kb[h], i);
                        const uint32_t kf[4] = {e4m3x2_f16x2(wa), e4m3x2_f16x2(wb), e4m3x2_f16x2(wa >> 16), e4m3x2_f16x2(wb >> 16)};
                        mma16816<MT>(i & 1 ? z[h] : x[h], kf, qf[v * 4 + i][0], qf[v * 4 + i][1]);
                    }
            }
        }
        const bool whole = t.whole(p0, T);
#pragma unroll
        for (int h = 0; h < kHB; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool see = whole || t.visible(p0 + 16 * h + g + (e >> 1) * 8);
                x[h][e] = see ? (x[h][e] + z[h][e]) * (e & 1 ? sl1 : sl0) : -INFINITY;
            }
        if (scores) {
#pragma unroll
            for (int h = 0; h < kHB; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (u.row0 + 2 * q4 + (e & 1) < u.group) scores[(2 * q4 + (e & 1)) * T + 16 * h + g + (e >> 1) * 8] = x[h][e];
        }
        float top0 = m0, top1 = m1, low = INFINITY;
#pragma unroll
        for (int h = 0; h < kHB; ++h) {
            top0 = fmaxf(top0, fmaxf(x[h][0], x[h][2]));
            top1 = fmaxf(top1, fmaxf(x[h][1], x[h][3]));
            low = fminf(low, fminf(fminf(x[h][0], x[h][1]), fminf(x[h][2], x[h][3])));
        }
        const bool some_inf = !FP8 && __any_sync(kFullMask, low == -INFINITY);
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) {
            top0 = fmaxf(top0, __shfl_xor_sync(kFullMask, top0, s));
            top1 = fmaxf(top1, __shfl_xor_sync(kFullMask, top1, s));
        }
        if (__any_sync(kFullMask, top0 != m0 || top1 != m1)) {
            const float f0 = shrink(m0, top0), f1 = shrink(m1, top1);
            m0 = top0;
            m1 = top1;
            l0 *= f0;
            l1 *= f1;
#pragma unroll
            for (int i = 0; i < kMT; ++i) {
                o[i][0] *= f0;
                o[i][1] *= f1;
                o[i][2] *= f0;
                o[i][3] *= f1;
            }
        }
        const float ref0 = m0 == -INFINITY ? 0.0f : m0 - kShift, ref1 = m1 == -INFINITY ? 0.0f : m1 - kShift;
#pragma unroll
        for (int h = 0; h < kHB; ++h) {
            const float a0 = exp2_fast(x[h][0] - ref0), a1 = exp2_fast(x[h][1] - ref1);
            const float b0 = exp2_fast(x[h][2] - ref0), b1 = exp2_fast(x[h][3] - ref1);
            l0 += a0 + b0;
            l1 += a1 + b1;
            // 8 positions x 8 heads, then transposed: a lane's pair is two positions of head g
            uint32_t ph[2], pl[2];
            if constexpr (kTwo) {
                split2<MT, !FP8>(a0, a1, ph[0], pl[0]);
                split2<MT, !FP8>(b0, b1, ph[1], pl[1]);
                if (!FP8 && some_inf) {
                    drop2(x[h][0], x[h][1], ph[0], pl[0]);
                    drop2(x[h][2], x[h][3], ph[1], pl[1]);
                }
                pl[0] = transpose8(pl[0]);
                pl[1] = transpose8(pl[1]);
            } else {
                ph[0] = pack2<MT>(a0, a1);
                ph[1] = pack2<MT>(b0, b1);
            }
            ph[0] = transpose8(ph[0]);
            ph[1] = transpose8(ph[1]);
            const uint32_t vh = vt + 16 * h * kRowBytes;
            if constexpr (!FP8) {
                const int row = (lane >> 4) * 8 + (lane & 7);
#pragma unroll
                for (int i = 0; i < kMT; ++i) {
                    uint32_t vf[4];
                    ldmatrix4_t(vf, vh + row * kRowBytes + v_vec<FP8, DP>(row, 2 * i + ((lane >> 3) & 1)) * 16);
                    mma16816<MT>(o[i], vf, ph[0], ph[1]);
                    if constexpr (kTwo) mma16816<MT>(o[i], vf, pl[0], pl[1]);
                }
            } else {
#pragma unroll
                for (int v = 0; v < Base::kValueVecs; ++v) {
                    uint4 w[4];  // positions 2 q4, 2 q4 + 1, and 8 later
#pragma unroll
                    for (int k = 0; k < 4; ++k) w[k] = Base::values(vh, 2 * q4 + (k & 1) + (k >> 1) * 8, g, v);
#pragma unroll
                    for (int i = 0; i < Base::kValueWords; ++i) {
                        uint32_t lo[4], hi[4];
                        pairs4(word(w[0], i), word(w[1], i), lo);
                        pairs4(word(w[2], i), word(w[3], i), hi);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {  // row g of product j is dimension g * DP / 8 + 2 j, row g + 8 the next
                            const uint32_t vf[4] = {lo[2 * k], lo[2 * k + 1], hi[2 * k], hi[2 * k + 1]};
                            mma16816<MT>(o[v * 8 + i * 2 + k], vf, ph[0], ph[1]);
                            if constexpr (kTwo) mma16816<MT>(o[v * 8 + i * 2 + k], vf, pl[0], pl[1]);
                        }
                    }
                }
            }
        }
    }

    static __device__ __forceinline__ float4 factors(float f0, float f1) { return make_float4(f0, f1, f0, f1); }
    __device__ __forceinline__ void gather() {
#pragma unroll
        for (int i = 4; i < 32; i <<= 1) {
            l0 += __shfl_xor_sync(kFullMask, l0, i);
            l1 += __shfl_xor_sync(kFullMask, l1, i);
        }
    }
    template <typename F> __device__ __forceinline__ void each_sum(const Unit& u, int lane, F&& f) const {
        if (lane >= 4) return;
        if (u.row0 + 2 * lane < u.group) f(2 * lane, m0 - kShift, l0);
        if (u.row0 + 2 * lane + 1 < u.group) f(2 * lane + 1, m1 - kShift, l1);
    }
    __device__ __forceinline__ void store_out(const KvAttention& a, const Unit& u, float vs, int dim, int lane) const {
        const int g = lane >> 2, q4 = lane & 3;
        const float f0 = vs / l0, f1 = vs / l1;
        const bool some0 = l0 != 0.0f, some1 = l1 != 0.0f;
        QT* out = static_cast<QT*>(a.out) + (int64_t)u.b * a.out_seq_stride + (int64_t)(u.head * u.group + u.row0 + 2 * q4) * a.out_head_stride;
        const bool in0 = u.row0 + 2 * q4 < u.group, in1 = u.row0 + 2 * q4 + 1 < u.group;
        if constexpr (FP8) {
#pragma unroll
            for (int i = 0; i < kMT; ++i) {
                const int d = g * (DP / 8) + 2 * i;
                if (d >= dim) continue;
                if (in0) *reinterpret_cast<uint32_t*>(out + d) = some0 ? pack2<QT>(o[i][0] * f0, o[i][2] * f0) : 0u;
                if (in1) *reinterpret_cast<uint32_t*>(out + a.out_head_stride + d) = some1 ? pack2<QT>(o[i][1] * f1, o[i][3] * f1) : 0u;
            }
        } else {
            // lanes g and g ^ 1 trade, so that each holds two dimensions of one head
            const bool odd = g & 1;
            QT* mine = out + (odd ? a.out_head_stride : 0);
            const bool in = odd ? in1 : in0, some = odd ? some1 : some0;
#pragma unroll
            for (int i = 0; i < kMT; ++i)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float x0 = o[i][2 * half] * f0, x1 = o[i][2 * half + 1] * f1;
                    const float other = __shfl_xor_sync(kFullMask, odd ? x0 : x1, 4);
                    const int d = 16 * i + 8 * half + (g & ~1);
                    if (in && d < dim) *reinterpret_cast<uint32_t*>(mine + d) = !some ? 0u : odd ? pack2<QT>(other, x1) : pack2<QT>(x0, other);
                }
        }
    }
    __device__ __forceinline__ void store_part(float* part, const Unit& u, int lane) const {
        const int g = lane >> 2, q4 = lane & 3;
        const bool in0 = u.row0 + 2 * q4 < u.group, in1 = u.row0 + 2 * q4 + 1 < u.group;
        float *p0 = part + 2 * q4 * DP, *p1 = p0 + DP;
#pragma unroll
        for (int i = 0; i < kMT; ++i) {
            if constexpr (FP8) {
                const int d = g * (DP / 8) + 2 * i;
                if (in0) *reinterpret_cast<float2*>(p0 + d) = make_float2(o[i][0], o[i][2]);
                if (in1) *reinterpret_cast<float2*>(p1 + d) = make_float2(o[i][1], o[i][3]);
            } else {
                const int d = 16 * i + g;
                if (in0) {
                    p0[d] = o[i][0];
                    p0[d + 8] = o[i][2];
                }
                if (in1) {
                    p1[d] = o[i][1];
                    p1[d + 8] = o[i][3];
                }
            }
        }
    }
};

// What a warp sets aside of its row: every lane its own vectors of O, and the
// largest X that they go with.
template <typename Rows> struct Aside {
    float4 o[Rows::kVectors][32];
    float2 most[32];
};
// Adds what was set aside to the row again.
template <typename Rows> __device__ __forceinline__ void add_aside(Rows& r, const Aside<Rows>& a, int lane) {
    const float2 m = a.most[lane];
    const float4 f = Rows::factors(shrink(m.x, r.m0), shrink(m.y, r.m1));
#pragma unroll
    for (int i = 0; i < Rows::kVectors; ++i) {
        const float4 x = a.o[i][lane];
        r.o[i][0] += x.x * f.x;
        r.o[i][1] += x.y * f.y;
        r.o[i][2] += x.z * f.z;
        r.o[i][3] += x.w * f.w;
    }
}
// Sets the row's O aside, with what already was (`some`), and goes on from zero.
template <typename Rows> __device__ __forceinline__ void put_aside(Rows& r, Aside<Rows>& a, bool some, int lane) {
    if (some) add_aside(r, a, lane);
    a.most[lane] = make_float2(r.m0, r.m1);
#pragma unroll
    for (int i = 0; i < Rows::kVectors; ++i) {
        a.o[i][lane] = make_float4(r.o[i][0], r.o[i][1], r.o[i][2], r.o[i][3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) r.o[i][e] = 0.0f;
    }
}

}  // namespace ss
