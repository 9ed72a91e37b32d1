// kv_attend.cu -- attention of one new token per sequence over a paged
// key-value cache (streamscan.h, ss_kv_attend), split over the cache's length
// and joined, in two launches.
//
// Mathematics.  For one key-value head, its `group` query heads are the rows
// of a 16-row matrix Q.  Over a tile of 16 positions, X = (Q K^T) scale log2 e
// is two m16n8 products per 16 of head_dim; with a running reference R per row
// (the largest X so far), P = 2^(X - R), l += rowsum(P), O += P V, and l and O
// shrink by 2^(R_old - R_new) where R grows.  Parts of one row over disjoint
// positions join by the same rule: R = max R_i, l = sum l_i 2^(R_i - R),
// O = sum O_i 2^(R_i - R); out = O / l and lse = (R + log2 l) ln 2.
//
// What bounds it.  Every key and value byte is read once from device memory
// and serves `group` query heads: 4 group / (element bytes) flops a byte, far
// below the ridge, so the kernel is a stream of 16-byte asynchronous copies
// that the arithmetic has to stay under.
//
// Split.  The tiles of every (sequence, unit), a unit being 16 query heads of
// one key-value head, form one long list; a warp takes one contiguous share
// of it, all shares equal to within a tile, whatever the lengths are.  So a
// single long sequence and a ragged batch both fill every SM, and the host
// needs no lengths.  A warp works alone: it owns a ring of tiles in shared
// memory that only it fills and reads, so the main loop has no barrier.  Rows
// that lie within one warp's share are written at once; a share's first and
// last row may be parts, which go to scratch, and the second launch joins
// them.  Where weights are kept, the first launch leaves X (fp32) in scratch
// and the second turns it into weights, since they need the joined sums.
#include "kv.cuh"

namespace ss {

namespace {

constexpr int kTile = 16;       // positions per tile (a page may end inside it)
constexpr int kMaxBatch = 512;  // sequences per launch: their tile counts' prefix sums are in shared memory
constexpr int kFinishThreads = 256;
constexpr int kFinishWarps = kFinishThreads / 32;
constexpr int kWeightChunk = 512;  // positions per CTA of the weights' part
constexpr int kMaxGroup = 128;
constexpr size_t kMaxLogits = (size_t)2 << 30;  // bytes of scores one launch may leave in scratch

// Which positions of a sequence are visible, and in which tiles they lie: the
// tiles of the first tokens, then those of the window.
struct Tiles {
    int len, start, sinks, nsink, first, count;
    __device__ Tiles(int len_, int window, int sinks_) : len(len_), start(0), sinks(sinks_), nsink(0), first(0) {
        if (window > 0 && window < len) {
            start = len - window;
            first = start / kTile;
            nsink = min((min(sinks, start) + kTile - 1) / kTile, first);
        }
        count = nsink + (len + kTile - 1) / kTile - first;
    }
    __device__ __forceinline__ int tile(int j) const { return j < nsink ? j : first + j - nsink; }
    __device__ __forceinline__ bool visible(int p) const { return p < len && (p < sinks || p >= start); }
};

struct Scratch {
    int* pre;       // batch + 1: tiles of the sequences before, per unit
    float* lse2;    // batch x q_heads: R + log2 l of the rows the first launch finished
    float2* ml;     // workers x 2 x 16: (R, l) of a part
    float* o;       // workers x 2 x rows x DP: its O
    float* logits;  // per (sequence, key-value head) tile: group x 16 scores, log2 units; or null
    int group, units, rows, workers;  // units per sequence; rows = min(group, 16)
};

// Worker w of n takes the tiles [share(w), share(w + 1)) of `total`.
__device__ __forceinline__ long long share_begin(int w, int n, long long total) { return (long long)w * total / n; }
// The worker whose share holds tile t.
__device__ __forceinline__ int share_of(long long t, int n, long long total) { return (int)(((t + 1) * n - 1) / total); }

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

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

// Two e4m3 bytes as two fp16 (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t lo16) {
    uint32_t r;
    asm("{.reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t;}" : "=r"(r) : "r"(lo16));
    return r;
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

// A place in the list of tiles.
struct Cursor {
    int b, u, j;
    Tiles t;
    __device__ Cursor() : b(0), u(0), j(0), t(0, 0, 0) {}
};

// DP: head_dim rounded up to 64, 128 or 256 (the rest is zeros in shared
// memory).  NW warps of a CTA, S stages of each warp's ring.
template <typename QT, bool FP8, int DP, int NW, int S>
struct Shape {
    static constexpr int kBytes = FP8 ? 1 : 2;
    static constexpr int kRowBytes = DP * kBytes;
    static constexpr int kVecs = kRowBytes / 16;
    static constexpr int kTileBytes = kTile * kRowBytes;    // of k, and of v
    static constexpr bool kQShared = DP == 256;             // Q's fragments in shared memory: registers are short
    static constexpr int kQBytes = kQShared ? DP / 16 * 32 * 16 : 0;
    static constexpr size_t kSmem = (size_t)NW * (S * 2 * kTileBytes + kQBytes) + (kMaxBatch + 1) * 4;
};

template <typename QT, bool FP8, int DP, int NW, int S>
__global__ void __launch_bounds__(NW * 32, 1) k_kv_attend(KvPages c, KvTable t, KvAttention a, Scratch sc, uint32_t* status) {
    using Sh = Shape<QT, FP8, DP, NW, S>;
    // 8-bit caches multiply in fp16, which holds every e4m3 value; P is kept
    // below 2^15 by the reference so that small weights stay normal numbers.
    using MT = typename std::conditional<FP8, __half, QT>::type;
    constexpr bool kF16 = std::is_same<MT, __half>::value;
    constexpr float kShift = kF16 ? 15.0f : 0.0f;
    // P is split into two 16-bit terms, so that rounding it adds nothing to the
    // rounding of out (2^-16 against 2^-9 for bf16), except under bf16 outputs
    // of 8-bit caches, where one fp16 term (2^-12) is already finer than out.
    constexpr bool kTwo = !(FP8 && std::is_same<QT, __nv_bfloat16>::value);
    constexpr int kKS = DP / 16, kNT = DP / 8;

    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, q4 = lane & 3;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // Prefix sums of the sequences' tile counts.
    int* pre = reinterpret_cast<int*>(smem + (size_t)NW * (S * 2 * Sh::kTileBytes + Sh::kQBytes));
    for (int i = tid; i < t.batch; i += NW * 32) pre[i + 1] = Tiles(kv_len(t, i, status), a.window, a.sinks).count;
    __syncthreads();
    if (warp == 0) {
        int run = 0;
        for (int i0 = 0; i0 < t.batch; i0 += 32) {
            const int i = i0 + lane;
            const int x = warp_inclusive_scan<int>(i < t.batch ? pre[i + 1] : 0, lane) + run;
            if (i < t.batch) pre[i + 1] = x;
            run = __shfl_sync(kFullMask, x, 31);
        }
        if (lane == 0) pre[0] = 0;
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int i = tid; i <= t.batch; i += NW * 32) sc.pre[i] = pre[i];

    const long long total = (long long)pre[t.batch] * sc.units;
    const int workers = (int)min((long long)gridDim.x * NW, total);
    const int me = warp * gridDim.x + blockIdx.x;  // the first workers are on different SMs
    if (me >= workers) return;
    const long long t0 = share_begin(me, workers, total);
    const int n = (int)(share_begin(me + 1, workers, total) - t0);

    // The sequence, unit and tile at t0.
    Cursor cur;
    {
        int lo = 0, hi = t.batch;
        while (hi - lo > 1) {  // the last b with pre[b] units <= t0: never an empty one
            const int mid = (lo + hi) / 2;
            if ((long long)pre[mid] * sc.units <= t0) lo = mid; else hi = mid;
        }
        cur.b = lo;
        cur.t = Tiles(kv_len(t, lo, status), a.window, a.sinks);
        const long long r = t0 - (long long)pre[lo] * sc.units;
        cur.u = (int)(r / cur.t.count);
        cur.j = (int)(r % cur.t.count);
    }
    auto advance = [&](Cursor& x) {
        if (++x.j < x.t.count) return;
        x.j = 0;
        if (++x.u < sc.units) return;
        x.u = 0;
        do ++x.b; while (x.b < t.batch && pre[x.b + 1] == pre[x.b]);
        if (x.b < t.batch) x.t = Tiles(kv_len(t, x.b, status), a.window, a.sinks);
    };
    const int units_per_head = sc.units / c.kv_heads;

    // ---- the ring: this warp's tiles, filled S - 1 ahead ----
    unsigned char* ring = smem + (size_t)warp * (S * 2 * Sh::kTileBytes);
    const uint32_t ring_a = smem_addr(ring);
    Cursor ld = cur;
    int ld_page;  // the page of this lane's row (lane % 16) of the next tile, fetched one tile ahead
    auto fetch_page = [&]() {
        const int p = ld.t.tile(ld.j) * kTile + (lane & 15);
        ld_page = ld.b < t.batch && ld.t.visible(p) ? t.pages[(int64_t)ld.b * t.row_stride + p / c.page_size] : -1;
    };
    auto issue = [&](int stage) {
        const int p = ld.t.tile(ld.j) * kTile + (lane & 15);
        int64_t off = -1;
        if (ld.t.visible(p)) {
            if (ld_page >= 0 && ld_page < c.num_pages)
                off = ((int64_t)ld_page * c.page_stride + (int64_t)(ld.u / units_per_head) * c.head_stride +
                       (int64_t)(p % c.page_size) * c.slot_stride) * Sh::kBytes;
            else
                record_error(status, kErrKvTable, (uint32_t)(t.first + ld.b));
        }
        constexpr int kRows = 32 / Sh::kVecs > 0 ? 32 / Sh::kVecs : 1;  // rows per copy instruction
        const int v = lane % Sh::kVecs;
        const bool in_row = v * 16 < c.head_dim * Sh::kBytes;
        const uint32_t dst = ring_a + stage * (2 * Sh::kTileBytes);
#pragma unroll
        for (int i = 0; i < kTile / kRows; ++i) {
            const int row = lane / Sh::kVecs + i * kRows;
            const int64_t o = __shfl_sync(kFullMask, off, row);
            const bool ok = o >= 0 && in_row;  // otherwise the vector is filled with zeros
            const int64_t at = ok ? o + v * 16 : 0;
            cp_async16(dst + row * Sh::kRowBytes + k_vec<FP8, DP>(row, v) * 16, c.k + at, ok ? 16 : 0);
            cp_async16(dst + Sh::kTileBytes + row * Sh::kRowBytes + v_vec<FP8, DP>(row, v) * 16, c.v + at, ok ? 16 : 0);
        }
    };
    fetch_page();
#pragma unroll
    for (int s = 0; s < S - 1; ++s) {
        if (s < n) {
            issue(s);
            advance(ld);
            fetch_page();
        }
        cp_commit();
    }

    // ---- this warp's rows ----
    uint32_t qf[Sh::kQShared ? 1 : kKS][4];
    unsigned char* qs = smem + (size_t)NW * (S * 2 * Sh::kTileBytes) + (size_t)warp * Sh::kQBytes;
    float o[kNT][4];
    float m0, m1, l0, l1;      // largest X of rows g and g + 8, and this lane's share of l
    float sl0 = 0, sl1 = 0;    // X per unit of q . k
    int began = 0;             // whether this row started in this share
    int head = 0, row0 = 0;    // key-value head, and the unit's first query head within it

    auto open_row = [&]() {
        head = cur.u / units_per_head;
        row0 = (cur.u % units_per_head) * 16;
        began = cur.j == 0;
        const QT* q = static_cast<const QT*>(a.q) + (int64_t)cur.b * a.q_seq_stride;
        const int ra = row0 + g, rb = ra + 8;
        const QT* pa = q + (int64_t)(head * sc.group + ra) * a.q_head_stride;
        const QT* pb = q + (int64_t)(head * sc.group + rb) * a.q_head_stride;
        const float sl = a.scale * 1.4426950408889634f * (FP8 && c.k_scale ? c.k_scale[head] : 1.0f);
        sl0 = sl1 = sl;
        auto put = [&](int ks, const uint32_t (&f)[4]) {
            if constexpr (Sh::kQShared) {
                *reinterpret_cast<uint4*>(qs + (ks * 32 + lane) * 16) = make_uint4(f[0], f[1], f[2], f[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) qf[ks][i] = f[i];
            }
        };
        if constexpr (!FP8) {
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks) {
                uint32_t f[4];
                const int d = ks * 16 + 2 * q4;
                f[0] = ra < sc.group && d < c.head_dim ? *reinterpret_cast<const uint32_t*>(pa + d) : 0u;
                f[1] = rb < sc.group && d < c.head_dim ? *reinterpret_cast<const uint32_t*>(pb + d) : 0u;
                f[2] = ra < sc.group && d + 8 < c.head_dim ? *reinterpret_cast<const uint32_t*>(pa + d + 8) : 0u;
                f[3] = rb < sc.group && d + 8 < c.head_dim ? *reinterpret_cast<const uint32_t*>(pb + d + 8) : 0u;
                put(ks, f);
            }
        } else {
            // The products' index runs over head_dim in another order: step ks
            // of lane q4 holds the four dimensions q4 * DP / 4 + 4 ks and on,
            // so that a lane's keys are consecutive bytes.
            auto load4 = [&](const QT* p, bool in, int ks) {
                const int d = q4 * (DP / 4) + 4 * ks;
                return in && d < c.head_dim ? *reinterpret_cast<const uint2*>(p + d) : make_uint2(0u, 0u);
            };
            float fa = 1.0f, fb = 1.0f;
            if constexpr (!std::is_same<QT, __half>::value) {
                // A power of two per row brings q into fp16's range (its largest
                // element to [2^7, 2^8); what falls below 2^-24 of that is lost
                // against sums that are rounded at 2^-24 themselves).
                float ma = 0.0f, mb = 0.0f;
                for (int ks = 0; ks < kKS; ++ks) {
                    const uint2 x = load4(pa, ra < sc.group, ks), y = load4(pb, rb < sc.group, ks);
                    const uint32_t wa[2] = {x.x, x.y}, wb[2] = {y.x, y.y};
                    for (int i = 0; i < 2; ++i) {
                        const float2 u = open2<QT>(wa[i]), v = open2<QT>(wb[i]);
                        ma = fmaxf(ma, fmaxf(isfinite(u.x) ? fabsf(u.x) : 0.0f, isfinite(u.y) ? fabsf(u.y) : 0.0f));
                        mb = fmaxf(mb, fmaxf(isfinite(v.x) ? fabsf(v.x) : 0.0f, isfinite(v.y) ? fabsf(v.y) : 0.0f));
                    }
                }
                for (int i = 1; i < 4; i <<= 1) {
                    ma = fmaxf(ma, __shfl_xor_sync(kFullMask, ma, i));
                    mb = fmaxf(mb, __shfl_xor_sync(kFullMask, mb, i));
                }
                const int ea = max((int)(__float_as_uint(ma) >> 23) - 127, -118);
                const int eb = max((int)(__float_as_uint(mb) >> 23) - 127, -118);
                fa = __uint_as_float((uint32_t)(127 + 7 - ea) << 23);
                fb = __uint_as_float((uint32_t)(127 + 7 - eb) << 23);
                sl0 *= __uint_as_float((uint32_t)(127 - 7 + ea) << 23);
                sl1 *= __uint_as_float((uint32_t)(127 - 7 + eb) << 23);
            }
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks) {
                const uint2 x = load4(pa, ra < sc.group, ks), y = load4(pb, rb < sc.group, ks);
                uint32_t f[4] = {x.x, y.x, x.y, y.y};
                if constexpr (!std::is_same<QT, __half>::value) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 u = open2<QT>(f[i]);
                        const float s = i & 1 ? fb : fa;
                        f[i] = pack2<__half>(u.x * s, u.y * s);
                    }
                }
                put(ks, f);
            }
        }
        m0 = m1 = -INFINITY;
        l0 = l1 = 0.0f;
#pragma unroll
        for (int i = 0; i < kNT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;
    };
    auto q_frag = [&](int ks, uint32_t (&f)[4]) {
        if constexpr (Sh::kQShared) {
            const uint4 x = lds128(smem_addr(qs) + (ks * 32 + lane) * 16);
            f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = qf[ks][i];
        }
    };
    // Visits this lane's outputs as (row half, first dimension, two values).
    auto each_pair = [&](auto&& f) {
        if constexpr (!FP8) {
#pragma unroll
            for (int i = 0; i < kNT; ++i) {
                f(0, i * 8 + 2 * q4, o[i][0], o[i][1]);
                f(1, i * 8 + 2 * q4, o[i][2], o[i][3]);
            }
        } else {  // column n of product i is dimension n * DP / 8 + i
#pragma unroll
            for (int i = 0; i < kNT; i += 2)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    f(0, (2 * q4 + e) * (DP / 8) + i, o[i][e], o[i + 1][e]);
                    f(1, (2 * q4 + e) * (DP / 8) + i, o[i][2 + e], o[i + 1][2 + e]);
                }
        }
    };
    auto close_row = [&](bool ended) {
        float la = l0, lb = l1;
#pragma unroll
        for (int i = 1; i < 4; i <<= 1) {
            la += __shfl_xor_sync(kFullMask, la, i);
            lb += __shfl_xor_sync(kFullMask, lb, i);
        }
        const int ra = row0 + g, rb = ra + 8;
        const bool in[2] = {ra < sc.group, rb < sc.group};
        if (began && ended) {
            const float vs = FP8 && c.v_scale ? c.v_scale[head] : 1.0f;
            const float f[2] = {la == 0.0f ? 0.0f : vs / la, lb == 0.0f ? 0.0f : vs / lb};
            QT* out = static_cast<QT*>(a.out) + (int64_t)cur.b * a.out_seq_stride;
            QT* po[2] = {out + (int64_t)(head * sc.group + ra) * a.out_head_stride, out + (int64_t)(head * sc.group + rb) * a.out_head_stride};
            each_pair([&](int half, int d, float x, float y) {
                if (in[half] && d < c.head_dim) *reinterpret_cast<uint32_t*>(po[half] + d) = pack2<QT>(x * f[half], y * f[half]);
            });
            if (q4 == 0) {
                const float z[2] = {la == 0.0f ? -INFINITY : m0 - kShift + log2f(la), lb == 0.0f ? -INFINITY : m1 - kShift + log2f(lb)};
                for (int half = 0; half < 2; ++half) {
                    const int64_t at = (int64_t)cur.b * a.q_heads + head * sc.group + (half ? rb : ra);
                    if (!in[half]) continue;
                    sc.lse2[at] = z[half];
                    if (a.lse) a.lse[at] = z[half] * 0.6931471805599453f;
                }
            }
            return;
        }
        const int slot = me * 2 + (began ? 1 : 0);
        if (q4 == 0) {
            if (in[0]) sc.ml[slot * 16 + g] = make_float2(m0 - kShift, la);
            if (in[1]) sc.ml[slot * 16 + g + 8] = make_float2(m1 - kShift, lb);
        }
        float* part = sc.o + (int64_t)slot * sc.rows * DP;
        each_pair([&](int half, int d, float x, float y) {
            if (in[half]) *reinterpret_cast<float2*>(part + (g + 8 * half) * DP + d) = make_float2(x, y);
        });
    };

    open_row();
    int stage = 0;
    for (int i = 0; i < n; ++i) {
        cp_wait<S - 2>();
        __syncwarp();  // every lane's copies have landed, and the stage to fill next has been read
        if (i + S - 1 < n) {
            issue(stage == 0 ? S - 1 : stage - 1);
            advance(ld);
            fetch_page();
        }
        cp_commit();
        const uint32_t kt = ring_a + stage * (2 * Sh::kTileBytes), vt = kt + Sh::kTileBytes;
        stage = stage + 1 == S ? 0 : stage + 1;

        float x[2][4] = {};
        if constexpr (!FP8) {
            const int row = (lane >> 4) * 8 + (lane & 7);
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks) {
                uint32_t kf[4], f[4];
                ldmatrix4(kf, kt + row * Sh::kRowBytes + k_vec<FP8, DP>(row, 2 * ks + ((lane >> 3) & 1)) * 16);
                q_frag(ks, f);
                mma16816<MT>(x[0], f, kf[0], kf[1]);
                mma16816<MT>(x[1], f, kf[2], kf[3]);
            }
        } else {
#pragma unroll
            for (int v = 0; v < DP / 64; ++v) {
                const int vec = q4 * (DP / 64) + v;
                const uint4 ka = lds128(kt + g * Sh::kRowBytes + k_vec<FP8, DP>(g, vec) * 16);
                const uint4 kb = lds128(kt + (g + 8) * Sh::kRowBytes + k_vec<FP8, DP>(g + 8, vec) * 16);
                const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                for (int i4 = 0; i4 < 4; ++i4) {
                    uint32_t f[4];
                    q_frag(v * 4 + i4, f);
                    mma16816<MT>(x[0], f, e4m3x2_f16x2(wa[i4]), e4m3x2_f16x2(wa[i4] >> 16));
                    mma16816<MT>(x[1], f, e4m3x2_f16x2(wb[i4]), e4m3x2_f16x2(wb[i4] >> 16));
                }
            }
        }
        const int p0 = cur.t.tile(cur.j) * kTile + 2 * q4;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const bool see = cur.t.visible(p0 + nt * 8 + e);
                x[nt][e] = see ? x[nt][e] * sl0 : -INFINITY;
                x[nt][2 + e] = see ? x[nt][2 + e] * sl1 : -INFINITY;
            }
        if (sc.logits) {
            const int64_t tile = (int64_t)pre[cur.b] * c.kv_heads + (int64_t)head * cur.t.count + cur.j;
            float* to = sc.logits + (tile * sc.group + row0 + g) * kTile + 2 * q4;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                if (row0 + g < sc.group) *reinterpret_cast<float2*>(to + nt * 8) = make_float2(x[nt][0], x[nt][1]);
                if (row0 + g + 8 < sc.group) *reinterpret_cast<float2*>(to + 8 * kTile + nt * 8) = make_float2(x[nt][2], x[nt][3]);
            }
        }
        float top0 = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1]));
        float top1 = fmaxf(fmaxf(x[0][2], x[0][3]), fmaxf(x[1][2], x[1][3]));
#pragma unroll
        for (int s = 1; s < 4; s <<= 1) {
            top0 = fmaxf(top0, __shfl_xor_sync(kFullMask, top0, s));
            top1 = fmaxf(top1, __shfl_xor_sync(kFullMask, top1, s));
        }
        top0 = fmaxf(top0, m0);
        top1 = fmaxf(top1, m1);
        if (__any_sync(kFullMask, top0 != m0 || top1 != m1)) {
            const float f0 = top0 == m0 ? 1.0f : exp2_fast(m0 - top0), f1 = top1 == m1 ? 1.0f : exp2_fast(m1 - top1);
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
        uint32_t ph[4], pl[4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            const float a0 = exp2_fast(x[nt][0] - ref0), a1 = exp2_fast(x[nt][1] - ref0);
            const float b0 = exp2_fast(x[nt][2] - ref1), b1 = exp2_fast(x[nt][3] - ref1);
            l0 += a0 + a1;
            l1 += b0 + b1;
            ph[nt * 2] = pack2<MT>(a0, a1);
            ph[nt * 2 + 1] = pack2<MT>(b0, b1);
            if constexpr (kTwo) {
                const float2 ra = open2<MT>(ph[nt * 2]), rb = open2<MT>(ph[nt * 2 + 1]);
                pl[nt * 2] = pack2<MT>(a0 - ra.x, a1 - ra.y);
                pl[nt * 2 + 1] = pack2<MT>(b0 - rb.x, b1 - rb.y);
            }
        }
        if constexpr (!FP8) {
            const int row = ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
            for (int nt = 0; nt < kNT; nt += 2) {
                uint32_t vf[4];
                ldmatrix4_t(vf, vt + row * Sh::kRowBytes + v_vec<FP8, DP>(row, nt + (lane >> 4)) * 16);
                mma16816<MT>(o[nt], ph, vf[0], vf[1]);
                mma16816<MT>(o[nt + 1], ph, vf[2], vf[3]);
                if constexpr (kTwo) {
                    mma16816<MT>(o[nt], pl, vf[0], vf[1]);
                    mma16816<MT>(o[nt + 1], pl, vf[2], vf[3]);
                }
            }
        } else {
            auto four = [&](int nt, uint32_t w0, uint32_t w1, uint32_t w8, uint32_t w9) {
                // bytes of positions (2 q4, 2 q4 + 1) and (2 q4 + 8, + 9) side by side, for products nt .. nt + 3
                const uint32_t a01 = __byte_perm(w0, w1, 0x5140), a23 = __byte_perm(w0, w1, 0x7362);
                const uint32_t b01 = __byte_perm(w8, w9, 0x5140), b23 = __byte_perm(w8, w9, 0x7362);
                const uint32_t va[4] = {a01, a01 >> 16, a23, a23 >> 16}, vb[4] = {b01, b01 >> 16, b23, b23 >> 16};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t f0 = e4m3x2_f16x2(va[k]), f1 = e4m3x2_f16x2(vb[k]);
                    mma16816<MT>(o[nt + k], ph, f0, f1);
                    if constexpr (kTwo) mma16816<MT>(o[nt + k], pl, f0, f1);
                }
            };
            const int r0 = 2 * q4;
            if constexpr (DP == 64) {
                uint2 w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int row = r0 + (k & 1) + (k >> 1) * 8;
                    w[k] = lds64(vt + row * Sh::kRowBytes + v_vec<FP8, DP>(row, g >> 1) * 16 + (g & 1) * 8);
                }
                four(0, w[0].x, w[1].x, w[2].x, w[3].x);
                four(4, w[0].y, w[1].y, w[2].y, w[3].y);
            } else {
#pragma unroll
                for (int v = 0; v < DP / 128; ++v) {
                    uint4 w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int row = r0 + (k & 1) + (k >> 1) * 8;
                        w[k] = lds128(vt + row * Sh::kRowBytes + v_vec<FP8, DP>(row, g * (DP / 128) + v) * 16);
                    }
                    four(v * 16, w[0].x, w[1].x, w[2].x, w[3].x);
                    four(v * 16 + 4, w[0].y, w[1].y, w[2].y, w[3].y);
                    four(v * 16 + 8, w[0].z, w[1].z, w[2].z, w[3].z);
                    four(v * 16 + 12, w[0].w, w[1].w, w[2].w, w[3].w);
                }
            }
        }
        if (cur.j + 1 == cur.t.count) {
            close_row(true);
            advance(cur);
            if (i + 1 < n) open_row();
        } else {
            advance(cur);
            if (i + 1 == n) close_row(false);
        }
    }
    cp_wait<0>();
}

// ---- the second launch: joins, empty rows, weights ----

// The parts of unit u of a sequence: workers [w0, w1]; one worker: no parts.
struct Parts {
    int w0, w1;
    long long s0;
    __device__ Parts(const Scratch& sc, const int* pre, int batch, int b, int u) {
        const int count = pre[b + 1] - pre[b];
        const long long total = (long long)pre[batch] * sc.units;
        const int n = (int)min((long long)sc.workers, total);
        s0 = (long long)pre[b] * sc.units + (long long)u * count;
        w0 = share_of(s0, n, total);
        w1 = share_of(s0 + count - 1, n, total);
    }
    // The first part is its worker's last row, the others are their workers' first ones.
    __device__ __forceinline__ int slot(int i) const { return (w0 + i) * 2 + (i == 0 ? 1 : 0); }
    __device__ __forceinline__ int count() const { return w1 - w0 + 1; }
};

// (R, l) of row `row` joined over the parts, by one warp.
__device__ __forceinline__ float2 join_ml(const Scratch& sc, const Parts& p, int row, int lane) {
    float top = -INFINITY, l = 0.0f;
    for (int i = lane; i < p.count(); i += 32) top = fmaxf(top, sc.ml[p.slot(i) * 16 + row].x);
    for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, s));
    for (int i = lane; i < p.count(); i += 32) {
        const float2 x = sc.ml[p.slot(i) * 16 + row];
        l += x.x == -INFINITY ? 0.0f : x.y * exp2_fast(x.x - top);
    }
    return make_float2(top, warp_sum<float>(l));
}

template <typename QT, int DP>
__global__ void __launch_bounds__(kFinishThreads) k_kv_finish(KvPages c, KvTable t, KvAttention a, Scratch sc, int chunks,
                                                             uint32_t* status) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float s_lse[kMaxGroup];
    __shared__ float4 s_o[kFinishWarps][DP / 4];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int units_per_head = sc.units / c.kv_heads;
    const int joins = t.batch * a.q_heads;
    if ((int)blockIdx.x < joins) {
        const int b = blockIdx.x / a.q_heads, j = blockIdx.x % a.q_heads;
        const int h = j / sc.group, r = j % sc.group;
        QT* out = static_cast<QT*>(a.out) + (int64_t)b * a.out_seq_stride + (int64_t)j * a.out_head_stride;
        if (sc.pre[b + 1] == sc.pre[b]) {  // no visible position
            for (int d = tid; d < c.head_dim; d += kFinishThreads) out[d] = from_f32<QT>(0.0f);
            if (tid == 0 && a.lse) a.lse[(int64_t)b * a.q_heads + j] = -INFINITY;
            return;
        }
        const Parts p(sc, sc.pre, t.batch, b, h * units_per_head + r / 16);
        if (p.count() == 1) return;
        const int row = r % 16;
        const float2 ml = join_ml(sc, p, row, lane);
        float4 acc[(DP + 127) / 128] = {};
        for (int i = warp; i < p.count(); i += kFinishWarps) {
            const int slot = p.slot(i);
            const float ref = sc.ml[slot * 16 + row].x;
            const float f = ref == -INFINITY ? 0.0f : exp2_fast(ref - ml.x);
            const float4* part = reinterpret_cast<const float4*>(sc.o + ((int64_t)slot * sc.rows + row) * DP);
#pragma unroll
            for (int k = 0; k < (DP + 127) / 128; ++k) {
                if (lane + k * 32 >= DP / 4) continue;
                const float4 x = part[lane + k * 32];
                acc[k].x += f * x.x;
                acc[k].y += f * x.y;
                acc[k].z += f * x.z;
                acc[k].w += f * x.w;
            }
        }
#pragma unroll
        for (int k = 0; k < (DP + 127) / 128; ++k)
            if (lane + k * 32 < DP / 4) s_o[warp][lane + k * 32] = acc[k];
        __syncthreads();
        const float vs = c.v_scale ? c.v_scale[h] : 1.0f;
        const float inv = ml.y == 0.0f ? 0.0f : vs / ml.y;
        for (int d = tid; d < c.head_dim; d += kFinishThreads) {
            float x = 0.0f;
            for (int w = 0; w < kFinishWarps; ++w) x += reinterpret_cast<const float*>(s_o[w])[d];
            out[d] = from_f32<QT>(ml.y == 0.0f ? 0.0f : x * inv);
        }
        if (tid == 0 && a.lse)
            a.lse[(int64_t)b * a.q_heads + j] = ml.y == 0.0f ? -INFINITY : (ml.x + log2f(ml.y)) * 0.6931471805599453f;
        return;
    }
    // Weights of kWeightChunk positions of one (sequence, key-value head).
    const int k = blockIdx.x - joins;
    const int chunk = k % chunks, bh = k / chunks;
    const int b = bh / c.kv_heads, h = bh % c.kv_heads;
    const Tiles tl(kv_len(t, b, status), a.window, a.sinks);
    if (chunk * kWeightChunk >= tl.len) return;
    for (int r = warp; r < sc.group; r += kFinishWarps) {
        const Parts p(sc, sc.pre, t.batch, b, h * units_per_head + r / 16);
        float lse;
        if (p.count() == 1) {
            lse = sc.lse2[(int64_t)b * a.q_heads + h * sc.group + r];
        } else {
            const float2 ml = join_ml(sc, p, r % 16, lane);
            lse = ml.y == 0.0f ? -INFINITY : ml.x + log2f(ml.y);
        }
        if (lane == 0) s_lse[r] = lse;
    }
    __syncthreads();
    const int64_t tile0 = (int64_t)sc.pre[b] * c.kv_heads + (int64_t)h * tl.count;
    for (int p = chunk * kWeightChunk + tid; p < min(tl.len, (chunk + 1) * kWeightChunk); p += kFinishThreads) {
        const bool see = tl.visible(p);
        if (!see && a.weight_in == a.weight_out) continue;  // accumulated in place: nothing to add
        const int page = kv_page(t, c.num_pages, b, p / c.page_size, status);
        if (page < 0) continue;
        float w = 0.0f;
        if (see) {
            const int tile = p / kTile;
            const int j = tile < tl.nsink ? tile : tl.nsink + tile - tl.first;
            const float* x = sc.logits + (tile0 + j) * sc.group * kTile + p % kTile;
            for (int r = 0; r < sc.group; ++r) {
                const float z = s_lse[r];
                w += z == -INFINITY ? 0.0f : exp2_fast(x[r * kTile] - z);
            }
        }
        const int64_t at = ((int64_t)page * c.kv_heads + h) * c.page_size + p % c.page_size;
        a.weight_out[at] = (a.weight_in ? a.weight_in[at] : 0.0f) + w;
    }
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

// How one call is cut into launches, and the scratch of the largest.
struct Plan {
    int batch;  // sequences per launch
    int dp, warps, grid;
    Scratch sc;
    size_t at_lse2, at_ml, at_o, at_logits, bytes;
};

Plan make_plan(const KvPages& c, const KvTable& t, const KvAttention& a, int warps, int dp, int sms) {
    Plan p{};
    p.dp = dp;
    p.warps = warps;
    p.sc.group = a.q_heads / c.kv_heads;
    p.sc.units = c.kv_heads * ((p.sc.group + 15) / 16);
    p.sc.rows = p.sc.group < 16 ? p.sc.group : 16;
    const size_t tiles = ((size_t)t.max_len + kTile - 1) / kTile;  // of one sequence and unit, at most
    const size_t seq_logits = a.weight_out ? tiles * a.q_heads * kTile * 4 : 0;
    size_t batch = (size_t)t.batch < kMaxBatch ? t.batch : kMaxBatch;
    if (seq_logits * batch > kMaxLogits) batch = kMaxLogits / seq_logits;
    while (batch > 1 && batch * tiles > 0x7fffffff) batch /= 2;
    p.batch = batch < 1 ? 1 : (int)batch;
    const size_t most = (size_t)p.batch * tiles * p.sc.units;
    p.grid = most < (size_t)sms ? (most < 1 ? 1 : (int)most) : sms;
    p.sc.workers = p.grid * warps;
    p.at_lse2 = round256((kMaxBatch + 1) * 4);
    p.at_ml = p.at_lse2 + round256((size_t)p.batch * a.q_heads * 4);
    p.at_o = p.at_ml + round256((size_t)p.sc.workers * 2 * 16 * 8);
    p.at_logits = p.at_o + round256((size_t)p.sc.workers * 2 * p.sc.rows * dp * 4);
    p.bytes = p.at_logits + round256(seq_logits * p.batch);
    return p;
}

template <typename QT, bool FP8, int DP, int NW, int S>
cudaError_t run(const KvPages& c, const KvTable& t, const KvAttention& a, void* scratch, size_t* bytes, uint32_t* status, cudaStream_t s) {
    auto* kern = k_kv_attend<QT, FP8, DP, NW, S>;
    constexpr size_t smem = Shape<QT, FP8, DP, NW, S>::kSmem;
    static_assert(smem <= 227 * 1024, "the ring does not fit in shared memory");
    KernelSetup su;
    cudaError_t e = kernel_setup(reinterpret_cast<const void*>(kern), NW * 32, smem, &su);
    if (e != cudaSuccess) return e;
    Plan p = make_plan(c, t, a, NW, DP, su.sms);
    if (scratch == nullptr) {
        *bytes = p.bytes;
        return cudaSuccess;
    }
    char* base = static_cast<char*>(scratch);
    p.sc.pre = reinterpret_cast<int*>(base);
    p.sc.lse2 = reinterpret_cast<float*>(base + p.at_lse2);
    p.sc.ml = reinterpret_cast<float2*>(base + p.at_ml);
    p.sc.o = reinterpret_cast<float*>(base + p.at_o);
    p.sc.logits = a.weight_out ? reinterpret_cast<float*>(base + p.at_logits) : nullptr;
    for (int b0 = 0; b0 < t.batch; b0 += p.batch) {
        KvTable u = t;
        KvAttention v = a;
        u.first = b0;
        u.batch = t.batch - b0 < p.batch ? t.batch - b0 : p.batch;
        u.pages += (int64_t)b0 * t.row_stride;
        u.lens += b0;
        v.q = static_cast<const QT*>(a.q) + (int64_t)b0 * a.q_seq_stride;
        v.out = static_cast<QT*>(a.out) + (int64_t)b0 * a.out_seq_stride;
        if (a.lse) v.lse = a.lse + (int64_t)b0 * a.q_heads;
        kern<<<p.grid, NW * 32, smem, s>>>(c, u, v, p.sc, status);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        const int chunks = (t.max_len + kWeightChunk - 1) / kWeightChunk;
        const size_t blocks = (size_t)u.batch * a.q_heads + (a.weight_out ? (size_t)u.batch * c.kv_heads * chunks : 0);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)blocks);
        cfg.blockDim = dim3(kFinishThreads);
        cfg.stream = s;
        cudaLaunchAttribute at;
        at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, k_kv_finish<QT, DP>, c, u, v, p.sc, chunks, status);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// Warps and stages by tile size: the ring takes about 192 KB of the SM, and
// the warps as many as their registers allow.
template <typename QT, bool FP8>
cudaError_t run_dim(const KvPages& c, const KvTable& t, const KvAttention& a, void* scratch, size_t* bytes, uint32_t* status, cudaStream_t s) {
    if (c.head_dim <= 64) return run<QT, FP8, 64, FP8 ? 16 : 12, FP8 ? 6 : 4>(c, t, a, scratch, bytes, status, s);
    if (c.head_dim <= 128) return run<QT, FP8, 128, FP8 ? 12 : 8, FP8 ? 4 : 3>(c, t, a, scratch, bytes, status, s);
    return run<QT, FP8, 256, FP8 ? 7 : 4, 3>(c, t, a, scratch, bytes, status, s);
}

cudaError_t run_any(const KvPages& c, const KvTable& t, const KvAttention& a, void* scratch, size_t* bytes, uint32_t* status, cudaStream_t s) {
    const bool bf = a.type == KvElem::BF16;
    if (c.type == KvElem::E4M3)
        return bf ? run_dim<__nv_bfloat16, true>(c, t, a, scratch, bytes, status, s) : run_dim<__half, true>(c, t, a, scratch, bytes, status, s);
    return bf ? run_dim<__nv_bfloat16, false>(c, t, a, scratch, bytes, status, s) : run_dim<__half, false>(c, t, a, scratch, bytes, status, s);
}

}  // namespace

cudaError_t kv_attend_scratch(const KvPages& c, const KvTable& t, const KvAttention& a, size_t* bytes) {
    return run_any(c, t, a, nullptr, bytes, nullptr, nullptr);
}

cudaError_t launch_kv_attend(const KvPages& c, const KvTable& t, const KvAttention& a, void* scratch, uint32_t* status, cudaStream_t s) {
    return run_any(c, t, a, scratch, nullptr, status, s);
}

}  // namespace ss
