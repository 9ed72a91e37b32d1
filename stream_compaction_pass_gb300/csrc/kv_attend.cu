// kv_attend.cu -- attention of one new token per sequence over a paged
// key-value cache (streamscan.h, ss_kv_attend), split over the cache's length
// and joined, in two launches, and a third where weights are kept.
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
// and the third turns it into weights, since they need the joined sums.
#include "kv.cuh"

namespace ss {

namespace {

// Sequences per launch: their tile counts' prefix sums are in shared memory,
// beside a ring that leaves little of it at head_dim 256.
template <int DP> constexpr int kMaxBatch = DP == 256 ? 512 : 4096;
constexpr int kJoinThreads = 512;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kWeightThreads = 256;
constexpr size_t kMaxLogits = (size_t)2 << 30;  // bytes of scores one launch may leave in scratch

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

struct Scratch {
    int* pre;       // batch + 1: tiles of the sequences before, per unit
    int* pre_all;   // the same of all positions, where those that are not visible get a weight too (else pre)
    float* lse2;    // batch x q_heads: R + log2 l of every row, for the weights
    float2* ml;     // workers x 2 x 16: (R, l) of a part
    float* o;       // workers x 2 x rows x DP: its O
    float* logits;  // per (sequence, key-value head) tile: group x 16 scores, log2 units; or null
    int group, units, rows, workers;  // units per sequence; rows = min(group, 16)
    int shift;                        // tiles have 2^shift positions
    FastDiv page;                     // by page_size
};

// A list of `total` tiles cut into n contiguous shares, the first ones a tile
// longer.  Lists are shorter than 2^31 (the launcher sees to it).
struct Shares {
    int quot, rem;
    __device__ __forceinline__ Shares(int total, int n) : quot(total / n), rem(total - total / n * n) {}
    __device__ __forceinline__ int begin(int w) const { return w * quot + min(w, rem); }
    __device__ __forceinline__ int holder(int t) const {  // the share that holds tile t
        const int split = rem * (quot + 1);
        return t < split ? t / (quot + 1) : rem + (t - split) / quot;
    }
};

// The last b with pre[b] * per <= at, for at < pre[n] * per: never an empty sequence.
__device__ __forceinline__ int find_sequence(const int* pre, int n, int per, int at) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (pre[mid] * per <= at) lo = mid; else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::128B [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes), "l"(policy) : "memory");
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

// x[1 .. n] become their running sums and x[0] zero, by one warp.
__device__ __forceinline__ void prefix_sums(int* x, int n, int lane) {
    int run = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        const int y = warp_inclusive_scan<int>(i < n ? x[i + 1] : 0, lane) + run;
        if (i < n) x[i + 1] = y;
        run = __shfl_sync(kFullMask, y, 31);
    }
    if (lane == 0) x[0] = 0;
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

// The sum of row `at` (sequence * q_heads + head): R and l.  A row without
// weights leaves +inf for the weights' pass, where 2^(X - inf) = 0.
__device__ __forceinline__ void store_lse(const Scratch& sc, const KvAttention& a, int64_t at, float ref, float l) {
    const float x = ref + log2f(l);
    sc.lse2[at] = l == 0.0f ? INFINITY : x;
    if (a.lse) a.lse[at] = l == 0.0f ? -INFINITY : x * 0.6931471805599453f;
}

// A place in the list of tiles: sequence, key-value head, 16 query heads of
// its group, tile.
struct Cursor {
    int b, head, part, j;
    Tiles t;
    __device__ __forceinline__ Cursor() : b(0), head(0), part(0), j(0), t(0, 0, 0, 0) {}
};

// DP: head_dim rounded up to 64, 128 or 256 (the rest is zeros in shared
// memory).  T positions per tile (16 or 32), NW warps of a CTA, S stages of
// each warp's ring.
template <bool FP8, int DP, int T, int NW, int S>
struct Shape {
    static constexpr int kBytes = FP8 ? 1 : 2;
    static constexpr int kRowBytes = DP * kBytes;
    static constexpr int kVecs = kRowBytes / 16;
    static constexpr int kTileBytes = T * kRowBytes;        // of k, and of v
    static constexpr bool kQShared = DP == 256;             // Q's fragments in shared memory: registers are short
    static constexpr int kQBytes = kQShared ? DP / 16 * 32 * 16 : 0;
    static constexpr size_t kSmem = (size_t)NW * (S * 2 * kTileBytes + kQBytes) + (kMaxBatch<DP> + 1) * 4;
};

template <typename QT, bool FP8, int DP, int T, int NW, int S>
__global__ void __launch_bounds__(NW * 32, 1) k_kv_attend(KvPages c, KvTable t, KvAttention a, Scratch sc, uint32_t* status) {
    using Sh = Shape<FP8, DP, T, NW, S>;
    constexpr int kShift2 = T == 16 ? 4 : 5;
    // 8-bit caches multiply in fp16, which holds every e4m3 value; P is kept
    // below 2^15 by the reference so that small weights stay normal numbers.
    using MT = typename std::conditional<FP8, __half, QT>::type;
    constexpr bool kF16 = std::is_same<MT, __half>::value;
    constexpr float kShift = kF16 ? 15.0f : 0.0f;
    // P is split into two 16-bit terms, so that rounding it adds nothing to the
    // rounding of out (2^-16 against 2^-9 for bf16), except under bf16 outputs
    // of 8-bit caches, where one fp16 term (2^-12) is already finer than out.
    constexpr bool kTwo = !(FP8 && std::is_same<QT, __nv_bfloat16>::value);
    constexpr int kKS = DP / 16, kNT = DP / 8, kPT = T / 8;  // steps along head_dim, products along it, along positions

    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, q4 = lane & 3;
    begin_dependent();

    // Prefix sums of the sequences' tile counts.
    int* pre = reinterpret_cast<int*>(smem + (size_t)NW * (S * 2 * Sh::kTileBytes + Sh::kQBytes));
    for (int i = tid; i < t.batch; i += NW * 32) pre[i + 1] = Tiles(kv_len(t, i, status), a.window, a.sinks, kShift2).count;
    __syncthreads();
    if (warp == 0) prefix_sums(pre, t.batch, lane);
    __syncthreads();
    if (blockIdx.x == 0)
        for (int i = tid; i <= t.batch; i += NW * 32) sc.pre[i] = pre[i];
    if (blockIdx.x == 0 && warp == 0 && sc.pre_all != sc.pre) {
        for (int i = lane; i < t.batch; i += 32) sc.pre_all[i + 1] = (kv_len(t, i, status) + T - 1) >> kShift2;
        __syncwarp();
        prefix_sums(sc.pre_all, t.batch, lane);
    }

    const int total = pre[t.batch] * sc.units;
    const int workers = min((int)gridDim.x * NW, total);
    const int me = warp * gridDim.x + blockIdx.x;  // the first workers are on different SMs
    if (me >= workers) return;
    const Shares shares(total, workers);
    const int t0 = shares.begin(me), n = shares.begin(me + 1) - t0;
    const int parts = sc.units / c.kv_heads;

    // The sequence, unit and tile at t0.
    Cursor cur;
    {
        cur.b = find_sequence(pre, t.batch, sc.units, t0);
        cur.t = Tiles(kv_len(t, cur.b, status), a.window, a.sinks, kShift2);
        const int r = t0 - pre[cur.b] * sc.units, u = r / cur.t.count;
        cur.j = r - u * cur.t.count;
        cur.head = u / parts;
        cur.part = u - cur.head * parts;
    }
    auto advance = [&](Cursor& x) {
        if (++x.j < x.t.count) return;
        x.j = 0;
        if (++x.part < parts) return;
        x.part = 0;
        if (++x.head < c.kv_heads) return;
        x.head = 0;
        do ++x.b; while (x.b < t.batch && pre[x.b + 1] == pre[x.b]);
        if (x.b < t.batch) x.t = Tiles(kv_len(t, x.b, status), a.window, a.sinks, kShift2);
    };

    // ---- the ring: this warp's tiles, filled S - 1 ahead ----
    unsigned char* ring = smem + (size_t)warp * (S * 2 * Sh::kTileBytes);
    const uint32_t ring_a = smem_addr(ring);
    constexpr int kRows = 32 / Sh::kVecs;  // rows per copy instruction
    const int cp_row = lane / Sh::kVecs, cp_v = lane % Sh::kVecs;
    const bool in_row = cp_v * 16 < c.head_dim * Sh::kBytes;
    const int64_t page_bytes = c.page_stride * Sh::kBytes, head_bytes = c.head_stride * Sh::kBytes, slot_bytes = c.slot_stride * Sh::kBytes;
    const int64_t cp_at = cp_row * slot_bytes + cp_v * 16;
    const bool paged_whole = c.page_size % T == 0;  // a tile lies in one page
    uint64_t policy;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    Cursor ld = cur;
    int ld_page = 0, ld_slot = 0;  // page and slot of this lane's row (lane % T) of the next tile, fetched one tile ahead
    auto fetch_page = [&]() {
        const int p = (ld.t.tile(ld.j) << kShift2) + (lane & (T - 1));
        const int index = sc.page.div(p);
        ld_slot = p - index * c.page_size;
        ld_page = ld.b < t.batch && ld.t.visible(p) ? t.pages[(int64_t)ld.b * t.row_stride + index] : -1;
    };
    auto issue = [&](int stage) {
        const uint32_t dst = ring_a + stage * (2 * Sh::kTileBytes);
        const int p0 = ld.t.tile(ld.j) << kShift2;
        const bool good = ld_page >= 0 && ld_page < c.num_pages;
        const int64_t off = ld_page * page_bytes + ld.head * head_bytes + ld_slot * slot_bytes;
        if (paged_whole && ld.t.whole(p0, T) && __all_sync(kFullMask, good)) {
            // every row is there, one slot after the other from row 0's
            const char *pk = c.k + cp_at, *pv = c.v + cp_at;
            const int64_t base = __shfl_sync(kFullMask, off, 0);
            pk += base;
            pv += base;
            const int size = in_row ? 16 : 0;
            if (!in_row) {  // nothing is read there: any address in the pool
                pk = c.k;
                pv = c.v;
            }
            const int64_t step = in_row ? kRows * slot_bytes : 0;
#pragma unroll
            for (int i = 0; i < T / kRows; ++i) {
                const int row = cp_row + i * kRows;
                cp_async16(dst + row * Sh::kRowBytes + k_vec<FP8, DP>(row, cp_v) * 16, pk, size, policy);
                cp_async16(dst + Sh::kTileBytes + row * Sh::kRowBytes + v_vec<FP8, DP>(row, cp_v) * 16, pv, size, policy);
                pk += step;
                pv += step;
            }
            return;
        }
        const bool see = ld.t.visible(p0 + (lane & (T - 1)));
        if (see && !good) record_error(status, kErrKvTable, (uint32_t)(t.first + ld.b));
        const int64_t mine = see && good ? off : -1;
#pragma unroll
        for (int i = 0; i < T / kRows; ++i) {
            const int row = cp_row + i * kRows;
            const int64_t o = __shfl_sync(kFullMask, mine, row);
            const bool ok = o >= 0 && in_row;  // otherwise the vector is filled with zeros
            const int64_t at = ok ? o + cp_v * 16 : 0;
            cp_async16(dst + row * Sh::kRowBytes + k_vec<FP8, DP>(row, cp_v) * 16, c.k + at, ok ? 16 : 0, policy);
            cp_async16(dst + Sh::kTileBytes + row * Sh::kRowBytes + v_vec<FP8, DP>(row, cp_v) * 16, c.v + at, ok ? 16 : 0, policy);
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
        head = cur.head;
        row0 = cur.part * 16;
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
                const int64_t at = (int64_t)cur.b * a.q_heads + head * sc.group;
                if (in[0]) store_lse(sc, a, at + ra, m0 - kShift, la);
                if (in[1]) store_lse(sc, a, at + rb, m1 - kShift, lb);
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

        float x[kPT][4] = {};
        if constexpr (!FP8) {
            const int row = (lane >> 4) * 8 + (lane & 7);
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks) {
                uint32_t f[4];
                q_frag(ks, f);
#pragma unroll
                for (int h = 0; h < kPT / 2; ++h) {
                    uint32_t kf[4];
                    ldmatrix4(kf, kt + (row + 16 * h) * Sh::kRowBytes + k_vec<FP8, DP>(row, 2 * ks + ((lane >> 3) & 1)) * 16);
                    mma16816<MT>(x[2 * h], f, kf[0], kf[1]);
                    mma16816<MT>(x[2 * h + 1], f, kf[2], kf[3]);
                }
            }
        } else {
#pragma unroll
            for (int v = 0; v < DP / 64; ++v) {
                const int vec = q4 * (DP / 64) + v;
                uint4 kw[kPT];
#pragma unroll
                for (int pt = 0; pt < kPT; ++pt) kw[pt] = lds128(kt + (g + 8 * pt) * Sh::kRowBytes + k_vec<FP8, DP>(g, vec) * 16);
#pragma unroll
                for (int i4 = 0; i4 < 4; ++i4) {
                    uint32_t f[4];
                    q_frag(v * 4 + i4, f);
#pragma unroll
                    for (int pt = 0; pt < kPT; ++pt) {
                        const uint32_t w = i4 == 0 ? kw[pt].x : i4 == 1 ? kw[pt].y : i4 == 2 ? kw[pt].z : kw[pt].w;
                        mma16816<MT>(x[pt], f, e4m3x2_f16x2(w), e4m3x2_f16x2(w >> 16));
                    }
                }
            }
        }
        const int p0 = cur.t.tile(cur.j) << kShift2;
        if (cur.t.whole(p0, T)) {
#pragma unroll
            for (int pt = 0; pt < kPT; ++pt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    x[pt][e] *= sl0;
                    x[pt][2 + e] *= sl1;
                }
        } else {
#pragma unroll
            for (int pt = 0; pt < kPT; ++pt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const bool see = cur.t.visible(p0 + 2 * q4 + pt * 8 + e);
                    x[pt][e] = see ? x[pt][e] * sl0 : -INFINITY;
                    x[pt][2 + e] = see ? x[pt][2 + e] * sl1 : -INFINITY;
                }
        }
        if (sc.logits) {
            const int64_t tile = (int64_t)pre[cur.b] * c.kv_heads + (int64_t)head * cur.t.count + cur.j;
            float* to = sc.logits + (tile * sc.group + row0 + g) * T + 2 * q4;
#pragma unroll
            for (int pt = 0; pt < kPT; ++pt) {
                if (row0 + g < sc.group) *reinterpret_cast<float2*>(to + pt * 8) = make_float2(x[pt][0], x[pt][1]);
                if (row0 + g + 8 < sc.group) *reinterpret_cast<float2*>(to + 8 * T + pt * 8) = make_float2(x[pt][2], x[pt][3]);
            }
        }
        float top0 = m0, top1 = m1;
#pragma unroll
        for (int pt = 0; pt < kPT; ++pt) {
            top0 = fmaxf(top0, fmaxf(x[pt][0], x[pt][1]));
            top1 = fmaxf(top1, fmaxf(x[pt][2], x[pt][3]));
        }
#pragma unroll
        for (int s = 1; s < 4; s <<= 1) {
            top0 = fmaxf(top0, __shfl_xor_sync(kFullMask, top0, s));
            top1 = fmaxf(top1, __shfl_xor_sync(kFullMask, top1, s));
        }
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
                ph[k * 2] = pack2<MT>(a0, a1);
                ph[k * 2 + 1] = pack2<MT>(b0, b1);
                if constexpr (kTwo) {
                    const float2 ra = open2<MT>(ph[k * 2]), rb = open2<MT>(ph[k * 2 + 1]);
                    pl[k * 2] = pack2<MT>(a0 - ra.x, a1 - ra.y);
                    pl[k * 2 + 1] = pack2<MT>(b0 - rb.x, b1 - rb.y);
                }
            }
            const uint32_t vh = vt + 16 * h * Sh::kRowBytes;
            if constexpr (!FP8) {
                const int row = ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
                for (int nt = 0; nt < kNT; nt += 2) {
                    uint32_t vf[4];
                    ldmatrix4_t(vf, vh + row * Sh::kRowBytes + v_vec<FP8, DP>(row, nt + (lane >> 4)) * 16);
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
                        w[k] = lds64(vh + row * Sh::kRowBytes + v_vec<FP8, DP>(row, g >> 1) * 16 + (g & 1) * 8);
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
                            w[k] = lds128(vh + row * Sh::kRowBytes + v_vec<FP8, DP>(row, g * (DP / 128) + v) * 16);
                        }
                        four(v * 16, w[0].x, w[1].x, w[2].x, w[3].x);
                        four(v * 16 + 4, w[0].y, w[1].y, w[2].y, w[3].y);
                        four(v * 16 + 8, w[0].z, w[1].z, w[2].z, w[3].z);
                        four(v * 16 + 12, w[0].w, w[1].w, w[2].w, w[3].w);
                    }
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

// ---- the second and third launch: joins, empty rows, weights ----

// The parts of one unit's rows: workers [w0, w0 + count); one worker: whole.
struct Parts {
    int w0, count;
    // `before` tiles precede the sequence in a unit's list, it has `tiles`, all sequences have `all`.
    __device__ __forceinline__ Parts(const Scratch& sc, int before, int tiles, int all, int unit) {
        const int total = all * sc.units;
        const Shares shares(total, min(sc.workers, total));
        const int s0 = before * sc.units + unit * tiles;
        w0 = shares.holder(s0);
        count = shares.holder(s0 + tiles - 1) - w0 + 1;
    }
    // The first part is its worker's last row, the others are their workers' first ones.
    __device__ __forceinline__ int slot(int i) const { return (w0 + i) * 2 + (i == 0 ? 1 : 0); }
};

__device__ __forceinline__ float rescale(float from, float to) { return from == -INFINITY ? 0.0f : exp2_fast(from - to); }

// One warp's share of a row's join: the parts team, team + teams, ..., with
// every load independent of the others.
template <int DP> struct RowSum {
    static constexpr int kVec = (DP + 127) / 128;
    float4 x[kVec];
    float top, l;
    __device__ __forceinline__ void add(const Scratch& sc, const Parts& p, int row, int team, int teams, int lane) {
        top = -INFINITY;
        l = 0.0f;
#pragma unroll
        for (int k = 0; k < kVec; ++k) x[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        constexpr int kAhead = DP == 256 ? 4 : 8;
        for (int i0 = team; i0 < p.count; i0 += teams * kAhead) {
            float2 ml[kAhead];
            float4 y[kAhead][kVec];
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                const int i = i0 + q * teams;
                ml[q] = make_float2(-INFINITY, 0.0f);
                if (i < p.count) ml[q] = sc.ml[p.slot(i) * 16 + row];
#pragma unroll
                for (int k = 0; k < kVec; ++k) {
                    y[q][k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (i < p.count && lane + k * 32 < DP / 4)
                        y[q][k] = reinterpret_cast<const float4*>(sc.o + ((int64_t)p.slot(i) * sc.rows + row) * DP)[lane + k * 32];
                }
            }
            float up = top;
#pragma unroll
            for (int q = 0; q < kAhead; ++q) up = fmaxf(up, ml[q].x);
            const float f = rescale(top, up);
            l *= f;
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
                x[k].x *= f;
                x[k].y *= f;
                x[k].z *= f;
                x[k].w *= f;
            }
            top = up;
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                const float e = rescale(ml[q].x, up);
                l += e * ml[q].y;
#pragma unroll
                for (int k = 0; k < kVec; ++k) {
                    x[k].x += e * y[q][k].x;
                    x[k].y += e * y[q][k].y;
                    x[k].z += e * y[q][k].z;
                    x[k].w += e * y[q][k].w;
                }
            }
        }
    }
};

constexpr int kTeamParts = 16;  // rows of more parts than this are joined by a whole CTA

// The second launch finishes the rows that were cut and those without a
// visible position: `per` rows a CTA, 1 or one per warp.
template <typename QT, int DP>
__global__ void __launch_bounds__(kJoinThreads) k_kv_join(KvPages c, KvTable t, KvAttention a, Scratch sc, int per) {
    __shared__ float4 s_o[kJoinWarps][DP / 4];
    __shared__ float2 s_ml[kJoinWarps];
    begin_dependent();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int units_per_head = sc.units / c.kv_heads;
    const int rows = t.batch * a.q_heads, all = sc.pre[t.batch];
    auto unit = [&](int j) { return j / sc.group * units_per_head + j % sc.group / 16; };
    // Adds up the sums of warps [w, w + n) and writes dimensions d0, d0 + step, ... of row r.
    auto store = [&](int r, int w, int n, int d0, int step) {
        const int b = r / a.q_heads, j = r % a.q_heads;
        float top = -INFINITY, l = 0.0f;
        for (int i = w; i < w + n; ++i) top = fmaxf(top, s_ml[i].x);
        for (int i = w; i < w + n; ++i) l += s_ml[i].y * rescale(s_ml[i].x, top);
        const float vs = c.v_scale ? c.v_scale[j / sc.group] : 1.0f;
        const float inv = l == 0.0f ? 0.0f : vs / l;
        QT* out = static_cast<QT*>(a.out) + (int64_t)b * a.out_seq_stride + (int64_t)j * a.out_head_stride;
        for (int d = d0; d < c.head_dim; d += step) {
            float x = 0.0f;
            for (int i = w; i < w + n; ++i) x += reinterpret_cast<const float*>(s_o[i])[d] * rescale(s_ml[i].x, top);
            out[d] = from_f32<QT>(l == 0.0f ? 0.0f : x * inv);
        }
        if (d0 == 0) store_lse(sc, a, r, top, l);
    };
    auto keep = [&](const RowSum<DP>& sum) {
#pragma unroll
        for (int k = 0; k < RowSum<DP>::kVec; ++k)
            if (lane + k * 32 < DP / 4) s_o[warp][lane + k * 32] = sum.x[k];
        if (lane == 0) s_ml[warp] = make_float2(sum.top, sum.l);
    };
    // Each warp looks at its row; long joins are left to the whole CTA.
    const int r = blockIdx.x * per + (per == 1 ? 0 : warp);
    bool wide = false;
    if (r < rows && (per > 1 || warp == 0)) {
        const int b = r / a.q_heads, j = r % a.q_heads, before = sc.pre[b], tiles = sc.pre[b + 1] - before;
        if (tiles == 0) {  // no visible position
            QT* out = static_cast<QT*>(a.out) + (int64_t)b * a.out_seq_stride + (int64_t)j * a.out_head_stride;
            for (int d = lane; d < c.head_dim; d += 32) out[d] = from_f32<QT>(0.0f);
            if (lane == 0 && a.lse) a.lse[r] = -INFINITY;
        } else {
            const Parts p(sc, before, tiles, all, unit(j));
            wide = p.count > (per == 1 ? 1 : kTeamParts);
            if (!wide && p.count > 1) {
                RowSum<DP> sum;
                sum.add(sc, p, j % sc.group % 16, 0, 1, lane);
                keep(sum);
                __syncwarp();
                store(r, warp, 1, lane, 32);
            }
        }
    }
    if (!__syncthreads_or(wide)) return;
    for (int k = 0; k < per; ++k) {
        if (!__syncthreads_or(wide && warp == k)) continue;
        const int rk = blockIdx.x * per + k, b = rk / a.q_heads, j = rk % a.q_heads, before = sc.pre[b];
        RowSum<DP> sum;
        sum.add(sc, Parts(sc, before, sc.pre[b + 1] - before, all, unit(j)), j % sc.group % 16, warp, kJoinWarps, lane);
        keep(sum);
        __syncthreads();
        store(rk, 0, kJoinWarps, tid, kJoinThreads);
    }
}

// The third launch, where weights are kept: every thread takes V consecutive
// positions of one tile, and every tile finds its sequence and head by itself,
// so that short sequences cost no more than long ones.  Accumulated in place,
// only visible positions change.
template <int V>
__global__ void __launch_bounds__(kWeightThreads) k_kv_weights(KvPages c, KvTable t, KvAttention a, Scratch sc, uint32_t* status) {
    __shared__ int s_pre[kMaxBatch<0> + 1];
    begin_dependent();
    for (int i = threadIdx.x; i <= t.batch; i += kWeightThreads) s_pre[i] = sc.pre_all[i];
    __syncthreads();
    const bool only_visible = sc.pre_all == sc.pre;
    const int T = 1 << sc.shift, total = s_pre[t.batch] * c.kv_heads;
    const int per_tile = T / V;
    const int64_t end = (int64_t)total * per_tile;
    for (int64_t at = (int64_t)blockIdx.x * kWeightThreads + threadIdx.x; at < end; at += (int64_t)gridDim.x * kWeightThreads) {
        const int tile_at = (int)(at / per_tile), in = (int)(at % per_tile) * V;
        const int b = find_sequence(s_pre, t.batch, c.kv_heads, tile_at);
        const int tiles = s_pre[b + 1] - s_pre[b];
        const int in_b = tile_at - s_pre[b] * c.kv_heads, h = in_b / tiles, j = in_b - h * tiles;
        const Tiles tl(kv_len(t, b, status), a.window, a.sinks, sc.shift);
        const int tile = only_visible ? tl.tile(j) : j;
        const int p = (tile << sc.shift) + in;
        if (p >= tl.len) continue;
        const int index = sc.page.div(p);
        const int page = kv_page(t, c.num_pages, b, index, status);
        if (page < 0) continue;
        const int64_t to = ((int64_t)page * c.kv_heads + h) * c.page_size + (p - index * c.page_size);
        float w[V], old[V];
#pragma unroll
        for (int e = 0; e < V; ++e) w[e] = old[e] = 0.0f;
        if constexpr (V == 4) {  // positions of one page, 16-byte aligned
            if (a.weight_in) {
                const float4 z = *reinterpret_cast<const float4*>(a.weight_in + to);
                old[0] = z.x; old[1] = z.y; old[2] = z.z; old[3] = z.w;
            }
        } else {
            if (a.weight_in) old[0] = a.weight_in[to];
        }
        if (tile < tl.nsink || tile >= tl.first) {  // the tile has scores
            const int before = only_visible ? s_pre[b] : sc.pre[b];
            const int64_t jv = (int64_t)before * c.kv_heads + (int64_t)h * tl.count + (tile < tl.nsink ? tile : tl.nsink + tile - tl.first);
            const float* x = sc.logits + jv * sc.group * T + in;
            const float* lse = sc.lse2 + (int64_t)b * a.q_heads + h * sc.group;
#pragma unroll 4
            for (int r = 0; r < sc.group; ++r) {
                const float z = lse[r];
                if constexpr (V == 4) {
                    const float4 y = __ldcs(reinterpret_cast<const float4*>(x + r * T));
                    w[0] += exp2_fast(y.x - z);
                    w[1] += exp2_fast(y.y - z);
                    w[2] += exp2_fast(y.z - z);
                    w[3] += exp2_fast(y.w - z);
                } else {
                    w[0] += exp2_fast(__ldcs(x + r * T) - z);
                }
            }
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (!tl.visible(p + e)) w[e] = 0.0f;  // also where a NaN row makes 2^(-inf - NaN)
        }
        if constexpr (V == 4) {
            if (p + 3 < tl.len) {
                *reinterpret_cast<float4*>(a.weight_out + to) = make_float4(old[0] + w[0], old[1] + w[1], old[2] + w[2], old[3] + w[3]);
                continue;
            }
        }
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (p + e < tl.len) a.weight_out[to + e] = old[e] + w[e];
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

Plan make_plan(const KvPages& c, const KvTable& t, const KvAttention& a, int most_batch, int warps, int dp, int tile, int sms) {
    Plan p{};
    p.dp = dp;
    p.warps = warps;
    p.sc.group = a.q_heads / c.kv_heads;
    p.sc.units = c.kv_heads * ((p.sc.group + 15) / 16);
    p.sc.rows = p.sc.group < 16 ? p.sc.group : 16;
    const size_t tiles = ((size_t)t.max_len + tile - 1) / tile;  // of one sequence and unit, at most
    const size_t seq_logits = a.weight_out ? tiles * a.q_heads * tile * 4 : 0;
    size_t batch = t.batch < most_batch ? t.batch : most_batch;
    if (seq_logits * batch > kMaxLogits) batch = kMaxLogits / seq_logits;
    while (batch > 1 && batch * tiles * p.sc.units > 0x7fffffff) batch /= 2;  // lists are counted in 32 bits
    p.batch = batch < 1 ? 1 : (int)batch;
    const size_t most = (size_t)p.batch * tiles * p.sc.units;
    p.grid = most < (size_t)sms ? (most < 1 ? 1 : (int)most) : sms;
    p.sc.workers = p.grid * warps;
    p.sc.shift = tile == 16 ? 4 : 5;
    p.sc.page = FastDiv(c.page_size);
    p.at_lse2 = 2 * round256(((size_t)p.batch + 1) * 4);
    p.at_ml = p.at_lse2 + round256((size_t)p.batch * a.q_heads * 4);
    p.at_o = p.at_ml + round256((size_t)p.sc.workers * 2 * 16 * 8);
    p.at_logits = p.at_o + round256((size_t)p.sc.workers * 2 * p.sc.rows * dp * 4);
    p.bytes = p.at_logits + round256(seq_logits * p.batch);
    return p;
}

template <typename QT, bool FP8, int DP, int T, int NW, int S>
cudaError_t run(const KvPages& c, const KvTable& t, const KvAttention& a, void* scratch, size_t* bytes, uint32_t* status, cudaStream_t s) {
    auto* kern = k_kv_attend<QT, FP8, DP, T, NW, S>;
    constexpr size_t smem = Shape<FP8, DP, T, NW, S>::kSmem;
    static_assert(smem <= 227 * 1024, "the ring does not fit in shared memory");
    KernelSetup su;
    cudaError_t e = kernel_setup(reinterpret_cast<const void*>(kern), NW * 32, smem, &su);
    if (e != cudaSuccess) return e;
    Plan p = make_plan(c, t, a, kMaxBatch<DP>, NW, DP, T, su.sms);
    if (scratch == nullptr) {
        *bytes = p.bytes;
        return cudaSuccess;
    }
    char* base = static_cast<char*>(scratch);
    p.sc.pre = reinterpret_cast<int*>(base);
    p.sc.pre_all = p.sc.pre;
    if (a.window > 0 && a.weight_out && a.weight_in != a.weight_out) p.sc.pre_all = reinterpret_cast<int*>(base + p.at_lse2 / 2);
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
        e = launch_dependent(kern, p.grid, NW * 32, smem, 1, s, c, u, v, p.sc, status);
        if (e != cudaSuccess) return e;
        // One row per warp, except where rows are few, or have so many parts on
        // average that a whole CTA joins each.
        const int rows = u.batch * a.q_heads;
        const int per = rows <= 2 * su.sms || p.sc.workers > kTeamParts * u.batch * p.sc.units ? 1 : kJoinWarps;
        e = launch_dependent(k_kv_join<QT, DP>, (rows + per - 1) / per, kJoinThreads, 0, 1, s, c, u, v, p.sc, per);
        if (e != cudaSuccess) return e;
        if (a.weight_out == nullptr) continue;
        const bool vec4 = c.page_size % 4 == 0 && ((reinterpret_cast<uintptr_t>(a.weight_in) | reinterpret_cast<uintptr_t>(a.weight_out)) & 15u) == 0;
        const size_t tiles = ((size_t)t.max_len + T - 1) / T * u.batch * c.kv_heads;
        const size_t blocks = (tiles * (vec4 ? T / 4 : T) + kWeightThreads - 1) / kWeightThreads, most = (size_t)su.sms * 8;
        e = launch_dependent(vec4 ? k_kv_weights<4> : k_kv_weights<1>, blocks < most ? blocks < 1 ? 1 : blocks : most, kWeightThreads, 0, 1, s, c, u, v, p.sc, status);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// Tile, warps and stages by row size: the ring takes about 192 KB of the SM,
// and the warps as many as their registers allow.  8-bit rows take tiles of 32
// positions, which spreads a tile's fixed instructions over as many bytes.
template <typename QT, bool FP8>
cudaError_t run_dim(const KvPages& c, const KvTable& t, const KvAttention& a, void* scratch, size_t* bytes, uint32_t* status, cudaStream_t s) {
    if (c.head_dim <= 64) return run<QT, FP8, 64, 32, FP8 ? 12 : 8, FP8 ? 4 : 3>(c, t, a, scratch, bytes, status, s);
    if (c.head_dim <= 128) return run<QT, FP8, 128, FP8 ? 32 : 16, 8, 3>(c, t, a, scratch, bytes, status, s);
    return run<QT, FP8, 256, 16, FP8 ? 7 : 4, 3>(c, t, a, scratch, bytes, status, s);
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
