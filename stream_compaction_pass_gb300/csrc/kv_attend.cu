// kv_attend.cu -- attention of one new token per sequence over a paged
// key-value cache (streamscan.h, ss_kv_attend), split over the cache's length
// and joined, in two launches, and a third where weights are kept; small calls
// take one.
//
// Mathematics.  With X = (q . k) scale log2 e and a running reference R per
// query head, P = 2^(X - R), l += sum P, O += P V, and l and O shrink by
// 2^(R_old - R_new) where R grows (kv_rows.cuh).  Parts of one row over
// disjoint positions join by the same rule: R = max R_i, l = sum l_i 2^(R_i - R),
// O = sum O_i 2^(R_i - R); out = O / l and lse = (R + log2 l) ln 2.
//
// What bounds it.  Every key and value byte is read once from device memory
// and serves `group` query heads: 4 group / (element bytes) flops a byte, far
// below the ridge, so the kernel is a stream of 16-byte asynchronous copies
// that the arithmetic has to stay under.  64 sequences of 155 thousand
// positions in all (8 x 4 heads of 128, bf16): 102 us for 634 MB, 6.2 TB/s,
// tensor pipe 12 %; without the arithmetic about 4 us less.
//
// Split.  The tiles of every (sequence, unit), a unit being 8 or 16 query
// heads of one key-value head, form one long list; a warp takes one contiguous
// share of it, all shares equal to within a tile, whatever the lengths are.  So
// a single long sequence and a ragged batch both fill every SM, and the host
// needs no lengths.  A warp works alone: it owns a ring of tiles in shared
// memory that only it fills and reads, so the main loop has no barrier.  Rows
// that lie within one warp's share are written at once; a share's first and
// last row may be parts, which go to scratch, and the second launch joins
// them (7 us for 2048 rows of 3.6 parts).  Where weights are kept, the first
// launch leaves X (fp32) in scratch and the third turns it into weights, since
// they need the joined sums (10 us for 1.2 million positions x 4 heads).
#include <cooperative_groups.h>

#include <algorithm>

#include "kv_rows.cuh"

namespace ss {

namespace {

// Sequences per launch: their tile counts' prefix sums are in shared memory,
// beside a ring that leaves little of it at head_dim 256.
template <int DP> constexpr int kMaxBatch = DP == 256 ? 512 : 4096;

namespace cg = cooperative_groups;

// Tiles of a warp up to which a call whose units fit the GPU takes the form of
// one launch, without and with weights (which that form adds up with the same
// warps).  Measured, one launch against three, in us:
//   8 heads of 128, bf16: 1 x 16000 positions (10 tiles) 15.1 / 16.7, 1 x 32000
//     (21) 26.2 / 30.0, 1 x 48000 (31) 37.2 / 39.3; with weights 1 x 8000 (5)
//     14.6 / 17.3, 1 x 16000 22.5 / 20.0, 4 x 8000 (10, on twice the SMs) 31.7 /
//     33.2, 1 x 32000 41.3 / 35.4, 1 head x 16000 22.2 / 23.8.
// 8-bit rows, groups above 8 and head_dim 256, whose tiles take a warp longer or
// whose CTAs have fewer warps (`slow`), have lower limits, but where the clusters
// hold three quarters of the SMs:
//   8-bit: 1 x 16000 (5) 16.9 / 20.6, 1 x 32000 (10) 25.0 / 23.2, 1 x 64000 41.5
//     / 32.9, 4 x 16000 (10) 26.9 / 31.8; with weights 1 x 8000 (3) 18.0 / 22.8,
//     1 x 16000 27.1 / 24.9, 1 x 32000 43.0 / 27.8, 4 x 8000 (5) 27.4 / 27.8.
//   256: 1 x 4000 (8) 11.5 / 13.1, 1 x 8000 (16) 18.0 / 15.2, 32 x 1000 (16) 23.4
//     / 31.4; with weights 1 x 2000 (4) 11.3 / 13.1, 1 x 6000 (12) 22.2 / 16.9.
//   group 12: 1 x 8000 (8) 13.8 / 16.8, 1 x 16000 (16) 21.1 / 17.7, 32 x 2000 (16)
//     24.2 / 33.9; with weights 4 x 2000 (4) 15.6 / 16.8, 4 x 4000 (8) 24.3 / 19.5.
struct SmallLimits {
    int few, many;  // on fewer SMs, and on three quarters of them
};
constexpr SmallLimits small_limits(bool slow, bool weights) {
    return slow ? (weights ? SmallLimits{5, 8} : SmallLimits{12, 24}) : weights ? SmallLimits{12, 12} : SmallLimits{24, 24};
}
constexpr int kSmallTiles = 24;  // the largest of them
constexpr int kJoinThreads = 512;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kWeightThreads = 256;
constexpr size_t kMaxLogits = (size_t)2 << 30;  // bytes of scores one launch may leave in scratch

struct Scratch {
    int* pre;       // batch + 1: tiles of the sequences before, per unit
    int* pre_all;   // the same of all positions, where those that are not visible get a weight too (else pre)
    float* lse2;    // batch x q_heads: R + log2 l of every row, for the weights
    float2* ml;     // workers x 2 x 16: (R, l) of a part
    float* o;       // workers x 2 x rows x DP: its O
    void* aside;    // workers: O of the row at hand while it is long (kv_rows.cuh)
    float* logits;  // per (sequence, key-value head) tile: group x 16 scores, log2 units; or null
    int group, units, rows, workers;  // units per sequence, of `heads` query heads; rows = min(group, heads)
    int heads;
    int ranks, max_tiles;             // small calls: CTAs of a unit's cluster, tiles of the longest sequence
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

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::128B [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes), "l"(policy) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

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

// The sum of row `at` (sequence * q_heads + head): R and l.  A row without
// weights leaves +inf for the weights' pass, where 2^(X - inf) = 0.
__device__ __forceinline__ void store_lse(const Scratch& sc, const KvAttention& a, int64_t at, float ref, float l) {
    const float x = ref + log2f(l);
    sc.lse2[at] = l == 0.0f ? INFINITY : x;
    if (a.lse) a.lse[at] = l == 0.0f ? -INFINITY : x * 0.6931471805599453f;
}

// Outputs of a row without a visible position.
template <typename QT> __device__ __forceinline__ void empty_row(const KvAttention& a, int b, int j, int dim, int first, int step) {
    QT* out = static_cast<QT*>(a.out) + (int64_t)b * a.out_seq_stride + (int64_t)j * a.out_head_stride;
    for (int d = first; d < dim; d += step) out[d] = from_f32<QT>(0.0f);
    if (first == 0 && a.lse) a.lse[(int64_t)b * a.q_heads + j] = -INFINITY;
}

// A part's O and l, by their factor.
__device__ __forceinline__ void add_part(float4& x, float& l, const float4& y, float l_part, float factor) {
    l += l_part * factor;
    x.x += y.x * factor;
    x.y += y.y * factor;
    x.z += y.z * factor;
    x.w += y.w * factor;
}

// A place in the list of tiles: sequence, key-value head, part of its group (8
// or 16 query heads), tile.
struct Cursor {
    int b, head, part, j;
    Tiles t;
    __device__ __forceinline__ Cursor() : b(0), head(0), part(0), j(0), t(0, 0, 0, 0) {}
};

// DP: head_dim rounded up to 64, 128 or 256 (the rest is zeros in shared
// memory).  T positions per tile (16 or 32), NW warps of a CTA, S stages of
// each warp's ring.  Rows: Rows8 or Rows16.
template <typename Rows, bool FP8, int DP, int T, int NW, int S>
struct Shape {
    static constexpr int kBytes = FP8 ? 1 : 2;
    static constexpr int kRowBytes = DP * kBytes;
    static constexpr int kVecs = kRowBytes / 16;
    static constexpr int kTileBytes = T * kRowBytes;  // of k, and of v
    static constexpr int kRing = S * 2 * kTileBytes;  // of a warp
    static constexpr size_t kSmem = (size_t)NW * (kRing + Rows::kQBytes) + (kMaxBatch<DP> + 1) * 4;
};

// SMALL: a call of few rows, a cluster of CTAs each.  The warps of a cluster
// share one unit's tiles; the parts are joined through shared memory, first of
// the CTA and then of the cluster, and the same warps add their tiles' weights:
// one launch in all.
template <typename Rows, bool FP8, int DP, int T, int NW, int S, bool SMALL>
__global__ void __launch_bounds__(NW * 32, 1) k_kv_attend(KvPages c, KvTable t, KvAttention a, Scratch sc, uint32_t* status) {
    using Sh = Shape<Rows, FP8, DP, T, NW, S>;
    constexpr int kShift2 = T == 16 ? 4 : 5;
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    begin_dependent();

    Cursor cur;
    int n, me = 0;
    const int parts = sc.units / c.kv_heads;
    int* pre = reinterpret_cast<int*>(smem + (size_t)NW * (Sh::kRing + Rows::kQBytes));
    if constexpr (SMALL) {
        const int row = blockIdx.x / sc.ranks, unit_no = row % sc.units;
        cur.b = row / sc.units;
        cur.t = Tiles(kv_len(t, cur.b, status), a.window, a.sinks, kShift2);
        cur.head = unit_no / parts;
        cur.part = unit_no % parts;
        if (cur.t.count == 0) {  // no visible position: the same for the whole cluster
            const int j0 = cur.head * sc.group + cur.part * Rows::kHeads, rows = min(Rows::kHeads, sc.group - cur.part * Rows::kHeads);
            for (int r = blockIdx.x % sc.ranks; r < rows; r += sc.ranks) empty_row<typename Rows::Query>(a, cur.b, j0 + r, c.head_dim, tid, NW * 32);
            return;
        }
        const int workers = min(sc.ranks * NW, cur.t.count);
        me = warp * sc.ranks + blockIdx.x % sc.ranks;
        const Shares shares(cur.t.count, workers);
        cur.j = me < workers ? shares.begin(me) : 0;
        n = me < workers ? shares.begin(me + 1) - cur.j : 0;
    } else {
        // Prefix sums of the sequences' tile counts.
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
        me = warp * gridDim.x + blockIdx.x;  // the first workers are on different SMs
        if (me >= workers) return;
        const Shares shares(total, workers);
        const int t0 = shares.begin(me);
        n = shares.begin(me + 1) - t0;

        // The sequence, unit and tile at t0.
        cur.b = find_sequence(pre, t.batch, sc.units, t0);
        cur.t = Tiles(kv_len(t, cur.b, status), a.window, a.sinks, kShift2);
        const int r = t0 - pre[cur.b] * sc.units, u = r / cur.t.count;
        cur.j = r - u * cur.t.count;
        cur.head = u / parts;
        cur.part = u - cur.head * parts;
    }
    auto advance = [&](Cursor& x) {
        if (++x.j < x.t.count || SMALL) return;
        x.j = 0;
        if (++x.part < parts) return;
        x.part = 0;
        if (++x.head < c.kv_heads) return;
        x.head = 0;
        do ++x.b; while (x.b < t.batch && pre[x.b + 1] == pre[x.b]);
        if (x.b < t.batch) x.t = Tiles(kv_len(t, x.b, status), a.window, a.sinks, kShift2);
    };

    // ---- the ring: this warp's tiles, filled S - 1 ahead ----
    const uint32_t ring_a = smem_addr(smem) + warp * Sh::kRing;
    const uint32_t queries = smem_addr(smem) + NW * Sh::kRing + warp * Rows::kQBytes;
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
    Rows rows;
    Unit unit{};
    bool began = false;  // whether this row started in this share
    int chain = 0;       // tiles since the row began, or since its O was set aside
    bool aside = false;
    auto open_row = [&]() {
        chain = 0;
        aside = false;
        unit = Unit{cur.b, cur.head, cur.part * Rows::kHeads, sc.group};
        began = cur.j == 0;
        rows.open(c, a, unit, queries, lane);
    };
    auto close_row = [&](bool ended) {
        if (aside) add_aside(rows, static_cast<const Aside<Rows>*>(sc.aside)[me], lane);
        rows.gather();
        if (began && ended) {
            const int64_t at = (int64_t)unit.b * a.q_heads + unit.head * sc.group + unit.row0;
            rows.store_out(a, unit, FP8 && c.v_scale ? c.v_scale[unit.head] : 1.0f, c.head_dim, lane);
            rows.each_sum(unit, lane, [&](int r, float ref, float l) { store_lse(sc, a, at + r, ref, l); });
            return;
        }
        const int slot = me * 2 + (began ? 1 : 0);
        rows.store_part(sc.o + (int64_t)slot * sc.rows * DP, unit, lane);
        rows.each_sum(unit, lane, [&](int r, float ref, float l) { sc.ml[slot * 16 + r] = make_float2(ref, l); });
    };

    auto tile_number = [&](const Cursor& x) -> int64_t {  // where its scores are
        if constexpr (SMALL) return ((int64_t)x.b * c.kv_heads + x.head) * sc.max_tiles + x.j;
        return (int64_t)pre[x.b] * c.kv_heads + (int64_t)x.head * x.t.count + x.j;
    };

    open_row();
    [[maybe_unused]] const int first = cur.j;
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
        const uint32_t kt = ring_a + stage * (2 * Sh::kTileBytes);
        stage = stage + 1 == S ? 0 : stage + 1;
        float* scores = nullptr;
        if (sc.logits) scores = sc.logits + (tile_number(cur) * sc.group + unit.row0) * T;
        rows.tile(kt, kt + Sh::kTileBytes, queries, cur.t, cur.t.tile(cur.j) << kShift2, scores, unit, lane);
        if (!SMALL && cur.j + 1 == cur.t.count) {
            close_row(true);
            advance(cur);
            if (i + 1 < n) open_row();
        } else {
            advance(cur);
            if constexpr (!SMALL) {
                if (++chain == Rows::kChain) {
                    put_aside(rows, static_cast<Aside<Rows>*>(sc.aside)[me], aside, lane);
                    chain = 0;
                    aside = true;
                }
                if (i + 1 == n) close_row(false);
            }
        }
    }
    cp_wait<0>();

    if constexpr (SMALL) {
        // Parts of the warps, then of the CTA, over the rings' shared memory.
        cg::cluster_group cluster = cg::this_cluster();
        const int nrows = min(Rows::kHeads, sc.group - unit.row0), rank = blockIdx.x % sc.ranks;
        float* w_o = reinterpret_cast<float*>(smem);             // NW x rows x DP
        float* c_o = w_o + NW * Rows::kHeads * DP;               // rows x DP
        float2* w_ml = reinterpret_cast<float2*>(c_o + Rows::kHeads * DP);  // NW x rows
        float2* c_ml = w_ml + NW * Rows::kHeads;                 // rows
        float* s_lse = reinterpret_cast<float*>(c_ml + Rows::kHeads);
        static_assert((size_t)(NW + 1) * Rows::kHeads * (DP * 4 + 8) + Rows::kHeads * 4 <= (size_t)NW * Sh::kRing, "the parts fit in the rings");
        rows.gather();
        __syncthreads();
        rows.store_part(w_o + warp * Rows::kHeads * DP, unit, lane);
        rows.each_sum(unit, lane, [&](int r, float ref, float l) { w_ml[warp * Rows::kHeads + r] = make_float2(ref, l); });
        __syncthreads();
        for (int i = tid; i < nrows * (DP / 4); i += NW * 32) {
            const int r = i / (DP / 4), d = i % (DP / 4);
            float top = -INFINITY, l = 0.0f;
            for (int w = 0; w < NW; ++w) top = fmaxf(top, w_ml[w * Rows::kHeads + r].x);
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int w = 0; w < NW; ++w) {
                const float2 ml = w_ml[w * Rows::kHeads + r];
                add_part(x, l, reinterpret_cast<const float4*>(w_o + (w * Rows::kHeads + r) * DP)[d], ml.y, shrink(ml.x, top));
            }
            reinterpret_cast<float4*>(c_o + r * DP)[d] = x;
            if (d == 0) c_ml[r] = make_float2(top, l);
        }
        cluster.sync();
        const float vs = FP8 && c.v_scale ? c.v_scale[unit.head] : 1.0f;
        const int64_t row0 = (int64_t)unit.b * a.q_heads + unit.head * sc.group + unit.row0;
        for (int i = rank * (NW * 32) + tid; i < nrows * (DP / 4); i += sc.ranks * (NW * 32)) {
            const int r = i / (DP / 4), d = i % (DP / 4);
            float top = -INFINITY, l = 0.0f;
            for (int k = 0; k < sc.ranks; ++k) top = fmaxf(top, cluster.map_shared_rank(c_ml, k)[r].x);
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int k = 0; k < sc.ranks; ++k) {
                const float2 ml = cluster.map_shared_rank(c_ml, k)[r];
                add_part(x, l, reinterpret_cast<const float4*>(cluster.map_shared_rank(c_o, k) + r * DP)[d], ml.y, shrink(ml.x, top));
            }
            using QT = typename Rows::Query;
            const float inv = l == 0.0f ? 0.0f : vs / l;
            if (l == 0.0f) x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            QT* out = static_cast<QT*>(a.out) + (int64_t)unit.b * a.out_seq_stride + (int64_t)(unit.head * sc.group + unit.row0 + r) * a.out_head_stride;
            if (4 * d < c.head_dim) *reinterpret_cast<uint2*>(out + 4 * d) = make_uint2(pack2<QT>(x.x * inv, x.y * inv), pack2<QT>(x.z * inv, x.w * inv));
            if (d == 0 && a.lse) a.lse[row0 + r] = l == 0.0f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
        }
        if (a.weight_out) {
            if (tid < nrows) {
                float top = -INFINITY, l = 0.0f;
                for (int k = 0; k < sc.ranks; ++k) top = fmaxf(top, cluster.map_shared_rank(c_ml, k)[tid].x);
                for (int k = 0; k < sc.ranks; ++k) {
                    const float2 ml = cluster.map_shared_rank(c_ml, k)[tid];
                    l += ml.y * shrink(ml.x, top);
                }
                s_lse[tid] = l == 0.0f ? INFINITY : top + log2f(l);
            }
            __syncthreads();
            auto add = [&](int p, float w) {
                const int index = sc.page.div(p), page = kv_page(t, c.num_pages, unit.b, index, status);
                if (page < 0) return;
                const int64_t at = ((int64_t)page * c.kv_heads + unit.head) * c.page_size + (p - index * c.page_size);
                a.weight_out[at] = (a.weight_in ? a.weight_in[at] : 0.0f) + w;
            };
            // the scores of this warp's own tiles
            for (int i = lane; i < n * T; i += 32) {
                const int j = first + i / T, p = (cur.t.tile(j) << kShift2) + i % T;
                if (!cur.t.visible(p)) continue;
                Cursor x = cur;
                x.j = j;
                const float* score = sc.logits + tile_number(x) * sc.group * T + i % T;
                float w = 0.0f;
                for (int r = 0; r < nrows; ++r) w += exp2_fast(score[r * T] - s_lse[r]);
                add(p, w);
            }
            if (a.weight_in != a.weight_out && a.window > 0)
                for (int p = rank * (NW * 32) + tid; p < cur.t.len; p += sc.ranks * (NW * 32))
                    if (!cur.t.visible(p)) add(p, 0.0f);
        }
        cluster.sync();  // no CTA leaves while another may read its shared memory
    }
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
            const float f = shrink(top, up);
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
                const float e = shrink(ml[q].x, up);
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

// The second launch finishes the rows that were cut and those without a
// visible position: a team of TEAM warps (1, 4 or all 16) a row.
template <typename QT, int DP, int TEAM>
__global__ void __launch_bounds__(kJoinThreads) k_kv_join(KvPages c, KvTable t, KvAttention a, Scratch sc) {
    __shared__ float4 s_o[kJoinWarps][DP / 4];
    __shared__ float2 s_ml[kJoinWarps];
    begin_dependent();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int units_per_head = sc.units / c.kv_heads;
    const int rows = t.batch * a.q_heads, all = sc.pre[t.batch];
    constexpr int kPer = kJoinWarps / TEAM;
    auto unit = [&](int j) { return j / sc.group * units_per_head + j % sc.group / sc.heads; };
    auto keep = [&](const RowSum<DP>& sum) {
#pragma unroll
        for (int k = 0; k < RowSum<DP>::kVec; ++k)
            if (lane + k * 32 < DP / 4) s_o[warp][lane + k * 32] = sum.x[k];
        if (lane == 0) s_ml[warp] = make_float2(sum.top, sum.l);
    };
    // Adds up the sums of warps [w, w + n) and writes dimensions d0, d0 + step, ... of row r.
    auto store = [&](int r, int w, int n, int d0, int step) {
        const int b = r / a.q_heads, j = r % a.q_heads;
        float top = -INFINITY, l = 0.0f;
        for (int i = w; i < w + n; ++i) top = fmaxf(top, s_ml[i].x);
        for (int i = w; i < w + n; ++i) l += s_ml[i].y * shrink(s_ml[i].x, top);
        const float vs = c.v_scale ? c.v_scale[j / sc.group] : 1.0f;
        const float inv = l == 0.0f ? 0.0f : vs / l;
        QT* out = static_cast<QT*>(a.out) + (int64_t)b * a.out_seq_stride + (int64_t)j * a.out_head_stride;
        for (int d = d0; d < c.head_dim; d += step) {
            float x = 0.0f;
            for (int i = w; i < w + n; ++i) x += reinterpret_cast<const float*>(s_o[i])[d] * shrink(s_ml[i].x, top);
            out[d] = from_f32<QT>(l == 0.0f ? 0.0f : x * inv);
        }
        if (d0 == 0) store_lse(sc, a, r, top, l);
    };
    // Each team looks at its row; a row of many more parts than others is left
    // to the whole CTA.
    const int mine = warp / TEAM, member = warp % TEAM, r = blockIdx.x * kPer + mine;
    bool joined = false, wide = false;
    if (r < rows) {
        const int b = r / a.q_heads, j = r % a.q_heads, before = sc.pre[b], tiles = sc.pre[b + 1] - before;
        if (tiles == 0) {
            empty_row<QT>(a, b, j, c.head_dim, member * 32 + lane, TEAM * 32);
        } else {
            const Parts p(sc, before, tiles, all, unit(j));
            wide = TEAM < kJoinWarps && p.count > 32 * TEAM;
            joined = p.count > 1 && !wide;
            if (joined) {
                RowSum<DP> sum;
                sum.add(sc, p, j % sc.group % sc.heads, member, TEAM, lane);
                keep(sum);
            }
        }
    }
    if constexpr (TEAM == 1) {
        __syncwarp();
        if (joined) store(r, warp, 1, lane, 32);
    }
    const bool any = __syncthreads_or(wide);
    if (TEAM > 1 && joined) store(r, mine * TEAM, TEAM, member * 32 + lane, TEAM * 32);
    if (!any) return;
    for (int k = 0; k < kPer; ++k) {
        if (!__syncthreads_or(wide && mine == k)) continue;
        const int rk = blockIdx.x * kPer + k, b = rk / a.q_heads, j = rk % a.q_heads, before = sc.pre[b];
        RowSum<DP> sum;
        sum.add(sc, Parts(sc, before, sc.pre[b + 1] - before, all, unit(j)), j % sc.group % sc.heads, warp, kJoinWarps, lane);
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

// Tiles of one sequence and unit, at most.
int most_tiles(const KvTable& t, const KvAttention& a, int tile) {
    const int all = (t.max_len + tile - 1) / tile;
    if (a.window <= 0 || a.window >= t.max_len) return all;
    const int64_t seen = ((int64_t)a.window + tile - 1) / tile + 1 + ((int64_t)a.sinks + tile - 1) / tile;
    return seen < all ? (int)seen : all;
}

// How one call is cut into launches, and the scratch of the largest.
struct Plan {
    int batch;  // sequences per launch
    int dp, warps, grid;
    Scratch sc;
    size_t at_lse2, at_ml, at_o, at_aside, at_logits, bytes;
};

Plan make_plan(const KvPages& c, const KvTable& t, const KvAttention& a, int most_batch, int heads, int warps, int dp, int tile, size_t aside, int sms) {
    Plan p{};
    p.dp = dp;
    p.warps = warps;
    p.sc.group = a.q_heads / c.kv_heads;
    p.sc.heads = heads;
    p.sc.units = c.kv_heads * ((p.sc.group + heads - 1) / heads);
    p.sc.rows = p.sc.group < heads ? p.sc.group : heads;
    const size_t tiles = most_tiles(t, a, tile);
    const size_t seq_logits = a.weight_out ? tiles * a.q_heads * tile * 4 : 0;
    const size_t seqs = t.batch < most_batch ? t.batch : most_batch;
    size_t batch = seqs;
    if (seq_logits * batch > kMaxLogits) batch = kMaxLogits / seq_logits;
    // lists are counted in 32 bits, also that of all positions, which the weights' launch may go over
    const size_t all = (size_t)((t.max_len + tile - 1) / tile) * c.kv_heads, longest = tiles * p.sc.units;
    while (batch > 1 && batch * (longest < all ? all : longest) > 0x7fffffff) batch /= 2;
    p.batch = batch < 1 ? 1 : (int)batch;
    // The scratch grows with the sequences, not with those that a launch takes:
    // a smaller call never needs more.
    const size_t most = seqs * tiles * p.sc.units, scores = seq_logits * seqs;
    p.grid = most < (size_t)sms ? (most < 1 ? 1 : (int)most) : sms;
    p.sc.workers = p.grid * warps;
    p.sc.shift = tile == 16 ? 4 : 5;
    p.sc.page = FastDiv(c.page_size);
    p.at_lse2 = 2 * round256((seqs + 1) * 4);
    p.at_ml = p.at_lse2 + round256(seqs * a.q_heads * 4);
    p.at_o = p.at_ml + round256((size_t)p.sc.workers * 2 * 16 * 8);
    p.at_aside = p.at_o + round256((size_t)p.sc.workers * 2 * p.sc.rows * dp * 4);
    p.at_logits = p.at_aside + round256(p.sc.workers * aside);
    p.bytes = p.at_logits + round256(scores <= kMaxLogits ? scores : seq_logits < kMaxLogits ? kMaxLogits : seq_logits);
    return p;
}

// Whether a call is small: a cluster of up to 8 CTAs for every key-value head of
// every sequence (whose group is one unit) fits the GPU at a time, with few
// tiles a warp.  ranks 0: it is not.
struct SmallPlan {
    int ranks;
    bool reserve;  // a smaller call may not be: scratch is kept for it
    Scratch sc;
    size_t bytes;
};

cudaError_t small_plan(const void* kern, size_t smem, const KvPages& c, const KvTable& t, const KvAttention& a, int heads, int warps, int tile,
                       bool slow, SmallPlan* out) {
    SmallPlan p{};
    *out = p;
    if (a.q_heads / c.kv_heads > heads) return cudaSuccess;
    const int tiles = most_tiles(t, a, tile);
    const int64_t units = (int64_t)t.batch * c.kv_heads;
    int ranks = 1;
    while (ranks < 8 && ranks * warps < tiles) ranks *= 2;
    for (; ranks > 0; ranks /= 2) {
        int most = 0;
        const cudaError_t e = cluster_limit(kern, warps * 32, smem, ranks, &most);
        if (e != cudaSuccess) return e;
        if (units <= most) break;
    }
    const SmallLimits limits = small_limits(slow, a.weight_out != nullptr);
    if (ranks == 0 || tiles > limits.many * ranks * warps) return cudaSuccess;
    if (tiles > limits.few * ranks * warps) {
        KernelSetup su;
        const cudaError_t e = kernel_setup(kern, warps * 32, smem, &su);
        if (e != cudaSuccess || units * ranks * 4 < (int64_t)su.sms * 3) return e;
        p.reserve = true;
    }
    p.ranks = p.sc.ranks = ranks;
    p.sc.group = a.q_heads / c.kv_heads;
    p.sc.units = c.kv_heads;
    p.sc.heads = heads;
    p.sc.max_tiles = tiles;
    p.sc.page = FastDiv(c.page_size);
    p.bytes = round256((size_t)units * tiles * p.sc.group * tile * 4);
    *out = p;
    return cudaSuccess;
}

template <typename QT, typename Rows, bool FP8, int DP, int T, int NW, int S>
cudaError_t run(const KvPages& c, const KvTable& t, const KvAttention& a, const KvScratch& mem, uint32_t* status, cudaStream_t s) {
    auto* kern = k_kv_attend<Rows, FP8, DP, T, NW, S, false>;
    constexpr size_t smem = Shape<Rows, FP8, DP, T, NW, S>::kSmem;
    static_assert(smem <= 227 * 1024, "the ring does not fit in shared memory");
    auto* one = k_kv_attend<Rows, FP8, DP, T, NW, S, true>;
    static_assert(kSmallTiles <= Rows::kChain, "a small call sets nothing aside");
    constexpr bool slow = FP8 || Rows::kHeads == 16 || DP == 256;
    SmallPlan small;
    cudaError_t e = small_plan(reinterpret_cast<const void*>(one), smem, c, t, a, Rows::kHeads, NW, T, slow, &small);
    if (e != cudaSuccess) return e;
    KernelSetup su;
    if (small.ranks == 0 || small.reserve) {
        e = kernel_setup(reinterpret_cast<const void*>(kern), NW * 32, smem, &su);
        if (e != cudaSuccess) return e;
    }
    if (small.ranks > 0) {
        size_t bytes = a.weight_out ? small.bytes : 0;  // 0 too where no sequence can have a position
        if (small.reserve) bytes = std::max(bytes, make_plan(c, t, a, kMaxBatch<DP>, Rows::kHeads, NW, DP, T, sizeof(Aside<Rows>), su.sms).bytes);
        if (bytes > 0) {
            void* base = mem.get(mem.owner, bytes);
            if (base == nullptr) return cudaErrorMemoryAllocation;
            if (a.weight_out) small.sc.logits = static_cast<float*>(base);
        }
        return launch_dependent(one, (size_t)t.batch * c.kv_heads * small.ranks, NW * 32, smem, small.ranks, s, c, t, a, small.sc, status);
    }
    Plan p = make_plan(c, t, a, kMaxBatch<DP>, Rows::kHeads, NW, DP, T, sizeof(Aside<Rows>), su.sms);
    char* base = static_cast<char*>(mem.get(mem.owner, p.bytes));
    if (base == nullptr) return cudaErrorMemoryAllocation;
    p.sc.pre = reinterpret_cast<int*>(base);
    p.sc.pre_all = p.sc.pre;
    if (a.window > 0 && a.weight_out && a.weight_in != a.weight_out) p.sc.pre_all = reinterpret_cast<int*>(base + p.at_lse2 / 2);
    p.sc.lse2 = reinterpret_cast<float*>(base + p.at_lse2);
    p.sc.ml = reinterpret_cast<float2*>(base + p.at_ml);
    p.sc.o = reinterpret_cast<float*>(base + p.at_o);
    p.sc.aside = base + p.at_aside;
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
        // Warps a row by the parts that rows have on average: most rows of more
        // units than workers are whole.
        const int64_t rows = (int64_t)u.batch * a.q_heads, units = (int64_t)u.batch * p.sc.units;
        const int team = units * 8 >= p.sc.workers ? 1 : units * 32 >= p.sc.workers ? 4 : kJoinWarps, per = kJoinWarps / team;
        auto* join = team == 1 ? k_kv_join<QT, DP, 1> : team == 4 ? k_kv_join<QT, DP, 4> : k_kv_join<QT, DP, kJoinWarps>;
        e = launch_dependent(join, (rows + per - 1) / per, kJoinThreads, 0, 1, s, c, u, v, p.sc);
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

// Rows8 up to 8 query heads a key-value head, Rows16 above.  Tile, warps and
// stages by row size: the ring takes about 192 KB of the SM, and the warps as
// many as their registers allow, since warps hide a tile's chain of products
// better than stages do (ragged batch in bf16, in a graph: 8 warps x 3 stages
// 113.6 us, 12 x 2 110.3, 13 x 2 spills 116.7).  8-bit and narrow rows take
// tiles of 32 positions, which spreads a tile's fixed instructions over as many
// bytes (8-bit rows in tiles of 16: 140.6 against 98.5 us).  Others, over 32 x
// 4000 to 8000 positions: Rows8 of 256 with 4 x 3 123.7 us, 6 x 2 121.6, 8-bit 8 x
// 3 124.7, 12 x 2 125.4; Rows16 of 64 with 8 x 3 131.6, 12 x 2 128.1 (spills),
// 8-bit 12 x 4 93.5, 16 x 3 92.3 (spills); of 128 with 8 x 3 126.6, 12 x 2 125.1
// (spills), 8-bit 84.0 / 106.4; of 256 in 8 bits with 7 x 3 114.6, 6 x 3 116.8.
template <typename QT, bool FP8>
cudaError_t run_dim(const KvPages& c, const KvTable& t, const KvAttention& a, const KvScratch& mem, uint32_t* status, cudaStream_t s) {
    if (a.q_heads / c.kv_heads <= 8) {
        if (c.head_dim <= 64) return run<QT, Rows8<QT, FP8, 64, 32>, FP8, 64, 32, FP8 ? 16 : 12, FP8 ? 3 : 2>(c, t, a, mem, status, s);
        if (c.head_dim <= 128) return run<QT, Rows8<QT, FP8, 128, FP8 ? 32 : 16>, FP8, 128, FP8 ? 32 : 16, 12, 2>(c, t, a, mem, status, s);
        return run<QT, Rows8<QT, FP8, 256, 16>, FP8, 256, 16, FP8 ? 8 : 4, 3>(c, t, a, mem, status, s);
    }
    if (c.head_dim <= 64) return run<QT, Rows16<QT, FP8, 64, 32>, FP8, 64, 32, FP8 ? 12 : 8, FP8 ? 4 : 3>(c, t, a, mem, status, s);
    if (c.head_dim <= 128) return run<QT, Rows16<QT, FP8, 128, FP8 ? 32 : 16>, FP8, 128, FP8 ? 32 : 16, 8, 3>(c, t, a, mem, status, s);
    return run<QT, Rows16<QT, FP8, 256, 16>, FP8, 256, 16, FP8 ? 7 : 4, 3>(c, t, a, mem, status, s);
}

}  // namespace

cudaError_t launch_kv_attend(const KvPages& c, const KvTable& t, const KvAttention& a, const KvScratch& mem, uint32_t* status, cudaStream_t s) {
    const bool bf = a.type == KvElem::BF16;
    if (c.type == KvElem::E4M3)
        return bf ? run_dim<__nv_bfloat16, true>(c, t, a, mem, status, s) : run_dim<__half, true>(c, t, a, mem, status, s);
    return bf ? run_dim<__nv_bfloat16, false>(c, t, a, mem, status, s) : run_dim<__half, false>(c, t, a, mem, status, s);
}

}  // namespace ss
