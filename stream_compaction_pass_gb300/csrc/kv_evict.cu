// kv_evict.cu -- eviction from a paged key-value cache by gathered attention
// weight (streamscan.h, ss_kv_evict), in two launches, or one where rows keep
// little.
//
// The selection is a compaction whose predicate is a rank: with weights as
// 32-bit keys, best first (kv.cuh, evict_key), it finds the m-th smallest key
// T of a row by its digits, 11, 11 and 10 bits from the top -- a histogram of
// the keys that share the digits found so far, and the bin that holds the m-th
// -- and then writes, in order, the positions whose key is below T and the
// first of those equal to it, ranked by a scan of the lanes' and the warps'
// counts.  The move copies the kept rows.
//
// What bounds it.  The move reads and writes every kept row once and is bound
// by memory: 2.1 GB of 8-bit rows in 326 us, 0.95 of the copy rate.  The
// selection reads 4 bytes a position and is bound by latency: three passes, each
// with a histogram, a scan and a barrier.  A row is one CTA's; where there are
// few rows it is split over a cluster of up to 8 CTAs, which add up their
// histograms in L2 and exchange counts through distributed shared memory.  128
// rows of 60 to 131 thousand positions take 77 us, 118 where all weights are
// equal, 192 rows of up to 9001 16 us, 8 rows of 2049 10 us.
#include <cooperative_groups.h>

#include "kv.cuh"

namespace ss {

namespace {

namespace cg = cooperative_groups;

constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kSplitFrom = 16384, kSplit = 2048;  // the shortest row that pays for a cluster's meetings, and its shortest share
constexpr int kStagedShare = 16384;            // the longest share whose keys are kept in shared memory
constexpr int kClassedShare = 256 * 1024;      // the longest share whose classes are
constexpr int kBlock = 1024;                   // positions a warp compacts at a time
// Bytes of a row's kept k and v up to which its selection moves them, in one
// launch, which also costs the host 3 to 4 us less: 300 rows of 141 x 512 bytes
// 12.5 against 15.0 us in a graph, 8 of 256 x 512 11.5 / 10.5, 8 of 512 x 512 16.2 / 10.5.
constexpr int64_t kFusedBytes = 128 * 1024;
constexpr int kListed = 16384;                 // candidates a long share keeps, 8 bytes each
static_assert((int64_t)kClassedShare * kMaxCluster == kKvMaxEvict, "the longest sequence is what a cluster can hold");

template <int N> struct SelectShared {
    uint32_t hist[3][kBins];  // one per pass
    uint32_t counts[2];       // this CTA's keys below T, and equal to it
    uint32_t warp_lt[N / 32], warp_eq[N / 32];
    uint32_t digit, before, listed;
};

// What the selection is asked for.
struct Choice {
    int keep, sinks, recent;
    int most_share;  // the longest share that the launch provides for, a multiple of 4
    FastDiv page;    // by src's page_size
    uint32_t* hist;  // of split rows: 3 x kBins words a row
};

// Shared memory of the selection before its classes, and in all.
__host__ __device__ constexpr int select_front(int threads, bool staged, int share) {
    const int blocks = threads / 32 * kBlock * 4, first = staged ? share * 4 : kListed * 8;
    return first > blocks ? first : blocks;
}
constexpr int select_bytes(int threads, bool staged, int share) { return select_front(threads, staged, share) + (share / 4 + 15) / 16 * 16; }

constexpr int kMoveThreads = 256;
constexpr int kMoveLoads = 8;  // 16-byte vectors that a thread has in flight

struct Move {
    int keep, rows, groups, vecs, elem_bytes;  // groups of `rows` kept rows per (sequence, head); `vecs` vectors a row
    FastDiv src_page, dst_page, by_vecs;
};

// Copies kept rows j0 .. j0 + mv.rows - 1 of one (sequence, head), k and v, by
// the N threads of a CTA: all of a thread's loads are issued before its first
// store.  `kept` is that row's list; s_place holds 2 mv.rows offsets.
template <int N, int LOADS>
__device__ __forceinline__ void move_rows(const KvPages& c, const KvTable& t, const KvPages& d, const KvTable& dt, const Move& mv,
                                          const int32_t* kept, int b, int h, int j0, int64_t* s_place, uint32_t* status) {
    const int tid = threadIdx.x, rows = mv.rows, vecs = mv.vecs;
    int64_t *s_src = s_place, *s_dst = s_place + rows;  // byte offsets, or -1
    for (int r = tid; r < rows; r += N) {
        const int j = j0 + r, p = j < mv.keep ? kept[j] : -1;
        int64_t src = -1, dst = -1;
        if (p >= 0) {
            const int fi = mv.src_page.div(p), ti = mv.dst_page.div(j);
            const int from = kv_page(t, c.num_pages, b, fi, status);
            const int to = kv_page(dt, d.num_pages, b, ti, status);
            if (from >= 0 && to >= 0) {
                const int fs = p - fi * c.page_size, ts = j - ti * d.page_size;
                src = ((int64_t)from * c.page_stride + (int64_t)h * c.head_stride + (int64_t)fs * c.slot_stride) * mv.elem_bytes;
                dst = ((int64_t)to * d.page_stride + (int64_t)h * d.head_stride + (int64_t)ts * d.slot_stride) * mv.elem_bytes;
                if (d.weight)
                    d.weight[((int64_t)to * d.kv_heads + h) * d.page_size + ts] = c.weight[((int64_t)from * c.kv_heads + h) * c.page_size + fs];
            }
        }
        s_src[r] = src;
        s_dst[r] = dst;
    }
    __syncthreads();
    const int half = rows * vecs;  // k's vectors, then v's
    for (int i0 = tid; i0 < 2 * half; i0 += N * LOADS) {
        uint4 x[LOADS];
        char* to[LOADS];
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
            const int i = i0 + l * N;
            to[l] = nullptr;
            if (i >= 2 * half) continue;
            const bool is_v = i >= half;
            const int k = is_v ? i - half : i, r = mv.by_vecs.div(k), v = k - r * vecs;
            if (s_src[r] < 0) continue;
            x[l] = ldg_vec((is_v ? c.v : c.k) + s_src[r] + v * 16);
            to[l] = (is_v ? d.v : d.k) + s_dst[r] + v * 16;
        }
#pragma unroll
        for (int l = 0; l < LOADS; ++l)
            if (to[l]) stg_vec(to[l], x[l]);
    }
}

// One cluster per (sequence, head); its CTAs take consecutive shares of the
// positions, each a multiple of 4 long.  N threads.  V: weights are read in
// fours, which lie in one page and are 16-byte aligned.
//
// A position is classed by what is known of its key: below T, possibly T,
// above; 2 bits, a byte for four positions (low half below T, high half
// possibly T).  STAGED: the keys of a share are read once and stay in shared
// memory, and the classes follow when T is known.  Otherwise two passes read
// every weight; the second one knows T's top digit, classes every position and
// lists those that share it with their keys.  The rest is done on the list,
// or, where that overflows (many equal weights), by reading the weights of
// the fours that may still hold T again.  128 long rows: 151 us when every pass
// read every weight, 95 with the classes, 70 with the list and the compaction
// in shared memory; keeping the keys of long rows too takes clusters of 8 and
// four waves of them, 130 us.
//
// FUSED: the CTA (one a row) also moves its row, where that is little.
template <int N, bool STAGED, int V, bool FUSED>
__global__ void __launch_bounds__(N, N == 512 ? 2 : 1) k_kv_select(KvPages c, KvTable t, KvPages d, KvTable dt, Move mv, Choice ch, int32_t* kept,
                                                                   int32_t* new_lens, uint32_t* status) {
    constexpr int kWarps = N / 32, kPer = kBins / N;  // bins a thread adds up
    __shared__ SelectShared<N> sh;
    extern __shared__ __align__(16) unsigned char s_share[];
    // Keys (STAGED) or the list, later the warps' compaction blocks; then the classes.
    uint32_t* s_keys = reinterpret_cast<uint32_t*>(s_share);
    uint2* s_list = reinterpret_cast<uint2*>(s_share);
    int32_t* s_block = reinterpret_cast<int32_t*>(s_share) + (threadIdx.x >> 5) * kBlock;
    unsigned char* s_class = s_share + select_front(N, STAGED, ch.most_share);
    begin_dependent();
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int row = blockIdx.x / ranks, b = row / c.kv_heads, h = row % c.kv_heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int len = kv_len(t, b, status);
    const int m = min(len, ch.keep);
    int32_t* out = kept + (int64_t)row * ch.keep;
    if (h == 0 && rank == 0 && tid == 0) new_lens[b] = m;
    auto move_row = [&]() {
        if constexpr (FUSED) {
            __syncthreads();  // the row's list is written, and shared memory free
            for (int j0 = 0; j0 < m; j0 += mv.rows) {
                move_rows<N, 4>(c, t, d, dt, mv, out, b, h, j0, reinterpret_cast<int64_t*>(s_share), status);
                __syncthreads();
            }
        }
    };
    if (len <= ch.keep) {  // the same for the whole cluster
        for (int64_t j = rank * N + tid; j < ch.keep; j += ranks * N) out[j] = j < m ? (int32_t)j : -1;  // keep may be up to 2^31 - 1
        move_row();
        return;
    }
    const int share = ((len + ranks - 1) / ranks + 3) / 4 * 4;
    const int begin = min(rank * share, len), count = min(share, len - begin);
    auto meet = [&]() {
        if (ranks == 1) __syncthreads(); else cluster.sync();
    };

    // Four keys of the share from position i < count on (a multiple of 4);
    // those past the share's end are the last of all.  A page out of range
    // reads page 0 and ranks last, so that no load waits for a branch; it is
    // reported at the end.
    bool bad = false;
    const int32_t* pages = t.pages + (int64_t)b * t.row_stride;
    const float* weight = c.weight + (int64_t)h * c.page_size;
    const int64_t per_page = (int64_t)c.kv_heads * c.page_size;
    auto place = [&](int p, bool& good) {
        const int index = ch.page.div(p), page = pages[index];
        good = (uint32_t)page < (uint32_t)c.num_pages;
        return weight + ((good ? page : 0) * per_page + (p - index * c.page_size));
    };
    auto read4 = [&](int i, uint32_t (&k)[4]) {
        const int p = begin + i;
        float w[4];
        bool good[4];
        if constexpr (V == 4) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(place(p, good[0])));
            w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
            good[1] = good[2] = good[3] = good[0];
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = __ldcg(place(min(p + e, len - 1), good[e]));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) k[e] = evict_key(w[e]);
        if (p >= ch.sinks && p + 4 <= len - ch.recent && i + 4 <= count && good[0] && good[1] && good[2] && good[3]) return;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            bad |= !good[e];
            if (!good[e] || i + e >= count) k[e] = 0xffffffffu;
            else if (p + e < ch.sinks || p + e >= len - ch.recent) k[e] = 0u;
        }
    };
    // Calls f(position) for this thread's fours, several at a time.
    constexpr int kAhead = STAGED ? 4 : 2;
    auto each_four = [&](auto&& f) {
        for (int i0 = tid * 4; i0 < count; i0 += N * 4 * kAhead) f(i0);
    };
    auto in_share = [&](int i0, int a) { return a == 0 || i0 + a * N * 4 < count; };

    for (int i = tid; i < 3 * kBins; i += N) (&sh.hist[0][0])[i] = 0;
    if (tid == 0) sh.listed = 0;
    uint32_t* row_hist = ch.hist + (int64_t)row * 3 * kBins;
    if (ranks > 1) {
        for (int i = rank * N + tid; i < 3 * kBins; i += ranks * N) row_hist[i] = 0;
        cluster.sync();
    }
    __syncthreads();
    uint32_t prefix = 0, want = (uint32_t)m;  // T's digits so far; which of the keys sharing them is T, from 1
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;  // of this pass's digit
        const int above = pass == 1 ? 21 : 10;                   // of the digits known
        const uint32_t digits = pass == 2 ? 1023u : 2047u;
        const bool on_list = !STAGED && pass == 2 && sh.listed <= kListed;
        if (on_list) {
            for (int i = tid; i < (int)sh.listed; i += N) {
                const uint32_t k = s_list[i].y;
                if (k >> above == prefix >> above) atomicAdd(&sh.hist[2][k & digits], 1u);
            }
        } else {
            each_four([&](int i0) {
                uint32_t k[kAhead][4];
                unsigned char cls[kAhead];
#pragma unroll
                for (int a = 0; a < kAhead; ++a) {
                    if (!in_share(i0, a)) continue;
                    const int i = i0 + a * N * 4;
                    cls[a] = 0xf0;
                    if (!STAGED && pass == 2) cls[a] = s_class[i / 4];
                    if (STAGED && pass > 0) {
                        const uint4 x = *reinterpret_cast<const uint4*>(s_keys + i);
                        k[a][0] = x.x; k[a][1] = x.y; k[a][2] = x.z; k[a][3] = x.w;
                    } else if (cls[a] & 0xf0) {
                        read4(i, k[a]);
                    }
                }
#pragma unroll
                for (int a = 0; a < kAhead; ++a) {
                    if (!in_share(i0, a)) continue;
                    const int i = i0 + a * N * 4;
                    if (STAGED && pass == 0) *reinterpret_cast<uint4*>(s_keys + i) = make_uint4(k[a][0], k[a][1], k[a][2], k[a][3]);
                    if (!(cls[a] & 0xf0)) continue;
                    uint32_t now = cls[a] & 0x0fu;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (pass == 0) {
                            if (i + e < count) atomicAdd(&sh.hist[0][k[a][e] >> 21], 1u);
                            continue;
                        }
                        const uint32_t known = k[a][e] >> above;
                        if (known > prefix >> above || i + e >= count || !(cls[a] >> (4 + e) & 1)) continue;
                        if (known == prefix >> above) {
                            atomicAdd(&sh.hist[pass][(k[a][e] >> shift) & digits], 1u);
                            now |= 0x10u << e;
                        } else {
                            now |= 1u << e;
                        }
                    }
                    if (!STAGED && pass > 0) s_class[i / 4] = (unsigned char)now;
                    if (!STAGED && pass == 1 && (now & 0xf0u)) {
                        uint32_t at = atomicAdd(&sh.listed, (uint32_t)__popc(now & 0xf0u));
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (now >> (4 + e) & 1u) {
                                if (at < (uint32_t)kListed) s_list[at] = make_uint2(i + e, k[a][e]);
                                ++at;
                            }
                    }
                }
            });
        }
        // A split row's histogram is added up in L2 (its bins are few that are
        // not empty).  Then every thread takes kPer consecutive bins, and a scan
        // over the block finds the bin of the want-th key.
        if (ranks > 1) {
            __syncthreads();
            for (int i = tid; i < kBins; i += N)
                if (const uint32_t x = sh.hist[pass][i]) atomicAdd(row_hist + pass * kBins + i, x);
        }
        meet();
        uint32_t s[kPer], mine = 0;
        const uint32_t* from_bins = (ranks > 1 ? row_hist + pass * kBins : &sh.hist[pass][0]) + tid * kPer;
#pragma unroll
        for (int e = 0; e < kPer; e += 2) {
            const uint2 x = ranks > 1 ? __ldcg(reinterpret_cast<const uint2*>(from_bins + e)) : *reinterpret_cast<const uint2*>(from_bins + e);
            s[e] = x.x;
            s[e + 1] = x.y;
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e) mine += s[e];
        const uint32_t incl = warp_inclusive_scan<uint32_t>(mine, lane);
        if (lane == 31) sh.warp_lt[warp] = incl;
        __syncthreads();
        uint32_t before = incl - mine;
        for (int w = 0; w < warp; ++w) before += sh.warp_lt[w];
        if (before < want && want <= before + mine) {  // one thread
            int digit = 0;
#pragma unroll
            for (int e = 0; e < kPer - 1; ++e)
                if (digit == e && before + s[e] < want) {
                    before += s[e];
                    digit = e + 1;
                }
            sh.digit = kPer * tid + digit;
            sh.before = before;
        }
        __syncthreads();
        prefix |= sh.digit << shift;
        want -= sh.before;
    }

    // T = prefix, and the first `want` of the positions that hold it stay.
    const bool listed = !STAGED && sh.listed <= kListed;
    if (listed) {
        for (int i = tid; i < (int)sh.listed; i += N) {
            const uint2 x = s_list[i];
            const uint32_t may = 0x10u << (x.x & 3u), below = 1u << (x.x & 3u), byte = (x.x >> 2 & 3u) * 8;
            if (x.y != prefix) atomicXor(reinterpret_cast<uint32_t*>(s_class) + (x.x >> 4), (x.y < prefix ? may | below : may) << byte);
        }
        __syncthreads();
    }
    // Each warp takes a consecutive part of the share.
    const int part = ((count + kWarps - 1) / kWarps + 127) / 128 * 128;
    const int from = min(warp * part, count), to = min(from + part, count);
    auto classes = [&](int i) -> uint32_t {  // of the four from i on, final
        uint32_t k[4], cls = 0xf0u;
        if constexpr (STAGED) {
            const uint4 x = *reinterpret_cast<const uint4*>(s_keys + i);
            k[0] = x.x; k[1] = x.y; k[2] = x.z; k[3] = x.w;
        } else {
            cls = s_class[i / 4];
            if (listed || !(cls & 0xf0u)) return cls;
            read4(i, k);
        }
        uint32_t now = cls & 0x0fu;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if ((cls >> (4 + e) & 1u) && i + e < to) now |= k[e] < prefix ? 1u << e : k[e] == prefix ? 0x10u << e : 0u;
        return now;
    };
    uint32_t lt = 0, eq = 0;
    for (int i = from + lane * 4; i < to; i += 128) {
        const uint32_t cls = classes(i);
        s_class[i / 4] = (unsigned char)cls;
        lt += __popc(cls & 0x0fu);
        eq += __popc(cls & 0xf0u);
    }
    lt = warp_sum<uint32_t>(lt);
    eq = warp_sum<uint32_t>(eq);
    if (lane == 0) {
        sh.warp_lt[warp] = lt;
        sh.warp_eq[warp] = eq;
    }
    __syncthreads();
    if (tid == 0) {
        uint32_t a = 0, e = 0;
        for (int w = 0; w < kWarps; ++w) {
            a += sh.warp_lt[w];
            e += sh.warp_eq[w];
        }
        sh.counts[0] = a;
        sh.counts[1] = e;
    }
    meet();
    lt = eq = 0;
    for (int r = 0; r < rank; ++r) {
        const uint32_t* x = cluster.map_shared_rank(&sh.counts[0], r);
        lt += x[0];
        eq += x[1];
    }
    for (int w = 0; w < warp; ++w) {
        lt += sh.warp_lt[w];
        eq += sh.warp_eq[w];
    }
    // kBlock positions at a time, 32 to a lane, compacted in shared memory and
    // written from there in order; the block's counts share a word.
    for (int i0 = from; i0 < to; i0 += kBlock) {
        const int i = i0 + lane * 32;
        uint32_t is_lt = 0, is_eq = 0;
        if (i < to) {
            const uint2 x = *reinterpret_cast<const uint2*>(s_class + i / 4);
            auto half = [](uint32_t w) {  // the low halves of four bytes, side by side
                w &= 0x0f0f0f0fu;
                w = (w | w >> 4) & 0x00ff00ffu;
                return (w | w >> 8) & 0xffffu;
            };
            const uint32_t here = to - i >= 32 ? 0xffffffffu : (1u << (to - i)) - 1u;
            is_lt = (half(x.x) | half(x.y) << 16) & here;
            is_eq = (half(x.x >> 4) | half(x.y >> 4) << 16) & here;
        }
        const uint32_t sum = __popc(is_lt) | __popc(is_eq) << 16;
        const uint32_t incl = warp_inclusive_scan<uint32_t>(sum, lane);
        const uint32_t my_lt = lt + ((incl - sum) & 0xffffu), my_eq = eq + ((incl - sum) >> 16);
        const uint32_t base = lt + min(eq, want);
        const int ties = my_eq < want ? (int)min(want - my_eq, sum >> 16) : 0;  // of this lane's that stay
        for (int drop = (int)(sum >> 16) - ties; drop > 0; --drop) is_eq &= ~(0x80000000u >> __clz(is_eq));
        uint32_t at = my_lt + min(my_eq, want) - base;
        for (uint32_t keep = is_lt | is_eq; keep; keep &= keep - 1) s_block[at++] = begin + i + __ffs(keep) - 1;
        const uint32_t all = __shfl_sync(kFullMask, incl, 31);
        lt += all & 0xffffu;
        eq += all >> 16;
        const uint32_t stay = lt + min(eq, want) - base;
        __syncwarp();
        for (uint32_t j = lane; j < stay; j += 32)
            if (base + j < (uint32_t)m) out[base + j] = s_block[j];
        __syncwarp();
    }
    if (bad) record_error(status, kErrKvTable, (uint32_t)(t.first + b));
    if (ranks > 1) cluster.sync();  // no CTA leaves while another may read its shared memory
    move_row();
}

// CTAs of a row's cluster: one per row where there are rows for half the SMs;
// otherwise a long row is split, into shares of kSplit positions or more, while
// the CTAs fit the SMs.  With the move, in a graph, one CTA / split, half kept:
//   1 row: 6000 positions 12.6 / 15.3 us, 14000 16.4 / 15.6, 20000 21.5 / 16.6,
//     131072 80.4 / 29.9;
//   8 rows: 10000 19.5 / 20.2, 14000 22.2 / 21.7, 20000 31.9 / 26.6, 131072 170 /
//     115, and with equal weights 240 / 128;
//   32 rows: 10000 46.8 / 46.0, 20000 78.2 / 75.5, 131072 411 / 362;
//   72 rows: 20000 136.0 / 136.9, 32000 208.4 / 207.7, 131072 810 / 780.
int select_ranks(const KvPages& c, const KvTable& t, int sms) {
    const int64_t rows = (int64_t)t.batch * c.kv_heads;
    int ranks = 1;
    auto split = [&](int r) { return rows * r * 2 <= sms && t.max_len >= kSplitFrom && t.max_len / (r * 2) >= kSplit; };
    while (ranks < kMaxCluster && (split(ranks) || t.max_len / ranks > kClassedShare - 4)) ranks *= 2;
    return ranks;
}

// One CTA per group of a row's kept positions.
__global__ void __launch_bounds__(kMoveThreads) k_kv_move(KvPages c, KvTable t, KvPages d, KvTable dt, Move mv, const int32_t* kept, uint32_t* status) {
    __shared__ int64_t s_place[2 * kMoveThreads];
    begin_dependent();
    const int row = blockIdx.x / mv.groups, j0 = (blockIdx.x - row * mv.groups) * mv.rows;
    kept += (int64_t)row * mv.keep;
    if (kept[j0] < 0) return;
    const int b = row / c.kv_heads;
    move_rows<kMoveThreads, kMoveLoads>(c, t, d, dt, mv, kept, b, row - b * c.kv_heads, j0, s_place, status);
}

}  // namespace

// For a smaller call (fewer rows, shorter ones) it is never more: the
// histograms of as many rows as can be split (select_ranks).
size_t kv_evict_scratch(const KvPages& c, const KvTable& t, int sms) {
    const int64_t rows = (int64_t)t.batch * c.kv_heads, few = sms / 2;
    const int64_t split = t.max_len > kClassedShare - 4 ? rows : t.max_len < kSplitFrom ? 0 : rows < few ? rows : few;
    return (size_t)split * 3 * kBins * 4;
}

cudaError_t launch_kv_evict(const KvPages& c, const KvTable& t, const KvPages& d, const KvTable& dt, int keep,
                            int sinks, int recent, int32_t* kept, uint32_t* scratch, int sms, uint32_t* status, cudaStream_t s) {
    const unsigned rows = (unsigned)t.batch * (unsigned)c.kv_heads;
    const int ranks = select_ranks(c, t, sms);
    const int share = ((t.max_len + ranks - 1) / ranks + 3) / 4 * 4;
    const bool staged = share <= kStagedShare;
    const bool vec4 = c.page_size % 4 == 0 && (reinterpret_cast<uintptr_t>(c.weight) & 15u) == 0;
    const int bytes = kv_elem_bytes(c.type), vecs = c.head_dim * bytes / 16;
    const int most = keep < t.max_len ? keep : t.max_len;
    const bool fused = staged && ranks == 1 && (int64_t)most * vecs * 32 <= kFusedBytes;
    auto* kern = !staged ? (vec4 ? k_kv_select<1024, false, 4, false> : k_kv_select<1024, false, 1, false>)
                 : fused ? (vec4 ? k_kv_select<512, true, 4, true> : k_kv_select<512, true, 1, true>)
                         : (vec4 ? k_kv_select<512, true, 4, false> : k_kv_select<512, true, 1, false>);
    const int threads = staged ? 512 : 1024, bytes_most = select_bytes(threads, staged, staged ? kStagedShare : kClassedShare);
    KernelSetup su;
    cudaError_t e = kernel_setup(reinterpret_cast<const void*>(kern), threads, (size_t)bytes_most, &su);
    if (e != cudaSuccess) return e;

    const int per = fused ? 256 : kv_rows_per_cta(kMoveThreads * kMoveLoads / (2 * vecs), kMoveThreads, (int64_t)rows * most, sms);
    const int groups = (most + per - 1) / per;
    const Move mv{keep, per, groups, vecs, bytes, FastDiv(c.page_size), FastDiv(d.page_size), FastDiv(vecs)};
    e = launch_dependent(kern, (size_t)rows * ranks, threads, (size_t)select_bytes(threads, staged, share), ranks, s, c, t, d, dt, mv,
                         Choice{keep, sinks, recent, share, FastDiv(c.page_size), scratch}, kept, dt.lens, status);
    if (e != cudaSuccess || fused || groups == 0) return e;
    return launch_dependent(k_kv_move, (size_t)rows * groups, kMoveThreads, 0, 1, s, c, t, d, dt, mv, kept, status);
}

}  // namespace ss
