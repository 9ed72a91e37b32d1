// kv_evict.cu -- eviction from a paged key-value cache by gathered attention
// weight (streamscan.h, ss_kv_evict), in two launches.
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
// by memory.  The selection reads 4 bytes a position; it is bound by latency
// (three passes, each with a histogram, a scan and a barrier).  A row is one
// CTA's; where there are few rows it is split over a cluster of up to 8 CTAs,
// which add up their histograms through distributed shared memory.  The keys
// of a share stay in shared memory where they fit; longer ones are read again
// in every pass, from L2.
#include <cooperative_groups.h>

#include "kv.cuh"

namespace ss {

namespace {

namespace cg = cooperative_groups;

constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kMaxStaged = 48 * 1024;  // keys a CTA can hold in shared memory

template <int N> struct SelectShared {
    uint32_t hist[3][kBins];  // one per pass: nobody clears what another CTA still reads
    uint32_t counts[2];       // this CTA's keys below T, and equal to it
    uint32_t warp_lt[N / 32], warp_eq[N / 32];
    uint32_t digit, before;
};

// What the selection is asked for.
struct Choice {
    int keep, sinks, recent;
    FastDiv page;  // by src's page_size
};

// One cluster per (sequence, head); its CTAs take consecutive shares of the
// positions, each a multiple of 4 long.  STAGED: the keys of a share fit in
// shared memory (otherwise every pass reads the weights again).  V: weights
// are read in fours, which lie in one page and are 16-byte aligned.
// N threads.
template <int N, bool STAGED, int V>
__global__ void __launch_bounds__(N) k_kv_select(KvPages c, KvTable t, Choice ch, int32_t* __restrict__ kept,
                                                             int32_t* __restrict__ new_lens, uint32_t* status) {
    constexpr int kWarps = N / 32, kPer = kBins / N;  // bins a thread adds up
    __shared__ SelectShared<N> sh;
    extern __shared__ __align__(16) uint32_t s_keys[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int row = blockIdx.x / ranks, b = row / c.kv_heads, h = row % c.kv_heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int len = kv_len(t, b, status);
    const int m = min(len, ch.keep);
    int32_t* out = kept + (int64_t)row * ch.keep;
    if (h == 0 && rank == 0 && tid == 0) new_lens[b] = m;
    if (len <= ch.keep) {  // the same for the whole cluster
        for (int j = rank * N + tid; j < ch.keep; j += ranks * N) out[j] = j < m ? j : -1;
        return;
    }
    const int share = ((len + ranks - 1) / ranks + 3) / 4 * 4;
    const int begin = min(rank * share, len), count = min(share, len - begin);
    auto meet = [&]() {
        if (ranks == 1) __syncthreads(); else cluster.sync();
    };

    // Four keys of the share from position i on (a multiple of 4); past the
    // share's end they are meaningless.  A page out of range reads page 0 and
    // ranks last, so that loads wait for no branch; it is reported at the end.
    bool bad = false;
    auto place = [&](int p, bool& good) {
        const int index = ch.page.div(p), page = __ldg(t.pages + (int64_t)b * t.row_stride + index);
        good = page >= 0 && page < c.num_pages;
        return ((int64_t)(good ? page : 0) * c.kv_heads + h) * c.page_size + (p - index * c.page_size);
    };
    auto read4 = [&](int i, uint32_t (&k)[4]) {
        const int p = begin + min(i, (count - 1) / 4 * 4);  // in range whatever i is
        float w[4];
        bool good[4];
        if constexpr (V == 4) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(c.weight + place(p, good[0])));
            w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
            good[1] = good[2] = good[3] = good[0];
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = __ldg(c.weight + place(min(p + e, len - 1), good[e]));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            k[e] = p + e < ch.sinks || p + e >= len - ch.recent ? 0u : good[e] ? evict_key(w[e]) : 0xffffffffu;
            bad |= !good[e];
        }
    };
    auto keys4 = [&](int i, uint32_t (&k)[4]) {
        if constexpr (STAGED) {
            const uint4 x = *reinterpret_cast<const uint4*>(s_keys + i);
            k[0] = x.x; k[1] = x.y; k[2] = x.z; k[3] = x.w;
        } else {
            read4(i, k);
        }
    };
    // Visits the share's keys as (position, key), several loads at a time.
    auto each_key = [&](auto&& read, auto&& f) {
        constexpr int kAhead = 4;
        for (int i0 = tid * 4; i0 < count; i0 += N * 4 * kAhead) {
            uint32_t k[kAhead][4];
#pragma unroll
            for (int a = 0; a < kAhead; ++a)
                if (a == 0 || i0 + a * N * 4 < count) read(i0 + a * N * 4, k[a]);
#pragma unroll
            for (int a = 0; a < kAhead; ++a)
                if (i0 + a * N * 4 < count) f(i0 + a * N * 4, k[a]);
        }
    };

    for (int i = tid; i < 3 * kBins; i += N) (&sh.hist[0][0])[i] = 0;
    __syncthreads();
    // First pass: the keys enter shared memory and their top digit is counted.
    each_key(read4, [&](int i, const uint32_t (&k)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i + e < count) atomicAdd(&sh.hist[0][k[e] >> 21], 1u);
        if constexpr (STAGED) *reinterpret_cast<uint4*>(s_keys + i) = make_uint4(k[0], k[1], k[2], k[3]);
    });

    uint32_t prefix = 0, want = (uint32_t)m;  // T's digits so far; which of the keys sharing them is T, from 1
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t bins = pass == 2 ? 1024u : 2048u;
        if (pass > 0) {
            const int above = pass == 1 ? 21 : 10;
            each_key(keys4, [&](int i, const uint32_t (&k)[4]) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (k[e] >> above == prefix >> above && i + e < count) atomicAdd(&sh.hist[pass][(k[e] >> shift) & (bins - 1)], 1u);
            });
        }
        meet();
        // Every thread sums kPer consecutive bins over the cluster; a scan over the block finds the bin of the want-th key.
        uint32_t s[kPer] = {}, mine = 0;
        for (int r = 0; r < ranks; ++r) {
            const uint32_t* from = (ranks == 1 ? &sh.hist[pass][0] : cluster.map_shared_rank(&sh.hist[pass][0], r)) + tid * kPer;
#pragma unroll
            for (int e = 0; e < kPer; e += 2) {
                const uint2 x = *reinterpret_cast<const uint2*>(from + e);
                s[e] += x.x;
                s[e + 1] += x.y;
            }
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
    // Each warp takes a consecutive part of the share, 128 positions at a
    // time, four to a lane; the 128 counts share a word, keys below T in the
    // low half and equal to T in the high half.
    const int part = ((count + kWarps - 1) / kWarps + 127) / 128 * 128;
    const int from = min(warp * part, count), to = min(from + part, count);
    auto classify = [&](int i, uint32_t (&k)[4], uint32_t (&is)[4]) {
        keys4(i, k);
        uint32_t sum = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            is[e] = i + e >= to ? 0u : k[e] < prefix ? 1u : k[e] == prefix ? 0x10000u : 0u;
            sum += is[e];
        }
        return sum;
    };
    uint32_t lt = 0, eq = 0;
    for (int i = from + lane * 4; i < to; i += 128) {
        uint32_t k[4], is[4];
        const uint32_t sum = classify(i, k, is);
        lt += sum & 0xffffu;
        eq += sum >> 16;
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
    for (int i0 = from; i0 < to; i0 += 128) {
        const int i = i0 + lane * 4;
        uint32_t k[4], is[4], sum = 0;
        is[0] = is[1] = is[2] = is[3] = 0;
        if (i < to) sum = classify(i, k, is);
        const uint32_t incl = warp_inclusive_scan<uint32_t>(sum, lane);
        uint32_t my_lt = lt + ((incl - sum) & 0xffffu), my_eq = eq + ((incl - sum) >> 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t at = my_lt + min(my_eq, want);
            if ((is[e] == 1u || (is[e] && my_eq < want)) && at < (uint32_t)m) out[at] = begin + i + e;
            my_lt += is[e] & 0xffffu;
            my_eq += is[e] >> 16;
        }
        const uint32_t all = __shfl_sync(kFullMask, incl, 31);
        lt += all & 0xffffu;
        eq += all >> 16;
    }
    if (bad) record_error(status, kErrKvTable, (uint32_t)(t.first + b));
    if (ranks > 1) cluster.sync();  // no CTA leaves while another may read its shared memory
}

constexpr int kMoveThreads = 256;
constexpr int kMoveLoads = 8;  // 16-byte vectors that a thread has in flight

// Copies `rows` kept rows of one (sequence, head) per CTA, k and v: all of a
// thread's loads are issued before its first store.
struct Move {
    int keep, rows, groups, vecs, elem_bytes;  // groups of `rows` kept rows per (sequence, head); `vecs` vectors a row
    FastDiv src_page, dst_page, by_vecs;
};
__global__ void __launch_bounds__(kMoveThreads) k_kv_move(KvPages c, KvTable t, KvPages d, KvTable dt, Move mv,
                                                         const int32_t* __restrict__ kept, uint32_t* status) {
    const int keep = mv.keep, rows = mv.rows, vecs = mv.vecs;
    __shared__ int64_t s_src[kMoveThreads], s_dst[kMoveThreads];  // byte offsets, or -1
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x;
    const int row = blockIdx.x / mv.groups, j0 = (blockIdx.x - row * mv.groups) * rows;
    const int b = row / c.kv_heads, h = row % c.kv_heads;
    if (kept[(int64_t)row * keep + j0] < 0) return;
    if (tid < rows) {
        const int j = j0 + tid;
        const int p = j < keep ? kept[(int64_t)row * keep + j] : -1;
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
        s_src[tid] = src;
        s_dst[tid] = dst;
    }
    __syncthreads();
    const int half = rows * vecs;  // k's vectors, then v's
    for (int i0 = tid; i0 < 2 * half; i0 += kMoveThreads * kMoveLoads) {
        uint4 x[kMoveLoads];
        char* to[kMoveLoads];
#pragma unroll
        for (int l = 0; l < kMoveLoads; ++l) {
            const int i = i0 + l * kMoveThreads;
            to[l] = nullptr;
            if (i >= 2 * half) continue;
            const bool is_v = i >= half;
            const int k = is_v ? i - half : i, r = mv.by_vecs.div(k), v = k - r * vecs;
            if (s_src[r] < 0) continue;
            x[l] = ldg_vec((is_v ? c.v : c.k) + s_src[r] + v * 16);
            to[l] = (is_v ? d.v : d.k) + s_dst[r] + v * 16;
        }
#pragma unroll
        for (int l = 0; l < kMoveLoads; ++l)
            if (to[l]) stg_vec(to[l], x[l]);
    }
}

}  // namespace

cudaError_t launch_kv_evict(const KvPages& c, const KvTable& t, const KvPages& d, const KvTable& dt, int keep,
                            int sinks, int recent, int32_t* kept, int sms, uint32_t* status, cudaStream_t s) {
    const unsigned rows = (unsigned)t.batch * (unsigned)c.kv_heads;
    // One CTA per row where there are rows for half the SMs; otherwise a row is
    // split, into shares of 2048 positions or more, while the CTAs fit the SMs.
    int ranks = 1;
    while (ranks < kMaxCluster && (int64_t)rows * ranks * 2 <= sms && t.max_len / (ranks * 2) >= 2048) ranks *= 2;
    const int share = ((t.max_len + ranks - 1) / ranks + 3) / 4 * 4;
    const bool staged = share <= kMaxStaged;
    const bool vec4 = c.page_size % 4 == 0 && (reinterpret_cast<uintptr_t>(c.weight) & 15u) == 0;
    const bool large = share > 16384;  // 32 keys a thread at 512 threads: twice the threads from here on
    auto* kern = large ? (staged ? (vec4 ? k_kv_select<1024, true, 4> : k_kv_select<1024, true, 1>) : (vec4 ? k_kv_select<1024, false, 4> : k_kv_select<1024, false, 1>))
                       : (vec4 ? k_kv_select<512, true, 4> : k_kv_select<512, true, 1>);
    const int threads = large ? 1024 : 512;
    KernelSetup su;
    cudaError_t e = kernel_setup(reinterpret_cast<const void*>(kern), threads, staged ? (size_t)kMaxStaged * 4 : 0, &su);
    if (e != cudaSuccess) return e;

    cudaLaunchAttribute at[1];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(rows * ranks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = staged ? (size_t)share * 4 : 0;
    cfg.stream = s;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ranks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, c, t, Choice{keep, sinks, recent, FastDiv(c.page_size)}, kept, dt.lens, status);
    if (e != cudaSuccess) return e;

    const int bytes = kv_elem_bytes(c.type), vecs = c.head_dim * bytes / 16;
    const int most = keep < t.max_len ? keep : t.max_len;
    const int per = kv_rows_per_cta(kMoveThreads * kMoveLoads / (2 * vecs), kMoveThreads, (int64_t)rows * most, sms);
    const int groups = (most + per - 1) / per;
    if (groups == 0) return cudaSuccess;
    cfg = {};
    cfg.gridDim = dim3(rows * (unsigned)groups);
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = s;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const Move mv{keep, per, groups, vecs, bytes, FastDiv(c.page_size), FastDiv(d.page_size), FastDiv(vecs)};
    return cudaLaunchKernelEx(&cfg, k_kv_move, c, t, d, dt, mv, (const int32_t*)kept, status);
}

}  // namespace ss
