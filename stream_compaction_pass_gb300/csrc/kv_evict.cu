// kv_evict.cu -- eviction from a paged key-value cache by gathered attention
// weight (streamscan.h, ss_kv_evict), in two launches.
//
// The selection is a compaction whose predicate is a rank: with weights as
// 32-bit keys, best first (kv.cuh, evict_key), it finds the m-th smallest key
// T of a row by its digits, 11, 11 and 10 bits from the top -- a histogram of
// the keys that share the digits found so far, and the bin that holds the m-th
// -- and then writes, in order, the positions whose key is below T and the
// first of those equal to it, ranked by ballots and a scan of the warps'
// counts.  The move copies the kept rows.
//
// What bounds it.  The move reads and writes every kept row once and is bound
// by memory.  The selection reads 4 bytes a position; it is bound by latency
// (three passes, each with a histogram, a scan and a barrier), so a row is
// split over a cluster of up to 8 CTAs that keep their share of the keys in
// shared memory, add up their histograms through distributed shared memory,
// and meet five times.
#include <cooperative_groups.h>

#include "kv.cuh"

namespace ss {

namespace {

namespace cg = cooperative_groups;

constexpr int kSelectThreads = 512;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kMaxStaged = 48 * 1024;  // keys a CTA can hold in shared memory

struct SelectShared {
    uint32_t hist[3][kBins];  // one per pass: nobody clears what another CTA still reads
    uint32_t counts[2];       // this CTA's keys below T, and equal to it
    uint32_t warp_lt[kSelectWarps], warp_eq[kSelectWarps];
    uint32_t digit, before;
};

// One cluster per (sequence, head); its CTAs take consecutive shares of the
// positions, each a multiple of 4 long.  `staged`: the keys of a share fit in
// shared memory (otherwise every pass reads the weights again).
__global__ void __launch_bounds__(kSelectThreads) k_kv_select(KvPages c, KvTable t, int keep, int sinks, int recent, int staged, int vec4,
                                                             int32_t* __restrict__ kept, int32_t* __restrict__ new_lens, uint32_t* status) {
    __shared__ SelectShared sh;
    extern __shared__ uint32_t s_keys[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int row = blockIdx.x / ranks, b = row / c.kv_heads, h = row % c.kv_heads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int len = kv_len(t, b, status);
    const int m = min(len, keep);
    int32_t* out = kept + (int64_t)row * keep;
    if (h == 0 && rank == 0 && tid == 0) new_lens[b] = m;
    if (len <= keep) {  // the same for the whole cluster
        for (int j = rank * kSelectThreads + tid; j < keep; j += ranks * kSelectThreads) out[j] = j < m ? j : -1;
        return;
    }
    const int share = ((len + ranks - 1) / ranks + 3) / 4 * 4;
    const int begin = min(rank * share, len), count = min(share, len - begin);

    auto forced = [&](int p) { return p < sinks || p >= len - recent; };
    auto read_key = [&](int i) -> uint32_t {
        const int p = begin + i;
        if (forced(p)) return 0u;
        const int page = kv_page(t, c.num_pages, b, p / c.page_size, status);
        if (page < 0) return 0xffffffffu;
        return evict_key(c.weight[((int64_t)page * c.kv_heads + h) * c.page_size + p % c.page_size]);
    };
    auto key = [&](int i) -> uint32_t { return staged ? s_keys[i] : read_key(i); };

    for (int i = tid; i < 3 * kBins; i += kSelectThreads) (&sh.hist[0][0])[i] = 0;
    __syncthreads();
    // First pass: the keys enter shared memory and their top digit is counted.
    if (staged && vec4) {  // four consecutive weights lie in one page, 16-byte aligned
        for (int i = tid * 4; i < count; i += kSelectThreads * 4) {
            const int p = begin + i;
            const int page = kv_page(t, c.num_pages, b, p / c.page_size, status);
            float4 w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (page >= 0)
                w = *reinterpret_cast<const float4*>(c.weight + ((int64_t)page * c.kv_heads + h) * c.page_size + p % c.page_size);
            const float x[4] = {w.x, w.y, w.z, w.w};
            uint32_t k[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                k[e] = forced(p + e) ? 0u : page < 0 ? 0xffffffffu : evict_key(x[e]);
                if (i + e < count) atomicAdd(&sh.hist[0][k[e] >> 21], 1u);
            }
            *reinterpret_cast<uint4*>(s_keys + i) = make_uint4(k[0], k[1], k[2], k[3]);
        }
    } else {
        for (int i = tid; i < count; i += kSelectThreads) {
            const uint32_t k = read_key(i);
            if (staged) s_keys[i] = k;
            atomicAdd(&sh.hist[0][k >> 21], 1u);
        }
    }

    uint32_t prefix = 0, want = (uint32_t)m;  // T's digits so far; which of the keys sharing them is T, from 1
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t bins = pass == 2 ? 1024u : 2048u;
        if (pass > 0) {
            const int above = pass == 1 ? 21 : 10;
            for (int i = tid; i < count; i += kSelectThreads) {
                const uint32_t k = key(i);
                if (k >> above == prefix >> above) atomicAdd(&sh.hist[pass][(k >> shift) & (bins - 1)], 1u);
            }
        }
        cluster.sync();
        // Thread i sums bins 4 i .. 4 i + 3 over the cluster; a scan over the block finds the bin of the want-th key.
        uint4 s = make_uint4(0, 0, 0, 0);
        for (int r = 0; r < ranks; ++r) {
            const uint4 x = reinterpret_cast<const uint4*>(cluster.map_shared_rank(&sh.hist[pass][0], r))[tid];
            s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
        }
        const uint32_t mine = s.x + s.y + s.z + s.w;
        const uint32_t incl = warp_inclusive_scan<uint32_t>(mine, lane);
        if (lane == 31) sh.warp_lt[warp] = incl;
        __syncthreads();
        uint32_t before = incl - mine;
        for (int w = 0; w < warp; ++w) before += sh.warp_lt[w];
        if (before < want && want <= before + mine) {  // one thread
            const uint32_t v[4] = {s.x, s.y, s.z, s.w};
            int e = 0;
            while (before + v[e] < want) before += v[e++];
            sh.digit = 4 * tid + e;
            sh.before = before;
        }
        __syncthreads();
        prefix |= sh.digit << shift;
        want -= sh.before;
    }

    // T = prefix, and the first `want` of the positions that hold it stay.
    // Each warp takes a consecutive part of the share, 32 positions at a time.
    const int part = ((count + kSelectWarps - 1) / kSelectWarps + 31) / 32 * 32;
    const int from = min(warp * part, count), to = min(from + part, count);
    uint32_t lt = 0, eq = 0;
    for (int i = from + lane; i - lane < to; i += 32) {
        const uint32_t k = i < to ? key(i) : 0xffffffffu;
        lt += __popc(__ballot_sync(kFullMask, i < to && k < prefix));
        eq += __popc(__ballot_sync(kFullMask, i < to && k == prefix));
    }
    if (lane == 0) {
        sh.warp_lt[warp] = lt;
        sh.warp_eq[warp] = eq;
    }
    __syncthreads();
    if (tid == 0) {
        uint32_t a = 0, e = 0;
        for (int w = 0; w < kSelectWarps; ++w) {
            a += sh.warp_lt[w];
            e += sh.warp_eq[w];
        }
        sh.counts[0] = a;
        sh.counts[1] = e;
    }
    cluster.sync();
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
    const uint32_t below = (1u << lane) - 1u;
    for (int i = from + lane; i - lane < to; i += 32) {
        const uint32_t k = i < to ? key(i) : 0xffffffffu;
        const uint32_t l = __ballot_sync(kFullMask, i < to && k < prefix);
        const uint32_t q = __ballot_sync(kFullMask, i < to && k == prefix);
        const uint32_t my_lt = lt + __popc(l & below), my_eq = eq + __popc(q & below);
        const uint32_t at = my_lt + min(my_eq, want);
        if (((l >> lane & 1u) || ((q >> lane & 1u) && my_eq < want)) && at < (uint32_t)m) out[at] = begin + i;
        lt += __popc(l);
        eq += __popc(q);
    }
    cluster.sync();  // no CTA leaves while another may read its shared memory
}

constexpr int kMoveThreads = 256;
constexpr int kMoveLoads = 8;  // 16-byte vectors that a thread has in flight

// Copies `rows` kept rows of one (sequence, head) per CTA, k and v: all of a
// thread's loads are issued before its first store.
__global__ void __launch_bounds__(kMoveThreads) k_kv_move(KvPages c, KvTable t, KvPages d, KvTable dt, int keep, int rows, int groups,
                                                         int vecs, int elem_bytes, const int32_t* __restrict__ kept, uint32_t* status) {
    __shared__ int64_t s_src[kMoveThreads], s_dst[kMoveThreads];  // byte offsets, or -1
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x;
    const int row = blockIdx.x / groups, j0 = blockIdx.x % groups * rows;
    const int b = row / c.kv_heads, h = row % c.kv_heads;
    if (kept[(int64_t)row * keep + j0] < 0) return;
    if (tid < rows) {
        const int j = j0 + tid;
        const int p = j < keep ? kept[(int64_t)row * keep + j] : -1;
        int64_t src = -1, dst = -1;
        if (p >= 0) {
            const int from = kv_page(t, c.num_pages, b, p / c.page_size, status);
            const int to = kv_page(dt, d.num_pages, b, j / d.page_size, status);
            if (from >= 0 && to >= 0) {
                const int fs = p % c.page_size, ts = j % d.page_size;
                src = ((int64_t)from * c.page_stride + (int64_t)h * c.head_stride + (int64_t)fs * c.slot_stride) * elem_bytes;
                dst = ((int64_t)to * d.page_stride + (int64_t)h * d.head_stride + (int64_t)ts * d.slot_stride) * elem_bytes;
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
            const int k = is_v ? i - half : i, r = k / vecs, v = k - r * vecs;
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
                            int sinks, int recent, int32_t* kept, uint32_t* status, cudaStream_t s) {
    const unsigned rows = (unsigned)t.batch * (unsigned)c.kv_heads;
    KernelSetup su;
    cudaError_t e = kernel_setup(reinterpret_cast<const void*>(k_kv_select), kSelectThreads, (size_t)kMaxStaged * 4, &su);
    if (e != cudaSuccess) return e;
    // A CTA for every 4096 positions, up to the portable cluster size.
    int ranks = 1;
    while (ranks < kMaxCluster && (t.max_len + ranks - 1) / ranks > 4096) ranks *= 2;
    const int share = ((t.max_len + ranks - 1) / ranks + 3) / 4 * 4;
    const int staged = share <= kMaxStaged;
    const int vec4 = c.page_size % 4 == 0 && (reinterpret_cast<uintptr_t>(c.weight) & 15u) == 0;

    cudaLaunchAttribute at[1];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(rows * ranks);
    cfg.blockDim = dim3(kSelectThreads);
    cfg.dynamicSmemBytes = staged ? (size_t)share * 4 : 0;
    cfg.stream = s;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ranks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_kv_select, c, t, keep, sinks, recent, staged, vec4, kept, dt.lens, status);
    if (e != cudaSuccess) return e;

    const int bytes = kv_elem_bytes(c.type), vecs = c.head_dim * bytes / 16;
    int per = kMoveThreads * kMoveLoads / (2 * vecs);  // rows whose vectors are one round of loads
    per = per > kMoveThreads ? kMoveThreads : per;
    const int most = keep < t.max_len ? keep : t.max_len;
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
    return cudaLaunchKernelEx(&cfg, k_kv_move, c, t, d, dt, keep, per, groups, vecs, bytes, (const int32_t*)kept, status);
}

}  // namespace ss
