// kv_assign.cu -- page tables and slot maps from the lengths that sequences
// grow by (streamscan.h, ss_kv_assign).
//
// Mathematics.  Three exclusive sums over the sequences place everything: of
// the new tokens (offsets), of the pages that a sequence needs beyond those it
// has, ceil((old + count) / page) - ceil(old / page) (its places in the ring of
// free pages), and of the pages that it gives back (its places behind the ring's
// end).  A sequence is served where its own sum does not pass the ring's count.
//
// What bounds it.  Latency, at decode sizes: one chain of loads (lengths, sums,
// the search of a token's sequence, its page).  So it is one launch: every CTA
// computes all sums (a few thousand sequences at most, in shared memory) and
// then takes its share of the table's entries and of the tokens, four tokens a
// thread, written as 16-byte vectors.  The ring's free part and the part behind
// it are disjoint, so pages are taken and given back side by side.  Only the
// lengths and the ring's state can be both read and written: where they are, the
// CTAs are one cluster, and its last step writes them, or, where tokens are too
// many for 8 CTAs, a second launch of one CTA.  64 sequences that get a token each
// take 4.9 us in a graph, 5.5 with lengths and state in place (the cluster); 512 of up
// to 8191 new tokens, whose 116 thousand fours of tokens are one and a half rounds of a
// CTA an SM, 7.2, in place 10.8 (two launches); 0.8 by their bytes.
#include <cooperative_groups.h>

#include <algorithm>
#include <climits>

#include "kv.cuh"

namespace ss {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32;

// Who writes the lengths, the state and the offsets.
enum class Finish : int {
    First,    // CTA 0: nothing that is read is written
    Cluster,  // CTA 0 of the grid's one cluster, when all have read
    Later,    // a launch of its own
    Only,     // this launch, of one CTA, does nothing else
};

struct Args : KvAssign {
    FastDiv page;  // by page_size
};

struct Sums {  // exclusive sums before a sequence
    int64_t tokens;
    int take, back, entries;
};

__device__ __forceinline__ int pages_of(const Args& a, int n) { return n == 0 ? 0 : a.page.div(n - 1) + 1; }

__device__ __forceinline__ int find(const int* x, int n, int at) {  // the last i < n with x[i] <= at
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (x[mid] <= at) lo = mid; else hi = mid;
    }
    return lo;
}

template <Finish F> __global__ void __launch_bounds__(kThreads) k_kv_assign(KvTable t, Args a, uint32_t* status) {
    extern __shared__ int s_sums[];
    __shared__ Sums s_warp[kWarps];
    __shared__ int s_taken;
    const int n = t.batch, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // Sums before sequence i: tokens (at most 2^31 - 1), pages taken, given back, table
    // entries; and its length before (0 where it is restarted), ~ of it where its new
    // length is not allowed.
    int *tokens = s_sums, *take = tokens + n + 1, *back = take + n + 1, *entries = back + n + 1, *before_of = entries + n + 1;
    begin_dependent();

    const int head_in = a.state[0], free_in = a.state[1];
    const bool sane = head_in >= 0 && free_in >= 0 && free_in <= a.capacity;
    const int head = sane ? (int)(head_in % a.capacity) : 0, free = sane ? free_in : 0;
    if (!sane && tid == 0) record_error(status, kErrKvTable, 0u);
    if (tid == 0) s_taken = 0;

    Sums run{0, 0, 0, 0};
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + tid;
        Sums mine{0, 0, 0, 0};
        if (i < n) {
            const int len = kv_len(t, i, status), asked = a.counts ? a.counts[i] : 1;
            const bool again = a.restart && a.restart[i];
            const int old = again ? 0 : len, had = pages_of(a, len), held = again ? 0 : had, count = max(asked, 0);
            const bool fits = asked >= 0 && (count == 0 || count <= a.limit - old);
            if (!fits) record_error(status, kErrKvTable, (uint32_t)i);
            before_of[i] = fits ? old : ~old;
            mine.tokens = count;
            mine.take = fits ? pages_of(a, old + count) - held : 0;
            mine.back = again ? had : 0;
            mine.entries = max(mine.back, held + mine.take) - (a.copy ? 0 : held);
        }
        Sums x;
        x.tokens = warp_inclusive_scan<int64_t>(mine.tokens, lane);
        x.take = warp_inclusive_scan<int>(mine.take, lane);
        x.back = warp_inclusive_scan<int>(mine.back, lane);
        x.entries = warp_inclusive_scan<int>(mine.entries, lane);
        if (lane == 31) s_warp[warp] = x;
        __syncthreads();
        Sums before = run;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const Sums y = s_warp[w];
            if (w < warp) {
                before.tokens += y.tokens;
                before.take += y.take;
                before.back += y.back;
                before.entries += y.entries;
            }
            run.tokens += y.tokens;
            run.take += y.take;
            run.back += y.back;
            run.entries += y.entries;
        }
        if (i < n) {
            tokens[i + 1] = (int)min(before.tokens + x.tokens, (int64_t)INT_MAX);
            take[i + 1] = before.take + x.take;
            back[i + 1] = before.back + x.back;
            entries[i + 1] = before.entries + x.entries;
        }
        __syncthreads();
    }
    if (tid < 4) s_sums[tid * (n + 1)] = 0;
    if (run.tokens > INT_MAX && tid == 0) record_error(status, kErrKvTable, (uint32_t)(n - 1));
    __syncthreads();

    // A sequence, from the sums.
    struct Seq {
        int old, held, need;
        bool served;
    };
    auto sequence = [&](int b) {
        const int x = before_of[b], first = take[b], last = take[b + 1];
        Seq q;
        q.old = x < 0 ? ~x : x;
        q.held = pages_of(a, q.old);
        q.need = last - first;
        q.served = x >= 0 && (q.need == 0 || last <= free);
        return q;
    };
    auto ring_at = [&](int i) {  // place i of the ring, counted from its head
        const int64_t x = (int64_t)head + i;
        return (int)(x < a.capacity ? x : x - a.capacity);
    };
    auto checked = [&](int page, int b) {
        if (page >= 0 && page < a.num_pages) return page;
        record_error(status, kErrKvTable, (uint32_t)b);
        return -1;
    };

    if constexpr (F != Finish::Only) {
        const int64_t threads = (int64_t)gridDim.x * kThreads, me = (int64_t)blockIdx.x * kThreads + tid;
        // ---- table entries: kept, given back, taken ----
        const int all = entries[n];
        for (int64_t e = me; e < all; e += threads) {
            const int b = find(entries, n, (int)e);
            const Seq q = sequence(b);
            const int col = (int)e - entries[b] + (a.copy ? 0 : q.held);
            const int mine = q.served ? q.held + q.need : q.held;
            const int had = back[b + 1] - back[b];
            int page = 0;
            if (col < had || (a.copy && col < q.held)) page = t.pages[(int64_t)b * t.row_stride + col];
            if (col < had) {
                checked(page, b);
                const int64_t to = (int64_t)free + back[b] + col;
                if (to < a.capacity) a.ring[ring_at((int)to)] = page;
                else record_error(status, kErrKvTable, (uint32_t)b);  // more pages than the ring can hold
            }
            if (col >= mine) continue;
            if (col >= q.held) page = a.ring[ring_at(take[b] + col - q.held)];
            if (a.copy || col >= q.held) a.pages[(int64_t)b * a.row_stride + col] = page;
        }
        // ---- tokens: four in a row a thread ----
        const int total = tokens[n];
        if (total > a.tokens && a.given && me == 0) record_error(status, kErrKvTable, (uint32_t)max(n - 1, 0));
        for (int64_t q0 = threads - 1 - me; q0 * 4 < a.tokens; q0 += threads) {  // threads without entries first
            const int t0 = (int)(q0 * 4), here = min(4, a.tokens - t0);
            int pos[4];
            int64_t slot[4];
            int b = -1, end = 0, first = 0, old = 0, held = 0, index = -1;
            int64_t base = 0;  // slot of the sequence's position 0, were all its pages like this one
            bool ok = false, on_page = false;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int at = t0 + k;
                pos[k] = 0;
                slot[k] = -1;
                if (k >= here || at >= total) continue;
                if (b < 0 || at >= end) {
                    if (b < 0) {
                        b = find(tokens, n, at);  // the last one that starts here: never an empty one
                    } else {
                        do ++b; while (tokens[b + 1] <= at);
                    }
                    first = tokens[b];
                    end = tokens[b + 1];
                    const Seq q = sequence(b);
                    ok = q.served;
                    old = q.old;
                    held = q.held;
                    index = -1;
                }
                pos[k] = (int)min((int64_t)old + at - first, (int64_t)INT_MAX);
                if (!ok) continue;
                const int i = a.page.div(pos[k]);
                if (i != index) {
                    index = i;
                    const int page = checked(i < held ? t.pages[(int64_t)b * t.row_stride + i] : a.ring[ring_at(take[b] + i - held)], b);
                    on_page = page >= 0;
                    base = ((int64_t)page - i) * a.page_size;
                }
                slot[k] = on_page ? base + pos[k] : -1;
            }
            if (a.vectors && here == 4) {
                if (a.positions) *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
                if (a.slots) {
                    reinterpret_cast<longlong2*>(a.slots + t0)[0] = make_longlong2(slot[0], slot[1]);
                    reinterpret_cast<longlong2*>(a.slots + t0)[1] = make_longlong2(slot[2], slot[3]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (k >= here) continue;
                    if (a.positions) a.positions[t0 + k] = pos[k];
                    if (a.slots) a.slots[t0 + k] = slot[k];
                }
            }
        }
    }

    // ---- the lengths, the ring's state and the offsets ----
    if constexpr (F == Finish::Later) return;
    if constexpr (F == Finish::Cluster) cg::this_cluster().sync();  // every CTA has read the old ones
    if (blockIdx.x != 0) return;
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + tid;
        if (i >= n) continue;
        const Seq q = sequence(i);
        if (q.served && q.need > 0) atomicMax(&s_taken, take[i + 1]);
        a.lens[i] = q.served ? q.old + tokens[i + 1] - tokens[i] : q.old;
    }
    if (a.offsets)
        for (int i = tid; i <= n; i += kThreads) a.offsets[i] = tokens[i];
    __syncthreads();
    if (tid == 0) {
        const int taken = s_taken;
        a.left[0] = ring_at(taken);
        a.left[1] = free - taken + (int)min((int64_t)back[n], a.capacity - free);
    }
}

}  // namespace

cudaError_t launch_kv_assign(const KvTable& t, const KvAssign& a, bool in_place, int sms, uint32_t* status, cudaStream_t s) {
    const size_t smem = (size_t)5 * (t.batch + 1) * 4, most = (size_t)5 * (kKvMaxAssign + 1) * 4;
    // A thread's four tokens, or its entries: those of the table where it is
    // copied, and else about as many as there are pages in the new tokens.
    const int64_t entries = a.copy ? (int64_t)t.batch * t.max_pages : t.batch;
    const int64_t work = (int64_t)(a.tokens + 3) / 4 + entries / 2;
    int grid = (int)std::min<int64_t>(sms, std::max<int64_t>(1, work / kThreads));
    const Finish f = !in_place ? Finish::First : grid <= 16 ? Finish::Cluster : Finish::Later;
    Args args;
    static_cast<KvAssign&>(args) = a;
    args.page = FastDiv(a.page_size);
    int cluster = 1;
    if (f == Finish::Cluster) {
        while (cluster < 8 && cluster < grid) cluster *= 2;
        grid = cluster;
    }
    auto* kern = f == Finish::First ? k_kv_assign<Finish::First> : f == Finish::Cluster ? k_kv_assign<Finish::Cluster> : k_kv_assign<Finish::Later>;
    KernelSetup su;
    cudaError_t e = kernel_setup(reinterpret_cast<const void*>(kern), kThreads, most, &su);
    if (e != cudaSuccess) return e;
    e = launch_dependent(kern, grid, kThreads, smem, cluster, s, t, args, status);
    if (e != cudaSuccess || f != Finish::Later) return e;
    e = kernel_setup(reinterpret_cast<const void*>(k_kv_assign<Finish::Only>), kThreads, most, &su);
    if (e != cudaSuccess) return e;
    return launch_dependent(k_kv_assign<Finish::Only>, 1, kThreads, smem, 1, s, t, args, status);
}

}  // namespace ss
