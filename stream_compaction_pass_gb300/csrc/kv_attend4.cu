// kv_attend4.cu -- attention over caches of 4 bits: the tiles, warps and stages
// of kv_attend.cuh's kernels for every row size.
#include "kv_attend.cuh"

namespace ss {

namespace {

template <typename QT> cudaError_t run_dim(const KvPages& c, const KvTable& t, const KvAttention& a, const KvScratch& mem, uint32_t* status, cudaStream_t s) {
    if (a.q_heads / c.kv_heads <= 8) {
        if (c.head_dim == 64) return run<QT, Rows8<QT, 4, 64, 32>, 4, 64, 32, 16, 4>(c, t, a, mem, status, s);
        if (c.head_dim == 128) return run<QT, Rows8<QT, 4, 128, 32>, 4, 128, 32, 12, 3>(c, t, a, mem, status, s);
        return run<QT, Rows8<QT, 4, 256, 16>, 4, 256, 16, 8, 4>(c, t, a, mem, status, s);
    }
    if (c.head_dim == 64) return run<QT, Rows16<QT, 4, 64, 32>, 4, 64, 32, 12, 4>(c, t, a, mem, status, s);
    if (c.head_dim == 128) return run<QT, Rows16<QT, 4, 128, 32>, 4, 128, 32, 8, 4>(c, t, a, mem, status, s);
    return run<QT, Rows16<QT, 4, 256, 16>, 4, 256, 16, 7, 5>(c, t, a, mem, status, s);
}

}  // namespace

cudaError_t launch_kv_attend4(const KvPages& c, const KvTable& t, const KvAttention& a, const KvScratch& mem, uint32_t* status, cudaStream_t s) {
    return a.type == KvElem::BF16 ? run_dim<__nv_bfloat16>(c, t, a, mem, status, s) : run_dim<__half>(c, t, a, mem, status, s);
}

}  // namespace ss
