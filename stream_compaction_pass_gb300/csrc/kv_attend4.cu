// kv_attend4.cu -- attention over caches of 4 bits: the tiles, warps and stages
// of kv_attend.cuh's kernels for every row size.
#include "kv_attend.cuh"

namespace ss {

namespace {

// A row is a quarter of a 16-bit one, but its codes take as many instructions to
// open as 16-bit values take bytes to load (issued in 61 % of the cycles at 0.76 of the
// copy rate), so large tiles spread what one costs at least: of 64 positions, with as
// many warps, in fours for the SM's four schedulers, as registers and shared memory
// allow, two stages each.  2.2 million positions of 8 x 8 heads of 128: tiles of 64
// with 12 warps 495 us, 11 548; of 32 with 16 warps 582, 12 570.  A ragged batch with
// weights 76.1, 79.1, 83.1, 78.3.  32 x 4000 to 8000 positions, tiles of 64 / 32: 16
// heads of 64 62.8 / 71.9 us (16 warps), 16 query heads a key-value head 83.9 / 86.1
// (8), of 64 91.4 / 97.5 (12); heads of 256, tiles of 32 with 8 warps 58.7, with 16
// query heads 110.9 / 109.1 (tiles of 32 / 16, 7 warps).
// Calls of one launch want few warps to start and more of them at work, hence
// tiles of 32 with 8 warps: 1021 positions 6.9 us (12 warps 6.9, 16 9.1), 4000 8.4
// (8.6, 9.2), 16,000 16.9 (16.0, 16.2).
template <typename QT> cudaError_t run_dim(const KvPages& c, const KvTable& t, const KvAttention& a, const KvScratch& mem, uint32_t* status, cudaStream_t s) {
    if (a.q_heads / c.kv_heads <= 8) {
        if (c.head_dim == 64) return run<QT, Rows8<QT, 4, 64, 64>, 4, 64, 64, 16, 2, Shape<Rows8<QT, 4, 64, 32>, 4, 64, 32, 8, 3>>(c, t, a, mem, status, s);
        if (c.head_dim == 128) return run<QT, Rows8<QT, 4, 128, 64>, 4, 128, 64, 12, 2, Shape<Rows8<QT, 4, 128, 32>, 4, 128, 32, 8, 3>>(c, t, a, mem, status, s);
        return run<QT, Rows8<QT, 4, 256, 32>, 4, 256, 32, 8, 2>(c, t, a, mem, status, s);
    }
    if (c.head_dim == 64) return run<QT, Rows16<QT, 4, 64, 64>, 4, 64, 64, 12, 2, Shape<Rows16<QT, 4, 64, 32>, 4, 64, 32, 8, 3>>(c, t, a, mem, status, s);
    if (c.head_dim == 128) return run<QT, Rows16<QT, 4, 128, 64>, 4, 128, 64, 8, 2, Shape<Rows16<QT, 4, 128, 32>, 4, 128, 32, 8, 3>>(c, t, a, mem, status, s);
    return run<QT, Rows16<QT, 4, 256, 32>, 4, 256, 32, 7, 2, Shape<Rows16<QT, 4, 256, 16>, 4, 256, 16, 7, 5>>(c, t, a, mem, status, s);
}

}  // namespace

cudaError_t launch_kv_attend4(const KvPages& c, const KvTable& t, const KvAttention& a, const KvScratch& mem, uint32_t* status, cudaStream_t s) {
    return a.type == KvElem::BF16 ? run_dim<__nv_bfloat16>(c, t, a, mem, status, s) : run_dim<__half>(c, t, a, mem, status, s);
}

}  // namespace ss
