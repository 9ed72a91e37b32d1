// kv_attend.cu -- attention over caches of 16 and 8 bits: the tiles, warps and
// stages of kv_attend.cuh's kernels for every row size.
#include "kv_attend.cuh"

namespace ss {

namespace {

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
template <typename QT, bool NARROW>
cudaError_t run_dim(const KvPages& c, const KvTable& t, const KvAttention& a, const KvScratch& mem, uint32_t* status, cudaStream_t s) {
    constexpr int kBits = NARROW ? 8 : 16;
    if (a.q_heads / c.kv_heads <= 8) {
        if (c.head_dim <= 64) return run<QT, Rows8<QT, kBits, 64, 32>, kBits, 64, 32, NARROW ? 16 : 12, NARROW ? 3 : 2>(c, t, a, mem, status, s);
        if (c.head_dim <= 128) return run<QT, Rows8<QT, kBits, 128, NARROW ? 32 : 16>, kBits, 128, NARROW ? 32 : 16, 12, 2>(c, t, a, mem, status, s);
        return run<QT, Rows8<QT, kBits, 256, 16>, kBits, 256, 16, NARROW ? 8 : 4, 3>(c, t, a, mem, status, s);
    }
    if (c.head_dim <= 64) return run<QT, Rows16<QT, kBits, 64, 32>, kBits, 64, 32, NARROW ? 12 : 8, NARROW ? 4 : 3>(c, t, a, mem, status, s);
    if (c.head_dim <= 128) return run<QT, Rows16<QT, kBits, 128, NARROW ? 32 : 16>, kBits, 128, NARROW ? 32 : 16, 8, 3>(c, t, a, mem, status, s);
    return run<QT, Rows16<QT, kBits, 256, 16>, kBits, 256, 16, NARROW ? 7 : 4, 3>(c, t, a, mem, status, s);
}

}  // namespace

cudaError_t launch_kv_attend(const KvPages& c, const KvTable& t, const KvAttention& a, const KvScratch& mem, uint32_t* status, cudaStream_t s) {
    const bool bf = a.type == KvElem::BF16;
    if (c.type == KvElem::E2M1) return launch_kv_attend4(c, t, a, mem, status, s);
    if (c.type == KvElem::E4M3)
        return bf ? run_dim<__nv_bfloat16, true>(c, t, a, mem, status, s) : run_dim<__half, true>(c, t, a, mem, status, s);
    return bf ? run_dim<__nv_bfloat16, false>(c, t, a, mem, status, s) : run_dim<__half, false>(c, t, a, mem, status, s);
}

}  // namespace ss
