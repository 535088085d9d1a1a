// Which attention kernel of the newest tokens runs: by head dimension, cache
// type, query rows of a key head, and whether some keys are masked for some rows.
#pragma once

#include "fa_decode_kernel.cuh"

namespace fa {

// What the host needs to know of a decode kernel.
struct DecodeKernel {
    const void *fn;
    int tile, ctas_per_sm, smem;
};
template <int D, int NT, int RW, bool F8, bool PARTLY>
DecodeKernel decode_kernel_of() {
    using C = DecodeConfig<D, NT, RW, F8>;
    return {reinterpret_cast<const void *>(fa_decode_kernel<D, NT, RW, F8, PARTLY>), C::kTile, C::kCtasPerSm, C::kSmemBytes};
}

// How a key head's query rows lie on warps: `tiles` of 8 rows to a warp, and
// `warps` warps that share a key range (and each load and convert all of it).
// More tiles need fewer loads and more registers, at three only two CTAs an SM
// at d = 128.  20 rows, d = 128, bf16 / E4M3: three tiles 170 / 110 us, two tiles
// on two warps 180 / 160; 32 rows: two on two 191 / 158, four on one 248 / 228;
// 40 rows: three on two 240 / 185, two on four 306 / 239.
struct DecodeLayout {
    int index, tiles, warps;
};
constexpr DecodeLayout kDecodeLayouts[6] = {{0, 1, 1}, {1, 2, 1}, {2, 3, 1}, {3, 2, 2}, {4, 3, 2}, {5, 2, 4}};
inline int decode_rows(const DecodeLayout &l) { return 8 * l.tiles * l.warps; }
// The first that holds the rows; more than the last one's go to further row
// blocks, which read the keys again.
inline DecodeLayout decode_layout(int rows) {
    for (const DecodeLayout &l : kDecodeLayouts)
        if (rows <= decode_rows(l)) return l;
    return kDecodeLayouts[5];
}
template <bool PARTLY, int D, bool F8>
DecodeKernel decode_kernel_with(const DecodeLayout &l) {
    constexpr const DecodeLayout *k = kDecodeLayouts;
    switch (l.index) {
        case 0: return decode_kernel_of<D, k[0].tiles, k[0].warps, F8, PARTLY>();
        case 1: return decode_kernel_of<D, k[1].tiles, k[1].warps, F8, PARTLY>();
        case 2: return decode_kernel_of<D, k[2].tiles, k[2].warps, F8, PARTLY>();
        case 3: return decode_kernel_of<D, k[3].tiles, k[3].warps, F8, PARTLY>();
        case 4: return decode_kernel_of<D, k[4].tiles, k[4].warps, F8, PARTLY>();
        default: return decode_kernel_of<D, k[5].tiles, k[5].warps, F8, PARTLY>();
    }
}
template <bool PARTLY>
DecodeKernel decode_kernel(int d, bool f8, const DecodeLayout &l) {
    return f8 ? (d == 64 ? decode_kernel_with<PARTLY, 64, true>(l) : decode_kernel_with<PARTLY, 128, true>(l))
              : (d == 64 ? decode_kernel_with<PARTLY, 64, false>(l) : decode_kernel_with<PARTLY, 128, false>(l));
}
// decode_kernel<true>, compiled apart (fa_decode_partly.cu): side by side with
// the others, and loaded by the calls that use it.
DecodeKernel decode_kernel_partly(int d, bool f8, const DecodeLayout &l);

}  // namespace fa
