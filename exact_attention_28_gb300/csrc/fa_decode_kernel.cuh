// Attention of the newest tokens of each sequence over the paged cache.
//
//   S_j = scale * q . k_j over the visible keys j of the sequence,
//   O = sum_j exp(S_j - m) v_j / l,  LSE = m + ln l,
// one pass with the running maximum m and sum l ("9.4 FlashAttention 与
// FlashMLA" section 9.4.2), the keys in parallel slices that are merged
// afterwards ("6. FlashAttention 分块逻辑" sections 11 and 13.2).
//
// What bounds it.  A key and a value (4 d bytes in bf16) meet the R = Hq / Hkv
// * Nq query rows of their head: 4 R d FLOPs, R FLOPs a byte, against about
// 290 that the tensor cores could do: the cache has to stream at the memory's
// rate, and everything else hides behind it.  So:
// * Work is dealt out by the lengths themselves, on the device.  A unit is one
//   tile of TK keys of one (sequence, key head, block of query rows), 32 KB of
//   cache whatever the type; the C CTAs take equal runs of the list of all
//   units, so a long sequence spreads over the GPU and short ones share a CTA.
// * A CTA has two tiles of 32 KB, one in use and one on its way by 16-byte
//   asynchronous copies, and three CTAs share an SM: 96 KB in flight on each
//   (DecodeConfig: where three do not fit, two, with a third tile if that fits).
//   (16 KB tiles cost 15 to 35% on 48 x 16 heads of up to 6007 keys in E4M3.)
//   Each warp copies and (with up to 24 rows) uses its own quarter of a tile,
//   so warps wait for nobody inside a segment.  An item's queries come the
//   same way with its first tile: loaded when they were needed, they cost 2 us
//   an item under the cache's traffic.
//   Copies of keys past the end or of unallocated blocks are zero-filled
//   instead: nothing behind a sequence's end is read.
// * The products run on mma.sync: up to 32 rows of a key head (E4M3: 16) the
//   tensor pipe is not what limits.  Scores and outputs are held transposed, with keys
//   (channels of O) down the 16 rows of a product and 8 query rows across: a
//   fragment of the cache, once loaded and converted, serves all of a warp's
//   rows, and their number is rounded up to 8 only.  (16 query rows down: 82.3
//   us on one sequence of 131,035 keys, now 81.2; 24 rows, E4M3: 137.6, 113.1.)
//   The scores never leave registers.
// * P is held as two bf16 terms (bf16 cache) or in fp16 (E4M3 cache, whose
//   codes are exact in fp16; q, scaled by a power of two per row, keeps all
//   its bits): the weights' rounding stays far below the output's.
// 64 sequences of 0 to 8192 keys, 32 query and 8 key heads, d = 128, bf16, 16-key
// blocks: 159.7 us, 6.73 TB/s (the measured copy rate is 6.69); one of 131,035
// keys 81.2 us (99%); 48 of 3 to 6007 keys, 16 heads, d = 64, E4M3, 4 new tokens
// 51.9 us, 5.71 TB/s (85%).  The 64 sequences with 64 query and 8 key heads and
// 2, 3, 4, 5 and 8 new tokens (16, 24, 32, 40 and 64 rows), d = 128, of the copy
// rate: bf16 95%, 92%, 87%, 65%, 55%; E4M3 83%, 71%, 55%, 43%, 35%.  From 32 rows
// on (E4M3: 24) mma.sync, at 8 cycles of an SM's quarter each, is what bounds it,
// with the conversions beside it, which each of a team's warps repeats; and from
// 33 rows on at d = 128 an SM holds two CTAs of two stages, 64 KB on the way.
#pragma once

#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx_sm103.cuh"

namespace fa {

constexpr int kDecodeThreads = 128;
constexpr int kDecodeWarps = kDecodeThreads / 32;
constexpr int kDecodeMaxCtas = 480;                                 // at most three per SM of 160
// What beginning and ending an item costs, in units: without it the CTAs with
// many short items finish last.  48 x 16 heads of 3 to 6007 keys, E4M3, d = 64:
// 51.7 us with 1, 51.8 with 2, 52.4 with 3; 24 query rows, E4M3, d = 128: 122.3,
// 113.1, 108.2; 160 sequences of up to 200 keys: 18.4, 18.5, 18.9.
constexpr int kDecodeItemUnits = 2;
// Two units arrive together at the start, so spreading work thinner only adds
// partial results: 8 sequences of up to 1000 keys 7.7 us, one unit each 8.8.
constexpr int kDecodeLeastUnits = 2;
constexpr float kDecodeTau = 8.0f;                                  // log2 units before a maximum is raised

// What a CTA leaves for the merge: the item whose first tiles it had but not
// its last ones (-1: none), its partial result's slot, and the CTA with the
// item's last tiles.  The CTAs between them left theirs in slots 2 c.
struct DecodeJob {
    int item, slot, last_cta, pad;
};

struct DecodeParams {
    const __nv_bfloat16 *q;
    __nv_bfloat16 *o;
    float *lse;
    int64_t qs[3], os[3];                 // batch, head, token strides in elements
    const void *k_cache, *v_cache;
    const float *k_descale, *v_descale;   // nullptr for a bf16 cache
    const int *block_table, *seq_lens;
    int B, Hq, Hkv, Nq, max_blocks, num_blocks, block_shift;
    int group;                            // Hq / Hkv
    int rows;                             // query rows of a key head: group * Nq
    int row_blocks;                       // blocks of 8 NT RW rows
    int part_rows;                        // rows of a partial result
    int causal;
    int whole_items;                      // no item is shared between CTAs: there is no merge
    float c2;                             // |scale| * log2(e), positive
    uint32_t q_sign;                      // sign bits to flip in q (scale < 0)
    DecodeJob *jobs;                      // [CTAs]
    float2 *part_ml;                      // [2 CTAs][part_rows]: m (log2 units), l
    float *part_o;                        // [2 CTAs][part_rows][D]
};

namespace dec {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// D += A B, 16 x 8 x 16, fp32 accumulator; F16: fp16 operands, else bf16.
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four E4M3 codes to two packed fp16 pairs, exactly; byte 0 is the first.
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// The 8 x 8 matrix of 16-bit elements whose row lane / 4 each lane holds two of, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
// 0xff.. at the elements of a word (two bf16, four E4M3 codes) that are NaN or infinite.
template <bool F8>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
    return F8 ? __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu) : __vcmpeq2(w & 0x7f807f80u, 0x7f807f80u);
}
// Over the eight lanes of a warp that have the same lane % 4.
__device__ __forceinline__ float column_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float column_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

}  // namespace dec

// a / b for b > 0, in 32 bits where a has them (a 64-bit division is a long
// chain of instructions, and a CTA's first copy waits for it).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

template <int D, int NT, int RW, bool F8>
struct DecodeConfig {
    static constexpr int kRowBytes = D * (F8 ? 1 : 2);
    static constexpr int kWarpBytes = 8192;                          // one warp's K and V of a stage
    static constexpr int kStageBytes = kDecodeWarps * kWarpBytes;
    static constexpr int kRows = 8 * NT;                             // query rows of a warp
    static constexpr int kQueryBytes = kRows * RW * D * 2 + 16;      // an item's queries and descales
    // three CTAs an SM where their registers and shared memory fit, else two with more tiles on their way
    static constexpr int kOtherBytes = 1024 + kDecodeWarps * kRows * 8 + kRows * RW * 12 + 256;   // the system's, static arrays
    static constexpr bool kThree = D * NT <= 256 && 3 * (2 * kStageBytes + kQueryBytes + kOtherBytes) <= 228 * 1024;
    static constexpr int kCtasPerSm = kThree ? 3 : 2;
    static constexpr int kStages = !kThree && 2 * (3 * kStageBytes + 2 * kQueryBytes + kOtherBytes) <= 228 * 1024 ? 3 : 2;
    static constexpr int kSmemBytes = kStages * kStageBytes + (kStages - 1) * kQueryBytes;
    static constexpr int kKeys = kWarpBytes / 2 / kRowBytes;         // keys of a warp's quarter: 16, 32 or 64
    static constexpr int kTile = kDecodeWarps * kKeys;               // keys of a tile
    static constexpr int kChunks = kRowBytes / 16;                   // 16-byte pieces of a row
    // Byte offset of piece c of row r: pieces permuted so that the 8 rows an
    // ldmatrix phase reads at one c lie in different banks.
    __device__ static __forceinline__ uint32_t at(int r, int c) {
        if constexpr (kRowBytes == 64) return (r >> 1) * 128 + ((((r & 1) * 4 + c) ^ ((r >> 1) & 7)) << 4);
        else return r * kRowBytes + ((c ^ (r & 7)) << 4);
    }
};

// A position in the list of units: tile j of the nt tiles of row block rb of
// key head h of sequence b.  An item (b, h, rb) takes up kDecodeItemUnits
// units of its own in front of its tiles, so that the CTAs with many short
// items get fewer tiles; `left` is how far the CTA's run goes on from here.
struct DecodeCursor {
    int b, h, rb, j, nt, len, left;
};

// Everything that an earlier kernel of the stream may have written is read
// with plain loads: the read-only path does not promise to see it here.
__device__ __forceinline__ int sequence_length(const DecodeParams &p, int b) {
    return min(max(p.seq_lens[b], 0), p.max_blocks << p.block_shift);
}

// The next tile (of this CTA, if `left` stays positive).
template <int TILE>
__device__ __forceinline__ void advance(const DecodeParams &p, DecodeCursor &c) {
    --c.left;
    if (++c.j < c.nt) return;
    c.j = 0;
    if (c.left <= (p.whole_items ? 0 : kDecodeItemUnits)) {
        c.left = 0;
        return;
    }
    if (++c.rb == p.row_blocks) {
        c.rb = 0;
        if (++c.h == p.Hkv) {
            c.h = 0;
            do {
                ++c.b;
                c.len = sequence_length(p, c.b);
                c.nt = (c.len + TILE - 1) / TILE;
            } while (c.nt == 0 && c.b + 1 < p.B);
        }
    }
    c.left -= kDecodeItemUnits;
    if (p.whole_items) c.left = max(c.left, c.nt);
}

// Units of one item of a sequence with this length, and of sequence b.
template <int TILE>
__device__ __forceinline__ int length_units(const DecodeParams &p, int len) {
    const int nt = (min(max(len, 0), p.max_blocks << p.block_shift) + TILE - 1) / TILE;
    return nt ? nt + kDecodeItemUnits : 0;
}
template <int TILE>
__device__ __forceinline__ int item_units(const DecodeParams &p, int b) {
    return length_units<TILE>(p, p.seq_lens[b]);
}

// What becomes of a row's sum of weights: the factor of its O, and its LSE
// from m in log2 units.  A sum is 0 where no key was visible (else it holds m's
// own weight, 1 or more), which leaves O = 0 and LSE = -inf; NaN, from a NaN
// among the row's query and keys, goes on to both.
__device__ __forceinline__ float over_sum(float x, float sum) { return sum == 0.f ? 0.f : x / sum; }
__device__ __forceinline__ float log_sum(float m, float sum) {
    return sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
}

// Adds the values that are not finite, of the newest keys that not every row
// sees, to the rows that see them: to O, or (part >= 0) to the partial results
// from row `part` on.  The whole CTA calls it, after rows [row0, row0 + n_rows)
// of this item were written; a thread has its channels to itself.
template <int D, bool F8>
__device__ __noinline__ void add_not_finite(const DecodeParams &p, int b, int h, int len, int64_t part, int row0, int n_rows) {
    const int first = len - p.Nq + 1;          // keys that row n sees end at first + n
    for (int c = threadIdx.x; c < D; c += kDecodeThreads)
        for (int r = 0; r < n_rows; ++r) {
            const int head = (row0 + r) / p.Nq, n = row0 + r - head * p.Nq;
            float x = 0.f;
            for (int key = max(first, 0); key < first + n; ++key) {
                const int page = p.block_table[static_cast<int64_t>(b) * p.max_blocks + (key >> p.block_shift)];
                if (page < 0 || page >= p.num_blocks) continue;
                const int64_t at = (((static_cast<int64_t>(page) * p.Hkv + h) << p.block_shift) +
                                    (key & ((1 << p.block_shift) - 1))) * D + c;
                const uint32_t v = F8 ? static_cast<const uint8_t *>(p.v_cache)[at] : static_cast<const uint16_t *>(p.v_cache)[at];
                if (dec::not_finite<F8>(v) & 1) x += __uint_as_float(F8 ? 0x7fc00000u : v << 16);
            }
            if (x == 0.f) continue;
            if (part >= 0) {
                p.part_o[(part + r) * D + c] += x;
            } else {
                __nv_bfloat16 &o = p.o[b * p.os[0] + (h * p.group + head) * p.os[1] + n * p.os[2] + c];
                o = __float2bfloat16_rn(__bfloat162float(o) + x);
            }
        }
}

// O = 0, LSE = -inf for every row of sequence b, which has no keys.
template <int D>
__device__ void write_empty_sequence(const DecodeParams &p, int b) {
    for (int i = threadIdx.x; i < p.Hq * p.Nq * (D / 8); i += kDecodeThreads) {
        const int row = i / (D / 8), h = row / p.Nq, n = row - h * p.Nq;
        *reinterpret_cast<uint4 *>(p.o + b * p.os[0] + h * p.os[1] + n * p.os[2] + (i % (D / 8)) * 8) =
            make_uint4(0, 0, 0, 0);
        if (i % (D / 8) == 0) p.lse[static_cast<int64_t>(b) * p.Hq * p.Nq + row] = -INFINITY;
    }
}

// RW warps of a team share their quarters of a tile; each has 8 NT of the
// 8 NT RW query rows.  RW = 1: four teams of one warp, each with its own keys.
// PARTLY: the newest keys are masked for some rows (several causal new tokens).
// One new token has no such keys, and pays nothing for them in a kernel of its
// own: one short sequence 4.5 us (with PARTLY's code 4.6), 4000 of up to 20
// keys 155 us (163).
template <int D, int NT, int RW, bool F8, bool PARTLY>
__global__ void __launch_bounds__(kDecodeThreads, (DecodeConfig<D, NT, RW, F8>::kCtasPerSm)) fa_decode_kernel(const __grid_constant__ DecodeParams p) {
    using C = DecodeConfig<D, NT, RW, F8>;
    constexpr int kTeams = kDecodeWarps / RW;
    constexpr int kRows = C::kRows;
    constexpr int kMT = D / 16;                // 16-channel tiles of O
    constexpr int kGroups = C::kKeys / 16;     // 16-key groups of a quarter
    // 16-key groups of a step, from the team's quarters: as many as registers
    // allow, for each step is a chain of scores, maximum and weights (12 to 16
    // rows, d = 64, E4M3: 57.4 us with one, 54.5 with two, 53.3 with four; d =
    // 128, 32 rows, where four do not fit: 156.7, 147.2, 175.3).
    constexpr int kMost = (C::kThree && D == 128 ? 4 : 8) / NT;
    constexpr int kStep = RW * kGroups < kMost ? RW * kGroups : kMost;
    // fp16 weights are lifted by 2^7, to at most 2^15: keys up to 2^-31 of the
    // row's largest weight then still count (a million at 2^-24 are 6% of it).
    constexpr float kLift = F8 ? 7.f : 0.f;
    extern __shared__ __align__(1024) uint8_t ring[];
    __shared__ float sm_m[kDecodeWarps][kRows], sm_l[kDecodeWarps][kRows];
    __shared__ float sm_factor[kRows * RW];
    __shared__ int64_t sm_out[kRows * RW];
    __shared__ uint32_t sm_alloc[C::kStages][kDecodeWarps];
    __shared__ int64_t sm_scan[kDecodeWarps];
    __shared__ int sm_first_b;
    __shared__ int64_t sm_first_u;
    __shared__ int sm_taken_out;               // values that are not finite were, in this segment (PARTLY)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const int cta = blockIdx.x, ctas = gridDim.x;

    ptx::griddep_wait();
    dec::launch_dependents();

    // ---- this CTA's run [u0, u1) of the units, and the sequence of the first
    const int64_t heads = static_cast<int64_t>(p.Hkv) * p.row_blocks;
    static_assert(kDecodeLeastUnits == 2, "a shift below");
    int active, first_b = 0;                   // CTAs with units: kDecodeLeastUnits or more each, one of them less if the total is odd
    int64_t units = 0, u0, u1, first_u = 0;    // first_u: where u0 lies among the units of sequence first_b
    const auto take_run = [&] {
        active = static_cast<int>(min(static_cast<int64_t>(ctas), p.whole_items ? units : (units + 1) >> 1));
        u0 = cta < active ? quotient(units * cta, active) : 0;
        u1 = cta < active ? quotient(units * (cta + 1), active) : 0;
    };
    const auto inclusive_sum = [&](int64_t x) {
        #pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        return x;
    };
    if (p.B <= 32) {
        // every warp for itself, a lane for each sequence: the start of a small call waits for no barrier
        const int len = lane < p.B ? sequence_length(p, lane) : 0;
        const int64_t mine = heads * length_units<C::kTile>(p, len), incl = inclusive_sum(mine), before = incl - mine;
        units = __shfl_sync(0xffffffffu, incl, 31);
        take_run();
        first_b = max(__ffs(__ballot_sync(0xffffffffu, before <= u0 && u0 < incl)) - 1, 0);
        first_u = u0 - __shfl_sync(0xffffffffu, before, first_b);
        for (int b = cta; b < p.B; b += ctas)
            if (__shfl_sync(0xffffffffu, len, b) == 0) write_empty_sequence<D>(p, b);
    } else {
        // a thread's sequences: one, or a multiple of four that come by 16-byte loads
        int per = (p.B + kDecodeThreads - 1) / kDecodeThreads;
        if (per > 1) per = (per + 3) & ~3;
        const int b_lo = min(tid * per, p.B), b_hi = min(b_lo + per, p.B);
        int64_t mine = 0;
        if (per > 1 && (reinterpret_cast<uintptr_t>(p.seq_lens) & 15) == 0) {
            #pragma unroll 4
            for (int b = b_lo; b < b_hi; b += 4) {
                if (b + 4 <= p.B) {
                    const int4 n = *reinterpret_cast<const int4 *>(p.seq_lens + b);
                    mine += length_units<C::kTile>(p, n.x) + length_units<C::kTile>(p, n.y) +
                            length_units<C::kTile>(p, n.z) + length_units<C::kTile>(p, n.w);
                } else {
                    for (int c = b; c < p.B; ++c) mine += item_units<C::kTile>(p, c);
                }
            }
        } else {
            for (int b = b_lo; b < b_hi; ++b) mine += item_units<C::kTile>(p, b);
        }
        mine *= heads;
        const int64_t incl = inclusive_sum(mine);
        if (lane == 31) sm_scan[warp] = incl;
        __syncthreads();
        int64_t before = incl - mine;
        #pragma unroll
        for (int w = 0; w < kDecodeWarps; ++w) {
            if (w < warp) before += sm_scan[w];
            units += sm_scan[w];
        }
        take_run();
        if (cta < active && before <= u0 && u0 < before + mine) {
            int b = b_lo;
            int64_t u = before;
            for (; b + 1 < b_hi; ++b) {
                const int64_t n = heads * item_units<C::kTile>(p, b);
                if (u0 < u + n) break;
                u += n;
            }
            sm_first_b = b;
            sm_first_u = u0 - u;
        }
        for (int b = cta; b < p.B; b += ctas)
            if (sequence_length(p, b) == 0) write_empty_sequence<D>(p, b);
        __syncthreads();
        first_b = sm_first_b;
        first_u = sm_first_u;
    }
    DecodeCursor cur;
    cur.left = 0;
    if (u0 < u1) {
        cur.b = first_b;
        cur.len = sequence_length(p, cur.b);
        cur.nt = (cur.len + C::kTile - 1) / C::kTile;
        const int cost = cur.nt + kDecodeItemUnits;
        const int hr = static_cast<int>(quotient(first_u, cost));
        const int at = static_cast<int>(first_u - static_cast<int64_t>(hr) * cost);
        const int skip = max(kDecodeItemUnits - at, 0);      // of the item's own units in front of the first tile
        cur.j = max(at - kDecodeItemUnits, 0);
        cur.h = hr / p.row_blocks;
        cur.rb = hr - cur.h * p.row_blocks;
        cur.left = static_cast<int>(u1 - u0) - skip;
        if (p.whole_items) {     // items that begin in the run, to their ends
            if (at == 0) {
                cur.left = max(cur.left, cur.nt);
            } else {             // the rest of this one is its beginner's
                cur.left = static_cast<int>(u1 - u0) - (cost - at) + 1;
                cur.j = cur.nt - 1;
                advance<C::kTile>(p, cur);
            }
        }
    }
    if (cur.left <= 0) {
        if (tid == 0) p.jobs[cta].item = -1;
        return;
    }

    // ---- copies: this warp's quarter of a unit's tile
    const uint32_t ring0 = ptx::smem_addr(ring);
    const int block_mask = (1 << p.block_shift) - 1;
    auto first_key = [&](const DecodeCursor &c) { return c.j * C::kTile + warp * C::kKeys; };
    // lane x < kKeys / 16 gets the block of this warp's x-th 16 keys (16 keys never straddle a block)
    auto lookup = [&](const DecodeCursor &c) {
        const int key = first_key(c) + 16 * lane;
        int page = -1;
        if (lane < C::kKeys / 16 && key < c.len)
            page = p.block_table[static_cast<int64_t>(c.b) * p.max_blocks + (key >> p.block_shift)];
        return page;
    };
    constexpr int kRowsPer = 512 / C::kRowBytes;       // rows one warp-wide copy covers
    const int my_row = lane / C::kChunks, my_piece = lane % C::kChunks;
    const uint32_t my_to = ring0 + warp * C::kWarpBytes + C::at(my_row, my_piece);
    const char *const my_k = static_cast<const char *>(p.k_cache) + lane * 16;
    const char *const my_v = static_cast<const char *>(p.v_cache) + lane * 16;
    auto copy = [&](const DecodeCursor &c, int stage, int page) {
        const uint32_t dst = my_to + stage * C::kStageBytes;
        const int key0 = first_key(c);
        #pragma unroll
        for (int x = 0; x < C::kKeys / 16; ++x) {
            const int pg = __shfl_sync(0xffffffffu, page, x);
            const bool there = pg >= 0 && pg < p.num_blocks;
            // not there: nothing is read, and the address is the cache's own first rows
            const int64_t off = there ? (((static_cast<int64_t>(pg) * p.Hkv + c.h) << p.block_shift) +
                                         ((key0 + 16 * x) & block_mask)) * C::kRowBytes : 0;
            const int rows = there ? c.len - (key0 + 16 * x) - my_row : 0;
            #pragma unroll
            for (int y = 0; y < 16 / kRowsPer; ++y) {
                // C::at(16 x + y kRowsPer + row, piece): y moves the lane's place by whole rows and flips its piece's bits
                constexpr int kHalf = C::kRowBytes == 64 ? 2 : 1;
                const uint32_t to = (dst ^ ((((16 * x + y * kRowsPer) / kHalf) & 7) << 4)) + (16 * x + y * kRowsPer) * C::kRowBytes;
                const bool in = y * kRowsPer < rows;
                dec::cp_async16(to, my_k + off + y * 512, in);
                dec::cp_async16(to + C::kWarpBytes / 2, my_v + off + y * 512, in);
            }
        }
        const uint32_t bits = __ballot_sync(0xffffffffu, page >= 0);
        if (lane == 0) sm_alloc[stage][warp] = bits;
    };
    const int team = warp / RW, row_tile = warp % RW;
    const uint32_t k_lane = C::at(lane & 15, lane >> 4);
    const uint32_t v_lane = C::kWarpBytes / 2 + (F8 ? k_lane : C::at((lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1));
    static_assert(kGroups % kStep == 0 || kStep % kGroups == 0, "a step begins with a group or a quarter");
    // Query row `row` of an item's row block; nullptr behind the last one.
    auto query_row = [&](const DecodeCursor &c, int row, int &n) -> const __nv_bfloat16 * {
        row += c.rb * kRows * RW;
        const int head = p.Nq == 1 ? row : row / p.Nq;
        n = row - head * p.Nq;
        return row < p.rows ? p.q + c.b * p.qs[0] + (c.h * p.group + head) * p.qs[1] + n * p.qs[2] : nullptr;
    };

    // Queries lie behind the ring, in the one or two buffers that items which
    // have begun to arrive need; pieces permuted as in C::at.
    const uint32_t queries0 = ring0 + C::kStages * C::kStageBytes;
    uint32_t queries = queries0, queries_next = queries0;
    const auto queries_at = [](uint32_t base, int row, int piece) { return base + row * D * 2 + ((piece ^ (row & 7)) << 4); };
    const auto other = [&](uint32_t base) {
        return C::kStages == 2 ? base : queries0 + (base == queries0 ? C::kQueryBytes : 0);
    };

    DecodeCursor ahead = cur;
    int page = lookup(ahead);
    bool new_item = true;
    auto issue = [&](int stage) {
        if (ahead.left > 0) {
            if (new_item) {      // its queries come with its first tile
                #pragma unroll
                for (int x = tid; x < kRows * RW * (D / 8); x += kDecodeThreads) {
                    int n;
                    const int row = x / (D / 8), piece = x % (D / 8);
                    const __nv_bfloat16 *q = query_row(ahead, row, n);
                    dec::cp_async16(queries_at(queries_next, row, piece), q ? q + piece * 8 : p.q, q != nullptr);
                }
                if constexpr (F8)
                    if (tid < 2)
                        dec::cp_async4(queries_next + C::kQueryBytes - 16 + tid * 4,
                                       (tid ? p.v_descale : p.k_descale) + ahead.h);
                queries_next = other(queries_next);
            }
            copy(ahead, stage, page);
            advance<C::kTile>(p, ahead);
            new_item = ahead.j == 0;
            if (ahead.left > 0) page = lookup(ahead);
        }
        dec::cp_commit();
    };
    #pragma unroll
    for (int s = 0; s < C::kStages - 1; ++s) issue(s);

    // ---- the segments of the run: all tiles here of one (sequence, key head, row block)
    uint32_t qf[NT][D / 16][2];  // of query row 8 t + g
    float crow[NT][2];           // of query rows 8 t + 2 t4 and the next, like m, l and o
    float o[NT][kMT][4], m[NT][2], l[NT][2];
    int lim[NT], lim_all = 0;    // visible keys of row 8 t + g, of every row
    float dv = 1.f;              // v_descale
    bool first_segment = true;
    int my_job_item = -1, my_job_slot = 0, my_job_last = 0;
    int segment_start = -1;      // the segment's first tile, -1 in front of it
    int stage = 0;
    for (; cur.left > 0; stage = stage + 1 == C::kStages ? 0 : stage + 1) {
        dec::cp_wait<C::kStages - 2>();
        if (segment_start < 0) {
            __syncthreads();     // every warp's part of the queries is there
            segment_start = cur.j;
            if (PARTLY && tid == 0) sm_taken_out = 0;
            lim_all = p.causal ? cur.len - p.Nq + 1 : cur.len;
            if constexpr (F8) {
                // q to fp16, scaled by a power of two so that the row's
                // largest element lies in [2^14, 2^15): every bf16 bit of
                // elements down to 2^-28 of it survives.  A thread has 8
                // elements; of every 16 those that a lane has codes of, four
                // in a row, go where the product wants their pairs, 8 apart.
                float kd;
                asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(kd), "=f"(dv) : "r"(queries + C::kQueryBytes - 16) : "memory");
                const float base = p.c2 * fabsf(kd), sign = (p.q_sign != 0) != (kd < 0.f) ? -1.f : 1.f;
                #pragma unroll
                for (int x = tid; x < kRows * RW * (D / 8); x += kDecodeThreads) {
                    const int row = x / (D / 8), piece = x % (D / 8);
                    const uint32_t at = queries_at(queries, row, piece);
                    uint32_t w[4];
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                 : "r"(at) : "memory");
                    float top = 0.f;
                    #pragma unroll
                    for (int i = 0; i < 4; ++i)
                        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
                    #pragma unroll
                    for (int i = 1; i < D / 8; i <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
                    const int e = static_cast<int>(__float_as_uint(top) >> 23);      // biased exponent
                    const int k = (e == 0 || e == 255) ? 0 : min(141 - e, 126);      // 2^k * top in [2^14, 2^15)
                    const float up = sign * __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
                    // kept a normal number: a masked score is -inf times it
                    if (piece == 0) sm_factor[row] = fmaxf(base * __uint_as_float(static_cast<uint32_t>(127 - k) << 23), 0x1p-126f);
                    #pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = dec::pack_f16x2(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xFFFF0000u) * up);
                    const bool odd = piece & 1;
                    const uint32_t g0 = __shfl_xor_sync(0xffffffffu, odd ? w[0] : w[1], 1);
                    const uint32_t g1 = __shfl_xor_sync(0xffffffffu, odd ? w[2] : w[3], 1);
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(odd ? g0 : w[0]), "r"(odd ? g1 : w[2]),
                                 "r"(odd ? w[1] : g0), "r"(odd ? w[3] : g1) : "memory");
                }
                __syncthreads();
            }
            #pragma unroll
            for (int t = 0; t < NT; ++t) {
                #pragma unroll
                for (int n = 0; n < kMT; ++n) o[t][n][0] = o[t][n][1] = o[t][n][2] = o[t][n][3] = 0.f;
                m[t][0] = m[t][1] = -INFINITY;
                l[t][0] = l[t][1] = 0.f;
                const int row = row_tile * kRows + 8 * t;
                int n;
                const bool there = query_row(cur, row + g, n) != nullptr;
                lim[t] = p.causal && there ? cur.len - p.Nq + 1 + n : cur.len;
                #pragma unroll
                for (int x = 0; x < 2; ++x) crow[t][x] = F8 ? sm_factor[row + 2 * t4 + x] : p.c2;
                #pragma unroll
                for (int kk = 0; kk < D / 16; kk += 2) {
                    uint32_t r[4];
                    dec::ldsm4(r, queries_at(queries, row + (lane & 7), 2 * kk + (lane >> 3)));
                    #pragma unroll
                    for (int x = 0; x < 4; ++x) qf[t][kk + (x >> 1)][x & 1] = F8 ? r[x] : r[x] ^ p.q_sign;
                }
            }
            queries = other(queries);
            __syncthreads();     // the buffer is free for a later item's
        } else if constexpr (RW == 1) __syncwarp();
        else if constexpr (RW == 4) __syncthreads();
        else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(RW * 32) : "memory");
        issue(stage == 0 ? C::kStages - 1 : stage - 1);      // the stage used up last

        // The newest keys, which only the later of several new tokens see: a
        // weight of 0 does not mask a value that is not finite.  Such values are
        // taken out of the tile, and added to the rows that see them at the
        // segment's end.  (The warps of a team do it side by side.)
        if (PARTLY && (cur.j + 1) * C::kTile > lim_all) {
            const int team0 = cur.j * C::kTile + team * RW * C::kKeys, lo = max(lim_all - team0, 0);
            const int pieces = (min(cur.len - team0, RW * C::kKeys) - lo) * C::kChunks;
            #pragma unroll 1
            for (int x = lane; x < pieces; x += 32) {
                const int k = lo + x / C::kChunks;
                const uint32_t at = ring0 + stage * C::kStageBytes + (team * RW + k / C::kKeys) * C::kWarpBytes +
                                    C::kWarpBytes / 2 + C::at(k % C::kKeys, x % C::kChunks);
                uint32_t w[4], bad[4];
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                             : "r"(at) : "memory");
                #pragma unroll
                for (int i = 0; i < 4; ++i) bad[i] = dec::not_finite<F8>(w[i]);
                if (bad[0] | bad[1] | bad[2] | bad[3]) {
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0] & ~bad[0]), "r"(w[1] & ~bad[1]),
                                 "r"(w[2] & ~bad[2]), "r"(w[3] & ~bad[3]) : "memory");
                    sm_taken_out = 1;
                }
            }
            __syncwarp();
        }

        // Scores and outputs are held transposed, keys and channels down the
        // 16 rows of a product and 8 query rows across: a key's or value's
        // fragment, once loaded (and converted), serves all of the warp's rows.
        uint32_t alloc_team = 0;
        #pragma unroll
        for (int x = 0; x < RW; ++x) alloc_team |= sm_alloc[stage][team * RW + x] << (x * kGroups);
        #pragma unroll 1
        for (int g0 = 0; g0 < RW * kGroups; g0 += kStep) {      // the 16-key groups of this team
            const int key0 = cur.j * C::kTile + team * RW * C::kKeys + 16 * g0;
            if (key0 >= cur.len) break;
            // This lane's bytes of its first piece of a group's keys and values;
            // piece c more is c << 4 flipped (C::at), the next groups are constants away.
            const uint32_t from = ring0 + stage * C::kStageBytes + (team * RW + g0 / kGroups) * C::kWarpBytes +
                                  g0 % kGroups * (16 * C::kRowBytes);
            const uint32_t from_k = from + k_lane, from_v = from + v_lane;
            const auto group_at = [](int n) { return n / kGroups * C::kWarpBytes + n % kGroups * (16 * C::kRowBytes); };
            const uint32_t alloc = alloc_team >> g0;
            float s[NT][kStep][4];
            #pragma unroll
            for (int t = 0; t < NT; ++t)
                #pragma unroll
                for (int n = 0; n < kStep; ++n) s[t][n][0] = s[t][n][1] = s[t][n][2] = s[t][n][3] = 0.f;
            #pragma unroll
            for (int c = 0; c < C::kChunks / 2; ++c)
                #pragma unroll
                for (int n = 0; n < kStep; ++n) {
                    uint32_t r[4];
                    dec::ldsm4(r, (from_k ^ (c << 5)) + group_at(n));
                    if constexpr (!F8) {
                        #pragma unroll
                        for (int t = 0; t < NT; ++t) dec::mma16816<false>(s[t][n], r, qf[t][c][0], qf[t][c][1]);
                    } else {
                        #pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            uint32_t a[4];
                            dec::e4m3x4_to_f16x2(r[2 * x], a[0], a[2]);
                            dec::e4m3x4_to_f16x2(r[2 * x + 1], a[1], a[3]);
                            #pragma unroll
                            for (int t = 0; t < NT; ++t)
                                dec::mma16816<true>(s[t][n], a, qf[t][2 * c + x][0], qf[t][2 * c + x][1]);
                        }
                    }
                }
            // masked where a key is not visible
            constexpr uint32_t kAll = (1u << kStep) - 1;
            if (key0 + 16 * kStep > lim_all || (alloc & kAll) != kAll) {
                #pragma unroll
                for (int t = 0; t < NT; ++t)
                    #pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int limit = __shfl_sync(0xffffffffu, lim[t], 8 * t4 + 4 * x);
                        #pragma unroll
                        for (int n = 0; n < kStep; ++n)
                            #pragma unroll
                            for (int y = 0; y < 2; ++y)
                                if (key0 + 16 * n + g + 8 * y >= limit || !((alloc >> n) & 1)) s[t][n][2 * y + x] = -INFINITY;
                    }
            }
            float top[NT][2];
            bool rises = false;
            #pragma unroll
            for (int t = 0; t < NT; ++t)
                #pragma unroll
                for (int x = 0; x < 2; ++x) {
                    top[t][x] = -INFINITY;
                    #pragma unroll
                    for (int n = 0; n < kStep; ++n) top[t][x] = fmaxf(top[t][x], fmaxf(s[t][n][x], s[t][n][2 + x]));
                    top[t][x] *= crow[t][x];      // log2 units from here on (crow > 0)
                    rises = rises || top[t][x] > m[t][x] + kDecodeTau;
                }
            // The reference maximum moves only when a score exceeds it by
            // more than kDecodeTau (weights stay below 2^8), as in the
            // forward: most steps then need neither the rows' maxima nor a
            // rescaled O.
            if (__any_sync(0xffffffffu, rises)) {
                #pragma unroll
                for (int t = 0; t < NT; ++t)
                    #pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float mn = fmaxf(m[t][x], dec::column_max(top[t][x]));
                        const float a = mn == -INFINITY ? 1.f : ptx::ex2(m[t][x] - mn);
                        const bool nothing = __all_sync(0xffffffffu, m[t][x] == -INFINITY);     // a segment's first keys
                        m[t][x] = mn;
                        if (nothing) continue;
                        l[t][x] *= a;
                        #pragma unroll
                        for (int n = 0; n < kMT; ++n) {
                            o[t][n][x] *= a;
                            o[t][n][2 + x] *= a;
                        }
                    }
            }
            // weights, and as operands of the second product: hi (+ lo) of 16 keys
            uint32_t hi[NT][kStep][2], lo[F8 ? 1 : NT][F8 ? 1 : kStep][2];
            #pragma unroll
            for (int t = 0; t < NT; ++t) {
                const auto ref = [&](int x) { return m[t][x] == -INFINITY ? 0.f : kLift - m[t][x]; };
                const uint64_t c2 = ptx::f2_pack(crow[t][0], crow[t][1]), r2 = ptx::f2_pack(ref(0), ref(1));
                uint64_t sum = ptx::f2_pack(l[t][0], l[t][1]);
                #pragma unroll
                for (int n = 0; n < kStep; ++n)
                    #pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float a = s[t][n][2 * x], b = s[t][n][2 * x + 1];
                        ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(a, b), c2, r2), a, b);
                        a = ptx::ex2(a);
                        b = ptx::ex2(b);
                        sum = ptx::f2_add(sum, ptx::f2_pack(a, b));
                        if constexpr (F8) {
                            hi[t][n][x] = dec::transposed(dec::pack_f16x2(a, b));
                        } else {
                            const uint32_t w = ptx::pack_bf16x2(a, b);
                            hi[t][n][x] = dec::transposed(w);
                            lo[t][n][x] = dec::transposed(ptx::pack_bf16x2(a - __uint_as_float(w << 16),
                                                                           b - __uint_as_float(w & 0xFFFF0000u)));
                        }
                    }
                ptx::f2_unpack(sum, l[t][0], l[t][1]);
            }
            // O += P V, 16 keys at a time
            #pragma unroll
            for (int n = 0; n < kStep; ++n)
                #pragma unroll
                for (int c = 0; c < C::kChunks; c += 2) {
                    uint32_t r[4];
                    dec::ldsm4_t(r, (from_v ^ (c << 4)) + group_at(n));
                    if constexpr (!F8) {
                        #pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            dec::mma16816<false>(o[t][c / 2], r, hi[t][n][0], hi[t][n][1]);
                            dec::mma16816<false>(o[t][c / 2], r, lo[t][n][0], lo[t][n][1]);
                        }
                    } else {
                        // a register holds channels (2g, 2g+1) of two keys: the
                        // even ones make rows 0 to 7 of a tile, the odd ones 8 to 15
                        #pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            uint32_t a[4];
                            dec::e4m3x4_to_f16x2(__byte_perm(r[2 * x], 0, 0x3120), a[0], a[1]);
                            dec::e4m3x4_to_f16x2(__byte_perm(r[2 * x + 1], 0, 0x3120), a[2], a[3]);
                            #pragma unroll
                            for (int t = 0; t < NT; ++t) dec::mma16816<true>(o[t][c + x], a, hi[t][n][0], hi[t][n][1]);
                        }
                    }
                }
        }

        const bool item_done = cur.j == cur.nt - 1;
        if (item_done || cur.left == 1) {
            // ---- the segment's end: the teams' results joined through this
            // stage's memory (its keys are used up, its next copy not issued),
            // as many rows at a time as a warp's quarter holds
            constexpr int kPass = C::kWarpBytes / (8 * D * 4) < NT ? C::kWarpBytes / (8 * D * 4) : NT;
            const int row0 = cur.rb * kRows * RW, n_rows = min(p.rows - row0, kRows * RW);
            const bool begun = segment_start == 0;            // the item's first tile was here
            const bool whole = item_done && begun;
            const int slot = 2 * cta + (first_segment ? 0 : 1);
            const int64_t part0 = static_cast<int64_t>(slot) * p.part_rows;
            #pragma unroll
            for (int t = 0; t < NT; ++t)
                #pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float sum = dec::column_sum(l[t][x]);
                    if (g == 0) {
                        sm_m[warp][8 * t + 2 * t4 + x] = m[t][x] - kLift;      // l and O carry the lift
                        sm_l[warp][8 * t + 2 * t4 + x] = sum;
                    }
                }
            __syncthreads();
            if (tid < n_rows) {      // a thread's row: the teams' weights in place of their maxima, LSE, and where O goes
                const int rt = tid / kRows, rr = tid % kRows;
                float mx = -INFINITY, sum = 0.f, a[kTeams];
                #pragma unroll
                for (int k = 0; k < kTeams; ++k) mx = fmaxf(mx, sm_m[k * RW + rt][rr]);
                #pragma unroll
                for (int k = 0; k < kTeams; ++k) {
                    a[k] = mx == -INFINITY ? 0.f : ptx::ex2(sm_m[k * RW + rt][rr] - mx);
                    sum = fmaf(a[k], sm_l[k * RW + rt][rr], sum);
                }
                float scale = dv;
                if (whole) {
                    const int row = row0 + tid, head = p.Nq == 1 ? row : row / p.Nq, n = row - head * p.Nq;
                    const int hq = cur.h * p.group + head;
                    scale = over_sum(dv, sum);
                    sm_out[tid] = cur.b * p.os[0] + hq * p.os[1] + n * p.os[2];
                    p.lse[(static_cast<int64_t>(cur.b) * p.Hq + hq) * p.Nq + n] = log_sum(mx, sum);
                } else {
                    p.part_ml[part0 + tid] = make_float2(mx, sum);
                }
                #pragma unroll
                for (int k = 0; k < kTeams; ++k) sm_m[k * RW + rt][rr] = a[k] * scale;
            }
            // Row r of a warp lies at r D, its channels c at c ^ 8 (r / 2 % 4),
            // so that the lanes of a store meet different banks.
            float *const mine_o = reinterpret_cast<float *>(ring + stage * C::kStageBytes + warp * C::kWarpBytes) + 2 * t4 * D;
            const int flip = (t4 >> 1) << 4, odd = (t4 & 1) << 3;
            #pragma unroll
            for (int t0 = 0; t0 < NT; t0 += kPass) {
                if (t0) __syncthreads();
                #pragma unroll
                for (int t = t0; t < NT && t < t0 + kPass; ++t)
                    #pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        if (row_tile * kRows + 8 * t + 2 * t4 + x >= n_rows) continue;
                        #pragma unroll
                        for (int n = 0; n < kMT; ++n) {
                            float *const to = mine_o + (n & 1 ? -flip : flip) + ((8 * (t - t0) + x) * D + 16 * n);
                            if constexpr (!F8) {
                                (to + (g + odd))[0] = o[t][n][x];
                                (to + (g - odd))[8] = o[t][n][2 + x];
                            } else {
                                *reinterpret_cast<float2 *>(to + ((2 * g) ^ odd)) = make_float2(o[t][n][x], o[t][n][2 + x]);
                            }
                        }
                    }
                __syncthreads();
                constexpr int kPassRows = 8 * kPass;
                for (int x = tid; x < RW * kPassRows * (D / 4); x += kDecodeThreads) {
                    const int y = x / (D / 4), c = x % (D / 4), rt = y / kPassRows, rr = y % kPassRows + 8 * t0;
                    const int r = rt * kRows + rr;
                    if (rr >= kRows || r >= n_rows) continue;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    #pragma unroll
                    for (int k = 0; k < kTeams; ++k) {
                        const int w = k * RW + rt;
                        const float a = sm_m[w][rr];
                        const float4 v = *reinterpret_cast<const float4 *>(
                            ring + stage * C::kStageBytes + w * C::kWarpBytes +
                            ((rr - 8 * t0) * D + ((4 * c) ^ (((rr >> 1) & 3) << 3))) * 4);
                        acc.x = fmaf(a, v.x, acc.x);
                        acc.y = fmaf(a, v.y, acc.y);
                        acc.z = fmaf(a, v.z, acc.z);
                        acc.w = fmaf(a, v.w, acc.w);
                    }
                    if (whole)
                        *reinterpret_cast<uint2 *>(p.o + sm_out[r] + c * 4) =
                            make_uint2(ptx::pack_bf16x2(acc.x, acc.y), ptx::pack_bf16x2(acc.z, acc.w));
                    else
                        *reinterpret_cast<float4 *>(p.part_o + (part0 + r) * D + c * 4) = acc;
                }
            }
            if (begun && !item_done) {
                const int64_t end = u1 - cur.left + (cur.nt - cur.j);      // its last unit's owner ends it
                my_job_item = (cur.b * p.Hkv + cur.h) * p.row_blocks + cur.rb;
                my_job_slot = slot;
                my_job_last = static_cast<int>(quotient(end * active + units - 1, units) - 1);
            }
            first_segment = false;
            segment_start = -1;
            __syncthreads();
            if (PARTLY && sm_taken_out) add_not_finite<D, F8>(p, cur.b, cur.h, cur.len, whole ? -1 : part0, row0, n_rows);
        }
        advance<C::kTile>(p, cur);
    }
    dec::cp_wait<0>();
    if (tid == 0) p.jobs[cta] = DecodeJob{my_job_item, my_job_slot, my_job_last, 0};
}

// Joins the partial results of an item that several CTAs shared: with
// M = max_c m_c and w_c = 2^(m_c - M), O = sum_c w_c O_c / sum_c w_c l_c and
// LSE = ln 2 (M + log2 sum_c w_c l_c).
//
// It is all latency (57 partials of 512 bytes for one of 8 heads of a single
// long sequence), so outputs are loaded before their weights are known.  One
// CTA per (CTA that began an item, query row), each warp taking every eighth
// partial, 8 at a time; where an item has at most 8 partials, as in a batch
// whose sequences cross a CTA's border once, a warp does a row alone and every
// eighth CTA has work (64 ragged sequences: 163.2 -> 161.8 us with that).
constexpr int kMergeThreads = 256;
constexpr int kMergeWarps = kMergeThreads / 32;
constexpr int kMergeBatch = 8;

template <int D>
__global__ void __launch_bounds__(kMergeThreads, 4) fa_decode_merge_kernel(const __grid_constant__ DecodeParams p) {
    constexpr int PER = D / 32;
    using Vec = typename std::conditional<PER == 4, float4, float2>::type;
    __shared__ float sm_w[kDecodeMaxCtas], sm_red[2][kMergeWarps], sm_o[kMergeWarps][D];
    ptx::griddep_wait();
    const int cta = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const DecodeJob job = p.jobs[cta];
    if (job.item < 0) return;
    const int parts = job.last_cta - cta + 1;
    const bool alone = parts <= kMergeBatch;                   // a warp for each row
    if (alone && blockIdx.y % kMergeWarps != 0) return;
    const int r = alone ? blockIdx.y + warp : blockIdx.y;      // row of the partial results
    const int rb = job.item % p.row_blocks, bh = job.item / p.row_blocks, h = bh % p.Hkv, b = bh / p.Hkv;
    const int row = rb * p.part_rows + r;
    if (r >= p.part_rows || row >= p.rows) return;             // the CTA, or a warp that works alone
    const int head = p.Nq == 1 ? row : row / p.Nq, n = row - head * p.Nq, hq = h * p.group + head;
    __nv_bfloat16 *const out = p.o + b * p.os[0] + hq * p.os[1] + n * p.os[2];
    float *const lse = p.lse + (static_cast<int64_t>(b) * p.Hq + hq) * p.Nq + n;
    const auto place = [&](int x) { return static_cast<int64_t>(x == 0 ? job.slot : 2 * (cta + x)) * p.part_rows + r; };
    const int step = alone ? 1 : kMergeWarps;
    Vec v[kMergeBatch];
    const auto fetch = [&](int first) {
        #pragma unroll
        for (int y = 0; y < kMergeBatch; ++y) {
            const int x = first + y * step;
            if (x < parts) v[y] = reinterpret_cast<const Vec *>(p.part_o + place(x) * D)[lane];
        }
    };
    const auto add = [&](float (&o)[PER], float w, int y) {
        const float *e = reinterpret_cast<const float *>(&v[y]);
        #pragma unroll
        for (int c = 0; c < PER; ++c) o[c] = fmaf(w, e[c], o[c]);
    };
    float o[PER] = {};

    if (alone) {
        fetch(0);
        const float2 ml = lane < parts ? p.part_ml[place(lane)] : make_float2(-INFINITY, 0.f);
        float mx = ml.x;
        #pragma unroll
        for (int x = kMergeBatch / 2; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        mx = __shfl_sync(0xffffffffu, mx, 0);
        const float w = ml.x == -INFINITY ? 0.f : ptx::ex2(ml.x - mx);
        float sum = w * ml.y;
        #pragma unroll
        for (int x = kMergeBatch / 2; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        sum = __shfl_sync(0xffffffffu, sum, 0);
        #pragma unroll
        for (int y = 0; y < kMergeBatch; ++y) {
            const float wy = __shfl_sync(0xffffffffu, w, y);
            if (y < parts) add(o, wy, y);
        }
        const float inv = over_sum(1.f, sum);
        uint32_t packed[PER / 2];
        #pragma unroll
        for (int c = 0; c < PER / 2; ++c) packed[c] = ptx::pack_bf16x2(o[2 * c] * inv, o[2 * c + 1] * inv);
        if constexpr (PER == 4) reinterpret_cast<uint2 *>(out)[lane] = make_uint2(packed[0], packed[1]);
        else reinterpret_cast<uint32_t *>(out)[lane] = packed[0];
        if (lane == 0) *lse = log_sum(mx, sum);
        return;
    }

    fetch(warp);
    // weights: at most kDecodeMaxCtas partials, a few to a thread
    constexpr int kMine = (kDecodeMaxCtas + kMergeThreads - 1) / kMergeThreads;
    float2 ml[kMine];
    float mx = -INFINITY;
    #pragma unroll
    for (int y = 0; y < kMine; ++y) {
        const int x = tid + y * kMergeThreads;
        ml[y] = x < parts ? p.part_ml[place(x)] : make_float2(-INFINITY, 0.f);
        mx = fmaxf(mx, ml[y].x);
    }
    #pragma unroll
    for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
    if (lane == 0) sm_red[0][warp] = mx;
    __syncthreads();
    #pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) mx = fmaxf(mx, sm_red[0][w]);
    float sum = 0.f;
    #pragma unroll
    for (int y = 0; y < kMine; ++y) {
        const int x = tid + y * kMergeThreads;
        const float w = ml[y].x == -INFINITY ? 0.f : ptx::ex2(ml[y].x - mx);
        if (x < parts) sm_w[x] = w;
        sum = fmaf(w, ml[y].y, sum);
    }
    #pragma unroll
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    if (lane == 0) sm_red[1][warp] = sum;
    __syncthreads();
    sum = 0.f;
    #pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) sum += sm_red[1][w];

    for (int first = warp;;) {
        #pragma unroll
        for (int y = 0; y < kMergeBatch; ++y) {
            const int x = first + y * kMergeWarps;
            if (x < parts) add(o, sm_w[x], y);
        }
        first += kMergeBatch * kMergeWarps;
        if (first >= parts) break;
        fetch(first);
    }
    #pragma unroll
    for (int c = 0; c < PER; ++c) sm_o[warp][lane * PER + c] = o[c];
    __syncthreads();
    if (tid < D / 2) {
        const float inv = over_sum(1.f, sum);
        float y0 = 0.f, y1 = 0.f;
        #pragma unroll
        for (int w = 0; w < kMergeWarps; ++w) {
            const float2 e = reinterpret_cast<const float2 *>(sm_o[w])[tid];
            y0 += e.x;
            y1 += e.y;
        }
        reinterpret_cast<uint32_t *>(out)[tid] = ptx::pack_bf16x2(y0 * inv, y1 * inv);
    }
    if (tid == 0) *lse = log_sum(mx, sum);
}

}  // namespace fa
