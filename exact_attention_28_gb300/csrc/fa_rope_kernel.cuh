// Rotary positions with several axes on q and k, and the write of rotated
// keys and of values into the paged cache.
//
// Pair c of a head, (x1, x2), turns by phi = pos[axis(c)] * f_c:
//   y1 = x1 cos phi - x2 sin phi,   y2 = x2 cos phi + x1 sin phi,
// and the gradient turns by -phi.
//
// The phase.  cos and sin need phi only modulo a turn.  f_c / (2 pi) is held
// as a 64-bit fraction of a turn, F_c = f_c / (2 pi) * 2^64 mod 2^64, rounded
// once (rotary_phase.h); then pos * F_c mod 2^64, one wrapping integer product,
// is the phase of any int32 position to within |pos| 2^-65 turns, with no range
// reduction in floating point (an fp32 angle is off by 0.06 rad at position
// 10^6).  Its upper 32 bits go on, cut off: up to 2^-32 turns (1.5e-9 rad) more.
// The nearest quarter turn is their top bits, and what is left, at most an
// eighth of a turn, goes through the Taylor polynomials of sin and cos.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "ptx_sm103.cuh"

namespace fa {

// The work.  A CTA takes a tile of tokens (32 at d = 128, 64 at d = 64) and a
// group of heads, up to 8; each thread one chunk of 8 pairs of one token, whose
// angles it forms once for all heads of the group.
//
// What bounds it: memory, each element read and written once.  A thread's
// pieces come through its own places in a ring of 16-byte asynchronous copies,
// so that the loads of the next heads are in flight while one is turned.  The
// order matters as much: all tiles of a group of heads come before the next
// group, so that CTAs that run together work on neighbouring rows of the same
// heads.  2 x 8192 tokens, 32 + 8 heads, d = 128, from token-major to
// head-major: 51.4 us with groups of 8 (6.5 TB/s, 97% of the measured copy rate), 58 us
// with persistent CTAs on equal runs of (tile, head), whatever the ring's depth.
// 16,411 tokens into a bf16 cache: 61.4 us (98%), into an E4M3 one 57.1 us (97%).
constexpr int kRopeThreads = 256;
constexpr int kRopeHeads = 8;                                // heads of a CTA, at most
constexpr int kRopeStages = 4;
constexpr int kRopeCtasPerSm = 3;
constexpr int kRopeStageBytes = kRopeThreads * 32;
constexpr int kRopeSmemBytes = kRopeStages * kRopeStageBytes;
constexpr int kMaxAxes = 4;
__host__ __device__ constexpr int rope_tokens(int d) { return kRopeThreads / (d / 16); }   // of a tile

// Frequencies of the rot/2 pairs (at most 64) as fractions of a turn per
// position, and the axis that each pair follows.
struct alignas(16) RotaryTable {
    uint64_t phase[64];
    uint8_t axis[64];
};

// A thread's chunk is 16 elements of a head in two 16-byte pieces, 8 pairs.
// Piece i of chunk c lies at 8 c in half i of the rotated elements (or, behind
// them, of the others), so that the chunks of a head fill whole sectors: of
// half-split pairs the pieces hold the first and second elements of pairs
// 8 c .. 8 c + 7, of interleaved ones pairs 4 c .. and rot/4 + 4 c .. .
__device__ __forceinline__ void chunk_offsets(int chunk, int rot, int d, int &a, int &b) {
    const int other = chunk - rot / 16;
    a = other < 0 ? chunk * 8 : rot + other * 8;
    b = a + (other < 0 ? rot : d - rot) / 2;
}

// cos, sin and -sin of a thread's 8 pairs as four packed twos.
struct Angles {
    uint64_t cs[4], sn[4], neg[4];
};

// sin and cos of p / 2^32 turns.  With q the nearest quarter and |t| <= pi / 4
// the angle from it, the Taylor terms that are left out are below t^11 / 11! =
// 1.8e-9 of the sine and t^10 / 10! = 2.5e-8; the rest is fp32 rounding.
__device__ __forceinline__ void sincos_turns(uint32_t p, float &sn, float &cs) {
    const uint32_t q = (p + 0x20000000u) >> 30;
    const float t = static_cast<float>(static_cast<int32_t>(p - (q << 30))) * 1.4629180792671596e-9f;   // 2 pi / 2^32
    const float z = t * t;
    const float s = fmaf(t * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), t);
    const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.f / 40320, -1.f / 720), 1.f / 24), -0.5f), 1.f);
    // q = 0 .. 3: (s, c), (c, -s), (-s, -c), (-c, s)
    sn = __uint_as_float(__float_as_uint(q & 1 ? c : s) ^ ((q & 2) << 30));
    cs = __uint_as_float(__float_as_uint(q & 1 ? s : c) ^ (((q + 1) & 2) << 30));
}

// The angles of a chunk's 8 pairs, at the positions of one token: those of
// axis a at positions[a * axis_stride].
template <bool INTERLEAVED>
__device__ __forceinline__ void chunk_angles(const RotaryTable &tab, int chunk, int rot, const int *positions,
                                             int64_t axis_stride, int axes, bool inverse, Angles &out) {
    int pos[kMaxAxes];
    #pragma unroll
    for (int a = 0; a < kMaxAxes; ++a) pos[a] = a < axes ? positions[a * axis_stride] : 0;
    // The table is a kernel parameter.  Constant-bank reads at different
    // places of a warp are served one after another, so these go through L1.
    uint64_t phase[8];
    uint32_t ax[2];
    const int first[2] = {INTERLEAVED ? chunk * 4 : chunk * 8, INTERLEAVED ? rot / 4 + chunk * 4 : chunk * 8 + 4};
    #pragma unroll
    for (int h = 0; h < 2; ++h) {
        #pragma unroll
        for (int i = 0; i < 4; i += 2)
            asm("ld.v2.b64 {%0, %1}, [%2];" : "=l"(phase[4 * h + i]), "=l"(phase[4 * h + i + 1])
                : "l"(&tab.phase[first[h] + i]));
        asm("ld.b32 %0, [%1];" : "=r"(ax[h]) : "l"(&tab.axis[first[h]]));
    }
    float cs[8], sn[8];
    #pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t a = (ax[i >> 2] >> (8 * (i & 3))) & 0xffu;
        int p = pos[0];
        #pragma unroll
        for (int k = 1; k < kMaxAxes; ++k) p = a == k ? pos[k] : p;
        const uint64_t turns = static_cast<uint64_t>(static_cast<int64_t>(p)) * phase[i];
        sincos_turns(static_cast<uint32_t>(turns >> 32), sn[i], cs[i]);
        if (inverse) sn[i] = -sn[i];
    }
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        out.cs[i] = ptx::f2_pack(cs[2 * i], cs[2 * i + 1]);
        out.sn[i] = ptx::f2_pack(sn[2 * i], sn[2 * i + 1]);
        out.neg[i] = ptx::f2_pack(-sn[2 * i], -sn[2 * i + 1]);
    }
}

__device__ __forceinline__ void rope_cp16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void rope_cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void rope_cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8]) {
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(r[i] << 16);
        x[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint4 pack8_bf16(const float (&x)[8]) {
    return make_uint4(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]), ptx::pack_bf16x2(x[4], x[5]),
                      ptx::pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8], float inv) {
    return make_uint2(ptx::pack_e4m3x4(__fmul_rn(x[0], inv), __fmul_rn(x[1], inv), __fmul_rn(x[2], inv),
                                       __fmul_rn(x[3], inv)),
                      ptx::pack_e4m3x4(__fmul_rn(x[4], inv), __fmul_rn(x[5], inv), __fmul_rn(x[6], inv),
                                       __fmul_rn(x[7], inv)));
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// The 8 pairs of a chunk, turned: x1 and x2 are read from the two pieces and
// y1, y2 put back into their places; two pairs at a time.
template <bool INTERLEAVED>
__device__ __forceinline__ void turn_chunk(float (&xa)[8], float (&xb)[8], const Angles &a) {
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        float *p = i < 2 ? xa + 4 * i : xb + 4 * (i - 2);     // interleaved: four elements, two pairs
        float &x1 = INTERLEAVED ? p[0] : xa[2 * i], &x1n = INTERLEAVED ? p[2] : xa[2 * i + 1];
        float &x2 = INTERLEAVED ? p[1] : xb[2 * i], &x2n = INTERLEAVED ? p[3] : xb[2 * i + 1];
        const uint64_t u = ptx::f2_pack(x1, x1n), v = ptx::f2_pack(x2, x2n);
        ptx::f2_unpack(fma2(v, a.neg[i], mul2(u, a.cs[i])), x1, x1n);
        ptx::f2_unpack(fma2(u, a.sn[i], mul2(v, a.cs[i])), x2, x2n);
    }
}
template <bool INTERLEAVED>
__device__ __forceinline__ void turn_bf16(uint4 &wa, uint4 &wb, const Angles &a) {
    float xa[8], xb[8];
    unpack8(wa, xa);
    unpack8(wb, xb);
    turn_chunk<INTERLEAVED>(xa, xb, a);
    wa = pack8_bf16(xa);
    wb = pack8_bf16(xb);
}

// Heads of one token that follow one another in memory: `count` rows, `step`
// elements (source) or bytes (target) apart.
struct SourceRun {
    const __nv_bfloat16 *x;
    int64_t step;
    int count;
};
struct TargetRun {
    char *y;                  // nullptr: nothing is written
    int64_t step;
    int count;
    bool turns, codes;        // rotated; E4M3 codes over descale[0], descale[1], ..
    const float *descale;
};

// fa_rope: bf16 [B, H, N, D] to the same, the heads of q and k one list.
struct RopeParams {
    const __nv_bfloat16 *q, *k;
    __nv_bfloat16 *qo, *ko;
    int64_t qs[3], ks[3], qos[3], kos[3];   // batch, head, token strides in elements
    const int *positions;
    int64_t pos_axis, pos_batch;
    int Hq, Hk, B, N, rot, axes;
    int tokens, heads, per_cta;             // B N, Hq + Hk
    bool inverse;
    RotaryTable tab;

    struct Token {
        int b, n;
    };
    __device__ __forceinline__ Token token(int i) const {
        const int b = B == 1 ? 0 : i / N;
        return {b, i - b * N};
    }
    __device__ __forceinline__ const int *position(const Token &t) const { return positions + t.b * pos_batch + t.n; }
    __device__ __forceinline__ SourceRun source(const Token &t, int h) const {
        if (h < Hq) return {q + t.b * qs[0] + h * qs[1] + t.n * qs[2], qs[1], Hq - h};
        return {k + t.b * ks[0] + (h - Hq) * ks[1] + t.n * ks[2], ks[1], heads - h};
    }
    template <int D>
    __device__ __forceinline__ TargetRun target(const Token &t, int h) const {
        const bool is_q = h < Hq;
        __nv_bfloat16 *y = is_q ? qo + t.b * qos[0] + h * qos[1] + t.n * qos[2]
                                : ko + t.b * kos[0] + (h - Hq) * kos[1] + t.n * kos[2];
        return {reinterpret_cast<char *>(y), 2 * (is_q ? qos[1] : kos[1]), (is_q ? Hq : heads) - h, true, false, nullptr};
    }
};

// fa_paged_append: bf16 [T, H, D] to q's output and the cache, the heads of
// q, k and v one list.
template <bool F8>
struct AppendParams {
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16 *qo;
    int64_t qs[2], ks[2], vs[2], qos[2];    // token, head strides in elements
    void *k_cache, *v_cache;
    const float *k_descale, *v_descale;     // of an E4M3 cache
    const int *slots, *positions;
    int64_t pos_axis;
    int64_t cache_rows;                     // num_blocks * block_size
    int block_shift;
    int Hq, Hkv, rot, axes;
    int tokens, heads, per_cta;             // T, Hq + 2 Hkv
    static constexpr bool inverse = false;
    RotaryTable tab;

    struct Token {
        int64_t t, slot;
    };
    __device__ __forceinline__ Token token(int i) const { return {i, slots[i]}; }
    __device__ __forceinline__ const int *position(const Token &t) const { return positions + t.t; }
    __device__ __forceinline__ SourceRun source(const Token &t, int h) const {
        const int kh = h - Hq, vh = kh - Hkv;
        if (kh < 0) return {q + t.t * qs[0] + h * qs[1], qs[1], -kh};
        if (vh < 0) return {k + t.t * ks[0] + kh * ks[1], ks[1], -vh};
        return {v + t.t * vs[0] + vh * vs[1], vs[1], heads - h};
    }
    template <int D>
    __device__ __forceinline__ TargetRun target(const Token &t, int h) const {
        const bool kept = t.slot >= 0 && t.slot < cache_rows;
        const int kh = h - Hq, vh = kh - Hkv;
        if (kh < 0) {
            __nv_bfloat16 *y = qo + t.t * qos[0] + h * qos[1];
            return {kept ? reinterpret_cast<char *>(y) : nullptr, 2 * qos[1], -kh, true, false, nullptr};
        }
        const bool is_k = vh < 0;
        const int64_t step = static_cast<int64_t>(D * (F8 ? 1 : 2)) << block_shift;     // from head to head of a block
        char *y = static_cast<char *>(is_k ? k_cache : v_cache) +
                  ((t.slot >> block_shift) * Hkv + (is_k ? kh : vh)) * step +
                  (t.slot & ((1 << block_shift) - 1)) * (D * (F8 ? 1 : 2));
        return {kept ? y : nullptr, step, is_k ? -vh : heads - h, is_k, F8,
                F8 ? (is_k ? k_descale + kh : v_descale + vh) : nullptr};
    }
};

// 16 codes of a chunk, pieces at bytes ea and eb of the row at y (nullptr:
// none).  The whole warp calls it.  A piece is 8 bytes; where the pieces of a
// pair of lanes fall on 16-byte boundaries they trade, so that the even lane
// stores both first pieces and the odd one both second ones.
__device__ __forceinline__ void store_codes(char *y, const float (&xa)[8], const float (&xb)[8], float inv, int ea, int eb,
                                            bool trades, bool odd) {
    const uint2 ca = pack8_e4m3(xa, inv), cb = pack8_e4m3(xb, inv), give = odd ? ca : cb;
    uint2 got;
    got.x = __shfl_xor_sync(0xffffffffu, give.x, 1);
    got.y = __shfl_xor_sync(0xffffffffu, give.y, 1);
    if (!y) return;
    if (trades) {
        if (odd) *reinterpret_cast<uint4 *>(y + eb - 8) = make_uint4(got.x, got.y, cb.x, cb.y);
        else *reinterpret_cast<uint4 *>(y + ea) = make_uint4(ca.x, ca.y, got.x, got.y);
    } else {
        *reinterpret_cast<uint2 *>(y + ea) = ca;
        *reinterpret_cast<uint2 *>(y + eb) = cb;
    }
}

template <int D, bool INTERLEAVED, class P>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtasPerSm) fa_rope_kernel(const __grid_constant__ P p) {
    extern __shared__ __align__(16) uint8_t rope_ring[];
    constexpr int kTokens = rope_tokens(D), kChunks = D / 16;
    const int token = threadIdx.x / kChunks, chunk = threadIdx.x % kChunks;
    const int tiles = (p.tokens + kTokens - 1) / kTokens, group = blockIdx.x / tiles, tile = blockIdx.x - group * tiles;
    const int head0 = group * p.per_cta, n_heads = min(p.per_cta, p.heads - head0);
    ptx::griddep_wait();

    int ea, eb;
    chunk_offsets(chunk, p.rot, D, ea, eb);
    const int row = tile * kTokens + token;
    const bool valid = row < p.tokens;
    const typename P::Token tok = p.token(valid ? row : p.tokens - 1);
    const uint32_t slot0 = ptx::smem_addr(rope_ring) + threadIdx.x * 16;
    SourceRun source = p.source(tok, head0);
    int ahead = 0;
    const auto issue = [&](uint32_t slot) {
        if (ahead < n_heads) {
            rope_cp16(slot, source.x + ea);
            rope_cp16(slot + kRopeStageBytes / 2, source.x + eb);
            ++ahead;
            source.x += source.step;
            if (--source.count == 0 && ahead < n_heads) source = p.source(tok, head0 + ahead);
        }
        rope_cp_commit();
    };
    #pragma unroll
    for (int s = 0; s < kRopeStages; ++s) issue(slot0 + s * kRopeStageBytes);

    const bool turned = chunk < p.rot / 16;
    const bool trades = p.rot % 32 == 0;       // both halves begin on 16-byte boundaries, chunks pair up
    Angles a;
    TargetRun target = p.template target<D>(tok, head0);
    // of a group that begins behind q and k, none are turned
    if (turned && target.turns)
        chunk_angles<INTERLEAVED>(p.tab, chunk, p.rot, p.position(tok), p.pos_axis, p.axes, p.inverse, a);
    uint32_t at = 0;                           // the stage in use, in bytes
    for (int h = 0; h < n_heads; ++h) {
        if (target.count == 0) target = p.template target<D>(tok, head0 + h);
        if (!valid) target.y = nullptr;
        rope_cp_wait<kRopeStages - 1>();       // a thread reads its own copies: no barrier
        const uint4 *from = reinterpret_cast<const uint4 *>(rope_ring + at) + threadIdx.x;
        uint4 wa = from[0], wb = from[kRopeThreads];
        if (!target.codes) {
            if (turned && target.turns) turn_bf16<INTERLEAVED>(wa, wb, a);
            if (target.y) {
                *reinterpret_cast<uint4 *>(target.y + 2 * ea) = wa;
                *reinterpret_cast<uint4 *>(target.y + 2 * eb) = wb;
                target.y += target.step;
            }
        } else {
            float xa[8], xb[8];
            unpack8(wa, xa);
            unpack8(wb, xb);
            if (turned && target.turns) turn_chunk<INTERLEAVED>(xa, xb, a);
            store_codes(target.y, xa, xb, __frcp_rn(*target.descale), ea, eb, trades, chunk & 1);
            ++target.descale;
            if (target.y) target.y += target.step;
        }
        --target.count;
        issue(slot0 + at);
        at = at + kRopeStageBytes == kRopeSmemBytes ? 0 : at + kRopeStageBytes;
    }
    rope_cp_wait<0>();
}

}  // namespace fa
