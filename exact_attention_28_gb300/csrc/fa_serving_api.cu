// Host side of the serving entry points (block tables, rotary positions, the
// write into the paged cache, attention of the newest tokens over it):
// argument checks and launches.  Implements that part of include/fa.h.
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <type_traits>

#include <cuda_runtime.h>

#include "../../include/fa.h"
#include "fa_block_tables_kernel.cuh"
#include "fa_decode_select.cuh"
#include "fa_rope_kernel.cuh"
#include "rotary_phase.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool block_size_ok(int bs) { return bs == 16 || bs == 32 || bs == 64 || bs == 128 || bs == 256; }
int log2_of(int power) { return 31 - __builtin_clz(static_cast<unsigned>(power)); }

fa_status launched() { return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// Launches with programmatic stream serialisation: the kernel may be set up
// while the stream's previous one drains, and waits for it (griddepcontrol.wait)
// before its first global access.
cudaError_t launch_dependent(cudaStream_t stream, dim3 grid, int threads, int smem, const void *kernel, void *param) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *args[1] = {param};
    return cudaLaunchKernelExC(&cfg, kernel, args);
}

template <class P>
int rope_index(int d, bool interleaved) {
    const int kind = std::is_same<P, fa::RopeParams>::value ? 0 : std::is_same<P, fa::AppendParams<false>>::value ? 1 : 2;
    return 48 + 4 * kind + (d == 128 ? 2 : 0) + (interleaved ? 1 : 0);
}
template <class P>
const void *rope_kernel(int d, bool interleaved) {
    return d == 128 ? (interleaved ? reinterpret_cast<const void *>(fa::fa_rope_kernel<128, true, P>)
                                   : reinterpret_cast<const void *>(fa::fa_rope_kernel<128, false, P>))
                    : (interleaved ? reinterpret_cast<const void *>(fa::fa_rope_kernel<64, true, P>)
                                   : reinterpret_cast<const void *>(fa::fa_rope_kernel<64, false, P>));
}

using fa::DecodeKernel;
using fa::DecodeLayout;
using fa::decode_layout;
using fa::decode_rows;

// SM count of a device, and which kernels have their shared-memory limits set
// there: at a kernel's first call, for it loads the file that the kernel is in
// (the 24 attention kernels of one file take 9 ms).
struct ServingDevice {
    int sms = 0;
    uint64_t ready = 0;
};
std::mutex g_serving_mu;
ServingDevice g_serving[64];

// The current device's SM count, with `kernel` ready to run there.  `index`
// numbers the kernels: 0 to 47 attention, 48 to 59 rotation.
fa_status serving_device(int &sms, int index, const void *kernel, int smem) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FA_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_serving_mu);
    ServingDevice &info = g_serving[dev];
    if (info.sms == 0 &&
        cudaDeviceGetAttribute(&info.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        info.sms = 0;
        return FA_ERR_CUDA;
    }
    if (!(info.ready >> index & 1)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
            cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100) != cudaSuccess)
            return FA_ERR_CUDA;
        info.ready |= uint64_t{1} << index;
    }
    sms = info.sms;
    return FA_OK;
}

// Memory that a call reads or writes, none at nullptr or without bytes.  Of a
// strided tensor only the first row: its others may lie between another's.
struct Span {
    const void *at;
    int64_t bytes;
    bool output;
};
// Whether no output lies on another span.
template <int N>
bool apart(const Span (&spans)[N]) {
    for (const Span &x : spans)
        for (const Span &y : spans) {
            const char *a = static_cast<const char *>(x.at), *b = static_cast<const char *>(y.at);
            if (&x != &y && x.output && a && b && x.bytes > 0 && y.bytes > 0 && a < b + y.bytes && b < a + x.bytes)
                return false;
        }
    return true;
}

// Strides of a tensor [extent_0, .., extent_{n-1}, d] (contiguous when given
// is NULL), checked: >= 0, rows on 16-byte boundaries, at most 2^40 elements;
// an output's rows must not lie on one another: each stride reaches past all
// that the smaller ones span.
fa_status take_strides(int64_t *out, const int64_t *given, const int *extent, int n, int d, bool output) {
    int64_t s = d;
    bool absent = false;   // no heads: the tensor is not there
    for (int i = 0; i < n; ++i) absent = absent || extent[i] == 0;
    for (int i = n - 1; i >= 0; --i) {
        out[i] = given ? given[i] : s;
        s *= extent[i];
    }
    for (int i = 0; i < n && !absent; ++i) {
        if (out[i] < 0 || out[i] > (int64_t{1} << 40)) return FA_ERR_INVALID_ARG;
        if (output && extent[i] > 1 && out[i] < d) return FA_ERR_INVALID_ARG;
        if (extent[i] > 1 && out[i] % 8 != 0) return FA_ERR_MISALIGNED;
    }
    if (output && !absent) {
        __int128 span = d;
        bool taken[3] = {};
        for (int k = 0; k < n; ++k) {
            int least = -1;
            for (int i = 0; i < n; ++i)
                if (!taken[i] && extent[i] > 1 && (least < 0 || out[i] < out[least])) least = i;
            if (least < 0) break;
            if (out[least] < span) return FA_ERR_INVALID_ARG;
            span += static_cast<__int128>(out[least]) * (extent[least] - 1);
            taken[least] = true;
        }
    }
    return FA_OK;
}

// An output that begins where its input does is the input itself: the same
// strides.  `in` then counts as no other memory.
bool in_place_ok(const void *&in, const int64_t *in_strides, const void *out, const int64_t *out_strides,
                 const int *extent, int n) {
    if (!in || in != out) return true;
    for (int i = 0; i < n; ++i)
        if (extent[i] > 1 && in_strides[i] != out_strides[i]) return false;
    in = nullptr;
    return true;
}

// Bytes of a bf16 tensor [extent_0, .., extent_{n-1}, d], of its first row unless it is contiguous.
int64_t span_bytes(const int64_t *strides, const int *extent, int n, int d) {
    int64_t s = d;
    for (int i = n - 1; i >= 0; --i) {
        if (extent[i] > 1 && strides[i] != s) return 2 * d;
        s *= extent[i];
    }
    return 2 * s;
}

// The rotation kernel for p: a CTA for each tile of tokens and group of heads,
// in as small groups as still run at once, up to 8 heads.  More CTAs than fit
// the GPU leave a second round half empty, fewer leave SMs idle: 3 x 1021
// tokens, 16 + 16 heads, d = 64: 192 CTAs (groups of 8) 7.9 us, 384 (4) 6.0,
// 768 (2) 7.9.
template <class P>
fa_status launch_rope(P &p, int d, bool interleaved, cudaStream_t stream) {
    const void *const kernel = rope_kernel<P>(d, interleaved);
    int sms;
    const fa_status st = serving_device(sms, rope_index<P>(d, interleaved), kernel, fa::kRopeSmemBytes);
    if (st != FA_OK) return st;
    const int64_t tiles = (static_cast<int64_t>(p.tokens) + fa::rope_tokens(d) - 1) / fa::rope_tokens(d);
    const auto groups = [&](int n) { return (static_cast<int64_t>(p.heads) + n - 1) / n; };
    int n = 1;
    while (n < fa::kRopeHeads && tiles * groups(n) > static_cast<int64_t>(fa::kRopeCtasPerSm) * sms) ++n;
    p.per_cta = static_cast<int>(groups(static_cast<int>(groups(n))));      // the same number of groups, evenly
    const int64_t ctas = tiles * groups(p.per_cta);
    if (ctas > 0x7fffffff) return FA_ERR_INVALID_ARG;
    if (launch_dependent(stream, dim3(static_cast<unsigned>(ctas)), fa::kRopeThreads, fa::kRopeSmemBytes,
                         kernel, &p) != cudaSuccess)
        return FA_ERR_CUDA;
    return launched();
}

// Checks the frequencies and axes and lays out the table.  The last table of
// each thread is kept with the numbers that it was made from, so that a
// program that turns by the same ones again pays a comparison of them (64
// phases take about 1 us).
fa_status take_rotary(fa::RotaryTable &tab, int d, int rot, int axes, const double *inv_freq, const int *pair_axis) {
    if (rot < 16 || rot > d || rot % 16 != 0) return FA_ERR_UNSUPPORTED;
    if (axes < 1 || axes > fa::kMaxAxes || !inv_freq) return FA_ERR_INVALID_ARG;
    struct Made {
        int pairs = 0, axes;
        double freq[64];
        int axis[64];
        fa::RotaryTable tab;
    };
    thread_local Made made;
    const int pairs = rot / 2;
    int axis[64] = {};
    if (pair_axis) std::memcpy(axis, pair_axis, pairs * sizeof(int));
    if (made.pairs != pairs || made.axes != axes || std::memcmp(made.freq, inv_freq, pairs * sizeof(double)) != 0 ||
        std::memcmp(made.axis, axis, pairs * sizeof(int)) != 0) {
        made.pairs = 0;
        std::memset(&made.tab, 0, sizeof made.tab);
        for (int c = 0; c < pairs; ++c) {
            if (!std::isfinite(inv_freq[c]) || axis[c] < 0 || axis[c] >= axes) return FA_ERR_INVALID_ARG;
            made.tab.phase[c] = fa::rotary_phase(inv_freq[c]);
            made.tab.axis[c] = static_cast<uint8_t>(axis[c]);
        }
        std::memcpy(made.freq, inv_freq, pairs * sizeof(double));
        std::memcpy(made.axis, axis, pairs * sizeof(int));
        made.axes = axes;
        made.pairs = pairs;
    }
    tab = made.tab;
    return FA_OK;
}

}  // namespace

extern "C" fa_status fa_block_tables(int *block_table, const int *ctx_lens, const int *new_lens,
                                     const int *free_blocks, int *seq_lens, int *query_start, int *slots,
                                     int *positions, int *counts, int B, int max_blocks, int block_size, int num_free,
                                     int num_tokens, fa_stream_t stream) {
    if (!block_table || !ctx_lens || !new_lens || !seq_lens || !query_start || !counts) return FA_ERR_INVALID_ARG;
    if (B < 1 || B > fa::kMaxRequests || max_blocks < 1 || num_free < 0 || num_tokens < 0 ||
        num_tokens > (1 << 30))
        return FA_ERR_INVALID_ARG;
    if ((num_free > 0 && !free_blocks) || (num_tokens > 0 && (!slots || !positions))) return FA_ERR_INVALID_ARG;
    if (!block_size_ok(block_size)) return FA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(max_blocks) * block_size > (int64_t{1} << 30)) return FA_ERR_INVALID_ARG;
    for (const void *x : {static_cast<const void *>(block_table), static_cast<const void *>(ctx_lens),
                          static_cast<const void *>(new_lens), static_cast<const void *>(free_blocks),
                          static_cast<const void *>(seq_lens), static_cast<const void *>(query_start),
                          static_cast<const void *>(slots), static_cast<const void *>(positions),
                          static_cast<const void *>(counts)})
        if (!aligned(x, 4)) return FA_ERR_MISALIGNED;
    // CTAs read the lengths and the free list while others write: no output may lie on another array
    if (!apart<9>({{ctx_lens, int64_t{4} * B, false}, {new_lens, int64_t{4} * B, false},
                   {free_blocks, int64_t{4} * num_free, false}, {block_table, int64_t{4} * B * max_blocks, true},
                   {seq_lens, int64_t{4} * B, true}, {query_start, int64_t{4} * B + 4, true},
                   {slots, int64_t{4} * num_tokens, true}, {positions, int64_t{4} * num_tokens, true}, {counts, 8, true}}))
        return FA_ERR_INVALID_ARG;
    fa::BlockTableParams p;
    p.table = block_table;
    p.ctx = ctx_lens;
    p.fresh = new_lens;
    p.free_blocks = free_blocks;
    p.seq_lens = seq_lens;
    p.query_start = query_start;
    p.slots = slots;
    p.positions = positions;
    p.counts = counts;
    p.B = B;
    p.max_blocks = max_blocks;
    p.block_shift = log2_of(block_size);
    p.num_free = num_free;
    p.num_tokens = num_tokens;
    p.wide = aligned(slots, 16) && aligned(positions, 16);
    const int smem = 3 * B * 4;
    if (smem > 32768 && cudaFuncSetAttribute(fa::fa_block_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             3 * fa::kMaxRequests * 4) != cudaSuccess)
        return FA_ERR_CUDA;
    // a CTA for each kTableTokens tokens; many requests with few tokens may
    // still need many blocks, which the CTAs take in turn
    const int64_t ctas = (static_cast<int64_t>(num_tokens) + fa::kTableTokens - 1) / fa::kTableTokens;
    if (launch_dependent(reinterpret_cast<cudaStream_t>(stream), dim3(static_cast<unsigned>(ctas > 0 ? ctas : 1)),
                         fa::kTableThreads, smem, reinterpret_cast<const void *>(fa::fa_block_tables_kernel), &p) !=
        cudaSuccess)
        return FA_ERR_CUDA;
    return launched();
}

extern "C" fa_status fa_rope(const void *Q, const int64_t *q_strides, void *Qr, const int64_t *qr_strides, int Hq,
                             const void *K, const int64_t *k_strides, void *Kr, const int64_t *kr_strides, int Hk,
                             const int *positions, int64_t pos_axis_stride, int64_t pos_batch_stride, int B, int N,
                             int d, int rot, int axes, const double *inv_freq, const int *pair_axis, int interleaved,
                             int inverse, fa_stream_t stream) {
    if (!Q || !Qr || !positions || Hq < 1 || Hk < 0 || B < 1 || N < 1) return FA_ERR_INVALID_ARG;
    if (Hk > 0 ? (!K || !Kr) : (K || Kr)) return FA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    const int64_t tokens = static_cast<int64_t>(B) * N, heads = static_cast<int64_t>(Hq) + Hk;
    if (tokens > (int64_t{1} << 30) || heads > 65535) return FA_ERR_INVALID_ARG;
    if (pos_axis_stride < 0 || pos_batch_stride < 0) return FA_ERR_INVALID_ARG;
    fa::RopeParams p;
    fa_status st = take_rotary(p.tab, d, rot, axes, inv_freq, pair_axis);
    if (st != FA_OK) return st;
    const int qe[3] = {B, Hq, N}, ke[3] = {B, Hk, N};
    for (const fa_status s : {take_strides(p.qs, q_strides, qe, 3, d, false),
                              take_strides(p.qos, qr_strides, qe, 3, d, true),
                              take_strides(p.ks, k_strides, ke, 3, d, false),
                              take_strides(p.kos, kr_strides, ke, 3, d, true)})
        if (s != FA_OK) return s;
    if (!aligned(Q, 16) || !aligned(Qr, 16) || !aligned(K, 16) || !aligned(Kr, 16) || !aligned(positions, 4))
        return FA_ERR_MISALIGNED;
    const void *q_in = Q, *k_in = K;
    if (!in_place_ok(q_in, p.qs, Qr, p.qos, qe, 3) || !in_place_ok(k_in, p.ks, Kr, p.kos, ke, 3) || Qr == Kr ||
        !apart<4>({{q_in, span_bytes(p.qs, qe, 3, d), false}, {k_in, span_bytes(p.ks, ke, 3, d), false},
                   {Qr, span_bytes(p.qos, qe, 3, d), true}, {Kr, span_bytes(p.kos, ke, 3, d), true}}))
        return FA_ERR_INVALID_ARG;
    p.q = static_cast<const __nv_bfloat16 *>(Q);
    p.k = static_cast<const __nv_bfloat16 *>(K);
    p.qo = static_cast<__nv_bfloat16 *>(Qr);
    p.ko = static_cast<__nv_bfloat16 *>(Kr);
    p.positions = positions;
    p.pos_axis = pos_axis_stride;
    p.pos_batch = pos_batch_stride;
    p.Hq = Hq;
    p.Hk = Hk;
    p.B = B;
    p.N = N;
    p.rot = rot;
    p.axes = axes;
    p.inverse = inverse != 0;
    p.tokens = static_cast<int>(tokens);
    p.heads = static_cast<int>(heads);
    return launch_rope(p, d, interleaved != 0, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" fa_status fa_paged_append(const void *Q, const int64_t *q_strides, void *Qr, const int64_t *qr_strides,
                                     int Hq, const void *K, const int64_t *k_strides, const void *V,
                                     const int64_t *v_strides, int Hkv, void *K_cache, void *V_cache, int cache_type,
                                     const float *k_descale, const float *v_descale, const int *slots,
                                     const int *positions, int64_t pos_axis_stride, int T, int num_blocks,
                                     int block_size, int d, int rot, int axes, const double *inv_freq,
                                     const int *pair_axis, int interleaved, fa_stream_t stream) {
    if (!K || !V || !K_cache || !V_cache || !slots || Hkv < 1 || Hq < 0 || T < 1 || num_blocks < 1)
        return FA_ERR_INVALID_ARG;
    if (Hq > 0 ? (!Q || !Qr) : (Q || Qr)) return FA_ERR_INVALID_ARG;
    if (cache_type != FA_CACHE_BF16 && cache_type != FA_CACHE_E4M3) return FA_ERR_INVALID_ARG;
    if (cache_type == FA_CACHE_E4M3 && (!k_descale || !v_descale)) return FA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    if (!block_size_ok(block_size)) return FA_ERR_UNSUPPORTED;
    const int64_t rows = static_cast<int64_t>(num_blocks) * block_size, heads = Hq + 2 * static_cast<int64_t>(Hkv);
    if (rows > 0x7fffffff || T > (1 << 30) || heads > 65535) return FA_ERR_INVALID_ARG;
    fa::RotaryTable tab;
    std::memset(&tab, 0, sizeof tab);
    if (rot != 0) {
        if (!positions || pos_axis_stride < 0) return FA_ERR_INVALID_ARG;
        const fa_status st = take_rotary(tab, d, rot, axes, inv_freq, pair_axis);
        if (st != FA_OK) return st;
    }
    const int qe[2] = {T, Hq}, ke[2] = {T, Hkv};
    int64_t strides[4][2];
    for (const fa_status s : {take_strides(strides[0], q_strides, qe, 2, d, false),
                              take_strides(strides[1], qr_strides, qe, 2, d, true),
                              take_strides(strides[2], k_strides, ke, 2, d, false),
                              take_strides(strides[3], v_strides, ke, 2, d, false)})
        if (s != FA_OK) return s;
    if (!aligned(Q, 16) || !aligned(Qr, 16) || !aligned(K, 16) || !aligned(V, 16) || !aligned(K_cache, 16) ||
        !aligned(V_cache, 16) || !aligned(slots, 4) || !aligned(positions, 4) || !aligned(k_descale, 4) ||
        !aligned(v_descale, 4))
        return FA_ERR_MISALIGNED;
    const void *q_in = Q;
    const int64_t cache = rows * Hkv * d * (cache_type == FA_CACHE_E4M3 ? 1 : 2);
    if (!in_place_ok(q_in, strides[0], Qr, strides[1], qe, 2) ||
        !apart<7>({{q_in, span_bytes(strides[0], qe, 2, d), false}, {K, span_bytes(strides[2], ke, 2, d), false},
                   {V, span_bytes(strides[3], ke, 2, d), false}, {slots, int64_t{4} * T, false},
                   {Qr, span_bytes(strides[1], qe, 2, d), true}, {K_cache, cache, true}, {V_cache, cache, true}}))
        return FA_ERR_INVALID_ARG;
    const auto run = [&](auto p) {
        p.q = static_cast<const __nv_bfloat16 *>(Q);
        p.k = static_cast<const __nv_bfloat16 *>(K);
        p.v = static_cast<const __nv_bfloat16 *>(V);
        p.qo = static_cast<__nv_bfloat16 *>(Qr);
        for (int i = 0; i < 2; ++i) {
            p.qs[i] = strides[0][i];
            p.qos[i] = strides[1][i];
            p.ks[i] = strides[2][i];
            p.vs[i] = strides[3][i];
        }
        p.k_cache = K_cache;
        p.v_cache = V_cache;
        p.k_descale = k_descale;
        p.v_descale = v_descale;
        p.slots = slots;
        p.positions = positions;
        p.pos_axis = rot ? pos_axis_stride : 0;
        p.cache_rows = rows;
        p.block_shift = log2_of(block_size);
        p.Hq = Hq;
        p.Hkv = Hkv;
        p.rot = rot;
        p.axes = axes;
        p.tokens = T;
        p.heads = static_cast<int>(heads);
        p.tab = tab;
        return launch_rope(p, d, interleaved != 0, reinterpret_cast<cudaStream_t>(stream));
    };
    return cache_type == FA_CACHE_E4M3 ? run(fa::AppendParams<true>()) : run(fa::AppendParams<false>());
}

namespace {

constexpr int kDecodeMaxNq = 16;
// Tables at most so many tiles wide: CTAs take whole items and there is no
// merge kernel.  One sequence, 8 key heads, d = 128, bf16, device time with
// whole items / shared ones: 77 keys (2 tiles) 4.5 / 5.3 us, 200 (4) 5.6 / 6.0,
// 480 (8) 7.9 / 6.2, 1000 (16) 12.7 / 6.4.
constexpr int kDecodeWholeTiles = 4;

fa_status validate_decode_sizes(int B, int Hq, int Hkv, int Nq, int d) {
    if (B < 1 || Hq < 1 || Hkv < 1 || Nq < 1 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
    if ((d != 64 && d != 128) || Nq > kDecodeMaxNq) return FA_ERR_UNSUPPORTED;
    if (Hq > 65535 || static_cast<int64_t>(B) * Hq * Nq > (int64_t{1} << 30)) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

// Workspace: the jobs, then m and l, then O of the partial results.
struct DecodeSpace {
    size_t ml, o, bytes;
};
DecodeSpace decode_space(int rows, int d) {
    const size_t cap = decode_rows(decode_layout(rows));
    const size_t part_rows = 2 * fa::kDecodeMaxCtas * (static_cast<size_t>(rows) < cap ? rows : cap);
    const auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
    DecodeSpace s;
    s.ml = up(fa::kDecodeMaxCtas * sizeof(fa::DecodeJob));
    s.o = up(s.ml + part_rows * sizeof(float2));
    s.bytes = up(s.o + part_rows * d * sizeof(float));
    return s;
}

}  // namespace

extern "C" fa_status fa_decode_paged_workspace(int B, int Hq, int Hkv, int Nq, int d, size_t *bytes) {
    if (!bytes) return FA_ERR_INVALID_ARG;
    const fa_status st = validate_decode_sizes(B, Hq, Hkv, Nq, d);
    if (st != FA_OK) return st;
    *bytes = decode_space(Hq / Hkv * Nq, d).bytes;
    return FA_OK;
}

extern "C" fa_status fa_decode_paged(const void *Q, const int64_t *q_strides, const void *K_cache,
                                     const void *V_cache, int cache_type, const float *k_descale,
                                     const float *v_descale, const int *block_table, const int *seq_lens, void *O,
                                     const int64_t *o_strides, float *LSE, int B, int Hq, int Hkv, int Nq,
                                     int max_blocks, int num_blocks, int block_size, int d, float scale, int causal,
                                     void *workspace, size_t workspace_bytes, fa_stream_t stream) {
    if (!Q || !K_cache || !V_cache || !block_table || !seq_lens || !O || !LSE || !workspace) return FA_ERR_INVALID_ARG;
    if (cache_type != FA_CACHE_BF16 && cache_type != FA_CACHE_E4M3) return FA_ERR_INVALID_ARG;
    if (cache_type == FA_CACHE_E4M3 && (!k_descale || !v_descale)) return FA_ERR_INVALID_ARG;
    if (max_blocks < 1 || num_blocks < 1 || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
    fa_status st = validate_decode_sizes(B, Hq, Hkv, Nq, d);
    if (st != FA_OK) return st;
    if (!block_size_ok(block_size)) return FA_ERR_UNSUPPORTED;
    fa::DecodeParams p;
    p.group = Hq / Hkv;
    p.rows = p.group * Nq;
    const DecodeSpace space = decode_space(p.rows, d);
    if (static_cast<int64_t>(max_blocks) * block_size > (int64_t{1} << 30) ||
        static_cast<int64_t>(num_blocks) * Hkv * block_size * d * 2 >= (int64_t{1} << 40) ||
        workspace_bytes < space.bytes)
        return FA_ERR_INVALID_ARG;
    const int e[3] = {B, Hq, Nq};
    for (const fa_status s : {take_strides(p.qs, q_strides, e, 3, d, false), take_strides(p.os, o_strides, e, 3, d, true)})
        if (s != FA_OK) return s;
    if (!aligned(Q, 16) || !aligned(K_cache, 16) || !aligned(V_cache, 16) || !aligned(O, 16) || !aligned(LSE, 4) ||
        !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(k_descale, 4) || !aligned(v_descale, 4) ||
        !aligned(workspace, 256))
        return FA_ERR_MISALIGNED;
    const bool f8 = cache_type == FA_CACHE_E4M3;
    const int64_t cache = static_cast<int64_t>(num_blocks) * Hkv * block_size * d * (f8 ? 1 : 2);
    // O may be Q: only an item's own CTAs read its queries, and its O is written when they are done
    const void *q_in = Q;
    if (!in_place_ok(q_in, p.qs, O, p.os, e, 3) ||
        !apart<8>({{q_in, span_bytes(p.qs, e, 3, d), false}, {K_cache, cache, false}, {V_cache, cache, false},
                   {block_table, int64_t{4} * B * max_blocks, false}, {seq_lens, int64_t{4} * B, false},
                   {O, span_bytes(p.os, e, 3, d), true}, {LSE, int64_t{4} * B * Hq * Nq, true},
                   {workspace, static_cast<int64_t>(space.bytes), true}}))
        return FA_ERR_INVALID_ARG;
    const DecodeLayout layout = decode_layout(p.rows);
    const int cap = decode_rows(layout);
    p.row_blocks = (p.rows + cap - 1) / cap;
    p.part_rows = p.rows < cap ? p.rows : cap;
    // at most so many units as the table is wide: a CTA each, up to as many as fit the GPU
    const bool partly = causal != 0 && Nq > 1;
    const DecodeKernel kernel = partly ? fa::decode_kernel_partly(d, f8, layout) : fa::decode_kernel<false>(d, f8, layout);
    const int64_t tiles = (static_cast<int64_t>(max_blocks) * block_size + kernel.tile - 1) / kernel.tile;
    p.whole_items = tiles <= kDecodeWholeTiles;
    const int64_t units = (p.whole_items ? 1 : tiles + fa::kDecodeItemUnits) * p.row_blocks * Hkv * B;
    if (units > (int64_t{1} << 38)) return FA_ERR_INVALID_ARG;   // a CTA counts its units in 31 bits
    // The kernel takes the maximum of raw scores, so it wants a positive
    // factor: a negative scale's sign goes to q, and zero runs as the
    // smallest normal number (every weight then rounds to the same value).
    p.c2 = static_cast<float>(std::fabs(static_cast<double>(scale)) * 1.4426950408889634);
    if (!std::isfinite(p.c2)) return FA_ERR_INVALID_ARG;
    if (p.c2 < 1.1754943508222875e-38f) p.c2 = 1.1754943508222875e-38f;
    p.q_sign = scale < 0.f ? 0x80008000u : 0u;
    int sms;
    st = serving_device(sms, 8 * layout.index + 4 * partly + 2 * f8 + (d == 128), kernel.fn, kernel.smem);
    if (st != FA_OK) return st;
    p.q = static_cast<const __nv_bfloat16 *>(Q);
    p.o = static_cast<__nv_bfloat16 *>(O);
    p.lse = LSE;
    p.k_cache = K_cache;
    p.v_cache = V_cache;
    p.k_descale = f8 ? k_descale : nullptr;
    p.v_descale = f8 ? v_descale : nullptr;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.Nq = Nq;
    p.max_blocks = max_blocks;
    p.num_blocks = num_blocks;
    p.block_shift = log2_of(block_size);
    p.causal = causal != 0;
    char *ws = static_cast<char *>(workspace);
    p.jobs = reinterpret_cast<fa::DecodeJob *>(ws);
    p.part_ml = reinterpret_cast<float2 *>(ws + space.ml);
    p.part_o = reinterpret_cast<float *>(ws + space.o);

    int64_t grid = static_cast<int64_t>(kernel.ctas_per_sm) * sms;
    if (grid > fa::kDecodeMaxCtas) grid = fa::kDecodeMaxCtas;
    if (grid > units) grid = units;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (launch_dependent(s, dim3(static_cast<unsigned>(grid)), fa::kDecodeThreads, kernel.smem, kernel.fn, &p) !=
        cudaSuccess)
        return FA_ERR_CUDA;
    if (p.whole_items) return launched();
    const void *merge = d == 64 ? reinterpret_cast<const void *>(fa::fa_decode_merge_kernel<64>)
                                : reinterpret_cast<const void *>(fa::fa_decode_merge_kernel<128>);
    if (launch_dependent(s, dim3(static_cast<unsigned>(grid), static_cast<unsigned>(p.part_rows)), fa::kMergeThreads, 0,
                         merge, &p) != cudaSuccess)
        return FA_ERR_CUDA;
    return launched();
}
