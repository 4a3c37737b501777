// What the chunked prefill's kernels share: parameters, key tiles and the merge
// of a query-tile pair's pieces. The kernel for
// a bf16 cache without a window is in prefill.cu, with its design; those for a
// window with sinks and for a block-scaled E4M3 cache are in prefill_win.cuh.
#pragma once

#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "tc_sm100.cuh"

struct PaPrefillParams {
    uint16_t* out;
    const uint16_t* q;
    const int32_t* tables;
    const int32_t* ctx;
    const int32_t* qsl;
    float scale_log2;
    int n_heads;
    int n_kv_heads;
    int max_blocks;
    int num_blocks;
    int oob_row;  // a TMA row coordinate past the end of the pool (zero fill)
    int splits;   // per-pair mode: pieces per query-tile pair (1: no split)
    float* part;  // partials of pieces: [item][piece] (per-pair mode) or [slot] (balanced mode),
                  // each [tile][row][kPartStride]
    // Balanced mode (work null in per-pair mode). Item it = (sequence *
    // n_kv_heads + kv head) * n_qp + pair. The planning kernel writes the
    // work list: every non-empty item whole, in item order, except the items
    // of the last partial wave, which are cut into sched[2] equal key ranges
    // (piece-major); CTAs take entries in order from the counter sched[0].
    int4* work;      // entries (item, first key tile, end key tile, partial slot or -1); sched[1] of them
    int* sched;      // counter, entries, pieces per cut item, cut items
    int n_items;
    int n_qp;
    int n_cta;
    unsigned int* err;
    int window;   // >= 0: a row at position p sees p - window .. p, and 0 .. n_sinks - 1
    int n_sinks;
    const float* k_scale;  // E4M3: [num_blocks][n_kv_heads]
    const float* v_scale;
    // pa_prefill_score_mod (reshape): scores are cap2 tanh(x), x = q.k * scale_log2 (scale / cap there) and
    // cap2 = cap * log2(e), 0: not capped, less slopes[head] * distance (null: none); prefix [n_seqs] (null:
    // none): keys before it are visible to earlier rows too
    int reshape;
    float cap2;
    float poly[4], small;  // cap2 tanh(x) = y (poly[0] + poly[1] y^2 + ..) for |x| <= small, y = q.k (bf16)
    const float* slopes;
    const int32_t* prefix;
};

// Launches of the windowed and of the E4M3 instantiations (translation units
// of their own): head_dim 64 or 128, G in {1, 2, 4, 8}.
int pa_prefill_dispatch_sinks(int head_dim, int G, const PaPrefillParams& P, const CUtensorMap& tk, const CUtensorMap& tv,
                              int n_seqs, int n_rows, cudaStream_t stream);
int pa_prefill_dispatch_fp8(int head_dim, int G, const PaPrefillParams& P, const CUtensorMap& tk, const CUtensorMap& tv,
                            int n_seqs, int n_rows, cudaStream_t stream);
// of reshaped scores: with a cap alone, a bias by distance or none, both
int pa_prefill_dispatch_cap(int head_dim, int G, const PaPrefillParams& P, const CUtensorMap& tk, const CUtensorMap& tv,
                            int n_seqs, int n_rows, cudaStream_t stream);
int pa_prefill_dispatch_cap_fp8(int head_dim, int G, const PaPrefillParams& P, const CUtensorMap& tk, const CUtensorMap& tv,
                                int n_seqs, int n_rows, cudaStream_t stream);
int pa_prefill_dispatch_bias(int head_dim, int G, const PaPrefillParams& P, const CUtensorMap& tk, const CUtensorMap& tv,
                             int n_seqs, int n_rows, cudaStream_t stream);
int pa_prefill_dispatch_bias_fp8(int head_dim, int G, const PaPrefillParams& P, const CUtensorMap& tk, const CUtensorMap& tv,
                                 int n_seqs, int n_rows, cudaStream_t stream);
int pa_prefill_dispatch_both(int head_dim, int G, const PaPrefillParams& P, const CUtensorMap& tk, const CUtensorMap& tv,
                             int n_seqs, int n_rows, cudaStream_t stream);
int pa_prefill_dispatch_both_fp8(int head_dim, int G, const PaPrefillParams& P, const CUtensorMap& tk, const CUtensorMap& tv,
                                 int n_seqs, int n_rows, cudaStream_t stream);

namespace {

constexpr int kBS = 16;          // tokens per block
constexpr int kKT = 128;         // keys per key tile
constexpr int kBPT = kKT / kBS;  // blocks per key tile
constexpr int kRows = 128;       // MMA M
constexpr unsigned kFull = 0xffffffffu;
constexpr uint32_t kTmemCols = 512;  // tile X: S at 256X, O at 256X + 128 (D columns)

using PrefillParams = PaPrefillParams;

// A sequence's prefix, at most its context; 0 without one (an entry below 0 is none).
__device__ __forceinline__ int prefix_of(const PrefillParams& P, int s, int ctx) {
    return P.prefix ? max(0, min(P.prefix[s], ctx)) : 0;
}

// The key tiles that the rows of a query-tile pair attend to: the cache blocks
// that some row sees, in order - the n_sink leading ones that hold sinks, then
// those from `first` on, the block of `lo`, the first position in the window of
// the pair's first row (all blocks without a window) - eight a tile, so that a
// tile may hold sinks and the window's beginning. n tiles.
struct KeyTiles {
    int lo, first, n_sink, n;
    __device__ __forceinline__ KeyTiles(const PrefillParams& P, int first_row_pos, int last_row_pos) {
        lo = P.window >= 0 ? max(0, first_row_pos - P.window) : 0;
        first = lo / kBS;
        n_sink = min((P.n_sinks + kBS - 1) / kBS, first);
        n = (n_sink + last_row_pos / kBS - first + kBPT) / kBPT;
    }
    __device__ __forceinline__ int block(int i) const { return i < n_sink ? i : i - n_sink + first; }
    // position of key k of tile j
    __device__ __forceinline__ int position(int j, int k) const { return block(j * kBPT + k / kBS) * kBS + k % kBS; }
};

// A block-scaled cache's scale, within the range the library works with.
__device__ __forceinline__ float clamp_scale(float s) { return fminf(fmaxf(s, 0x1p-32f), 0x1p32f); }

// Four E4M3 codes -> four fp16 values (exact), two a register.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t codes, uint32_t& a, uint32_t& b) {
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(a), "=r"(b)
        : "r"(codes));
}

// A piece's partial for one row: the un-normalised O (head_dim floats from
// offset 0), and at offset 128 the reference maximum m (base-2 units) and the
// sum l of 2^(s*scale - m); the same row size for both head dims.
constexpr int kPartStride = 132;  // floats, 16-byte aligned rows
constexpr int kPartML = 128;      // offset of (m, l) in a partial row

// Key tiles [kt0, kt1) of piece sp out of `splits` over a pair's n_kt tiles.
__host__ __device__ inline void piece_range(int n_kt, int sp, int splits, int& kt0, int& kt1) {
    kt0 = (int)((long long)sp * n_kt / splits);
    kt1 = (int)((long long)(sp + 1) * n_kt / splits);
}

// fp32 -> fp16 round to nearest even; a in the low half, b in the high half
// (beyond the fp16 range: infinity).
__device__ __forceinline__ uint32_t float2_to_f16x2(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Instruction descriptor of tcgen05.mma kind::f16 with fp16 A and B (the
// kind takes one type for both operands) and an fp32 accumulator; fields as
// in tc::idesc_bf16_f32 with the A and B format fields 0 (fp16).
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, int a_mn_major, int b_mn_major) {
    return (1u << 4) | ((uint32_t)a_mn_major << 15) | ((uint32_t)b_mn_major << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Whether a sequence of L > 0 rows is left out and flagged: its chunk is not in
// the cache yet, or (calls with a window, over E4M3 or of reshaped scores) its context runs past its
// table or its chunk past max_chunk_len.
template <int G>
__device__ __forceinline__ bool left_out(const PrefillParams& P, int L, int ctx) {
    constexpr int QT = kRows / G;
    if (ctx < L) return true;
    return (P.window >= 0 || P.k_scale || P.reshape) && ((ctx - 1) / kBS >= P.max_blocks || (L - 1) / (2 * QT) >= P.n_qp);
}

// Key tiles of item it = (sequence * n_kv_heads + kv head) * n_qp + pair:
// 0 if the pair has no rows. A sequence that is left out has none either, and
// flags the device error once.
template <int G>
__device__ int item_tiles(const PrefillParams& P, int it) {
    constexpr int QT = kRows / G;
    const int per_seq = P.n_kv_heads * P.n_qp;
    const int s = it / per_seq, qp = it % P.n_qp;
    const int q0 = P.qsl[s], L = P.qsl[s + 1] - q0, i0 = qp * 2 * QT;
    if (i0 >= L) return 0;
    const int ctx = P.ctx[s];
    if (left_out<G>(P, L, ctx)) {
        if (it % per_seq == 0) pa::set_error(P.err, PA_DEVERR_CONTEXT);
        return 0;
    }
    return KeyTiles(P, ctx - L + i0, max(ctx - L + min(i0 + 2 * QT, L), prefix_of(P, s, ctx)) - 1).n;
}

// Combines the pieces of one output row: O = sum_k O_k 2^(m_k - M),
// l = sum_k l_k 2^(m_k - M), out = O / l (lane: D / 32 consecutive dims).
// Piece k covers key tiles piece_range(n_kt_all, k, n_pieces); empty ones
// wrote nothing and are skipped. Up to 8 pieces: every lane loads every
// piece's (m, l) (one broadcast load each) and its O slices, all at once, so
// the row costs one round of memory latency. More pieces (n_pieces <= 64):
// lane k reads piece k's (m, l), then the O slices are loaded 8 pieces at a
// time.
template <int NV>
__device__ __forceinline__ void store_row(const float (&acc)[NV], float inv, int lane, uint16_t* out_row) {
    if constexpr (NV == 4) {
        uint2 pk;
        pk.x = pa::float2_to_bf16x2(acc[0] * inv, acc[1] * inv);
        pk.y = pa::float2_to_bf16x2(acc[2] * inv, acc[3] * inv);
        *reinterpret_cast<uint2*>(out_row + lane * 4) = pk;
    } else {
        *reinterpret_cast<uint32_t*>(out_row + lane * 2) = pa::float2_to_bf16x2(acc[0] * inv, acc[1] * inv);
    }
}
template <int NV>
__device__ __forceinline__ void load_slice(const float* src, int lane, float (&v)[NV]) {
    if constexpr (NV == 4) {
        const float4 t = *reinterpret_cast<const float4*>(src + lane * 4);
        v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
    } else {
        const float2 t = *reinterpret_cast<const float2*>(src + lane * 2);
        v[0] = t.x; v[1] = t.y;
    }
}
template <int D, typename PartOf>
__device__ __forceinline__ void merge_row(int n_pieces, int n_kt_all, PartOf part_of, int lane, uint16_t* out_row) {
    constexpr int NV = D / 32;  // dims per lane: 4 or 2
    if (n_pieces <= 8) {
        float v[8][NV];
        float2 ml[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            int a = 0, b = 0;
            if (k < n_pieces) piece_range(n_kt_all, k, n_pieces, a, b);
            ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int e = 0; e < NV; ++e) v[k][e] = 0.f;
            if (b > a) {
                const float* src = part_of(k);
                ml[k] = *reinterpret_cast<const float2*>(src + kPartML);
                load_slice<NV>(src, lane, v[k]);
            }
        }
        float M = -INFINITY;
#pragma unroll
        for (int k = 0; k < 8; ++k) M = fmaxf(M, ml[k].x);
        float l = 0.f, acc[NV] = {};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float f = ml[k].x == -INFINITY ? 0.f : pa::fast_exp2(ml[k].x - M);
            l += ml[k].y * f;
#pragma unroll
            for (int e = 0; e < NV; ++e) acc[e] += v[k][e] * f;
        }
        store_row<NV>(acc, 1.f / l, lane, out_row);
        return;
    }
    float m_mine = -INFINITY, l_mine = 0.f;
    for (int k = lane; k < n_pieces; k += 32) {
        int a, b;
        piece_range(n_kt_all, k, n_pieces, a, b);
        if (b > a) {
            const float2 ml = *reinterpret_cast<const float2*>(part_of(k) + kPartML);
            if (ml.x > m_mine) {  // keep the larger reference; rescale the other sum
                l_mine = l_mine * (m_mine == -INFINITY ? 0.f : pa::fast_exp2(m_mine - ml.x)) + ml.y;
                m_mine = ml.x;
            } else {
                l_mine += ml.x == -INFINITY ? 0.f : ml.y * pa::fast_exp2(ml.x - m_mine);
            }
        }
    }
    float M = m_mine;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
    float l = m_mine == -INFINITY ? 0.f : l_mine * pa::fast_exp2(m_mine - M);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
    float acc[NV] = {};
    for (int k0 = 0; k0 < n_pieces; k0 += 8) {
        float v[8][NV];
        float f[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int k = k0 + u;
            int a = 0, b = 0;
            if (k < n_pieces) piece_range(n_kt_all, k, n_pieces, a, b);
            f[u] = 0.f;
#pragma unroll
            for (int e = 0; e < NV; ++e) v[u][e] = 0.f;
            if (b > a) {
                const float* src = part_of(k);
                const float m = src[kPartML];
                f[u] = m == -INFINITY ? 0.f : pa::fast_exp2(m - M);
                load_slice<NV>(src, lane, v[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
            for (int e = 0; e < NV; ++e) acc[e] += v[u][e] * f[u];
    }
    store_row<NV>(acc, 1.f / l, lane, out_row);
}

// Per-pair mode with splits > 1: one warp per (chunk row, query head).
template <int G, int D>
__global__ void __launch_bounds__(128)
pa_prefill_merge_kernel(const PrefillParams P, int n_seqs, int n_rows_total, int n_qp) {
    constexpr int QT = kRows / G;
    pa::grid_dependency_wait();  // every piece's partial is written
    const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int H = P.n_heads, Hk = P.n_kv_heads;
    if (w >= (long long)n_rows_total * H) return;
    const int t = (int)(w / H), h = (int)(w % H);
    // the sequence whose chunk holds row t: the last s with qsl[s] <= t
    int lo = 0, hi = n_seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (P.qsl[mid] <= t) lo = mid; else hi = mid - 1;
    }
    const int s = lo;
    const int q0 = P.qsl[s], L = P.qsl[s + 1] - q0, ctx = P.ctx[s];
    const int i = t - q0;
    if (i < 0 || i >= L || left_out<G>(P, L, ctx)) return;
    const int qp = i / (2 * QT), x = (i % (2 * QT)) / QT, r = (i % QT) * G + h % G, kvh = h / G;
    if (qp >= n_qp) return;  // a chunk beyond max_chunk_len: no partials
    const int i0 = qp * 2 * QT;
    const int n_kt_all = KeyTiles(P, ctx - L + i0, max(ctx - L + min(i0 + 2 * QT, L), prefix_of(P, s, ctx)) - 1).n;
    const size_t item = ((size_t)s * Hk + kvh) * n_qp + qp;
    merge_row<D>(P.splits, n_kt_all,
                 [&](int k) { return P.part + (((item * P.splits + k) * 2 + x) * 128 + r) * kPartStride; }, lane,
                 P.out + ((size_t)t * H + h) * D);
}

}  // namespace
