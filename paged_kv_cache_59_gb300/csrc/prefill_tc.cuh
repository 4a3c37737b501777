// Chunked causal prefill over the paged KV cache on the tcgen05 tensor cores.
//
// What is computed ("Modern AI Infrastructure and Agentic System Design",
// 9.1 "Two workloads wearing one name": a long prompt is processed in chunks
// interleaved with decode; "KV Cache Explained Like You're an LLM Engineer",
// "Prefill Phase vs. Decode Phase"; causal masking as in "What Happens Inside
// an LLM During Inference ...", "Self-Attention Mechanism"): sequence s's
// chunk of L new tokens occupies the last L of its context_lens[s] cached
// positions; chunk row i sits at position p = ctx - L + i and
//     out[i][h] = sum_{t <= p} softmax_t(scale * q[i][h] . K[t]) V[t].
//
// Design (GB300), for head_dim D = 64 or 128 (one instantiation each; the
// K/V block rows are D bf16 values, moved as D/64 boxes of 64 dims). A query
// tile is 128 matrix rows = QT = 128/G chunk tokens x
// the G query heads of one KV head's group, so every K/V byte staged in
// shared memory feeds all G heads. One CTA owns two query tiles (A and B) of
// the same (sequence, KV head): both use every K/V tile it loads, and the
// tensor core alternates between them so that one tile's MMAs run while the
// other tile's softmax works. Per key tile j of 128 keys (8 blocks of 16),
// five roles in 14 warps, each waiting only on mbarriers or, for the
// hand-over of P, on a named barrier:
//   - a producer warp moves the 8 K and 8 V blocks with 2-D TMA loads into
//     128B-swizzled shared memory: two K stages and three V stages, each
//     refilled as soon as the tensor core is done with it (blocks past the
//     end of the sequence load out of bounds and arrive as zeros);
//   - four converter warps (one per scheduler) rewrite each landed V tile in
//     place as fp16 values of v * 2^-8 (rows past the context, which hold
//     whatever the pool has there, become zeros);
//   - one thread of an MMA warp issues, per query tile X, S_X = Q_X K_j^T
//     (tcgen05.mma kind::f16, bf16 in, fp32 accumulator in tensor memory,
//     M = N = 128, K = D) and, once X's softmax has written P, O_X += P V_j (fp16
//     in: P read from tensor memory, V as an MN-major shared-memory operand)
//     with S_X(j+1) right behind it. The MMAs of one thread execute in issue
//     order, so S_X(j+1) may follow the PV MMA that still reads P(j) out of
//     the same columns, and the completion of S_X(j+1) covers that PV MMA;
//   - one softmax warpgroup per query tile (thread = row) reads S_X from
//     tensor memory once, a quarter of 32 columns at a time, applies the
//     scale, the causal mask (diagonal tiles only) and an online softmax in
//     fp32 (base 2) against the row's integer reference maximum m (changed
//     only on a row's first visible keys or before any p = 2^(s*scale - m)
//     could leave the fp16 range, so every rescale of O, l and the tile's
//     earlier P is an exact power of two), and writes P back into S_X's
//     columns as fp16 (rounded to nearest: within 2^-12 of p relative).
//     A bf16 P (within 2^-9) would exceed an absolute error of 2e-3 on short
//     causal rows with cancelling values; the tensor core takes A and B of
//     one type, hence V in fp16 too. Every bf16 value is an fp16 value
//     inside fp16's exponent range; the factor 2^-8 moves that range up to
//     |v| <= 65504 * 2^8 (larger values become infinite and the output
//     non-finite, which is flagged), at an absolute error of at most 2^-17
//     for |v| < 2^-6, where the scaled value is subnormal. The four warps
//     hand P over to the MMA warp through a named barrier (arrive/sync).
// The normalised output 2^8 O / l is written once at the end.
//
// Window with sinks (WIN): a row at position p sees p - window .. p and the
// first n_sinks positions. Only the key tiles that a row of the pair sees are
// walked (KeyTiles), so the work of a long prompt's chunk is that of its
// window; the tiles at the window's and the sinks' edges take the masking code.
//
// E4M3 cache with a scale per (block, KV head) (EB = 1): the codes of a K and
// of a V tile (half the bytes) land in a buffer each, and the converter warps
// widen both to fp16, exactly; Q is converted to fp16 once. Scales never touch
// the operands: the softmax threads apply them to S and to the exponent.
//
// Scheduling. Per-pair mode: one CTA per (pair, KV head, sequence), or per
// piece of its key range. Balanced mode: one CTA per SM takes entries of a
// work list in order (whole pairs for the full waves, pieces of the pairs of
// the last partial wave) and runs them one after another, re-initialising
// its barriers between entries; pieces leave partials for a merge kernel.
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
};

// Launches of the windowed and of the E4M3 instantiations (translation units
// of their own): head_dim 64 or 128, G in {1, 2, 4, 8}.
int pa_prefill_dispatch_sinks(int head_dim, int G, const PaPrefillParams& P, const CUtensorMap& tk, const CUtensorMap& tv,
                              int n_seqs, int max_chunk_len, int n_rows, cudaStream_t stream);
int pa_prefill_dispatch_fp8(int head_dim, int G, const PaPrefillParams& P, const CUtensorMap& tk, const CUtensorMap& tv,
                            int n_seqs, int max_chunk_len, int n_rows, cudaStream_t stream);

namespace {

constexpr int kBS = 16;          // tokens per block
constexpr int kKT = 128;         // keys per key tile
constexpr int kBPT = kKT / kBS;  // blocks per key tile
constexpr int kRows = 128;       // MMA M
constexpr unsigned kFull = 0xffffffffu;

constexpr int kKS = 2;  // K tile stages
constexpr int kThreads = 448;  // 8 softmax warps, MMA warp (8), producer (9), 4 converter warps (10..13)
// Shared memory map for head_dim D (64 or 128): a Q tile (128 rows) and a
// K or V tile (128 keys) are 128 x D bf16 values each, stored as D / 64
// 128B-swizzled halves of 64 dims (16 KiB each). The dynamic shared memory
// base must be 1024-byte aligned (swizzle atoms of TMA and of the matrix
// descriptors): checked. EB = bytes per cached element: 2 (bf16), or 1 (E4M3),
// where the codes of a K and of a V tile land in a buffer of their own (128
// rows of D bytes) and the stages hold them widened to fp16; that room costs
// the third V stage.
template <int D, int EB>
struct PfLay {
    static_assert(D == 64 || D == 128, "head_dim 64 or 128");
    static constexpr int kVS = EB == 2 ? 3 : 2;          // V tile stages
    static constexpr int kHalves = D / 64;               // 64-dim halves of a row
    static constexpr uint32_t kTile = kKT * D * 2;       // K or V tile bytes
    static constexpr uint32_t kQTile = kRows * D * 2;    // Q tile bytes
    static constexpr uint32_t kQ = 0;                    // Q_A, Q_B
    static constexpr uint32_t kK0 = 2 * kQTile;          // K stages
    static constexpr uint32_t kV0 = kK0 + kKS * kTile;   // V stages
    static constexpr uint32_t kRaw = kV0 + kVS * kTile;  // E4M3: codes of a K tile, of a V tile
    static constexpr uint32_t kRawTile = kKT * D;
    static constexpr uint32_t kBars = kRaw + (EB == 1 ? 2 * kRawTile : 0);  // mbarriers
    static constexpr uint32_t kMisc = kBars + 256;       // tmem slot, abort flag, segment entries
    static constexpr uint32_t kSmem = kMisc + 64;
    static_assert(kSmem <= 227 * 1024, "shared memory budget");
};
constexpr uint32_t kTmemCols = 512;  // tile X: S at 256X, O at 256X + 128 (D columns)

using PrefillParams = PaPrefillParams;

// The key tiles that the rows of a query-tile pair attend to, numbered 0 ..
// n-1: the n_sink leading tiles that hold sinks, then tiles `first` .. from
// the window of the pair's first row to its last row (all without a window).
// `lo`: the first position in that row's window.
struct KeyTiles {
    int lo, first, n_sink, n;
    __device__ __forceinline__ KeyTiles(const PrefillParams& P, int first_row_pos, int last_row_pos) {
        lo = P.window >= 0 ? max(0, first_row_pos - P.window) : 0;
        first = lo / kKT;
        n_sink = min((P.n_sinks + kKT - 1) / kKT, first);
        n = n_sink + last_row_pos / kKT + 1 - first;
    }
    __device__ __forceinline__ int tile(int j) const { return j < n_sink ? j : j - n_sink + first; }
    // whether some row of the pair sees one of the positions a .. b-1 (past the context aside)
    __device__ __forceinline__ bool seen(const PrefillParams& P, int a, int b) const { return b > lo || a < P.n_sinks; }
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

// Bounded wait (1 s) that also gives up once another role has aborted. A
// waiting thread sleeps inside try_wait (up to 20 us per try, woken when the
// phase completes), so idle roles take no issue slots from busy ones.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, unsigned int* err,
                                         volatile int* abort_flag) {
    if (pa::mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    const uint64_t t0 = pa::globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (pa::mbar_try_wait_sleep(bar, parity, 20000u)) return true;
        if ((it & 15u) == 0) {
            if (*abort_flag) return false;
            if (pa::globaltimer_ns() - t0 > PA_WAIT_LIMIT_NS) {
                pa::set_error(err, PA_DEVERR_TIMEOUT);
                *abort_flag = 1;
                return false;
            }
        }
    }
}

// Even mode: a warp's 32 rows (thread = row) of a cut item. There is no merge
// launch: whichever piece of these rows comes last joins all of them, so no
// CTA ever waits for another. A piece that finds the others' partials complete
// keeps its own in tensor memory and joins; any other writes its partial, and
// joins if the rest became complete meanwhile. The sum over pieces runs in
// their order, whoever makes it, so the result does not depend on timing.
// (About 40 MB of partials less to read than with a merge kernel, and a launch
// less: the piece a CTA passes on is its last, the rest its successor's first,
// so it nearly always is the last one and never writes.)
// Partial of a slot's tile x: float4 [D / 4][128 rows] of O, then float2 [128]
// of (m, l). `own(c, v)` gives columns 32 c .. 32 c + 31 of this row's O (warp-
// collective); `put(c, v)` takes the joined ones, normalised.
__device__ __forceinline__ float* slot_part(const PrefillParams& P, int slot, int x) {
    return P.part + ((size_t)slot * 2 + x) * 128 * kPartStride;
}
template <int D, typename Own, typename Put>
__device__ __forceinline__ void join_pieces(const PrefillParams& P, int slot, int x, int r, int warp, int lane, float m,
                                            float l, Own own, Put put) {
    const int4* cta = P.work + P.n_items + P.n_cta;
    const int c = slot >> 1;
    const int4 info = cta[slot & 1 ? c + 1 : c];
    const int ca = info.z, n = info.w, me = c - ca;
    int* count = const_cast<int*>(reinterpret_cast<const int*>(cta + P.n_cta)) + (ca + 1) * 8 + warp;
    auto counted = [&]() {  // every lane acquires: it reads other CTAs' partials itself
        int v;
        asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(count) : "memory");
        return v;
    };
    bool last = __all_sync(kFull, counted() == n - 1);
    if (!last) {
        float* dst = slot_part(P, slot, x);
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
            float v[32];
            own(q, v);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                reinterpret_cast<float4*>(dst)[(8 * q + k) * 128 + r] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        }
        reinterpret_cast<float2*>(dst + 128 * D)[r] = make_float2(m, l);
        __threadfence();
        __syncwarp();
        int before = 0;
        if (lane == 0) before = atomicAdd(count, 1);
        last = __shfl_sync(kFull, before, 0) == n - 1;
        if (last) last = __all_sync(kFull, counted() == n);  // (always: all have been counted)
    }
    if (!last) return;
    auto ml = [&](int k) {
        return k == me ? make_float2(m, l)
                       : __ldcg(reinterpret_cast<const float2*>(slot_part(P, k == 0 ? 2 * ca + 1 : 2 * (ca + k), x) + 128 * D) + r);
    };
    float M = -INFINITY, sum = 0.f;
    for (int k = 0; k < n; ++k) M = fmaxf(M, ml(k).x);
    auto factor = [&](float mk) { return mk == -INFINITY ? 0.f : pa::fast_exp2(mk - M); };
    for (int k = 0; k < n; ++k) {
        const float2 p = ml(k);
        sum += p.y * factor(p.x);
    }
    const float inv = 1.f / sum;
#pragma unroll 1
    for (int q = 0; q < D / 32; ++q) {
        float acc[32] = {};
#pragma unroll 1
        for (int k = 0; k < n; ++k) {
            const float f = factor(ml(k).x);
            float v[32];
            if (k == me) {  // warp-uniform
                own(q, v);
            } else {
                const float4* src = reinterpret_cast<const float4*>(slot_part(P, k == 0 ? 2 * ca + 1 : 2 * (ca + k), x));
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float4 w = __ldcg(src + (8 * q + u) * 128 + r);
                    v[4 * u] = w.x;
                    v[4 * u + 1] = w.y;
                    v[4 * u + 2] = w.z;
                    v[4 * u + 3] = w.w;
                }
            }
#pragma unroll
            for (int u = 0; u < 32; ++u) acc[u] += v[u] * f;
        }
#pragma unroll
        for (int u = 0; u < 32; ++u) acc[u] *= inv;
        put(q, acc);
    }
}

// WIN: rows may have a lower bound (a window with sinks). EB = 1: an E4M3 cache
// with a scale per (block, KV head).
template <int G, int D, int EB, bool WIN>
__global__ void __launch_bounds__(kThreads, 1)
pa_prefill_tc_kernel(const PrefillParams P, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV) {
    using L_ = PfLay<D, EB>;
    constexpr int kVS = L_::kVS;
    constexpr uint32_t kQ = L_::kQ, kK0 = L_::kK0, kV0 = L_::kV0, kBars = L_::kBars, kMisc = L_::kMisc;
    constexpr uint32_t kTile = L_::kTile, kQTile = L_::kQTile;
    constexpr int kNH = L_::kHalves;
    constexpr int QT = kRows / G;  // chunk tokens per query tile
    extern __shared__ __align__(1024) unsigned char sm[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kBars);
    // E4M3: k_full[0], v_full[0] are the landed codes, k_free and v_free the fp16 stages' as here
    uint64_t* k_full = bars;          // [kKS] K tile landed
    uint64_t* k_free = k_full + kKS;  // [kKS] QK_B, the last reader of the K stage, is done
    uint64_t* v_full = k_free + kKS;  // [kVS] V tile landed (bf16)
    uint64_t* v_free = v_full + kVS;  // [kVS] PV_B, the last reader of the V stage, is done
    uint64_t* s_full = v_free + kVS;  // [2] per query tile: S_X(j) and every earlier MMA done
    uint64_t* pv_done = s_full + 2;   // [2] per query tile
    uint64_t* drain = pv_done + 2;    // every MMA issued in the segment is done
    uint64_t* v_conv = drain + 1;     // [kVS] V tile rewritten as fp16, 4 arrivals (one per converter warp)
    uint64_t* k_conv = v_conv + kVS;  // E4M3: [kKS] K tile widened to fp16, 4 arrivals
    uint64_t* raw_free = k_conv + (EB == 1 ? kKS : 0);  // E4M3: [2] the codes of K, of V are read, 4 arrivals
    constexpr int kNumBars = 2 * kKS + 3 * kVS + 5 + (EB == 1 ? kKS + 2 : 0);
    static_assert(kNumBars * 8 <= 256, "barrier area");
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + kMisc + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int H = P.n_heads, Hk = P.n_kv_heads;
    if (pa::smem_u32(sm) & 1023u) {  // never expected; refuse rather than mis-swizzle
        if (threadIdx.x == 0) pa::set_error(P.err, PA_DEVERR_LAYOUT);
        return;
    }
    // Segments. Per-pair mode: piece sp of pair (qp, kv head, sequence) from
    // the grid position. Balanced mode: the work-list entries this CTA takes
    // from the counter, one at a time.
    int* next = reinterpret_cast<int*>(sm + kMisc + 8);  // [2] the entry taken, by segment parity
    int entry_at = 0, entry_end = 0;                     // even mode
    int4 entry_next = make_int4(0, 0, 0, 0);
    bool have_tmem = false;
    uint32_t tbase = 0;
    if constexpr (WIN) {
        pa::launch_dependents();     // the next kernel may be scheduled
        pa::grid_dependency_wait();  // the plan, and whatever wrote the cache, is complete
    }
    int n_run = 0;  // segments run so far
    for (int seg = 0;; ++seg) {
        int s, kvh, qp, kt0 = 0, kt1 = 0;
        bool direct = true;
        int slot = -1;  // even mode: this piece's slot, or a whole item
        float* part_base = nullptr;
        if (WIN && P.work) {
            // even mode: this CTA's run of entries; the next one is loaded ahead
            if (seg == 0) {
                const int4 c = P.work[P.n_items + P.n_cta + blockIdx.x];
                entry_at = c.x;
                entry_end = c.y;
                if (entry_at < entry_end) entry_next = P.work[entry_at];
            }
            if (entry_at >= entry_end) break;
            const int4 e = entry_next;
            if (++entry_at < entry_end) entry_next = P.work[entry_at];
            kt0 = e.y;
            kt1 = e.z;
            slot = e.w;
            s = e.x / (Hk * P.n_qp);
            kvh = (e.x / P.n_qp) % Hk;
            qp = e.x % P.n_qp;
        } else if (P.work) {
            if (threadIdx.x == 0) next[seg & 1] = atomicAdd(&P.sched[0], 1);
            __syncthreads();
            const int w = next[seg & 1];
            if (w >= P.sched[1]) break;
            const int4 e = P.work[w];
            kt0 = e.y;
            kt1 = e.z;
            direct = e.w < 0;
            if (!direct) part_base = P.part + (size_t)e.w * 2 * 128 * kPartStride;
            s = e.x / (Hk * P.n_qp);
            kvh = (e.x / P.n_qp) % Hk;
            qp = e.x % P.n_qp;
        } else {
            if (seg > 0) break;
            qp = blockIdx.x / P.splits;
            kvh = blockIdx.y;
            s = blockIdx.z;
        }
        const int h0 = kvh * G;
        const int q0 = P.qsl[s];
        const int L = P.qsl[s + 1] - q0;
        const int i0 = qp * 2 * QT;  // first chunk token of query tile A; tile B follows
        if (i0 >= L) continue;       // segment-uniform, before any barrier or TMEM use
        const int ctx = P.ctx[s];
        if (ctx < L) {  // the chunk must be in the cache already
            if (threadIdx.x == 0) pa::set_error(P.err, PA_DEVERR_CONTEXT);
            continue;
        }
        const int nblk = min((ctx + kBS - 1) / kBS, P.max_blocks);
        const int first_pos = ctx - L;
        // both tiles walk the key tiles up to the last row of the pair (tile A's
        // extra tiles beyond its own rows are fully masked)
        const int p_last = first_pos + min(i0 + 2 * QT, L) - 1;
        const KeyTiles keys(P, first_pos + i0, p_last);
        const int n_kt_all = keys.n;
        if (!P.work) {  // this CTA's piece of the key tiles (all of them when not split)
            const int sp = blockIdx.x % P.splits;
            piece_range(n_kt_all, sp, P.splits, kt0, kt1);
            direct = P.splits <= 1;
            if (!direct) {
                const size_t item = ((size_t)s * Hk + kvh) * (gridDim.x / P.splits) + qp;
                part_base = P.part + (item * P.splits + sp) * 2 * 128 * kPartStride;
            }
        }
        kt1 = min(kt1, n_kt_all);
        const int n_kt = kt1 - kt0;  // tiles this segment walks; local tile j is key tile keys.tile(kt0 + j)
        if (n_kt <= 0) continue;     // segment-uniform; the merge skips empty pieces

        if (threadIdx.x == 0) {
            if (n_run > 0) {  // every phase of the last segment has completed
                for (int b = 0; b < kNumBars; ++b) pa::mbar_inval(&bars[b]);
            } else {
                *abort_flag = 0;
            }
            for (int i = 0; i < kKS; ++i) {
                pa::mbar_init(&k_full[i], 1);
                pa::mbar_init(&k_free[i], 1);
            }
            for (int i = 0; i < kVS; ++i) {
                pa::mbar_init(&v_full[i], 1);
                pa::mbar_init(&v_free[i], 1);
                pa::mbar_init(&v_conv[i], 4);
            }
            if constexpr (EB == 1) {
                for (int i = 0; i < kKS; ++i) pa::mbar_init(&k_conv[i], 4);
                for (int i = 0; i < 2; ++i) pa::mbar_init(&raw_free[i], 4);
            }
            for (int x = 0; x < 2; ++x) {
                pa::mbar_init(&s_full[x], 1);
                pa::mbar_init(&pv_done[x], 1);
            }
            pa::mbar_init(drain, 1);
            pa::fence_mbar_init();
        }
        if (warp == 0 && !have_tmem) {
            tc::tmem_alloc(tslot, kTmemCols);
            tc::tmem_relinquish();
        }
        // ---- Q tiles: tile X row r = (chunk token i0 + X*QT + r/G, head h0 + r%G)
        if (warp < 8) {
            const int x = warp >> 2, r = threadIdx.x & 127;
            const int i = i0 + x * QT + r / G;
            const uint4* src = reinterpret_cast<const uint4*>(P.q + ((size_t)(q0 + i) * H + h0 + r % G) * D);
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                uint4 v = i < L ? src[c] : make_uint4(0, 0, 0, 0);
                if constexpr (EB == 1) {  // fp16 operands: exact for |q| in fp16's normal range
                    uint32_t* u = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 f = pa::bf16x2_to_float2(u[k]);
                        u[k] = float2_to_f16x2(f.x, f.y);
                    }
                }
                *reinterpret_cast<uint4*>(sm + kQ + x * kQTile + (c >> 3) * 16384 + tc::sw128_offset(r, c & 7)) = v;
            }
        }
        tc::fence_async_smem();
        tc::fence_before_sync();
        __syncthreads();
        tc::fence_after_sync();
        tbase = *tslot;
        have_tmem = true;

        constexpr uint32_t ID_QK = EB == 2 ? tc::idesc_bf16_f32(128, 128, 0, 0) : idesc_f16_f32(128, 128, 0, 0);
        constexpr uint32_t ID_PV = idesc_f16_f32(128, D, 0, 1);

        if (warp == 9) {
            // ------------------------------------------------------- TMA producer
            // K(j) goes to K stage j%2 once both QKs of K(j-2) are done (k_free);
            // V(j) to V stage j%3 once PV_B(j-3), the last reader of V(j-3), is
            // done. K(j) is issued before V(j), and V(j) before K(j+1).
            const int32_t* trow = P.tables + (size_t)s * P.max_blocks;
            struct Ids { int ids = -1, group = -1; };  // block ids of key tiles 4g..4g+3, one per lane
            Ids idk, idv;
            auto issue_tile = [&](Ids& w, const CUtensorMap* map, unsigned char* dst, uint64_t* bar, int j) {
                if ((j >> 2) != w.group) {  // warp-collective
                    w.group = j >> 2;
                    const int blk = w.group * 32 + lane;
                    w.ids = blk < nblk ? trow[blk] : -1;
                }
                // lane l < 8 * NB moves box (block b = l / NB, dims 64 g .. 64 g + 63, g = l % NB);
                // E4M3: NB = 1, a box is a block's 16 x D codes
                constexpr int NB = EB == 2 ? kNH : 1;
                const int b = (lane / NB) & (kBPT - 1), g = lane % NB;
                const int bid = __shfl_sync(kFull, w.ids, (j & 3) * kBPT + b);
                const int blk = j * kBPT + b;
                // blocks between the sinks and the window may be released: zeros too
                bool ok = blk < nblk && (!WIN || keys.seen(P, blk * kBS, blk * kBS + kBS));
                if (ok && (bid < 0 || bid >= P.num_blocks)) {
                    if (lane < NB * kBPT && g == 0) pa::set_error(P.err, PA_DEVERR_BLOCK_ID);
                    ok = false;
                }
                const int y = ok ? (bid * Hk + kvh) * kBS : P.oob_row;  // out of range: zero fill
                if (lane == 0) pa::mbar_arrive_expect_tx(bar, EB == 2 ? kTile : L_::kRawTile);
                __syncwarp();
                if (lane < NB * kBPT)
                    tc::tma_load_2d(dst + (EB == 2 ? g * 16384 + b * 2048 : b * (kBS * D)), map, g * 64, y, bar);
                __syncwarp();
            };
            if constexpr (EB == 2) {
                auto issue_k = [&](int j) {
                    issue_tile(idk, &tmK, sm + kK0 + (j % kKS) * kTile, &k_full[j % kKS], keys.tile(kt0 + j));
                };
                auto issue_v = [&](int j) {
                    issue_tile(idv, &tmV, sm + kV0 + (j % kVS) * kTile, &v_full[j % kVS], keys.tile(kt0 + j));
                };
                int nk = 0, nv = 0;  // loads issued
                bool ok = true;
                for (; nk < kKS && nk < n_kt; ++nk) issue_k(nk);
                for (; nv < kVS && nv < n_kt; ++nv) issue_v(nv);
                while (ok && (nk < n_kt || nv < n_kt)) {
                    if (nk < n_kt && nk <= nv) {  // K(nk) replaces K(nk-2)
                        ok = wait_bar(&k_free[nk % kKS], (uint32_t)(((nk - kKS) / kKS) & 1), P.err, abort_flag);
                        if (!ok) break;
                        issue_k(nk++);
                    } else {  // V(nv) replaces V(nv-3)
                        ok = wait_bar(&v_free[nv % kVS], (uint32_t)(((nv - kVS) / kVS) & 1), P.err, abort_flag);
                        if (!ok) break;
                        issue_v(nv++);
                    }
                }
                // every issued copy has landed before the CTA may exit (bounded; in
                // the normal case the MMA warp has already consumed them all)
                for (int t = (nk > kKS ? nk - kKS : 0); t < nk; ++t)
                    pa::mbar_wait(&k_full[t % kKS], (uint32_t)((t / kKS) & 1), nullptr, 5000000ull);
                for (int t = (nv > kVS ? nv - kVS : 0); t < nv; ++t)
                    pa::mbar_wait(&v_full[t % kVS], (uint32_t)((t / kVS) & 1), nullptr, 5000000ull);
            } else {
                // K(j)'s codes replace K(j-1)'s once those are widened, V's likewise
                bool ok = true;
                int n = 0;  // loads issued: K(0), V(0), K(1), ...
                for (; ok && n < 2 * n_kt; ++n) {
                    const int x = n & 1, j = n >> 1;
                    if (j > 0) ok = wait_bar(&raw_free[x], (uint32_t)((j - 1) & 1), P.err, abort_flag);
                    ok = __all_sync(kFull, ok);
                    if (!ok) break;
                    issue_tile(x ? idv : idk, x ? &tmV : &tmK, sm + L_::kRaw + x * L_::kRawTile, x ? v_full : k_full,
                               keys.tile(kt0 + j));
                }
                // every issued copy has landed before the CTA may exit (bounded, as above)
                for (int x = 0; x < 2; ++x) {
                    const int loads = (n + 1 - x) / 2;
                    if (loads > 0)
                        pa::mbar_wait(x ? v_full : k_full, (uint32_t)((loads - 1) & 1), nullptr, 5000000ull);
                }
            }
        } else if (warp == 8) {
            // ---------------------------------------------------------- MMA issuer
            // One thread issues every MMA. Its waits for data that is normally
            // ready long before (the V tile's conversion, the next K tile) come
            // before its wait for a tile's P, so that P.V and the next Q.K^T of a
            // tile are issued back to back once the softmax hands P over.
            // Matrix descriptors differ only in the start-address field (bits
            // 0-13, byte address / 16); every operand lies inside the shared
            // allocation, so offsets added to the low word never leave the field.
            // The hand-over of each tile's P is a named barrier (ids 1 and 2, the
            // four softmax warps arrive, this warp syncs): every segment has
            // exactly n_kt arrivals of each softmax warpgroup and n_kt syncs here,
            // also after a failed wait, so neither side can be left waiting.
            const uint64_t dq = tc::smem_desc(pa::smem_u32(sm + kQ), 16, 1024);
            const uint64_t dk = tc::smem_desc(pa::smem_u32(sm + kK0), 16, 1024);
            const uint64_t dv = tc::smem_desc(pa::smem_u32(sm + kV0), 16384, 1024);
            auto at = [](uint64_t d, uint32_t off16) {
                return ((uint64_t)(uint32_t)(d >> 32) << 32) | (uint32_t)((uint32_t)d + off16);
            };
            auto issue_qk = [&](int x, int kst) {  // S_x = Q_x K^T, K in stage kst (one thread)
                const uint32_t qo = x * (kQTile >> 4), ko = kst * (kTile >> 4);
                const uint32_t dst = tbase + x * 256;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t o = ((ks >> 2) * 16384 + (ks & 3) * 32) >> 4;
                    tc::mma_bf16(dst, at(dq, qo + o), at(dk, ko + o), ID_QK, ks > 0 ? 1u : 0u);
                }
                if (x == 1) tc::mma_commit(&k_free[kst]);  // the stage's last reader
                tc::mma_commit(&s_full[x]);
            };
            auto issue_pv = [&](int x, int vst, bool first) {  // O_x += P V (fp16), V in stage vst (one thread)
                const uint32_t vo = vst * (kTile >> 4);
                const uint32_t pcol = tbase + x * 256, dst = pcol + 128;
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    tc::mma_bf16_ts(dst, pcol + (ks >> 1) * 32 + (ks & 1) * 8, at(dv, vo + ks * (2048 >> 4)),
                                    ID_PV, (!first || ks > 0) ? 1u : 0u);  // fp16 operands per ID_PV
                if (x == 1) tc::mma_commit(&v_free[vst]);  // the stage's last reader
                tc::mma_commit(&pv_done[x]);
            };
            // The tensor core runs the MMAs of this thread in issue order, so
            // QK_x(j+1) may follow PV_x(j) (which reads P out of S_x's columns)
            // without a wait.
            uint64_t* k_ready = EB == 2 ? k_full : k_conv;
            bool ok = wait_bar(&k_ready[0], 0, P.err, abort_flag);
            ok = __all_sync(kFull, ok);
            if (ok && lane == 0) {
                tc::fence_after_sync();
                issue_qk(0, 0);
                issue_qk(1, 0);
            }
            __syncwarp();
            int kst = 1, kph = 0;  // stage and phase parity of K(j+1)
            int vst = 0, vph = 0;  // stage and phase parity of V(j)
            for (int j = 0; j < n_kt; ++j) {
                const bool more = j + 1 < n_kt;
                if (ok) ok = wait_bar(&v_conv[vst], (uint32_t)vph, P.err, abort_flag);
                if (ok && more) ok = wait_bar(&k_ready[kst], (uint32_t)kph, P.err, abort_flag);
                ok = __all_sync(kFull, ok);
                asm volatile("bar.sync 1, 160;" ::: "memory");  // tile A's P is in tensor memory
                if (ok && lane == 0) {
                    tc::fence_after_sync();
                    issue_pv(0, vst, j == 0);
                    if (more) issue_qk(0, kst);
                }
                __syncwarp();
                asm volatile("bar.sync 2, 160;" ::: "memory");  // tile B's P
                if (ok && lane == 0) {
                    tc::fence_after_sync();
                    issue_pv(1, vst, j == 0);
                    if (more) issue_qk(1, kst);
                }
                __syncwarp();
                if (++vst == kVS) { vst = 0; vph ^= 1; }
                if (++kst == kKS) { kst = 0; kph ^= 1; }
            }
            // drain: every issued MMA has completed before the CTA can release its
            // shared and tensor memory (bounded wait)
            if (lane == 0) tc::mma_commit(drain);
            __syncwarp();
            pa::mbar_wait(drain, 0, nullptr, 10000000ull);
            if (ok && lane == 0) {  // the stages' last frees (never waited for) land before the barriers are reused
                for (int t = max(0, n_kt - kKS); t < n_kt; ++t)
                    pa::mbar_wait(&k_free[t % kKS], (uint32_t)((t / kKS) & 1), nullptr, 10000000ull);
                for (int t = max(0, n_kt - kVS); t < n_kt; ++t)
                    pa::mbar_wait(&v_free[t % kVS], (uint32_t)((t / kVS) & 1), nullptr, 10000000ull);
            }
            __syncwarp();
        } else if (warp >= 10) {
            // ------------------------------------------------------ V converters
            // Thread t of 128 (four warps, one per scheduler) rewrites the 16-byte
            // chunks t, t + 128, ... of the landed tile (consecutive threads,
            // consecutive chunks). A chunk holds
            // 8 consecutive values of one key row: row (chunk % 1024) / 8 of
            // either 64-dim half, wherever the swizzle put the chunk in the row.
            const int t = threadIdx.x - 320;  // 0..127
            if constexpr (EB == 2) {
                const float2 k2 = make_float2(0.00390625f, 0.00390625f);  // 2^-8
                auto cvt = [&](uint32_t u) {  // bf16 pair -> fp16 pair of v * 2^-8
                    const float2 f = __fmul2_rn(make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)), k2);
                    return float2_to_f16x2(f.x, f.y);
                };
                bool ok = true;
                for (int j = 0; j < n_kt && ok; ++j) {
                    ok = wait_bar(&v_full[j % kVS], (uint32_t)((j / kVS) & 1), P.err, abort_flag);
                    ok = __all_sync(kFull, ok);
                    if (!ok) break;
                    const int kb = keys.tile(kt0 + j) * kKT;
                    uint4* vs = reinterpret_cast<uint4*>(sm + kV0 + (j % kVS) * kTile);
                    const int valid = ctx - kb;  // key rows of this tile inside the context (may exceed 128)
                    auto hidden = [&](int row) {  // a row that no query of the pair sees
                        return row >= valid || (WIN && !keys.seen(P, kb + row, kb + row + 1));
                    };
                    auto convert = [&](auto partial) {
    #pragma unroll 4
                        for (int c = 0; c < (int)(kTile / 2048); ++c) {
                            const int e = t + 128 * c;
                            uint4 w = vs[e];
                            if constexpr (decltype(partial)::value)
                                if (hidden((e & 1023) >> 3)) w = make_uint4(0, 0, 0, 0);
                            w.x = cvt(w.x);
                            w.y = cvt(w.y);
                            w.z = cvt(w.z);
                            w.w = cvt(w.w);
                            vs[e] = w;
                        }
                    };
                    if (valid < kKT || (WIN && kb < keys.lo && kb + kKT > P.n_sinks))  // the context or the window ends inside
                        convert(std::true_type{});
                    else convert(std::false_type{});
                    tc::fence_async_smem();  // generic-proxy writes, read next by the tensor core
                    __syncwarp();
                    if (lane == 0) pa::mbar_arrive(&v_conv[j % kVS]);
                }
            } else {
                // E4M3: 16 codes (one 16-byte chunk of a row) become two 16-byte fp16 chunks of
                // the stage. Eight threads that access shared memory together should touch
                // eight different bank groups in the read and in both writes, whose chunks
                // are 2 c and 2 c + 1 of a row (XOR the row, modulo 8). D = 64: two rows of
                // four chunks, read in a run; the rows differ in parity, so their chunks do.
                // D = 128: chunks c .. c + 3 (of one 64-dim half) of rows r and r ^ 5; TMA
                // stored the codes with the same XOR, so the reads differ in bit 2, and the
                // writes in bit 0.
                int row0, c16;
                if constexpr (D == 64) {
                    row0 = t >> 2;
                    c16 = t & 3;
                } else {
                    const int u = t >> 4;  // 0..7: rows {0, 5}, {1, 4}, {2, 7}, {3, 6} and the same plus 8
                    c16 = (t & 3) + ((t >> 1) & 4);
                    row0 = (u & 4) * 2 + ((t & 4) ? (u & 3) ^ 5 : (u & 3));
                }
                constexpr int kStep = D == 64 ? 32 : 16;  // rows per pass
                const uint32_t src0 = row0 * D + (D == 64 ? c16 * 16 : ((c16 ^ (row0 & 7)) << 4));
                const uint32_t half = (c16 >> 2) * 16384, ch = 2 * (c16 & 3);
                const uint32_t dst0 = half + tc::sw128_offset(row0, ch), dst1 = half + tc::sw128_offset(row0, ch + 1);
                auto widen = [&](int x, unsigned char* dst, int kb) {
                    const unsigned char* raw = sm + L_::kRaw + x * L_::kRawTile + src0;
                    const int valid = ctx - kb;
                    auto pass = [&](auto partial) {
#pragma unroll 4
                        for (int c = 0; c < kKT / kStep; ++c) {
                            uint4 w = *reinterpret_cast<const uint4*>(raw + c * kStep * D);
                            // V rows that no query of the pair sees are zero (p = 0 must not meet a NaN)
                            if constexpr (decltype(partial)::value) {
                                const int row = row0 + c * kStep;
                                if (row >= valid || !keys.seen(P, kb + row, kb + row + 1)) w = make_uint4(0, 0, 0, 0);
                            }
                            uint4 lo, hi;
                            e4m3x4_to_f16x4(w.x, lo.x, lo.y);
                            e4m3x4_to_f16x4(w.y, lo.z, lo.w);
                            e4m3x4_to_f16x4(w.z, hi.x, hi.y);
                            e4m3x4_to_f16x4(w.w, hi.z, hi.w);
                            *reinterpret_cast<uint4*>(dst + dst0 + c * kStep * 128) = lo;
                            *reinterpret_cast<uint4*>(dst + dst1 + c * kStep * 128) = hi;
                        }
                    };
                    if (x == 1 && (valid < kKT || (kb < keys.lo && kb + kKT > P.n_sinks))) pass(std::true_type{});
                    else pass(std::false_type{});
                    tc::fence_async_smem();  // generic-proxy writes, read next by the tensor core
                    __syncwarp();
                    if (lane == 0) pa::mbar_arrive(&raw_free[x]);
                };
                bool ok = true;
                for (int j = 0; j < n_kt && ok; ++j) {
                    const int kb = keys.tile(kt0 + j) * kKT, ks = j % kKS, vs = j % kVS;
                    ok = wait_bar(k_full, (uint32_t)(j & 1), P.err, abort_flag);
                    if (ok && j >= kKS) ok = wait_bar(&k_free[ks], (uint32_t)(((j - kKS) / kKS) & 1), P.err, abort_flag);
                    ok = __all_sync(kFull, ok);
                    if (!ok) break;
                    widen(0, sm + kK0 + ks * kTile, kb);
                    if (lane == 0) pa::mbar_arrive(&k_conv[ks]);
                    ok = wait_bar(v_full, (uint32_t)(j & 1), P.err, abort_flag);
                    if (ok && j >= kVS) ok = wait_bar(&v_free[vs], (uint32_t)(((j - kVS) / kVS) & 1), P.err, abort_flag);
                    ok = __all_sync(kFull, ok);
                    if (!ok) break;
                    widen(1, sm + kV0 + vs * kTile, kb);
                    if (lane == 0) pa::mbar_arrive(&v_conv[vs]);
                }
            }
        } else {
            // --------------------------------------- softmax warpgroup of tile x
            // warp w serves TMEM lanes 32*(w%4) .. +31 (rows). After a failed wait
            // (timeout) the warps keep iterating without waiting.
            //
            // One pass over S per key tile, a quarter of 32 columns at a time:
            // p = 2^(s*scale - m) against the row's current reference m, which is
            // an integer (or -inf before the row has seen a key), so every change
            // of m rescales by an exact power of two. m changes only when a
            // quarter's sum of p exceeds 2^15, i.e. before any p could leave the
            // fp16 range (65504), and on a row's first visible quarter (m = -inf
            // gives p = inf): the quarter is then recomputed against
            // m = ceil(max s*scale of the quarter) (its p <= 1), and the P of the
            // tile's earlier quarters, already in tensor memory, is rescaled in
            // place (fp16 times a power of two: exact down to the subnormals).
            const int x = warp >> 2;
            const int r = threadIdx.x & 127;  // matrix row = TMEM lane
            const int i = i0 + x * QT + r / G;
            const int pos = first_pos + i;  // this row's position (padding rows: beyond the chunk)
            const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t tS = tbase + x * 256 + lane_base;
            const uint32_t tO = tS + 128;
            const float sc = P.scale_log2;
            float m_used = -INFINITY, l = 0.f;
            bool ok = true;
            // E4M3: lane l holds the scales of block l % 8 of a key tile; those of
            // tile j + 1 and the block id of tile j + 2 are loaded while tile j is
            // worked on. As in the decode, K's scale multiplies the block's scores
            // and V's enters the exponent, w = 2^(s*scale*k + log2 v - m), and the
            // sum takes w / v.
            auto block_id = [&](int j) {
                const int blk = j < n_kt ? keys.tile(kt0 + j) * kBPT + (lane & (kBPT - 1)) : nblk;
                return blk < nblk && keys.seen(P, blk * kBS, blk * kBS + kBS) ? P.tables[(size_t)s * P.max_blocks + blk] : -1;
            };
            auto scale_of = [&](const float* scales, int bid) {
                return bid >= 0 && bid < P.num_blocks ? scales[(size_t)bid * Hk + kvh] : 1.f;
            };
            float ks_next = 1.f, vs_next = 1.f;
            int bid_next = -1;
            if constexpr (EB == 1) {
                const int bid = block_id(0);
                ks_next = scale_of(P.k_scale, bid);
                vs_next = scale_of(P.v_scale, bid);
                bid_next = block_id(1);
            }
            for (int j = 0; j < n_kt; ++j) {
                float my_k = 0.f, my_e = 0.f, my_inv = 0.f;
                if constexpr (EB == 1) {  // the approximate log2 and reciprocal are off by 2^-22, far below w's rounding
                    const float vs = clamp_scale(vs_next);
                    my_k = clamp_scale(ks_next) * sc;
                    my_e = __log2f(vs);
                    my_inv = __fdividef(1.f, vs);
                    ks_next = scale_of(P.k_scale, bid_next);
                    vs_next = scale_of(P.v_scale, bid_next);
                    bid_next = block_id(j + 2);
                }
                if (ok) ok = wait_bar(&s_full[x], (uint32_t)(j & 1), P.err, abort_flag);
                ok = __all_sync(kFull, ok);
                tc::fence_after_sync();
                const int kb = keys.tile(kt0 + j) * kKT;
                // Keys beyond a row's position are masked. Only the tiles on the
                // diagonal have such keys; a warp takes the masking code only when
                // one of its rows needs it (a warp-uniform branch), so the other
                // tiles run the plain loop.
                const int lim0 = pos - kb;  // keys k > lim0 of the tile are not visible
                // WIN: nor keys k < lim1, sinks (k < sink1) apart
                const int lim1 = P.window >= 0 ? lim0 - P.window : 0, sink1 = P.n_sinks - kb;
                const bool mask_warp = __any_sync(kFull, lim0 < kKT - 1 || (WIN && lim1 > 0 && sink1 < kKT));
                auto is_visible = [&](int k) { return k <= lim0 && (!WIN || k >= lim1 || k < sink1); };
                float2 psum2 = make_float2(0.f, 0.f);  // this tile's sum of p against m_used
                float alpha = 1.f;                     // this tile's rescale of l and O
                const float2 sc2 = make_float2(sc, sc);
                // p of one quarter (raw scores in columns 32q..32q+31) -> fp16 pairs;
                // P of keys 2w, 2w+1 goes to column 32q + w, so a quarter only
                // overwrites columns it has already read.
                // Returns the quarter's sum of p; `add` is what it adds to the row's sum
                // (E4M3: each block's sum over its V scale).
                float qk[2] = {sc, sc}, qe[2] = {0.f, 0.f}, qi[2] = {1.f, 1.f};  // E4M3: the quarter's two blocks
                auto exps = [&](auto masked, const uint32_t (&raw)[32], int qd, uint32_t (&ph)[16], float& add) {
                    float2 qs[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int w = 0; w < 16; ++w) {
                        const int b = EB == 1 ? w >> 3 : 0;
                        const float nm = EB == 1 ? qe[b] - m_used : -m_used;
                        float2 e = __ffma2_rn(make_float2(__uint_as_float(raw[2 * w]), __uint_as_float(raw[2 * w + 1])),
                                              EB == 1 ? make_float2(qk[b], qk[b]) : sc2, make_float2(nm, nm));
                        if constexpr (decltype(masked)::value) {  // masked keys give p = 0 (also for a zero scale)
                            const int k = 32 * qd + 2 * w;
                            if (!is_visible(k)) e.x = -INFINITY;
                            if (!is_visible(k + 1)) e.y = -INFINITY;
                        }
                        e.x = pa::fast_exp2(e.x);
                        e.y = pa::fast_exp2(e.y);
                        qs[b] = __fadd2_rn(qs[b], e);
                        ph[w] = float2_to_f16x2(e.x, e.y);
                    }
                    const float s0 = qs[0].x + qs[0].y;
                    if constexpr (EB == 2) return add = s0;
                    const float s1 = qs[1].x + qs[1].y;
                    add = s0 * qi[0] + s1 * qi[1];
                    return s0 + s1;
                };
                auto sweep = [&](auto masked) {
#pragma unroll 1
                    for (int qd = 0; qd < 4; ++qd) {
                        uint32_t raw[32];
                        tc::tmem_ld32(tS + 32 * qd, raw);
                        tc::tmem_wait_ld();
                        if constexpr (EB == 1) {
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
                                qk[b] = __shfl_sync(kFull, my_k, 2 * qd + b);
                                qe[b] = __shfl_sync(kFull, my_e, 2 * qd + b);
                                qi[b] = __shfl_sync(kFull, my_inv, 2 * qd + b);
                            }
                        }
                        uint32_t ph[16];
                        float add;
                        const float qs = exps(masked, raw, qd, ph, add);
                        const bool big = !(qs <= 32768.f);  // also inf (no reference yet) and NaN
                        if (__any_sync(kFull, big)) {
                            // rare: a new reference for the rows that need one
                            float a = 1.f;
                            if (big) {
                                float qmax = -INFINITY;
#pragma unroll
                                for (int k = 0; k < 32; ++k) {
                                    const bool vis = !decltype(masked)::value || is_visible(32 * qd + k);
                                    const float r = __uint_as_float(raw[k]);
                                    if (vis) qmax = fmaxf(qmax, EB == 1 ? fmaf(r, qk[k >> 4], qe[k >> 4]) : r);
                                }
                                const float mq = ceilf(EB == 1 ? qmax : qmax * sc);
                                if (mq > m_used) {
                                    // 2^(m_used - mq) built from its exponent bits (0 below 2^-126)
                                    const float d = m_used - mq;
                                    a = d < -126.f ? 0.f : __int_as_float(((int)d + 127) << 23);
                                    m_used = mq;
                                    exps(masked, raw, qd, ph, add);
                                }
                            }
                            psum2.x *= a;
                            psum2.y *= a;
                            alpha *= a;
                            if (qd > 0) {  // P of the earlier quarters, in place (warp-collective)
                                tc::tmem_wait_st();
                                // in fp32: the factor itself may lie below fp16's range
                                // (2^-25 would round to 0 as a half) while the products
                                // (P <= 2^15) do not
#pragma unroll 1
                                for (int q2 = 0; q2 < qd; ++q2) {
                                    uint32_t pp[16];
                                    tc::tmem_ld16(tS + 32 * q2, pp);
                                    tc::tmem_wait_ld();
#pragma unroll
                                    for (int w = 0; w < 16; ++w) {
                                        const float2 f = __half22float2(*reinterpret_cast<__half2*>(&pp[w]));
                                        pp[w] = float2_to_f16x2(f.x * a, f.y * a);
                                    }
                                    tc::tmem_st16(tS + 32 * q2, pp);
                                }
                            }
                        }
                        psum2.x += add;
                        tc::tmem_st16(tS + 32 * qd, ph);
                    }
                };
                if (mask_warp) sweep(std::true_type{});
                else sweep(std::false_type{});
                l = l * alpha + (psum2.x + psum2.y);
                // a new reference rescales O_x: PV_x(j-1) must have landed first
                if (j > 0 && __any_sync(kFull, alpha != 1.f)) {
                    if (ok) ok = wait_bar(&pv_done[x], (uint32_t)((j - 1) & 1), P.err, abort_flag);
                    ok = __all_sync(kFull, ok);
                    tc::fence_after_sync();
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t raw[32];
                        tc::tmem_ld32(tO + c * 32, raw);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k) raw[k] = __float_as_uint(__uint_as_float(raw[k]) * alpha);
                        tc::tmem_st32(tO + c * 32, raw);
                    }
                }
                tc::tmem_wait_st();
                tc::fence_before_sync();
                __syncwarp();
                asm volatile("bar.arrive %0, 160;" ::"r"(1 + x) : "memory");  // P handed to the MMA warp
            }
            tc::tmem_wait_st();  // no store may be pending when the columns are released
            if (ok) ok = wait_bar(&pv_done[x], (uint32_t)((n_kt - 1) & 1), P.err, abort_flag);
            ok = __all_sync(kFull, ok);
            if (WIN && ok && slot >= 0) {
                tc::fence_after_sync();
                bool finite = true;
                uint4* dst = reinterpret_cast<uint4*>(P.out + ((size_t)(q0 + i) * H + h0 + r % G) * D);
                join_pieces<D>(
                    P, slot, x, r, warp, lane, m_used, l,
                    [&](int c, float (&v)[32]) {
                        uint32_t raw[32];
                        tc::tmem_ld32(tO + c * 32, raw);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(raw[k]) * (EB == 2 ? 256.f : 1.f);  // undo V's 2^-8
                    },
                    [&](int c, const float (&v)[32]) {
                        if (i >= L) return;
#pragma unroll
                        for (int k = 0; k < 32; ++k) finite &= fabsf(v[k]) < INFINITY;
#pragma unroll
                        for (int k = 0; k < 32; k += 8)
                            dst[(c * 32 + k) / 8] =
                                make_uint4(pa::float2_to_bf16x2(v[k], v[k + 1]), pa::float2_to_bf16x2(v[k + 2], v[k + 3]),
                                           pa::float2_to_bf16x2(v[k + 4], v[k + 5]), pa::float2_to_bf16x2(v[k + 6], v[k + 7]));
                    });
                if (!finite) pa::set_error(P.err, PA_DEVERR_RANGE);
            } else if (ok && !direct) {
                // a piece: keep O, m and l for the merge
                tc::fence_after_sync();
                float* dst = part_base + ((size_t)x * 128 + r) * kPartStride;
                bool finite = true;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t raw[32];
                    tc::tmem_ld32(tO + c * 32, raw);
                    tc::tmem_wait_ld();
                    if (i < L) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            if constexpr (EB == 2) raw[k] = __float_as_uint(__uint_as_float(raw[k]) * 256.f);  // undo V's 2^-8
                            finite &= (raw[k] & 0x7f800000u) != 0x7f800000u;
                        }
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            *reinterpret_cast<float4*>(dst + c * 32 + k) =
                                make_float4(__uint_as_float(raw[k]), __uint_as_float(raw[k + 1]),
                                            __uint_as_float(raw[k + 2]), __uint_as_float(raw[k + 3]));
                    }
                }
                if (!finite) pa::set_error(P.err, PA_DEVERR_RANGE);
                if (i < L) *reinterpret_cast<float2*>(dst + kPartML) = make_float2(m_used, l);
            } else if (ok) {
                tc::fence_after_sync();
                const float inv = (EB == 2 ? 256.f : 1.f) / l;  // bf16: with V's 2^-8 undone
                uint4* dst = reinterpret_cast<uint4*>(P.out + ((size_t)(q0 + i) * H + h0 + r % G) * D);
                bool finite = true;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t raw[32];
                    tc::tmem_ld32(tO + c * 32, raw);
                    tc::tmem_wait_ld();
                    if (i < L) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) finite &= (raw[k] & 0x7f800000u) != 0x7f800000u;
#pragma unroll
                        for (int k = 0; k < 32; k += 8) {
                            uint4 w;
                            w.x = pa::float2_to_bf16x2(__uint_as_float(raw[k]) * inv, __uint_as_float(raw[k + 1]) * inv);
                            w.y = pa::float2_to_bf16x2(__uint_as_float(raw[k + 2]) * inv, __uint_as_float(raw[k + 3]) * inv);
                            w.z = pa::float2_to_bf16x2(__uint_as_float(raw[k + 4]) * inv, __uint_as_float(raw[k + 5]) * inv);
                            w.w = pa::float2_to_bf16x2(__uint_as_float(raw[k + 6]) * inv, __uint_as_float(raw[k + 7]) * inv);
                            dst[(c * 32 + k) / 8] = w;
                        }
                    }
                }
                if (!finite) pa::set_error(P.err, PA_DEVERR_RANGE);
            }
        }
        tc::fence_before_sync();
        __syncthreads();  // end of the segment: every role is done with smem, TMEM and the barriers
        ++n_run;
    }  // segments
    if (have_tmem && warp == 0) tc::tmem_dealloc(tbase, kTmemCols);
}

// Key tiles of item it = (sequence * n_kv_heads + kv head) * n_qp + pair:
// 0 if the pair has no rows. A chunk that is not in the cache (ctx < L) has
// none either, and flags the device error once per sequence.
template <int G>
__device__ int item_tiles(const PrefillParams& P, int it) {
    constexpr int QT = kRows / G;
    const int per_seq = P.n_kv_heads * P.n_qp;
    const int s = it / per_seq, qp = it % P.n_qp;
    const int q0 = P.qsl[s], L = P.qsl[s + 1] - q0, i0 = qp * 2 * QT;
    if (i0 >= L) return 0;
    const int ctx = P.ctx[s];
    if (ctx < L) {
        if (it % per_seq == 0) pa::set_error(P.err, PA_DEVERR_CONTEXT);
        return 0;
    }
    return KeyTiles(P, ctx - L + i0, ctx - L + min(i0 + 2 * QT, L) - 1).n;
}

// Balanced mode: the work list. One block of 1024 threads, each a run of
// consecutive items. With P non-empty items and C CTAs (one per SM), the
// first P - R items run whole (full waves, in item order so that the pairs of
// one KV head run side by side and share their K/V tiles in L2); the last
// R = P mod C items would fill only part of a wave, so each is cut into S
// equal key ranges, S (1..8, R*S <= 4C) minimising ceil(R*S/C)/S + 0.03 S
// (the wave fraction the tail takes plus a per-piece cost); its pieces are
// listed piece-major, so the pieces running together again share key ranges.
template <int G>
__global__ void __launch_bounds__(1024) pa_prefill_plan_kernel(const PrefillParams P) {
    __shared__ int wsum[32];
    __shared__ int sh[3];  // P, R, S
    const int n = P.n_items, t = threadIdx.x, lane = t & 31, wid = t >> 5;
    const int per = (n + 1023) / 1024;
    const int b0 = min(n, t * per), b1 = min(n, b0 + per);
    int mine = 0;
    for (int it = b0; it < b1; ++it) mine += item_tiles<G>(P, it) > 0;
    int incl = mine;  // inclusive count within the warp
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) wsum[wid] = incl;
    __syncthreads();
    if (wid == 0) {
        int v = wsum[lane];
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, v, o);
            if (lane >= o) v += y;
        }
        wsum[lane] = v;  // inclusive over warps
    }
    __syncthreads();
    if (t == 0) {
        const int np = wsum[31], C = P.n_cta;
        int R = np % C, S = 1;
        float best = 2.f;
        for (int c = 1; c <= 8 && R * c <= 4 * C; ++c) {
            const float cost = (float)((R * c + C - 1) / C) / c + 0.03f * c;
            if (cost < best) {
                best = cost;
                S = c;
            }
        }
        if (S == 1) R = 0;  // no cut: the tail runs whole
        sh[0] = np;
        sh[1] = R;
        sh[2] = S;
        P.sched[0] = 0;
        P.sched[1] = np - R + R * S;
        P.sched[2] = S;
        P.sched[3] = R;
    }
    __syncthreads();
    const int np = sh[0], R = sh[1], S = sh[2], whole = np - R;
    int rank = incl - mine + (wid > 0 ? wsum[wid - 1] : 0);
    for (int it = b0; it < b1; ++it) {
        const int nk = item_tiles<G>(P, it);
        if (nk <= 0) continue;
        if (rank < whole) {
            P.work[rank] = make_int4(it, 0, nk, -1);
        } else {
            const int ti = rank - whole;
            for (int sp = 0; sp < S; ++sp) {
                int a, b;
                piece_range(nk, sp, S, a, b);
                P.work[whole + sp * R + ti] = make_int4(it, a, b, ti * S + sp);
            }
        }
        ++rank;
    }
}

// Even mode (windowed and E4M3 instantiations): the work list. An item costs
// its key tiles plus kStart, what starting and finishing a segment takes in
// units of a tile (Q, the pipeline's fill, the epilogue: about 10 us against
// 1.9). The costs of all non-empty items, in item order, are cut into C runs of
// equal length, C the CTAs (fewer when a run would be shorter than kStart + 4),
// so that all CTAs finish together: each has at most one piece of an item begun
// by the CTA before, whole items, and one piece of an item that the next CTA
// goes on with. (A window makes the items equally long and few waves deep: 256
// items of 35 tiles on 152 CTAs take 4 segments on the busiest CTA with whole
// waves and cut tails, 2 or 3 here, and no CTA idles.) A cut that would leave
// fewer than kLeast tiles on one side moves to that end of the item. When the
// items are at most the CTAs and none is much longer than the mean, each runs
// whole, which saves joining pieces.
// Item r (its rank among the non-empty ones) and CTA c share at most one
// entry, number r + c; a CTA's entries are consecutive. P.work[n_items + n_cta
// + c] = (first entry, end entry, the CTA ca that begins the item cut between
// CTA c - 1 and c, its pieces or 0). Piece k of that item: slot 2 ca + 1 for
// k = 0, else 2 (ca + k). Behind that table, 8 counters for each CTA (see
// join_pieces), zeroed here.
constexpr int kStart = 5, kLeast = 3;
template <int G>
__global__ void __launch_bounds__(1024) pa_prefill_plan_even_kernel(const PrefillParams P) {
    __shared__ long long wsum[32];
    __shared__ int wcnt[32], wmax[32];
    pa::launch_dependents();     // the prefill kernel may be scheduled
    pa::grid_dependency_wait();  // the lengths are written
    const int n = P.n_items, t = threadIdx.x, lane = t & 31, wid = t >> 5;
    const int per = (n + 1023) / 1024;
    const int b0 = (int)min((long long)n, (long long)t * per), b1 = min(n, b0 + per);
    int4* cta = P.work + n + P.n_cta;
    for (int c = t; c < P.n_cta; c += 1024) {
        cta[c] = make_int4(0x7fffffff, 0, -1, 0);
        cta[P.n_cta + 2 * c] = cta[P.n_cta + 2 * c + 1] = make_int4(0, 0, 0, 0);
    }
    long long mine = 0;
    int cnt = 0, most = 0;
    for (int it = b0; it < b1; ++it) {
        const int nk = item_tiles<G>(P, it);
        mine += nk > 0 ? nk + kStart : 0;
        cnt += nk > 0;
        most = max(most, nk);
    }
    long long incl = mine;  // inclusive sums within the warp
    int icnt = cnt;
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(kFull, incl, o);
        const int u = __shfl_up_sync(kFull, icnt, o);
        if (lane >= o) {
            incl += v;
            icnt += u;
        }
        most = max(most, __shfl_xor_sync(kFull, most, o));
    }
    if (lane == 31) {
        wsum[wid] = incl;
        wcnt[wid] = icnt;
        wmax[wid] = most;
    }
    __syncthreads();
    if (wid == 0) {
        long long v = wsum[lane];
        int u = wcnt[lane], m = wmax[lane];
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(kFull, v, o);
            const int z = __shfl_up_sync(kFull, u, o);
            if (lane >= o) {
                v += y;
                u += z;
            }
            m = max(m, __shfl_xor_sync(kFull, m, o));
        }
        wsum[lane] = v;  // inclusive over warps
        wcnt[lane] = u;
        wmax[lane] = m;
    }
    __syncthreads();
    const long long T = wsum[31];
    const int np = wcnt[31];
    const bool whole = np <= P.n_cta && wmax[0] <= T / P.n_cta + 2 * kStart;
    const long long C = max(1LL, min((long long)P.n_cta, T / (kStart + 4)));
    long long off = incl - mine + (wid > 0 ? wsum[wid - 1] : 0);
    int r = icnt - cnt + (wid > 0 ? wcnt[wid - 1] : 0);
    for (int it = b0; it < b1; ++it) {
        const int nk = item_tiles<G>(P, it);
        if (nk <= 0) continue;
        if (whole) {
            P.work[r] = make_int4(it, 0, nk, -1);
            cta[r] = make_int4(r, r + 1, -1, 0);
        } else {
            // run c: costs [c T / C, (c + 1) T / C); the item's costs are [off, off + nk + kStart)
            const int c0 = (int)(((off + 1) * C - 1) / T), c1 = (int)(((off + nk + kStart) * C - 1) / T);
            auto cut = [&](int c) {  // the item's tile at which run c begins
                if (c <= c0) return 0;
                if (c > c1) return nk;
                const int x = (int)(c * T / C - off) - kStart;
                return x < kLeast ? 0 : x > nk - kLeast ? nk : x;
            };
            int ca = c0, cb = c1;  // the CTAs that get tiles
            while (cut(ca + 1) == 0) ++ca;
            while (cut(cb) == nk) --cb;
            for (int c = ca; c <= cb; ++c) {
                P.work[r + c] = make_int4(it, cut(c), cut(c + 1), ca == cb ? -1 : c == ca ? 2 * c + 1 : 2 * c);
                atomicMin(&cta[c].x, r + c);
                atomicMax(&cta[c].y, r + c + 1);
            }
            for (int c = ca + 1; c <= cb; ++c) {
                cta[c].z = ca;
                cta[c].w = cb - ca + 1;
            }
        }
        off += nk + kStart;
        ++r;
    }
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
    if (i < 0 || i >= L || ctx < L) return;
    const int qp = i / (2 * QT), x = (i % (2 * QT)) / QT, r = (i % QT) * G + h % G, kvh = h / G;
    const int i0 = qp * 2 * QT;
    const int n_kt_all = KeyTiles(P, ctx - L + i0, ctx - L + min(i0 + 2 * QT, L) - 1).n;
    const size_t item = ((size_t)s * Hk + kvh) * n_qp + qp;
    merge_row<D>(P.splits, n_kt_all,
                 [&](int k) { return P.part + (((item * P.splits + k) * 2 + x) * 128 + r) * kPartStride; }, lane,
                 P.out + ((size_t)t * H + h) * D);
}

// Balanced mode: one warp per (row, head) of the cut pairs, warp w = 256 *
// (cut pair) + 128 * (query tile) + (tile row); the cut pairs are the
// piece-0 entries of the work list's tail.
template <int G, int D>
__global__ void __launch_bounds__(128) pa_prefill_merge_cut_kernel(const PrefillParams P) {
    constexpr int QT = kRows / G;
    pa::grid_dependency_wait();  // every piece's partial is written
    const int w = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int S = P.sched[2], R = P.sched[3];
    const int t = w >> 8, x = (w >> 7) & 1, r = w & 127;
    if (t >= R) return;
    const int item = P.work[P.sched[1] - R * S + t].x;
    const int Hk = P.n_kv_heads;
    const int s = item / (Hk * P.n_qp), kvh = (item / P.n_qp) % Hk, qp = item % P.n_qp;
    const int q0 = P.qsl[s], L = P.qsl[s + 1] - q0, ctx = P.ctx[s];
    const int i0 = qp * 2 * QT, i = i0 + x * QT + r / G;
    if (i >= L) return;
    const int n_kt_all = KeyTiles(P, ctx - L + i0, ctx - L + min(i0 + 2 * QT, L) - 1).n;
    const size_t slot0 = (size_t)t * S;
    merge_row<D>(S, n_kt_all, [&](int k) { return P.part + (((slot0 + k) * 2 + x) * 128 + r) * kPartStride; },
                 lane, P.out + ((size_t)(q0 + i) * P.n_heads + kvh * G + r % G) * D);
}

template <int G, int D, int EB, bool WIN>
int launch_prefill(const PrefillParams& Pp, const CUtensorMap& tk, const CUtensorMap& tv, int n_seqs,
                   int max_chunk_len, int n_rows, cudaStream_t stream) {
    auto kern = pa_prefill_tc_kernel<G, D, EB, WIN>;
    constexpr uint32_t kSmemBytes = PfLay<D, EB>::kSmem;
    static bool attr_done[64] = {false};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_done[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes) !=
            cudaSuccess)
            return PA_ERR_CUDA;
        attr_done[dev] = true;
    }
    constexpr int QT = kRows / G;
    const int n_qp = (max_chunk_len + 2 * QT - 1) / (2 * QT);
    if (WIN && Pp.work) {  // even mode: plan, then one CTA per SM, launched ahead of the plan's end
        const int st = pa_launch_pdl(pa_prefill_plan_even_kernel<G>, dim3(1), dim3(1024), 0, stream, Pp);
        if (st != PA_OK) return st;
        return pa_launch_pdl(kern, dim3((unsigned)Pp.n_cta), dim3(kThreads), kSmemBytes, stream, Pp, tk, tv);
    }
    if (Pp.work) {  // balanced mode: plan, then one CTA per SM taking work-list entries
        pa_prefill_plan_kernel<G><<<1, 1024, 0, stream>>>(Pp);
        kern<<<Pp.n_cta, kThreads, kSmemBytes, stream>>>(Pp, tk, tv);
    } else {
        dim3 grid(n_qp * Pp.splits, Pp.n_kv_heads, n_seqs);
        kern<<<grid, kThreads, kSmemBytes, stream>>>(Pp, tk, tv);
    }
    if (cudaGetLastError() != cudaSuccess) return PA_ERR_CUDA;
    if (Pp.work)  // the cut pairs (fewer than one per CTA): 256 rows each
        return pa_launch_pdl(pa_prefill_merge_cut_kernel<G, D>, dim3((unsigned)Pp.n_cta * 64), dim3(128), 0, stream,
                             Pp);
    if (Pp.splits <= 1) return PA_OK;
    // rows of all chunks: the merge finds each row's sequence in q_start_loc
    const long long warps = (long long)n_rows * Pp.n_heads;
    return pa_launch_pdl(pa_prefill_merge_kernel<G, D>, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0, stream, Pp,
                         n_seqs, n_rows, n_qp);
}

template <int D, int EB, bool WIN>
int dispatch_prefill(int G, const PrefillParams& P, const CUtensorMap& tk, const CUtensorMap& tv, int n_seqs,
                     int max_chunk_len, int n_rows, cudaStream_t stream) {
    switch (G) {
        case 1: return launch_prefill<1, D, EB, WIN>(P, tk, tv, n_seqs, max_chunk_len, n_rows, stream);
        case 2: return launch_prefill<2, D, EB, WIN>(P, tk, tv, n_seqs, max_chunk_len, n_rows, stream);
        case 4: return launch_prefill<4, D, EB, WIN>(P, tk, tv, n_seqs, max_chunk_len, n_rows, stream);
        default: return launch_prefill<8, D, EB, WIN>(P, tk, tv, n_seqs, max_chunk_len, n_rows, stream);
    }
}

}  // namespace
