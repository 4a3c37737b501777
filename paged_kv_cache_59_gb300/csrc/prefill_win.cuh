// Chunked causal prefill under a sliding window with sinks (bf16 cache), and over
// an E4M3 cache with a scale per (block, KV head), on the tcgen05 tensor cores.
//
//     out[i][h] = sum_t softmax_t(scale * q[i][h] . K[t]) V[t]
// over t <= p with t >= p - window or t < n_sinks, p the row's position (window
// -1: t <= p). The arithmetic of a key tile is that of prefill.cu: query tiles of
// 128 rows (tokens x the group's heads), two of them (A and B) per CTA, key
// tiles of 128, S and P in tensor memory, fp32 softmax against an integer
// reference, fp16 P; see there for its design and its bounds. What differs:
//
// Work. Only the key tiles that a row of the pair sees are walked (KeyTiles). A
// window makes items short - a few tens of tiles - so starting one is what
// costs. (a) The items' tiles are cut evenly over the SMs, pieces joined by the
// last of them (see below). (b) The roles run over a CTA's segments each at its
// own pace, without a block-wide barrier between segments: rings and barrier
// phases go on from one segment to the next. While the softmax warps work on a
// segment's last tile and write its output, the producer loads the next
// segment's K and V, and the converter warps its Q as soon as the last Q.K^T has
// read the old one; the tensor core then starts on it at once.
//
// Measured (32/8 heads of 128, 19 pairs a KV head, so one item a CTA): 1.75 us a
// key tile in bf16 (1,460 TFLOP/s of its two tiles' four products over 152 SMs,
// 0.75 of a cuBLAS burst) and 1.80 with E4M3, and 11 us a call beside the tiles:
// the plan and launches 6, the first tile's loads, softmax and the epilogue 5.
// What bounds the tile loop is a chain: S and P share 128 of the 512 tensor-
// memory columns for each of the two query tiles, so a tile's P.V and next
// Q.K^T (1,350 cycles, the shared memory's bandwidth being shared with V's
// conversion) and its softmax (1,650 to 1,900) follow each other. Without the
// exponentials a tile takes 1.56 us, without V's conversion 1.61, without both
// 1.47. Converters that load V (E4M3: K and V) themselves, a tile ahead in
// registers instead of by TMA, took 1.82, and 270 us instead of 201 for four
// chunks whose cache comes from HBM.
// Reshaped scores (MOD, pa_prefill_score_mod): the same kernel, each score capped by a tanh, biased by
// its key's distance, or both, before the exponential, and prefixes that lift the causal limit. 2,048
// rows, window 4,096, scores of a spread of 6, on one cache again and again: 177 us with a cap of 50, 152 with
// biases (caches in turn 180 and 155).
// 2,048 rows, window 4,096 + 4 sinks (256 items of 33 tiles on 152 SMs): 129.1 us on
// one cache, 1,066 TFLOP/s of visible pairs, 132.6 over three in turn; 179 us with
// whole waves, cut tails and a block-wide barrier between segments.
//
// bf16 V (EB = 2) is staged in fp16, whose range begins 2^-24: as v 2^-8, as in
// prefill.cu, elements below 2^-6 lose bits, and a layer whose values are all of
// magnitude 2^-12 would keep 2 or 3 of 8. So the rows of every 32 keys (a quarter
// of the softmax) are staged as v 2^(-8 - e), e = min(0, exponent of their largest
// magnitude), -64 at least: an element is off by at most 2^-17 of that magnitude,
// 1/32 of a weight's rounding. As with a block's scale below, e enters the
// exponent, w = 2^(s*scale + e - m), and the sum takes w 2^-e. Where e = 0 the bits
// are those of prefill.cu. Looking for the magnitude costs 0.5 to 1% where the
// first rows hold an element of 2 or more, which settles it, else 4 (2,048 rows,
// window 4,096 + 4 sinks: 128.5 us without it, 129.1 and 132.6 with).
//
// E4M3 (EB = 1). The codes of a K and of a V tile (half the bytes) land in a
// buffer each, and the converter warps widen both to fp16, exactly; Q is
// converted to fp16 once. Scales never touch the operands: a block's K scale
// multiplies its scores, and V's enters the exponent,
//     w = 2^(s*scale*k + log2 v - m),  out = sum w code / sum w / v,
// as in the decode, so P.V runs on the codes with one reference for loud and
// quiet blocks alike.
#pragma once

#include "prefill_tc.cuh"

namespace {

// 8 softmax warps, MMA warp (8), producer (9; bf16: of K), 4 converter warps
// (10..13), bf16: V producer (14); four warps a scheduler at most, so 128
// registers each.
template <int EB>
constexpr int kWinThreads = EB == 2 ? 480 : 448;

constexpr int kLeastExp = -64;  // of 32 keys' V rows (all zero, or too small for every purpose)

// Shared memory, as PfLay: EB = bytes per cached element. With an E4M3 cache the
// codes of a K and of a V tile land in a buffer of their own (128 rows of D
// bytes), and the stages hold them widened to fp16.
template <int D, int EB>
struct WinLay {
    static constexpr int kKS = 2;                     // K tile stages
    static constexpr int kVS = EB == 2 ? 3 : 2;  // V tile stages
    static constexpr int kHalves = D / 64;               // 64-dim halves of a row
    static constexpr uint32_t kTile = kKT * D * 2;       // K or V tile bytes
    static constexpr uint32_t kQTile = kRows * D * 2;    // Q tile bytes
    static constexpr uint32_t kQ = 0;                    // Q_A, Q_B
    static constexpr uint32_t kK0 = 2 * kQTile;          // K stages
    static constexpr uint32_t kV0 = kK0 + kKS * kTile;   // V stages
    static constexpr uint32_t kRaw = kV0 + kVS * kTile;  // E4M3: codes of a K tile, of a V tile
    static constexpr uint32_t kRawTile = kKT * D;
    static constexpr uint32_t kBars = kRaw + (EB == 1 ? 2 * kRawTile : 0);  // mbarriers
    static constexpr uint32_t kMisc = kBars + 256;       // tmem slot, abort flag
    static constexpr uint32_t kVExp = kMisc + 64;        // bf16: (e, 2^-e) of each V stage's 4 x 32 keys
    static constexpr uint32_t kSmem = kVExp + (EB == 2 ? kVS * 4 * 8 : 0);
    static_assert(kSmem <= 227 * 1024, "shared memory budget");
};

// One piece of work of a CTA: key tiles [kt0, kt0 + n_kt) of a query-tile pair,
// numbered as in KeyTiles.
struct Segment {
    int s, kvh, qp;           // sequence, KV head, pair
    int q0, L, ctx;           // first row, rows, context of the sequence
    int kt0, n_kt;
    int slot;                 // even mode: this piece's slot, or -1 for a whole item
};

// The segments of this CTA, the same for every thread. Even mode: its run of the
// work list. Per-pair mode (P.work null): the one piece that the grid position
// names.
template <int G>
struct Segments {
    const PrefillParams& P;
    int at, end;
    __device__ __forceinline__ explicit Segments(const PrefillParams& P_) : P(P_), at(0), end(1) {
        if (P.work) {
            const int4 c = P.work[P.n_items + P.n_cta + blockIdx.x];
            at = c.x;
            end = c.y;
        }
    }
    // The next segment with rows and tiles; false at the end.
    __device__ __forceinline__ bool next(Segment& g) {
        while (at < end) {
            const int4 e = P.work ? P.work[at]
                                  : make_int4(((int)blockIdx.z * P.n_kv_heads + (int)blockIdx.y) * P.n_qp +
                                                  (int)blockIdx.x / P.splits, 0, 0, -1);
            ++at;
            g.s = e.x / (P.n_kv_heads * P.n_qp);
            g.kvh = (e.x / P.n_qp) % P.n_kv_heads;
            g.qp = e.x % P.n_qp;
            g.q0 = P.qsl[g.s];
            g.L = P.qsl[g.s + 1] - g.q0;
            g.ctx = P.ctx[g.s];
            g.kt0 = e.y;
            g.slot = e.w;
            int kt1 = e.z;
            if (!P.work) {
                constexpr int QT = kRows / G;
                if (g.qp * 2 * QT >= g.L) continue;
                if (left_out<G>(P, g.L, g.ctx)) {
                    if (threadIdx.x == 0) pa::set_error(P.err, PA_DEVERR_CONTEXT);
                    continue;
                }
                piece_range(keys(g).n, (int)blockIdx.x % P.splits, P.splits, g.kt0, kt1);
            }
            g.n_kt = kt1 - g.kt0;
            if (g.n_kt > 0) return true;
        }
        return false;
    }
    __device__ __forceinline__ KeyTiles keys(const Segment& g) const {
        constexpr int QT = kRows / G;
        const int i0 = g.qp * 2 * QT, first = g.ctx - g.L;
        return KeyTiles(P, first + i0, max(first + min(i0 + 2 * QT, g.L), prefix_of(P, g.s, g.ctx)) - 1);
    }
};

// mbarriers (all phases run on from segment to segment): tile J counts the
// CTA's key tiles over all its segments.
//   k_full, v_full [stage]  bf16: the K (V) tile landed; E4M3: [0] its codes landed
//   raw_free [2]            E4M3: K's, V's codes are read (4 converter warps)
//   k_conv, v_conv [stage]  the converted tile is in its stage (4 converter warps)
//   v_exp [stage]           bf16: the tile's exponents of V are in their place (4 converter warps)
//   k_free, v_free [stage]  the last MMA that reads the stage is done
//   q_full, q_free          the segment's Q is in place (4 converter warps), its last Q.K^T done
// A wait for a phase passes at once when the barrier is two phases behind, so a
// role waits for every phase of a barrier, or for one that other waits order.
//   s_full [x], pv_done [x] S_x of tile J, O_x including tile J
template <int D, int EB>
struct Bars {
    static constexpr int kKS = WinLay<D, EB>::kKS, kVS = WinLay<D, EB>::kVS;
    uint64_t* b;
    static constexpr int kCount = 3 * kKS + 3 * kVS + 2 + 1 + 4 + 1 + 1 + kVS;
    static_assert(kCount * 8 <= 256, "barrier area");
    __device__ __forceinline__ uint64_t* k_full(int i) const { return b + i; }
    __device__ __forceinline__ uint64_t* k_conv(int i) const { return b + kKS + i; }
    __device__ __forceinline__ uint64_t* k_free(int i) const { return b + 2 * kKS + i; }
    __device__ __forceinline__ uint64_t* v_full(int i) const { return b + 3 * kKS + i; }
    __device__ __forceinline__ uint64_t* v_conv(int i) const { return b + 3 * kKS + kVS + i; }
    __device__ __forceinline__ uint64_t* v_free(int i) const { return b + 3 * kKS + 2 * kVS + i; }
    __device__ __forceinline__ uint64_t* raw_free(int i) const { return b + 3 * kKS + 3 * kVS + i; }
    __device__ __forceinline__ uint64_t* q_full() const { return b + 3 * kKS + 3 * kVS + 2; }
    __device__ __forceinline__ uint64_t* s_full(int x) const { return b + 3 * kKS + 3 * kVS + 3 + x; }
    __device__ __forceinline__ uint64_t* pv_done(int x) const { return b + 3 * kKS + 3 * kVS + 5 + x; }
    __device__ __forceinline__ uint64_t* drain() const { return b + 3 * kKS + 3 * kVS + 7; }
    __device__ __forceinline__ uint64_t* q_free() const { return b + 3 * kKS + 3 * kVS + 8; }
    __device__ __forceinline__ uint64_t* v_exp(int i) const { return b + 3 * kKS + 3 * kVS + 9 + i; }
};

// Whether no query of the pair sees the position (its V row is zeroed), and
// whether tile j may have such a row.
__device__ __forceinline__ bool hidden_row(const PrefillParams& P, const KeyTiles& keys, int ctx, int pos) {
    return pos >= ctx || (pos < keys.lo && pos >= P.n_sinks);
}
__device__ __forceinline__ bool hides_rows(const KeyTiles& keys, int ctx, int j) {
    return keys.position(j, kKT - 1) >= ctx || (keys.lo > 0 && j * kBPT <= keys.n_sink);
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
// (m, l). `own(c, v)` gives columns 32 c .. 32 c + 31 of this row's O, `put(c, v)`
// takes the joined ones, normalised (both warp-collective), and put_row(rr, v)
// columns 4 lane .. of the warp's row rr. `valid`: the row is in the chunk (the
// valid rows of a warp are its first).
__device__ __forceinline__ float* slot_part(const PrefillParams& P, int slot, int x) {
    return P.part + ((size_t)slot * 2 + x) * 128 * kPartStride;
}
template <int D, typename Own, typename Put, typename PutRow>
__device__ __forceinline__ void join_pieces(const PrefillParams& P, int slot, int x, int r, int warp, int lane, bool valid,
                                            float m, float l, Own own, Put put, PutRow put_row) {
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
    auto piece_part = [&](int k) { return slot_part(P, k == 0 ? 2 * ca + 1 : 2 * (ca + k), x); };
    // A few rows in many pieces (a chunk of a token or two behind a long context) are joined row by
    // row, the lanes along the columns and eight pieces' loads in flight, when that takes fewer
    // rounds of memory latency than 32 columns of a piece at a time.
    const int rows = __popc(__ballot_sync(kFull, valid));
    const bool by_row = rows * ((n + 7) / 8) < D / 32 * (n - 1);
    // only the item's first piece, its CTA's last segment, can expect the others to be complete
    bool last = me == 0 && !by_row && __all_sync(kFull, counted() == n - 1);
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
    if (by_row) {
        for (int rr = 0; rr < rows; ++rr) {
            const int row = (r & ~31) + rr;
            auto row_ml = [&](int k) { return __ldcg(reinterpret_cast<const float2*>(piece_part(k) + 128 * D) + row); };
            float M = -INFINITY, sum = 0.f;
            for (int k = lane; k < n; k += 32) M = fmaxf(M, row_ml(k).x);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
            for (int k = lane; k < n; k += 32) {
                const float2 p = row_ml(k);
                sum += p.x == -INFINITY ? 0.f : p.y * pa::fast_exp2(p.x - M);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k0 = 0; k0 < n; k0 += 8) {
                float4 v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    v[u] = k0 + u < n && lane < D / 4
                               ? __ldcg(reinterpret_cast<const float4*>(piece_part(k0 + u)) + lane * 128 + row)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
                const int k = k0 + (lane & 7);
                const float m_k = k < n ? row_ml(k).x : -INFINITY, f = m_k == -INFINITY ? 0.f : pa::fast_exp2(m_k - M);
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float fu = __shfl_sync(kFull, f, u);
                    acc.x += v[u].x * fu;
                    acc.y += v[u].y * fu;
                    acc.z += v[u].z * fu;
                    acc.w += v[u].w * fu;
                }
            }
            const float inv = 1.f / sum;
            put_row(rr, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
        }
        return;
    }
    float2 ml01[2];  // (m, l) of the first two pieces (nearly always all of them)
    auto load_ml = [&](int k) {
        return k == me ? make_float2(m, l) : __ldcg(reinterpret_cast<const float2*>(piece_part(k) + 128 * D) + r);
    };
    ml01[0] = load_ml(0);
    ml01[1] = load_ml(1);
    auto ml = [&](int k) { return k == 0 ? ml01[0] : k == 1 ? ml01[1] : load_ml(k); };
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
            float v[32];
            if (k == me) {  // warp-uniform
                own(q, v);
            } else {
                const float4* src = reinterpret_cast<const float4*>(piece_part(k));
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float4 w = __ldcg(src + (8 * q + u) * 128 + r);
                    v[4 * u] = w.x;
                    v[4 * u + 1] = w.y;
                    v[4 * u + 2] = w.z;
                    v[4 * u + 3] = w.w;
                }
            }
            const float f = factor(ml(k).x);
#pragma unroll
            for (int u = 0; u < 32; ++u) acc[u] += v[u] * f;
        }
#pragma unroll
        for (int u = 0; u < 32; ++u) acc[u] *= inv;
        put(q, acc);
    }
}

// Kernels of reshaped scores (pa_prefill_score_mod), one for each way to reshape them, as the
// instructions of the others cost even where they are not taken (2,048 rows under a window of
// 4,096, 32 heads: a bias 176 us in a kernel for all, 144 in its own): a cap alone, a bias by
// distance or none (a prefix over plain scores), and both, or a cap above 128.
enum { kPlain, kCap, kBias, kCapBias };

// The largest |q.k * k| of a quarter's products; k: the factors of its two blocks.
__device__ __forceinline__ float largest_of(const uint32_t (&raw)[32], const float (&k)[2]) {
    float most[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 32; i += 2)
        asm("max.abs.f32 %0, %0, %1, %2;" : "+f"(most[i >> 4]) : "f"(__uint_as_float(raw[i])), "f"(__uint_as_float(raw[i + 1])));
    return fmaxf(most[0] * fabsf(k[0]), most[1] * fabsf(k[1]));
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 pair_of(const uint32_t (&raw)[32], int w) {
    return make_float2(__uint_as_float(raw[2 * w]), __uint_as_float(raw[2 * w + 1]));
}
__device__ __forceinline__ void put_pair(uint32_t (&raw)[32], int w, float2 v) {
    raw[2 * w] = __float_as_uint(v.x);
    raw[2 * w + 1] = __float_as_uint(v.y);
}

// A quarter's 32 products q.k, capped in place: cap2 tanh(x), x = q.k * k, in base-2 units.
// k: the factors of the two blocks; largest: at least this lane's largest |x|.
// tanh x = 1 - 2 / (1 + e^(2x)), an exponential a score and one reciprocal for four: r = 1 / (abcd)
// gives 1 / a = r b cd and so on (2,048 rows under a window of 4,096, no other form taken: 218 us;
// one for two 233, for each 255). Off by a few 2^-23 of the cap, so for caps up to 128. |x| is
// cut at 10, where tanh is 1 to 2^-28 and the product of four still finite.
constexpr float kWideCap2 = 128.f * 1.4426950408889634f;
__device__ __forceinline__ void cap_scores(uint32_t (&raw)[32], const float (&k)[2], float cap2, float largest) {
    if (__any_sync(kFull, largest > 10.f)) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float most = 10.f / fabsf(k[i >> 4]);
            asm("min.NaN.f32 %0, %0, %1;\n\tmax.NaN.f32 %0, %0, %2;" : "+r"(raw[i]) : "r"(__float_as_uint(most)), "r"(__float_as_uint(-most)));
        }
    }
#pragma unroll
    for (int w = 0; w < 16; w += 2) {
        const float2 f = both(k[w >> 3] * 2.8853900817779268f);
        float2 a = __fmul2_rn(pair_of(raw, w), f), c = __fmul2_rn(pair_of(raw, w + 1), f);
        a = __fadd2_rn(make_float2(pa::fast_exp2(a.x), pa::fast_exp2(a.y)), both(1.f));
        c = __fadd2_rn(make_float2(pa::fast_exp2(c.x), pa::fast_exp2(c.y)), both(1.f));
        const float2 ac = __fmul2_rn(a, c);  // (a.x c.x, a.y c.y)
        const float r = pa::fast_rcp(ac.x * ac.y);
        const float2 rr = __fmul2_rn(make_float2(ac.y, ac.x), both(r));  // 1 / (a.x c.x), 1 / (a.y c.y)
        put_pair(raw, w, __ffma2_rn(__fmul2_rn(rr, c), both(-2.f * cap2), both(cap2)));
        put_pair(raw, w + 1, __ffma2_rn(__fmul2_rn(rr, a), both(-2.f * cap2), both(cap2)));
    }
}

// What a quarter's registers hold: products q.k (to be scaled; to be scaled and capped; to be
// scaled and biased), or scores (the exponent block by block; score by score, see the new reference).
enum { kProducts, kCapped, kBiased, kScores, kEachScore };
template <int X>
using Form = std::integral_constant<int, X>;

// MOD: how scores are reshaped. A segment's tiles are then walked from its last to its
// first: under a bias by distance the nearest keys, usually the heaviest, set a row's
// reference, and far ones seldom raise it. With a cap alone the first is the last one that
// all rows see whole, which gives a row 128 keys' largest score for a reference.
template <int G, int D, int EB, int MOD>
__global__ void __launch_bounds__(kWinThreads<EB>, 1)
pa_prefill_win_kernel(const PrefillParams P, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV) {
    using L_ = WinLay<D, EB>;
    constexpr int kKS = L_::kKS, kVS = L_::kVS, kNH = L_::kHalves, QT = kRows / G;
    constexpr uint32_t kTile = L_::kTile, kQTile = L_::kQTile;
    extern __shared__ __align__(1024) unsigned char sm[];
    const Bars<D, EB> bars{reinterpret_cast<uint64_t*>(sm + L_::kBars)};
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + L_::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L_::kMisc + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int H = P.n_heads, Hk = P.n_kv_heads;
    if (pa::smem_u32(sm) & 1023u) {  // never expected; refuse rather than mis-swizzle
        if (threadIdx.x == 0) pa::set_error(P.err, PA_DEVERR_LAYOUT);
        return;
    }
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int i = 0; i < Bars<D, EB>::kCount; ++i) {
            uint64_t* b = bars.b + i;
            // the converter warps' barriers take 4 arrivals
            const bool four = (b >= bars.k_conv(0) && b < bars.k_conv(kKS)) || (b >= bars.v_conv(0) && b < bars.v_conv(kVS)) ||
                              (b >= bars.raw_free(0) && b < bars.raw_free(2)) || b >= bars.v_exp(0) || b == bars.q_full();
            pa::mbar_init(b, four ? 4 : 1);
        }
        pa::fence_mbar_init();
    }
    pa::launch_dependents();     // the next kernel may be scheduled
    pa::grid_dependency_wait();  // the plan, and whatever wrote q and the cache, is complete
    if (warp == 0) {  // only now: tensor memory is not held while waiting for another kernel
        tc::tmem_alloc(tslot, kTmemCols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tbase = *tslot;
    Segments<G> segments(P);
    Segment g;
    bool ok = true;  // after a failed wait a role goes on without waiting, so that no other role is left alone
    int J0 = 0;      // tiles of the segments before
    auto tile_of = [](const Segment& seg, int j) {  // a segment's j-th tile
        if constexpr (MOD == kPlain) return seg.kt0 + j;
        constexpr int kEnd = (2 * QT + 2 * kKT - 2) / kKT;  // tiles that hold the rows' own positions, or one more
        const int lead = MOD != kCap || seg.n_kt <= kEnd ? 0 : kEnd;
        return seg.kt0 + seg.n_kt - 1 - (j == 0 ? lead : j <= lead ? j - 1 : j);
    };

    if (warp == 9 || warp == 14) {
        // ----------------------------------------------------------- TMA producers
        // A stage is refilled as soon as its last reader is done. bf16: K and V have a warp each:
        // when a tile's load waits in line behind the other operand's, the tensor core waits for it
        // (one warp for both: 11% more a tile). E4M3, half the bytes and boxes: one warp for both
        // (a second one takes issue slots from the softmax: 5% more a tile); K(J)'s codes replace
        // K(J-1)'s once those are widened, V's likewise.
        constexpr int kBoth = EB == 1;
        constexpr uint32_t kBytes = EB == 2 ? kTile : L_::kRawTile;
        // bf16: lane l < 8 kNH moves box (block l / kNH, dims 64 g .., g = l % kNH); E4M3: lane
        // l < 8 block l's 16 x D codes
        constexpr int NB = EB == 2 ? kNH : 1;
        const int b = (lane / NB) & (kBPT - 1), half = lane % NB;
        const uint32_t box = EB == 2 ? half * 16384 + b * 2048 : b * (kBS * D);
        struct Ring {  // one operand's
            const CUtensorMap* map;
            unsigned char* mem;
            uint64_t *full, *free;
            int n_stages;
            int st = 0, ph = 1;  // the next stage; the parity of the phase that frees it (for a first fill: of
                                 // the phase before the barrier's first, which passes)
            int ids, group;      // block ids of key tiles 4 group .. + 3, one per lane
        };
        auto ring = [&](int x) {
            Ring r;
            r.map = x ? &tmV : &tmK;
            r.mem = sm + (EB == 1 ? L_::kRaw + x * L_::kRawTile : x ? L_::kV0 : L_::kK0);
            r.full = x ? bars.v_full(0) : bars.k_full(0);
            r.free = EB == 1 ? bars.raw_free(x) : x ? bars.v_free(0) : bars.k_free(0);
            r.n_stages = EB == 1 ? 1 : x ? kVS : kKS;
            return r;
        };
        Ring first = ring(warp == 14), second = ring(1);
        while (ok && segments.next(g)) {
            const KeyTiles keys = segments.keys(g);
            const int nblk = min((g.ctx + kBS - 1) / kBS, P.max_blocks);
            const int32_t* trow = P.tables + (size_t)g.s * P.max_blocks;
            first.group = second.group = -1;
            auto load = [&](Ring& r, int tile) {
                if ((tile >> 2) != r.group) {  // warp-collective
                    r.group = tile >> 2;
                    const int blk = keys.block(r.group * 32 + lane);
                    r.ids = blk < nblk ? trow[blk] : -1;
                }
                const int bid = __shfl_sync(kFull, r.ids, (tile & 3) * kBPT + b);
                bool in = keys.block(tile * kBPT + b) < nblk;  // blocks past the context: zeros
                if (in && (bid < 0 || bid >= P.num_blocks)) {
                    if (lane < NB * kBPT && half == 0) pa::set_error(P.err, PA_DEVERR_BLOCK_ID);
                    in = false;
                }
                const int y = in ? (bid * Hk + g.kvh) * kBS : P.oob_row;  // out of range: zero fill
                ok = __all_sync(kFull, pa::mbar_wait(r.free + r.st, (uint32_t)r.ph, P.err, abort_flag));
                if (!ok) return;
                if (lane == 0) pa::mbar_arrive_expect_tx(r.full + r.st, kBytes);
                __syncwarp();
                if (lane < NB * kBPT)
                    tc::tma_load_2d(r.mem + r.st * kBytes + box, r.map, half * 64, y, r.full + r.st);
                __syncwarp();
                if (++r.st == r.n_stages) {
                    r.st = 0;
                    r.ph ^= 1;
                }
            };
            for (int j = 0; ok && j < g.n_kt; ++j) {
                load(first, tile_of(g, j));
                if (kBoth && ok) load(second, tile_of(g, j));
            }
        }
        // Every issued copy lands before the CTA exits: normally the converters and the tensor
        // core have consumed them all; after an abort, give those in flight time (bounded).
        if (!ok) {
            const uint64_t t0 = pa::globaltimer_ns();
            while (pa::globaltimer_ns() - t0 < 5000000ull) __nanosleep(10000);
        }
    } else if (warp == 8) {
        // -------------------------------------------------------------- MMA issuer
        // One thread issues every MMA. The tensor core runs them in issue order, so Q.K^T of tile
        // J + 1 may follow P.V of tile J (which reads P out of the same columns) without a wait, also
        // across segments. P is handed over by named barriers (ids 1 and 2: four softmax warps arrive,
        // this warp syncs), n_kt times per segment and tile on both sides, whatever fails.
        constexpr uint32_t ID_QK = EB == 2 ? tc::idesc_bf16_f32(128, 128, 0, 0) : idesc_f16_f32(128, 128, 0, 0);
        constexpr uint32_t ID_PV = idesc_f16_f32(128, D, 0, 1);
        const uint64_t dq = tc::smem_desc(pa::smem_u32(sm + L_::kQ), 16, 1024);
        const uint64_t dk = tc::smem_desc(pa::smem_u32(sm + L_::kK0), 16, 1024);
        const uint64_t dv = tc::smem_desc(pa::smem_u32(sm + L_::kV0), 16384, 1024);
        auto at = [](uint64_t d, uint32_t off16) {
            return ((uint64_t)(uint32_t)(d >> 32) << 32) | (uint32_t)((uint32_t)d + off16);
        };
        auto issue_qk = [&](int x, int kst) {  // S_x = Q_x K^T, K in stage kst (one thread)
            const uint32_t qo = x * (kQTile >> 4), ko = kst * (kTile >> 4);
            const uint32_t dst = tbase + x * 256;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t o = ((ks >> 2) * 16384 + (ks & 3) * 32) >> 4;
                tc::mma_bf16(dst, at(dq, qo + o), at(dk, ko + o), ID_QK, ks > 0 ? 1u : 0u);  // types per ID_QK
            }
            if (x == 1) tc::mma_commit(bars.k_free(kst));  // the stage's last reader
            tc::mma_commit(bars.s_full(x));
        };
        auto issue_pv = [&](int x, int vst, bool first) {  // O_x += P V (fp16), V in stage vst (one thread)
            const uint32_t vo = vst * (kTile >> 4);
            const uint32_t pcol = tbase + x * 256, dst = pcol + 128;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
                tc::mma_bf16_ts(dst, pcol + (ks >> 1) * 32 + (ks & 1) * 8, at(dv, vo + ks * (2048 >> 4)), ID_PV,
                                (!first || ks > 0) ? 1u : 0u);  // fp16 operands per ID_PV
            if (x == 1) tc::mma_commit(bars.v_free(vst));  // the stage's last reader
            tc::mma_commit(bars.pv_done(x));
        };
        int kst = 0, kph = 0, vst = 0, vph = 0;  // next K and V stage, phase parity
        auto k_ready = [&]() {
            return pa::mbar_wait(EB == 2 ? bars.k_full(kst) : bars.k_conv(kst), (uint32_t)kph, P.err, abort_flag);
        };
        auto k_next = [&]() {
            if (++kst == kKS) {
                kst = 0;
                kph ^= 1;
            }
        };
        for (int n_seg = 0; segments.next(g); ++n_seg) {
            if (ok) ok = pa::mbar_wait(bars.q_full(), (uint32_t)(n_seg & 1), P.err, abort_flag);
            if (ok) ok = k_ready();
            ok = __all_sync(kFull, ok);
            if (ok && lane == 0) {
                tc::fence_after_sync();
                issue_qk(0, kst);
                issue_qk(1, kst);
                if (g.n_kt == 1) tc::mma_commit(bars.q_free());
            }
            __syncwarp();
            k_next();
            for (int j = 0; j < g.n_kt; ++j) {
                const bool more = j + 1 < g.n_kt;
                if (ok) ok = pa::mbar_wait(bars.v_conv(vst), (uint32_t)vph, P.err, abort_flag);
                if (ok && more) ok = k_ready();
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
                    if (j + 2 == g.n_kt) tc::mma_commit(bars.q_free());  // that was the segment's last Q.K^T
                }
                __syncwarp();
                if (++vst == kVS) {
                    vst = 0;
                    vph ^= 1;
                }
                if (more) k_next();
            }
            J0 += g.n_kt;
        }
        // every issued MMA, and every arrival it makes, completes before the CTA releases its
        // shared and tensor memory (bounded waits)
        if (lane == 0) {
            tc::mma_commit(bars.drain());
            pa::mbar_wait(bars.drain(), 0, nullptr, 10000000ull);
            if (ok) {
                for (int J = max(0, J0 - kKS); J < J0; ++J)
                    pa::mbar_wait(bars.k_free(J % kKS), (uint32_t)((J / kKS) & 1), nullptr, 10000000ull);
                for (int J = max(0, J0 - kVS); J < J0; ++J)
                    pa::mbar_wait(bars.v_free(J % kVS), (uint32_t)((J / kVS) & 1), nullptr, 10000000ull);
            }  // (q_free, of the last segment: before drain)
        }
        __syncwarp();
    } else if (warp >= 10) {
        // -------------------------------------------------------------- converters
        // Four warps, one per scheduler: each segment's Q, then its V tiles to fp16 (bf16 cache:
        // in place, v * 2^-8; E4M3: K and V, from the codes to their stages).
        const int t = threadIdx.x - 320;  // 0..127
        auto arrive = [&](uint64_t* bar) {  // after generic writes that the tensor core reads next
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) pa::mbar_arrive(bar);
        };
        for (int n_seg = 0; ok && segments.next(g); ++n_seg) {
            const KeyTiles keys = segments.keys(g);
            // ---- Q: tile X row r = (chunk token i0 + X*QT + r/G, head h0 + r%G). Thread t takes chunk
            // t % (D / 8) of every (1024 / D)-th row: a warp reads whole rows. The first half is in
            // registers before the old Q is free.
            {
                constexpr int CPR = D / 8, RPP = 128 / CPR, NP = kRows / RPP;  // chunks per row, rows per pass, passes
                const int c = t % CPR, r0 = t / CPR, i0 = g.qp * 2 * QT;
                auto fetch = [&](int x, int p) {
                    const int r = r0 + p * RPP, i = i0 + x * QT + r / G;
                    return i < g.L ? reinterpret_cast<const uint4*>(P.q + ((size_t)(g.q0 + i) * H + g.kvh * G + r % G) * D)[c]
                                   : make_uint4(0, 0, 0, 0);
                };
                auto put = [&](int x, int p, uint4 v) {
                    const int r = r0 + p * RPP;
                    if constexpr (EB == 1) {  // fp16 operands: exact for |q| in fp16's normal range
                        uint32_t* u = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 f = pa::bf16x2_to_float2(u[k]);
                            u[k] = float2_to_f16x2(f.x, f.y);
                        }
                    }
                    *reinterpret_cast<uint4*>(sm + L_::kQ + x * kQTile + (c >> 3) * 16384 + tc::sw128_offset(r, c & 7)) = v;
                };
                uint4 v[8];
#pragma unroll
                for (int p = 0; p < 8; ++p) v[p] = fetch(0, p);
                if (n_seg > 0) ok = pa::mbar_wait(bars.q_free(), (uint32_t)((n_seg - 1) & 1), P.err, abort_flag);
                ok = __all_sync(kFull, ok);
                if (!ok) break;
#pragma unroll
                for (int b = 0; b < 2 * NP; b += 8) {
#pragma unroll
                    for (int p = 0; p < 8; ++p) put((b + p) / NP, (b + p) % NP, v[p]);
                    if (b + 8 < 2 * NP) {
#pragma unroll
                        for (int p = 0; p < 8; ++p) v[p] = fetch((b + 8 + p) / NP, (b + 8 + p) % NP);
                    }
                }
                arrive(bars.q_full());
            }
            if constexpr (EB == 2) {
                // A warp converts the 32 keys that a quarter of the softmax takes: their largest magnitude
                // gives the quarter's exponent e. Loops of a few chunks: unrolled further, or with the rows
                // held in registers from one pass to the other, the code took 3 to 8% more of the whole
                // kernel's time.
                const int w4 = warp - 10;
                for (int j = 0; j < g.n_kt; ++j) {
                    const int J = J0 + j, st = J % kVS, tile = tile_of(g, j);
                    ok = pa::mbar_wait(bars.v_full(st), (uint32_t)((J / kVS) & 1), P.err, abort_flag);
                    ok = __all_sync(kFull, ok);
                    if (!ok) break;
                    // chunk c of the lane: 16 bytes of row 32 w4 + 4 (c % 8) + lane / 8, 64-dim half c / 8
                    constexpr int NC = (int)(kTile / 2048);
                    uint4* vs = reinterpret_cast<uint4*>(sm + L_::kV0 + st * kTile) + w4 * 256 + lane;
                    auto at = [](int c) { return (c >> 3) * 1024 + (c & 7) * 32; };
                    if (hides_rows(keys, g.ctx, tile)) {  // no query of the pair sees: zero (p = 0 must not meet a NaN)
#pragma unroll 1
                        for (int c = 0; c < NC; ++c)
                            if (hidden_row(P, keys, g.ctx, keys.position(tile, 32 * w4 + 4 * (c & 7) + (lane >> 3))))
                                vs[at(c)] = make_uint4(0, 0, 0, 0);
                    }
                    uint32_t most = 0;  // the largest magnitude of either half-word, signs undefined
                    auto larger = [&](uint32_t u) { asm("max.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(most) : "r"(u)); };
#pragma unroll 1
                    for (int c = 0; c < NC && !__any_sync(kFull, (most & 0x40004000u) != 0); c += 2) {  // one of 2 or more settles it
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint4 w = vs[at(c + k)];
                            larger(w.x);
                            larger(w.y);
                            larger(w.z);
                            larger(w.w);
                        }
                    }
                    most = __reduce_max_sync(kFull, max(most >> 16 & 0x7fffu, most & 0x7fffu));
                    const int e = max(kLeastExp, min(0, (int)(most >> 7) - 127));
                    if (lane == 0) {
                        reinterpret_cast<float2*>(sm + L_::kVExp)[st * 4 + w4] = make_float2((float)e, __int_as_float((127 - e) << 23));
                        pa::mbar_arrive(bars.v_exp(st));
                    }
                    const float f = __int_as_float((119 - e) << 23);  // 2^(-8 - e)
                    const float2 f2 = make_float2(f, f);
                    auto cvt = [&](uint32_t u) {  // bf16 pair -> fp16 pair of v * 2^(-8 - e)
                        const float2 x = __fmul2_rn(make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)), f2);
                        return float2_to_f16x2(x.x, x.y);
                    };
#pragma unroll 4
                    for (int c = 0; c < NC; ++c) {
                        const uint4 w = vs[at(c)];
                        vs[at(c)] = make_uint4(cvt(w.x), cvt(w.y), cvt(w.z), cvt(w.w));
                    }
                    arrive(bars.v_conv(st));
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
                auto widen = [&](int x, unsigned char* dst, int tile) {
                    const unsigned char* raw = sm + L_::kRaw + x * L_::kRawTile + src0;
                    auto pass = [&](auto partial) {
#pragma unroll 4
                        for (int c = 0; c < kKT / kStep; ++c) {
                            uint4 w = *reinterpret_cast<const uint4*>(raw + c * kStep * D);
                            // V rows that no query of the pair sees are zero (p = 0 must not meet a NaN)
                            if constexpr (decltype(partial)::value) {
                                if (hidden_row(P, keys, g.ctx, keys.position(tile, row0 + c * kStep))) w = make_uint4(0, 0, 0, 0);
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
                    if (x == 1 && hides_rows(keys, g.ctx, tile)) pass(std::true_type{});
                    else pass(std::false_type{});
                    arrive(bars.raw_free(x));
                };
                for (int j = 0; j < g.n_kt; ++j) {
                    const int J = J0 + j, tile = tile_of(g, j), ks = J % kKS, vs = J % kVS;
                    ok = pa::mbar_wait(bars.k_full(0), (uint32_t)(J & 1), P.err, abort_flag);
                    if (ok && J >= kKS) ok = pa::mbar_wait(bars.k_free(ks), (uint32_t)(((J - kKS) / kKS) & 1), P.err, abort_flag);
                    ok = __all_sync(kFull, ok);
                    if (!ok) break;
                    widen(0, sm + L_::kK0 + ks * kTile, tile);
                    if (lane == 0) pa::mbar_arrive(bars.k_conv(ks));
                    ok = pa::mbar_wait(bars.v_full(0), (uint32_t)(J & 1), P.err, abort_flag);
                    if (ok && J >= kVS) ok = pa::mbar_wait(bars.v_free(vs), (uint32_t)(((J - kVS) / kVS) & 1), P.err, abort_flag);
                    ok = __all_sync(kFull, ok);
                    if (!ok) break;
                    widen(1, sm + L_::kV0 + vs * kTile, tile);
                    if (lane == 0) pa::mbar_arrive(bars.v_conv(vs));
                }
            }
            J0 += g.n_kt;
        }
    } else {
        // ------------------------------------------- softmax warpgroup of tile x
        // As in prefill.cu: thread = row, one pass over S per key tile, a quarter of 32 columns at a
        // time, p = 2^(s*scale - m) against the row's integer reference m, which changes on a row's
        // first visible keys and before a quarter's sum could leave fp16's range.
        const int x = warp >> 2, r = threadIdx.x & 127;  // matrix row = TMEM lane
        const uint32_t tS = tbase + x * 256 + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t tO = tS + 128;
        const float sc = P.scale_log2;
        int vst = 0, vph = 0;  // bf16: V stage and phase parity of the tile
        Segment after;  // the next segment, read while the last P.V of this one runs
        for (bool more = segments.next(g); more; g = after) {
            const KeyTiles keys = segments.keys(g);
            const int i = g.qp * 2 * QT + x * QT + r / G;
            const int pos = g.ctx - g.L + i;  // this row's position (padding rows: beyond the chunk)
            const int limit = MOD ? max(pos, prefix_of(P, g.s, g.ctx) - 1) : pos;  // the last position it sees
            float slope2 = 0.f;
            if constexpr (MOD >= kBias) slope2 = P.slopes ? pa::slope_log2(P.slopes[g.kvh * G + r % G]) : 0.f;
            float m_used = -INFINITY, l = 0.f;
            // Key k of tile j is at position 128 j + k + kb_sinks if it is a sink, else + kb_win. In tiles
            // from j_win on, the limits below are those of the window's keys: where such a tile begins
            // with sinks, they precede every row's window, so each row sees them by their number alone.
            const int kb_sinks = g.kt0 * kKT, kb_win = kb_sinks + (keys.first - keys.n_sink) * kBS;
            const int j_win = keys.n_sink / kBPT - g.kt0;
            // E4M3: lane l holds the scales of block l % 8 of a key tile; those of
            // tile j + 1 and the block id of tile j + 2 are loaded while tile j is
            // worked on.
            const int nblk = min((g.ctx + kBS - 1) / kBS, P.max_blocks);
            auto block_id = [&](int j) {
                const int blk = j < g.n_kt ? keys.block(tile_of(g, j) * kBPT + (lane & (kBPT - 1))) : nblk;
                return blk < nblk ? P.tables[(size_t)g.s * P.max_blocks + blk] : -1;
            };
            auto scale_of = [&](const float* scales, int bid) {
                return bid >= 0 && bid < P.num_blocks ? scales[(size_t)bid * Hk + g.kvh] : 1.f;
            };
            float ks_next = 1.f, vs_next = 1.f;
            int bid_next = -1;
            if constexpr (EB == 1) {
                const int bid = block_id(0);
                ks_next = scale_of(P.k_scale, bid);
                vs_next = scale_of(P.v_scale, bid);
                bid_next = block_id(1);
            }
            for (int j = 0; j < g.n_kt; ++j) {
                const int J = J0 + j;
                float my_k = 0.f, my_e = 0.f;
                if constexpr (EB == 1) {  // the approximate log2 and reciprocal are off by 2^-22, far below w's rounding
                    const float vs = clamp_scale(vs_next);
                    my_k = clamp_scale(ks_next) * sc;
                    my_e = __log2f(vs);
                    ks_next = scale_of(P.k_scale, bid_next);
                    vs_next = scale_of(P.v_scale, bid_next);
                    bid_next = block_id(j + 2);
                }
                // bf16: the tile's exponents; nearly always there, as V is loaded ahead. A barrier of their own:
                // waiting for the converted tile took up to 1% longer.
                if (EB == 2 && ok) ok = pa::mbar_wait(bars.v_exp(vst), (uint32_t)vph, P.err, abort_flag);
                if (ok) ok = pa::mbar_wait(bars.s_full(x), (uint32_t)(J & 1), P.err, abort_flag);
                ok = __all_sync(kFull, ok);
                tc::fence_after_sync();
                const float2* v_exp = reinterpret_cast<const float2*>(sm + L_::kVExp) + vst * 4;
                if (++vst == kVS) {
                    vst = 0;
                    vph ^= 1;
                }
                const int jt = tile_of(g, j) - g.kt0;
                const int kb = jt * kKT + (jt < j_win ? kb_sinks : kb_win);
                // A row does not see keys beyond its position or, sinks apart, before its window. A warp
                // takes the masking code only for a tile where that hides a key from one of its rows (a
                // warp-uniform branch): a tile or two at either end of a window, and that of the sinks.
                // Key k of a quarter is bit k of the quarter's mask: two instructions an element (as
                // three comparisons, a masked tile took twice a plain one's time).
                const int lim0 = limit - kb;  // keys k > lim0 of the tile are not visible
                // (A prefix may end any distance behind a row, so that the window's beginning comes first.)
                const int lim1 = P.window >= 0 ? (MOD ? max(pos - P.window, 0) - kb : pos - kb - P.window) : 0, sink1 = P.n_sinks - kb_sinks - jt * kKT;  // nor k < lim1, k >= sink1
                // (With a bias also for one with a key after a row's own position, which a prefix may show.)
                const bool mask_warp = __any_sync(kFull, (MOD >= kBias && P.slopes ? pos - kb : lim0) < kKT - 1 || (lim1 > 0 && sink1 < kKT));
                auto below = [](int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; };  // bits 0 .. n-1
                auto visible_of = [&](int qd) {
                    const int k0 = 32 * qd;
                    return below(lim0 + 1 - k0) & (~below(lim1 - k0) | below(sink1 - k0));
                };
                float2 psum2 = make_float2(0.f, 0.f);  // this tile's sum of p against m_used
                float alpha = 1.f;                     // this tile's rescale of l and O
                const float2 sc2 = make_float2(sc, sc);
                // p of one quarter (raw scores in columns 32q..32q+31) -> fp16 pairs;
                // P of keys 2w, 2w+1 goes to column 32q + w, so a quarter only
                // overwrites columns it has already read.
                // Returns the quarter's sum of w; `add` is what it adds to the row's sum
                // (E4M3: each block's sum over its V scale; bf16: the quarter's times 2^-e).
                float qk[2] = {sc, sc}, qe[2] = {0.f, 0.f}, qi[2] = {1.f, 1.f};  // E4M3: the quarter's two blocks; bf16: [0]
                // `form`: what raw holds
                auto exps = [&](auto masked, auto form, const uint32_t (&raw)[32], uint32_t visible, uint32_t (&ph)[16], float& add) {
                    float2 qs[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int w = 0; w < 16; ++w) {
                        const int b = EB == 1 ? w >> 3 : 0;
                        const float nm = qe[MOD >= kBias ? w >> 3 : b] - m_used;
                        float2 e = make_float2(__uint_as_float(raw[2 * w]), __uint_as_float(raw[2 * w + 1]));
                        if constexpr (decltype(form)::value == kScores) {
                            e = __fadd2_rn(e, both(nm));
                        } else if constexpr (decltype(form)::value == kEachScore) {
                            e = __fadd2_rn(__fadd2_rn(e, both(qe[MOD >= kBias ? w >> 3 : b])), both(-m_used));
                        } else if constexpr (decltype(form)::value == kCapped) {
                            const float2 z = __fmul2_rn(e, e);
                            float2 q = both(P.poly[3]);
#pragma unroll
                            for (int i = 2; i >= 0; --i) q = __ffma2_rn(q, z, both(P.poly[i]));
                            e = __ffma2_rn(e, q, both(nm));
                        } else if constexpr (decltype(form)::value == kBiased) {
                            e = __ffma2_rn(e, both(qk[b]), __ffma2_rn(make_float2(2 * w & 15, (2 * w & 15) + 1), both(slope2), both(nm)));
                        } else {
                            e = __ffma2_rn(e, EB == 1 ? both(qk[b]) : sc2, both(nm));
                        }
                        if constexpr (decltype(masked)::value) {  // masked keys give p = 0 (also for a zero scale)
                            if (!(visible & (1u << (2 * w)))) e.x = -INFINITY;
                            if (!(visible & (1u << (2 * w + 1)))) e.y = -INFINITY;
                        }
                        e.x = pa::fast_exp2(e.x);
                        e.y = pa::fast_exp2(e.y);
                        qs[b] = __fadd2_rn(qs[b], e);
                        ph[w] = float2_to_f16x2(e.x, e.y);
                    }
                    const float s0 = qs[0].x + qs[0].y;
                    if constexpr (EB == 2) {
                        add = s0 * qi[0];
                        return s0;
                    }
                    const float s1 = qs[1].x + qs[1].y;
                    add = s0 * qi[0] + s1 * qi[1];
                    return s0 + s1;
                };
                auto sweep = [&](auto masked) {
#pragma unroll 1
                    for (int qd = 0; qd < 4; ++qd) {
                        uint32_t raw[32];
                        float2 ve;  // (read here, its latency is covered by that of the scores)
                        if constexpr (EB == 2) ve = v_exp[qd];
                        tc::tmem_ld32(tS + 32 * qd, raw);
                        tc::tmem_wait_ld();
                        if constexpr (EB == 2) {
                            qe[0] = ve.x;
                            qi[0] = ve.y;
                        } else {
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
                                qk[b] = __shfl_sync(kFull, my_k, 2 * qd + b);
                                qe[b] = __shfl_sync(kFull, my_e, 2 * qd + b);
                                qi[b] = pa::fast_exp2(-qe[b]);
                            }
                        }
                        const uint32_t visible = decltype(masked)::value ? visible_of(qd) : 0xffffffffu;
                        // A bias -slope2 (back - at): the keys' places `at` in their block with the scores, the
                        // row's distance `back` to the block's first key with the exponent.
                        float back[2] = {0.f, 0.f};
                        if constexpr (MOD >= kBias) {
                            if constexpr (EB == 2) qe[1] = qe[0];
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
                                back[b] = (float)(pos - keys.position(tile_of(g, j), 32 * qd + kBS * b));
                                qe[b] = fmaf(-slope2, back[b], qe[b]);
                            }
                        }
                        float largest = 0.f;
                        auto scores_of = [&]() {  // of raw's products, the bias's `at` among them
                            // keys hidden from the row may hold anything, and cap_scores mixes four of them
                            if constexpr (decltype(masked)::value) {
#pragma unroll
                                for (int k = 0; k < 32; ++k)
                                    if (!(visible & (1u << k))) raw[k] = 0u;
                            }
                            if constexpr (MOD == kCap) {
                                cap_scores(raw, qk, P.cap2, largest);
                            } else if (MOD == kCapBias && P.cap2 <= kWideCap2) {
                                cap_scores(raw, qk, P.cap2, largest_of(raw, qk));
                            } else if (MOD == kCapBias && !__any_sync(kFull, largest_of(raw, qk) >= pa::kTanhSmall)) {
#pragma unroll
                                for (int w = 0; w < 16; ++w) {  // the polynomial of pa::tanh_f32
                                    const float2 x = __fmul2_rn(pair_of(raw, w), both(qk[w >> 3])), z = __fmul2_rn(x, x);
                                    float2 q = both(pa::tanh_coef(4));
#pragma unroll
                                    for (int i = 3; i >= 0; --i) q = __ffma2_rn(q, z, both(pa::tanh_coef(i)));
                                    put_pair(raw, w, __fmul2_rn(__fmul2_rn(x, both(P.cap2)), __ffma2_rn(q, z, both(1.f))));
                                }
                            } else {
#pragma unroll
                                for (int k = 0; k < 32; ++k) {
                                    const float v = __uint_as_float(raw[k]) * qk[k >> 4];
                                    raw[k] = __float_as_uint(MOD == kCapBias ? P.cap2 * pa::tanh_f32(v) : v);
                                }
                            }
                            if constexpr (MOD >= kBias) {
#pragma unroll
                                for (int w = 0; w < 16; ++w) {
                                    const float at = 2 * w & 15, bk = back[w >> 3];
                                    float2 v = __ffma2_rn(make_float2(at, at + 1.f), both(slope2), pair_of(raw, w));
                                    if (decltype(masked)::value && P.prefix)  // a key after the row, at > bk: its distance is at - bk
                                        v = __ffma2_rn(make_float2(fmaxf(at - bk, 0.f), fmaxf(at + 1.f - bk, 0.f)), both(-2.f * slope2), v);
                                    put_pair(raw, w, v);
                                }
                            }
                        };
                        // Products go straight into the exponent while that is one form for all of them: with a
                        // cap, scores that a short polynomial covers (P.small: 0.6 of the cap; 2^-18.6 of the
                        // score, 2^-13.7 of a weight at a cap of 50, half of P's own rounding); with a bias,
                        // where no key can come after the row. Not over E4M3 with a cap: loud blocks' scores are
                        // often beyond it, and taking turns costs more than cap_scores alone (three prompts of
                        // 1,000 to 1,600 rows, scores of a spread of 6: 250 us, 205; of a spread of 1: 158, 178).
                        bool whole = (MOD == kCap && EB == 2) || (MOD == kBias && !(decltype(masked)::value && P.prefix));
                        if constexpr (MOD == kCap) {
                            largest = largest_of(raw, qk);
                            if (EB == 2) whole = !__any_sync(kFull, !(largest <= P.small));
                        }
                        uint32_t ph[16];
                        float add, qs;
                        constexpr int kForm = MOD == kCap ? kCapped : MOD == kBias ? kBiased : kProducts;
                        if constexpr (MOD == kPlain) {
                            qs = exps(masked, Form<kProducts>{}, raw, visible, ph, add);
                        } else if (MOD != kCapBias && whole) {
                            qs = exps(masked, Form<kForm>{}, raw, visible, ph, add);
                        } else {
                            scores_of();
                            qs = exps(masked, Form<kScores>{}, raw, visible, ph, add);
                        }
                        const bool big = !(qs <= 32768.f);  // also inf (no reference yet) and NaN
                        if (__any_sync(kFull, big)) {
                            // rare: a new reference for the rows that need one
                            if (MOD != kPlain && whole) scores_of();
                            float a = 1.f;
                            if (big) {
                                float qmax = -INFINITY;
#pragma unroll
                                for (int k = 0; k < 32; ++k) {
                                    const bool vis = !decltype(masked)::value || (visible & (1u << k));
                                    const float r = __uint_as_float(raw[k]);
                                    const int b = EB == 1 ? k >> 4 : 0;
                                    if (vis) qmax = fmaxf(qmax, MOD != kPlain ? r + qe[MOD >= kBias ? k >> 4 : b] : fmaf(r, qk[b], qe[b]));
                                }
                                const float mq = ceilf(qmax);
                                if (mq > m_used) {
                                    // 2^(m_used - mq) built from its exponent bits (0 below 2^-126)
                                    const float d = m_used - mq;
                                    a = d < -126.f ? 0.f : __int_as_float(((int)d + 127) << 23);
                                    m_used = mq;
                                    if constexpr (MOD < kBias) exps(masked, Form<MOD != kPlain ? kScores : kProducts>{}, raw, visible, ph, add);
                                }
                                // Steep biases make scores whose roundings, of a block's bias less the reference, are
                                // above fp16's range (of 2^27 and up; also without a new reference). Rounded as the
                                // largest was, no score is above it.
                                if constexpr (MOD >= kBias) exps(masked, Form<kEachScore>{}, raw, visible, ph, add);
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
                auto quarter_factors = [&](int qd, float (&k)[2], float (&e)[2]) {
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        k[b] = EB == 2 ? sc : __shfl_sync(kFull, my_k, 2 * qd + b);
                        e[b] = EB == 2 ? v_exp[qd].x : __shfl_sync(kFull, my_e, 2 * qd + b);
                    }
                };
                // The segment's first tile, seen whole: its largest score is the row's reference. From 32
                // keys alone, as below, scores of a wide spread (6 either way) outgrew it again and again.
                if (MOD == kCap && j == 0 && !mask_warp && sc >= 0.f) {
                    float top = -INFINITY;
#pragma unroll 1
                    for (int qd = 0; qd < 4; ++qd) {
                        uint32_t raw[32];
                        tc::tmem_ld32(tS + 32 * qd, raw);
                        tc::tmem_wait_ld();
                        float k[2], e[2], most[2] = {-INFINITY, -INFINITY};
                        quarter_factors(qd, k, e);
#pragma unroll
                        for (int i = 0; i < 32; ++i) most[i >> 4] = fmaxf(most[i >> 4], __uint_as_float(raw[i]));
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const float v = most[b] * k[b];
                            top = fmaxf(top, fmaf(P.cap2, pa::tanh_f32(v), e[b]));
                        }
                    }
                    m_used = ceilf(top);
                }
                if (mask_warp) sweep(std::true_type{});
                else sweep(std::false_type{});
                l = l * alpha + (psum2.x + psum2.y);
                // a new reference rescales O_x: PV_x(j-1) must have landed first
                if (j > 0 && __any_sync(kFull, alpha != 1.f)) {
                    if (ok) ok = pa::mbar_wait(bars.pv_done(x), (uint32_t)((J - 1) & 1), P.err, abort_flag);
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
            more = segments.next(after);
            if (ok) ok = pa::mbar_wait(bars.pv_done(x), (uint32_t)((J0 + g.n_kt - 1) & 1), P.err, abort_flag);
            ok = __all_sync(kFull, ok);
            J0 += g.n_kt;
            if (!ok) continue;
            tc::fence_after_sync();
            constexpr float kUndo = EB == 2 ? 256.f : 1.f;  // V's 2^-8
            bool finite = true;
            auto own = [&](int c, float (&v)[32]) {
                uint32_t raw[32];
                tc::tmem_ld32(tO + c * 32, raw);
                tc::tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(raw[k]) * kUndo;
            };
            auto row_out = [&](int rr) {  // output row of matrix row rr
                return reinterpret_cast<uint4*>(P.out + ((size_t)(g.q0 + i - r / G + rr / G) * H + g.kvh * G + rr % G) * D);
            };
            // The normalised output: 32 columns, 64 bytes of each row. Four lanes exchange theirs
            // so that each of their stores covers a row's 64 bytes: as 16 bytes a row, 32 rows an
            // instruction, the stores took 2 us a segment.
            auto put = [&](int c, const float (&v)[32]) {
                if (i < g.L) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) finite &= fabsf(v[k]) < INFINITY;
                }
                uint32_t w[4][4];  // [16-byte chunk][word]
#pragma unroll
                for (int k = 0; k < 16; ++k) w[k >> 2][k & 3] = pa::float2_to_bf16x2(v[2 * k], v[2 * k + 1]);
#pragma unroll
                for (int o = 1; o <= 2; o <<= 1) {  // transposes the 4 x 4 chunks of a lane quad
                    const bool up = (lane & o) != 0;
#pragma unroll
                    for (int a = 0; a < 4; ++a) {
                        if (a & o) continue;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t got = __shfl_xor_sync(kFull, up ? w[a][e] : w[a + o][e], o);
                            if (up) w[a][e] = got;
                            else w[a + o][e] = got;
                        }
                    }
                }
#pragma unroll
                for (int a = 0; a < 4; ++a) {  // chunk lane % 4 of the quad's row a
                    const int rr = (r & ~3) + a;
                    if (i - r / G + rr / G < g.L)
                        row_out(rr)[4 * c + (lane & 3)] = make_uint4(w[a][0], w[a][1], w[a][2], w[a][3]);
                }
            };
            if (!__any_sync(kFull, i < g.L)) {
                // no row of this warp is in the chunk: nothing to keep, here and in other pieces of the item
            } else if (g.slot >= 0) {
                join_pieces<D>(P, g.slot, x, r, warp, lane, i < g.L, m_used, l, own, put, [&](int rr, float4 v) {
                    uint2* row = reinterpret_cast<uint2*>(row_out((r & ~31) + rr));
                    if (lane >= D / 4) return;
                    finite &= fabsf(v.x) < INFINITY && fabsf(v.y) < INFINITY && fabsf(v.z) < INFINITY && fabsf(v.w) < INFINITY;
                    row[lane] = make_uint2(pa::float2_to_bf16x2(v.x, v.y), pa::float2_to_bf16x2(v.z, v.w));
                });
            } else if (P.work || P.splits <= 1) {
                const float inv = 1.f / l;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float v[32];
                    own(c, v);
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] *= inv;
                    put(c, v);
                }
            } else {  // per-pair mode: keep O, m and l for the merge kernel
                const size_t item = ((size_t)g.s * Hk + g.kvh) * P.n_qp + g.qp;
                float* part = P.part + (((item * P.splits + blockIdx.x % P.splits) * 2 + x) * 128 + r) * kPartStride;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float v[32];
                    own(c, v);
                    if (i < g.L) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) finite &= fabsf(v[k]) < INFINITY;
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            *reinterpret_cast<float4*>(part + c * 32 + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                    }
                }
                if (i < g.L) *reinterpret_cast<float2*>(part + kPartML) = make_float2(m_used, l);
            }
            if (!finite) pa::set_error(P.err, PA_DEVERR_RANGE);
        }
    }
    tc::fence_before_sync();
    __syncthreads();  // every role is done with shared memory, tensor memory and the barriers
    if (warp == 0) tc::tmem_dealloc(tbase, kTmemCols);
}

// Even mode: the work list. An item costs
// its key tiles plus kStart, what starting and finishing a segment takes in
// units of a tile (the pipeline's fill, the epilogue: 4 us for an item run whole
// against 1.78 us a tile, 5 and 8 us for the two pieces of a cut one; 3 was the
// best of 1, 2, 3 and 5 for chunks of several lengths together: 190, 188, 189
// and 190 us for two of 1,024 rows, 231, 204, 202 and 207 us for four of 512
// rows behind 700 .. 16,384 tokens). The costs of all non-empty items, in item
// order, are cut into C runs of equal length, C the CTAs (fewer when a run would
// be shorter than kStart + 4), so that all CTAs finish together: each has at most
// one piece of an item begun by the CTA before, whole items, and one piece of an
// item that the next CTA goes on with. (A window makes the items equally long and few waves deep: 256
// items of 33 tiles on 152 CTAs take 4 segments on the busiest CTA with whole
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
// Capped scores over a bf16 cache take 1.5 of a plain tile's time, and starting no more: two
// of theirs (2,048 rows under a window of 4,096, on one cache again and again: 184 and 177 us; over E4M3, whose segments take
// longer to start, three remain: 205, with two 211).
constexpr int kStart = 3, kLeast = 3;
constexpr int kStartCap = 2;
template <int G>
__global__ void __launch_bounds__(1024) pa_prefill_plan_even_kernel(const PrefillParams P) {
    __shared__ long long wsum[32];
    __shared__ int wcnt[32], wmax[32];
    pa::launch_dependents();     // the prefill kernel may be scheduled
    pa::grid_dependency_wait();  // the lengths are written
    const int start = P.cap2 > 0.f && !P.k_scale ? kStartCap : kStart;
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
        mine += nk > 0 ? nk + start : 0;
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
    const bool whole = np <= P.n_cta && wmax[0] <= T / P.n_cta + 2 * start;
    const long long C = max(1LL, min((long long)P.n_cta, T / (start + 4)));
    long long off = incl - mine + (wid > 0 ? wsum[wid - 1] : 0);
    int r = icnt - cnt + (wid > 0 ? wcnt[wid - 1] : 0);
    for (int it = b0; it < b1; ++it) {
        const int nk = item_tiles<G>(P, it);
        if (nk <= 0) continue;
        if (whole) {
            P.work[r] = make_int4(it, 0, nk, -1);
            cta[r] = make_int4(r, r + 1, -1, 0);
        } else {
            // run c: costs [c T / C, (c + 1) T / C); the item's costs are [off, off + nk + start)
            const int c0 = (int)(((off + 1) * C - 1) / T), c1 = (int)(((off + nk + start) * C - 1) / T);
            auto cut = [&](int c) {  // the item's tile at which run c begins
                if (c <= c0) return 0;
                if (c > c1) return nk;
                const int x = (int)(c * T / C - off) - start;
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
        off += nk + start;
        ++r;
    }
}

template <int G, int D, int EB, int MOD>
int launch_prefill_win(const PrefillParams& Pp, const CUtensorMap& tk, const CUtensorMap& tv, int n_seqs,
                       int n_rows, cudaStream_t stream) {
    auto kern = pa_prefill_win_kernel<G, D, EB, MOD>;
    constexpr uint32_t kSmemBytes = WinLay<D, EB>::kSmem;
    static bool attr_done[64] = {false};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_done[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes) != cudaSuccess)
            return PA_ERR_CUDA;
        attr_done[dev] = true;
    }
    if (Pp.work) {  // even mode: plan, then one CTA per SM, launched ahead of the plan's end
        const int st = pa_launch_pdl(pa_prefill_plan_even_kernel<G>, dim3(1), dim3(1024), 0, stream, Pp);
        if (st != PA_OK) return st;
        return pa_launch_pdl(kern, dim3((unsigned)Pp.n_cta), dim3(kWinThreads<EB>), kSmemBytes, stream, Pp, tk, tv);
    }
    const int st = pa_launch_pdl(kern, dim3(Pp.n_qp * Pp.splits, Pp.n_kv_heads, n_seqs), dim3(kWinThreads<EB>), kSmemBytes, stream,
                                 Pp, tk, tv);
    if (st != PA_OK || Pp.splits <= 1) return st;
    // rows of all chunks: the merge finds each row's sequence in q_start_loc
    const long long warps = (long long)n_rows * Pp.n_heads;
    return pa_launch_pdl(pa_prefill_merge_kernel<G, D>, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0, stream, Pp, n_seqs,
                         n_rows, Pp.n_qp);
}

template <int D, int EB, int MOD = kPlain>
int dispatch_prefill_win(int G, const PrefillParams& P, const CUtensorMap& tk, const CUtensorMap& tv, int n_seqs,
                         int n_rows, cudaStream_t stream) {
    switch (G) {
        case 1: return launch_prefill_win<1, D, EB, MOD>(P, tk, tv, n_seqs, n_rows, stream);
        case 2: return launch_prefill_win<2, D, EB, MOD>(P, tk, tv, n_seqs, n_rows, stream);
        case 4: return launch_prefill_win<4, D, EB, MOD>(P, tk, tv, n_seqs, n_rows, stream);
        default: return launch_prefill_win<8, D, EB, MOD>(P, tk, tv, n_seqs, n_rows, stream);
    }
}

}  // namespace
