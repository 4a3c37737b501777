// Cache write with the position rotation applied on the way.
//
// A new token's q and k are rotated by its position p before attention sees
// them (rotary position embedding): each pair of dims (x, y) of a head turns
// by the angle p * f_i of its frequency i,
//     x' = x cos - y sin,    y' = y cos + x sin,
// with cos and sin read from the caller's fp32 table row of p. Pairs are dims
// (i, i + r/2) or, interleaved, (2i, 2i + 1), i < r/2; dims from r on pass
// through. k' and v then go to the token's slot ("KV Cache Explained Like
// You're an LLM Engineer", section "What KV Cache Stores"; "Inference serving:
// the KV-cache machine", section "Paged KV: virtual memory for tokens": slot =
// block table[p / 16] * 16 + p % 16), as bf16, as E4M3 with a scale per KV
// head, or as E4M3 with a scale per (block, KV head). One launch replaces the
// rotation of q, the rotation of k and the scatter, so q, k and v are read
// once and written once.
//
// Products and sums are rounded one by one in fp32 (no contraction), and the
// result once to its stored type.
#include <math.h>

#include "pa_common.cuh"

namespace {

constexpr int kBS = 16;        // tokens per block
constexpr int kThreads = 128;  // threads per CTA
constexpr unsigned kFull = 0xffffffffu;

enum Mode { kBf16 = 0, kHeadScale = 1, kBlockScale = 2 };

struct RopeParams {
    uint16_t* q_out;
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    unsigned char* k_pool;
    unsigned char* v_pool;
    const float* cos_sin;  // [max_position][rot]: rot/2 cosines, rot/2 sines
    const int64_t* pos;
    const int64_t* slots;
    const float* k_head_scale;  // kHeadScale: [n_kv_heads]
    const float* v_head_scale;
    float* k_block_scale;  // kBlockScale: [num_blocks][n_kv_heads], updated
    float* v_block_scale;
    long long qo_stride, q_stride, k_stride, v_stride;  // elements between tokens
    long long pool_slots;
    int n_tokens;
    int n_heads;  // query heads to rotate (0: none)
    int n_kv_heads;
    int rot;
    int max_position;
    int interleaved;
    int rows_per_thread;   // head rows of its token a thread handles
    int row_groups;        // CTAs per token tile
    int kv_ctas;           // kBlockScale: leading CTAs that write K and V
    int tokens_per_warp;   // kBlockScale: tokens a K/V warp looks at
    unsigned int* err;
};

// A token's position: -1 if the token is to be skipped (a negative position,
// or one beyond the table, which is flagged). Without rotation every token is
// taken.
__device__ __forceinline__ int token_position(const RopeParams& P, int t, bool flag) {
    if (P.rot == 0) return 0;
    const int64_t p = P.pos[t];
    if (p < 0) return -1;
    if (p >= P.max_position) {
        if (flag) pa::set_error(P.err, PA_DEVERR_POSITION);
        return -1;
    }
    return (int)p;
}

// The pair of 8-dim chunks (a, b) that lane c of a row's D / 16 lanes holds:
// the two halves of eight rotation pairs, eight whole interleaved pairs each,
// or two chunks past the rotated dims.
__device__ __forceinline__ void chunk_pair(int c, int rot, bool interleaved, int& a, int& b) {
    if (interleaved) {
        a = 2 * c;
        b = a + 1;
    } else if (c < rot / 16) {
        a = c;
        b = c + rot / 16;
    } else {
        a = rot / 8 + 2 * (c - rot / 16);
        b = a + 1;
    }
}

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
    const float4 x = *reinterpret_cast<const float4*>(p), y = *reinterpret_cast<const float4*>(p + 4);
    f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
    f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
}

__device__ __forceinline__ void widen8(const uint4 w, float* f) {
    const float2 a = pa::bf16x2_to_float2(w.x), b = pa::bf16x2_to_float2(w.y);
    const float2 c = pa::bf16x2_to_float2(w.z), d = pa::bf16x2_to_float2(w.w);
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
    f[4] = c.x; f[5] = c.y; f[6] = d.x; f[7] = d.y;
}

__device__ __forceinline__ uint4 narrow8(const float* f) {
    return make_uint4(pa::float2_to_bf16x2(f[0], f[1]), pa::float2_to_bf16x2(f[2], f[3]),
                      pa::float2_to_bf16x2(f[4], f[5]), pa::float2_to_bf16x2(f[6], f[7]));
}

// Eight values -> E4M3 codes (nearest even, saturating at +-448; NaN stays NaN).
__device__ __forceinline__ uint2 codes8(const float* f) {
    uint2 r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r.x)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]));
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r.y)
        : "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
    return r;
}

__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
    const float x = a, y = b;
    a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
    b = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
}

// x[0..7], x[8..15]: the lane's two chunks, rotated in place by its eight angles.
__device__ __forceinline__ void rotate16(float (&x)[16], const float (&cs)[8], const float (&sn)[8], bool interleaved) {
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn_pair(x[2 * i], x[2 * i + 1], cs[i], sn[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn_pair(x[i], x[i + 8], cs[i], sn[i]);
    }
}

// Rows of q (and, in bf16 and per-head mode, of k and v). A CTA takes a tile
// of kThreads / (D / 16) tokens and `rows_per_thread` head rows of each; a
// thread keeps its token's eight angles in registers over its rows, U rows'
// loads in flight at a time.
template <int D, int MODE, int U>
__device__ __forceinline__ void rotate_rows(const RopeParams& P, int cta) {
    constexpr int LPR = D / 16, TPC = kThreads / LPR;
    const int c = threadIdx.x % LPR;
    const long long t64 = (long long)(cta / P.row_groups) * TPC + threadIdx.x / LPR;
    if (t64 >= P.n_tokens) return;
    const int t = (int)t64;
    const int group = cta % P.row_groups;
    const int n_rows = MODE == kBlockScale ? P.n_heads : P.n_heads + 2 * P.n_kv_heads;
    const int r0 = group * P.rows_per_thread, r1 = min(r0 + P.rows_per_thread, n_rows);
    const int pos = token_position(P, t, group == 0 && c == 0);
    if (pos < 0) return;
    const bool il = P.interleaved != 0;
    int ca, cb;
    chunk_pair(c, P.rot, il, ca, cb);
    const bool turn = c < P.rot / 16;
    float cs[8], sn[8];
    if (turn) {
        const float* row = P.cos_sin + (long long)pos * P.rot;
        load8(row + 8 * c, cs);
        load8(row + P.rot / 2 + 8 * c, sn);
    }
    long long slot = -1;
    if (MODE != kBlockScale && r1 > P.n_heads) {
        slot = P.slots[t];
        if (slot >= P.pool_slots) {
            if (c == 0 && r1 == n_rows) pa::set_error(P.err, PA_DEVERR_SLOT);
            slot = -1;
        }
    }
    for (int rb = r0; rb < r1; rb += U) {
        uint4 w[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = rb + u;
            if (r >= r1 || (r >= P.n_heads && slot < 0)) continue;
            const uint16_t* src = r < P.n_heads ? P.q + t * P.q_stride + r * D
                                  : r < P.n_heads + P.n_kv_heads
                                      ? P.k + t * P.k_stride + (r - P.n_heads) * D
                                      : P.v + t * P.v_stride + (r - P.n_heads - P.n_kv_heads) * D;
            w[u][0] = reinterpret_cast<const uint4*>(src)[ca];
            w[u][1] = reinterpret_cast<const uint4*>(src)[cb];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = rb + u;
            if (r >= r1 || (r >= P.n_heads && slot < 0)) continue;
            const bool is_q = r < P.n_heads, is_v = r >= P.n_heads + P.n_kv_heads;
            float x[16];
            if (MODE == kHeadScale || (turn && !is_v)) {
                widen8(w[u][0], x);
                widen8(w[u][1], x + 8);
                if (turn && !is_v) rotate16(x, cs, sn, il);
            }
            if (MODE != kHeadScale || is_q) {
                if (turn && !is_v) {
                    w[u][0] = narrow8(x);
                    w[u][1] = narrow8(x + 8);
                }
                uint16_t* dst;
                if (is_q) {
                    dst = P.q_out + t * P.qo_stride + r * D;
                } else {
                    const int h = is_v ? r - P.n_heads - P.n_kv_heads : r - P.n_heads;
                    dst = reinterpret_cast<uint16_t*>(is_v ? P.v_pool : P.k_pool) +
                          ((slot / kBS * P.n_kv_heads + h) * kBS + slot % kBS) * D;
                }
                reinterpret_cast<uint4*>(dst)[ca] = w[u][0];
                reinterpret_cast<uint4*>(dst)[cb] = w[u][1];
            } else {
                const int h = is_v ? r - P.n_heads - P.n_kv_heads : r - P.n_heads;
                const float s = (is_v ? P.v_head_scale : P.k_head_scale)[h];
                unsigned char* dst = (is_v ? P.v_pool : P.k_pool) +
                                     ((slot / kBS * P.n_kv_heads + h) * kBS + slot % kBS) * D;
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = __fdiv_rn(x[i], s);
                reinterpret_cast<uint2*>(dst)[ca] = codes8(x);
                reinterpret_cast<uint2*>(dst)[cb] = codes8(x + 8);
            }
        }
    }
}

// The smallest 2^e, -32 <= e <= 32, with amax <= 448 * 2^e; 448 = 1.75 * 2^8.
__device__ __forceinline__ float power_scale(float amax) {
    const uint32_t b = __float_as_uint(amax);
    int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = min(32, max(-32, e));
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// K and V of a block-scaled cache. The scale of a (block, head) covers all of
// its tokens, so a call's tokens of one block - a run - belong to one warp, which
// finds their largest magnitude and encodes them. They lie within 16 consecutive
// entries of the call, in any order, skipped entries between them. The entry
// without another of its block in the 15 before it leads, and its warp takes
// those in the 15 behind it. One behind these that an entry of the run precedes
// by less than 16 belongs to nobody: it is not written, and flagged.
// A run with the block's first slot gives the block its scale; any other run
// raises the scale if it must, and then also encodes the block's other tokens
// again. As scales are powers of two, that is exact for every code whose new
// value is not an E4M3 subnormal, and off by at most 2^-10 of the new scale (half
// a subnormal step) there: tokens do not lose a bit each time the block's scale
// grows.
// One warp per (tokens_per_warp tokens, KV head, K or V). Finding the runs by
// their blocks takes 0.1 us of a small call and 2 to 7% of a large one more than
// by slots that follow each other without a gap, where a skipped token left two
// warps with one block. (LARGE: passes without a token are jumped over one by
// one; leaving the loop after the last, as small calls do, spilled 100 bytes.)
template <int D, bool LARGE>
__device__ __forceinline__ void write_block_scaled(const RopeParams& P, int cta) {
    constexpr int LPR = D / 16, TPP = 32 / LPR, NP = kBS / TPP;  // lanes per row, rows per pass, passes
    const int lane = threadIdx.x & 31;
    const long long w = (long long)cta * (kThreads / 32) + (threadIdx.x >> 5);
    const bool is_v = w & 1;
    const int h = (int)((w >> 1) % P.n_kv_heads);
    const long long t0 = (w >> 1) / P.n_kv_heads * P.tokens_per_warp;
    if (t0 >= P.n_tokens) return;
    // The warp's own entries, t0 .. t0 + tokens_per_warp - 1 (at most 16), and those around them: lane l holds
    // entry t0 + l, where every run of its own ends, and of one of the 16 entries before t0 (lanes 0 .. 15) and
    // the 16 from t0 + 32 on (16 .. 31) the block. Block -1: nothing is written.
    const long long e1 = t0 + lane, e2 = lane < 16 ? e1 - 16 : e1 + 16, last = P.n_tokens - 1;
    const bool here = e1 <= last, here2 = e2 >= 0 && e2 <= last;
    const long long t1 = min(e1, last), t2 = max(0LL, min(e2, last));  // no branch before any of the loads
    const int64_t slot = P.slots[t1], slot2 = P.slots[t2];
    int64_t at = 0, at2 = 0;
    if (P.rot > 0) {
        at = P.pos[t1];
        at2 = P.pos[t2];
    }
    const bool mine = here && lane < P.tokens_per_warp;
    if (mine && h == 0 && !is_v) {
        if (slot >= P.pool_slots) pa::set_error(P.err, PA_DEVERR_SLOT);
        if (P.rot > 0 && at >= P.max_position) pa::set_error(P.err, PA_DEVERR_POSITION);
    }
    auto block_of = [&](bool in, int64_t slot, int64_t at) {
        in &= (uint64_t)slot < (uint64_t)P.pool_slots && (P.rot == 0 || (uint64_t)at < (uint64_t)P.max_position);
        return in ? (int)(slot >> 4) : -1;  // slot / kBS
    };
    const int block = block_of(here, slot, at), block2 = block_of(here2, slot2, at2);
    const int off = (int)slot & (kBS - 1), pos = (int)at;
    unsigned todo = __ballot_sync(kFull, mine && block >= 0);
    const bool il = P.interleaved != 0;
    const int c = lane % LPR, tg = lane / LPR;
    int ca, cb;
    chunk_pair(c, P.rot, il, ca, cb);
    const bool turn = !is_v && c < P.rot / 16;
    const uint16_t* src = is_v ? P.v : P.k;
    const long long stride = is_v ? P.v_stride : P.k_stride;
    unsigned char* pool = is_v ? P.v_pool : P.k_pool;
    float* scales = is_v ? P.v_block_scale : P.k_block_scale;
    while (todo) {
        const int l0 = __ffs(todo) - 1;  // 0 .. 15
        const int blk_id = __shfl_sync(kFull, block, l0);
        const unsigned alike = __ballot_sync(kFull, block == blk_id), alike2 = __ballot_sync(kFull, block2 == blk_id);
        todo &= ~alike;
        if ((alike2 & 0xffffu) >> (l0 + 1)) continue;  // an entry before t0 leads
        const unsigned run = alike >> l0 & 0xffffu;    // bit i: entry e0 + i
        const long long e0 = t0 + l0;
        if (((unsigned long long)(alike2 >> 16) << 16 | alike >> 16) >> l0 && lane == 0 && h == 0 && !is_v)
            pa::set_error(P.err, PA_DEVERR_SLOT);
        const bool fresh = __ballot_sync(kFull, off == 0) >> l0 & run;
        const long long tile = (long long)blk_id * P.n_kv_heads + h;
        const float stored = scales[tile];
        // the run's rows are read twice, the second time from L1: holding 16 rotated
        // rows in registers would halve the warps that hide the loads' latency
        auto row_of = [&](int i) { return reinterpret_cast<const uint4*>(src + (e0 + i) * stride + h * D); };
        auto rotated = [&](const uint4 a, const uint4 b, int i, bool use, float (&x)[16]) {  // lanes of a row: entry i
            const int at = __shfl_sync(kFull, pos, l0 + i);
            widen8(a, x);
            widen8(b, x + 8);
            if (turn && use) {
                float cs[8], sn[8];
                const float* row = P.cos_sin + (long long)at * P.rot;
                load8(row + 8 * c, cs);
                load8(row + P.rot / 2 + 8 * c, sn);
                rotate16(x, cs, sn, il);
            }
        };
        float amax = 0.f;  // over finite values
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            if (LARGE && !(run >> (p * TPP) & ((1u << TPP) - 1))) continue;
            if (!LARGE && !(run >> (p * TPP))) break;
            const int i = p * TPP + tg;
            const bool use = run >> i & 1;
            uint4 a = make_uint4(0, 0, 0, 0), b = a;
            if (use) {
                a = row_of(i)[ca];
                b = row_of(i)[cb];
            }
            float x[16];
            rotated(a, b, i, use, x);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float v = fabsf(x[k]);
                if (v < INFINITY) amax = fmaxf(amax, v);
            }
        }
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, m));
        const float need = power_scale(amax);
        // as the attention calls read it: a scale from elsewhere may be out of range or NaN
        const float old = fminf(fmaxf(stored, 0x1p-32f), 0x1p32f);
        // the next power of two of old: the same, unless it is from elsewhere (to divide by any scale, rather
        // than multiply by the exact inverse of a power of two, took 15% longer)
        const float least = __uint_as_float((__float_as_uint(old) + 0x7fffffu) & 0x7f800000u);
        const float s = fresh ? need : fmaxf(least, need);
        const float inv = 1.f / s;  // exact: a power of two
        unsigned char* blk = pool + tile * (kBS * D);
        if (!fresh && s != old) {
            const float ratio = old * inv;
            const unsigned written = __reduce_or_sync(kFull, lane >= l0 && run >> (lane - l0) & 1 ? 1u << off : 0u);  // slots
#pragma unroll
            for (int j = 0; j < kBS * D / 16 / 32; ++j) {
                const int piece = lane + 32 * j, row = piece / (D / 16);
                if (written >> row & 1) continue;
                uint4* at = reinterpret_cast<uint4*>(blk) + piece;
                const uint4 u = *at;
                const uint32_t in[4] = {u.x, u.y, u.z, u.w};
                float f[16];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float2 lo, hi;
                    pa::e4m3x4_to_float2x2(in[k], lo, hi);
                    f[4 * k] = lo.x * ratio;
                    f[4 * k + 1] = lo.y * ratio;
                    f[4 * k + 2] = hi.x * ratio;
                    f[4 * k + 3] = hi.y * ratio;
                }
                const uint2 a = codes8(f), b = codes8(f + 8);
                *at = make_uint4(a.x, a.y, b.x, b.y);
            }
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            if (LARGE && !(run >> (p * TPP) & ((1u << TPP) - 1))) continue;
            if (!LARGE && !(run >> (p * TPP))) break;
            const int i = p * TPP + tg;
            const bool use = run >> i & 1;
            uint4 a = make_uint4(0, 0, 0, 0), b = a;
            if (use) {
                a = row_of(i)[ca];
                b = row_of(i)[cb];
            }
            float x[16];
            rotated(a, b, i, use, x);
            const int to = __shfl_sync(kFull, off, l0 + i);
            if (use) {
#pragma unroll
                for (int k = 0; k < 16; ++k) x[k] *= inv;
                uint2* row = reinterpret_cast<uint2*>(blk + to * D);
                row[ca] = codes8(x);
                row[cb] = codes8(x + 8);
            }
        }
        if (lane == 0) scales[tile] = s;
    }
}

// Two forms of each kernel. A small call is one wave of short-lived CTAs, where
// spilled registers would only add latency: up to 102 registers a thread, four
// rows in flight. A large one is bound by HBM (K/V warps: by latency) and wants
// warps: 80 registers, or 64 and two rows in flight for the block-scaled
// cache, whatever spills. Measured small / large (64 / 8,192 tokens of 64/8
// heads of 128 in bf16; 64 tokens / 6,742 in ragged chunks of 32/8 heads in
// E4M3): 2.2 / 54.1 us and 2.9 / 35.4 us in the first form, 2.4 / 52.6 and 3.8 /
// 30.8 in the second (E4M3 before runs were found by block: 3.0 and 32.0 us now).
template <int MODE, bool LARGE>
struct Form {
    static constexpr int U = LARGE && MODE == kBlockScale ? 2 : 4;
    static constexpr int kCtasPerSm = !LARGE ? 5 : MODE == kBlockScale ? 8 : 6;
};

template <int D, int MODE, bool LARGE>
__global__ void __launch_bounds__(kThreads, Form<MODE, LARGE>::kCtasPerSm) rope_cache_kernel(const RopeParams P) {
    pa::launch_dependents();     // the next kernel (decode, prefill) may be scheduled
    pa::grid_dependency_wait();  // earlier readers and writers of q and the pool are complete
    int cta = blockIdx.x;
    if (MODE == kBlockScale) {
        if (cta < P.kv_ctas) {
            write_block_scaled<D, LARGE>(P, cta);
            return;
        }
        cta -= P.kv_ctas;
    }
    rotate_rows<D, MODE, Form<MODE, LARGE>::U>(P, cta);
}

int sm_count() {
    static int cached[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (!cached[dev]) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        cached[dev] = n;  // every thread that races here writes the same value
    }
    return cached[dev];
}

bool stride_ok(long long stride, int heads, int head_dim) {
    return stride >= (long long)heads * head_dim && stride % 8 == 0;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <int D, int MODE>
int launch(RopeParams& P, cudaStream_t stream) {
    constexpr int TPC = kThreads / (D / 16), kWarps = kThreads / 32;
    const int sms = sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    const long long tiles = ((long long)P.n_tokens + TPC - 1) / TPC;
    const int n_rows = MODE == kBlockScale ? P.n_heads : P.n_heads + 2 * P.n_kv_heads;
    // one row a thread while that still fits in one wave of 16 CTAs per SM;
    // beyond it eight, which read a token's angles an eighth as often
    const bool large = tiles * (P.n_heads + 2LL * P.n_kv_heads) > 16LL * sms;
    P.rows_per_thread = large ? 8 : 1;
    P.row_groups = (n_rows + P.rows_per_thread - 1) / P.rows_per_thread;
    long long ctas = tiles * P.row_groups, kv = 0;
    if (MODE == kBlockScale) {
        const long long units = 2LL * P.n_kv_heads;
        // K/V warps look at one token each while that is one wave of them. Beyond it a warp
        // takes several: 16 suit prompt chunks, where a warp finds one run (6,742 tokens: 32.0 us,
        // 35 with 4), but a decode batch has a run per token and its warps would work through
        // 16 of them (1,024 and 2,048 sequences: 38.1 and 44.0 us, 12.8 and 24.4 with 4). The
        // host cannot tell one from the other, so calls that can still be a batch take 4, which
        // costs a prompt of 2,048 tokens 4% and one of 4,096 15% (13.2 and 23.5 us, 12.8 and
        // 20.4 with 16).
        P.tokens_per_warp = P.n_tokens * units <= 16LL * kWarps * sms ? 1 : P.n_tokens <= 4096 ? 4 : 16;
        const long long warps = ((long long)P.n_tokens + P.tokens_per_warp - 1) / P.tokens_per_warp * units;
        kv = (warps + kWarps - 1) / kWarps;
    }
    if (ctas + kv > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    P.kv_ctas = (int)kv;
    const dim3 grid((unsigned)(ctas + kv));
    return large ? pa_launch_pdl(rope_cache_kernel<D, MODE, true>, grid, dim3(kThreads), 0, stream, P)
                 : pa_launch_pdl(rope_cache_kernel<D, MODE, false>, grid, dim3(kThreads), 0, stream, P);
}

template <int MODE>
int rope_impl(RopeParams& P, int head_dim, int block_size, int num_blocks, pa_stream_t stream) {
    if (P.n_tokens < 0 || P.n_kv_heads <= 0 || num_blocks < 0 || P.rot < 0 || P.max_position < 0) return PA_ERR_INVALID_ARG;
    if (block_size != kBS || (head_dim != 64 && head_dim != 128)) return PA_ERR_UNSUPPORTED;
    if (P.rot > head_dim) return PA_ERR_INVALID_ARG;
    if (P.rot % 16 != 0) return PA_ERR_UNSUPPORTED;
    if ((P.q == nullptr) != (P.q_out == nullptr)) return PA_ERR_INVALID_ARG;
    if (P.q && P.n_heads <= 0) return PA_ERR_INVALID_ARG;
    if (P.n_tokens == 0) return PA_OK;
    if (!P.k || !P.v || !P.k_pool || !P.v_pool || !P.slots) return PA_ERR_INVALID_ARG;
    if (P.rot > 0 && (!P.cos_sin || !P.pos || !pa_aligned16(P.cos_sin) || !aligned(P.pos, 8))) return PA_ERR_INVALID_ARG;
    if (!pa_aligned16(P.k) || !pa_aligned16(P.v) || !pa_aligned16(P.k_pool) || !pa_aligned16(P.v_pool) ||
        !aligned(P.slots, 8))
        return PA_ERR_INVALID_ARG;
    if (!stride_ok(P.k_stride, P.n_kv_heads, head_dim) || !stride_ok(P.v_stride, P.n_kv_heads, head_dim))
        return PA_ERR_INVALID_ARG;
    if (P.q) {
        if (!pa_aligned16(P.q) || !pa_aligned16(P.q_out) || !stride_ok(P.q_stride, P.n_heads, head_dim) ||
            !stride_ok(P.qo_stride, P.n_heads, head_dim) || (P.q == P.q_out && P.q_stride != P.qo_stride))
            return PA_ERR_INVALID_ARG;
    } else {
        P.n_heads = 0;
    }
    // K's and V's warps work on one block at the same time
    if (MODE == kBlockScale && (P.k_pool == P.v_pool || P.k_block_scale == P.v_block_scale)) return PA_ERR_INVALID_ARG;
    P.pool_slots = (long long)num_blocks * kBS;
    P.err = pa_device_error_ptr();
    if (!P.err) return PA_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return head_dim == 128 ? launch<128, MODE>(P, s) : launch<64, MODE>(P, s);
}

RopeParams make_params(void* q_out, const void* q, const void* k, const void* v, void* k_pool, void* v_pool,
                       const float* cos_sin, const int64_t* positions, const int64_t* slot_mapping,
                       int64_t q_out_stride, int64_t q_stride, int64_t k_stride, int64_t v_stride, int n_tokens,
                       int n_heads, int n_kv_heads, int rot_dim, int max_position, int interleaved) {
    RopeParams P = {};
    P.q_out = static_cast<uint16_t*>(q_out);
    P.q = static_cast<const uint16_t*>(q);
    P.k = static_cast<const uint16_t*>(k);
    P.v = static_cast<const uint16_t*>(v);
    P.k_pool = static_cast<unsigned char*>(k_pool);
    P.v_pool = static_cast<unsigned char*>(v_pool);
    P.cos_sin = cos_sin;
    P.pos = positions;
    P.slots = slot_mapping;
    P.qo_stride = q_out_stride;
    P.q_stride = q_stride;
    P.k_stride = k_stride;
    P.v_stride = v_stride;
    P.n_tokens = n_tokens;
    P.n_heads = n_heads;
    P.n_kv_heads = n_kv_heads;
    P.rot = rot_dim;
    P.max_position = max_position;
    P.interleaved = interleaved;
    return P;
}

}  // namespace

extern "C" int pa_rope_and_cache(void* q_out, const void* q, const void* k, const void* v, void* k_pool, void* v_pool,
                                 const float* cos_sin, const int64_t* positions, const int64_t* slot_mapping,
                                 const float* k_scale, const float* v_scale, int64_t q_out_stride, int64_t q_stride,
                                 int64_t k_stride, int64_t v_stride, int n_tokens, int n_heads, int n_kv_heads,
                                 int head_dim, int rot_dim, int max_position, int interleaved, int block_size,
                                 int num_blocks, pa_stream_t stream) {
    RopeParams P = make_params(q_out, q, k, v, k_pool, v_pool, cos_sin, positions, slot_mapping, q_out_stride, q_stride,
                               k_stride, v_stride, n_tokens, n_heads, n_kv_heads, rot_dim, max_position, interleaved);
    if ((k_scale == nullptr) != (v_scale == nullptr)) return PA_ERR_INVALID_ARG;
    if (!k_scale) return rope_impl<kBf16>(P, head_dim, block_size, num_blocks, stream);
    if (!aligned(k_scale, 4) || !aligned(v_scale, 4)) return PA_ERR_INVALID_ARG;
    P.k_head_scale = k_scale;
    P.v_head_scale = v_scale;
    return rope_impl<kHeadScale>(P, head_dim, block_size, num_blocks, stream);
}

extern "C" int pa_rope_and_cache_fp8_block(void* q_out, const void* q, const void* k, const void* v, void* k_pool,
                                           void* v_pool, float* k_scale, float* v_scale, const float* cos_sin,
                                           const int64_t* positions, const int64_t* slot_mapping, int64_t q_out_stride,
                                           int64_t q_stride, int64_t k_stride, int64_t v_stride, int n_tokens,
                                           int n_heads, int n_kv_heads, int head_dim, int rot_dim, int max_position,
                                           int interleaved, int block_size, int num_blocks, pa_stream_t stream) {
    RopeParams P = make_params(q_out, q, k, v, k_pool, v_pool, cos_sin, positions, slot_mapping, q_out_stride, q_stride,
                               k_stride, v_stride, n_tokens, n_heads, n_kv_heads, rot_dim, max_position, interleaved);
    if (n_tokens > 0 && (!k_scale || !v_scale || !aligned(k_scale, 4) || !aligned(v_scale, 4))) return PA_ERR_INVALID_ARG;
    P.k_block_scale = k_scale;
    P.v_block_scale = v_scale;
    return rope_impl<kBlockScale>(P, head_dim, block_size, num_blocks, stream);
}
