// Compaction of paged sequences: the tokens that stay move, in place, to the
// sequence's first positions, so that its last blocks come free
// ("Inference serving: the KV-cache machine", section "Paged KV: virtual memory for
// tokens": blocks are the unit that is freed; a token dropped from the middle of a
// block frees nothing until those that stay are moved together).
//
//     new position j of a sequence := its old position keep[j],  keep ascending,
// for K and V, for every KV head (or by a list for each one).
//
// In place and without a copy of the cache: keep[j] >= j, so whoever writes position j
// last reads from positions >= j. A CTA, or a cluster of CTAs that share a step's
// tokens, takes one (sequence, KV head, K or V) from the first position on, a step of
// tokens at a time: a step is stored when all of its tokens are loaded (a barrier of the
// cluster), and later steps read only positions beyond those it writes, so their loads
// are in flight meanwhile. No CTA waits for one that may not be running. Positions before
// the block of the first moved one (keep[j] == j) are not touched.
//
// With block-scaled E4M3 a block takes the largest scale of its new tokens and codes
// of tokens from quieter blocks are encoded again: code * old / new, exact unless the
// result is an E4M3 subnormal (scales are powers of two). A step's scales are read
// before the barrier of an earlier step, and so before any that it reads is replaced.
//
// Bound by HBM: every moved byte is read once and written once. 32 chats of 2,000 to
// 8,192 tokens that keep a third, a list for each of 8 heads (128 dims, bf16): 72 us,
// 5.5 TB/s, 0.81 of a copy. One document of 131,072 tokens that keeps 0.6: 108 us,
// 6.0 TB/s (16 clusters of 12; a CTA for each slice of the rows' columns, each with all the
// look-ups, took 302). 6 documents of 23,000 to 65,000 tokens in block-scaled E4M3: 84 us,
// 5.4 TB/s. 100 chats, a list for all heads: 143 us, 6.3 TB/s.
#include "compact_clusters.h"
#include "pa_common.cuh"

namespace {

constexpr int kBS = 16;
constexpr int kThreads = 256;
constexpr int kUnroll = 8;    // 16-byte copies a thread and step
// Steps in the ring of copies: two CTAs' rings and notes fill an SM's shared memory. Rows of
// 64 bytes with block scales are more tokens a step, with more notes (64 chats of 2,000 to
// 8,000 tokens: 83 us, 119 with three steps and one CTA an SM).
template <int C, bool BSC>
constexpr int kSteps = BSC && C == 4 ? 2 : 3;
constexpr int kNotes = 8;     // steps whose places are held
constexpr uint32_t kNone = 0xffffffffu;
constexpr unsigned kFull = 0xffffffffu;

struct CompactParams {
    unsigned char* pool[2];  // K, V
    float* scale[2];
    int n_kept;
    const int32_t* tables;
    const int32_t* keep;
    const int32_t* starts;
    long long keep_stride;  // from one KV head's list to the next; 0: one list
    int n_kv_heads;
    int max_blocks;
    int num_blocks;
    unsigned int* err;
};

__device__ __forceinline__ float clamp_scale(float s) { return fminf(fmaxf(s, 0x1p-32f), 0x1p32f); }

// Four E4M3 codes times f, each rounded to nearest even once.
__device__ __forceinline__ uint32_t scale_codes(uint32_t w, float f) {
    float2 a, b;
    pa::e4m3x4_to_float2x2(w, a, b);
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 t;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 t, %2, %1;\n\t"
        "cvt.u32.u16 %0, t;\n\t}"
        : "=r"(lo)
        : "f"(a.x * f), "f"(a.y * f));
    asm("{\n\t.reg .b16 t;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 t, %2, %1;\n\t"
        "cvt.u32.u16 %0, t;\n\t}"
        : "=r"(hi)
        : "f"(b.x * f), "f"(b.y * f));
    return lo | (hi << 16);
}

// A barrier of the cluster's threads, in two halves. Nothing is published by it: what it
// orders are copies that have arrived, before the arrival, against stores after the wait.
// (A releasing arrival waits until a thread's earlier stores are performed, a round trip
// a step.)
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait;" ::: "memory"); }

// The first position of a list that moves (n: none does). Whether keep[j] == j holds
// for a leading part of an ascending list only, so samples narrow it down by the
// number of threads a round. Every thread of the CTA calls; all get the same answer.
__device__ int first_moved(const int32_t* keep, int n) {
    int lo = 0, len = n;  // the answer lies in [lo, lo + len]
    if (n > kThreads) {   // the usual place is near the beginning
        const int stays = __syncthreads_count(keep[threadIdx.x] == (int)threadIdx.x);
        if (stays < kThreads) return stays;
        lo = kThreads;
        len = n - kThreads;
    }
    while (len > 0) {
        const int step = (len + kThreads - 1) / kThreads;
        const long long at = (long long)threadIdx.x * step;
        const int stays = __syncthreads_count(at < len && keep[lo + at] == lo + (int)at);
        if (step == 1) return lo + stays;
        // sample `stays` is the first that moved (or lies behind the end), the one before did not
        if (stays == 0) return lo;
        const int a = (stays - 1) * step, b = min((long long)stays * step, (long long)len);
        lo += a + 1;
        len = b - a - 1;
    }
    return lo;
}

// Whether one of the positions j < n that this thread looks at, as one of `threads`, is not j. Sixteen are
// in flight, four a load (8 sequences of 131,008 tokens of which the last 16 move: 9.8 us, a list for each of 8
// heads 12.2; without a look 8.7).
__device__ bool changed(const int32_t* keep, int n, int thread, int threads) {
    const int lead = min(n, (int)(-(reinterpret_cast<uintptr_t>(keep) >> 2) & 3)), quads = (n - lead) / 4;
    const int4* four = reinterpret_cast<const int4*>(keep + lead);
    bool bad = false;
    auto differs = [&](long long i) {
        const int4 v = four[i];
        const int j = lead + 4 * (int)i;
        return v.x != j || v.y != j + 1 || v.z != j + 2 || v.w != j + 3;
    };
    long long i = thread;
    for (; i + 3LL * threads < quads; i += 4LL * threads) {
        const bool a = differs(i), b = differs(i + threads), c = differs(i + 2LL * threads), d = differs(i + 3LL * threads);
        bad |= a | b | c | d;
    }
    for (; i < quads; i += threads) bad |= differs(i);
    const int j = thread < lead ? thread : thread + 4 * quads;  // the ends, up to three each
    return bad || (j < n && keep[j] != j);
}

// C: 16-byte chunks of a row; grid (CTAs of a cluster, 2 * KV heads, sequences).
template <int C, bool BSC>
__global__ void __launch_bounds__(kThreads, 2) compact_blocks_kernel(const CompactParams P) {
    constexpr int kPerPass = kThreads / C, T = kPerPass * kUnroll;  // tokens a pass, a CTA's share of a step
    constexpr int F = (T + kThreads - 1) / kThreads;                // tokens a thread looks up a step
    constexpr int kRow = C * 16, S = kSteps<C, BSC>;                // bytes of a row, steps of the ring
    __shared__ uint32_t src[kNotes][T], dst[kNotes][T / kBS];       // rows of the pool (dst: a block's first) or kNone
    __shared__ float factor[BSC ? kNotes : 1][BSC ? T : 1], new_scale[BSC ? kNotes : 1][BSC ? T / kBS : 1];
    extern __shared__ __align__(16) uint4 ring[];                   // [S][kUnroll][kThreads]
    static_assert(kNotes >= S + 2, "places noted S steps ahead replace those of a step that all have stored");
    const int tid = threadIdx.x, side = blockIdx.y & 1, h = blockIdx.y >> 1, b = blockIdx.z;
    pa::launch_dependents();
    pa::grid_dependency_wait();
    const int first = P.starts[b], end = P.starts[b + 1];
    // every CTA of a cluster takes the same branches: they share the sequence and the head
    if (first < 0 || end < first || end > P.n_kept) {
        if (tid == 0) pa::set_error(P.err, PA_DEVERR_POSITION);
        return;
    }
    const int n = end - first;
    if (n == 0) return;
    const int32_t* keep = P.keep + h * P.keep_stride + first;
    const int32_t* table = P.tables + (size_t)b * P.max_blocks;
    const int moved = first_moved(keep, n);
    // What stays is looked at too, as the search went by samples.
    const int still = moved >= n ? n : moved / kBS * kBS;
    // (A list for all heads is shared out among them.)
    const int part = (P.keep_stride ? 0 : h * (int)gridDim.x * 2) + blockIdx.x * 2 + side;
    const int parts = gridDim.x * 2 * (P.keep_stride ? 1 : P.n_kv_heads);
    if (changed(keep, still, part * kThreads + tid, parts * kThreads) || (tid == 0 && (still - 1) / kBS >= P.max_blocks))
        pa::set_error(P.err, PA_DEVERR_POSITION);
    if (moved >= n) return;
    const int stride = (int)gridDim.x * T;  // tokens of a step
    const int j0 = moved / kBS * kBS + (int)blockIdx.x * T;
    const int steps = (int)(((long long)n - moved / kBS * kBS + stride - 1) / stride);
    unsigned char* pool = side ? P.pool[1] : P.pool[0];
    float* scales = side ? P.scale[1] : P.scale[0];

    // Where the tokens of a step come from and go to: list, table and scale are three loads deep, so
    // each is issued a step after the one it needs, and none is waited for at once.
    int kept[F], before[F];
    int from[F], src_block[F], dst_block[F];
    int from2[F], src2[F], dst2[F];
    float scale[F];
    auto position = [&](int s, int f) {  // of the token, or -1
        const int t = f * kThreads + tid;
        const long long j = j0 + (long long)s * stride + t;
        return s < steps && t < T && j < n ? (int)j : -1;
    };
    auto ask_list = [&](int s) {
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const int j = position(s, f);
            kept[f] = j >= 0 ? keep[j] : -1;
            before[f] = j > 0 ? keep[j - 1] : -1;
        }
    };
    auto ask_table = [&](int s) {
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const int j = position(s, f), k = kept[f];
            const bool good = j >= 0 && k >= j && k > before[f] && k / kBS < P.max_blocks;
            if (j >= 0 && !good) pa::set_error(P.err, PA_DEVERR_POSITION);
            from[f] = good ? k % kBS : -1;
            src_block[f] = good ? table[k / kBS] : 0;
            dst_block[f] = good ? table[j / kBS] : 0;
        }
    };
    auto ask_scale = [&]() {
#pragma unroll
        for (int f = 0; f < F; ++f) {
            from2[f] = from[f];
            src2[f] = src_block[f];
            dst2[f] = dst_block[f];
            if (from2[f] >= 0 && !(src2[f] >= 0 && src2[f] < P.num_blocks && dst2[f] >= 0 && dst2[f] < P.num_blocks)) {
                pa::set_error(P.err, PA_DEVERR_BLOCK_ID);
                from2[f] = -1;
            }
            if constexpr (BSC) scale[f] = from2[f] >= 0 ? scales[(size_t)src2[f] * P.n_kv_heads + h] : 0.f;
        }
    };
    auto note = [&](int s) {
        const int buf = s % kNotes;
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const int t = f * kThreads + tid;
            if (T < kThreads && t >= T) break;  // whole warps
            src[buf][t] = from2[f] >= 0 ? ((uint32_t)src2[f] * P.n_kv_heads + h) * kBS + from2[f] : kNone;
            // the block's first good token (all of them have the same destination) notes it
            const unsigned good = __ballot_sync(kFull, from2[f] >= 0) & (0xffffu << (tid & 16));
            if (good && (tid & 31) == __ffs(good) - 1) dst[buf][t / kBS] = ((uint32_t)dst2[f] * P.n_kv_heads + h) * kBS;
            if constexpr (BSC) {
                const float old = from2[f] >= 0 ? clamp_scale(scale[f]) : 0.f;
                float most = old;
#pragma unroll
                for (int o = 1; o < kBS; o <<= 1) most = fmaxf(most, __shfl_xor_sync(kFull, most, o));
                factor[buf][t] = old == most ? 1.f : __fdiv_rn(old, most);
                if (t % kBS == 0) new_scale[buf][t / kBS] = most;
            }
        }
    };
    const int c = tid % C, tp = tid / C;
    unsigned char* column = pool + c * 16;
    auto load = [&](int s) {  // a thread's chunks of a step into its places of the ring
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint32_t row = s < steps ? src[s % kNotes][u * kPerPass + tp] : kNone;
            if (row != kNone)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(pa::smem_u32(&ring[(s % S * kUnroll + u) * kThreads + tid])),
                             "l"(column + (size_t)row * kRow)
                             : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto store = [&](int s) {
        const int buf = s % kNotes;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int t = u * kPerPass + tp;
            if (src[buf][t] == kNone) continue;
            uint4 v = ring[(s % S * kUnroll + u) * kThreads + tid];
            if constexpr (BSC) {
                const float f = factor[buf][t];
                if (f != 1.f) v = make_uint4(scale_codes(v.x, f), scale_codes(v.y, f), scale_codes(v.z, f), scale_codes(v.w, f));
            }
            *reinterpret_cast<uint4*>(column + (size_t)(dst[buf][t / kBS] + tp % kBS) * kRow) = v;
        }
        if constexpr (BSC) {
            if (tid < T / kBS && new_scale[buf][tid] > 0.f) scales[dst[buf][tid] / kBS] = new_scale[buf][tid];  // [block][KV head]
        }
    };
    // During step s: its tokens are stored; copies of the next S - 1 are in flight; the places of step
    // s + S are noted, its successors looked up.
    ask_list(0);
    ask_table(0);
    ask_list(1);
    ask_scale();
    ask_table(1);
    ask_list(2);
#pragma unroll 1
    for (int s = 0; s < S; ++s) {
        note(s);
        ask_scale();
        ask_table(s + 2);
        ask_list(s + 3);
    }
    __syncthreads();
#pragma unroll 1
    for (int s = 0; s < S - 1; ++s) load(s);
#pragma unroll 1
    for (int s = 0; s < steps; ++s) {
        note(s + S);
        ask_scale();
        ask_table(s + S + 2);
        ask_list(s + S + 3);
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");  // this thread's part of step s is here
        __syncthreads();  // and every thread's, and the notes
        if (gridDim.x > 1) cluster_arrive();
        load(s + S - 1);
        if (gridDim.x > 1) cluster_wait();
        store(s);
    }
}

template <int C, bool BSC>
int launch_compact(const CompactParams& P, int sms, int n_seqs, cudaStream_t stream) {
    auto kern = compact_blocks_kernel<C, BSC>;
    constexpr int kRing = kSteps<C, BSC> * kUnroll * kThreads * 16;
    cudaLaunchConfig_t cfg = {};
    cfg.dynamicSmemBytes = kRing;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    static int largest_of[64] = {0};  // clusters that the device's context holds (above 8: not everywhere); 0: not asked yet
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PA_ERR_CUDA;
    int largest = largest_of[dev];
    if (!largest) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing) != cudaSuccess ||
            cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
            return PA_ERR_CUDA;
        cfg.numAttrs = 1;
        for (largest = 16; largest > 1; --largest) {
            int fit = 0;
            cfg.gridDim = dim3(largest);
            attr[0].val.clusterDim.x = largest;
            const cudaError_t asked = cudaOccupancyMaxActiveClusters(&fit, kern, &cfg);
            if (asked == cudaSuccess && fit > 0) break;
            if (asked != cudaSuccess) cudaGetLastError();  // a size that the device does not know
        }
        largest_of[dev] = largest;
    }
    const int ctas = pa_compact_ctas(2LL * P.n_kv_heads * n_seqs, sms, P.n_kept, n_seqs, kThreads / C * kUnroll, largest);
    cfg.gridDim = dim3(ctas, 2 * P.n_kv_heads, n_seqs);
    attr[0].val.clusterDim.x = ctas;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, P) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int sm_count() {
    static int cached[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (!cached[dev] && cudaDeviceGetAttribute(&cached[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) cached[dev] = 0;
    return cached[dev];
}

}  // namespace

extern "C" int pa_compact_blocks(void* k_pool, void* v_pool, float* k_scale, float* v_scale, const int32_t* block_tables,
                                 const int32_t* keep, const int32_t* keep_start_loc, int keep_heads, int n_kept,
                                 int n_kv_heads, int head_dim, int block_size, int elem_bytes, int n_seqs,
                                 int max_blocks_per_seq, int num_blocks, pa_stream_t stream) {
    if (n_seqs < 0 || n_kept < 0 || n_kv_heads <= 0 || head_dim <= 0 || num_blocks < 0 || max_blocks_per_seq < 0 ||
        (keep_heads != 1 && keep_heads != n_kv_heads) || (elem_bytes != 1 && elem_bytes != 2) ||
        (k_scale == nullptr) != (v_scale == nullptr) || (k_scale && elem_bytes != 1))
        return PA_ERR_INVALID_ARG;
    if (block_size != kBS || (head_dim != 64 && head_dim != 128)) return PA_ERR_UNSUPPORTED;
    if (n_kv_heads > 32767 || n_seqs > 65535 || (long long)num_blocks * n_kv_heads * kBS >= (long long)kNone) return PA_ERR_UNSUPPORTED;
    if (n_seqs == 0 || n_kept == 0) return PA_OK;
    if (!k_pool || !v_pool || !block_tables || !keep || !keep_start_loc) return PA_ERR_INVALID_ARG;
    if (!pa_aligned16(k_pool) || !pa_aligned16(v_pool) || k_pool == v_pool || (k_scale && k_scale == v_scale) ||
        ((reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale) | reinterpret_cast<uintptr_t>(block_tables) |
          reinterpret_cast<uintptr_t>(keep) | reinterpret_cast<uintptr_t>(keep_start_loc)) & 3u))
        return PA_ERR_INVALID_ARG;
    unsigned int* err = pa_device_error_ptr();
    const int sms = sm_count();
    if (!err || sms <= 0) return PA_ERR_CUDA;
    CompactParams P;
    P.pool[0] = static_cast<unsigned char*>(k_pool);
    P.pool[1] = static_cast<unsigned char*>(v_pool);
    P.scale[0] = k_scale;
    P.scale[1] = v_scale;
    P.n_kept = n_kept;
    P.tables = block_tables;
    P.keep = keep;
    P.starts = keep_start_loc;
    P.keep_stride = keep_heads > 1 ? n_kept : 0;
    P.n_kv_heads = n_kv_heads;
    P.max_blocks = max_blocks_per_seq;
    P.num_blocks = num_blocks;
    P.err = err;
    const int chunks = head_dim * elem_bytes / 16;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (k_scale) return chunks == 8 ? launch_compact<8, true>(P, sms, n_seqs, st) : launch_compact<4, true>(P, sms, n_seqs, st);
    switch (chunks) {
        case 4: return launch_compact<4, false>(P, sms, n_seqs, st);
        case 8: return launch_compact<8, false>(P, sms, n_seqs, st);
        default: return launch_compact<16, false>(P, sms, n_seqs, st);
    }
}
