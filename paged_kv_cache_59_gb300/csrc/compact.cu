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
// last reads from positions >= j. A CTA takes one (sequence, KV head, K or V) - or a
// slice of the rows' columns, which move independently - from the first position on, a
// step of T tokens at a time: step s is stored after every thread has loaded steps up
// to s + 1, and later steps read only positions beyond those that step s writes. So no
// CTA waits for another, and a step's loads are in flight while the one before is
// stored. Positions before the first moved one (keep[j] == j) are not touched.
//
// With block-scaled E4M3 a block takes the largest scale of its new tokens and codes
// of tokens from quieter blocks are encoded again: code * old / new, exact unless the
// result is an E4M3 subnormal (scales are powers of two). Column slices of one head
// then form a cluster, so that no slice's block scales are replaced while another reads
// them.
#include "pa_common.cuh"

namespace {

constexpr int kBS = 16;
constexpr int kThreads = 256;
constexpr int kUnroll = 8;  // 16-byte loads in flight a thread and step
constexpr uint32_t kNone = 0xffffffffu;
constexpr unsigned kFull = 0xffffffffu;

struct CompactParams {
    unsigned char* pool[2];  // K, V
    float* scale[2];
    const int32_t* tables;
    const int32_t* keep;
    const int32_t* starts;
    long long keep_stride;  // from one KV head's list to the next; 0: one list
    int n_kv_heads;
    int row_bytes;
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

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

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

// C: 16-byte chunks of a row that the CTA moves; grid (column slices, 2 * KV heads, sequences).
template <int C, bool BSC>
__global__ void __launch_bounds__(kThreads, 2) compact_blocks_kernel(const CompactParams P) {
    constexpr int kPerPass = kThreads / C, T = kPerPass * kUnroll;  // tokens a pass, a step
    __shared__ uint32_t src[4][T], dst[4][T];                       // slots (block * 16 + offset) or kNone
    __shared__ float factor[BSC ? 4 : 1][BSC ? T : 1], new_scale[BSC ? 4 : 1][BSC ? T / kBS : 1];
    const int tid = threadIdx.x, side = blockIdx.y & 1, h = blockIdx.y >> 1, b = blockIdx.z;
    pa::launch_dependents();
    pa::grid_dependency_wait();
    const int first = P.starts[b], n = P.starts[b + 1] - first;
    // every CTA of a cluster takes the same branches: they share the sequence and the head
    if (n <= 0) return;
    const int32_t* keep = P.keep + h * P.keep_stride + first;
    const int32_t* table = P.tables + (size_t)b * P.max_blocks;
    const int moved = first_moved(keep, n);
    if (moved >= n) return;
    const int j0 = moved / kBS * kBS;
    const int steps = (n - j0 + T - 1) / T;
    unsigned char* pool = side ? P.pool[1] : P.pool[0];
    float* scales = side ? P.scale[1] : P.scale[0];

    // where the tokens of a step come from and go to
    auto fetch = [&](int s) {
        const int buf = s & 3;
#pragma unroll
        for (int t0 = 0; t0 < T; t0 += kThreads) {
            const int t = t0 + tid;
            if (T < kThreads && t >= T) break;  // whole warps
            const int j = j0 + s * T + t;
            uint32_t from = kNone, to = kNone;
            float old = 0.f;
            if (s < steps && j < n) {
                const int k = keep[j], before = j > 0 ? keep[j - 1] : -1;
                if (k < j || k <= before || k / kBS >= P.max_blocks) {
                    pa::set_error(P.err, PA_DEVERR_POSITION);
                } else {
                    const int sb = table[k / kBS], db = table[j / kBS];
                    if (sb < 0 || sb >= P.num_blocks || db < 0 || db >= P.num_blocks) {
                        pa::set_error(P.err, PA_DEVERR_BLOCK_ID);
                    } else {
                        from = (uint32_t)sb * kBS + k % kBS;
                        to = (uint32_t)db * kBS + j % kBS;
                        if constexpr (BSC) old = clamp_scale(scales[(size_t)sb * P.n_kv_heads + h]);
                    }
                }
            }
            src[buf][t] = from;
            dst[buf][t] = to;
            if constexpr (BSC) {
                float most = old;
#pragma unroll
                for (int o = 1; o < kBS; o <<= 1) most = fmaxf(most, __shfl_xor_sync(kFull, most, o));
                factor[buf][t] = old == most ? 1.f : __fdiv_rn(old, most);
                if (t % kBS == 0) new_scale[buf][t / kBS] = most;
            }
        }
    };
    const int c = tid % C, tp = tid / C;
    const size_t column = (size_t)blockIdx.x * (C * 16) + c * 16;
    auto row = [&](uint32_t slot) {
        return pool + (((size_t)(slot / kBS) * P.n_kv_heads + h) * kBS + slot % kBS) * P.row_bytes + column;
    };
    auto load = [&](int s, uint4 (&v)[kUnroll]) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint32_t from = src[s & 3][u * kPerPass + tp];
            v[u] = from != kNone ? __ldcg(reinterpret_cast<const uint4*>(row(from))) : make_uint4(0, 0, 0, 0);
        }
    };
    auto store = [&](int s, uint4 (&v)[kUnroll]) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int t = u * kPerPass + tp;
            const uint32_t to = dst[s & 3][t];
            if (to == kNone) continue;
            if constexpr (BSC) {
                const float f = factor[s & 3][t];
                if (f != 1.f) v[u] = make_uint4(scale_codes(v[u].x, f), scale_codes(v[u].y, f), scale_codes(v[u].z, f), scale_codes(v[u].w, f));
            }
            *reinterpret_cast<uint4*>(row(to)) = v[u];
        }
        if constexpr (BSC) {
            if (blockIdx.x == 0 && tid < T / kBS && new_scale[s & 3][tid] > 0.f) {
                // a token of the block is valid, so the block is in the table's and the pool's range
                const int db = table[(j0 + s * T) / kBS + tid];
                scales[(size_t)db * P.n_kv_heads + h] = new_scale[s & 3][tid];
            }
        }
    };
    // Buffer s & 3 is filled two steps ahead and read until step s is stored, a barrier before it is filled again.
    auto sync = [&]() {
        if constexpr (BSC) cluster_sync();
        else __syncthreads();
    };
    uint4 even[kUnroll], odd[kUnroll];
    fetch(0);
    fetch(1);
    __syncthreads();
    load(0, even);
    for (int s = 0; s < steps; s += 2) {
        load(s + 1, odd);
        fetch(s + 2);
        sync();
        store(s, even);
        if (s + 1 < steps) {
            load(s + 2, even);
            fetch(s + 3);
            sync();
            store(s + 1, odd);
        }
    }
}

template <int C, bool BSC>
int launch_compact(const CompactParams& P, int slices, int n_seqs, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(slices, 2 * P.n_kv_heads, n_seqs);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = slices;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = BSC ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, compact_blocks_kernel<C, BSC>, P) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
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
    if (n_kv_heads > 32767 || n_seqs > 65535 || (long long)num_blocks * kBS >= (long long)kNone) return PA_ERR_UNSUPPORTED;
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
    P.tables = block_tables;
    P.keep = keep;
    P.starts = keep_start_loc;
    P.keep_stride = keep_heads > 1 ? n_kept : 0;
    P.n_kv_heads = n_kv_heads;
    P.row_bytes = head_dim * elem_bytes;
    P.max_blocks = max_blocks_per_seq;
    P.num_blocks = num_blocks;
    P.err = err;
    // Few (sequence, head, K or V) are sliced by columns until there are two CTAs for each SM: rows of
    // 64 bytes at the least with block scales, 32 without.
    int chunks = P.row_bytes / 16, slices = 1;
    const int least = k_scale ? 4 : 2;
    while (chunks > least && 2LL * n_kv_heads * n_seqs * slices < 2LL * sms) {
        chunks /= 2;
        slices *= 2;
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (k_scale) return chunks == 8 ? launch_compact<8, true>(P, slices, n_seqs, st) : launch_compact<4, true>(P, slices, n_seqs, st);
    switch (chunks) {
        case 2: return launch_compact<2, false>(P, slices, n_seqs, st);
        case 4: return launch_compact<4, false>(P, slices, n_seqs, st);
        case 8: return launch_compact<8, false>(P, slices, n_seqs, st);
        default: return launch_compact<16, false>(P, slices, n_seqs, st);
    }
}
