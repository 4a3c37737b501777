// Host side of the chunked prefill: argument checks, workspaces, tensor maps and
// the launches (the kernels are in prefill_tc.cuh), and the instantiations for a
// bf16 cache without a window.
#include "prefill_tc.cuh"

namespace {

int sm_count() {
    static int cached[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (!cached[dev] && cudaDeviceGetAttribute(&cached[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        cached[dev] = 0;
    return cached[dev];
}

int pairs_per_seq(int G, int max_chunk_len) {
    const int QT = kRows / G;
    return (max_chunk_len + 2 * QT - 1) / (2 * QT);
}

size_t part_bytes(long long n_items, int splits) {
    return splits > 1 ? (size_t)n_items * splits * 2 * 128 * kPartStride * sizeof(float) : 0;
}

// Balanced mode (splits = 0): partial slots for the cut items (at most 4
// per CTA), the work list (n_items + 4 * n_cta entries) and the counters,
// each part 16-byte aligned.
struct BalancedLayout {
    size_t part, work, sched, total;
};
BalancedLayout balanced_layout(long long n_items, int n_cta) {
    BalancedLayout b;
    b.part = 0;
    b.work = (size_t)4 * n_cta * 2 * 128 * kPartStride * sizeof(float);
    b.sched = b.work + (size_t)(n_items + 4LL * n_cta) * sizeof(int4);
    b.total = b.sched + 16;
    return b;
}

int prefill_impl(void* out, const void* q, const void* k_pool, const void* v_pool, const int32_t* block_tables,
                 const int32_t* context_lens, const int32_t* q_start_loc, float scale, int n_heads,
                 int n_kv_heads, int head_dim, int block_size, int n_seqs, int max_blocks_per_seq,
                 int max_chunk_len, int num_blocks, int splits, void* workspace, size_t workspace_bytes,
                 pa_stream_t stream, int eb = 2, const float* k_scale = nullptr, const float* v_scale = nullptr,
                 int window = -1, int n_sinks = 0) {
    if (n_seqs < 0 || max_chunk_len < 0 || num_blocks < 0 || max_blocks_per_seq < 0 || n_heads <= 0 ||
        n_kv_heads <= 0 || splits < 0 || splits > 64)
        return PA_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128) || block_size != kBS) return PA_ERR_UNSUPPORTED;
    if (n_heads % n_kv_heads != 0) return PA_ERR_INVALID_ARG;
    const int G = n_heads / n_kv_heads;
    if (G != 1 && G != 2 && G != 4 && G != 8) return PA_ERR_UNSUPPORTED;
    if (n_seqs == 0 || max_chunk_len == 0) return PA_OK;
    if (n_kv_heads > 65535 || n_seqs > 65535) return PA_ERR_UNSUPPORTED;
    if (!out || !q || !k_pool || !v_pool || !block_tables || !context_lens || !q_start_loc)
        return PA_ERR_INVALID_ARG;
    if (!pa_aligned16(out) || !pa_aligned16(q) || !pa_aligned16(k_pool) || !pa_aligned16(v_pool))
        return PA_ERR_INVALID_ARG;
    if (out == q) return PA_ERR_INVALID_ARG;
    if (eb == 1 && (!k_scale || !v_scale || (reinterpret_cast<uintptr_t>(k_scale) & 3u) ||
                    (reinterpret_cast<uintptr_t>(v_scale) & 3u)))
        return PA_ERR_INVALID_ARG;
    // the kernel adds up to a few key tiles to these; no context reaches the limit
    constexpr int kMost = 0x7fffffff - 65536;
    if (window > kMost) window = kMost;
    if (n_sinks > kMost) n_sinks = kMost;
    const long long rows = (long long)num_blocks * n_kv_heads * kBS;
    if (rows + kBS > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;  // TMA row coordinates are int32
    const int n_qp = pairs_per_seq(G, max_chunk_len);
    const long long n_items = (long long)n_qp * n_kv_heads * n_seqs;
    if (n_items > 0x3fffffffLL) return PA_ERR_UNSUPPORTED;
    const int n_cta = splits == 0 ? sm_count() : 0;
    if (splits == 0 && n_cta <= 0) return PA_ERR_CUDA;
    if ((long long)n_qp * (splits > 0 ? splits : 1) > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    const size_t need = splits == 0 ? balanced_layout(n_items, n_cta).total : part_bytes(n_items, splits);
    if (need > 0 && (!workspace || workspace_bytes < need || !pa_aligned16(workspace))) return PA_ERR_WORKSPACE;
    unsigned int* err = pa_device_error_ptr();
    if (!err) return PA_ERR_CUDA;
    CUtensorMap tk, tv;
    const bool maps = eb == 2 ? pa_make_tmap_2d_bf16(&tk, k_pool, head_dim, (uint64_t)rows, head_dim * 2, 64, kBS) &&
                                    pa_make_tmap_2d_bf16(&tv, v_pool, head_dim, (uint64_t)rows, head_dim * 2, 64, kBS)
                              : pa_make_tmap_2d_u8(&tk, k_pool, head_dim, (uint64_t)rows, head_dim, head_dim, kBS, head_dim == 128) &&
                                    pa_make_tmap_2d_u8(&tv, v_pool, head_dim, (uint64_t)rows, head_dim, head_dim, kBS, head_dim == 128);
    if (!maps) return PA_ERR_CUDA;
    PrefillParams Pp;
    Pp.out = static_cast<uint16_t*>(out);
    Pp.q = static_cast<const uint16_t*>(q);
    Pp.tables = block_tables;
    Pp.ctx = context_lens;
    Pp.qsl = q_start_loc;
    Pp.scale_log2 = scale * 1.4426950408889634f;
    Pp.n_heads = n_heads;
    Pp.n_kv_heads = n_kv_heads;
    Pp.max_blocks = max_blocks_per_seq;
    Pp.num_blocks = num_blocks;
    Pp.oob_row = (int)rows;
    Pp.splits = splits > 0 ? splits : 1;
    Pp.part = need ? static_cast<float*>(workspace) : nullptr;
    Pp.work = nullptr;
    Pp.sched = nullptr;
    if (splits == 0) {
        const BalancedLayout bl = balanced_layout(n_items, n_cta);
        char* w = static_cast<char*>(workspace);
        Pp.work = reinterpret_cast<int4*>(w + bl.work);
        Pp.sched = reinterpret_cast<int*>(w + bl.sched);
    }
    Pp.n_items = (int)n_items;
    Pp.n_qp = n_qp;
    Pp.n_cta = n_cta;
    Pp.err = err;
    Pp.window = window;
    Pp.n_sinks = n_sinks;
    Pp.k_scale = k_scale;
    Pp.v_scale = v_scale;
    // chunk rows bound for the merge grid (rows past the last chunk exit)
    const long long n_rows = (long long)n_seqs * max_chunk_len;
    if (n_rows > 0x7fffffffLL || n_rows * n_heads > 0x7fffffffLL * 4LL) return PA_ERR_UNSUPPORTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int nr = (int)n_rows;
    if (eb == 1) return pa_prefill_dispatch_fp8(head_dim, G, Pp, tk, tv, n_seqs, max_chunk_len, nr, st);
    if (window >= 0) return pa_prefill_dispatch_sinks(head_dim, G, Pp, tk, tv, n_seqs, max_chunk_len, nr, st);
    return head_dim == 64 ? dispatch_prefill<64, 2, false>(G, Pp, tk, tv, n_seqs, max_chunk_len, nr, st)
                          : dispatch_prefill<128, 2, false>(G, Pp, tk, tv, n_seqs, max_chunk_len, nr, st);
}

}  // namespace

extern "C" size_t pa_prefill_workspace_bytes(int n_seqs, int n_heads, int n_kv_heads, int max_chunk_len,
                                             int splits) {
    if (n_seqs <= 0 || n_heads <= 0 || n_kv_heads <= 0 || max_chunk_len <= 0 || splits < 0 || splits > 64 ||
        n_heads % n_kv_heads != 0)
        return 0;
    const int G = n_heads / n_kv_heads;
    if (G != 1 && G != 2 && G != 4 && G != 8) return 0;
    const long long n_items = (long long)pairs_per_seq(G, max_chunk_len) * n_kv_heads * n_seqs;
    if (splits > 0) return part_bytes(n_items, splits);
    const int n_cta = sm_count();
    return n_cta > 0 ? balanced_layout(n_items, n_cta).total : 0;
}

extern "C" int pa_prefill_paged_ex(void* out, const void* q, const void* k_pool, const void* v_pool,
                                   const int32_t* block_tables, const int32_t* context_lens,
                                   const int32_t* q_start_loc, float scale, int n_heads, int n_kv_heads,
                                   int head_dim, int block_size, int n_seqs, int max_blocks_per_seq,
                                   int max_chunk_len, int num_blocks, int splits, void* workspace,
                                   size_t workspace_bytes, pa_stream_t stream) {
    return prefill_impl(out, q, k_pool, v_pool, block_tables, context_lens, q_start_loc, scale, n_heads,
                        n_kv_heads, head_dim, block_size, n_seqs, max_blocks_per_seq, max_chunk_len, num_blocks,
                        splits, workspace, workspace_bytes, stream);
}

extern "C" int pa_prefill_paged(void* out, const void* q, const void* k_pool, const void* v_pool,
                                const int32_t* block_tables, const int32_t* context_lens,
                                const int32_t* q_start_loc, float scale, int n_heads, int n_kv_heads,
                                int head_dim, int block_size, int n_seqs, int max_blocks_per_seq,
                                int max_chunk_len, int num_blocks, pa_stream_t stream) {
    return prefill_impl(out, q, k_pool, v_pool, block_tables, context_lens, q_start_loc, scale, n_heads,
                        n_kv_heads, head_dim, block_size, n_seqs, max_blocks_per_seq, max_chunk_len, num_blocks,
                        1, nullptr, 0, stream);
}

extern "C" int pa_prefill_sinks(void* out, const void* q, const void* k_pool, const void* v_pool,
                                const int32_t* block_tables, const int32_t* context_lens, const int32_t* q_start_loc,
                                float scale, int n_heads, int n_kv_heads, int head_dim, int block_size, int n_seqs,
                                int max_blocks_per_seq, int max_chunk_len, int num_blocks, int window, int n_sinks,
                                int splits, void* workspace, size_t workspace_bytes, pa_stream_t stream) {
    if (window < 0 || n_sinks < 0) return PA_ERR_INVALID_ARG;
    return prefill_impl(out, q, k_pool, v_pool, block_tables, context_lens, q_start_loc, scale, n_heads, n_kv_heads,
                        head_dim, block_size, n_seqs, max_blocks_per_seq, max_chunk_len, num_blocks, splits, workspace,
                        workspace_bytes, stream, 2, nullptr, nullptr, window, n_sinks);
}

extern "C" int pa_prefill_fp8_block(void* out, const void* q, const void* k_pool, const void* v_pool,
                                    const float* k_scale, const float* v_scale, const int32_t* block_tables,
                                    const int32_t* context_lens, const int32_t* q_start_loc, float scale, int n_heads,
                                    int n_kv_heads, int head_dim, int block_size, int n_seqs, int max_blocks_per_seq,
                                    int max_chunk_len, int num_blocks, int window, int n_sinks, int splits,
                                    void* workspace, size_t workspace_bytes, pa_stream_t stream) {
    if (window < -1 || n_sinks < 0) return PA_ERR_INVALID_ARG;
    if (window < 0) n_sinks = 0;  // everything is visible
    return prefill_impl(out, q, k_pool, v_pool, block_tables, context_lens, q_start_loc, scale, n_heads, n_kv_heads,
                        head_dim, block_size, n_seqs, max_blocks_per_seq, max_chunk_len, num_blocks, splits, workspace,
                        workspace_bytes, stream, 1, k_scale, v_scale, window, n_sinks);
}
