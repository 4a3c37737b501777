// The chunked prefill's instantiations for an E4M3 cache with a scale per (block, KV head), with or without a window.
#include "prefill_win.cuh"

int pa_prefill_dispatch_fp8(int head_dim, int G, const PaPrefillParams& P, const CUtensorMap& tk, const CUtensorMap& tv,
                       int n_seqs, int n_rows, cudaStream_t stream) {
    return head_dim == 64 ? dispatch_prefill_win<64, 1>(G, P, tk, tv, n_seqs, n_rows, stream)
                          : dispatch_prefill_win<128, 1>(G, P, tk, tv, n_seqs, n_rows, stream);
}
