// The chunked prefill's instantiations for scores with a cap and a bias by distance over an E4M3 cache with a scale per (block, KV head).
#include "prefill_win.cuh"

int pa_prefill_dispatch_both_fp8(int head_dim, int G, const PaPrefillParams& P, const CUtensorMap& tk, const CUtensorMap& tv,
                                 int n_seqs, int n_rows, cudaStream_t stream) {
    return head_dim == 64 ? dispatch_prefill_win<64, 1, kCapBias>(G, P, tk, tv, n_seqs, n_rows, stream)
                          : dispatch_prefill_win<128, 1, kCapBias>(G, P, tk, tv, n_seqs, n_rows, stream);
}
