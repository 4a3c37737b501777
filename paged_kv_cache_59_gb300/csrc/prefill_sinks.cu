// The chunked prefill's instantiations for a bf16 cache under a window with sinks.
#include "prefill_tc.cuh"

int pa_prefill_dispatch_sinks(int head_dim, int G, const PaPrefillParams& P, const CUtensorMap& tk, const CUtensorMap& tv,
                       int n_seqs, int max_chunk_len, int n_rows, cudaStream_t stream) {
    return head_dim == 64 ? dispatch_prefill<64, 2, true>(G, P, tk, tv, n_seqs, max_chunk_len, n_rows, stream)
                          : dispatch_prefill<128, 2, true>(G, P, tk, tv, n_seqs, max_chunk_len, n_rows, stream);
}
