// The chunked prefill's instantiations for a bf16 cache under a window with sinks.
#include "prefill_win.cuh"

int pa_prefill_dispatch_sinks(int head_dim, int G, const PaPrefillParams& P, const CUtensorMap& tk, const CUtensorMap& tv,
                       int n_seqs, int n_rows, cudaStream_t stream) {
    return head_dim == 64 ? dispatch_prefill_win<64, 2>(G, P, tk, tv, n_seqs, n_rows, stream)
                          : dispatch_prefill_win<128, 2>(G, P, tk, tv, n_seqs, n_rows, stream);
}
