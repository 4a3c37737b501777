// How many CTAs share a compaction's steps (host).
#pragma once

#include <algorithm>

// CTAs of a cluster, one cluster for each of `units` (sequence, KV head, K or V): until there are two CTAs for
// each SM, as far as a sequence's tokens (on average) give each a step's share (`tokens`). Up to 8, and up to 16
// where few clusters leave SMs idle, which moves as many bytes a second as an SM's share of HBM: 1.3 CTAs for
// each SM, as clusters of CTAs that share SMs with others hold all of theirs back. (One document's 16 units: 125
// us with 8, 107 with 10, 109 with 12, 133 with 16; in E4M3 72, 61, 53, 72; 8 units of 4 sequences: 45 with 8, 33
// with 12, 27 with 16.) `largest`: the largest cluster that the context can hold.
inline int pa_compact_ctas(long long units, int sms, long long n_kept, long long n_seqs, int tokens, int largest) {
    const int most = (int)std::min<long long>(largest, std::min(16LL, std::max(8LL, 13LL * sms / (10 * units))));
    int ctas = 1;
    while (ctas < most && units * ctas < 2LL * sms && n_kept > n_seqs * ctas * tokens) ctas = std::min(2 * ctas, most);
    return ctas;
}
