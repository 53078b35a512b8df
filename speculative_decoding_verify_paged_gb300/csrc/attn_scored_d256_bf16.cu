// Attention with modified scores: heads of 256 values, bf16 caches (attn_scored.cuh).
#include <algorithm>

#include "attn_scored.cuh"

namespace sv {
template cudaError_t scored::pick<256, false>(const ScoredArgs &, void *, size_t *, cudaStream_t, bool);
}
