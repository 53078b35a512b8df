// Attention with modified scores: heads of 128 values, e4m3 caches (attn_scored.cuh).
#include <algorithm>

#include "attn_scored.cuh"

namespace sv {
template cudaError_t scored::pick<128, true>(const ScoredArgs &, void *, size_t *, cudaStream_t, bool);
}
