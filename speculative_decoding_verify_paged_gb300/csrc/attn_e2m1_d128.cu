// Attention with modified scores: heads of 128 values, E2M1 caches (attn_e2m1.cuh).
#include <algorithm>

#include "attn_e2m1.cuh"

namespace sv {
template cudaError_t scored::pick4<128>(const ScoredArgs &, void *, size_t *, cudaStream_t, bool);
}
