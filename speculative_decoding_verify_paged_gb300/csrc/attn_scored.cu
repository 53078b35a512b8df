// Which kernel takes a call of sv_spec_verify_attn_scored.
#include <algorithm>

#include <cuda.h>

#include "sv_internal.cuh"

namespace sv {
namespace scored {
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn tensor_map_encoder() {
  static const EncodeTiledFn fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}
template <int D, bool F8>
cudaError_t pick(const ScoredArgs &sa, void *workspace, size_t *bytes, cudaStream_t st, bool go);
template <int D>
cudaError_t pick4(const ScoredArgs &sa, void *workspace, size_t *bytes, cudaStream_t st, bool go);
}

// bf16, E4M3 and E2M1 caches with heads of 64, 128 or 256 values in blocks of 8 tokens and more
// (attn_scored.cuh, attn_e2m1.cuh); a row of a pool is a 32-bit number there, and so are a unit's rows.
size_t attn_scored_mma_workspace(const ScoredArgs &sa) {
  const KV &kv = sa.a.kv;
  if (kv.elem_bytes == 4 || (kv.head_dim != 64 && kv.head_dim != 128 && kv.head_dim != 256)) return 0;
  if (kv.block_size < 8 || (long long)kv.num_blocks * kv.num_kv_heads * kv.block_size >= (1LL << 31)) return 0;
  if ((long long)(sa.a.num_q_heads / kv.num_kv_heads) * sa.a.max_q >= (1LL << 30)) return 0;
  size_t bytes = 0;
  launch_attn_scored_mma(sa, nullptr, &bytes, nullptr, false);
  return bytes;
}

cudaError_t launch_attn_scored_mma(const ScoredArgs &sa, void *workspace, size_t *bytes, cudaStream_t st, bool go) {
  const bool f8 = sa.a.kv.fp8;
  if (sa.a.kv.fp4)
    return sa.a.kv.head_dim == 64    ? scored::pick4<64>(sa, workspace, bytes, st, go)
           : sa.a.kv.head_dim == 128 ? scored::pick4<128>(sa, workspace, bytes, st, go)
                                     : scored::pick4<256>(sa, workspace, bytes, st, go);
  switch (sa.a.kv.head_dim) {
    case 64: return f8 ? scored::pick<64, true>(sa, workspace, bytes, st, go) : scored::pick<64, false>(sa, workspace, bytes, st, go);
    case 128: return f8 ? scored::pick<128, true>(sa, workspace, bytes, st, go) : scored::pick<128, false>(sa, workspace, bytes, st, go);
    default: return f8 ? scored::pick<256, true>(sa, workspace, bytes, st, go) : scored::pick<256, false>(sa, workspace, bytes, st, go);
  }
}

}  // namespace sv
