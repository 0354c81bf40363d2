// bfp8_kvweigh.cuh -- what the kernels share that sum the attention weight of
// cached tokens.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "bfp8_attn.cuh"

namespace bfp8 {

struct WeighArgs {
  AttnArgs a;                         // lse is an input here; few_rows: as there
  float* w;
  int64_t ws_page, ws_head;           // floats
  int32_t add;                        // 0: every sum begins here
};

// Does token j's sum begin with this call (new tokens have none yet)?
__device__ __forceinline__ bool begins_here(const WeighArgs& p, int32_t j, int32_t pos0) {
  return p.add == 0 || (p.a.causal != 0 && j >= pos0);
}

// Sequences of at most 8 * groups (1 or 2) rows, `ctas` SMs (bfp8_kvweigh.cu).
cudaError_t launch_weigh_few(const WeighArgs& p, int groups, int ctas, cudaStream_t stream);

// The others (bfp8_kvweigh_tile.cu); counters[2 * ctas] zero.  q: tensor map of the queries as bytes [dim, head, token],
// 128-byte swizzle, boxes of 128 bytes x group x weigh_tile_tokens(group, max_q).
int weigh_tile_tokens(int group, int max_q);
size_t weigh_tile_partial_bytes(int ctas);
cudaError_t launch_weigh_tile(const CUtensorMap& q, const WeighArgs& p, int ctas, int32_t* counters, float* partials,
                              cudaStream_t stream);

}  // namespace bfp8
