// Causal full attention over packed prompts (the kernel is in full_fwd.cuh).
#include "full_fwd.cuh"

namespace nsa {

cudaError_t launch_full_prefill(const FullArgs& a, const FullMaps& m, int nt, cudaStream_t st) {
  const int grid = a.n_items < kFullBlocks ? (int)a.n_items : kFullBlocks;
  return nt == 2 ? launch_full_d<2, false>(a, m, grid, st) : launch_full_d<1, false>(a, m, grid, st);
}

}  // namespace nsa
