// Full attention of drafted tokens (a tree, a chain or one token) over a cache:
// the kernel of full_fwd.cuh with the cache's keys cut into equal runs for all
// SMs, and the merge of the units that a border cut.
#include "full_fwd.cuh"

namespace nsa {

namespace {

// Joins the runs' (O, max, sum) of a row in block order, so the result does not
// depend on timing. Block x: the unit that begins in run x and ends beyond it (every
// unit that a border cut begins in one run), if there is one; a warp takes kMergeRows
// rows at once, since each waits for two loads in turn.
constexpr int kMergeRows = 4;
template <int DV>
__global__ void __launch_bounds__(256) nsa_full_merge_kernel(const FullArgs a, int rows) {
  constexpr int E = DV / 32;
  pdl_wait();   // launched while the attention kernel runs
  const int c0 = blockIdx.x;
  const int4 cut = a.cut[c0];
  if (cut.x < 0) return;
  const int b = cut.x, c1 = cut.w, n = a.nodes ? a.nodes[b] : a.M;
  const int lane = threadIdx.x & 31;
  const int r0 = (blockIdx.y * 8 + (threadIdx.x >> 5)) * kMergeRows;
  const int have = min(rows, (n - cut.z) * a.G);   // row r of the unit is head r % G of node cut.z + r / G
  if (r0 >= have) return;
  const int64_t ld = (int64_t)rows * (DV + 4);
  auto slot = [&](int c, int k) -> const float* {   // row r0 + k (the last one again past the end) of run c
    return a.part + (2 * (int64_t)c + (c == c0 ? 1 : 0)) * ld + (int64_t)min(r0 + k, have - 1) * (DV + 4);
  };
  float m[kMergeRows], l[kMergeRows], acc[kMergeRows][E];
#pragma unroll
  for (int k = 0; k < kMergeRows; ++k) {
    m[k] = -INFINITY;
    l[k] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[k][e] = 0.f;
  }
  for (int cb = c0; cb <= c1; cb += 32) {
    const int c = cb + lane;
    const bool has = c <= c1;
    const int cnt = min(32, c1 - cb + 1);
    float w[kMergeRows];
#pragma unroll
    for (int k = 0; k < kMergeRows; ++k) {
      float2 ml = make_float2(-INFINITY, 0.f);
      if (has) ml = *reinterpret_cast<const float2*>(slot(c, k) + DV);
      float mx = ml.x;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float mn = fmaxf(m[k], mx), mz = mn == -INFINITY ? 0.f : mn;
      const float wm = ex2(m[k] - mz);   // 0 before the first run
      w[k] = has ? ex2(ml.x - mz) : 0.f;
      float ls = has ? ml.y * w[k] : 0.f;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
      l[k] = l[k] * wm + ls;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[k][e] *= wm;
      m[k] = mn;
    }
#pragma unroll 4
    for (int i = 0; i < cnt; ++i) {
#pragma unroll
      for (int k = 0; k < kMergeRows; ++k) {
        const float wi = __shfl_sync(0xffffffffu, w[k], i);
        const float* po = slot(cb + i, k) + lane * E;
        if constexpr (E == 4) {
          const float4 v = *reinterpret_cast<const float4*>(po);
          acc[k][0] = fmaf(v.x, wi, acc[k][0]);
          acc[k][1] = fmaf(v.y, wi, acc[k][1]);
          acc[k][2] = fmaf(v.z, wi, acc[k][2]);
          acc[k][3] = fmaf(v.w, wi, acc[k][3]);
        } else {
          const float2 v = *reinterpret_cast<const float2*>(po);
          acc[k][0] = fmaf(v.x, wi, acc[k][0]);
          acc[k][1] = fmaf(v.y, wi, acc[k][1]);
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kMergeRows; ++k) {
    const int r = r0 + k;
    if (r >= have) break;
    const int64_t row = ((int64_t)b * a.M + cut.z + r / a.G) * a.H_q + cut.y * a.G + r % a.G;
    const float inv = l[k] == 0.f ? 0.f : 1.f / l[k];
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + row * DV + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e >> 1] = l[k] == 0.f ? 0u : pack_bf16x2(acc[k][e] * inv, acc[k][e + 1] * inv);
    if (a.lse && lane == 0) a.lse[row] = l[k] == 0.f ? -INFINITY : 0.69314718055994531f * (m[k] + log2f(l[k]));
  }
}

}  // namespace

cudaError_t launch_full_tree(const FullArgs& a, const FullMaps& m, int nt, cudaStream_t st) {
  const int grid = kFullBlocks;
  cudaError_t e = nt == 2 ? launch_full_d<2, true>(a, m, grid, st) : launch_full_d<1, true>(a, m, grid, st);
  if (e != cudaSuccess) return e;
  const int TOK = nt * 128 / a.G, rows = nt * 128;
  const int used = a.M < TOK ? a.M * a.G : rows;
  const dim3 mg(grid, (used + 8 * kMergeRows - 1) / (8 * kMergeRows));
  return a.d_v == 128 ? launch_after(nsa_full_merge_kernel<128>, mg, 256, 0, st, a, rows)
                      : launch_after(nsa_full_merge_kernel<64>, mg, 256, 0, st, a, rows);
}

}  // namespace nsa
