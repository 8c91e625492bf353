// Full attention of drafted tokens (a tree, a chain or one token) over a cache:
// the kernel of full_fwd.cuh with the cache's keys cut into equal runs for all
// SMs, and the merge of the units that a border cut.
#include "full_fwd.cuh"

namespace nsa {

namespace {

// One warp joins one row: the runs' (O, max, sum) in block order, so the result
// does not depend on timing. grid.x: (sequence, key head, row block).
template <int DV, int NT>
__global__ void __launch_bounds__(256) nsa_full_merge_kernel(const FullArgs a, int blocks) {
  constexpr int E = DV / 32;
  const int TOK = NT * 128 / a.G;
  const int rb_max = (a.M + TOK - 1) / TOK;
  const int b = blockIdx.x / (a.H_kv * rb_max);
  const int L = a.lens[b], n = a.nodes ? a.nodes[b] : a.M;
  const int32_t p0 = a.prefix_out[b], p1 = a.prefix_out[b + 1];
  if (p0 == p1) return;   // nothing to do (or refused) in this sequence
  const int rb = (n + TOK - 1) / TOK;
  const int gi = blockIdx.x - b * a.H_kv * rb_max, g = gi / rb_max, ri = gi - g * rb_max;
  if (ri >= rb) return;
  const int r = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int tt = r / a.G;   // row r of the block is head r % G of its token tt
  if (tt >= min(TOK, n - ri * TOK)) return;
  const int ntile = (L + kFaKeys - 1) / kFaKeys;
  const int64_t W = a.prefix_out[a.B];
  const int64_t start = p0 + (int64_t)(g * rb + ri) * ntile, last = start + ntile - 1;
  const int c0 = (int)(((start + 1) * blocks - 1) / W), c1 = (int)(((last + 1) * blocks - 1) / W);
  if (c0 == c1) return;   // one block did the whole unit
  const float* part = a.part + (int64_t)r * (DV + 4);
  const int64_t ld = (int64_t)NT * 128 * (DV + 4);
  float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int cb = c0; cb <= c1; cb += 32) {
    const int c = cb + lane;
    // a block without tiles (fewer tiles than blocks) left nothing
    const bool has = c <= c1 && W * c / blocks < W * (c + 1) / blocks;
    const float* p = part + (2 * (int64_t)c + (c == c0 ? 1 : 0)) * ld;
    float mc = -INFINITY, lc = 0.f;
    if (has) {
      mc = p[DV];
      lc = p[DV + 1];
    }
    float mx = mc;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mn = fmaxf(m, mx), mz = mn == -INFINITY ? 0.f : mn;
    const float wm = ex2(m - mz);   // 0 before the first run
    const float w = has ? ex2(mc - mz) : 0.f;
    float ls = has ? lc * w : 0.f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
    l = l * wm + ls;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= wm;
    m = mn;
    const uint32_t live = __ballot_sync(0xffffffffu, has);
    const int cnt = min(32, c1 - cb + 1);
#pragma unroll 4
    for (int i = 0; i < cnt; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      if (!((live >> i) & 1u)) continue;
      const float* po = part + (2 * (int64_t)(cb + i) + (cb + i == c0 ? 1 : 0)) * ld + lane * E;
      if constexpr (E == 4) {
        const float4 v = *reinterpret_cast<const float4*>(po);
        acc[0] = fmaf(v.x, wi, acc[0]);
        acc[1] = fmaf(v.y, wi, acc[1]);
        acc[2] = fmaf(v.z, wi, acc[2]);
        acc[3] = fmaf(v.w, wi, acc[3]);
      } else {
        const float2 v = *reinterpret_cast<const float2*>(po);
        acc[0] = fmaf(v.x, wi, acc[0]);
        acc[1] = fmaf(v.y, wi, acc[1]);
      }
    }
  }
  const int64_t row = ((int64_t)b * a.M + ri * TOK + tt) * a.H_q + g * a.G + r % a.G;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + row * DV + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2)
    dst[e >> 1] = l == 0.f ? 0u : pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : 0.69314718055994531f * (m + log2f(l));
}

}  // namespace

cudaError_t launch_full_tree(const FullArgs& a, const FullMaps& m, int nt, cudaStream_t st) {
  const int grid = kFullBlocks;
  cudaError_t e = nt == 2 ? launch_full_d<2, true>(a, m, grid, st) : launch_full_d<1, true>(a, m, grid, st);
  if (e != cudaSuccess) return e;
  const int TOK = nt * 128 / a.G, rb = (a.M + TOK - 1) / TOK;
  const int rows = a.M < TOK ? a.M * a.G : nt * 128;
  const dim3 mg(a.B * a.H_kv * rb, (rows + 7) / 8);
  if (nt == 2) {
    if (a.d_v == 128) nsa_full_merge_kernel<128, 2><<<mg, 256, 0, st>>>(a, grid);
    else nsa_full_merge_kernel<64, 2><<<mg, 256, 0, st>>>(a, grid);
  } else {
    if (a.d_v == 128) nsa_full_merge_kernel<128, 1><<<mg, 256, 0, st>>>(a, grid);
    else nsa_full_merge_kernel<64, 1><<<mg, 256, 0, st>>>(a, grid);
  }
  return cudaGetLastError();
}

}  // namespace nsa
