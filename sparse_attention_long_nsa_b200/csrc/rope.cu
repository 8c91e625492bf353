// Per-head RMS norm of queries and keys with the rotary position in the same
// pass, and its backward.
//
// Forward, for every token n and head (x = the projection's d_k channels):
//   y = x * rsqrt(mean(x^2) + eps) * w
//   each pair (a, b) of the first d_rot channels of y turns by the angle
//   positions[n] * inv_freq[i]:  (a cos - b sin, a sin + b cos)
// pairs are (2i, 2i + 1) or (i, i + d_rot / 2). fp32 throughout, rounded to bf16
// once. The angle is formed and brought into [-pi, pi] in fp64: in fp32 the
// product alone would be off by position * 2^-24 radians.
//
// Backward: dn = the incoming gradient turned by the opposite angle,
//   u = dn w,  h = x r  (r = rsqrt(mean(x^2) + eps), recomputed),
//   dx = r (u - h mean(u h)),  dw = sum over tokens and heads of dn h.
//
// Both are bound by memory: 4 bytes per element forward, 6 backward. Four lanes
// own a head: a lane holds d_k / 64 units, a unit being two 16-byte chunks of 8
// channels. For pairs (i, i + d_rot / 2) the two chunks of a rotating unit are
// partners, so that every rotation stays inside a thread. The sines and cosines
// of a block's tokens are computed once into shared memory and serve all heads.
#include "common.cuh"
#include "kernels.h"

namespace nsa {

namespace {

constexpr int kThreads = 256;
constexpr int kGroups = kThreads / 4;   // heads in work at a time

struct Chunks {
  int c0, c1;   // the two 8-channel chunks of a unit
  bool rot;
};
// unit u of a head of which R = d_rot / 8 chunks rotate
__device__ __forceinline__ Chunks unit_chunks(int u, int R) {
  const int half = R >> 1;
  Chunks c;
  c.rot = u < half;
  c.c0 = c.rot ? u : R + 2 * (u - half);
  c.c1 = c.rot ? u + half : c.c0 + 1;
  return c;
}

__device__ __forceinline__ void unpack8(const uint4& w, float* f) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ float sum4(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// (cos, sin) of pair i of tokens n0 .. n0 + nt - 1 into cs[tok * half + i]
__device__ __forceinline__ void fill_angles(const RopeArgs& a, int64_t n0, int nt, int half, float2* cs) {
  constexpr double k2Pi = 6.283185307179586476925286766559, kInv2Pi = 0.15915494309189533576888376337251;
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int tok = i / half;
    const double x = (double)a.positions[n0 + tok] * (double)a.inv_freq[i - tok * half];
    const float r = (float)fma(-rint(x * kInv2Pi), k2Pi, x);
    float s, c;
    sincosf(r, &s, &c);
    cs[i] = make_float2(c, s);
  }
}

// turn the pairs of a unit (SIGN -1: by the opposite angle); f[0..7] and f[8..15]
// are its two chunks, first channel 8 * c0 / 8 * c1
template <bool INTER, int SIGN>
__device__ __forceinline__ void turn_unit(float* f, const Chunks& ch, const float2* cs) {
  if constexpr (INTER) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 t = cs[(i < 4 ? ch.c0 * 4 : ch.c1 * 4 - 4) + i];
      const float s = SIGN * t.y, p = f[2 * i], q = f[2 * i + 1];
      f[2 * i] = p * t.x - q * s;
      f[2 * i + 1] = p * s + q * t.x;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 t = cs[ch.c0 * 8 + i];
      const float s = SIGN * t.y, p = f[i], q = f[8 + i];
      f[i] = p * t.x - q * s;
      f[8 + i] = p * s + q * t.x;
    }
  }
}

}  // namespace

// One block: `tok` tokens, all their query, key (and value) heads. Values are
// copied. Head items are dealt to the 64 lane groups in turn.
template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads) nsa_qk_norm_rope_kernel(const RopeArgs a) {
  constexpr int U = D / 64;
  extern __shared__ float2 cs[];
  const int64_t n0 = (int64_t)blockIdx.x * a.tok;
  const int nt = (int)min((int64_t)a.tok, a.N - n0);
  const int half = a.d_rot >> 1, R = a.d_rot >> 3;
  const int sub = threadIdx.x & 3, grp = threadIdx.x >> 2;
  fill_angles(a, n0, nt, half, cs);
  __syncthreads();
  const int H = a.H_q + a.H_kv + a.H_v;
  const int total = nt * H;
  for (int base = 0; base < total; base += kGroups) {
    const int item = base + grp;
    const bool on = item < total;
    const int tok = on ? item / H : 0;
    const int h = on ? item - tok * H : 0;
    const int64_t n = n0 + tok;
    const bool is_q = h < a.H_q, is_v = h >= a.H_q + a.H_kv;
    int64_t row = n;
    bool write = on;
    if (!is_q && a.cache_rows) {   // a row outside the cache is not written
      row = a.cache_rows[n];
      write = on && row >= 0 && row < a.n_rows;
    }
    if (is_v) {
      const int hv = h - a.H_q - a.H_kv;
      if (write) {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.v) + n * a.v_stride +
                                                          (int64_t)hv * a.d_v);
        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.v_out) + (row * a.H_kv + hv) * a.d_v);
        for (int c = sub; c < a.d_v / 8; c += 4) dst[c] = src[c];
      }
    }
    const bool work = on && !is_v;
    const int hk = h - a.H_q;
    const __nv_bfloat16* x = is_q ? static_cast<const __nv_bfloat16*>(a.q) + n * a.q_stride + (int64_t)h * D
                                  : static_cast<const __nv_bfloat16*>(a.k) + n * a.k_stride + (int64_t)hk * D;
    uint4 raw[U][2];
    if (work) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const Chunks ch = unit_chunks(sub + 4 * j, R);
        raw[j][0] = reinterpret_cast<const uint4*>(x)[ch.c0];
        raw[j][1] = reinterpret_cast<const uint4*>(x)[ch.c1];
      }
    } else {
#pragma unroll
      for (int j = 0; j < U; ++j) raw[j][0] = raw[j][1] = make_uint4(0, 0, 0, 0);
    }
    float f[U][16];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      unpack8(raw[j][0], f[j]);
      unpack8(raw[j][1], f[j] + 8);
#pragma unroll
      for (int i = 0; i < 16; ++i) ss = fmaf(f[j][i], f[j][i], ss);
    }
    ss = sum4(ss);
    if (!work || !write) continue;   // the shuffles above were the last ones of this item
    const float r = rsqrtf(ss * (1.f / D) + a.eps);
    const float* w = is_q ? a.w_q : a.w_k;
    __nv_bfloat16* y = is_q ? static_cast<__nv_bfloat16*>(a.q_out) + (n * a.H_q + h) * D
                            : static_cast<__nv_bfloat16*>(a.k_out) + (row * a.H_kv + hk) * D;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const Chunks ch = unit_chunks(sub + 4 * j, R);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 wv = *reinterpret_cast<const float4*>(w + (q < 2 ? ch.c0 : ch.c1) * 8 + (q & 1) * 4);
        f[j][4 * q] *= r * wv.x;
        f[j][4 * q + 1] *= r * wv.y;
        f[j][4 * q + 2] *= r * wv.z;
        f[j][4 * q + 3] *= r * wv.w;
      }
      if (ch.rot) turn_unit<INTER, 1>(f[j], ch, cs + tok * half);
      reinterpret_cast<uint4*>(y)[ch.c0] = pack8(f[j]);
      reinterpret_cast<uint4*>(y)[ch.c1] = pack8(f[j] + 8);
    }
  }
}

// Backward. grid.x blocks walk the token groups; blocks below `q_blocks` take the
// query heads, the others the key heads, so that a thread's dw sums belong to one
// weight. part[block][D]: this block's dw, its groups summed in a fixed order.
template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 2) nsa_qk_norm_rope_bwd_kernel(const RopeBwdArgs b) {
  constexpr int U = D / 64;
  extern __shared__ float2 cs[];
  const RopeArgs& a = b.f;
  const int half = a.d_rot >> 1, R = a.d_rot >> 3;
  const int sub = threadIdx.x & 3, grp = threadIdx.x >> 2;
  const bool is_q = (int)blockIdx.x < b.q_blocks;
  const int blk = is_q ? blockIdx.x : blockIdx.x - b.q_blocks;
  const int nblk = is_q ? b.q_blocks : (int)gridDim.x - b.q_blocks;
  const int H = is_q ? a.H_q : a.H_kv;
  const float* w = is_q ? a.w_q : a.w_k;
  const __nv_bfloat16* xb = static_cast<const __nv_bfloat16*>(is_q ? a.q : a.k);
  const __nv_bfloat16* gb = static_cast<const __nv_bfloat16*>(is_q ? b.dq_out : b.dk_out);
  __nv_bfloat16* ob = static_cast<__nv_bfloat16*>(is_q ? b.dq : b.dk);
  const int64_t xs = is_q ? a.q_stride : a.k_stride, os = is_q ? b.dq_stride : b.dk_stride;
  float dw[U][16];
#pragma unroll
  for (int j = 0; j < U; ++j)
#pragma unroll
    for (int i = 0; i < 16; ++i) dw[j][i] = 0.f;
  for (int64_t n0 = (int64_t)blk * a.tok; n0 < a.N; n0 += (int64_t)nblk * a.tok) {
    const int nt = (int)min((int64_t)a.tok, a.N - n0);
    __syncthreads();
    fill_angles(a, n0, nt, half, cs);
    __syncthreads();
    const int total = nt * H;
    for (int base = 0; base < total; base += kGroups) {
      const int item = base + grp;
      const bool on = item < total;
      const int tok = on ? item / H : 0;
      const int h = on ? item - tok * H : 0;
      const int64_t n = n0 + tok;
      const uint4* x = reinterpret_cast<const uint4*>(xb + n * xs + (int64_t)h * D);
      const uint4* g = reinterpret_cast<const uint4*>(gb + (n * H + h) * D);
      uint4 rx[U][2], rg[U][2];
      if (on) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const Chunks ch = unit_chunks(sub + 4 * j, R);
          rx[j][0] = x[ch.c0];
          rx[j][1] = x[ch.c1];
          rg[j][0] = g[ch.c0];
          rg[j][1] = g[ch.c1];
        }
      } else {
#pragma unroll
        for (int j = 0; j < U; ++j) rx[j][0] = rx[j][1] = rg[j][0] = rg[j][1] = make_uint4(0, 0, 0, 0);
      }
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        float f[16];
        unpack8(rx[j][0], f);
        unpack8(rx[j][1], f + 8);
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = fmaf(f[i], f[i], ss);
      }
      const float r = rsqrtf(sum4(ss) * (1.f / D) + a.eps);
      // dn = the gradient turned back; u = dn w; dw += dn h; m = sum(u h)
      float u[U][16];
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const Chunks ch = unit_chunks(sub + 4 * j, R);
        float f[16];
        unpack8(rg[j][0], u[j]);
        unpack8(rg[j][1], u[j] + 8);
        unpack8(rx[j][0], f);
        unpack8(rx[j][1], f + 8);
        if (ch.rot) turn_unit<INTER, -1>(u[j], ch, cs + tok * half);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 w4 = *reinterpret_cast<const float4*>(w + (q < 2 ? ch.c0 : ch.c1) * 8 + (q & 1) * 4);
          const float wv[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
          for (int i = 4 * q; i < 4 * q + 4; ++i) {
            const float hx = f[i] * r;
            dw[j][i] = fmaf(u[j][i], hx, dw[j][i]);
            u[j][i] *= wv[i - 4 * q];
            m = fmaf(u[j][i], hx, m);
          }
        }
      }
      m = sum4(m) * (1.f / D) * r;   // mean(u h) r: h = x r below
      if (on) {
        uint4* dst = reinterpret_cast<uint4*>(ob + n * os + (int64_t)h * D);
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const Chunks ch = unit_chunks(sub + 4 * j, R);
          float f[16];
          unpack8(rx[j][0], f);
          unpack8(rx[j][1], f + 8);
#pragma unroll
          for (int i = 0; i < 16; ++i) f[i] = r * fmaf(-f[i], m, u[j][i]);
          dst[ch.c0] = pack8(f);
          dst[ch.c1] = pack8(f + 8);
        }
      }
    }
  }
  // this block's dw: over the 8 lane groups of a warp by shuffles, then over the warps
  __syncthreads();
  float* red = reinterpret_cast<float*>(cs);   // [8 warps][D]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const Chunks ch = unit_chunks(sub + 4 * j, R);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = dw[j][i];
      s += __shfl_xor_sync(0xffffffffu, s, 4);
      s += __shfl_xor_sync(0xffffffffu, s, 8);
      s += __shfl_xor_sync(0xffffffffu, s, 16);
      if (lane < 4) red[warp * D + (i < 8 ? ch.c0 * 8 + i : ch.c1 * 8 + i - 8)] = s;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < D; e += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < kThreads / 32; ++v) s += red[v * D + e];
    b.part[(size_t)blockIdx.x * D + e] = s;
  }
}

// dw = the blocks' parts summed in a fixed order: 32 channels x 8 slices of the
// blocks per block; grid (D / 32, 2): queries, keys
__global__ void __launch_bounds__(256) nsa_rope_dw_kernel(const float* part, int q_blocks, int blocks, int D,
                                                          float* dw_q, float* dw_k) {
  __shared__ float red[8][32];
  const int e = blockIdx.x * 32 + (threadIdx.x & 31), sl = threadIdx.x >> 5;
  const int lo = blockIdx.y == 0 ? 0 : q_blocks, hi = blockIdx.y == 0 ? q_blocks : blocks;
  float s = 0.f;
  for (int i = lo + sl; i < hi; i += 8) s += part[(size_t)i * D + e];
  red[sl][threadIdx.x & 31] = s;
  __syncthreads();
  if (sl == 0) {
#pragma unroll
    for (int v = 1; v < 8; ++v) s += red[v][threadIdx.x & 31];
    (blockIdx.y == 0 ? dw_q : dw_k)[e] = s;
  }
}

// tokens per block: enough blocks for two per SM when there are few tokens, at
// most 8 tokens (the angles of a block serve its tokens' heads only)
static int rope_tok(int64_t N) {
  const int64_t t = N / (2 * 148);
  return t < 1 ? 1 : (t > 8 ? 8 : (int)t);
}

cudaError_t launch_qk_norm_rope(RopeArgs a, int d_k, cudaStream_t st) {
  a.tok = rope_tok(a.N);
  const unsigned grid = (unsigned)((a.N + a.tok - 1) / a.tok);
  const size_t smem = (size_t)a.tok * (a.d_rot / 2) * sizeof(float2);
#define NSA_ROPE(D)                                                                            \
  case D:                                                                                      \
    if (a.interleaved) nsa_qk_norm_rope_kernel<D, true><<<grid, kThreads, smem, st>>>(a);      \
    else nsa_qk_norm_rope_kernel<D, false><<<grid, kThreads, smem, st>>>(a);                   \
    break;
  switch (d_k) {
    NSA_ROPE(64)
    NSA_ROPE(128)
    NSA_ROPE(192)
    default: return cudaErrorInvalidValue;
  }
#undef NSA_ROPE
  return cudaGetLastError();
}

cudaError_t launch_qk_norm_rope_bwd(RopeBwdArgs b, int d_k, cudaStream_t st) {
  RopeArgs& a = b.f;
  a.tok = rope_tok(a.N);
  // two blocks per SM, dealt to queries and keys by their heads
  const int64_t groups = (a.N + a.tok - 1) / a.tok;
  int kb = (int)((int64_t)kRopeBwdBlocks * a.H_kv / (a.H_q + a.H_kv));
  if (kb < 1) kb = 1;
  int qb = kRopeBwdBlocks - kb;
  if (qb > groups) qb = (int)groups;
  if (kb > groups) kb = (int)groups;
  b.q_blocks = qb;
  const size_t ang = (size_t)a.tok * (a.d_rot / 2) * sizeof(float2), red = (size_t)(kThreads / 32) * d_k * 4;
  const size_t smem = ang > red ? ang : red;
#define NSA_ROPE(D)                                                                                   \
  case D:                                                                                             \
    if (a.interleaved) nsa_qk_norm_rope_bwd_kernel<D, true><<<qb + kb, kThreads, smem, st>>>(b);      \
    else nsa_qk_norm_rope_bwd_kernel<D, false><<<qb + kb, kThreads, smem, st>>>(b);                   \
    break;
  switch (d_k) {
    NSA_ROPE(64)
    NSA_ROPE(128)
    NSA_ROPE(192)
    default: return cudaErrorInvalidValue;
  }
#undef NSA_ROPE
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  nsa_rope_dw_kernel<<<dim3(d_k / 32, 2), 256, 0, st>>>(b.part, qb, qb + kb, d_k, b.dw_q, b.dw_k);
  return cudaGetLastError();
}

}  // namespace nsa
