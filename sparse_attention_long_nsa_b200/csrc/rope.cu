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
// Both are bound by memory: 4 bytes per element forward, 6 backward. Eight lanes own
// a head: a lane holds d_k / 64 units, a unit being two 8-byte chunks of 4 channels
// (with 16-byte chunks and four lanes the backward's sums of dw alone took 48
// registers and it spilled). For pairs (i, i + d_rot / 2) the two chunks of a
// rotating unit are partners, so that every rotation stays inside a thread. The
// sines and cosines of a block's tokens are computed once into shared memory and
// serve all heads; a head's channels are loaded while the head before is worked on.
#include "common.cuh"
#include "kernels.h"

namespace nsa {

namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 8;                       // of a head
constexpr int kGroups = kThreads / kLanes;      // heads in work at a time

struct Chunks {
  int c0, c1;   // the two 4-channel chunks of a unit
  bool rot;
};
// unit u of a head of which R = d_rot / 4 chunks rotate
__device__ __forceinline__ Chunks unit_chunks(int u, int R) {
  const int half = R >> 1;
  Chunks c;
  c.rot = u < half;
  c.c0 = c.rot ? u : R + 2 * (u - half);
  c.c1 = c.rot ? u + half : c.c0 + 1;
  return c;
}

__device__ __forceinline__ void unpack4(const uint2& w, float* f) {
  f[0] = __uint_as_float(w.x << 16);
  f[1] = __uint_as_float(w.x & 0xffff0000u);
  f[2] = __uint_as_float(w.y << 16);
  f[3] = __uint_as_float(w.y & 0xffff0000u);
}
__device__ __forceinline__ uint2 pack4(const float* f) {
  return make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
}
__device__ __forceinline__ float sum8(float x) {
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// cosine and sine of pair i of tokens n0 .. n0 + nt - 1 into cosv / sinv[tok * half + i]
__device__ __forceinline__ void fill_angles(const RopeArgs& a, int64_t n0, int nt, int half, float* cosv, float* sinv) {
  constexpr double k2Pi = 6.283185307179586476925286766559, kInv2Pi = 0.15915494309189533576888376337251;
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int tok = i / half;
    const double x = (double)a.positions[n0 + tok] * (double)a.inv_freq[i - tok * half];
    const float r = (float)fma(-rint(x * kInv2Pi), k2Pi, x);
    float s, c;
    sincosf(r, &s, &c);
    cosv[i] = c;
    sinv[i] = s;
  }
}

// turn the pairs of a unit (SIGN -1: by the opposite angle); f[0..3] and f[4..7]
// are its two chunks, first channel 4 * c0 / 4 * c1; cv, sv: the token's row
template <bool INTER, int SIGN>
__device__ __forceinline__ void turn_unit(float* f, const Chunks& ch, const float* cv, const float* sv) {
  if constexpr (INTER) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = (h == 0 ? ch.c0 : ch.c1) * 2;
      const float2 c2 = *reinterpret_cast<const float2*>(cv + at), s2 = *reinterpret_cast<const float2*>(sv + at);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float c = i == 0 ? c2.x : c2.y, s = SIGN * (i == 0 ? s2.x : s2.y);
        const float p = f[4 * h + 2 * i], q = f[4 * h + 2 * i + 1];
        f[4 * h + 2 * i] = fmaf(q, -s, p * c);
        f[4 * h + 2 * i + 1] = fmaf(p, s, q * c);
      }
    }
  } else {
    const float4 c4 = *reinterpret_cast<const float4*>(cv + ch.c0 * 4), s4 = *reinterpret_cast<const float4*>(sv + ch.c0 * 4);
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      const float2 c = k == 0 ? make_float2(c4.x, c4.y) : make_float2(c4.z, c4.w);
      const float2 s = k == 0 ? make_float2(SIGN * s4.x, SIGN * s4.y) : make_float2(SIGN * s4.z, SIGN * s4.w);
      const float2 p = make_float2(f[k], f[k + 1]), q = make_float2(f[4 + k], f[5 + k]);
      const float2 y = fma2(q, make_float2(-s.x, -s.y), mul2(p, c)), z = fma2(p, s, mul2(q, c));
      f[k] = y.x;
      f[k + 1] = y.y;
      f[4 + k] = z.x;
      f[5 + k] = z.y;
    }
  }
}

// squares of a unit's 8 bf16 channels, added to the two partial sums of ss
__device__ __forceinline__ float2 square_sum(const uint2* raw, float2 ss) {
  float f[8];
  unpack4(raw[0], f);
  unpack4(raw[1], f + 4);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 v = make_float2(f[i], f[i + 1]);
    ss = fma2(v, v, ss);
  }
  return ss;
}

// the 8 weights of a unit
__device__ __forceinline__ void load_w(const float* w, const Chunks& ch, float* wv) {
  *reinterpret_cast<float4*>(wv) = *reinterpret_cast<const float4*>(w + ch.c0 * 4);
  *reinterpret_cast<float4*>(wv + 4) = *reinterpret_cast<const float4*>(w + ch.c1 * 4);
}

// a lane's units of the head at x (zeros without one)
template <int U>
__device__ __forceinline__ void load_head(const __nv_bfloat16* x, bool on, int sub, int R, uint2 raw[U][2]) {
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const Chunks ch = unit_chunks(sub + kLanes * j, R);
    raw[j][0] = on ? reinterpret_cast<const uint2*>(x)[ch.c0] : make_uint2(0, 0);
    raw[j][1] = on ? reinterpret_cast<const uint2*>(x)[ch.c1] : make_uint2(0, 0);
  }
}

}  // namespace

// One block: `tok` tokens, all their query, key (and value) heads, dealt to the 32
// lane groups in turn. Values are copied.
template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads) nsa_qk_norm_rope_kernel(const RopeArgs a) {
  constexpr int U = D / 64;
  extern __shared__ float4 sm_angles[];   // cosines, then sines
  float* cosv = reinterpret_cast<float*>(sm_angles);
  const int64_t n0 = (int64_t)blockIdx.x * a.tok;
  const int nt = (int)min((int64_t)a.tok, a.N - n0);
  const int half = a.d_rot >> 1, R = a.d_rot >> 2;
  float* sinv = cosv + a.tok * half;
  const int sub = threadIdx.x & (kLanes - 1), grp = threadIdx.x / kLanes;
  const int H = a.H_q + a.H_kv, HA = H + a.H_v;
  const int total = nt * HA;
  struct Item {
    int64_t n;
    int tok, h;
    bool on;
  };
  auto item_of = [&](int i) -> Item {
    Item it;
    it.on = i < total;
    it.tok = it.on ? i / HA : 0;
    it.h = it.on ? i - it.tok * HA : 0;
    it.n = n0 + it.tok;
    return it;
  };
  auto src = [&](const Item& it) -> const __nv_bfloat16* {
    return it.h < a.H_q ? static_cast<const __nv_bfloat16*>(a.q) + it.n * a.q_stride + (int64_t)it.h * D
                        : static_cast<const __nv_bfloat16*>(a.k) + it.n * a.k_stride + (int64_t)(it.h - a.H_q) * D;
  };
  Item it = item_of(grp);
  uint2 raw[U][2], nxt[U][2];
  load_head<U>(src(it), it.on && it.h < H, sub, R, raw);
  fill_angles(a, n0, nt, half, cosv, sinv);
  __syncthreads();
  for (int base = 0; base < total; base += kGroups) {
    const Item ni = item_of(base + kGroups + grp);
    load_head<U>(src(ni), ni.on && ni.h < H, sub, R, nxt);
    const bool is_q = it.h < a.H_q, is_v = it.h >= H;
    int64_t row = it.n;
    bool write = it.on;
    if (!is_q && a.cache_rows) {   // a row outside the cache is not written
      row = a.cache_rows[it.n];
      write = it.on && row >= 0 && row < a.n_rows;
    }
    if (is_v && write) {
      const int hv = it.h - H;
      const uint4* s4 = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.v) + it.n * a.v_stride +
                                                       (int64_t)hv * a.d_v);
      uint4* d4 = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.v_out) + (row * a.H_kv + hv) * a.d_v);
      for (int c = sub; c < a.d_v / 8; c += kLanes) d4[c] = s4[c];
    }
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < U; ++j) s2 = square_sum(raw[j], s2);
    const float r = rsqrtf(sum8(s2.x + s2.y) * (1.f / D) + a.eps);
    if (write && !is_v) {
      const float* w = is_q ? a.w_q : a.w_k;
      __nv_bfloat16* y = is_q ? static_cast<__nv_bfloat16*>(a.q_out) + (it.n * a.H_q + it.h) * D
                              : static_cast<__nv_bfloat16*>(a.k_out) + (row * a.H_kv + it.h - a.H_q) * D;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const Chunks ch = unit_chunks(sub + kLanes * j, R);
        float f[8], wv[8];
        unpack4(raw[j][0], f);
        unpack4(raw[j][1], f + 4);
        load_w(w, ch, wv);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float2 v = mul2(make_float2(f[i], f[i + 1]), mul2(make_float2(wv[i], wv[i + 1]), make_float2(r, r)));
          f[i] = v.x;
          f[i + 1] = v.y;
        }
        if (ch.rot) turn_unit<INTER, 1>(f, ch, cosv + it.tok * half, sinv + it.tok * half);
        reinterpret_cast<uint2*>(y)[ch.c0] = pack4(f);
        reinterpret_cast<uint2*>(y)[ch.c1] = pack4(f + 4);
      }
    }
    it = ni;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      raw[j][0] = nxt[j][0];
      raw[j][1] = nxt[j][1];
    }
  }
}

// Backward. grid.x blocks walk the token groups; blocks below `q_blocks` take the
// query heads, the others the key heads, so that a thread's dw sums belong to one
// weight. part[block][D]: this block's dw, its groups summed in a fixed order.
template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 2) nsa_qk_norm_rope_bwd_kernel(const RopeBwdArgs b) {
  constexpr int U = D / 64;
  extern __shared__ float4 sm_angles[];   // cosines, then sines; at the end the warps' dw
  float* cosv = reinterpret_cast<float*>(sm_angles);
  const RopeArgs& a = b.f;
  const int half = a.d_rot >> 1, R = a.d_rot >> 2;
  float* sinv = cosv + a.tok * half;
  const int sub = threadIdx.x & (kLanes - 1), grp = threadIdx.x / kLanes;
  const bool is_q = (int)blockIdx.x < b.q_blocks;
  const int blk = is_q ? blockIdx.x : blockIdx.x - b.q_blocks;
  const int nblk = is_q ? b.q_blocks : (int)gridDim.x - b.q_blocks;
  const int H = is_q ? a.H_q : a.H_kv;
  const float* w = is_q ? a.w_q : a.w_k;
  const __nv_bfloat16* xb = static_cast<const __nv_bfloat16*>(is_q ? a.q : a.k);
  const __nv_bfloat16* gb = static_cast<const __nv_bfloat16*>(is_q ? b.dq_out : b.dk_out);
  __nv_bfloat16* ob = static_cast<__nv_bfloat16*>(is_q ? b.dq : b.dk);
  const int64_t xs = is_q ? a.q_stride : a.k_stride, os = is_q ? b.dq_stride : b.dk_stride;
  float dw[U][8];
#pragma unroll
  for (int j = 0; j < U; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.f;
  for (int64_t n0 = (int64_t)blk * a.tok; n0 < a.N; n0 += (int64_t)nblk * a.tok) {
    const int nt = (int)min((int64_t)a.tok, a.N - n0);
    const int total = nt * H;
    uint2 rx[U][2], rg[U][2];
    auto load = [&](int i) {
      const bool on = i < total;
      const int tok = on ? i / H : 0, h = on ? i - tok * H : 0;
      load_head<U>(xb + (n0 + tok) * xs + (int64_t)h * D, on, sub, R, rx);
      load_head<U>(gb + ((n0 + tok) * H + h) * D, on, sub, R, rg);
    };
    load(grp);
    __syncthreads();
    fill_angles(a, n0, nt, half, cosv, sinv);
    __syncthreads();
    for (int base = 0; base < total; base += kGroups) {
      const int item = base + grp;
      const bool on = item < total;
      const int tok = on ? item / H : 0;
      const int h = on ? item - tok * H : 0;
      const int64_t n = n0 + tok;
      uint2 cx[U][2], cg[U][2];
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          cx[j][i] = rx[j][i];
          cg[j][i] = rg[j][i];
        }
      if (base + kGroups < total) load(item + kGroups);
      float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < U; ++j) s2 = square_sum(cx[j], s2);
      const float r = rsqrtf(sum8(s2.x + s2.y) * (1.f / D) + a.eps);
      const float2 r2 = make_float2(r, r);
      // u = dn w (dn: the gradient turned back); dw += dn h; m = sum(u h), h = x r
      float u[U][8];
      float2 m2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const Chunks ch = unit_chunks(sub + kLanes * j, R);
        float f[8], wv[8];
        unpack4(cg[j][0], u[j]);
        unpack4(cg[j][1], u[j] + 4);
        unpack4(cx[j][0], f);
        unpack4(cx[j][1], f + 4);
        if (ch.rot) turn_unit<INTER, -1>(u[j], ch, cosv + tok * half, sinv + tok * half);
        load_w(w, ch, wv);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float2 hx = mul2(make_float2(f[i], f[i + 1]), r2), dn = make_float2(u[j][i], u[j][i + 1]);
          const float2 t = fma2(dn, hx, make_float2(dw[j][i], dw[j][i + 1]));
          dw[j][i] = t.x;
          dw[j][i + 1] = t.y;
          const float2 v = mul2(dn, make_float2(wv[i], wv[i + 1]));
          m2 = fma2(v, hx, m2);
          u[j][i] = v.x;
          u[j][i + 1] = v.y;
        }
      }
      const float m = -sum8(m2.x + m2.y) * (1.f / D) * r;   // -mean(u h) r: h = x r below
      if (on) {
        uint2* dst = reinterpret_cast<uint2*>(ob + n * os + (int64_t)h * D);
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const Chunks ch = unit_chunks(sub + kLanes * j, R);
          float f[8];
          unpack4(cx[j][0], f);
          unpack4(cx[j][1], f + 4);
#pragma unroll
          for (int i = 0; i < 8; i += 2) {   // r (u - h mean(u h))
            const float2 v = mul2(r2, fma2(make_float2(f[i], f[i + 1]), make_float2(m, m), make_float2(u[j][i], u[j][i + 1])));
            f[i] = v.x;
            f[i + 1] = v.y;
          }
          dst[ch.c0] = pack4(f);
          dst[ch.c1] = pack4(f + 4);
        }
      }
    }
  }
  // this block's dw: over the 4 lane groups of a warp by shuffles, then over the warps
  __syncthreads();
  float* red = cosv;   // [8 warps][D]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const Chunks ch = unit_chunks(sub + kLanes * j, R);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s = dw[j][i];
      s += __shfl_xor_sync(0xffffffffu, s, 8);
      s += __shfl_xor_sync(0xffffffffu, s, 16);
      if (lane < kLanes) red[warp * D + (i < 4 ? ch.c0 * 4 + i : ch.c1 * 4 + i - 4)] = s;
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
  const size_t smem = (size_t)a.tok * a.d_rot * sizeof(float);
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
  const size_t ang = (size_t)a.tok * a.d_rot * sizeof(float), red = (size_t)(kThreads / 32) * d_k * 4;
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
