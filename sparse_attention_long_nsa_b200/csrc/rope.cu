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
// rotating unit are partners, so that every rotation stays inside a thread. A warp
// takes one token and four heads at a time: it forms the token's sines and cosines
// (and, forward, their products with the weights) once, in registers, for all of its
// heads; formed per head their loads and the index arithmetic bound the kernel.
// 8192 tokens of 64 + 4 heads of 192, calls in a row: forward 90 us (4.7 TB/s of 6.55
// measured), backward 142 us (4.5 TB/s).
#include "common.cuh"
#include "kernels.h"

namespace nsa {

namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 8;                       // of a head
constexpr int kWarps = kThreads / 32;
constexpr int kWarpHeads = 32 / kLanes;         // heads a warp works on at a time

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

// cosine and sine of a token's pairs into cosv / sinv (one warp)
__device__ __forceinline__ void fill_angles(const RopeArgs& a, int64_t n, int half, float* cosv, float* sinv) {
  constexpr double k2Pi = 6.283185307179586476925286766559, kInv2Pi = 0.15915494309189533576888376337251;
  const double pos = (double)a.positions[n];
  __syncwarp();   // the token before is done with them
  for (int i = threadIdx.x & 31; i < half; i += 32) {
    const double x = pos * (double)a.inv_freq[i];
    const float r = (float)fma(-rint(x * kInv2Pi), k2Pi, x);
    float s, c;
    sincosf(r, &s, &c);
    cosv[i] = c;
    sinv[i] = s;
  }
  __syncwarp();
}

// the cosines and sines of a unit's four pairs ((1, 0) when it does not rotate):
// pair i is channels (i, 4 + i), interleaved (2i, 2i + 1)
template <bool INTER>
__device__ __forceinline__ void unit_angles(const Chunks& ch, const float* cv, const float* sv, float* c, float* s) {
  if (!ch.rot) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = 1.f;
      s[i] = 0.f;
    }
  } else if constexpr (INTER) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = (h == 0 ? ch.c0 : ch.c1) * 2;
      *reinterpret_cast<float2*>(c + 2 * h) = *reinterpret_cast<const float2*>(cv + at);
      *reinterpret_cast<float2*>(s + 2 * h) = *reinterpret_cast<const float2*>(sv + at);
    }
  } else {
    *reinterpret_cast<float4*>(c) = *reinterpret_cast<const float4*>(cv + ch.c0 * 4);
    *reinterpret_cast<float4*>(s) = *reinterpret_cast<const float4*>(sv + ch.c0 * 4);
  }
}

// out pair i = (a A_i + b B_i, a C_i + b D_i) of a unit's pairs (a, b), co = A, B, C, D
template <bool INTER>
__device__ __forceinline__ void mix_unit(float* f, const float (*co)[4]) {
  if constexpr (INTER) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p = f[2 * i], q = f[2 * i + 1];
      f[2 * i] = fmaf(q, co[1][i], p * co[0][i]);
      f[2 * i + 1] = fmaf(p, co[2][i], q * co[3][i]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      const float2 p = make_float2(f[k], f[k + 1]), q = make_float2(f[4 + k], f[5 + k]);
      const float2 y = fma2(q, make_float2(co[1][k], co[1][k + 1]), mul2(p, make_float2(co[0][k], co[0][k + 1])));
      const float2 z = fma2(p, make_float2(co[2][k], co[2][k + 1]), mul2(q, make_float2(co[3][k], co[3][k + 1])));
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

// `wpt` warps share a token's heads; a block has 8 / wpt tokens. Values are copied.
template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 2) nsa_qk_norm_rope_kernel(const RopeArgs a) {
  constexpr int U = D / 64;
  extern __shared__ float4 sm_angles[];   // cosines and sines of each warp's token
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane & (kLanes - 1), grp = lane / kLanes;
  const int64_t n = (int64_t)blockIdx.x * (kWarps / a.wpt) + warp / a.wpt;
  if (n >= a.N) return;   // the whole warp; the warps of a block do not meet
  const int first = (warp % a.wpt) * kWarpHeads + grp, step = a.wpt * kWarpHeads;
  const int half = a.d_rot >> 1, R = a.d_rot >> 2;
  float* cosv = reinterpret_cast<float*>(sm_angles) + warp * a.d_rot;
  float* sinv = cosv + half;
  int64_t row = n;   // of the key and value; a row outside the cache is not written
  if (a.cache_rows) row = a.cache_rows[n];
  const bool store_kv = row >= 0 && (!a.cache_rows || row < a.n_rows);
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + n * a.q_stride;
  const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k) + n * a.k_stride;
  uint2 raw[U][2];
  load_head<U>(q + (int64_t)first * D, first < a.H_q, sub, R, raw);
  fill_angles(a, n, half, cosv, sinv);
#pragma unroll 1
  for (int role = 0; role < (store_kv ? 2 : 1); ++role) {   // queries, keys
    const int H = role == 0 ? a.H_q : a.H_kv;
    const float* w = role == 0 ? a.w_q : a.w_k;
    const __nv_bfloat16* x = role == 0 ? q : k;
    __nv_bfloat16* y = role == 0 ? static_cast<__nv_bfloat16*>(a.q_out) + n * a.H_q * D
                                 : static_cast<__nv_bfloat16*>(a.k_out) + row * a.H_kv * D;
    if (role == 1) load_head<U>(x + (int64_t)first * D, first < H, sub, R, raw);
    if (first - grp >= H) continue;   // none for this warp
    // norm weight and rotation of a pair (a, b) in one: (a w_a c - b w_b s, a w_a s + b w_b c)
    float co[U][4][4];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const Chunks ch = unit_chunks(sub + kLanes * j, R);
      float wv[8], c[4], s[4];
      load_w(w, ch, wv);
      unit_angles<INTER>(ch, cosv, sinv, c, s);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float wa = INTER ? wv[2 * i] : wv[i], wb = INTER ? wv[2 * i + 1] : wv[4 + i];
        co[j][0][i] = wa * c[i];
        co[j][1][i] = -wb * s[i];
        co[j][2][i] = wa * s[i];
        co[j][3][i] = wb * c[i];
      }
    }
#pragma unroll 1
    for (int h = first; h - grp < H; h += step) {
      uint2 cur[U][2];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        cur[j][0] = raw[j][0];
        cur[j][1] = raw[j][1];
      }
      load_head<U>(x + (int64_t)(h + step) * D, h + step < H, sub, R, raw);
      float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < U; ++j) s2 = square_sum(cur[j], s2);
      const float r = rsqrtf(sum8(s2.x + s2.y) * (1.f / D) + a.eps);
      const float2 r2 = make_float2(r, r);
      if (h < H) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const Chunks ch = unit_chunks(sub + kLanes * j, R);
          float f[8];
          unpack4(cur[j][0], f);
          unpack4(cur[j][1], f + 4);
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float2 v = mul2(make_float2(f[i], f[i + 1]), r2);
            f[i] = v.x;
            f[i + 1] = v.y;
          }
          if (ch.rot) {
            mix_unit<INTER>(f, co[j]);
          } else {   // A and D only: 0 x (infinity or NaN) of the other channel is not 0
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              f[INTER ? 2 * i : i] *= co[j][0][i];
              f[INTER ? 2 * i + 1 : 4 + i] *= co[j][3][i];
            }
          }
          uint2* dst = reinterpret_cast<uint2*>(y + (int64_t)h * D);
          dst[ch.c0] = pack4(f);
          dst[ch.c1] = pack4(f + 4);
        }
      }
      __syncwarp();
    }
  }
  if (a.H_v > 0 && store_kv)
    for (int h = first; h < a.H_v; h += step) {
      const uint4* s4 = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.v) + n * a.v_stride +
                                                       (int64_t)h * a.d_v);
      uint4* d4 = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.v_out) + (row * a.H_kv + h) * a.d_v);
      for (int c = sub; c < a.d_v / 8; c += kLanes) d4[c] = s4[c];
    }
}

// Backward. A thread sums the query weight's gradient of its channels in registers
// and the key weight's (few heads) in shared memory of its own. part[block]: this
// block's dw_q and dw_k, its lanes summed in a fixed order. At d_k = 192 a thread takes
// 196 registers, one block an SM: held to two blocks it spilled, 177 us for 8K tokens
// against 143. The narrower heads keep that setting though they would fit twice (8K tokens
// of 32 + 4 heads: 56 us at d_k = 64 and 67 at 128; two blocks an SM 41 and 54).
template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 1) nsa_qk_norm_rope_bwd_kernel(const RopeBwdArgs b) {
  constexpr int U = D / 64;
  extern __shared__ float4 sm_angles[];   // cosines and sines of each warp's token; at the end the warps' dw
  __shared__ float4 w_s[2][D / 4];
  __shared__ float4 dwk_s[U][2][kThreads];
  const RopeArgs& a = b.f;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane & (kLanes - 1), grp = lane / kLanes;
  const int half = a.d_rot >> 1, R = a.d_rot >> 2;
  float* cosv = reinterpret_cast<float*>(sm_angles) + warp * a.d_rot;
  float* sinv = cosv + half;
  for (int i = threadIdx.x; i < D; i += kThreads) {
    reinterpret_cast<float*>(w_s[0])[i] = a.w_q[i];
    reinterpret_cast<float*>(w_s[1])[i] = a.w_k[i];
  }
  float dw[U][8];
#pragma unroll
  for (int j = 0; j < U; ++j) {
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.f;
    dwk_s[j][0][threadIdx.x] = dwk_s[j][1][threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncthreads();
  const int first = (warp % a.wpt) * kWarpHeads + grp, step = a.wpt * kWarpHeads;
  const int per = kWarps / a.wpt;   // tokens of a block at a time
  // one head: cx, cg its channels of x and of the gradient, dst its dx; adds dn h to acc
  auto head = [&](const uint2 (*cx)[2], const uint2 (*cg)[2], const float* w, bool on, uint2* dst, float (*acc)[8]) {
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < U; ++j) s2 = square_sum(cx[j], s2);
    const float r = rsqrtf(sum8(s2.x + s2.y) * (1.f / D) + a.eps);
    const float2 r2 = make_float2(r, r);
    // dn: the gradient turned back; u = dn w; m = sum(u h), h = x r
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
      if (ch.rot) {
        float c[4], s[4];
        unit_angles<INTER>(ch, cosv, sinv, c, s);
        const float co[4][4] = {{c[0], c[1], c[2], c[3]}, {s[0], s[1], s[2], s[3]},
                                {-s[0], -s[1], -s[2], -s[3]}, {c[0], c[1], c[2], c[3]}};
        mix_unit<INTER>(u[j], co);
      }
      load_w(w, ch, wv);
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float2 hx = mul2(make_float2(f[i], f[i + 1]), r2), dn = make_float2(u[j][i], u[j][i + 1]);
        const float2 t = fma2(dn, hx, make_float2(acc[j][i], acc[j][i + 1]));
        acc[j][i] = t.x;
        acc[j][i + 1] = t.y;
        const float2 v = mul2(dn, make_float2(wv[i], wv[i + 1]));
        m2 = fma2(v, hx, m2);
        u[j][i] = v.x;
        u[j][i + 1] = v.y;
      }
    }
    const float m = -sum8(m2.x + m2.y) * (1.f / D) * r;   // -mean(u h) r: h = x r below
    if (on) {
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
    __syncwarp();
  };
#pragma unroll 1
  for (int64_t n = (int64_t)blockIdx.x * per + warp / a.wpt; n < a.N; n += (int64_t)gridDim.x * per) {
    uint2 rx[U][2], rg[U][2];
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.q) + n * a.q_stride;
    const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(b.dq_out) + n * a.H_q * D;
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(b.dq) + n * b.dq_stride;
    load_head<U>(x + (int64_t)first * D, first < a.H_q, sub, R, rx);
    load_head<U>(g + (int64_t)first * D, first < a.H_q, sub, R, rg);
    fill_angles(a, n, half, cosv, sinv);
#pragma unroll 1
    for (int h = first; h - grp < a.H_q; h += step) {
      uint2 cx[U][2], cg[U][2];
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          cx[j][i] = rx[j][i];
          cg[j][i] = rg[j][i];
        }
      load_head<U>(x + (int64_t)(h + step) * D, h + step < a.H_q, sub, R, rx);
      load_head<U>(g + (int64_t)(h + step) * D, h + step < a.H_q, sub, R, rg);
      head(cx, cg, reinterpret_cast<const float*>(w_s[0]), h < a.H_q, reinterpret_cast<uint2*>(o + (int64_t)h * D), dw);
    }
    x = static_cast<const __nv_bfloat16*>(a.k) + n * a.k_stride;
    g = static_cast<const __nv_bfloat16*>(b.dk_out) + n * a.H_kv * D;
    o = static_cast<__nv_bfloat16*>(b.dk) + n * b.dk_stride;
#pragma unroll 1
    for (int h = first; h - grp < a.H_kv; h += step) {
      load_head<U>(x + (int64_t)h * D, h < a.H_kv, sub, R, rx);
      load_head<U>(g + (int64_t)h * D, h < a.H_kv, sub, R, rg);
      float acc[U][8];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        *reinterpret_cast<float4*>(acc[j]) = dwk_s[j][0][threadIdx.x];
        *reinterpret_cast<float4*>(acc[j] + 4) = dwk_s[j][1][threadIdx.x];
      }
      head(rx, rg, reinterpret_cast<const float*>(w_s[1]), h < a.H_kv, reinterpret_cast<uint2*>(o + (int64_t)h * D), acc);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        dwk_s[j][0][threadIdx.x] = *reinterpret_cast<const float4*>(acc[j]);
        dwk_s[j][1][threadIdx.x] = *reinterpret_cast<const float4*>(acc[j] + 4);
      }
    }
  }
  // this block's dw: over the 4 lane groups of a warp by shuffles, then over the warps
  float* red = reinterpret_cast<float*>(sm_angles);   // [8 warps][D]
#pragma unroll 1
  for (int role = 0; role < 2; ++role) {
    if (role == 1) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        *reinterpret_cast<float4*>(dw[j]) = dwk_s[j][0][threadIdx.x];
        *reinterpret_cast<float4*>(dw[j] + 4) = dwk_s[j][1][threadIdx.x];
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const Chunks ch = unit_chunks(sub + kLanes * j, R);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float t = dw[j][i];
        t += __shfl_xor_sync(0xffffffffu, t, 8);
        t += __shfl_xor_sync(0xffffffffu, t, 16);
        if (lane < kLanes) red[warp * D + (i < 4 ? ch.c0 * 4 + i : ch.c1 * 4 + i - 4)] = t;
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < D; e += kThreads) {
      float t = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) t += red[v * D + e];
      b.part[((size_t)blockIdx.x * 2 + role) * D + e] = t;
    }
  }
}

// dw = the blocks' parts summed in a fixed order: 32 channels x 8 slices of the
// blocks per block; grid (D / 32, 2): queries, keys
__global__ void __launch_bounds__(256) nsa_rope_dw_kernel(const float* part, int blocks, int D, float* dw_q, float* dw_k) {
  __shared__ float red[8][32];
  const int e = blockIdx.x * 32 + (threadIdx.x & 31), sl = threadIdx.x >> 5;
  float s = 0.f;
#pragma unroll 8
  for (int i = sl; i < blocks; i += 8) s += part[((size_t)i * 2 + blockIdx.y) * D + e];
  red[sl][threadIdx.x & 31] = s;
  __syncthreads();
  if (sl == 0) {
#pragma unroll
    for (int v = 1; v < 8; ++v) s += red[v][threadIdx.x & 31];
    (blockIdx.y == 0 ? dw_q : dw_k)[e] = s;
  }
}

// Warps that share a token: as many as its heads can use while the tokens alone do
// not give every SM two blocks (a decode step of 32 tokens: 8; from 2368 tokens on 1).
static int rope_wpt(int64_t N, int H) {
  int wpt = 1;
  while (wpt < kWarps && wpt * kWarpHeads < H && N * wpt < 2 * 148 * kWarps) wpt *= 2;
  return wpt;
}

cudaError_t launch_qk_norm_rope(RopeArgs a, int d_k, cudaStream_t st) {
  a.wpt = rope_wpt(a.N, a.H_q);
  const int per = kWarps / a.wpt;
  const unsigned grid = (unsigned)((a.N + per - 1) / per);
  const size_t smem = (size_t)kWarps * a.d_rot * sizeof(float);
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
  a.wpt = rope_wpt(a.N, a.H_q);
  const int per = kWarps / a.wpt;
  const int64_t groups = (a.N + per - 1) / per;
  const int grid = groups < kRopeBwdBlocks ? (int)groups : kRopeBwdBlocks;
  const size_t ang = (size_t)kWarps * a.d_rot * sizeof(float), red = (size_t)kWarps * d_k * 4;
  const size_t smem = ang > red ? ang : red;
#define NSA_ROPE(D)                                                                                   \
  case D:                                                                                             \
    if (a.interleaved) nsa_qk_norm_rope_bwd_kernel<D, true><<<grid, kThreads, smem, st>>>(b);      \
    else nsa_qk_norm_rope_bwd_kernel<D, false><<<grid, kThreads, smem, st>>>(b);                   \
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
  nsa_rope_dw_kernel<<<dim3(d_k / 32, 2), 256, 0, st>>>(b.part, grid, d_k, b.dw_q, b.dw_k);
  return cudaGetLastError();
}

}  // namespace nsa
