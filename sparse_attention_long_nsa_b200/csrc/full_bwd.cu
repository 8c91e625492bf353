// Backward of the causal full attention over packed prompts, on tcgen05.
//
// With P = exp(scale q K^T - lse) recomputed from the forward's lse,
//   dV = P^T dO,  dP = dO V^T,  dS = P o (dP - delta),  delta = rowsum(dO o O),
//   dQ = scale dS K,  dK = scale dS^T Q.
// P and dS are rounded to bf16 for their products (as P in the forward); sums,
// delta and the exponent stay in fp32, the results are rounded once.
//
// Three kernels, none of which adds into memory that another block adds into, so
// the results do not depend on timing:
//   bwd_row     (lse in log2 units, delta) of every row
//   bwd_kv      a block of 128 keys of one key head against all (token, head) rows
//               that see it, 128 rows at a time: S^T = K Q^T, dP^T = V dO^T (keys in
//               the tensor-memory lanes), so that P^T and dS^T are written where they
//               are the A operand of dV += P^T dO and dK += dS^T Q. The heads that
//               share the key head are rows like any others.
//   bwd_q       128 rows against the keys they see: S, dP, dQ += dS K
// S and dP are formed twice, seven products instead of five: one pass that also
// accumulated dQ would add fp32 atomics in an order that differs between runs.
//
// Tensor memory (512 columns) of bwd_kv: S^T 0-127, over whose first half P^T is
// written; dP^T 64-191, over whose second half dS^T is written; dV 128, dK 192. That
// leaves S^T of the next row tile free to be formed while dS^T of this one is: the
// products run dP, dV, next S, dK, and each waits for work that the one or two before
// it hid (without the look-ahead every tile waited for its whole chain).
// bwd_q: S 128, dP 128, dQ 192, dS 64; the next tile's S is issued before dQ.
//
// Measured, 4096 tokens, 64 heads on 4 key heads, 192 / 128, each kernel alone (single
// launches under the profiler): bwd_kv 655 us (four of the seven products, 1.05 PFLOP/s,
// tensor pipe 57 % active), bwd_q 570 us (three, 0.96 PFLOP/s, 50 %), bwd_row 24 us, the
// merge 11 us.
#include "common.cuh"
#include "kernels.h"

namespace nsa {

namespace {

constexpr int kThreads = 608;   // 16 warps of elementwise work, loads, products, row values
constexpr int kEl = 512;        // elementwise threads: four warps share a row's columns, 32 each
constexpr int kPiece = 16384;   // 128 rows x 64 channels, 128-byte swizzled
constexpr int kRows = 128;

// Streamed operands: two stages of the d_k wide one, and of the d_v wide one as many
// as fit beside them and the resident tiles (one at 192 + 128: its next tile is
// loaded while the two products after its last use run). A stage's pieces are
// adjacent, so that it is one operand of 64, 128 or 192 columns: products of 64
// columns that take their other operand from tensor memory run at half the rate.
__host__ __device__ constexpr int wide_stages(int dk, int dv) {
  return (232448 - 1024 - 4096 - (dk + dv) * 256 - 2 * dk * 256) / (dv * 256) >= 2 ? 2 : 1;
}
__host__ __device__ constexpr int bwd_smem(int dk, int dv) {
  return 1024 + (dk + dv) * 256 + 2 * dk * 256 + wide_stages(dk, dv) * dv * 256 + 4096;
}

struct BwdBars {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];   // stages of the d_k / d_v wide operand
  uint64_t fix_full, fix_empty;               // the block's resident operands
  uint64_t s_full, s_read, p_full, dp_full, dp_read, ds_full, ds_free, acc_full, drain;
  uint64_t row_full[2], row_empty[2];
  uint32_t tmem_base;
  int abort;
};

// zeros from row `from` of a piece on (one warp)
__device__ __forceinline__ void clear_rows(uint8_t* piece, int from, int lane) {
  for (int i = from * 8 + lane; i < kRows * 8; i += 32) *reinterpret_cast<uint4*>(piece + i * 16) = make_uint4(0, 0, 0, 0);
}

// one lane waits for the copies in flight before its block exits
__device__ __forceinline__ void drain_loads(BwdBars* bars, int segs, uint32_t k_n, uint32_t v_n, uint32_t vs) {
  if (segs > 0) mbar_wait_drain(&bars->fix_full, (segs - 1) & 1);
  for (uint32_t i = k_n < 2 ? 0 : k_n - 2; i < k_n; ++i) mbar_wait_drain(&bars->k_full[i & 1], (i >> 1) & 1);
  for (uint32_t i = v_n < vs ? 0 : v_n - vs; i < v_n; ++i) mbar_wait_drain(&bars->v_full[i % vs], (i / vs) & 1);
}

// dO o O summed over a row, beside the row's lse in log2 units: 8 channels a lane
template <int DV>
__global__ void __launch_bounds__(256) nsa_full_bwd_row_kernel(const FullBwdArgs a) {
  constexpr int L = DV / 8;   // lanes of a row
  const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) / L;
  const int sub = threadIdx.x % L;
  if (row >= a.n_rows) return;   // whole rows: the lanes of a row leave together
  const uint4 o = reinterpret_cast<const uint4*>(a.out)[row * L + sub];
  const uint4 g = reinterpret_cast<const uint4*>(a.dout)[row * L + sub];
  const uint32_t ov[4] = {o.x, o.y, o.z, o.w}, gv[4] = {g.x, g.y, g.z, g.w};
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(__uint_as_float(ov[i] << 16), __uint_as_float(gv[i] << 16), s);
    s = fmaf(__uint_as_float(ov[i] & 0xffff0000u), __uint_as_float(gv[i] & 0xffff0000u), s);
  }
  const uint32_t mask = L == 32 ? 0xffffffffu : ((1u << L) - 1u) << ((threadIdx.x & 31) & ~(L - 1));
#pragma unroll
  for (int w = L / 2; w >= 1; w >>= 1) s += __shfl_xor_sync(mask, s, w);
  if (sub == 0) a.row[row] = make_float2(a.lse[row] * 1.4426950408889634f, s);
}

// ---- key blocks: the row tiles of all units in a row, cut into equal runs ----
struct KvSeg {
  int b, g, kt;       // sequence, key head, key block
  int L;              // tokens of the sequence
  int64_t tok0;       // its first row
  int r0, n;          // first row tile (of 128 / G tokens) and how many
  int slot;           // partial slot, -1: the whole unit
};
struct KvPlace {
  int b, g, kt;
  int64_t start, cnt; // first tile and number of tiles of the unit
};
// the unit that holds tile `pos`; a unit of sequence b has R - kt G tiles (R row
// tiles in the sequence, of which the first kt G lie before the key block)
__device__ __forceinline__ KvPlace kv_place(const FullBwdArgs& a, int64_t pos) {
  int lo = 0, hi = a.batch - 1;
  while (lo < hi) {   // last b with kv_prefix[b] <= pos
    const int mid = (lo + hi + 1) >> 1;
    if (a.kv_prefix[mid] <= pos) lo = mid; else hi = mid - 1;
  }
  KvPlace p;
  p.b = lo;
  const int L = a.len[lo], TOK = kRows / a.G;
  const int64_t R = (L + TOK - 1) / TOK, T = (L + kRows - 1) / kRows;
  const int64_t per_g = T * R - (int64_t)a.G * (T * (T - 1) / 2);
  const int64_t in_b = pos - a.kv_prefix[lo];
  p.g = (int)(in_b / per_g);
  const int64_t rem = in_b - p.g * per_g;
  int k0 = 0, k1 = (int)T - 1;
  while (k0 < k1) {   // last kt with kt R - G kt (kt - 1) / 2 <= rem
    const int64_t mid = (k0 + k1 + 1) >> 1;
    if (mid * R - (int64_t)a.G * (mid * (mid - 1) / 2) <= rem) k0 = (int)mid; else k1 = (int)mid - 1;
  }
  p.kt = k0;
  const int64_t first = (int64_t)k0 * R - (int64_t)a.G * ((int64_t)k0 * (k0 - 1) / 2);
  p.start = a.kv_prefix[lo] + p.g * per_g + first;
  p.cnt = R - (int64_t)k0 * a.G;
  return p;
}
__device__ __forceinline__ int64_t run_begin(const FullBwdArgs& a, int c, int blocks) {
  const int64_t W = a.kv_prefix[a.batch];
  return W / blocks * c + W % blocks * c / blocks;   // no product of W and c: W may be large
}

struct KvSched {
  const FullBwdArgs& a;
  int64_t pos, end;
  __device__ explicit KvSched(const FullBwdArgs& a_) : a(a_) {
    pos = run_begin(a, blockIdx.x, gridDim.x);
    end = run_begin(a, blockIdx.x + 1, gridDim.x);
  }
  __device__ bool next(KvSeg& s) {
    if (pos >= end) return false;
    const KvPlace p = kv_place(a, pos);
    const int64_t off = pos - p.start;
    const int64_t n = min(p.cnt - off, end - pos);
    s.b = p.b;
    s.g = p.g;
    s.kt = p.kt;
    s.L = a.len[p.b];
    s.tok0 = a.tok_off[p.b];
    s.r0 = p.kt * a.G + (int)off;
    s.n = (int)n;
    s.slot = n == p.cnt ? -1 : 2 * (int)blockIdx.x + (off == 0 ? 1 : 0);
    pos += n;
    return true;
  }
};

__device__ __forceinline__ void bwd_init(BwdBars* bars) {
  for (int i = 0; i < 2; ++i) {
    mbar_init(&bars->k_full[i], 1);
    mbar_init(&bars->k_empty[i], 1);
    mbar_init(&bars->v_full[i], 1);
    mbar_init(&bars->v_empty[i], 1);
  }
  mbar_init(&bars->fix_full, 1);
  mbar_init(&bars->fix_empty, 1);
  mbar_init(&bars->s_full, 1);
  mbar_init(&bars->s_read, kEl);
  mbar_init(&bars->p_full, kEl);
  mbar_init(&bars->dp_full, 1);
  mbar_init(&bars->dp_read, kEl);
  mbar_init(&bars->ds_full, kEl);
  mbar_init(&bars->ds_free, 1);
  mbar_init(&bars->acc_full, 1);
  mbar_init(&bars->drain, 1);
  for (int i = 0; i < 2; ++i) {
    mbar_init(&bars->row_full[i], 32);
    mbar_init(&bars->row_empty[i], kEl);
  }
  bars->abort = 0;
  fence_mbar_init();
}

__device__ __forceinline__ uint4 pack_out(const float* v, float f) {
  return make_uint4(pack_bf16x2(v[0] * f, v[1] * f), pack_bf16x2(v[2] * f, v[3] * f), pack_bf16x2(v[4] * f, v[5] * f),
                    pack_bf16x2(v[6] * f, v[7] * f));
}

}  // namespace

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1) nsa_full_bwd_kv_kernel(const FullBwdArgs a,
                                                                      const __grid_constant__ FullBwdMaps mp) {
  constexpr int KC = DK / 64, VC = DV / 64, VS = wide_stages(DK, DV);
  constexpr int kKStage = KC * kPiece, kVStage = VC * kPiece;
  constexpr uint32_t kColDP = 64, kColDS = 128, kColDV = 192, kColDK = 320;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* Ks = smem;                       // K pieces, then V pieces
  uint8_t* Vs = Ks + KC * kPiece;
  uint8_t* Qr = Vs + kVStage;               // streamed Q, dO
  uint8_t* Gr = Qr + 2 * kKStage;
  float* rowv = reinterpret_cast<float*>(Gr + VS * kVStage);      // [2][-lse | -delta][128] of the row tile
  BwdBars* bars = reinterpret_cast<BwdBars*>(rowv + 4 * kRows);
  volatile int* abort_flag = &bars->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) bwd_init(bars);
  if (warp == 0) tmem_alloc(&bars->tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t tmem = bars->tmem_base;
  const int TOK = kRows / a.G;
  KvSched sched(a);
  KvSeg sg;
  sg.slot = -1;
  bool ok = true;
  auto uwait = [&](uint64_t* bar, uint32_t parity, uint32_t site) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity & 1u, abort_flag, a.status, site));
  };

  if (warp == 16) {
    // ------------------------------------------------------------ loads
    uint32_t k_n = 0, v_n = 0;   // stages filled
    uint32_t tiles = 0;
    int segs = 0;
    while (ok && sched.next(sg)) {
      if (segs > 0) ok = uwait(&bars->fix_empty, segs - 1, 641);
      if (!ok) break;
      if (lane == 0) {
        const int row = (int)(sg.tok0 + (int64_t)sg.kt * kRows);
        mbar_arrive_expect_tx(&bars->fix_full, (KC + VC) * kPiece);
        for (int c = 0; c < KC; ++c) tma_load_3d(Ks + c * kPiece, &mp.k, &bars->fix_full, c * 64, sg.g, row);
        for (int c = 0; c < VC; ++c) tma_load_3d(Vs + c * kPiece, &mp.v, &bars->fix_full, c * 64, sg.g, row);
      }
      ++segs;
      for (int j = 0; j < sg.n && ok; ++j, ++tiles) {
        const int row = (int)(sg.tok0 + (int64_t)(sg.r0 + j) * TOK);
        const uint32_t ks = tiles & 1, vs = tiles % VS;
        if (tiles >= 2) ok = uwait(&bars->k_empty[ks], (tiles >> 1) - 1, 642);
        if (!ok) break;
        if (lane == 0 && !(tiles == 0 && NSA_INJECT(a, FAULT_FULL_BWD_TILE))) {   // checking build: withhold the first
          mbar_arrive_expect_tx(&bars->k_full[ks], kKStage);
          for (int c = 0; c < KC; ++c)
            tma_load_3d(Qr + ks * kKStage + c * kPiece, &mp.q, &bars->k_full[ks], c * 64, sg.g * a.G, row);
        }
        ++k_n;
        if (tiles >= VS) ok = uwait(&bars->v_empty[vs], tiles / VS - 1, 643);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars->v_full[vs], kVStage);
          for (int c = 0; c < VC; ++c)
            tma_load_3d(Gr + vs * kVStage + c * kPiece, &mp.dout, &bars->v_full[vs], c * 64, sg.g * a.G, row);
        }
        ++v_n;
      }
    }
    if (!ok && lane == 0) drain_loads(bars, segs, k_n, v_n, VS);
  } else if (warp == 17) {
    // ------------------------------------------------------------ products
    // (operands uniform over the warp, see the forward kernel)
    const uint32_t tm = uni(tmem);
    const uint32_t id_s = umma_idesc_bf16(128, 128, false, false);
    const uint32_t id_v = umma_idesc_bf16(128, DV, false, true), id_k = umma_idesc_bf16(128, DK, false, true);
    const uint64_t kd = umma_desc_sw128(uni(smem_u32(Ks)), 16, 1024), vd = umma_desc_sw128(uni(smem_u32(Vs)), 16, 1024);
    const uint32_t q_a = uni(smem_u32(Qr)), g_a = uni(smem_u32(Gr));
    const uint64_t qs = umma_desc_sw128(q_a, 16, 1024), gs = umma_desc_sw128(g_a, 16, 1024);             // rows x channels
    const uint64_t qt = umma_desc_sw128(q_a, kPiece, 1024), gt = umma_desc_sw128(g_a, kPiece, 1024);     // channels x rows
    uint32_t tiles = 0;
    int segs = 0;
    while (ok && sched.next(sg)) {
      const int n = uni(sg.n), L = uni(sg.L), r0 = uni(sg.r0);
      ok = uwait(&bars->fix_full, segs, 651);
      if (!ok) break;
      ++segs;
      // S^T of a tile = K Q^T at stage ks (one lane)
      auto scores = [&](uint32_t ks) {
        const uint64_t q = qs + (uint64_t)(ks * (kKStage >> 4));
#pragma unroll
        for (int kk = 0; kk < KC * 4; ++kk) {
          const uint64_t o = (uint64_t)((kk >> 2) * (kPiece >> 4) + (kk & 3) * 2);
          umma_ss(tm, kd + o, q + o, id_s, kk ? 1u : 0u);
        }
        umma_commit(&bars->s_full);
      };
      auto clear_q = [&](int j, uint32_t ks) {   // rows of tile j past the last token
        const int left = min(L - (r0 + j) * TOK, TOK) * a.G;
        if (left < kRows) {
          for (int c = 0; c < KC; ++c) clear_rows(Qr + ks * kKStage + c * kPiece, left, lane);
          fence_proxy_async_smem();
          __syncwarp();
        }
      };
      ok = uwait(&bars->k_full[tiles & 1], tiles >> 1, 652);
      if (!ok) break;
      clear_q(0, tiles & 1);
      if (elect_one()) {
        tc_fence_after();
        scores(tiles & 1);
      }
      __syncwarp();
      // step j: dP of tile j; dV of tile j and S of tile j + 1; dK of tile j
#pragma unroll 1
      for (int j = 0; j < n && ok; ++j, ++tiles) {
        const uint32_t ks = tiles & 1, vs = tiles % VS;   // of tile j
        const int left = min(L - (r0 + j) * TOK, TOK) * a.G;
        // dP^T = V dO^T beside P: the upper columns of S^T have to be read
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->v_full[vs], (tiles / VS) & 1, abort_flag, a.status, 653) &&
                                         mbar_wait(&bars->s_read, tiles & 1, abort_flag, a.status, 654));
        if (!ok) break;
        if (left < kRows) {
          for (int c = 0; c < VC; ++c) clear_rows(Gr + vs * kVStage + c * kPiece, left, lane);
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (elect_one()) {
          tc_fence_after();
          const uint64_t g = gs + (uint64_t)(vs * (kVStage >> 4));
#pragma unroll
          for (int kk = 0; kk < VC * 4; ++kk) {
            const uint64_t o = (uint64_t)((kk >> 2) * (kPiece >> 4) + (kk & 3) * 2);
            umma_ss(tm + kColDP, vd + o, g + o, id_s, kk ? 1u : 0u);
          }
          umma_commit(&bars->dp_full);
          if (j + 1 == n) umma_commit(&bars->fix_empty);
        }
        __syncwarp();
        // dV += P^T dO; then S over P and the half of dP that has been read
        ok = __all_sync(0xffffffffu,
                        mbar_wait(&bars->p_full, tiles & 1, abort_flag, a.status, 655) &&
                            (j + 1 == n || (mbar_wait(&bars->k_full[ks ^ 1], ((tiles + 1) >> 1) & 1, abort_flag, a.status, 652) &&
                                            mbar_wait(&bars->dp_read, tiles & 1, abort_flag, a.status, 657))));
        if (!ok) break;
        if (j + 1 < n) clear_q(j + 1, ks ^ 1);
        if (elect_one()) {
          tc_fence_after();
          const uint64_t g = gt + (uint64_t)(vs * (kVStage >> 4));
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_ts(tm + kColDV, tm + kk * 8, g + (uint64_t)(kk * (2048 >> 4)), id_v, (j | kk) ? 1u : 0u);
          umma_commit(&bars->v_empty[vs]);
          if (j + 1 < n) scores(ks ^ 1);
        }
        __syncwarp();
        // dK += dS^T Q
        ok = uwait(&bars->ds_full, tiles, 656);
        if (!ok) break;
        if (elect_one()) {
          tc_fence_after();
          const uint64_t q = qt + (uint64_t)(ks * (kKStage >> 4));
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_ts(tm + kColDK, tm + kColDS + kk * 8, q + (uint64_t)(kk * (2048 >> 4)), id_k, (j | kk) ? 1u : 0u);
          umma_commit(&bars->k_empty[ks]);
          if (j + 1 == n) umma_commit(&bars->acc_full);
        }
        __syncwarp();
      }
    }
    if (elect_one()) {   // every product has finished before tensor memory is released
      umma_commit(&bars->drain);
      mbar_wait_drain(&bars->drain, 0);
    }
    __syncwarp();
  } else if (warp == 18) {
    // ------------------------------------------------------------ (lse, delta) of the row tiles
    uint32_t tiles = 0;
    while (ok && sched.next(sg)) {
      for (int j = 0; j < sg.n && ok; ++j, ++tiles) {
        const uint32_t st = tiles & 1;
        if (tiles >= 2) ok = uwait(&bars->row_empty[st], (tiles >> 1) - 1, 661);
        if (!ok) break;
        const int t0 = (sg.r0 + j) * TOK;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = i * 32 + lane, t = t0 + r / a.G;
          const float2 v = t < sg.L ? a.row[(sg.tok0 + t) * a.H_q + sg.g * a.G + r % a.G] : make_float2(0.f, 0.f);
          rowv[st * 2 * kRows + r] = -v.x;
          rowv[(st * 2 + 1) * kRows + r] = -v.y;
        }
        mbar_arrive(&bars->row_full[st]);
      }
    }
  } else if (warp < 16) {
    // ------------------------------------------------------------ P, dS; results
    const int wq = warp >> 2;                        // rows 32 wq .. + 31 of the tile
    const int r = (warp & 3) * 32 + lane;            // key = tensor-memory lane
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
    uint32_t tiles = 0;
    int segs = 0;
    while (ok && sched.next(sg)) {
      const int key = sg.kt * kRows + r;
#pragma unroll 1
      for (int j = 0; j < sg.n && ok; ++j, ++tiles) {
        const int t0 = (sg.r0 + j) * TOK;
        const bool edge = t0 < sg.kt * kRows + kRows - 1 || t0 + TOK > sg.L;
        // rows lo <= c < hi of these see the key
        const int lo = max(key - t0, 0) * a.G - 32 * wq, hi = min(sg.L - t0, TOK) * a.G - 32 * wq;
        const float* rv = rowv + (tiles & 1) * 2 * kRows + 32 * wq;
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->row_full[tiles & 1], (tiles >> 1) & 1, abort_flag, a.status, 671) &&
                                         mbar_wait(&bars->s_full, tiles & 1, abort_flag, a.status, 672));
        if (!ok) break;
        tc_fence_after();
        float p[32];
        tmem_ld32(tmem + lane_base + 32 * wq, p);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 32; ++c) asm volatile("" : "+f"(p[c]));   // no use before the wait
        tc_fence_before();
        mbar_arrive(&bars->s_read);
        uint32_t w[16];
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const float4 v = *reinterpret_cast<const float4*>(rv + c);
          const float2 e0 = fma2(make_float2(p[c], p[c + 1]), sc2, make_float2(v.x, v.y));
          const float2 e1 = fma2(make_float2(p[c + 2], p[c + 3]), sc2, make_float2(v.z, v.w));
          p[c] = ex2(e0.x);
          p[c + 1] = ex2(e0.y);
          p[c + 2] = ex2(e1.x);
          p[c + 3] = ex2(e1.y);
        }
        if (edge) {
#pragma unroll
          for (int c = 0; c < 32; ++c) p[c] = (c >= lo && c < hi) ? p[c] : 0.f;
        }
#pragma unroll
        for (int c = 0; c < 16; ++c) w[c] = pack_bf16x2(p[2 * c], p[2 * c + 1]);
        // P^T lies over columns that other warps read
        ok = uwait(&bars->s_read, tiles, 673);
        if (!ok) break;
        tc_fence_after();
        tmem_st16(tmem + lane_base + 16 * wq, w);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bars->p_full);
        ok = uwait(&bars->dp_full, tiles, 674);
        if (!ok) break;
        tc_fence_after();
        float d[32];
        tmem_ld32(tmem + lane_base + kColDP + 32 * wq, d);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 32; ++c) asm volatile("" : "+f"(d[c]));
        tc_fence_before();
        mbar_arrive(&bars->dp_read);
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const float4 v = *reinterpret_cast<const float4*>(rv + kRows + c);
          const float2 d0 = mul2(make_float2(p[c], p[c + 1]), add2(make_float2(d[c], d[c + 1]), make_float2(v.x, v.y)));
          const float2 d1 =
              mul2(make_float2(p[c + 2], p[c + 3]), add2(make_float2(d[c + 2], d[c + 3]), make_float2(v.z, v.w)));
          d[c] = d0.x;
          d[c + 1] = d0.y;
          d[c + 2] = d1.x;
          d[c + 3] = d1.y;
        }
        mbar_arrive(&bars->row_empty[tiles & 1]);
        if (edge) {
#pragma unroll
          for (int c = 0; c < 32; ++c) d[c] = (c >= lo && c < hi) ? d[c] : 0.f;
        }
#pragma unroll
        for (int c = 0; c < 16; ++c) w[c] = pack_bf16x2(d[2 * c], d[2 * c + 1]);
        ok = uwait(&bars->dp_read, tiles, 675);   // dS^T lies over columns that other warps read
        if (!ok) break;
        tc_fence_after();
        tmem_st16(tmem + lane_base + kColDS + 16 * wq, w);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bars->ds_full);
      }
      if (!ok) break;
      ok = uwait(&bars->acc_full, segs++, 676);
      if (!ok) break;
      tc_fence_after();
      // 32 columns at a time of dV and dK, dealt to the warps that share the rows
      const bool valid = key < sg.L;
      const int64_t row = (sg.tok0 + key) * a.H_kv + sg.g;
      float* part = a.part + ((int64_t)sg.slot * kRows + r) * (DK + DV);
#pragma unroll 1
      for (int c = 32 * wq; c < DV + DK; c += 128) {
        const bool is_v = c < DV;
        float d[32];
        tmem_ld32(tmem + lane_base + (is_v ? kColDV + c : kColDK + c - DV), d);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) asm volatile("" : "+f"(d[i]));
        if (valid) {
          if (sg.slot >= 0) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<float4*>(part + c + i) = make_float4(d[i], d[i + 1], d[i + 2], d[i + 3]);
          } else {
            __nv_bfloat16* dst = is_v ? static_cast<__nv_bfloat16*>(a.dv) + row * DV + c
                                      : static_cast<__nv_bfloat16*>(a.dk) + row * DK + c - DV;
            const float f = is_v ? 1.f : a.scale;
#pragma unroll
            for (int i = 0; i < 32; i += 8) *reinterpret_cast<uint4*>(dst + i) = pack_out(d + i, f);
          }
        }
        __syncwarp();   // the tensor-memory loads are warp-wide
      }
      tc_fence_before();   // the next unit's products wait for this thread's next arrivals
    }
  }
  if (tid == 0) {   // for the merge: {sequence, key head, key block, last run} of the unit cut by this run's end
    int4 cut = make_int4(-1, 0, 0, 0);
    if (sg.slot == 2 * (int)blockIdx.x + 1) {
      const int blocks = gridDim.x;
      const int64_t end = run_begin(a, blockIdx.x + 1, blocks) - sg.n + ((sg.L + TOK - 1) / TOK - sg.kt * a.G);
      int c1 = blockIdx.x + 1;
      while (c1 + 1 < blocks && run_begin(a, c1 + 1, blocks) < end) ++c1;
      cut = make_int4(sg.b, sg.g, sg.kt, c1);
    }
    a.cut[blockIdx.x] = cut;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// The units that a border between runs cut: their parts in block order. Block x: the
// unit that begins in run x and ends beyond it, if there is one; a warp takes four keys.
template <int DK, int DV>
__global__ void __launch_bounds__(256) nsa_full_bwd_merge_kernel(const FullBwdArgs a) {
  constexpr int E = (DK + DV) / 64;   // pairs of channels per lane
  pdl_wait();   // every block of a kernel in a chain of early launches waits, before any exit
  const int c0 = blockIdx.x;
  const int4 cut = a.cut[c0];
  if (cut.x < 0) return;
  const int lane = threadIdx.x & 31, r0 = (blockIdx.y * 8 + (threadIdx.x >> 5)) * 4;
  const int have = min(a.len[cut.x] - cut.z * kRows, kRows);   // keys of the block
  if (r0 >= have) return;
  const int64_t ld = (int64_t)kRows * (DK + DV);
  float2 s[4][E];
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) s[k][e] = make_float2(0.f, 0.f);
#pragma unroll 2
  for (int c = c0; c <= cut.w; ++c) {
    const float* slot = a.part + (2 * c + (c == c0 ? 1 : 0)) * ld;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2* src = reinterpret_cast<const float2*>(slot + (int64_t)min(r0 + k, have - 1) * (DK + DV));
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float2 v = src[e * 32 + lane];
        s[k][e].x += v.x;
        s[k][e].y += v.y;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (r0 + k >= have) break;
    const int64_t row = (a.tok_off[cut.x] + cut.z * kRows + r0 + k) * a.H_kv + cut.y;
#pragma unroll
    for (int e = 0; e < E; ++e) {   // channels 0 .. DV - 1: dV, then dK
      const int ch = e * 64 + lane * 2;
      if (e * 64 < DV)
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.dv) + row * DV + ch) =
            pack_bf16x2(s[k][e].x, s[k][e].y);
      else
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.dk) + row * DK + ch - DV) =
            pack_bf16x2(s[k][e].x * a.scale, s[k][e].y * a.scale);
    }
  }
}

// ---- query rows ----
template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1) nsa_full_bwd_q_kernel(const FullBwdArgs a,
                                                                     const __grid_constant__ FullBwdMaps mp) {
  constexpr int KC = DK / 64, VC = DV / 64, VS = wide_stages(DK, DV);
  constexpr int kKStage = KC * kPiece, kVStage = VC * kPiece;
  constexpr uint32_t kColDP = 128, kColDQ = 256, kColDS = 448;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* Qs = smem;                       // Q pieces, then dO pieces
  uint8_t* Gs = Qs + KC * kPiece;
  uint8_t* Kr = Gs + kVStage;               // streamed K, V
  uint8_t* Vr = Kr + 2 * kKStage;
  BwdBars* bars = reinterpret_cast<BwdBars*>(Vr + VS * kVStage);
  volatile int* abort_flag = &bars->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) bwd_init(bars);
  if (warp == 0) tmem_alloc(&bars->tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  const uint32_t tmem = bars->tmem_base;
  const int TOK = kRows / a.G;
  bool ok = true;
  auto uwait = [&](uint64_t* bar, uint32_t parity, uint32_t site) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity & 1u, abort_flag, a.status, site));
  };
  // items: row tiles, longest first, in snake order (levels as in the forward)
  int it = 0, b, g, i0, L, nkt;
  int64_t tok0;
  auto next = [&]() -> bool {
    const int64_t grid = gridDim.x, c = blockIdx.x;
    const int64_t x = it * grid + ((it & 1) ? grid - 1 - c : c);
    ++it;
    if (x >= a.n_items) return false;
    const int u = (int)(x / a.H_kv);
    g = (int)(x - (int64_t)u * a.H_kv);
    int lo = 0, hi = a.seqs.n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.seqs.tile_prefix[mid] <= u) lo = mid; else hi = mid - 1;
    }
    const int rem = u - a.seqs.tile_prefix[lo];
    const int tile = (a.seqs.len[lo] + TOK - 1) / TOK - 1 - rem / (lo + 1);
    b = rem % (lo + 1);
    L = a.seqs.len[b];
    tok0 = a.seqs.tok_off[b];
    i0 = tile * TOK;
    nkt = (min(i0 + TOK, L) + kRows - 1) / kRows;
    return true;
  };

  if (warp == 16) {
    // ------------------------------------------------------------ loads
    uint32_t k_n = 0, v_n = 0;   // stages filled
    uint32_t tiles = 0;
    int segs = 0;
    while (ok && next()) {
      if (segs > 0) ok = uwait(&bars->fix_empty, segs - 1, 681);
      if (!ok) break;
      if (lane == 0) {
        const int row = (int)(tok0 + i0);
        mbar_arrive_expect_tx(&bars->fix_full, (KC + VC) * kPiece);
        for (int c = 0; c < KC; ++c) tma_load_3d(Qs + c * kPiece, &mp.q, &bars->fix_full, c * 64, g * a.G, row);
        for (int c = 0; c < VC; ++c) tma_load_3d(Gs + c * kPiece, &mp.dout, &bars->fix_full, c * 64, g * a.G, row);
      }
      ++segs;
      for (int j = 0; j < nkt && ok; ++j, ++tiles) {
        const int row = (int)(tok0 + (int64_t)j * kRows);
        const uint32_t ks = tiles & 1, vs = tiles % VS;
        if (tiles >= VS) ok = uwait(&bars->v_empty[vs], tiles / VS - 1, 683);   // V is free before K
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars->v_full[vs], kVStage);
          for (int c = 0; c < VC; ++c)
            tma_load_3d(Vr + vs * kVStage + c * kPiece, &mp.v, &bars->v_full[vs], c * 64, g, row);
        }
        ++v_n;
        if (tiles >= 2) ok = uwait(&bars->k_empty[ks], (tiles >> 1) - 1, 682);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars->k_full[ks], kKStage);
          for (int c = 0; c < KC; ++c)
            tma_load_3d(Kr + ks * kKStage + c * kPiece, &mp.k, &bars->k_full[ks], c * 64, g, row);
        }
        ++k_n;
      }
    }
    if (!ok && lane == 0) drain_loads(bars, segs, k_n, v_n, VS);
  } else if (warp == 17) {
    // ------------------------------------------------------------ products
    // S of tile j + 1 is issued before dQ of tile j: both stages of K are in use then
    const uint32_t tm = uni(tmem);
    const uint32_t id_s = umma_idesc_bf16(128, 128, false, false), id_k = umma_idesc_bf16(128, DK, false, true);
    const uint64_t qd = umma_desc_sw128(uni(smem_u32(Qs)), 16, 1024), gd = umma_desc_sw128(uni(smem_u32(Gs)), 16, 1024);
    const uint32_t k_a = uni(smem_u32(Kr)), v_a = uni(smem_u32(Vr));
    const uint64_t kd = umma_desc_sw128(k_a, 16, 1024), vd = umma_desc_sw128(v_a, 16, 1024);
    const uint64_t kt = umma_desc_sw128(k_a, kPiece, 1024);   // channels x keys
    uint32_t tiles = 0;    // of the segments before
    int segs = 0;
    while (ok && next()) {
      const int n = uni(nkt), keys = uni(min(i0 + TOK, L));
      ok = uwait(&bars->fix_full, segs, 691);
      if (!ok) break;
      ++segs;
      auto scores = [&](int j) {   // S of tile j
        const uint32_t t = tiles + j, ks = t & 1;
        const int left = keys - j * kRows;   // keys in sight
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->k_full[ks], (t >> 1) & 1, abort_flag, a.status, 693) &&
                                         (t == 0 || mbar_wait(&bars->s_read, (t - 1) & 1, abort_flag, a.status, 692)));
        if (!ok) return;
        if (left < kRows) {   // dS is zero there, but 0 x NaN is not
          for (int c = 0; c < KC; ++c) clear_rows(Kr + ks * kKStage + c * kPiece, left, lane);
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (elect_one()) {
          tc_fence_after();
          const uint64_t k = kd + (uint64_t)(ks * (kKStage >> 4));
#pragma unroll
          for (int kk = 0; kk < KC * 4; ++kk) {
            const uint64_t o = (uint64_t)((kk >> 2) * (kPiece >> 4) + (kk & 3) * 2);
            umma_ss(tm, qd + o, k + o, id_s, kk ? 1u : 0u);
          }
          umma_commit(&bars->s_full);
        }
        __syncwarp();
      };
      auto weights = [&](int j) {   // dP of tile j
        const uint32_t t = tiles + j, vs = t % VS;
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->v_full[vs], (t / VS) & 1, abort_flag, a.status, 695) &&
                                         (t == 0 || mbar_wait(&bars->dp_read, (t - 1) & 1, abort_flag, a.status, 694)));
        if (!ok) return;
        if (elect_one()) {
          tc_fence_after();
          const uint64_t v = vd + (uint64_t)(vs * (kVStage >> 4));
#pragma unroll
          for (int kk = 0; kk < VC * 4; ++kk) {
            const uint64_t o = (uint64_t)((kk >> 2) * (kPiece >> 4) + (kk & 3) * 2);
            umma_ss(tm + kColDP, gd + o, v + o, id_s, kk ? 1u : 0u);
          }
          umma_commit(&bars->v_empty[vs]);
          umma_commit(&bars->dp_full);
          if (j + 1 == n) umma_commit(&bars->fix_empty);
        }
        __syncwarp();
      };
      auto gradient = [&](int j) {   // dQ += dS K of tile j
        const uint32_t t = tiles + j;
        ok = uwait(&bars->ds_full, t, 696);
        if (!ok) return;
        if (elect_one()) {
          tc_fence_after();
          const uint64_t k = kt + (uint64_t)((t & 1) * (kKStage >> 4));
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_ts(tm + kColDQ, tm + kColDS + kk * 8, k + (uint64_t)(kk * (2048 >> 4)), id_k, (j | kk) ? 1u : 0u);
          umma_commit(&bars->k_empty[t & 1]);
          umma_commit(&bars->ds_free);
          if (j + 1 == n) umma_commit(&bars->acc_full);
        }
        __syncwarp();
      };
      // S of a tile before dQ of the tile before. dP after that dQ where V has two stages
      // (128 / 64: 19.5 us against 22 for the small training case), before it where it has
      // one, so that its next tile is asked for early (192 / 128: 570 us against 599).
#pragma unroll 1
      for (int j = 0; j <= n && ok; ++j) {
        if (j < n) scores(j);
        if (VS == 1 && ok && j < n) weights(j);
        if (ok && j > 0) gradient(j - 1);
        if (VS > 1 && ok && j < n) weights(j);
      }
      tiles += n;
    }
    if (elect_one()) {
      umma_commit(&bars->drain);
      mbar_wait_drain(&bars->drain, 0);
    }
    __syncwarp();
  } else if (warp < 16) {
    // ------------------------------------------------------------ dS; dQ
    const int wq = warp >> 2;                        // keys 32 wq .. + 31 of the tile
    const int r = (warp & 3) * 32 + lane;            // row = tensor-memory lane
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
    uint32_t tiles = 0;
    int segs = 0;
    while (ok && next()) {
      const int t = i0 + r / a.G, hq = g * a.G + r % a.G;
      const bool valid = t < L;
      const int64_t row = (tok0 + t) * a.H_q + hq;
      const float2 rv = valid ? a.row[row] : make_float2(0.f, 0.f);
      const float2 nl = make_float2(-rv.x, -rv.x), nd = make_float2(-rv.y, -rv.y);
#pragma unroll 1
      for (int j = 0; j < nkt && ok; ++j, ++tiles) {
        const bool edge = j * kRows + kRows - 1 > i0;   // some key of the tile is past the first token
        const int hi = t - (j * kRows + 32 * wq);       // keys c <= hi are seen
        ok = uwait(&bars->s_full, tiles, 701);
        if (!ok) break;
        tc_fence_after();
        float p[32];
        tmem_ld32(tmem + lane_base + 32 * wq, p);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 32; ++c) asm volatile("" : "+f"(p[c]));
        tc_fence_before();
        mbar_arrive(&bars->s_read);
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const float2 e = fma2(make_float2(p[c], p[c + 1]), sc2, nl);
          p[c] = ex2(e.x);
          p[c + 1] = ex2(e.y);
        }
        ok = uwait(&bars->dp_full, tiles, 702);
        if (!ok) break;
        tc_fence_after();
        float d[32];
        tmem_ld32(tmem + lane_base + kColDP + 32 * wq, d);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 32; ++c) asm volatile("" : "+f"(d[c]));
        tc_fence_before();
        mbar_arrive(&bars->dp_read);
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const float2 v = mul2(make_float2(p[c], p[c + 1]), add2(make_float2(d[c], d[c + 1]), nd));
          d[c] = v.x;
          d[c + 1] = v.y;
        }
        if (edge) {
#pragma unroll
          for (int c = 0; c < 32; ++c) d[c] = c <= hi ? d[c] : 0.f;
        }
        uint32_t w[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) w[c] = pack_bf16x2(d[2 * c], d[2 * c + 1]);
        if (tiles > 0) {   // the product that reads the tile before has finished
          ok = uwait(&bars->ds_free, tiles - 1, 703);
          if (!ok) break;
          tc_fence_after();
        }
        tmem_st16(tmem + lane_base + kColDS + 16 * wq, w);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bars->ds_full);
      }
      if (!ok) break;
      ok = uwait(&bars->acc_full, segs++, 704);
      if (!ok) break;
      tc_fence_after();
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.dq) + row * DK;
#pragma unroll 1
      for (int c = 32 * wq; c < DK; c += 128) {
        float d[32];
        tmem_ld32(tmem + lane_base + kColDQ + c, d);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) asm volatile("" : "+f"(d[i]));
        if (valid) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) *reinterpret_cast<uint4*>(dst + c + i) = pack_out(d + i, a.scale);
        }
        __syncwarp();
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

template <int DK, int DV>
static cudaError_t launch_bwd_t(const FullBwdArgs& a, const FullBwdMaps& m, cudaStream_t st) {
  constexpr int smem = bwd_smem(DK, DV);
  auto kv = nsa_full_bwd_kv_kernel<DK, DV>;
  auto kq = nsa_full_bwd_q_kernel<DK, DV>;
  cudaError_t e = cudaFuncSetAttribute(kv, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kq, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t threads = a.n_rows * (DV / 8), W = a.kv_prefix[a.batch];
  nsa_full_bwd_row_kernel<DV><<<(unsigned)((threads + 255) / 256), 256, 0, st>>>(a);
  // no more runs than give each about four row tiles (rounded up: 5 tiles are runs of two
  // and three): the merge of many parts costs more than the SMs save (1024 tokens, 4 heads
  // of 64, a training step: 54 us with four, 69 with one, 57 with two, 60 with six)
  const int64_t want = (W + 3) / 4;
  const int runs = want < kFullBlocks ? (int)want : kFullBlocks;
  const int grid = a.n_items < kFullBlocks ? (int)a.n_items : kFullBlocks;
  e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_after(kv, dim3(runs), kThreads, smem, st, a, m);
  if (e == cudaSuccess)
    e = launch_after(nsa_full_bwd_merge_kernel<DK, DV>, dim3(runs, kRows / 32), 256, 0, st, a);
  if (e == cudaSuccess) e = launch_after(kq, dim3(grid), kThreads, smem, st, a, m);
  return e;
}

cudaError_t launch_full_bwd(const FullBwdArgs& a, const FullBwdMaps& m, int d_k, int d_v, cudaStream_t st) {
  if (d_k == 192 && d_v == 128) return launch_bwd_t<192, 128>(a, m, st);
  if (d_k == 128 && d_v == 128) return launch_bwd_t<128, 128>(a, m, st);
  if (d_k == 64 && d_v == 64) return launch_bwd_t<64, 64>(a, m, st);
  if (d_k == 64 && d_v == 128) return launch_bwd_t<64, 128>(a, m, st);
  if (d_k == 128 && d_v == 64) return launch_bwd_t<128, 64>(a, m, st);
  if (d_k == 192 && d_v == 64) return launch_bwd_t<192, 64>(a, m, st);
  return cudaErrorInvalidValue;
}

}  // namespace nsa
