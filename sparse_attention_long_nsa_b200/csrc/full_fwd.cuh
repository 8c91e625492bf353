// Full (dense) attention on tcgen05: the kernel behind the causal prompt
// attention (full_prefill.cu) and the drafted-token attention over a cache
// (full_tree.cu).
//
//   o = softmax(scale q K^T + mask) V,  lse = log sum exp(scale q K^T + mask)
//
// A work item ("segment") is a block of query rows of one key head and a run of
// 128-key tiles. Rows are (token, head of the group): the G heads that share a
// key head lie in one row block, so a key tile is fetched once for all of them.
// Scores, the running maximum and the sum stay in fp32; P is rounded to bf16 for
// the product with V (as the sparse kernels do), the output once at the end.
//
// Tensor memory: two score buffers S0, S1 (128 columns each, P written over the
// columns already read) and two accumulators O0, O1. With NT = 2 the block holds
// 256 rows, buffer x serves rows 128 x .. + 127, and every key tile is used by
// both; while one half's softmax runs, the tensor core works for the other. With
// NT = 1 (128 rows or fewer) both buffers serve the same rows and the key tiles
// alternate between them; their results are merged at the end.
//
// Roles (576 threads): warps 0-7 softmax of buffer 0, warps 8-15 of buffer 1, warp
// 16 loads Q, K and V by TMA, warp 17 issues the products. A softmax warp owns 16
// rows; its half-warps hold alternating runs of 32 keys of them and trade maxima and
// sums by shuffles. With a thread to a whole row (8 warps) the kernel waited on its
// own latencies: two warps a scheduler issued in 24% of the cycles.
// K arrives in chunks of 128 keys x 64 channels and V in pieces of the
// same 16 KB, through one ring in the order of use (V of a tile and the next tile's
// K make a group with one barrier): the room that is left beside
// Q holds about one and a half tiles, and a common ring of small pieces keeps
// more bytes in flight than separate rings of whole tiles would.
//
// The product with V rows that no row of the block sees (past the last key; nodes that
// no mask of the block's rows names): P is zero there, but 0 x (infinity or NaN) is not,
// so the issuing warp clears those rows in shared memory first. A node that only some of
// the rows see stays: a value of it that is not finite reaches the others too. Every wait
// is bounded; on a timeout the block stops, lets its copies and products land and leaves.
//
// Measured, this kernel alone (single launches under the profiler): 8192 tokens, 64 heads
// on 4 key heads, 192 / 128: 1.09 ms (1.26 PFLOP/s of 1.62 measured, tensor pipe 63 %
// active); calls in a row, under the power cap, take 1.23 to 1.27 ms. 32 x 16 nodes over
// 16384 keys: 293 us (tensor pipe 51 %, 4.6 TB/s); 16 single tokens over 8K to 128K keys:
// 500 us (6.0 TB/s).
#pragma once

#include <limits.h>

#include "common.cuh"
#include "kernels.h"

namespace nsa {

constexpr int kFaThreads = 576;
constexpr int kFaKeys = 128;
constexpr int kFaSlot = 16384;
constexpr float kFaRescaleLog2 = 8.f;   // O is rescaled only when a row max grows by more (log2 units)

template <int DK, int NT>
struct FaShape {
  static constexpr int kQBytes = NT * 128 * DK * 2;
  static constexpr int kMisc = 2048 + (NT == 1 ? 2048 : 0);
  static constexpr int kFit = (232448 - 1024 - kQBytes - kMisc) / kFaSlot;
  // a power of two for 256 rows (the slot of a piece is found by a mask: d = 128 205 -> 200
  // us for ragged prompts); with 128 rows the deeper ring is worth more
  static constexpr int kSlots = NT == 2 ? (kFit > 8 ? 8 : kFit) : kFit > 12 ? 12 : kFit;
  static constexpr int kSmem = 1024 + kQBytes + kSlots * kFaSlot + kMisc;
};

struct FaBars {
  uint64_t full[16], empty[12];  // full: by group of pieces (at most 13 are under way); empty: by ring slot
  uint64_t q_full, q_empty, s_full[2], p_full[2], o_full[2], drain, merge;
  uint32_t tmem_base;
  int abort;
};

// one work item
struct FaSeg {
  int b, g;
  int i0, ntok;        // first query token (within the sequence) and how many exist from there
  int kt0, nt[2];      // first key tile; tiles of buffer 0 / 1 (NT = 1: nt[0] = all of them)
  int nkeys;           // keys in sight of the block: later ones are masked, their V rows cleared
  int prefix;          // tree: keys below it are seen by every row
  int64_t q_row;       // row of token i0 in q / out (token units)
  int64_t kv_row;      // first row of the sequence in k / v (contiguous layouts)
  int slot;            // >= 0: partial result slot; -1: the item covers all keys, write the output
};

// ---- schedules: next() gives a block's items in order, the same to every role ----

// Causal prompts: query blocks of NT * 128 / G tokens, longest first over all
// sequences (each level of tiles names the sequences long enough to have it),
// dealt to the blocks in snake order.
template <int NT>
struct PrefillSched {
  const FullArgs& a;
  int it = 0;
  __device__ explicit PrefillSched(const FullArgs& a_) : a(a_) {}
  __device__ bool next(FaSeg& s) {
    const int64_t grid = gridDim.x, c = blockIdx.x;
    const int64_t x = it * grid + ((it & 1) ? grid - 1 - c : c);
    ++it;
    if (x >= a.n_items) return false;
    const int u = (int)(x / a.H_kv);
    s.g = (int)(x - (int64_t)u * a.H_kv);
    int lo = 0, hi = a.seqs.n - 1;   // sequences are sorted by length, longest first
    while (lo < hi) {                // last i with tile_prefix[i] <= u
      const int mid = (lo + hi + 1) >> 1;
      if (a.seqs.tile_prefix[mid] <= u) lo = mid; else hi = mid - 1;
    }
    // in the stretch of sequence `lo`, lo + 1 sequences are long enough
    const int TOK = NT * 128 / a.G, r = u - a.seqs.tile_prefix[lo];
    const int tile = (a.seqs.len[lo] + TOK - 1) / TOK - 1 - r / (lo + 1);
    s.b = r % (lo + 1);
    const int L = a.seqs.len[s.b];
    s.i0 = tile * TOK;
    s.ntok = min(TOK, L - s.i0);
    s.kt0 = 0;
    s.nkeys = s.i0 + s.ntok;
    const int n0 = NT == 1 ? s.nkeys : min(s.nkeys, s.i0 + TOK / 2);
    s.nt[0] = (n0 + kFaKeys - 1) / kFaKeys;
    s.nt[1] = (NT == 2 && s.ntok > TOK / 2) ? (s.nkeys + kFaKeys - 1) / kFaKeys : 0;
    s.prefix = 0;
    s.q_row = a.seqs.tok_off[s.b] + s.i0;
    s.kv_row = a.seqs.tok_off[s.b];
    s.slot = -1;
    return true;
  }
};

// Runs that W key tiles are cut into: one a block, and no more than give each about two
// tiles (8 sequences of 1000 tokens: 14.9 us with two, 18.6 with one, 18.8 with three; one
// of 8192: 24.5, 27.7, 25.0). The count is rounded up: 3 tiles are runs of one and two.
constexpr int kMinRun = 2;
__device__ __forceinline__ int64_t tree_runs(int64_t W) {
  return min((int64_t)gridDim.x, (W + kMinRun - 1) / kMinRun);
}

// Drafted tokens over a cache: all (sequence, key head, row block) units' key
// tiles in a row, cut into equal runs, one for each block; a unit cut by a
// border leaves partial results (slot 2 c: the run starts inside the unit; slot
// 2 c + 1: the unit ends beyond the run) that the merge kernel joins.
template <int NT>
struct TreeSched {
  const FullArgs& a;
  const int* prefix;   // [B + 1] key tiles of the sequences before
  int pos, end, b = 0;
  __device__ TreeSched(const FullArgs& a_, const int* p) : a(a_), prefix(p) {
    const int64_t W = p[a.B], c = blockIdx.x, n = tree_runs(W);
    pos = c < n ? (int)(W * c / n) : 0;
    end = c < n ? (int)(W * (c + 1) / n) : 0;
  }
  __device__ bool next(FaSeg& s) {
    if (pos >= end) return false;
    while (prefix[b + 1] <= pos) ++b;
    const int L = a.lens[b], n = a.nodes ? a.nodes[b] : a.M;
    const int TOK = NT * 128 / a.G;
    const int ntile = (L + kFaKeys - 1) / kFaKeys, rb = (n + TOK - 1) / TOK;
    const int unit = (pos - prefix[b]) / ntile;
    s.b = b;
    s.g = unit / rb;
    s.i0 = (unit - s.g * rb) * TOK;
    s.ntok = min(TOK, n - s.i0);
    s.kt0 = pos - prefix[b] - unit * ntile;
    const int cnt = min(ntile - s.kt0, end - pos);
    s.nkeys = L;
    s.nt[0] = cnt;
    // A block of at most 128 rows in the 256-row kernel (few nodes in a call made for many)
    // has one buffer at work: its scores, softmax and product with V take turns. Of 32
    // sequences with up to 16 nodes of 16 heads half are such blocks, and the calls reach
    // 0.55 of their memory floor.
    s.nt[1] = (NT == 2 && s.ntok > TOK / 2) ? cnt : 0;
    s.prefix = L - n;
    s.q_row = (int64_t)b * a.M + s.i0;
    s.kv_row = (int64_t)b * a.Lmax;
    s.slot = cnt == ntile ? -1 : 2 * (int)blockIdx.x + (s.kt0 == 0 ? 1 : 0);
    pos += cnt;
    return true;
  }
};

template <int NT, bool TREE>
struct FaSched : PrefillSched<NT> {
  __device__ FaSched(const FullArgs& a, const int*) : PrefillSched<NT>(a) {}
};
template <int NT>
struct FaSched<NT, true> : TreeSched<NT> {
  __device__ FaSched(const FullArgs& a, const int* p) : TreeSched<NT>(a, p) {}
};

// key tiles of the sequences before each sequence (a sequence with lengths out of
// range is recorded in the status word and has none)
template <int NT>
__device__ __forceinline__ void tree_prefix(const FullArgs& a, int* prefix) {
  // one warp, four sequences a lane (B <= 128)
  const int lane = threadIdx.x & 31;
  int v[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = lane * 4 + i;
    v[i] = 0;
    if (b < a.B) {
      const int L = a.lens[b], n = a.nodes ? a.nodes[b] : a.M;
      if (n < 0 || n > a.M || L < n || L > a.max_len) {
        if (blockIdx.x == 0 && a.status) {
          atomicOr(a.status, DEV_ERR_BOUNDS);
          atomicExch(a.status + 1, 601u);
        }
      } else if (n > 0) {
        const int TOK = NT * 128 / a.G;
        v[i] = (L + kFaKeys - 1) / kFaKeys * ((n + TOK - 1) / TOK) * a.H_kv;
      }
    }
    sum += v[i];
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  int run = inc - sum;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = lane * 4 + i;
    if (b <= a.B) prefix[b] = run;
    run += v[i];
    if (b == 127 && a.B == 128) prefix[128] = run;
  }
}

template <int DK, int DV, int NT, bool TREE>
__global__ void __launch_bounds__(kFaThreads, 1) nsa_full_attn_kernel(const FullArgs a,
                                                                      const __grid_constant__ FullMaps mp) {
  using Sh = FaShape<DK, NT>;
  constexpr int NS = Sh::kSlots;
  constexpr int KC = DK / 64;               // ring pieces of a K tile
  constexpr int VC = DV / 64;               // ring pieces of a V tile: 64 keys x 128 or 128 keys x 64
  constexpr int A = NT == 2 ? 1 : 2;        // S of tile t + A follows P.V of tile t
  constexpr uint32_t kColO = 256;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* Qs = smem;
  uint8_t* ring = smem + Sh::kQBytes;
  FaBars* bars = reinterpret_cast<FaBars*>(ring + NS * kFaSlot);
  int* prefix = reinterpret_cast<int*>(bars + 1);                                            // [129]
  float2* ml_s = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(bars) + 2048);         // NT = 1: [2][128]
  volatile int* abort_flag = &bars->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < 16; ++i) mbar_init(&bars->full[i], 1);
    for (int i = 0; i < NS; ++i) mbar_init(&bars->empty[i], 1);
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars->s_full[x], 1);
      mbar_init(&bars->p_full[x], 256);
      mbar_init(&bars->o_full[x], 1);
    }
    mbar_init(&bars->drain, 1);
    mbar_init(&bars->merge, 512);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&bars->tmem_base, 512);
  if (TREE && warp == 1) tree_prefix<NT>(a, prefix);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  if (TREE) pdl_launch_dependents();   // the merge may be scheduled; it waits for this grid's end
  FaSched<NT, TREE> sched(a, prefix);
  FaSeg sg;
  sg.slot = -1;
  bool ok = true;

  if (warp == 16) {
    // ------------------------------------------------------------ loads
    if (lane == 0) {
      prefetch_tmap(&mp.q);
      prefetch_tmap(&mp.k);
      prefetch_tmap(&mp.v);
    }
    uint32_t pos = 0;      // ring pieces issued
    uint32_t groups = 0;   // groups begun
    int q_n = 0;           // Q tiles issued
    int blk, brow = 0, blk2, brow2 = 0;   // page table windows: lane i holds the row of 64-key block blk + i
    while (ok && sched.next(sg)) {
      blk = blk2 = INT_MAX;   // another sequence: read anew
      if (q_n > 0) ok = __all_sync(0xffffffffu, mbar_wait(&bars->q_empty, (q_n - 1) & 1, abort_flag, a.status, 611));
      if (!ok) break;
      const int n = max(sg.nt[0], sg.nt[1]);
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars->q_full, (uint32_t)Sh::kQBytes);
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int kb = 0; kb < KC; ++kb)
            tma_load_3d(Qs + (x * KC + kb) * 16384, &mp.q, &bars->q_full, kb * 64, sg.g * a.G,
                        (int)sg.q_row + x * (128 / a.G));
      }
      ++q_n;
      // rows of the two 64-key halves of key tile `t` (the second only if it has keys)
      auto rows_of = [&](int t, int& r0, int& r1, int& first, int& rows) {
        const int key = (sg.kt0 + t) * kFaKeys;
        if (TREE && a.pt.table) {
          const int kb = key >> 6;
          if (kb < first || kb - first >= 32) {
            first = kb;
            const int e = (kb + lane) * 64;
            rows = e < sg.nkeys ? (int)paged_row(a.pt, sg.b, e, a.status) : 0;
          }
          r0 = __shfl_sync(0xffffffffu, rows, kb - first);
          r1 = __shfl_sync(0xffffffffu, rows, (kb - first + 1) & 31);   // kb - first is even: never wraps
        } else {
          r0 = (int)(sg.kv_row + key);
          r1 = r0 + 64;
        }
      };
      auto acquire = [&]() -> uint32_t {   // the next ring slot, free
        const uint32_t st = pos % NS;
        if (pos >= NS)
          ok = ok && __all_sync(0xffffffffu, mbar_wait(&bars->empty[st], ((pos / NS) - 1) & 1, abort_flag, a.status, 612));
        if (ok) ++pos;
        return st;
      };
      // group: V of tile tv (none when < 0) and K of tile tk (none when >= n)
      auto push = [&](int tv, int tk) {
        uint64_t* bar = &bars->full[groups & 15];
        if (groups == 0 && NSA_INJECT(a, FAULT_FULL_TILE)) {   // checking build: withhold the first tile
          ++groups;
          return;
        }
        const bool v2 = tv >= 0 && (sg.kt0 + tv) * kFaKeys + 64 < sg.nkeys;   // the second 64 keys exist
        const bool k2 = tk < n && (sg.kt0 + tk) * kFaKeys + 64 < sg.nkeys;
        if (lane == 0)
          mbar_arrive_expect_tx(bar, (tv < 0 ? 0u : (v2 ? 16384u : 8192u) * VC) + (tk >= n ? 0u : (k2 ? 16384u : 8192u) * KC));
        ++groups;
        int r0, r1;
        if (tv >= 0) {
          rows_of(tv, r0, r1, blk, brow);
#pragma unroll
          for (int c = 0; c < VC; ++c) {
            uint8_t* dst = ring + acquire() * kFaSlot;
            if (!ok) return;
            if (lane == 0) {
              if (VC == 1) {          // 128 keys x 64 channels
                tma_load_3d(dst, &mp.v, bar, 0, sg.g, r0);
                if (v2) tma_load_3d(dst + 8192, &mp.v, bar, 0, sg.g, r1);
              } else if (c == 0 || v2) {   // 64 keys x 128 channels
                tma_load_3d(dst, &mp.v, bar, 0, sg.g, c == 0 ? r0 : r1);
                tma_load_3d(dst + 8192, &mp.v, bar, 64, sg.g, c == 0 ? r0 : r1);
              }
            }
          }
        }
        if (tk < n) {
          rows_of(tk, r0, r1, blk, brow);
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            uint8_t* dst = ring + acquire() * kFaSlot;
            if (!ok) return;
            if (lane == 0) {
              tma_load_3d(dst, &mp.k, bar, c * 64, sg.g, r0);
              if (k2) tma_load_3d(dst + 8192, &mp.k, bar, c * 64, sg.g, r1);
            }
          }
        }
      };
      // A cache comes from memory: beside 256 rows of Q the ring does not cover its latency,
      // and the tile after the next is asked into L2 (32 x 16 nodes over 16K, calls in a
      // row: 397 -> 356 us; with 128 rows the ring is deeper and it costs 1%, two tiles
      // ahead cost 5%).
      auto prefetch = [&](int t) {
        int r0, r1;
        rows_of(t, r0, r1, blk2, brow2);
        if (lane < KC + VC) {
          const CUtensorMap* m = lane < KC ? &mp.k : &mp.v;
          const int c = (lane < KC ? lane : lane - KC) * 64;
          tma_prefetch_3d(m, c, sg.g, r0);
          if ((sg.kt0 + t) * kFaKeys + 64 < sg.nkeys) tma_prefetch_3d(m, c, sg.g, r1);
        }
        __syncwarp();
      };
#pragma unroll 1
      for (int t = -A; t < n && ok; ++t) {
        if (t >= 0 || t + A < n) push(t < 0 ? -1 : t, t + A);
        if (TREE && NT == 2 && t + A + 1 < n) prefetch(t + A + 1);
      }
    }
    if (!ok && lane == 0) {   // let the copies still in flight land before the block exits
      if (q_n > 0) mbar_wait_drain(&bars->q_full, (q_n - 1) & 1);
      // (a group cut short by the abort never completes: its wait runs into its limit,
      // by when its copies have landed)
      for (uint32_t v = groups < 13 ? 0 : groups - 13; v < groups; ++v) mbar_wait_drain(&bars->full[v & 15], (v >> 4) & 1);
    }
  } else if (warp == 17) {
    // ------------------------------------------------------------ products
    // operands are kept uniform over the warp: as per-lane values each product would
    // first move six of them, longer than the product itself takes
    const uint32_t tm = uni(tmem), ring_a = uni(smem_u32(ring)), q_a = uni(smem_u32(Qs));
    const uint32_t idesc_s = umma_idesc_bf16(128, 128, false, false);
    const uint32_t idesc_o = umma_idesc_bf16(128, DV, false, true);
    const uint64_t qdesc = umma_desc_sw128(q_a, 16, 1024);
    const uint64_t kdesc = umma_desc_sw128(ring_a, 16, 1024);
    const uint64_t vdesc = umma_desc_sw128(ring_a, 8192, 1024);
    uint32_t base = 0;     // ring piece after the last segment's
    uint32_t groups = 0;   // groups waited for
    uint32_t segs = 0;
    uint32_t p_par = 0;    // bit x: parity of the next P of buffer x
    auto wait_group = [&]() -> bool {
      const uint32_t gi = groups++;
      return mbar_wait(&bars->full[gi & 15], (gi >> 4) & 1, abort_flag, a.status, 622);
    };
    // S of buffer x = Q (rows of half xq) . K at ring piece p; `rel`: its last use (one lane)
    auto qk = [&](int x, int xq, uint32_t p, bool rel) {
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const uint32_t st = (p + c) % NS;
        const uint64_t qd = qdesc + (uint64_t)((xq * KC + c) * (16384 >> 4));
        const uint64_t kd = kdesc + (uint64_t)(st * (kFaSlot >> 4));
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) umma_ss(tm + 128 * x, qd + kk * 2, kd + kk * 2, idesc_s, (c | kk) ? 1u : 0u);
        if (rel) umma_commit(&bars->empty[st]);
      }
      umma_commit(&bars->s_full[x]);
    };
    while (ok && sched.next(sg)) {
      const int n0 = uni(sg.nt[0]), n1 = uni(sg.nt[1]), n = max(n0, n1), nkeys = uni(sg.nkeys), kt0 = uni(sg.kt0);
      const int pre = uni(sg.prefix), seen_to = uni(sg.i0 + sg.ntok);   // nodes of the block's rows end there
      uint64_t named = 0;   // tree: nodes that a row of the block sees (their words are read beside the tile's copies)
      if (TREE && a.mask && (kt0 + n) * kFaKeys > pre)
        for (int i = sg.i0 + lane; i < seen_to; i += 32) named |= a.mask[(int64_t)sg.b * a.M + i];
      ok = __all_sync(0xffffffffu, mbar_wait(&bars->q_full, segs & 1, abort_flag, a.status, 621));
      if (!ok) break;
      ++segs;
      if (TREE) {
        if (a.mask)
          named = (uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(named >> 32)) << 32 |
                  __reduce_or_sync(0xffffffffu, (uint32_t)named);
        else
          named = seen_to >= 64 ? ~0ull : (1ull << seen_to) - 1ull;
        if (nkeys - pre < 64) named &= (1ull << (nkeys - pre)) - 1ull;
      }
      // the first S of each buffer
#pragma unroll 1
      for (int x = 0; x < 2 && ok; ++x) {
        if (NT == 2 ? (x == 1 && n1 == 0) : x >= n) continue;
        if (NT == 1 || x == 0) ok = __all_sync(0xffffffffu, wait_group());
        if (!ok) break;
        if (elect_one()) {
          tc_fence_after();
          qk(x, NT == 2 ? x : 0, base + (NT == 2 ? 0 : x * KC), NT == 1 || x == 1 || n1 == 0);
          if (NT == 1 ? n <= 2 && x == n - 1 : n == 1 && (x == 1 || n1 == 0)) umma_commit(&bars->q_empty);
        }
        __syncwarp();
      }
      uint32_t p = base + (NT == 2 ? 1 : min(n, 2)) * KC;   // V of tile t, then K of tile t + A
      // One instance of the step in the loop: its code has to stay in the instruction
      // cache beside the softmax's. All that a step needs is waited for at once, while
      // the products before it are still in the tensor core's queue.
#pragma unroll 1
      for (int i = 0; i < (NT == 2 ? 2 * n : n) && ok; ++i) {
        const int x = i & 1, t = NT == 2 ? i >> 1 : i;
        const int nx = NT == 1 ? n : x == 0 ? n0 : n1;      // tiles of this buffer (NT = 1: of both)
        const bool fresh = NT == 1 || x == 0 || t >= n0;    // first use of the group
        const bool last = NT == 1 || x == 1 || t >= n1;     // last use of V
        if (t < nx) {
          ok = __all_sync(0xffffffffu, (!fresh || wait_group()) &&
                                           mbar_wait(&bars->p_full[x], (p_par >> x) & 1, abort_flag, a.status, 624));
          p_par ^= 1u << x;
          if (!ok) break;
          const int key0 = (kt0 + t) * kFaKeys, left = nkeys - key0;   // keys of this tile (may exceed 128)
          if (fresh && (TREE ? key0 + kFaKeys > pre : left < kFaKeys)) {   // clear the V rows no row sees
#pragma unroll
            for (int h = 0; h < 2; ++h) {                   // 64 keys each
              const int have = left - 64 * h;
              if (have <= 0) continue;                      // not loaded
              int first = have;                             // prompts: the rows from there on
              uint64_t dead = 0;                            // trees: bit i for key 64 h + i
              if (TREE) {
                const int j = key0 + 64 * h - pre;          // node of the first key
                dead = j >= 64 ? ~0ull : j >= 0 ? ~(named >> j) : j > -64 ? ~named << -j : 0ull;
                first = dead ? __ffsll((long long)dead) - 1 : 64;
              }
              uint8_t* vs = ring + (VC == 2 ? (p + h) % NS * kFaSlot : p % NS * kFaSlot + h * 8192);
              for (int k = first * 8 + lane; k < 64 * 8; k += 32) {
                if (TREE && !(dead >> (k >> 3) & 1)) continue;
                *reinterpret_cast<uint4*>(vs + k * 16) = make_uint4(0, 0, 0, 0);
                if (VC == 2) *reinterpret_cast<uint4*>(vs + 8192 + k * 16) = make_uint4(0, 0, 0, 0);
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (elect_one()) {
            tc_fence_after();
            // O (+)= P . V, keys 64 h .. + 63: piece h (VC = 2) or rows 64 h of the one piece
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint64_t vd = vdesc + (uint64_t)((p + (VC == 2 ? h : 0)) % NS * (kFaSlot >> 4)) +
                                  (VC == 1 ? (uint64_t)(h * (8192 >> 4)) : 0);
              if (h == 0 || left > 64) {                    // else no keys there: V was not loaded
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  umma_ts(tm + kColO + 128 * x, tm + 128 * x + (h * 4 + kk) * 8, vd + kk * (2048 >> 4), idesc_o,
                          (t < A && h == 0 && kk == 0) ? 0u : 1u);
              }
              if (last && (VC == 2 || h == 1)) umma_commit(&bars->empty[(p + (VC == 2 ? h : 0)) % NS]);
            }
            if (t + A < nx) {
              const bool last_k = NT == 1 || x == 1 || t + A >= n1;
              qk(x, NT == 2 ? x : 0, p + VC, last_k);
              if (t + A + 1 == n && last_k) umma_commit(&bars->q_empty);   // the last S is on its way
            } else {
              umma_commit(&bars->o_full[x]);
            }
          }
          __syncwarp();
        }
        if (NT == 1 || x == 1) p += VC + (t + A < n ? KC : 0);
      }
      base = p;
    }
    // every product has finished before tensor memory is released
    if (elect_one()) {
      umma_commit(&bars->drain);
      mbar_wait_drain(&bars->drain, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax, output
    const int x = warp >> 3;
    const int kh = lane >> 4;                        // half-warp
    const int r = (warp & 3) * 32 + ((warp >> 2) & 1) * 16 + (lane & 15);   // row of this buffer = tensor-memory lane
    const uint32_t lane_base = (uint32_t)(r - (lane & 15)) << 16;
    const uint32_t s_col = tmem + lane_base + 128 * x;
    const int TOK1 = 128 / a.G;
    const int xr = NT == 2 ? x : 0;                  // which 128 rows of the block
    const int tt = xr * TOK1 + r / a.G, hh = r % a.G;
    const int tt_w0 = xr * TOK1 + (r - (lane & 15)) / a.G;   // first token of the warp's rows
    const float sc = a.scale_log2;
    const float thr = kFaRescaleLog2 / sc;
    uint32_t s_n = 0, o_n[2] = {0, 0}, m_n = 0;
    auto uwait = [&](uint64_t* bar, uint32_t parity, uint32_t site) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity & 1u, abort_flag, a.status, site));
    };
    auto other = [&](float v) -> float { return __shfl_xor_sync(0xffffffffu, v, 16); };   // the other half-warp's
    while (ok && sched.next(sg)) {
      const int n = sg.nt[NT == 2 ? x : 0];
      if (NT == 2 && n == 0) continue;
      const bool valid = tt < sg.ntok;
      const bool warp_on = tt_w0 < sg.ntok;          // some row of the warp exists
      const int t_abs = sg.i0 + tt;                  // prefill: position of the row's token
      uint64_t bits = 0;
      if (TREE && valid) {
        const int nn = sg.nkeys - sg.prefix;         // nodes of the sequence
        bits = a.mask ? a.mask[(int64_t)sg.b * a.M + t_abs] : (t_abs >= 63 ? ~0ull : (2ull << t_abs) - 1ull);
        if (nn < 64) bits &= (1ull << nn) - 1ull;
      }
      float m = -INFINITY, l = 0.f;                  // l: this half-warp's keys
      bool any = false;                              // this buffer got a tile
      for (int t = NT == 2 ? 0 : x; t < n; t += NT == 2 ? 1 : 2) {
        if (ok) ok = uwait(&bars->s_full[x], s_n, 631);
        if (!ok) break;
        ++s_n;
        tc_fence_after();
        if (warp_on) {
          // keys 32 kh .. + 31 of the first 64, then of the second 64
          float s[64];
          tmem_ld32_h<32>(s_col, s);
          tmem_ld32_h<32>(s_col + 64, s + 32);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 64; ++c) asm volatile("" : "+f"(s[c]));   // no use before the wait
          const int key0 = (sg.kt0 + t) * kFaKeys;
          if (TREE ? key0 + kFaKeys > sg.prefix : key0 + kFaKeys - 1 > sg.i0 + tt_w0) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {            // bit c of `see`: key k0 + c is seen
              const int k0 = key0 + 64 * i + 32 * kh;
              uint32_t see;
              if (TREE) {
                const int j = k0 - sg.prefix;        // node of the first key
                if (j >= 64) see = 0u;
                else if (j >= 0) see = (uint32_t)(bits >> j);
                else if (j > -32) see = ((uint32_t)bits << -j) | ((1u << -j) - 1u);
                else see = ~0u;
              } else {
                const int nv = t_abs + 1 - k0;
                see = nv >= 32 ? ~0u : nv <= 0 ? 0u : (1u << nv) - 1u;
              }
#pragma unroll
              for (int c = 0; c < 32; ++c) s[32 * i + c] = (see >> c) & 1u ? s[32 * i + c] : -INFINITY;
            }
          }
          float mx[4] = {max_nan(s[0], s[4]), max_nan(s[1], s[5]), max_nan(s[2], s[6]), max_nan(s[3], s[7])};
#pragma unroll
          for (int c = 8; c < 64; c += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i) mx[i] = max_nan(mx[i], s[c + i], s[c + 4 + i]);
          float tmx = max_nan(max_nan(mx[0], mx[1]), mx[2], mx[3]);
          tmx = max_nan(tmx, other(tmx));
          float alpha = 1.f;
          if (!(tmx <= m + thr)) {                   // a NaN makes the whole row one
            alpha = ex2((m - tmx) * sc);             // 0 on a row's first visible keys
            m = tmx;
          }
          if (any && __any_sync(0xffffffffu, alpha != 1.f)) {
            // S of this tile is complete, so the product before it is too
#pragma unroll 1
            for (int c = 0; c < DV / 2; c += 16) {
              float o[16];
              const uint32_t col = tmem + lane_base + kColO + 128 * x + c;
              tmem_ld16_h<DV / 2>(col, o);
              tmem_ld_wait();
              uint32_t w[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(o[i] * alpha);
              tmem_st16_h<DV / 2>(col, w);
            }
          }
          l *= alpha;
          const float mo = m == -INFINITY ? 0.f : -m * sc;   // nothing in sight yet: p = 2^-inf = 0
          const float2 sc2 = make_float2(sc, sc), mo2 = make_float2(mo, mo);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t w[16];
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              const float2 e = fma2(make_float2(s[32 * i + c], s[32 * i + c + 1]), sc2, mo2);
              const float2 p = make_float2(ex2(e.x), ex2(e.y));
              sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], p);
              w[c >> 1] = pack_bf16x2(p.x, p.y);
            }
            tmem_st16_h<16>(s_col + 32 * i, w);
          }
          const float2 sm = add2(sum[0], sum[1]);
          l += sm.x + sm.y;
          tmem_st_wait();
        }
        tc_fence_before();
        mbar_arrive(&bars->p_full[x]);
        any = true;
      }
      if (!ok) break;
      // ---- the segment's result
      l += other(l);
      if (NT == 2) {
        ok = uwait(&bars->o_full[x], o_n[x], 632);
        ++o_n[x];
      } else {
        ok = uwait(&bars->o_full[0], o_n[0], 633);
        ++o_n[0];
        if (ok && n > 1) {
          ok = uwait(&bars->o_full[1], o_n[1], 634);
          ++o_n[1];
        }
        if (ok) {   // publish (m, l), meet, merge columns x * DV / 2 .. of both accumulators
          if (kh == 0) ml_s[x * 128 + r] = make_float2(m, l);
          mbar_arrive(&bars->merge);
          ok = uwait(&bars->merge, m_n++, 635);
        }
      }
      if (!ok) break;
      tc_fence_after();
      constexpr int NC = NT == 2 ? DV / 2 : DV / 4;  // columns this thread writes
      const int c0 = (NT == 2 ? 0 : x * (DV / 2)) + kh * NC;
      const uint32_t o_base = tmem + lane_base + kColO + (NT == 2 ? 128 * x : x * (DV / 2));
      float w0 = 1.f, w1 = 0.f, mm = m, ll = l;
      if (NT == 1) {
        const float2 A = ml_s[r], Bv = ml_s[128 + r];
        mm = fmaxf(A.x, Bv.x);
        const float mz = mm == -INFINITY ? 0.f : mm;
        w0 = ex2((A.x - mz) * sc);
        w1 = n > 1 ? ex2((Bv.x - mz) * sc) : 0.f;
        ll = A.y * w0 + (n > 1 ? Bv.y * w1 : 0.f);
      }
      if (warp_on) {
        const int64_t row = ((sg.q_row + tt) * a.H_q) + sg.g * a.G + hh;
        const bool empty = ll == 0.f;                // no key in sight: zeros
        const float inv = empty ? 0.f : 1.f / ll;
        float* po = TREE && sg.slot >= 0 ? a.part + ((int64_t)sg.slot * (NT * 128) + xr * 128 + r) * (DV + 4) : nullptr;
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + row * DV;
#pragma unroll 1
        for (int c = 0; c < NC; c += 16) {
          float o[16];
          tmem_ld16_h<NC>(o_base + c, o);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) asm volatile("" : "+f"(o[i]));
          if (NT == 1) {
            if (n > 1) {
              float o1[16];
              tmem_ld16_h<NC>(o_base + 128 + c, o1);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) asm volatile("" : "+f"(o1[i]));
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = o[i] * w0 + o1[i] * w1;
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= w0;
            }
          }
          if (valid) {
            if (TREE && po) {
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<float4*>(po + c0 + c + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = empty ? 0.f : o[i] * inv;
#pragma unroll
              for (int i = 0; i < 16; i += 8)
                *reinterpret_cast<uint4*>(dst + c0 + c + i) =
                    make_uint4(pack_bf16x2(o[i], o[i + 1]), pack_bf16x2(o[i + 2], o[i + 3]),
                               pack_bf16x2(o[i + 4], o[i + 5]), pack_bf16x2(o[i + 6], o[i + 7]));
            }
          }
          __syncwarp();   // the tensor-memory loads are warp-wide
        }
        if (valid && kh == 0 && (NT == 2 || x == 0)) {
          if (TREE && po) {
            po[DV] = mm * sc;
            po[DV + 1] = ll;
          } else if (a.lse) {
            a.lse[row] = empty ? -INFINITY : 0.69314718055994531f * (mm * sc + log2f(ll));
          }
        }
      }
      if (NT == 1) {   // both accumulators are read before the next segment's products overwrite them
        tc_fence_before();
        mbar_arrive(&bars->merge);
        ok = uwait(&bars->merge, m_n++, 636);
        tc_fence_after();
      }
    }
  }

  if (TREE && tid == 0) {
    // for the merge: {sequence, key head, first row's node, last run} of the unit that
    // begins in this run and ends beyond it; sequence -1: none
    int4 cut = make_int4(-1, 0, 0, 0);
    if (sg.slot == 2 * (int)blockIdx.x + 1) {
      const int64_t W = prefix[a.B], nb = tree_runs(W);
      const int64_t end = W * (blockIdx.x + 1) / nb - sg.nt[0] + (sg.nkeys + kFaKeys - 1) / kFaKeys;   // behind the unit
      cut = make_int4(sg.b, sg.g, sg.i0, (int)((end * nb - 1) / W));
    }
    a.cut[blockIdx.x] = cut;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

template <int DK, int DV, int NT, bool TREE>
static cudaError_t launch_full_t(const FullArgs& a, const FullMaps& m, int grid, cudaStream_t st) {
  auto kern = nsa_full_attn_kernel<DK, DV, NT, TREE>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, FaShape<DK, NT>::kSmem);
  if (e != cudaSuccess) return e;
  kern<<<grid, kFaThreads, FaShape<DK, NT>::kSmem, st>>>(a, m);
  return cudaGetLastError();
}

template <int NT, bool TREE>
static cudaError_t launch_full_d(const FullArgs& a, const FullMaps& m, int grid, cudaStream_t st) {
  if (a.d_k == 192 && a.d_v == 128) return launch_full_t<192, 128, NT, TREE>(a, m, grid, st);
  if (a.d_k == 128 && a.d_v == 128) return launch_full_t<128, 128, NT, TREE>(a, m, grid, st);
  if (a.d_k == 64 && a.d_v == 64) return launch_full_t<64, 64, NT, TREE>(a, m, grid, st);
  if (a.d_k == 64 && a.d_v == 128) return launch_full_t<64, 128, NT, TREE>(a, m, grid, st);
  if (a.d_k == 128 && a.d_v == 64) return launch_full_t<128, 64, NT, TREE>(a, m, grid, st);
  if (a.d_k == 192 && a.d_v == 64) return launch_full_t<192, 64, NT, TREE>(a, m, grid, st);
  return cudaErrorInvalidValue;
}

}  // namespace nsa
