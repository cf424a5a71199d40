// Attention in fp32 of rows that see a window, or selected pages: chunks and single
// tokens, one launch.
//
// A tile is 16 query rows of one (sequence, kv head): 16 / G consecutive tokens
// by the G heads of the group (row = token * G + head); a single token fills G
// of them.  A warp computes a tile against runs of 8 keys (half a page),
//   S = Q K^T   m16n8k8, rows x keys
//   O += P V    m16n8k8, rows x dims, one k-step of 8 keys
// on the tensor cores with fp32's precision, every operand as the sum of two tf32
// values (tf32_split.cuh).  Sums, softmax and outputs are fp32.
//
// K and V go from global memory straight into the operands' registers; which
// dim stands at which k, and which key of the eight, is free as long as the
// other operand follows: dims so that a lane's elements are whole 16-byte
// words, keys so that S's layout is at once P's layout as an operand.  The next
// eight keys are on their way while the present ones are computed: K's as soon
// as S has used K's registers, V's after O has used V's (registers for both
// halves twice would spill at head_dim 128).  Q waits in shared memory, split,
// in the order of the operands.
//
// Two shapes of a CTA of four warps (template ROWS): four tiles of consecutive
// rows against all their keys (the warps read the same pages at about the same
// time, from L1), where there are tiles enough to fill the SMs; or one tile
// whose keys are split over the warps and over a cluster of CTAs, joined through
// shared memory.
#include <algorithm>

#include <cooperative_groups.h>

#include "cpa_internal.cuh"
#include "ptx.cuh"
#include "tf32_split.cuh"

namespace cg = cooperative_groups;

namespace cpa {
namespace {

constexpr int kPageKeys = 16, kUnitKeys = 8;
constexpr int kWarps = 4;
constexpr int kRows = 16;
// The tensor cores cut what they add up off towards zero: a sum of all of a row's
// keys in one place loses some 2^-24 with each product, in one direction (2.9e-5 of
// the output over 4096 keys).  So a sum takes the products of kSumUnits units, and
// is then added, rounded to nearest, to the one in shared memory: 6.5e-7 over 4096
// keys, what a plain fp32 product gives.  (4 tokens and a 1000-token chunk, 8 kv heads
// of 128, window 1024 / 4096: 406 / 1525 us without this, 422 / 1572 with 8 units,
// 413 / 1540 with 16, which lose 1.0e-6; a new sum for every unit, added in
// registers, 466 / 1782.  1000 tokens of 2 kv heads of 64 over 64 / 128 pages 75 / 114
// and 79 / 128 us, the longest loss: less L1 beside the larger shared memory.)
constexpr int kSumUnits = 8;
constexpr float kMoveThreshold = 8.0f;  // log2 units, as in the step kernel

// Eight keys of K and V of one kv head as a lane holds them.  With r = lane / 4
// and c = lane % 4: of K, row r, 16 bytes of each 64 (at 16 c); of V, rows 2c
// and 2c + 1, 16 bytes of each 128 (at 16 r).
template <int D>
struct UnitRegs {
  float k[D / 4];
  float v[2][D / 8];

  // (not the read-only path: the append launched just before may still write the
  // cache when this kernel starts)
  __device__ __forceinline__ void load_k(const float *kp, int r, int c) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const float4 x = *reinterpret_cast<const float4 *>(kp + r * D + i * 16 + c * 4);
      k[4 * i] = x.x;
      k[4 * i + 1] = x.y;
      k[4 * i + 2] = x.z;
      k[4 * i + 3] = x.w;
    }
  }
  __device__ __forceinline__ void load_v(const float *vp, int r, int c) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const float4 x = *reinterpret_cast<const float4 *>(vp + (2 * c + j) * D + i * 32 + r * 4);
        v[j][4 * i] = x.x;
        v[j][4 * i + 1] = x.y;
        v[j][4 * i + 2] = x.z;
        v[j][4 * i + 3] = x.w;
      }
  }
};

template <int D, bool ROWS, int VIS>
__global__ void __launch_bounds__(kWarps * 32, 2) window_f32_kernel(const AttnParams p) {
  constexpr int KS = D / 8;               // k-steps of S, and 8-dim tiles of O
  constexpr int TILES = ROWS ? kWarps : 1;  // tiles of the CTA
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank(), g = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const int G = p.Hq / p.Hkv, TM = TILES * kRows / G;  // tokens per CTA
  // Q, split: [tile][k-step][hi, lo][lane], 16 bytes; later the CTA's O.  Then the
  // warps' O
  extern __shared__ __align__(16) float sm[];
  float *sm_o = sm + TILES * kRows * D * 2;

  // Sequence s owns the CTA numbers from query_start_loc[s] / TM + s on: at
  // least one per TM tokens begun, and some left over.  The last s whose first
  // number is not above this CTA's, 32 candidates at a time.
  const int z = blockIdx.x / nc;
  int s = 0;
  for (int n = p.num_seqs; n > 1;) {  // the answer is in [s, s + n)
    const int step = (n + 31) / 32, i = s + lane * step;
    const bool le = lane * step < n && __ldg(p.query_start_loc + i) / TM + i <= z;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int last = m ? 31 - __clz(m) : 0;
    const int end = s + n;
    s += last * step;
    n = min(step, end - s);
  }
  const int qs = __ldg(p.query_start_loc + s);
  const int q_len = min(__ldg(p.query_start_loc + s + 1), p.num_tokens) - qs;
  int ctx = __ldg(p.seq_lens + s);
  const int cap = p.max_pages * kPageKeys;
  if (ctx > cap) {
    if (threadIdx.x == 0) atomicOr(p.status, STATUS_BAD_PAGE);
    ctx = cap;
  }
  const int first = (z - (qs / TM + s)) * TM;  // the CTA's first token of the sequence
  if (qs < 0 || first < 0 || first >= q_len) {
    // (the whole cluster; in a malformed batch every one, and what comes next on
    // the stream must still find the append done)
    ptx::grid_dependency_wait();
    return;
  }

  for (int i = threadIdx.x; i < TILES * KS * 32; i += kWarps * 32) {
    const int tile = i / (KS * 32), ks = i / 32 % KS, l = i % 32;
    const int dim = (ks >> 1) * 16 + (l & 3) * 4 + (ks & 1) * 2;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = tile * kRows + (l >> 2) + 8 * h, tok = first + row / G;
      float2 x = make_float2(0.f, 0.f);
      if (tok < q_len)
        x = __ldg(reinterpret_cast<const float2 *>(static_cast<const float *>(p.q) +
                                                   ((int64_t)(qs + tok) * p.Hq + g * G + row % G) * D + dim));
      split(x.x, hi[h], lo[h]);
      split(x.y, hi[2 + h], lo[2 + h]);
    }
    uint4 *to = reinterpret_cast<uint4 *>(sm) + (tile * KS + ks) * 64 + l;
    to[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    to[32] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  __syncthreads();

  // the warp's tile: its first token, the positions of this lane's two rows
  const int tok0 = first + (ROWS ? warp * kRows / G : 0);
  const int base = ctx - q_len;
  const int ta = tok0 + r / G, tb = tok0 + (r + 8) / G;
  const int xa = base + ta, xb = base + tb;
  const int x0 = base + tok0, x1 = base + min(tok0 + kRows / G, q_len) - 1;  // first and last
  // the keys that rows of the tile see: [0, near) and [far, x1]; kSelected:
  // [far, x1] and the whole pages listed for the tile's unit
  const bool any = tok0 < q_len && base >= 0;
  int far, near, front;  // front: virtual pages before the gap
  const int32_t *listed = nullptr;
  if constexpr (VIS == kSelected) {
    const int unit = tok0 / (kUnitRows / G) * (kUnitRows / G);
    const int limit = unit_limit(p, max(0, base + unit));
    far = limit * kPageKeys;
    front = min(limit, p.budget);
    near = front * kPageKeys;
    listed = p.selected + ((int64_t)(qs + unit) * p.Hkv + g) * p.budget;
  } else {
    far = max(0, x0 - p.window + 1);
    near = min(p.sinks, far);
    front = (near + kPageKeys - 1) / kPageKeys;
  }
  const int gap = max(0, far / kPageKeys - front);
  const int units = any ? 2 * ((x1 + kPageKeys) / kPageKeys - gap) : 0;
  const int wi = ROWS ? 0 : rank * kWarps + warp, nw = ROWS ? 1 : nc * kWarps;
  const int u0 = (int)((int64_t)units * wi / nw), u1 = (int)((int64_t)units * (wi + 1) / nw);
  const uint4 *q = reinterpret_cast<const uint4 *>(sm) + (ROWS ? warp : 0) * KS * 64 + lane;

  const int32_t *bt = p.block_table + (int64_t)s * p.max_pages;
  const int64_t page_floats = (int64_t)kPageKeys * D;
  const float *kc = static_cast<const float *>(p.k_cache) + g * page_floats;
  const float *vc = static_cast<const float *>(p.v_cache) + g * page_floats;
  const int pg0 = u0 >> 1, pg1 = (u1 + 1) >> 1;
  int entry = -1;  // lane l: the entry of the l-th page from the last look-up on
  auto look_up = [&](int from) {
    entry = -1;
    if (from + lane < pg1) {
      const int v = from + lane;
      int col = v < front ? v : v + gap;
      if (VIS == kSelected && v < front) {
        col = __ldg(listed + v);
        if (col >= front + gap) col = -1;  // not one of the list's candidates
      }
      if (VIS != kSelected || col >= 0) entry = __ldg(bt + col);
      if (entry < 0 || entry >= p.num_pages) {
        atomicOr(p.status, STATUS_BAD_PAGE);
        entry = -1;
      }
    }
  };
  auto find = [&](int u, int64_t &at) -> int {  // unit u's place in the caches, its page's entry
    const int pg = (u >> 1) - pg0;
    if (pg && (u & 1) == 0 && (pg & 31) == 0) look_up(u >> 1);
    const int e = __shfl_sync(0xffffffffu, entry, pg & 31);
    at = (int64_t)max(e, 0) * p.Hkv * page_floats + (u & 1) * kUnitKeys * D;
    return e;
  };

  float o[KS][4];
#pragma unroll
  for (int i = 0; i < KS; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  // The sums of the last units are in `o`, at most kSumUnits, and those of the others
  // in shared memory, in 16-byte words of the lane's own, still to be multiplied by
  // ka and kb (rows r and r + 8)
  float4 *kept = reinterpret_cast<float4 *>(sm_o + warp * kRows * D) + lane;
  bool any_kept = false;
  float ka = 1.f, kb = 1.f;
  auto join_kept = [&](bool keep) {
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      if (any_kept) {
        const float4 y = kept[i * 32];
        o[i][0] = fmaf(y.x, ka, o[i][0]);
        o[i][1] = fmaf(y.y, ka, o[i][1]);
        o[i][2] = fmaf(y.z, kb, o[i][2]);
        o[i][3] = fmaf(y.w, kb, o[i][3]);
      }
      if (keep) {
        kept[i * 32] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
      }
    }
    any_kept = true;
    ka = kb = 1.f;
  };
  float ma = -INFINITY, mb = -INFINITY, la = 0.f, lb = 0.f;  // rows r and r + 8
  const float sl2 = p.scale_log2;

  ptx::grid_dependency_wait();  // the append that may have been launched just before
  UnitRegs<D> x;
  int64_t at = 0;
  int e = -1;
  if (u0 < u1) {
    look_up(pg0);
    e = find(u0, at);
    x.load_k(kc + at, r, c);
    x.load_v(vc + at, r, c);
  }
  for (int u = u0; u < u1; ++u) {
    float acc[4][4] = {};  // hi hi of even and of odd k-steps, hi lo, lo hi
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const uint4 h = q[ks * 64], l = q[ks * 64 + 32];
      uint32_t h0, l0, h1, l1;
      split(x.k[2 * ks], h0, l0);
      split(x.k[2 * ks + 1], h1, l1);
      mma_tf32(acc[ks & 1], h.x, h.y, h.z, h.w, h0, h1);
      mma_tf32(acc[2], h.x, h.y, h.z, h.w, l0, l1);
      mma_tf32(acc[3], l.x, l.y, l.z, l.w, h0, h1);
    }
    int next = -1;
    if (u + 1 < u1) {
      next = find(u + 1, at);
      x.load_k(kc + at, r, c);
    }
    float sc[4];  // (row r, keys 2c, 2c + 1), (row r + 8, the same)
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[i] = ((acc[2][i] + acc[3][i]) + (acc[0][i] + acc[1][i])) * sl2;
    // (a listed page's place among the front pages stands for its column: its
    // keys are all seen)
    const int v = u >> 1, key0 = (v < front ? v : v + gap) * kPageKeys + (u & 1) * kUnitKeys;
    // all rows of the tile see all eight keys: up to the first row's position,
    // and sinks or inside the last row's window
    const int key1 = key0 + kUnitKeys - 1;
    if (e < 0 || key1 > x0 || (VIS == kWindow && key1 >= p.sinks && key0 <= x1 - p.window)) {
      auto sees = [&](int x, int k) {
        return e >= 0 && k <= x && (VIS == kSelected || k < p.sinks || k > x - p.window);
      };
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int k = key0 + 2 * c + j;
        if (!sees(xa, k)) sc[j] = -INFINITY;
        if (!sees(xb, k)) sc[2 + j] = -INFINITY;
        // a key no row sees may hold anything
        if (e < 0 || k > x1 || (k >= near && k < far)) {
#pragma unroll
          for (int i = 0; i < KS; ++i) x.v[j][i] = 0.f;
        }
      }
    }
    const float ya = fmaxf(sc[0], sc[1]), yb = fmaxf(sc[2], sc[3]);
    if (__any_sync(0xffffffffu, ya > ma + kMoveThreshold || yb > mb + kMoveThreshold)) {
      float na = ya, nb = yb;
#pragma unroll
      for (int k = 1; k < 4; k <<= 1) {
        na = fmaxf(na, __shfl_xor_sync(0xffffffffu, na, k));
        nb = fmaxf(nb, __shfl_xor_sync(0xffffffffu, nb, k));
      }
      na = fmaxf(na, ma);
      nb = fmaxf(nb, mb);
      const float fa = ma == -INFINITY ? 0.f : ptx::ex2(ma - na);
      const float fb = mb == -INFINITY ? 0.f : ptx::ex2(mb - nb);
      ma = na;
      mb = nb;
      la *= fa;
      lb *= fb;
      ka *= fa;
      kb *= fb;
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        o[i][0] *= fa;
        o[i][1] *= fa;
        o[i][2] *= fb;
        o[i][3] *= fb;
      }
    }
    const float ra = ma == -INFINITY ? 0.f : ma, rb = mb == -INFINITY ? 0.f : mb;
    const float p0 = ptx::ex2(sc[0] - ra), p1 = ptx::ex2(sc[1] - ra);
    const float p2 = ptx::ex2(sc[2] - rb), p3 = ptx::ex2(sc[3] - rb);
    la += p0 + p1;
    lb += p2 + p3;
    // P as the A operand: key 2c stands at k = c, key 2c + 1 at k = c + 4
    uint32_t h0, h1, h2, h3, l0, l1, l2, l3;
    split(p0, h0, l0);
    split(p2, h1, l1);
    split(p1, h2, l2);
    split(p3, h3, l3);
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      uint32_t vh0, vl0, vh1, vl1;
      split(x.v[0][i], vh0, vl0);
      split(x.v[1][i], vh1, vl1);
      mma_tf32(o[i], h0, h1, h2, h3, vl0, vl1);
      mma_tf32(o[i], l0, l1, l2, l3, vh0, vh1);
      mma_tf32(o[i], h0, h1, h2, h3, vh0, vh1);
    }
    if (u + 1 < u1) x.load_v(vc + at, r, c);
    e = next;
    if ((u - u0) % kSumUnits == kSumUnits - 1 && u + 1 < u1) join_kept(true);
  }
  if (any_kept) join_kept(false);
#pragma unroll
  for (int k = 1; k < 4; k <<= 1) {
    la += __shfl_xor_sync(0xffffffffu, la, k);
    lb += __shfl_xor_sync(0xffffffffu, lb, k);
  }
  // O tile i: column n stands for dim i / 4 * 32 + 4 n + i % 4; this lane has
  // columns 2c and 2c + 1
  auto row_out = [&](int tok, int row) {
    return static_cast<float *>(p.out) + ((int64_t)(qs + tok) * p.Hq + g * G + row % G) * D;
  };
  if constexpr (ROWS) {
    if (!any) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if ((h ? tb : ta) >= q_len) continue;
      float *to = row_out(h ? tb : ta, r + 8 * h);
      const float l = h ? lb : la;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < KS; i += 4)
          *reinterpret_cast<float4 *>(to + i * 8 + (2 * c + n) * 4) =
              make_float4(o[i][2 * h + n] / l, o[i + 1][2 * h + n] / l, o[i + 2][2 * h + n] / l,
                          o[i + 3][2 * h + n] / l);
    }
    return;
  }
  // join the warps, then the cluster's CTAs
  __shared__ float2 sm_ml[kWarps][kRows], cl_ml[kRows];
  float *cl_o = sm;  // (sm_o: [warp][row][D])
  __syncthreads();  // Q and what the lanes kept have been read
  if (c == 0) {
    sm_ml[warp][r] = make_float2(ma, la);
    sm_ml[warp][r + 8] = make_float2(mb, lb);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < KS; i += 4)
        *reinterpret_cast<float4 *>(sm_o + (warp * kRows + r + 8 * h) * D + i * 8 + (2 * c + n) * 4) =
            make_float4(o[i][2 * h + n], o[i + 1][2 * h + n], o[i + 2][2 * h + n], o[i + 3][2 * h + n]);
  __syncthreads();
  struct State {
    float M, L, O;
  };
  auto join = [&](int n, auto ml, auto val) {
    State x = {-INFINITY, 0.f, 0.f};
    for (int i = 0; i < n; ++i) x.M = fmaxf(x.M, ml(i).x);
    for (int i = 0; i < n; ++i) {
      const float2 y = ml(i);
      const float f = y.x == -INFINITY ? 0.f : ptx::ex2(y.x - x.M);
      x.L = fmaf(y.y, f, x.L);
      x.O = fmaf(val(i), f, x.O);
    }
    return x;
  };
  const int rows = any ? min(kRows, (q_len - tok0) * G) : 0;
  auto of_warps = [&](int row, int d) {
    return join(kWarps, [&](int w) { return sm_ml[w][row]; }, [&](int w) { return sm_o[(w * kRows + row) * D + d]; });
  };
  auto store = [&](int row, int d, const State &x) { row_out(tok0 + row / G, row)[d] = x.O / x.L; };
  if (nc == 1) {
    for (int i = threadIdx.x; i < rows * D; i += kWarps * 32) store(i / D, i % D, of_warps(i / D, i % D));
    return;
  }
  for (int i = threadIdx.x; i < rows * D; i += kWarps * 32) {
    const State x = of_warps(i / D, i % D);
    cl_o[i] = x.O;
    if (i % D == 0) cl_ml[i / D] = make_float2(x.M, x.L);
  }
  cluster.sync();
  for (int i = rank * kWarps * 32 + threadIdx.x; i < rows * D; i += nc * kWarps * 32) {
    const int row = i / D;
    store(row, i % D, join(nc, [&](int b) { return *cluster.map_shared_rank(&cl_ml[row], b); },
                           [&](int b) { return *cluster.map_shared_rank(cl_o + i, b); }));
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
}

// Q of four tiles, or of one, later the CTA's O; and the warps' O.
template <int D, bool ROWS>
constexpr int smem_bytes() {
  return ((ROWS ? kWarps : 1) * 2 + kWarps) * kRows * D * (int)sizeof(float);
}

// Lets the kernel have that much.
template <int D, bool ROWS, int VIS>
cudaError_t allow_smem() {
  return cudaFuncSetAttribute(window_f32_kernel<D, ROWS, VIS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              smem_bytes<D, ROWS>());
}

// CTAs resident on an SM of the current device at a time (one tile per CTA).
template <int D, int VIS>
int resident() {
  static PerDevice ctas;
  return std::max(1, ctas.get(current_device(), [] {
    int n = 0;
    if (allow_smem<D, false, VIS>() != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, window_f32_kernel<D, false, VIS>, kWarps * 32,
                                                      smem_bytes<D, false>()) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    return n;
  }));
}

template <int D, bool ROWS, int VIS>
cudaError_t launch(const AttnParams &p, int nc, cudaStream_t stream) {
  constexpr int smem = smem_bytes<D, ROWS>();
  const cudaError_t e = allow_smem<D, ROWS, VIS>();
  if (e != cudaSuccess) return e;
  const int TM = (ROWS ? kWarps : 1) * kRows / (p.Hq / p.Hkv);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(nc * (p.num_tokens / TM + p.num_seqs), p.Hkv);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = nc;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.fused ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, window_f32_kernel<D, ROWS, VIS>, p);
}

template <int VIS>
cudaError_t launch_seeing(const AttnParams &p, int sms, cudaStream_t stream) {
  const int G = p.Hq / p.Hkv;
  const int64_t tiles = (int64_t)p.Hkv * (((int64_t)p.num_tokens * G + kRows - 1) / kRows);
  if (p.num_tokens > p.num_seqs && tiles >= 8 * sms)  // two CTAs of four tiles on every SM
    return p.D == 128 ? launch<128, true, VIS>(p, 1, stream) : launch<64, true, VIS>(p, 1, stream);
  // CTAs per tile: the number with the fewest rounds of resident CTAs, counted
  // in a warp's pages, a start and a join costing about three
  const int64_t pages = std::min<int64_t>(
      p.max_pages, VIS == kSelected ? (int64_t)p.budget + p.local_pages + kUnitRows / kPageKeys / G
                                    : (int64_t)(p.window + kPageKeys - 1) / kPageKeys + 2 +
                                          (p.sinks + kPageKeys - 1) / kPageKeys);
  const int64_t ctas = std::max<int64_t>(tiles, (int64_t)p.Hkv * p.num_seqs);
  const int64_t slots = (int64_t)sms * (p.D == 128 ? resident<128, VIS>() : resident<64, VIS>());
  int nc = 1;
  int64_t least = INT64_MAX;
  for (int n = 1; n <= 8; n *= 2) {
    const int64_t cost = (ctas * n + slots - 1) / slots * ((pages + n * kWarps - 1) / (n * kWarps) + 3);
    if (cost < least) {
      least = cost;
      nc = n;
    }
  }
  return p.D == 128 ? launch<128, false, VIS>(p, nc, stream) : launch<64, false, VIS>(p, nc, stream);
}

}  // namespace

cudaError_t launch_window_f32(const AttnParams &p, int sms, cudaStream_t stream) {
  return p.vis == kSelected ? launch_seeing<kSelected>(p, sms, stream)
                            : launch_seeing<kWindow>(p, sms, stream);
}

}  // namespace cpa
