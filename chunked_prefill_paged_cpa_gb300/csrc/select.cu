// Page summaries and the selection of pages by them.
//
// A page's summary bounds its keys per kv head: hi_d and lo_d, the largest and the
// smallest of element d over its 16 keys, as whole numbers of at most 127 times one
// scale.  For a query q no key of the page has a larger product than
// sum_d max(q_d hi_d, q_d lo_d); summed over the rows of a unit (the tokens that
// share a selection, by the heads of the group) that is
//   sum_d A_d hi_d + B_d lo_d,   A_d = sum_rows max(q_d, 0), B_d = sum_rows min(q_d, 0),
// one product of 2 D terms per page however many rows the unit has.  The queries
// are made whole numbers too, and so the sums are exact and their order is free:
// the selection depends on the inputs alone, and ties, which go to the lower page,
// are ties everywhere.
//
// Both are bound by HBM: a summary reads 16 keys, a selection reads 1/15 of the
// keys' bytes of a 16-bit cache.
#include <algorithm>

#include <cooperative_groups.h>

#include "cpa_internal.cuh"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace cpa {
namespace {

constexpr int kPageTokens = 16;
constexpr float kTiny = 0x1p-100f;  // smaller magnitudes count as zero: 127 / x stays finite

// ---------------------------------------------------------------------------
// Summaries.  A warp makes one page's row of one kv head: the lanes of a row of
// keys hold 16 bytes of it each, and the groups of lanes take different keys.
constexpr int kSumThreads = 256;

enum { KEYS_BF16 = 0, KEYS_F16 = 1, KEYS_E4M3 = 2, KEYS_F32 = 3 };

// The elements of 16 bytes.
template <int KT>
__device__ __forceinline__ void widen(const uint4 &x, float *f) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (KT == KEYS_F32) {
      f[i] = __uint_as_float(w[i]);
    } else if constexpr (KT == KEYS_BF16) {
      f[2 * i] = bf16_lo(w[i]);
      f[2 * i + 1] = bf16_hi(w[i]);
    } else if constexpr (KT == KEYS_F16) {
      const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
      f[2 * i] = y.x;
      f[2 * i + 1] = y.y;
    } else {
      uint32_t h[2];
      ptx::e4m3x4_to_f16x4(w[i], h[0], h[1]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&h[j]));
        f[4 * i + 2 * j] = y.x;
        f[4 * i + 2 * j + 1] = y.y;
      }
    }
  }
}

// The scale and the factor to whole numbers of values whose largest magnitude is
// `most`; fine: all of them are finite.
__device__ __forceinline__ float whole_factor(float most, bool fine) {
  return fine && most >= kTiny ? __fdiv_rn(127.f, most) : 0.f;
}
__device__ __forceinline__ int whole(float x, float factor) {
  return factor == 0.f ? 0 : __float2int_rn(__fmul_rn(x, factor));
}

struct SummariseArgs {
  const unsigned char *k_cache;
  const int32_t *table, *starts, *lens;
  int num_seqs, max_pages, Hkv;
  int64_t num_pages;
  unsigned char *summaries;
  uint32_t *status;
};

template <int KT, int D>
__global__ void __launch_bounds__(kSumThreads) summarise_kernel(const SummariseArgs a) {
  constexpr int EB = KT == KEYS_F32 ? 4 : KT == KEYS_E4M3 ? 1 : 2;
  constexpr int N = 16 / EB;             // elements of a lane
  constexpr int LANES = D * EB / 16;     // lanes of a row: 4 .. 32
  constexpr int ROWS = 32 / LANES;       // rows of a load
  constexpr int ROW_BYTES = 2 * D + 16;  // of a summary
  // every CTA: pages completed before each sequence's
  extern __shared__ int before[];  // [num_seqs + 1]
  __shared__ int warps[kSumThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, S = a.num_seqs;
  auto pages_of = [&](int s, int &first) {
    const int q = __ldg(a.starts + s + 1) - __ldg(a.starts + s);
    const int len = min(__ldg(a.lens + s), a.max_pages * kPageTokens);
    first = max(0, len - q) / kPageTokens;
    return q > 0 && len >= q ? len / kPageTokens - first : 0;
  };
  int sum = 0;
  for (int s0 = 0; s0 < S; s0 += kSumThreads) {
    const int s = s0 + tid;
    int first, n = s < S ? pages_of(s, first) : 0, in = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) in += y;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = in;
    __syncthreads();
    for (int w = 0; w < kSumThreads / 32; ++w) {
      if (w < warp) in += warps[w];
    }
    if (s < S) before[s] = sum + in - n;
    for (int w = 0; w < kSumThreads / 32; ++w) sum += warps[w];
  }
  if (tid == 0) before[S] = sum;
  __syncthreads();

  const int64_t items = (int64_t)sum * a.Hkv;
  for (int64_t i = (int64_t)blockIdx.x * (kSumThreads / 32) + warp; i < items;
       i += (int64_t)gridDim.x * (kSumThreads / 32)) {
    const int n = (int)(i / a.Hkv), g = (int)(i - (int64_t)n * a.Hkv);
    int lo = 0, hi = S - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (before[mid] <= n) lo = mid; else hi = mid - 1;
    }
    int first;
    pages_of(lo, first);
    const int page = __ldg(a.table + (int64_t)lo * a.max_pages + first + n - before[lo]);
    if (page < 0 || page >= a.num_pages) {
      if (a.status && lane == 0) atomicOr(a.status, STATUS_BAD_PAGE);
      continue;
    }
    const unsigned char *keys = a.k_cache + ((int64_t)page * a.Hkv + g) * (kPageTokens * D * EB) + lane * 16;
    uint4 x[kPageTokens / ROWS];
#pragma unroll
    for (int r = 0; r < kPageTokens / ROWS; ++r) x[r] = __ldg(reinterpret_cast<const uint4 *>(keys + r * 512));
    float up[N], down[N];
    bool fine = true;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      up[e] = -INFINITY;
      down[e] = INFINITY;
    }
#pragma unroll
    for (int r = 0; r < kPageTokens / ROWS; ++r) {
      float f[N];
      widen<KT>(x[r], f);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        fine &= fabsf(f[e]) < INFINITY;
        up[e] = fmaxf(up[e], f[e]);
        down[e] = fminf(down[e], f[e]);
      }
    }
    float most = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) {
#pragma unroll
      for (int o = LANES; o < 32; o <<= 1) {
        up[e] = fmaxf(up[e], __shfl_xor_sync(0xffffffffu, up[e], o));
        down[e] = fminf(down[e], __shfl_xor_sync(0xffffffffu, down[e], o));
      }
      most = fmaxf(most, fmaxf(fabsf(up[e]), fabsf(down[e])));
    }
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    fine = __all_sync(0xffffffffu, fine);
    const float factor = whole_factor(most, fine);
    // the first group of lanes stores the largest, and the second (the same one,
    // where there is no second) the smallest
    unsigned char *row = a.summaries + ((int64_t)page * a.Hkv + g) * ROW_BYTES;
    const int l = lane % LANES;
    auto store = [&](unsigned char *to, const float *f) {
      uint32_t w[N / 4];
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        w[i] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[i] |= (uint32_t)(whole(f[4 * i + j], factor) & 255) << (8 * j);
      }
      if constexpr (N == 4) *reinterpret_cast<uint32_t *>(to + l * 4) = w[0];
      if constexpr (N == 8) *reinterpret_cast<uint2 *>(to + l * 8) = make_uint2(w[0], w[1]);
      if constexpr (N == 16) *reinterpret_cast<uint4 *>(to + l * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    };
    if (lane < LANES) store(row, up);
    if (LANES == 32 || (lane >= LANES && lane < 2 * LANES)) store(row + D, down);
    if (lane == 0) {
      const float scale = !fine ? INFINITY : most >= kTiny ? __fdiv_rn(most, 127.f) : 0.f;
      *reinterpret_cast<uint4 *>(row + 2 * D) = make_uint4(__float_as_uint(scale), 0u, 0u, 0u);
    }
  }
}

// ---------------------------------------------------------------------------
// Selection.  A cluster of CTAs per (unit, kv head); each CTA scores a run of the
// candidate pages and keeps the scores in its shared memory; the n-th largest is
// found by its digits, eight bits at a time from the first that differs, over all
// of the cluster's scores.
constexpr int kDigits = 256;
constexpr int kMaxCluster = 8;  // (portable)

struct SelectArgs {
  const void *q;
  const unsigned char *summaries;
  const int32_t *table, *starts, *lens;
  int num_seqs, num_tokens, max_pages, Hkv, G;
  int64_t num_pages;
  int budget, sink_pages, local_pages;
  int32_t *selected;
  uint32_t *status;
  int capacity;  // scores of a CTA
};

// A score as a key whose order as a whole number is the score's (-0 as +0); never 0.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
constexpr uint32_t kTopKey = 0xff800000u;  // of +infinity

template <int QT, int D, int THREADS>
__global__ void __launch_bounds__(THREADS) select_kernel(const SelectArgs a) {
  constexpr int WARPS = THREADS / 32;
  constexpr int QB = QT == KEYS_F32 ? 4 : 2;
  constexpr int QN = 16 / QB;            // elements of 16 bytes of a query
  constexpr int ROW_BYTES = 2 * D + 16;  // of a summary
  constexpr int CW = 2 * D / 64;         // 16-byte words of a lane's part of it
  extern __shared__ uint32_t keys[];     // [capacity]
  __shared__ int s_up[D], s_down[D];
  __shared__ __align__(16) int8_t s_codes[2 * D];
  __shared__ int s_red[WARPS][3];
  __shared__ __align__(16) int s_hist[4][kDigits], s_all[kDigits];
  __shared__ uint32_t s_range[3];  // this CTA's ordinary keys: least, largest; its top keys
  __shared__ int s_more[2];        // this CTA's keys above the threshold, and at it
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank(), g = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto sync = [&] { if (nc > 1) cluster.sync(); else __syncthreads(); };

  // The unit.  Number c < num_seqs is the first of sequence c; number num_seqs + m
  // a later one whose first token is among TU w .. TU w + TU - 1, w = m + 1: at most
  // one is, and its sequence holds token TU w - 1.
  const int TU = kUnitRows / a.G, c = blockIdx.x / nc;
  int s = c, first = 0;
  if (c >= a.num_seqs) {
    const int64_t t = (int64_t)TU * (c - a.num_seqs + 1) - 1;
    int lo = 0, hi = a.num_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(a.starts + mid) <= t) lo = mid; else hi = mid - 1;
    }
    s = lo;
    const int64_t at = t + 1 - __ldg(a.starts + s);
    first = at > 0 && at < a.num_tokens ? (int)((at + TU - 1) / TU * TU) : a.num_tokens;
  }
  const int qs = __ldg(a.starts + s);
  const int q_len = min(__ldg(a.starts + s + 1), a.num_tokens) - qs;
  if (qs < 0 || first >= q_len) return;  // (the whole cluster)
  const int t0 = qs + first, tokens = min(TU, q_len - first);
  int ctx = __ldg(a.lens + s);
  if (ctx > a.max_pages * kPageTokens) {
    if (tid == 0 && a.status) atomicOr(a.status, STATUS_BAD_PAGE);
    ctx = a.max_pages * kPageTokens;
  }
  const int limit = unit_limit(max(0, ctx - q_len + first), a.local_pages);
  const int n = min(limit, a.budget);
  int32_t *list = a.selected + ((int64_t)t0 * a.Hkv + g) * a.budget;
  for (int i = n + rank * THREADS + tid; i < a.budget; i += nc * THREADS) list[i] = -1;
  if (n == limit) {
    for (int i = rank * THREADS + tid; i < n; i += nc * THREADS) list[i] = i;
    return;
  }

  // The unit's rows as whole numbers: the largest magnitude, then the sums.  A short
  // last unit's last token counts for the tokens that it lacks.
  for (int i = tid; i < D; i += THREADS) s_up[i] = s_down[i] = 0;
  for (int i = tid; i < 4 * kDigits; i += THREADS) s_hist[0][i] = 0;
  constexpr int QL = D / QN;  // 16-byte words of a query
  const int words = tokens * a.G * QL;
  const int last_weight = first > 0 ? 1 + TU - tokens : 1;
  auto load = [&](int w, float *f) {
    const int row = w / QL, tok = t0 + row / a.G, head = g * a.G + row % a.G;
    const uint4 x = __ldg(reinterpret_cast<const uint4 *>(
        static_cast<const unsigned char *>(a.q) + (((int64_t)tok * a.Hkv * a.G + head) * D) * QB) + w % QL);
    widen<QT>(x, f);
  };
  float most = 0.f;
  bool fine = true;
  for (int w = tid; w < words; w += THREADS) {
    float f[QN];
    load(w, f);
#pragma unroll
    for (int e = 0; e < QN; ++e) {
      fine &= fabsf(f[e]) < INFINITY;
      most = fmaxf(most, fabsf(f[e]));
    }
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  if (lane == 0) s_red[warp][0] = __float_as_int(most);
  fine = __syncthreads_and(fine);
  for (int w = 0; w < WARPS; ++w) most = fmaxf(most, __int_as_float(s_red[w][0]));
  const float factor = whole_factor(most, fine);
  for (int w = tid; w < words; w += THREADS) {
    float f[QN];
    load(w, f);
    const int weight = w / (QL * a.G) == tokens - 1 ? last_weight : 1;
#pragma unroll
    for (int e = 0; e < QN; ++e) {
      const int x = whole(f[e], factor);
      if (x) atomicAdd((x > 0 ? s_up : s_down) + w % QL * QN + e, weight * abs(x));
    }
  }
  __syncthreads();
  // seven bits of each sum, by the same shift
  int top = 0;
  for (int i = tid; i < D; i += THREADS) top = max(top, max(s_up[i], s_down[i]));
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) s_red[warp][1] = top;
  __syncthreads();
  for (int w = 0; w < WARPS; ++w) top = max(top, s_red[w][1]);
  const int shift = max(0, 25 - __clz(top)), half = (1 << shift) >> 1;
  for (int i = tid; i < D; i += THREADS) {
    s_codes[i] = (int8_t)min((s_up[i] + half) >> shift, 127);
    s_codes[D + i] = (int8_t)-min((s_down[i] + half) >> shift, 127);
  }
  __syncthreads();

  // Scores of pages j0 .. j1 - 1: four lanes to a page, a warp 32 pages at a time.
  const int per = (limit + nc - 1) / nc;
  const int j0 = min(limit, rank * per), j1 = min(limit, j0 + per);
  int4 qc[CW];
#pragma unroll
  for (int i = 0; i < CW; ++i) qc[i] = *reinterpret_cast<const int4 *>(s_codes + i * 64 + (lane & 3) * 16);
  const int32_t *bt = a.table + (int64_t)s * a.max_pages;
  uint32_t least = 0xffffffffu, largest = 0u;
  int tops = 0;
  for (int j = j0 + warp * 32; j < j1; j += THREADS) {
    int entry = -1;
    if (j + lane < j1) {
      entry = __ldg(bt + j + lane);
      if (entry < 0 || entry >= a.num_pages) {
        if (a.status) atomicOr(a.status, STATUS_BAD_PAGE);
        entry = -1;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int e = __shfl_sync(0xffffffffu, entry, k * 8 + (lane >> 2));
      const unsigned char *row = a.summaries + ((int64_t)max(e, 0) * a.Hkv + g) * ROW_BYTES;
      int sum = 0;
#pragma unroll
      for (int i = 0; i < CW; ++i) {
        const int4 x = __ldg(reinterpret_cast<const int4 *>(row + i * 64 + (lane & 3) * 16));
        sum = __dp4a(x.x, qc[i].x, sum);
        sum = __dp4a(x.y, qc[i].y, sum);
        sum = __dp4a(x.z, qc[i].z, sum);
        sum = __dp4a(x.w, qc[i].w, sum);
      }
      const float scale = __ldg(reinterpret_cast<const float *>(row + 2 * D));
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const int page = j + k * 8 + (lane >> 2);
      if ((lane & 3) == 0 && page < j1) {
        uint32_t key = scale < INFINITY ? order_key(__fmul_rn(scale, (float)sum)) : kTopKey;
        if (page < a.sink_pages) key = kTopKey;
        if (e < 0) key = 0u;
        keys[page - j0] = key;
        if (key == kTopKey) {
          ++tops;
        } else {
          least = min(least, key);
          largest = max(largest, key);
        }
      }
    }
  }
  least = __reduce_min_sync(0xffffffffu, least);
  largest = __reduce_max_sync(0xffffffffu, largest);
  tops = __reduce_add_sync(0xffffffffu, tops);
  if (lane == 0) {
    s_red[warp][0] = (int)least;
    s_red[warp][1] = (int)largest;
    s_red[warp][2] = tops;
  }
  __syncthreads();
  tops = 0;
  for (int w = 0; w < WARPS; ++w) {
    least = min(least, (uint32_t)s_red[w][0]);
    largest = max(largest, (uint32_t)s_red[w][1]);
    tops += s_red[w][2];
  }
  if (nc > 1) {
    if (tid == 0) {
      s_range[0] = least;
      s_range[1] = largest;
      s_range[2] = (uint32_t)tops;
    }
    cluster.sync();
    tops = 0;
    for (int b = 0; b < nc; ++b) {
      const uint32_t *r = cluster.map_shared_rank(s_range, b);
      least = min(least, r[0]);
      largest = max(largest, r[1]);
      tops += (int)r[2];
    }
  }

  // The n-th largest key: found under the mask, the `want` first of those that have
  // its bits belong to the selection.  The digits from the highest bit in which the
  // ordinary keys differ; until no key is left out of those with the bits found.
  uint32_t found = kTopKey, mask = 0xffffffffu;
  int want = n;
  if (tops < n) {
    want = n - tops;
    int bits = 32 - __clz(least ^ largest);  // that differ
    mask = bits == 32 ? 0u : 0xffffffffu << bits;
    found = largest & mask;
    for (int pass = 0; bits > 0; ++pass) {
      const int d = max(0, bits - 8);
      for (int i = tid; i < j1 - j0; i += THREADS) {
        const uint32_t key = keys[i];
        if (key != kTopKey && (key & mask) == found) atomicAdd(s_hist[pass] + ((key & ~mask) >> d), 1);
      }
      sync();
      const int *counts = s_hist[pass];
      if (nc > 1) {
        for (int i = tid; i < kDigits; i += THREADS) {
          int x[kMaxCluster], sum = 0;
#pragma unroll
          for (int b = 0; b < kMaxCluster; ++b) x[b] = b < nc ? *cluster.map_shared_rank(s_hist[pass] + i, b) : 0;
#pragma unroll
          for (int b = 0; b < kMaxCluster; ++b) sum += x[b];
          s_all[i] = sum;
        }
        __syncthreads();
        counts = s_all;
      }
      // every warp finds the digit for itself: a lane holds eight, from the top
      const int4 hi = *reinterpret_cast<const int4 *>(counts + 252 - lane * 8),
                 lo = *reinterpret_cast<const int4 *>(counts + 248 - lane * 8);
      const int count[8] = {hi.w, hi.z, hi.y, hi.x, lo.w, lo.z, lo.y, lo.x};
      int sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += count[i];
      int upto = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const int owner = __ffs(__ballot_sync(0xffffffffu, upto >= want)) - 1;
      int left = want - (upto - sum), digit = 0, here = 0;
      bool done = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (!done) {
          digit = 255 - lane * 8 - i;
          here = count[i];
          done = left <= here;
          if (!done) left -= here;
        }
      }
      digit = __shfl_sync(0xffffffffu, digit, owner);
      here = __shfl_sync(0xffffffffu, here, owner);
      want = __shfl_sync(0xffffffffu, left, owner);
      found |= (uint32_t)digit << d;
      mask = 0xffffffffu << d;
      bits = d;
      if (here == want) break;
      if (nc > 1) __syncthreads();  // (s_all has been read)
    }
  }

  // All keys above it, and the first `want` of those at it, in the pages' order.
  // A warp has a run of the pages.
  auto at_it = [&](uint32_t key) { return (key & mask) == found && (key != kTopKey || found == kTopKey); };
  const int run = ((j1 - j0 + WARPS - 1) / WARPS + 31) / 32 * 32;
  const int r0 = min(j1 - j0, warp * run), r1 = min(j1 - j0, r0 + run);
  int above = 0, at = 0;
  for (int i = r0 + lane; i < r1; i += 32) {
    const uint32_t key = keys[i];
    const bool eq = at_it(key);
    above += !eq && key > found;
    at += eq;
  }
  above = __reduce_add_sync(0xffffffffu, above);
  at = __reduce_add_sync(0xffffffffu, at);
  __syncthreads();  // (s_red has been read)
  if (lane == 0) {
    s_red[warp][0] = above;
    s_red[warp][1] = at;
  }
  __syncthreads();
  above = at = 0;
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) {
      above += s_red[w][0];
      at += s_red[w][1];
    }
  }
  if (nc > 1) {
    if (warp == WARPS - 1 && lane == 0) {
      s_more[0] = above + s_red[warp][0];
      s_more[1] = at + s_red[warp][1];
    }
    cluster.sync();
    for (int b = 0; b < rank; ++b) {
      above += *cluster.map_shared_rank(s_more, b);
      at += *cluster.map_shared_rank(s_more + 1, b);
    }
    cluster.sync();  // no CTA leaves while another reads its counts
  }
  for (int i = r0; i < r1; i += 32) {
    const uint32_t key = i + lane < r1 ? keys[i + lane] : 0u;
    const bool eq = i + lane < r1 && at_it(key), gt = i + lane < r1 && !eq && key > found;
    const unsigned mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
    const unsigned low = (1u << lane) - 1u;
    const int eq_before = at + __popc(me & low);
    if (gt || (eq && eq_before < want))
      list[above + __popc(mg & low) + min(eq_before, want)] = j0 + i + lane;
    above += __popc(mg);
    at += __popc(me);
  }
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// The status word of a workspace that may be there.
int status_of(const cpa_desc *d, uint32_t **status) {
  *status = nullptr;
  if (!d->workspace) return CPA_OK;
  if (!aligned(d->workspace, 256) || d->workspace_bytes < 256) return CPA_ERR_WORKSPACE;
  *status = static_cast<uint32_t *>(d->workspace);
  return CPA_OK;
}

// Checks of a packed batch's metadata.
int check_batch(const cpa_desc *d, int num_seqs, const void *table, const void *starts, const void *lens) {
  if (d->max_pages_per_seq <= 0 || !table || !starts || !lens || !aligned(table, 4) || !aligned(starts, 4) ||
      !aligned(lens, 4))
    return CPA_ERR_ARG;
  if ((int64_t)d->max_pages_per_seq * kPageTokens > (1 << 30) || d->num_pages > INT32_MAX / kPageTokens ||
      num_seqs > kDecodeMaxSeqs)
    return CPA_ERR_UNSUPPORTED;
  return CPA_OK;
}

template <int KT, int D>
cudaError_t launch_summarise(const SummariseArgs &a, int sms, cudaStream_t stream) {
  // (48 KB of shared memory at most: 4097 words)
  const size_t smem = sizeof(int) * ((size_t)a.num_seqs + 1);
  summarise_kernel<KT, D><<<4 * sms, kSumThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

// CTAs of a kernel resident on an SM with this much shared memory each.
template <int QT, int D, int THREADS>
int select_resident(int smem) {
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, select_kernel<QT, D, THREADS>, THREADS, smem) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  return n;
}

constexpr int kMaxScores = 48 * 1024;  // of a CTA: 192 KB

template <int QT, int D, int THREADS>
cudaError_t launch_select_on(SelectArgs a, int64_t units, int sms, cudaStream_t stream) {
  const int device = current_device();
  static PerDevice configured;
  cudaError_t e = cudaSuccess;
  if (configured.get(device, [&] {
        e = cudaFuncSetAttribute(select_kernel<QT, D, THREADS>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxScores * 4);
        return e == cudaSuccess ? 1 : 0;
      }) < 1)
    return e;
  // CTAs per (unit, kv head): the number with the fewest rounds of resident CTAs,
  // counted in a warp's turns of 32 pages, all else costing about ten
  int nc = 0;
  int64_t least = INT64_MAX;
  for (int n = 1; n <= kMaxCluster; n *= 2) {
    const int per = (a.max_pages + n - 1) / n;
    if (per > kMaxScores) continue;
    const int64_t slots = (int64_t)std::max(1, select_resident<QT, D, THREADS>(per * 4)) * sms;
    const int64_t cost = (units * a.Hkv * n + slots - 1) / slots * ((per + THREADS - 1) / THREADS + 10);
    if (cost < least) {
      least = cost;
      nc = n;
    }
  }
  a.capacity = (a.max_pages + nc - 1) / nc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * nc), a.Hkv);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = (size_t)a.capacity * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = nc;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, select_kernel<QT, D, THREADS>, a);
}

template <int QT, int D>
cudaError_t launch_select(const SelectArgs &a, int sms, cudaStream_t stream) {
  const int TU = kUnitRows / a.G;
  const int64_t units = a.num_seqs + (a.num_tokens > a.num_seqs ? (a.num_tokens - 1) / TU : 0);
  // units whose clusters leave SMs idle: as many loads on their way as an SM takes
  return units * a.Hkv * kMaxCluster <= sms ? launch_select_on<QT, D, 512>(a, units, sms, stream)
                                            : launch_select_on<QT, D, 128>(a, units, sms, stream);
}

}  // namespace
}  // namespace cpa

using namespace cpa;

extern "C" size_t cpa_summary_bytes(const cpa_desc *desc) {
  if (check_shape(desc) != CPA_OK) return 0;
  return (size_t)desc->num_pages * desc->num_kv_heads * summary_row_bytes(desc->head_dim);
}

extern "C" int cpa_summarise_pages(const void *k_cache, const int32_t *block_table,
                                   const int32_t *query_start_loc, const int32_t *seq_lens,
                                   int32_t num_seqs, void *summaries, const cpa_desc *desc,
                                   void *stream) {
  int rc = check_shape(desc);
  if (rc != CPA_OK) return rc;
  if (num_seqs < 0) return CPA_ERR_ARG;
  if (num_seqs == 0) return CPA_OK;
  if (!k_cache || !summaries || !aligned(k_cache, 16) || !aligned(summaries, 16)) return CPA_ERR_ARG;
  if ((rc = check_batch(desc, num_seqs, block_table, query_start_loc, seq_lens)) != CPA_OK) return rc;
  SummariseArgs a{};
  if ((rc = status_of(desc, &a.status)) != CPA_OK) return rc;
  a.k_cache = static_cast<const unsigned char *>(k_cache);
  a.table = block_table;
  a.starts = query_start_loc;
  a.lens = seq_lens;
  a.num_seqs = num_seqs;
  a.max_pages = desc->max_pages_per_seq;
  a.Hkv = desc->num_kv_heads;
  a.num_pages = desc->num_pages;
  a.summaries = static_cast<unsigned char *>(summaries);
  const int sms = sm_count(current_device());
  if (sms <= 0) return CPA_ERR_CUDA;
  cudaStream_t st = (cudaStream_t)stream;
  const int kt = desc->kv_dtype == CPA_KV_E4M3 ? KEYS_E4M3
                 : desc->dtype == CPA_F32      ? KEYS_F32
                 : desc->dtype == CPA_F16      ? KEYS_F16
                                               : KEYS_BF16;
  const bool wide = desc->head_dim == 128;
  cudaError_t e;
  if (kt == KEYS_E4M3) e = wide ? launch_summarise<KEYS_E4M3, 128>(a, sms, st) : launch_summarise<KEYS_E4M3, 64>(a, sms, st);
  else if (kt == KEYS_F32) e = wide ? launch_summarise<KEYS_F32, 128>(a, sms, st) : launch_summarise<KEYS_F32, 64>(a, sms, st);
  else if (kt == KEYS_F16) e = wide ? launch_summarise<KEYS_F16, 128>(a, sms, st) : launch_summarise<KEYS_F16, 64>(a, sms, st);
  else e = wide ? launch_summarise<KEYS_BF16, 128>(a, sms, st) : launch_summarise<KEYS_BF16, 64>(a, sms, st);
  return e == cudaSuccess ? CPA_OK : CPA_ERR_CUDA;
}

extern "C" int cpa_select_pages(const void *q, const void *summaries, const int32_t *block_table,
                                const int32_t *query_start_loc, const int32_t *seq_lens,
                                int32_t num_seqs, int32_t num_selected, int32_t sink_pages,
                                int32_t local_pages, int32_t *selected, void *stream,
                                const cpa_desc *desc) {
  int rc = check_shape(desc);
  if (rc != CPA_OK) return rc;
  if (num_seqs < 0 || num_selected < 0 || sink_pages < 0 || local_pages < 1) return CPA_ERR_ARG;
  if (num_selected > kMaxSelected) return CPA_ERR_UNSUPPORTED;
  if (num_seqs == 0 || desc->num_tokens == 0 || num_selected == 0) return CPA_OK;
  if (desc->num_tokens < num_seqs) return CPA_ERR_ARG;  // every sequence has q_len >= 1
  if (!q || !summaries || !selected || !aligned(q, 16) || !aligned(summaries, 16) || !aligned(selected, 4))
    return CPA_ERR_ARG;
  if ((rc = check_batch(desc, num_seqs, block_table, query_start_loc, seq_lens)) != CPA_OK) return rc;
  if (desc->max_pages_per_seq > kMaxCluster * kMaxScores) return CPA_ERR_UNSUPPORTED;
  SelectArgs a{};
  if ((rc = status_of(desc, &a.status)) != CPA_OK) return rc;
  a.q = q;
  a.summaries = static_cast<const unsigned char *>(summaries);
  a.table = block_table;
  a.starts = query_start_loc;
  a.lens = seq_lens;
  a.num_seqs = num_seqs;
  a.num_tokens = (int)desc->num_tokens;
  a.max_pages = desc->max_pages_per_seq;
  a.Hkv = desc->num_kv_heads;
  a.G = desc->num_q_heads / desc->num_kv_heads;
  a.num_pages = desc->num_pages;
  a.budget = num_selected;
  a.sink_pages = sink_pages;
  a.local_pages = std::min(local_pages, 1 << 26);
  a.selected = selected;
  const int sms = sm_count(current_device());
  if (sms <= 0) return CPA_ERR_CUDA;
  cudaStream_t st = (cudaStream_t)stream;
  const bool wide = desc->head_dim == 128;
  cudaError_t e;
  if (desc->dtype == CPA_F32) e = wide ? launch_select<KEYS_F32, 128>(a, sms, st) : launch_select<KEYS_F32, 64>(a, sms, st);
  else if (desc->dtype == CPA_F16) e = wide ? launch_select<KEYS_F16, 128>(a, sms, st) : launch_select<KEYS_F16, 64>(a, sms, st);
  else e = wide ? launch_select<KEYS_BF16, 128>(a, sms, st) : launch_select<KEYS_BF16, 64>(a, sms, st);
  return e == cudaSuccess ? CPA_OK : CPA_ERR_CUDA;
}
