// Page summaries and the selection of pages by them.
//
// Let hi_d and lo_d be the largest and the smallest of element d over a page's 16 keys
// of a kv head.  For a query q no key of the page has a larger product than
// sum_d max(q_d hi_d, q_d lo_d); summed over the rows of a unit (the tokens that
// share a selection, by the heads of the group) that is
//   sum_d A_d hi_d + B_d lo_d,   A_d = sum_rows max(q_d, 0), B_d = sum_rows min(q_d, 0),
// one product of 2 D terms per page however many rows the unit has.  The score is
// that with hi and lo, the queries and the sums each rounded to whole numbers of at
// most 127: an estimate of the bound.  In whole numbers sums are exact and their order
// is free: the selection depends on the inputs alone, and ties, which go to the lower
// page, are ties everywhere.
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
// keys hold 16 bytes of it each, and the groups of lanes take different keys.  The
// extremes are taken in the keys' own 16 bits, two to an instruction, and the next
// page's keys are on their way meanwhile.  (8 prompts of 8192 tokens, 8 kv heads of
// 128, bf16: 134 MB in 25 us, 5.4 TB/s; element by element in fp32, without the next
// page's loads, 33 us.  The pages' places are looked up 32 at a time, a lane each.)
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

// The larger and the smaller of the elements of two words, NaN where either is:
// fp32, or 16-bit pairs (E4M3 keys as binary16).
template <int KT>
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
  uint32_t y;
  if constexpr (KT == KEYS_F32) asm("max.NaN.f32 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  else if constexpr (KT == KEYS_BF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
template <int KT>
__device__ __forceinline__ uint32_t smaller(uint32_t a, uint32_t b) {
  uint32_t y;
  if constexpr (KT == KEYS_F32) asm("min.NaN.f32 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  else if constexpr (KT == KEYS_BF16) asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  else asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
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
    int len = __ldg(a.lens + s);
    if (len > a.max_pages * kPageTokens) {
      if (a.status) atomicOr(a.status, STATUS_BAD_PAGE);
      len = a.max_pages * kPageTokens;
    }
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
  const int64_t i0 = (int64_t)blockIdx.x * (kSumThreads / 32) + warp, stride = (int64_t)gridDim.x * (kSumThreads / 32);
  // the warp's k-th item: its page and kv head's place in the caches, -1 for none;
  // lane l looks up the l-th from the last look-up on
  int64_t place = -1;
  auto find = [&](int k) -> int64_t {
    if ((k & 31) == 0) {
      const int64_t i = i0 + (k + lane) * stride;
      place = -1;
      if (i < items) {
        const int n = (int)(i / a.Hkv), g = (int)(i - (int64_t)n * a.Hkv);
        int lo = 0, hi = S - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (before[mid] <= n) lo = mid; else hi = mid - 1;
        }
        int first;
        pages_of(lo, first);
        const int page = __ldg(a.table + (int64_t)lo * a.max_pages + first + n - before[lo]);
        if (page >= 0 && page < a.num_pages) place = (int64_t)page * a.Hkv + g;
        else if (a.status) atomicOr(a.status, STATUS_BAD_PAGE);
      }
    }
    return __shfl_sync(0xffffffffu, place, k & 31);
  };
  constexpr int LOADS = kPageTokens / ROWS;
  auto load = [&](int64_t at, uint4 (&x)[LOADS]) {
    const unsigned char *keys = a.k_cache + (at < 0 ? 0 : at) * (kPageTokens * D * EB) + lane * 16;
#pragma unroll
    for (int r = 0; r < LOADS; ++r) x[r] = __ldg(reinterpret_cast<const uint4 *>(keys + r * 512));
  };
  if (i0 >= items) return;
  const int count = (int)((items - i0 + stride - 1) / stride);
  uint4 x[LOADS];
  int64_t at = find(0);
  load(at, x);
  for (int k = 0; k < count; ++k) {
    // (words of extremes: of E4M3 keys twice as many as were loaded)
    constexpr int W = KT == KEYS_E4M3 ? 8 : 4;
    uint32_t hi[W], lo[W];
#pragma unroll
    for (int r = 0; r < LOADS; ++r) {
      uint32_t w[W];
      if constexpr (KT == KEYS_E4M3) {
        ptx::e4m3x4_to_f16x4(x[r].x, w[0], w[1]);
        ptx::e4m3x4_to_f16x4(x[r].y, w[2], w[3]);
        ptx::e4m3x4_to_f16x4(x[r].z, w[4], w[5]);
        ptx::e4m3x4_to_f16x4(x[r].w, w[6], w[7]);
      } else {
        w[0] = x[r].x;
        w[1] = x[r].y;
        w[2] = x[r].z;
        w[3] = x[r].w;
      }
#pragma unroll
      for (int i = 0; i < W; ++i) {
        hi[i] = r ? larger<KT>(hi[i], w[i]) : w[i];
        lo[i] = r ? smaller<KT>(lo[i], w[i]) : w[i];
      }
    }
    const int64_t now = at;
    if (k + 1 < count) {
      at = find(k + 1);
      load(at, x);
    }
    if (now < 0) continue;
#pragma unroll
    for (int i = 0; i < W; ++i) {
#pragma unroll
      for (int o = LANES; o < 32; o <<= 1) {
        hi[i] = larger<KT>(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
        lo[i] = smaller<KT>(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
      }
    }
    float up[N], down[N], most = 0.f;
    bool fine = true;
    constexpr int WIDE = KT == KEYS_E4M3 ? KEYS_F16 : KT;
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      widen<WIDE>(make_uint4(hi[i], hi[i + 1], hi[i + 2], hi[i + 3]), up + i * (N / W));
      widen<WIDE>(make_uint4(lo[i], lo[i + 1], lo[i + 2], lo[i + 3]), down + i * (N / W));
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float y = fmaxf(fabsf(up[e]), fabsf(down[e]));
      fine &= fabsf(up[e]) < INFINITY && fabsf(down[e]) < INFINITY;
      most = fmaxf(most, y);
    }
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    fine = __all_sync(0xffffffffu, fine);
    const float factor = whole_factor(most, fine);
    // the first group of lanes stores the largest, and the second (the same one,
    // where there is no second) the smallest
    unsigned char *row = a.summaries + now * ROW_BYTES;
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
//
// What reads HBM at its rate is many warps with a whole turn of 32 summaries on its
// way each, few instructions per summary, and CTAs enough on an SM that some read
// while others search.  The turns go to shared memory by cp.async with consecutive
// lanes on consecutive bytes, and are read a lane to a page.  (256 tokens of 8 kv
// heads of 128, 256 to 1024 pages each, one CTA per list: 68 us, 5.2 TB/s; 1024
// tokens of 640 pages 230 us, 6.2 TB/s.  With the words in registers, four lanes to
// a page, 77 and 305 us; with the pages' places computed for every 16 bytes 79 us;
// with two turns on their way, and so half the CTAs, 115 and 396 us; CTAs of 64, 96
// and 256 threads 71, 67 and 88 us, and a hybrid step's selection, where a chunk's
// units take longest, 40, 35 and 33 us against 28; clusters of two 102 us.)
// A single unit waits for its chain: metadata, entries, summaries, then five or six
// barriers of the cluster (6247 pages, 8 kv heads: 13 us; 63 us before every lane
// fetched another CTA's counts).
constexpr int kSelThreads = 128, kWideThreads = 256;
constexpr int kDigits = 256;
constexpr int kMaxCluster = 8;  // (portable)

struct SelectArgs {
  const void *q;
  const unsigned char *summaries;
  const int32_t *table, *starts, *lens;
  int num_seqs, num_tokens, max_pages, Hkv, G, log_g;
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
  constexpr int CH = ROW_BYTES / 16;
  // room for 32 summaries for every warp, then the keys [capacity]
  extern __shared__ uint4 sm_select[];
  uint32_t *keys = reinterpret_cast<uint32_t *>(sm_select + WARPS * 32 * CH);
  __shared__ int s_sums[2 * D];
  __shared__ __align__(16) int8_t s_codes[WARPS][2 * D];
  __shared__ int s_red[WARPS][3];
  // (once the scores are there, in the summaries' place)
  int(*s_hist)[kDigits] = reinterpret_cast<int(*)[kDigits]>(sm_select), *s_all = s_hist[4];
  __shared__ uint32_t s_range[3];  // this CTA's ordinary keys: least, largest; its top keys
  __shared__ int s_more[2];        // this CTA's keys above the threshold, and at it
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  // the kv heads of a unit side by side: their rows of a page are neighbours in memory
  const int number = blockIdx.x / nc, g = (gridDim.x / nc - 1 - number) % a.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto sync = [&] { if (nc > 1) cluster.sync(); else __syncthreads(); };

  // The unit.  Number c < num_seqs is the first of sequence c; number num_seqs + m
  // a later one whose first token is among TU w .. TU w + TU - 1, w = m + 1: at most
  // one is, and its sequence holds token TU w - 1.
  // (The last numbers first: units of chunks take longer.)
  const int TU = kUnitRows / a.G, c = (gridDim.x / nc - 1 - number) / a.Hkv;
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

  // The CTA scores pages j0 .. j1 - 1, a warp 32 at a time; their entries are looked
  // up one turn ahead.
  const int per = (limit + nc - 1) / nc;  // (limit <= max_pages: at most the capacity)
  const int j0 = min(limit, rank * per), j1 = min(limit, j0 + per);
  const int32_t *bt = a.table + (int64_t)s * a.max_pages;
  auto look_up = [&](int j) {
    if (j + lane >= j1) return -1;
    const int entry = __ldg(bt + j + lane);
    if (entry >= 0 && entry < a.num_pages) return entry;
    if (a.status) atomicOr(a.status, STATUS_BAD_PAGE);
    return -1;
  };
  uint4 *mine32 = sm_select + warp * 32 * CH;  // the warp's 32 summaries
  // 32 summaries on their way: the codes of 32 / CL of them at a time, consecutive
  // lanes taking consecutive 16 bytes, then a scale for each lane
  constexpr int CL = CH - 1;
  auto fetch = [&](int entry) {
    const unsigned char *from = a.summaries + (lane % CL) * 16;
    uint4 *to = mine32 + lane / CL * CH + lane % CL;
    const int mine = entry < 0 ? -1 : entry * a.Hkv + g;  // (at most num_pages Hkv - 1, see the host's checks)
#pragma unroll
    for (int i = 0; i < CL; ++i) {
      const int row = __shfl_sync(0xffffffffu, mine, i * (32 / CL) + lane / CL);
      ptx::cp_async16(to + i * (32 / CL) * CH, from + (int64_t)max(row, 0) * ROW_BYTES, row < 0 ? 0 : 16);
    }
    ptx::cp_async16(mine32 + lane * CH + CL, a.summaries + (int64_t)max(mine, 0) * ROW_BYTES + 2 * D, mine < 0 ? 0 : 16);
    ptx::cp_async_commit();
  };
  int entry = look_up(j0 + warp * 32), next = look_up(j0 + warp * 32 + THREADS);
  fetch(entry);

  // The unit's rows as whole numbers: the largest magnitude, then the sums, then
  // seven bits of each by the same shift.  A short last unit's last token counts for
  // the tokens that it lacks, as the operator is defined; that gives it more than its
  // share (36 tokens of 4 heads of N(0, 1): 6 to 8 of 32 pages differ from the sum
  // over the rows).
  constexpr int QL = D / QN;  // 16-byte words of a query; a lane's stand at the same dims
  static_assert(QL <= 32, "a row fits a warp");
  const int rows = tokens << a.log_g;
  const float last_weight = first > 0 ? (float)(1 + TU - tokens) : 1.f;
  auto load = [&](int row) {  // (zeros past the last one)
    if (row >= rows) return make_uint4(0u, 0u, 0u, 0u);
    const int64_t head = ((int64_t)(t0 + (row >> a.log_g)) * a.Hkv + g << a.log_g) + (row & (a.G - 1));
    return __ldg(reinterpret_cast<const uint4 *>(static_cast<const unsigned char *>(a.q) + head * (D * QB)) + lane % QL);
  };
  // The largest magnitude of the words seen, word by word, NaN where there was one.
  uint32_t high[4] = {0u, 0u, 0u, 0u};
  auto raise = [&](const uint4 &x) {
    constexpr uint32_t kMagnitude = QT == KEYS_F32 ? 0x7fffffffu : 0x7fff7fffu;
    high[0] = larger<QT>(high[0], x.x & kMagnitude);
    high[1] = larger<QT>(high[1], x.y & kMagnitude);
    high[2] = larger<QT>(high[2], x.z & kMagnitude);
    high[3] = larger<QT>(high[3], x.w & kMagnitude);
  };
  auto highest = [&](bool &fine) {  // over the warp
    float f[QN], most = 0.f;
    widen<QT>(make_uint4(high[0], high[1], high[2], high[3]), f);
    fine = true;
#pragma unroll
    for (int e = 0; e < QN; ++e) {
      fine &= f[e] < INFINITY;
      most = fmaxf(most, f[e]);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    fine = __all_sync(0xffffffffu, fine);
    return most;
  };
  // Sums of the whole numbers and of their magnitudes, in fp32: at most 127 * 256
  // rows, exact.  (Rounding to a whole number by adding 1.5 * 2^23.)
  float sum[QN] = {}, size[QN] = {};
  auto add = [&](const uint4 &x, float factor, float weight) {
    constexpr float kRound = 12582912.f;
    float f[QN];
    widen<QT>(x, f);
#pragma unroll
    for (int e = 0; e < QN; ++e) {
      const float c = __fadd_rn(__fadd_rn(__fmul_rn(f[e], factor), kRound), -kRound);
      sum[e] = fmaf(c, weight, sum[e]);
      size[e] = fmaf(fabsf(c), weight, size[e]);
    }
  };
  int up[QN], down[QN];
  auto join_lanes = [&] {  // those of a warp at the same dims
#pragma unroll
    for (int e = 0; e < QN; ++e) {
#pragma unroll
      for (int o = QL; o < 32; o <<= 1) {
        sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], o);
        size[e] += __shfl_xor_sync(0xffffffffu, size[e], o);
      }
      up[e] = (int)(0.5f * (size[e] + sum[e]));
      down[e] = (int)(0.5f * (size[e] - sum[e]));
    }
  };
  if (tokens == 1) {
    // a single token: every warp for itself, nothing to wait for
    constexpr int MOST = 8 * QL / 32;  // rows of a lane: 8 heads at most
    uint4 x[MOST];
#pragma unroll
    for (int i = 0; i < MOST; ++i) x[i] = load(i * (32 / QL) + lane / QL);
#pragma unroll
    for (int i = 0; i < MOST; ++i) raise(x[i]);
    bool fine;
    const float most = highest(fine), factor = whole_factor(most, fine);
    if (factor != 0.f) {  // (0: all codes 0, whatever the queries hold)
#pragma unroll
      for (int i = 0; i < MOST; ++i) add(x[i], factor, last_weight);
    }
    join_lanes();
  } else {
    constexpr int STEP = THREADS / QL;  // rows of the CTA at a time
    const int row0 = warp * (32 / QL) + lane / QL;
#pragma unroll 4
    for (int row = row0; row < rows; row += STEP) raise(load(row));
    bool fine;
    float most = highest(fine);
    if (lane == 0) s_red[warp][0] = __float_as_int(most);
    for (int i = tid; i < 2 * D; i += THREADS) s_sums[i] = 0;
    fine = __syncthreads_and(fine);
    for (int w = 0; w < WARPS; ++w) most = fmaxf(most, __int_as_float(s_red[w][0]));
    const float factor = whole_factor(most, fine);
    if (factor != 0.f) {
#pragma unroll 4
      for (int row = row0; row < rows; row += STEP)
        add(load(row), factor, row >> a.log_g == tokens - 1 ? last_weight : 1.f);
    }
    join_lanes();
    if (lane < QL) {
#pragma unroll
      for (int e = 0; e < QN; ++e) {
        atomicAdd(s_sums + lane * QN + e, up[e]);
        atomicAdd(s_sums + D + lane * QN + e, down[e]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < QN; ++e) {
      up[e] = s_sums[lane % QL * QN + e];
      down[e] = s_sums[D + lane % QL * QN + e];
    }
  }
  int8_t *codes = s_codes[warp];
  {
    int top = 0;
#pragma unroll
    for (int e = 0; e < QN; ++e) top = max(top, max(up[e], down[e]));
    top = __reduce_max_sync(0xffffffffu, top);
    const int shift = max(0, 25 - __clz(top)), half = (1 << shift) >> 1;
    if (lane < QL) {
#pragma unroll
      for (int e = 0; e < QN; ++e) {
        codes[lane * QN + e] = (int8_t)min((up[e] + half) >> shift, 127);
        codes[D + lane * QN + e] = (int8_t)-min((down[e] + half) >> shift, 127);
      }
    }
    __syncwarp();
  }

  // The scores, a lane to a page (its 16-byte words 4 banks from the next lane's).
  uint32_t least = 0xffffffffu, largest = 0u;
  int tops = 0;
  for (int j = j0 + warp * 32; j < j1; j += THREADS) {
    ptx::cp_async_wait<0>();
    __syncwarp();
    const uint4 *row = mine32 + lane * CH;
    int sum[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < CH - 1; ++i) {
      const uint4 x = row[i], q = reinterpret_cast<const uint4 *>(codes)[i];
      sum[0] = __dp4a((int)x.x, (int)q.x, sum[0]);
      sum[1] = __dp4a((int)x.y, (int)q.y, sum[1]);
      sum[0] = __dp4a((int)x.z, (int)q.z, sum[0]);
      sum[1] = __dp4a((int)x.w, (int)q.w, sum[1]);
    }
    const float scale = __uint_as_float(row[CH - 1].x);
    const int page = j + lane;
    if (page < j1) {
      uint32_t key = scale < INFINITY ? order_key(__fmul_rn(scale, (float)(sum[0] + sum[1]))) : kTopKey;
      if (page < a.sink_pages) key = kTopKey;
      if (entry < 0) key = 0u;
      keys[page - j0] = key;
      if (key == kTopKey) {
        ++tops;
      } else {
        least = min(least, key);
        largest = max(largest, key);
      }
    }
    __syncwarp();
    entry = next;
    if (j + THREADS < j1) {
      fetch(entry);
      next = look_up(j + 2 * THREADS);
    }
  }
  least = __reduce_min_sync(0xffffffffu, least);
  largest = __reduce_max_sync(0xffffffffu, largest);
  tops = __reduce_add_sync(0xffffffffu, tops);
  // (a warp without a page has not waited for its fetch of zeros; the counts take
  // the summaries' place)
  ptx::cp_async_wait<0>();
  __syncthreads();  // (s_red and the summaries have been read)
  for (int i = tid; i < 4 * kDigits; i += THREADS) s_hist[0][i] = 0;
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
    // (a lane to a CTA: one round trip)
    const uint32_t *r = cluster.map_shared_rank(s_range, min(lane, nc - 1));
    least = __reduce_min_sync(0xffffffffu, r[0]);
    largest = __reduce_max_sync(0xffffffffu, r[1]);
    tops = __reduce_add_sync(0xffffffffu, lane < nc ? (int)r[2] : 0);
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
    const int *more = cluster.map_shared_rank(s_more, min(lane, nc - 1));
    above += __reduce_add_sync(0xffffffffu, lane < rank ? more[0] : 0);
    at += __reduce_add_sync(0xffffffffu, lane < rank ? more[1] : 0);
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
  // (16 KB of shared memory at most: 4097 words)
  const size_t smem = sizeof(int) * ((size_t)a.num_seqs + 1);
  // as many CTAs as are resident at once
  static PerDevice ctas;
  const int resident = std::max(1, ctas.get(current_device(), [] {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, summarise_kernel<KT, D>, kSumThreads, 0) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    return n;
  }));
  summarise_kernel<KT, D><<<resident * sms, kSumThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

// CTAs of the selection's kernel resident on an SM of the current device, each with
// this much shared memory of its own choice: what registers and the kernel's own
// shared memory allow, found once, and what the shared memory does.
template <int QT, int D, int THREADS>
int64_t select_resident(int smem) {
  constexpr int kSm = 228 * 1024, kOwn = 5 * 1024;  // an SM's; a CTA's static part and the system's 1 KB
  static PerDevice ctas;
  const int most = std::max(1, ctas.get(current_device(), [] {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, select_kernel<QT, D, THREADS>, THREADS, 0) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    return n;
  }));
  return std::max(1, std::min(most, kSm / (smem + kOwn)));
}

constexpr int kMaxScores = 32 * 1024;  // of a CTA: 128 KB
constexpr int kSharedLimit = 216 * 1024;  // beside the static part

template <int QT, int D, int THREADS>
cudaError_t launch_select_on(SelectArgs a, int64_t units, int sms, cudaStream_t stream) {
  constexpr int room = THREADS * (2 * D + 16);  // for the summaries
  static_assert(room >= 5 * kDigits * 4, "the counts fit in the summaries' place");
  const int device = current_device();
  static PerDevice configured;
  cudaError_t e = cudaSuccess;
  if (configured.get(device, [&] {
        e = cudaFuncSetAttribute(select_kernel<QT, D, THREADS>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedLimit);
        return e == cudaSuccess ? 1 : 0;
      }) < 1)
    return e;
  // CTAs per (unit, kv head): the number with the fewest rounds of resident CTAs,
  // counted in a warp's turns of 32 pages, all else costing about ten.  The host
  // knows no context: all of this goes by the table's columns (256 tokens of 256 to
  // 1024 pages in 1025 / 8192 / 65536 columns: 68 / 98 / 377 us)
  int nc = 0;
  int64_t least = INT64_MAX;
  for (int n = 1; n <= kMaxCluster; n *= 2) {
    const int per = (a.max_pages + n - 1) / n;
    if (per > kMaxScores || room + per * 4 > kSharedLimit) continue;
    const int64_t slots = select_resident<QT, D, THREADS>(room + per * 4) * sms;
    const int64_t cost = (units * a.Hkv * n + slots - 1) / slots * ((per + THREADS - 1) / THREADS + 10);
    if (cost < least) {
      least = cost;
      nc = n;
    }
  }
  if (units * a.Hkv * nc > INT32_MAX) return cudaErrorInvalidConfiguration;
  a.capacity = (a.max_pages + nc - 1) / nc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * a.Hkv * nc));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = room + (size_t)a.capacity * 4;
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
  const bool few = units * a.Hkv * kMaxCluster <= sms &&
                   kWideThreads * (2 * D + 16) + (a.max_pages + kMaxCluster - 1) / kMaxCluster * 4 <= kSharedLimit;
  return few ? launch_select_on<QT, D, kWideThreads>(a, units, sms, stream)
             : launch_select_on<QT, D, kSelThreads>(a, units, sms, stream);
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
  if ((int64_t)num_seqs * desc->max_pages_per_seq > INT32_MAX) return CPA_ERR_UNSUPPORTED;
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
  if (desc->max_pages_per_seq > kMaxCluster * kMaxScores || desc->num_pages * desc->num_kv_heads > INT32_MAX)
    return CPA_ERR_UNSUPPORTED;
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
  a.log_g = a.G == 1 ? 0 : a.G == 2 ? 1 : a.G == 4 ? 2 : 3;  // (check_shape: no others)
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
