// A step's packed metadata from a list of requests: what the attention calls and
// the append take, gathered from the rows of a table that holds every request.
//
// One launch.  Every CTA sums up the requests' new tokens for itself (a few words
// per request, from L2), so nothing is handed from CTA to CTA; then the table's
// rows and the tokens are shared out over the grid.  The operator is bound by a
// launch and a chain of three dependent loads.  (8 requests 3.0 us; 1024 requests
// and 19 K tokens of a 2048-column table 7.8 us, four rounds of the sum; with
// one CTA of 1024 threads on an SM 4.5 and 9.1 us.  The grid follows the rows and
// columns: 32 K tokens of one request are on one CTA, 39 us.)
#include <algorithm>

#include "cpa_internal.cuh"

namespace cpa {
namespace {

constexpr int kPageTokens = 16;
constexpr int kPackThreads = 256, kPackWarps = kPackThreads / 32;
constexpr int kPackCols = 512;  // columns of a row that a warp copies at a time

struct PackArgs {
  const int32_t *requests, *took;
  int num_requests;
  const int32_t *table, *lens;
  int num_rows, max_pages;
  int64_t num_pages, num_tokens;
  int32_t *starts, *seq_lens, *block_table, *positions;
  int64_t *slots;
  int32_t *counts;
  uint32_t *status;
};

// Shared memory per request: packed start, row, length.
inline size_t pack_smem(int num_requests) { return sizeof(int) * (3 * (size_t)num_requests + 1); }

__global__ void __launch_bounds__(kPackThreads) pack_kernel(const PackArgs a) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, R = a.num_requests;
  extern __shared__ int sm[];
  int *s_start = sm, *s_row = s_start + R + 1, *s_len = s_row + R;
  __shared__ int64_t warps[kPackWarps];
  auto raise = [&](uint32_t bit) {
    if (a.status) atomicOr(a.status, bit);
  };
  // requests with tokens so far in the upper half, their tokens in the lower one
  int64_t sum = 0;
  for (int i0 = 0; i0 < R; i0 += kPackThreads) {
    const int i = i0 + tid;
    int row = 0, q = 0, len = 0;
    if (i < R) {
      row = a.requests ? __ldg(a.requests + i) : i;
      q = __ldg(a.took + i);
      bool ok = q >= 0 && row >= 0 && row < a.num_rows;
      if (ok) {
        len = __ldg(a.lens + row);
        ok = len >= q && len <= (int64_t)a.max_pages * kPageTokens;
      }
      if (!ok) {
        if (blockIdx.x == 0) raise(STATUS_BAD_ROW);
        q = 0;
      }
    }
    const int64_t mine = q > 0 ? ((int64_t)1 << 48) + q : 0;
    int64_t in = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) in += y;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = in;
    __syncthreads();
    int64_t before = sum + in - mine;
    for (int w = 0; w < kPackWarps; ++w) {
      if (w < warp) before += warps[w];
      sum += warps[w];
    }
    if (q > 0) {
      const int at = (int)(before >> 48);
      // (starts past 2^31 are of a step that is refused below)
      s_start[at] = (int)(before & (((int64_t)1 << 48) - 1));
      s_row[at] = row;
      s_len[at] = len;
    }
  }
  const int n = (int)(sum >> 48);
  const int64_t tokens = sum & (((int64_t)1 << 48) - 1);
  if (tokens > a.num_tokens) {
    if (blockIdx.x == 0 && tid == 0) {
      a.counts[0] = 0;
      a.counts[1] = (int)-(tokens < INT32_MAX ? tokens : (int64_t)INT32_MAX);
      raise(STATUS_BAD_ROW);
    }
    return;
  }
  if (tid == 0) s_start[n] = (int)tokens;
  __syncthreads();
  const int first = blockIdx.x * kPackThreads + tid, stride = gridDim.x * kPackThreads;
  for (int i = first; i <= n; i += stride) {
    a.starts[i] = s_start[i];
    if (i < n) a.seq_lens[i] = s_len[i];
  }
  if (first == 0) {
    a.counts[0] = n;
    a.counts[1] = (int)tokens;
  }
  // the tokens' positions and slots
  for (int64_t t = first; t < tokens; t += stride) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_start[mid] <= t) lo = mid; else hi = mid - 1;
    }
    const int pos = s_len[lo] - s_start[lo + 1] + (int)t;
    const int page = __ldg(a.table + (int64_t)s_row[lo] * a.max_pages + pos / kPageTokens);
    const bool ok = page >= 0 && page < a.num_pages;
    if (!ok) raise(STATUS_BAD_PAGE);
    a.positions[t] = pos;
    a.slots[t] = ok ? (int64_t)page * kPageTokens + pos % kPageTokens : -1;
  }
  // the rows' pages
  const int runs = (a.max_pages + kPackCols - 1) / kPackCols;
  for (int64_t i = (int64_t)blockIdx.x * kPackWarps + warp; i < (int64_t)n * runs; i += (int64_t)gridDim.x * kPackWarps) {
    const int s = (int)(i / runs), c0 = (int)(i - (int64_t)s * runs) * kPackCols;
    const int c1 = min(c0 + kPackCols, (s_len[s] + kPageTokens - 1) / kPageTokens);
    const int32_t *from = a.table + (int64_t)s_row[s] * a.max_pages;
    int32_t *to = a.block_table + (int64_t)s * a.max_pages;
    for (int c = c0 + lane; c < c1; c += 32) to[c] = __ldg(from + c);
  }
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

}  // namespace
}  // namespace cpa

using namespace cpa;

extern "C" int cpa_pack_step(const int32_t *requests, const int32_t *new_tokens, int32_t num_requests,
                             const int32_t *table, const int32_t *table_lens, int32_t num_rows,
                             int32_t *query_start_loc, int32_t *seq_lens, int32_t *block_table,
                             int32_t *positions, int64_t *slot_mapping, int32_t *counts,
                             const cpa_desc *desc, void *stream) {
  if (!desc || num_requests < 0 || num_rows < 0) return CPA_ERR_ARG;
  if (desc->num_pages <= 0 || desc->max_pages_per_seq <= 0 || desc->page_size <= 0 || desc->num_tokens < 0)
    return CPA_ERR_ARG;
  if (!requests && num_requests > num_rows) return CPA_ERR_ARG;
  if (desc->page_size != kPageTokens || desc->num_pages > INT32_MAX / kPageTokens ||
      (int64_t)desc->max_pages_per_seq * kPageTokens > (1 << 30) || num_requests > kDecodeMaxSeqs ||
      desc->num_tokens > INT32_MAX / 2)
    return CPA_ERR_UNSUPPORTED;
  if (!query_start_loc || !counts || !aligned(query_start_loc, 4) || !aligned(counts, 4)) return CPA_ERR_ARG;
  if (num_requests > 0 && (!new_tokens || !table || !table_lens || !seq_lens || !block_table)) return CPA_ERR_ARG;
  if (desc->num_tokens > 0 && (!positions || !slot_mapping)) return CPA_ERR_ARG;
  if (!aligned(requests, 4) || !aligned(new_tokens, 4) || !aligned(table, 4) || !aligned(table_lens, 4) ||
      !aligned(seq_lens, 4) || !aligned(block_table, 4) || !aligned(positions, 4) || !aligned(slot_mapping, 8))
    return CPA_ERR_ARG;
  uint32_t *status = nullptr;
  if (desc->workspace) {
    if (!aligned(desc->workspace, 256) || desc->workspace_bytes < 256) return CPA_ERR_WORKSPACE;
    status = static_cast<uint32_t *>(desc->workspace);
  }
  const int device = current_device(), sms = sm_count(device);
  if (sms <= 0) return CPA_ERR_CUDA;
  static PerDevice configured;
  if (configured.get(device, [&] {
        return cudaFuncSetAttribute(pack_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)pack_smem(kDecodeMaxSeqs)) == cudaSuccess;
      }) < 1)
    return CPA_ERR_CUDA;
  const PackArgs a = {requests, new_tokens, num_requests, table, table_lens, num_rows,
                      desc->max_pages_per_seq, desc->num_pages, desc->num_tokens, query_start_loc, seq_lens,
                      block_table, positions, slot_mapping, counts, status};
  // a warp for every 512 columns of every request, two CTAs on an SM at most
  const int64_t runs = ((int64_t)desc->max_pages_per_seq + kPackCols - 1) / kPackCols;
  const int64_t ctas = std::max<int64_t>(1, (num_requests * runs + kPackWarps - 1) / kPackWarps);
  pack_kernel<<<(unsigned)std::min<int64_t>(ctas, 2 * sms), kPackThreads, pack_smem(num_requests),
                (cudaStream_t)stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? CPA_OK : CPA_ERR_CUDA;
}
