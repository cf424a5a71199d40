// Page operators of the paged cache: copy, fork, extend, release, compact.
//
// State, all on the device and owned by the caller: block_table (int32, one row
// per sequence, -1 where a row holds no page), seq_lens, and page_refs[page],
// the number of block_table entries that hold the page; 0 means free.  There is
// no free list: a page is free when nothing refers to it, and new pages are the
// lowest free ones, so that the state after a call depends on the state before
// it alone, never on the order in which blocks run (references are added and
// dropped by integer atomics, whose order changes nothing).
//
// The table operators touch a few words per page and are bound by latency: a
// launch, and the chain of dependent loads in it.  The copies move whole pages
// and are bound by HBM.
#include <algorithm>

#include <cooperative_groups.h>

#include "cpa_internal.cuh"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace cpa {
namespace {

constexpr int kPageTokens = 16;

__device__ __forceinline__ int div_up(int a, int b) { return (a + b - 1) / b; }

// These calls come one after another on a stream, each waiting for the one
// before, and most are shorter than a launch: they are launched with
// programmatic serialisation, let the next one in at once, and wait for the one
// before (its writes visible) before they read or write anything.  What they
// read, another may be writing until then: no load takes the read-only path.  A copy, which
// fills the SMs, lets the next one in when it ends.  (Release,
// release, compact and copy on 96 rows 98.7 -> 95.4 us, on 6 rows 15.2 -> 12.1 us.)
__device__ __forceinline__ void chain() {
  ptx::grid_launch_dependents();
  ptx::grid_dependency_wait();
}

__device__ __forceinline__ int ld32(const int32_t *p) {
  int x;
  asm volatile("ld.global.ca.s32 %0, [%1];" : "=r"(x) : "l"(p) : "memory");
  return x;
}

// kernel<<<grid, threads, smem, stream>>>(args...), in clusters along x, so.
template <class... Params, class... Args>
int launch_chained(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                   int cluster, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...) == cudaSuccess ? CPA_OK : CPA_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// Copies.  The 16-byte words of all pairs' K and V pages are numbered through
// (pair, then K or V, then the word within the page); a block takes 1024
// consecutive words at a time, four per thread, all four loads before the
// stores.
constexpr int kCopyThreads = 256, kCopyWords = 4;

__global__ void __launch_bounds__(kCopyThreads)
copy_pages_kernel(const int32_t *__restrict__ src, const int32_t *__restrict__ dst,
                  const int32_t *__restrict__ num_pairs, int max_pairs, uint4 *k_cache,
                  uint4 *v_cache, int page_words, int64_t num_pages, uint32_t *status) {
  ptx::grid_dependency_wait();
  int n = max_pairs;
  if (num_pairs) n = min(max(ld32(num_pairs), 0), max_pairs);
  const int pair_words = 2 * page_words;
  const int64_t total = (int64_t)n * pair_words;
  constexpr int kStep = kCopyThreads * kCopyWords;
  for (int64_t base = (int64_t)blockIdx.x * kStep; base < total; base += (int64_t)gridDim.x * kStep) {
    const int64_t pair0 = base / pair_words;
    const int in0 = (int)(base - pair0 * pair_words);
    uint4 x[kCopyWords];
    uint4 *to[kCopyWords];
#pragma unroll
    for (int i = 0; i < kCopyWords; ++i) {
      const int in = in0 + i * kCopyThreads + (int)threadIdx.x;
      const int64_t pair = pair0 + in / pair_words;
      int word = in % pair_words;
      to[i] = nullptr;
      if (pair >= n) continue;
      const int a = ld32(src + pair), b = ld32(dst + pair);
      if (a < 0 || a >= num_pages || b < 0 || b >= num_pages) {
        if (word == 0 && status) atomicOr(status, STATUS_BAD_PAGE);
        continue;
      }
      uint4 *cache = k_cache;
      if (word >= page_words) {
        cache = v_cache;
        word -= page_words;
      }
      x[i] = cache[(int64_t)a * page_words + word];
      to[i] = cache + (int64_t)b * page_words + word;
    }
#pragma unroll
    for (int i = 0; i < kCopyWords; ++i)
      if (to[i]) *to[i] = x[i];
  }
}

// ---------------------------------------------------------------------------
// Fork: one block per (parent, child).
constexpr int kRowThreads = 256;

__global__ void __launch_bounds__(kRowThreads)
fork_kernel(const int32_t *__restrict__ parents, const int32_t *__restrict__ children, int n,
            int32_t *table, int max_pages, int32_t *seq_lens, int num_rows, int32_t *refs,
            int64_t num_pages, uint32_t *status) {
  chain();
  const int i = blockIdx.x, tid = threadIdx.x;
  const int parent = ld32(parents + i), child = ld32(children + i);
  int bad = parent < 0 || parent >= num_rows || child < 0 || child >= num_rows;
  if (!bad) {
    // the child is no other fork's child and nobody's parent, and holds nothing:
    // its row is then this block's alone
    for (int j = tid; j < n; j += kRowThreads)
      bad |= (j != i && ld32(children + j) == child) || ld32(parents + j) == child;
    const int32_t *row = table + (int64_t)child * max_pages;
    for (int c = tid; c < max_pages; c += kRowThreads) bad |= row[c] >= 0;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) atomicOr(status, STATUS_BAD_ROW);
    return;
  }
  const int32_t *from = table + (int64_t)parent * max_pages;
  int32_t *to = table + (int64_t)child * max_pages;
  for (int c = tid; c < max_pages; c += kRowThreads) {
    const int page = from[c];
    if (page >= num_pages) {
      atomicOr(status, STATUS_BAD_PAGE);
    } else if (page >= 0) {
      to[c] = page;
      atomicAdd(refs + page, 1);
    }
  }
  if (tid == 0) seq_lens[child] = seq_lens[parent];
}

// ---------------------------------------------------------------------------
// Release: blockIdx.x is the row's place in the list, blockIdx.y a run of its
// columns.
constexpr int kReleaseCols = 4 * kRowThreads;

__global__ void __launch_bounds__(kRowThreads)
release_kernel(const int32_t *__restrict__ rows, int32_t *table, int max_pages, int32_t *seq_lens,
               int num_rows, int window, int sinks, int32_t *refs, int64_t num_pages,
               uint32_t *status) {
  chain();
  const int row = rows ? ld32(rows + blockIdx.x) : (int)blockIdx.x;
  if (row < 0 || row >= num_rows) {
    if (threadIdx.x == 0) atomicOr(status, STATUS_BAD_ROW);
    return;
  }
  int c0 = 0, c1 = max_pages;
  if (window > 0) {
    // the next query, at position seq_lens[row], sees j < sinks and j > len - window
    const int len = min(max(seq_lens[row], 0), max_pages * kPageTokens);
    c0 = div_up(sinks, kPageTokens);
    c1 = max(0, len - window + 1) / kPageTokens;
  } else if (blockIdx.y == 0 && threadIdx.x == 0) {
    seq_lens[row] = 0;
  }
  const int first = blockIdx.y * kReleaseCols;
  c1 = min(c1, first + kReleaseCols);
  for (int c = max(c0, first) + (int)threadIdx.x; c < c1; c += kRowThreads) {
    int32_t *at = table + (int64_t)row * max_pages + c;
    if (*at < 0) continue;
    // (exchanged, so that a row named twice gives its pages back once)
    const int page = atomicExch(at, -1);
    if (page < 0) continue;
    if (page >= num_pages) {
      atomicOr(status, STATUS_BAD_PAGE);
    } else if (atomicSub(refs + page, 1) <= 0) {
      atomicAdd(refs + page, 1);  // the table held a page that counted as free
      atomicOr(status, STATUS_BAD_PAGE);
    }
  }
}

// ---------------------------------------------------------------------------
// Extend: one cluster.  Every CTA works out every row's needs (a few loads per
// row), the free pages are searched in turns of 16 pages per thread of the
// cluster, and then rows and tokens are shared out.
constexpr int kExtThreads = 1024;
constexpr int kExtPages = 16;  // pages per thread and turn of the search

// Exclusive sum over the block; `total` on every thread.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t *warps, int64_t &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int64_t in = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, in, o);
    if (lane >= o) in += y;
  }
  __syncthreads();
  if (lane == 31) warps[warp] = in;
  __syncthreads();
  int64_t w = lane < nw ? warps[lane] : 0, wi = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, wi, o);
    if (lane >= o) wi += y;
  }
  total = __shfl_sync(0xffffffffu, wi, 31);
  const int64_t before = __shfl_sync(0xffffffffu, wi - w, warp);
  return before + in - x;
}

struct ExtendArgs {
  const int32_t *starts, *lens;
  int num_seqs;
  int64_t num_tokens;
  int32_t *table;
  int max_pages;
  int32_t *refs;
  int64_t num_pages;
  int64_t *slots;
  int32_t *copy_src, *copy_dst, *counts;
  int32_t *free_list;  // workspace [num_pages]
  uint32_t *status;
  int hash_bits;
};

// Shared memory per row: first token, first position, length, new pages (then
// their base), and the hash of shared pages (page, writers, last writer).
inline size_t extend_smem(int num_seqs, int hash_bits) {
  return sizeof(int) * (5 * (size_t)num_seqs + 1 + 3 * ((size_t)1 << hash_bits));
}

__global__ void __launch_bounds__(kExtThreads) extend_kernel(const ExtendArgs a) {
  chain();
  cg::cluster_group cluster = cg::this_cluster();
  const int nb = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, S = a.num_seqs;
  extern __shared__ int sm[];
  int *s_qs = sm, *s_len = s_qs + S + 1, *s_head = s_len + S, *s_base = s_head + S,
      *s_copy = s_base + S;  // head: the shared page the row writes to, or -1
  const int H = 1 << a.hash_bits;
  int *h_page = s_copy + S, *h_count = h_page + H, *h_last = h_count + H;
  __shared__ int64_t warps[32];
  __shared__ int found[2];  // free pages in this CTA's piece, by turn

  // the first turn's references, on their way while the rows are looked at
  const int64_t first = ((int64_t)rank * kExtThreads + tid) * kExtPages;
  const bool whole = first + kExtPages <= a.num_pages;
  int4 head_refs[kExtPages / 4];
#pragma unroll
  for (int i = 0; i < kExtPages / 4; ++i)
    head_refs[i] = whole ? *reinterpret_cast<const int4 *>(a.refs + first + 4 * i) : make_int4(1, 1, 1, 1);
  for (int i = tid; i < H; i += kExtThreads) {
    h_page[i] = -1;
    h_count[i] = 0;
    h_last[i] = -1;
  }
  __syncthreads();

  // A page without earlier tokens of the row is replaced where there is none, or
  // where another entry holds it too.  (The references stay as they were before
  // the call until every row is done.)
  auto replaced = [&](int e) { return e < 0 || (e < a.num_pages && __ldcg(a.refs + e) > 1); };

  // A1: what each row needs.  A row of at most four pages is one thread's; a
  // longer one is counted by its whole warp.
  auto slot_of = [&](int page) {  // the page's place in the hash (it is there, or inserted)
    unsigned h = (unsigned)page * 2654435761u >> (32 - a.hash_bits);
    for (;; h = (h + 1) & (H - 1)) {
      const int was = atomicCAS(h_page + h, -1, page);
      if (was == -1 || was == page) return (int)h;
    }
  };
  for (int s0 = 0; s0 < S; s0 += kExtThreads) {
    const int s = s0 + tid;
    int c0 = 0, c1 = 0, need = 0, head = -1;
    bool partial = false;  // the first page holds earlier tokens
    if (s < S) {
      const int qs = ld32(a.starts + s), q = ld32(a.starts + s + 1) - qs;
      int len = ld32(a.lens + s);
      const bool ok = qs >= 0 && q >= 0 && qs + (int64_t)q <= a.num_tokens && len >= q &&
                      len <= (int64_t)a.max_pages * kPageTokens;
      if (!ok && rank == 0) atomicOr(a.status, STATUS_BAD_ROW);
      if (!ok) len = -1;
      s_qs[s] = qs;
      if (s == S - 1) s_qs[S] = qs + max(q, 0);
      s_len[s] = len;
      if (ok && q > 0) {
        c0 = (len - q) / kPageTokens;
        c1 = (len - 1) / kPageTokens + 1;
        if ((len - q) % kPageTokens) {
          const int e = a.table[(int64_t)s * a.max_pages + c0];
          partial = true;
          need = e < 0;
          if (e >= 0 && e < a.num_pages && a.refs[e] > 1) {
            head = e;
            const int h = slot_of(e);
            atomicAdd(h_count + h, 1);
            atomicMax(h_last + h, s);
          }
        }
      }
      s_head[s] = head;
    }
    // pages of the new tokens alone: the row's first, where it writes to a page
    // that holds earlier tokens, is A2's
    if (partial) ++c0;
    const bool wide = c1 - c0 > 4;
    if (!wide)
      for (int c = c0; c < c1; ++c) need += replaced(a.table[(int64_t)s * a.max_pages + c]);
    for (unsigned m = __ballot_sync(0xffffffffu, wide); m; m &= m - 1) {
      const int l = __ffs(m) - 1;
      const int row = __shfl_sync(0xffffffffu, s, l), b = __shfl_sync(0xffffffffu, c0, l),
                e = __shfl_sync(0xffffffffu, c1, l);
      int sum = 0;
      for (int c = b + lane; c < e; c += 32) sum += replaced(a.table[(int64_t)row * a.max_pages + c]);
      sum = __reduce_add_sync(0xffffffffu, sum);
      if (lane == l) need += sum;
    }
    if (s < S) s_base[s] = need;
  }
  __syncthreads();
  // A2: a row that writes to a shared page copies it, unless it is the last
  // row to do so and every reference is a row that writes to it in this step:
  // the rows before it have then given up theirs.  s_head keeps the copies.
  for (int s = tid; s < S; s += kExtThreads) {
    const int page = s_head[s];
    if (page < 0) continue;
    const int h = slot_of(page);
    if (h_last[h] == s && h_count[h] == a.refs[page]) s_head[s] = -1;
    else s_base[s] += 1;
  }
  __syncthreads();
  // A3: exclusive sums, new pages in the low 40 bits, copies above: 4096 rows need
  // at most 2^38 pages, where their tokens overlap (a malformed step).  A row's
  // sum is kept in 32 bits: it is used where all fit into the pool.
  constexpr int kCopyShift = 40;
  constexpr int64_t kPagesMask = ((int64_t)1 << kCopyShift) - 1;
  const int per = div_up(S, kExtThreads);
  const int sa = min(S, tid * per), sb = min(S, sa + per);
  int64_t mine = 0;
  for (int s = sa; s < sb; ++s) mine += s_base[s] + ((int64_t)(s_head[s] >= 0) << kCopyShift);
  int64_t sum = 0, at = block_scan(mine, warps, sum);
  for (int s = sa; s < sb; ++s) {
    const int n = s_base[s], copy = s_head[s] >= 0;
    s_base[s] = (int)(at & kPagesMask);
    s_copy[s] = (int)(at >> kCopyShift);
    at += n + ((int64_t)copy << kCopyShift);
  }
  const int64_t needed = sum & kPagesMask;
  const int copies = (int)(sum >> kCopyShift);

  // B: the lowest free pages, in turns of 16 K pages per CTA (skipped where
  // nothing is needed)
  int64_t have = 0;
  int turn = 0;
  for (int64_t p0 = 0; p0 < a.num_pages && have < needed; p0 += (int64_t)nb * kExtThreads * kExtPages, ++turn) {
    const int64_t p = p0 + ((int64_t)rank * kExtThreads + tid) * kExtPages;
    unsigned zero = 0;
    if (p + kExtPages <= a.num_pages) {
#pragma unroll
      for (int i = 0; i < kExtPages / 4; ++i) {
        const int4 r = turn ? *reinterpret_cast<const int4 *>(a.refs + p + 4 * i) : head_refs[i];
        zero |= ((r.x == 0) | (r.y == 0) << 1 | (r.z == 0) << 2 | (r.w == 0) << 3) << (4 * i);
      }
    } else {
      for (int i = 0; i < kExtPages && p + i < a.num_pages; ++i) zero |= (a.refs[p + i] == 0) << i;
    }
    int64_t total = 0, place = block_scan(__popc(zero), warps, total);
    if (tid == 0) found[turn & 1] = (int)total;
    cluster.sync();  // (a CTA is at most one turn ahead: two places)
    int64_t all = 0;
    for (int b = 0; b < nb; ++b) {
      const int f = *cluster.map_shared_rank(found + (turn & 1), b);
      if (b < rank) place += f;
      all += f;
    }
    for (place += have; zero && place < needed; zero &= zero - 1, ++place)
      a.free_list[place] = (int)(p + __ffs(zero) - 1);
    have += all;
  }
  cluster.sync();

  // C: new entries and references, row by row over the cluster
  const bool fits = have >= needed;
  if (rank == 0 && tid == 0) {
    a.counts[0] = fits ? copies : 0;
    a.counts[1] = (int)(fits ? needed : -min(needed, (int64_t)INT32_MAX));
    if (!fits) atomicOr(a.status, STATUS_NO_PAGES);
  }
  // entry *e becomes the r-th free page; what it held is noted in its place
  auto take = [&](int32_t *e, int r) {
    const int page = __ldcg(a.free_list + r), old = *e;
    a.free_list[r] = old;
    *e = page;
    a.refs[page] = 1;
  };
  if (fits) {
    const int nt = nb * kExtThreads;
    for (int s0 = rank * kExtThreads; s0 < S; s0 += nt) {
      const int s = s0 + tid;
      int c0 = 0, c1 = 0, r = 0, old = -1;
      if (s < S && s_len[s] >= 0) {
        const int q = s_qs[s + 1] - s_qs[s], len = s_len[s];
        if (q > 0) {
          c0 = (len - q) / kPageTokens;
          c1 = (len - 1) / kPageTokens + 1;
        }
        r = s_base[s];
        old = s_head[s];
        if (old >= 0) {
          a.copy_src[s_copy[s]] = old;
          a.copy_dst[s_copy[s]] = __ldcg(a.free_list + r);
          take(a.table + (int64_t)s * a.max_pages + c0, r++);
        }
        if (q > 0 && (len - q) % kPageTokens) {
          int32_t *e = a.table + (int64_t)s * a.max_pages + c0;
          if (old < 0 && *e < 0) take(e, r++);
          ++c0;
        }
      }
      const bool wide = c1 - c0 > 4;
      if (!wide)
        for (int c = c0; c < c1; ++c) {
          int32_t *e = a.table + (int64_t)s * a.max_pages + c;
          if (replaced(*e)) take(e, r++);
        }
      for (unsigned m = __ballot_sync(0xffffffffu, wide); m; m &= m - 1) {
        const int l = __ffs(m) - 1;
        const int row = __shfl_sync(0xffffffffu, s, l), b = __shfl_sync(0xffffffffu, c0, l),
                  e = __shfl_sync(0xffffffffu, c1, l);
        int at2 = __shfl_sync(0xffffffffu, r, l);
        for (int c = b; c < e; c += 32) {
          int32_t *x = a.table + (int64_t)row * a.max_pages + c + lane;
          const bool mine2 = c + lane < e && replaced(*x);
          const unsigned who = __ballot_sync(0xffffffffu, mine2);
          if (mine2) take(x, at2 + __popc(who & ((1u << lane) - 1u)));
          at2 += __popc(who);
        }
      }
    }
  }
  cluster.sync();
  // ... and the references given up
  if (fits)
    for (int i = rank * kExtThreads + tid; i < needed; i += nb * kExtThreads) {
      const int old = __ldcg(a.free_list + i);
      if (old >= 0) atomicSub(a.refs + old, 1);
    }

  // D: the new tokens' slots
  for (int64_t t = (int64_t)rank * kExtThreads + tid; t < a.num_tokens; t += (int64_t)nb * kExtThreads) {
    int64_t slot = -1;
    if (fits && S > 0 && t < s_qs[S]) {
      int lo = 0, hi = S - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_qs[mid] <= t) lo = mid; else hi = mid - 1;
      }
      const int q = s_qs[lo + 1] - s_qs[lo], i = (int)(t - s_qs[lo]);
      if (s_len[lo] >= 0 && i >= 0 && i < q) {
        const int pos = s_len[lo] - q + i;
        const int page = a.table[(int64_t)lo * a.max_pages + pos / kPageTokens];
        if (page >= 0 && page < a.num_pages) slot = (int64_t)page * kPageTokens + pos % kPageTokens;
        else atomicOr(a.status, STATUS_BAD_PAGE);
      }
    }
    a.slots[t] = slot;
  }
}

// ---------------------------------------------------------------------------
// Compact.  With m live pages, the free pages below m take the live pages from
// m on.  Three steps: live pages counted; the places of both kinds listed; the
// references and the tables changed.  A pool of up to 128 K pages is one
// cluster's, 4 or 16 pages per thread, which does the first two steps at once, and the
// third too where the tables are small; others take a launch for each step, over
// blocks of 4096 pages.  (568 pages and 6 rows of 79 columns: three launches of
// 3.8, 7.6 and 4.5 us against one of 8.1 us; 24 584 pages and 96 rows of 259: 3.1,
// 7.8 and 5.0 us against 11.7 us.)
constexpr int kCompactThreads = 256, kCompactPages = 16;
constexpr int kCompactBlock = kCompactThreads * kCompactPages;

// Bit i: page p + i is live, i < N.
template <int N>
__device__ __forceinline__ unsigned live_bits(const int32_t *refs, int64_t p, int64_t num_pages) {
  unsigned live = 0;
  if (p + N <= num_pages) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const int4 r = *reinterpret_cast<const int4 *>(refs + p + 4 * i);
      live |= ((r.x > 0) | (r.y > 0) << 1 | (r.z > 0) << 2 | (r.w > 0) << 3) << (4 * i);
    }
  } else {
    for (int i = 0; i < N && p + i < num_pages; ++i) live |= (refs[p + i] > 0) << i;
  }
  return live;
}

__global__ void __launch_bounds__(kCompactThreads)
compact_count_kernel(const int32_t *refs, int64_t num_pages, int32_t *block_live) {
  chain();
  __shared__ int64_t warps[32];
  const int64_t p = (int64_t)blockIdx.x * kCompactBlock + threadIdx.x * kCompactPages;
  int64_t total;
  block_scan(__popc(live_bits<kCompactPages>(refs, p, num_pages)), warps, total);
  if (threadIdx.x == 0) block_live[blockIdx.x] = (int)total;
}

// Pages p .. p + N - 1, the first of which has before_p live pages before it, into
// the lists and place (see compact_place_kernel).
template <int N>
__device__ __forceinline__ void list_pages(int64_t p, unsigned live, int64_t num_pages, int64_t m,
                                           int64_t packed, int64_t before_p, int32_t *copy_src,
                                           int32_t *copy_dst, int32_t *place) {
#pragma unroll
  for (int g = 0; g < N; g += 4) {
    int at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool l = live >> (g + i) & 1u;
      const int64_t page = p + g + i;
      at[i] = l ? 0 : -1;
      if (page < num_pages) {
        if (page >= m) {
          if (l) copy_src[at[i] = (int)(before_p - packed)] = (int)page;
        } else if (!l) {
          copy_dst[page - before_p] = (int)page;
        }
      }
      before_p += l;
    }
    if (p + g + 4 <= num_pages) {
      *reinterpret_cast<int4 *>(place + p + g) = make_int4(at[0], at[1], at[2], at[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (p + g + i < num_pages) place[p + g + i] = at[i];
    }
  }
}

// Lists: the j-th free page below m (all live pages) takes the j-th live page
// from m on.  place[page]: -1 for a free page, else the j of a live page from m
// on, and 0 for a live page that stays.
__global__ void __launch_bounds__(kCompactThreads)
compact_place_kernel(const int32_t *refs, int64_t num_pages, const int32_t *block_live,
                     int32_t *copy_src, int32_t *copy_dst, int32_t *counts, int32_t *place) {
  chain();
  __shared__ int64_t warps[32];
  const int tid = threadIdx.x, nblocks = gridDim.x;
  // live pages in all, and before this block
  int64_t mine = 0, before = 0;
  for (int b = tid; b < nblocks; b += kCompactThreads) {
    const int64_t x = block_live[b];
    mine += x;
    if (b < (int)blockIdx.x) before += x;
  }
  int64_t m, base;
  block_scan(mine, warps, m);
  block_scan(before, warps, base);
  // live pages before m: the blocks before m's block, and a part of that block
  const int mb = (int)(m / kCompactBlock);
  int64_t below = 0;
  for (int b = tid; b < mb; b += kCompactThreads) below += block_live[b];
  {
    const int64_t p = (int64_t)mb * kCompactBlock + tid * kCompactPages;
    unsigned live = p < num_pages ? live_bits<kCompactPages>(refs, p, num_pages) : 0u;
    if (p + kCompactPages > m) live &= p < m ? (1u << (int)(m - p)) - 1u : 0u;
    below += __popc(live);
  }
  int64_t packed;  // live pages that stay
  block_scan(below, warps, packed);
  const int64_t p = (int64_t)blockIdx.x * kCompactBlock + tid * kCompactPages;
  const unsigned live = live_bits<kCompactPages>(refs, p, num_pages);
  int64_t total;
  int64_t before_p = base + block_scan(__popc(live), warps, total);
  list_pages<kCompactPages>(p, live, num_pages, m, packed, before_p, copy_src, copy_dst, place);
  if (blockIdx.x == 0 && tid == 0) {
    counts[0] = (int)(m - packed);
    counts[1] = (int)m;
  }
}

// References and tables, by threads first, first + stride, ...
__device__ __forceinline__ void compact_apply(int32_t *table, int64_t entries, int32_t *refs,
                                              int64_t num_pages, const int32_t *copy_src,
                                              const int32_t *copy_dst, int moves, int m,
                                              const int32_t *place, uint32_t *status, int64_t first,
                                              int64_t stride) {
  for (int64_t i = first; i < moves; i += stride) {
    const int a = __ldcg(copy_src + i), b = __ldcg(copy_dst + i);
    refs[b] = refs[a];
    refs[a] = 0;
  }
  for (int64_t i = first; i < entries; i += stride) {
    const int page = table[i];
    if (page < 0) continue;
    // (not from the references, which change meanwhile)
    const int j = page < num_pages ? __ldcg(place + page) : -1;
    if (j < 0) atomicOr(status, STATUS_BAD_PAGE);  // an entry whose page counts as free, or is none
    else if (page >= m) table[i] = __ldcg(copy_dst + j);
  }
}

__global__ void __launch_bounds__(256)
compact_apply_kernel(int32_t *table, int64_t entries, int32_t *refs, int64_t num_pages,
                     const int32_t *copy_src, const int32_t *copy_dst, const int32_t *counts,
                     const int32_t *place, uint32_t *status) {
  chain();
  compact_apply(table, entries, refs, num_pages, copy_src, copy_dst, counts[0], counts[1], place, status,
                (int64_t)blockIdx.x * blockDim.x + threadIdx.x, (int64_t)gridDim.x * blockDim.x);
}

template <int N>
__global__ void __launch_bounds__(kExtThreads)
compact_cluster_kernel(int32_t *refs, int64_t num_pages, int32_t *copy_src, int32_t *copy_dst,
                       int32_t *counts, int32_t *place, int32_t *table, int64_t entries, int apply,
                       uint32_t *status) {
  chain();
  cg::cluster_group cluster = cg::this_cluster();
  const int nb = (int)cluster.num_blocks(), rank = (int)cluster.block_rank(), tid = threadIdx.x;
  __shared__ int64_t warps[32];
  __shared__ int here[2];  // this CTA's live pages, and those of them below m
  const int64_t p = ((int64_t)rank * kExtThreads + tid) * N;
  const unsigned live = p < num_pages ? live_bits<N>(refs, p, num_pages) : 0u;
  int64_t total;
  int64_t before_p = block_scan(__popc(live), warps, total);
  if (tid == 0) here[0] = (int)total;
  cluster.sync();
  int64_t m = 0;
  for (int b = 0; b < nb; ++b) {
    const int x = *cluster.map_shared_rank(here, b);
    if (b < rank) before_p += x;
    m += x;
  }
  unsigned low = live;
  if (p + N > m) low &= p < m ? (1u << (int)(m - p)) - 1u : 0u;
  block_scan(__popc(low), warps, total);
  if (tid == 0) here[1] = (int)total;
  cluster.sync();
  int64_t packed = 0;  // live pages that stay
  for (int b = 0; b < nb; ++b) packed += *cluster.map_shared_rank(here + 1, b);
  list_pages<N>(p, live, num_pages, m, packed, before_p, copy_src, copy_dst, place);
  if (rank == 0 && tid == 0) {
    counts[0] = (int)(m - packed);
    counts[1] = (int)m;
  }
  cluster.sync();  // (the lists are written, and no CTA leaves while another reads its counts)
  if (apply)
    compact_apply(table, entries, refs, num_pages, copy_src, copy_dst, (int)(m - packed), (int)m, place,
                  status, rank * kExtThreads + tid, nb * kExtThreads);
}

// Workspace: the status word's 256 bytes, a word per page, a word per block of 4096 pages.
size_t pages_workspace(int64_t num_pages) {
  const int64_t blocks = (num_pages + kCompactBlock - 1) / kCompactBlock;
  return 256 + ((size_t)(num_pages + blocks) * 4 + 255) / 256 * 256;
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Description, table and reference checks shared by the table operators.
int check_pool(const cpa_desc *d, const void *table, int rows, const void *refs) {
  if (!d || rows < 0) return CPA_ERR_ARG;
  if (d->num_pages <= 0 || d->max_pages_per_seq <= 0 || d->page_size <= 0) return CPA_ERR_ARG;
  if (d->page_size != kPageTokens) return CPA_ERR_UNSUPPORTED;
  if (d->num_pages > INT32_MAX / kPageTokens) return CPA_ERR_UNSUPPORTED;
  if ((int64_t)d->max_pages_per_seq * kPageTokens > (1 << 30)) return CPA_ERR_UNSUPPORTED;
  if ((!table && rows > 0) || !refs || !aligned(table, 4) || !aligned(refs, 16)) return CPA_ERR_ARG;
  if (!d->workspace || !aligned(d->workspace, 256) ||
      d->workspace_bytes < pages_workspace(d->num_pages))
    return CPA_ERR_WORKSPACE;
  return CPA_OK;
}

}  // namespace
}  // namespace cpa

using namespace cpa;

extern "C" size_t cpa_pages_workspace_bytes(int64_t num_pages) {
  return num_pages <= 0 || num_pages > INT32_MAX / kPageTokens ? 0 : pages_workspace(num_pages);
}

extern "C" int cpa_copy_pages(const int32_t *src, const int32_t *dst, const int32_t *num_pairs,
                              int32_t max_pairs, void *k_cache, void *v_cache,
                              const cpa_desc *desc, void *stream) {
  const int rc = check_shape(desc);
  if (rc != CPA_OK) return rc;
  if (max_pairs < 0) return CPA_ERR_ARG;
  if (max_pairs == 0) return CPA_OK;
  if (!src || !dst || !k_cache || !v_cache || !aligned(src, 4) || !aligned(dst, 4) ||
      !aligned(num_pairs, 4) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return CPA_ERR_ARG;
  uint32_t *status = nullptr;
  if (desc->workspace) {
    if (!aligned(desc->workspace, 256) || desc->workspace_bytes < 256) return CPA_ERR_WORKSPACE;
    status = static_cast<uint32_t *>(desc->workspace);
  }
  const int eb = desc->kv_dtype == CPA_KV_E4M3 ? 1 : desc->dtype == CPA_F32 ? 4 : 2;
  const int64_t words = (int64_t)desc->num_kv_heads * kPageTokens * desc->head_dim * eb / 16;
  if (words > INT32_MAX / 4) return CPA_ERR_UNSUPPORTED;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return CPA_ERR_CUDA;
  const int sms = sm_count(dev);
  if (sms <= 0) return CPA_ERR_CUDA;
  const int64_t step = kCopyThreads * kCopyWords;
  const int64_t blocks = ((int64_t)max_pairs * 2 * words + step - 1) / step;
  return launch_chained(
      copy_pages_kernel, dim3((unsigned)std::min<int64_t>(blocks, 16 * sms)), kCopyThreads, 0, (cudaStream_t)stream, 0, src, dst, num_pairs, max_pairs, static_cast<uint4 *>(k_cache), static_cast<uint4 *>(v_cache),
      (int)words, desc->num_pages, status);
}

extern "C" int cpa_fork_sequences(const int32_t *parents, const int32_t *children,
                                  int32_t num_forks, int32_t *block_table, int32_t *seq_lens,
                                  int32_t num_rows, int32_t *page_refs, const cpa_desc *desc,
                                  void *stream) {
  const int rc = check_pool(desc, block_table, num_rows, page_refs);
  if (rc != CPA_OK) return rc;
  if (num_forks < 0 || num_forks > num_rows) return CPA_ERR_ARG;
  if (num_forks == 0) return CPA_OK;
  if (num_forks > kDecodeMaxSeqs) return CPA_ERR_UNSUPPORTED;
  if (!parents || !children || !seq_lens || !aligned(parents, 4) || !aligned(children, 4) ||
      !aligned(seq_lens, 4))
    return CPA_ERR_ARG;
  return launch_chained(
      fork_kernel, dim3(num_forks), kRowThreads, 0, (cudaStream_t)stream, 0, parents, children, num_forks, block_table, desc->max_pages_per_seq, seq_lens, num_rows,
      page_refs, desc->num_pages, static_cast<uint32_t *>(desc->workspace));
}

extern "C" int cpa_release_pages(const int32_t *rows, int32_t num_released, int32_t *block_table,
                                 int32_t *seq_lens, int32_t num_rows, int32_t window,
                                 int32_t sinks, int32_t *page_refs, const cpa_desc *desc,
                                 void *stream) {
  const int rc = check_pool(desc, block_table, num_rows, page_refs);
  if (rc != CPA_OK) return rc;
  if (num_released < 0 || window < 0 || sinks < 0) return CPA_ERR_ARG;
  if (window == 0 && sinks != 0) return CPA_ERR_ARG;
  if (!rows && num_released > num_rows) return CPA_ERR_ARG;
  if (num_released == 0) return CPA_OK;
  if (!seq_lens || !aligned(rows, 4) || !aligned(seq_lens, 4)) return CPA_ERR_ARG;
  const int64_t runs = ((int64_t)desc->max_pages_per_seq + kReleaseCols - 1) / kReleaseCols;
  if (runs > 65535) return CPA_ERR_UNSUPPORTED;
  return launch_chained(
      release_kernel, dim3(num_released, (unsigned)runs), kRowThreads, 0, (cudaStream_t)stream, 0, rows, block_table, desc->max_pages_per_seq, seq_lens, num_rows, std::min(window, 1 << 30),
      std::min(sinks, 1 << 30), page_refs, desc->num_pages,
      static_cast<uint32_t *>(desc->workspace));
}

extern "C" int cpa_extend_sequences(const int32_t *query_start_loc, const int32_t *seq_lens,
                                    int32_t num_seqs, int32_t *block_table, int32_t *page_refs,
                                    int64_t *slot_mapping, int32_t *copy_src, int32_t *copy_dst,
                                    int32_t *counts, const cpa_desc *desc, void *stream) {
  const int rc = check_pool(desc, block_table, num_seqs, page_refs);
  if (rc != CPA_OK) return rc;
  if (desc->num_tokens < 0) return CPA_ERR_ARG;
  if (num_seqs > kDecodeMaxSeqs || desc->num_tokens > INT32_MAX / 2) return CPA_ERR_UNSUPPORTED;
  if (!query_start_loc || !counts || (num_seqs > 0 && (!seq_lens || !copy_src || !copy_dst)) ||
      (!slot_mapping && desc->num_tokens > 0) || !aligned(query_start_loc, 4) ||
      !aligned(seq_lens, 4) || !aligned(copy_src, 4) || !aligned(copy_dst, 4) ||
      !aligned(counts, 4) || !aligned(slot_mapping, 8))
    return CPA_ERR_ARG;
  ExtendArgs a{};
  a.starts = query_start_loc;
  a.lens = seq_lens;
  a.num_seqs = num_seqs;
  a.num_tokens = desc->num_tokens;
  a.table = block_table;
  a.max_pages = desc->max_pages_per_seq;
  a.refs = page_refs;
  a.num_pages = desc->num_pages;
  a.slots = slot_mapping;
  a.copy_src = copy_src;
  a.copy_dst = copy_dst;
  a.counts = counts;
  a.free_list = reinterpret_cast<int32_t *>(static_cast<char *>(desc->workspace) + 256);
  a.status = static_cast<uint32_t *>(desc->workspace);
  a.hash_bits = 5;  // at least two places per row
  while ((1 << a.hash_bits) < 2 * num_seqs) ++a.hash_bits;
  const size_t smem = extend_smem(num_seqs, a.hash_bits);
  if (cudaFuncSetAttribute(extend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)extend_smem(kDecodeMaxSeqs, 13)) != cudaSuccess)
    return CPA_ERR_CUDA;
  // A CTA for every 16 K pages of the pool (one turn of the search) and every
  // 4 K tokens, at most eight, the largest portable cluster.
  const int64_t want = std::max((desc->num_pages + 16383) / 16384, (desc->num_tokens + 4095) / 4096);
  const int nb = want <= 1 ? 1 : want <= 2 ? 2 : want <= 4 ? 4 : 8;
  return launch_chained(extend_kernel, dim3(nb), kExtThreads, smem, (cudaStream_t)stream, nb, a);
}

extern "C" int cpa_compact_pages(int32_t *block_table, int32_t num_rows, int32_t *page_refs,
                                 int32_t *copy_src, int32_t *copy_dst, int32_t *counts,
                                 const cpa_desc *desc, void *stream) {
  const int rc = check_pool(desc, block_table, num_rows, page_refs);
  if (rc != CPA_OK) return rc;
  if (!counts || (desc->num_pages > 1 && (!copy_src || !copy_dst)) || !aligned(copy_src, 4) || !aligned(copy_dst, 4) ||
      !aligned(counts, 4))
    return CPA_ERR_ARG;
  int32_t *place = reinterpret_cast<int32_t *>(static_cast<char *>(desc->workspace) + 256);
  int32_t *block_live = place + desc->num_pages;
  cudaStream_t st = (cudaStream_t)stream;
  const int64_t entries = (int64_t)num_rows * desc->max_pages_per_seq;
  uint32_t *status = static_cast<uint32_t *>(desc->workspace);
  constexpr int kFew = 4;  // pages per thread of a cluster
  const bool few = desc->num_pages <= 8 * kExtThreads * kFew;
  if (few || desc->num_pages <= 8 * kExtThreads * kCompactPages) {
    int nb = 8;
    while (few && nb > 1 && desc->num_pages <= nb / 2 * kExtThreads * kFew) nb /= 2;
    // the tables here too, up to four entries per thread (a round of dependent
    // loads each; a launch of its own is as quick from there on)
    const int apply = entries <= (int64_t)nb * kExtThreads * 4;
    const int e = launch_chained(few ? compact_cluster_kernel<kFew> : compact_cluster_kernel<kCompactPages>,
                                 dim3(nb), kExtThreads, 0, st, nb, page_refs, desc->num_pages, copy_src,
                                 copy_dst, counts, place, block_table, entries, apply, status);
    if (e != CPA_OK) return e;
    if (apply) return CPA_OK;
  } else {
    const int blocks = (int)((desc->num_pages + kCompactBlock - 1) / kCompactBlock);
    int e = launch_chained(compact_count_kernel, dim3(blocks), kCompactThreads, 0, st, 0, page_refs,
                           desc->num_pages, block_live);
    if (e != CPA_OK) return e;
    e = launch_chained(compact_place_kernel, dim3(blocks), kCompactThreads, 0, st, 0, page_refs,
                       desc->num_pages, block_live, copy_src, copy_dst, counts, place);
    if (e != CPA_OK) return e;
  }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return CPA_ERR_CUDA;
  const int sms = sm_count(dev);
  if (sms <= 0) return CPA_ERR_CUDA;
  const int64_t work = std::max(entries, desc->num_pages);
  return launch_chained(compact_apply_kernel, dim3((unsigned)std::min<int64_t>((work + 255) / 256, 8 * sms)), 256,
                        0, st, 0, block_table, entries, page_refs, desc->num_pages, copy_src, copy_dst,
                        counts, place, status);
}
