// Attention of a batch of single tokens that see a window, or selected pages, with
// 16-bit queries, or selected pages in fp32: one launch, no plan.
//
// Either way every row sees about the same number of keys and the host knows a
// bound on it, so the step kernel's queue has nothing to balance.  Work
// is split evenly instead: a cluster of CTAs per (token, kv head), its warps
// taking equal runs of the row's pages.  Per page of 16 keys a warp runs
//   S = K Q^T      m16n8k16, keys x the G heads of the group (padded to 8)
//   O^T += V^T P^T m16n8k16, dims x heads, one k-step of 16 keys
// with K and V loaded from global memory straight into the operands' registers.
// Which dim stands at which k of an MMA is free as long as Q follows, and so is
// the order of O's dims: both are chosen so that a lane's elements of a row are
// whole 16-byte words and a warp's loads whole rows.  P turns from S's layout
// (keys down the lanes) into an operand's (heads down the lanes) by movmatrix.
//
// The operator is bound by HBM: 16-row tensor instructions reach a fraction of
// the tcgen05 rate, but a page costs about 120 of a warp's instructions, and
// nothing waits: no barrier, no shared memory until the warps' states are
// joined at the end (through shared memory, then the cluster's).
//
// fp32 (KVM 3): m16n8k8 with every operand as two tf32 values (tf32_split.cuh), Q's
// halves in shared memory, P turned by shuffles.  A page is some 900 instructions,
// and as keys are the 16 rows of S and dims those of O^T, each element of K and V
// is split once.  A page's products are added up on their own and then, rounded to
// nearest, to O: the tensor cores cut off towards zero (attn_window_f32.cu).  (8 kv
// heads of 128 with 4 query heads each, 68 pages: 20 / 60 tokens 51 / 105 us, 5.0
// TB/s, and 50 / 104 us with the products added to O; on the kernel of mixed fp32
// steps, whose 16 rows a token fills with its 4, 65 / 128 us.)
#include <algorithm>

#include <cooperative_groups.h>

#include "cpa_internal.cuh"
#include "ptx.cuh"
#include "tf32_split.cuh"

namespace cg = cooperative_groups;

namespace cpa {
namespace {

constexpr int kPageKeys = 16;
constexpr int kWarps = 4;                  // of a CTA that may share its row with a cluster
constexpr int kMaxCluster = 8;            // (portable)
constexpr int kHeads = 8;                 // N of the MMAs
constexpr float kMoveThreshold = 8.0f;    // log2 units, as in the step kernel

template <bool F16>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The 8x8 matrix of 16-bit elements, two per lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// (Not the read-only path: the append launched just before may still write the
// cache when this kernel starts.)
__device__ __forceinline__ uint4 load16(const unsigned char *p) {
  uint4 x;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(p));
  return x;
}
__device__ __forceinline__ uint2 load8(const unsigned char *p) {
  uint2 x;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(x.x), "=r"(x.y) : "l"(p));
  return x;
}

// One page of K and V of one kv head as a lane holds it.  With r = lane / 4 and
// c = lane % 4: of K, rows r and r + 8, 16 bytes of each 64 (at 16 c); of V,
// rows 2c, 2c + 1, 2c + 8 and 2c + 9, the dims r D / 8 .. (r + 1) D / 8 - 1.
// (Of V in 16 bits a lane could take 16 bytes of each 128 instead, so that every
// load reads whole lines: measured 1.5 % slower.  Of V in fp32 it does.)
template <int KVM, int D>
struct PageRegs {
  static constexpr int EB = KVM == 2 ? 1 : KVM == 3 ? 4 : 2;
  static constexpr int KC = D * EB / 64;   // 16-byte words per row of K
  static constexpr int VW = D * EB / 32;   // 4-byte words per row of V: 2 .. 16
  uint32_t k[2][KC * 4];
  uint32_t v[4][VW];

  __device__ __forceinline__ void load_k(const unsigned char *kp, int r, int c) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < KC; ++i) {
        const uint4 x = load16(kp + (r + 8 * h) * (D * EB) + i * 64 + c * 16);
        k[h][4 * i] = x.x;
        k[h][4 * i + 1] = x.y;
        k[h][4 * i + 2] = x.z;
        k[h][4 * i + 3] = x.w;
      }
  }
  __device__ __forceinline__ void load_v(const unsigned char *vp, int r, int c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const unsigned char *row =
          vp + (2 * c + (j & 1) + 8 * (j >> 1)) * (D * EB) + r * (KVM == 3 ? 16 : VW * 4);
      if constexpr (VW == 2) {
        const uint2 x = load8(row);
        v[j][0] = x.x;
        v[j][1] = x.y;
      } else {
#pragma unroll
        for (int i = 0; i < VW / 4; ++i) {
          const uint4 x = load16(row + i * (KVM == 3 ? 128 : 16));
          v[j][4 * i] = x.x;
          v[j][4 * i + 1] = x.y;
          v[j][4 * i + 2] = x.z;
          v[j][4 * i + 3] = x.w;
        }
      }
    }
  }
};

template <int KVM, int D, int W, int VIS>
__global__ void __launch_bounds__(W * 32) window_decode_kernel(const AttnParams p) {
  constexpr bool F16 = KVM != 0;
  constexpr int EB = KVM == 2 ? 1 : KVM == 3 ? 4 : 2;
  constexpr int KS = D / 16;   // k-steps of S (of 8 dims in fp32: twice as many), and 16-dim tiles of O^T
  __shared__ uint2 sm_q[KVM == 3 ? 2 * KS * 64 : 1];  // fp32: [k-step][hi, lo][lane]
  using Page = PageRegs<KVM, D>;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = blockIdx.x, nc = gridDim.x, g = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const int G = p.Hq / p.Hkv;

  // blockIdx.z is the token, or the sequence in a step that has chunks too
  int t = blockIdx.z, s = t, qs, q_len;
  if (p.rows_mode == 2) {
    qs = __ldg(p.query_start_loc + s);
    q_len = __ldg(p.query_start_loc + s + 1) - qs;
    if (q_len != 1 || qs < 0 || qs >= p.num_tokens) {
      ptx::grid_dependency_wait();
      return;  // (the whole cluster)
    }
    t = qs;
  } else {
    // the token's sequence: t itself when every sequence has one token
    if (t >= p.num_seqs || __ldg(p.query_start_loc + t) != t || __ldg(p.query_start_loc + t + 1) != t + 1) {
      int lo = 0, hi = p.num_seqs - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(p.query_start_loc + mid) <= t) lo = mid; else hi = mid - 1;
      }
      s = lo;
    }
    qs = __ldg(p.query_start_loc + s);
    q_len = __ldg(p.query_start_loc + s + 1) - qs;
  }
  int ctx = __ldg(p.seq_lens + s);
  const int cap = p.max_pages * kPageKeys;
  if (ctx > cap) {
    if (threadIdx.x == 0) atomicOr(p.status, STATUS_BAD_PAGE);
    ctx = cap;
  }
  // kWindow: keys [0, near) and [far, vis); page v of the row's pages is
  // block-table column v, or v + gap behind the `front` pages of the sinks.
  // kSelected: keys [far, vis) and whole pages; the front pages are columns listed[v].
  const int vis = t - qs < q_len ? max(0, ctx - q_len + (t - qs) + 1) : 0;
  int far, near, front;
  const int32_t *listed = nullptr;
  if constexpr (VIS == kSelected) {
    const int unit = (t - qs) / (kUnitRows / G) * (kUnitRows / G);  // 0: a token of its own
    const int limit = unit_limit(p, max(0, vis - 1 - (t - qs - unit)));
    far = limit * kPageKeys;
    front = qs + unit < 0 || qs + unit >= p.num_tokens ? 0 : min(limit, p.budget);  // (0: a malformed batch)
    near = front * kPageKeys;
    listed = p.selected + ((int64_t)(qs + unit) * p.Hkv + g) * p.budget;
  } else {
    far = max(0, vis - p.window);
    near = min(p.sinks, far);
    front = (near + kPageKeys - 1) / kPageKeys;
  }
  const int gap = max(0, far / kPageKeys - front);
  const int np = (vis + kPageKeys - 1) / kPageKeys - gap;
  const int wi = rank * W + warp, nw = nc * W;
  const int v0 = (int)((int64_t)np * wi / nw), v1 = (int)((int64_t)np * (wi + 1) / nw);

  // Q as the B operand: head r, the dims that K's lanes with this c hold, in
  // the order in which the k-steps use them
  uint32_t qb[KVM == 3 ? 1 : KS][2];
  if constexpr (KVM == 3) {
    for (int i = threadIdx.x; i < 2 * KS * 32; i += W * 32) {
      const int ks = i / 32, l = i % 32, head = l >> 2;
      const int dim = (ks >> 1) * 16 + (l & 3) * 4 + (ks & 1) * 2;
      float2 x = make_float2(0.f, 0.f);
      if (head < G && vis > 0)
        x = __ldg(reinterpret_cast<const float2 *>(static_cast<const float *>(p.q) +
                                                   ((int64_t)t * p.Hq + g * G + head) * D + dim));
      uint2 hi, lo;
      split(x.x, hi.x, lo.x);
      split(x.y, hi.y, lo.y);
      sm_q[ks * 64 + l] = hi;
      sm_q[ks * 64 + 32 + l] = lo;
    }
    __syncthreads();
  } else {
    const bool have = r < G && vis > 0;
    const unsigned short *q =
        static_cast<const unsigned short *>(p.q) + ((int64_t)t * p.Hq + g * G + (r < G ? r : 0)) * D;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      // E4M3: 16 codes per 16-byte word, 4 k-steps; 16-bit: 8 elements, 2 k-steps
      const int dim = KVM == 2 ? (ks >> 2) * 64 + c * 16 + (ks & 3) * 4 : (ks >> 1) * 32 + c * 8 + (ks & 1) * 4;
      uint2 x = make_uint2(0u, 0u);
      if (have) x = __ldg(reinterpret_cast<const uint2 *>(q + dim));
      if (KVM == 2 && !p.act_f16) {
        x.x = ptx::pack_f16x2(bf16_lo(x.x), bf16_hi(x.x));
        x.y = ptx::pack_f16x2(bf16_lo(x.y), bf16_hi(x.y));
      }
      qb[ks][0] = x.x;
      qb[ks][1] = x.y;
    }
  }

  const int32_t *bt = p.block_table + (int64_t)s * p.max_pages;
  const int64_t page_bytes = (int64_t)kPageKeys * D * EB;
  const unsigned char *kc = static_cast<const unsigned char *>(p.k_cache) + g * page_bytes;
  const unsigned char *vc = static_cast<const unsigned char *>(p.v_cache) + g * page_bytes;
  // lane l holds the entry of page base + l; -1 where there is none to read
  int entry = -1;
  auto look_up = [&](int base) {
    entry = -1;
    if (base + lane < v1) {
      const int v = base + lane;
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
  auto find = [&](int v, int64_t &at) -> int {  // page v's place in the caches; its entry
    if (((v - v0) & 31) == 0) look_up(v);
    const int e = __shfl_sync(0xffffffffu, entry, (v - v0) & 31);
    at = (int64_t)max(e, 0) * p.Hkv * page_bytes;
    return e;
  };

  float o[KS][4];
#pragma unroll
  for (int i = 0; i < KS; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // heads 2c and 2c + 1
  const float sl2 = p.scale_log2;

  // Page v, held in x: S, then after_s(); softmax and O, then after_o().
  auto page = [&](Page &x, int v, int e, auto after_s, auto after_o) {
    float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
    if constexpr (KVM == 3) {
      float small[2][4] = {};  // hi lo, lo hi
#pragma unroll
      for (int ks = 0; ks < 2 * KS; ++ks) {
        const uint2 qh = sm_q[ks * 64 + lane], ql = sm_q[ks * 64 + 32 + lane];
        uint32_t h[4], l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split(__uint_as_float(x.k[e & 1][2 * ks + (e >> 1)]), h[e], l[e]);
        mma_tf32((ks & 1) ? sb : sa, h[0], h[1], h[2], h[3], qh.x, qh.y);
        mma_tf32(small[0], h[0], h[1], h[2], h[3], ql.x, ql.y);
        mma_tf32(small[1], l[0], l[1], l[2], l[3], qh.x, qh.y);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sa[e] += small[0][e] + small[1][e];
    }
#pragma unroll
    for (int ks = 0; ks < (KVM == 3 ? 0 : KS); ++ks) {
      uint32_t a[4];
      if constexpr (KVM == 2) {
        ptx::e4m3x4_to_f16x4(x.k[0][ks], a[0], a[2]);
        ptx::e4m3x4_to_f16x4(x.k[1][ks], a[1], a[3]);
      } else {
        a[0] = x.k[0][2 * ks];
        a[2] = x.k[0][2 * ks + 1];
        a[1] = x.k[1][2 * ks];
        a[3] = x.k[1][2 * ks + 1];
      }
      mma16<F16>((ks & 1) ? sb : sa, a, qb[ks][0], qb[ks][1]);
    }
    after_s();
    float sc[4];  // (key r, heads 2c, 2c + 1), (key r + 8, the same)
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[i] = (sa[i] + sb[i]) * sl2;
    // pages at the edges of what the row sees: other keys get no weight, and
    // their V, which may hold anything, becomes zero
    // (a listed page's keys are all seen: its place among the front pages stands
    // for its column)
    const int key0 = (v < front ? v : v + gap) * kPageKeys;
    if (e < 0 || key0 + kPageKeys > vis || (key0 < far && key0 + kPageKeys > near)) {
      auto seen = [&](int k) { return e >= 0 && k < vis && (k < near || k >= far); };
      if (!seen(key0 + r)) sc[0] = sc[1] = -INFINITY;
      if (!seen(key0 + r + 8)) sc[2] = sc[3] = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (!seen(key0 + 2 * c + (j & 1) + 8 * (j >> 1))) {
#pragma unroll
          for (int i = 0; i < Page::VW; ++i) x.v[j][i] = 0u;
        }
    }
    const float x0 = fmaxf(sc[0], sc[2]), x1 = fmaxf(sc[1], sc[3]);
    if (__any_sync(0xffffffffu, x0 > m0 + kMoveThreshold || x1 > m1 + kMoveThreshold)) {
      // the maximum over the page's keys: lanes of the same heads
      float y0 = x0, y1 = x1;
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) {
        y0 = fmaxf(y0, __shfl_xor_sync(0xffffffffu, y0, k));
        y1 = fmaxf(y1, __shfl_xor_sync(0xffffffffu, y1, k));
      }
      y0 = fmaxf(y0, m0);
      y1 = fmaxf(y1, m1);
      const float f0 = m0 == -INFINITY ? 0.f : ptx::ex2(m0 - y0);
      const float f1 = m1 == -INFINITY ? 0.f : ptx::ex2(m1 - y1);
      m0 = y0;
      m1 = y1;
      l0 *= f0;
      l1 *= f1;
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        o[i][0] *= f0;
        o[i][1] *= f1;
        o[i][2] *= f0;
        o[i][3] *= f1;
      }
    }
    const float r0 = m0 == -INFINITY ? 0.f : m0, r1 = m1 == -INFINITY ? 0.f : m1;
    const float p0 = ptx::ex2(sc[0] - r0), p1 = ptx::ex2(sc[1] - r1);
    const float p2 = ptx::ex2(sc[2] - r0), p3 = ptx::ex2(sc[3] - r1);
    l0 += p0 + p2;
    l1 += p1 + p3;
    if constexpr (KVM == 3) {
      // P^T as the B operand: head r, keys 2c and 2c + 1, then 8 more of each
      const int from = 8 * c + (r >> 1);
      uint32_t ph[4], pl[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float even = __shfl_sync(0xffffffffu, j < 2 ? p0 : p2, from + 4 * (j & 1));
        const float odd = __shfl_sync(0xffffffffu, j < 2 ? p1 : p3, from + 4 * (j & 1));
        split((r & 1) ? odd : even, ph[j], pl[j]);
      }
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        float t[4];
#pragma unroll
        for (int m = 0; m < 4; m += 2) {
          uint32_t h[4], l[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split(__uint_as_float(x.v[m + (e >> 1)][2 * i + (e & 1)]), h[e], l[e]);
          if (m == 0) mma_tf32_first(t, h[0], h[1], h[2], h[3], pl[m], pl[m + 1]);
          else mma_tf32(t, h[0], h[1], h[2], h[3], pl[m], pl[m + 1]);
          mma_tf32(t, l[0], l[1], l[2], l[3], ph[m], ph[m + 1]);
          mma_tf32(t, h[0], h[1], h[2], h[3], ph[m], ph[m + 1]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] += t[e];
      }
      after_o();
      return;
    }
    const uint32_t b0 = transpose8(F16 ? ptx::pack_f16x2(p0, p1) : ptx::pack_bf16x2(p0, p1));
    const uint32_t b1 = transpose8(F16 ? ptx::pack_f16x2(p2, p3) : ptx::pack_bf16x2(p2, p3));
    // O^T tile i: dims 2i and 2i + 1 of those that the lane holds (rows r and r + 8)
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      uint32_t a[4];
      if constexpr (KVM == 2) {
        const unsigned sel = (i & 1) ? 0x7362u : 0x5140u;
        ptx::e4m3x4_to_f16x4(__byte_perm(x.v[0][i >> 1], x.v[1][i >> 1], sel), a[0], a[1]);
        ptx::e4m3x4_to_f16x4(__byte_perm(x.v[2][i >> 1], x.v[3][i >> 1], sel), a[2], a[3]);
      } else {
        a[0] = __byte_perm(x.v[0][i], x.v[1][i], 0x5410);
        a[1] = __byte_perm(x.v[0][i], x.v[1][i], 0x7632);
        a[2] = __byte_perm(x.v[2][i], x.v[3][i], 0x5410);
        a[3] = __byte_perm(x.v[2][i], x.v[3][i], 0x7632);
      }
      mma16<F16>(o[i], a, b0, b1);
    }
    after_o();
  };

  // the append that may have been launched just before
  if (p.rows_mode != 2) ptx::grid_dependency_wait();
  // The next page is on its way while a page is computed.  16-bit caches: into
  // a second set of registers.  8-bit caches, whose pages are half as long:
  // K's words as soon as S has used K's registers, V's after O has used V's; the
  // registers saved hold a third more warps.  (256 and 64 tokens of 8 kv heads,
  // window 4096, head_dim 128: bf16 612 / 163 us with a second set, 619 / 206
  // without; E4M3 337 / 120 and 341 / 87 us.)  fp32: as 8-bit caches, since a second
  // set does not fit.
  if constexpr (KVM < 2) {
    auto none = [] {};
    auto fetch = [&](Page &x, int v) {
      int64_t at;
      const int e = find(v, at);
      x.load_k(kc + at, r, c);
      x.load_v(vc + at, r, c);
      return e;
    };
    if (v0 < v1) {
      Page a, b;
      int ea = fetch(a, v0), eb = -1;
      for (int v = v0; v < v1; v += 2) {
        if (v + 1 < v1) eb = fetch(b, v + 1);
        page(a, v, ea, none, none);
        if (v + 1 < v1) {
          if (v + 2 < v1) ea = fetch(a, v + 2);
          page(b, v + 1, eb, none, none);
        }
      }
    }
  } else if (v0 < v1) {
    Page x;
    int64_t at;
    int e = find(v0, at), next = -1;
    x.load_k(kc + at, r, c);
    x.load_v(vc + at, r, c);
    for (int v = v0; v < v1; ++v) {
      const bool more = v + 1 < v1;
      page(x, v, e,
           [&] {
             if (more) {
               next = find(v + 1, at);
               x.load_k(kc + at, r, c);
             }
           },
           [&] {
             if (more) x.load_v(vc + at, r, c);
           });
      e = next;
    }
  }

  // join the warps, then the cluster's CTAs
  __shared__ float sm_o[W][kHeads][D];
  __shared__ float2 sm_ml[W][kHeads];
#pragma unroll
  for (int k = 4; k < 32; k <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, k);
    l1 += __shfl_xor_sync(0xffffffffu, l1, k);
  }
  if (r == 0) {
    sm_ml[warp][2 * c] = make_float2(m0, l0);
    sm_ml[warp][2 * c + 1] = make_float2(m1, l1);
  }
#pragma unroll
  for (int i = 0; i < KS; ++i) {
    const int dim = KVM == 3 ? (i >> 1) * 32 + 4 * r + 2 * (i & 1) : r * (D / 8) + 2 * i;
    if (2 * c < G) *reinterpret_cast<float2 *>(&sm_o[warp][2 * c][dim]) = make_float2(o[i][0], o[i][2]);
    if (2 * c + 1 < G) *reinterpret_cast<float2 *>(&sm_o[warp][2 * c + 1][dim]) = make_float2(o[i][1], o[i][3]);
  }
  __syncthreads();
  // (max, sum) and sum of V of one head and dim over n states
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
  auto store = [&](int h, int d, const State &x) {
    if (vis <= 0) return;  // a malformed row: not owned, or longer than its context
    const float y = KVM == 2 ? x.O * (p.v_scale / x.L) : x.O / x.L;
    if (KVM == 3) {
      static_cast<float *>(p.out)[((int64_t)t * p.Hq + g * G + h) * D + d] = y;
      return;
    }
    const bool f16 = KVM == 1 || (KVM == 2 && p.act_f16);
    static_cast<uint16_t *>(p.out)[((int64_t)t * p.Hq + g * G + h) * D + d] =
        f16 ? __half_as_ushort(__float2half_rn(y)) : __bfloat16_as_ushort(__float2bfloat16_rn(y));
  };
  auto of_warps = [&](int h, int d) {
    return join(W, [&](int w) { return sm_ml[w][h]; }, [&](int w) { return sm_o[w][h][d]; });
  };
  if (nc == 1) {
    for (int i = threadIdx.x; i < G * D; i += W * 32) store(i / D, i % D, of_warps(i / D, i % D));
    ptx::grid_dependency_wait();
    return;
  }
  __shared__ float cl_o[kHeads][D];
  __shared__ float2 cl_ml[kHeads];
  for (int i = threadIdx.x; i < G * D; i += W * 32) {
    const State x = of_warps(i / D, i % D);
    cl_o[i / D][i % D] = x.O;
    if (i % D == 0) cl_ml[i / D] = make_float2(x.M, x.L);
  }
  cluster.sync();
  for (int i = rank * W * 32 + threadIdx.x; i < G * D; i += nc * W * 32) {
    const int h = i / D, d = i % D;
    store(h, d, join(nc, [&](int b) { return *cluster.map_shared_rank(&cl_ml[h], b); },
                     [&](int b) { return *cluster.map_shared_rank(&cl_o[h][d], b); }));
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
  // Behind a step kernel (rows_mode 2) this grid starts before that one has
  // ended, but ends after it: what comes next on the stream sees both.
  ptx::grid_dependency_wait();
}

// Pages that a row sees at most.
int64_t page_bound(const AttnParams &p) {
  if (p.vis == kSelected) return std::min<int64_t>(p.max_pages, (int64_t)p.budget + p.local_pages);
  return std::min<int64_t>(p.max_pages, (int64_t)(p.window + kPageKeys - 1) / kPageKeys + 1 +
                                            (p.sinks + kPageKeys - 1) / kPageKeys);
}

template <int KVM, int D, int W, int VIS>
int resident() {  // CTAs on an SM of the current device at a time
  static PerDevice ctas;
  return std::max(1, ctas.get(current_device(), [] {
    int n = 0;
    // The words on their way sit in L1: an SM that the step kernel has left comes
    // with nearly all of it as shared memory, and is to be set up anew.  (64
    // tokens of window 4096 beside a 480-token chunk, 8-bit cache: 192 us without
    // this hint, 151 us with it.)
    if (cudaFuncSetAttribute(window_decode_kernel<KVM, D, W, VIS>,
                             cudaFuncAttributePreferredSharedMemoryCarveout, 40) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, window_decode_kernel<KVM, D, W, VIS>, W * 32, 0) !=
            cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    return n;
  }));
}

template <int KVM, int D, int W, int VIS>
cudaError_t launch_on(const AttnParams &p, int nc, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(nc, p.Hkv, p.rows_mode == 2 ? p.num_seqs : p.num_tokens);
  cfg.blockDim = dim3(W * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = nc;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.rows_mode == 2 || p.fused ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, window_decode_kernel<KVM, D, W, VIS>, p);
}

template <int KVM, int D, int VIS>
cudaError_t launch(const AttnParams &p, int sms, cudaStream_t stream) {
  // CTAs per (token, kv head): the number with the fewest rounds of resident
  // CTAs, counted in a warp's pages, a start and a join costing about three
  const int64_t rows = (int64_t)(p.rows_mode == 2 ? p.num_seqs : p.num_tokens) * p.Hkv;
  const int64_t slots = (int64_t)resident<KVM, D, kWarps, VIS>() * sms, pages = page_bound(p);
  if constexpr (KVM == 2) {
    // Rows for more than one round, over an 8-bit cache: CTAs of two warps, since
    // starts and joins weigh more beside the shorter pages (256 tokens of 8 kv
    // heads: window 1024 97 / 90 us, 4096 339 / 320 us with four and with two warps;
    // 64 tokens, one round, 85 / 89 us).
    if (rows > slots) {
      resident<KVM, D, 2, VIS>();
      return launch_on<KVM, D, 2, VIS>(p, 1, stream);
    }
  }
  int nc = 1;
  if constexpr (VIS == kSelected) {
    // Lists are short beside a start and a join: as many CTAs as are resident at
    // once, a page for each warp at least, one CTA where there are more rows.
    // (bf16, 132 pages, 8 kv heads, tokens: 8 with 2 / 4 / 8 CTAs 20.6 / 17.0 / 22.9 us,
    // 32 with 1 / 2 / 4 46 / 53 / 63, 128 with 1 / 2 / 4 179 / 189 / 214; 8-bit cache, 68
    // pages: 8 with 4 / 8 9.5 / 9.1 us, 64 with 1 / 2 28 / 35.)
    while (nc < kMaxCluster && rows * 2 * nc <= slots && 2 * nc * kWarps <= pages) nc *= 2;
    return launch_on<KVM, D, kWarps, VIS>(p, nc, stream);
  }
  int64_t least = INT64_MAX;
  for (int n = 1; n <= kMaxCluster; n *= 2) {
    const int64_t cost = (rows * n + slots - 1) / slots * ((pages + n * kWarps - 1) / (n * kWarps) + 3);
    if (cost < least) {
      least = cost;
      nc = n;
    }
  }
  return launch_on<KVM, D, kWarps, VIS>(p, nc, stream);
}

}  // namespace

// A cluster has at most eight CTAs: few rows with a long window leave SMs idle,
// which the step kernel, whose splits have no such bound, does not.  Measured
// (one token of 8 kv heads, head_dim 128, bf16; one of 1 kv head; this kernel
// against the step kernel): window 4096 11 / 18 us and 11 / 20 us, window 16384
// 30 / 24 and 26 / 36, window 65536 104 / 60 and 100 / 70.  Where the clusters
// fill half the SMs or more (4 tokens of 8 kv heads, window 65536) 160 / 281 us.
bool window_decode_takes(const AttnParams &p, int sms) {
  const int64_t rows = (int64_t)p.num_tokens * p.Hkv;
  return rows * kMaxCluster > sms || page_bound(p) <= 32 * kMaxCluster * kWarps;
}

// Mixed steps: over an 8-bit cache the step kernel spends more on widening a
// decode's pages than HBM on reading them, and the single tokens are better
// computed here, on the SMs that the chunks leave, once they are enough to pay
// for two more launches.  Measured (this kernel beside the step kernel against
// the step kernel alone, window 1024, a 480-token chunk, 8 kv heads): 16 tokens
// 48 / 48 us, 32 tokens (111 pages per SM) 54 / 64, 64 tokens 60 / 93; window 4096
// and 16 tokens 104 / 134.  16-bit caches gain little (64 tokens 78 / 82 us) and
// lose it again on a cold start: with a window they stay in the step kernel's queue.
// Over lists, behind the selection that made them (append, summaries, selection and
// attention of a 512-token chunk beside 16 / 32 / 64 / 128 / 256 tokens with 68 pages
// each, bf16, this kernel beside against the step kernel alone): 74 / 89 / 125 / 174 /
// 283 us against 76 / 93 / 125 / 184 / 311; 16 tokens and a 128-token chunk 69 / 66.
// (Whether clusters fill the SMs is asked of all the step's tokens.  Asked of its
// sequences alone, 8-bit caches of 1 kv head, window 65536 beside 480 tokens:
// 4 tokens 242 / 293 us, 8 tokens 275 / 239 us, 16 tokens 318 / 293 us; of 2 kv
// heads, 4 tokens 391 / 484 us, 7 tokens 392 / 375 us.)
bool window_decode_beside(const AttnParams &p, int sms) {
  constexpr int kLeastPages = 96;  // per SM
  return (p.kv_e4m3 || p.vis == kSelected) && window_decode_takes(p, sms) &&
         (int64_t)p.num_seqs * p.Hkv * page_bound(p) >= (int64_t)kLeastPages * sms;
}

template <int VIS>
static cudaError_t launch_seeing(const AttnParams &p, int sms, cudaStream_t stream) {
  if constexpr (VIS == kSelected) {
    if (p.act_f32) return p.D == 128 ? launch<3, 128, VIS>(p, sms, stream) : launch<3, 64, VIS>(p, sms, stream);
  }
  if (p.D == 128) {
    if (p.kv_e4m3) return launch<2, 128, VIS>(p, sms, stream);
    return p.act_f16 ? launch<1, 128, VIS>(p, sms, stream) : launch<0, 128, VIS>(p, sms, stream);
  }
  if (p.kv_e4m3) return launch<2, 64, VIS>(p, sms, stream);
  return p.act_f16 ? launch<1, 64, VIS>(p, sms, stream) : launch<0, 64, VIS>(p, sms, stream);
}

cudaError_t launch_window_decode(const AttnParams &p, int sms, cudaStream_t stream) {
  return p.vis == kSelected ? launch_seeing<kSelected>(p, sms, stream)
                            : launch_seeing<kWindow>(p, sms, stream);
}

}  // namespace cpa
