// cache8_tree.cu — attention for trees of drafted tokens over the uniform 8-bit
// cache (include/dkv.h: dkv_cache8_tree).
#include <algorithm>

#include "cache8.cuh"
#include "dkv_kernels.cuh"
#include "dkv_tc.cuh"

namespace dkv {
namespace {

constexpr int kT8Rows = 128;        // query rows of a unit: (node, head of the group), nodes first
constexpr int kT8Walkers = 8;       // warps of a block of the second kernel
constexpr int kT8Step = 4;          // tiles of a step
constexpr int kT8Least = 2;         // steps that make a CTA worth its start
constexpr int kT8Conv = 7;          // warps that convert
constexpr int kT8Threads = 32 * (8 + kT8Conv + 1);
constexpr int kT8Stages = 5;
constexpr int kT8Stage = 32768;     // K, then V of a step in 16 bits
constexpr int kT8Descs = 64;        // ring of a converting warp
constexpr float kT8Lazy = 8.0f, kT8LazySum = 5.0f;     // how far x may pass m, y pass u
constexpr float kT8Up = 7.0f;       // log2 of a weight at its maximum

// A request of the call: N tokens stored, M drafts (0: padding).
struct TreeReq {
  int N, M, slot;
};
__device__ __forceinline__ TreeReq tree_req(const Cache8View& c, const Tree8Args& a, int i) {
  TreeReq r;
  r.M = a.n_nodes ? a.n_nodes[i] : a.max_nodes;
  r.N = max(a.seq_lens[i], 0);
  r.slot = a.slots ? a.slots[i] : i;
  int err = 0;
  if (r.M <= 0) r.M = 0;
  else if (r.M > a.max_nodes || (unsigned)r.slot >= (unsigned)c.n_slots) err = DKV_ERR_ARG;
  else if ((long long)r.N > (long long)c.width * c.T) err = DKV_ERR_TABLE_FULL;
  if (err) {
    c.latch(err, i);
    r.M = 0;
  }
  return r;
}

// The 16-token tiles of a request in order: stored ones [0, head) and [win, end) of
// which those from `full` on lie in the tail, then the drafts; `count` in all. A stored tile
// is left out if no node of any depth sees a token of it.
struct TreeTiles {
  int head, win, end, full, stored, count;
  __device__ __forceinline__ int tile(int x) const { return x < head ? x : x - head + win; }
};
__device__ __forceinline__ TreeTiles tree_tiles(int N, int M, int T, int window, int sinks) {
  TreeTiles t;
  t.end = (N + kSub - 1) / kSub;
  t.full = N / T * (T / kSub);
  t.head = t.win = 0;
  if (window > 0 && window <= N) {          // a root (position N) sees those above N - window
    const int from = N - window + 1;
    t.win = from >= N ? t.end : from / kSub;
    t.head = min((min(sinks, N) + kSub - 1) / kSub, t.win);
  }
  t.stored = t.head + t.end - t.win;
  t.count = t.stored + (M + kSub - 1) / kSub;
  return t;
}

// Which drafts a node sees (bits of 128) and its depth.
struct Node {
  uint32_t over[kMaxNodes / 32];
  int depth;
};
__device__ __forceinline__ Node node_of(const Cache8View& c, const Tree8Args& a, const int* parents, int i, int N, int m) {
  Node n;
#pragma unroll
  for (int w = 0; w < kMaxNodes / 32; w++) n.over[w] = 0;
  auto up = [&](int x) {        // x's parent
    int p = parents ? parents[x] : x - 1;
    if (p < -1 || p >= x) {
      c.latch(DKV_ERR_ARG, i);
      p = -1;
    }
    return p;
  };
  auto sees = [&](int x) {
#pragma unroll
    for (int w = 0; w < kMaxNodes / 32; w++)
      if (x >> 5 == w) n.over[w] |= 1u << (x & 31);
  };
  n.depth = 0;
  for (int x = m; (x = up(x)) >= 0;) n.depth++;
  sees(m);
  int back = 1;
  for (int x = m; (x = up(x)) >= 0; back++)
    if (a.window <= 0 || back < a.window || N + n.depth - back < a.sinks) sees(x);
  return n;
}
// bits [0, n)
__device__ __forceinline__ uint32_t below(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }
// Which of the 16 stored tokens from pos0 on a node sees, as bits.
__device__ __forceinline__ uint32_t sees_stored(const Tree8Args& a, int N, int depth, int pos0) {
  uint32_t s = below(min(N - pos0, kSub));
  if (a.window > 0) s &= ~below(N + depth + 1 - a.window - pos0) | below(a.sinks - pos0);
  return s;
}

// ---- one row by one warp, from the formula: what the products below are checked
// against, and what computes rows that come out infinite or NaN (a value that a row does
// not see may have met its weight of 0) ----
// A lane's share of a tile in the stored order, as values: K of tokens g and g + 8,
// features 16 m + 2 t + {0, 1, 8, 9}; V of features 16 m + g, + 8 and tokens 2t, 2t + 1,
// 2t + 8, 2t + 9.
template <int ELEM, int CODE>
struct Walk {
  const Cache8View& c;
  const Tree8Args& a;
  int i, h, lane;
  TreeReq r;
  TreeTiles t;

  // words of m-step m: [0], [1] row g, columns 2t and 2t + 8; [2], [3] row g + 8
  __device__ __forceinline__ void words(const uint8_t* codes, const uint8_t* tail, int op, int m, float (&v)[8]) const {
    if (codes) {
      const uint2 w = *reinterpret_cast<const uint2*>(codes + op * kTile + 512 * (m >> 1) + 16 * lane + 8 * (m & 1));
      uint32_t x[4];
      code_halves<CODE>(w.x, x[0], x[1]);
      code_halves<CODE>(w.y, x[2], x[3]);
#pragma unroll
      for (int e = 0; e < 4; e++) {
        v[2 * e] = lo_elem<DKV_F16>(x[e]);
        v[2 * e + 1] = hi_elem<DKV_F16>(x[e]);
      }
    } else {
      const uint4 w = *reinterpret_cast<const uint4*>(tail + 2 * op * kTile + 512 * m + 16 * lane);
      const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 4; e++) {
        v[2 * e] = lo_elem<ELEM>(x[e]);
        v[2 * e + 1] = hi_elem<ELEM>(x[e]);
      }
    }
  }
  // the same of drafts, of which those from n on are not read
  __device__ __forceinline__ void draft_k(int m0, int n, int m, float (&v)[8]) const {
    const int g = lane >> 2, tt = lane & 3;
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const int x = g + 8 * (e >> 1);
      uint32_t w = 0;
      if (x < n)
        w = *reinterpret_cast<const uint32_t*>(a.k + ((long long)i * a.max_nodes + m0 + x) * a.ks + h * (2 * kD) +
                                               2 * (16 * m + 2 * tt + 8 * (e & 1)));
      v[2 * e] = lo_elem<ELEM>(w);
      v[2 * e + 1] = hi_elem<ELEM>(w);
    }
  }
  __device__ __forceinline__ void draft_v(int m0, int n, int m, float (&v)[8]) const {
    const int g = lane >> 2, tt = lane & 3;
#pragma unroll
    for (int e = 0; e < 8; e++) {
      const int x = 2 * tt + (e & 1) + 8 * (e >> 1 & 1), f = 16 * m + g + 8 * (e >> 2);
      v[e] = x < n ? elem_float<ELEM>(*reinterpret_cast<const uint16_t*>(
                         a.v + ((long long)i * a.max_nodes + m0 + x) * a.vs + h * (2 * kD) + 2 * f))
                   : 0.0f;
    }
  }
  struct At {
    const uint8_t *codes, *tail;
    float2 sc;
    int m0, n;        // drafts
    uint32_t see;
  };
  __device__ __forceinline__ At at(int x, const Node& node) const {
    At p{nullptr, nullptr, make_float2(1.0f, 1.0f), 0, 0, 0};
    if (x >= t.stored) {
      p.m0 = (x - t.stored) * kSub;
      p.n = min(r.M - p.m0, kSub);
      const int w = p.m0 >> 5;
      p.see = (w == 0 ? node.over[0] : w == 1 ? node.over[1] : w == 2 ? node.over[2] : node.over[3]) >> (p.m0 & 31) & 0xffffu;
      return p;
    }
    const int tile = t.tile(x);
    p.see = sees_stored(a, r.N, node.depth, tile * kSub);
    if (tile < t.full) {
      const int per = c.T / kSub;
      int page = c.table[(size_t)r.slot * c.width + tile / per];
      if ((unsigned)page >= (unsigned)c.n_pages) {
        c.latch(DKV_ERR_CHECK, i);
        page = 0;
      }
      p.sc = *reinterpret_cast<const float2*>(c.scales + 2 * ((size_t)page * c.hkv + h));
      p.codes = c.pages + c.page_head(page, h) + (size_t)(tile % per) * (2 * kTile);
    } else {
      p.tail = c.tail + c.tail_head(r.slot, h) + (size_t)(tile - t.full) * (4 * kTile);
    }
    return p;
  }

  // base-2 logits of tokens g and g + 8 (-Inf where they are not seen); q: the lane's
  // features in the order of `words`, over a power of two that qs brings back
  __device__ __forceinline__ float2 logits(const At& p, const float (&q)[32], float qs) const {
    float x = 0.0f, y = 0.0f;
    // bf16 keys may be as large as fp32: 2^-8 of them
    constexpr float kIn = ELEM == DKV_BF16 ? 0.00390625f : 1.0f;
#pragma unroll
    for (int m = 0; m < 8; m++) {
      float v[8];
      if (p.codes || p.tail) words(p.codes, p.tail, 0, m, v);
      else draft_k(p.m0, p.n, m, v);
#pragma unroll
      for (int e = 0; e < 4; e++) {
        x = fmaf(q[4 * m + e], v[e] * kIn, x);
        y = fmaf(q[4 * m + e], v[4 + e] * kIn, y);
      }
    }
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    y += __shfl_xor_sync(0xffffffffu, y, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    y += __shfl_xor_sync(0xffffffffu, y, 2);
    const float f = p.sc.x * (1.0f / kIn) * kLogitScale * qs;
    const int g = lane >> 2;
    return make_float2(p.see >> g & 1u ? x * f : -INFINITY, p.see >> (g + 8) & 1u ? y * f : -INFINITY);
  }

  __device__ void row(int m, int g8, uint8_t* out) const {
    const int g = lane >> 2, tt = lane & 3;
    const Node node = node_of(c, a, a.parents ? a.parents + (size_t)i * a.max_nodes : nullptr, i, r.N, m);
    float q[32], am = 0.0f;
    const uint8_t* qp = a.q + ((long long)i * a.max_nodes + m) * a.qs + ((size_t)h * c.G + g8) * (2 * kD);
#pragma unroll
    for (int e = 0; e < 16; e++) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(qp + 2 * (16 * (e >> 1) + 8 * (e & 1) + 2 * tt));
      q[2 * e] = lo_elem<ELEM>(w);
      q[2 * e + 1] = hi_elem<ELEM>(w);
      am = amax_finite(amax_finite(am, q[2 * e]), q[2 * e + 1]);
    }
    float qs = 1.0f;
    if (ELEM == DKV_BF16) {
      am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
      const int ex = max(-126, min(126, (int)(__float_as_uint(am) >> 23) - 127));
      const float inv = __uint_as_float((uint32_t)(127 - ex) << 23);
      qs = __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
      for (int e = 0; e < 32; e++) q[e] *= inv;
    }
    float top = -INFINITY, l = 0.0f;
#pragma unroll 1
    for (int x = 0; x < t.count; x++) {
      const At p = at(x, node);
      if (!p.see) continue;
      const float2 y = logits(p, q, qs);
      const float now = fmaxf(top, fmaxf(y.x, y.y));
      if (now > -INFINITY) l = l * fast_exp2(top - now) + fast_exp2(y.x - now) + fast_exp2(y.y - now);
      else l += y.x + y.y == -INFINITY ? 0.0f : y.x + y.y;      // NaN
      top = now;
    }
    // the warp's maximum and sum: lanes of one t hold the tokens once
    float all = top;
#pragma unroll
    for (int d = 4; d <= 16; d <<= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, d));
    l = top == all ? l : l * fast_exp2(top - all);
#pragma unroll
    for (int d = 4; d <= 16; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    const float inv = __fdiv_rn(1.0f, l);
    float o[16];
#pragma unroll
    for (int e = 0; e < 16; e++) o[e] = 0.0f;
#pragma unroll 1
    for (int x = 0; x < t.count; x++) {
      const At p = at(x, node);
      if (!p.see) continue;
      const float2 y = logits(p, q, qs);
      const float px = fast_exp2(y.x - all) * inv, py = fast_exp2(y.y - all) * inv;
      float w[4];
      w[0] = __shfl_sync(0xffffffffu, px, 8 * tt);
      w[1] = __shfl_sync(0xffffffffu, px, 8 * tt + 4);
      w[2] = __shfl_sync(0xffffffffu, py, 8 * tt);
      w[3] = __shfl_sync(0xffffffffu, py, 8 * tt + 4);
      bool see[4];
#pragma unroll
      for (int e = 0; e < 4; e++) see[e] = p.see >> (2 * tt + (e & 1) + 8 * (e >> 1)) & 1u;
#pragma unroll
      for (int f = 0; f < 8; f++) {
        float v[8];
        if (p.codes || p.tail) words(p.codes, p.tail, 1, f, v);
        else draft_v(p.m0, p.n, f, v);
#pragma unroll
        for (int e = 0; e < 8; e++)
          if (see[e & 3]) o[2 * f + (e >> 2)] = fmaf(w[e & 3], v[e] * p.sc.y, o[2 * f + (e >> 2)]);
      }
    }
#pragma unroll
    for (int e = 0; e < 16; e++) {
      o[e] += __shfl_xor_sync(0xffffffffu, o[e], 1);
      o[e] += __shfl_xor_sync(0xffffffffu, o[e], 2);
      if (tt == (e & 3)) reinterpret_cast<uint16_t*>(out)[8 * e + g] = float_elem<ELEM>(in_range<ELEM>(o[e]));
    }
  }
};

// ---- the call's plan, the same in every block: prefix sums of the requests' steps ----
// A unit is a (request, KV head, 128 query rows); its steps of 64 tokens follow one
// another, and the units of all requests form one sequence that is cut into equal
// ranges, one a CTA.
struct TreePlan {
  int pre[kMaxCallReq + 1], N[kMaxCallReq], M[kMaxCallReq], slot[kMaxCallReq];
};
__device__ __forceinline__ int unit_rows(int M, int G) { return (M * G + kT8Rows - 1) / kT8Rows; }
__device__ __forceinline__ int make_plan(const Cache8View& c, const Tree8Args& a, TreePlan& p, int* scan) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  int carry = 0;
  for (int base = 0; base < a.n_req; base += blockDim.x) {
    const int i = base + threadIdx.x;
    int cost = 0;
    if (i < a.n_req) {
      const TreeReq r = tree_req(c, a, i);
      p.N[i] = r.N;
      p.M[i] = r.M;
      p.slot[i] = r.slot;
      if (r.M > 0) {
        const TreeTiles t = tree_tiles(r.N, r.M, c.T, a.window, a.sinks);
        cost = c.hkv * unit_rows(r.M, c.G) * ((t.count + kT8Step - 1) / kT8Step);
      }
    }
    int x = cost;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    const int sum = lane < warps ? scan[lane] : 0;
    const int before = carry + __reduce_add_sync(0xffffffffu, lane < warp ? sum : 0);
    carry += __reduce_add_sync(0xffffffffu, sum);
    if (i < a.n_req) p.pre[i] = before + x - cost;
    if (threadIdx.x == 0) p.pre[min(base + (int)blockDim.x, a.n_req)] = carry;
    __syncthreads();
  }
  return carry;
}
__device__ __forceinline__ int tree_ctas(int total, int grid) { return max(1, min(grid, (total + kT8Least - 1) / kT8Least)); }
__device__ __forceinline__ int range_start(int total, int cta, int ctas) { return (int)((long long)total * cta / ctas); }
__device__ __forceinline__ int range_of(int total, int pos, int ctas) { return (int)((((long long)pos + 1) * ctas - 1) / total); }

// Part of a unit in a CTA's range: steps s0 .. s0 + n - 1 of `per`.
struct TreeItem {
  int i, h, t, s0, n, per, N, M, slot;
  TreeTiles tiles;
};
__device__ __forceinline__ TreeItem tree_item(const Cache8View& c, const Tree8Args& a, const TreePlan& p, int pos, int hi) {
  TreeItem it;
  int i = 0, end = a.n_req;
  while (end - i > 1) {        // the last request that starts at or before pos
    const int mid = (i + end) >> 1;
    if (p.pre[mid] <= pos) i = mid; else end = mid;
  }
  it.i = i;
  it.N = p.N[i];
  it.M = p.M[i];
  it.slot = p.slot[i];
  it.tiles = tree_tiles(it.N, it.M, c.T, a.window, a.sinks);
  it.per = (it.tiles.count + kT8Step - 1) / kT8Step;
  const int x = pos - p.pre[i], unit = x / it.per, rt = unit_rows(it.M, c.G);
  it.s0 = x - unit * it.per;
  it.h = unit / rt;
  it.t = unit - it.h * rt;
  it.n = min(it.per - it.s0, hi - pos);
  return it;
}

// What a converting warp knows of one of its tiles. kind: of codes, of which every
// node sees every token (0) or not (1), of the tail (2), drafts (3), none (4).
struct TileDesc {
  const uint8_t* src;
  float ks;
  union {
    float lv;       // log2 of V's scale
    int req_head;   // kinds 2 and 3: request << 12 | KV head
  };
  int pos0, kind;   // first token, first draft
};
// What the softmax has to know of it. kind: seen by all (0), stored (1), drafts (2), none (3).
struct TileMeta {
  float ks, lv;
  int pos0, kind;
};

struct TreeSmem {
  TileDesc desc[kT8Conv][kT8Descs];
  TileMeta meta[kT8Stages][kT8Step];
  float4 ex[2][kT8Rows];       // m, u, l of the halves
  TreePlan plan;
  int parents[kMaxNodes];
  float qs[kT8Rows];
  int scan[32];
  uint64_t bar[2 * kT8Stages + 10];
  uint32_t taddr;
  int fail;
};
constexpr int kT8Smem = 1024 + kT8Stages * kT8Stage + (int)sizeof(TreeSmem);

__device__ __forceinline__ uint4 ld_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ void stmatrix4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void stmatrix4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}
__device__ __forceinline__ void loaded32(float* v) {
#pragma unroll
  for (int e = 0; e < 32; e++) asm volatile("" : "+f"(v[e]));
}
// largest finite magnitude of bf16 pairs, as bits
__device__ __forceinline__ uint32_t amax2_finite(uint32_t m, uint32_t w) {
  w &= 0x7fff7fffu;
  return __vmaxu2(m, w & ~__vcmpgeu2(w, 0x7f807f80u));
}
// exponent of the power of two that brings the largest magnitude (of a warp) to [128, 256)
__device__ __forceinline__ int scale_exp(uint32_t m) {
  const uint32_t top = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
  return max(-120, (int)(top >> 7) - (127 + 7));
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
__device__ __forceinline__ uint32_t half_of_bf16(uint32_t w, float f) {
  return pack_half2(lo_elem<DKV_BF16>(w) * f, hi_elem<DKV_BF16>(w) * f);
}

template <int ELEM, int CODE>
__global__ void __launch_bounds__(kT8Threads, 1) k_tree8(Cache8View c, Tree8Args a, int part_rows) {
  pdl_launch_dependents();
  pdl_wait();
  if (c.stopped()) return;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TreeSmem& sm = *reinterpret_cast<TreeSmem*>(smem + kT8Stages * kT8Stage);
  const int total = make_plan(c, a, sm.plan, sm.scan);
  if (total == 0) return;
  const int ctas = tree_ctas(total, gridDim.x);
  if ((int)blockIdx.x >= ctas) return;
  const int lo = range_start(total, blockIdx.x, ctas), hi = range_start(total, blockIdx.x + 1, ctas);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, G = c.G;
  // step j of the CTA: half j & 1, its step j >> 1, stage j % kT8Stages
  const uint32_t b0 = smem_u32(sm.bar);
  auto full = [&](int s) { return b0 + 8u * s; };
  auto empty = [&](int s) { return b0 + 8u * (kT8Stages + s); };
  auto sfull = [&](int h) { return b0 + 8u * (2 * kT8Stages + h); };
  auto sfree = [&](int h) { return b0 + 8u * (2 * kT8Stages + 2 + h); };
  auto pfull = [&](int h) { return b0 + 8u * (2 * kT8Stages + 4 + h); };
  auto pvdone = [&](int h) { return b0 + 8u * (2 * kT8Stages + 6 + h); };
  const uint32_t ready = b0 + 8u * (2 * kT8Stages + 8), drain = ready + 8u;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kT8Stages; s++) {
      mbar_init(full(s), kT8Step);
      mbar_init(empty(s), 1);
    }
    for (int h = 0; h < 2; h++) {
      mbar_init(sfull(h), 1);
      mbar_init(sfree(h), 4);
      mbar_init(pfull(h), 4);
      mbar_init(pvdone(h), 1);
    }
    mbar_init(ready, 8);
    mbar_init(drain, 1);
    sm.fail = 0;
    fence_mbar_init();
  }
  if (warp == 8 + kT8Conv) tmem_alloc(smem_u32(&sm.taddr), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = __shfl_sync(0xffffffffu, sm.taddr, 0);
  // O of the halves, S of the halves, P of the halves, Q
  auto t_o = [&](int h) { return tbase + 128u * h; };
  auto t_s = [&](int h) { return tbase + 256u + 64u * h; };
  auto t_p = [&](int h) { return tbase + 384u + 32u * h; };
  const uint32_t t_q = tbase + 448u;
  auto fail = [&]() {
    c.latch(DKV_ERR_TIMEOUT, -1);
    *(volatile int*)&sm.fail = 1;
  };
  auto wait = [&](uint32_t bar, int phase) {       // the same for every lane
    return __all_sync(0xffffffffu, *(volatile int*)&sm.fail == 0 && mbar_wait_bounded(bar, phase & 1)) != 0;
  };
  bool ok = true;

  if (warp < 8) {
    // ---- softmax: a thread per query row, a half takes every other step ----
    const int half = warp >> 2, lg = warp & 3, r = 32 * lg + lane;
    const uint32_t tl = (uint32_t)(32 * lg) << 16;
    Node node;
    int have_i = -1, have_t = -1;
    for (int pos = lo, j0 = 0; pos < hi;) {
      const TreeItem it = tree_item(c, a, sm.plan, pos, hi);
      const int rows = it.M * G - it.t * kT8Rows, row = it.t * kT8Rows + r, m = row / G;
      const bool real = r < rows, busy = 32 * lg < rows;
      const bool fresh = it.i != have_i || it.t != have_t;
      have_i = it.i;
      have_t = it.t;
      if (fresh && half == 1 && r < it.M && a.parents) sm.parents[r] = a.parents[(size_t)it.i * a.max_nodes + r];
      if (half == 0 && busy) {
        // the queries as fp16 (bf16: over a power of two of their row)
        uint32_t q[64];
        const uint4* src = reinterpret_cast<const uint4*>(a.q + ((long long)it.i * a.max_nodes + m) * a.qs +
                                                          ((size_t)it.h * G + (row - m * G)) * (2 * kD));
#pragma unroll
        for (int e = 0; e < 16; e++) {
          const uint4 w = real ? src[e] : make_uint4(0, 0, 0, 0);
          q[4 * e] = w.x;
          q[4 * e + 1] = w.y;
          q[4 * e + 2] = w.z;
          q[4 * e + 3] = w.w;
        }
        if (ELEM == DKV_BF16) {
          uint32_t am = 0;
#pragma unroll
          for (int e = 0; e < 64; e++) am = amax2_finite(am, q[e]);
          const int ex = max(-126, min(126, (int)(max(am & 0xffffu, am >> 16) >> 7) - 127));
          const float inv = pow2(-ex);
          sm.qs[r] = pow2(ex);
#pragma unroll
          for (int e = 0; e < 64; e++) q[e] = half_of_bf16(q[e], inv);
        }
        tmem_st32(t_q + tl, q);
        tmem_st32(t_q + tl + 32, q + 32);
        tmem_wait_st();
      }
      tc_fence_before();
      named_sync(1, 256);
      if (lane == 0) mbar_arrive(ready);
      if (fresh && real) node = node_of(c, a, a.parents ? sm.parents : nullptr, it.i, it.N, m);
      const float scale = ELEM == DKV_BF16 && real ? sm.qs[r] : 1.0f;
      float mx = -INFINITY, u = -INFINITY, l = 0.0f;
      int j = j0 + ((j0 & 1) != half), n = j >> 1;
      const int end = j0 + it.n;
      bool first = true;
      for (; ok && j < end; j += 2, n++) {
        ok = wait(sfull(half), n);
        if (!ok) break;
        float s[64];
        tc_fence_after();
        if (busy) {
          tmem_ld32_nowait(t_s(half) + tl, s);
          tmem_ld32_nowait(t_s(half) + tl + 32, s + 32);
          tmem_wait_ld();
          loaded32(s);
          loaded32(s + 32);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sfree(half));
        uint32_t p[32];
        if (busy) {
          const TileMeta* meta = sm.meta[j % kT8Stages];
          float f[4], lv[4], ym[4];
#pragma unroll
          for (int b = 0; b < 4; b++) {
            const TileMeta d = meta[b];
            f[b] = d.ks * scale;
            lv[b] = d.lv;
            if (d.kind != 0) {
              uint32_t see = 0;
              if (real && d.kind == 1) see = sees_stored(a, it.N, node.depth, d.pos0);
              if (real && d.kind == 2) {
                const int w = d.pos0 >> 5;
                see = (w == 0 ? node.over[0] : w == 1 ? node.over[1] : w == 2 ? node.over[2] : node.over[3]) >> (d.pos0 & 31);
              }
#pragma unroll
              for (int e = 0; e < 16; e++) s[16 * b + e] = see & (1u << e) ? s[16 * b + e] : -INFINITY;
            }
            float y0 = s[16 * b], y1 = s[16 * b + 1];
#pragma unroll
            for (int e = 2; e < 16; e += 2) {
              y0 = fmaxf(y0, s[16 * b + e]);
              y1 = fmaxf(y1, s[16 * b + e + 1]);
            }
            ym[b] = fmaxf(y0, y1) * f[b];
          }
          const float yt = fmaxf(fmaxf(ym[0], ym[1]), fmaxf(ym[2], ym[3]));
          const float xt = fmaxf(fmaxf(ym[0] + lv[0], ym[1] + lv[1]), fmaxf(ym[2] + lv[2], ym[3] + lv[3]));
          if (__any_sync(0xffffffffu, real && (xt > mx + kT8Lazy || yt > u + kT8LazySum))) {
            const float nm = fmaxf(mx, xt), nu = fmaxf(u, yt);
            l *= nu == -INFINITY ? 1.0f : fast_exp2(u - nu);
            if (!first) {
              ok = wait(pvdone(half), n - 1);
              if (!ok) break;
              tc_fence_after();
              const float fo = nm == -INFINITY ? 1.0f : fast_exp2(mx - nm);
#pragma unroll 1
              for (int q = 0; q < 8; q++) {
                float o[16];
                tmem_ld16_nowait(t_o(half) + tl + 16 * q, o);
                tmem_wait_ld();
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; e++) {
                  asm volatile("" : "+f"(o[e]));
                  w[e] = __float_as_uint(o[e] * fo);
                }
                tmem_st16(t_o(half) + tl + 16 * q, w);
              }
              tmem_wait_st();
            }
            mx = nm;
            u = nu;
          }
          const float ur = u == -INFINITY ? 0.0f : u, mr = mx == -INFINITY ? 0.0f : mx;
          float sum = 0.0f;
#pragma unroll
          for (int b = 0; b < 4; b++) {
            const float g = fast_exp2(fminf(ur + lv[b] - mr + kT8Up, 127.0f));
            float part = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; e++) {
              const float p0 = fast_exp2(fmaf(s[16 * b + 2 * e], f[b], -ur)), p1 = fast_exp2(fmaf(s[16 * b + 2 * e + 1], f[b], -ur));
              part += p0 + p1;
              p[8 * b + e] = pack_half2(p0 * g, p1 * g);
            }
            sum += part;
          }
          l += sum;
        }
        // P of the step before is read, and its arrivals are complete (warps without rows
        // are here early)
        if (n > 0) ok = wait(pvdone(half), n - 1);
        if (!ok) break;
        tc_fence_after();
        if (busy) {
          tmem_st32(t_p(half) + tl, p);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull(half));
        first = false;
      }
      if (ok && !first) ok = wait(pvdone(half), n - 1);
      if (!ok) fail();
      sm.ex[half][r] = make_float4(mx, u, l, first ? 0.0f : 1.0f);
      tc_fence_before();
      named_sync(2, 256);
      tc_fence_after();
      if (ok && busy) {
        // both halves' rows, 64 features by each half's warps
        const float4 e0 = sm.ex[0][r], e1 = sm.ex[1][r];
        const float top = fmaxf(e0.y, e1.y);
        auto weight = [&](const float4& e) { return e.z == 0.0f ? 0.0f : e.z * (e.y == top ? 1.0f : fast_exp2(e.y - top)); };
        const float lsum = weight(e0) + weight(e1);
        auto factor = [&](const float4& e) {
          return e.z == 0.0f ? 0.0f : __fdiv_rn(fast_exp2(e.x - kT8Up - top), lsum);
        };
        const float f0 = factor(e0), f1 = factor(e1);
        const bool whole = it.n == it.per, two0 = e0.w != 0.0f, two1 = e1.w != 0.0f;
        uint8_t* out = a.out + (((long long)it.i * a.max_nodes + m) * c.hkv * G + (size_t)it.h * G + (row - m * G)) * (2 * kD) + 128 * half;
        float* part = a.part + (size_t)(2 * blockIdx.x + (it.s0 > 0 ? 0 : 1)) * part_rows * (kD + 2);
#pragma unroll 1
        for (int q = 0; q < 4; q++) {
          float o0[16], o1[16];
          tmem_ld16_nowait(t_o(0) + tl + 64 * half + 16 * q, o0);
          tmem_ld16_nowait(t_o(1) + tl + 64 * half + 16 * q, o1);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; e++) {
            asm volatile("" : "+f"(o0[e]));
            asm volatile("" : "+f"(o1[e]));
            o0[e] = (two0 ? o0[e] * f0 : 0.0f) + (two1 ? o1[e] * f1 : 0.0f);
          }
          if (real && whole) {
            uint32_t w[8], bad = 0;
#pragma unroll
            for (int e = 0; e < 8; e++) {
              w[e] = pack_elems<ELEM>(o0[2 * e], o0[2 * e + 1]);
              find_not_finite<ELEM>(bad, w[e]);
            }
            if (__builtin_expect(found_not_finite(bad), 0)) {
#pragma unroll
              for (int e = 0; e < 8; e++) w[e] = pack_elems<ELEM>(in_range<ELEM>(o0[2 * e]), in_range<ELEM>(o0[2 * e + 1]));
            }
            reinterpret_cast<uint4*>(out)[2 * q] = make_uint4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<uint4*>(out)[2 * q + 1] = make_uint4(w[4], w[5], w[6], w[7]);
          } else if (real) {
#pragma unroll
            for (int e = 0; e < 4; e++)
              reinterpret_cast<float4*>(part + r * kD + 64 * half + 16 * q)[e] =
                  make_float4(o0[4 * e], o0[4 * e + 1], o0[4 * e + 2], o0[4 * e + 3]);
          }
        }
        if (real && !whole && half == 0) reinterpret_cast<float2*>(part + part_rows * kD)[r] = make_float2(top, lsum);
      }
      tc_fence_before();
      pos += it.n;
      j0 += it.n;
    }
  } else if (warp < 8 + kT8Conv) {
    // ---- codes, tails and drafts to 16-bit operands: the tiles of the steps are dealt
    // out to the warps in turn ----
    const int cw = warp - 8;
    const int steps = (kT8Step * (hi - lo) - cw + kT8Conv - 1) / kT8Conv;      // tiles cw, cw + kT8Conv, ..
    const int mat = lane >> 3, mrow = lane & 7, me = mat & 1, ms = mat >> 1;
    const uint32_t stage0 = smem_u32(smem);
    TileDesc* desc = sm.desc[cw];
    auto describe = [&](int batch) {       // tiles 32 batch ..: a lane each
      const int k = 32 * batch + lane;
      if (k < steps) {
        const int tile_of = cw + kT8Conv * k, pos = lo + tile_of / kT8Step;
        const TreeItem it = tree_item(c, a, sm.plan, pos, pos + 1);
        const int x = kT8Step * it.s0 + tile_of % kT8Step;
        TileDesc d{nullptr, kLogitScale, {0.0f}, 0, 4};
        if (x < it.tiles.stored) {
          const int tile = it.tiles.tile(x);
          d.pos0 = tile * kSub;
          if (tile < it.tiles.full) {
            const int per = c.T / kSub;
            int page = c.table[(size_t)it.slot * c.width + tile / per];
            if ((unsigned)page >= (unsigned)c.n_pages) {
              c.latch(DKV_ERR_CHECK, it.i);
              page = 0;
            }
            const float2 sc = *reinterpret_cast<const float2*>(c.scales + 2 * ((size_t)page * c.hkv + it.h));
            d.src = c.pages + c.page_head(page, it.h) + (size_t)(tile % per) * (2 * kTile);
            d.ks = sc.x * kLogitScale;
            d.lv = log2f(sc.y);
            // every depth sees all of it
            d.kind = a.window <= 0 || d.pos0 >= it.N + it.M - a.window || d.pos0 + kSub <= a.sinks ? 0 : 1;
          } else {
            d.src = c.tail + c.tail_head(it.slot, it.h) + (size_t)(tile - it.tiles.full) * (4 * kTile);
            d.req_head = it.i << 12 | it.h;
            d.kind = 2;
          }
        } else if (x < it.tiles.count) {
          d.pos0 = (x - it.tiles.stored) * kSub;
          d.req_head = it.i << 12 | it.h;
          d.kind = 3;
        }
        desc[k & (kT8Descs - 1)] = d;
      }
      __syncwarp();
    };
    auto fetch = [&](int k, uint4 (&w)[8]) {
      if (k >= steps) return;
      const TileDesc d = desc[k & (kT8Descs - 1)];
      if (d.kind > 1) return;
#pragma unroll
      for (int e = 0; e < 8; e++) w[e] = ld_stream(d.src + 512 * e + 16 * lane);
    };
    auto put = [&](int k, const uint4 (&w)[8]) {
      const int tile_of = cw + kT8Conv * k, j = tile_of / kT8Step, sub = tile_of % kT8Step, stage = j % kT8Stages;
      if (j >= kT8Stages) ok = wait(empty(stage), j / kT8Stages - 1);
      if (!ok) return;
      const uint32_t base = stage0 + stage * kT8Stage;
      // the lane's row of the four 8 x 8 matrices of a store: K, V, V of drafts
      const uint32_t k_off = (2 * sub + ms) * 1024 + mrow * 128 + ((me ^ mrow) << 4);
      const uint32_t v_off = 16384 + ms * 1024 + mrow * 128 + (((2 * sub + me) ^ mrow) << 4);
      const uint32_t vt_off = 16384 + me * 1024 + mrow * 128 + (((2 * sub + ms) ^ mrow) << 4);
      const TileDesc d = desc[k & (kT8Descs - 1)];
      TileMeta meta{d.ks, d.lv, d.pos0, d.kind > 2 ? d.kind - 1 : d.kind == 2 ? 1 : d.kind};
      if (d.kind <= 1) {
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const uint32_t at0 = e < 4 ? base + ((k_off + (e >> 1) * 8192) ^ ((e & 1) << 6)) : base + v_off + (e - 4) * 4096;
          const uint32_t at1 = e < 4 ? at0 ^ 32u : at0 + 2048;
          uint32_t x[4];
          code_halves<CODE>(w[e].x, x[0], x[1]);
          code_halves<CODE>(w[e].y, x[2], x[3]);
          stmatrix4(at0, x[0], x[1], x[2], x[3]);
          code_halves<CODE>(w[e].z, x[0], x[1]);
          code_halves<CODE>(w[e].w, x[2], x[3]);
          stmatrix4(at1, x[0], x[1], x[2], x[3]);
        }
      } else if (d.kind <= 3) {
        const int i = d.req_head >> 12, h = d.req_head & 4095, g = lane >> 2, t = lane & 3;
        const int n = min(d.kind == 2 ? sm.plan.N[i] - d.pos0 : sm.plan.M[i] - d.pos0, kSub);      // valid tokens
        meta.lv = 0.0f;
        uint32_t x[32];
        const long long drow = (long long)i * a.max_nodes + d.pos0;
#pragma unroll 1
        for (int op = 0; op < 2; op++) {
          if (d.kind == 2) {
            // what lies behind the request's tokens becomes 0 (0 times what it may hold is not)
            const bool v = op == 1;
            const uint32_t lo_t = v ? (2 * t < n ? 0xffffu : 0u) | (2 * t + 1 < n ? 0xffff0000u : 0u) : g < n ? 0xffffffffu : 0u;
            const uint32_t hi_t = v ? (2 * t + 8 < n ? 0xffffu : 0u) | (2 * t + 9 < n ? 0xffff0000u : 0u) : g + 8 < n ? 0xffffffffu : 0u;
#pragma unroll
            for (int f = 0; f < 8; f++) {
              const uint4 y = *reinterpret_cast<const uint4*>(d.src + 2 * op * kTile + 512 * f + 16 * lane);
              x[4 * f] = y.x & lo_t;
              x[4 * f + 1] = y.y & (v ? hi_t : lo_t);
              x[4 * f + 2] = y.z & (v ? lo_t : hi_t);
              x[4 * f + 3] = y.w & hi_t;
            }
          } else {
            const uint8_t* p = op == 0 ? a.k + drow * a.ks : a.v + drow * a.vs;
            const long long stride = op == 0 ? a.ks : a.vs;
#pragma unroll
            for (int f = 0; f < 32; f++) {      // rows g, g + 8; features 16 m + 8 e + 2 t
              const int row = g + 8 * (f >> 1 & 1);
              x[f] = row < n ? *reinterpret_cast<const uint32_t*>(p + row * stride + h * (2 * kD) + 2 * (16 * (f >> 2) + 8 * (f & 1) + 2 * t))
                             : 0u;
            }
          }
          if (ELEM == DKV_BF16) {
            uint32_t am = 0;
#pragma unroll
            for (int f = 0; f < 32; f++) am = amax2_finite(am, x[f]);
            const int ex = scale_exp(am);
            const float inv = pow2(-ex);
#pragma unroll
            for (int f = 0; f < 32; f++) x[f] = half_of_bf16(x[f], inv);
            if (op == 0) meta.ks = kLogitScale * pow2(ex);
            else meta.lv = (float)ex;
          }
#pragma unroll
          for (int f = 0; f < 8; f++) {
            if (op == 0)
              stmatrix4(base + ((k_off + (f >> 2) * 8192) ^ ((f & 3) << 5)), x[4 * f], x[4 * f + 1], x[4 * f + 2], x[4 * f + 3]);
            else if (d.kind == 2)
              stmatrix4(base + v_off + f * 2048, x[4 * f], x[4 * f + 1], x[4 * f + 2], x[4 * f + 3]);
            else
              stmatrix4_trans(base + vt_off + f * 2048, x[4 * f], x[4 * f + 1], x[4 * f + 2], x[4 * f + 3]);
          }
        }
      }
      if (lane == 0) sm.meta[stage][sub] = meta;
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(full(stage));
    };
    if (steps > 0) {
      uint4 w0[8], w1[8];
      describe(0);
      fetch(0, w0);
      fetch(1, w1);
#pragma unroll 1
      for (int k = 0; ok && k < steps; k += 2) {
        if ((k & 31) == 0) describe((k >> 5) + 1);
        put(k, w0);
        fetch(k + 2, w0);
        if (ok && k + 1 < steps) {
          put(k + 1, w1);
          fetch(k + 3, w1);
        }
      }
      if (!ok) fail();
    }
  } else {
    // ---- products: S of the steps to come, then O += P V; the whole warp walks, one
    // lane issues ----
    constexpr uint32_t id_s = umma_idesc_f16(128, 64), id_pv = umma_idesc_f16(128, 128);
    const uint64_t kd = umma_desc_sw128(smem_u32(smem)), vd = umma_desc_sw128(smem_u32(smem + 16384));
    auto product_s = [&](int j) {
      const int h = j & 1, n = j >> 1, stage = j % kT8Stages;
      ok = wait(full(stage), j / kT8Stages) && (n == 0 || wait(sfree(h), n - 1));
      if (!ok) return;
      tc_fence_after();
      if (lane == 0) {
#pragma unroll
        for (int e = 0; e < 8; e++)
          umma_f16_tmem_a(t_s(h), t_q + 8 * e, kd + ((stage * kT8Stage + (e >> 2) * 8192 + (e & 3) * 32) >> 4), id_s, e > 0);
        umma_commit(sfull(h));
      }
      __syncwarp();
    };
    auto product_v = [&](int j, int tiles, bool start) {
      const int h = j & 1, n = j >> 1, stage = j % kT8Stages;
      ok = wait(pfull(h), n);
      if (!ok) return;
      tc_fence_after();
      if (lane == 0) {
#pragma unroll
        for (int e = 0; e < kT8Step; e++)
          if (e < tiles)
            umma_f16_tmem_a(t_o(h), t_p(h) + 8 * e, vd + ((stage * kT8Stage + e * 32) >> 4), id_pv, !start || e > 0);
        umma_commit(pvdone(h));
        umma_commit(empty(stage));
      }
      __syncwarp();
    };
    int item = 0;
    for (int pos = lo, j0 = 0; ok && pos < hi; item++) {
      const TreeItem it = tree_item(c, a, sm.plan, pos, hi);
      ok = wait(ready, item);
      if (!ok) break;
      tc_fence_after();
      product_s(j0);
      if (ok && it.n > 1) product_s(j0 + 1);
      for (int x = 0; ok && x < it.n; x++) {
        if (x + 2 < it.n) product_s(j0 + x + 2);
        if (ok) product_v(j0 + x, min(kT8Step, it.tiles.count - kT8Step * (it.s0 + x)), x < 2);
      }
      pos += it.n;
      j0 += it.n;
    }
    if (!ok) fail();
    if (lane == 0) {
      umma_commit(drain);                // every MMA issued so far has completed
      mbar_wait_bounded(drain, 0);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8 + kT8Conv) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// ---- rows of units that several CTAs hold parts of, and rows that came out infinite or
// NaN: a warp a row ----
template <int ELEM, int CODE>
__global__ void __launch_bounds__(32 * kT8Walkers) k_tree8_join(Cache8View c, Tree8Args a, int part_rows, int main_grid) {
  __shared__ TreePlan plan;
  __shared__ int scan[32];
  pdl_launch_dependents();
  pdl_wait();
  if (c.stopped()) return;
  const int total = make_plan(c, a, plan, scan);
  if (total == 0) return;
  const int ctas = tree_ctas(total, main_grid);
  const int lane = threadIdx.x & 31, G = c.G, hq = c.hkv * G;
  const long long rows = (long long)a.n_req * a.max_nodes * hq;
#pragma unroll 1
  for (long long x = (long long)blockIdx.x * kT8Walkers + (threadIdx.x >> 5); x < rows; x += (long long)gridDim.x * kT8Walkers) {
    const int q = (int)(x % hq), y = (int)(x / hq), i = y / a.max_nodes, m = y - i * a.max_nodes, h = q / G;
    const TreeReq req{plan.N[i], plan.M[i], plan.slot[i]};
    if (m >= req.M) continue;
    uint8_t* out = a.out + x * (2 * kD);
    const TreeTiles tiles = tree_tiles(req.N, req.M, c.T, a.window, a.sinks);
    const int per = (tiles.count + kT8Step - 1) / kT8Step, row = m * G + (q - h * G), t = row / kT8Rows, r = row - t * kT8Rows;
    const int us = plan.pre[i] + (h * unit_rows(req.M, G) + t) * per;
    const int c0 = range_of(total, us, ctas), c1 = range_of(total, us + per - 1, ctas);
    uint2 w;
    uint32_t bad = 0;
    if (c0 == c1) {
      w = *reinterpret_cast<const uint2*>(out + 8 * lane);
    } else {
      // the first part begins its unit (place 1), the others go on with it (place 0)
      auto part = [&](int cta) { return a.part + (size_t)(2 * cta + (cta == c0 ? 1 : 0)) * part_rows * (kD + 2); };
      float top = -INFINITY, sum = 0.0f;
      for (int b = c0; b <= c1; b += 32) {
        float2 ul = make_float2(-INFINITY, 0.0f);
        if (b + lane <= c1) ul = reinterpret_cast<const float2*>(part(b + lane) + part_rows * kD)[r];
        float now = ul.x;
#pragma unroll
        for (int d = 16; d; d >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, d));
        now = fmaxf(now, top);
        sum = sum == 0.0f ? 0.0f : sum * (top == now ? 1.0f : fast_exp2(top - now));
        sum += ul.y == 0.0f ? 0.0f : ul.y * (ul.x == now ? 1.0f : fast_exp2(ul.x - now));
        top = now;
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int b = c0; b <= c1; b += 32) {
        float f = 0.0f;
        if (b + lane <= c1) {
          const float2 ul = reinterpret_cast<const float2*>(part(b + lane) + part_rows * kD)[r];
          f = ul.y == 0.0f ? 0.0f : __fdiv_rn(ul.y * (ul.x == top ? 1.0f : fast_exp2(ul.x - top)), sum);
        }
        const int n = min(c1 - b + 1, 32);
#pragma unroll 4
        for (int e = 0; e < n; e++) {
          const float4 v = reinterpret_cast<const float4*>(part(b + e) + r * kD)[lane];
          const float fe = __shfl_sync(0xffffffffu, f, e);
          o.x = fmaf(v.x, fe, o.x);
          o.y = fmaf(v.y, fe, o.y);
          o.z = fmaf(v.z, fe, o.z);
          o.w = fmaf(v.w, fe, o.w);
        }
      }
      w = make_uint2(pack_elems<ELEM>(in_range<ELEM>(o.x), in_range<ELEM>(o.y)), pack_elems<ELEM>(in_range<ELEM>(o.z), in_range<ELEM>(o.w)));
      *reinterpret_cast<uint2*>(out + 8 * lane) = w;
    }
    find_not_finite<ELEM>(bad, w.x);
    find_not_finite<ELEM>(bad, w.y);
    if (__any_sync(0xffffffffu, found_not_finite(bad))) {
      const Walk<ELEM, CODE> walk{c, a, i, h, lane, req, tiles};
      walk.row(m, q - h * G, out);
    }
  }
}

int part_rows_of(int G, int max_nodes) { return std::min(kT8Rows, (max_nodes * G + 31) / 32 * 32); }

template <int ELEM, int CODE>
cudaError_t tree_typed(const Cache8View& c, const Tree8Args& a, int sm_count, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(k_tree8<ELEM, CODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kT8Smem);
  if (e != cudaSuccess) return e;
  const int part_rows = part_rows_of(c.G, a.max_nodes);
  // no more CTAs than the longest lengths that the table holds could use
  const long long tiles = ((long long)c.width * c.T + a.max_nodes) / kSub + 3;
  const long long steps = (long long)a.n_req * c.hkv * ((a.max_nodes * c.G + kT8Rows - 1) / kT8Rows) * (tiles / kT8Step + 1);
  const int grid = (int)std::min<long long>(sm_count, (steps + kT8Least - 1) / kT8Least);
  e = launch_dependent(k_tree8<ELEM, CODE>, dim3(grid), dim3(kT8Threads), kT8Smem, st, c, a, part_rows);
  if (e != cudaSuccess) return e;
  const long long rows = (long long)a.n_req * a.max_nodes * c.hkv * c.G;
  const int blocks = (int)std::min<long long>((rows + kT8Walkers - 1) / kT8Walkers, (long long)sm_count * 6);
  return launch_dependent(k_tree8_join<ELEM, CODE>, dim3(blocks), dim3(32 * kT8Walkers), 0, st, c, a, part_rows, grid);
}

}  // namespace

size_t tree8_workspace(int G, int max_nodes, int sm_count) {
  return (size_t)sm_count * 2 * part_rows_of(G, max_nodes) * (kD + 2) * 4;
}

cudaError_t launch_tree8(const Cache8View& c, int elem, int code, int sm_count, const Tree8Args& a, cudaStream_t st) {
  if (elem == DKV_F16)
    return code == DKV_E4M3 ? tree_typed<DKV_F16, DKV_E4M3>(c, a, sm_count, st) : tree_typed<DKV_F16, DKV_INT8>(c, a, sm_count, st);
  return code == DKV_E4M3 ? tree_typed<DKV_BF16, DKV_E4M3>(c, a, sm_count, st) : tree_typed<DKV_BF16, DKV_INT8>(c, a, sm_count, st);
}

}  // namespace dkv
