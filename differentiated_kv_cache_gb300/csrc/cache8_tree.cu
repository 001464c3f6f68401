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
// registers a thread: launched with 128; 256 x 168 + 256 x 88 = 512 x 128
constexpr int kT8RegsFew = 88, kT8RegsMany = 168;
constexpr int kT8Stages = 4;        // even: a stage is of one half, which has seen its phases
constexpr int kT8Stage = 32768;     // K, then V of a step in 16 bits
constexpr int kT8Descs = 64;        // descriptors of a converting warp, a ring
constexpr int kT8Ring = 2;          // copies that it has on their way
constexpr int kT8Pitch = 272;       // bytes from draft row to draft row (no bank conflicts)
constexpr int kT8Entry = 16 * kT8Pitch;     // K and V codes of a tile, or K or V of a 16-bit one
constexpr float kT8Up = 7.0f;       // log2 of a weight at its row's maximum
constexpr float kT8Most = 32768.0f; // largest sum of a row's weights of one tile (fp16 holds 65504)

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
  const int lt = __ffs(T) - 1;      // T is a power of two, at least 16
  t.full = N >> lt << (lt - 4);
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
  uint32_t qmax[2][kT8Rows];   // bits of the largest |q| of the features that a half's warps load
  int scan[32];
  uint64_t bar[2 * kT8Stages + 10];
  uint64_t rbar[kT8Conv][kT8Ring];
  uint32_t taddr;
  int fail;
};
constexpr int kT8OffRing = kT8Stages * kT8Stage, kT8OffSmem = kT8OffRing + kT8Conv * kT8Ring * kT8Entry;
constexpr int kT8Smem = 1024 + kT8OffSmem + (int)sizeof(TreeSmem);

__device__ __forceinline__ void stmatrix4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void stmatrix4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
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

// One lane of the warp. A branch on it, not on the lane's number, leaves the products'
// operands in uniform registers: an M = 128, K = 16 product with A in tensor memory
// takes 42 (N = 64) and 74 cycles (N = 128) to issue, and 100 otherwise.
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ bool wait_long(uint32_t bar, uint32_t parity) { return mbar_wait_bounded(bar, parity); }

// Tile x of a CTA whose range begins at step lo.
__device__ __forceinline__ void describe_tile(const Cache8View& c, const Tree8Args& a, const TreePlan& plan, int lo, int x, TileDesc& out) {
  const int pos = lo + x / kT8Step;
  const TreeItem it = tree_item(c, a, plan, pos, pos + 1);
  x = kT8Step * it.s0 + x % kT8Step;
  TileDesc d{nullptr, kLogitScale, {0.0f}, 0, 4};
  if (x < it.tiles.stored) {
    const int tile = it.tiles.tile(x);
    d.pos0 = tile * kSub;
    if (tile < it.tiles.full) {
      const int per = __ffs(c.T) - 5;      // log2 of a block's tiles
      int page = c.table[(size_t)it.slot * c.width + (tile >> per)];
      if ((unsigned)page >= (unsigned)c.n_pages) {
        c.latch(DKV_ERR_CHECK, it.i);
        page = 0;
      }
      const float2 sc = *reinterpret_cast<const float2*>(c.scales + 2 * ((size_t)page * c.hkv + it.h));
      d.src = c.pages + c.page_head(page, it.h) + (size_t)(tile & ((1 << per) - 1)) * (2 * kTile);
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
  out = d;
}

// K (op 0) or V of a tile of the tail (op + 0) or of drafts (op + 2), n tokens of it valid,
// from its copy `src` in shared memory to fp16 operands (`at`: the lane's row of the first
// four matrices). Returns the exponent of the power of two that the values were divided by.
template <int ELEM>
__device__ __noinline__ int put_elems(const uint8_t* src, int op, int n, uint32_t at) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const bool v = op & 1, draft = op & 2;
  uint32_t x[32];
  int ex = 0;
  if (!draft) {
    // what lies behind the request's tokens becomes 0 (0 times what it may hold is not)
    const uint32_t lo_t = v ? (2 * t < n ? 0xffffu : 0u) | (2 * t + 1 < n ? 0xffff0000u : 0u) : g < n ? 0xffffffffu : 0u;
    const uint32_t hi_t = v ? (2 * t + 8 < n ? 0xffffu : 0u) | (2 * t + 9 < n ? 0xffff0000u : 0u) : g + 8 < n ? 0xffffffffu : 0u;
#pragma unroll
    for (int f = 0; f < 8; f++) {
      const uint4 y = *reinterpret_cast<const uint4*>(src + 512 * f + 16 * lane);
      x[4 * f] = y.x & lo_t;
      x[4 * f + 1] = y.y & (v ? hi_t : lo_t);
      x[4 * f + 2] = y.z & (v ? lo_t : hi_t);
      x[4 * f + 3] = y.w & hi_t;
    }
  } else {
#pragma unroll
    for (int f = 0; f < 32; f++) {      // rows g, g + 8; features 16 m + 8 e + 2 t
      const int row = g + 8 * (f >> 1 & 1);
      const uint32_t y = *reinterpret_cast<const uint32_t*>(src + row * kT8Pitch + 2 * (16 * (f >> 2) + 8 * (f & 1) + 2 * t));
      x[f] = row < n ? y : 0u;
    }
  }
  if (ELEM == DKV_BF16) {
    uint32_t am = 0;
#pragma unroll
    for (int f = 0; f < 32; f++) am = amax2_finite(am, x[f]);
    ex = scale_exp(am);
    const float inv = pow2(-ex);
#pragma unroll
    for (int f = 0; f < 32; f++) x[f] = half_of_bf16(x[f], inv);
  }
#pragma unroll
  for (int f = 0; f < 8; f++) {
    if (!v)
      stmatrix4((at + (f >> 2) * 8192) ^ ((f & 3) << 5), x[4 * f], x[4 * f + 1], x[4 * f + 2], x[4 * f + 3]);
    else if (!draft)
      stmatrix4(at + f * 2048, x[4 * f], x[4 * f + 1], x[4 * f + 2], x[4 * f + 3]);
    else
      stmatrix4_trans(at + f * 2048, x[4 * f], x[4 * f + 1], x[4 * f + 2], x[4 * f + 3]);
  }
  return ex;
}

template <int ELEM, int CODE>
__global__ void __launch_bounds__(kT8Threads, 1) k_tree8(const __grid_constant__ Cache8View c, const __grid_constant__ Tree8Args a, int part_rows) {
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TreeSmem& sm = *reinterpret_cast<TreeSmem*>(smem + kT8OffSmem);
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
    for (int w = 0; w < kT8Conv * kT8Ring; w++) mbar_init(smem_u32(&sm.rbar[0][0]) + 8 * w, 1);
    sm.fail = 0;
    fence_mbar_init();
  }
  if (warp == 8 + kT8Conv) tmem_alloc(smem_u32(&sm.taddr), 512);
  pdl_wait();
  // an error of an earlier call (its load is in flight with the plan's)
  const int halted = threadIdx.x == 0 ? *(volatile int*)c.status : 0;
  const int total = make_plan(c, a, sm.plan, sm.scan);
  tc_fence_before();
  const bool stopped = __syncthreads_or(halted);
  tc_fence_after();
  const int ctas = tree_ctas(total, gridDim.x);
  if (stopped || total == 0 || (int)blockIdx.x >= ctas) {
    if (warp == 8 + kT8Conv) tmem_dealloc(__shfl_sync(0xffffffffu, sm.taddr, 0), 512);
    return;
  }
  const int lo = range_start(total, blockIdx.x, ctas), hi = range_start(total, blockIdx.x + 1, ctas);
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
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, phase & 1))) return true;
    return __all_sync(0xffffffffu, *(volatile int*)&sm.fail == 0 && wait_long(bar, phase & 1)) != 0;
  };
  bool ok = true;

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kT8RegsMany));
    // ---- softmax: a thread per query row, a half takes every other step ----
    const int half = warp >> 2, lg = warp & 3, r = 32 * lg + lane;
    const uint32_t tl = (uint32_t)(32 * lg) << 16;
    Node node;
    TreeItem it = tree_item(c, a, sm.plan, lo, hi);
    int last_i = -1, last_t = -1, parent = 0;
    uint4 qr[8];              // 64 features of the row, the other half's warps have the others
    auto row_of = [&](const TreeItem& x) { return x.t * kT8Rows + r; };
    auto real_of = [&](const TreeItem& x) { return row_of(x) < x.M * G; };
    auto q_of = [&](const TreeItem& x) {
      const int row = row_of(x), m = row / G;
      return a.q + ((long long)x.i * a.max_nodes + m) * a.qs + ((size_t)x.h * G + (row - m * G)) * (2 * kD) + 128 * half;
    };
    auto load_row = [&](const TreeItem& x) {
      const uint4* src = reinterpret_cast<const uint4*>(q_of(x));
      const bool real = real_of(x);
#pragma unroll
      for (int e = 0; e < 8; e++) qr[e] = real ? src[e] : make_uint4(0, 0, 0, 0);
      if (half == 1 && a.parents && r < x.M) parent = a.parents[(size_t)x.i * a.max_nodes + r];
    };
    load_row(it);
    for (int pos = lo, j0 = 0;;) {
      const int row = row_of(it), m = row / G;
      const bool real = real_of(it), busy = 32 * lg + it.t * kT8Rows < it.M * G;
      if (half == 1 && r < it.M) sm.parents[r] = parent;
      if (ELEM == DKV_BF16) {
        uint32_t am = 0;
#pragma unroll
        for (int e = 0; e < 8; e++) am = amax2_finite(amax2_finite(amax2_finite(amax2_finite(am, qr[e].x), qr[e].y), qr[e].z), qr[e].w);
        sm.qmax[half][r] = max(am & 0xffffu, am >> 16);
      }
      named_sync(1, 256);
      // the queries as fp16 (bf16: over a power of two of their row)
      float scale = 1.0f, inv = 1.0f;
      if (ELEM == DKV_BF16) {
        const int ex = max(-126, min(126, (int)(max(sm.qmax[0][r], sm.qmax[1][r]) >> 7) - 127));
        inv = pow2(-ex);
        scale = pow2(ex);
      }
      if (busy) {
#pragma unroll
        for (int e = 0; e < 2; e++) {
          uint32_t q[16];
#pragma unroll
          for (int x = 0; x < 4; x++) {
            q[4 * x] = qr[4 * e + x].x;
            q[4 * x + 1] = qr[4 * e + x].y;
            q[4 * x + 2] = qr[4 * e + x].z;
            q[4 * x + 3] = qr[4 * e + x].w;
          }
          if (ELEM == DKV_BF16) {
#pragma unroll
            for (int x = 0; x < 16; x++) q[x] = half_of_bf16(q[x], inv);
          }
          tmem_st16(t_q + tl + 32 * half + 16 * e, q);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ready);
      if (real && (it.i != last_i || it.t != last_t)) node = node_of(c, a, a.parents ? sm.parents : nullptr, it.i, it.N, m);
      last_i = it.i;
      last_t = it.t;
      float mx = -INFINITY, u = -INFINITY, l = 0.0f;
      int j = j0 + ((j0 & 1) != half), n = j >> 1, stage = j % kT8Stages;
      const int end = j0 + it.n;
      bool first = true, raise = true, have = false;
      float s[64];
      auto load_s = [&]() {
        tc_fence_after();
        if (busy) {
          tmem_ld32_nowait(t_s(half) + tl, s);
          tmem_ld32_nowait(t_s(half) + tl + 32, s + 32);
        }
      };
      for (; ok && j < end; j += 2, n++) {
        if (!have) {
          ok = wait(sfull(half), n);
          if (!ok) break;
          load_s();
        }
        if (busy) {
          tmem_wait_ld();
          loaded32(s);
          loaded32(s + 32);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sfree(half));
        uint32_t p[32];
        if (busy) {
          const TileMeta* meta = sm.meta[stage];
          float f[4], lv[4];
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
          }
          float sum;
#pragma unroll 1
          for (bool again = raise;; again = true) {
            if (again) {
              float ym[4];
#pragma unroll
              for (int b = 0; b < 4; b++) {
                float y0 = s[16 * b], y1 = s[16 * b + 1];
#pragma unroll
                for (int e = 2; e < 16; e += 2) {
                  y0 = fmaxf(y0, s[16 * b + e]);
                  y1 = fmaxf(y1, s[16 * b + e + 1]);
                }
                ym[b] = fmaxf(y0, y1) * f[b];
              }
              const float nu = fmaxf(u, fmaxf(fmaxf(ym[0], ym[1]), fmaxf(ym[2], ym[3])));
              const float nm = fmaxf(mx, fmaxf(fmaxf(ym[0] + lv[0], ym[1] + lv[1]), fmaxf(ym[2] + lv[2], ym[3] + lv[3])));
              l *= nu == -INFINITY ? 1.0f : fast_exp2(u - nu);
              if (!first) {        // O is still once the last product is done
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
              raise = __any_sync(0xffffffffu, real && u == -INFINITY);      // a row that has seen nothing so far
            }
            const float ur = u == -INFINITY ? 0.0f : u, up = kT8Up + ur - (mx == -INFINITY ? 0.0f : mx);
            float most = 0.0f;
            sum = 0.0f;
#pragma unroll
            for (int b = 0; b < 4; b++) {
              const float g = fast_exp2(fminf(up + lv[b], 127.0f));
              const uint64_t f2 = f32x2(f[b], f[b]), u2 = f32x2(-ur, -ur), g2 = f32x2(g, g);
              uint64_t part[2] = {0, 0};
#pragma unroll
              for (int e = 0; e < 8; e++) {
                const uint64_t y = fma_f32x2(f32x2(s[16 * b + 2 * e], s[16 * b + 2 * e + 1]), f2, u2);
                const uint64_t pr = f32x2(fast_exp2(__uint_as_float((uint32_t)y)), fast_exp2(__uint_as_float((uint32_t)(y >> 32))));
                part[e & 1] = add_f32x2(part[e & 1], pr);
                const uint64_t w = mul_f32x2(pr, g2);
                p[8 * b + e] = pack_half2(__uint_as_float((uint32_t)w), __uint_as_float((uint32_t)(w >> 32)));
              }
              part[0] = add_f32x2(part[0], part[1]);
              const float tile = __uint_as_float((uint32_t)part[0]) + __uint_as_float((uint32_t)(part[0] >> 32));
              sum += tile;
              most = tile * g <= kT8Most ? most : INFINITY;
            }
            if (again || !__any_sync(0xffffffffu, real && most != 0.0f)) break;
          }
          if (!ok) break;
          l += sum;
        }
        // the next S, if it is there, comes while P goes
        have = j + 2 < end && __all_sync(0xffffffffu, mbar_test(sfull(half), (n + 1) & 1));
        if (have) load_s();
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
        stage += 2;
        if (stage >= kT8Stages) stage -= kT8Stages;
      }
      // the next item's queries, while the last product is awaited
      pos += it.n;
      j0 += it.n;
      const TreeItem then = pos < hi ? tree_item(c, a, sm.plan, pos, hi) : it;
      if (pos < hi && real_of(then)) asm volatile("prefetch.global.L2 [%0];\n" ::"l"(q_of(then)));
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
        // a part: [feature / 4][row][4], whose lanes' stores are neighbours, then (u, l) of the rows
        float4* part = reinterpret_cast<float4*>(a.part + (size_t)(2 * blockIdx.x + (it.s0 > 0 ? 0 : 1)) * part_rows * (kD + 2));
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
              part[(16 * half + 4 * q + e) * part_rows + r] = make_float4(o0[4 * e], o0[4 * e + 1], o0[4 * e + 2], o0[4 * e + 3]);
          }
        }
        if (real && !whole && half == 0) reinterpret_cast<float2*>(part + part_rows * (kD / 4))[r] = make_float2(top, lsum);
      }
      tc_fence_before();
      if (pos >= hi) break;
      it = then;
      load_row(it);
    }
  } else {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kT8RegsFew));
  if (warp < 8 + kT8Conv) {
    // ---- codes, tails and drafts to 16-bit operands: the tiles of the steps are dealt
    // out to the warps in turn ----
    const int cw = warp - 8;
    const int steps = (kT8Step * (hi - lo) - cw + kT8Conv - 1) / kT8Conv;      // tiles cw, cw + kT8Conv, ..
    const int mat = lane >> 3, mrow = lane & 7, me = mat & 1, ms = mat >> 1;
    const uint32_t stage0 = smem_u32(smem);
    TileDesc* desc = sm.desc[cw];
    auto describe = [&](int batch) {       // tiles 32 batch ..: a lane each
      const int k = 32 * batch + lane;
      if (k < steps) describe_tile(c, a, sm.plan, lo, cw + kT8Conv * k, desc[k & (kT8Descs - 1)]);
      __syncwarp();
    };
    // The next copy: codes of a tile, or K, then V of a 16-bit one.
    uint8_t* ring = smem + kT8OffRing + cw * (kT8Ring * kT8Entry);
    const uint32_t rbar = smem_u32(sm.rbar[cw]);
    int at = 0, at_v = 0, ahead = 0, entry = 0, parity = 0, flying = 0;
    auto issue = [&]() {
      TileDesc d;
      for (;; at++) {
        if (at >= steps) return;
        d = desc[at & (kT8Descs - 1)];
        if (d.kind < 4) break;
      }
      const uint32_t dst = smem_u32(ring + ahead * kT8Entry), bar = rbar + 8 * ahead;
      if (d.kind <= 2) {
        if (lane == 0) {
          mbar_expect_tx(bar, 2 * kTile);
          bulk_g2s(dst, d.src + at_v * (2 * kTile), 2 * kTile, bar);
        }
      } else {
        const int i = d.req_head >> 12, h = d.req_head & 4095, n = min(sm.plan.M[i] - d.pos0, kSub);
        const long long row = (long long)i * a.max_nodes + d.pos0 + lane;
        if (lane == 0) mbar_expect_tx(bar, n * (2 * kD));
        __syncwarp();
        if (lane < n)
          bulk_g2s(dst + lane * kT8Pitch, (at_v ? a.v + row * a.vs : a.k + row * a.ks) + h * (2 * kD), 2 * kD, bar);
      }
      flying++;
      ahead = ahead == kT8Ring - 1 ? 0 : ahead + 1;
      at_v = d.kind >= 2 ? at_v ^ 1 : 0;
      at += at_v ^ 1;
    };
    auto arrived = [&]() {               // the next copy
      const uint8_t* p = ring + entry * kT8Entry;
      ok = wait(rbar + 8 * entry, parity);
      if (!ok) return p;
      flying--;
      if (++entry == kT8Ring) {
        entry = 0;
        parity ^= 1;
      }
      return p;
    };
    int described = 0;
    if (steps > 0) {
      describe(0);
      for (int e = 0; e < kT8Ring; e++) issue();
    }
#pragma unroll 1
    for (int k = 0; ok && k < steps; k++) {
      // descriptors up to 32 tiles ahead
      if (32 * (described + 1) < steps && k >= 32 * described + 4 * cw) describe(++described);
      const int tile_of = cw + kT8Conv * k, j = tile_of / kT8Step, sub = tile_of % kT8Step, stage = j % kT8Stages;
      // (P V of step j - 8, the phase before, is done: this warp's last tile was of step
      // j - 1 or j - 2, so P V of j - 5, whose S waited for it, or of j - 6 is)
      if (j >= kT8Stages) ok = wait(empty(stage), j / kT8Stages - 1);
      if (!ok) break;
      const uint32_t base = stage0 + stage * kT8Stage;
      // the lane's row of the four 8 x 8 matrices of a store: K, V, V of drafts
      const uint32_t k_at = base + (2 * sub + ms) * 1024 + mrow * 128 + ((me ^ mrow) << 4);
      const uint32_t v_at = base + 16384 + ms * 1024 + mrow * 128 + (((2 * sub + me) ^ mrow) << 4);
      const TileDesc d = desc[k & (kT8Descs - 1)];
      TileMeta meta{d.ks, d.lv, d.pos0, d.kind < 2 ? d.kind : d.kind - 1};
      if (d.kind <= 1) {
        const uint8_t* p = arrived() + 16 * lane;
        if (!ok) break;
        uint4 w[8];
#pragma unroll
        for (int e = 0; e < 8; e++) w[e] = *reinterpret_cast<const uint4*>(p + 512 * e);
        __syncwarp();
        issue();
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const uint32_t at0 = e < 4 ? (k_at + (e >> 1) * 8192) ^ ((e & 1) << 6) : v_at + (e - 4) * 4096;
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
        const int i = d.req_head >> 12, draft = d.kind == 3 ? 2 : 0;
        const int n = min((draft ? sm.plan.M[i] : sm.plan.N[i]) - d.pos0, kSub);      // valid tokens
        const uint8_t* p = arrived();
        if (!ok) break;
        meta.ks = kLogitScale * pow2(put_elems<ELEM>(p, draft, n, k_at));
        __syncwarp();
        issue();
        p = arrived();
        if (!ok) break;
        const uint32_t vt_at = base + 16384 + me * 1024 + mrow * 128 + (((2 * sub + ms) ^ mrow) << 4);
        meta.lv = (float)put_elems<ELEM>(p, draft + 1, n, draft ? vt_at : v_at);
        __syncwarp();
        issue();
      }
      if (lane == 0) sm.meta[stage][sub] = meta;
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(full(stage));
    }
    if (!ok) fail();
    // no copy may be in flight at the exit
    for (; flying > 0; flying--) {
      wait_long(rbar + 8 * entry, parity);
      if (++entry == kT8Ring) {
        entry = 0;
        parity ^= 1;
      }
    }
  } else {
    // ---- products: S of the steps to come, then O += P V; the whole warp walks, one
    // lane issues (counters, so that operands stay in uniform registers) ----
    constexpr uint32_t id_s = umma_idesc_f16(128, 64), id_pv = umma_idesc_f16(128, 128);
    const uint64_t kd = umma_desc_sw128(smem_u32(smem)), vd = umma_desc_sw128(smem_u32(smem + 16384));
    // Of each half: steps whose S, whose P V are issued, whose P V are done, and their
    // stages. Whatever can be issued is, but S of step j waits for P V of step j - 3, so that
    // stages are freed nearly in order (a converting warp waits for those of its tiles only).
    int ns[2] = {0, 0}, nv[2] = {0, 0}, done[2] = {0, 0}, s_stage[2] = {0, 1}, s_round[2] = {0, 0}, v_stage[2] = {0, 1};
    auto test = [&](uint32_t bar, int phase) { return __all_sync(0xffffffffu, mbar_test(bar, phase & 1)) != 0; };
    auto next = [](int& stage) {          // two steps on; true behind the last stage
      stage += 2;
      if (stage < kT8Stages) return false;
      stage -= kT8Stages;
      return true;
    };
    int item = 0, j0 = 0;
    for (int pos = lo; ok && pos < hi; item++) {
      const TreeItem it = tree_item(c, a, sm.plan, pos, hi);
      const int n = __shfl_sync(0xffffffffu, it.n, 0);
      // tiles of the part's last step
      const int rest = __shfl_sync(0xffffffffu, min(kT8Step, it.tiles.count - kT8Step * (it.s0 + it.n - 1)), 0);
      const int begin[2] = {(j0 + 1) >> 1, j0 >> 1};
      j0 += n;
      pos += n;
      const int end[2] = {(j0 + 1) >> 1, j0 >> 1};
      ok = wait(ready, item);
      if (!ok) break;
      tc_fence_after();
      long long since = 0;
      int idle = 0;
#pragma unroll 1
      while (nv[0] < end[0] || nv[1] < end[1]) {
        bool none = true;
#pragma unroll
        for (int h = 0; h < 2; h++) {
          if (done[h] < nv[h] && test(pvdone(h), nv[h] - 1)) done[h] = nv[h];
          if (ns[h] < end[h] && done[h ^ 1] >= ns[h] - 1 + h && test(full(s_stage[h]), s_round[h]) && (ns[h] == 0 || test(sfree(h), ns[h] - 1))) {
            tc_fence_after();
            if (elected()) {
              const uint64_t bd = kd + s_stage[h] * (kT8Stage >> 4);
#pragma unroll
              for (int e = 0; e < 8; e++)
                umma_f16_tmem_a(t_s(h), t_q + 8 * e, bd + (((e >> 2) * 8192 + (e & 3) * 32) >> 4), id_s, e > 0);
              umma_commit(sfull(h));
            }
            __syncwarp();
            ns[h]++;
            if (next(s_stage[h])) s_round[h] ^= 1;
            none = false;
          }
          if (nv[h] < ns[h] && test(pfull(h), nv[h])) {
            tc_fence_after();
            const bool start = nv[h] == begin[h];
            const int tiles = 2 * nv[h] + h == j0 - 1 ? rest : kT8Step;
            if (elected()) {
              const uint64_t bd = vd + v_stage[h] * (kT8Stage >> 4);
#pragma unroll
              for (int e = 0; e < kT8Step; e++)
                if (e < tiles) umma_f16_tmem_a(t_o(h), t_p(h) + 8 * e, bd + (e * 32 >> 4), id_pv, !start || e > 0);
              umma_commit(pvdone(h));
              umma_commit(empty(v_stage[h]));
            }
            __syncwarp();
            done[h] = nv[h]++;       // P came after the step before was done
            next(v_stage[h]);
            none = false;
          }
        }
        // bounded: about a second without anything to issue
        if (!none) idle = 0;
        else if (++idle == 1) since = clock64();
        else if ((idle & 1023) == 0 && __any_sync(0xffffffffu, *(volatile int*)&sm.fail != 0 || clock64() - since > 2000000000LL)) {
          ok = false;
          break;
        }
      }
    }
    if (!ok) fail();
    if (elected()) {
      umma_commit(drain);                // every MMA issued so far has completed
      mbar_wait_bounded(drain, 0);
    }
    __syncwarp();
  }
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
          const float4 v = reinterpret_cast<const float4*>(part(b + e))[lane * part_rows + r];
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
