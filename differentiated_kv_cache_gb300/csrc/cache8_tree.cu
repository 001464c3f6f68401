// cache8_tree.cu — attention for trees of drafted tokens over the uniform 8-bit
// cache (include/dkv.h: dkv_cache8_tree).
#include <algorithm>

#include "cache8.cuh"
#include "dkv_kernels.cuh"

namespace dkv {
namespace {

constexpr int kT8Rows = 128;        // query rows of a unit: (node, head of the group), nodes first
constexpr int kT8Walkers = 8;       // warps of a block that walks rows

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

template <int ELEM, int CODE>
__global__ void __launch_bounds__(32 * kT8Walkers) k_tree8_rows(Cache8View c, Tree8Args a) {
  pdl_launch_dependents();
  pdl_wait();
  if (c.stopped()) return;
  const int lane = threadIdx.x & 31, hq = c.hkv * c.G;
  const long long rows = (long long)a.n_req * a.max_nodes * hq;
  for (long long x = (long long)blockIdx.x * kT8Walkers + (threadIdx.x >> 5); x < rows; x += (long long)gridDim.x * kT8Walkers) {
    const int q = (int)(x % hq), y = (int)(x / hq), i = y / a.max_nodes, m = y - i * a.max_nodes, h = q / c.G;
    const TreeReq r = tree_req(c, a, i);
    if (m >= r.M) continue;
    const Walk<ELEM, CODE> w{c, a, i, h, lane, r, tree_tiles(r.N, r.M, c.T, a.window, a.sinks)};
    w.row(m, q - h * c.G, a.out + x * (2 * kD));
  }
}

}  // namespace

size_t tree8_workspace(int G, int max_nodes, int sm_count) {
  const size_t rows = std::min(kT8Rows, (max_nodes * G + 31) / 32 * 32);
  return (size_t)sm_count * 2 * rows * (kD + 2) * 4;
}

cudaError_t launch_tree8(const Cache8View& c, int elem, int code, int sm_count, const Tree8Args& a, cudaStream_t st) {
  auto kernel = elem == DKV_F16 ? (code == DKV_E4M3 ? k_tree8_rows<DKV_F16, DKV_E4M3> : k_tree8_rows<DKV_F16, DKV_INT8>)
                                : (code == DKV_E4M3 ? k_tree8_rows<DKV_BF16, DKV_E4M3> : k_tree8_rows<DKV_BF16, DKV_INT8>);
  const long long rows = (long long)a.n_req * a.max_nodes * c.hkv * c.G;
  const int grid = (int)std::min<long long>((rows + kT8Walkers - 1) / kT8Walkers, (long long)sm_count * 8);
  return launch_dependent(kernel, dim3(grid), dim3(32 * kT8Walkers), 0, st, c, a);
}

}  // namespace dkv
