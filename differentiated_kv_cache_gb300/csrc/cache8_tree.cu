// cache8_tree.cu — attention for trees of drafted tokens over the uniform 8-bit
// cache (include/dkv.h: dkv_cache8_tree).
//
// o = sum_t w_t v_t / sum_t w_t, w_t = exp(q k_t / sqrt(128)), over the stored tokens in a
// node's window and the drafts on its way to the root. All nodes of a request and all heads
// of a group (M G query rows) read the same K and V, so the cache is read once for 128
// rows; the products, 4 * 128 operations a row and token, go to tcgen05. Both take fp16
// operands and sum in fp32: codes are exact in fp16; queries in bf16 come into its range by a
// power of two of their row, whose 8 bits stay down to 2^-17 of the largest (what lies under 2^-25
// of it is lost), bf16 K and all V of tails and drafts by one of each token, whose bits stay down
// to 2^-24 (lost under 2^-32), and so V of codes whose block some node sees a part of. K's scale joins the logits, V's joins the weights as an addend of
// their exponent. Weights are rounded to fp16 (2^-11), as probabilities are in the attention of
// single tokens.
//
// Units (request, KV head, 128 rows) of steps (128 tokens) follow one another; the sequence
// of all is cut into ranges of equal time, one for each SM, so ragged batches and one long
// request alike fill the GPU. A unit that is cut leaves parts (O over its sum, maximum, sum),
// which the second kernel joins. The way of a step, of which several are in flight:
//   lookups -> bulk copies of codes -> conversion to swizzled fp16 operands -> S = Q K^T
//   -> weights -> O += P V, with Q, S, P and O in tensor memory.
// What bounds a step of 128 rows (2500 to 2600 cycles) are the softmax warps, busy for nine
// tenths of it: logits out of tensor memory 390 cycles, weights 1350 (16384 exponentials, 4 cycles
// for a warp's 32, a quarter of them for each quarter of an SM: 512; sums and roundings), weights
// into tensor memory 350, and 300 until the next S. All eight share a step, so none of these
// hides another's; the products are done ahead of them. A step with exponents for each token takes
// 1800 to 6000: these, a second exponential, masks, V's conversion beside it. Between two units
// of a CTA lie 6000 to 12000 cycles, ahead of the first weights 24000 to 32000: the launch,
// the plan, a chain of four loads, queries, and code that all SMs fetch at once. Measured:
//   8 heads, G = 4, fp16, e4m3, 16 requests of 4096 tokens, 26 drafts    60 us (by bytes 21)
//   8 heads, G = 8, bf16, int8, 8 of 32768, 64 drafts                   552 us, 1000 TFLOP/s
//     (52 % of a plain matrix product's rate)
//   4 heads, G = 7, bf16, e4m3, 32 of 1024 to 16384, window 4096         55 us
//   8 heads, G = 5, fp16, int8, 64 of 1 to 3000, chains of 5             92 us
//   8 heads, G = 4, fp16, e4m3, one of 300 tokens, 8 drafts              11.6 us
// Tried and slower: 64 tokens a step (the second: 0.92 ms); conversion by the softmax warps
// (the chains: 196 us); maxima of each step ahead of its weights (the second: 0.66 ms; now
// they are taken when a weight could leave fp16's range); conversion unrolled over its tiles
// (0.62 ms: it leaves the instruction caches); ranges of equal steps (the chains: 126 us); the
// tails' and drafts' largest values looked for ahead of all copies (the third: 68 us); tiles of 16
// bits through the body of the other steps, with exponents of tokens (the third: 70 us).
#include <algorithm>

#include "cache8.cuh"
#include "dkv_kernels.cuh"
#include "dkv_tc.cuh"

namespace dkv {
namespace {

constexpr int kT8Rows = 128;        // query rows of a unit: (node, head of the group), nodes first
constexpr int kT8Walkers = 8;       // warps (and rows) of a block of the second kernel
constexpr int kT8Step = 8;          // tiles of a step, in two parts of four
// warps: 0 .. 7 softmax, 8 .. 11 convert K, 12 .. 15 V, 16 products, 17 lookups, 18
// copies of K codes, 19 of V codes
constexpr int kT8Threads = 640;
// registers a thread: launched with 96; 256 x 144 + 384 x 64 = 640 x 96
constexpr int kT8RegsFew = 64, kT8RegsMany = 144;
constexpr int kT8Slots = 2;         // steps whose K (V) is kept as operands
constexpr int kT8Ring = 2;          // steps whose K (V) codes are there or on their way
constexpr int kT8Entry = kT8Step * kTile;   // K or V codes of a step
constexpr int kT8Slot = 32768;      // K or V of a step in 16 bits
constexpr int kT8Batch = 4;         // steps that are looked up at once
constexpr int kT8Descs = 4 * kT8Batch;      // steps whose descriptors are kept, a ring
constexpr int kT8Metas = 8;         // steps whose scales are kept for the softmax, a ring
// steps in whose time a CTA goes from one unit to the next (2: 64 chains of 1 to 3000 tokens take
// 96 us, 32 windows 57; 3: 91 and 54; 4: 91 and 55; 6: 92 and 55)
constexpr int kT8Turn = 4;
constexpr float kT8Up = 7.0f;       // log2 of a weight at its row's maximum
constexpr float kT8Most = 32768.0f; // largest sum of a row's weights of one tile (fp16 holds 65504)
constexpr float kT8Far = 60.0f;     // log2 of how far weights may be from probabilities
constexpr float kT8Sum = 1.15292150460684698e18f;    // largest sum of probabilities under an earlier maximum, 2^kT8Far

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

// The 16-token tiles of a request: stored ones [0, head) and [win, end), of which those from `full`
// on lie in the tail, then the drafts; `count` in all. A stored tile is left out if no node of any
// depth sees a token of it. Their order: `codes` tiles of blocks that every node sees all of, [0,
// firsts) and [whole, full); other codes up to `tails`, whose block's scale may be set by what a node
// does not see; the tail's; the drafts. In the steps of the kernel below places [0, codes) hold the
// first kind; all others, whose tokens have exponents of their own (and, in 16 bits, whose copies
// need twice the room), lie from `elems` on at every second place, so that the four places of a softmax
// warp are of one sort.
struct TreeTiles {
  int head, win, end, full, firsts, whole, stored, count;
  int codes, tails, elems, places;
  __device__ __forceinline__ int tile(int x) const {
    if (x < codes) return x < firsts ? x : x - firsts + whole;
    const int mid = min(head, full);
    x -= codes;
    if (x < mid - firsts) return x + firsts;
    x -= mid - firsts;
    if (x < whole - win) return x + win;
    x -= whole - win;
    return x < head - mid ? x + mid : x - (head - mid) + max(win, full);
  }
};
__device__ __forceinline__ TreeTiles tree_tiles(int N, int M, int T, int window, int sinks) {
  TreeTiles t;
  t.end = (N + kSub - 1) / kSub;
  const int lt = __ffs(T) - 1;      // T is a power of two, at least 16
  t.full = N >> lt << (lt - 4);
  t.head = t.win = t.firsts = t.whole = 0;
  if (window > 0 && window <= N) {          // a root (position N) sees those above N - window
    const int from = N - window + 1;
    t.win = from >= N ? t.end : from / kSub;
    t.head = min((min(sinks, N) + kSub - 1) / kSub, t.win);
    t.firsts = min(sinks >> lt << (lt - 4), min(t.head, t.full));
  }
  if (window > 0 && N + M > window)         // the deepest node may see those from N + M - window on
    t.whole = (N + M - window + T - 1) >> lt << (lt - 4);
  t.whole = min(max(t.whole, t.win), max(t.win, t.full));
  t.stored = t.head + t.end - t.win;
  t.count = t.stored + (M + kSub - 1) / kSub;
  t.codes = t.firsts + max(t.win, t.full) - t.whole;
  t.tails = t.codes + min(t.head, t.full) - t.firsts + t.whole - t.win;
  t.elems = (t.codes + 3) & ~3;
  t.places = t.elems + 2 * (t.count - t.codes);
  return t;
}

// Which drafts a node sees (bits of 128) and its depth. By a whole warp, a node a lane (those
// without one: m = -1): a walk up from lanes of their own, each with its own number of steps,
// leaves the warp in pieces that run one after another (24 requests with chains of up to 110
// drafts: 355 us, 29 so).
struct Node {
  uint32_t over[kMaxNodes / 32];
  int depth;
};
__device__ __forceinline__ Node node_of(const Cache8View& c, const Tree8Args& a, const int* parents, int i, int N, int m) {
  Node n;
  n.depth = max(m, 0);
  const int w = a.window > 0 ? a.window : kMaxNodes, first = a.window > 0 ? a.sinks - N : 0;   // of a path, besides the last w: those of depth under `first`
  if (!parents) {              // a chain
#pragma unroll
    for (int e = 0; e < kMaxNodes / 32; e++)
      n.over[e] = m < 0 ? 0u : below(m + 1 - 32 * e) & (~below(m + 1 - w - 32 * e) | below(first - 32 * e));
    return n;
  }
  auto up = [&](int x) {       // x's parent (-1: none)
    int p = x >= 0 ? parents[x] : -1;
    if (p < -1 || p >= max(x, 0)) {
      c.latch(DKV_ERR_ARG, i);
      p = -1;
    }
    return p;
  };
  // a path from its end: all of it where no window cuts it, else again once its length is known
  int len = kMaxNodes;
  bool whole = true;
#pragma unroll 1
  while (true) {
#pragma unroll
    for (int e = 0; e < kMaxNodes / 32; e++) n.over[e] = 0;
    int back = 0;
#pragma unroll 1
    for (int x = m; __any_sync(0xffffffffu, x >= 0); x = up(x)) {
      const bool see = x >= 0 && (whole || back < w || len - back < first);
      const uint32_t bit = see ? 1u << (x & 31) : 0u;
#pragma unroll
      for (int e = 0; e < kMaxNodes / 32; e++) n.over[e] |= x >> 5 == e ? bit : 0u;
      back += x >= 0;
    }
    len = back - 1;            // its depth
    if (!whole || !__any_sync(0xffffffffu, back > w)) break;
    whole = false;
  }
  n.depth = max(len, 0);
  return n;
}
// Which of the 16 stored tokens from pos0 on a node sees, as bits.
__device__ __forceinline__ uint32_t sees_stored(const Tree8Args& a, int N, int depth, int pos0) {
  uint32_t s = below(min(N - pos0, kSub));
  if (a.window > 0) s &= ~below(N + depth + 1 - a.window - pos0) | below(a.sinks - pos0);
  return s;
}

// ---- one row by a block of the second kernel, from the formula in fp32, over what the row sees:
// rows that came out infinite or NaN (a code that a row does not see may have met its weight of
// 0). A warp takes every eighth tile, 32 of which it looks up at once, a lane each; the eight join.
// O is the mean so far, not a sum over weights of up to 1 each: bf16 values of the type's largest
// size leave fp32's range as the sum of two.
// 4096 tokens take a row 64 us (sums: 55); a warp a row, its code unrolled over all kinds of tiles, took 3300:
// a tile was 100 KB of instructions. ----
// A lane's share of a tile in the stored order: K of tokens g and g + 8, features
// 16 m + 2 t + {0, 1, 8, 9}; V of features 16 m + g, + 8 and tokens 2t, 2t + 1, 2t + 8, 2t + 9.
struct WalkSmem {
  float q[kD], o[kT8Walkers][kD], top[kT8Walkers], sum[kT8Walkers];
};
template <int ELEM, int CODE>
struct Walk {
  const Cache8View& c;
  const Tree8Args& a;
  int i, h;
  TreeReq r;
  TreeTiles t;

  // Words 4 m + (0 .. 3) of K or V (op): the four pairs of m-step m, in fp16 where they were codes.
  __device__ __forceinline__ void words(unsigned long long at, int kind, int n, bool op, uint32_t (&x)[32]) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, tt = lane & 3;
    const uint8_t* p = reinterpret_cast<const uint8_t*>(at);
    if (kind < 2) {
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const uint4 w = *reinterpret_cast<const uint4*>(p + op * kTile + 512 * e + 16 * lane);
        code_halves<CODE>(w.x, x[8 * e], x[8 * e + 1]);
        code_halves<CODE>(w.y, x[8 * e + 2], x[8 * e + 3]);
        code_halves<CODE>(w.z, x[8 * e + 4], x[8 * e + 5]);
        code_halves<CODE>(w.w, x[8 * e + 6], x[8 * e + 7]);
      }
    } else if (kind == 2) {
#pragma unroll
      for (int m = 0; m < 8; m++) {
        const uint4 w = *reinterpret_cast<const uint4*>(p + 2 * op * kTile + 512 * m + 16 * lane);
        x[4 * m] = w.x;
        x[4 * m + 1] = w.y;
        x[4 * m + 2] = w.z;
        x[4 * m + 3] = w.w;
      }
    } else if (!op) {             // drafts, of which those from n on are not read
#pragma unroll
      for (int f = 0; f < 32; f++) {
        const int row = f & 2 ? g + 8 : g;
        x[f] = row < n ? *reinterpret_cast<const uint32_t*>(p + row * a.ks + 32 * (f >> 2) + 16 * (f & 1) + 4 * tt) : 0u;
      }
    } else {
#pragma unroll
      for (int f = 0; f < 32; f++) {
        const int row = 2 * tt + 8 * (f & 1), at2 = 2 * (16 * (f >> 2) + 8 * (f >> 1 & 1) + g);
        const uint32_t lo = row < n ? *reinterpret_cast<const uint16_t*>(p + row * a.vs + at2) : 0u;
        const uint32_t hi = row + 1 < n ? *reinterpret_cast<const uint16_t*>(p + (row + 1) * a.vs + at2) : 0u;
        x[f] = lo | hi << 16;
      }
    }
  }

  __device__ __noinline__ void row(int m, int g8, uint8_t* out, WalkSmem& sm) const {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tt = lane & 3;
    const Node node = node_of(c, a, a.parents ? a.parents + (size_t)i * a.max_nodes : nullptr, i, r.N, m);
    // the query over a power of two (bf16), which `back` brings back
    const uint8_t* qp = a.q + ((long long)i * a.max_nodes + m) * a.qs + ((size_t)h * c.G + g8) * (2 * kD);
    const uint2 qw = *reinterpret_cast<const uint2*>(qp + 8 * lane);
    float q[4] = {lo_elem<ELEM>(qw.x), hi_elem<ELEM>(qw.x), lo_elem<ELEM>(qw.y), hi_elem<ELEM>(qw.y)}, qs = 1.0f;
    // bf16 keys may be as large as fp32: 2^-8 of them
    constexpr float kIn = ELEM == DKV_BF16 ? 0.00390625f : 1.0f;
    if (ELEM == DKV_BF16) {
      const float am = amax_finite(amax_finite(amax_finite(amax_finite(0.0f, q[0]), q[1]), q[2]), q[3]);
      const int ex = max(-126, min(118, (int)(__reduce_max_sync(0xffffffffu, __float_as_uint(am)) >> 23) - 127));
      const float inv = __uint_as_float((uint32_t)(127 - ex) << 23);
      qs = __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
      for (int e = 0; e < 4; e++) q[e] *= inv;
    }
    __syncthreads();             // (the row before has been written)
    if (warp == 0) reinterpret_cast<float4*>(sm.q)[lane] = make_float4(q[0], q[1], q[2], q[3]);
    __syncthreads();
    const float back = qs * (1.0f / kIn);
    float top = -INFINITY, l = 0.0f, o[16];
#pragma unroll
    for (int e = 0; e < 16; e++) o[e] = 0.0f;
#pragma unroll 1
    for (int b = warp; b < t.count; b += 32 * kT8Walkers) {
      // the lane's tile: where it lies, what scales it, which of its tokens the row sees
      const int mine = b + kT8Walkers * lane;
      unsigned long long k_at = 0, v_at = 0;
      float2 sc = make_float2(1.0f, 1.0f);
      uint32_t see = 0;
      int kind = 2, n = kSub;
      if (mine >= t.stored && mine < t.count) {
        const int m0 = (mine - t.stored) * kSub, w = m0 >> 5;
        kind = 3;
        n = min(r.M - m0, kSub);
        see = (w == 0 ? node.over[0] : w == 1 ? node.over[1] : w == 2 ? node.over[2] : node.over[3]) >> (m0 & 31) & 0xffffu;
        k_at = reinterpret_cast<unsigned long long>(a.k + ((long long)i * a.max_nodes + m0) * a.ks + h * (2 * kD));
        v_at = reinterpret_cast<unsigned long long>(a.v + ((long long)i * a.max_nodes + m0) * a.vs + h * (2 * kD));
      } else if (mine < t.stored) {
        const int tile = t.tile(mine), per = c.T / kSub;
        see = sees_stored(a, r.N, node.depth, tile * kSub);
        if (tile < t.full) {
          int page = c.table[(size_t)r.slot * c.width + tile / per];
          if ((unsigned)page >= (unsigned)c.n_pages) {
            c.latch(DKV_ERR_CHECK, i);
            page = 0;
          }
          kind = 0;
          sc = *reinterpret_cast<const float2*>(c.scales + 2 * ((size_t)page * c.hkv + h));
          k_at = reinterpret_cast<unsigned long long>(c.pages + c.page_head(page, h) + (size_t)(tile % per) * (2 * kTile));
        } else {
          k_at = reinterpret_cast<unsigned long long>(c.tail + c.tail_head(r.slot, h) + (size_t)(tile - t.full) * (4 * kTile));
        }
        v_at = k_at;
      }
#pragma unroll 1
      for (unsigned left = __ballot_sync(0xffffffffu, see != 0); left; left &= left - 1) {
        const int who = __ffs(left) - 1;
        const unsigned long long kp = __shfl_sync(0xffffffffu, k_at, who), vp = __shfl_sync(0xffffffffu, v_at, who);
        const float ks = __shfl_sync(0xffffffffu, sc.x, who) * kLogitScale, vs = __shfl_sync(0xffffffffu, sc.y, who);
        const uint32_t seen = __shfl_sync(0xffffffffu, see, who);
        const int kd = __shfl_sync(0xffffffffu, kind, who), valid = __shfl_sync(0xffffffffu, n, who);
        const bool halves = ELEM == DKV_F16 || kd < 2;
        auto lo = [&](uint32_t w) { return halves ? lo_elem<DKV_F16>(w) : lo_elem<DKV_BF16>(w); };
        auto hi = [&](uint32_t w) { return halves ? hi_elem<DKV_F16>(w) : hi_elem<DKV_BF16>(w); };
        uint32_t x[32];
        words(kp, kd, valid, false, x);
        float y0 = 0.0f, y1 = 0.0f;
#pragma unroll
        for (int f = 0; f < 16; f++) {            // pair f of the lane's features, tokens g and g + 8
          const float2 qv = *reinterpret_cast<const float2*>(sm.q + 16 * (f >> 1) + 8 * (f & 1) + 2 * tt);
          const uint32_t w0 = x[4 * (f >> 1) + (f & 1)], w1 = x[4 * (f >> 1) + 2 + (f & 1)];
          y0 = fmaf(qv.y, hi(w0) * kIn, fmaf(qv.x, lo(w0) * kIn, y0));
          y1 = fmaf(qv.y, hi(w1) * kIn, fmaf(qv.x, lo(w1) * kIn, y1));
        }
        words(vp, kd, valid, true, x);
        y0 += __shfl_xor_sync(0xffffffffu, y0, 1);
        y1 += __shfl_xor_sync(0xffffffffu, y1, 1);
        y0 += __shfl_xor_sync(0xffffffffu, y0, 2);
        y1 += __shfl_xor_sync(0xffffffffu, y1, 2);
        // (neither factor is infinite, nor a sum by the first: a logit is infinite only if the formula's is)
        y0 = seen >> g & 1u ? y0 * ks * back : -INFINITY;
        y1 = seen >> (g + 8) & 1u ? y1 * ks * back : -INFINITY;
        float now = fmaxf(top, fmaxf(y0, y1));
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, d));
        if (now > top) {
          l *= fast_exp2(top - now);
          top = now;
        }
        const float under = top == -INFINITY ? 0.0f : top;
        const float p0 = fast_exp2(y0 - under), p1 = fast_exp2(y1 - under);
        float more = p0 + p1;            // lanes of one t hold the tokens once
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) more += __shfl_xor_sync(0xffffffffu, more, d);
        const float before = l;
        l += more;
        const float part = l == 0.0f ? 0.0f : __frcp_rn(l), keep = before * part, scaled = part * vs;
#pragma unroll
        for (int e = 0; e < 16; e++) o[e] *= keep;
        float w[4];
        w[0] = __shfl_sync(0xffffffffu, p0, 8 * tt) * scaled;
        w[1] = __shfl_sync(0xffffffffu, p0, 8 * tt + 4) * scaled;
        w[2] = __shfl_sync(0xffffffffu, p1, 8 * tt) * scaled;
        w[3] = __shfl_sync(0xffffffffu, p1, 8 * tt + 4) * scaled;
        const uint32_t at = seen >> (2 * tt);
#pragma unroll
        for (int f = 0; f < 16; f++) {            // features 16 (f / 2) + 8 (f % 2) + g
          const uint32_t v0 = x[4 * (f >> 1) + 2 * (f & 1)], v1 = x[4 * (f >> 1) + 2 * (f & 1) + 1];
          if (at & 1u) o[f] = fmaf(w[0], lo(v0), o[f]);
          if (at & 2u) o[f] = fmaf(w[1], hi(v0), o[f]);
          if (at & 256u) o[f] = fmaf(w[2], lo(v1), o[f]);
          if (at & 512u) o[f] = fmaf(w[3], hi(v1), o[f]);
        }
      }
    }
    // lanes of one g hold a feature's tokens
#pragma unroll
    for (int e = 0; e < 16; e++) {
      o[e] += __shfl_xor_sync(0xffffffffu, o[e], 1);
      o[e] += __shfl_xor_sync(0xffffffffu, o[e], 2);
      if (tt == (e & 3)) sm.o[warp][8 * e + g] = o[e];
    }
    if (lane == 0) {
      sm.top[warp] = top;
      sm.sum[warp] = l;
    }
    __syncthreads();
    if (threadIdx.x < kD) {
      float all = -INFINITY, sum = 0.0f, y = 0.0f;
#pragma unroll
      for (int w = 0; w < kT8Walkers; w++) all = fmaxf(all, sm.top[w]);
#pragma unroll
      for (int w = 0; w < kT8Walkers; w++) sum = fmaf(sm.sum[w], sm.top[w] == all ? 1.0f : fast_exp2(sm.top[w] - all), sum);
#pragma unroll
      for (int w = 0; w < kT8Walkers; w++)
        if (sm.top[w] > -INFINITY || sm.sum[w] != 0.0f)
          y = fmaf(sm.o[w][threadIdx.x], __fdiv_rn(sm.sum[w] * (sm.top[w] == all ? 1.0f : fast_exp2(sm.top[w] - all)), sum), y);
      if (sum == 0.0f) y = __uint_as_float(0x7fffffffu);         // no logit above -Inf
      reinterpret_cast<uint16_t*>(out)[threadIdx.x] = float_elem<ELEM>(in_range<ELEM>(y));
    }
  }
};

// ---- the call's plan, the same in every block ----
// A unit is a (request, KV head, 128 query rows); its steps of 128 tokens follow one
// another, and the units of all requests form one sequence that is cut into ranges, one a
// CTA. For the cuts a unit counts `turn` steps more than it has, ahead of its first: what a CTA
// spends on results, queries and first maxima between two units, at most a quarter of its range.
struct TreePlan {
  int pre[kMaxCallReq + 1], units[kMaxCallReq + 1];      // steps, units of the requests before
  int N[kMaxCallReq], M[kMaxCallReq], slot[kMaxCallReq];
};
struct TreeTotal {
  int steps, units;
  __device__ __forceinline__ int ctas(int grid) const { return max(1, min(grid, steps)); }
  __device__ __forceinline__ int turn(int grid) const { return min(kT8Turn, steps / (4 * grid)); }
};
__device__ __forceinline__ int unit_rows(int M, int G) { return (M * G + kT8Rows - 1) / kT8Rows; }
__device__ __forceinline__ TreeTotal make_plan(const Cache8View& c, const Tree8Args& a, TreePlan& p, int2* scan) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  TreeTotal carry{0, 0};
  for (int base = 0; base < a.n_req; base += blockDim.x) {
    const int i = base + threadIdx.x;
    int cost = 0, units = 0;
    if (i < a.n_req) {
      const TreeReq r = tree_req(c, a, i);
      p.N[i] = r.N;
      p.M[i] = r.M;
      p.slot[i] = r.slot;
      if (r.M > 0) {
        const TreeTiles t = tree_tiles(r.N, r.M, c.T, a.window, a.sinks);
        units = c.hkv * unit_rows(r.M, c.G);
        cost = units * ((t.places + kT8Step - 1) / kT8Step);
      }
    }
    int x = cost, y = units;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x2 = __shfl_up_sync(0xffffffffu, x, d), y2 = __shfl_up_sync(0xffffffffu, y, d);
      if (lane >= d) {
        x += x2;
        y += y2;
      }
    }
    if (lane == 31) scan[warp] = make_int2(x, y);
    __syncthreads();
    const int2 sum = lane < warps ? scan[lane] : make_int2(0, 0);
    const int before = carry.steps + __reduce_add_sync(0xffffffffu, lane < warp ? sum.x : 0);
    const int units_before = carry.units + __reduce_add_sync(0xffffffffu, lane < warp ? sum.y : 0);
    carry.steps += __reduce_add_sync(0xffffffffu, sum.x);
    carry.units += __reduce_add_sync(0xffffffffu, sum.y);
    if (i < a.n_req) {
      p.pre[i] = before + x - cost;
      p.units[i] = units_before + y - units;
    }
    if (threadIdx.x == 0) {
      p.pre[min(base + (int)blockDim.x, a.n_req)] = carry.steps;
      p.units[min(base + (int)blockDim.x, a.n_req)] = carry.units;
    }
    __syncthreads();
  }
  return carry;
}
__device__ __forceinline__ int range_start(int total, int cta, int ctas) {       // floor(total * cta / ctas)
  const int q = total / ctas;
  return q * cta + (total - q * ctas) * cta / ctas;
}
__device__ __forceinline__ int range_of(int total, int pos, int ctas) {     // the CTA whose range holds pos
  int x = min((int)((float)pos * ((float)ctas / (float)total)), ctas - 1);   // within a few of it
  while (x > 0 && (long long)x * total > (long long)pos * ctas + (ctas - 1)) x--;
  while (x < ctas - 1 && (long long)(x + 1) * total <= (long long)pos * ctas + (ctas - 1)) x++;
  return x;
}
// The first step at or behind a cut, which counts turns.
__device__ __forceinline__ int step_at(const Cache8View& c, const Tree8Args& a, const TreePlan& p, const TreeTotal& all, int cut, int turn) {
  if (turn == 0) return cut;
  if (cut >= all.steps + turn * all.units) return all.steps;
  int i = 0, end = a.n_req;
#pragma unroll 1
  while (end - i > 1) {        // the last request that starts at or before the cut
    const int mid = (i + end) >> 1;
    if (p.pre[mid] + turn * p.units[mid] <= cut) i = mid; else end = mid;
  }
  const int per = (tree_tiles(p.N[i], p.M[i], c.T, a.window, a.sinks).places + kT8Step - 1) / kT8Step;
  const int x = cut - p.pre[i] - turn * p.units[i], unit = x / (per + turn);
  return p.pre[i] + unit * per + max(x - unit * (per + turn) - turn, 0);
}

// Part of a unit in a CTA's range: steps s0 .. s0 + n - 1 of `per`.
struct TreeItem {
  int i, h, t, s0, n, per, N, M, slot;
  TreeTiles tiles;
};
__device__ __forceinline__ TreeItem tree_item(const Cache8View& c, const Tree8Args& a, const TreePlan& p, int pos, int hi) {
  TreeItem it;
  int i = 0, end = a.n_req;
#pragma unroll 1
  while (end - i > 1) {        // the last request that starts at or before pos
    const int mid = (i + end) >> 1;
    if (p.pre[mid] <= pos) i = mid; else end = mid;
  }
  it.i = i;
  it.N = p.N[i];
  it.M = p.M[i];
  it.slot = p.slot[i];
  it.tiles = tree_tiles(it.N, it.M, c.T, a.window, a.sinks);
  it.per = (it.tiles.places + kT8Step - 1) / kT8Step;
  const int x = pos - p.pre[i], unit = x / it.per, rt = unit_rows(it.M, c.G);
  it.s0 = x - unit * it.per;
  it.h = unit / rt;
  it.t = unit - it.h * rt;
  it.n = min(it.per - it.s0, hi - pos);
  return it;
}

// What a CTA leaves for the second kernel: whether it begins a unit that others go on with (1;
// request, KV head, rows, the last of those others), and whether rows of whole units came out
// infinite or NaN (2; its steps).
struct __align__(16) TreeRecord {
  int flags, i, h, t, M, last, lo, hi;
};

// What is known of a tile. kind: codes of a block that every node sees all of (0), other codes (1),
// the tail's (2), drafts (3), none (4).
struct TileDesc {
  const uint8_t* src;       // (drafts: K)
  float ks;
  union {
    float lv;       // log2 of V's scale
    int req_head;   // kinds 2 and 3, on the way: request << 12 | KV head
  };
  int pos0, kind;   // first token, first draft
  int n;            // kinds 2 and 3: valid tokens
  const uint8_t* vsrc;
};
// What the softmax has to know of it; kind as above.
struct TileMeta {
  float ks, lv;
  int pos0, kind;
};

struct TreeSmem {
  TileDesc desc[kT8Descs][kT8Step];
  unsigned there[2 * kT8Descs];        // places of a step that hold a tile (the products are behind the conversion)
  TileMeta meta[kT8Metas][kT8Step];    // (K of step j comes when the softmax has read that of step j - 5)
  // of a step's tiles from `elems` on: K's powers of two, V's exponents (there with V, not with S)
  alignas(16) uint16_t kexp[kT8Metas][kT8Step / 2][kSub];
  alignas(16) float vexp[kT8Slots][kT8Step / 2][kSub];
  TreePlan plan;
  int parents[kMaxNodes];
  float2 pair[2][2][kT8Rows];      // what the two warps of a row tell each other
  int2 scan[32];
  int runs[4];                     // ends of items of the products
  int begun[4];                    // the unit that the CTA's last item begins: 1, request, KV head, rows
  int bad, any_taken;
  int2 taken[16][4];               // of a step's tiles of 16 bits: first token, kind << 16 | tokens whose V was taken out
  // K, V of a step there, no longer needed; S, P, P V of a step there, queries there (two of
  // each, of P V four: a wait is for the last of them, the one before in its place long over);
  // drain
  uint64_t bar[4 * kT8Slots + 11];
  uint64_t rfull[2][kT8Ring], rfree[2][kT8Ring];      // copies of K, of V codes
  uint64_t dfull[4], dfree[4];     // batches of descriptors
  uint32_t taddr;
  int fail;
};
constexpr int kT8OffV = kT8Slots * kT8Slot, kT8OffRing = 2 * kT8Slots * kT8Slot;
constexpr int kT8OffSmem = kT8OffRing + 2 * kT8Ring * kT8Entry;
constexpr int kT8Smem = 1024 + kT8OffSmem + (int)sizeof(TreeSmem);
static_assert(kT8Smem <= 232448, "a block's shared memory");

__device__ __forceinline__ void stmatrix4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void stmatrix4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"r"(addr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void lds128(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// Largest finite magnitude of a lane's bf16 values, as bits: with the exponent's last bit added to
// the bits of the magnitudes, infinities and NaN are negative numbers of 16 bits.
template <int N>
__device__ __forceinline__ uint32_t amax_bits(const uint32_t (&x)[N]) {
  uint32_t m = 0x00800080u;
#pragma unroll
  for (int f = 0; f < N; f++) asm("max.s16x2 %0, %0, %1;\n" : "+r"(m) : "r"((x[f] & 0x7fff7fffu) + 0x00800080u));
  return max(m & 0xffffu, m >> 16) - 0x80u;
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

// Place x of a CTA whose range begins at step lo, but for its page's scales.
__device__ __forceinline__ TileDesc describe_tile(const Cache8View& c, const Tree8Args& a, const TreePlan& plan, int lo, int x,
                                                  const float2*& scales) {
  const int pos = lo + x / kT8Step;
  const TreeItem it = tree_item(c, a, plan, pos, pos + 1);
  x = kT8Step * it.s0 + x % kT8Step;
  TileDesc d{nullptr, kLogitScale, {0.0f}, 0, 4, 0, nullptr};
  const bool own = x >= it.tiles.elems;
  if (own ? x & 1 : x >= it.tiles.codes) return d;
  if (own) x = it.tiles.codes + ((x - it.tiles.elems) >> 1);
  if (x < it.tiles.tails) {
    const int tile = it.tiles.tile(x), per = __ffs(c.T) - 5;      // log2 of a block's tiles
    d.pos0 = tile * kSub;
    int page = c.table[(size_t)it.slot * c.width + (tile >> per)];
    if ((unsigned)page >= (unsigned)c.n_pages) {
      c.latch(DKV_ERR_CHECK, it.i);
      page = 0;
    }
    scales = reinterpret_cast<const float2*>(c.scales + 2 * ((size_t)page * c.hkv + it.h));
    d.src = c.pages + c.page_head(page, it.h) + (size_t)(tile & ((1 << per) - 1)) * (2 * kTile);
    d.kind = own ? 1 : 0;
  } else if (x < it.tiles.stored) {
    const int tile = it.tiles.tile(x);
    d.req_head = it.i << 12 | it.h;
    d.pos0 = tile * kSub;
    d.src = c.tail + c.tail_head(it.slot, it.h) + (size_t)(tile - it.tiles.full) * (4 * kTile);
    d.kind = 2;
  } else if (x < it.tiles.count) {
    d.req_head = it.i << 12 | it.h;
    d.pos0 = (x - it.tiles.stored) * kSub;
    d.src = a.k + ((long long)it.i * a.max_nodes + d.pos0) * a.ks + it.h * (2 * kD);
    d.kind = 3;
  }
  return d;
}

// ---- powers of two: K of each bf16 token and V of each token of 16 bits, or of a block that some node
// sees a part of only, are divided by one of their own, which brings the token's largest value to
// [128, 256). (One for the tile, or the block's scale: what a row does not see would set the power for
// what it does. A sibling's V 2^30 above the others left rows that do
// not see it wrong by 25 %, one 2^60 above left zeros. V in fp16 as it is: the weights of codes, which
// carry their scale, lie 2^-20 below and lose their bits beside a heavier token of small V in the same
// step; 64 codes beside a draft with V of 1e-4 were off by 7 times the bound of rounded weights.) ----
// Largest finite magnitudes so far of the low and of the high values: with the exponent's last
// bit added to the bits of the magnitudes, infinities and NaN are negative numbers of 16 bits.
template <int ELEM>
constexpr uint32_t kT8Bias = ELEM == DKV_F16 ? 0x0400u : 0x0080u;
__device__ __forceinline__ uint32_t max_s16x2(uint32_t a, uint32_t b) {
  uint32_t m;
  asm("max.s16x2 %0, %1, %2;\n" : "=r"(m) : "r"(a), "r"(b));
  return m;
}
template <int ELEM>
__device__ __forceinline__ uint32_t top_pair(uint32_t m, uint32_t w) {
  return max_s16x2(m, (w & 0x7fff7fffu) + kT8Bias<ELEM> * 0x10001u);
}
__device__ __forceinline__ uint32_t swap_halves(uint32_t x) { return prmt(x, x, 0x1032u); }
// The exponent for one of the two. Not below -112: results come back by that and kT8Up; the smallest
// normal V then comes to 2^-14, where fp16 keeps what bf16 holds.
template <int ELEM>
__device__ __forceinline__ int exp_of(uint32_t top) {
  const uint32_t x = __float_as_uint(elem_float<ELEM>((uint16_t)((top & 0xffffu) - kT8Bias<ELEM>)));
  return max(ELEM == DKV_F16 ? -29 : -112, (int)(x >> 23) - (127 + 7));
}
// What brings two values there, by 2^-lo and 2^-hi: bf16 in fp32; fp16 in two steps, since one
// factor of fp16 is 2^15 at most (the first of two that enlarge is exact).
struct Factors {
  uint32_t a, b;
};
template <int ELEM>
__device__ __forceinline__ Factors factors(int lo, int hi) {
  if (ELEM == DKV_BF16) return Factors{__float_as_uint(pow2(-lo)), __float_as_uint(pow2(-hi))};
  const int l1 = min(-lo, 14), h1 = min(-hi, 14), l2 = min(-lo - l1, 15), h2 = min(-hi - h1, 15);
  return Factors{(uint32_t)(15 + l1) << 10 | (uint32_t)(15 + h1) << 26, (uint32_t)(15 + l2) << 10 | (uint32_t)(15 + h2) << 26};
}
template <int ELEM>
__device__ __forceinline__ uint32_t half_of(uint32_t w, const Factors& f) {
  if (ELEM == DKV_BF16) return pack_half2(lo_elem<DKV_BF16>(w) * __uint_as_float(f.a), hi_elem<DKV_BF16>(w) * __uint_as_float(f.b));
  uint32_t x;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(x) : "r"(w), "r"(f.a));
  asm("mul.rn.f16x2 %0, %0, %1;\n" : "+r"(x) : "r"(f.b));
  return x;
}
// What the softmax has to know of the 16 tokens: K's powers of two (bf16), V's exponents.
struct TileExps {
  uint16_t* k;
  float* v;
};
__device__ __forceinline__ void put_exp(const TileExps& e, bool v, int token, int ex) {
  if (v) e.v[token] = (float)ex;
  else e.k[token] = (uint16_t)((127 + ex) << 7);
}
// V that is not finite would meet the weights of rows that do not see it, and 0 times it is not 0:
// it becomes 0 where it lies in shared memory, and whoever sees its token (bits of 16) is computed
// again. (Out of the way: instructions fetched with the usual case cost it 5%.)
template <int ELEM>
__device__ __noinline__ uint32_t take_out(uint8_t* src, bool draft, int n) {
  constexpr uint32_t kExp = ELEM == DKV_F16 ? 0x0400u : 0x0080u;
  const int lane = threadIdx.x & 31;
  uint32_t bits = 0;
#pragma unroll 1
  for (int e = 0; e < 32; e++) {             // word e % 4 of the lane's 16 bytes of 512
    uint32_t* at = reinterpret_cast<uint32_t*>(src + 512 * (e >> 2) + 16 * lane) + (e & 3);
    const int token = draft ? 2 * (e >> 2) + (lane >> 4) : 2 * (lane & 3) + 8 * (e & 1);
    uint32_t w = *at;
    if (((w & 0x7fffu) + kExp) & 0x8000u) {
      w &= 0xffff0000u;
      bits |= 1u << token;
    }
    if (((w >> 16 & 0x7fffu) + kExp) & 0x8000u) {
      w &= 0xffffu;
      bits |= 1u << (draft ? token : token + 1);
    }
    *at = w;
  }
  __syncwarp();
  return __reduce_or_sync(0xffffffffu, bits) & below(n);
}
// A tile of the tail, or of codes (FMT: what they are read as; lv: log2 of V's scale), as fp16 operands,
// of which n tokens are valid; at: the lane's row of the first four matrices. Returns the tokens of the
// tail whose V has values that are not finite. Two passes over the
// lane's 16 bytes of every m-step in short loops: this code runs once or twice a unit and comes from
// far (unrolled, all eight m-steps at once: 59.9 us for the window, 57.3 so).
template <int FMT, bool CODES, int CODE>
__device__ __noinline__ uint32_t put_tile(uint8_t* src, bool v, int n, uint32_t at, TileExps exps, float lv) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const bool scaled = v || FMT == DKV_BF16;         // (K in fp16 stays as it is)
  // The four 8 x 8 matrices of m-step f, of K the first eight features' first: even words are of token
  // g (K) or tokens 2t and 2t + 1 (V, low and high halves), odd ones of those eight tokens on. What
  // lies behind the valid tokens becomes 0 (0 times what it may hold is not).
  const uint32_t valid_a = v ? (2 * t < n ? 0xffffu : 0u) | (2 * t + 1 < n ? 0xffff0000u : 0u) : g < n ? 0xffffffffu : 0u;
  const uint32_t valid_b = v ? (2 * t + 8 < n ? 0xffffu : 0u) | (2 * t + 9 < n ? 0xffff0000u : 0u) : g + 8 < n ? 0xffffffffu : 0u;
  auto load = [&](int f) {
    uint4 y;
    if (CODES) {
      const uint2 w = *reinterpret_cast<const uint2*>(src + 512 * (f >> 1) + 16 * lane + 8 * (f & 1));
      code_halves<CODE>(w.x, y.x, y.y);
      code_halves<CODE>(w.y, y.z, y.w);
    } else {
      y = *reinterpret_cast<const uint4*>(src + 512 * f + 16 * lane);
    }
    return make_uint4(y.x & valid_a, (v ? y.y : y.z) & valid_b, (v ? y.z : y.y) & valid_a, y.w & valid_b);
  };
  uint32_t a = 0, b = 0, out = 0;
#pragma unroll 1
  while (scaled) {
    uint32_t acc = 0;
    a = b = kT8Bias<FMT> * 0x10001u;
#pragma unroll 2
    for (int f = 0; f < 8; f++) {
      const uint4 x = load(f);
      a = top_pair<FMT>(top_pair<FMT>(a, x.x), x.z);
      b = top_pair<FMT>(top_pair<FMT>(b, x.y), x.w);
      find_not_finite<FMT>(acc, x.x);
      find_not_finite<FMT>(acc, x.y);
      find_not_finite<FMT>(acc, x.z);
      find_not_finite<FMT>(acc, x.w);
    }
    if (CODES || !v || __builtin_expect(!__any_sync(0xffffffffu, found_not_finite(acc)), 1)) break;
    out = take_out<FMT>(src, false, n);
  }
  Factors fa{}, fb{};
  if (scaled) {
    if (!v) {
      a = max_s16x2(a, swap_halves(a));
      b = max_s16x2(b, swap_halves(b));
    }
#pragma unroll 1
    for (int d = v ? 4 : 1; d < (v ? 32 : 4); d <<= 1) {
      a = max_s16x2(a, __shfl_xor_sync(0xffffffffu, a, d));
      b = max_s16x2(b, __shfl_xor_sync(0xffffffffu, b, d));
    }
    const int a0 = exp_of<FMT>(a), a1 = exp_of<FMT>(a >> 16), b0 = exp_of<FMT>(b), b1 = exp_of<FMT>(b >> 16);
    if (v ? g == 0 : t == 0) {
      // (a code is 0 or at least 2^-9; a token of zeros counts as one of the smallest scale)
      auto put = [&](int token, int ex) {
        if (CODES) exps.v[token] = ex < -16 ? -100.0f : (float)ex + lv;
        else put_exp(exps, v, token, ex);
      };
      put(v ? 2 * t : g, a0);
      put(v ? 2 * t + 8 : g + 8, b0);
      if (v) {
        put(2 * t + 1, a1);
        put(2 * t + 9, b1);
      }
    }
    fa = factors<FMT>(a0, a1);
    fb = factors<FMT>(b0, b1);
  } else if (CODES && lane < kSub) {
    put_exp(exps, false, lane, 0);
  }
#pragma unroll 2
  for (int f = 0; f < 8; f++) {
    uint4 x = load(f);
    if (scaled) x = make_uint4(half_of<FMT>(x.x, fa), half_of<FMT>(x.y, fb), half_of<FMT>(x.z, fa), half_of<FMT>(x.w, fb));
    if (!v) stmatrix4((at + (f >> 2) * 16384) ^ ((f & 3) << 5), x.x, x.z, x.y, x.w);
    else stmatrix4(at + f * 2048, x.x, x.y, x.z, x.w);
  }
  return out;
}
// Drafts, whose rows of 256 bytes lie in shared memory: a lane half a row, 16 bytes at a time in an
// order that keeps eight lanes apart in the banks, there (where column y lies in the same banks for
// every row) and in the operand (where y xor the row does). K goes to its operand rows (to: row 0),
// V back to where it was, then once more with row r turned by r times 16 bytes, so that the same features of
// eight rows lie in different banks, and from there as transposed matrices (to: as for put_tail).
// (Both by words straight from the rows, eight lanes on a bank: a step of four draft tiles 4000
// cycles.)
template <int ELEM>
__device__ __noinline__ uint32_t put_drafts(uint8_t* rows, bool v, int n, uint32_t to, TileExps exps) {
  const int lane = threadIdx.x & 31, row = lane & 15, half = lane >> 4, r = row & 7;
  const bool scaled = v || ELEM == DKV_BF16;
  const uint32_t src = smem_u32(rows);
  // y -> column, such that r -> column and r -> column xor r are one to one
  const int turn = (r << 1 & 7) ^ (r & 4 ? 3 : 0);
  const uint32_t mine = src + row * (2 * kD) + 128 * half;
  auto load = [&](int y) {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (row < n) lds128(mine + ((y ^ turn) << 4), x.x, x.y, x.z, x.w);
    return x;
  };
  uint32_t top = 0, out = 0;
#pragma unroll 1
  while (scaled) {
    uint32_t acc = 0;
    top = kT8Bias<ELEM> * 0x10001u;
#pragma unroll 2
    for (int y = 0; y < 8; y++) {
      const uint4 x = load(y);
      top = top_pair<ELEM>(top_pair<ELEM>(top_pair<ELEM>(top_pair<ELEM>(top, x.x), x.y), x.z), x.w);
      find_not_finite<ELEM>(acc, x.x);
      find_not_finite<ELEM>(acc, x.y);
      find_not_finite<ELEM>(acc, x.z);
      find_not_finite<ELEM>(acc, x.w);
    }
    if (!v || __builtin_expect(!__any_sync(0xffffffffu, found_not_finite(acc)), 1)) break;
    out = take_out<ELEM>(rows, true, n);
  }
  Factors f{};
  if (scaled) {
    top = max_s16x2(top, swap_halves(top));
    const int ex = exp_of<ELEM>(max_s16x2(top, __shfl_xor_sync(0xffffffffu, top, 16)));
    if (half == 0) put_exp(exps, v, row, ex);
    f = factors<ELEM>(ex, ex);
  }
#pragma unroll 2
  for (int y = 0; y < 8; y++) {
    uint4 x = load(y);
    if (scaled) x = make_uint4(half_of<ELEM>(x.x, f), half_of<ELEM>(x.y, f), half_of<ELEM>(x.z, f), half_of<ELEM>(x.w, f));
    sts128(v ? mine + ((y ^ turn) << 4) : to + half * 16384 + row * 128 + ((y ^ turn ^ r) << 4), x.x, x.y, x.z, x.w);
  }
  if (v) {
    const int c = lane & 15;
    uint32_t x[32];
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 8; e++) lds128(src + (2 * e + half) * (2 * kD) + 16 * c, x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 8; e++)
      sts128(src + (2 * e + half) * (2 * kD) + (((c + 2 * e + half) & 15) << 4), x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
    __syncwarp();
    const int at = (lane & 7) + 8 * half;      // matrices: features 0 .. 7, 8 .. 15 of rows 0 .. 7, of rows 8 .. 15
#pragma unroll 2
    for (int m = 0; m < 8; m++) {
      uint32_t w[4];
      ldmatrix_x4(w, src + at * (2 * kD) + (((2 * m + (lane >> 3 & 1) + at) & 15) << 4));
      stmatrix4_trans(to + m * 2048, w[0], w[1], w[2], w[3]);
    }
  }
  return out;
}

template <int ELEM, int CODE>
__global__ void __launch_bounds__(kT8Threads, 1) k_tree8(const __grid_constant__ Cache8View c, const __grid_constant__ Tree8Args a, int part_rows,
                                                         int* plan, TreeRecord* records) {
  pdl_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  // (an offset, not a rounded pointer: the compiler still knows that this is shared memory)
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  TreeSmem& sm = *reinterpret_cast<TreeSmem*>(smem + kT8OffSmem);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, G = c.G;
  // step j of the CTA: K and V in slot j % kT8Slots, S and P in place j & 1
  const uint32_t b0 = smem_u32(sm.bar);
  auto kfull = [&](int s) { return b0 + 8u * s; };
  auto kfree = [&](int s) { return b0 + 8u * (kT8Slots + s); };
  auto vfull = [&](int s) { return b0 + 8u * (2 * kT8Slots + s); };
  auto vfree = [&](int s) { return b0 + 8u * (3 * kT8Slots + s); };
  auto sfull = [&](int s) { return b0 + 8u * (4 * kT8Slots + s); };
  auto pfull = [&](int s) { return b0 + 8u * (4 * kT8Slots + 2 + s); };
  auto qfull = [&](int s) { return b0 + 8u * (4 * kT8Slots + 4 + s); };
  auto pvdone = [&](int s) { return b0 + 8u * (4 * kT8Slots + 6 + s); };
  const uint32_t drain = b0 + 8u * (4 * kT8Slots + 10);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kT8Slots; s++) {
      mbar_init(kfull(s), 4);
      mbar_init(kfree(s), 1);
      mbar_init(vfull(s), 4);
      mbar_init(vfree(s), 1);
    }
    for (int s = 0; s < 2; s++) {
      mbar_init(sfull(s), 1);
      mbar_init(pfull(s), 8);
      mbar_init(qfull(s), 8);
    }
    for (int s = 0; s < 4; s++) mbar_init(pvdone(s), 1);
    mbar_init(drain, 1);
    for (int s = 0; s < 4; s++) {
      mbar_init(smem_u32(&sm.dfull[s]), 1);
      mbar_init(smem_u32(&sm.dfree[s]), 10);
    }
    for (int s = 0; s < 2 * kT8Ring; s++) {
      mbar_init(smem_u32(&sm.rfull[0][0]) + 8 * s, 1);
      mbar_init(smem_u32(&sm.rfree[0][0]) + 8 * s, 4);
    }
    sm.fail = sm.bad = sm.any_taken = sm.begun[0] = 0;
    fence_mbar_init();
  }
  if (warp == 16) tmem_alloc(smem_u32(&sm.taddr), 512);
  pdl_wait();
  // an error of an earlier call (its load is in flight with the plan's)
  const int halted = threadIdx.x == 0 ? *(volatile int*)c.status : 0;
  const TreeTotal all = make_plan(c, a, sm.plan, sm.scan);
  tc_fence_before();
  const bool stopped = __syncthreads_or(halted);
  tc_fence_after();
  if (blockIdx.x == 0)           // for the second kernel
    for (int i = threadIdx.x; i <= a.n_req; i += blockDim.x) plan[i] = sm.plan.pre[i];
  const int ctas = all.ctas(gridDim.x), turn = all.turn(gridDim.x);
  int lo = 0, hi = 0;
  if (all.steps > 0 && (int)blockIdx.x < ctas) {
    const int mine = step_at(c, a, sm.plan, all, range_start(all.steps + turn * all.units, blockIdx.x + (lane & 1), ctas), turn);
    lo = __shfl_sync(0xffffffffu, mine, 0);
    hi = __shfl_sync(0xffffffffu, mine, 1);
  }
  if (stopped || lo == hi) {
    if (threadIdx.x == 0) records[blockIdx.x] = TreeRecord{};
    if (warp == 16) tmem_dealloc(__shfl_sync(0xffffffffu, sm.taddr, 0), 512);
    return;
  }
  const uint32_t tbase = __shfl_sync(0xffffffffu, sm.taddr, 0);
  // O, two S (and P over them), two Q
  const uint32_t t_o = tbase;
  auto t_s = [&](int s) { return tbase + 128u + 128u * s; };
  auto t_q = [&](int s) { return tbase + 384u + 64u * s; };
  // Bounded: by the products' warp, which gives up after a second without any, and by its own
  // attempts; then the block's other waits give up, too. The same for every lane. (Short:
  // the kernel's hot code has to fit the instruction caches.)
  auto wait = [&](uint32_t bar, int phase) {
#pragma unroll 1
    for (int n = 1 << 25; !__all_sync(0xffffffffu, mbar_try_wait(bar, phase & 1)); n--)
      if (n == 0 || ((n & 255) == 0 && *(volatile int*)&sm.fail)) {
        *(volatile int*)&sm.fail = 1;
        return false;
      }
    return true;
  };
  bool ok = true;

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kT8RegsMany));
    // ---- softmax: a thread per query row and part of a step, so two warps for 32 rows,
    // which agree on the rows' maxima ----
    const int part = warp >> 2, lg = warp & 3, r = 32 * lg + lane, pair_bar = 4 + lg;
    const uint32_t tl = (uint32_t)(32 * lg) << 16;
    Node node;
    TreeItem it = tree_item(c, a, sm.plan, lo, hi);
    int told = 0;              // place of `pair` to use next
    auto row_of = [&](const TreeItem& x) { return x.t * kT8Rows + r; };
    auto real_of = [&](const TreeItem& x) { return row_of(x) < x.M * G; };
    auto busy_of = [&](const TreeItem& x) { return 32 * lg + x.t * kT8Rows < x.M * G; };
    auto q_of = [&](const TreeItem& x) {         // 64 features of the row; the other warp has the others
      const int row = row_of(x), m = row / G;
      return a.q + ((long long)x.i * a.max_nodes + m) * a.qs + ((size_t)x.h * G + (row - m * G)) * (2 * kD) + 128 * part;
    };
    // The queries of item n (bf16: over a power of two of their row, which is returned).
    auto put_row = [&](const TreeItem& x, int n) {
      float scale = 1.0f;
      if (busy_of(x)) {
        const uint4* src = reinterpret_cast<const uint4*>(q_of(x));
        const bool real = real_of(x);
        uint4 qr[8];
#pragma unroll
        for (int e = 0; e < 8; e++) qr[e] = real ? src[e] : make_uint4(0, 0, 0, 0);
        float inv = 1.0f;
        if (ELEM == DKV_BF16) {
          uint32_t x[32];
#pragma unroll
          for (int e = 0; e < 8; e++) {
            x[4 * e] = qr[e].x;
            x[4 * e + 1] = qr[e].y;
            x[4 * e + 2] = qr[e].z;
            x[4 * e + 3] = qr[e].w;
          }
          const float mine = __uint_as_float(amax_bits(x));
          sm.pair[told][part][r].x = mine;
          named_sync(pair_bar, 64);
          const uint32_t most = max(__float_as_uint(mine), __float_as_uint(sm.pair[told][part ^ 1][r].x));
          told ^= 1;
          const int ex = most ? max(-126, min(126, (int)(most >> 7) - 127)) : 0;
          inv = pow2(-ex);
          scale = pow2(ex);
        }
#pragma unroll
        for (int e = 0; e < 2; e++) {
          uint32_t q[16];
#pragma unroll
          for (int y = 0; y < 4; y++) {
            q[4 * y] = qr[4 * e + y].x;
            q[4 * y + 1] = qr[4 * e + y].y;
            q[4 * y + 2] = qr[4 * e + y].z;
            q[4 * y + 3] = qr[4 * e + y].w;
          }
          if (ELEM == DKV_BF16) {
#pragma unroll
            for (int y = 0; y < 16; y++) q[y] = half_of_bf16(q[y], inv);
          }
          tmem_st16(t_q(n & 1) + tl + 32 * part + 16 * e, q);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(qfull(n & 1));
      return scale;
    };
    float scale = put_row(it, 0);
    int last_i = -1, last_t = -1;
    for (int pos = lo, j = 0, item = 0;; item++) {
      const int row = row_of(it), m = row / G;
      const bool real = real_of(it), busy = busy_of(it);
      if (it.i != last_i || it.t != last_t) {      // the same for all eight warps
        if (a.parents && it.i != last_i) {
          named_sync(1, 256);
          if (part == 1 && r < it.M) sm.parents[r] = a.parents[(size_t)it.i * a.max_nodes + r];
          named_sync(1, 256);
        }
        if (busy) node = node_of(c, a, a.parents ? sm.parents : nullptr, it.i, it.N, real ? m : -1);
        last_i = it.i;
        last_t = it.t;
      }
      pos += it.n;
      TreeItem then = it;
      if (pos < hi) {
        then = tree_item(c, a, sm.plan, pos, hi);
        if (real_of(then)) asm volatile("prefetch.global.L2 [%0];\n" ::"l"(q_of(then)));
      }
      float mx = -INFINITY, u = -INFINITY, l = 0.0f;
      const int end = j + it.n;
      bool first = true, raise = true;
      // The rows' running maxima take in yt, xt of a step over both parts.
      auto raise_to = [&](float yt, float xt, int j, bool first) {
        sm.pair[told][part][r] = make_float2(yt, xt);
        named_sync(pair_bar, 64);
        const float2 other = sm.pair[told][part ^ 1][r];
        told ^= 1;
        const float nu = fmaxf(u, fmaxf(yt, other.x)), nm = fmaxf(mx, fmaxf(xt, other.y));
        l *= nu == -INFINITY ? 1.0f : fast_exp2(u - nu);
        if (!first) {        // O is still once the last product is done
          ok = wait(pvdone((j - 1) & 3), (j - 1) >> 2) && ok;
          tc_fence_after();
          const float fo = nm == -INFINITY ? 1.0f : fast_exp2(mx - nm);
#pragma unroll 1
          for (int q = 0; q < 4; q++) {
            float o[16];
            tmem_ld16_nowait(t_o + tl + 64 * part + 16 * q, o);
            tmem_wait_ld();
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; e++) {
              asm volatile("" : "+f"(o[e]));
              w[e] = __float_as_uint(o[e] * fo);
            }
            tmem_st16(t_o + tl + 64 * part + 16 * q, w);
          }
        }
        mx = nm;
        u = nu;
        raise = __any_sync(0xffffffffu, real && u == -INFINITY);      // a row that has seen nothing so far
      };
      for (; j < end; j++) {
        // (after a wait that gave up the warps walk on, through the same barriers)
        ok = wait(sfull(j & 1), j >> 1) && ok;
        tc_fence_after();
        if (busy) {
          const uint32_t ts = t_s(j & 1) + tl + 64 * part;
          const TileMeta* meta = sm.meta[j & (kT8Metas - 1)] + 4 * part;
          float sum = 0.0f;
          if (kT8Step * (it.s0 + it.n - (end - j)) + 4 * part >= it.tiles.elems) {
            // two tiles whose tokens have exponents of their own
            float y[2][16];
            bool is[2];
            auto vexp = [&](int b, int e) { return *reinterpret_cast<const ulonglong2*>(&sm.vexp[j & 1][2 * part + b][4 * e]); };
            tmem_ld16_nowait(ts, y[0]);
            tmem_ld16_nowait(ts + 32, y[1]);
            ok = wait(vfull(j & 1), j >> 1) && ok;      // (V of step j + 2 waits for these weights)
            tmem_wait_ld();
#pragma unroll
            for (int b = 0; b < 2; b++) {
              const TileMeta d = meta[2 * b];
              is[b] = d.kind != 4;
              if (!is[b]) continue;
              const int w = d.pos0 >> 5;
              const uint32_t see = !real ? 0xffffu : d.kind != 3 ? sees_stored(a, it.N, node.depth, d.pos0)
                                   : (w == 0 ? node.over[0] : w == 1 ? node.over[1] : w == 2 ? node.over[2] : node.over[3]) >> (d.pos0 & 31) & 0xffffu;
              const float f = d.ks * scale;
              const uint4* kp = reinterpret_cast<const uint4*>(sm.kexp[j & (kT8Metas - 1)][2 * part + b]);      // (bf16)
#pragma unroll
              for (int e = 0; e < 2; e++) {
                const uint4 x = ELEM == DKV_BF16 ? kp[e] : make_uint4(0, 0, 0, 0);
                const uint32_t k[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int z = 0; z < 8; z++) {
                  float& o = y[b][8 * e + z];
                  asm volatile("" : "+f"(o));
                  o *= ELEM == DKV_BF16 ? f * __uint_as_float(z & 1 ? k[z >> 1] & 0xffff0000u : k[z >> 1] << 16) : f;
                }
              }
              if (!__all_sync(0xffffffffu, see == 0xffffu)) {
#pragma unroll
                for (int e = 0; e < 16; e++) y[b][e] = see & (1u << e) ? y[b][e] : -INFINITY;
              }
            }
#pragma unroll 1
            for (bool again = raise;; again = true) {
              if (again) {
                float yt = -INFINITY, xt = -INFINITY;
#pragma unroll
                for (int b = 0; b < 2; b++)
                  if (is[b]) {
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                      const ulonglong2 v = vexp(b, e >> 2);
#pragma unroll
                      for (int z = 0; z < 4; z++) {
                        asm volatile("" : "+f"(y[b][e + z]));
                        const unsigned long long v2 = z & 2 ? v.y : v.x;
                        yt = fmaxf(yt, y[b][e + z]);
                        xt = fmaxf(xt, y[b][e + z] + __uint_as_float((uint32_t)(z & 1 ? v2 >> 32 : v2)));
                      }
                    }
                  }
                raise_to(yt, xt, j, first);
              }
              const float ur = u == -INFINITY ? 0.0f : u, mr = kT8Up - (mx == -INFINITY ? 0.0f : mx);
              const uint64_t ur2 = f32x2(-ur, -ur), mr2 = f32x2(mr, mr);
              bool fits = true;
              uint64_t own = 0;         // probabilities under u: their exponentials by themselves
#pragma unroll
              for (int b = 0; b < 2; b++) {
                if (!is[b]) continue;
                uint64_t acc = 0;
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; e++) {
                  const ulonglong2 v = vexp(b, e >> 1);
                  const uint64_t y2 = f32x2(y[b][2 * e], y[b][2 * e + 1]), t = add_f32x2(y2, ur2);
                  const uint64_t x = add_f32x2(y2, add_f32x2(e & 1 ? v.y : v.x, mr2));
                  own = add_f32x2(own, f32x2(fast_exp2(__uint_as_float((uint32_t)t)), fast_exp2(__uint_as_float((uint32_t)(t >> 32)))));
                  const float w0 = fast_exp2(__uint_as_float((uint32_t)x)), w1 = fast_exp2(__uint_as_float((uint32_t)(x >> 32)));
                  acc = add_f32x2(acc, f32x2(w0, w1));
                  w[e] = pack_half2(w0, w1);
                }
                fits = fits && __uint_as_float((uint32_t)acc) + __uint_as_float((uint32_t)(acc >> 32)) <= kT8Most;
                tmem_st8(ts + 16 * b, w);
              }
              sum = __uint_as_float((uint32_t)own) + __uint_as_float((uint32_t)(own >> 32));
              fits = fits && sum <= kT8Sum;
              if (again || named_all(pair_bar, 64, fits || !real)) break;
            }
            l += sum;
          } else {
            float s[64];
            tmem_ld32_nowait(ts, s);
            tmem_ld32_nowait(ts + 32, s + 32);
            float f[4], lv[4];
            int kind[4];
#pragma unroll
            for (int b = 0; b < 4; b++) {
              const TileMeta d = meta[b];
              f[b] = d.ks * scale;
              lv[b] = d.lv;
              kind[b] = d.kind;
            }
            tmem_wait_ld();
            loaded32(s);
            loaded32(s + 32);
            // (every node sees all of what there is)
#pragma unroll
            for (int b = 1; b < 4; b++)
              if (kind[b]) {
#pragma unroll
                for (int e = 0; e < 16; e++) s[16 * b + e] = -INFINITY;
              }
            uint32_t p[32];
#pragma unroll 1
            for (bool again = raise;; again = true) {
              if (again) {
                // (the maxima are not to be taken ahead of the question)
#pragma unroll
                for (int e = 0; e < 64; e++) asm volatile("" : "+f"(s[e]));
                float yt = -INFINITY, xt = -INFINITY;
#pragma unroll
                for (int b = 0; b < 4; b++) {
                  float y0 = s[16 * b], y1 = s[16 * b + 1];
#pragma unroll
                  for (int e = 2; e < 16; e += 2) {
                    y0 = fmaxf(y0, s[16 * b + e]);
                    y1 = fmaxf(y1, s[16 * b + e + 1]);
                  }
                  y0 = fmaxf(y0, y1) * f[b];
                  yt = fmaxf(yt, y0);
                  xt = fmaxf(xt, y0 + lv[b]);
                }
                raise_to(yt, xt, j, first);
              }
              // weights 2^(x - m + kT8Up), to be rounded to fp16; their sum of a tile over
              // 2^(kT8Up + u - m) s_v is that of the probabilities under u, except where these
              // are so far apart that one of them may vanish
              const float ur = u == -INFINITY ? 0.0f : u, mr = kT8Up - (mx == -INFINITY ? 0.0f : mx);
              bool fits = true, far = false;
              sum = 0.0f;
#pragma unroll
              for (int b = 0; b < 4; b++) {
                const float up = lv[b] + mr;
                const uint64_t f2 = f32x2(f[b], f[b]), up2 = f32x2(up, up);
                uint64_t acc[2] = {0, 0};
#pragma unroll
                for (int e = 0; e < 8; e++) {
                  const uint64_t y = fma_f32x2(f32x2(s[16 * b + 2 * e], s[16 * b + 2 * e + 1]), f2, up2);
                  const float w0 = fast_exp2(__uint_as_float((uint32_t)y)), w1 = fast_exp2(__uint_as_float((uint32_t)(y >> 32)));
                  acc[e & 1] = add_f32x2(acc[e & 1], f32x2(w0, w1));
                  p[8 * b + e] = pack_half2(w0, w1);
                }
                acc[0] = add_f32x2(acc[0], acc[1]);
                const float tile = __uint_as_float((uint32_t)acc[0]) + __uint_as_float((uint32_t)(acc[0] >> 32));
                const float back = up + ur;
                sum = fmaf(tile, fast_exp2(-back), sum);
                fits = fits && tile <= kT8Most;
                far = far || !(fabsf(back) <= kT8Far);      // (these rows take the longer way every time)
              }
              if (again) {
                if (__any_sync(0xffffffffu, real && far)) {
                  sum = 0.0f;
#pragma unroll
                  for (int e = 0; e < 64; e++) sum += fast_exp2(fmaf(s[e], f[e >> 4], -ur));
                }
                break;
              }
              if (named_all(pair_bar, 64, (fits && !far) || !real)) break;
            }
            l += sum;
            tmem_st32(ts, p);
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull(j & 1));
        first = false;
      }
      // the next item's queries ahead of this one's results
      if (pos < hi) scale = put_row(then, item + 1);
      ok = wait(pvdone((end - 1) & 3), (end - 1) >> 2) && ok;
      if (busy) {
        tc_fence_after();
        sm.pair[told][part][r].x = l;
        named_sync(pair_bar, 64);
        const float lsum = l + sm.pair[told][part ^ 1][r].x;
        told ^= 1;
        // a sum that left fp32's range, or a factor that is not a normal number (only values below
        // 2^-100 need one; two factors one after the other for every value: the chains 94 us, 90 so):
        // NaN, which the second kernel looks into; as is a row without a logit above -Inf
        const bool whole = it.n == it.per;
        float f = lsum == 0.0f ? 0.0f : __fdiv_rn(fast_exp2(mx - kT8Up - u), lsum);
        if ((lsum != 0.0f || whole) && !(f >= 1.17549435e-38f)) f = __uint_as_float(0x7fffffffu);
        if (__builtin_expect(*(volatile int*)&sm.any_taken, 0)) {
          // tiles of 16 bits are a unit's last ones, in five steps at most
#pragma unroll 1
          for (int x = 4 * max(end - it.n, end - 8); x < 4 * end; x++) {
            const int2 d = sm.taken[x >> 2 & 15][x & 3];
            const int kind = d.y >> 16, w = d.x >> 5;
            const uint32_t see = kind == 2 ? sees_stored(a, it.N, node.depth, d.x)
                                 : kind == 3 ? (w == 0 ? node.over[0] : w == 1 ? node.over[1] : w == 2 ? node.over[2] : node.over[3]) >> (d.x & 31)
                                             : 0u;
            if (see & d.y & 0xffffu) f = __uint_as_float(0x7fffffffu);
          }
        }
        uint8_t* out = a.out + (((long long)it.i * a.max_nodes + m) * c.hkv * G + (size_t)it.h * G + (row - m * G)) * (2 * kD) + 128 * part;
        // a part: [feature / 4][row][4], whose lanes' stores are neighbours, then (u, l) of the rows
        float4* dst = reinterpret_cast<float4*>(a.part + (size_t)(2 * blockIdx.x + (it.s0 > 0 ? 0 : 1)) * part_rows * (kD + 2));
        // (loops, and short ones: code that runs once an item comes from far)
        auto load = [&](int q, float (&o)[16]) {
          tmem_ld16_nowait(t_o + tl + 64 * part + 16 * q, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; e++) {
            asm volatile("" : "+f"(o[e]));
            o[e] *= f;
          }
        };
        if (whole) {
          uint32_t bad = 0;
#pragma unroll 1
          for (int q = 0; q < 4; q++) {
            float o[16];
            load(q, o);
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; e++) {
              w[e] = pack_elems<ELEM>(o[2 * e], o[2 * e + 1]);
              find_not_finite<ELEM>(bad, w[e]);
            }
            if (real) {
              reinterpret_cast<uint4*>(out)[2 * q] = make_uint4(w[0], w[1], w[2], w[3]);
              reinterpret_cast<uint4*>(out)[2 * q + 1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
          if (__builtin_expect(__any_sync(0xffffffffu, real && found_not_finite(bad)), 0)) {
            sm.bad = 1;
#pragma unroll 1
            for (int q = 0; q < 4; q++) {
              float o[16];
              load(q, o);
#pragma unroll
              for (int e = 0; e < 8; e++)
                if (real) reinterpret_cast<uint32_t*>(out)[8 * q + e] = pack_elems<ELEM>(in_range<ELEM>(o[2 * e]), in_range<ELEM>(o[2 * e + 1]));
            }
          }
        } else {
#pragma unroll 1
          for (int q = 0; q < 4; q++) {
            float o[16];
            load(q, o);
#pragma unroll
            for (int e = 0; e < 4; e++)
              if (real) dst[(16 * part + 4 * q + e) * part_rows + r] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
          if (real && part == 0) reinterpret_cast<float2*>(dst + part_rows * (kD / 4))[r] = make_float2(u, lsum);
          if (threadIdx.x == 0 && it.s0 == 0) {
            sm.begun[0] = 1;
            sm.begun[1] = it.i;
            sm.begun[2] = it.h;
            sm.begun[3] = it.t;
          }
        }
      }
      tc_fence_before();
      if (pos >= hi) break;
      it = then;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kT8RegsFew));
    const int steps = hi - lo;
    if (warp < 16) {
      // ---- codes, tails and drafts to 16-bit operands: a warp two tiles of each step ----
      const int op = warp >= 12, first = 2 * (warp & 3);
      const int mat = lane >> 3, mrow = lane & 7, me = mat & 1, ms = mat >> 1;
      // the lane's row of the four 8 x 8 matrices of a store, tile t of the step: K (rows of 64
      // features, 16 KB on the others), V (rows: features, of 64 tokens), V of drafts (the
      // matrices the other way round)
      const uint32_t base = smem_u32(smem) + (op ? kT8OffV : 0);
      auto place = [&](int t) {
        return op ? base + (t >> 2) * 16384 + ms * 1024 + mrow * 128 + (((2 * (t & 3) + me) ^ mrow) << 4)
                  : base + (2 * t + ms) * 1024 + mrow * 128 + ((me ^ mrow) << 4);
      };
      auto draft_place = [&](int t) { return base + (t >> 2) * 16384 + me * 1024 + mrow * 128 + (((2 * (t & 3) + ms) ^ mrow) << 4); };
      const uint32_t full = op ? vfull(0) : kfull(0), free = op ? vfree(0) : kfree(0);
      uint8_t* ring = smem + kT8OffRing + op * (kT8Ring * kT8Entry) + first * kTile;
      const uint32_t rfull = smem_u32(sm.rfull[op]), rfree = smem_u32(sm.rfree[op]);
#pragma unroll 1
      for (int j = 0; ok && j < steps; j++) {
        const int slot = j & 1;
        const TileDesc* desc = sm.desc[j & (kT8Descs - 1)] + first;
        uint32_t out = 0;
        ok = wait(rfull + 8 * slot, j >> 1);               // (the descriptors are there, too)
        if (ok && j >= kT8Slots) ok = wait(free + 8 * slot, (j >> 1) - 1);
        if (!ok) break;
        const uint32_t to0 = place(first) + slot * kT8Slot, to1 = place(first + 1) + slot * kT8Slot;
        const int kind = desc->kind;
        if (kind >= 1 && kind <= 3) {
          // (the second place is none)
          const TileExps exps{sm.kexp[j & (kT8Metas - 1)][warp & 3], sm.vexp[slot][warp & 3]};
          if (kind == 1) put_tile<DKV_F16, true, CODE>(ring + slot * kT8Entry, op, kSub, to0, exps, desc->lv);
          else if (kind == 2) out = put_tile<ELEM, false, CODE>(ring + slot * kT8Entry, op, desc->n, to0, exps, 0.0f);
          else out = put_drafts<ELEM>(ring + slot * kT8Entry, op, desc->n, (op ? draft_place(first) : base + 2 * first * 1024) + slot * kT8Slot, exps);
        } else {
#pragma unroll 1
          for (int t = 0; t < 2; t++)
            if (desc[t].kind == 0) {
              const uint8_t* p = ring + slot * kT8Entry + t * kTile + 16 * lane;
              uint4 w[4];
#pragma unroll
              for (int e = 0; e < 4; e++) w[e] = *reinterpret_cast<const uint4*>(p + 512 * e);
              // K: 16 features on are 32 bytes of a row (swizzled); V: 2 KB
              const uint32_t to = t ? to1 : to0;
#pragma unroll
              for (int e = 0; e < 4; e++) {
                const uint32_t at0 = op ? to + e * 4096 : (to + (e >> 1) * 16384) ^ ((e & 1) << 6);
                const uint32_t at1 = op ? at0 + 2048 : at0 ^ 32u;
                uint32_t y[4];
                code_halves<CODE>(w[e].x, y[0], y[1]);
                code_halves<CODE>(w[e].y, y[2], y[3]);
                stmatrix4(at0, y[0], y[1], y[2], y[3]);
                code_halves<CODE>(w[e].z, y[0], y[1]);
                code_halves<CODE>(w[e].w, y[2], y[3]);
                stmatrix4(at1, y[0], y[1], y[2], y[3]);
              }
            }
        }
        if (op && lane == 0) {
          sm.taken[j & 15][warp & 3] = make_int2(desc->pos0, kind << 16 | (int)out);
          if (out) sm.any_taken = 1;
        }
        if (op == 0 && lane < 2) {
          const TileDesc* d = desc + lane;
          sm.meta[j & (kT8Metas - 1)][first + lane] = TileMeta{d->ks, d->lv, d->pos0, d->kind};
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(full + 8 * slot);
          mbar_arrive(rfree + 8 * slot);
          if (j % kT8Batch == kT8Batch - 1) mbar_arrive(smem_u32(&sm.dfree[j / kT8Batch & 3]));
        }
      }
    } else if (warp == 17) {
      // ---- where the tiles lie and what scales them, a lane a tile, a batch of steps at a
      // time (at most four are kept) ----
      const int batches = (steps + kT8Batch - 1) / kT8Batch;
#pragma unroll 1
      for (int b = 0; ok && b < batches; b++) {
        const float2* scales = nullptr;
        TileDesc d{nullptr, kLogitScale, {0.0f}, 0, 4, 0, nullptr};
        const int x = kT8Step * kT8Batch * b + lane;
        if (x < kT8Step * steps) d = describe_tile(c, a, sm.plan, lo, x, scales);
        if (scales) {
          const float2 sc = *scales;
          d.ks = sc.x * kLogitScale;
          d.lv = log2f(sc.y);
        }
        if (d.kind == 2 || d.kind == 3) {
          const int i = d.req_head >> 12, h = d.req_head & 4095;
          d.n = min((d.kind == 2 ? sm.plan.N[i] : sm.plan.M[i]) - d.pos0, kSub);
          d.vsrc = d.kind == 2 ? d.src + 2 * kTile : a.v + ((long long)i * a.max_nodes + d.pos0) * a.vs + h * (2 * kD);
          d.lv = 0.0f;
        }
        if (b >= 4) ok = wait(smem_u32(&sm.dfree[b & 3]), (b >> 2) - 1);
        if (!ok) break;
        const int at = (kT8Batch * b + lane / kT8Step) & (kT8Descs - 1);
        sm.desc[at][lane % kT8Step] = d;
        const unsigned there = __ballot_sync(0xffffffffu, d.kind < 4);
        if (lane % kT8Step == 0) sm.there[(kT8Batch * b + lane / kT8Step) & (2 * kT8Descs - 1)] = there >> lane & 0xffu;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.dfull[b & 3]));
      }
    } else if (warp >= 18) {
      // ---- copies of codes ----
      const int op = warp - 18;
      const uint32_t ring = smem_u32(smem + kT8OffRing + op * (kT8Ring * kT8Entry));
      int issued = 0;
#pragma unroll 1
      for (int j = 0; ok && j < steps; j++) {
        if (j % kT8Batch == 0) ok = wait(smem_u32(&sm.dfull[j / kT8Batch & 3]), j / kT8Batch >> 2);
        if (ok && j >= kT8Ring) ok = wait(smem_u32(&sm.rfree[op][j & 1]), (j >> 1) - 1);
        if (!ok) break;
        const TileDesc* d = &sm.desc[j & (kT8Descs - 1)][lane & (kT8Step - 1)];
        const int kind = d->kind;
        const unsigned who = __ballot_sync(0xffffffffu, lane < kT8Step && kind <= 2);
        // codes: 2 KB of a tile, K then V; the tail: 4 KB; drafts: their rows
        const unsigned long long src = reinterpret_cast<unsigned long long>(d->src) + (kind == 2 ? 2 * op * kTile : op * kTile);
        const int size = kind == 2 ? 2 * kTile : kind == 3 ? d->n * 2 * kD : kind < 2 ? kTile : 0;
        const int bytes = __reduce_add_sync(0xffffffffu, lane < kT8Step ? size : 0);
        const uint32_t bar = smem_u32(&sm.rfull[op][j & 1]), dst = ring + (j & 1) * kT8Entry;
        if (lane == 0) {
          if (bytes) mbar_expect_tx(bar, bytes);
          else mbar_arrive(bar);
        }
        __syncwarp();
#pragma unroll
        for (int t = 0; t < kT8Step; t++) {
          const unsigned long long p = __shfl_sync(0xffffffffu, src, t);
          const int n = __shfl_sync(0xffffffffu, size, t);
          if (who >> t & 1u)
            if (elected()) bulk_g2s(dst + t * kTile, reinterpret_cast<const void*>(p), n, bar);
        }
        for (unsigned rows = __ballot_sync(0xffffffffu, lane < kT8Step && kind == 3); rows; rows &= rows - 1) {
          const int t = __ffs(rows) - 1;
          const TileDesc* e = &sm.desc[j & (kT8Descs - 1)][t];
          if (lane < e->n) bulk_g2s(dst + t * kTile + lane * (2 * kD), op ? e->vsrc + lane * a.vs : e->src + lane * a.ks, 2 * kD, bar);
        }
        __syncwarp();
        if (lane == 0 && j % kT8Batch == kT8Batch - 1) mbar_arrive(smem_u32(&sm.dfree[j / kT8Batch & 3]));
        issued = j + 1;
      }
      // no copy may be in flight at the exit
      for (int j = max(issued - kT8Ring, 0); j < issued; j++) mbar_wait_bounded(smem_u32(&sm.rfull[op][j & 1]), j >> 1 & 1);
    } else if (warp == 16) {
      // ---- products: S of the steps to come, O += P V; the whole warp walks, one lane
      // issues (counters, so that operands stay in uniform registers). Products run in the
      // order of their issue, so S may follow the P V that read its place ----
      constexpr uint32_t id_half = umma_idesc_f16(128, 64), id = umma_idesc_f16(128, 128);
      const uint64_t kd = umma_desc_sw128(smem_u32(smem)), vd = umma_desc_sw128(smem_u32(smem + kT8OffV));
      auto test = [&](uint32_t bar, int phase) { return __all_sync(0xffffffffu, mbar_test(bar, phase & 1)) != 0; };
      auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
      // S walks the items; their ends are kept for P V, which is at most two items behind
      int s_end = 0, item = -1, v_end = 0, v_item = -1;
      int js = 0, jv = 0;              // next step of S, of P V
      bool begin = true, q_there = false;
      const int last = uniform(steps);
      int s_slot = 0, s_round = 0, v_slot = 0, v_round = 0, idle = 0;
      auto next_slot = [](int& slot, int& round) {
        if (++slot == kT8Slots) {
          slot = 0;
          round ^= 1;
        }
      };
      long long since = 0;
#pragma unroll 1
      while (jv < last) {
        bool none = true;
        if (js < last && js < jv + 2) {
          if (js == s_end) {
            const TreeItem it = tree_item(c, a, sm.plan, lo + js, hi);
            s_end = js + uniform(it.n);
            item++;
            q_there = false;
            if (lane == 0) sm.runs[item & 3] = s_end;
            __syncwarp();
          }
          if (!q_there) q_there = test(qfull(item & 1), item >> 1);
          if (q_there && test(kfull(s_slot), s_round)) {
            tc_fence_after();
            const uint32_t d = uniform(t_s(js & 1)), q = uniform(t_q(item & 1));
            const uint32_t kind = uniform(sm.there[js & (2 * kT8Descs - 1)] >> 4 ? id : id_half);
            const int at = uniform(s_slot * (kT8Slot >> 4)), bar_s = uniform(sfull(js & 1)), bar_k = uniform(kfree(s_slot));
            if (elected()) {
              const uint64_t bd = kd + at;
#pragma unroll
              for (int e = 0; e < 8; e++)
                umma_f16_tmem_a(d, q + 8 * e, bd + (((e >> 2) * 16384 + (e & 3) * 32) >> 4), kind, e > 0);
              umma_commit(bar_s);
              umma_commit(bar_k);
            }
            __syncwarp();
            next_slot(s_slot, s_round);
            js++;
            none = false;
          }
        }
        if (jv < js && jv == v_end) {
          v_end = uniform(sm.runs[++v_item & 3]);
          begin = true;
        }
        if (jv < js && test(pfull(jv & 1), jv >> 1) && test(vfull(v_slot), v_round)) {
          tc_fence_after();
          const uint32_t p = uniform(t_s(jv & 1));
          const int who = uniform(sm.there[jv & (2 * kT8Descs - 1)]), go_on = uniform(!begin), at = uniform(v_slot * (kT8Slot >> 4));
          const int bar_pv = uniform(pvdone(jv & 3)), bar_v = uniform(vfree(v_slot));
          if (elected()) {
            const uint64_t bd = vd + at;
#pragma unroll
            for (int e = 0; e < kT8Step; e++)
              if (who >> e & 1)       // (place 0 always holds a tile)
                umma_f16_tmem_a(t_o, p + 64 * (e >> 2) + 8 * (e & 3), bd + (((e >> 2) * 16384 + (e & 3) * 32) >> 4), id, go_on || e > 0);
            umma_commit(bar_pv);
            umma_commit(bar_v);
          }
          __syncwarp();
          next_slot(v_slot, v_round);
          begin = false;
          jv++;
          none = false;
        }
        // bounded: about a second without anything to issue
        if (!none) idle = 0;
        else if (++idle == 1) since = clock64();
        else if ((idle & 1023) == 0 && __any_sync(0xffffffffu, *(volatile int*)&sm.fail != 0 || clock64() - since > 2000000000LL)) {
          *(volatile int*)&sm.fail = 1;
          ok = false;
          break;
        }
      }
      if (elected()) {
        umma_commit(drain);                // every MMA issued so far has completed
        mbar_wait_bounded(drain, 0);
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
    if (lane == 0 && sm.fail) c.latch(DKV_ERR_TIMEOUT, -1);
  } else if (threadIdx.x == 0) {
    TreeRecord d{sm.begun[0] | sm.bad << 1, sm.begun[1], sm.begun[2], sm.begun[3], 0, 0, lo, hi};
    if (sm.begun[0]) {
      d.M = sm.plan.M[d.i];
      const int per = (tree_tiles(sm.plan.N[d.i], d.M, c.T, a.window, a.sinks).places + kT8Step - 1) / kT8Step;
      const int unit = d.h * unit_rows(d.M, G) + d.t;
      d.last = range_of(all.steps + turn * all.units, sm.plan.pre[d.i] + unit * per + turn * (sm.plan.units[d.i] + unit + 1) + per - 1, ctas);
    }
    records[blockIdx.x] = d;
  }
}

// ---- units that several CTAs hold parts of, and rows that came out infinite or NaN ----
// o = sum_p l_p 2^(u_p - u) o_p / sum_p l_p 2^(u_p - u) over a unit's parts p. A block looks at what
// one CTA has left and takes eight rows of the unit that it began, if others went on with it; a
// lane four features of one of them, so that the loads of a warp are whole 128-byte lines (a warp
// for each row, with the part's rows 16 bytes a lane: 5 us more for 16 requests of 4096 tokens with 26
// drafts). It waits for memory, not for its bandwidth: the first three parts are sent for before
// their weights are known, and four blocks fit an SM (five spill: 1.5 us more; three: 2 us).
template <int ELEM, int CODE>
__global__ void __launch_bounds__(32 * kT8Walkers, 4) k_tree8_join(const __grid_constant__ Cache8View c, const __grid_constant__ Tree8Args a,
                                                                   int part_rows, const int* plan, const TreeRecord* records) {
  __shared__ WalkSmem walk_sm;
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, lr = lane & 7, lq = lane >> 3, G = c.G;
  const int octets = part_rows / 8, c0 = blockIdx.x / octets, o8 = 8 * (blockIdx.x - c0 * octets);
  pdl_wait();
  const TreeRecord rec = records[c0];
  // (an error of this call or an earlier one: results are undefined)
  if (rec.flags == 0 || c.stopped()) return;
  auto out_of = [&](int i, int h, int row) {
    const int m = row / G;
    return a.out + (((size_t)i * a.max_nodes + m) * (c.hkv * G) + (size_t)h * G + (row - m * G)) * (2 * kD);
  };
  // of eight rows from `first` on those that came out infinite or NaN, one by one
  auto again = [&](int i, int h, int first, bool bad, const TreeReq& req, const TreeTiles& tiles) {
    const Walk<ELEM, CODE> walk{c, a, i, h, req, tiles};
#pragma unroll 1
    for (int x = 0; x < 8; x++)
      if (__syncthreads_or(bad && lr == x)) walk.row((first + x) / G, (first + x) % G, out_of(i, h, first + x), walk_sm);
  };
  const int row0 = rec.t * kT8Rows + o8, row = row0 + lr;
  if ((rec.flags & 1) && row0 < rec.M * G) {
    const int c1 = rec.last, r = o8 + lr;
    const bool real = row < rec.M * G;
    uint8_t* out = out_of(rec.i, rec.h, row) + 8 * (4 * warp + lq);
    // the first part begins its unit (place 1), the others go on with it (place 0)
    const size_t place = (size_t)part_rows * (kD + 2) / 4;
    const float4* parts = reinterpret_cast<const float4*>(a.part);
    auto part = [&](int cta) { return parts + (size_t)(2 * cta + (cta == c0 ? 1 : 0)) * place; };
    auto weight_of = [&](int cta) { return reinterpret_cast<const float2*>(part(cta) + part_rows * (kD / 4))[real ? r : 0]; };
    const int at = (4 * warp + lq) * part_rows + (real ? r : 0);
    // most units have few parts: their rows are on their way while the weights are
    constexpr int kNear = 3;
    float4 v[kNear];
    float2 ul[kNear];
#pragma unroll
    for (int e = 0; e < kNear; e++) {
      v[e] = part(min(c0 + e, c1))[at];
      ul[e] = weight_of(min(c0 + e, c1));
    }
    float top = -INFINITY, sum = 0.0f;
    auto more = [&](float2 z) {
      const float now = fmaxf(top, z.x);
      sum = sum == 0.0f ? 0.0f : sum * (top == now ? 1.0f : fast_exp2(top - now));
      sum += z.y == 0.0f ? 0.0f : z.y * (z.x == now ? 1.0f : fast_exp2(z.x - now));
      top = now;
    };
    if (c1 - c0 < kNear) {
#pragma unroll
      for (int e = 0; e < kNear; e++)
        if (c0 + e <= c1) more(ul[e]);
    } else {
      for (int b = c0 + lq; b <= c1; b += 4) more(weight_of(b));
#pragma unroll
      for (int d = 8; d <= 16; d <<= 1) {
        const float ot = __shfl_xor_sync(0xffffffffu, top, d), os = __shfl_xor_sync(0xffffffffu, sum, d);
        more(make_float2(ot, os));
      }
    }
    // (no logit above -Inf: no softmax)
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (sum == 0.0f) o.x = __uint_as_float(0x7fffffffu);
    auto add = [&](const float4& y, const float2& z) {
      const float f = z.y == 0.0f ? 0.0f : __fdiv_rn(z.y * (z.x == top ? 1.0f : fast_exp2(z.x - top)), sum);
      o.x = fmaf(y.x, f, o.x);
      o.y = fmaf(y.y, f, o.y);
      o.z = fmaf(y.z, f, o.z);
      o.w = fmaf(y.w, f, o.w);
    };
#pragma unroll
    for (int e = 0; e < kNear; e++)
      if (c0 + e <= c1) add(v[e], ul[e]);
#pragma unroll 4
    for (int b = c0 + kNear; b <= c1; b++) add(part(b)[at], weight_of(b));
    const uint2 w = make_uint2(pack_elems<ELEM>(in_range<ELEM>(o.x), in_range<ELEM>(o.y)), pack_elems<ELEM>(in_range<ELEM>(o.z), in_range<ELEM>(o.w)));
    if (real) *reinterpret_cast<uint2*>(out) = w;
    uint32_t bad = 0;
    find_not_finite<ELEM>(bad, w.x);
    find_not_finite<ELEM>(bad, w.y);
    if (__builtin_expect(__syncthreads_or(real && found_not_finite(bad)), 0)) {
      const TreeReq req = tree_req(c, a, rec.i);
      again(rec.i, rec.h, row0, real && found_not_finite(bad), req, tree_tiles(req.N, req.M, c.T, a.window, a.sinks));
    }
  }
  if (__builtin_expect(rec.flags & 2, 0)) {
#pragma unroll 1
    for (int pos = rec.lo; pos < rec.hi;) {
      int i = 0, end = a.n_req;
#pragma unroll 1
      while (end - i > 1) {      // as in tree_item
        const int mid = (i + end) >> 1;
        if (plan[mid] <= pos) i = mid; else end = mid;
      }
      const TreeReq req = tree_req(c, a, i);
      const TreeTiles tiles = tree_tiles(req.N, req.M, c.T, a.window, a.sinks);
      const int per = (tiles.places + kT8Step - 1) / kT8Step, x = pos - plan[i], unit = x / per, s0 = x - unit * per, n = min(per - s0, rec.hi - pos);
      const int rt = unit_rows(req.M, G), h = unit / rt, first = (unit - h * rt) * kT8Rows + o8;
      pos += n;
      if (n < per) continue;
      uint32_t bad = 0;
      if (first + lr < req.M * G) {
        const uint2 w = *reinterpret_cast<const uint2*>(out_of(i, h, first + lr) + 8 * (4 * warp + lq));
        find_not_finite<ELEM>(bad, w.x);
        find_not_finite<ELEM>(bad, w.y);
      }
      if (__syncthreads_or(found_not_finite(bad))) again(i, h, first, found_not_finite(bad), req, tiles);
    }
  }
}

int part_rows_of(int G, int max_nodes) { return std::min(kT8Rows, (max_nodes * G + 31) / 32 * 32); }

// The workspace: the steps' prefix sums, then a record and two parts a CTA.
constexpr size_t kT8PlanBytes = ((kMaxCallReq + 1) * 4 + 255) / 256 * 256;

template <int ELEM, int CODE>
cudaError_t tree_typed(const Cache8View& c, Tree8Args a, int sm_count, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(k_tree8<ELEM, CODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kT8Smem);
  if (e != cudaSuccess) return e;
  const int part_rows = part_rows_of(c.G, a.max_nodes);
  int* plan = reinterpret_cast<int*>(a.part);
  TreeRecord* records = reinterpret_cast<TreeRecord*>(a.part + kT8PlanBytes / 4);
  a.part += kT8PlanBytes / 4 + sm_count * (sizeof(TreeRecord) / 4);
  // no more CTAs than the longest lengths that the table holds could use
  const long long tiles = ((long long)c.width * c.T + a.max_nodes) / kSub + 3;
  const long long steps = (long long)a.n_req * c.hkv * ((a.max_nodes * c.G + kT8Rows - 1) / kT8Rows) * (tiles / kT8Step + 1);
  const int grid = (int)std::min<long long>(sm_count, steps);
  e = launch_dependent(k_tree8<ELEM, CODE>, dim3(grid), dim3(kT8Threads), kT8Smem, st, c, a, part_rows, plan, records);
  if (e != cudaSuccess) return e;
  return launch_dependent(k_tree8_join<ELEM, CODE>, dim3(grid * (part_rows / 8)), dim3(32 * kT8Walkers), 0, st, c, a, part_rows, plan, records);
}

}  // namespace

size_t tree8_workspace(int G, int max_nodes, int sm_count) {
  return kT8PlanBytes + (size_t)sm_count * (sizeof(TreeRecord) + 2 * part_rows_of(G, max_nodes) * (kD + 2) * 4);
}

cudaError_t launch_tree8(const Cache8View& c, int elem, int code, int sm_count, const Tree8Args& a, cudaStream_t st) {
  if (elem == DKV_F16)
    return code == DKV_E4M3 ? tree_typed<DKV_F16, DKV_E4M3>(c, a, sm_count, st) : tree_typed<DKV_F16, DKV_INT8>(c, a, sm_count, st);
  return code == DKV_E4M3 ? tree_typed<DKV_BF16, DKV_E4M3>(c, a, sm_count, st) : tree_typed<DKV_BF16, DKV_INT8>(c, a, sm_count, st);
}

}  // namespace dkv
