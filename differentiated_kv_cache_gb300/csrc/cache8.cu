// cache8.cu — host side of the uniform 8-bit cache's entry points
// (include/dkv.h) and the append kernels: rotation of keys and queries by one
// position or one of each axis, 16-bit tails, quantisation of completed blocks,
// accepted drafts.
#include <algorithm>
#include <type_traits>

#include "cache8.cuh"
#include "dkv_kernels.cuh"

namespace dkv {
namespace {

// Requests of an append with several tokens each: first token row, tokens,
// first job and the number of blocks a request can touch.
constexpr int kQGroup = 4;       // query heads whose loads are in flight together
constexpr int kAppendReq = 1024;
struct AppendCall {
  int tok0[kAppendReq + 1];
  int blk0[kAppendReq + 1];
};

// Four pair slots of a 128-feature row: features a0..a0+3 turn with
// b0..b0+3 (rows split in halves) or the pairs lie inside a0..b0+3
// (interleaved); past rotary_dim eight features pass unchanged.
struct Quad {
  int a0, b0, pair0;
  bool turn;
};
__device__ __forceinline__ Quad quad_of(int j, int rot, int inter) {
  Quad x;
  x.turn = 8 * j < rot;
  x.pair0 = 4 * j;
  const bool split = x.turn && !inter;
  x.a0 = split ? 4 * j : 8 * j;
  x.b0 = split ? rot / 2 + 4 * j : 8 * j + 4;
  return x;
}

struct Rot4 {
  float2 cs[4];
};
__device__ __forceinline__ Rot4 load_rot(const float2* rope, int rot, int pos, const Quad& x) {
  Rot4 r;
  if (x.turn) {
    const float4* p = reinterpret_cast<const float4*>(rope + (size_t)pos * (rot / 2) + x.pair0);
    const float4 u = __ldg(p), w = __ldg(p + 1);
    r.cs[0] = make_float2(u.x, u.y);
    r.cs[1] = make_float2(u.z, u.w);
    r.cs[2] = make_float2(w.x, w.y);
    r.cs[3] = make_float2(w.z, w.w);
  }
  return r;
}

// The same with a position of its own for each pair (four axes in the bytes of
// axes, pairs pair0 onwards): token `row` of the call. Pairs of one axis, the usual
// case where axes take parts of the head, lie together in the table.
__device__ __forceinline__ Rot4 load_rot_at(const Cache8View& c, const Append8Args& a, uint32_t axes, long long row,
                                            int info, const Quad& x) {
  Rot4 r = {};
  if (!x.turn) return r;
  auto position = [&](int i) {
    int p = __ldg(a.pos + (axes >> (8 * i) & 0xffu) * a.n_tok + row);
    if ((unsigned)p >= (unsigned)a.rope_len) {
      c.latch(DKV_ERR_ARG, info);
      p = 0;
    }
    return p;
  };
  if (axes == (axes & 0xffu) * 0x01010101u) return load_rot(a.rope, c.rot, position(0), x);
  int p[4];
#pragma unroll
  for (int i = 0; i < 4; i++) p[i] = position(i);
#pragma unroll
  for (int i = 0; i < 4; i++) r.cs[i] = __ldg(a.rope + (size_t)p[i] * (c.rot / 2) + x.pair0 + i);
  return r;
}
__device__ __forceinline__ uint32_t axes_of(const Append8Args& a, int j) {
  return *reinterpret_cast<const uint32_t*>(a.axis + 4 * j);
}

// (a c - b s, b c + a s), every operation rounded by itself
__device__ __forceinline__ void turn_pair(float& a, float& b, float2 cs) {
  const float y = __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
  b = __fadd_rn(__fmul_rn(b, cs.x), __fmul_rn(a, cs.y));
  a = y;
}

// The eight features of a quad, turned and rounded: u = features a0..a0+3,
// w = b0..b0+3.
template <int ELEM>
__device__ __forceinline__ void turn_quad(uint2& u, uint2& w, const Quad& x, const Rot4& r, int inter) {
  if (!x.turn) return;
  float a[4] = {lo_elem<ELEM>(u.x), hi_elem<ELEM>(u.x), lo_elem<ELEM>(u.y), hi_elem<ELEM>(u.y)};
  float b[4] = {lo_elem<ELEM>(w.x), hi_elem<ELEM>(w.x), lo_elem<ELEM>(w.y), hi_elem<ELEM>(w.y)};
  if (inter) {
    turn_pair(a[0], a[1], r.cs[0]);
    turn_pair(a[2], a[3], r.cs[1]);
    turn_pair(b[0], b[1], r.cs[2]);
    turn_pair(b[2], b[3], r.cs[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++) turn_pair(a[i], b[i], r.cs[i]);
  }
  u = make_uint2(pack_elems<ELEM>(a[0], a[1]), pack_elems<ELEM>(a[2], a[3]));
  w = make_uint2(pack_elems<ELEM>(b[0], b[1]), pack_elems<ELEM>(b[2], b[3]));
}

__device__ __forceinline__ uint2 ld8(const uint8_t* p) { return *reinterpret_cast<const uint2*>(p); }
__device__ __forceinline__ void st8(uint8_t* p, uint2 v) { *reinterpret_cast<uint2*>(p) = v; }

// What one job finds out about its request; not valid: nothing to do.
struct Where {
  int slot, before, n;
};
__device__ __forceinline__ Where where_of(const Append8Args& a, int i, int n) {
  return Where{a.slots ? a.slots[i] : i, a.before[i], n};
}
__device__ __forceinline__ bool valid(const Cache8View& c, const Append8Args& a, int i, const Where& w) {
  if (w.before < 0) return false;
  if ((unsigned)w.slot >= (unsigned)c.n_slots) {
    c.latch(DKV_ERR_ARG, i);
    return false;
  }
  const long long end = (long long)w.before + w.n;
  if (end > (long long)c.width * c.T) {
    c.latch(DKV_ERR_TABLE_FULL, i);
    return false;
  }
  if (c.rot && !a.pos && end > a.rope_len) {
    c.latch(DKV_ERR_ARG, i);
    return false;
  }
  return true;
}

// Slots given twice or outside the cache (one block, beside the others), but for
// requests that are padding.
template <typename Padding>
__device__ void check_slots(const Cache8View& c, const int* slots, int n_req, uint32_t* bits, Padding padding) {
  if (!slots) return;
  for (int x = threadIdx.x; x < (c.n_slots + 31) / 32; x += blockDim.x) bits[x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n_req; i += blockDim.x) {
    const int s = slots[i];
    if (padding(i)) continue;
    if ((unsigned)s >= (unsigned)c.n_slots) {
      c.latch(DKV_ERR_ARG, i);
      continue;
    }
    if (atomicOr(&bits[s >> 5], 1u << (s & 31)) >> (s & 31) & 1u) c.latch(DKV_ERR_ARG, i);
  }
}

// Quantise a complete block of one head from its 16-bit entries (tile order)
// in shared memory and write codes and scales. All threads of the block.
template <int ELEM, int CODE>
__device__ void quantise_block(const Cache8View& c, const uint16_t* buf, int page, int h, uint32_t* red) {
  const int nt = blockDim.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = nt >> 5;
  const int per = c.T * kD;      // entries of one operand
  // magnitudes order like their bits: packed maxima of every value, and again of
  // the finite ones only where the first pass finds that some are not
  constexpr uint32_t kInf = ELEM == DKV_F16 ? 0x7c00u : 0x7f80u;
  uint32_t top[2];
  bool all = true;
#pragma unroll 1
  for (;; all = false) {
    uint32_t m[2] = {0, 0};
    for (int x = 8 * threadIdx.x; x < 2 * per; x += 8 * nt) {
      const uint4 w = *reinterpret_cast<const uint4*>(buf + x);
      const int o = (x / kTile) & 1;
      uint32_t v[4] = {w.x & 0x7fff7fffu, w.y & 0x7fff7fffu, w.z & 0x7fff7fffu, w.w & 0x7fff7fffu};
      if (!all) {
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] &= ~__vcmpgeu2(v[i], kInf << 16 | kInf);
      }
      const uint32_t mm = __vmaxu2(__vmaxu2(v[0], v[1]), __vmaxu2(v[2], v[3]));
      if (o == 0) m[0] = __vmaxu2(m[0], mm);
      else m[1] = __vmaxu2(m[1], mm);
    }
#pragma unroll
    for (int o = 0; o < 2; o++) {
      const uint32_t r = __reduce_max_sync(0xffffffffu, max(m[o] & 0xffffu, m[o] >> 16));
      if (lane == 0) red[32 * o + warp] = r;
    }
    __syncthreads();
    top[0] = top[1] = 0;
    for (int w = 0; w < nw; w++) {
      top[0] = max(top[0], red[w]);
      top[1] = max(top[1], red[32 + w]);
    }
    if (!all || max(top[0], top[1]) < kInf) break;
    __syncthreads();
  }
  const float s0 = block_scale(elem_float<ELEM>((uint16_t)top[0]), CODE);
  const float s1 = block_scale(elem_float<ELEM>((uint16_t)top[1]), CODE);
  const float i0 = __fdiv_rn(1.0f, s0), i1 = __fdiv_rn(1.0f, s1);
  if (threadIdx.x == 0) {
    float* sc = c.scales + 2 * ((size_t)page * c.hkv + h);
    sc[0] = s0;
    sc[1] = s1;
  }
  uint8_t* dst = c.pages + c.page_head(page, h);
  // 16 codes a thread: m-steps 2j and 2j + 1 of one lane's operands
  auto encode = [&](auto finite) {
    constexpr bool FINITE = decltype(finite)::value;
    for (int g = threadIdx.x; g < 2 * per / 16; g += nt) {
      const int tile = g >> 7, j = (g >> 5) & 3, l = g & 31;
      const float inv = tile & 1 ? i1 : i0;
      const uint16_t* src = buf + tile * kTile + 512 * j + 8 * l;
      uint32_t r[4];
#pragma unroll
      for (int e = 0; e < 2; e++) {
        const uint4 w = *reinterpret_cast<const uint4*>(src + 256 * e);
        const uint32_t x = code_pair<CODE, FINITE>(lo_elem<ELEM>(w.x), hi_elem<ELEM>(w.x), inv);
        const uint32_t y = code_pair<CODE, FINITE>(lo_elem<ELEM>(w.y), hi_elem<ELEM>(w.y), inv);
        const uint32_t z = code_pair<CODE, FINITE>(lo_elem<ELEM>(w.z), hi_elem<ELEM>(w.z), inv);
        const uint32_t u = code_pair<CODE, FINITE>(lo_elem<ELEM>(w.w), hi_elem<ELEM>(w.w), inv);
        r[2 * e] = FINITE ? prmt(x, y, 0x5410u) : x | y << 16;
        r[2 * e + 1] = FINITE ? prmt(z, u, 0x5410u) : z | u << 16;
      }
      *reinterpret_cast<uint4*>(dst + tile * kTile + 512 * j + 16 * l) = make_uint4(r[0], r[1], r[2], r[3]);
    }
  };
  // integers of finite values need no conversion instruction: 16 x 4096 tokens
  // with 8 / 8 heads 176 us, 196 with
  if (CODE == DKV_INT8 && all) encode(std::true_type());
  else encode(std::false_type());
}

// Entries of one token's quad: K (rows = tokens) or V (columns = tokens) of a
// [T/16][2][2048] buffer, in shared memory or in the tail.
__device__ __forceinline__ void put_k(uint16_t* buf, int i, const Quad& x, uint2 u, uint2 w) {
  uint16_t* t = buf + (i >> 4) * 2 * kTile;
  const int r = i & 15;
  // features f, f + 1 (f even) are neighbours
  *reinterpret_cast<uint32_t*>(t + tile16(r, x.a0 & 15, x.a0 >> 4)) = u.x;
  *reinterpret_cast<uint32_t*>(t + tile16(r, (x.a0 + 2) & 15, x.a0 >> 4)) = u.y;
  *reinterpret_cast<uint32_t*>(t + tile16(r, x.b0 & 15, x.b0 >> 4)) = w.x;
  *reinterpret_cast<uint32_t*>(t + tile16(r, (x.b0 + 2) & 15, x.b0 >> 4)) = w.y;
}
__device__ __forceinline__ void put_v(uint16_t* buf, int i, int f0, uint4 v) {
  uint16_t* t = buf + (i >> 4) * 2 * kTile + kTile;
  const int col = i & 15;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 8; e++) {
    const int f = f0 + e;
    t[tile16(f & 15, col, f >> 4)] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
  }
}

// One token per request, a block per request and KV head: 16 threads turn a row
// (K, V, then the G query heads) of 8 features each, so that every row's load is
// in flight at once. The call is bound by its launch and its chain of dependent
// loads (request, angles; tail and page where a block is complete), not by
// bytes: one request 2.1 us, 128 with 28 / 4 heads 5.2 us (7.5 with a row after
// the other).
constexpr int kStepThreads = 160;     // 16 x (2 + G) at most
template <int ELEM, int CODE, bool AT>
__global__ void __launch_bounds__(kStepThreads) k_append8_step(Cache8View c, Append8Args a, int n_req) {
  extern __shared__ __align__(16) uint8_t sm[];
  pdl_launch_dependents();
  pdl_wait();
  const int i = blockIdx.x / c.hkv, h = blockIdx.x % c.hkv;
  if (i == n_req) {
    if (!c.stopped()) check_slots(c, a.slots, n_req, reinterpret_cast<uint32_t*>(sm), [&](int x) { return a.before[x] < 0; });
    return;
  }
  const int r = threadIdx.x >> 4, j = threadIdx.x & 15;
  const Where w = where_of(a, i, 1);
  const Quad qd = quad_of(j, r == 1 ? 0 : c.rot, c.inter);      // V passes unchanged
  const uint8_t* src = nullptr;
  if (r == 0) src = a.k + i * a.ks + h * (2 * kD);
  else if (r == 1) src = a.v + i * a.vs + h * (2 * kD);
  else if (a.q && r - 2 < c.G) src = a.q + i * a.qs + ((size_t)h * c.G + r - 2) * (2 * kD);
  uint2 u = make_uint2(0, 0), v = u;
  if (src) {
    u = ld8(src + 2 * qd.a0);
    v = ld8(src + 2 * qd.b0);
  }
  if (c.stopped()) return;             // its load is in flight with the others
  if (!valid(c, a, i, w)) return;
  const int T = c.T, b = w.before / T, p = w.before - b * T;
  const bool full = p == T - 1;
  uint16_t* tail = reinterpret_cast<uint16_t*>(c.tail + c.tail_head(w.slot, h));
  uint16_t* buf = reinterpret_cast<uint16_t*>(sm);
  const Rot4 rot = AT ? load_rot_at(c, a, axes_of(a, j), i, i, qd) : load_rot(a.rope, c.rot, w.before, qd);
  int page = 0;
  if (full) {
    page = c.table[(size_t)w.slot * c.width + b];
    if ((unsigned)page >= (unsigned)c.n_pages) {
      if (threadIdx.x == 0) c.latch(DKV_ERR_CHECK, i);
      return;
    }
    const uint4* from = reinterpret_cast<const uint4*>(tail);      // tokens of earlier calls
    uint4* to = reinterpret_cast<uint4*>(buf);
    for (int x = threadIdx.x; x < T * 2 * kD / 8; x += blockDim.x) to[x] = from[x];
    __syncthreads();
  }
  uint16_t* to = full ? buf : tail;
  if (src) turn_quad<ELEM>(u, v, qd, rot, c.inter);
  if (r == 0) {
    put_k(to, p, qd, u, v);
    if (a.k_rot) {
      uint8_t* kr = a.k_rot + ((size_t)i * c.hkv + h) * (2 * kD);
      st8(kr + 2 * qd.a0, u);
      st8(kr + 2 * qd.b0, v);
    }
  } else if (r == 1) {
    put_v(to, p, 8 * j, make_uint4(u.x, u.y, v.x, v.y));
  } else if (src) {
    uint8_t* dq = a.q_rot + (((size_t)i * c.hkv + h) * c.G + r - 2) * (2 * kD);
    st8(dq + 2 * qd.a0, u);
    st8(dq + 2 * qd.b0, v);
  }
  if (full) {
    __syncthreads();
    quantise_block<ELEM, CODE>(c, buf, page, h, reinterpret_cast<uint32_t*>(sm + (size_t)T * 4 * kD));
  }
}

// One block of one KV head: a job takes the call's tokens that fall into it. The
// block's 16-bit entries gather in shared memory if this call completes it, else
// the new ones go to the tail. The G query heads of the KV head turn with the
// same angles. Bound by bytes: 32 x 4096 tokens (3.22 GB) take 479 us, 99% of
// the measured copy rate, with 4 T threads and the loads of K, V and four query
// rows in flight together (8 T threads: 786 us, two blocks an SM do not cover
// each other's barriers; 2 T threads: 635 us). Half of the query heads in a block of
// their own: 555 us instead of 490, and 143 us instead of 126 us for ragged pieces
// in blocks of 128; V's neighbouring tokens exchanged to store pairs: 531 us
// instead of 479 (spills). With positions of several axes (AT) a row's angles hang on two
// loads after one another, issued behind those of K, V and the queries: 8 prompts of 8000
// tokens with 40 / 8 heads, adjacent pairs of half a head (1.87 GB), 331 us, 83% of the copy
// rate (341 with the angles first); ragged pieces in blocks of 64 tokens 80 us, 77%.
template <int ELEM, int CODE, bool AT>
__global__ void __launch_bounds__(512, 2)
    k_append8(Cache8View c, Append8Args a, int n_req, const __grid_constant__ AppendCall call) {
  extern __shared__ __align__(16) uint8_t sm[];
  pdl_launch_dependents();
  pdl_wait();
  if (c.stopped()) return;
  if ((int)blockIdx.x == call.blk0[n_req] * c.hkv) {
    check_slots(c, a.slots, n_req, reinterpret_cast<uint32_t*>(sm), [&](int x) { return a.before[x] < 0; });
    return;
  }
  const int job = blockIdx.x / c.hkv, h = blockIdx.x % c.hkv;
  int i = 0;
  for (int end = n_req; end - i > 1;) {      // the request whose jobs hold this one
    const int mid = (i + end) >> 1;
    if (call.blk0[mid] <= job) i = mid; else end = mid;
  }
  const int row0 = call.tok0[i], n = call.tok0[i + 1] - row0, jb = job - call.blk0[i];
  const Where w = where_of(a, i, n);
  if (!valid(c, a, i, w)) return;
  const int T = c.T, first = w.before / T, open = (w.before + n) / T, used = w.before % T;
  int b = first + jb;
  // The tokens left in the open block overwrite tail places that the first
  // block still reads (its earlier tokens): the job of the first block takes
  // the open block too, after its own.
  const bool both = used > 0 && open > first;
  if (both && b == open) return;
  const int gq = a.q ? c.G : 0;
  uint16_t* tail = reinterpret_cast<uint16_t*>(c.tail + c.tail_head(w.slot, h));
  uint16_t* buf = reinterpret_cast<uint16_t*>(sm);
  const uint32_t axes = AT ? axes_of(a, threadIdx.x & 15) : 0u;
  while (true) {
    const int start = b * T;
    // tokens of this call inside the block: places [lo, hi)
    const int lo = max(w.before - start, 0), hi = min(w.before + n - start, T);
    if (hi <= lo) return;        // fewer blocks touched than the host allowed for
    const bool full = hi == T;
    int page = 0;
    if (full) {
      page = c.table[(size_t)w.slot * c.width + b];
      if ((unsigned)page >= (unsigned)c.n_pages) {
        if (threadIdx.x == 0) c.latch(DKV_ERR_CHECK, i);
        return;
      }
      if (lo > 0) {              // tokens of earlier calls
        const uint4* src = reinterpret_cast<const uint4*>(tail);
        uint4* dst = reinterpret_cast<uint4*>(buf);
        for (int x = threadIdx.x; x < T * 2 * kD / 8; x += blockDim.x) dst[x] = src[x];
        __syncthreads();
      }
    }
    uint16_t* to = full ? buf : tail;
    const long long r0 = row0 + (long long)start - w.before;     // token row of place 0
    for (int x = threadIdx.x; x < (hi - lo) * 16; x += blockDim.x) {
      const int p = lo + (x >> 4), j = x & 15;
      const long long row = r0 + p;
      const Quad qd = quad_of(j, c.rot, c.inter);
      Rot4 rot;
      if (!AT) rot = load_rot(a.rope, c.rot, start + p, qd);
      const uint8_t* ks = a.k + row * a.ks + h * (2 * kD);
      const uint8_t* qs = a.q + row * a.qs + (size_t)h * c.G * (2 * kD);
      uint8_t* dq = a.q_rot + (row * c.hkv + h) * (size_t)c.G * (2 * kD);
      uint2 u = ld8(ks + 2 * qd.a0), v = ld8(ks + 2 * qd.b0);
      const uint4 vv = *reinterpret_cast<const uint4*>(a.v + row * a.vs + h * (2 * kD) + 16 * j);
      // the loads of a group of query heads are on their way with K's and V's
      uint2 y[kQGroup], z[kQGroup];
      auto load_q = [&](int g0) {
#pragma unroll
        for (int g = 0; g < kQGroup; g++)
          if (g0 + g < gq) {
            y[g] = ld8(qs + (g0 + g) * (2 * kD) + 2 * qd.a0);
            z[g] = ld8(qs + (g0 + g) * (2 * kD) + 2 * qd.b0);
          }
      };
      load_q(0);
      if (AT) rot = load_rot_at(c, a, axes, row, i, qd);      // two loads after one another: behind the others
      turn_quad<ELEM>(u, v, qd, rot, c.inter);
      if (a.k_rot) {
        uint8_t* kr = a.k_rot + (row * c.hkv + h) * (2 * kD);
        st8(kr + 2 * qd.a0, u);
        st8(kr + 2 * qd.b0, v);
      }
      put_k(to, p, qd, u, v);
      put_v(to, p, 8 * j, vv);
      for (int g0 = 0; g0 < gq; g0 += kQGroup) {
        if (g0 > 0) load_q(g0);
#pragma unroll
        for (int g = 0; g < kQGroup; g++)
          if (g0 + g < gq) {
            turn_quad<ELEM>(y[g], z[g], qd, rot, c.inter);
            st8(dq + (g0 + g) * (2 * kD) + 2 * qd.a0, y[g]);
            st8(dq + (g0 + g) * (2 * kD) + 2 * qd.b0, z[g]);
          }
      }
    }
    if (full) {
      __syncthreads();
      quantise_block<ELEM, CODE>(c, buf, page, h, reinterpret_cast<uint32_t*>(sm + (size_t)T * 4 * kD));
    }
    if (!both || b != first) return;
    b = open;
    __syncthreads();
  }
}

// Accepted drafts: a block of threads per request, KV head and block of tokens that
// a path can touch; the keys are turned already. Paths are short, so the call is bound by its
// launch and a chain of loads (request, path, rows, then tail or page), not by bytes: 4 tokens
// of one request 7.5 us, up to 9 of each of 128 requests 7.5 us (0.5 by their bytes), as the
// append of one token takes.
constexpr int kAcceptThreads = 256;
constexpr int kStoreSmem = 128 * 4 * kD + 256;      // the largest block
template <int ELEM, int CODE>
__global__ void __launch_bounds__(kAcceptThreads) k_accept8(Cache8View c, Accept8Args a, int n_req, int jobs) {
  extern __shared__ __align__(16) uint8_t sm[];
  pdl_launch_dependents();
  pdl_wait();
  if (c.stopped()) return;
  const int h = blockIdx.x % c.hkv, job = blockIdx.x / c.hkv, i = job / jobs, jb = job - i * jobs;
  auto tokens = [&](int x) { return a.n_path ? a.n_path[x] : a.width; };
  if (i == n_req) {
    check_slots(c, a.slots, n_req, reinterpret_cast<uint32_t*>(sm), [&](int x) { return a.before[x] < 0 || tokens(x) <= 0; });
    return;
  }
  const int n = tokens(i);
  const int before = a.before[i], slot = a.slots ? a.slots[i] : i;
  if (before < 0 || n <= 0) return;
  int err = 0;
  if ((unsigned)slot >= (unsigned)c.n_slots || n > a.width) err = DKV_ERR_ARG;
  else if ((long long)before + n > (long long)c.width * c.T) err = DKV_ERR_TABLE_FULL;
  if (err) {
    c.latch(err, i);
    return;
  }
  const int T = c.T, first = before / T, open = (before + n) / T, used = before - first * T;
  int b = first + jb;
  const bool both = used > 0 && open > first;     // as in k_append8
  if (both && b == open) return;
  uint16_t* tail = reinterpret_cast<uint16_t*>(c.tail + c.tail_head(slot, h));
  uint16_t* buf = reinterpret_cast<uint16_t*>(sm);
  while (true) {
    const int start = b * T, lo = max(before - start, 0), hi = min(before + n - start, T);
    if (hi <= lo) return;
    const bool full = hi == T;
    int page = 0;
    if (full) {
      page = c.table[(size_t)slot * c.width + b];
      if ((unsigned)page >= (unsigned)c.n_pages) {
        if (threadIdx.x == 0) c.latch(DKV_ERR_CHECK, i);
        return;
      }
      if (lo > 0) {
        const uint4* src = reinterpret_cast<const uint4*>(tail);
        uint4* dst = reinterpret_cast<uint4*>(buf);
        for (int x = threadIdx.x; x < T * 2 * kD / 8; x += blockDim.x) dst[x] = src[x];
        __syncthreads();
      }
    }
    uint16_t* to = full ? buf : tail;
    for (int x = threadIdx.x; x < (hi - lo) * 16; x += blockDim.x) {
      const int p = lo + (x >> 4), j = x & 15;
      int node = a.path[(size_t)i * a.width + (start + p - before)];
      if ((unsigned)node >= (unsigned)a.max_nodes) {
        c.latch(DKV_ERR_ARG, i);
        node = 0;
      }
      const long long row = (long long)i * a.max_nodes + node;
      const uint4 u = *reinterpret_cast<const uint4*>(a.k + row * a.ks + h * (2 * kD) + 16 * j);
      const uint4 v = *reinterpret_cast<const uint4*>(a.v + row * a.vs + h * (2 * kD) + 16 * j);
      put_k(to, p, quad_of(j, 0, 0), make_uint2(u.x, u.y), make_uint2(u.z, u.w));
      put_v(to, p, 8 * j, v);
    }
    if (full) {
      __syncthreads();
      quantise_block<ELEM, CODE>(c, buf, page, h, reinterpret_cast<uint32_t*>(sm + (size_t)T * 4 * kD));
    }
    if (!both || b != first) return;
    b = open;
    __syncthreads();
  }
}

// Keys and queries turned without being stored: 16 threads a token, each with the
// angles of eight features for kRotHeads heads, whose loads are in flight together and ahead of
// the two after one another that the angles take. Bound by bytes: 60 600 tokens of 48 heads in
// bf16, three axes in turn (1.46 GB) 219 us, 98% of the copy rate; 16 x 26 drafts of 40
// heads 8.5 us, the latency of a launch and three loads.
constexpr int kRotHeads = 8, kRotThreads = 256;
template <int ELEM>
__global__ void __launch_bounds__(kRotThreads) k_rotate8(Cache8View c, Append8Args a) {
  pdl_launch_dependents();
  pdl_wait();
  if (c.stopped()) return;
  const int hk = a.k ? c.hkv : 0, heads = hk + (a.q ? c.hkv * c.G : 0), parts = (heads + kRotHeads - 1) / kRotHeads;
  const int j = threadIdx.x & 15;
  const long long row = (long long)(blockIdx.x / parts) * (kRotThreads / 16) + (threadIdx.x >> 4);
  const int h0 = (blockIdx.x % parts) * kRotHeads;
  if (row >= a.n_tok || a.pos[row] < 0) return;       // below 0: padding
  const Quad qd = quad_of(j, c.rot, c.inter);
  uint2 u[kRotHeads], v[kRotHeads];
  auto place = [&](int h, const uint8_t* k, long long ks, const uint8_t* q, long long qs) {
    return h < hk ? k + row * ks + h * (2 * kD) : q + row * qs + (h - hk) * (2 * kD);
  };
#pragma unroll
  for (int e = 0; e < kRotHeads; e++)
    if (h0 + e < heads) {
      const uint8_t* p = place(h0 + e, a.k, a.ks, a.q, a.qs);
      u[e] = ld8(p + 2 * qd.a0);
      v[e] = ld8(p + 2 * qd.b0);
    }
  const Rot4 rot = load_rot_at(c, a, axes_of(a, j), row, (int)min(row, 0x7fffffffll), qd);
#pragma unroll
  for (int e = 0; e < kRotHeads; e++)
    if (h0 + e < heads) {
      turn_quad<ELEM>(u[e], v[e], qd, rot, c.inter);
      uint8_t* p = const_cast<uint8_t*>(place(h0 + e, a.k_rot, c.hkv * (2 * kD), a.q_rot, (long long)c.hkv * c.G * (2 * kD)));
      st8(p + 2 * qd.a0, u[e]);
      st8(p + 2 * qd.b0, v[e]);
    }
}

template <int ELEM, int CODE, bool AT>
cudaError_t append_typed(const Cache8View& c, const Append8Args& a, int n_req, const int32_t* n_new, cudaStream_t st) {
  const size_t smem = std::max<size_t>((size_t)c.T * 4 * kD + 256, a.slots ? (size_t)(c.n_slots + 31) / 32 * 4 : 0);
  const unsigned hkv = (unsigned)c.hkv;
  cudaError_t e = cudaSuccess;
  if (!n_new) {
    auto kernel = k_append8_step<ELEM, CODE, AT>;
    if (smem > 48 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(n_req * hkv + 1), dim3(kStepThreads), smem, st, c, a, n_req);
  }
  AppendCall call;
  call.tok0[0] = call.blk0[0] = 0;
  for (int i = 0; i < n_req; i++) {
    call.tok0[i + 1] = call.tok0[i] + n_new[i];
    call.blk0[i + 1] = call.blk0[i] + (n_new[i] + c.T - 2) / c.T + 1;     // blocks that n tokens can touch
  }
  auto kernel = k_append8<ELEM, CODE, AT>;
  if (smem > 48 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, dim3(call.blk0[n_req] * hkv + 1), dim3(4 * c.T), smem, st, c, a, n_req, call);
}

template <int ELEM, int CODE>
cudaError_t append_typed(const Cache8View& c, const Append8Args& a, int n_req, const int32_t* n_new, cudaStream_t st) {
  return a.pos ? append_typed<ELEM, CODE, true>(c, a, n_req, n_new, st)
               : append_typed<ELEM, CODE, false>(c, a, n_req, n_new, st);
}

template <int ELEM, int CODE>
cudaError_t accept_typed(const Cache8View& c, const Accept8Args& a, int n_req, cudaStream_t st) {
  const int jobs = (a.width + c.T - 2) / c.T + 1;     // blocks that a path can touch
  const size_t smem = std::max<size_t>((size_t)c.T * 4 * kD + 256, a.slots ? (size_t)(c.n_slots + 31) / 32 * 4 : 0);
  auto kernel = k_accept8<ELEM, CODE>;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStoreSmem);
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(kernel, dim3((unsigned)(n_req * jobs * c.hkv + 1)), dim3(kAcceptThreads), smem, st, c, a, n_req, jobs);
}

}  // namespace

cudaError_t launch_append8(const Cache8View& c, int elem, int code, const Append8Args& a, int n_req,
                           const int32_t* n_new, cudaStream_t st) {
  if (elem == DKV_F16)
    return code == DKV_E4M3 ? append_typed<DKV_F16, DKV_E4M3>(c, a, n_req, n_new, st)
                            : append_typed<DKV_F16, DKV_INT8>(c, a, n_req, n_new, st);
  return code == DKV_E4M3 ? append_typed<DKV_BF16, DKV_E4M3>(c, a, n_req, n_new, st)
                          : append_typed<DKV_BF16, DKV_INT8>(c, a, n_req, n_new, st);
}

cudaError_t launch_accept8(const Cache8View& c, int elem, int code, const Accept8Args& a, int n_req, cudaStream_t st) {
  if (elem == DKV_F16)
    return code == DKV_E4M3 ? accept_typed<DKV_F16, DKV_E4M3>(c, a, n_req, st) : accept_typed<DKV_F16, DKV_INT8>(c, a, n_req, st);
  return code == DKV_E4M3 ? accept_typed<DKV_BF16, DKV_E4M3>(c, a, n_req, st) : accept_typed<DKV_BF16, DKV_INT8>(c, a, n_req, st);
}

cudaError_t launch_rotate8(const Cache8View& c, int elem, const Append8Args& a, cudaStream_t st) {
  const int heads = (a.k ? c.hkv : 0) + (a.q ? c.hkv * c.G : 0);
  const long long tokens = (a.n_tok + kRotThreads / 16 - 1) / (kRotThreads / 16), parts = (heads + kRotHeads - 1) / kRotHeads;
  return launch_dependent(elem == DKV_F16 ? k_rotate8<DKV_F16> : k_rotate8<DKV_BF16>, dim3((unsigned)(tokens * parts)),
                          dim3(kRotThreads), 0, st, c, a);
}

}  // namespace dkv

// ---------------------------------------------------------------------------
// C ABI
// ---------------------------------------------------------------------------
using namespace dkv;

namespace {

struct Device8 {
  int prev = -1;
  bool ok = true;
  explicit Device8(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
    if (prev != dev) ok = cudaSetDevice(dev) == cudaSuccess;
    want = dev;
  }
  ~Device8() {
    if (prev >= 0 && prev != want) cudaSetDevice(prev);
  }
  int want;
};

// The caller's own next check of CUDA's last error is not to find this call's.
int result(cudaError_t e) {
  if (e == cudaSuccess) return DKV_OK;
  cudaGetLastError();
  return DKV_ERR_CUDA;
}

bool at(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Shape fields only (the pointers may be NULL).
int check_shape(const dkv_cache8* c) {
  if (!c || c->n_kv_heads < 1 || c->n_kv_heads > 4096 || c->n_pages < 1 || c->n_slots < 1 || c->table_width < 1)
    return DKV_ERR_ARG;
  if (c->n_slots > kMaxSlots || c->device < 0) return DKV_ERR_ARG;
  if (c->elem_type != DKV_F16 && c->elem_type != DKV_BF16) return DKV_ERR_ARG;
  if (c->code_type != DKV_E4M3 && c->code_type != DKV_INT8) return DKV_ERR_ARG;
  if (c->rotary_dim < 0 || c->rotary_dim > kD || c->rotary_dim % 16) return DKV_ERR_ARG;
  if (c->rotary_interleaved != 0 && c->rotary_interleaved != 1) return DKV_ERR_ARG;
  const int t = c->block_tokens;
  if (t != 16 && t != 32 && t != 64 && t != 128) return DKV_ERR_UNSUPPORTED;
  if (c->head_dim != kD || c->group_size < 1 || c->group_size > kMaxG) return DKV_ERR_UNSUPPORTED;
  // positions and lengths are 32-bit
  if ((long long)c->table_width * t > 0x7fffff00ll) return DKV_ERR_ARG;
  return DKV_OK;
}

int check_cache(const dkv_cache8* c, bool store) {
  const int rc = check_shape(c);
  if (rc) return rc;
  if (!c->status || !at(c->status, 4)) return DKV_ERR_ARG;
  if (store) {
    if (!c->pages || !c->scales || !c->tail || !c->page_table) return DKV_ERR_ARG;
    if (!at(c->pages, 16) || !at(c->tail, 16) || !at(c->scales, 8) || !at(c->page_table, 4)) return DKV_ERR_ARG;
  }
  return DKV_OK;
}

// Vector rows: 16-byte aligned, rows of at least `heads` heads.
bool rows_ok(const void* p, int64_t stride, int heads) {
  return p && at(p, 16) && stride >= (int64_t)heads * kD && stride % 8 == 0 && stride < (1ll << 38);
}

Cache8View view(const dkv_cache8* c) {
  Cache8View v;
  v.pages = static_cast<uint8_t*>(c->pages);
  v.scales = c->scales;
  v.tail = static_cast<uint8_t*>(c->tail);
  v.table = c->page_table;
  v.status = c->status;
  v.hkv = c->n_kv_heads;
  v.G = c->group_size;
  v.T = c->block_tokens;
  v.n_pages = c->n_pages;
  v.n_slots = c->n_slots;
  v.width = c->table_width;
  v.rot = c->rotary_dim;
  v.inter = c->rotary_interleaved;
  return v;
}

// Positions of a call's tokens and the axis of each pair of features.
struct Turn {
  const int32_t* positions;
  int32_t n_axes;
  const uint8_t* pair_axis;
  int fill(const dkv_cache8* c, long long n_tok, Append8Args& a) const {
    if (!c->rotary_dim || !positions || !at(positions, 4) || n_axes < 1 || n_axes > kMaxAxes || (n_axes > 1 && !pair_axis))
      return DKV_ERR_ARG;
    for (int i = 0; i < kD / 2; i++) a.axis[i] = 0;
    for (int i = 0; pair_axis && i < c->rotary_dim / 2; i++) {
      if (pair_axis[i] >= n_axes) return DKV_ERR_ARG;
      a.axis[i] = pair_axis[i];
    }
    a.pos = positions;
    a.n_tok = n_tok;
    return DKV_OK;
  }
};

int sm_count(int device) {
  int n = 0;
  return cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) == cudaSuccess ? n : 0;
}

int append(const dkv_cache8* cache, int32_t n_req, const int32_t* n_new, const int32_t* slots, const int32_t* before,
           const Turn* turn, const void* k, int64_t k_stride, const void* v, int64_t v_stride, const void* q,
           int64_t q_stride, const float* rope, int32_t rope_len, void* k_rot, void* q_rot, void* stream) {
  const int rc = check_cache(cache, true);
  if (rc) return rc;
  if (n_req < 1 || n_req > kMaxCallReq || !before || !at(before, 4) || !at(slots, 4)) return DKV_ERR_ARG;
  if (!slots && n_req > cache->n_slots) return DKV_ERR_ARG;
  const int hkv = cache->n_kv_heads, hq = hkv * cache->group_size;
  if (!rows_ok(k, k_stride, hkv) || !rows_ok(v, v_stride, hkv)) return DKV_ERR_ARG;
  if ((q != nullptr) != (q_rot != nullptr) || (q && !rows_ok(q, q_stride, hq))) return DKV_ERR_ARG;
  if (!at(k_rot, 16) || !at(q_rot, 16)) return DKV_ERR_ARG;
  if (k_rot == k && k_stride != (int64_t)hkv * kD) return DKV_ERR_ARG;
  if (q && q_rot == q && q_stride != (int64_t)hq * kD) return DKV_ERR_ARG;
  if ((cache->rotary_dim != 0) != (rope != nullptr) || !at(rope, 16)) return DKV_ERR_ARG;
  if (rope && rope_len < 1) return DKV_ERR_ARG;
  long long tok = n_req, blk = 0;
  if (n_new) {
    tok = 0;
    const int t = cache->block_tokens;
    for (int i = 0; i < n_req; i++) {
      if (n_new[i] < 1 || n_new[i] > (long long)cache->table_width * t) return DKV_ERR_ARG;
      tok += n_new[i];
      blk += (n_new[i] + t - 2) / t + 1;
      if (tok > 0x7fffffffll || blk * hkv > 0x7ffffff0ll) return DKV_ERR_ARG;   // rows and jobs are 32-bit
    }
  }
  Append8Args a;
  if (turn) {
    const int e = turn->fill(cache, tok, a);
    if (e) return e;
  } else {
    a.pos = nullptr;
  }
  Device8 dev(cache->device);
  if (!dev.ok) return result(cudaErrorInvalidDevice);
  a.k = static_cast<const uint8_t*>(k);
  a.v = static_cast<const uint8_t*>(v);
  a.q = static_cast<const uint8_t*>(q);
  a.ks = 2 * k_stride;
  a.vs = 2 * v_stride;
  a.qs = 2 * q_stride;
  a.rope = reinterpret_cast<const float2*>(rope);
  a.rope_len = rope_len;
  a.k_rot = static_cast<uint8_t*>(k_rot);
  a.q_rot = static_cast<uint8_t*>(q_rot);
  a.slots = slots;
  a.before = before;
  const cudaError_t e = launch_append8(view(cache), cache->elem_type, cache->code_type, a, n_req, n_new,
                                       reinterpret_cast<cudaStream_t>(stream));
  return result(e);
}

}  // namespace

extern "C" {

int dkv_cache8_workspace(const dkv_cache8* cache, int32_t max_req, int64_t* bytes) {
  const int rc = check_shape(cache);
  if (rc) return rc;
  if (!bytes || max_req < 1 || max_req > kMaxCallReq) return DKV_ERR_ARG;
  const int sms = sm_count(cache->device);
  if (!sms) return result(cudaErrorInvalidDevice);
  *bytes = (int64_t)attention8_workspace(cache->n_kv_heads, cache->group_size, max_req, sms);
  return DKV_OK;
}

int dkv_cache8_append(const dkv_cache8* cache, int32_t n_req, const int32_t* n_new, const int32_t* slots,
                      const int32_t* before, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                      const void* q, int64_t q_stride, const float* rope, int32_t rope_len, void* k_rot,
                      void* q_rot, void* stream) {
  return append(cache, n_req, n_new, slots, before, nullptr, k, k_stride, v, v_stride, q, q_stride, rope, rope_len, k_rot,
                q_rot, stream);
}

int dkv_cache8_append_at(const dkv_cache8* cache, int32_t n_req, const int32_t* n_new, const int32_t* slots,
                         const int32_t* before, const int32_t* positions, int32_t n_axes, const uint8_t* pair_axis,
                         const void* k, int64_t k_stride, const void* v, int64_t v_stride, const void* q, int64_t q_stride,
                         const float* rope, int32_t rope_len, void* k_rot, void* q_rot, void* stream) {
  const Turn turn{positions, n_axes, pair_axis};
  return append(cache, n_req, n_new, slots, before, &turn, k, k_stride, v, v_stride, q, q_stride, rope, rope_len, k_rot,
                q_rot, stream);
}

int dkv_cache8_rotate(const dkv_cache8* cache, int32_t n_tok, const int32_t* positions, int32_t n_axes,
                      const uint8_t* pair_axis, const void* k, int64_t k_stride, const void* q, int64_t q_stride,
                      const float* rope, int32_t rope_len, void* k_rot, void* q_rot, void* stream) {
  const int rc = check_cache(cache, false);
  if (rc) return rc;
  const int hkv = cache->n_kv_heads, hq = hkv * cache->group_size;
  if (n_tok < 1 || (!k && !q) || (k != nullptr) != (k_rot != nullptr) || (q != nullptr) != (q_rot != nullptr)) return DKV_ERR_ARG;
  if ((k && !rows_ok(k, k_stride, hkv)) || (q && !rows_ok(q, q_stride, hq)) || !at(k_rot, 16) || !at(q_rot, 16)) return DKV_ERR_ARG;
  if (k && k_rot == k && k_stride != (int64_t)hkv * kD) return DKV_ERR_ARG;
  if (q && q_rot == q && q_stride != (int64_t)hq * kD) return DKV_ERR_ARG;
  if (!rope || !at(rope, 16) || rope_len < 1) return DKV_ERR_ARG;
  // blocks of 16 tokens and 8 heads are numbered in 32 bits
  if (((long long)n_tok / 16 + 1) * ((hkv + hq) / 8 + 1) > 0x7ffffff0ll) return DKV_ERR_ARG;
  Append8Args a;
  const int e = Turn{positions, n_axes, pair_axis}.fill(cache, n_tok, a);
  if (e) return e;
  Device8 dev(cache->device);
  if (!dev.ok) return result(cudaErrorInvalidDevice);
  a.k = static_cast<const uint8_t*>(k);
  a.v = nullptr;
  a.q = static_cast<const uint8_t*>(q);
  a.ks = 2 * k_stride;
  a.vs = 0;
  a.qs = 2 * q_stride;
  a.rope = reinterpret_cast<const float2*>(rope);
  a.rope_len = rope_len;
  a.k_rot = static_cast<uint8_t*>(k_rot);
  a.q_rot = static_cast<uint8_t*>(q_rot);
  a.slots = a.before = nullptr;
  return result(launch_rotate8(view(cache), cache->elem_type, a, reinterpret_cast<cudaStream_t>(stream)));
}

int dkv_cache8_accept(const dkv_cache8* cache, int32_t n_req, const int32_t* slots, const int32_t* before,
                      int32_t max_nodes, const int32_t* path, int32_t path_width, const int32_t* n_path, const void* k,
                      int64_t k_stride, const void* v, int64_t v_stride, void* stream) {
  const int rc = check_cache(cache, true);
  if (rc) return rc;
  if (n_req < 1 || n_req > kMaxCallReq || !before || !at(before, 4) || !at(slots, 4)) return DKV_ERR_ARG;
  if (!slots && n_req > cache->n_slots) return DKV_ERR_ARG;
  if (max_nodes < 1 || max_nodes > kMaxNodes || path_width < 1 || path_width > kMaxNodes) return DKV_ERR_ARG;
  if (!path || !at(path, 4) || !at(n_path, 4)) return DKV_ERR_ARG;
  const int hkv = cache->n_kv_heads;
  if (!rows_ok(k, k_stride, hkv) || !rows_ok(v, v_stride, hkv)) return DKV_ERR_ARG;
  Device8 dev(cache->device);
  if (!dev.ok) return result(cudaErrorInvalidDevice);
  const Accept8Args a{static_cast<const uint8_t*>(k), static_cast<const uint8_t*>(v), 2 * k_stride, 2 * v_stride,
                      slots, before, path, n_path, max_nodes, path_width};
  return result(launch_accept8(view(cache), cache->elem_type, cache->code_type, a, n_req, reinterpret_cast<cudaStream_t>(stream)));
}

int dkv_cache8_tree_workspace(const dkv_cache8* cache, int32_t max_nodes, int64_t* bytes) {
  const int rc = check_shape(cache);
  if (rc) return rc;
  if (!bytes || max_nodes < 1 || max_nodes > kMaxNodes) return DKV_ERR_ARG;
  const int sms = sm_count(cache->device);
  if (!sms) return result(cudaErrorInvalidDevice);
  *bytes = (int64_t)tree8_workspace(cache->group_size, max_nodes, sms);
  return DKV_OK;
}

int dkv_cache8_tree(const dkv_cache8* cache, int32_t n_req, const int32_t* slots, const int32_t* seq_lens,
                    int32_t max_nodes, const int32_t* n_nodes, const int32_t* parents, const void* q, int64_t q_stride,
                    const void* k, int64_t k_stride, const void* v, int64_t v_stride, void* out, int32_t window,
                    int32_t sinks, void* workspace, int64_t workspace_bytes, void* stream) {
  const int rc = check_cache(cache, true);
  if (rc) return rc;
  if (n_req < 1 || n_req > kMaxCallReq || !seq_lens || !at(seq_lens, 4) || !at(slots, 4)) return DKV_ERR_ARG;
  if (!slots && n_req > cache->n_slots) return DKV_ERR_ARG;
  if (max_nodes < 1 || max_nodes > kMaxNodes || !at(n_nodes, 4) || !at(parents, 4)) return DKV_ERR_ARG;
  const int hkv = cache->n_kv_heads, hq = hkv * cache->group_size;
  if (!rows_ok(q, q_stride, hq) || !rows_ok(k, k_stride, hkv) || !rows_ok(v, v_stride, hkv)) return DKV_ERR_ARG;
  if (!out || !at(out, 16) || out == q || out == k || out == v || window < 0 || sinks < 0) return DKV_ERR_ARG;
  const long long most = (long long)cache->table_width * cache->block_tokens;
  // steps of 128 tokens (and a few for each unit) and rows of the whole call are numbered in 32 bits
  const long long tiles = (max_nodes * cache->group_size + 127) / 128, steps = (most + 2 * kSub + max_nodes + 63) / 64 + 8;
  if ((long long)n_req * hkv * tiles > 0x7ffffff0ll / steps || (long long)n_req * max_nodes * hq > 0x7ffffff0ll) return DKV_ERR_ARG;
  if (!workspace || !at(workspace, 16)) return DKV_ERR_ARG;
  Device8 dev(cache->device);
  if (!dev.ok) return result(cudaErrorInvalidDevice);
  const int sms = sm_count(cache->device);
  if (!sms) return result(cudaErrorInvalidDevice);
  if (workspace_bytes < (int64_t)tree8_workspace(cache->group_size, max_nodes, sms)) return DKV_ERR_SCRATCH;
  // a window that no position exceeds is none (and positions minus it stay in 32 bits)
  if (window >= most + max_nodes) window = 0;
  const Tree8Args a{slots, seq_lens, n_nodes, parents, static_cast<const uint8_t*>(q), static_cast<const uint8_t*>(k),
                    static_cast<const uint8_t*>(v), 2 * q_stride, 2 * k_stride, 2 * v_stride, static_cast<uint8_t*>(out),
                    n_req, max_nodes, window, sinks, static_cast<float*>(workspace)};
  return result(launch_tree8(view(cache), cache->elem_type, cache->code_type, sms, a, reinterpret_cast<cudaStream_t>(stream)));
}

int dkv_cache8_attention(const dkv_cache8* cache, int32_t n_req, const int32_t* slots, const int32_t* seq_lens,
                         const void* q, int64_t q_stride, void* out, int32_t window, int32_t sinks,
                         void* stream) {
  const int rc = check_cache(cache, true);
  if (rc) return rc;
  if (n_req < 1 || n_req > kMaxCallReq || !seq_lens || !at(seq_lens, 4) || !at(slots, 4)) return DKV_ERR_ARG;
  if (!slots && n_req > cache->n_slots) return DKV_ERR_ARG;
  const int hkv = cache->n_kv_heads, hq = hkv * cache->group_size;
  if (!rows_ok(q, q_stride, hq) || !out || out == q || !at(out, 16) || window < 0 || sinks < 0) return DKV_ERR_ARG;
  // tiles of the whole call are numbered in 32 bits
  if ((long long)n_req * hkv * ((long long)cache->table_width * cache->block_tokens / kSub + 1) > 0x7ffffff0ll)
    return DKV_ERR_ARG;
  if (!cache->workspace || !at(cache->workspace, 16)) return DKV_ERR_ARG;
  Device8 dev(cache->device);
  if (!dev.ok) return result(cudaErrorInvalidDevice);
  const int sms = sm_count(cache->device);
  if (!sms) return result(cudaErrorInvalidDevice);
  if (cache->workspace_bytes < (int64_t)attention8_workspace(hkv, cache->group_size, n_req, sms)) return DKV_ERR_SCRATCH;
  // a window that no length exceeds is none (and positions minus it stay in 32 bits)
  if (window >= (long long)cache->table_width * cache->block_tokens) window = 0;
  const cudaError_t e =
      launch_attention8(view(cache), cache->elem_type, cache->code_type, sms, slots, seq_lens, n_req, q, q_stride, out,
                        window, sinks, cache->workspace, reinterpret_cast<cudaStream_t>(stream));
  return result(e);
}

int dkv_cache8_prefill(const dkv_cache8* cache, int32_t n_req, const int32_t* seq_lens, const void* q,
                       int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                       void* out, int32_t window, int32_t sinks, void* stream) {
  const int rc = check_cache(cache, false);
  if (rc) return rc;
  if (n_req < 1 || n_req > kMaxCallReq || !seq_lens || window < 0 || sinks < 0) return DKV_ERR_ARG;
  const int hkv = cache->n_kv_heads, hq = hkv * cache->group_size;
  if (!rows_ok(q, q_stride, hq) || !rows_ok(k, k_stride, hkv) || !rows_ok(v, v_stride, hkv)) return DKV_ERR_ARG;
  if (!out || !at(out, 16) || out == q || out == k || out == v) return DKV_ERR_ARG;
  long long tok = 0, tiles = 0;
  int longest = 0;
  const int tq = 128 / cache->group_size;
  for (int i = 0; i < n_req; i++) {
    if (seq_lens[i] < 1) return DKV_ERR_ARG;
    longest = std::max(longest, seq_lens[i]);
    tok += seq_lens[i];
    tiles += (seq_lens[i] + (long long)tq - 1) / tq;
    if (tok > 0x7fffff00ll || tiles * hkv > 0x7ffffff0ll) return DKV_ERR_ARG;   // rows and tiles are 32-bit
  }
  Device8 dev(cache->device);
  if (!dev.ok) return result(cudaErrorInvalidDevice);
  const int sms = sm_count(cache->device);
  if (!sms) return result(cudaErrorInvalidDevice);
  if (window >= longest) window = 0;   // as above
  const cudaError_t e = launch_prefill8(view(cache), cache->elem_type, seq_lens, n_req, q, q_stride, k, k_stride, v,
                                        v_stride, out, window, sinks, sms, reinterpret_cast<cudaStream_t>(stream));
  return result(e);
}

}  // extern "C"
