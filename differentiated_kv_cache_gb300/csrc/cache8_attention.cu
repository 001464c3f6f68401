// cache8_attention.cu — decode attention over the uniform 8-bit cache, in full
// or through a sliding window with first tokens that stay visible
// (include/dkv.h: dkv_cache8_attention).
//
// The tiles of all (request, KV head) units, 16 tokens of 4 KB of codes each,
// form one sequence that is cut into equal contiguous ranges, one per CTA of a
// persistent grid and of those one per warp: a long unit spreads over the GPU,
// short ones share a warp, and lengths are read on the device (a captured call
// replays with others). A warp streams its tiles through a ring of bulk
// copies; a unit inside one warp's range is written by it, one inside a CTA is
// joined in shared memory, and one that crosses CTAs leaves a partial per CTA
// in the workspace, which the CTA that arrives last joins in order (the result
// does not depend on who that is).
//
// Bound by DRAM: 32 requests of 4096 tokens with 8 KV heads (273 MB) take 48 us,
// 5.7 TB/s or 84% of the measured copy rate; 35 of them stream at 7.7 TB/s, the
// rest is launch, the chain lengths - page table - first tile (3.5 us), CTAs
// that DRAM serves at uneven rates (4 us) and the joins (3 us). 8 x 32768 with 64
// query heads: 89 us, 89%. One CTA of 12 warps with two 4 KB copies each on
// their way: three copies queue up at DRAM and part the CTAs' ends further
// (50.4 us), 8 warps leave the matrix and conversion chain of a tile exposed
// (54 us), 16 have too few registers (52 us, 8 x 32768: 119 us). One CTA per
// (request, KV head) took 52 and 297 us. Both sums under one maximum, which loses
// tokens of zero values beside large ones, took 0.3 us less (269 instructions a tile
// instead of 289).
//
// A warp's step on a tile of codes, S^T = K Q^T and O^T += V^T P^T with
// mma.sync m16n8k16 (tokens / features on M, the G <= 8 queries on N; at most
// 8 rows of queries cannot fill a tcgen05 tile, and the kernel is bound by
// memory, not by matrix rate):
//   y_j  = s_k (q . code_j) log2(e) / sqrt(128),   x_j = y_j + log2(s_v)
//   w_j  = 2^(x_j - m)        the probability times V's scale, up to 2^-m
//   O   += w_j code_j,   l += 2^(y_j - u),   out = O 2^(m - u) / l
// so that blocks with different V scales need no rescaling of O. m and u are
// running maxima of x and y. Each sum has its own: s_v lies in 2^-100 .. 2^121,
// and a block of zeros, which adds nothing to O, has its full weight in l beside
// blocks of any size. They are raised (O, l rescaled) only when some x_j exceeds m
// by more than 8 (w stays below 2^8, in fp16's range) or some y_j exceeds u by
// more than 5 (2^(m - u) stays below 2^127). w enters the second product rounded
// to fp16 (relative 2^-11, the size of the output's own rounding); l sums the
// unrounded fp32 values.
// Tiles of the 16-bit tail take s_k = s_v = 1 where there are no codes to mix
// with; else s_v is the power of two that brings their largest |v| to
// [128, 256), the size of codes, so that equal weights stand for equal
// contributions; their values are divided by it (exact but for values 2^-20 and
// less of the largest).
#include <algorithm>

#include "cache8.cuh"
#include "dkv_kernels.cuh"

namespace dkv {
namespace {

constexpr int kA8Warps = 12;
constexpr int kA8Stages = 2;        // ring entries of a warp
constexpr int kA8Entry = 2 * kTile; // 4 KB: K and V codes of a tile, or K or V of a tail tile
constexpr int kA8Row = kD + 4;      // floats of a query's row in a shared partial (no bank conflicts)
constexpr int kA8Cta = 2 * kA8Warps;    // tiles that make a CTA worth its start
constexpr float kA8Lazy = 8.0f, kA8LazySum = 5.0f;     // how far x may pass m, y pass u
// bf16 values of a tail alone, which are not scaled: m lies this much above the
// maximum, so that 127 weights of up to 2^8 sum to less than 1 and their
// products stay in fp32's range
constexpr float kA8Above = 15.0f;

struct Attn8Args {
  const int *slots, *seq_lens;
  const uint8_t* q;
  long long qs;      // bytes
  uint8_t* out;
  int n_req, window, sinks;
  unsigned* count;   // arrivals of CTAs, per query row; zero between calls
  float* part;       // [CTA][2]: G rows of 128, then 8 maxima, 8 sums
};

// Tiles of one request: [0, head) from its start, [win, end) behind them; the
// tiles from `full` on lie in the tail.
struct Tiles {
  int head, win, end, full, count;
};
__device__ __forceinline__ Tiles tiles_of(int N, int T, int window, int sinks) {
  Tiles t;
  t.end = (N + kSub - 1) / kSub;
  t.full = N / T * (T / kSub);
  t.head = 0;
  t.win = 0;
  if (window > 0 && window < N) {
    t.win = (N - window) / kSub;
    t.head = min((min(sinks, N) + kSub - 1) / kSub, t.win);
  }
  t.count = t.head + t.end - t.win;
  return t;
}

template <int CODE>
__device__ __forceinline__ void code_halves(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (CODE == DKV_E4M3) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    // byte b + 128 under the exponent of 1024, then 1152 off: exact
    const uint32_t u = w ^ 0x80808080u;
    lo = hsub2_u(prmt(u, 0x64646464u, 0x4140u), 0x64806480u);
    hi = hsub2_u(prmt(u, 0x64646464u, 0x4342u), 0x64806480u);
  }
}

// Running state of a warp for one (request, KV head): lane 4g + t holds
// queries 2t, 2t + 1; O rows are features 16 m + g and 16 m + g + 8.
struct State {
  float o[8][4];
  float m[2], u[2], l[2];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; i++)
#pragma unroll
      for (int e = 0; e < 4; e++) o[i][e] = 0.0f;
    m[0] = m[1] = u[0] = u[1] = -INFINITY;
    l[0] = l[1] = 0.0f;
  }
};

// Raise the running maxima where some x or y = x - lv exceeds them by more than
// the slack. x: tokens g (x[0], x[1]) and g + 8 (x[2], x[3]) for the lane's two
// queries; above: how far m lies above the maximum.
__device__ __forceinline__ void raise(State& s, const float* x, float lv, float above) {
  float a = fmaxf(x[0], x[2]), b = fmaxf(x[1], x[3]);
  if (!__any_sync(0xffffffffu, a > fminf(s.m[0] + (kA8Lazy - above), s.u[0] + (lv + kA8LazySum)) ||
                                   b > fminf(s.m[1] + (kA8Lazy - above), s.u[1] + (lv + kA8LazySum))))
    return;
#pragma unroll
  for (int d = 4; d <= 16; d <<= 1) {
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
    b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, d));
  }
  auto up = [](float& top, float x) {      // the factor of what was summed below the old maximum
    const float old = top;
    top = fmaxf(old, x);
    return top == -INFINITY ? 1.0f : fast_exp2(old - top);
  };
  const float fa = up(s.m[0], a + above), fb = up(s.m[1], b + above);
  s.l[0] *= up(s.u[0], a - lv);
  s.l[1] *= up(s.u[1], b - lv);
#pragma unroll
  for (int i = 0; i < 8; i++) {
    s.o[i][0] *= fa;
    s.o[i][1] *= fb;
    s.o[i][2] *= fa;
    s.o[i][3] *= fb;
  }
}

// w = 2^(x - m) in place of x, and 2^(x - lv - u) summed into l.
__device__ __forceinline__ void weights(State& s, float* x, float lv) {
#pragma unroll
  for (int e = 0; e < 2; e++) {
    const float m = s.m[e] == -INFINITY ? 0.0f : s.m[e], u = s.u[e] == -INFINITY ? 0.0f : s.u[e] + lv;
    s.l[e] += fast_exp2(x[e] - u) + fast_exp2(x[e + 2] - u);
    x[e] = fast_exp2(x[e] - m);
    x[e + 2] = fast_exp2(x[e + 2] - m);
  }
}

// Which tokens of a tile the query sees, for this lane: logits of tokens g and
// g + 8, and the V entries of tokens 2t, 2t+1, 2t+8, 2t+9 (one byte each).
struct See {
  bool lo, hi;
  uint32_t v;
};
// every token of a tile
__device__ __forceinline__ bool sees_all(int pos0, int N, int window) {
  return pos0 + kSub <= N && (window <= 0 || pos0 >= N - window);
}
__device__ __forceinline__ See see_of(int pos0, int N, int window, int sinks, int lane) {
  See s;
  const int from = window > 0 ? N - window : 0;
  auto sees = [&](int i) { return pos0 + i < N && (pos0 + i >= from || pos0 + i < sinks); };
  const int g = lane >> 2, t = lane & 3;
  s.lo = sees(g);
  s.hi = sees(g + 8);
  s.v = (sees(2 * t) ? 0xffu : 0u) | (sees(2 * t + 1) ? 0xff00u : 0u) | (sees(2 * t + 8) ? 0xff0000u : 0u) |
        (sees(2 * t + 9) ? 0xff000000u : 0u);
  return s;
}

// A lane's 64 bytes of K or V codes from shared memory.
__device__ __forceinline__ void load_codes(const uint8_t* p, uint4 (&w)[4]) {
#pragma unroll
  for (int j = 0; j < 4; j++) w[j] = *reinterpret_cast<const uint4*>(p + 512 * j);
}

// A tile of codes at p (K, then V); edge: some token may not be visible.
template <int CODE>
__device__ __forceinline__ void code_tile(State& s, const uint32_t (&qf)[16], const uint8_t* p, bool edge,
                                          const See& see, const float (&ks)[2], float lv) {
  uint4 kw[4];
  load_codes(p, kw);
  float x[4] = {0.0f, 0.0f, 0.0f, 0.0f}, y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < 4; j++) {
    uint32_t a[4];
    code_halves<CODE>(kw[j].x, a[0], a[2]);
    code_halves<CODE>(kw[j].y, a[1], a[3]);
    mma16816(x, a, qf[4 * j], qf[4 * j + 1]);
    code_halves<CODE>(kw[j].z, a[0], a[2]);
    code_halves<CODE>(kw[j].w, a[1], a[3]);
    mma16816(y, a, qf[4 * j + 2], qf[4 * j + 3]);
  }
#pragma unroll
  for (int e = 0; e < 4; e++) x[e] = fmaf(x[e] + y[e], ks[e & 1], lv);
  uint4 vw[4];
  load_codes(p + kTile, vw);
  if (edge) {
#pragma unroll
    for (int e = 0; e < 4; e++) x[e] = (e < 2 ? see.lo : see.hi) ? x[e] : -INFINITY;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      vw[j].x &= see.v;
      vw[j].y &= see.v;
      vw[j].z &= see.v;
      vw[j].w &= see.v;
    }
  }
  raise(s, x, lv, 0.0f);
  weights(s, x, lv);
  const uint32_t b0 = movmatrix_trans(pack_half2(x[0], x[1])), b1 = movmatrix_trans(pack_half2(x[2], x[3]));
#pragma unroll
  for (int j = 0; j < 4; j++) {
    uint32_t a[4];
    code_halves<CODE>(vw[j].x, a[0], a[2]);
    code_halves<CODE>(vw[j].y, a[1], a[3]);
    mma16816(s.o[2 * j], a, b0, b1);
    code_halves<CODE>(vw[j].z, a[0], a[2]);
    code_halves<CODE>(vw[j].w, a[1], a[3]);
    mma16816(s.o[2 * j + 1], a, b0, b1);
  }
}

template <int ELEM>
__device__ __forceinline__ uint32_t scale_pair(uint32_t w, float f) {   // f: a power of two
  if (ELEM == DKV_F16) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&w), __float2half2_rn(f));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), __float2bfloat162_rn(f));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Query fragments of a (request, KV head).
template <int ELEM>
__device__ __forceinline__ void load_q(const uint8_t* q, int G, int lane, uint32_t (&raw)[16]) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int m = 0; m < 8; m++) {
    const uint8_t* p = q + (size_t)g * (2 * kD) + 2 * (16 * m + 2 * t);
    raw[2 * m] = g < G ? *reinterpret_cast<const uint32_t*>(p) : 0u;
    raw[2 * m + 1] = g < G ? *reinterpret_cast<const uint32_t*>(p + 16) : 0u;
  }
}
__device__ __forceinline__ uint32_t umax2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// A tile of the 16-bit tail: kp points to the lane's first 16 bytes of K,
// after_k() gives V's once K is read; the next steps lie 512 bytes on. qf: the
// queries in elem_type.
template <int ELEM, typename AfterK>
__device__ __forceinline__ void tail_tile(State& s, const uint32_t (&qf)[16], const uint8_t* kp, AfterK after_k,
                                          bool edge, const See& see, bool mixed, float ks) {
  float x[4] = {0.0f, 0.0f, 0.0f, 0.0f}, y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int m = 0; m < 8; m++) {
    const uint4 w = *reinterpret_cast<const uint4*>(kp + 512 * m);
    const uint32_t a[4] = {w.x, w.z, w.y, w.w};
    mma_elem<ELEM>(m & 1 ? y : x, a, qf[2 * m], qf[2 * m + 1]);
  }
  const uint8_t* vp = after_k();
  uint4 v[8];
#pragma unroll
  for (int m = 0; m < 8; m++) v[m] = *reinterpret_cast<const uint4*>(vp + 512 * m);
#pragma unroll
  for (int e = 0; e < 4; e++) x[e] = (x[e] + y[e]) * ks;
  if (edge) {
    // entries of tokens that are not visible (unwritten ones too) become 0
    const uint32_t lo = prmt(see.v, 0, 0x1100u), hi = prmt(see.v, 0, 0x3322u);
#pragma unroll
    for (int m = 0; m < 8; m++) {
      v[m].x &= lo;
      v[m].y &= hi;
      v[m].z &= lo;
      v[m].w &= hi;
    }
#pragma unroll
    for (int e = 0; e < 4; e++) x[e] = (e < 2 ? see.lo : see.hi) ? x[e] : -INFINITY;
  }
  float lv = 0.0f, above = ELEM == DKV_BF16 ? kA8Above : 0.0f;
  if (mixed) {
    above = 0.0f;
    uint32_t am2 = 0;        // magnitudes order like their bits
#pragma unroll
    for (int m = 0; m < 8; m++)
      am2 = umax2(umax2(am2, v[m].x & 0x7fff7fffu), umax2(umax2(v[m].y & 0x7fff7fffu, v[m].z & 0x7fff7fffu), v[m].w & 0x7fff7fffu));
    const float am = elem_float<ELEM>((uint16_t)__reduce_max_sync(0xffffffffu, max(am2 & 0xffffu, am2 >> 16)));
    // exponents that fp16 factors (or the scale floor) allow; infinite or NaN
    // values leave 1
    const int low = ELEM == DKV_F16 ? -14 : -100, high = ELEM == DKV_F16 ? 14 : 100;
    const int ex = am < INFINITY ? max(low, min(high, (int)(__float_as_uint(am) >> 23) - (127 + 7))) : 0;
    const float inv = __uint_as_float((uint32_t)(127 - ex) << 23);
    lv = (float)ex;
#pragma unroll
    for (int e = 0; e < 4; e++) x[e] += lv;
#pragma unroll
    for (int m = 0; m < 8; m++) {
      v[m].x = scale_pair<ELEM>(v[m].x, inv);
      v[m].y = scale_pair<ELEM>(v[m].y, inv);
      v[m].z = scale_pair<ELEM>(v[m].z, inv);
      v[m].w = scale_pair<ELEM>(v[m].w, inv);
    }
  }
  raise(s, x, lv, above);
  weights(s, x, lv);
  uint32_t p0 = pack_elems<ELEM>(x[0], x[1]), p1 = pack_elems<ELEM>(x[2], x[3]);
  const uint32_t b0 = movmatrix_trans(p0), b1 = movmatrix_trans(p1);
  uint32_t r0 = 0, r1 = 0;
  if (ELEM == DKV_BF16) {   // what bf16 rounds away (8 bits are fewer than the fp16 of the other tiles keep)
    r0 = movmatrix_trans(pack_elems<ELEM>(x[0] - lo_elem<ELEM>(p0), x[1] - hi_elem<ELEM>(p0)));
    r1 = movmatrix_trans(pack_elems<ELEM>(x[2] - lo_elem<ELEM>(p1), x[3] - hi_elem<ELEM>(p1)));
  }
#pragma unroll
  for (int m = 0; m < 8; m++) {
    const uint32_t a[4] = {v[m].x, v[m].z, v[m].y, v[m].w};
    mma_elem<ELEM>(s.o[m], a, b0, b1);
    if (ELEM == DKV_BF16) mma_elem<ELEM>(s.o[m], a, r0, r1);
  }
}

// bf16 queries as fp16 after division by the power of two below the row's
// largest |q| (8 bits fit; what falls below fp16's range is under 2^-24 of that
// largest). scale: the power of two of the lane's queries 2t, 2t + 1.
__device__ __forceinline__ void half_q(uint32_t (&qf)[16], int lane, float (&scale)[2]) {
  float am = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; i++)
    am = amax_finite(amax_finite(am, lo_elem<DKV_BF16>(qf[i])), hi_elem<DKV_BF16>(qf[i]));
  am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
  am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
  const int ex = max(-126, min(126, (int)(__float_as_uint(am) >> 23) - 127));     // both powers are normal numbers
  const float inv = __uint_as_float((uint32_t)(127 - ex) << 23), sc = __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
  for (int i = 0; i < 16; i++) qf[i] = pack_half2(lo_elem<DKV_BF16>(qf[i]) * inv, hi_elem<DKV_BF16>(qf[i]) * inv);
  const int t = lane & 3;      // row of query 2t: lanes 4 (2t) ..
  scale[0] = __shfl_sync(0xffffffffu, sc, 8 * t);
  scale[1] = __shfl_sync(0xffffffffu, sc, 8 * t + 4);
}

// A unit that one warp holds whole: out = O 2^(m - u) / l, two features a store.
template <int ELEM>
__device__ __forceinline__ void write_unit(const State& s, uint8_t* out, int G, int lane) {
  const int g = lane >> 2, t = lane & 3, odd = g & 1, q = 2 * t + odd;
  const float ia = __fdiv_rn(fast_exp2(s.m[0] - s.u[0]), s.l[0]), ib = __fdiv_rn(fast_exp2(s.m[1] - s.u[1]), s.l[1]);
  uint32_t bad = 0;
#pragma unroll
  for (int m = 0; m < 8; m++)
#pragma unroll
    for (int e = 0; e < 2; e++) {
      const float a = s.o[m][2 * e] * ia, b = s.o[m][2 * e + 1] * ib;
      const float other = __shfl_xor_sync(0xffffffffu, odd ? a : b, 4);
      const uint32_t w = odd ? pack_elems<ELEM>(other, b) : pack_elems<ELEM>(a, other);
      find_not_finite<ELEM>(bad, w);
      if (q < G) *reinterpret_cast<uint32_t*>(out + (size_t)q * (2 * kD) + 2 * (16 * m + 8 * e + g - odd)) = w;
    }
  if (__builtin_expect(__any_sync(0xffffffffu, found_not_finite(bad)), 0)) {
    // seldom: each lane its own features, within the type's range
    __syncwarp();
#pragma unroll
    for (int m = 0; m < 8; m++)
#pragma unroll
      for (int e = 0; e < 4; e++)
        if (2 * t + (e & 1) < G)
          reinterpret_cast<uint16_t*>(out)[(2 * t + (e & 1)) * kD + 16 * m + 8 * (e >> 1) + g] =
              float_elem<ELEM>(in_range<ELEM>(s.o[m][e] * (e & 1 ? ib : ia)));
  }
}

// A partial: the part's own result, so that its size is that of its values, and
// its weight as l 2^m with l in [2^-9, 2^-8): a row's weights sum to less than 2
// under their joint maximum (304 parts at most), values of any size stay in
// fp32's range times them. l = 0: no visible token with a logit above -Inf.
__device__ __forceinline__ void split_weight(float& m, float& l) {
  if (l > 0.0f && l < INFINITY) {
    const int e = (int)(__float_as_uint(l) >> 23) - (127 - 9);      // l: of the order of 1 and more, never subnormal
    m += (float)e;
    l = __uint_as_float(__float_as_uint(l) - ((uint32_t)e << 23));
  }
}
// In shared memory: G rows of kA8Row, then 8 maxima and 8 sums.
__device__ __forceinline__ void put_partial(const State& s, float* p, int G, int lane) {
  const int g = lane >> 2, t = lane & 3;
  float f[2], m[2] = {s.u[0], s.u[1]}, l[2] = {s.l[0], s.l[1]};
#pragma unroll
  for (int e = 0; e < 2; e++) {
    f[e] = l[e] == 0.0f ? 0.0f : __fdiv_rn(fast_exp2(s.m[e] - s.u[e]), l[e]);
    split_weight(m[e], l[e]);
  }
#pragma unroll
  for (int m8 = 0; m8 < 8; m8++)
#pragma unroll
    for (int e = 0; e < 4; e++)
      if (2 * t + (e & 1) < G) p[(2 * t + (e & 1)) * kA8Row + 16 * m8 + g + 8 * (e >> 1)] = s.o[m8][e] * f[e & 1];
  if (g == 0) {
    float* ml = p + G * kA8Row;
    ml[2 * t] = m[0];
    ml[2 * t + 1] = m[1];
    ml[8 + 2 * t] = l[0];
    ml[8 + 2 * t + 1] = l[1];
  }
}
// weight of a partial with maximum m under the joint maximum M: 1 where they
// are equal, infinite ones too
__device__ __forceinline__ float join(float m, float M) { return m == M ? 1.0f : fast_exp2(m - M); }

// largest of the lanes' values, in one instruction (NaN is passed over)
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(y) : "f"(x));
  return y;
}
// Row q of several parts: lane x holds the address of part x where bit x of set
// is on; rows of `row` floats, then G maxima from G * row and G sums from
// G * row + 8. o is the sum of the parts' results by weight, l of the weights.
struct Row {
  float4 o;
  float m, l;
};
__device__ __noinline__ Row join_row(unsigned set, const float* p, int row, int G, int q, int lane) {
  const bool has = set >> lane & 1u;
  const float m = has ? p[G * row + q] : -INFINITY, pl = has ? p[G * row + 8 + q] : 0.0f;
  Row r{make_float4(0.0f, 0.0f, 0.0f, 0.0f), warp_max(m), 0.0f};
  const float f = has ? pl * join(m, r.m) : 0.0f;
  const unsigned long long mine = reinterpret_cast<unsigned long long>(p + q * row);
  // two parts at a time
#pragma unroll 1
  while (set) {
    const int x0 = __ffs(set) - 1;
    set &= set - 1;
    const int x1 = set ? __ffs(set) - 1 : x0;
    const bool two = set != 0;
    set &= set - 1;
    const float4 v0 = reinterpret_cast<const float4*>(__shfl_sync(0xffffffffu, mine, x0))[lane];
    const float4 v1 = reinterpret_cast<const float4*>(__shfl_sync(0xffffffffu, mine, x1))[lane];
    const float f0 = __shfl_sync(0xffffffffu, f, x0), f1 = __shfl_sync(0xffffffffu, f, x1);
    r.l += f0;
    r.o.x = fmaf(v0.x, f0, r.o.x);
    r.o.y = fmaf(v0.y, f0, r.o.y);
    r.o.z = fmaf(v0.z, f0, r.o.z);
    r.o.w = fmaf(v0.w, f0, r.o.w);
    if (two) {
      r.l += f1;
      r.o.x = fmaf(v1.x, f1, r.o.x);
      r.o.y = fmaf(v1.y, f1, r.o.y);
      r.o.z = fmaf(v1.z, f1, r.o.z);
      r.o.w = fmaf(v1.w, f1, r.o.w);
    }
  }
  return r;
}

// Row q of the parts that CTAs c0 .. c1 left in the workspace (the first one's
// second place, the others' first), kFar at a time in flight: one request of
// 131072 tokens with one KV head (152 parts) takes 21 us, 26 with four at a time,
// 38 with two; sixteen (20 us) cost every other call half a percent.
constexpr int kFar = 8;
__device__ __noinline__ Row join_far(const float* part, int stride, int c0, int c1, int G, int q, int lane) {
  Row r{make_float4(0.0f, 0.0f, 0.0f, 0.0f), -INFINITY, 0.0f};
#pragma unroll 1
  for (int x = c0; x <= c1; x += 32) {
    const int n = min(c1 - x + 1, 32), cta = min(x + lane, c1);
    const float* p = part + (size_t)(2 * cta + (cta == c0 ? 1 : 0)) * stride;
    const float m = lane < n ? __ldcg(p + G * kD + q) : -INFINITY, pl = lane < n ? __ldcg(p + G * kD + 8 + q) : 0.0f;
    const unsigned long long mine = reinterpret_cast<unsigned long long>(p + q * kD);
    float4 v[kFar];
    auto load = [&](int b) {
#pragma unroll
      for (int i = 0; i < kFar; i++)
        v[i] = __ldcg(reinterpret_cast<const float4*>(__shfl_sync(0xffffffffu, mine, min(b + i, 31))) + lane);
    };
    load(0);
    const float now = fmaxf(r.m, warp_max(m));
    const float f = lane < n ? pl * join(m, now) : 0.0f, g = join(r.m, now);
    r.m = now;
    r.l *= g;
    r.o.x *= g;
    r.o.y *= g;
    r.o.z *= g;
    r.o.w *= g;
#pragma unroll 1
    for (int b = 0;;) {
#pragma unroll
      for (int i = 0; i < kFar; i++) {
        const float fi = __shfl_sync(0xffffffffu, f, min(b + i, 31));
        if (b + i < n) {
          r.l += fi;
          r.o.x = fmaf(v[i].x, fi, r.o.x);
          r.o.y = fmaf(v[i].y, fi, r.o.y);
          r.o.z = fmaf(v[i].z, fi, r.o.z);
          r.o.w = fmaf(v[i].w, fi, r.o.w);
        }
      }
      b += kFar;
      if (b >= n) break;
      load(b);
    }
  }
  return r;
}

template <int ELEM>
__device__ __forceinline__ void write_row(uint8_t* out, int lane, float4 o, float l) {
  const float inv = __fdiv_rn(1.0f, l);
  uint2 w = make_uint2(pack_elems<ELEM>(o.x * inv, o.y * inv), pack_elems<ELEM>(o.z * inv, o.w * inv));
  uint32_t bad = 0;
  find_not_finite<ELEM>(bad, w.x);
  find_not_finite<ELEM>(bad, w.y);
  if (__builtin_expect(found_not_finite(bad), 0))
    w = make_uint2(pack_elems<ELEM>(in_range<ELEM>(o.x * inv), in_range<ELEM>(o.y * inv)),
                   pack_elems<ELEM>(in_range<ELEM>(o.z * inv), in_range<ELEM>(o.w * inv)));
  *reinterpret_cast<uint2*>(out + 8 * lane) = w;
}

// What a lane finds out about one tile of the sequence.
struct Desc {
  const uint8_t* src;    // its 4 KB of codes, or its 8 KB of the tail
  float2 sc;             // s_k, s_v
  int tile;
  int head;              // request << 12 | KV head (4096 at most)
  int start;             // first position of its unit
  bool tail, edge;
};

// Copies of codes that no later work of this layer's step reads again: first
// to leave L2, which keeps the tables, the scales and the kernel's own code.
__device__ __forceinline__ uint64_t stream_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;\n" : "=l"(p));
  return p;
}
__device__ __forceinline__ void bulk_g2s_hint(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;\n" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar), "l"(pol)
      : "memory");
}
__device__ __noinline__ bool slow_wait(uint32_t bar, uint32_t parity) { return mbar_wait_bounded(bar, parity); }

// One kernel, and each of its phases once in the code: what runs once a call
// (plan, descriptors, joins) is bound by instruction fetches that miss the
// caches behind a cold L2.
template <int ELEM, int CODE>
__global__ void __launch_bounds__(kA8Warps * 32)
    k_attention8(Cache8View c, Attn8Args a) {
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ int s_pre[kMaxCallReq + 1], s_len[kMaxCallReq], s_slot[kMaxCallReq], s_scan[32];
  __shared__ int s_unit[2 * kA8Warps];
  __shared__ int2 s_span[2 * kA8Warps];     // its positions
  __shared__ __align__(8) uint64_t s_bar[kA8Warps * kA8Stages];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = c.G, hkv = c.hkv;
  const int first_off = kA8Warps * kA8Stages * kA8Entry, part_bytes = (G * kA8Row + 16) * 4;
  uint8_t* ring = sm + warp * (kA8Stages * kA8Entry);
  const uint32_t bar0 = smem_u32(s_bar + warp * kA8Stages);
  if (lane == 0) {
    for (int s = 0; s < kA8Stages; s++) mbar_init(bar0 + 8 * s, 1);
    fence_mbar_init();
  }
  if (threadIdx.x < 2 * kA8Warps) s_unit[threadIdx.x] = -1;
  const uint64_t policy = stream_policy();
  pdl_launch_dependents();
  pdl_wait();

  // ---- lengths, and the prefix sums of the requests' tiles over all heads ----
  int carry = 0;
  bool stopped = false;
  for (int base = 0; base < a.n_req; base += blockDim.x) {
    const int i = base + threadIdx.x;
    int n = 0, cost = 0, slot = i;
    if (i < a.n_req) {
      n = a.seq_lens[i];
      if (a.slots) slot = a.slots[i];
    }
    if (base == 0) stopped = c.stopped();       // its load is in flight with theirs
    if (i < a.n_req) {
      n = max(n, 0);
      int err = 0;
      if (n > 0 && (unsigned)slot >= (unsigned)c.n_slots) err = DKV_ERR_ARG;
      else if ((long long)n > (long long)c.width * c.T) err = DKV_ERR_TABLE_FULL;
      if (err) {
        c.latch(err, i);
        n = 0;
      }
      s_len[i] = n;
      s_slot[i] = slot;
      cost = tiles_of(n, c.T, a.window, a.sinks).count * hkv;
    }
    int x = cost;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) s_scan[warp] = x;
    __syncthreads();
    int sum = lane < kA8Warps ? s_scan[lane] : 0;
    const int before = carry + __reduce_add_sync(0xffffffffu, lane < warp ? sum : 0);
    carry += __reduce_add_sync(0xffffffffu, sum);
    if (i < a.n_req) s_pre[i] = before + x - cost;
    if (threadIdx.x == 0) s_pre[min(base + (int)blockDim.x, a.n_req)] = carry;
    __syncthreads();
  }
  const int total = carry, units = a.n_req * hkv;
  // CTAs that take part: not so many that warps have no tile, but one a unit
  // (and no CTA without a tile: the join counts on that)
  const int ctas = max(1, min(min((int)gridDim.x, total), max(units, (total + kA8Cta - 1) / kA8Cta)));
  if ((int)blockIdx.x >= ctas && total > 0) return;

  auto start_of = [&](int cta) { return (int)((long long)total * cta / ctas); };
  const int lo = start_of(blockIdx.x), hi = start_of(blockIdx.x + 1);
  const int w0 = lo + (int)((unsigned)(hi - lo) * warp / kA8Warps);
  const int w1 = lo + (int)((unsigned)(hi - lo) * (warp + 1) / kA8Warps);
  auto cta_of = [&](int x) { return (int)((((long long)x + 1) * ctas - 1) / total); };
  if (stopped) {
    // The error may be one of this call, and CTAs that began before it count on
    // this one's arrival for the units that cross its ends: that is all it does.
    if (warp < 2 && total > 0 && lane < G) {
      const int pos = warp ? hi - 1 : lo;
      int r = 0, end = a.n_req;
      while (end - r > 1) {
        const int mid = (r + end) >> 1;
        if (s_pre[mid] <= pos) r = mid; else end = mid;
      }
      const int n = tiles_of(s_len[r], c.T, a.window, a.sinks).count, h = (pos - s_pre[r]) / n;
      const int us = s_pre[r] + h * n, ue = us + n;
      if (warp ? us >= lo && ue > hi : us < lo)
        atomicInc(a.count + ((size_t)r * hkv + h) * G + lane, (unsigned)(cta_of(ue - 1) - cta_of(us)));
    }
    return;
  }
  const int per = __ffs(c.T / kSub) - 1;     // log2 of the tiles of a block

  // ---- the warp's tiles, 32 descriptors at a time, a lane each ----
  Desc cur, nxt;
  nxt.src = nullptr;
  nxt.head = nxt.tile = nxt.start = 0;
  nxt.tail = nxt.edge = false;
  nxt.sc = make_float2(1.0f, 1.0f);
  unsigned cur_tail = 0, nxt_tail = 0;
  bool ok = true;
  int ahead = 0;                       // ring entry to fill next
  int at = w0, half = 0;               // tile to issue next, and which half of a tail tile
  int base = w0;                       // first tile of `cur`
  int stage = 0, parity = 0;           // ring entry to read next
  // The next `n` entries; the lane that holds a tile's descriptor issues its copy.
  auto issue = [&](int n) {
#pragma unroll 1
    for (; n > 0 && at < w1; n--) {
      const bool in = at - base < 32;
      const int from = (at - w0) & 31;
      const bool tail = (in ? cur_tail : nxt_tail) >> from & 1u;
      if (lane == from && ok) {
        mbar_expect_tx(bar0 + 8 * ahead, kA8Entry);
        bulk_g2s_hint(smem_u32(ring + ahead * kA8Entry), (in ? cur.src : nxt.src) + half * kA8Entry, kA8Entry,
                      bar0 + 8 * ahead, policy);
      }
      ahead = ahead == kA8Stages - 1 ? 0 : ahead + 1;
      half = tail ? half ^ 1 : 0;
      at += half ^ 1;
    }
  };
  auto wait = [&]() {                  // the next entry, in shared memory
    if (!mbar_try_wait(bar0 + 8 * stage, parity) && ok && !slow_wait(bar0 + 8 * stage, parity)) {
      ok = false;
      c.latch(DKV_ERR_TIMEOUT, -1);
    }
    const uint8_t* p = ring + stage * kA8Entry + 16 * lane;
    if (++stage == kA8Stages) {
      stage = 0;
      parity ^= 1;
    }
    return p;
  };

  State s;
  s.clear();
  uint32_t qf[16];
  const uint8_t* q_at = nullptr;
  float qs[2] = {1.0f, 1.0f};
  bool mixed = false;                  // the unit may have tiles of codes
  int unit = -1, N = 0, ustart = 0, uend = 0, last_start = -1;
#pragma unroll 1
  for (int k = 0; w0 < w1; k++) {
    // descriptors of batch k; the tiles of batch k - 1 follow
    cur = nxt;
    cur_tail = nxt_tail;
    const int pos = w0 + 32 * k + lane;
    nxt.tail = false;
    if (pos < w1) {
      int r = 0, end = a.n_req;        // the request: the last that starts at or before pos
      while (end - r > 1) {
        const int mid = (r + end) >> 1;
        if (s_pre[mid] <= pos) r = mid; else end = mid;
      }
      const int n = s_len[r], slot = s_slot[r];
      const Tiles t = tiles_of(n, c.T, a.window, a.sinks);
      const int rem = pos - s_pre[r], h = (unsigned)rem / (unsigned)t.count, x = rem - h * t.count;
      nxt.head = r << 12 | h;
      nxt.start = pos - x;
      nxt.tile = x < t.head ? x : x - t.head + t.win;
      nxt.edge = !sees_all(nxt.tile * kSub, n, a.window);
      if (nxt.tile < t.full) {
        int page = c.table[(size_t)slot * c.width + (nxt.tile >> per)];
        if ((unsigned)page >= (unsigned)c.n_pages) {
          c.latch(DKV_ERR_CHECK, r);
          page = 0;
        }
        nxt.sc = *reinterpret_cast<const float2*>(c.scales + 2 * ((size_t)page * hkv + h));
        nxt.src = c.pages + c.page_head(page, h) + (size_t)(nxt.tile & ((1 << per) - 1)) * (2 * kTile);
      } else {
        nxt.src = c.tail + c.tail_head(slot, h) + (size_t)(nxt.tile - t.full) * (4 * kTile);
        nxt.tail = true;
      }
    }
    nxt_tail = __ballot_sync(0xffffffffu, nxt.tail);
    if (k == 0) {
      base = w0 - 32;                  // nothing in `cur` yet
      issue(kA8Stages);
      base = w0;
      if (w1 - w0 > 32) continue;
      cur = nxt;
      cur_tail = nxt_tail;
    } else if (k == 1) {
      base = w0;
    } else {
      base += 32;
    }
    const float my_ks = cur.sc.x * kLogitScale, my_lv = log2f(cur.sc.y);
    const int before = __shfl_up_sync(0xffffffffu, cur.start, 1);
    const unsigned edges = __ballot_sync(0xffffffffu, cur.edge);
    const unsigned begins = __ballot_sync(0xffffffffu, cur.start != (lane == 0 ? last_start : before));
    const int n = min(32, w1 - base);
    const bool last = base + 32 >= w1;
#pragma unroll 1
    for (int from = 0; from < n + (last ? 1 : 0); from++) {
      if (from == n || (begins >> from & 1u)) {
        if (unit >= 0) {
          // the end of the warp's part of a unit
#pragma unroll
          for (int d = 4; d <= 16; d <<= 1) {
            s.l[0] += __shfl_xor_sync(0xffffffffu, s.l[0], d);
            s.l[1] += __shfl_xor_sync(0xffffffffu, s.l[1], d);
          }
          if (ustart >= w0 && base + from == uend) {
            write_unit<ELEM>(s, a.out + (size_t)unit * G * (2 * kD), G, lane);
          } else {
            // begun before the range: a place of its own; else it goes on
            // behind the range, and the ring is drained
            const int slot = ustart < w0 ? 0 : 1;
            put_partial(s, reinterpret_cast<float*>(slot ? ring : sm + first_off + warp * part_bytes), G, lane);
            if (lane == 0) {
              s_unit[2 * warp + slot] = unit;
              s_span[2 * warp + slot] = make_int2(ustart, uend);
            }
          }
        }
        if (from == n) break;
        const int rh = __shfl_sync(0xffffffffu, cur.head, from), r = rh >> 12, h = rh & 4095;
        ustart = last_start = __shfl_sync(0xffffffffu, cur.start, from);
        unit = r * hkv + h;
        N = s_len[r];
        mixed = N >= c.T;
        uend = ustart + tiles_of(N, c.T, a.window, a.sinks).count;
        s.clear();
        q_at = a.q + r * a.qs + (size_t)h * G * (2 * kD);
        load_q<ELEM>(q_at, G, lane, qf);
        if (ELEM == DKV_BF16) half_q(qf, lane, qs);
      }
      const float ks = __shfl_sync(0xffffffffu, my_ks, from), lv = __shfl_sync(0xffffffffu, my_lv, from);
      const bool edge = edges >> from & 1u, tail = cur_tail >> from & 1u;
      See see{true, true, 0xffffffffu};
      if (edge) see = see_of(__shfl_sync(0xffffffffu, cur.tile, from) * kSub, N, a.window, a.sinks, lane);
      const uint8_t* p = wait();
      if (!tail) {
        const float k2[2] = {ks * qs[0], ks * qs[1]};
        code_tile<CODE>(s, qf, p, edge, see, k2, lv);
      } else {
        auto after_k = [&]() {      // the next tile's K follows while V is awaited
          __syncwarp();
          issue(1);
          return wait();
        };
        if (ELEM == DKV_F16) {
          tail_tile<ELEM>(s, qf, p, after_k, edge, see, mixed, kLogitScale);
        } else {
          uint32_t raw[16];    // the other tiles' fragments are scaled
          load_q<ELEM>(q_at, G, lane, raw);
          tail_tile<ELEM>(s, raw, p, after_k, edge, see, mixed, kLogitScale);
        }
      }
      __syncwarp();
      issue(1);
    }
    if (last) break;
  }
  // a wait that gave up: no copy may still be in flight at the exit
  if (!ok)
    for (int e = 0; e < kA8Stages; e++) {
      slow_wait(bar0 + 8 * stage, parity);
      if (++stage == kA8Stages) {
        stage = 0;
        parity ^= 1;
      }
    }
  __syncthreads();

  // ---- joins: the rows of the units that several warps hold parts of, a warp a
  // row in turn; where the unit crosses CTAs, each leaves its part, and the CTA
  // that arrives last joins those. The rows of such units, which are the CTA's
  // first or last, come first: each waits through a fence, an atomic and loads, a
  // few us in which the other warps do the rest (200 requests of 2 tiles with 8 KV
  // heads and G = 5 take 13 us, with a warp a unit 16; 200 of 1 .. 160 tokens 20
  // and 23; but 8 x 32768 tokens, with few units of many parts, 89.2 and 87.8) ----
  const int mine = lane < 2 * kA8Warps ? s_unit[lane] : -1;
  // slots lie in the order of positions: those of a unit are neighbours
  const unsigned used = __ballot_sync(0xffffffffu, mine >= 0), below = used & ((1u << lane) - 1u);
  const int before = __shfl_sync(0xffffffffu, mine, below ? 31 - __clz(below) : lane);
  const unsigned leaders = __ballot_sync(0xffffffffu, mine >= 0 && (below == 0 || before != mine));
  const int rank = __popc(leaders & ((1u << lane) - 1u));       // of a leader
  const float* my_part = reinterpret_cast<const float*>(
      sm + ((lane & 1) ? (lane >> 1) * (kA8Stages * kA8Entry) : first_off + (lane >> 1) * part_bytes));
  const int stride = G * kD + 16;      // floats of a part in the workspace
  const int n_units = __popc(leaders);
#pragma unroll 1
  for (int job = warp; job < n_units * G; job += kA8Warps) {
    // the first unit, the last, then those between
    const int t = job / G, q = job - t * G, nth = t == 0 ? 0 : t == 1 ? n_units - 1 : t - 1;
    const int lead = __ffs(__ballot_sync(0xffffffffu, (leaders >> lane & 1u) && rank == nth)) - 1;
    const unsigned next = lead < 31 ? leaders >> (lead + 1) << (lead + 1) : 0u;
    const unsigned set = used & ~((1u << lead) - 1u) & (next ? (next & -next) - 1u : 0xffffffffu);
    const int u = __shfl_sync(0xffffffffu, mine, lead);
    const int us = s_span[lead].x, ue = s_span[lead].y;
    uint8_t* out = a.out + ((size_t)u * G + q) * (2 * kD);
    Row r = join_row(set, my_part, kA8Row, G, q, lane);
    if (us < lo || ue > hi) {
      float* dst = a.part + (size_t)(2 * blockIdx.x + (us < lo ? 0 : 1)) * stride;
      const float inv = r.l == 0.0f ? 0.0f : __fdiv_rn(1.0f, r.l);
      r.o = make_float4(r.o.x * inv, r.o.y * inv, r.o.z * inv, r.o.w * inv);
      split_weight(r.m, r.l);
      *reinterpret_cast<float4*>(dst + q * kD + 4 * lane) = r.o;
      if (lane == 0) {
        dst[G * kD + q] = r.m;
        dst[G * kD + 8 + q] = r.l;
      }
      const int c0 = cta_of(us), c1 = cta_of(ue - 1);
      __threadfence();
      __syncwarp();
      // a counter per row, back to zero by itself
      const unsigned old = lane == 0 ? atomicInc(a.count + (size_t)u * G + q, (unsigned)(c1 - c0)) : 0u;
      if (__shfl_sync(0xffffffffu, old, 0) != (unsigned)(c1 - c0)) continue;
      __threadfence();
      r = join_far(a.part, stride, c0, c1, G, q, lane);
    }
    write_row<ELEM>(out, lane, r.o, r.l);
  }

  // requests without tokens: zeros
  for (int i = blockIdx.x; i < a.n_req; i += ctas)
    if (s_pre[i + 1] == s_pre[i])
      for (int x = threadIdx.x; x < hkv * G * (kD / 8); x += blockDim.x)
        reinterpret_cast<uint4*>(a.out + (size_t)i * hkv * G * (2 * kD))[x] = make_uint4(0, 0, 0, 0);
}

// a counter per query row: rows of one unit are joined apart
size_t count_bytes(int hq, int n_req) { return ((size_t)hq * n_req * 4 + 255) / 256 * 256; }
size_t attention8_smem(int G) {
  return (size_t)kA8Warps * kA8Stages * kA8Entry + (size_t)kA8Warps * (G * kA8Row + 16) * 4;
}

}  // namespace

// The partials first: their place does not depend on the call's requests.
size_t attention8_workspace(int hkv, int G, int max_req, int sm_count) {
  return (size_t)sm_count * 2 * ((size_t)G * kD + 16) * 4 + count_bytes(hkv * G, max_req);
}

cudaError_t launch_attention8(const Cache8View& c, int elem, int code, int sm_count, const int* slots,
                              const int* seq_lens, int n_req, const void* q, long long q_stride, void* out,
                              int window, int sinks, void* workspace, cudaStream_t st) {
  float* part = static_cast<float*>(workspace);
  const Attn8Args a{slots, seq_lens, static_cast<const uint8_t*>(q), 2 * q_stride, static_cast<uint8_t*>(out),
                    n_req, window, sinks, reinterpret_cast<unsigned*>(part + (size_t)sm_count * 2 * (c.G * kD + 16)), part};
  auto kernel = elem == DKV_F16 ? (code == DKV_E4M3 ? k_attention8<DKV_F16, DKV_E4M3> : k_attention8<DKV_F16, DKV_INT8>)
                                : (code == DKV_E4M3 ? k_attention8<DKV_BF16, DKV_E4M3> : k_attention8<DKV_BF16, DKV_INT8>);
  // the limit belongs to the kernel, which calls of other group sizes on other
  // host threads launch too: always the largest
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)attention8_smem(kMaxG));
  if (e != cudaSuccess) return e;
  // no more CTAs than the longest lengths that the table holds could use
  const long long units = (long long)n_req * c.hkv, tiles = units * ((long long)c.width * c.T / kSub);
  const int grid = (int)std::min<long long>(sm_count, std::max(units, (tiles + kA8Cta - 1) / kA8Cta));
  return launch_dependent(kernel, dim3(grid), dim3(kA8Warps * 32), attention8_smem(c.G), st, c, a);
}

}  // namespace dkv
