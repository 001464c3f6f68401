// cache8_attention.cu — decode attention over the uniform 8-bit cache, in full
// or through a sliding window with first tokens that stay visible
// (include/dkv.h: dkv_cache8_attention).
//
// One CTA per (request, KV head); its warps take 16-token tiles in turn and
// join their partial results in shared memory.
//
// A warp's step on a tile of codes, S^T = K Q^T and O^T += V^T P^T with
// mma.sync m16n8k16 (tokens / features on M, the G <= 8 queries on N; at most
// 8 rows of queries cannot fill a tcgen05 tile, and the kernel is bound by
// memory, not by matrix rate):
//   x_j  = s_k (q . code_j) log2(e) / sqrt(128) + log2(s_v)
//   w_j  = 2^(x_j - m)        the probability times V's scale, up to 2^-m
//   O   += w_j code_j,   l += w_j / s_v,   out = O / l
// so that one running maximum m serves both and blocks with different V
// scales need no rescaling of O. m is raised (O, l rescaled) only when some
// x_j exceeds it by more than 8: w stays below 2^8, in fp16's range. w enters
// the second product rounded to fp16 (relative 2^-11, the size of the
// output's own rounding); l sums the unrounded fp32 values.
// Tiles of the 16-bit tail take s_k = 1 and, for s_v, the power of two below
// their largest |v|, by which their values are divided (exact but for values
// 2^-14 and less of the largest).
#include "cache8.cuh"
#include "dkv_kernels.cuh"

namespace dkv {
namespace {

constexpr int kA8Warps = 8;
constexpr float kA8Lazy = 8.0f;

struct Attn8Args {
  const int *slots, *seq_lens;
  const uint8_t* q;
  long long qs;      // bytes
  uint8_t* out;
  int n_req, window, sinks;
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

template <int ELEM>
__device__ __forceinline__ void mma_elem(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if (ELEM == DKV_F16) {
    mma16816(c, a, b0, b1);
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

// Running state of a warp for one (request, KV head): lane 4g + t holds
// queries 2t, 2t + 1; O rows are features 16 m + g and 16 m + g + 8.
struct State {
  float o[8][4];
  float m[2], l[2];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; i++)
#pragma unroll
      for (int e = 0; e < 4; e++) o[i][e] = 0.0f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.0f;
  }
};

// Raise the running maxima where some x exceeds them by more than the slack.
// x: tokens g (x[0], x[1]) and g + 8 (x[2], x[3]) for the lane's two queries.
__device__ __forceinline__ void raise(State& s, const float* x) {
  float a = fmaxf(x[0], x[2]), b = fmaxf(x[1], x[3]);
  if (!__any_sync(0xffffffffu, a > s.m[0] + kA8Lazy || b > s.m[1] + kA8Lazy)) return;
#pragma unroll
  for (int d = 4; d <= 16; d <<= 1) {
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
    b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, d));
  }
  const float na = fmaxf(s.m[0], a), nb = fmaxf(s.m[1], b);
  const float fa = na == -INFINITY ? 1.0f : fast_exp2(s.m[0] - na), fb = nb == -INFINITY ? 1.0f : fast_exp2(s.m[1] - nb);
  s.m[0] = na;
  s.m[1] = nb;
  s.l[0] *= fa;
  s.l[1] *= fb;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    s.o[i][0] *= fa;
    s.o[i][1] *= fb;
    s.o[i][2] *= fa;
    s.o[i][3] *= fb;
  }
}

// w = 2^(x - m) in place of x, summed into l.
__device__ __forceinline__ void weights(State& s, float* x, float inv) {
  const float ma = s.m[0] == -INFINITY ? 0.0f : s.m[0], mb = s.m[1] == -INFINITY ? 0.0f : s.m[1];
  x[0] = fast_exp2(x[0] - ma);
  x[1] = fast_exp2(x[1] - mb);
  x[2] = fast_exp2(x[2] - ma);
  x[3] = fast_exp2(x[3] - mb);
  s.l[0] = fmaf(x[0] + x[2], inv, s.l[0]);
  s.l[1] = fmaf(x[1] + x[3], inv, s.l[1]);
}

// Which tokens of a tile the query sees, for this lane: logits of tokens g and
// g + 8, and the V entries of tokens 2t, 2t+1, 2t+8, 2t+9 (one byte each).
struct See {
  bool all, lo, hi;
  uint32_t v;
};
__device__ __forceinline__ See see_of(int pos0, int N, int window, int sinks, int lane) {
  See s;
  const int from = window > 0 ? N - window : 0;
  s.all = pos0 + kSub <= N && pos0 >= from;
  if (s.all) {
    s.lo = s.hi = true;
    s.v = 0xffffffffu;
    return s;
  }
  auto sees = [&](int i) { return pos0 + i < N && (pos0 + i >= from || pos0 + i < sinks); };
  const int g = lane >> 2, t = lane & 3;
  s.lo = sees(g);
  s.hi = sees(g + 8);
  s.v = (sees(2 * t) ? 0xffu : 0u) | (sees(2 * t + 1) ? 0xff00u : 0u) | (sees(2 * t + 8) ? 0xff0000u : 0u) |
        (sees(2 * t + 9) ? 0xff000000u : 0u);
  return s;
}

// A tile of codes: kw, vw are the lane's 64 bytes of K and of V.
template <int CODE>
__device__ __forceinline__ void code_tile(State& s, const uint32_t (&qf)[16], const uint4 (&kw)[4], const uint4 (&vw)[4],
                                          const See& see, const float (&ks)[2], float lv, float inv) {
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
  for (int e = 0; e < 4; e++) x[e] = (e < 2 ? see.lo : see.hi) ? fmaf(x[e] + y[e], ks[e & 1], lv) : -INFINITY;
  raise(s, x);
  weights(s, x, inv);
  const uint32_t b0 = movmatrix_trans(pack_half2(x[0], x[1])), b1 = movmatrix_trans(pack_half2(x[2], x[3]));
#pragma unroll
  for (int j = 0; j < 4; j++) {
    uint32_t a[4];
    code_halves<CODE>(see.all ? vw[j].x : vw[j].x & see.v, a[0], a[2]);
    code_halves<CODE>(see.all ? vw[j].y : vw[j].y & see.v, a[1], a[3]);
    mma16816(s.o[2 * j], a, b0, b1);
    code_halves<CODE>(see.all ? vw[j].z : vw[j].z & see.v, a[0], a[2]);
    code_halves<CODE>(see.all ? vw[j].w : vw[j].w & see.v, a[1], a[3]);
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

// A tile of the 16-bit tail: kp, vp point to the lane's first 16 bytes of K
// and V, the next steps 512 bytes on.
template <int ELEM>
__device__ __forceinline__ void tail_tile(State& s, const uint32_t (&qf)[16], const uint8_t* kp, const uint8_t* vp,
                                          const See& see, float ks) {
  float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int m = 0; m < 8; m++) {
    const uint4 w = *reinterpret_cast<const uint4*>(kp + 512 * m);
    const uint32_t a[4] = {w.x, w.z, w.y, w.w};
    mma_elem<ELEM>(x, a, qf[2 * m], qf[2 * m + 1]);
  }
  // entries of tokens that are not visible (unwritten ones too) become 0
  const uint32_t lo = prmt(see.v, 0, 0x1100u), hi = prmt(see.v, 0, 0x3322u);
  uint4 v[8];
  float am = 0.0f;
#pragma unroll
  for (int m = 0; m < 8; m++) {
    v[m] = *reinterpret_cast<const uint4*>(vp + 512 * m);
    v[m].x &= lo;
    v[m].y &= hi;
    v[m].z &= lo;
    v[m].w &= hi;
    const uint32_t w[4] = {v[m].x, v[m].y, v[m].z, v[m].w};
#pragma unroll
    for (int e = 0; e < 4; e++) am = amax_finite(amax_finite(am, lo_elem<ELEM>(w[e])), hi_elem<ELEM>(w[e]));
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, d));
  // power of two below am, its exponent within what fp16 factors (or the
  // scale floor) allow
  const int low = ELEM == DKV_F16 ? -14 : -100, high = ELEM == DKV_F16 ? 14 : 100;
  const int ex = max(low, min(high, (int)(__float_as_uint(am) >> 23) - 127));
  const float inv = __uint_as_float((uint32_t)(127 - ex) << 23);
#pragma unroll
  for (int e = 0; e < 4; e++) x[e] = (e < 2 ? see.lo : see.hi) ? fmaf(x[e], ks, (float)ex) : -INFINITY;
  raise(s, x);
  weights(s, x, inv);
  uint32_t p0 = pack_elems<ELEM>(x[0], x[1]), p1 = pack_elems<ELEM>(x[2], x[3]);
  const uint32_t b0 = movmatrix_trans(p0), b1 = movmatrix_trans(p1);
  uint32_t r0 = 0, r1 = 0;
  if (ELEM == DKV_BF16) {   // what bf16 rounds away (8 bits are fewer than the fp16 of the other tiles keep)
    r0 = movmatrix_trans(pack_elems<ELEM>(x[0] - lo_elem<ELEM>(p0), x[1] - hi_elem<ELEM>(p0)));
    r1 = movmatrix_trans(pack_elems<ELEM>(x[2] - lo_elem<ELEM>(p1), x[3] - hi_elem<ELEM>(p1)));
  }
#pragma unroll
  for (int m = 0; m < 8; m++) {
    const uint32_t a[4] = {scale_pair<ELEM>(v[m].x, inv), scale_pair<ELEM>(v[m].z, inv), scale_pair<ELEM>(v[m].y, inv),
                           scale_pair<ELEM>(v[m].w, inv)};
    mma_elem<ELEM>(s.o[m], a, b0, b1);
    if (ELEM == DKV_BF16) mma_elem<ELEM>(s.o[m], a, r0, r1);
  }
}

// Query fragments of a (request, KV head): raw, and for bf16 also as fp16
// after division by the power of two below the row's largest |q| (8 bits fit;
// what falls below fp16's range is under 2^-24 of that largest). scale: the
// power of two of the lane's queries 2t, 2t + 1.
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
__device__ __forceinline__ void half_q(const uint32_t (&raw)[16], int lane, uint32_t (&qf)[16], float (&scale)[2]) {
  float am = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; i++)
    am = amax_finite(amax_finite(am, lo_elem<DKV_BF16>(raw[i])), hi_elem<DKV_BF16>(raw[i]));
  am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
  am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
  const int ex = max(-100, min(100, (int)(__float_as_uint(am) >> 23) - 127));
  const float inv = __uint_as_float((uint32_t)(127 - ex) << 23), sc = __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
  for (int i = 0; i < 16; i++) qf[i] = pack_half2(lo_elem<DKV_BF16>(raw[i]) * inv, hi_elem<DKV_BF16>(raw[i]) * inv);
  const int t = lane & 3;      // row of query 2t: lanes 4 (2t) ..
  scale[0] = __shfl_sync(0xffffffffu, sc, 8 * t);
  scale[1] = __shfl_sync(0xffffffffu, sc, 8 * t + 4);
}

template <int ELEM, int CODE>
__global__ void __launch_bounds__(kA8Warps * 32)
    k_attention8(Cache8View c, Attn8Args a) {
  __shared__ float s_o[kA8Warps][kMaxG][kD];
  __shared__ float s_m[kA8Warps][kMaxG], s_l[kA8Warps][kMaxG];
  pdl_launch_dependents();
  pdl_wait();
  if (c.noop()) return;
  const int i = blockIdx.x / c.hkv, h = blockIdx.x % c.hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t4 = lane & 3, g4 = lane >> 2;
  int slot = a.slots ? a.slots[i] : i, N = max(a.seq_lens[i], 0);
  int err = 0;
  if ((unsigned)slot >= (unsigned)c.n_slots) err = DKV_ERR_ARG;
  else if ((long long)N > (long long)c.width * c.T) err = DKV_ERR_TABLE_FULL;
  if (err) {
    if (threadIdx.x == 0) c.latch(err, i);
    return;
  }
  const Tiles tl = tiles_of(N, c.T, a.window, a.sinks);
  uint32_t raw[16], qf[16];
  float qs[2] = {1.0f, 1.0f};
  load_q<ELEM>(a.q + i * a.qs + (size_t)h * c.G * (2 * kD), c.G, lane, raw);
  if (ELEM == DKV_BF16) {
    half_q(raw, lane, qf, qs);
  } else {
#pragma unroll
    for (int e = 0; e < 16; e++) qf[e] = raw[e];
  }
  State s;
  s.clear();
  const int per = c.T / kSub;
  for (int x = warp; x < tl.count; x += kA8Warps) {
    const int tile = x < tl.head ? x : x - tl.head + tl.win;
    const See see = see_of(tile * kSub, N, a.window, a.sinks, lane);
    if (tile < tl.full) {
      int page = c.table[(size_t)slot * c.width + tile / per];
      if ((unsigned)page >= (unsigned)c.n_pages) {
        if (lane == 0) c.latch(DKV_ERR_CHECK, i);
        page = 0;
      }
      const float* sc = c.scales + 2 * ((size_t)page * c.hkv + h);
      const float sk = sc[0], sv = sc[1];
      const uint4* p = reinterpret_cast<const uint4*>(c.pages + c.page_head(page, h) + (size_t)(tile % per) * 2 * kTile) + lane;
      uint4 kw[4], vw[4];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        kw[j] = p[32 * j];
        vw[j] = p[128 + 32 * j];
      }
      const float ks[2] = {sk * kLogitScale * qs[0], sk * kLogitScale * qs[1]};
      code_tile<CODE>(s, qf, kw, vw, see, ks, log2f(sv), __fdiv_rn(1.0f, sv));
    } else {
      const uint8_t* p = c.tail + c.tail_head(slot, h) + (size_t)(tile - tl.full) * 4 * kTile + 16 * lane;
      tail_tile<ELEM>(s, raw, p, p + 2 * kTile, see, kLogitScale);
    }
  }
#pragma unroll
  for (int d = 4; d <= 16; d <<= 1) {
    s.l[0] += __shfl_xor_sync(0xffffffffu, s.l[0], d);
    s.l[1] += __shfl_xor_sync(0xffffffffu, s.l[1], d);
  }
  if (g4 == 0) {
    s_m[warp][2 * t4] = s.m[0];
    s_m[warp][2 * t4 + 1] = s.m[1];
    s_l[warp][2 * t4] = s.l[0];
    s_l[warp][2 * t4 + 1] = s.l[1];
  }
#pragma unroll
  for (int m = 0; m < 8; m++)
#pragma unroll
    for (int e = 0; e < 4; e++) s_o[warp][2 * t4 + (e & 1)][16 * m + g4 + 8 * (e >> 1)] = s.o[m][e];
  __syncthreads();
  for (int x = threadIdx.x; x < c.G * kD / 2; x += blockDim.x) {
    const int g = x / (kD / 2), f = 2 * (x % (kD / 2));
    float M = -INFINITY;
    for (int w = 0; w < kA8Warps; w++) M = fmaxf(M, s_m[w][g]);
    float u = 0.0f, v = 0.0f, l = 0.0f;
    for (int w = 0; w < kA8Warps; w++) {
      const float fw = s_m[w][g] == M ? 1.0f : fast_exp2(s_m[w][g] - M);   // 0 for a warp without tiles
      u = fmaf(s_o[w][g][f], fw, u);
      v = fmaf(s_o[w][g][f + 1], fw, v);
      l = fmaf(s_l[w][g], fw, l);
    }
    const bool none = tl.count == 0;
    reinterpret_cast<uint32_t*>(a.out)[(((size_t)i * c.hkv + h) * c.G + g) * (kD / 2) + f / 2] =
        none ? 0u : pack_elems<ELEM>(__fdiv_rn(u, l), __fdiv_rn(v, l));
  }
}

}  // namespace

size_t attention8_workspace(int, int, int, int) { return 256; }

cudaError_t launch_attention8(const Cache8View& c, int elem, int code, int, const int* slots, const int* seq_lens,
                              int n_req, const void* q, long long q_stride, void* out, int window, int sinks, void*,
                              cudaStream_t st) {
  const Attn8Args a{slots, seq_lens, static_cast<const uint8_t*>(q), 2 * q_stride, static_cast<uint8_t*>(out),
                    n_req, window, sinks};
  auto kernel = elem == DKV_F16 ? (code == DKV_E4M3 ? k_attention8<DKV_F16, DKV_E4M3> : k_attention8<DKV_F16, DKV_INT8>)
                                : (code == DKV_E4M3 ? k_attention8<DKV_BF16, DKV_E4M3> : k_attention8<DKV_BF16, DKV_INT8>);
  return launch_dependent(kernel, dim3((unsigned)(n_req * c.hkv)), dim3(kA8Warps * 32), 0, st, c, a);
}

}  // namespace dkv
