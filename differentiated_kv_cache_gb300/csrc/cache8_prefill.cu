// cache8_prefill.cu — causal attention over whole prompts with an optional
// sliding window and first tokens that stay visible (include/dkv.h:
// dkv_cache8_prefill), fp16 or bf16, on the fifth-generation tensor cores.
//
// A CTA takes 128 query rows of one request and KV head: row r is token
// r / G of the CTA's floor(128 / G), query head r % G of the group, so one
// K / V tile serves the whole group and a tile of rows spans few positions
// (the keys that only part of its rows see stay few). Warp 0 issues the TMA
// copies (the queries once, 128-key K and V tiles through two stages each),
// warp 1 the MMAs, warps 2..5 run the softmax with one thread per row:
//   S = Q K^T        tcgen05, D in tensor memory, three buffers
//   P = 2^(S - m)    lazily raised row maximum, written over S in 16 bits
//   O += P V         tcgen05, A = P from tensor memory, V MN-major
// Only key tiles with a visible key are visited: [0, first) of the first
// tokens, then the window's up to the diagonal. Every wait is bounded; on
// expiry the kernel latches DKV_ERR_TIMEOUT, waits (bounded) for its own
// copies and MMAs, frees its tensor memory and returns.
#include <algorithm>
#include <cudaTypedefs.h>

#include "cache8.cuh"
#include "dkv_kernels.cuh"
#include "dkv_tc.cuh"

namespace dkv {

cudaError_t tma_encoder(PFN_cuTensorMapEncodeTiled_v12000* fn);

namespace {

constexpr int kW8T = 128;                  // query rows per CTA, keys per tile
constexpr int kW8Threads = 192;
constexpr int kW8Half = kW8T * 128;        // 64 features of 128 rows: 16 KB
constexpr int kW8Tile = 2 * kW8Half;
constexpr int kW8Stages = 2;
constexpr int kW8OffK = kW8Tile;
constexpr int kW8OffV = kW8OffK + kW8Stages * kW8Tile;
constexpr int kW8OffBar = kW8OffV + kW8Stages * kW8Tile;
constexpr int kW8Smem = 1024 + kW8OffBar + 256;
constexpr int kW8SBufs = 3;
constexpr uint32_t kW8OCol = kW8SBufs * 128;
constexpr uint32_t kW8Cols = 512;
constexpr float kW8Lazy = 8.0f;

constexpr int kW8Req = 1024;
struct W8Call {
  int n_req;
  int tok0[kW8Req + 1];
  int tile0[kW8Req + 1];     // first query tile of a request
};

struct W8Args {
  uint8_t* out;
  int window, sinks, tq;     // tq: tokens of a query tile
};

template <int ELEM>
__global__ void __launch_bounds__(kW8Threads, 1)
    k_prefill8(Cache8View c, const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
               const __grid_constant__ CUtensorMap tv, W8Args a, const __grid_constant__ W8Call call) {
  pdl_launch_dependents();
  pdl_wait();
  if (c.stopped()) return;
  const int G = c.G, h = blockIdx.x % c.hkv;
  const int qtile = call.tile0[call.n_req] - 1 - (int)(blockIdx.x / c.hkv);   // later rows first: more keys
  int i = 0;
  {
    int hi = call.n_req;
    while (hi - i > 1) {
      const int mid = (i + hi) >> 1;
      if (call.tile0[mid] <= qtile) i = mid; else hi = mid;
    }
  }
  const int t0 = call.tok0[i], n0 = call.tok0[i + 1] - t0;
  const int p0 = (qtile - call.tile0[i]) * a.tq, p1 = min(p0 + a.tq, n0) - 1;   // positions of the CTA
  // key tiles: [0, first), then [from, last]
  const int last = p1 / kW8T;
  int from = 0, first = 0;
  if (a.window > 0) {
    from = max(p0 - a.window + 1, 0) / kW8T;
    first = min((min(a.sinks, n0) + kW8T - 1) / kW8T, from);
  }
  const int nkt = first + last - from + 1;
  auto key_tile = [&](int j) { return j < first ? j : j - first + from; };
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kW8OffBar);
  const uint32_t b0 = smem_u32(bars);
  const uint32_t qfull = b0, ofull = b0 + 8u * 18;
  auto kfull = [&](int s) { return b0 + 8u * (1 + s); };
  auto kempty = [&](int s) { return b0 + 8u * (3 + s); };
  auto vfull = [&](int s) { return b0 + 8u * (5 + s); };
  auto vempty = [&](int s) { return b0 + 8u * (7 + s); };
  auto sfull = [&](int b) { return b0 + 8u * (9 + b); };
  auto pfull = [&](int b) { return b0 + 8u * (12 + b); };
  auto pvdone = [&](int b) { return b0 + 8u * (15 + b); };
  uint32_t* s_taddr = reinterpret_cast<uint32_t*>(bars + 19);
  int* s_fail = reinterpret_cast<int*>(s_taddr + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(qfull, 1);
    mbar_init(ofull, 1);
    for (int s = 0; s < kW8Stages; s++) {
      mbar_init(kfull(s), 1);
      mbar_init(kempty(s), 1);
      mbar_init(vfull(s), 1);
      mbar_init(vempty(s), 1);
    }
    for (int b = 0; b < kW8SBufs; b++) {
      mbar_init(sfull(b), 1);
      mbar_init(pfull(b), 128);
      mbar_init(pvdone(b), 1);
    }
    *s_fail = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(smem_u32(s_taddr), kW8Cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *s_taddr;
  auto fail = [&]() {
    c.latch(DKV_ERR_TIMEOUT, i);
    *(volatile int*)s_fail = 1;
  };
  auto failed = [&]() { return *(volatile int*)s_fail != 0; };

  if (warp == 0) {
    if (lane == 0) {
      mbar_expect_tx(qfull, (uint32_t)(2 * 128 * a.tq * G));
      for (int f = 0; f < 2; f++)
        tma_load_3d(smem_u32(smem + f * kW8Half), &tq, 64 * f, h * G, t0 + p0, qfull);
      int last_k[kW8Stages] = {-1, -1}, last_v[kW8Stages] = {-1, -1};
      auto load = [&](int j, bool is_k) {
        const int s = j & 1;
        const uint32_t full = is_k ? kfull(s) : vfull(s);
        if (j >= 2 && !mbar_wait_bounded(is_k ? kempty(s) : vempty(s), ((j >> 1) - 1) & 1)) return false;
        mbar_expect_tx(full, kW8Tile);
        for (int f = 0; f < 2; f++)
          tma_load_3d(smem_u32(smem + (is_k ? kW8OffK : kW8OffV) + s * kW8Tile + f * kW8Half), is_k ? &tk : &tv,
                      64 * f, h, t0 + key_tile(j) * kW8T, full);
        (is_k ? last_k : last_v)[s] = j;
        return true;
      };
      bool ok = load(0, true);
      for (int j = 0; ok && j < nkt && !failed(); j++) {
        if (j + 1 < nkt) ok = load(j + 1, true);
        if (ok) ok = load(j, false);
      }
      if (!ok) fail();
      // no copy of this CTA may still be in flight when it exits
      mbar_wait_bounded(qfull, 0);
      for (int s = 0; s < kW8Stages; s++) {
        if (last_k[s] >= 0) mbar_wait_bounded(kfull(s), (last_k[s] >> 1) & 1);
        if (last_v[s] >= 0) mbar_wait_bounded(vfull(s), (last_v[s] >> 1) & 1);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t type = ELEM == DKV_BF16 ? (1u << 7) | (1u << 10) : 0u;   // A and B formats
      constexpr uint32_t id_qk = umma_idesc_f16(128, 128) | type;
      constexpr uint32_t id_pv = umma_idesc_f16(128, 128) | type | (1u << 16);   // B (V) MN-major
      const uint32_t qs = smem_u32(smem);
      bool ok = mbar_wait_bounded(qfull, 0);
      auto issue_qk = [&](int t) {
        const int b = t % kW8SBufs, s = t & 1;
        if (t >= kW8SBufs && !mbar_wait_bounded(pvdone(b), ((t / kW8SBufs) - 1) & 1)) return false;
        if (!mbar_wait_bounded(kfull(s), (t >> 1) & 1)) return false;
        tc_fence_after();
        const uint32_t ks = smem_u32(smem + kW8OffK + s * kW8Tile);
#pragma unroll
        for (int k = 0; k < 8; k++) {
          const uint32_t off = (k >> 2) * kW8Half + (k & 3) * 32;
          umma_f16(tbase + b * 128, umma_desc_sw128(qs + off), umma_desc_sw128(ks + off), id_qk, k > 0);
        }
        umma_commit(kempty(s));
        umma_commit(sfull(b));
        return true;
      };
      auto issue_pv = [&](int t) {
        const int b = t % kW8SBufs, s = t & 1;
        if (!mbar_wait_bounded(pfull(b), (t / kW8SBufs) & 1)) return false;
        if (!mbar_wait_bounded(vfull(s), (t >> 1) & 1)) return false;
        tc_fence_after();
        const uint32_t vs = smem_u32(smem + kW8OffV + s * kW8Tile);
#pragma unroll
        for (int kk = 0; kk < 8; kk++)
          umma_f16_tmem_a(tbase + kW8OCol, tbase + b * 128 + 8 * kk, umma_desc_sw128_mn(vs + kk * 2048, kW8Half), id_pv,
                          t > 0 || kk > 0);
        umma_commit(vempty(s));
        umma_commit(pvdone(b));
        return true;
      };
      if (ok && !issue_qk(0)) ok = false;
      for (int j = 0; ok && j < nkt && !failed(); j++) {
        if (j + 1 < nkt && !issue_qk(j + 1)) { ok = false; break; }
        if (!issue_pv(j)) { ok = false; break; }
      }
      if (!ok) fail();
      umma_commit(ofull);
      mbar_wait_bounded(ofull, 0);
    }
  } else {
    const int lg = warp & 3, row = 32 * lg + lane, pos = p0 + row / G;
    const bool real = row < a.tq * G && pos < n0;
    const uint32_t tl = tbase + ((uint32_t)(32 * lg) << 16);
    float m = -INFINITY, l = 0.0f;
    bool ok = true;
    for (int j = 0; j < nkt; j++) {
      const int b = j % kW8SBufs, kt = key_tile(j) * kW8T;
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(sfull(b), (j / kW8SBufs) & 1) && !failed());
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(vfull(j & 1), (j >> 1) & 1));
      if (!ok) break;
      tc_fence_after();
      if (kt + kW8T > n0) {
        // V rows behind the request belong to others: zero them, whatever they
        // hold (their weight is 0, but 0 * Inf is not)
        uint8_t* vs = smem + kW8OffV + (j & 1) * kW8Tile;
        for (int x = threadIdx.x - 64; x < 2 * (kt + kW8T - n0) * 8; x += 128) {
          const int f = x & 1, r = n0 - kt + (x >> 4), o = (x >> 1) & 7;
          *reinterpret_cast<uint4*>(vs + f * kW8Half + r * 128 + 16 * o) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async();
      }
      float x[128];
#pragma unroll
      for (int q = 0; q < 4; q++) tmem_ld32_nowait(tl + b * 128 + 32 * q, x + 32 * q);
      tmem_wait_ld();
      const bool edge = kt + kW8T - 1 > p0 || (a.window > 0 && kt <= p1 - a.window);
      if (edge) {
        // keys [lo, hi] of the window, or below the number of first tokens
        const int hi = pos - kt, lo = a.window > 0 ? pos - a.window + 1 - kt : 0, early = a.window > 0 ? a.sinks - kt : 0;
#pragma unroll
        for (int q = 0; q < 128; q++)
          if (q > hi || (q < lo && q >= early)) x[q] = -INFINITY;
      }
      float mx = x[0];
#pragma unroll
      for (int q = 1; q < 128; q++) mx = fmaxf(mx, x[q]);
      const float mxs = mx * kLogitScale;
      if (__any_sync(0xffffffffu, mxs > m + kW8Lazy)) {
        const float mn = fmaxf(m, mxs);
        if (j > 0) {
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(pvdone((j - 1) % kW8SBufs), ((j - 1) / kW8SBufs) & 1));
          if (!ok) break;
          tc_fence_after();
          const float f = mn == -INFINITY ? 1.0f : fast_exp2(m - mn);
          l *= f;
#pragma unroll 1
          for (int q = 0; q < 4; q++) {
            float o[32];
            tmem_ld32_nowait(tl + kW8OCol + 32 * q, o);
            tmem_wait_ld();
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 32; e++) w[e] = __float_as_uint(o[e] * f);
            tmem_st32(tl + kW8OCol + 32 * q, w);
          }
          tmem_wait_st();
        }
        m = mn;
      }
      const float mr = m == -INFINITY ? 0.0f : m;     // no visible key so far
#pragma unroll
      for (int q = 0; q < 4; q++) {
        uint32_t ph[16];
#pragma unroll
        for (int e = 0; e < 16; e++) {
          const float u = fast_exp2(fmaf(x[32 * q + 2 * e], kLogitScale, -mr));
          const float v = fast_exp2(fmaf(x[32 * q + 2 * e + 1], kLogitScale, -mr));
          l += u + v;
          ph[e] = pack_elems<ELEM>(u, v);
        }
        tmem_st16(tl + b * 128 + 16 * q, ph);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(pfull(b));
    }
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(ofull, 0) && !failed());
    if (ok) {
      tc_fence_after();
      const float inv = __fdiv_rn(1.0f, l);
      uint8_t* dst = a.out + (((size_t)(t0 + pos) * c.hkv + h) * G + row % G) * (2 * kD);
#pragma unroll 1
      for (int q = 0; q < 4; q++) {
        float o[32];
        tmem_ld32_nowait(tl + kW8OCol + 32 * q, o);
        tmem_wait_ld();
        if (real) {
          uint4* d4 = reinterpret_cast<uint4*>(dst + 64 * q);
#pragma unroll
          for (int e = 0; e < 4; e++)
            d4[e] = make_uint4(pack_elems<ELEM>(o[8 * e] * inv, o[8 * e + 1] * inv),
                               pack_elems<ELEM>(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                               pack_elems<ELEM>(o[8 * e + 4] * inv, o[8 * e + 5] * inv),
                               pack_elems<ELEM>(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tbase, kW8Cols);
  }
}

// [n_tok][heads][128] 16-bit vectors, token rows `stride` elements apart; box
// = tokens x heads x 64 features, 128-byte swizzle.
cudaError_t rows_map(PFN_cuTensorMapEncodeTiled_v12000 enc, int elem, const void* base, int heads, long long n_tok,
                     long long stride, int box_heads, int box_tok, CUtensorMap* m) {
  const cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)heads, (cuuint64_t)n_tok};
  const cuuint64_t str[2] = {(cuuint64_t)kD * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tok};
  const cuuint32_t es[3] = {1, 1, 1};
  if (enc(m, elem == DKV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
          const_cast<void*>(base), dims, str, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_prefill8(const Cache8View& c, int elem, const int32_t* seq_lens, int n_req, const void* q,
                            long long qs, const void* k, long long ks, const void* v, long long vs, void* out,
                            int window, int sinks, cudaStream_t st) {
  PFN_cuTensorMapEncodeTiled_v12000 enc;
  cudaError_t e = tma_encoder(&enc);
  if (e != cudaSuccess) return e;
  W8Call call;
  call.n_req = n_req;
  call.tok0[0] = call.tile0[0] = 0;
  const int tq = kW8T / c.G;
  for (int i = 0; i < n_req; i++) {
    call.tok0[i + 1] = call.tok0[i] + seq_lens[i];
    call.tile0[i + 1] = call.tile0[i] + (seq_lens[i] + tq - 1) / tq;
  }
  const long long n = call.tok0[n_req];
  CUtensorMap mq, mk, mv;
  if ((e = rows_map(enc, elem, q, c.hkv * c.G, n, qs, c.G, tq, &mq)) != cudaSuccess) return e;
  if ((e = rows_map(enc, elem, k, c.hkv, n, ks, 1, kW8T, &mk)) != cudaSuccess) return e;
  if ((e = rows_map(enc, elem, v, c.hkv, n, vs, 1, kW8T, &mv)) != cudaSuccess) return e;
  auto kernel = elem == DKV_F16 ? k_prefill8<DKV_F16> : k_prefill8<DKV_BF16>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kW8Smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, dim3((unsigned)call.tile0[n_req] * c.hkv), dim3(kW8Threads), kW8Smem, st, c, mq, mk,
                          mv, W8Args{static_cast<uint8_t*>(out), window, sinks, tq}, call);
}

}  // namespace dkv
