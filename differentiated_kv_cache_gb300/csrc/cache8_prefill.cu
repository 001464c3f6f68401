// cache8_prefill.cu — causal attention over whole prompts with an optional
// sliding window and first tokens that stay visible (include/dkv.h:
// dkv_cache8_prefill), fp16 or bf16, on the fifth-generation tensor cores.
//
// A work item is 256 query rows of one request and KV head in two halves of
// 128: row r of a half is token r / G of its floor(128 / G), query head r % G of
// the group, so one K / V tile serves the whole group twice and a half spans few
// positions (keys that only part of its rows see stay few). The grid has a CTA an
// item; one is on each SM, and when it comes to its item it asks for one whose
// CTA has not begun (clusterlaunchcontrol), the latest rows first: items differ
// much in their keys (8 x 4096 tokens with 56 / 8 heads 1.51 ms, dealt out in turn
// 1.80; one prompt of 8192 0.41 and 0.46). warp 0 issues the TMA copies (an item's queries, 128-key K and V tiles
// through two stages each), warps 1 and 2 the MMAs of a half each, warps 4..7
// and 8..11 run the softmax of the halves with one thread per row (and most of
// the registers):
//   S = Q K^T        tcgen05, D in tensor memory, 64 keys a step, two buffers
//   P = 2^(S - m)    written over S in 16 bits; m is a maximum of earlier keys,
//                    raised (O, l rescaled) only when a row's P of a step sum
//                    to over 2^12, so that most steps need no maximum at all
//   O += P V         tcgen05, A = P from tensor memory, V MN-major
// S of step n + 2 is issued once P V of step n is done, while the softmax takes
// step n + 1, and the halves do not wait for one another: products run while
// either half's softmax does, and the next item's first products while this
// item's results are written. (Tensor memory holds two S of 64 columns and an O
// of 128 for each half. With one S of 128 columns a half, each softmax waited
// for P V and the next S in turn; that layout was timed only while an MMA took
// 100 cycles to issue, see below, so there is no figure for it as things are.)
// Only key tiles with a visible key are visited, the window's from the diagonal
// back (the nearest keys give a good first m), then the first tokens'; of each,
// a half takes the 32-key parts that some of its rows may see.
//
// Bound by the tensor cores: 32 prompts of 4096 tokens, 32 / 8 heads, window 1024
// take 1.85 ms (1.93 TFLOP, 53% of the measured bf16 burst rate; the steps at the
// window's edges and the diagonal add 5% to the columns of the products), 16384
// tokens with 64 / 8 heads and window 4096 take 1.50 ms (66%; 0.8%). (Other runs
// of the same code: 1.76 and 1.44.) In a step of 64 keys the products of both
// halves take about 1400 of 1650 cycles; S has N = 64, for which the queries are
// read from shared memory again (48 instead of 32 cycles an MMA), the price of the
// second S buffer. With one thread in the MMA warps' loop, whose operands then are
// no uniform registers, an MMA took 100 cycles to issue (2.25 ms); results written
// by warps of their own left the softmax too few registers (2.25 ms); queries
// fetched per half, the second half started a step late: no difference.
//
// 0 * Inf is not 0: an infinite or NaN value makes NaN of every row of its step,
// those that do not see it too. A second kernel computes rows that came out so
// again over what they see (in this kernel the code for it cost 3%, though it
// never ran, and a look at V ahead of the products 5%).
//
// Every wait is bounded; on expiry the kernel latches DKV_ERR_TIMEOUT, waits
// (bounded) for its own copies and MMAs, frees its tensor memory and returns.
#include <algorithm>
#include <cudaTypedefs.h>

#include "cache8.cuh"
#include "dkv_kernels.cuh"
#include "dkv_tc.cuh"

namespace dkv {

cudaError_t tma_encoder(PFN_cuTensorMapEncodeTiled_v12000* fn);

namespace {

constexpr int kW8T = 128;                  // query rows of a half, keys of a tile
constexpr int kW8Threads = 384;
// registers a thread: launched with 168; 128 x 88 + 256 x 208 = 384 x 168
constexpr int kW8RegsFew = 88, kW8RegsMany = 208;
constexpr int kW8Half = kW8T * 128;        // 64 features of 128 rows: 16 KB
constexpr int kW8Tile = 2 * kW8Half;
constexpr int kW8OffK = 2 * kW8Tile;       // after the queries of both halves
constexpr int kW8OffV = kW8OffK + 2 * kW8Tile;
constexpr int kW8OffOut = kW8OffV + 2 * kW8Tile;      // 4 KB a softmax warp, to write whole lines
constexpr int kW8OffBar = kW8OffOut + 8 * 4096;
constexpr int kW8Next = 8;                 // places of the ring of items
constexpr int kW8OffNext = kW8OffBar + 256;           // their barriers, then the answers of 16 bytes
constexpr int kW8Smem = 1024 + kW8OffNext + 24 * kW8Next;
constexpr uint32_t kW8OCol = 256;          // S of the halves, then O of the halves
constexpr uint32_t kW8Cols = 512;
constexpr float kW8Most = 4096.0f;         // largest sum of a row's P of one tile (fp16 holds 65504)

// status[3], zero between calls: a row of this call came out infinite or NaN; the
// blocks of the second kernel then count themselves in the bits below, and the last
// one puts the zero back.
constexpr int kLook = 1 << 30;

constexpr int kW8Req = 1024;
struct W8Call {
  int n_req;
  int tok0[kW8Req + 1];
  int tile0[kW8Req + 1];     // first query tile of a request
};

struct W8Args {
  uint8_t* out;
  int window, sinks, tq;     // tq: tokens of a half
};

// A work item: 2 tq positions from p0 of request i (its tokens at row t0, n0 of
// them) and KV head h; `near` key tiles back from `last`, then the first tiles,
// `count` in all.
struct Item {
  int h, t0, n0, p0, last, near, count;
  int lo, hi, early;   // keys that some row sees: [lo, hi], and below early
  __device__ __forceinline__ int key(int j) const { return (j < near ? last - j : j - near) * kW8T; }
  // 64 keys from kt; every tile of an item has such a step
  __device__ __forceinline__ bool step(int kt) const { return (kt <= hi && kt + 63 >= lo) || kt < early; }
};
__device__ __forceinline__ Item item_of(int x, const Cache8View& c, const W8Args& a, const W8Call& call) {
  Item it;
  it.h = x % c.hkv;
  const int qtile = call.tile0[call.n_req] - 1 - x / c.hkv;     // later rows first: more keys
  int i = 0, hi = call.n_req;
  while (hi - i > 1) {
    const int mid = (i + hi) >> 1;
    if (call.tile0[mid] <= qtile) i = mid; else hi = mid;
  }
  it.t0 = call.tok0[i];
  it.n0 = call.tok0[i + 1] - it.t0;
  it.p0 = (qtile - call.tile0[i]) * 2 * a.tq;
  it.hi = min(it.p0 + 2 * a.tq, it.n0) - 1;
  it.last = it.hi / kW8T;
  it.lo = a.window > 0 ? max(it.p0 - a.window + 1, 0) : 0;
  it.early = a.window > 0 ? min(a.sinks, it.n0) : 0;
  const int from = it.lo / kW8T, first = min((it.early + kW8T - 1) / kW8T, from);
  it.near = it.last - from + 1;
  it.count = it.near + first;
  return it;
}

// The steps of an item in order: its tiles, and in each the 64-key halves that
// some row sees. n: steps, t: tiles of the CTA's sequence so far.
struct Cursor {
  int j, u, n, t;
  __device__ __forceinline__ int key(const Item& it) const { return it.key(j) + 64 * u; }
  __device__ __forceinline__ void begin(const Item& it) {
    j = 0;
    u = it.step(it.key(0)) ? 0 : 1;
  }
  // to the next step; false (with the tile counted): the item's last one it was
  __device__ __forceinline__ bool next(const Item& it) {
    n++;
    if (u == 0 && it.step(it.key(j) + 64)) {
      u = 1;
      return true;
    }
    t++;
    if (++j == it.count) return false;
    u = it.step(it.key(j)) ? 0 : 1;
    return true;
  }
};

// The 32-key parts [c0, c1) of the 64 keys from kt that a half's rows may see
// (one at least).
struct Parts {
  int c0, c1;
};
__device__ __forceinline__ Parts parts_of(const Item& it, const W8Args& a, int half, int kt) {
  const int q0 = it.p0 + half * a.tq, q1 = max(min(q0 + a.tq, it.n0) - 1, q0);
  const int hi = min(q1 - kt, 63), lo = a.window > 0 ? max(q0 - a.window + 1 - kt, 0) : 0;
  const int early = a.window > 0 ? min(a.sinks - kt, 64) : 0;
  Parts p{2, 0};
  if (lo <= hi) p = Parts{lo >> 5, (hi >> 5) + 1};
  if (early > 0) p = Parts{0, max(p.c1, (early + 31) >> 5)};
  if (p.c1 <= p.c0) p = Parts{0, 1};
  return p;
}

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {     // without waiting
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// A block of the grid that has not begun yet is asked for, so that this one does
// its work; the answer (16 bytes) completes the barrier.
__device__ __forceinline__ void ask_item(uint32_t answer, uint32_t bar) {
  mbar_expect_tx(bar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];\n" ::"r"(answer),
               "r"(bar)
               : "memory");
}
// The block's index, -1 if every block has begun (then none may be asked for again).
__device__ __forceinline__ int told_item(uint32_t answer) {
  int x;
  asm volatile(
      "{\n .reg .pred p;\n .reg .b128 h;\n ld.shared.b128 h, [%1];\n mov.s32 %0, -1;\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, h;\n}\n"
      : "=r"(x)
      : "r"(answer)
      : "memory");
  return x;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// bits [0, n)
__device__ __forceinline__ uint32_t below(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }
// Values of a tensor-memory load are used after the wait only.
__device__ __forceinline__ void loaded32(float* v) {
#pragma unroll
  for (int e = 0; e < 32; e++) asm volatile("" : "+f"(v[e]));
}

template <int ELEM>
__global__ void __launch_bounds__(kW8Threads, 1)
    k_prefill8(Cache8View c, const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
               const __grid_constant__ CUtensorMap tv, W8Args a, const __grid_constant__ W8Call call) {
  pdl_launch_dependents();
  pdl_wait();
  if (c.stopped()) return;
  const int G = c.G;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kW8OffBar);
  const uint32_t b0 = smem_u32(bars);
  // S and P V of step n (64 keys) signal sdone and pvdone of (half, n & 3); a K
  // (V) stage is free when both halves' S (P V) of its tile's last step are done,
  // the queries when both halves' last S of an item are. (Four of each: step
  // n + 4 needs a tile or queries that are not loaded before everyone has seen
  // step n's phase.)
  const uint32_t qfull = b0;
  auto kfull = [&](int s) { return b0 + 16u + 8u * s; };
  auto vfull = [&](int s) { return b0 + 32u + 8u * s; };
  auto pfull = [&](int h, int n) { return b0 + 48u + 16u * h + 8u * (n & 1); };
  auto sdone = [&](int h, int n) { return b0 + 80u + 32u * h + 8u * (n & 3); };
  auto pvdone = [&](int h, int n) { return b0 + 144u + 32u * h + 8u * (n & 3); };
  auto drain = [&](int h) { return b0 + 208u + 8u * h; };
  // Item r + 1 of this CTA (item 0 is its own block): place r & 7. Its index is
  // asked for when item r begins, whose first K tile waits for S of the tile
  // two before; every warp has then read the indices up to item r - 3, so a
  // place is free long before it is used again.
  auto told = [&](int r) { return b0 + 256u + 8u * (r & (kW8Next - 1)); };
  auto answer = [&](int r) { return b0 + 256u + 8u * kW8Next + 16u * (r & (kW8Next - 1)); };
  auto item_told = [&](int r, bool& ok) {      // the same for every lane
    ok = __all_sync(0xffffffffu, mbar_wait_bounded(told(r), (r / kW8Next) & 1));
    return ok ? told_item(answer(r)) : -1;
  };
  uint32_t* s_taddr = reinterpret_cast<uint32_t*>(bars + 28);
  int* s_fail = reinterpret_cast<int*>(s_taddr + 1);
  // (broadcasts: uniform over a warp for the compiler too)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 28; s++)      // pfull: a lane of each warp
      mbar_init(b0 + 8u * s, s >= 6 && s < 10 ? 4 : 1);
    for (int r = 0; r < kW8Next; r++) mbar_init(told(r), 1);
    *s_fail = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(smem_u32(s_taddr), kW8Cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = __shfl_sync(0xffffffffu, *s_taddr, 0);
  auto fail = [&]() {
    c.latch(DKV_ERR_TIMEOUT, -1);
    *(volatile int*)s_fail = 1;
  };
  auto failed = [&]() { return *(volatile int*)s_fail != 0; };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kW8RegsFew));
    if (warp == 0) {
      // ---- copies: an item's first K tile, its queries, then K(j + 1) ahead of V(j) ----
      if (lane == 0) {
        int nk = 0, nv = 0, nq = 0;      // K tiles, V tiles and items so far
        int done = 0;                    // steps of the tiles whose K is loaded
        int end[2] = {0, 0};             // last step of the latest tile of each stage
        int vend[2] = {0, 0};
        bool ok = true;
        auto load = [&](const Item& it, int j, bool is_k) {
          const int t = is_k ? nk : nv, s = t & 1;
          const uint32_t full = is_k ? kfull(s) : vfull(s);
          const int e = is_k ? end[s] : vend[s];
          if (t >= 2)          // tile t - 2 of the stage is done with
            for (int h = 0; h < 2; h++)
              if (!mbar_wait_bounded(is_k ? sdone(h, e) : pvdone(h, e), (e >> 2) & 1)) return false;
          mbar_expect_tx(full, kW8Tile);
          for (int f = 0; f < 2; f++)
            tma_load_3d(smem_u32(smem + (is_k ? kW8OffK : kW8OffV) + s * kW8Tile + f * kW8Half), is_k ? &tk : &tv,
                        64 * f, it.h, it.t0 + it.key(j), full);
          if (is_k) {
            nk++;
            done += (it.step(it.key(j)) ? 1 : 0) + (it.step(it.key(j) + 64) ? 1 : 0);
            end[s] = done - 1;
          } else {
            nv++;
            vend[s] = end[s];            // K of the tile after next is not loaded yet
          }
          return true;
        };
        int asked = 0;
        for (int x = blockIdx.x; x >= 0 && !failed();) {
          fence_proxy_async();
          ask_item(answer(asked), told(asked));
          asked++;
          const Item it = item_of(x, c, a, call);
          const int last = done - 1;     // the last step of the item before
          ok = load(it, 0, true);
          if (nq > 0)
            for (int h = 0; h < 2; h++) ok = ok && mbar_wait_bounded(sdone(h, last), (last >> 2) & 1);
          if (!ok) break;
          mbar_expect_tx(qfull, (uint32_t)(4 * 128 * a.tq * G));
          for (int f = 0; f < 4; f++)
            tma_load_3d(smem_u32(smem + f * kW8Half), &tq, 64 * (f & 1), it.h * G, it.t0 + it.p0 + (f >> 1) * a.tq, qfull);
          nq++;
          for (int j = 0; ok && j < it.count && !failed(); j++) {
            if (j + 1 < it.count) ok = load(it, j + 1, true);
            if (ok) ok = load(it, j, false);
          }
          if (!ok) break;
          ok = mbar_wait_bounded(told(asked - 1), ((asked - 1) / kW8Next) & 1);
          if (!ok) break;
          x = told_item(answer(asked - 1));
        }
        if (!ok) fail();
        // no copy of this CTA, and no answer, may still be in flight when it exits
        if (asked > 0) mbar_wait_bounded(told(asked - 1), ((asked - 1) / kW8Next) & 1);
        if (nq > 0) mbar_wait_bounded(qfull, (nq - 1) & 1);
        for (int t = max(nk - 2, 0); t < nk; t++) mbar_wait_bounded(kfull(t & 1), (t >> 1) & 1);
        for (int t = max(nv - 2, 0); t < nv; t++) mbar_wait_bounded(vfull(t & 1), (t >> 1) & 1);
      }
    } else if (warp < 3) {
      // ---- MMAs of a half: S of step n once P V of step n - 1 is done, then P V ----
      // The whole warp walks the steps, one lane issues: operands stay in uniform
      // registers.
      constexpr uint32_t type = ELEM == DKV_BF16 ? (1u << 7) | (1u << 10) : 0u;   // A and B formats
      constexpr uint32_t id_pv = umma_idesc_f16(128, 128) | type | (1u << 16);   // B (V) MN-major
      const int h = warp - 1;
      const uint32_t ts = tbase + h * 128, to = tbase + kW8OCol + h * 128;
      const uint64_t qd = umma_desc_sw128(smem_u32(smem + h * kW8Tile));
      const uint64_t kd = umma_desc_sw128(smem_u32(smem + kW8OffK)), vd = umma_desc_sw128_mn(smem_u32(smem + kW8OffV), kW8Half);
      Cursor sc{0, 0, 0, 0}, pc{0, 0, 0, 0};     // steps of S and, two behind, of P V
      int ii = 0;
      bool ok = true;
      for (int x = blockIdx.x, next = -1; x >= 0; x = ok ? next : -1, ii++) {
        const Item it = item_of(x, c, a, call);
        sc.begin(it);
        pc.begin(it);
        bool more_s = true, more_p = true;
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(qfull, ii & 1));
        for (int ahead = 0; ok && more_p; ahead++) {
          if (ahead >= 2) {
            const Parts p = parts_of(it, a, h, pc.key(it));
            const int st = pc.t & 1, n = pc.n;
            const bool first = ahead == 2;
            const uint64_t bd = vd + ((st * kW8Tile + pc.u * 8192) >> 4);
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(vfull(st), (pc.t >> 1) & 1) &&
                                             mbar_wait_bounded(pfull(h, n), (n >> 1) & 1));
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
              for (int kk = 0; kk < 4; kk++)
                if (kk >= 2 * p.c0 && kk < 2 * p.c1)
                  umma_f16_tmem_a(to, ts + 64 * (n & 1) + 8 * kk, bd + kk * (2048 >> 4), id_pv, !first || kk > 2 * p.c0);
              umma_commit(pvdone(h, n));
            }
            __syncwarp();
            more_p = pc.next(it);
          }
          if (more_s) {
            const Parts p = parts_of(it, a, h, sc.key(it));
            const int st = sc.t & 1, n = sc.n;
            const uint32_t id = umma_idesc_f16(128, 32 * (p.c1 - p.c0)) | type;
            const uint64_t bd = kd + ((st * kW8Tile + sc.u * 8192 + 4096 * p.c0) >> 4);
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(kfull(st), (sc.t >> 1) & 1) &&
                                             (n < 2 || mbar_wait_bounded(pvdone(h, n - 2), ((n - 2) >> 2) & 1)));
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
              for (int k = 0; k < 8; k++) {
                const int off = ((k >> 2) * kW8Half + (k & 3) * 32) >> 4;      // half of the features, 16 of them
                umma_f16(ts + 64 * (n & 1) + 32 * p.c0, qd + off, bd + off, id, k > 0);
              }
              umma_commit(sdone(h, n));
            }
            __syncwarp();
            more_s = sc.next(it);
            if (!more_s) next = item_told(ii, ok);     // while its P is awaited
          }
        }
      }
      if (!ok) fail();
      if (lane == 0) {
        umma_commit(drain(h));                 // every MMA issued so far has completed
        mbar_wait_bounded(drain(h), 0);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kW8RegsMany));
    // ---- softmax: a thread per row of a half ----
    const int half = warp >= 8 ? 1 : 0, lg = warp & 3, row = 32 * lg + lane, token = row / G;
    const uint32_t tl = tbase + ((uint32_t)(32 * lg) << 16);
    const uint32_t ts = tl + half * 128, to = tl + kW8OCol + half * 128;
    Cursor cu{0, 0, 0, 0};
    bool ok = true;
    int ii = 0;
    Item it = item_of(blockIdx.x, c, a, call);
    for (int next = 0; next >= 0; ii++) {
      const int q0 = it.p0 + half * a.tq, q1 = max(min(q0 + a.tq, it.n0) - 1, q0), pos = q0 + token;
      // rows behind the request, or of no token, hold what happened to be there:
      // they take no part in what the warp decides
      const bool real = token < a.tq && pos < it.n0;
      float m = -INFINITY, l = 0.0f;
      cu.begin(it);
      bool first = true, more = true, have = false, raise = true;
      float s[64];
      for (; more; first = false) {
        const int kt = cu.key(it), n = cu.n, stage = cu.t & 1, stage_par = (cu.t >> 1) & 1, u = cu.u;
        const uint32_t tb = ts + 64 * (n & 1);
        if (!have) {
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(sdone(half, n), (n >> 2) & 1));
          if (!ok) break;
          tc_fence_after();
          tmem_ld32_nowait(tb, s);
          tmem_ld32_nowait(tb + 32, s + 32);
        }
        if (kt + 64 > it.n0) {
          // V rows behind the request belong to others: zero them, whatever they
          // hold (their weight is 0, but 0 * Inf is not). Both halves do, each
          // ahead of its own product
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(vfull(stage), stage_par));
          if (!ok) break;
          const int own = max(it.n0 - kt, 0);
          uint8_t* vs = smem + kW8OffV + stage * kW8Tile + u * 8192;
          for (int y = row; y < 2 * (64 - own) * 8; y += 128) {
            const int f = y & 1, r = own + (y >> 4), o = (y >> 1) & 7;
            *reinterpret_cast<uint4*>(vs + f * kW8Half + r * 128 + 16 * o) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async();
        }
        tmem_wait_ld();
        loaded32(s);
        loaded32(s + 32);
        // some row does not see all 64 keys: those of the window, or below the
        // number of first tokens
        if (!(kt + 63 <= q0 && (a.window <= 0 || kt > q1 - a.window || kt + 64 <= a.sinks))) {
          const int hi = pos - kt + 1, lo = a.window > 0 ? pos - a.window + 1 - kt : 0, early = a.window > 0 ? a.sinks - kt : 0;
          const uint32_t see0 = below(hi) & (~below(lo) | below(early));
          const uint32_t see1 = below(hi - 32) & (~below(lo - 32) | below(early - 32));
#pragma unroll
          for (int e = 0; e < 32; e++) {
            s[e] = see0 & (1u << e) ? s[e] : -INFINITY;
            s[32 + e] = see1 & (1u << e) ? s[32 + e] : -INFINITY;
          }
        }
        uint32_t ph[32];
        float sum;
#pragma unroll 1
        for (bool again = raise;; again = true) {
          if (again) {
            float y[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int e = 4; e < 64; e++) y[e & 3] = fmaxf(y[e & 3], s[e]);
            const float mn = fmaxf(m, fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])) * kLogitScale);
            if (!first) {      // O is still once the last P V is done
              ok = __all_sync(0xffffffffu, mbar_wait_bounded(pvdone(half, n - 1), ((n - 1) >> 2) & 1));
              if (!ok) break;
              tc_fence_after();
              const float f = mn == -INFINITY ? 1.0f : fast_exp2(m - mn);
              l *= f;
#pragma unroll 1
              for (int q = 0; q < 4; q++) {
                float o[32];
                tmem_ld32_nowait(to + 32 * q, o);
                tmem_wait_ld();
                loaded32(o);
                uint32_t w[32];
#pragma unroll
                for (int e = 0; e < 32; e++) w[e] = __float_as_uint(o[e] * f);
                tmem_st32(to + 32 * q, w);
              }
              tmem_wait_st();
            }
            m = mn;
            raise = __any_sync(0xffffffffu, real && m == -INFINITY);     // a row that has seen no key so far
          }
          const float mr = m == -INFINITY ? 0.0f : m;
          const uint64_t sc2 = f32x2(kLogitScale, kLogitScale), nm2 = f32x2(-mr, -mr);
          uint64_t l2[4] = {0, 0, 0, 0};
#pragma unroll
          for (int e = 0; e < 32; e++) {
            const uint64_t y = fma_f32x2(f32x2(s[2 * e], s[2 * e + 1]), sc2, nm2);
            const float v0 = fast_exp2(__uint_as_float((uint32_t)y)), v1 = fast_exp2(__uint_as_float((uint32_t)(y >> 32)));
            l2[e & 3] = add_f32x2(l2[e & 3], f32x2(v0, v1));
            ph[e] = pack_elems<ELEM>(v0, v1);
          }
          const uint64_t t2 = add_f32x2(add_f32x2(l2[0], l2[1]), add_f32x2(l2[2], l2[3]));
          sum = __uint_as_float((uint32_t)t2) + __uint_as_float((uint32_t)(t2 >> 32));
          if (again || !__any_sync(0xffffffffu, real && !(sum <= kW8Most))) break;
        }
        if (!ok) break;
        l += sum;
        tmem_st16(tb, ph);
        tmem_st16(tb + 16, ph + 16);
        // the next S, if it is there, comes while P goes
        more = cu.next(it);
        have = more && __all_sync(0xffffffffu, mbar_test(sdone(half, n + 1), ((n + 1) >> 2) & 1));
        if (have) {
          tc_fence_after();
          tmem_ld32_nowait(ts + 64 * ((n + 1) & 1), s);
          tmem_ld32_nowait(ts + 64 * ((n + 1) & 1) + 32, s + 32);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull(half, n));
      }
      // the next item, while P V of the last step is awaited
      next = ok ? item_told(ii, ok) : -1;
      const Item then = next >= 0 ? item_of(next, c, a, call) : it;
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(pvdone(half, cu.n - 1), ((cu.n - 1) >> 2) & 1));
      if (!ok) break;
      tc_fence_after();
      const float inv = __fdiv_rn(1.0f, l);
      // through shared memory, 64 features at a time: eight lanes write a line
      const unsigned long long dst = real ? reinterpret_cast<unsigned long long>(a.out) +
          (((size_t)(it.t0 + pos) * c.hkv + it.h) * G + row % G) * (2 * kD) : 0ull;
      uint8_t* stage = smem + kW8OffOut + (warp - 4) * 4096;
      uint32_t bad[4] = {0, 0, 0, 0};
#pragma unroll 1
      for (int q = 0; q < 2; q++) {
#pragma unroll
        for (int r = 0; r < 2; r++) {
          float o[32];
          tmem_ld32_nowait(to + 64 * q + 32 * r, o);
          tmem_wait_ld();
          loaded32(o);
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const uint4 w = make_uint4(pack_elems<ELEM>(o[8 * e] * inv, o[8 * e + 1] * inv),
                                       pack_elems<ELEM>(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                                       pack_elems<ELEM>(o[8 * e + 4] * inv, o[8 * e + 5] * inv),
                                       pack_elems<ELEM>(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
            find_not_finite<ELEM>(bad[0], w.x);
            find_not_finite<ELEM>(bad[1], w.y);
            find_not_finite<ELEM>(bad[2], w.z);
            find_not_finite<ELEM>(bad[3], w.w);
            *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 * r + e) ^ (lane & 7)) << 4)) = w;
          }
        }
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const int r = 4 * e + (lane >> 3);
          const unsigned long long to_row = __shfl_sync(0xffffffffu, dst, r);
          const uint4 w = *reinterpret_cast<const uint4*>(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
          if (to_row) *reinterpret_cast<uint4*>(to_row + 128 * q + 16 * (lane & 7)) = w;
        }
        __syncwarp();
      }
      if (real && found_not_finite(bad[0] | bad[1] | bad[2] | bad[3])) {
        c.status[2] = 1;
        c.status[3] = kLook;
      }
      it = then;
      tc_fence_before();
    }
    if (!ok) fail();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tbase, kW8Cols);
  }
}

// ---- Rows that came out infinite or NaN ----
// A feature of a row is NaN by right where the row sees a NaN value of it,
// infinite ones of both signs, an infinite one under a weight of 0, or a key whose
// logit is NaN or +Inf. It is wrong where a value that the row does not see, in a
// step beside its keys, made 0 * NaN or 0 * Inf of it, and where an infinite value
// that it does see met a weight that rounds to 0 in 16 bits. What is infinite is
// right where the row sees an infinite value of that feature (nothing makes a
// number of NaN again). Else a mean of values of the type's largest size was
// rounded up, or a sum of bf16 values left fp32's range: weights of up to 2^12 make
// that possible above 2^122 / tokens.
//
// A block takes the halves of the kernel above in turn (128 / G tokens, all heads
// of a group). Of one that holds such a feature it looks through the keys and
// values that its rows see, and those that the steps beside them hold, for what is
// not finite, 512 keys at a time, the first ones first and then from the diagonal
// back, until all is seen to be right. Where some is not, it computes the half
// again with mma.sync, with zeros for the values that are not finite, and writes
// the features that are not right, and only those. So a call that meets such a
// value costs a look through its results, and through keys and values as far as
// that value; and each value the computing of the few halves that hold it in a step
// but not in their rows' sight. 16384 tokens, 64 / 8 heads, window 4096 + 64, bf16 (1.45
// ms without such a value): one NaN in a first token's key or value 1.95 ms, in the
// middle 2.1, a feature infinite in every token 10.8, one value in 10^4 NaN 10.4
// (with 64 / 64 heads 20.8: every half again, at 110 TFLOP/s). A walk of a warp a
// row through its keys, nearest first, took 244 ms for one NaN in 4096 tokens with
// window 1024 (0.14 ms without).
//
// The launch that finds nothing adds 1.5 us to a call.
struct Again8 {
  uint8_t* out;
  const uint8_t *q, *k, *v;
  long long qs, ks, vs;      // row strides in bytes
  W8Args w;
};
constexpr int kAgThreads = 256;            // a warp for 16 rows
constexpr int kAgKeys = 64;                // keys of a tile
constexpr int kAgLook = 512;               // keys between two looks at what is left

// Bits of features: NaN by right, +Inf and -Inf among the values that are seen.
enum { kNan, kUp, kDown, kKinds };
struct AgShared {
  uint4 k[kAgKeys * 16], v[kAgKeys * 16];          // 16-byte pieces, swizzled by row % 8
  uint32_t seen[kKinds][kW8T][4];                  // by a token
  uint32_t all[kKinds][4];                         // by every token
  uint32_t unseen[4];                              // any value that some token does not see
  uint32_t need[kW8T][4], inf[kW8T][4];            // per row: infinite or NaN, then what is to be computed again; infinite
};
// A bit for each of eight 16-bit places that are on in m0 .. m3.
__device__ __forceinline__ uint32_t bits8(uint32_t m0, uint32_t m1, uint32_t m2, uint32_t m3) {
  auto two = [](uint32_t m) { return (m & 1u) | (m >> 31 << 1); };
  return two(m0) | two(m1) << 2 | two(m2) << 4 | two(m3) << 6;
}
template <int ELEM>
struct Elem {
  static constexpr uint32_t kInf = ELEM == DKV_F16 ? 0x7c007c00u : 0x7f807f80u;
  static __device__ __forceinline__ uint32_t mag(uint32_t w) { return w & 0x7fff7fffu; }
  static __device__ __forceinline__ bool all_finite(uint4 w) {
    return (__vcmpgeu2(mag(w.x), kInf) | __vcmpgeu2(mag(w.y), kInf) | __vcmpgeu2(mag(w.z), kInf) | __vcmpgeu2(mag(w.w), kInf)) == 0;
  }
  static __device__ __forceinline__ uint32_t nans(uint4 w) {
    return bits8(__vcmpgtu2(mag(w.x), kInf), __vcmpgtu2(mag(w.y), kInf), __vcmpgtu2(mag(w.z), kInf), __vcmpgtu2(mag(w.w), kInf));
  }
  static __device__ __forceinline__ uint32_t equal(uint4 w, uint32_t x) {
    return bits8(__vcmpeq2(w.x, x), __vcmpeq2(w.y, x), __vcmpeq2(w.z, x), __vcmpeq2(w.w, x));
  }
  // zeros in place of what is not finite
  static __device__ __forceinline__ uint4 finite_of(uint4 w) {
    return make_uint4(w.x & __vcmpltu2(mag(w.x), kInf), w.y & __vcmpltu2(mag(w.y), kInf), w.z & __vcmpltu2(mag(w.z), kInf),
                      w.w & __vcmpltu2(mag(w.w), kInf));
  }
};

// Keys [0, first) and [lo, hi), numbered in a row.
struct AgKeys {
  int first, lo, total;
  __device__ __forceinline__ AgKeys(int first_, int lo_, int hi) : first(min(first_, lo_)), lo(lo_), total(first + hi - lo_) {}
  __device__ __forceinline__ int operator()(int x) const { return x < first ? x : lo + x - first; }
};

// The bits of piece c (eight features) of key j, for the tokens that see it.
// Seldom reached.
__device__ __noinline__ void mark(AgShared& sh, int q0, int nt, const W8Args& a, int j, int c, uint32_t nan, uint32_t up,
                                  uint32_t down) {
  const int word = c >> 2, shift = 8 * (c & 3);
  const uint32_t b[kKinds] = {nan << shift, up << shift, down << shift};
  auto put = [](uint32_t& w, uint32_t x) {
    if ((*(volatile uint32_t*)&w & x) != x) atomicOr(&w, x);
  };
  const int t0 = max(j - q0, 0);      // the tokens [t0, t1) see it
  const int t1 = a.window <= 0 || j < a.sinks ? nt : (int)min((long long)nt, (long long)j - q0 + a.window);
  const bool all = t0 == 0 && t1 == nt;
  if (!all) put(sh.unseen[word], b[kNan] | b[kUp] | b[kDown]);
  for (int i = 0; i < kKinds; i++)
    if (all) put(sh.all[i][word], b[i]);
    else if (b[i])
      for (int t = t0; t < t1; t++) put(sh.seen[i][t][word], b[i]);
}
struct AgRow {
  uint32_t nan, up, down;
};
// Of a word of features of a token.
__device__ __forceinline__ AgRow row_of(const AgShared& sh, int t, int w) {
  AgRow r{sh.seen[kNan][t][w] | sh.all[kNan][w], sh.seen[kUp][t][w] | sh.all[kUp][w], sh.seen[kDown][t][w] | sh.all[kDown][w]};
  r.nan |= r.up & r.down;
  return r;
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// The half again: S = Q K^T and O += P V with mma.sync m16n8k16, 16 rows a warp,
// in the manner and the types of the kernel above; weights are at most 2^-above.
template <int ELEM>
__device__ __noinline__ void half_again(AgShared& sh, const Cache8View& c, const Again8& a, const Item& it, int q0, int nt,
                                        float above) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, G = c.G;
  const int window = a.w.window, q1 = q0 + nt - 1;
  const AgKeys key(window > 0 ? min(a.w.sinks, it.n0) : 0, window > 0 ? max(q0 - window + 1, 0) : 0, q1 + 1);
  const uint32_t* need = sh.need[16 * warp + (lane & 15)];
  const bool mine = __any_sync(0xffffffffu, (need[0] | need[1] | need[2] | need[3]) != 0);
  int pos[2];
  long long row[2];            // of the output and the queries: token, head
  uint32_t qf[8][4];
#pragma unroll
  for (int e = 0; e < 2; e++) {
    const int r = 16 * warp + g + 8 * e;
    pos[e] = q0 + r / G;
    const bool in = r < nt * G;
    const long long tok = (long long)it.t0 + pos[e];
    row[e] = in ? (tok * c.hkv + it.h) * G + r % G : -1;
    const uint8_t* p = a.q + tok * a.qs + ((size_t)it.h * G + r % G) * (2 * kD) + 4 * t;
#pragma unroll
    for (int k = 0; k < 8; k++) {
      qf[k][e] = in ? *reinterpret_cast<const uint32_t*>(p + 32 * k) : 0u;
      qf[k][2 + e] = in ? *reinterpret_cast<const uint32_t*>(p + 32 * k + 16) : 0u;
    }
  }
  float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 16; i++)
#pragma unroll
    for (int e = 0; e < 4; e++) o[i][e] = 0.0f;
  const uint32_t ks = smem_u32(sh.k), vs = smem_u32(sh.v);
  auto piece = [](uint32_t base, int r, int ch) { return base + 16 * (16 * r + (ch ^ (r & 7))); };
#pragma unroll 1
  for (int base = 0; base < key.total; base += kAgKeys) {
    __syncthreads();
    for (int i = threadIdx.x; i < kAgKeys * 16; i += kAgThreads) {
      const int r = i >> 4, ch = i & 15, at = 16 * r + (ch ^ (r & 7));
      uint4 kw = make_uint4(0, 0, 0, 0), vw = kw;
      const int j = key(min(base + r, key.total - 1));
      if (base + r < key.total) {
        kw = *reinterpret_cast<const uint4*>(a.k + ((long long)it.t0 + j) * a.ks + it.h * (2 * kD) + 16 * ch);
        vw = *reinterpret_cast<const uint4*>(a.v + ((long long)it.t0 + j) * a.vs + it.h * (2 * kD) + 16 * ch);
      }
      sh.k[at] = kw;
      sh.v[at] = Elem<ELEM>::finite_of(vw);
    }
    __syncthreads();
    if (!mine) continue;
    float s[8][4];
#pragma unroll
    for (int n = 0; n < 8; n++) {
#pragma unroll
      for (int e = 0; e < 4; e++) s[n][e] = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; k++) {
        uint32_t b[4];
        ldmatrix_x4(b, piece(ks, 8 * n + (lane & 7), 4 * k + (lane >> 3)));
        mma_elem<ELEM>(s[n], qf[2 * k], b[0], b[1]);
        mma_elem<ELEM>(s[n], qf[2 * k + 1], b[2], b[3]);
      }
    }
    float top[2] = {m[0], m[1]};
    const int j0 = key(base), j1 = key(base + kAgKeys - 1);
    if (base + kAgKeys > key.total || j1 > q0 || !(window <= 0 || j0 > q1 - window || j1 < a.w.sinks)) {
#pragma unroll
      for (int n = 0; n < 8; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) {        // some token does not see every key
          const int x = base + 8 * n + 2 * t + (e & 1), j = key(x), p = pos[e >> 1];
          if (!(x < key.total && j <= p && (window <= 0 || j > p - window || j < a.w.sinks))) s[n][e] = -INFINITY;
        }
    }
#pragma unroll
    for (int n = 0; n < 8; n++)
#pragma unroll
      for (int e = 0; e < 4; e++) {
        s[n][e] *= kLogitScale;
        top[e >> 1] = fmaxf(top[e >> 1], s[n][e]);
      }
    float f[2], off[2];
#pragma unroll
    for (int e = 0; e < 2; e++) {
      top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
      top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
      f[e] = top[e] == -INFINITY ? 1.0f : fast_exp2(m[e] - top[e]);
      off[e] = top[e] == -INFINITY ? 0.0f : top[e] + above;
      m[e] = top[e];
      l[e] *= f[e];
    }
#pragma unroll
    for (int i = 0; i < 16; i++)
#pragma unroll
      for (int e = 0; e < 4; e++) o[i][e] *= f[e >> 1];
#pragma unroll
    for (int n = 0; n < 8; n++)
#pragma unroll
      for (int e = 0; e < 4; e++) {
        s[n][e] = fast_exp2(s[n][e] - off[e >> 1]);
        l[e >> 1] += s[n][e];
      }
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const uint32_t p[4] = {pack_elems<ELEM>(s[2 * k][0], s[2 * k][1]), pack_elems<ELEM>(s[2 * k][2], s[2 * k][3]),
                             pack_elems<ELEM>(s[2 * k + 1][0], s[2 * k + 1][1]), pack_elems<ELEM>(s[2 * k + 1][2], s[2 * k + 1][3])};
#pragma unroll
      for (int n = 0; n < 8; n++) {
        uint32_t b[4];
        ldmatrix_x4_trans(b, piece(vs, 16 * k + (lane & 15), 2 * n + (lane >> 4)));
        mma_elem<ELEM>(o[2 * n], p, b[0], b[1]);
        mma_elem<ELEM>(o[2 * n + 1], p, b[2], b[3]);
      }
    }
  }
  if (!mine) return;
#pragma unroll
  for (int e = 0; e < 2; e++) {
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    if (row[e] < 0) continue;
    const int r = 16 * warp + g + 8 * e;
    const float inv = __fdiv_rn(1.0f, l[e]);
    uint16_t* out = reinterpret_cast<uint16_t*>(a.out + row[e] * (2 * kD));
#pragma unroll
    for (int i = 0; i < 16; i++) {
      const int w = i >> 2;
      if ((sh.need[r][w] >> (8 * (i & 3)) & 0xffu) == 0) continue;
      const AgRow x = row_of(sh, r / G, w);
#pragma unroll
      for (int y = 0; y < 2; y++) {
        const int at = 8 * (i & 3) + 2 * t + y;
        if (!((sh.need[r][w] & ~x.nan) >> at & 1u)) continue;
        // an infinite sum is infinite, unless the weights are NaN
        const float v = (x.up | x.down) >> at & 1u ? (x.up >> at & 1u ? INFINITY : -INFINITY) * inv : o[i][2 * e + y] * inv;
        out[8 * i + 2 * t + y] = float_elem<ELEM>(in_range<ELEM>(v));
      }
    }
  }
}

template <int ELEM>
__global__ void __launch_bounds__(kAgThreads, 1) k_prefill8_again(Cache8View c, Again8 a, const __grid_constant__ W8Call call) {
  pdl_launch_dependents();
  pdl_wait();
  if (c.stopped() || (*(volatile int*)(c.status + 3) & kLook) == 0) return;
  __shared__ AgShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x, G = c.G, tq = a.w.tq;
  const long long halves = 2ll * call.tile0[call.n_req] * c.hkv;
#pragma unroll 1
  for (long long x = blockIdx.x; x < halves; x += gridDim.x) {
    const Item it = item_of((int)(x >> 1), c, a.w, call);
    const int q0 = it.p0 + (int)(x & 1) * tq, nt = min(tq, it.n0 - q0);      // its tokens
    if (nt <= 0) continue;
    // what its rows hold
    __syncthreads();           // the half before is done with
    uint32_t some = 0;
    uint4 w[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const int r = 16 * warp + 2 * i + (lane >> 4);
      w[i] = make_uint4(0, 0, 0, 0);
      if (r < nt * G)
        w[i] = *reinterpret_cast<const uint4*>(a.out + (((long long)(it.t0 + q0 + r / G) * c.hkv + it.h) * G + r % G) * (2 * kD) +
                                               16 * (lane & 15));
    }
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const int r = 16 * warp + 2 * i + (lane >> 4);
      uint32_t inf = (Elem<ELEM>::equal(w[i], Elem<ELEM>::kInf) | Elem<ELEM>::equal(w[i], Elem<ELEM>::kInf | 0x80008000u)) << (8 * (lane & 3));
      uint32_t b = inf | Elem<ELEM>::nans(w[i]) << (8 * (lane & 3));
      some |= b;
#pragma unroll
      for (int d = 1; d <= 2; d <<= 1) {
        b |= __shfl_xor_sync(0xffffffffu, b, d);
        inf |= __shfl_xor_sync(0xffffffffu, inf, d);
      }
      if ((lane & 3) == 0) {
        sh.need[r][lane >> 2 & 3] = b;
        sh.inf[r][lane >> 2 & 3] = inf;
      }
    }
    for (int i = tid; i < kKinds * kW8T * 4; i += kAgThreads) (&sh.seen[0][0][0])[i] = 0;
    if (tid < kKinds * 4) (&sh.all[0][0])[tid] = 0;
    if (tid < 4) sh.unseen[tid] = 0;
    if (!__syncthreads_or(some != 0)) continue;
    // what is not finite: of every key that some token sees, or that a step beside
    // those holds (no step of the item's lies outside the tiles of 128 keys that its
    // 2 tq rows see some of)
    const int beside = 2 * tq + kW8T, q1 = q0 + nt - 1;
    const int lo = a.w.window > 0 ? max(q0 - a.w.window + 1 - beside, 0) : 0;
    const int first = a.w.window > 0 && a.w.sinks > 0 ? min(a.w.sinks, it.n0 - kW8T) + kW8T : 0;
    const AgKeys key(first, lo, (int)min((long long)q1 + 1 + beside, (long long)it.n0));
    const int looks = (key.total + kAgLook - 1) / kAgLook;
    bool left = true;
#pragma unroll 1
    for (int n = 0; left && n < looks; n++) {
      const int from = (n == 0 ? 0 : looks - n) * kAgLook, end = min(from + kAgLook, key.total);
#pragma unroll 1
      for (int y = from; y < end; y += 8 * (kAgThreads / 16)) {
        uint4 z[8];
        bool bad = false;
        auto at = [&](int i) { return key(min(y + i * (kAgThreads / 16) + (tid >> 4), end - 1)); };   // the last one several times
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const long long j = (long long)it.t0 + at(i);
          w[i] = *reinterpret_cast<const uint4*>(a.k + j * a.ks + it.h * (2 * kD) + 16 * (tid & 15));
          z[i] = *reinterpret_cast<const uint4*>(a.v + j * a.vs + it.h * (2 * kD) + 16 * (tid & 15));
        }
#pragma unroll
        for (int i = 0; i < 8; i++) bad |= !Elem<ELEM>::all_finite(w[i]) || !Elem<ELEM>::all_finite(z[i]);
        if (!__any_sync(0xffffffffu, bad)) continue;
#pragma unroll
        for (int i = 0; i < 8; i++) {
          // of the whole key: a NaN makes its logit NaN, an infinite entry NaN or
          // infinite, and then what it gives of an infinite value is NaN
          const bool none = __ballot_sync(0xffffffffu, Elem<ELEM>::nans(w[i]) != 0) >> (lane & 16) & 0xffffu;
          const bool odd = __ballot_sync(0xffffffffu, !Elem<ELEM>::all_finite(w[i])) >> (lane & 16) & 0xffffu;
          uint32_t nan = Elem<ELEM>::nans(z[i]), up = Elem<ELEM>::equal(z[i], Elem<ELEM>::kInf);
          uint32_t down = Elem<ELEM>::equal(z[i], Elem<ELEM>::kInf | 0x80008000u);
          if (odd) nan |= up | down;
          if (none) nan = 0xffu;
          if (nan | up | down) mark(sh, q0, nt, a.w, at(i), tid & 15, nan, up, down);
        }
      }
      __syncthreads();
      bool open = false;
      if (tid < nt * G)
        for (int e = 0; e < 4; e++) {
          const AgRow r = row_of(sh, tid / G, e);
          open |= (sh.need[tid][e] & ~r.nan & ~(sh.inf[tid][e] & (r.up | r.down))) != 0;
        }
      left = __syncthreads_or(open);
    }
    if (!left) continue;
    bool again = false, wide = false;
    if (tid < nt * G) {
      uint32_t* need = sh.need[tid];
      // a row with a feature that is not NaN has weights that are not: what is
      // infinite of it needs no computing, and other NaN came of sums
      bool sure = false;
      for (int e = 0; e < 4; e++) sure |= (need[e] & ~sh.inf[tid][e]) != 0xffffffffu;
      uint16_t* out = reinterpret_cast<uint16_t*>(
          a.out + (((long long)(it.t0 + q0 + tid / G) * c.hkv + it.h) * G + tid % G) * (2 * kD));
      for (int e = 0; e < 4; e++) {
        const AgRow r = row_of(sh, tid / G, e);
        const uint32_t x = need[e] & ~r.nan & ~(sh.inf[tid][e] & (r.up | r.down)), inf = x & (r.up | r.down);
        if (sure) {
          for (uint32_t f = inf; f; f &= f - 1) {
            const int b = __ffs(f) - 1;
            out[32 * e + b] = float_elem<ELEM>(r.up >> b & 1u ? INFINITY : -INFINITY);
          }
          need[e] = x & ~inf;
          wide |= (need[e] & (sh.inf[tid][e] | ~sh.unseen[e])) != 0;
        } else {
          need[e] = x & (inf | sh.unseen[e]);
        }
        again |= need[e] != 0;
      }
    }
    if (!__syncthreads_or(again)) continue;
    // 2^32 tokens' weights of 2^-32 sum to 1 (bf16 keeps them whole); fp16 values
    // need no such room
    wide = __syncthreads_or(wide) && ELEM == DKV_BF16;
    half_again<ELEM>(sh, c, a, it, q0, nt, wide ? 32.0f : 0.0f);
  }
  __syncthreads();             // every thread has read the word
  if (tid == 0 && atomicAdd(c.status + 3, 1) == (kLook | ((int)gridDim.x - 1))) c.status[3] = 0;
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
                            int window, int sinks, int sm_count, cudaStream_t st) {
  PFN_cuTensorMapEncodeTiled_v12000 enc;
  cudaError_t e = tma_encoder(&enc);
  if (e != cudaSuccess) return e;
  W8Call call;
  call.n_req = n_req;
  call.tok0[0] = call.tile0[0] = 0;
  const int tq = kW8T / c.G;
  for (int i = 0; i < n_req; i++) {
    call.tok0[i + 1] = call.tok0[i] + seq_lens[i];
    call.tile0[i + 1] = call.tile0[i] + (seq_lens[i] + 2 * tq - 1) / (2 * tq);
  }
  const long long n = call.tok0[n_req];
  CUtensorMap mq, mk, mv;
  if ((e = rows_map(enc, elem, q, c.hkv * c.G, n, qs, c.G, tq, &mq)) != cudaSuccess) return e;
  if ((e = rows_map(enc, elem, k, c.hkv, n, ks, 1, kW8T, &mk)) != cudaSuccess) return e;
  if ((e = rows_map(enc, elem, v, c.hkv, n, vs, 1, kW8T, &mv)) != cudaSuccess) return e;
  auto kernel = elem == DKV_F16 ? k_prefill8<DKV_F16> : k_prefill8<DKV_BF16>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kW8Smem);
  if (e != cudaSuccess) return e;
  e = launch_dependent(kernel, dim3(call.tile0[n_req] * c.hkv), dim3(kW8Threads), kW8Smem, st, c, mq, mk, mv,
                       W8Args{static_cast<uint8_t*>(out), window, sinks, tq}, call);
  if (e != cudaSuccess) return e;
  const Again8 again{static_cast<uint8_t*>(out),       static_cast<const uint8_t*>(q), static_cast<const uint8_t*>(k),
                     static_cast<const uint8_t*>(v), 2 * qs, 2 * ks, 2 * vs, W8Args{static_cast<uint8_t*>(out), window, sinks, tq}};
  return launch_dependent(elem == DKV_F16 ? k_prefill8_again<DKV_F16> : k_prefill8_again<DKV_BF16>, dim3(sm_count),
                          dim3(kAgThreads), 0, st, c, again, call);
}

}  // namespace dkv
