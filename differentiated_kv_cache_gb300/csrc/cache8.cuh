// cache8.cuh — shared definitions of the uniform 8-bit cache (include/dkv.h):
// element and code types, the stored tile order, the device view of a
// descriptor.
#pragma once

#include <cuda_bf16.h>

#include "dkv_common.cuh"

namespace dkv {

constexpr int kSub = 16;            // tokens of one stored tile
constexpr int kTile = kSub * kD;    // entries of K or V in a tile
constexpr int kMaxSlots = 1 << 18;
// smallest block scale: keeps 1 / s and products of scales finite in fp32
constexpr float kScaleFloor = 7.888609052210118e-31f;   // 2^-100
constexpr float kLogitScale = 1.4426950408889634f * 0.08838834764831845f;   // log2(e) / sqrt(128)

// Device view of a dkv_cache8.
struct Cache8View {
  uint8_t* pages;
  float* scales;
  uint8_t* tail;
  const int* table;
  int* status;
  int hkv, G, T, n_pages, n_slots, width, rot, inter;

  // bytes of one (page, head) and of one (slot, head)
  __device__ __forceinline__ size_t page_head(int page, int h) const {
    return ((size_t)page * hkv + h) * ((size_t)T * 2 * kD);
  }
  __device__ __forceinline__ size_t tail_head(int slot, int h) const {
    return ((size_t)slot * hkv + h) * ((size_t)T * 4 * kD);
  }
  // an error of an earlier call; the same for every thread of the block,
  // whatever other blocks latch meanwhile
  __device__ __forceinline__ bool stopped() const {
    return __syncthreads_or(threadIdx.x == 0 && *(volatile int*)status != 0);
  }
  __device__ __forceinline__ void latch(int code, int info) const {
    if (atomicCAS(status, 0, code) == 0) status[1] = info;
  }
};

// Entry of a tile (include/dkv.h): (r, c, m) = (token, feature % 16,
// feature / 16) for K, (feature % 16, token, feature / 16) for V.
__host__ __device__ __forceinline__ int tile16(int r, int c, int m) {
  return 256 * m + 8 * (4 * (r & 7) + ((c & 7) >> 1)) + 4 * (r >> 3) + 2 * (c >> 3) + (c & 1);
}

template <int ELEM>
__device__ __forceinline__ float elem_float(uint16_t b) {
  return ELEM == DKV_F16 ? __half2float(__ushort_as_half(b)) : __uint_as_float((uint32_t)b << 16);
}
template <int ELEM>
__device__ __forceinline__ uint16_t float_elem(float x) {
  return ELEM == DKV_F16 ? __half_as_ushort(__float2half_rn(x)) : __bfloat16_as_ushort(__float2bfloat16_rn(x));
}
// two values, the first in the lower half
template <int ELEM>
__device__ __forceinline__ uint32_t pack_elems(float a, float b) {
  if (ELEM == DKV_F16) return pack_half2(a, b);
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// A mean of values of the type whose weights were rounded on the way can come out
// just above the type's largest: that largest value, unless it is infinite.
template <int ELEM>
__device__ __forceinline__ float in_range(float x) {
  const float top = ELEM == DKV_F16 ? 65504.0f : 3.3895313892515355e38f;
  return fabsf(x) < INFINITY ? fminf(fmaxf(x, -top), top) : x;
}
// acc + 0 * x: NaN from the first infinite or NaN value on (never in the sign).
template <int ELEM>
__device__ __forceinline__ void find_not_finite(uint32_t& acc, uint32_t x) {
  if (ELEM == DKV_F16) asm("fma.rn.f16x2 %0, %1, %2, %0;\n" : "+r"(acc) : "r"(x), "r"(0u));
  else asm("fma.rn.bf16x2 %0, %1, %2, %0;\n" : "+r"(acc) : "r"(x), "r"(0u));
}
__device__ __forceinline__ bool found_not_finite(uint32_t acc) { return (acc & 0x7fff7fffu) != 0; }
template <int ELEM>
__device__ __forceinline__ float lo_elem(uint32_t w) { return elem_float<ELEM>((uint16_t)(w & 0xffffu)); }
template <int ELEM>
__device__ __forceinline__ float hi_elem(uint32_t w) { return elem_float<ELEM>((uint16_t)(w >> 16)); }

// c += a b, 16 x 16 by 16 x 8 (mma.sync), fp32 sums
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

// largest finite |x| so far
__device__ __forceinline__ float amax_finite(float m, float x) {
  const float a = fabsf(x);
  return a < INFINITY ? fmaxf(m, a) : m;      // false for infinities and NaN
}

// amax times the fp32 nearest 1 / Q (a code can then exceed Q by a rounding:
// code_pair clamps it)
__device__ __forceinline__ float block_scale(float amax, int code_type) {
  return fmaxf(__fmul_rn(amax, code_type == DKV_E4M3 ? 1.0f / 448.0f : 1.0f / 127.0f), kScaleFloor);
}

// Codes of two values (the first in the lower byte; FINITE leaves the upper half
// undefined). FINITE: neither is infinite or NaN, and |x inv| exceeds Q by a
// rounding at most.
template <int CODE, bool FINITE>
__device__ __forceinline__ uint32_t code_pair(float a, float b, float inv) {
  a = __fmul_rn(a, inv);
  b = __fmul_rn(b, inv);
  if (CODE == DKV_E4M3) {
    uint16_t r;   // round to nearest even, saturating; NaN stays NaN
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(b), "f"(a));
    return r;
  }
  if (FINITE) {   // the sum's ulp is 1: rounds to nearest even, the low byte is the code
    const float big = 12582912.0f;
    return prmt(__float_as_uint(__fadd_rn(a, big)), __float_as_uint(__fadd_rn(b, big)), 0x0040u);
  }
  // NaN gives 0
  const int x = a == a ? (int)rintf(fminf(fmaxf(a, -127.0f), 127.0f)) : 0;
  const int y = b == b ? (int)rintf(fminf(fmaxf(b, -127.0f), 127.0f)) : 0;
  return (uint32_t)(x & 0xff) | ((uint32_t)(y & 0xff) << 8);
}

struct Append8Args {
  const uint8_t *k, *v, *q;
  long long ks, vs, qs;      // row strides in bytes
  const float2* rope;
  int rope_len;
  uint8_t *k_rot, *q_rot;
  const int *slots, *before;
};

cudaError_t launch_append8(const Cache8View& c, int elem, int code, const Append8Args& a, int n_req,
                           const int32_t* n_new, cudaStream_t st);
cudaError_t launch_attention8(const Cache8View& c, int elem, int code, int sm_count, const int* slots,
                              const int* seq_lens, int n_req, const void* q, long long q_stride, void* out,
                              int window, int sinks, void* workspace, cudaStream_t st);
size_t attention8_workspace(int hkv, int G, int max_req, int sm_count);
cudaError_t launch_prefill8(const Cache8View& c, int elem, const int32_t* seq_lens, int n_req, const void* q,
                            long long qs, const void* k, long long ks, const void* v, long long vs, void* out,
                            int window, int sinks, int sm_count, cudaStream_t st);

}  // namespace dkv
