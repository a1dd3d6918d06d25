// Internal interface of the 8-bit block-scaled cache (tq_cache8*.cu).
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tq.h"
#include "tq_internal.h"

namespace tq {

// Sequences one launch handles: their prefix sums live in shared memory. Calls
// with more are split into launches over slices of the batch.
constexpr int kC8Slice = 1024;

// Validates a cache descriptor (host); `what` names the entry point.
tq_status check_cache8(const tq_cache8* c, const char* what);
// Validates a block table: stride, and that every token position fits int32.
tq_status check_table8(const tq_cache8* c, int32_t batch, int64_t table_stride, const char* what);

// A stride's check passes where its dimension has one index: it is never used.
inline bool stride_ok(int64_t n, int64_t stride, int64_t unit) { return n <= 1 || (stride >= 0 && stride % unit == 0); }

// Whether rows of d elements at sum i_k * stride_k (i_k < n_k) can overlap: from the smallest stride up, what lies below a
// stride must fit within it. (Strides that interleave without that, 2 d beside 3 d, count as overlapping.)
struct RowDim {
  int64_t n, stride;
};
template <int K>
inline bool rows_overlap(RowDim (&dim)[K], int64_t d) {
  for (int i = 1; i < K; ++i)                        // by stride; a dimension of one index has none that matters
    for (int j = i; j > 0 && dim[j].stride < dim[j - 1].stride; --j) {
      const RowDim x = dim[j];
      dim[j] = dim[j - 1];
      dim[j - 1] = x;
    }
  int64_t extent = d;
  for (const RowDim& x : dim) {
    if (x.n <= 1) continue;
    if (x.stride < extent) return true;
    if (x.n - 1 > (INT64_MAX - extent) / x.stride) return true;
    extent += (x.n - 1) * x.stride;
  }
  return false;
}
inline bool rows_overlap(int64_t ni, int64_t si, int64_t nj, int64_t sj, int64_t d) {
  RowDim dim[2] = {{ni, si}, {nj, sj}};
  return rows_overlap(dim, d);
}

// The driver's tensor-map encoder, looked up once; NULL where the driver lacks it.
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled_fn();

namespace c8 {

// Largest magnitude that takes part in a block's scale; what lies beyond
// (infinities included) is stored as the largest code.
constexpr float kMost = 1.7014118346046923e38f;      // 2^127

// Scale of a block whose largest magnitude is amax <= 2^127: the smallest
// power of two 2^e with amax <= M 2^e, M = 448 = 1.75 * 2^8 (e4m3) or
// 127 = 1.984375 * 2^6 (int8), and e >= -100. From the bits of amax: its
// exponent, and whether its mantissa is above M's.
template <bool INT8>
__device__ __forceinline__ float block_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int E = static_cast<int>(u >> 23) - 127;
  const uint32_t frac = u & 0x7fffffu;
  int e = INT8 ? E - 6 + (frac > 0x7e0000u ? 1 : 0) : E - 8 + (frac > 0x600000u ? 1 : 0);
  e = max(e, -100);                                  // zero and tiny blocks (E = -127) too
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// 1 / scale for a scale that is a power of two in [2^-100, 2^121]: exact.
__device__ __forceinline__ float inv_pow2(float s) {
  return __uint_as_float((254u << 23) - (__float_as_uint(s) & 0x7f800000u));
}

// Code of a value already divided by the scale: nearest, ties to even,
// saturating. NaN has no code of its own and is stored as zero.
template <bool INT8>
__device__ __forceinline__ uint32_t encode(float y) {
  if (!(y == y)) return 0u;
  if (INT8) return static_cast<uint32_t>(__float2int_rn(fminf(fmaxf(y, -127.f), 127.f))) & 0xffu;
  return __nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
}

template <bool INT8>
__device__ __forceinline__ float decode(uint32_t code) {
  if (INT8) return static_cast<float>(static_cast<int8_t>(code));
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3)));
}

// The low / high two e4m3 codes of a word as two halves.
template <bool HI>
__device__ __forceinline__ uint32_t halves_e4m3(uint32_t w) {
  uint32_t r;
  if (HI)
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(w));
  else
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

template <bool INT8>
__device__ __forceinline__ void decode4(uint32_t w, float* v) {
  if (INT8) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = static_cast<float>(static_cast<int8_t>(w >> (8 * k)));
  } else {
    const uint32_t lo = halves_e4m3<false>(w), hi = halves_e4m3<true>(w);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    v[0] = a.x;
    v[1] = a.y;
    v[2] = b.x;
    v[3] = b.y;
  }
}

// Largest b in [0, n) with cum[b] <= u, for cum[0] = 0 <= u < cum[n].
__device__ __forceinline__ int find_seq(const int* cum, int n, int u) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cum[mid] <= u) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// cum[0..n] = exclusive prefix sums of count(b) >= 0, b < n <= kC8Slice, by a CTA of T threads (T a multiple of 32, T <=
// 1024). `part` holds T / 32 ints. Lengths that fall and overlap may add up to any number: sums stay at kMostUnits, so
// that cum never falls and a walk over the units in steps below 2^20 stays within 32 bits.
constexpr int kMostUnits = 0x7fffffff - (1 << 20);
template <int T, typename F>
__device__ __forceinline__ void scan_counts(int* cum, int* part, int n, F count) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  int base = 0;
  for (int at = 0; at < n; at += T) {
    const int b = at + tid;
    uint32_t v = b < n ? count(b) : 0;               // two sums below 2^31 are below 2^32
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = min(v + x, static_cast<uint32_t>(kMostUnits));
    }
    if (lane == 31) part[w] = static_cast<int>(v);
    __syncthreads();
    int64_t before = base, all = base;
    for (int k = 0; k < T / 32; ++k) {
      const int x = part[k];
      if (k < w) before += x;
      all += x;
    }
    if (b < n) cum[b + 1] = static_cast<int>(min(before + v, static_cast<int64_t>(kMostUnits)));
    base = static_cast<int>(min(all, static_cast<int64_t>(kMostUnits)));
    __syncthreads();
  }
  if (tid == 0) cum[0] = 0;
  __syncthreads();
}

}  // namespace c8
}  // namespace tq
