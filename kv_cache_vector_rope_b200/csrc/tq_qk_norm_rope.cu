// tq_qk_norm_rope: RMS norm of every query and key head and the rotate-half
// position rotation, in one pass.
//
// gist.science "TurboESM ..." section 2A: RoPE comes before everything else
// that happens to a key. Models that norm their heads do so before the
// rotation; both act on one head's d values, so one pass reads each value once
// and writes it once:
//   y = x * rsqrt(mean x^2 + eps) * w,
//   (y_i, y_{i+rot/2}) -> (y_i cos a - y_{i+rot/2} sin a, y_i sin a + y_{i+rot/2} cos a),
//   a = pos * base^(-2i/rot), i < rot/2; elements rot .. d-1 are not turned.
//
// A lane holds V consecutive values of a row (16 bytes; 8 in bf16 where the
// alignment is for four only) and the V they are paired with, so no value
// changes lanes. A warp takes rows of one token, several side by side and two
// sets of them in flight: the token's angles are formed once by the warp (fp64
// turns pos * base^(-2i/rot) / 2 pi, whose remainder goes through sincospif:
// far positions lose whole turns only) and then sit in registers, as the
// weights do, while the warp walks the token's heads.
#include "tq_device.cuh"
#include "tq_cache8.h"

namespace tq {
namespace {

struct NormRopeArgs {
  int d, rot;
  int64_t n;
  int hq, hkv;
  const void* q;
  const void* k;
  int64_t q_ts, q_hs, k_ts, k_hs;
  void* qo;
  void* ko;
  int64_t qo_ts, qo_hs, ko_ts, ko_hs;
  const float* qw;
  const float* kw;
  float eps;
  const int32_t* pos;
  double base;
  int32_t* d_status;
  int parts, rows_per_part;                          // a token's rows are dealt to this many warps
};

constexpr int kNrThreads = 256;

// V values as loaded.
template <typename T, int V>
struct Vec;
template <>
struct Vec<float, 4> {
  float4 x;
  __device__ __forceinline__ void load(const float* p) { x = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void get(float* v) const { v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w; }
  static __device__ __forceinline__ void store(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
__device__ __forceinline__ uint32_t two_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
struct Vec<__nv_bfloat16, 4> {
  uint2 x;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { x = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = __uint_as_float(x.x << 16), v[1] = __uint_as_float(x.x & 0xffff0000u);
    v[2] = __uint_as_float(x.y << 16), v[3] = __uint_as_float(x.y & 0xffff0000u);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(two_bf16(v[0], v[1]), two_bf16(v[2], v[3]));
  }
};
template <>
struct Vec<__nv_bfloat16, 8> {
  uint4 x;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { x = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = __uint_as_float(x.x << 16), v[1] = __uint_as_float(x.x & 0xffff0000u);
    v[2] = __uint_as_float(x.y << 16), v[3] = __uint_as_float(x.y & 0xffff0000u);
    v[4] = __uint_as_float(x.z << 16), v[5] = __uint_as_float(x.z & 0xffff0000u);
    v[6] = __uint_as_float(x.w << 16), v[7] = __uint_as_float(x.w & 0xffff0000u);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* v) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(two_bf16(v[0], v[1]), two_bf16(v[2], v[3]), two_bf16(v[4], v[5]), two_bf16(v[6], v[7]));
  }
};

// Rows [r0, r1) of one side (q or k) of a token. LPR: lanes per row, the power
// of two >= d / 2V; a lane's values start at e0 and e1.
template <typename T, int V, int LPR>
__device__ __forceinline__ void side_rows(const T* src, int64_t hs, T* dst, int64_t ohs, int r0, int r1, const float* w,
                                          float eps, float inv_d, int e0, int e1, bool on, bool turned, const float2* cs) {
  constexpr int kRows = 32 / LPR;                    // rows of a warp side by side
  constexpr int kSets = 2;
  const int sub = (threadIdx.x & 31) / LPR;
  float w0[V], w1[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    w0[k] = w && on ? __ldg(w + e0 + k) : 1.f;
    w1[k] = w && on ? __ldg(w + e1 + k) : 1.f;
  }
  for (int r = r0 + sub; r - sub < r1; r += kRows * kSets) {
    Vec<T, V> a[kSets], b[kSets];
#pragma unroll
    for (int s = 0; s < kSets; ++s) {
      const int row = r + s * kRows;
      if (on && row < r1) {
        a[s].load(src + row * hs + e0);
        b[s].load(src + row * hs + e1);
      }
    }
#pragma unroll
    for (int s = 0; s < kSets; ++s) {
      const int row = r + s * kRows;
      const bool live = on && row < r1;
      float x0[V], x1[V];
      if (live) {
        a[s].get(x0);
        b[s].get(x1);
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) x0[k] = x1[k] = 0.f;
      }
      if (w) {
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < V; ++k) ss = fmaf(x0[k], x0[k], fmaf(x1[k], x1[k], ss));
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float f = rsqrtf(ss * inv_d + eps);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          x0[k] *= f * w0[k];
          x1[k] *= f * w1[k];
        }
      }
      if (turned) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float u = x0[k], v = x1[k];
          x0[k] = u * cs[k].x - v * cs[k].y;
          x1[k] = u * cs[k].y + v * cs[k].x;
        }
      }
      if (live) {
        Vec<T, V>::store(dst + row * ohs + e0, x0);
        Vec<T, V>::store(dst + row * ohs + e1, x1);
      }
    }
  }
}

template <typename T, int V, int LPR>
__global__ void __launch_bounds__(kNrThreads) qk_norm_rope_kernel(NormRopeArgs a) {
  __shared__ float2 turn[kNrThreads / 32][128];      // (cos, sin) of pair i of each warp's token
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, part_lane = lane & (LPR - 1);
  const int half = a.rot / 2, pass = (a.d - a.rot) / 2;
  const bool on = part_lane < a.d / (2 * V);
  const bool rope = a.pos != nullptr && half > 0;
  const bool first = V * part_lane < half;           // values that are turned come first
  const int e0 = first ? V * part_lane : a.rot + V * part_lane - half;
  const int e1 = e0 + (first ? half : pass);
  const bool turned = rope && first;
  double freq[4];                                    // turns per position of pairs lane, lane + 32, ...
#pragma unroll
  for (int s = 0; s < 4; ++s)
    freq[s] = rope && lane + 32 * s < half ? pow(a.base, -2.0 * (lane + 32 * s) / a.rot) * 0.15915494309189533577 : 0.0;
  const float inv_d = 1.f / a.d;
  const int64_t units = a.n * a.parts;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + w; u < units;
       u += static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5)) {
    const int64_t tok = a.parts == 1 ? u : u / a.parts;
    const int r0 = static_cast<int>(u - tok * a.parts) * a.rows_per_part, r1 = min(a.hq + a.hkv, r0 + a.rows_per_part);
    float2 cs[V];
    if (rope) {
      const int p = a.pos[tok];
      if (p < 0 && lane == 0 && a.d_status) atomicOr(a.d_status, TQ_DEV_BAD_POSITION);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (32 * s >= half) break;
        const double x = static_cast<double>(p) * freq[s];
        float sn, c;
        sincospif(static_cast<float>(2.0 * (x - rint(x))), &sn, &c);
        turn[w][lane + 32 * s] = make_float2(c, sn);
      }
      __syncwarp();
      if (turned) {
#pragma unroll
        for (int k = 0; k < V; ++k) cs[k] = turn[w][e0 + k];
      }
      __syncwarp();                                  // read before the next token's are written
    }
    if (r0 < a.hq)
      side_rows<T, V, LPR>(static_cast<const T*>(a.q) + tok * a.q_ts, a.q_hs, static_cast<T*>(a.qo) + tok * a.qo_ts,
                           a.qo_hs, r0, min(r1, a.hq), a.qw, a.eps, inv_d, e0, e1, on, turned, cs);
    if (r1 > a.hq)
      side_rows<T, V, LPR>(static_cast<const T*>(a.k) + tok * a.k_ts, a.k_hs, static_cast<T*>(a.ko) + tok * a.ko_ts,
                           a.ko_hs, max(r0 - a.hq, 0), r1 - a.hq, a.kw, a.eps, inv_d, e0, e1, on, turned, cs);
  }
}

template <typename T, int V>
cudaError_t launch_norm_rope(NormRopeArgs a, cudaStream_t st) {
  const int lanes = a.d / (2 * V), rows = a.hq + a.hkv;
  int lpr = 1;
  while (lpr < lanes) lpr *= 2;
  // Warps: one per token, or several where the tokens alone would leave SMs idle
  // (a part has at least as many rows as a warp holds side by side).
  const int side = 32 / lpr, most = (rows + side - 1) / side;
  const int64_t want = (148 * 8 + a.n - 1) / a.n;
  a.parts = static_cast<int>(want < most ? want : most);
  a.rows_per_part = ((rows + a.parts - 1) / a.parts + side - 1) / side * side;
  a.parts = (rows + a.rows_per_part - 1) / a.rows_per_part;
  const int64_t units = a.n * a.parts;
  // Small calls take two warps per CTA, so that they reach every SM.
  const int threads = units <= 148 * 8 ? 64 : kNrThreads;
  const int64_t ctas = (units + threads / 32 - 1) / (threads / 32);
  const unsigned grid = static_cast<unsigned>(ctas < 148 * 8 ? ctas : 148 * 8);
  switch (lpr) {
    case 1: qk_norm_rope_kernel<T, V, 1><<<grid, threads, 0, st>>>(a); break;
    case 2: qk_norm_rope_kernel<T, V, 2><<<grid, threads, 0, st>>>(a); break;
    case 4: qk_norm_rope_kernel<T, V, 4><<<grid, threads, 0, st>>>(a); break;
    case 8: qk_norm_rope_kernel<T, V, 8><<<grid, threads, 0, st>>>(a); break;
    case 16: qk_norm_rope_kernel<T, V, 16><<<grid, threads, 0, st>>>(a); break;
    default: qk_norm_rope_kernel<T, V, 32><<<grid, threads, 0, st>>>(a); break;
  }
  count_launch();
  return cudaGetLastError();
}

}  // namespace
}  // namespace tq

extern "C" tq_status tq_qk_norm_rope(int32_t d, int32_t rot_dim, int64_t n_tokens, int32_t hq, int32_t hkv,
                                     tq_dtype dtype, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                     const void* k, int64_t k_token_stride, int64_t k_head_stride, void* q_out,
                                     int64_t q_out_token_stride, int64_t q_out_head_stride, void* k_out,
                                     int64_t k_out_token_stride, int64_t k_out_head_stride, const float* q_weight,
                                     const float* k_weight, float eps, const int32_t* positions, float rope_base,
                                     int32_t* d_status, void* stream) {
  using namespace tq;
  clear_error();
  if (d < 8 || d > kMaxD || d % 8 != 0)
    return fail(TQ_ERR_INVALID_ARG, "d must be a multiple of 8 in [8, %d] (got %d)", kMaxD, d);
  if (rot_dim < 0 || rot_dim > d || rot_dim % 8 != 0)
    return fail(TQ_ERR_INVALID_ARG, "rot_dim must be a multiple of 8 in [0, d] (got %d)", rot_dim);
  if (n_tokens < 0 || hq < 0 || hkv < 0 || hq > 65536 || hkv > 65536)
    return fail(TQ_ERR_INVALID_ARG, "n_tokens, hq and hkv must not be negative, heads at most 65536");
  if (dtype != TQ_F32 && dtype != TQ_BF16) return fail(TQ_ERR_INVALID_ARG, "dtype must be TQ_F32 or TQ_BF16");
  if (!(eps >= 0.f)) return fail(TQ_ERR_INVALID_ARG, "eps must not be negative");
  const bool rope = positions != nullptr && rot_dim > 0;
  if (rope && !(rope_base > 0.f && rope_base < INFINITY))
    return fail(TQ_ERR_INVALID_ARG, "rope_base must be positive and finite");
  if (n_tokens == 0 || hq + hkv == 0) return TQ_OK;
  const size_t vec = dtype == TQ_F32 ? 16 : 8;       // bytes of the four values a lane loads at once
  struct Side {
    const char* name;
    int heads;
    const void* p;
    int64_t ts, hs;
  } sides[4] = {{"q", hq, q, q_token_stride, q_head_stride},
                {"k", hkv, k, k_token_stride, k_head_stride},
                {"q_out", hq, q_out, q_out_token_stride, q_out_head_stride},
                {"k_out", hkv, k_out, k_out_token_stride, k_out_head_stride}};
  for (const Side& s : sides) {
    if (s.heads == 0) continue;
    if (!s.p) return fail(TQ_ERR_INVALID_ARG, "%s is NULL", s.name);
    if (!aligned(s.p, vec) || !stride_ok(n_tokens, s.ts, 4) || !stride_ok(s.heads, s.hs, 4))
      return fail(TQ_ERR_INVALID_ARG, "%s must be aligned to four elements, base and strides (not negative)", s.name);
  }
  for (int i = 2; i < 4; ++i)
    if (sides[i].heads > 0 && rows_overlap(n_tokens, sides[i].ts, sides[i].heads, sides[i].hs, d))
      return fail(TQ_ERR_INVALID_ARG, "%s: its strides make rows overlap", sides[i].name);
  if ((q_weight && !aligned(q_weight, 16)) || (k_weight && !aligned(k_weight, 16)))
    return fail(TQ_ERR_INVALID_ARG, "weights must be 16-byte aligned");
  NormRopeArgs a{d, rot_dim, n_tokens, hq, hkv, q, k, q_token_stride, q_head_stride, k_token_stride, k_head_stride,
                 q_out, k_out, q_out_token_stride, q_out_head_stride, k_out_token_stride, k_out_head_stride, q_weight,
                 k_weight, eps, rope ? positions : nullptr, static_cast<double>(rope_base), d_status, 0, 0};
  // bf16 rows go eight values at a time where bases, strides and halves allow it.
  bool eight = dtype == TQ_BF16 && d % 16 == 0 && rot_dim % 16 == 0;
  for (const Side& s : sides)
    if (s.heads > 0)
      eight = eight && aligned(s.p, 16) && (n_tokens == 1 || s.ts % 8 == 0) && (s.heads == 1 || s.hs % 8 == 0);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == TQ_F32 ? launch_norm_rope<float, 4>(a, st)
                        : eight         ? launch_norm_rope<__nv_bfloat16, 8>(a, st)
                                        : launch_norm_rope<__nv_bfloat16, 4>(a, st);
  if (e != cudaSuccess) return fail(TQ_ERR_CUDA, "tq_qk_norm_rope launch: %s", cudaGetErrorString(e));
  return TQ_OK;
}
