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
// A lane holds four values of a row and the four they are paired with, so no
// value changes lanes; a row takes d / 8 lanes (rounded up to a power of two)
// and its sum of squares a few shuffles. The angle is formed in fp64 as turns
// (pos * base^(-2i/rot) / 2 pi; far positions lose whole turns only) and its
// remainder goes through sincospif; one set per token serves all heads.
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
  int rows_per_cta;                                  // rows (heads) of a token one CTA takes
};

constexpr int kNrThreads = 256;
constexpr int kNrTile = 4;                           // tokens whose angles are formed together

struct F4 {
  float v[4];
};
__device__ __forceinline__ F4 load4(const float* p) {
  const float4 x = *reinterpret_cast<const float4*>(p);
  return {{x.x, x.y, x.z, x.w}};
}
__device__ __forceinline__ F4 load4(const __nv_bfloat16* p) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  return {{__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u), __uint_as_float(x.y << 16),
           __uint_as_float(x.y & 0xffff0000u)}};
}
__device__ __forceinline__ void store4(float* p, const F4& x) {
  *reinterpret_cast<float4*>(p) = make_float4(x.v[0], x.v[1], x.v[2], x.v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const F4& x) {
  __nv_bfloat162 a = __floats2bfloat162_rn(x.v[0], x.v[1]), b = __floats2bfloat162_rn(x.v[2], x.v[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}

// LPR: lanes per row, the power of two >= d / 8.
template <typename T, int LPR>
__global__ void __launch_bounds__(kNrThreads) qk_norm_rope_kernel(NormRopeArgs a) {
  __shared__ float2 turn[kNrTile][128];              // (cos, sin) of pair i of each token of the tile
  const int tid = threadIdx.x;
  const int half = a.rot / 2, pass = (a.d - a.rot) / 2;
  const int rows = a.hq + a.hkv;
  const int r0 = blockIdx.y * a.rows_per_cta, r1 = min(rows, r0 + a.rows_per_cta);
  const bool rope = a.pos != nullptr && half > 0;
  // Thread i forms pair i % 128 of token i / 128 (+2, ...) of a tile.
  const int pair = tid & 127;
  const double freq = rope && pair < half ? pow(a.base, -2.0 * pair / a.rot) * 0.15915494309189533577 : 0.0;
  const int lane = tid & (LPR - 1), slot = tid / LPR;
  constexpr int kSlots = kNrThreads / LPR;
  const bool on = lane < a.d / 8;
  const bool turned = 4 * lane < half;
  const int e0 = turned ? 4 * lane : a.rot + 4 * lane - half;
  const int e1 = e0 + (turned ? half : pass);
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kNrTile; t0 < a.n;
       t0 += static_cast<int64_t>(gridDim.x) * kNrTile) {
    const int nt = static_cast<int>(min(static_cast<int64_t>(kNrTile), a.n - t0));
    if (rope && pair < half) {
      for (int t = tid >> 7; t < nt; t += kNrThreads / 128) {
        const int p = a.pos[t0 + t];
        if (p < 0 && pair == 0 && a.d_status) atomicOr(a.d_status, TQ_DEV_BAD_POSITION);
        const double x = static_cast<double>(p) * freq;
        float s, c;
        sincospif(static_cast<float>(2.0 * (x - rint(x))), &s, &c);
        turn[t][pair] = make_float2(c, s);
      }
    }
    __syncthreads();
    const int count = nt * (r1 - r0);
    for (int at = slot; at - slot < count; at += kSlots) {      // whole warps stay together for the shuffles
      const bool live = at < count && on;
      const int t = at < count ? at / (r1 - r0) : 0;
      const int r = at < count ? r0 + at % (r1 - r0) : r0;
      const bool is_q = r < a.hq;
      const int h = is_q ? r : r - a.hq;
      const int64_t tok = t0 + t;
      const T* src = static_cast<const T*>(is_q ? a.q : a.k) +
                     (is_q ? tok * a.q_ts + h * a.q_hs : tok * a.k_ts + h * a.k_hs);
      const float* w = is_q ? a.qw : a.kw;
      F4 x0{{0.f, 0.f, 0.f, 0.f}}, x1 = x0;
      if (live) {
        x0 = load4(src + e0);
        x1 = load4(src + e1);
      }
      if (w != nullptr || LPR < 32) {
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) ss = fmaf(x0.v[k], x0.v[k], fmaf(x1.v[k], x1.v[k], ss));
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (w != nullptr && live) {
          const float f = rsqrtf(ss / a.d + a.eps);
          const float4 w0 = __ldg(reinterpret_cast<const float4*>(w + e0));
          const float4 w1 = __ldg(reinterpret_cast<const float4*>(w + e1));
          x0 = {{x0.v[0] * f * w0.x, x0.v[1] * f * w0.y, x0.v[2] * f * w0.z, x0.v[3] * f * w0.w}};
          x1 = {{x1.v[0] * f * w1.x, x1.v[1] * f * w1.y, x1.v[2] * f * w1.z, x1.v[3] * f * w1.w}};
        }
      }
      if (!live) continue;
      if (rope && turned) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 cs = turn[t][e0 + k];
          const float u = x0.v[k], v = x1.v[k];
          x0.v[k] = u * cs.x - v * cs.y;
          x1.v[k] = u * cs.y + v * cs.x;
        }
      }
      T* dst = static_cast<T*>(is_q ? a.qo : a.ko) +
               (is_q ? tok * a.qo_ts + h * a.qo_hs : tok * a.ko_ts + h * a.ko_hs);
      store4(dst + e0, x0);
      store4(dst + e1, x1);
    }
    __syncthreads();                                 // the tile's angles are read
  }
}

template <typename T>
cudaError_t launch_norm_rope(const NormRopeArgs& a, dim3 grid, cudaStream_t st) {
  const int lanes = a.d / 8;
  if (lanes <= 1) qk_norm_rope_kernel<T, 1><<<grid, kNrThreads, 0, st>>>(a);
  else if (lanes <= 2) qk_norm_rope_kernel<T, 2><<<grid, kNrThreads, 0, st>>>(a);
  else if (lanes <= 4) qk_norm_rope_kernel<T, 4><<<grid, kNrThreads, 0, st>>>(a);
  else if (lanes <= 8) qk_norm_rope_kernel<T, 8><<<grid, kNrThreads, 0, st>>>(a);
  else if (lanes <= 16) qk_norm_rope_kernel<T, 16><<<grid, kNrThreads, 0, st>>>(a);
  else qk_norm_rope_kernel<T, 32><<<grid, kNrThreads, 0, st>>>(a);
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
                 k_weight, eps, rope ? positions : nullptr, static_cast<double>(rope_base), d_status, 0};
  const int rows = hq + hkv;
  const int64_t tiles = (n_tokens + kNrTile - 1) / kNrTile;
  const int64_t most = 148 * 8;
  const unsigned gx = static_cast<unsigned>(tiles < most ? tiles : most);
  // Few tokens: the heads of a token are spread over CTAs too.
  int parts = 1;
  while (parts < rows && parts < 64 && static_cast<int64_t>(gx) * parts < 148 && (rows + parts - 1) / parts > 4)
    parts *= 2;
  a.rows_per_cta = (rows + parts - 1) / parts;
  dim3 grid(gx, static_cast<unsigned>((rows + a.rows_per_cta - 1) / a.rows_per_cta));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == TQ_F32 ? launch_norm_rope<float>(a, grid, st) : launch_norm_rope<__nv_bfloat16>(a, grid, st);
  if (e != cudaSuccess) return fail(TQ_ERR_CUDA, "tq_qk_norm_rope launch: %s", cudaGetErrorString(e));
  return TQ_OK;
}
