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
// A lane holds four consecutive values of a row and the four they are paired
// with, so no value changes lanes. A warp takes the rows of one token, several
// side by side and several sets of them in flight: the token's angles are formed
// once by the warp (fp64 turns pos * base^(-2i/rot) / 2 pi, whose remainder goes
// through sincospif: far positions lose whole turns only) and stay in registers
// as products with the weights while the warp walks the token's heads.
//
// Bound by memory: 16384 tokens of 40 bf16 heads of 128 64.9 us (51.3 at the
// copy's rate; more CTAs per SM 72 to 91 us), 1021
// tokens of 40 fp32 heads of 64 6.0 us (3.2), 8 tokens 2.9 us, which is launch,
// one load, the angles and one store, each waiting for the last.
#include <cmath>

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
  int64_t q_ts, k_ts;
  int q_hs, k_hs;                                    // a token's heads lie within 2^31 elements
  void* qo;
  void* ko;
  int64_t qo_ts, ko_ts;
  int qo_hs, ko_hs;
  const float* qw;
  const float* kw;
  float eps;
  const int32_t* pos;
  double log2_base;
  int32_t* d_status;
  int parts, rows_per_part;                          // a token's rows are dealt to this many warps
};

constexpr int kNrThreads = 256, kNrCtas = 3;         // resident CTAs per SM

// Four values as loaded.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  float4 x;
  __device__ __forceinline__ void load(const float* p) { x = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void get(float2 (&v)[2]) const { v[0] = make_float2(x.x, x.y), v[1] = make_float2(x.z, x.w); }
  static __device__ __forceinline__ void store(float* p, const float2 (&v)[2]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  uint2 x;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { x = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void get(float2 (&v)[2]) const {
    v[0] = make_float2(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u));
    v[1] = make_float2(__uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u));
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float2 (&v)[2]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0].x, v[0].y), b = __floats2bfloat162_rn(v[1].x, v[1].y);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
};

// Two fp32 products (sums) per instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return r;
}

// Rows [r0, r1) of one side (q or k) of a token. LPR: lanes per row, the power
// of two >= d / 8; a lane's values start at e0 and e1. With w0, w1 the weights
// and (c, s) the angle of a pair (u, v) and f the row's norm factor:
//   f (u w0 c - v w1 s),  f (u w0 s + v w1 c),
// and f u w0, f v w1 where the pair is not turned: not by an angle of 0, whose sine would carry an infinity or NaN of one
// into the other.
template <typename T, int LPR>
__device__ __forceinline__ void side_rows(const T* src, int hs, T* dst, int ohs, int r0, int r1, const float* w,
                                          float eps, float inv_d, int e0, int e1, bool on, bool turned, const float2 (&c)[2],
                                          const float2 (&sn)[2]) {
  constexpr int kRows = 32 / LPR;                    // rows of a warp side by side
  // bf16: two sets of rows while the next two are on their way; fp32, with twice the registers a set: four at once.
  // (A prompt of 16384 tokens, 40 heads of 128: bf16 64.2 us against 68.3 with four at once; 8192 fp32 ones 64 us against
  // 72 with two ahead.)
  constexpr bool kAhead = sizeof(T) == 2;
  constexpr int kSets = kAhead ? 2 : 4;
  const int sub = (threadIdx.x & 31) / LPR;
  float2 uc[2], vs[2], us[2], vc[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float2 w0 = make_float2(1.f, 1.f), w1 = w0;
    if (w && on) {
      w0 = __ldg(reinterpret_cast<const float2*>(w + e0) + k);
      w1 = __ldg(reinterpret_cast<const float2*>(w + e1) + k);
    }
    uc[k] = mul2(w0, c[k]);
    us[k] = mul2(w0, sn[k]);
    vc[k] = mul2(w1, c[k]);
    vs[k] = mul2(w1, make_float2(-sn[k].x, -sn[k].y));
  }
  src += e0;
  dst += e0;
  const int gap = e1 - e0;
  Vec<T> na[kSets], nb[kSets];
  const auto load = [&](int r) {
#pragma unroll
    for (int s = 0; s < kSets; ++s) {
      const int row = r + s * kRows;
      if (on && row < r1) {
        const T* p = src + row * hs;
        na[s].load(p);
        nb[s].load(p + gap);
      }
    }
  };
  if (kAhead) load(r0 + sub);
#pragma unroll 1
  for (int r = r0 + sub; r - sub < r1; r += kRows * kSets) {
    if (!kAhead) load(r);
    Vec<T> a[kSets], b[kSets];
#pragma unroll
    for (int s = 0; s < kSets; ++s) {
      a[s] = na[s];
      b[s] = nb[s];
    }
    if (kAhead) load(r + kRows * kSets);
#pragma unroll
    for (int s = 0; s < kSets; ++s) {
      const int row = r + s * kRows;
      const bool live = on && row < r1;
      float2 u[2], v[2];
      if (live) {
        a[s].get(u);
        b[s].get(v);
      } else {
        u[0] = u[1] = v[0] = v[1] = make_float2(0.f, 0.f);
      }
      float f = 1.f;
      if (w) {
        const float2 s2 = fma2(u[0], u[0], fma2(u[1], u[1], fma2(v[0], v[0], mul2(v[1], v[1]))));
        float ss = s2.x + s2.y;
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        f = rsqrtf(ss * inv_d + eps);
      }
      if (live) {
        const float2 ff = make_float2(f, f);
        float2 y0[2], y1[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          y0[k] = turned ? fma2(u[k], uc[k], mul2(v[k], vs[k])) : mul2(u[k], uc[k]);
          y1[k] = turned ? fma2(u[k], us[k], mul2(v[k], vc[k])) : mul2(v[k], vc[k]);
          y0[k] = mul2(ff, y0[k]);
          y1[k] = mul2(ff, y1[k]);
        }
        T* p = dst + row * ohs;
        Vec<T>::store(p, y0);
        Vec<T>::store(p + gap, y1);
      }
    }
  }
}

template <typename T, int LPR>
__global__ void __launch_bounds__(kNrThreads, kNrCtas) qk_norm_rope_kernel(NormRopeArgs a) {
  __shared__ float2 turn[kNrThreads / 32][128];      // (cos, sin) of pair i of each warp's token
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, part_lane = lane & (LPR - 1);
  const int half = a.rot / 2, pass = (a.d - a.rot) / 2;
  const bool on = part_lane < a.d / 8;
  const bool rope = a.pos != nullptr && half > 0;
  const bool first = 4 * part_lane < half;           // values that are turned come first
  const int e0 = first ? 4 * part_lane : a.rot + 4 * part_lane - half;
  const int e1 = e0 + (first ? half : pass);
  const bool turned = rope && first;
  __shared__ double freq[128];                       // turns per position of each pair
  for (int i = threadIdx.x; rope && i < half; i += blockDim.x)
    freq[i] = exp2(-2.0 * i / a.rot * a.log2_base) * 0.15915494309189533577;
  __syncthreads();
  const float inv_d = 1.f / a.d;
  const int64_t units = a.n * a.parts;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + w; u < units;
       u += static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5)) {
    const int64_t tok = a.parts == 1 ? u : u / a.parts;
    const int r0 = static_cast<int>(u - tok * a.parts) * a.rows_per_part, r1 = min(a.hq + a.hkv, r0 + a.rows_per_part);
    float2 c[2] = {make_float2(1.f, 1.f), make_float2(1.f, 1.f)}, sn[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    if (rope) {
      const int p = a.pos[tok];
      if (p < 0 && lane == 0 && a.d_status) atomicOr(a.d_status, TQ_DEV_BAD_POSITION);
#pragma unroll 1
      for (int i = lane; i < half; i += 32) {
        const double x = static_cast<double>(p) * freq[i];
        float2 y;
        sincospif(static_cast<float>(2.0 * (x - rint(x))), &y.y, &y.x);
        turn[w][i] = y;
      }
      __syncwarp();
      if (turned) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 x = turn[w][e0 + 2 * k], y = turn[w][e0 + 2 * k + 1];
          c[k] = make_float2(x.x, y.x);
          sn[k] = make_float2(x.y, y.y);
        }
      }
      __syncwarp();                                  // read before the next token's are written
    }
    if (r0 < a.hq)
      side_rows<T, LPR>(static_cast<const T*>(a.q) + tok * a.q_ts, a.q_hs, static_cast<T*>(a.qo) + tok * a.qo_ts,
                           a.qo_hs, r0, min(r1, a.hq), a.qw, a.eps, inv_d, e0, e1, on, turned, c, sn);
    if (r1 > a.hq)
      side_rows<T, LPR>(static_cast<const T*>(a.k) + tok * a.k_ts, a.k_hs, static_cast<T*>(a.ko) + tok * a.ko_ts,
                           a.ko_hs, max(r0 - a.hq, 0), r1 - a.hq, a.kw, a.eps, inv_d, e0, e1, on, turned, c, sn);
  }
}

template <typename T>
cudaError_t launch_norm_rope(NormRopeArgs a, cudaStream_t st) {
  const int lanes = a.d / 8, rows = a.hq + a.hkv;
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
  const int cap = 148 * (threads == kNrThreads ? kNrCtas : 16);   // as many as are resident at once
  const unsigned grid = static_cast<unsigned>(ctas < cap ? ctas : cap);
  switch (lpr) {
    case 1: qk_norm_rope_kernel<T, 1><<<grid, threads, 0, st>>>(a); break;
    case 2: qk_norm_rope_kernel<T, 2><<<grid, threads, 0, st>>>(a); break;
    case 4: qk_norm_rope_kernel<T, 4><<<grid, threads, 0, st>>>(a); break;
    case 8: qk_norm_rope_kernel<T, 8><<<grid, threads, 0, st>>>(a); break;
    case 16: qk_norm_rope_kernel<T, 16><<<grid, threads, 0, st>>>(a); break;
    default: qk_norm_rope_kernel<T, 32><<<grid, threads, 0, st>>>(a); break;
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
  for (Side& s : sides) {
    if (s.heads <= 1) s.hs = 0;                      // never used
    if (s.heads > 1 && s.hs > 0x7fffffff / s.heads)
      return fail(TQ_ERR_UNSUPPORTED, "%s: the heads of a token span 2^31 elements or more", s.name);
  }
  for (int i = 2; i < 4; ++i)
    if (sides[i].heads > 0 && rows_overlap(n_tokens, sides[i].ts, sides[i].heads, sides[i].hs, d))
      return fail(TQ_ERR_INVALID_ARG, "%s: its strides make rows overlap", sides[i].name);
  if ((q_weight && !aligned(q_weight, 16)) || (k_weight && !aligned(k_weight, 16)))
    return fail(TQ_ERR_INVALID_ARG, "weights must be 16-byte aligned");
  const auto head_stride = [&](int i) { return static_cast<int>(sides[i].hs); };
  NormRopeArgs a{d, rot_dim, n_tokens, hq, hkv, q, k, q_token_stride, k_token_stride, head_stride(0), head_stride(1),
                 q_out, k_out, q_out_token_stride, k_out_token_stride, head_stride(2), head_stride(3), q_weight,
                 k_weight, eps, rope ? positions : nullptr, rope ? std::log2(static_cast<double>(rope_base)) : 0.0, d_status, 0, 0};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == TQ_F32 ? launch_norm_rope<float>(a, st) : launch_norm_rope<__nv_bfloat16>(a, st);
  if (e != cudaSuccess) return fail(TQ_ERR_CUDA, "tq_qk_norm_rope launch: %s", cudaGetErrorString(e));
  return TQ_OK;
}
