// tq_cache8_attention: attention of the newest queries of each sequence over
// an 8-bit paged cache (tq_cache8_write's layout).
//
// For query row i of nq, at position len - nq + i, and the KV head its query
// head belongs to:
//   s_t = scale * k_scale[page(t)] * <q, kcode_t>,  p_t = e^(s_t - m),
//   out = sum_t p_t v_scale[page(t)] vcode_t / sum_t p_t,   lse = m + ln sum_t p_t.
// gist.science "TurboESM ..." section 2E: one pass over the packed cache with a
// running maximum and sum, no dequantised intermediate in memory.
//
// A decode step is bound by the cache's bytes (2 d per key and KV head), so the
// work is cut along the keys: all (sequence, KV head, row tile, 64-key tile)
// units in that order are dealt in equal contiguous ranges to the CTAs, however
// long or ragged the sequences are. A range that ends inside a sequence leaves
// a partial record (m, l, sum) that cache8_combine_kernel merges; a CTA writes
// at most two of them.
//
// Each warp takes groups of 16 keys of its CTA's range and keeps its own
// running (m, l, sum). The products run on 16x8x16 half-precision matrix
// instructions with the keys (then the value coordinates) as the 16 rows and
// eight query rows as the columns, which suits the few rows of a step: every
// 8-bit code is exactly a half, and a query row is scaled by a power of two
// into half's range (exact for bf16; fp32 queries and fp32 outputs use two
// half limbs for q and for p). The contraction index of both products is
// permuted so that a lane's operands are 16 contiguous bytes of the cache.
#include <cuda.h>

#include "tq_cache8.h"
#include "tq_device.cuh"

namespace tq {
namespace {

using namespace c8;

constexpr int kAtThreads = 256;
constexpr int kAtWarps = kAtThreads / 32;
constexpr int kAtGrid = 148 * 2;                     // two CTAs per SM
constexpr int kUnit = 64;                            // keys per unit of the split
constexpr int kMinUnits = 2;                         // a CTA takes at least this many units
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Weights are kept as 2^(s - m + kLift): halves hold them to 2^-24, and the
// running maximum m is moved only when a score exceeds it by kSlack octaves.
constexpr float kLift = 6.f;
constexpr float kSlack = 8.f;

struct AttnArgs {
  int heads, block, batch;
  int64_t n_blocks;
  const uint8_t* k;
  const uint8_t* v;
  const float* ks;
  const float* vs;
  const void* q;
  int64_t q_bs, q_hs, q_rs;
  int group, nq, rows;                               // rows = group * nq per KV head
  int row_tiles;
  const int32_t* lens;                               // of this slice
  const int32_t* table;
  int64_t table_stride;
  int64_t first_seq;
  int causal;
  int window;
  float scale2;                                      // softmax scale * log2 e
  void* out;
  int64_t o_bs, o_hs, o_rs;
  float* lse;                                        // [batch][hq][nq] or NULL
  float* rec;                                        // [grid][2][rows of a tile][2 + d]
  int* cum_out;                                      // [batch + 1], for the combine kernel
  int32_t* d_status;
};

__device__ __forceinline__ int seq_len(const AttnArgs& a, int b, bool tell) {
  const int64_t n = a.lens[b], cap = a.table_stride * a.block;
  if (n < 0 || n > cap) {
    if (tell && a.d_status) atomicOr(a.d_status, TQ_DEV_BAD_LENGTH);
    return n < 0 ? 0 : static_cast<int>(cap);
  }
  return static_cast<int>(n);
}
// First key any row of the sequence sees.
__device__ __forceinline__ int seq_first(const AttnArgs& a, int n) {
  return a.window > 0 ? max(0, n - a.nq + 1 - a.window) : 0;
}
__device__ __forceinline__ int seq_tiles(const AttnArgs& a, int n) {
  return n == 0 ? 0 : (n + kUnit - 1) / kUnit - seq_first(a, n) / kUnit;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The low / high two codes of a word as two halves.
template <bool INT8, bool HI>
__device__ __forceinline__ uint32_t two_halves(uint32_t w) {
  if (INT8) {
    // 0x64uu is 1024 + u; u = code + 128.
    const uint32_t x = __byte_perm(w ^ 0x80808080u, 0x64646464u, HI ? 0x4342 : 0x4140);
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&x), __floats2half2_rn(1152.f, 1152.f));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(HI ? w >> 16 : w & 0xffffu), __NV_E4M3);
  return static_cast<uint32_t>(h.x) | static_cast<uint32_t>(h.y) << 16;
}

template <int D>
struct Chunk;                                        // bytes a lane loads of one key / value row
template <>
struct Chunk<64> {
  static constexpr int kK = 1, kVWords = 2;
};
template <>
struct Chunk<128> {
  static constexpr int kK = 2, kVWords = 4;
};
template <>
struct Chunk<256> {
  static constexpr int kK = 4, kVWords = 8;
};

// One (sequence, KV head, row tile, key range) of a CTA's range.
struct Seg {
  int b, kv, rt, n, t0, t1;                          // keys [t0, t1)
  bool whole;                                        // all keys of the stream
  bool head;                                         // the stream's first keys
};

__device__ __forceinline__ Seg seg_at(const AttnArgs& a, const int* cum, int u, int uend, int* next) {
  Seg s;
  s.b = find_seq(cum, a.batch, u);
  s.n = seq_len(a, s.b, false);
  const int tiles = seq_tiles(a, s.n), rel = u - cum[s.b];
  const int stream = rel / tiles, tile0 = rel % tiles;
  s.kv = stream / a.row_tiles;
  s.rt = stream % a.row_tiles;
  const int nt = min(tiles - tile0, uend - u);
  const int first = seq_first(a, s.n);
  s.t0 = (first / kUnit + tile0) * kUnit;
  s.t1 = min(s.t0 + nt * kUnit, s.n);
  if (tile0 == 0) s.t0 = first / 16 * 16;
  s.head = tile0 == 0;
  s.whole = nt == tiles;
  *next = u + nt;
  return s;
}

__device__ __forceinline__ int64_t page_of(const AttnArgs& a, int b, int blk) {
  return a.table ? static_cast<int64_t>(a.table[b * a.table_stride + blk]) : (a.first_seq + b) * a.table_stride + blk;
}

__device__ __forceinline__ float load_q(const void* p, bool f32, int64_t i) {
  return f32 ? reinterpret_cast<const float*>(p)[i] : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}

// NT: eight-row query tiles a CTA handles together. QF / OF: fp32 queries /
// outputs, two half limbs each.
template <int D, bool INT8, int NT, bool QF, bool OF>
__global__ void __launch_bounds__(kAtThreads, 2) cache8_attn_kernel(AttnArgs a) {
  constexpr int KC = Chunk<D>::kK, KS = KC * 4;      // 16-byte chunks, k-steps of the score product
  constexpr int VW = Chunk<D>::kVWords, MT = VW * 2; // words per value row of a lane, 16-row tiles of the value product
  constexpr int QL = QF ? 2 : 1;
  constexpr int kRows = 8 * NT;
  __shared__ int cum[kC8Slice + 1];
  __shared__ int part[kAtWarps];
  __shared__ float sm_m[kAtWarps][kRows], sm_l[kAtWarps][kRows];
  __shared__ float4 sm_acc[kAtWarps][4][32];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  scan_counts<kAtThreads>(cum, part, a.batch, [&](int b) {
    return seq_tiles(a, seq_len(a, b, blockIdx.x == 0)) * a.heads * a.row_tiles;
  });
  if (blockIdx.x == 0)
    for (int b = tid; b <= a.batch; b += kAtThreads) a.cum_out[b] = cum[b];
  const int total = cum[a.batch];
  const int per = max((total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x), kMinUnits);
  const int u0 = min(static_cast<int>(blockIdx.x) * per, total), u1 = min(u0 + per, total);
  for (int u = u0; u < u1;) {
    int next;
    const Seg sg = seg_at(a, cum, u, u1, &next);
    // Queries: lane (g, t) holds row g's coordinates of its chunks.
    uint32_t qh[NT][KS][QL][2];
    float cq[NT][2];
    int lo[NT][2], hi[NT][2];
    int lo_max = 0, hi_min = 0x7fffffff;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = sg.rt * kRows + nt * 8 + g;
      const bool live = r < a.rows;
      const int i = live ? r / a.group : 0, hq = sg.kv * a.group + (live ? r % a.group : 0);
      const int64_t base = (a.first_seq + sg.b) * a.q_bs + hq * a.q_hs + i * a.q_rs;
      float amax = 0.f;
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          amax = fmaxf(amax, live ? fabsf(load_q(a.q, QF, base + 16 * (t + 4 * c) + e)) : 0.f);
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // Times a power of two: the largest coordinate lands in [2^14, 2^15).
      const int E = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -100);
      const float up = __uint_as_float(static_cast<uint32_t>(14 - min(E, 127) + 127) << 23);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[e] = live ? load_q(a.q, QF, base + 16 * (t + 4 * (s / 4)) + 4 * (s % 4) + e) * up : 0.f;
        qh[nt][s][0][0] = pack_half(x[0], x[1]);
        qh[nt][s][0][1] = pack_half(x[2], x[3]);
        if (QF) {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] -= __half2float(__float2half_rn(x[e]));
          qh[nt][s][QL - 1][0] = pack_half(x[0], x[1]);
          qh[nt][s][QL - 1][1] = pack_half(x[2], x[3]);
        }
      }
      const float mine = a.scale2 / up;
      const int my_hi = !live ? 0 : a.causal ? max(0, sg.n - a.nq + i + 1) : sg.n;
      const int my_lo = a.window > 0 ? max(0, my_hi - a.window) : 0;
      int x = live ? my_hi : 0x7fffffff, y = live ? my_lo : 0;
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        x = min(x, __shfl_xor_sync(0xffffffffu, x, o));
        y = max(y, __shfl_xor_sync(0xffffffffu, y, o));
      }
      hi_min = min(hi_min, x);
      lo_max = max(lo_max, y);
#pragma unroll
      for (int j = 0; j < 2; ++j) {                  // the score columns of this lane are rows 2t and 2t + 1
        cq[nt][j] = __shfl_sync(0xffffffffu, mine, (2 * t + j) * 4);
        hi[nt][j] = __shfl_sync(0xffffffffu, my_hi, (2 * t + j) * 4);
        lo[nt][j] = __shfl_sync(0xffffffffu, my_lo, (2 * t + j) * 4);
      }
    }
    float acc[NT][MT][4];
    float m[NT][2], l[NT][2];
    float vrun = 1.17549435e-38f;                    // the sums are in units of this value scale
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int x = 0; x < MT; ++x) acc[nt][x][0] = acc[nt][x][1] = acc[nt][x][2] = acc[nt][x][3] = 0.f;
    }
    for (int k0 = sg.t0 + 16 * w; k0 < sg.t1; k0 += 16 * kAtWarps) {
      const int64_t page = page_of(a, sg.b, k0 / a.block);
      const bool ok = page >= 0 && page < a.n_blocks;
      if (!ok) {
        if (lane == 0 && a.d_status) atomicOr(a.d_status, TQ_DEV_BAD_BLOCK);
        continue;
      }
      const int64_t ph = page * a.heads + sg.kv;
      const float ks = a.ks[ph], vs = a.vs[ph];
      const uint8_t* kp = a.k + (ph * a.block + k0 % a.block) * D;
      const uint8_t* vp = a.v + (ph * a.block + k0 % a.block) * D;
      const int left = sg.n - k0;                    // keys of the group that the sequence has
      uint4 kw[2][KC];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < KC; ++c)
          kw[h][c] = *reinterpret_cast<const uint4*>(kp + (g + 8 * h) * D + 16 * (t + 4 * c));
      uint32_t vw[4][VW];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = 2 * t + (j & 1) + 8 * (j >> 1);
        const bool in = row < left;                  // what lies behind the sequence may be any byte
#pragma unroll
        for (int c = 0; c < VW / 2; ++c) {
          const uint2 x = in ? *reinterpret_cast<const uint2*>(vp + row * D + (VW >= 4 ? 16 * (g + 8 * (c / 2)) + 8 * (c % 2) : 8 * g))
                             : make_uint2(0u, 0u);
          vw[j][2 * c] = x.x;
          vw[j][2 * c + 1] = x.y;
        }
      }
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
      for (int st = 0; st < KS; ++st) {
        const uint32_t w0 = (&kw[0][st / 4].x)[st % 4], w1 = (&kw[1][st / 4].x)[st % 4];
        const uint32_t a0 = two_halves<INT8, false>(w0), a2 = two_halves<INT8, true>(w0);
        const uint32_t a1 = two_halves<INT8, false>(w1), a3 = two_halves<INT8, true>(w1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (QF) {
            // Each step's products are added in fp32: the matrix unit's own sums are cut, not rounded.
            float x[4] = {0.f, 0.f, 0.f, 0.f};
            mma_f16(x, a0, a1, a2, a3, qh[nt][st][QL - 1][0], qh[nt][st][QL - 1][1]);
            mma_f16(x, a0, a1, a2, a3, qh[nt][st][0][0], qh[nt][st][0][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][e] += x[e];
          } else {
            mma_f16(s[nt], a0, a1, a2, a3, qh[nt][st][0][0], qh[nt][st][0][1]);
          }
        }
      }
      const bool full = k0 >= lo_max && k0 + 16 <= hi_min;
      bool rise = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[nt][e] *= cq[nt][e & 1] * ks;
          if (!full) {
            const int key = k0 + g + 8 * (e >> 1);
            if (key < lo[nt][e & 1] || key >= hi[nt][e & 1]) s[nt][e] = -INFINITY;
          }
          rise |= s[nt][e] > m[nt][e & 1] + kSlack;
        }
      }
      if (__any_sync(0xffffffffu, rise || vs > vrun)) {
        const float fv = vs > vrun ? vrun / vs : 1.f;
        vrun = fmaxf(vrun, vs);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float f[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float x = fmaxf(s[nt][j], s[nt][j + 2]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
            const float mn = fmaxf(m[nt][j], x);
            f[j] = mn == m[nt][j] ? 1.f : fast_exp2(m[nt][j] - mn);
            m[nt][j] = mn;
            l[nt][j] *= f[j];
            f[j] *= fv;
          }
#pragma unroll
          for (int x = 0; x < MT; ++x) {
            acc[nt][x][0] *= f[0];
            acc[nt][x][1] *= f[1];
            acc[nt][x][2] *= f[0];
            acc[nt][x][3] *= f[1];
          }
        }
      }
      const float vr = vs / vrun;
      uint32_t ph0[NT][2], ph1[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // A row that has seen no key yet has m = -inf: its weights are 0, not e^(-inf + inf).
          p[e] = s[nt][e] == -INFINITY ? 0.f : fast_exp2(s[nt][e] - m[nt][e & 1] + kLift);
          l[nt][e & 1] += p[e];
          p[e] *= vr;
        }
        const uint32_t h0 = pack_half(p[0], p[1]), h1 = pack_half(p[2], p[3]);
        ph0[nt][0] = transpose8(h0);
        ph0[nt][1] = transpose8(h1);
        if (OF) {
          const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h0));
          const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&h1));
          ph1[nt][0] = transpose8(pack_half(p[0] - x.x, p[1] - x.y));
          ph1[nt][1] = transpose8(pack_half(p[2] - y.x, p[3] - y.y));
        }
      }
#pragma unroll
      for (int x = 0; x < VW; ++x) {
        // Coordinate pairs of two keys side by side: (key 2t, key 2t + 1) per half pair.
        const uint32_t p0 = __byte_perm(vw[0][x], vw[1][x], 0x5140), p1 = __byte_perm(vw[0][x], vw[1][x], 0x7362);
        const uint32_t q0 = __byte_perm(vw[2][x], vw[3][x], 0x5140), q1 = __byte_perm(vw[2][x], vw[3][x], 0x7362);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t a0 = two_halves<INT8, false>(h ? p1 : p0), a1 = two_halves<INT8, true>(h ? p1 : p0);
          const uint32_t a2 = two_halves<INT8, false>(h ? q1 : q0), a3 = two_halves<INT8, true>(h ? q1 : q0);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (OF) {
              float y[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16(y, a0, a1, a2, a3, ph1[nt][0], ph1[nt][1]);
              mma_f16(y, a0, a1, a2, a3, ph0[nt][0], ph0[nt][1]);
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[nt][2 * x + h][e] += y[e];
            } else {
              mma_f16(acc[nt][2 * x + h], a0, a1, a2, a3, ph0[nt][0], ph0[nt][1]);
            }
          }
        }
      }
    }
    // Merge the warps: maxima and sums, then the value sums a piece at a time.
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x = l[nt][j];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (g == 0) {
          sm_m[w][nt * 8 + 2 * t + j] = m[nt][j];
          sm_l[w][nt * 8 + 2 * t + j] = x;
        }
      }
    __syncthreads();
    float f[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float M = -INFINITY;
        for (int k = 0; k < kAtWarps; ++k) M = fmaxf(M, sm_m[k][nt * 8 + 2 * t + j]);
        f[nt][j] = m[nt][j] == -INFINITY ? 0.f : fast_exp2(m[nt][j] - M) * vrun;
      }
    float* rec = a.rec + (static_cast<int64_t>(blockIdx.x) * 2 + (sg.head && u != u0 ? 1 : 0)) * kRows * (D + 2);
    constexpr int kPairs = NT * MT;
#pragma unroll
    for (int p0 = 0; p0 < kPairs; p0 += 4) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int nt = (p0 + p) / MT, x = (p0 + p) % MT;
        sm_acc[w][p][lane] = make_float4(acc[nt][x][0] * f[nt][0], acc[nt][x][1] * f[nt][1], acc[nt][x][2] * f[nt][0],
                                         acc[nt][x][3] * f[nt][1]);
      }
      __syncthreads();
      {
        const int p = tid >> 6, ln = (tid & 63) >> 1, c = tid & 1;   // two values: coordinate + c, rows 2t' and 2t' + 1
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kAtWarps; ++k) {
          const float2 y = reinterpret_cast<const float2*>(&sm_acc[k][p][ln])[c];
          sum.x += y.x;
          sum.y += y.y;
        }
        const int nt = (p0 + p) / MT, x = (p0 + p) % MT;
        const int wd = x >> 1, gg = ln >> 2, tt = ln & 3;
        const int dim = (VW >= 4 ? 16 * (gg + 8 * (wd / 4)) + 4 * (wd % 4) : 8 * gg + 4 * wd) + 2 * (x & 1) + c;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int row = nt * 8 + 2 * tt + j, r = sg.rt * kRows + row;
          if (r >= a.rows) continue;
          const float val = j ? sum.y : sum.x;
          float M = -INFINITY, L = 0.f;
          for (int k = 0; k < kAtWarps; ++k) M = fmaxf(M, sm_m[k][row]);
          for (int k = 0; k < kAtWarps; ++k)
            if (sm_m[k][row] != -INFINITY) L += sm_l[k][row] * fast_exp2(sm_m[k][row] - M);
          if (sg.whole) {
            const int i = r / a.group, hq = sg.kv * a.group + r % a.group;
            const int64_t at = (a.first_seq + sg.b) * a.o_bs + hq * a.o_hs + i * a.o_rs + dim;
            const float o = L == 0.f ? 0.f : val / L;
            if (OF) static_cast<float*>(a.out)[at] = o;
            else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(o);
            if (a.lse && dim == 0)
              a.lse[((a.first_seq + sg.b) * a.heads * a.group + hq) * a.nq + i] =
                  L == 0.f ? -INFINITY : (M - kLift + log2f(L)) * kLn2;
          } else {
            rec[row * (D + 2) + 2 + dim] = val;
            if (dim == 0) {
              rec[row * (D + 2)] = M;
              rec[row * (D + 2) + 1] = L;
            }
          }
        }
      }
      __syncthreads();
    }
    u = next;
  }
}

// Merges the records of every stream that more than one CTA worked on, and
// writes the rows of streams with no key at all. One CTA per (sequence, KV
// head and row tile); a warp per row.
template <int D, int NT, bool OF>
__global__ void __launch_bounds__(256) cache8_combine_kernel(AttnArgs a, int grid) {
  constexpr int kRows = 8 * NT;
  const int b = blockIdx.y, stream = blockIdx.x;
  const int c0 = a.cum_out[b], tiles = (a.cum_out[b + 1] - c0) / (a.heads * a.row_tiles);
  const int total = a.cum_out[a.batch];
  const int per = max((total + grid - 1) / grid, kMinUnits);
  const int u0 = c0 + stream * tiles, u1 = u0 + tiles;
  const int first = u0 / per, last = tiles > 0 ? (u1 - 1) / per : first;
  if (tiles > 0 && first == last) return;            // one CTA had it all and wrote the rows
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kv = stream / a.row_tiles, rt = stream % a.row_tiles;
  for (int row = w; row < kRows; row += 8) {
    const int r = rt * kRows + row;
    if (r >= a.rows) break;
    float M = -INFINITY, L = 0.f, sum[D / 32];
#pragma unroll
    for (int x = 0; x < D / 32; ++x) sum[x] = 0.f;
    for (int c = first; tiles > 0 && c <= last; ++c) {
      const int slot = c == first && u0 != c * per ? 1 : 0;
      const float* rec = a.rec + ((static_cast<int64_t>(c) * 2 + slot) * kRows + row) * (D + 2);
      const float m = rec[0], l = rec[1];
      if (m == -INFINITY) continue;
      const float mn = fmaxf(M, m), f = M == -INFINITY ? 0.f : fast_exp2(M - mn), h = fast_exp2(m - mn);
      L = L * f + l * h;
#pragma unroll
      for (int x = 0; x < D / 32; ++x) sum[x] = sum[x] * f + rec[2 + x * 32 + lane] * h;
      M = mn;
    }
    const int i = r / a.group, hq = kv * a.group + r % a.group;
    const int64_t at = (a.first_seq + b) * a.o_bs + hq * a.o_hs + i * a.o_rs;
    const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int x = 0; x < D / 32; ++x) {
      if (OF) static_cast<float*>(a.out)[at + x * 32 + lane] = sum[x] * inv;
      else static_cast<__nv_bfloat16*>(a.out)[at + x * 32 + lane] = __float2bfloat16_rn(sum[x] * inv);
    }
    if (a.lse && lane == 0)
      a.lse[((a.first_seq + b) * a.heads * a.group + hq) * a.nq + i] =
          L == 0.f ? -INFINITY : (M - kLift + log2f(L)) * kLn2;
  }
}

template <int D, bool INT8, int NT, bool QF, bool OF>
cudaError_t launch_attn(const AttnArgs& a, cudaStream_t st) {
  cache8_attn_kernel<D, INT8, NT, QF, OF><<<kAtGrid, kAtThreads, 0, st>>>(a);
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cache8_combine_kernel<D, NT, OF><<<dim3(a.heads * a.row_tiles, a.batch), 256, 0, st>>>(a, kAtGrid);
  count_launch();
  return cudaGetLastError();
}

template <int D, bool INT8, int NT>
cudaError_t launch_types(bool qf, bool of, const AttnArgs& a, cudaStream_t st) {
  if (qf && of) return launch_attn<D, INT8, NT, true, true>(a, st);
  if (qf) return launch_attn<D, INT8, NT, true, false>(a, st);
  if (of) return launch_attn<D, INT8, NT, false, true>(a, st);
  return launch_attn<D, INT8, NT, false, false>(a, st);
}

// Query rows a CTA takes together: 8, or 16 where a KV head has more and the
// sums of 16 rows fit the registers (d up to 128, not both fp32).
int rows_of(int d, int rows, bool f32) { return rows > 8 && d <= 128 && !f32 ? 16 : 8; }

constexpr size_t kCumBytes = (sizeof(int) * (kC8Slice + 1) + 255) / 256 * 256;

size_t attn_workspace(int d) { return kCumBytes + sizeof(float) * kAtGrid * 2 * 16 * static_cast<size_t>(d + 2); }

}  // namespace
}  // namespace tq

extern "C" size_t tq_cache8_attention_workspace_bytes(const tq_cache8* cache, int32_t batch, int32_t hq, int32_t nq) {
  if (tq::check_cache8(cache, "tq_cache8_attention_workspace_bytes") != TQ_OK || batch < 0 || hq < 1 || nq < 1) return 0;
  return tq::attn_workspace(cache->d);
}

extern "C" tq_status tq_cache8_attention(const tq_cache8* cache, const void* q, tq_dtype q_dtype, int64_t q_batch_stride,
                                         int64_t q_head_stride, int64_t q_row_stride, int32_t batch, int32_t hq,
                                         int32_t nq, const int32_t* seq_lens, const int32_t* block_table,
                                         int64_t table_stride, int32_t causal, int32_t window, float scale, void* out,
                                         tq_dtype out_dtype, int64_t out_batch_stride, int64_t out_head_stride,
                                         int64_t out_row_stride, float* lse_out, void* workspace, size_t workspace_bytes,
                                         int32_t* d_status, void* stream) {
  using namespace tq;
  const char* what = "tq_cache8_attention";
  clear_error();
  tq_status st = check_cache8(cache, what);
  if (st != TQ_OK) return st;
  const int d = cache->d;
  if ((q_dtype != TQ_F32 && q_dtype != TQ_BF16) || (out_dtype != TQ_F32 && out_dtype != TQ_BF16))
    return fail(TQ_ERR_INVALID_ARG, "%s: q and out must be TQ_F32 or TQ_BF16", what);
  if (batch < 0 || hq < 1 || nq < 1) return fail(TQ_ERR_INVALID_ARG, "%s: batch < 0, hq < 1 or nq < 1", what);
  if (hq % cache->heads != 0)
    return fail(TQ_ERR_INVALID_ARG, "%s: hq (%d) is not a multiple of the cache's heads (%d)", what, hq, cache->heads);
  if (static_cast<int64_t>(hq) * nq > 0x3fffffff) return fail(TQ_ERR_INVALID_ARG, "%s: hq * nq too large", what);
  if (window < 0) return fail(TQ_ERR_INVALID_ARG, "%s: window must not be negative", what);
  if (window > 0 && !causal) return fail(TQ_ERR_INVALID_ARG, "%s: a window needs causal attention", what);
  if (!(scale > -INFINITY && scale < INFINITY)) return fail(TQ_ERR_INVALID_ARG, "%s: scale must be finite", what);
  if (batch == 0) return TQ_OK;
  if (!q || !out || !seq_lens) return fail(TQ_ERR_INVALID_ARG, "%s: NULL q, out or seq_lens", what);
  st = check_table8(cache, batch, table_stride, what);
  if (st != TQ_OK) return st;
  if (!block_table && table_stride * batch > cache->n_blocks)
    return fail(TQ_ERR_INVALID_ARG, "%s: without a block table the cache needs batch * table_stride blocks", what);
  if (!aligned(q, 16) || !aligned(out, 16) || q_batch_stride % 8 || q_head_stride % 8 || q_row_stride % 8 ||
      out_batch_stride % 8 || out_head_stride % 8 || out_row_stride % 8)
    return fail(TQ_ERR_INVALID_ARG, "%s: q and out must be 16-byte aligned, strides multiples of 8 elements", what);
  if (q_batch_stride < 0 || q_head_stride < 0 || q_row_stride < 0 || out_batch_stride < 0 || out_head_stride < 0 ||
      out_row_stride < 0)
    return fail(TQ_ERR_INVALID_ARG, "%s: negative stride", what);
  if ((batch > 1 && out_batch_stride < d) || rows_overlap(hq, out_head_stride, nq, out_row_stride, d))
    return fail(TQ_ERR_INVALID_ARG, "%s: the strides of out make rows overlap", what);
  if (d != 64 && d != 128 && d != 256)
    return fail(TQ_ERR_UNSUPPORTED, "%s: d=%d not built (64, 128, 256)", what, d);
  if (!workspace || workspace_bytes < attn_workspace(d))
    return fail(TQ_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", what, workspace_bytes, attn_workspace(d));
  if (!aligned(workspace, 256)) return fail(TQ_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", what);
  const bool qf = q_dtype == TQ_F32, of = out_dtype == TQ_F32;
  const int group = hq / cache->heads, rows = group * nq;
  const int tile = rows_of(d, rows, qf || of), row_tiles = (rows + tile - 1) / tile;
  // Units of one launch stay below 2^30: batches are cut into slices.
  const int64_t per_seq = ((table_stride * cache->block + kUnit - 1) / kUnit) * cache->heads * row_tiles;
  if (per_seq > (1 << 25))
    return fail(TQ_ERR_UNSUPPORTED, "%s: heads x query rows x capacity of one sequence too large", what);
  int64_t slice = (1 << 30) / per_seq;
  if (slice > kC8Slice) slice = kC8Slice;
  AttnArgs a{cache->heads, cache->block, 0, cache->n_blocks, cache->k, cache->v, cache->k_scale, cache->v_scale, q,
             q_batch_stride, q_head_stride, q_row_stride, group, nq, rows, row_tiles, nullptr, nullptr, table_stride, 0,
             causal ? 1 : 0, window, scale * kLog2e, out, out_batch_stride, out_head_stride, out_row_stride, lse_out,
             reinterpret_cast<float*>(static_cast<char*>(workspace) + kCumBytes), static_cast<int*>(workspace), d_status};
  const bool i8 = cache->code == TQ_INT8;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  for (int64_t b0 = 0; b0 < batch; b0 += slice) {
    a.batch = static_cast<int>(batch - b0 < slice ? batch - b0 : slice);
    a.first_seq = b0;
    a.lens = seq_lens + b0;
    a.table = block_table ? block_table + b0 * table_stride : nullptr;
    cudaError_t e;
#define TQ_C8(D, NT) (i8 ? launch_types<D, true, NT>(qf, of, a, s) : launch_types<D, false, NT>(qf, of, a, s))
    if (d == 64) e = tile == 16 ? TQ_C8(64, 2) : TQ_C8(64, 1);
    else if (d == 128) e = tile == 16 ? TQ_C8(128, 2) : TQ_C8(128, 1);
    else e = TQ_C8(256, 1);
#undef TQ_C8
    if (e != cudaSuccess) return fail(TQ_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
  }
  return TQ_OK;
}
