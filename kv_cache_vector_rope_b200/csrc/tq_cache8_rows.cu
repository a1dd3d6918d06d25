// tq_cache8_attention for many query rows where tensor memory cannot hold or
// round them: fp32 queries or outputs, and d = 256.
//
// The formulas are those of tq_cache8_attn.cu. A CTA takes 128 query rows,
// sixteen to a warp, and walks 64 keys at a time. Codes come by asynchronous
// copies, each thread converts its own once for all 128 rows into halves (an
// 8-bit code is exactly one), and the warps read them as operands of 16x8x16
// half products: scores with the query rows as the 16 rows, then the weights,
// whose registers already lie as the second product's operand, times the values.
// WIDE, for fp32: queries and weights are two half limbs each (2^-22 of the
// row's largest), and the products of a step are added in fp32, because the
// matrix unit cuts its own sums instead of rounding them; that is why these rows
// do not go the way of tq_cache8_chunk.cu, whose sums stay in tensor memory.
//
// Bound by the matrix instructions: 2 x 128 of them a warp and tile at d = 128,
// fp32, or at d = 256, 1.23 ns each per SM, half of the time; the rest is the
// conversion, the weights and the barriers between them. Measured, 512 rows of
// two sequences of 8192 tokens: 8 KV heads of 4 fp32 heads, d = 128, 1118 us (by
// eights of rows 2040), d = 64 568 us; 4 KV heads, d = 256, bf16 641 us, fp32 989 us.
#include "tq_cache8_attn.cuh"

namespace tq {
namespace {

using namespace c8;
using namespace sm100;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kTile = kRowsUnit;                     // keys at a time
static_assert(kTile == 64 && kRowsTile == 16 * kWarps, "four groups of 16 keys, 16 rows a warp");

// CTAs per SM: at d = 64 two, whose barriers and products overlap (512 fp32 rows of 2 x 8192 tokens 657 -> 559 us when it was chosen,
// though 128 registers spill 200 bytes); at d = 128 two do not fit shared memory.
constexpr int rows_ctas(int d) { return d <= 64 ? 2 : 1; }

template <int D, bool WIDE>
struct Smem {
  static constexpr int kOffQ = 0;                    // [limbs][128][D] halves
  static constexpr int kLimb = 128 * D * 2;
  static constexpr int kOffK = kOffQ + (WIDE ? 2 : 1) * kLimb;
  static constexpr int kOffV = kOffK + kTile * D * 2;
  static constexpr int kOffRaw = kOffV + kTile * D * 2;          // K, V: [64][D] codes
  static constexpr int kOffScale = kOffRaw + 2 * kTile * D;      // float [2][K, V][4]
  static constexpr int kOffOk = kOffScale + 64;                  // int [2][4]
  static constexpr int kOffSome = kOffOk + 32;                   // bytes [64]: whether the key has a value code that is not zero
  static constexpr int kOffRow = kOffSome + kTile;               // float [128]: score factors
  static constexpr int kOffPart = kOffRow + 4 * 128;
  static constexpr int kOffCum = kOffPart + 4 * kWarps;
  static constexpr int kBytes = kOffCum + 4 * (kRowsSlice + 1) + 128;  // and room to align the base
};

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Byte offset of 16-byte chunk c of a row of D halves: eight rows' chunks c lie in eight different bank groups.
template <int D>
__device__ __forceinline__ int chunk_at(int row, int c) {
  return row * (2 * D) + ((c ^ (row & 7)) << 4);
}

template <int D, bool INT8, bool WIDE>
__global__ void __launch_bounds__(kThreads, rows_ctas(D)) cache8_rows_kernel(AttnArgs a) {
  using L = Smem<D, WIDE>;
  constexpr int kLimbs = WIDE ? 2 : 1;
  constexpr int kPer = D / 64;                       // 16-byte pieces of K (and of V) a thread copies of a tile
  constexpr int kRowsPer = 4096 / D;                 // keys that all threads' first pieces cover
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + (128 - (smem_u32(smem_raw) & 127)) % 128;
  const uint32_t base = smem_u32(smem);
  float* sm_scale = reinterpret_cast<float*>(smem + L::kOffScale);
  int* sm_ok = reinterpret_cast<int*>(smem + L::kOffOk);
  unsigned char* sm_some = smem + L::kOffSome;
  float* sm_cq = reinterpret_cast<float*>(smem + L::kOffRow);
  int* cum = reinterpret_cast<int*>(smem + L::kOffCum);
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  scan_counts<kThreads>(cum, reinterpret_cast<int*>(smem + L::kOffPart), a.batch, [&](int b) {
    return head_units(a, seq_len(a, b, blockIdx.x == 0)) * a.heads;
  });
  if (tid == 0) a.cuts[blockIdx.x].n = 0;
  let_next_start();
  const int total = cum[a.batch];
  const int per = units_per_cta(a, total, gridDim.x);
  const int u0 = min(static_cast<int>(blockIdx.x) * per, total), u1 = min(u0 + per, total);
  // A thread copies and converts pieces of the same keys and coordinates of every tile.
  const int piece_row = tid / (D / 16), piece = tid % (D / 16);
  const uint32_t raw = base + L::kOffRaw + piece_row * D + piece * 16;
  Seg sg;
  for (int u = u0, next; u < u1; u = next) {
    if (u == u0) sg = seg_at(a, cum, u, u1, &next);
    else seg_after(a, cum, sg, u, u1, &next);
    if (sg.t1 <= sg.t0) continue;
    const int key0 = sg.t0 / kTile * kTile, tiles = (sg.t1 - key0 + kTile - 1) / kTile;
    // Pages of the thread's pieces, and of group tid of a tile: -1 for keys the segment does not reach.
    int pg[kPer], pg_group = -1;
    const auto page_at = [&](int key) {
      return key >= sg.t0 && key < sg.t1 ? static_cast<int>(page_of(a, sg.b, key >> a.block_log2)) : -1;
    };
    const auto pages = [&](int j) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) pg[i] = page_at(key0 + j * kTile + (piece_row + i * kRowsPer) / 16 * 16);
      if (tid < 4) pg_group = page_at(key0 + j * kTile + 16 * tid);
    };
    const auto ok = [&](int page) { return page >= 0 && page < a.n_blocks; };
    const auto issue = [&](int j) {                  // tile j's codes and scales set out, the next tile's pages looked up
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (ok(pg[i])) {
          const int key = key0 + j * kTile + piece_row + i * kRowsPer;
          const int64_t at = ((static_cast<int64_t>(pg[i]) * a.heads + sg.kv) * a.block + (key & (a.block - 1))) * D + 16 * piece;
          copy16(raw + i * 4096, a.k + at);
          copy16(raw + i * 4096 + kTile * D, a.v + at);
        }
      if (tid < 4) {
        const bool good = ok(pg_group);
        const int key = key0 + j * kTile + 16 * tid;
        float* to = sm_scale + (j & 1) * 8 + tid;
        sm_ok[(j & 1) * 4 + tid] = good;
        if (good) {
          copy4(smem_u32(to), a.ks + static_cast<int64_t>(pg_group) * a.heads + sg.kv);
          copy4(smem_u32(to + 4), a.vs + static_cast<int64_t>(pg_group) * a.heads + sg.kv);
        } else {
          to[0] = to[4] = 0.f;
          if (key >= sg.t0 && key < sg.t1 && a.d_status) atomicOr(a.d_status, TQ_DEV_BAD_BLOCK);
        }
      }
      pages(j + 1);
    };
    __syncthreads();                                 // the last segment's readers of the queries and scales are done
    pages(0);
    issue(0);
    // Queries: two threads to a row, half of its coordinates each. Times a power of two the largest coordinate of a row
    // lands in [2^14, 2^15).
    {
      const int row = tid >> 1, r = sg.rt * kRowsTile + row, c0 = (tid & 1) * (D / 32);
      const bool live = r < a.rows;
      const int i = live ? a.group_div.of(r) : 0, hq = sg.kv * a.group + (live ? r - i * a.group : 0);
      const int64_t from = (a.first_seq + sg.b) * a.q_bs + hq * a.q_hs + i * a.q_rs;
      const auto load = [&](int c, float (&x)[16]) {
        if (!live) {
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = 0.f;
        } else if (a.q_f32) {
          load_q16<true>(a.q, from + 16 * c, x);
        } else {
          load_q16<false>(a.q, from + 16 * c, x);
        }
      };
      float amax = 0.f;
#pragma unroll 2
      for (int c = c0; c < c0 + D / 32; ++c) {
        float x[16];
        load(c, x);
#pragma unroll
        for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e]));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      const int E = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -100);
      const float up = __uint_as_float(static_cast<uint32_t>(14 - min(E, 127) + 127) << 23);
      if (!(tid & 1)) sm_cq[row] = a.scale2 / up;
#pragma unroll 2
      for (int c = c0; c < c0 + D / 32; ++c) {
        float x[16];
        load(c, x);
#pragma unroll
        for (int limb = 0; limb < kLimbs; ++limb) {
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (limb == 0) {
              x[2 * e] *= up;
              x[2 * e + 1] *= up;
            } else {
              x[2 * e] -= __half2float(__float2half_rn(x[2 * e]));
              x[2 * e + 1] -= __half2float(__float2half_rn(x[2 * e + 1]));
            }
            h[e] = pack_half(x[2 * e], x[2 * e + 1]);
          }
          unsigned char* q = smem + L::kOffQ + limb * L::kLimb;
          *reinterpret_cast<uint4*>(q + chunk_at<D>(row, 2 * c)) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(q + chunk_at<D>(row, 2 * c + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
        }
      }
    }
    // The lane's two rows, g and g + 8 of the warp's sixteen.
    const int r0 = sg.rt * kRowsTile + 16 * w;
    int lo[2], hi[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = r0 + g + 8 * x;
      hi[x] = r < a.rows ? row_hi(a, sg.n, a.group_div.of(r)) : 0;
      lo[x] = row_lo(a, hi[x]);
    }
    const bool any_row = r0 < a.rows;
    const int last = any_row ? a.group_div.of(min(r0 + 15, a.rows - 1)) : 0;
    const int hi_min = any_row ? row_hi(a, sg.n, a.group_div.of(r0)) : 0, hi_max = any_row ? row_hi(a, sg.n, last) : 0;
    const int lo_min = row_lo(a, hi_min), lo_max = row_lo(a, hi_max);
    float acc[D / 8][4];
    float m[2] = {-INFINITY, -INFINITY}, unit[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int x = 0; x < D / 8; ++x) acc[x][0] = acc[x][1] = acc[x][2] = acc[x][3] = 0.f;
    float cq[2] = {0.f, 0.f};
    for (int j = 0; j < tiles; ++j) {
      const int tile0 = key0 + j * kTile;
      const float* scale = sm_scale + (j & 1) * 8;
      const int* good = sm_ok + (j & 1) * 4;
      copies_done();
      __syncthreads();                               // tile j's scales are there; the last tile's operands have been read
      if (j == 0) {
        cq[0] = sm_cq[16 * w + g];
        cq[1] = sm_cq[16 * w + g + 8];
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int row = piece_row + i * kRowsPer;
        const bool real = good[row >> 4] && tile0 + row < sg.n;      // what lies elsewhere may be any byte
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          uint4 y = *reinterpret_cast<const uint4*>(smem + (raw - base) + i * 4096 + kv * kTile * D);
          if (!real) y = make_uint4(0u, 0u, 0u, 0u);
          const uint32_t in[4] = {y.x, y.y, y.z, y.w};
          if (kv) {                                  // D / 16 lanes side by side hold a key
            const uint32_t any = __ballot_sync(0xffffffffu, ((y.x | y.y | y.z | y.w) & (INT8 ? 0xffffffffu : 0x7f7f7f7fu)) != 0u);
            if (piece == 0) sm_some[row] = ((any >> lane) & ((1u << (D / 16)) - 1u)) != 0u;
          }
          uint32_t h[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            h[2 * k] = two_halves<INT8, false>(in[k]);
            h[2 * k + 1] = two_halves<INT8, true>(in[k]);
          }
          unsigned char* to = smem + (kv ? L::kOffV : L::kOffK);
          *reinterpret_cast<uint4*>(to + chunk_at<D>(row, 2 * piece)) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(to + chunk_at<D>(row, 2 * piece + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
        }
      }
      if (j + 1 < tiles) issue(j + 1);               // each thread's codes have become halves
      __syncthreads();
      if (!any_row || tile0 >= hi_max || tile0 + kTile <= lo_min) continue;
      // Scores: tile nt of 8 keys, rows g (0, 1) and g + 8 (2, 3), keys 2 t and 2 t + 1.
      float s[8][4];
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
      const int qrow = 16 * w + (lane & 15);
#pragma unroll 2
      for (int ks = 0; ks < D / 16; ks += 2) {       // two steps of 16 coordinates
        uint32_t qa[kLimbs][2][4];
#pragma unroll
        for (int limb = 0; limb < kLimbs; ++limb)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            ldsm4(qa[limb][x], base + L::kOffQ + limb * L::kLimb + chunk_at<D>(qrow, 2 * (ks + x) + (lane >> 4)));
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
          uint32_t kb[4];
          ldsm4(kb, base + L::kOffK + chunk_at<D>(8 * nt + (lane & 7), 2 * ks + (lane >> 3)));
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if constexpr (WIDE) {
              float y[4] = {0.f, 0.f, 0.f, 0.f};
              mma(y, qa[kLimbs - 1][x], kb[2 * x], kb[2 * x + 1]);
              mma(y, qa[0][x], kb[2 * x], kb[2 * x + 1]);
#pragma unroll
              for (int e = 0; e < 4; ++e) s[nt][e] += y[e];
            } else {
              mma(s[nt], qa[0][x], kb[2 * x], kb[2 * x + 1]);
            }
          }
        }
      }
      const bool full = tile0 >= lo_max && tile0 + kTile <= hi_min && good[0] && good[1] && good[2] && good[3];
      bool rise = false;
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        const float ks = scale[nt >> 1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[nt][e] *= cq[e >> 1] * ks;
          if (!full) {
            const int key = tile0 + 8 * nt + 2 * t + (e & 1);
            if (key < lo[e >> 1] || key >= hi[e >> 1] || !good[nt >> 1]) s[nt][e] = -INFINITY;
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
          rise |= fmaxf(s[nt][2 * x], s[nt][2 * x + 1]) > weigh(m[x], unit[x], octaves(scale[4 + (nt >> 1)])).lim;
      }
      if (__any_sync(0xffffffffu, rise)) {
        float f[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float top = -INFINITY, topv = -INFINITY;
#pragma unroll
          for (int nt = 0; nt < 8; ++nt) top = fmaxf(top, fmaxf(s[nt][2 * x], s[nt][2 * x + 1]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const float mn = fmaxf(m[x], rintf(top)), by = below(m[x], mn);
#pragma unroll
          for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (sm_some[8 * nt + 2 * t + e] && s[nt][2 * x + e] > -INFINITY)
                topv = fmaxf(topv, below(s[nt][2 * x + e], mn) + octaves(scale[4 + (nt >> 1)]));
          topv = fmaxf(topv, __shfl_xor_sync(0xffffffffu, topv, 1));
          topv = fmaxf(topv, __shfl_xor_sync(0xffffffffu, topv, 2));
          const float en = next_unit(unit[x], by, topv);
          f[x] = unit_step(m[x], unit[x], mn, en);
          l[x] *= fast_exp2(by);
          m[x] = mn;
          unit[x] = en;
          // Keys without a value: counted here, then left out.
#pragma unroll
          for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float& y = s[nt][2 * x + e];
              if (sm_some[8 * nt + 2 * t + e] || y == -INFINITY) continue;
              l[x] += fast_exp2((y - base_of(mn)) + kLift);
              y = -INFINITY;
            }
        }
#pragma unroll
        for (int x = 0; x < D / 8; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[x][e] *= f[e >> 1];
      }
      // Weights: the scores' registers of 16 keys are the next product's operand as they lie.
      uint32_t pa[kLimbs][4][4];
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        const float lv = octaves(scale[4 + (nt >> 1)]);
        float p[4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const Weigh y = weigh(m[x], unit[x], lv);
          const float base = base_of(m[x]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            p[2 * x + e] = fast_exp2((s[nt][2 * x + e] - base) + y.lift);
            l[x] = fmaf(p[2 * x + e], y.inv, l[x]);
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t h = pack_half(p[2 * x], p[2 * x + 1]);
          pa[0][nt >> 1][2 * (nt & 1) + x] = h;
          if constexpr (WIDE) {
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&h));
            pa[kLimbs - 1][nt >> 1][2 * (nt & 1) + x] = pack_half((p[2 * x] - y.x) * kLimb, (p[2 * x + 1] - y.y) * kLimb);
          }
        }
      }
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {             // 16 coordinates: two tiles of 8
        float y[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}}, z[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          uint32_t vb[4];
          ldsm4_trans(vb, base + L::kOffV + chunk_at<D>(16 * kk + (lane & 15), 2 * c + (lane >> 4)));
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if constexpr (WIDE) {
              mma(z[x], pa[kLimbs - 1][kk], vb[2 * x], vb[2 * x + 1]);
              mma(y[x], pa[0][kk], vb[2 * x], vb[2 * x + 1]);
            } else {
              mma(acc[2 * c + x], pa[0][kk], vb[2 * x], vb[2 * x + 1]);
            }
          }
        }
        if constexpr (WIDE) {
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[2 * c + x][e] = fmaf(z[x][e], 1.f / kLimb, acc[2 * c + x][e] + y[x][e]);
        }
      }
    }
    // Out, or to the record of a stream that other CTAs share.
    const bool second = sg.head && u != u0;          // the record's slot
    if (tid == 0 && sg.head && !sg.whole) a.cuts[blockIdx.x] = cut_of(a, sg, second, per);
    float* rec = a.rec + (static_cast<int64_t>(blockIdx.x) * 2 + (second ? 1 : 0)) * kRowsTile * (kRecHead + D);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
      const int row = 16 * w + g + 8 * x, r = sg.rt * kRowsTile + row;
      if (r >= a.rows) continue;
      const int i = a.group_div.of(r), hq = sg.kv * a.group + r - i * a.group;
      const int64_t at = (a.first_seq + sg.b) * a.o_bs + hq * a.o_hs + i * a.o_rs + 2 * t;
      const float e = unit_of(unit[x]), by = sg.whole ? (l[x] == 0.f ? 0.f : 1.f / l[x] * pow2_whole(e)) : 1.f;
      float* to = rec + row * (kRecHead + D);
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const float2 y = make_float2(l[x] == 0.f ? 0.f : acc[c][2 * x] * by, l[x] == 0.f ? 0.f : acc[c][2 * x + 1] * by);
        if (!sg.whole) *reinterpret_cast<float2*>(to + kRecHead + 8 * c + 2 * t) = y;
        else if (a.out_f32) *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at + 8 * c) = y;
        else *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(a.out) + at + 8 * c) = __floats2bfloat162_rn(y.x, y.y);
      }
      if (t == 0) {
        if (!sg.whole) {
          to[0] = m[x];
          to[1] = l[x];
          to[2] = e;
        } else if (a.lse) {
          a.lse[((a.first_seq + sg.b) * a.heads * a.group + hq) * a.nq + i] =
              l[x] == 0.f ? -INFINITY : (m[x] - kLift + log2f(l[x])) * kLn2;
        }
      }
    }
  }
}

template <int D, bool INT8, bool WIDE>
cudaError_t launch_one(const AttnArgs& a, cudaStream_t st) {
  constexpr int smem = Smem<D, WIDE>::kBytes;
  static_assert(smem * rows_ctas(D) <= 233472 - 1024 * rows_ctas(D), "shared memory plan exceeds an SM's");
  constexpr int grid = kSms * rows_ctas(D);
  static_assert(grid <= kMaxRecs, "CTAs that the merge knows");
  cudaError_t e = cudaFuncSetAttribute(cache8_rows_kernel<D, INT8, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cache8_rows_kernel<D, INT8, WIDE><<<grid, kThreads, smem, st>>>(a);
  count_launch();
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_merge<D>(a, grid, st);
}

template <int D, bool WIDE>
cudaError_t launch_code(bool int8, const AttnArgs& a, cudaStream_t st) {
  return int8 ? launch_one<D, true, WIDE>(a, st) : launch_one<D, false, WIDE>(a, st);
}

}  // namespace

// Up to 64 rows the few-row kernel is the faster: two sequences of 8192 tokens, 8 KV heads, d = 128, fp32: 64 us with 64
// rows against 79 here, d = 64 50 against 54; 4 KV heads of d = 256, bf16 54 against 82. From 256 rows on this one is: 168
// us against 202, 102 against 150, 122 against 162. Between them they cross twice, a tile of 128 rows costing the same
// however full (128 rows 103 against 111, 132 rows 167 against 116).
constexpr int kRowsFrom = 64;
bool rows_supported(int d, bool f32, int rows) { return (f32 || d == 256) && rows > kRowsFrom; }

size_t rows_record_bytes(int d) { return sizeof(float) * kSms * rows_ctas(d) * 2 * kRowsTile * static_cast<size_t>(kRecHead + d); }

cudaError_t launch_rows(int d, bool int8, const AttnArgs& a, cudaStream_t st) {
  if (d == 64) return launch_code<64, true>(int8, a, st);
  if (d == 128) return launch_code<128, true>(int8, a, st);
  return a.q_f32 || a.out_f32 ? launch_code<256, true>(int8, a, st) : launch_code<256, false>(int8, a, st);
}

}  // namespace tq
