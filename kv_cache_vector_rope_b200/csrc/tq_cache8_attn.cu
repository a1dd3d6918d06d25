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
// units in that order are dealt to the CTAs in contiguous ranges of equal cost,
// a stream's start counting as several units, however long or ragged the
// sequences are. A range that ends inside a sequence leaves a partial record
// (m, l, unit, sum) that cache8_combine_kernel merges; a CTA writes at most two of
// them.
//
// Each warp takes groups of 16 keys of its CTA's range and keeps its own
// running (m, l, sum). A group lies in one page; its keys and values come by two
// TMA copies (128-byte swizzle, the cache seen as rows of 128 bytes) into the
// warp's own ring in shared memory, several groups ahead, so the loads never
// wait for the arithmetic and no warp waits for another until the range ends.
// The products run on 16x8x16 half-precision matrix
// instructions with the keys (then the value coordinates) as the 16 rows and
// eight query rows as the columns, which suits the few rows of a step: every
// 8-bit code is exactly a half, and a query row is scaled by a power of two
// into half's range (exact for bf16; fp32 queries and fp32 outputs use two
// half limbs for q and for p). Weights carry the octaves of the value scale over a
// unit of the row's own (Weigh). The contraction index of both products is
// permuted so that a lane's operands are 16 contiguous bytes of the cache.
//
// Up to four rows over int8 codes multiply the bytes as they are (16x8x32): q in
// units of its power of two is four 7-bit limbs, exact to 2^-27 of the largest
// coordinate, two limbs of each of the four rows in a tile's eight columns, so a
// score costs a quarter of the keys' conversions and half the instructions.
//
// Bound by instruction issue beside the memory: unpacking 8-bit codes for the
// matrix unit, softmax and the two products fill 52% of the issue slots and 50%
// of the integer pipe at d = 128. Measured, floor of the cache's bytes in brackets: a
// step of 8 sequences of 32768 keys, 8 KV heads, 4 rows each, d = 128, 101 us (82),
// d = 64 64 us (41); one sequence of 131072 keys 56 us (41); four drafted fp32 rows
// of 32 ragged sequences, 20 KV heads, d = 64, 77 us (40).
#include <cuda.h>

#include "tq_cache8_attn.cuh"

namespace tq {
namespace {

using namespace c8;
using namespace sm100;

constexpr int kAtThreads = 256;
constexpr int kAtWarps = kAtThreads / 32;
constexpr int kAtGrid = kMaxRecs;                    // at most two CTAs per SM
constexpr int kUnit = 64;                            // keys per unit of the split
constexpr int kMinUnits = 2;                         // a CTA takes at least this many units
// What a segment's start and merge cost a CTA beside its keys, in units. Four drafted fp32 rows of 32 ragged sequences,
// 20 KV heads, d = 64: 79 us at 8, 77 at 12 and 16, 78 at 24; d = 128: one sequence of 131072 keys 56.4 at 8 and 12, 55.8
// at 24, 16 rows of 32 ragged sequences 105, 102 and 110; 4 heads of d = 256, 32 ragged sequences: 66 at 4, 62 at 8, 60
// at 14, 66 at 24.
constexpr int lead_of(int d) { return d == 64 ? 16 : d == 128 ? 8 : 14; }
constexpr int kSlice = 512;                          // sequences of one launch
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same into fresh sums.
__device__ __forceinline__ void mma_f16_new(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// D = A B (+ C) of signed bytes, 16x8x32, in whole numbers.
__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_s8_new(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                           uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(0));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Per head dim: 16-byte chunks a lane reads of each of its two keys, 4-byte
// words it reads of each of its four values, groups in a warp's ring (three of
// 4 KB for each of 16 warps are 192 KB at d = 128), groups it takes together
// with one query tile (d = 64: two, which share the wait, the look at the
// maximum and the value sums: 8 x 32768 keys 69 -> 63 us; with two query tiles
// their operands no longer fit the registers, 91 -> 100 us) and CTAs per SM.
template <int D>
struct Plan;
template <>
struct Plan<64> {
  static constexpr int kK = 1, kVWords = 2, kGroups = 6, kPair = 2, kCtas = 2;
};
template <>
struct Plan<128> {
  static constexpr int kK = 2, kVWords = 4, kGroups = 3, kPair = 1, kCtas = 2;
};
template <>
struct Plan<256> {
  static constexpr int kK = 4, kVWords = 8, kGroups = 3, kPair = 1, kCtas = 1;
};

// Dynamic shared memory: the warps' rings first (1024-byte aligned).
// ROWS: query rows; QN: 8-byte query operands per lane.
template <int D, int ROWS, int QN>
struct Smem {
  static constexpr int kHalfStage = 16 * D;          // 16 keys (or values)
  static constexpr int kGroup = 2 * kHalfStage;
  static constexpr int kRing = kGroup * Plan<D>::kGroups;
  static constexpr int kRows = ROWS;
  // uint2 [2][QN][32], the query operands of this segment and the next; float4
  // [warps][2][32], a piece of the value sums, over this segment's and what
  // lies between the two, while the warps are merged.
  static constexpr int kOffQ = kAtWarps * kRing;
  static constexpr int kQBytes = QN * 32 * 8, kAccBytes = kAtWarps * 2 * 32 * 16;
  static constexpr int kBetween = kQBytes > kAccBytes ? 0 : kAccBytes - kQBytes;
  static constexpr int kOffM = kOffQ + 2 * kQBytes + kBetween;
  static constexpr int kOffL = kOffM + 4 * kAtWarps * kRows;
  static constexpr int kOffUnit = kOffL + 4 * kAtWarps * kRows;  // bytes [kRows][warps]: octaves of the sums' units, and 128
  static constexpr int kOffTop = kOffUnit + kAtWarps * kRows;    // float [3][kRows]: merged maximum, sum and unit
  static constexpr int kOffRow = kOffTop + 12 * kRows;           // [2] per row: score factor, first key, end
  static constexpr int kOffBar = kOffRow + 24 * kRows;
  static constexpr int kOffPart = kOffBar + 8 * kAtWarps * Plan<D>::kGroups;
  static constexpr int kOffCum = kOffPart + 4 * kAtWarps;
  static constexpr int kBytes = kOffCum + 4 * (kSlice + 1) + 1024;   // and room to align the base
};

// Where byte `at` of a half stage lies: 16-byte chunk c of 128-byte row r sits at chunk c ^ (r % 8).
__host__ __device__ constexpr int swizzled(int at) { return at ^ ((at >> 3) & 0x70); }
// The swizzle is linear in the bits of an offset: from the place of `a` that of a + b, with no bit in common, is one
// XOR and one addition away. The half stages lie on 1024 bytes.
__device__ __forceinline__ uint32_t swizzled_on(uint32_t place, int b) {
  return (place ^ (swizzled(b) & 1023)) + (swizzled(b) & ~1023);
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 x;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at) : "memory");
  return x;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 x;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(at) : "memory");
  return x;
}

// NT: query tiles a CTA handles together, of eight rows, or of four with two
// limbs each (QUAD). QF / OF: fp32 queries / outputs, two half limbs each.
template <int D, bool QUAD, int NT, bool QF>
struct Tiling {
  static constexpr int kTile = QUAD ? 4 : 8;         // rows of a tile
  static constexpr int kCols = QUAD ? 1 : 2;         // rows of a tile that a lane's columns belong to
  static constexpr int kRows = kTile * NT;
  static constexpr int kOps = QUAD || !QF ? D / 16 : D / 8;      // query operands per tile: k-steps x limbs (x pairs of limbs)
  using Plan = Smem<D, kRows, NT * kOps>;
};
template <int D, bool INT8, bool QUAD, int NT, bool QF, bool OF>
__global__ void __launch_bounds__(kAtThreads, Plan<D>::kCtas)
    cache8_attn_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, AttnArgs a) {
  constexpr int KC = Plan<D>::kK, KS = KC * 4;       // 16-byte chunks, k-steps of the score product
  constexpr int VW = Plan<D>::kVWords, MT = VW * 2;  // words per value row of a lane, 16-row tiles of the value product
  constexpr int G = NT == 1 ? Plan<D>::kPair : 1;    // groups a warp takes together
  constexpr int ST = Plan<D>::kGroups / G;           // such turns in its ring
  constexpr int kStep = 16 * G * kAtWarps;           // keys the warps take together
  static_assert(INT8 || !QUAD, "byte products are for int8 codes");
  using T = Tiling<D, QUAD, NT, QF>;
  constexpr int QL = QF ? 2 : 1, QN = T::kOps, NJ = T::kCols, kTile = T::kTile, kRows = T::kRows;
  constexpr int NE = 2 * NJ;                         // scores of a lane per tile: keys g and g + 8
  constexpr bool kQRegs = NT * QN <= 8;              // few enough to hold in registers
  constexpr uint32_t kMagnitude = INT8 ? 0xffffffffu : 0x7f7f7f7fu;      // the bits that say whether a code is zero
  using L = typename T::Plan;
  constexpr int kStage = G * L::kGroup;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
  float* sm_m = reinterpret_cast<float*>(smem + L::kOffM);
  float* sm_l = reinterpret_cast<float*>(smem + L::kOffL);
  unsigned char* sm_unit = smem + L::kOffUnit;       // octaves within [-127, 122]
  float* sm_top = reinterpret_cast<float*>(smem + L::kOffTop);
  int* cum = reinterpret_cast<int*>(smem + L::kOffCum);
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  unsigned char* ring = smem + w * L::kRing;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::kOffBar) + w * ST;
  const uint32_t k_first = smem_u32(ring) + swizzled(g * D + 16 * t);
  const uint32_t v_first = smem_u32(ring) + L::kHalfStage + swizzled(2 * t * D + (VW == 2 ? 8 : 16) * g);
  if (lane == 0) {
    for (int s = 0; s < ST; ++s) mbar_init(bar + s, 1);
    mbar_fence_init();
  }
  int per = 1, u0 = 0, u1 = 1;                       // alone: one segment
  if (!a.alone) {
    scan_counts<kAtThreads>(cum, reinterpret_cast<int*>(smem + L::kOffPart), a.batch, [&](int b) {
      return head_units(a, seq_len(a, b, blockIdx.x == 0)) * a.heads;
    });
    if (tid == 0) a.cuts[blockIdx.x].n = 0;
    let_next_start();
    const int total = cum[a.batch];
    per = units_per_cta(a, total, gridDim.x);
    u0 = min(static_cast<int>(blockIdx.x) * per, total);
    u1 = min(u0 + per, total);
  }
  int at = 0;                                        // ring stage of the next group
  uint32_t phase = 0;                                // of stage `at`
  bool dead = false;                                 // a wait gave up
  // The segment at hand and what this warp has on its way of it: `turns` times G groups at k0, k0 + kStep, ..., of
  // which `issued` are being copied. Pages and scales of 32 groups at a time, one per lane, the next 32 loaded ahead.
  Seg sg{};
  int u = u0, next = u0, k0 = 0, turns = 0, issued = 0, pg = 0, pg_next = 0;
  float sc_k = 0.f, sc_v = 0.f;                      // the value scale as its octaves
  const auto key_of = [&](int x) { return k0 + x / G * kStep + x % G * 16; };
  const auto load_page = [&](int x) {
    return key_of(x) < sg.t1 ? static_cast<int>(page_of(a, sg.b, key_of(x) >> a.block_log2)) : -1;
  };
  const auto ok = [&](int page) { return page >= 0 && page < a.n_blocks; };
  const auto load_scale = [&](const float* p, int page) {
    return ok(page) ? p[static_cast<int64_t>(page) * a.heads + sg.kv] : 0.f;
  };
  const auto step = [&](int& st) { return ++st == ST ? (st = 0, true) : false; };
  const auto issue = [&](int i, int rel, int st) {   // turn i, whose groups' pages are lanes G rel... of pg, then pg_next
    int page[G];
#pragma unroll
    for (int x = 0; x < G; ++x) page[x] = __shfl_sync(0xffffffffu, G * rel < 32 ? pg : pg_next, (G * rel + x) & 31);
    if (lane == 0) {
      mbar_expect_tx(bar + st, key_of(G * i + G - 1) < sg.t1 ? kStage : L::kGroup);
#pragma unroll
      for (int x = 0; x < G; ++x) {
        const int key = key_of(G * i + x);
        if (x > 0 && key >= sg.t1) break;
        // A bad page's group is masked; page 0 is copied in its place.
        const int64_t ph = static_cast<int64_t>(ok(page[x]) ? page[x] : 0) * a.heads + sg.kv;
        const int row = static_cast<int>((ph * a.block + (key & (a.block - 1))) * D / 128);
        unsigned char* to = ring + st * kStage + x * L::kGroup;
        tma_load_2d(to, &kmap, bar + st, 0, row);
        tma_load_2d(to + L::kHalfStage, &vmap, bar + st, 0, row);
      }
    }
  };
  // The next segment with keys, if the range has one: its first groups set out.
  const auto open = [&] {
    for (u = next; u < u1; u = next) {
      if (a.alone) sg = seg_alone(a, blockIdx.x), next = u1;
      else if (u == u0) sg = seg_at(a, cum, u, u1, &next);
      else seg_after(a, cum, sg, u, u1, &next);
      if (sg.t1 > sg.t0) break;
    }
    if (u >= u1) return;
    k0 = sg.t0 + 16 * G * w;
    turns = sg.t1 > k0 ? (sg.t1 - k0 + kStep - 1) / kStep : 0;
    pg = load_page(lane);
    pg_next = load_page(32 + lane);
    issued = 0;
    if (!dead)
      for (int st = at; issued < ST && issued < turns; ++issued) {
        issue(issued, issued, st);
        step(st);
      }
    sc_k = load_scale(a.ks, pg);
    sc_v = octaves(load_scale(a.vs, pg));
  };
  // Queries of the segment at hand, for buffer `buf`: the last NT warps, which have the fewest keys, prepare a tile's
  // operands each; lane (g, t) holds column g's coordinates of its chunks.
  const auto q_of = [&](int buf) { return reinterpret_cast<uint2*>(smem + L::kOffQ + buf * (L::kQBytes + L::kBetween)); };
  const auto rows_at = [&](int buf) { return reinterpret_cast<float*>(smem + L::kOffRow) + buf * 3 * kRows; };
  const auto prepare = [&](int buf) {
    if (w < kAtWarps - NT) return;
    uint2* sm_q = q_of(buf);
    float* sm_cq = rows_at(buf);
    int* sm_lo = reinterpret_cast<int*>(sm_cq + kRows);
    int* sm_hi = sm_lo + kRows;
    const int nt = w - (kAtWarps - NT), row = nt * kTile + (QUAD ? g >> 1 : g), r = sg.rt * kRows + row;
    const bool live = r < a.rows;
    const int i = live ? a.group_div.of(r) : 0, hq = sg.kv * a.group + (live ? r - i * a.group : 0);
    const int64_t base = (a.first_seq + sg.b) * a.q_bs + hq * a.q_hs + i * a.q_rs;
    float x[KC][16];
    float amax = 0.f;
    bool finite = true;
#pragma unroll
    for (int c = 0; c < KC; ++c) {
      if (live) load_q16<QF>(a.q, base + 16 * (t + 4 * c), x[c]);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if (!live) x[c][e] = 0.f;
        amax = fmaxf(amax, fabsf(x[c][e]));
        finite &= fabsf(x[c][e]) < INFINITY;
      }
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // Times a power of two: the largest coordinate lands in [2^14, 2^15), or for limbs of bytes in [2^5, 2^6).
    constexpr int kTop = QUAD ? 5 : 14;
    const int E = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -100);
    const float up = __uint_as_float(static_cast<uint32_t>(kTop - min(E, 127) + 127) << 23);
#pragma unroll
    for (int c = 0; c < KC; ++c)
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        float* y = x[c] + 4 * s;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] *= up;
        if constexpr (QUAD) {
          // y = l0 + l1 / 2^7 + l2 / 2^14 + l3 / 2^21: column g takes limbs g % 2 and 2 + g % 2 of its row.
          uint32_t limb[4] = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float z = rintf(y[e]);
              limb[k] |= (static_cast<uint32_t>(static_cast<int>(z)) & 0xffu) << (8 * e);
              y[e] = (y[e] - z) * 128.f;
            }
          uint32_t* to = reinterpret_cast<uint32_t*>(sm_q + (nt * QN + 2 * c + (s >> 1)) * 32 + lane) + (s & 1);
          to[0] = g & 1 ? limb[1] : limb[0];
          to[KS / 2 * 64] = g & 1 ? limb[3] : limb[2];
        } else {
          sm_q[(nt * QN + 4 * c + s) * 32 + lane] = make_uint2(pack_half(y[0], y[1]), pack_half(y[2], y[3]));
          if (QF) {
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] -= __half2float(__float2half_rn(y[e]));
            sm_q[(nt * QN + (QL - 1) * KS + 4 * c + s) * 32 + lane] =
                make_uint2(pack_half(y[0], y[1]), pack_half(y[2], y[3]));
          }
        }
      }
    // Bytes cannot carry an infinity or NaN of q: the score factor does.
    finite = __shfl_xor_sync(0xffffffffu, finite, 1) && finite;
    finite = __shfl_xor_sync(0xffffffffu, finite, 2) && finite;
    if (t == 0 && (!QUAD || !(g & 1))) {
      const int end = live ? row_hi(a, sg.n, i) : 0;
      sm_cq[row] = QUAD && !finite ? __uint_as_float(0x7fffffffu) : a.scale2 / up * (QUAD ? 1.f / 128.f : 1.f);
      sm_hi[row] = end;
      sm_lo[row] = row_lo(a, end);
    }
  };
  open();
  if (a.alone && u >= u1) {                          // no row sees a key
    if (sg.kv == 0) put_empty<D>(a, sg.b * a.row_tiles + sg.rt, w, kAtWarps, 1);
    return;
  }
  if (u < u1) prepare(0);
  __syncthreads();
  for (int buf = 0; u < u1; buf ^= 1) {
    float nx_k = 0.f, nx_v = 0.f;
    const uint2* sm_q = q_of(buf);
    const float* sm_cq = rows_at(buf);
    const int* sm_lo = reinterpret_cast<const int*>(sm_cq + kRows);
    const int* sm_hi = sm_lo + kRows;
    const auto row_of = [&](int nt, int j) { return nt * kTile + (QUAD ? t : 2 * t + j); };   // of a lane's columns
    float cq[NT][NJ];
    int lo_max = 0, hi_min = 0x7fffffff;             // keys in [lo_max, hi_min) are seen by every row
    for (int r = 0; r < kRows && sg.rt * kRows + r < a.rows; ++r) {
      lo_max = max(lo_max, sm_lo[r]);
      hi_min = min(hi_min, sm_hi[r]);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < NJ; ++j) cq[nt][j] = sm_cq[row_of(nt, j)];
    uint2 qr[kQRegs ? NT * QN : 1];
    if (kQRegs) {
#pragma unroll
      for (int x = 0; x < NT * QN; ++x) qr[x] = sm_q[x * 32 + lane];
    }
    float acc[NT][MT][4];
    float l[NT][NJ];
    // The rows' m and e, and what follows from them: two tiles' do not fit the registers and lie where the warp's maxima
    // and sums go at the end (twelve rows over 8 x 32768 keys: 149 us in registers).
    constexpr bool kHold = NT == 1;
    float mh[kHold ? NT : 1][kHold ? NJ : 1] = {}, eh[kHold ? NT : 1][kHold ? NJ : 1] = {};
    const auto m_of = [&](int nt, int j) { return kHold ? mh[kHold ? nt : 0][kHold ? j : 0] : sm_m[w * kRows + row_of(nt, j)]; };
    const auto e_of = [&](int nt, int j) { return kHold ? eh[kHold ? nt : 0][kHold ? j : 0] : sm_l[w * kRows + row_of(nt, j)]; };
    const auto set_m = [&](int nt, int j, float x, float y) {
      if (kHold) {
        mh[kHold ? nt : 0][kHold ? j : 0] = x;
        eh[kHold ? nt : 0][kHold ? j : 0] = y;
      } else if (g == 0) {
        sm_m[w * kRows + row_of(nt, j)] = x;
        sm_l[w * kRows + row_of(nt, j)] = y;
      }
    };
    Weigh wg[kHold ? G : 1][kHold ? NT : 1][kHold ? NJ : 1] = {};        // for value scales of 2^lv
    float lv[G] = {};
    const auto weigh_of = [&](int x, int nt, int j) {
      return kHold ? wg[kHold ? x : 0][kHold ? nt : 0][kHold ? j : 0] : weigh(m_of(nt, j), e_of(nt, j), lv[x]);
    };
    const auto weigh_all = [&] {
      if constexpr (kHold) {
#pragma unroll
        for (int x = 0; x < G; ++x)
#pragma unroll
          for (int j = 0; j < NJ; ++j) wg[x][0][j] = weigh(m_of(0, j), e_of(0, j), lv[x]);
      }
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        set_m(nt, j, -INFINITY, -INFINITY);
        l[nt][j] = 0.f;
      }
#pragma unroll
      for (int x = 0; x < MT; ++x) acc[nt][x][0] = acc[nt][x][1] = acc[nt][x][2] = acc[nt][x][3] = 0.f;
    }
    if (!kHold) __syncwarp();
    weigh_all();
    for (int i = 0; i < turns; ++i) {
      constexpr int kBatch = 32 / G;                 // turns of a batch of pages
      const int rel = i % kBatch;
      if (rel == 0 && i > 0) {
        pg = pg_next;
        sc_k = nx_k;
        sc_v = nx_v;
        pg_next = load_page(G * i + 32 + lane);
      }
      if (rel == kBatch / 4) {
        nx_k = load_scale(a.ks, pg_next);
        nx_v = octaves(load_scale(a.vs, pg_next));
      }
      if (!dead && !mbar_wait(bar + at, phase, a.wait_ns)) {
        dead = true;
        if (a.d_status) atomicOr(a.d_status, TQ_DEV_TIMEOUT);
      }
      dead = __any_sync(0xffffffffu, dead);
      if (dead) {                                    // the copies on their way land before the CTA ends
        for (; i < issued; ++i) {
          mbar_wait(bar + at, phase);
          phase ^= step(at) ? 1u : 0u;
        }
        break;
      }
      const int key0 = k0 + i * kStep;               // group x: 16 keys from key0 + 16 x
      float ks[G];
      bool same = true;
      int known[G];                                  // the end of the keys that may be read; 0 with a bad page
#pragma unroll
      for (int x = 0; x < G; ++x) {
        ks[x] = __shfl_sync(0xffffffffu, sc_k, G * rel + x);
        const float to = __shfl_sync(0xffffffffu, sc_v, G * rel + x);
        same &= to == lv[x];
        lv[x] = to;
        const bool good = ok(__shfl_sync(0xffffffffu, pg, G * rel + x));
        known[x] = good ? sg.n : 0;
        if (!good && key0 + 16 * x < sg.t1 && lane == 0 && a.d_status) atomicOr(a.d_status, TQ_DEV_BAD_BLOCK);
      }
      const uint32_t ka = k_first + at * kStage, va = v_first + at * kStage;
      uint32_t vw[G][4][VW];
      const auto values = [&] {
#pragma unroll
        for (int x = 0; x < G; ++x)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int row = (j & 1) + 8 * (j >> 1);
            uint32_t* to = vw[x][j];
            if constexpr (VW == 2) {
              const uint2 y = lds64(swizzled_on(va + x * L::kGroup, row * D));
              to[0] = y.x;
              to[1] = y.y;
            } else {
#pragma unroll
              for (int c = 0; c < VW / 4; ++c) {
                const uint4 y = lds128(swizzled_on(va + x * L::kGroup, row * D + 128 * c));
                to[4 * c] = y.x;
                to[4 * c + 1] = y.y;
                to[4 * c + 2] = y.z;
                to[4 * c + 3] = y.w;
              }
            }
          }
#pragma unroll
        for (int x = 0; x < G; ++x)
          if (key0 + 16 * x + 16 > known[x]) {       // what lies behind the sequence, or in no page, may be any byte
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (key0 + 16 * x + 2 * t + (j & 1) + 8 * (j >> 1) >= known[x])
#pragma unroll
                for (int y = 0; y < VW; ++y) vw[x][j][y] = 0u;
          }
      };
      float s[G][NT][NE];
#pragma unroll
      for (int x = 0; x < G; ++x) {
        uint4 kw[2][KC];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int c = 0; c < KC; ++c) kw[h][c] = lds128(swizzled_on(ka + x * L::kGroup, 8 * h * D + 64 * c));
        if constexpr (QUAD) {
          int c[NT][2][4];
#pragma unroll
          for (int k = 0; k < KS / 2; ++k) {
            const uint32_t* w0 = &kw[0][k / 2].x + 2 * (k % 2);
            const uint32_t* w1 = &kw[1][k / 2].x + 2 * (k % 2);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int at = nt * QN + h * (KS / 2) + k;
                const uint2 b = kQRegs ? qr[at] : sm_q[at * 32 + lane];
                if (k == 0) mma_s8_new(c[nt][h], w0[0], w1[0], w0[1], w1[1], b.x, b.y);
                else mma_s8(c[nt][h], w0[0], w1[0], w0[1], w1[1], b.x, b.y);
              }
          }
          // Of each key the four limbs' sums: exact but for the two conversions (|128 c0 + c1| < 2^29).
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              s[x][nt][e] = fmaf(static_cast<float>(c[nt][1][2 * e] * 128 + c[nt][1][2 * e + 1]), 1.f / 16384.f,
                              static_cast<float>(c[nt][0][2 * e] * 128 + c[nt][0][2 * e + 1]));
        } else {
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const uint32_t w0 = (&kw[0][k / 4].x)[k % 4], w1 = (&kw[1][k / 4].x)[k % 4];
            const uint32_t a0 = two_halves<INT8, false>(w0), a2 = two_halves<INT8, true>(w0);
            const uint32_t a1 = two_halves<INT8, false>(w1), a3 = two_halves<INT8, true>(w1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const int at = nt * QN + k;
              const uint2 b = kQRegs ? qr[at] : sm_q[at * 32 + lane];
              if (QF) {
                // Each step's products are added in fp32: the matrix unit's own sums are cut, not rounded.
                const uint2 b2 = kQRegs ? qr[at + (QL - 1) * KS] : sm_q[(at + (QL - 1) * KS) * 32 + lane];
                float y[4];
                mma_f16_new(y, a0, a1, a2, a3, b2.x, b2.y);
                mma_f16(y, a0, a1, a2, a3, b.x, b.y);
#pragma unroll
                for (int e = 0; e < 4; ++e) s[x][nt][e] = k == 0 ? y[e] : s[x][nt][e] + y[e];
              } else if (k == 0) {
                mma_f16_new(s[x][nt], a0, a1, a2, a3, b.x, b.y);
              } else {
                mma_f16(s[x][nt], a0, a1, a2, a3, b.x, b.y);
              }
            }
          }
        }
      }
      values();                                      // behind the scores: the keys' registers are free
      if (!same) weigh_all();
      bool rise = false;
#pragma unroll
      for (int x = 0; x < G; ++x) {
        const int key1 = key0 + 16 * x;
        const bool full = key1 >= lo_max && key1 + 16 <= min(hi_min, known[x]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float lim[NJ];
#pragma unroll
          for (int j = 0; j < NJ; ++j) lim[j] = weigh_of(x, nt, j).lim;
#pragma unroll
          for (int e = 0; e < NE; ++e) {
            s[x][nt][e] *= cq[nt][e % NJ] * ks[x];
            if (!full) {
              const int key = key1 + g + 8 * (e / NJ), row = row_of(nt, e % NJ);
              if (key < sm_lo[row] || key >= min(sm_hi[row], known[x])) s[x][nt][e] = -INFINITY;
            }
            rise |= s[x][nt][e] > lim[e % NJ];
          }
        }
      }
      if (__any_sync(0xffffffffu, rise)) {
        // Where each lane finds a code in its part of every value that may be read, no key is without one.
        bool plain = true;
#pragma unroll
        for (int x = 0; x < G; ++x) {
          plain &= lv[x] == lv[0];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t any = 0u;
#pragma unroll
            for (int y = 0; y < VW; ++y) any |= vw[x][j][y];
            plain &= (any & kMagnitude) != 0u || key0 + 16 * x + 2 * t + (j & 1) + 8 * (j >> 1) >= known[x];
          }
        }
        plain = __all_sync(0xffffffffu, plain);
        uint32_t none = 0u;                          // bits 2 x + h: the lane's key g + 8 h of group x has no such code
        if (__builtin_expect(!plain, 0)) {
#pragma unroll
          for (int x = 0; x < G; ++x)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t some[2];                        // bit t of some[j]: key 2 t + j + 8 h
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                uint32_t any = 0u;
#pragma unroll
                for (int y = 0; y < VW; ++y) any |= vw[x][2 * h + j][y];
                some[j] = __ballot_sync(0xffffffffu, (any & kMagnitude) != 0u);
                some[j] |= some[j] >> 16;
                some[j] |= some[j] >> 8;
                some[j] |= some[j] >> 4;
              }
              none |= (~(((g & 1) ? some[1] : some[0]) >> (g >> 1)) & 1u) << (2 * x + h);
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float f[NJ];
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            float top = -INFINITY;
#pragma unroll
            for (int x = 0; x < G; ++x) top = fmaxf(top, fmaxf(s[x][nt][j], s[x][nt][j + NJ]));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float m = m_of(nt, j), e = e_of(nt, j), mn = fmaxf(m, rintf(top)), by = below(m, mn);
            float topv = top == -INFINITY ? -INFINITY : below(top, mn) + lv[0];
            if (!plain) {
              topv = -INFINITY;
#pragma unroll
              for (int x = 0; x < G; ++x)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  if (!((none >> (2 * x + h)) & 1) && s[x][nt][j + NJ * h] > -INFINITY)
                    topv = fmaxf(topv, below(s[x][nt][j + NJ * h], mn) + lv[x]);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) topv = fmaxf(topv, __shfl_xor_sync(0xffffffffu, topv, o));
            }
            const float en = next_unit(e, by, topv);
            f[j] = unit_step(m, e, mn, en);
            l[nt][j] *= fast_exp2(by);
            if (!kHold) __syncwarp();
            set_m(nt, j, mn, en);
            // Keys without a value: counted here, then left out.
            if (none != 0u) {
#pragma unroll
              for (int x = 0; x < G; ++x)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  float& y = s[x][nt][j + NJ * h];
                  if (!((none >> (2 * x + h)) & 1) || y == -INFINITY) continue;
                  l[nt][j] += fast_exp2((y - base_of(mn)) + kLift);
                  y = -INFINITY;
                }
            }
          }
#pragma unroll
          for (int x = 0; x < MT; ++x) {
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][x][e] *= f[e % NJ];
          }
        }
        weigh_all();
        if (!kHold) __syncwarp();
      }
      uint32_t ph0[G][NT][2], ph1[G][NT][2];
#pragma unroll
      for (int x = 0; x < G; ++x) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float p[NE];
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const Weigh y = weigh_of(x, nt, j);
            const float base = base_of(m_of(nt, j));
#pragma unroll
            for (int e = j; e < NE; e += NJ) {
              p[e] = fast_exp2((s[x][nt][e] - base) + y.lift);
              l[nt][j] = fmaf(p[e], y.inv, l[nt][j]);
            }
          }
          if constexpr (QUAD) {
            // A row's two columns: the weight and what its half leaves of it.
#pragma unroll
            for (int e = 0; e < 2; ++e)
              ph0[x][nt][e] = transpose8(pack_half(p[e], OF ? (p[e] - __half2float(__float2half_rn(p[e]))) * kLimb : 0.f));
          } else {
            const uint32_t h0 = pack_half(p[0], p[1]), h1 = pack_half(p[2], p[3]);
            ph0[x][nt][0] = transpose8(h0);
            ph0[x][nt][1] = transpose8(h1);
            if (OF) {
              const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&h0));
              const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&h1));
              ph1[x][nt][0] = transpose8(pack_half((p[0] - y.x) * kLimb, (p[1] - y.y) * kLimb));
              ph1[x][nt][1] = transpose8(pack_half((p[2] - z.x) * kLimb, (p[3] - z.y) * kLimb));
            }
          }
        }
      }
#pragma unroll
      for (int c = 0; c < VW; ++c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float y[NT][4], z[NT][4];                    // of the weights' halves, and of their second ones
#pragma unroll
          for (int x = 0; x < G; ++x) {
            // Coordinate pairs of two keys side by side: (key 2t, key 2t + 1) per half pair.
            const uint32_t p = __byte_perm(vw[x][0][c], vw[x][1][c], h ? 0x7362 : 0x5140);
            const uint32_t q = __byte_perm(vw[x][2][c], vw[x][3][c], h ? 0x7362 : 0x5140);
            const uint32_t a0 = two_halves<INT8, false>(p), a1 = two_halves<INT8, true>(p);
            const uint32_t a2 = two_halves<INT8, false>(q), a3 = two_halves<INT8, true>(q);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (OF) {
                if (x == 0) mma_f16_new(y[nt], a0, a1, a2, a3, ph0[x][nt][0], ph0[x][nt][1]);
                else mma_f16(y[nt], a0, a1, a2, a3, ph0[x][nt][0], ph0[x][nt][1]);
                if (!QUAD) {
                  if (x == 0) mma_f16_new(z[nt], a0, a1, a2, a3, ph1[x][nt][0], ph1[x][nt][1]);
                  else mma_f16(z[nt], a0, a1, a2, a3, ph1[x][nt][0], ph1[x][nt][1]);
                }
              } else {
                mma_f16(acc[nt][2 * c + h], a0, a1, a2, a3, ph0[x][nt][0], ph0[x][nt][1]);
              }
            }
          }
          if (OF) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                acc[nt][2 * c + h][e] += y[nt][e];
                if (!QUAD) acc[nt][2 * c + h][e] = fmaf(z[nt][e], 1.f / kLimb, acc[nt][2 * c + h][e]);
              }
          }
        }
      }
      // Every lane's operands have gone into products: the stage is free. (Right behind the loads, with nothing in
      // between that waits for their data, a copy could overtake them.)
      const int freed = at;
      phase ^= step(at) ? 1u : 0u;
      __syncwarp();
      if (issued < turns) {
        issue(issued, issued - (i - rel), freed);
        ++issued;
      }
    }
    const Seg was = sg;                              // merged while the next segment's first groups are on their way
    const int was_u = u;
    open();
    if (u < u1) prepare(buf ^ 1);
    // Merge the warps: maxima and sums, then the value sums a piece at a time.
    float m[NT][NJ], unit[NT][NJ];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        m[nt][j] = m_of(nt, j);
        unit[nt][j] = unit_of(e_of(nt, j));
      }
    if (!kHold) __syncwarp();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        float x = l[nt][j];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (g == 0) {
          sm_m[w * kRows + row_of(nt, j)] = m[nt][j];
          sm_l[w * kRows + row_of(nt, j)] = x;
          sm_unit[row_of(nt, j) * kAtWarps + w] = static_cast<unsigned char>(__float_as_uint(unit[nt][j] + 12583040.f));
        }
      }
    __syncthreads();
    if (tid < kRows) {
      float M = -INFINITY, sum = 0.f, top = kNoUnit;
#pragma unroll
      for (int k = 0; k < kAtWarps; ++k) M = fmaxf(M, sm_m[k * kRows + tid]);
      const uint2 units = reinterpret_cast<const uint2*>(sm_unit)[tid];
      static_assert(kAtWarps == 8, "a byte for each warp");
#pragma unroll
      for (int k = 0; k < kAtWarps; ++k)
        if (sm_l[k * kRows + tid] != 0.f) {          // also with a NaN in the row, whose maximum is -inf
          const float by = below(sm_m[k * kRows + tid], M);
          sum += sm_l[k * kRows + tid] * fast_exp2(by);
          top = fmaxf(top, by + (__uint_as_float(__byte_perm(k < 4 ? units.x : units.y, 0x4b000000u, 0x7550 + k % 4)) - 8388736.f));
        }
      sm_top[tid] = M;
      sm_top[kRows + tid] = sum;
      sm_top[2 * kRows + tid] = rintf(top);
    }
    __syncthreads();
    float f[NT][NJ];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int row = row_of(nt, j);
        f[nt][j] = m[nt][j] == -INFINITY
                       ? 0.f
                       : fast_exp2(below(m[nt][j], sm_top[row]) + (unit[nt][j] - sm_top[2 * kRows + row]));
      }
    const bool second = was.head && was_u != u0;     // the record's slot
    if (tid == 0 && was.head && !was.whole) a.cuts[blockIdx.x] = cut_of(a, was, second, per);
    float* rec = a.rec + (static_cast<int64_t>(blockIdx.x) * 2 + (second ? 1 : 0)) * kRows * (kRecHead + D);
    constexpr int kPieces = 4 / NJ, kVals = 2 * NJ;  // 16-row tiles at a time, and values of a lane in each
    static_assert(NT * MT % kPieces == 0, "whole pieces");
    float* sums = reinterpret_cast<float*>(smem + L::kOffQ + buf * L::kQBytes);
#pragma unroll
    for (int p0 = 0; p0 < NT * MT; p0 += kPieces) {
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        const int nt = (p0 + p) / MT, x = (p0 + p) % MT;
        float* to = sums + ((w * kPieces + p) * 32 + lane) * kVals;
        if constexpr (QUAD)                          // the two limbs' columns are one row's
          *reinterpret_cast<float2*>(to) = make_float2(fmaf(acc[nt][x][1], 1.f / kLimb, acc[nt][x][0]) * f[nt][0],
                                                       fmaf(acc[nt][x][3], 1.f / kLimb, acc[nt][x][2]) * f[nt][0]);
        else
          *reinterpret_cast<float4*>(to) = make_float4(acc[nt][x][0] * f[nt][0], acc[nt][x][1] * f[nt][NJ - 1],
                                                       acc[nt][x][2] * f[nt][0], acc[nt][x][3] * f[nt][NJ - 1]);
      }
      __syncthreads();
      {
        // One value per thread: coordinate + c / NJ, the c % NJ-th of its lane's rows.
        const int p = tid / (32 * kVals), ln = tid % (32 * kVals) / kVals, c = tid % kVals;
        float val = 0.f;
#pragma unroll
        for (int k = 0; k < kAtWarps; ++k) val += sums[((k * kPieces + p) * 32 + ln) * kVals + c];
        const int nt = (p0 + p) / MT, x = (p0 + p) % MT;
        const int wd = x >> 1, gg = ln >> 2;
        const int dim = (VW >= 4 ? 16 * (gg + 8 * (wd / 4)) + 4 * (wd % 4) : 8 * gg + 4 * wd) + 2 * (x & 1) + c / NJ;
        const int row = nt * kTile + (QUAD ? ln & 3 : 2 * (ln & 3) + c % NJ), r = was.rt * kRows + row;
        if (r < a.rows) {
          const float M = sm_top[row], sum = sm_top[kRows + row], octaves = sm_top[2 * kRows + row];
          if (was.whole) {
            const int i = a.group_div.of(r), hq = was.kv * a.group + r - i * a.group;
            const int64_t at = (a.first_seq + was.b) * a.o_bs + hq * a.o_hs + i * a.o_rs + dim;
            const float o = sum == 0.f ? 0.f : val / sum * pow2_whole(octaves);
            if (OF) static_cast<float*>(a.out)[at] = o;
            else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(o);
            if (a.lse && dim == 0)
              a.lse[((a.first_seq + was.b) * a.heads * a.group + hq) * a.nq + i] =
                  sum == 0.f ? -INFINITY : (M - kLift + log2f(sum)) * kLn2;
          } else {
            rec[row * (kRecHead + D) + kRecHead + dim] = val;
            if (dim == 0) {
              rec[row * (kRecHead + D)] = M;
              rec[row * (kRecHead + D) + 1] = sum;
              rec[row * (kRecHead + D) + 2] = octaves;
            }
          }
        }
      }
      __syncthreads();
    }
  }
}

struct Maps {
  CUtensorMap k, v;
};

// The code arrays as rows of 128 bytes, copied in boxes of one group of 16 keys.
tq_status encode_maps(const tq_cache8* c, Maps* m, const char* what) {
  const EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return fail(TQ_ERR_CUDA, "%s: cuTensorMapEncodeTiled not found", what);
  const cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(c->n_blocks) * c->heads * c->block * c->d / 128};
  const cuuint64_t strides[1] = {128};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(16 * c->d / 128)};
  const cuuint32_t estr[2] = {1, 1};
  if (dims[1] > 0x7fffffffu) return fail(TQ_ERR_UNSUPPORTED, "%s: cache beyond 2^38 bytes of keys", what);
  CUtensorMap* maps[2] = {&m->k, &m->v};
  uint8_t* base[2] = {c->k, c->v};
  for (int i = 0; i < 2; ++i) {
    const CUresult r = fn(maps[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base[i], dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(TQ_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed (%d)", what, static_cast<int>(r));
  }
  return TQ_OK;
}

template <int D, bool INT8, bool QUAD, int NT, bool QF, bool OF>
cudaError_t launch_attn(const Maps& maps, const AttnArgs& a, cudaStream_t st) {
  constexpr int smem = Tiling<D, QUAD, NT, QF>::Plan::kBytes;
  static_assert(smem * Plan<D>::kCtas <= 233472 - 1024 * Plan<D>::kCtas, "shared memory plan exceeds an SM's");
  auto kernel = cache8_attn_kernel<D, INT8, QUAD, NT, QF, OF>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  constexpr int grid = kSms * Plan<D>::kCtas;         // every CTA resident at once
  static_assert(grid <= kAtGrid, "the workspace holds kAtGrid CTAs' records");
  kernel<<<a.alone ? a.batch * a.heads * a.row_tiles : grid, kAtThreads, smem, st>>>(maps.k, maps.v, a);
  count_launch();
  e = cudaGetLastError();
  return e != cudaSuccess || a.alone ? e : launch_combine<D, OF>(a, grid, st);
}

template <int D, bool INT8, bool QUAD, int NT>
cudaError_t launch_types(bool qf, bool of, const Maps& m, const AttnArgs& a, cudaStream_t st) {
  if (qf && of) return launch_attn<D, INT8, QUAD, NT, true, true>(m, a, st);
  if (qf) return launch_attn<D, INT8, QUAD, NT, true, false>(m, a, st);
  if (of) return launch_attn<D, INT8, QUAD, NT, false, true>(m, a, st);
  return launch_attn<D, INT8, QUAD, NT, false, false>(m, a, st);
}

// Query rows a CTA takes together: 16 where a KV head has more than 8 and their
// sums fit the registers (d up to 128, not fp32; twelve rows over 8 x 32768 keys,
// d = 128: 141 us, by eights 190; d = 64 98, 116). Over int8 codes up to four rows
// are one tile of byte products with two of q's limbs a column where that is the
// faster: one step of a decode of 8 x 32768 keys took, against the half products'
// eight columns, 62 against 71 us (d = 64), and with fp32 queries 64 against 84 (d =
// 64), 104 against 117 (d = 128), 108 against 112 (d = 256); with bf16 queries 102
// against 97 (d = 128) and 109 against 98 (d = 256), so there they stay away, as they
// do from 5 to 8 rows (two such tiles: 125 against 98 us).
int rows_of(int d, int rows, bool qf, bool of, bool int8) {
  if (int8 && rows <= 4 && (qf || d == 64)) return 4;
  return rows > 8 && d <= 128 && !qf && !of ? 16 : 8;
}

// Whether each CTA takes one stream by itself, without the lengths' sums before it and the merge behind: where there are
// a few streams per CTA at most and none can be long. One token, d = 128, 8 streams of 100 keys: 6.9 us against 9.6 split
// over the CTAs, of 400 9.7 against 10.6, of 777 13.0 against 10.8; 240 streams of 1000 keys 21 against 27; 512 of 100 14
// against 18, of 1000 39 against 42; 2048 streams of 60 keys 46 against 44.
bool streams_alone(int d, int64_t streams, int64_t most_keys) {
  const int ctas = kSms * (d == 256 ? Plan<256>::kCtas : Plan<128>::kCtas);
  return streams <= 4 * ctas && most_keys * d <= (2 * streams > ctas ? 1024 : 512) * 128;
}

template <int D>
cudaError_t launch_few(bool int8, int tile, bool qf, bool of, const Maps& m, const AttnArgs& a, cudaStream_t st) {
  if (tile == 4) {
    if constexpr (D == 64) return launch_types<D, true, true, 1>(qf, of, m, a, st);
    else return of ? launch_attn<D, true, true, 1, true, true>(m, a, st) : launch_attn<D, true, true, 1, true, false>(m, a, st);
  }
  if constexpr (D <= 128)
    if (tile == 16)                                  // bf16 queries and outputs
      return int8 ? launch_attn<D, true, false, 2, false, false>(m, a, st) : launch_attn<D, false, false, 2, false, false>(m, a, st);
  return int8 ? launch_types<D, true, false, 1>(qf, of, m, a, st) : launch_types<D, false, false, 1>(qf, of, m, a, st);
}

int log2_of(int x) {
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

constexpr size_t kCutBytes = (sizeof(CutInfo) * kMaxRecs + 255) / 256 * 256;

size_t attn_workspace(int d, int64_t rows) {
  const size_t few = sizeof(float) * kAtGrid * 2 * 16 * static_cast<size_t>(kRecHead + d);
  const size_t chunk = chunk_supported(d, false, static_cast<int>(rows)) ? chunk_record_bytes(d) : 0;
  const size_t wide = rows_supported(d, true, static_cast<int>(rows)) ? rows_record_bytes(d) : 0;
  const size_t many = chunk > wide ? chunk : wide;
  return kCutBytes + (few > many ? few : many);
}

}  // namespace
}  // namespace tq

extern "C" size_t tq_cache8_attention_workspace_bytes(const tq_cache8* cache, int32_t batch, int32_t hq, int32_t nq) {
  if (tq::check_cache8(cache, "tq_cache8_attention_workspace_bytes") != TQ_OK || batch < 0 || hq < 1 || nq < 1 ||
      hq % cache->heads != 0 || static_cast<int64_t>(hq) * nq > 0x3fffffff)
    return 0;
  return tq::attn_workspace(cache->d, static_cast<int64_t>(hq / cache->heads) * nq);
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
  if (table_stride * cache->block > (1 << 30))       // keys ahead of the last one are counted in 32 bits
    return fail(TQ_ERR_UNSUPPORTED, "%s: sequences beyond 2^30 tokens", what);
  if (!block_table && table_stride * batch > cache->n_blocks)
    return fail(TQ_ERR_INVALID_ARG, "%s: without a block table the cache needs batch * table_stride blocks", what);
  if (!aligned(q, 16) || !aligned(out, 16) || !stride_ok(batch, q_batch_stride, 8) || !stride_ok(hq, q_head_stride, 8) ||
      !stride_ok(nq, q_row_stride, 8) || !stride_ok(batch, out_batch_stride, 8) || !stride_ok(hq, out_head_stride, 8) ||
      !stride_ok(nq, out_row_stride, 8))
    return fail(TQ_ERR_INVALID_ARG, "%s: q and out must be 16-byte aligned, strides multiples of 8 elements, not negative",
                what);
  RowDim out_dims[3] = {{batch, out_batch_stride}, {hq, out_head_stride}, {nq, out_row_stride}};
  if (rows_overlap(out_dims, d))
    return fail(TQ_ERR_INVALID_ARG, "%s: the strides of out make rows overlap", what);
  if (d != 64 && d != 128 && d != 256)
    return fail(TQ_ERR_UNSUPPORTED, "%s: d=%d not built (64, 128, 256)", what, d);
  const int group = hq / cache->heads, rows = group * nq;
  const bool qf = q_dtype == TQ_F32, of = out_dtype == TQ_F32;
  const bool chunk = chunk_supported(d, qf || of, rows), wide = rows_supported(d, qf || of, rows);
  const int tile = chunk ? kChunkRows : wide ? kRowsTile : rows_of(d, rows, qf, of, cache->code == TQ_INT8);
  const int row_tiles = (rows + tile - 1) / tile;
  const int unit = chunk ? kChunkUnit : wide ? kRowsUnit : kUnit, lead = chunk ? kChunkLead : wide ? kRowsLead : lead_of(d);
  const int most = chunk ? kChunkSlice : wide ? kRowsSlice : kSlice;
  // Units of one launch stay within 2^30: batches are cut into slices.
  const int64_t per_head = ((table_stride * cache->block + unit - 1) / unit + 1 + lead) * row_tiles, per_seq = per_head * cache->heads;
  if (per_head > (1 << 30) || per_seq > (1 << 30))
    return fail(TQ_ERR_UNSUPPORTED, "%s: KV heads x query rows x capacity of one sequence too large", what);
  if (!workspace || workspace_bytes < attn_workspace(d, rows))
    return fail(TQ_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", what, workspace_bytes, attn_workspace(d, rows));
  if (!aligned(workspace, 256)) return fail(TQ_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", what);
  int64_t slice = (1 << 30) / per_seq;
  if (slice > most) slice = most;
  const int64_t streams = static_cast<int64_t>(batch) * cache->heads * row_tiles;
  const bool alone = !chunk && !wide && streams_alone(d, streams, table_stride * cache->block);
  AttnArgs a{Div(cache->heads), Div(group), Div(row_tiles), cache->heads, cache->block, 0, log2_of(cache->block), cache->n_blocks, cache->k, cache->v, cache->k_scale, cache->v_scale, q, qf, of,
             q_batch_stride, q_head_stride, q_row_stride, group, nq, rows, tile, row_tiles, log2_of(unit), chunk ? kChunkMinUnits : wide ? kRowsMinUnits : kMinUnits,
             lead,
             nullptr, nullptr, table_stride, 0,
             causal ? 1 : 0, window, alone, scale * kLog2e, out, out_batch_stride, out_head_stride, out_row_stride, lse_out,
             reinterpret_cast<float*>(static_cast<char*>(workspace) + kCutBytes), reinterpret_cast<CutInfo*>(workspace), pipeline_wait_ns(), d_status};
  Maps maps;
  if (!chunk && !wide) {
    st = encode_maps(cache, &maps, what);
    if (st != TQ_OK) return st;
  }
  const bool i8 = cache->code == TQ_INT8;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  for (int64_t b0 = 0; b0 < batch; b0 += slice) {
    a.batch = static_cast<int>(batch - b0 < slice ? batch - b0 : slice);
    a.first_seq = b0;
    a.lens = seq_lens + b0;
    a.table = block_table ? block_table + b0 * table_stride : nullptr;
    cudaError_t e;
    if (chunk) e = launch_chunk(d, i8, a, s);
    else if (wide) e = launch_rows(d, i8, a, s);
    else if (d == 64) e = launch_few<64>(i8, tile, qf, of, maps, a, s);
    else if (d == 128) e = launch_few<128>(i8, tile, qf, of, maps, a, s);
    else e = launch_few<256>(i8, tile, qf, of, maps, a, s);
    if (e != cudaSuccess) return fail(TQ_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
  }
  return TQ_OK;
}
