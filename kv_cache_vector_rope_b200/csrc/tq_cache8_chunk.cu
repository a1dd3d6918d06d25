// tq_cache8_attention for many query rows: a chunk of a prompt over the 8-bit
// cache it extends (bf16 queries and outputs, d 64 or 128).
//
// The formulas are those of tq_cache8_attn.cu. With hundreds of rows per KV head
// the products bound the call, so they run on the tensor cores' tcgen05 path: a
// CTA takes 256 rows (two query tiles of 128) and walks 128 keys at a time,
//   S = Q K^T   both operands in shared memory, S (128 x 128 fp32) in tensor memory,
//   O += P V    P (halves) in tensor memory over S, O (128 x d fp32) in tensor memory.
// Two query tiles alternate, and each takes the 128 keys in two halves: while the
// weights of one half are formed, the values of the half before and the scores
// of the half after run, so that neither side waits for the other. Warps 0-3 and 4-7 form weights (one row per thread), warps 8-11
// turn codes into halves, warp 12 issues the products, warp 13 copies codes in
// (a bulk copy per 16 keys, which lie in one page) and looks pages and scales up.
//
// Codes become halves once per CTA for all 256 rows; an 8-bit code is exactly a
// half. The scales stay out of the products: a group's key scale goes into the
// factor of its scores, its value scale into the exponent of its weights, over a
// unit of the row's own (Weigh), which rescales O where it moves. Queries are
// scaled by a power of two into half's range (exact), weights are rounded to
// halves (2^-11).
//
// Bound by the wait from a half's weights to its next scores (values, scores,
// two looks at barriers: about 2100 cycles, of which the other half's weights
// cover 1400) beside shared memory (about 3000 of 4700 cycles a step). Measured:
// 1024 tokens of two sequences of 8192, 8 KV heads of 4 query heads, d = 128,
// 296 us (the products alone 158 at the library's rate), d = 64 260 us; a prompt
// of 4 x 2048 tokens, d = 128, 248 us.
#include "tq_cache8_attn.cuh"

namespace tq {
namespace {

using namespace c8;
using namespace sm100;

constexpr int kThreads = 512;                        // four warpgroups: weights, weights, codes, products
constexpr int kTile = kChunkUnit;                    // keys per step
static_assert(kTile == 128 && kChunkRows == 256, "tiles of 128 x 128");
constexpr int kRegsWeights = 152, kRegsCodes = 104, kRegsProducts = 104;
static_assert((2 * kRegsWeights + kRegsCodes + kRegsProducts) * 128 <= 128 * kThreads, "within the launch's registers");

// What the copying warp says of a tile: each group of 16 keys' key scale and octaves of the value scale, which groups are
// in the tile (loaded) and which of them lie outside the cache (bad).
struct TileInfo {
  float ks[8], lv[8];
  uint32_t loaded, bad;
};

template <int D>
struct Smem {
  static constexpr int kTileBytes = 128 * D * 2;     // 128 rows of halves: D / 64 atoms of [128][128 B], 128-byte swizzle
  static constexpr int kRawBytes = 128 * D;          // 128 rows of codes
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = 2 * kTileBytes;       // two stages
  static constexpr int kOffV = kOffK + 2 * kTileBytes;
  static constexpr int kOffRawK = kOffV + 2 * kTileBytes;
  static constexpr int kOffRawV = kOffRawK + kRawBytes;
  static constexpr int kOffInfo = kOffRawV + kRawBytes;          // TileInfo [4]
  static constexpr int kOffBar = kOffInfo + 4 * static_cast<int>(sizeof(TileInfo));
  static constexpr int kBars = 27;
  static constexpr int kOffTmem = kOffBar + 8 * (kBars + 1);
  static constexpr int kOffPart = kOffTmem + 16;
  static constexpr int kOffCum = kOffPart + 4 * (kThreads / 32);
  static constexpr int kBytes = kOffCum + 4 * (kChunkSlice + 1) + 1024;
};

enum Bar {
  kKFull = 0, kVFull = 2, kKEmpty = 4, kVEmpty = 6, kQFull = 8, kRawFull = 10, kRawEmpty = 12,   // raw: K, V
  // Query tile q, half h at 2 q + h. One barrier per half and a phase per tile: a wait tells a phase from the one
  // before it only, and up to two halves of one query tile are under way.
  kSFull = 14, kPFull = 18, kPvDone = 22, kDrain = 26
};

// Tensor memory columns: S of tile q, half h at 128 q + 64 h (its first 32 become P), O at 256 + D q.
constexpr uint32_t kTmemCols = 512;

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
// An operand whose rows run along the contraction (V: one row of coordinates
// per key), 128-byte swizzle: groups of 8 keys 1024 B apart, the next 64
// coordinates `next` bytes on.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t next) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(next >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred P;\n\t.reg .b32 r;\n\t"
      "elect.sync r|P, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, P;\n\t}"
      : "=r"(p));
  return p != 0;
}

template <int R>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 16 codes as halves, to two 16-byte chunks of a tile. Lanes of odd
// 64-coordinate atoms store their second chunk first (the caller gives the two
// addresses and words in that order), so that eight lanes meet eight different
// bank groups.
template <bool INT8>
__device__ __forceinline__ void put_codes(uint32_t at0, uint32_t at1, const uint32_t (&w)[4]) {
  uint32_t h[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    h[2 * k] = two_halves<INT8, false>(w[k]);
    h[2 * k + 1] = two_halves<INT8, true>(w[k]);
  }
  sts128(at0, h[0], h[1], h[2], h[3]);
  sts128(at1, h[4], h[5], h[6], h[7]);
}

// Two fp32 operations per instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return r;
}

// Which of 32 keys a row sees: those in [from, end), but of bad groups of 16.
__device__ __forceinline__ uint32_t seen(int from, int end, uint32_t bad) {
  uint32_t see = end >= 32 ? 0xffffffffu : end <= 0 ? 0u : (1u << end) - 1u;
  see &= from >= 32 ? 0u : from <= 0 ? 0xffffffffu : ~((1u << from) - 1u);
  return see & ((bad & 1 ? 0u : 0xffffu) | (bad & 2 ? 0u : 0xffff0000u));
}
// The others' scores become -inf.
__device__ __forceinline__ void hide(uint32_t (&x)[32], uint32_t see) {
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (!(see & (1u << e))) x[e] = 0xff800000u;
}
// Weights 2^(x f + off) of 32 scores, two groups of 16: as halves to 16 columns, and their sums times 2^-d to l.
__device__ __forceinline__ void weights(const uint32_t (&x)[32], const float (&f)[4], const float (&d)[4], float off0, int first,
                                        float& l, uint32_t at) {
  uint32_t pk[16];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float fk = f[first + h], off = d[first + h] + off0;
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int e = 8 * h; e < 8 * h + 8; ++e) {
      float2 y = fma2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), make_float2(fk, fk),
                      make_float2(off, off));
      y.x = fast_exp2(y.x);
      y.y = fast_exp2(y.y);
      sum = add2(sum, y);
      pk[e] = pack_half(y.x, y.y);
    }
    l = fmaf(sum.x + sum.y, pow2_whole(-fminf(d[first + h], 126.f)), l);
  }
  tmem_st16(at, pk);
}
// Largest of 16 scores from x[at] on.
__device__ __forceinline__ float top16(const uint32_t (&x)[32], int at) {
  float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
  for (int e = at; e < at + 16; e += 4) {
    t0 = fmaxf(t0, fmaxf(__uint_as_float(x[e]), __uint_as_float(x[e + 1])));
    t1 = fmaxf(t1, fmaxf(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])));
  }
  return fmaxf(t0, t1);
}

constexpr float kSteep = 4194304.f;
// A query row's maximum of scores, unit of its value sums (Weigh) and sum of weights. Weights are 2^(s f + (lift - m)),
// one rounding each, while scores are below 2^22 octaves. Beyond (steep, for the warp) the product, which is not rounded
// before the sum, may differ from m by more than halves have room for: the scores are made to count from `from` first. by:
// what the last move scaled O by.
struct Row {
  float m, unit, l, from, by;
  bool steep;
};
// A half of a tile: its scores in tensor memory, the factors of their groups, and the keys that the row sees.
struct Half {
  uint32_t at;
  float cq;
  const float *ks, *lv;                              // of the four groups of 16 keys
  uint32_t see0, see1;
  uint2 some;                                        // the keys with a value code that is not zero
};
// Which of 64 keys have a value code that is not zero: their halves lie at `at` in shared memory, D / 64 times [64 keys]
// [128 bytes], 16 KB apart. A lane takes two keys, 16 bytes at a time, lanes side by side in different banks.
template <int D>
__device__ __noinline__ uint2 keys_with_values(uint32_t at) {
  const int lane = threadIdx.x & 31;
  uint32_t any[2] = {0u, 0u};
#pragma unroll
  for (int c = 0; c < D / 8; ++c)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint32_t y[4];
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3])
                   : "r"(at + (c >> 3) * (128 * 128) + (32 * x + lane) * 128 + ((c ^ lane) & 7) * 16)
                   : "memory");
      any[x] |= (y[0] | y[1]) | (y[2] | y[3]);
    }
  return make_uint2(__ballot_sync(0xffffffffu, (any[0] & 0x7fff7fffu) != 0u), __ballot_sync(0xffffffffu, (any[1] & 0x7fff7fffu) != 0u));
}
// The common move's counterpart for a half in which rows see keys without a value, or for steep scores: the weights of such
// keys go into l here and their scores become -inf in tensor memory, where the others count from `from` then, as m does.
// top: the half's largest score as it comes from the products. A call, so that the hot path stays short.
__device__ __noinline__ void move_row(Row* row, const Half& h, float top) {
  Row r = *row;
  const float mn = fmaxf(r.m, rintf(top - r.from)), by = below(r.m, mn);
  const bool far = fabsf(mn) > kSteep && fabsf(mn) < INFINITY;
  const bool steep = __any_sync(0xffffffffu, r.steep || far);
  const float shift = steep && fabsf(mn) < INFINITY ? mn : 0.f;
  float topv = -INFINITY;
  r.l *= fast_exp2(by);
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {
    const uint32_t see = (k < 2 ? h.see0 : h.see1) >> (16 * (k & 1)), some = (k < 2 ? h.some.x : h.some.y) >> (16 * (k & 1));
    const float f = fmaxf(h.cq * h.ks[k], 1.17549435e-38f);
    uint32_t y[16];
    tmem_ld16(h.at + 16 * k, y);
    tmem_ld_wait();
    float top16 = -INFINITY;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float z = __fsub_rn(__fmul_rn(__uint_as_float(y[e]), f), r.from);
      const bool sees = (see >> e) & 1;
      if ((some >> e) & 1) {
        if (sees) top16 = fmaxf(top16, z);
        if (steep) y[e] = __float_as_uint((z - shift) / f);
      } else {
        if (sees) r.l += fast_exp2((z - base_of(mn)) + kLift);
        y[e] = 0xff800000u;
      }
    }
    tmem_st16(h.at + 16 * k, y);
    if (top16 > -INFINITY) topv = fmaxf(topv, below(top16, mn) + h.lv[k]);
  }
  tmem_st_wait();
  const float en = next_unit(r.unit, by, topv);
  r.by = r.unit == -INFINITY ? 1.f : fast_exp2(by + (r.unit - en));
  r.from += shift;
  r.m = mn - shift;
  r.unit = en;
  r.steep = steep;
  *row = r;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

template <int D, bool INT8>
__global__ void __launch_bounds__(kThreads, 1) cache8_chunk_kernel(AttnArgs a) {
  using L = Smem<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
  const uint32_t base = smem_u32(smem);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  TileInfo* info = reinterpret_cast<TileInfo*>(smem + L::kOffInfo);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + L::kOffTmem);
  int* cum = reinterpret_cast<int*>(smem + L::kOffCum);
  const int tid = threadIdx.x, lane = tid & 31;
  const int w = __shfl_sync(0xffffffffu, tid >> 5, 0);   // known to be the same for the warp
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar + kKFull + s, 4);
      mbar_init(bar + kVFull + s, 4);
      mbar_init(bar + kKEmpty + s, 1);
      mbar_init(bar + kVEmpty + s, 1);
      mbar_init(bar + kQFull + s, 4);
      mbar_init(bar + kSFull + 2 * s, 1);
      mbar_init(bar + kSFull + 2 * s + 1, 1);
      mbar_init(bar + kPFull + 2 * s, 4);
      mbar_init(bar + kPFull + 2 * s + 1, 4);
      mbar_init(bar + kPvDone + 2 * s, 1);
      mbar_init(bar + kPvDone + 2 * s + 1, 1);
      mbar_init(bar + kRawFull + s, 1);
      mbar_init(bar + kRawEmpty + s, 4);
    }
    mbar_init(bar + kDrain, 1);
    mbar_fence_init();
  }
  if (w == 12) {
    tmem_alloc(tmem_at, kTmemCols);
    tmem_relinquish();
  }
  scan_counts<kThreads>(cum, reinterpret_cast<int*>(smem + L::kOffPart), a.batch, [&](int b) {
    return head_units(a, seq_len(a, b, blockIdx.x == 0)) * a.heads;
  });
  if (tid == 0) a.cuts[blockIdx.x].n = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_at, 0);
  let_next_start();
  const int total = cum[a.batch];
  const int per = units_per_cta(a, total, gridDim.x);
  const int u0 = min(static_cast<int>(blockIdx.x) * per, total), u1 = min(u0 + per, total);
  // Every role walks the same segments; a wait that gives up ends the role's walk (the others' waits give up too).
  const auto wait = [&](int which, uint32_t parity) {
    if (mbar_wait(bar + which, parity & 1, a.wait_ns)) return true;
    if (a.d_status) atomicOr(a.d_status, TQ_DEV_TIMEOUT);
    return false;
  };
  // One arrival per warp: 32 lanes' arrivals at one barrier queue up for hundreds of cycles.
  const auto arrive = [&](int which) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar + which);
  };
  bool alive = true;
  const auto walk = [&](Seg& sg, int u, int& next) {
    if (u == u0) sg = seg_at(a, cum, u, u1, &next);
    else seg_after(a, cum, sg, u, u1, &next);
  };

  if (w < 8) {
    // ------------------------------------------------------------ weights: one row per thread
    regs_up<kRegsWeights>();
    const int q = w >> 2, wr = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((w & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + 128 * q, o_at = tmem + lanes + 256 + D * q;
    uint32_t tiles_seen = 0;                         // tiles of this query tile so far
    uint32_t walked = 0;                             // tiles of all segments: the info ring's count
    Seg sg;
    for (int u = u0, next; alive && u < u1;) {
      walk(sg, u, next);
      if (sg.t1 <= sg.t0) {
        u = next;
        continue;
      }
      const int key0 = sg.t0 / kTile * kTile, tiles = (sg.t1 - key0 + kTile - 1) / kTile;
      const int r0 = sg.rt * kChunkRows + 128 * q, r = r0 + wr;
      if (r0 >= a.rows) {                            // this query tile has no row
        walked += tiles;
        u = next;
        continue;
      }
      const bool live = r < a.rows;
      const int i = live ? a.group_div.of(r) : 0, hq = sg.kv * a.group + (live ? r - i * a.group : 0);
      float cq;
      {
        // The row's halves of words are bf16: read once, all loads in flight, the maximum by its magnitude bits.
        const uint4* from = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                           (a.first_seq + sg.b) * a.q_bs + hq * a.q_hs + i * a.q_rs);
        uint4 raw[D / 8];
#pragma unroll
        for (int c = 0; c < D / 8; ++c) raw[c] = live ? from[c] : make_uint4(0u, 0u, 0u, 0u);
        uint32_t most = 0u;                          // two 16-bit maxima
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          most = __vmaxu2(most, __vmaxu2(__vmaxu2(raw[c].x & 0x7fff7fffu, raw[c].y & 0x7fff7fffu),
                                         __vmaxu2(raw[c].z & 0x7fff7fffu, raw[c].w & 0x7fff7fffu)));
        }
        const int E = max(static_cast<int>(max(most >> 16, most & 0xffffu) >> 7) - 127, -100);
        float up = __uint_as_float(static_cast<uint32_t>(14 - min(E, 127) + 127) << 23);
        cq = fabsf(a.scale2) / up;
        if (a.scale2 < 0.f) up = -up;                // the factor of the scores stays positive
        const uint32_t row = base + L::kOffQ + q * L::kTileBytes + wr * 128;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint32_t x[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            h[e] = pack_half(__uint_as_float(x[e] << 16) * up, __uint_as_float(x[e] & 0xffff0000u) * up);
          sts128(row + (c >> 3) * (128 * 128) + (((c & 7) ^ (wr & 7)) << 4), h[0], h[1], h[2], h[3]);
        }
        fence_proxy_async_smem();
        arrive(kQFull + q);
      }
      const int hi = live ? row_hi(a, sg.n, i) : 0, lo = row_lo(a, hi);
      // Keys in [lo_max, hi_min) are seen by every row of the tile.
      const int hi_min = row_hi(a, sg.n, a.group_div.of(r0));
      const int lo_max = row_lo(a, row_hi(a, sg.n, a.group_div.of(min(r0 + 127, a.rows - 1))));
      float from = 0.f;                              // what m counts from (steep)
      bool steep = false, again = false;             // again: a half whose m and unit have been moved
      float m = -INFINITY, unit = kNoUnit, l = 0.f;
      for (int j = 0; j < 2 * tiles; ++j) {          // halves of 64 keys
        const int half = j & 1, k0 = key0 + j * 64;
        const uint32_t at = s_at + 64 * half;
        alive = __all_sync(0xffffffffu, wait(kSFull + 2 * q + half, tiles_seen + (j >> 1)));
        if (!alive) break;
        tc_fence_after();
        const uint32_t now = walked + (j >> 1);
        const TileInfo& inf = info[now & 3];
        const uint32_t bad = inf.bad >> (4 * half);
        const bool masked = k0 < lo_max || k0 + 64 > hi_min || (bad & 15);
        uint32_t x0[32], x1[32];
        float f[4], d[4];                            // of the half's four groups of 16 keys: factors, octaves over the unit
        tmem_ld32(at, x0);
        tmem_ld32(at + 32, x1);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          f[k] = fmaxf(cq * inf.ks[4 * half + k], 1.17549435e-38f);
          d[k] = fmaxf(inf.lv[4 * half + k] - unit, -60.f);
        }
        tmem_ld_wait();
        if (masked) {
          hide(x0, seen(lo - k0, hi - k0, bad));
          hide(x1, seen(lo - k0 - 32, hi - k0 - 32, bad >> 2));
        }
        float top[4];
        bool rise = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          top[k] = top16(k < 2 ? x0 : x1, 16 * (k & 1)) * f[k];
          rise |= top[k] > __fadd_rd(unit == kNoUnit ? -INFINITY : m + kSlack, fminf(-d[k], 0.f));
        }
        if (__any_sync(0xffffffffu, (rise || steep) && !again)) {
          // A score is too high for m, or an addend for the unit: both are moved, and what has been summed up, in l and
          // in O, with them.
          const float all = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), mn = fmaxf(m, rintf(all));
          alive = __all_sync(0xffffffffu, wait(kVFull + (now & 1), now >> 1));
          if (!alive) break;
          Half h{at, cq, inf.ks + 4 * half, inf.lv + 4 * half, 0xffffffffu, 0xffffffffu,
                 keys_with_values<D>(base + L::kOffV + (now & 1) * L::kTileBytes + half * 64 * 128)};
          if (masked) {
            h.see0 = seen(lo - k0, hi - k0, bad);
            h.see1 = seen(lo - k0 - 32, hi - k0 - 32, bad >> 2);
          }
          const bool odd = __any_sync(0xffffffffu, steep || (h.see0 & ~h.some.x) || (h.see1 & ~h.some.y) ||
                                                       (fabsf(mn) > kSteep && fabsf(mn) < INFINITY));
          float fo;
          if (odd) {
            Row row{m, unit == kNoUnit ? -INFINITY : unit, l, from, 1.f, steep};
            move_row(&row, h, all);
            steep = row.steep;
            from = row.from;
            l = row.l;
            m = row.m;
            unit = unit_of(row.unit);
            fo = row.by;
          } else {
            const float by = below(m, mn);
            float topv = -INFINITY;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (top[k] > -INFINITY) topv = fmaxf(topv, below(top[k], mn) + inf.lv[4 * half + k]);
            const float en = next_unit(unit == kNoUnit ? -INFINITY : unit, by, topv);
            fo = unit == kNoUnit ? 1.f : fast_exp2(by + (unit - en));
            l *= fast_exp2(by);
            m = mn;
            unit = unit_of(en);
          }
          if (j > 0) {
            // O holds the half before, and with it all others: the products end in order.
            alive = __all_sync(0xffffffffu, wait(kPvDone + 2 * q + (half ^ 1), tiles_seen + ((j - 1) >> 1)));
            if (!alive) break;
            tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < D / 16; ++k) {
              uint32_t o[16];
              tmem_ld16(o_at + 16 * k, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fo);
              tmem_st16(o_at + 16 * k, o);
            }
          }
          if (odd) {                                 // read the scores again
            again = true;
            --j;
            continue;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) d[k] = fmaxf(inf.lv[4 * half + k] - unit, -60.f);
        }
        again = false;
        const float off0 = kLift - base_of(m);
        weights(x0, f, d, off0, 0, l, at);
        weights(x1, f, d, off0, 2, l, at + 16);
        tmem_st_wait();
        tc_fence_before();
        arrive(kPFull + 2 * q + half);
      }
      if (alive) alive = __all_sync(0xffffffffu, wait(kPvDone + 2 * q + 1, tiles_seen + tiles - 1));
      if (!alive) break;
      tiles_seen += tiles;
      walked += tiles;
      tc_fence_after();
      float* rec = a.rec + (static_cast<int64_t>(blockIdx.x) * 2 + (sg.head && u != u0 ? 1 : 0)) * kChunkRows * (kRecHead + D) +
                   static_cast<int64_t>(128 * q + wr) * (kRecHead + D);
      m += from;
      const float by = sg.whole ? (l == 0.f ? 0.f : 1.f / l * pow2_whole(unit)) : 1.f;
      const int64_t at = (a.first_seq + sg.b) * a.o_bs + hq * a.o_hs + i * a.o_rs;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(o_at + 32 * c, o);
        tmem_ld_wait();
        float y[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) y[e] = l == 0.f ? 0.f : __uint_as_float(o[e]) * by;
        if (!live) continue;
        if (sg.whole) {
          __nv_bfloat16* to = static_cast<__nv_bfloat16*>(a.out) + at + 32 * c;
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __nv_bfloat162 z = __floats2bfloat162_rn(y[e + 2 * k], y[e + 2 * k + 1]);
              h[k] = *reinterpret_cast<const uint32_t*>(&z);
            }
            *reinterpret_cast<uint4*>(to + e) = make_uint4(h[0], h[1], h[2], h[3]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(rec + kRecHead + 32 * c + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
        }
      }
      tc_fence_before();                             // O is read before the next segment's first product writes it
      if (live) {
        if (!sg.whole) {
          rec[0] = m;
          rec[1] = l;
          rec[2] = unit;
        } else if (a.lse) {
          a.lse[((a.first_seq + sg.b) * a.heads * a.group + hq) * a.nq + i] =
              l == 0.f ? -INFINITY : (m - kLift + log2f(l)) * kLn2;
        }
      }
      u = next;
    }
  } else if (w < 12) {
    // ------------------------------------------------------------ codes to halves
    regs_down<kRegsCodes>();
    constexpr int kPer = D / 16;                     // 16-byte pieces of a row, and of a thread per tile
    constexpr int kStepRows = 128 / kPer;            // rows that the 128 threads take at a time
    const int ct = tid - 256, row = ct / kPer, c = ct % kPer;
    // A thread's pieces: rows row, row + kStepRows, ... (a multiple of 8 rows on: the same swizzle).
    const bool odd = (c >> 2) & 1;
    const uint32_t to = (c >> 2) * (128 * 128) + row * 128;
    const uint32_t at0 = to + ((((c & 3) * 2 + (odd ? 1 : 0)) ^ (row & 7)) << 4);
    const uint32_t at1 = to + ((((c & 3) * 2 + (odd ? 0 : 1)) ^ (row & 7)) << 4);
    uint32_t it = 0;
    Seg sg;
    for (int u = u0, next; alive && u < u1;) {
      walk(sg, u, next);
      if (sg.t1 <= sg.t0) {
        u = next;
        continue;
      }
      const int key0 = sg.t0 / kTile * kTile, tiles = (sg.t1 - key0 + kTile - 1) / kTile;
      for (int j = 0; alive && j < tiles; ++j, ++it) {
        const uint32_t st = it & 1, parity = (it >> 1) & 1;
        const int left = sg.n - (key0 + j * kTile);  // what lies behind the sequence may be any byte
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          alive = __all_sync(0xffffffffu, wait(kRawFull + kv, it) && wait((kv ? kVEmpty : kKEmpty) + st, parity ^ 1));
          if (!alive) break;
          const uint32_t loaded = info[it & 3].loaded;
          const uint4* raw = reinterpret_cast<const uint4*>(smem + (kv ? L::kOffRawV : L::kOffRawK)) + ct;
          const uint32_t tile = base + (kv ? L::kOffV : L::kOffK) + st * L::kTileBytes;
          const bool clean = left >= kTile && loaded == 0xffu;
          uint4 codes[kPer];
#pragma unroll
          for (int x = 0; x < kPer; ++x) codes[x] = raw[x * 128];
#pragma unroll
          for (int x = 0; x < kPer; ++x) {
            const int group = (x * kStepRows + row) >> 4;
            uint4 y = codes[x];
            if (!clean && (!((loaded >> group) & 1) || x * kStepRows + row >= left)) y = make_uint4(0u, 0u, 0u, 0u);
            const uint32_t words[4] = {odd ? y.z : y.x, odd ? y.w : y.y, odd ? y.x : y.z, odd ? y.y : y.w};
            put_codes<INT8>(tile + at0 + x * kStepRows * 128, tile + at1 + x * kStepRows * 128, words);
          }
          fence_proxy_async_smem();
          __syncwarp();
          // The raw codes are given back only here, when what was read has been used: an arrival right behind the
          // loads, with nothing that waits for their data, let the next copy overwrite codes not yet read.
          if (lane == 0) {
            mbar_arrive(bar + kRawEmpty + kv);
            mbar_arrive(bar + (kv ? kVFull : kKFull) + st);
          }
        }
      }
      u = next;
    }
  } else {
    // ------------------------------------------------------------ products
    regs_down<kRegsProducts>();
    if (w == 12) {
      // The whole warp walks the loop, so that descriptors stay warp-uniform,
      // and one elected lane issues: from a single-lane branch each product
      // took 390 cycles to issue (a chunk of 2 x 1024 tokens 1417 us).
      const bool leader = elect_one();
      constexpr uint32_t kIdS = idesc_f16(128, 64, false), kIdO = idesc_f16(128, D, true);
      const uint64_t q_desc = desc_k_sw128(base + L::kOffQ), k_desc = desc_k_sw128(base + L::kOffK);
      const uint64_t v_desc = desc_mn_sw128(base + L::kOffV, 128 * 128);
      uint32_t it = 0, segs[2] = {0, 0}, done[2] = {0, 0};
      const auto ready = [&](int which, uint32_t parity) { return __all_sync(0xffffffffu, wait(which, parity)); };
      const auto scores = [&](int q, int half, uint32_t st, bool last) {
        const uint64_t qd = q_desc + ((q * L::kTileBytes) >> 4), kd = k_desc + ((st * L::kTileBytes + half * 64 * 128) >> 4);
        if (leader) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            constexpr int kAtom = 128 * 128;
            const uint64_t off = static_cast<uint64_t>(((k >> 2) * kAtom + (k & 3) * 32) >> 4);
            umma_ss(tmem + 128 * q + 64 * half, qd + off, kd + off, kIdS, k != 0);
          }
          umma_commit(bar + kSFull + 2 * q + half);
          if (last) umma_commit(bar + kKEmpty + st);
        }
      };
      const auto values = [&](int q, int half, uint32_t st, bool first, bool last) {
        const uint64_t vd = v_desc + ((st * L::kTileBytes + half * 64 * 128) >> 4);
        if (leader) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_ts(tmem + 256 + D * q, tmem + 128 * q + 64 * half + 8 * k, vd + static_cast<uint64_t>((k * 16 * 128) >> 4),
                    kIdO, !(first && k == 0));
          umma_commit(bar + kPvDone + 2 * q + half);
          if (last) umma_commit(bar + kVEmpty + st);
        }
      };
      Seg sg;
      for (int u = u0, next; alive && u < u1;) {
        walk(sg, u, next);
        if (sg.t1 <= sg.t0) {
          u = next;
          continue;
        }
        const int key0 = sg.t0 / kTile * kTile, tiles = (sg.t1 - key0 + kTile - 1) / kTile;
        const int nq = __shfl_sync(0xffffffffu, a.rows - sg.rt * kChunkRows > 128 ? 2 : 1, 0);
        const int steps = __shfl_sync(0xffffffffu, tiles, 0);
        for (int j = 0; alive && j <= steps; ++j) {
          // Step j: half by half and query tile by query tile, the values of tile j - 1, then the scores of tile j.
          const uint32_t st = (it + j) & 1, was = st ^ 1;
          if (j < steps) alive = ready(kKFull + st, (it + j) >> 1);
          if (alive && j > 0) alive = ready(kVFull + was, (it + j - 1) >> 1);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int half = x >> 1, q = x & 1;
            if (!alive || q >= nq) continue;
            const bool last = half == 1 && q == nq - 1;
            if (j > 0) {
              alive = ready(kPFull + 2 * q + half, done[q] + j - 1);
              if (!alive) continue;
              tc_fence_after();
              values(q, half, was, j == 1 && half == 0, last);
            } else if (half == 0) {
              alive = ready(kQFull + q, segs[q]);
              if (!alive) continue;
              ++segs[q];
            }
            if (j < steps) {
              tc_fence_after();
              scores(q, half, st, last);
            }
          }
          __syncwarp();
        }
        it += steps;
        done[0] += steps;
        if (nq > 1) done[1] += steps;
        u = next;
      }
      // What was issued ends, and its last arrivals land, before tensor memory is freed and the CTA ends.
      if (leader) umma_commit(bar + kDrain);
      __syncwarp();
      mbar_wait(bar + kDrain, 0);
    } else if (w == 13) {
      // ---------------------------------------------------------- codes in: lane g < 8 takes keys 16 g .. of each tile
      uint32_t it = 0;
      const uint32_t bytes = 16 * D;
      Seg sg;
      for (int u = u0, next; alive && u < u1;) {
        walk(sg, u, next);
        if (sg.t1 <= sg.t0) {
          u = next;
          continue;
        }
        if (lane == 0 && sg.head && !sg.whole) a.cuts[blockIdx.x] = cut_of(a, sg, u != u0, per);
        const int key0 = sg.t0 / kTile * kTile, tiles = (sg.t1 - key0 + kTile - 1) / kTile;
        // -1: keys the segment does not reach, -2: a page outside the cache.
        const auto load_page = [&](int j) {
          const int key = key0 + j * kTile + 16 * lane;
          if (j >= tiles || lane >= 8 || key < sg.t0 || key >= sg.t1) return -1;
          const int64_t p = page_of(a, sg.b, key >> a.block_log2);
          return p >= 0 && p < a.n_blocks ? static_cast<int>(p) : -2;
        };
        const auto load_scale = [&](const float* p, int page) {
          return page >= 0 ? p[static_cast<int64_t>(page) * a.heads + sg.kv] : 0.f;
        };
        int page = load_page(0), page1 = load_page(1);
        float ks = load_scale(a.ks, page), vs = load_scale(a.vs, page);
        for (int j = 0; j < tiles; ++j, ++it) {
          const int page2 = load_page(j + 2);
          const float ks1 = load_scale(a.ks, page1), vs1 = load_scale(a.vs, page1);
          const uint32_t loaded = __ballot_sync(0xffffffffu, page >= 0), bad = __ballot_sync(0xffffffffu, page == -2);
          if (bad && lane == 0 && a.d_status) atomicOr(a.d_status, TQ_DEV_BAD_BLOCK);
          const int64_t at = ((static_cast<int64_t>(page) * a.heads + sg.kv) * a.block + ((key0 + j * kTile + 16 * lane) & (a.block - 1))) * D;
          const uint32_t sum = __popc(loaded) * bytes;
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            alive = __all_sync(0xffffffffu, wait(kRawEmpty + kv, it + 1));
            if (!alive) break;
            if (kv == 0) {
              TileInfo& inf = info[it & 3];
              if (lane == 0) {
                inf.loaded = loaded;
                inf.bad = bad;
              }
              if (lane < 8) {
                inf.ks[lane] = ks;
                inf.lv[lane] = octaves(vs);
              }
            }
            __syncwarp();
            if (lane == 0) mbar_expect_tx(bar + kRawFull + kv, sum);
            __syncwarp();
            if (page >= 0)
              bulk_load(base + (kv ? L::kOffRawV : L::kOffRawK) + lane * bytes, (kv ? a.v : a.k) + at, bytes, bar + kRawFull + kv);
          }
          if (!alive) break;
          page = page1;
          page1 = page2;
          ks = ks1;
          vs = vs1;
        }
        u = next;
      }
      // Copies in flight land before the CTA ends (bar kRawFull's phase `it - 1` is the last one armed, if any).
      if (it > 0 || !alive)
        for (int kv = 0; kv < 2; ++kv) {
          mbar_wait(bar + kRawFull + kv, (it - 1) & 1);
          if (!alive) mbar_wait(bar + kRawFull + kv, it & 1, 1000000ull);
        }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (w == 12) tmem_dealloc(tmem, kTmemCols);
}

template <int D, bool INT8>
cudaError_t launch_one(const AttnArgs& a, cudaStream_t st) {
  constexpr int smem = Smem<D>::kBytes;
  static_assert(smem <= 232448, "shared memory plan exceeds 227 KB");
  cudaError_t e = cudaFuncSetAttribute(cache8_chunk_kernel<D, INT8>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cache8_chunk_kernel<D, INT8><<<kSms, kThreads, smem, st>>>(a);
  count_launch();
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_merge<D>(a, kSms, st);
}

}  // namespace

// Up to 64 rows go to the few-row kernel, which a short sequence wants: one of 1000 keys, 8 KV heads, 64 rows, 21.6 us
// against 23.4 here (d = 64: 16.6 against 21.2). Over long ones this kernel would be the faster from 17 rows on, d = 128 (8 x
// 32768 keys: 16 rows 143 there, 205 here, 24 rows 257 and 207, 64 rows 500 and 212; 8 x 2048 keys, 24 rows 42 and 34),
// and from 33 on, d = 64 (32 rows 181 and 189, 48 rows 260 and 190).
bool chunk_supported(int d, bool f32, int rows) { return (d == 64 || d == 128) && !f32 && rows > 64; }

size_t chunk_record_bytes(int d) { return sizeof(float) * kSms * 2 * kChunkRows * static_cast<size_t>(kRecHead + d); }

cudaError_t launch_chunk(int d, bool int8, const AttnArgs& a, cudaStream_t st) {
  if (d == 64) return int8 ? launch_one<64, true>(a, st) : launch_one<64, false>(a, st);
  return int8 ? launch_one<128, true>(a, st) : launch_one<128, false>(a, st);
}

}  // namespace tq
