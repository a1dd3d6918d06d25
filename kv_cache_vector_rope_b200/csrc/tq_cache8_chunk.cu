// tq_cache8_attention for many query rows: a chunk of a prompt over the 8-bit
// cache it extends (bf16 queries and outputs, d 64 or 128).
//
// The formulas are those of tq_cache8_attn.cu. With hundreds of rows per KV head
// the products bound the call, so they run on the tensor cores' tcgen05 path: a
// CTA takes 256 rows (two query tiles of 128) and walks 128 keys at a time,
//   S = Q K^T   both operands in shared memory, S (128 x 128 fp32) in tensor memory,
//   O += P V    P (halves) in tensor memory over S, O (128 x d fp32) in tensor memory.
// Two query tiles alternate: while one's weights are formed, the other's two
// products run. Warps 0-3 and 4-7 form weights (one row per thread), warps 8-11
// turn codes into halves, warp 12 issues the products.
//
// Codes become halves once per CTA for all 256 rows. An 8-bit code is exactly a
// half; a block's scale is a power of two, and so is its ratio to the largest
// scale of the 128 keys (K) or so far (V), so the halves carry the ratio and the
// reference scale goes into the softmax factor (K) or, where it grows, into a
// rescaling of O (V). A ratio below 2^-15 loses bits that lie 2^-24 below the
// largest code of the tile. Queries are scaled by a power of two into half's
// range (exact), weights are rounded to halves (2^-12).
#include "tq_cache8_attn.cuh"

namespace tq {
namespace {

using namespace c8;
using namespace sm100;

constexpr int kThreads = 512;                        // four warpgroups: weights, weights, codes, products
constexpr int kTile = kChunkUnit;                    // keys per step
static_assert(kTile == 128 && kChunkRows == 256, "tiles of 128 x 128");
constexpr int kRegsWeights = 176, kRegsCodes = 112, kRegsProducts = 40;
static_assert((2 * kRegsWeights + kRegsCodes + kRegsProducts) * 128 <= 128 * kThreads, "within the launch's registers");

template <int D>
struct Smem {
  static constexpr int kTileBytes = 128 * D * 2;     // 128 rows of halves: D / 64 atoms of [128][128 B], 128-byte swizzle
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = 2 * kTileBytes;       // two stages
  static constexpr int kOffV = kOffK + 2 * kTileBytes;
  static constexpr int kOffInfo = kOffV + 2 * kTileBytes;        // float4 [4]: K scale, V scale, bad groups
  static constexpr int kOffBar = kOffInfo + 64;
  static constexpr int kBars = 17;
  static constexpr int kOffTmem = kOffBar + 8 * (kBars + 1);
  static constexpr int kOffPart = kOffTmem + 16;
  static constexpr int kOffCum = kOffPart + 4 * (kThreads / 32);
  static constexpr int kBytes = kOffCum + 4 * (kC8Slice + 1) + 1024;
};

enum Bar { kKFull = 0, kVFull = 2, kKEmpty = 4, kVEmpty = 6, kQFull = 8, kSFull = 10, kPFull = 12, kPvDone = 14, kDrain = 16 };

// Tensor memory columns: S of tile q at 128 q (its first 64 become P), O at 256 + D q.
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

// 16 codes of row `row`, coordinates 16 c .., as halves times `ratio` into a tile.
template <int D, bool INT8>
__device__ __forceinline__ void put_codes(uint32_t tile, int row, int c, const uint4& w, bool scaled, __half2 ratio) {
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
  uint32_t h[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    h[2 * k] = two_halves<INT8, false>(ws[k]);
    h[2 * k + 1] = two_halves<INT8, true>(ws[k]);
  }
  if (scaled) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&h[k]), ratio);
      h[k] = *reinterpret_cast<const uint32_t*>(&x);
    }
  }
  const int atom = c >> 2, at = (c & 3) * 2;
  const uint32_t base = tile + atom * (128 * 128) + row * 128;
  // Lanes of odd atoms store their second half first, so that eight lanes meet eight different bank groups.
  const bool odd = atom & 1;
  const int first = at + (odd ? 1 : 0), second = at + (odd ? 0 : 1);
  sts128(base + ((first ^ (row & 7)) << 4), odd ? h[4] : h[0], odd ? h[5] : h[1], odd ? h[6] : h[2], odd ? h[7] : h[3]);
  sts128(base + ((second ^ (row & 7)) << 4), odd ? h[0] : h[4], odd ? h[1] : h[5], odd ? h[2] : h[6], odd ? h[3] : h[7]);
}

template <int D, bool INT8>
__global__ void __launch_bounds__(kThreads, 1) cache8_chunk_kernel(AttnArgs a) {
  using L = Smem<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
  const uint32_t base = smem_u32(smem);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  float4* info = reinterpret_cast<float4*>(smem + L::kOffInfo);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + L::kOffTmem);
  int* cum = reinterpret_cast<int*>(smem + L::kOffCum);
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar + kKFull + s, 128);
      mbar_init(bar + kVFull + s, 128);
      mbar_init(bar + kKEmpty + s, 1);
      mbar_init(bar + kVEmpty + s, 1);
      mbar_init(bar + kQFull + s, 128);
      mbar_init(bar + kSFull + s, 1);
      mbar_init(bar + kPFull + s, 128);
      mbar_init(bar + kPvDone + s, 1);
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
  if (blockIdx.x == 0)
    for (int b = tid; b <= a.batch; b += kThreads) a.cum_out[b] = cum[b];
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  const int total = cum[a.batch];
  const int per = units_per_cta(a, total, gridDim.x);
  const int u0 = min(static_cast<int>(blockIdx.x) * per, total), u1 = min(u0 + per, total);
  // Every role walks the same segments; a wait that gives up ends the role's walk (the others' waits give up too).
  const auto wait = [&](int which, uint32_t parity) {
    if (mbar_wait(bar + which, parity & 1, a.wait_ns)) return true;
    if (a.d_status) atomicOr(a.d_status, TQ_DEV_TIMEOUT);
    return false;
  };
  bool alive = true;

  if (w < 8) {
    // ------------------------------------------------------------ weights: one row per thread
    regs_up<kRegsWeights>();
    const int q = w >> 2, wr = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((w & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + 128 * q, o_at = tmem + lanes + 256 + D * q;
    uint32_t tiles_seen = 0;                         // tiles of this query tile so far
    uint32_t walked = 0;                             // tiles of all segments: the info ring's count
    for (int u = u0; alive && u < u1;) {
      int next;
      const Seg sg = seg_at(a, cum, u, u1, &next);
      const int key0 = sg.t0 / kTile * kTile, tiles = (sg.t1 - key0 + kTile - 1) / kTile;
      const int r0 = sg.rt * kChunkRows + 128 * q, r = r0 + wr;
      if (r0 >= a.rows) {                            // this query tile has no row
        walked += tiles;
        u = next;
        continue;
      }
      const bool live = r < a.rows;
      const int i = live ? r / a.group : 0, hq = sg.kv * a.group + (live ? r % a.group : 0);
      float cq;
      {
        const int64_t at = (a.first_seq + sg.b) * a.q_bs + hq * a.q_hs + i * a.q_rs;
        float amax = 0.f;
        if (live)
#pragma unroll 2
          for (int c = 0; c < D / 16; ++c) {
            float x[16];
            load_q16<false>(a.q, at + 16 * c, x);
#pragma unroll
            for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e]));
          }
        const int E = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -100);
        float up = __uint_as_float(static_cast<uint32_t>(14 - min(E, 127) + 127) << 23);
        cq = fabsf(a.scale2) / up;
        if (a.scale2 < 0.f) up = -up;                // the factor of the scores stays positive
        const uint32_t row = base + L::kOffQ + q * L::kTileBytes + wr * 128;
#pragma unroll 2
        for (int c = 0; c < D / 16; ++c) {
          float x[16];
          if (live) load_q16<false>(a.q, at + 16 * c, x);
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) h[e] = live ? pack_half(x[2 * e] * up, x[2 * e + 1] * up) : 0u;
          const uint32_t to = row + (c >> 2) * (128 * 128);
          const int c0 = (c & 3) * 2;
          sts128(to + ((c0 ^ (wr & 7)) << 4), h[0], h[1], h[2], h[3]);
          sts128(to + (((c0 + 1) ^ (wr & 7)) << 4), h[4], h[5], h[6], h[7]);
        }
        fence_proxy_async_smem();
        mbar_arrive(bar + kQFull + q);
      }
      const int hi = live ? row_hi(a, sg.n, i) : 0, lo = row_lo(a, hi);
      // Keys in [lo_max, hi_min) are seen by every row of the tile.
      const int hi_min = row_hi(a, sg.n, r0 / a.group);
      const int lo_max = row_lo(a, row_hi(a, sg.n, min(r0 + 127, a.rows - 1) / a.group));
      float m = -INFINITY, l = 0.f, vrun = 0.f;
      for (int j = 0; j < tiles; ++j) {
        const int k0 = key0 + j * kTile;
        alive = __all_sync(0xffffffffu, wait(kSFull + q, tiles_seen + j));
        if (!alive) break;
        tc_fence_after();
        uint32_t sr[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_at + 32 * c, sr[c]);
        tmem_ld_wait();
        const float4 inf = info[(walked + j) & 3];
        const float f = fmaxf(cq * inf.x, 1.17549435e-38f);   // not 0: masked scores stay -inf
        const uint32_t bad = __float_as_uint(inf.z);
        if (k0 < lo_max || k0 + kTile > hi_min || bad) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int key = k0 + 32 * c + e;
              if (key < lo || key >= hi || (bad >> (2 * c + e / 16)) & 1) sr[c][e] = 0xff800000u;
            }
        }
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            top[c] = fmaxf(top[c], fmaxf(__uint_as_float(sr[c][e]), __uint_as_float(sr[c][e + 1])));
        const float mt = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * f;
        if (__any_sync(0xffffffffu, mt > m + kSlack || inf.y != vrun)) {
          const float mn = fmaxf(m, mt);
          const float fm = mn == m ? 1.f : fast_exp2(m - mn);
          m = mn;
          l *= fm;
          if (j > 0) {
            // O of the tiles before is complete before it is scaled.
            alive = __all_sync(0xffffffffu, wait(kPvDone + q, tiles_seen + j - 1));
            if (!alive) break;
            tc_fence_after();
            const float fo = fm * (vrun / inf.y);
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(o_at + 32 * c, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fo);
              tmem_st32(o_at + 32 * c, o);
            }
          }
          vrun = inf.y;
        }
        // p = 2^(s f - m + kLift); a row that has seen no key yet has m = -inf, and every s is -inf too.
        const float off = m == -INFINITY ? 0.f : kLift - m;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float p0 = fast_exp2(fmaf(__uint_as_float(sr[c][2 * e]), f, off));
            const float p1 = fast_exp2(fmaf(__uint_as_float(sr[c][2 * e + 1]), f, off));
            sum[e & 3] += p0 + p1;
            pk[e] = pack_half(p0, p1);
          }
          tmem_st16(s_at + 16 * c, pk);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar + kPFull + q);
      }
      if (alive) alive = __all_sync(0xffffffffu, wait(kPvDone + q, tiles_seen + tiles - 1));
      if (!alive) break;
      tiles_seen += tiles;
      walked += tiles;
      tc_fence_after();
      float* rec = a.rec + (static_cast<int64_t>(blockIdx.x) * 2 + (sg.head && u != u0 ? 1 : 0)) * kChunkRows * (kRecHead + D) +
                   static_cast<int64_t>(128 * q + wr) * (kRecHead + D);
      const float by = sg.whole ? (l == 0.f ? 0.f : vrun / l) : vrun;
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
    const int ct = tid - 256;
    uint32_t it = 0;
    float vref = 0.f;
    for (int u = u0; alive && u < u1;) {
      int next;
      const Seg sg = seg_at(a, cum, u, u1, &next);
      const int key0 = sg.t0 / kTile * kTile, tiles = (sg.t1 - key0 + kTile - 1) / kTile;
      vref = 0.f;
      // Lane g of each warp keeps page and scales of keys 16 g .. of the tile (lanes 8.. idle); keys the segment does
      // not reach have page -1, pages outside the cache -2.
      const auto load_page = [&](int j) {
        const int key = key0 + j * kTile + 16 * lane;
        if (lane >= 8 || key < sg.t0 || key >= sg.t1) return -1;
        const int64_t p = page_of(a, sg.b, key / a.block);
        return p >= 0 && p < a.n_blocks ? static_cast<int>(p) : -2;
      };
      const auto load_scale = [&](const float* p, int page) {
        return page >= 0 ? p[static_cast<int64_t>(page) * a.heads + sg.kv] : 0.f;
      };
      const auto load_raw = [&](const uint8_t* codes, int page, int j, uint4 (&raw)[kPer]) {
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
          const int row = (x * 128 + ct) / kPer, c = (x * 128 + ct) % kPer;
          const int pg = __shfl_sync(0xffffffffu, page, row >> 4);
          const int key = key0 + j * kTile + row;
          const bool in = pg >= 0 && key < sg.n;     // what lies behind the sequence may be any byte
          raw[x] = in ? *reinterpret_cast<const uint4*>(
                            codes + ((static_cast<int64_t>(pg) * a.heads + sg.kv) * a.block + key % a.block) * D + 16 * c)
                      : make_uint4(0u, 0u, 0u, 0u);
        }
      };
      int pg = load_page(0);
      uint4 kraw[kPer], vraw[kPer];
      load_raw(a.k, pg, 0, kraw);
      load_raw(a.v, pg, 0, vraw);
      float ks = load_scale(a.ks, pg), vs = load_scale(a.vs, pg);
      for (int j = 0; j < tiles; ++j, ++it) {
        const int pg_next = j + 1 < tiles ? load_page(j + 1) : -1;
        const uint32_t bad = __ballot_sync(0xffffffffu, pg == -2);
        if (bad && ct == 0 && a.d_status) atomicOr(a.d_status, TQ_DEV_BAD_BLOCK);
        float kref = dev::warp_max(ks);
        if (!(kref > 0.f)) kref = 1.f;               // no page at all
        vref = fmaxf(vref, dev::warp_max(vs));
        if (!(vref > 0.f)) vref = 1.17549435e-38f;
        const float rk = pg >= 0 ? ks / kref : 0.f, rv = pg >= 0 ? vs / vref : 0.f;
        const bool k_scaled = __any_sync(0xffffffffu, lane < 8 && rk != 1.f);
        const bool v_scaled = __any_sync(0xffffffffu, lane < 8 && rv != 1.f);
        if (ct == 0) info[it & 3] = make_float4(kref, vref, __uint_as_float(bad), 0.f);
        const uint32_t st = it & 1, parity = (it >> 1) & 1;
        alive = __all_sync(0xffffffffu, wait(kKEmpty + st, parity ^ 1));
        if (!alive) break;
        const uint32_t kt = base + L::kOffK + st * L::kTileBytes, vt = base + L::kOffV + st * L::kTileBytes;
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
          const int row = (x * 128 + ct) / kPer, c = (x * 128 + ct) % kPer;
          const __half2 ratio = __float2half2_rn(__shfl_sync(0xffffffffu, rk, row >> 4));
          put_codes<D, INT8>(kt, row, c, kraw[x], k_scaled, ratio);
        }
        fence_proxy_async_smem();
        mbar_arrive(bar + kKFull + st);
        float ks_next = 0.f, vs_next = 0.f;
        if (j + 1 < tiles) {
          load_raw(a.k, pg_next, j + 1, kraw);
          ks_next = load_scale(a.ks, pg_next);
          vs_next = load_scale(a.vs, pg_next);
        }
        alive = __all_sync(0xffffffffu, wait(kVEmpty + st, parity ^ 1));
        if (!alive) break;
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
          const int row = (x * 128 + ct) / kPer, c = (x * 128 + ct) % kPer;
          const __half2 ratio = __float2half2_rn(__shfl_sync(0xffffffffu, rv, row >> 4));
          put_codes<D, INT8>(vt, row, c, vraw[x], v_scaled, ratio);
        }
        fence_proxy_async_smem();
        mbar_arrive(bar + kVFull + st);
        if (j + 1 < tiles) load_raw(a.v, pg_next, j + 1, vraw);
        pg = pg_next;
        ks = ks_next;
        vs = vs_next;
      }
      u = next;
    }
  } else {
    // ------------------------------------------------------------ products
    regs_down<kRegsProducts>();
    if (w == 12 && lane == 0) {
      constexpr uint32_t kIdS = idesc_f16(128, 128, false), kIdO = idesc_f16(128, D, true);
      uint32_t it = 0, segs[2] = {0, 0}, done[2] = {0, 0};
      const auto scores = [&](int q, uint32_t st) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k >> 2) * (128 * 128) + (k & 3) * 32;
          umma_ss(tmem + 128 * q, desc_k_sw128(base + L::kOffQ + q * L::kTileBytes + off),
                  desc_k_sw128(base + L::kOffK + st * L::kTileBytes + off), kIdS, k != 0);
        }
        umma_commit(bar + kSFull + q);
      };
      const auto values = [&](int q, uint32_t st, bool first) {
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          umma_ts(tmem + 256 + D * q, tmem + 128 * q + 8 * k,
                  desc_mn_sw128(base + L::kOffV + st * L::kTileBytes + k * 16 * 128, 128 * 128), kIdO, !(first && k == 0));
        umma_commit(bar + kPvDone + q);
      };
      for (int u = u0; alive && u < u1;) {
        int next;
        const Seg sg = seg_at(a, cum, u, u1, &next);
        const int key0 = sg.t0 / kTile * kTile, tiles = (sg.t1 - key0 + kTile - 1) / kTile;
        const int nq = a.rows - sg.rt * kChunkRows > 128 ? 2 : 1;
        for (int j = 0; alive && j <= tiles; ++j) {
          // Step j: the values of tile j - 1, then the scores of tile j, query tile by query tile.
          const uint32_t st = (it + j) & 1, was = st ^ 1;
          if (j < tiles && !wait(kKFull + st, (it + j) >> 1)) alive = false;
          for (int q = 0; alive && q < nq; ++q) {
            if (j > 0) {
              if (q == 0 && !wait(kVFull + was, (it + j - 1) >> 1)) alive = false;
              if (alive && !wait(kPFull + q, done[q])) alive = false;
              if (!alive) break;
              tc_fence_after();
              values(q, was, j == 1);
              ++done[q];
              if (q == nq - 1) umma_commit(bar + kVEmpty + was);
            } else {
              if (!wait(kQFull + q, segs[q])) alive = false;
              if (!alive) break;
              ++segs[q];
            }
            if (j < tiles) {
              tc_fence_after();
              scores(q, st);
              if (q == nq - 1) umma_commit(bar + kKEmpty + st);
            }
          }
        }
        it += tiles;
        u = next;
      }
      // What was issued ends, and its last arrivals land, before tensor memory is freed and the CTA ends.
      umma_commit(bar + kDrain);
      mbar_wait(bar + kDrain, 0);
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
  return e != cudaSuccess ? e : launch_combine<D, false>(a, kSms, st);
}

}  // namespace

bool chunk_supported(int d, bool f32, int rows) { return (d == 64 || d == 128) && !f32 && rows > 64; }

size_t chunk_record_bytes(int d) { return sizeof(float) * kSms * 2 * kChunkRows * static_cast<size_t>(kRecHead + d); }

cudaError_t launch_chunk(int d, bool int8, const AttnArgs& a, cudaStream_t st) {
  if (d == 64) return int8 ? launch_one<64, true>(a, st) : launch_one<64, false>(a, st);
  return int8 ? launch_one<128, true>(a, st) : launch_one<128, false>(a, st);
}

}  // namespace tq
