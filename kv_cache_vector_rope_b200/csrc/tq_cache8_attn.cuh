// What the kernels of tq_cache8_attention share: their arguments, how the work
// is dealt to the CTAs, operand loads, and the merge of partial results.
#pragma once

#include "tq_cache8.h"
#include "tq_device.cuh"
#include "tq_sm100.cuh"

namespace tq {
namespace c8 {

constexpr int kSms = 148;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Weights are kept as 2^(s - m + kLift): halves hold them to 2^-24, and the
// running maximum m is moved only when a score exceeds it by kSlack octaves.
constexpr float kLift = 6.f;
constexpr float kSlack = 8.f;
// A partial record: per row its maximum, its sum, the exponent of its value sums' unit, an unused float, d value sums.
constexpr int kRecHead = 4;
constexpr int kMaxRecs = 2 * kSms;                   // CTAs that may leave records of one stream

// Programmatic launches: a kernel lets the one behind it be set up, and waits for the end of the one before it.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// x / d for 0 <= x < 2^31 by a product and a shift (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994): the walk over a sequence's row tiles is a chain of them.
struct Div {
  int d;
  uint32_t mul;
  int shift;
  explicit Div(int d_) : d(d_), shift(0) {
    while ((1ll << shift) < d) ++shift;
    mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << shift) - static_cast<uint64_t>(d))) / static_cast<uint64_t>(d) + 1);
  }
  __device__ __forceinline__ int of(int x) const {
    return static_cast<int>((__umulhi(static_cast<uint32_t>(x), mul) + static_cast<uint32_t>(x)) >> shift);
  }
};

struct AttnArgs {
  Div heads_div, group_div, tiles_div;               // of heads, group and row_tiles
  int heads, block, batch;
  int block_log2;
  int64_t n_blocks;
  const uint8_t* k;
  const uint8_t* v;
  const float* ks;
  const float* vs;
  const void* q;
  bool q_f32, out_f32;
  int64_t q_bs, q_hs, q_rs;
  int group, nq, rows;                               // rows = group * nq per KV head, row r: position r / group
  int tile_rows, row_tiles;                          // rows a CTA takes together
  int unit_log2, min_units;                          // keys per unit of the split, units a CTA takes at least
  int lead;                                          // what a stream costs beside its keys, in units
  const int32_t* lens;                               // of this slice
  const int32_t* table;
  int64_t table_stride;
  int64_t first_seq;
  int causal;
  int window;
  bool alone;                                        // a CTA per stream, whole
  float scale2;                                      // softmax scale * log2 e
  void* out;
  int64_t o_bs, o_hs, o_rs;
  float* lse;                                        // [batch][hq][nq] or NULL
  float* rec;                                        // [grid][2][tile_rows][kRecHead + d]
  struct CutInfo* cuts;                              // [grid], for the merge
  uint64_t wait_ns;
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

// Keys [lo, hi) that row position i sees of a sequence of n keys.
__device__ __forceinline__ int row_hi(const AttnArgs& a, int n, int i) { return a.causal ? max(0, n - a.nq + i + 1) : n; }
__device__ __forceinline__ int row_lo(const AttnArgs& a, int hi) { return a.window > 0 ? max(0, hi - a.window) : 0; }

// First key and end of what the rows of row tile rt see together, and how many
// units of the split that is (units start at multiples of their size).
struct KeyRange {
  int lo, hi, units;
};
__device__ __forceinline__ KeyRange tile_range(const AttnArgs& a, int n, int rt) {
  KeyRange r;
  const int r0 = rt * a.tile_rows, r1 = min(a.rows, r0 + a.tile_rows) - 1;
  r.hi = row_hi(a, n, a.group_div.of(r1));
  r.lo = row_lo(a, row_hi(a, n, a.group_div.of(r0)));
  r.units = r.hi > r.lo ? ((r.hi + (1 << a.unit_log2) - 1) >> a.unit_log2) - (r.lo >> a.unit_log2) : 0;
  return r;
}
// A stream costs its units and a lead (operands, the merge of the warps); a
// stream without keys costs nothing.
__device__ __forceinline__ int stream_cost(const AttnArgs& a, const KeyRange& r) { return r.units > 0 ? r.units + a.lead : 0; }
// Cost of one KV head of a sequence.
__device__ __forceinline__ int head_units(const AttnArgs& a, int n) {
  int u = 0;
  if (n > 0)
    for (int rt = 0; rt < a.row_tiles; ++rt) u += stream_cost(a, tile_range(a, n, rt));
  return u;
}

// The costs of all (sequence, KV head, row tile) streams, in that order, are
// dealt to the CTAs in equal contiguous ranges (a stream's lead comes first).
__device__ __forceinline__ int units_per_cta(const AttnArgs& a, int total, int grid) {
  return max((total + grid - 1) / grid, a.min_units);
}

// One stream's part of a CTA's range.
struct Seg {
  int b, kv, rt, n, t0, t1;                          // keys [t0, t1); t0 is a multiple of 16; none where t1 <= t0
  bool whole;                                        // all keys of the stream
  bool head;                                         // the stream's first keys
  int start, units;                                  // of the whole stream: where its cost begins, its units
};
__device__ __forceinline__ void seg_fill(const AttnArgs& a, Seg& s, const KeyRange& r, int rel, int u, int uend, int* next) {
  s.start = u - rel;
  s.units = r.units;
  const int take = min(stream_cost(a, r) - rel, uend - u);
  const int from = max(rel - a.lead, 0), to = rel + take - a.lead;       // units of the stream
  s.head = from == 0;
  s.whole = s.head && to == r.units;
  s.t0 = s.head ? r.lo / 16 * 16 : ((r.lo >> a.unit_log2) + from) << a.unit_log2;
  s.t1 = to > from ? min(((r.lo >> a.unit_log2) + to) << a.unit_log2, r.hi) : s.t0;
  *next = u + take;
}
__device__ __forceinline__ Seg seg_at(const AttnArgs& a, const int* cum, int u, int uend, int* next) {
  Seg s;
  s.b = find_seq(cum, a.batch, u);
  s.n = seq_len(a, s.b, false);
  const int per_head = a.heads_div.of(cum[s.b + 1] - cum[s.b]);
  int rel = u - cum[s.b];
  s.kv = rel / per_head;
  rel -= s.kv * per_head;
  s.rt = 0;
  KeyRange r = tile_range(a, s.n, 0);
  while (rel >= stream_cost(a, r)) {
    rel -= stream_cost(a, r);
    r = tile_range(a, s.n, ++s.rt);
  }
  seg_fill(a, s, r, rel, u, uend, next);
  return s;
}
// All of stream x, in the order of (sequence, KV head, row tile).
__device__ __forceinline__ Seg seg_alone(const AttnArgs& a, int x) {
  Seg s;
  int next;
  const int h = a.tiles_div.of(x);
  s.rt = x - h * a.row_tiles;
  s.b = a.heads_div.of(h);
  s.kv = h - s.b * a.heads;
  s.n = seq_len(a, s.b, s.kv == 0 && s.rt == 0);
  seg_fill(a, s, tile_range(a, s.n, s.rt), 0, 0, 0x7fffffff, &next);
  return s;
}
// The segment behind `s`, which ends its stream at u < uend: the next stream that costs anything, from its start.
__device__ __forceinline__ void seg_after(const AttnArgs& a, const int* cum, Seg& s, int u, int uend, int* next) {
  KeyRange r;
  do {
    if (++s.rt == a.row_tiles) {
      s.rt = 0;
      if (++s.kv == a.heads) {
        s.kv = 0;
        do ++s.b;
        while (cum[s.b + 1] <= u);
        s.n = seq_len(a, s.b, false);
      }
    }
    r = tile_range(a, s.n, s.rt);
  } while (r.units <= 0);
  seg_fill(a, s, r, 0, u, uend, next);
}
// What a CTA whose range ends inside a stream that it began leaves for the merge: the CTAs from this one on that hold a
// record of the stream (0: there is no such stream), whether its own is in its second slot, and which stream it is.
struct CutInfo {
  int n, slot, b, kv, rt;
};
__device__ __forceinline__ CutInfo cut_of(const AttnArgs& a, const Seg& s, bool second, int per) {
  CutInfo c;
  c.n = (s.start + a.lead + s.units - 1) / per - static_cast<int>(blockIdx.x) + 1;
  c.slot = second;
  c.b = s.b;
  c.kv = s.kv;
  c.rt = s.rt;
  return c;
}

__device__ __forceinline__ int64_t page_of(const AttnArgs& a, int b, int blk) {
  return a.table ? static_cast<int64_t>(a.table[b * a.table_stride + blk]) : (a.first_seq + b) * a.table_stride + blk;
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

// Value scales. A row's value sums take the weights 2^(s - m + kLift) times the block's value scale, as halves, which
// end at 2^-24: what a key adds must be small beside the row's largest addend, not beside the largest scale, whose keys
// may weigh nothing or lie where the row does not look. So the sums are in units of 2^e: m is the maximum of the scores
// s (in octaves) over the keys that the row has seen, e that of s - m plus the octaves of the value scale over those of
// them with a code that is not zero (a large token can leave others of its block none), both rounded to whole numbers,
// whose differences are exact. The largest addend is then about 2^kLift, later ones exceed it by kSlack octaves at most
// before m and e are moved, and a key is off by 2^-25 of a unit, 2^-30 of the largest addend with codes of the type's
// largest. Where a weight has a second half, that is kept times 2^11 and ends as far below. A row that has seen no key
// has m = -inf, one without an addend e = -inf.
constexpr float kLimb = 2048.f;
constexpr float kNoUnit = -127.f;                    // of sums without an addend: below every other
__device__ __forceinline__ float octaves(float scale) {          // of a power of two; below all of them for 0
  return __uint_as_float(0x4b000000u | (__float_as_uint(scale) >> 23)) - (8388608.f + 127.f);
}
__device__ __forceinline__ float pow2_whole(float x) {           // 2^x for a whole number x in [-126, 127], 0 for -127
  return __uint_as_float(__float_as_uint(x + (12582912.f + 127.f)) << 23);
}
__device__ __forceinline__ float unit_of(float e) { return fmaxf(e, kNoUnit); }
// How the weights of keys under a value scale of 2^lv are formed: 2^((s - m) + lift) goes into the value sums and, times
// inv, into the sum of weights (one exponential for both: lift carries d, the octaves of the scale over the unit, and inv
// is 2^-d). d is at least -60, where nothing is left of a half and the weights of keys that count are still normal
// numbers. A score above lim asks for a new m and e: before the first addend every score.
struct Weigh {
  float lift, lim, inv;
};
__device__ __forceinline__ Weigh weigh(float m, float e, float lv) {
  const float d = fmaxf(lv - unit_of(e), -60.f);
  Weigh w;
  w.lift = d + kLift;
  w.lim = e == -INFINITY ? -INFINITY : __fadd_rd(m, kSlack - fmaxf(d, 0.f));   // where it is not exact, not too high
  w.inv = pow2_whole(-fminf(d, 126.f));
  return w;
}
// m as it is taken from scores: of a row that has seen no key all are -inf.
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.f : m; }
// The unit of sums in units of 2^e whose m has moved by `by`, with further addends of up to 2^top: at least 2^-126, which
// outputs cannot tell from less.
__device__ __forceinline__ float next_unit(float e, float by, float top) {
  return fmaxf(e, top) == -INFINITY ? -INFINITY : fmaxf(fmaxf(e + by, rintf(top)), -126.f);
}
// a - b of two maxima, the first at most the second (which may be -inf too).
__device__ __forceinline__ float below(float a, float b) { return a == b ? 0.f : a - b; }
// Factor of the value sums where (m, e) become (mn, en).
__device__ __forceinline__ float unit_step(float m, float e, float mn, float en) {
  if (e == -INFINITY) return 1.f;                    // no addend so far
  return fast_exp2(below(m, mn) + (e - en));
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
  return halves_e4m3<HI>(w);
}

// Sixteen consecutive values of a query row.
template <bool F32>
__device__ __forceinline__ void load_q16(const void* p, int64_t i, float* x) {
  if (F32) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 y = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i)[k];
      x[4 * k] = y.x;
      x[4 * k + 1] = y.y;
      x[4 * k + 2] = y.z;
      x[4 * k + 3] = y.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint4 y = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i)[k];
      const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        x[8 * k + 2 * h] = __uint_as_float(w[h] << 16);
        x[8 * k + 2 * h + 1] = __uint_as_float(w[h] & 0xffff0000u);
      }
    }
  }
}

// A warp's part of the rows without a key: it looks at `pairs` (sequence, row tile) pairs from `pair` on and writes
// zeros for rows row0, row0 + step, ... of those where no row sees a key, all heads.
constexpr int kEmptyPairs = 4;
template <int D>
__device__ __forceinline__ void put_empty(const AttnArgs& a, int pair, int row0, int step, int pairs = kEmptyPairs) {
  const int lane = threadIdx.x & 31;
  for (int end = min(pair + pairs, a.batch * a.row_tiles); pair < end; ++pair) {
    const int b = a.tiles_div.of(pair), rt = pair - b * a.row_tiles;
    const int n = seq_len(a, b, false);
    if (n > 0 && tile_range(a, n, rt).units > 0) continue;
    const int pieces = a.out_f32 ? D / 4 : D / 8, log2 = 31 - __clz(pieces);     // of 16 bytes
    for (int row = row0; row < a.tile_rows && rt * a.tile_rows + row < a.rows; row += step) {
      const int r = rt * a.tile_rows + row, i = a.group_div.of(r);
      for (int x = lane; x < a.heads * pieces; x += 32) {
        const int hq = (x >> log2) * a.group + r - i * a.group, piece = x & (pieces - 1);
        const int64_t at = (a.first_seq + b) * a.o_bs + hq * a.o_hs + i * a.o_rs;
        char* to = static_cast<char*>(a.out) + at * (a.out_f32 ? 4 : 2);
        reinterpret_cast<uint4*>(to)[piece] = make_uint4(0u, 0u, 0u, 0u);
        if (a.lse && piece == 0) a.lse[((a.first_seq + b) * a.heads * a.group + hq) * a.nq + i] = -INFINITY;
      }
    }
  }
}

// Merges the records of every stream that more than one CTA worked on, and
// writes the rows of streams with no key at all. Block x < grid - 1 takes the
// stream that CTA x began and others ended, if there is one, and a row of it:
// the records' maxima and sums are read side by side, then D / 4 lanes walk the
// coordinates with the other threads dealing the records out among themselves,
// so that a stream in hundreds of records (one long sequence) costs a few rounds
// of loads, not one per record. The blocks behind look for rows without keys.
constexpr int kCbThreads = 256;
template <int D, bool OF>
__global__ void __launch_bounds__(kCbThreads) cache8_combine_kernel(AttnArgs a, int grid) {
  constexpr int kParts = kCbThreads / (D / 4);       // records in flight side by side
  __shared__ float wt[kMaxRecs];                     // octaves of the records' weights
  __shared__ float red[3][kCbThreads / 32];
  __shared__ float4 sums[kParts][D / 4];
  const int x0 = blockIdx.x, row = blockIdx.y, tid = threadIdx.x;
  wait_before();
  if (x0 >= grid - 1) return put_empty<D>(a, ((x0 - (grid - 1)) * (kCbThreads / 32) + tid / 32) * kEmptyPairs, row, a.tile_rows);
  const CutInfo cut = a.cuts[x0];
  const int b = cut.b, kv = cut.kv, r = cut.rt * a.tile_rows + row, n = cut.n;
  if (n == 0 || r >= a.rows) return;
  const auto record = [&](int k) {
    return a.rec + ((static_cast<int64_t>(x0 + k) * 2 + (k == 0 ? cut.slot : 0)) * a.tile_rows + row) * (kRecHead + D);
  };
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, e[2] = {0.f, 0.f};   // n <= kMaxRecs <= 2 * kCbThreads
#pragma unroll
  for (int y = 0; y < 2; ++y)
    if (tid + y * kCbThreads < n) {
      const float4 h = *reinterpret_cast<const float4*>(record(tid + y * kCbThreads));
      m[y] = h.x;
      l[y] = h.y;
      e[y] = h.z;
    }
  static_assert(kMaxRecs <= 2 * kCbThreads, "two records per thread");
  const float mw = dev::warp_max(fmaxf(m[0], m[1]));
  if ((tid & 31) == 0) red[0][tid >> 5] = mw;
  __syncthreads();
  float M = -INFINITY;
#pragma unroll
  for (int k = 0; k < kCbThreads / 32; ++k) M = fmaxf(M, red[0][k]);
  float lw = 0.f, ew = -INFINITY;
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const float by = m[y] == -INFINITY ? -INFINITY : below(m[y], M);
    lw += l[y] * fast_exp2(by);                      // a NaN of a row, whose maximum is -inf, stays
    ew = fmaxf(ew, by + e[y]);
    if (tid + y * kCbThreads < n) wt[tid + y * kCbThreads] = by + e[y];
  }
  lw = dev::warp_sum(lw);
  ew = dev::warp_max(ew);
  if ((tid & 31) == 0) {
    red[1][tid >> 5] = lw;
    red[2][tid >> 5] = ew;
  }
  __syncthreads();
  float L = 0.f, unit = kNoUnit;                     // of the merged sums
#pragma unroll
  for (int k = 0; k < kCbThreads / 32; ++k) {
    L += red[1][k];
    unit = fmaxf(unit, rintf(red[2][k]));
  }
  const int x = tid % (D / 4), part = tid / (D / 4);
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = part; k < n; k += kParts) {
    const float w = fast_exp2(wt[k] - unit);
    const float4 y = reinterpret_cast<const float4*>(record(k) + kRecHead)[x];
    sum.x = fmaf(y.x, w, sum.x);
    sum.y = fmaf(y.y, w, sum.y);
    sum.z = fmaf(y.z, w, sum.z);
    sum.w = fmaf(y.w, w, sum.w);
  }
  sums[part][x] = sum;
  __syncthreads();
  if (tid >= D / 4) return;
#pragma unroll
  for (int k = 1; k < kParts; ++k) {
    const float4 y = sums[k][x];
    sum.x += y.x;
    sum.y += y.y;
    sum.z += y.z;
    sum.w += y.w;
  }
  const int i = a.group_div.of(r), hq = kv * a.group + r - i * a.group;
  const int64_t at = (a.first_seq + b) * a.o_bs + hq * a.o_hs + i * a.o_rs + 4 * x;
  const float o[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float y = L == 0.f ? 0.f : o[k] / L * pow2_whole(unit);
    if (OF) static_cast<float*>(a.out)[at + k] = y;
    else static_cast<__nv_bfloat16*>(a.out)[at + k] = __float2bfloat16_rn(y);
  }
  if (a.lse && x == 0)
    a.lse[((a.first_seq + b) * a.heads * a.group + hq) * a.nq + i] =
        L == 0.f ? -INFINITY : (M - kLift + log2f(L)) * kLn2;
}

// Launches a kernel that begins while the one before it on the stream ends: its
// CTAs are set up meanwhile and wait_before() lets them on once that one's
// results are there.
template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// Blocks that look for rows without keys, `pairs` (sequence, row tile) pairs each.
inline int empty_blocks(const AttnArgs& a, int pairs) { return (a.batch * a.row_tiles + pairs - 1) / pairs; }
template <int D, bool OF>
cudaError_t launch_combine(const AttnArgs& a, int grid, cudaStream_t st) {
  const int rows = a.rows < a.tile_rows ? a.rows : a.tile_rows;
  const cudaError_t e = launch_behind(cache8_combine_kernel<D, OF>, dim3(grid - 1 + empty_blocks(a, kCbThreads / 32 * kEmptyPairs), rows),
                                      kCbThreads, st, a, grid);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

// The same for tiles of 128 or 256 rows: block x looks at CTA x's stream and a part of its rows, a warp at four rows side
// by side (lanes 8 y + k: row y's record k).
constexpr int kMergeThreads = 256, kMergeRows = 4, kMergeSplit = 4;
template <int D>
__global__ void __launch_bounds__(kMergeThreads, D == 256 ? 3 : 4) cache8_merge_kernel(AttnArgs a, int grid) {
  constexpr int E = D / 32;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int x0 = blockIdx.x, from = (blockIdx.y * 8 + w) * kMergeRows, step = gridDim.y * 8 * kMergeRows;
  wait_before();
  if (x0 >= grid - 1) return put_empty<D>(a, (x0 - (grid - 1)) * kEmptyPairs, blockIdx.y * 8 + w, gridDim.y * 8);
  const CutInfo cut = a.cuts[x0];
  const int n = cut.n;
  if (n == 0) return;
  for (int row0 = from; row0 < a.tile_rows && cut.rt * a.tile_rows + row0 < a.rows; row0 += step) {
    const auto record = [&](int k, int x) {
      return a.rec + ((static_cast<int64_t>(x0 + k) * 2 + (k == 0 ? cut.slot : 0)) * a.tile_rows + row0 + x) * (kRecHead + D);
    };
    float M[kMergeRows], unit[kMergeRows];
    {
      float top = -INFINITY, e = -INFINITY;
      const auto join = [&](float m, float y) {
        const float mn = fmaxf(top, m);
        e = fmaxf(e + below(top, mn), y + below(m, mn));
        top = mn;
      };
      for (int k = lane & 7; k < n; k += 8) {
        const float4 h = *reinterpret_cast<const float4*>(record(k, lane >> 3));
        join(h.x, h.x == -INFINITY ? -INFINITY : h.z);
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) {
        const float m = __shfl_xor_sync(0xffffffffu, top, o), y = __shfl_xor_sync(0xffffffffu, e, o);
        join(m, y);
      }
      e = fmaxf(rintf(e), kNoUnit);
#pragma unroll
      for (int x = 0; x < kMergeRows; ++x) {
        M[x] = __shfl_sync(0xffffffffu, top, 8 * x);
        unit[x] = __shfl_sync(0xffffffffu, e, 8 * x);
      }
    }
    float y[kMergeRows][E], l[kMergeRows];
#pragma unroll
    for (int x = 0; x < kMergeRows; ++x) {
      l[x] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) y[x][e] = 0.f;
    }
#pragma unroll 2
    for (int k = 0; k < n; ++k)
#pragma unroll
      for (int x = 0; x < kMergeRows; ++x) {
        const float* p = record(k, x);
        const float4 h = *reinterpret_cast<const float4*>(p);
        const float by = h.x == -INFINITY ? -INFINITY : below(h.x, M[x]), f = fast_exp2(by + (h.z - unit[x]));
        l[x] = fmaf(h.y, fast_exp2(by), l[x]);       // a NaN of a row, whose maximum is -inf, stays
        float z[E];
        if constexpr (E == 2) {
          *reinterpret_cast<float2*>(z) = *reinterpret_cast<const float2*>(p + kRecHead + lane * 2);
        } else {
#pragma unroll
          for (int e = 0; e < E; e += 4)
            *reinterpret_cast<float4*>(z + e) = *reinterpret_cast<const float4*>(p + kRecHead + lane * E + e);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) y[x][e] = fmaf(z[e], f, y[x][e]);
      }
#pragma unroll
    for (int x = 0; x < kMergeRows; ++x) {
      const int r = cut.rt * a.tile_rows + row0 + x;
      if (r >= a.rows) continue;
      const int i = a.group_div.of(r), hq = cut.kv * a.group + r - i * a.group;
      const int64_t at = (a.first_seq + cut.b) * a.o_bs + hq * a.o_hs + i * a.o_rs + lane * E;
      const float inv = l[x] == 0.f ? 0.f : 1.f / l[x] * pow2_whole(unit[x]);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        if (a.out_f32) *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at + e) = make_float2(y[x][e] * inv, y[x][e + 1] * inv);
        else *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(a.out) + at + e) = __floats2bfloat162_rn(y[x][e] * inv, y[x][e + 1] * inv);
      }
      if (a.lse && lane == 0)
        a.lse[((a.first_seq + cut.b) * a.heads * a.group + hq) * a.nq + i] =
            l[x] == 0.f ? -INFINITY : (M[x] - kLift + log2f(l[x])) * kLn2;
    }
  }
}
template <int D>
cudaError_t launch_merge(const AttnArgs& a, int grid, cudaStream_t st) {
  const cudaError_t e = launch_behind(cache8_merge_kernel<D>, dim3(grid - 1 + empty_blocks(a, kEmptyPairs), kMergeSplit),
                                      kMergeThreads, st, a, grid);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace c8

// The tensor-memory kernel for many query rows (tq_cache8_chunk.cu): bf16
// queries and outputs, d 64 or 128.
constexpr int kChunkRows = 256;                      // rows a CTA takes together
constexpr int kChunkUnit = 128;                      // keys per unit
constexpr int kChunkMinUnits = 4;
constexpr int kChunkLead = 4;                        // a segment's start and end, in units
constexpr int kChunkSlice = 256;                     // sequences per launch
bool chunk_supported(int d, bool f32, int rows);
size_t chunk_record_bytes(int d);
cudaError_t launch_chunk(int d, bool int8, const c8::AttnArgs& a, cudaStream_t st);

// The kernel for many query rows that are fp32, or d = 256 (tq_cache8_rows.cu).
constexpr int kRowsTile = 128;                       // rows a CTA takes together
constexpr int kRowsUnit = 64;                        // keys per unit
constexpr int kRowsMinUnits = 4;
constexpr int kRowsLead = 4;                         // a segment's start and end, in units
constexpr int kRowsSlice = 512;                      // sequences per launch
bool rows_supported(int d, bool f32, int rows);
size_t rows_record_bytes(int d);
cudaError_t launch_rows(int d, bool int8, const c8::AttnArgs& a, cudaStream_t st);

}  // namespace tq
