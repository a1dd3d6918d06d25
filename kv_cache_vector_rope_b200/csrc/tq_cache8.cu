// tq_cache8_write / tq_cache8_read: an 8-bit paged KV cache with one
// power-of-two scale for each block of tokens and head.
//
// The work item is one (block that a sequence touches, head), K and V of it:
// its rows are one contiguous piece of each code array and their scales are
// theirs alone, so an item needs nothing from another and no atomics. The
// blocks follow from prefix sums over the sequences, which every CTA forms for
// itself from the lengths in device memory (a call needs no host copy of them).
//
// The scale is the least power of two that brings the block's largest value
// into the codes' range, so that a code times its scale is exact in fp32 and
// bf16 and a block whose values grow is coded anew from its codes alone. New rows stay in registers between the search for the largest
// value and the rounding: each is read once.
//
// Bound by memory, less what the dependent start of an item costs (span, page,
// old scale, rows). Measured, floor of the bytes at the copy's rate in brackets:
// bf16 prompt of 8 x 8192 tokens, 8 heads of 128, written 45.6 us (35.7), read
// back 43.9 us (35.7); one new token of 64 sequences 3.7 us, which is launch and
// that chain of loads; 1000 tokens of 20 heads of 64 read as fp32 4.2 us (2.0).
#include <type_traits>

#include "tq_cache8.h"
#include "tq_device.cuh"

namespace tq {
namespace {

using namespace c8;

struct RowsArgs {
  int d, heads, block, batch;
  int64_t n_blocks;
  uint8_t* code[2];                                  // K, V
  float* scale[2];
  void* x[2];                                        // rows outside the cache: read by write, written by read
  int64_t ts[2], hs[2];
  int64_t n;
  const int32_t* cu;                                 // [batch + 1] of this slice
  const int32_t* start;                              // [batch]
  const int32_t* table;                              // [batch][table_stride] or NULL
  int64_t table_stride;
  int64_t first_seq;                                 // of this slice (table == NULL: pages follow the sequence)
  int32_t* d_status;
  int row_magic;                                     // 2^20 / (pieces per row) + 1
};

// Threads of a CTA whose warps (G = 32) or all of whose threads take an item.
__host__ __device__ constexpr int cta_threads(int G) { return G == 32 ? 64 : 256; }
constexpr int kGroup = 256;                          // G where a CTA takes an item
constexpr int kWriteCtas = 4, kWriteCtasF32 = 2, kReadCtas = 4;   // such CTAs per SM

__device__ __forceinline__ void report(int32_t* d_status, int bit) {
  if (d_status) atomicOr(d_status, bit);
}

// The tokens of sequence b of the slice that this call may touch: rows
// [at, at + n) of x at positions [start, start + n), cut to what x and the
// block table hold.
struct Span {
  int at, n, start;
};
__device__ __forceinline__ Span seq_span(const RowsArgs& a, int b, bool tell) {
  int64_t lo = a.cu[b], hi = a.cu[b + 1];
  const int64_t st = a.start[b];
  bool bad = lo < 0 || hi < lo || hi > a.n || st < 0;
  if (lo < 0 || hi < lo || st < 0) {
    lo = hi = 0;
  } else {
    hi = min(hi, a.n);
    lo = min(lo, hi);
    const int64_t cap = a.table_stride * a.block - st;
    if (hi - lo > cap) {
      bad = true;
      hi = lo + max(cap, static_cast<int64_t>(0));
    }
  }
  if (bad && tell) report(a.d_status, TQ_DEV_BAD_LENGTH);
  return {static_cast<int>(lo), static_cast<int>(hi - lo), st < 0 ? 0 : static_cast<int>(st)};
}

// The sequences' spans, in shared memory: cum[b] is the first block-unit of
// sequence b, a unit being one block that the call touches.
struct Spans {
  int cum[kC8Slice + 1], at[kC8Slice], start[kC8Slice], end[kC8Slice];
  int part[32];
};
template <int T>
__device__ __forceinline__ void scan_spans(const RowsArgs& a, Spans& s) {
  scan_counts<T>(s.cum, s.part, a.batch, [&](int b) {
    const Span x = seq_span(a, b, blockIdx.x == 0);
    s.at[b] = x.at;
    s.start[b] = x.start;
    s.end[b] = x.start + x.n;
    return x.n > 0 ? (x.start % a.block + x.n + a.block - 1) / a.block : 0;
  });
}

// One unit of the walk: rows [r0, r1) of a page; row r0 is row x0 of x.
struct Unit {
  int r0, r1, page;                                  // page -1: outside the cache
  int64_t x0;
};
// b: the unit's sequence, found by moving on from the last unit's.
__device__ __forceinline__ Unit unit_at(const RowsArgs& a, const Spans& s, int u, int& b) {
  while (u >= s.cum[b + 1]) ++b;
  Unit it;
  const int start = s.start[b];
  const int j = start / a.block + (u - s.cum[b]), p0 = j * a.block;
  it.r0 = max(start - p0, 0);
  it.r1 = min(s.end[b] - p0, a.block);
  it.x0 = static_cast<int64_t>(s.at[b]) + p0 + it.r0 - start;
  const int64_t page = a.table ? static_cast<int64_t>(a.table[b * a.table_stride + j]) : (a.first_seq + b) * a.table_stride + j;
  it.page = page >= 0 && page < a.n_blocks ? static_cast<int>(page) : -1;
  return it;
}

// 16 bytes of a row.
__device__ __forceinline__ void store16(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
    w[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight values as loaded, kept in registers between the scale and the codes.
// top: the largest magnitude, as the bits of a float: whole-number order, in
// which infinities and NaN come after every finite value.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ uint32_t top() const {
    float v[8];
    get(v);
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(v[k]) & 0x7fffffffu);
    return m;
  }
};
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = __vmaxu2(__vmaxu2(a.x & 0x7fff7fffu, a.y & 0x7fff7fffu), __vmaxu2(a.z & 0x7fff7fffu, a.w & 0x7fff7fffu));
    return max(m << 16, m & 0xffff0000u);
  }
};

// The two largest values (K's, V's) over the G threads of a group.
template <int G>
__device__ __forceinline__ void group_max(uint32_t (&m)[2], uint2* red) {
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) m[kv] = __reduce_max_sync(0xffffffffu, m[kv]);
  if (G == 32) return;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_uint2(m[0], m[1]);
  __syncthreads();
#pragma unroll
  for (int k = 0; k < G / 32; ++k) {
    m[0] = max(m[0], red[k].x);
    m[1] = max(m[1], red[k].y);
  }
  __syncthreads();
}

// Four codes of finite values that are within the code's range once divided by
// the scale. int8: adding 1.5 * 2^23 rounds to a whole number (ties to even),
// which is then the low byte of the sum.
template <bool INT8>
__device__ __forceinline__ uint32_t encode4_finite(const float* x, float inv) {
  if (INT8) {
    uint32_t y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = __float_as_uint(fmaf(x[k], inv, 12582912.f));
    return __byte_perm(__byte_perm(y[0], y[1], 0x0040), __byte_perm(y[2], y[3], 0x0040), 0x5410);
  }
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0] * inv, x[1] * inv), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2] * inv, x[3] * inv), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

// A group of G threads (the CTA, or a warp) takes an item. Each thread keeps up
// to kKeep pieces of eight values of K and of V in registers from the pass that
// finds the blocks' largest magnitudes to the pass that codes them (all of a
// 64 x 128 block for a CTA); what lies beyond is read again, from L2. The
// largest magnitude is found on the bits, two bf16 values at a time, and says
// whether the block has a value that is not finite; only then does the pass that
// looks at each value run.
constexpr int kKeep = 4;
template <typename T, bool INT8, int G>
__global__ void __launch_bounds__(cta_threads(G), G == 32 ? 1 : sizeof(T) == 2 ? kWriteCtas : kWriteCtasF32) cache8_write_kernel(RowsArgs a) {
  __shared__ Spans spans;
  __shared__ uint2 red[cta_threads(G) / 32];
  const int gt = threadIdx.x % G;                    // thread of the group
  scan_spans<cta_threads(G)>(a, spans);
  const int units = spans.cum[a.batch], step = gridDim.x * (cta_threads(G) / G), head = blockIdx.y;
  const int per_row = a.d / 8;
  int u = blockIdx.x * (cta_threads(G) / G) + threadIdx.x / G;
  int b = u < units ? find_seq(spans.cum, a.batch, u) : 0;
  Unit next;
  if (u < units) next = unit_at(a, spans, u, b);
  for (; u < units; u += step) {
    const Unit it = next;
    if (u + step < units) next = unit_at(a, spans, u + step, b);         // its page is on the way meanwhile
    const int chunks = (it.r1 - it.r0) * per_row;
    const T* x[2];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) x[kv] = static_cast<const T*>(a.x[kv]) + it.x0 * a.ts[kv] + head * a.hs[kv];
    // c / per_row for c < 4096, per_row <= 32: exact, the error is at most c / 2^20 < 1 / 32.
    const auto where = [&](int kv, int c) {
      const int row = (c * a.row_magic) >> 20;
      return x[kv] + row * a.ts[kv] + (c - row * per_row) * 8;
    };
    Raw8<T> raw[2][kKeep];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
      for (int k = 0; k < kKeep; ++k)
        if (gt + k * G < chunks) raw[kv][k].load(where(kv, gt + k * G));
    // The rows do not wait for the page, which a step's one item has just asked for.
    if (it.page < 0) {
      if (gt == 0 && head == 0) report(a.d_status, TQ_DEV_BAD_BLOCK);
      continue;
    }
    const int64_t ph = static_cast<int64_t>(it.page) * a.heads + head;
    float old[2] = {0.f, 0.f};
    if (it.r0 > 0) {
      old[0] = a.scale[0][ph];
      old[1] = a.scale[1][ph];
    }
    uint32_t m[2] = {0u, 0u};
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
      for (int k = 0; k < kKeep; ++k)
        if (gt + k * G < chunks) m[kv] = max(m[kv], raw[kv][k].top());
      for (int c = gt + kKeep * G; c < chunks; c += G) {
        Raw8<T> r;
        r.load(where(kv, c));
        m[kv] = max(m[kv], r.top());
      }
    }
    group_max<G>(m, red);
    const uint32_t most = __float_as_uint(kMost);
    const bool odd = max(m[0], m[1]) > most;         // a value that is not finite (or beyond 2^127): for all threads alike
    if (odd) {
      if (gt == 0) report(a.d_status, TQ_DEV_NONFINITE);
      m[0] = m[1] = 0u;
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv)
#pragma unroll 1
        for (int c = gt; c < chunks; c += G) {
          Raw8<T> r;
          r.load(where(kv, c));
          float v[8];
          r.get(v);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t y = __float_as_uint(v[e]) & 0x7fffffffu;
            if (y <= most) m[kv] = max(m[kv], y);
          }
        }
      group_max<G>(m, red);
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint8_t* dst = a.code[kv] + ph * a.block * a.d;
      float scale = block_scale<INT8>(__uint_as_float(m[kv]));
      if (it.r0 > 0) {                               // the block holds tokens: its scale may only grow
        if (old[kv] >= scale) {
          scale = old[kv];
        } else {
          const float ratio = old[kv] * inv_pow2(scale);
#pragma unroll 1
          for (int c = gt; c < it.r0 * per_row; c += G) {
            uint2* p = reinterpret_cast<uint2*>(dst) + c;
            const uint2 w = *p;
            const uint32_t ws[2] = {w.x, w.y};
            uint32_t o[2] = {0u, 0u};
#pragma unroll
            for (int e = 0; e < 8; ++e)
              o[e >> 2] |= encode<INT8>(decode<INT8>((ws[e >> 2] >> (8 * (e & 3))) & 0xffu) * ratio) << (8 * (e & 3));
            *p = make_uint2(o[0], o[1]);
          }
        }
      }
      const float inv = inv_pow2(scale);
      uint2* row0 = reinterpret_cast<uint2*>(dst + static_cast<int64_t>(it.r0) * a.d);
      const auto put = [&](const Raw8<T>& r, int c) {
        float v[8];
        r.get(v);
        row0[c] = make_uint2(encode4_finite<INT8>(v, inv), encode4_finite<INT8>(v + 4, inv));
      };
      if (odd) {
#pragma unroll 1
        for (int c = gt; c < chunks; c += G) {
          Raw8<T> r;
          r.load(where(kv, c));
          float v[8];
          r.get(v);
          uint32_t o[2] = {0u, 0u};
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e >> 2] |= encode<INT8>(v[e] * inv) << (8 * (e & 3));
          row0[c] = make_uint2(o[0], o[1]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < kKeep; ++k)
          if (gt + k * G < chunks) put(raw[kv][k], gt + k * G);
        for (int c = gt + kKeep * G; c < chunks; c += G) {
          Raw8<T> r;
          r.load(where(kv, c));
          put(r, c);
        }
      }
      if (gt == 0) a.scale[kv][ph] = scale;          // every thread has read the old one: group_max lies between
    }
  }
}

// Reading back: a piece is what makes 16 bytes of output (8 codes for bf16, 4
// for fp32), so that a warp's loads and stores are both contiguous; 4 KB of
// codes of K and of V are in flight per CTA and pass.
template <typename T, bool INT8, int G>
__global__ void __launch_bounds__(cta_threads(G), G == 32 ? 1 : kReadCtas) cache8_read_kernel(RowsArgs a) {
  constexpr int P = 16 / sizeof(T);
  constexpr int kPieces = 32 / P;                    // 32 codes a thread
  using Raw = typename std::conditional<P == 8, uint2, uint32_t>::type;
  __shared__ Spans spans;
  const int gt = threadIdx.x % G;
  scan_spans<cta_threads(G)>(a, spans);
  const int units = spans.cum[a.batch], step = gridDim.x * (cta_threads(G) / G), head = blockIdx.y;
  const int per_row = a.d / P;
  int u = blockIdx.x * (cta_threads(G) / G) + threadIdx.x / G;
  int b = u < units ? find_seq(spans.cum, a.batch, u) : 0;
  Unit next;
  if (u < units) next = unit_at(a, spans, u, b);
  for (; u < units; u += step) {
    const Unit it = next;
    if (u + step < units) next = unit_at(a, spans, u + step, b);
    const bool ok = it.page >= 0;
    if (!ok && gt == 0 && head == 0) report(a.d_status, TQ_DEV_BAD_BLOCK);
    const int64_t ph = static_cast<int64_t>(ok ? it.page : 0) * a.heads + head;
    const int chunks = (it.r1 - it.r0) * per_row;
    for (int c0 = gt; c0 < chunks; c0 += kPieces * G) {
      Raw raw[2][kPieces];
      float scale[2];
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        if (!a.x[kv]) continue;
        const Raw* src = reinterpret_cast<const Raw*>(a.code[kv] + (ph * a.block + it.r0) * a.d);
        scale[kv] = ok ? a.scale[kv][ph] : 0.f;
#pragma unroll
        for (int k = 0; k < kPieces; ++k)
          if (c0 + k * G < chunks) raw[kv][k] = ok ? src[c0 + k * G] : Raw();
      }
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        if (!a.x[kv]) continue;
        T* x = static_cast<T*>(a.x[kv]) + it.x0 * a.ts[kv] + head * a.hs[kv];
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
          const int c = c0 + k * G;
          if (c >= chunks) break;
          const int row = (c * a.row_magic) >> 20;   // c / per_row, as above (c < 8192, per_row <= 64)
          const uint32_t* ws = reinterpret_cast<const uint32_t*>(&raw[kv][k]);
          float v[P];
#pragma unroll
          for (int h = 0; h < P / 4; ++h) decode4<INT8>(ws[h], v + 4 * h);
#pragma unroll
          for (int e = 0; e < P; ++e) v[e] *= scale[kv];
          store16(x + row * a.ts[kv] + (c - row * per_row) * P, v);
        }
      }
    }
  }
}

template <bool WRITE, typename T, bool INT8>
void launch_group(bool warps, dim3 grid, const RowsArgs& a, cudaStream_t st) {
  if (WRITE) {
    if (warps) cache8_write_kernel<T, INT8, 32><<<grid, cta_threads(32), 0, st>>>(a);
    else cache8_write_kernel<T, INT8, kGroup><<<grid, cta_threads(kGroup), 0, st>>>(a);
  } else {
    if (warps) cache8_read_kernel<T, INT8, 32><<<grid, cta_threads(32), 0, st>>>(a);
    else cache8_read_kernel<T, INT8, kGroup><<<grid, cta_threads(kGroup), 0, st>>>(a);
  }
}

template <bool WRITE>
cudaError_t launch_rows(const tq_cache8* c, tq_dtype dtype, RowsArgs a, int64_t batch, cudaStream_t st) {
  const int32_t *cu = a.cu, *start = a.start, *table = a.table;
  const int per_row = a.d / (WRITE || dtype == TQ_BF16 ? 8 : 4);
  a.row_magic = (1 << 20) / per_row + 1;
  // A warp per item where a warp holds an item's new rows in registers, since blocks are that small or the call's
  // sequences bring so few tokens; else a CTA per item. (1000 tokens in blocks of 16, 20 heads of 64, read back: 4.3 us
  // against 8.3 with a CTA per item.)
  const int64_t tokens = a.n / batch < c->block ? a.n / batch : c->block;
  const bool warps = tokens * a.d <= 32 * kKeep * 8;
  for (int64_t b0 = 0; b0 < batch; b0 += kC8Slice) {
    const int64_t nb = batch - b0 < kC8Slice ? batch - b0 : kC8Slice;
    a.batch = static_cast<int>(nb);
    a.first_seq = b0;
    a.cu = cu + b0;
    a.start = start + b0;
    a.table = table ? table + b0 * a.table_stride : nullptr;
    // Blocks touched: at most one per token, and two partial ones per sequence beside the full ones.
    const int64_t full = a.n / c->block + 2 * nb, units = a.n < full ? a.n : full;
    const int64_t ctas = warps ? (units + cta_threads(32) / 32 - 1) / (cta_threads(32) / 32) : units;
    // About three waves of CTAs, a few blocks each (at three CTAs per SM a prompt write took 50.4 us, with 1, 2 and 8 waves 67, 52 and 55).
    const int64_t most = (148 * 12 + c->heads - 1) / c->heads;
    const dim3 grid(static_cast<unsigned>(ctas < most ? ctas : most), static_cast<unsigned>(c->heads));
    if (dtype == TQ_F32) {
      if (c->code == TQ_INT8) launch_group<WRITE, float, true>(warps, grid, a, st);
      else launch_group<WRITE, float, false>(warps, grid, a, st);
    } else {
      if (c->code == TQ_INT8) launch_group<WRITE, __nv_bfloat16, true>(warps, grid, a, st);
      else launch_group<WRITE, __nv_bfloat16, false>(warps, grid, a, st);
    }
    count_launch();
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <bool WRITE>
tq_status rows_call(const char* what, const tq_cache8* cache, tq_dtype dtype, const void* k, int64_t k_ts, int64_t k_hs,
                    const void* v, int64_t v_ts, int64_t v_hs, int64_t n_tokens, int32_t batch, const int32_t* cu_tokens,
                    const int32_t* start, const int32_t* block_table, int64_t table_stride, int32_t* d_status,
                    void* stream) {
  clear_error();
  tq_status st = check_cache8(cache, what);
  if (st != TQ_OK) return st;
  if (dtype != TQ_F32 && dtype != TQ_BF16) return fail(TQ_ERR_INVALID_ARG, "%s: dtype must be TQ_F32 or TQ_BF16", what);
  if (n_tokens < 0 || n_tokens > 0x7fffffff || batch < 0)
    return fail(TQ_ERR_INVALID_ARG, "%s: n_tokens must be in [0, 2^31) and batch >= 0", what);
  if (n_tokens == 0 || batch == 0) return TQ_OK;
  if (!cu_tokens || !start) return fail(TQ_ERR_INVALID_ARG, "%s: NULL cu_tokens or start", what);
  if (WRITE ? (!k || !v) : (!k && !v)) return fail(TQ_ERR_INVALID_ARG, "%s: NULL rows", what);
  st = check_table8(cache, batch, table_stride, what);
  if (st != TQ_OK) return st;
  if (!block_table && table_stride * batch > cache->n_blocks)
    return fail(TQ_ERR_INVALID_ARG, "%s: without a block table the cache needs batch * table_stride blocks", what);
  const struct {
    const void* p;
    int64_t ts, hs;
  } side[2] = {{k, k_ts, k_hs}, {v, v_ts, v_hs}};
  for (const auto& s : side) {
    if (!s.p) continue;
    if (!aligned(s.p, 16) || !stride_ok(n_tokens, s.ts, 8) || !stride_ok(cache->heads, s.hs, 8))
      return fail(TQ_ERR_INVALID_ARG, "%s: rows must be 16-byte aligned, strides multiples of 8 elements, not negative",
                  what);
    if (!WRITE && rows_overlap(n_tokens, s.ts, cache->heads, s.hs, cache->d))
      return fail(TQ_ERR_INVALID_ARG, "%s: the strides make rows overlap", what);
  }
  RowsArgs a{cache->d, cache->heads, cache->block, 0, cache->n_blocks, {cache->k, cache->v},
             {cache->k_scale, cache->v_scale}, {const_cast<void*>(k), const_cast<void*>(v)}, {k_ts, v_ts}, {k_hs, v_hs},
             n_tokens, cu_tokens, start, block_table, table_stride, 0, d_status, 0};
  const cudaError_t e = launch_rows<WRITE>(cache, dtype, a, batch, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(TQ_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
  return TQ_OK;
}

}  // namespace

EncodeTiledFn encode_tiled_fn() {
  static const EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool got = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                     q == cudaDriverEntryPointSuccess;
    return got ? reinterpret_cast<EncodeTiledFn>(p) : nullptr;
  }();
  return fn;
}

// The sizes of a cache; a code array stays below 2^62 bytes.
static tq_status check_sizes8(int32_t d, int32_t heads, int32_t block, int64_t n_blocks, int64_t least, const char* what) {
  if (d < 16 || d > kMaxD || d % 16 != 0)
    return fail(TQ_ERR_INVALID_ARG, "%s: d must be a multiple of 16 in [16, %d] (got %d)", what, kMaxD, d);
  if (block != 16 && block != 32 && block != 64 && block != 128)
    return fail(TQ_ERR_INVALID_ARG, "%s: block must be 16, 32, 64 or 128 tokens (got %d)", what, block);
  if (heads < 1 || heads > 65535) return fail(TQ_ERR_INVALID_ARG, "%s: heads must be in [1, 65535]", what);
  if (n_blocks < least || n_blocks > 0x7fffffff)
    return fail(TQ_ERR_INVALID_ARG, "%s: n_blocks must be in [%d, 2^31)", what, static_cast<int>(least));
  return TQ_OK;
}

tq_status check_cache8(const tq_cache8* c, const char* what) {
  if (!c) return fail(TQ_ERR_INVALID_ARG, "%s: cache is NULL", what);
  const tq_status st = check_sizes8(c->d, c->heads, c->block, c->n_blocks, 1, what);
  if (st != TQ_OK) return st;
  if (c->code != TQ_E4M3 && c->code != TQ_INT8)
    return fail(TQ_ERR_INVALID_ARG, "%s: code must be TQ_E4M3 or TQ_INT8", what);
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return fail(TQ_ERR_INVALID_ARG, "%s: NULL cache pointer", what);
  if (!aligned(c->k, 128) || !aligned(c->v, 128) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return fail(TQ_ERR_INVALID_ARG, "%s: code arrays must be 128-byte aligned", what);
  return TQ_OK;
}

tq_status check_table8(const tq_cache8* c, int32_t batch, int64_t table_stride, const char* what) {
  if (batch < 1) return fail(TQ_ERR_INVALID_ARG, "%s: batch must be positive", what);
  if (table_stride < 1 || table_stride > 0x7fffff80 / c->block)
    return fail(TQ_ERR_INVALID_ARG, "%s: table_stride * block must be in [block, 2^31)", what);
  return TQ_OK;
}

}  // namespace tq

extern "C" {

int64_t tq_cache8_bytes(int32_t d, int32_t heads, int32_t block, int64_t n_blocks) {
  tq::clear_error();
  if (tq::check_sizes8(d, heads, block, n_blocks, 0, "tq_cache8_bytes") != TQ_OK) return -1;
  const int64_t page = 2 * static_cast<int64_t>(heads) * (static_cast<int64_t>(block) * d + static_cast<int64_t>(sizeof(float)));
  if (n_blocks > INT64_MAX / page) {
    tq::fail(TQ_ERR_INVALID_ARG, "tq_cache8_bytes: 2^63 bytes or more");
    return -1;
  }
  return n_blocks * page;
}

tq_status tq_cache8_write(const tq_cache8* cache, tq_dtype dtype, const void* k, int64_t k_token_stride,
                          int64_t k_head_stride, const void* v, int64_t v_token_stride, int64_t v_head_stride,
                          int64_t n_tokens, int32_t batch, const int32_t* cu_tokens, const int32_t* start,
                          const int32_t* block_table, int64_t table_stride, int32_t* d_status, void* stream) {
  return tq::rows_call<true>("tq_cache8_write", cache, dtype, k, k_token_stride, k_head_stride, v, v_token_stride,
                             v_head_stride, n_tokens, batch, cu_tokens, start, block_table, table_stride, d_status,
                             stream);
}

tq_status tq_cache8_read(const tq_cache8* cache, tq_dtype dtype, void* k_out, int64_t k_token_stride,
                         int64_t k_head_stride, void* v_out, int64_t v_token_stride, int64_t v_head_stride,
                         int64_t n_tokens, int32_t batch, const int32_t* cu_tokens, const int32_t* start,
                         const int32_t* block_table, int64_t table_stride, int32_t* d_status, void* stream) {
  return tq::rows_call<false>("tq_cache8_read", cache, dtype, k_out, k_token_stride, k_head_stride, v_out,
                              v_token_stride, v_head_stride, n_tokens, batch, cu_tokens, start, block_table,
                              table_stride, d_status, stream);
}

}  // extern "C"
