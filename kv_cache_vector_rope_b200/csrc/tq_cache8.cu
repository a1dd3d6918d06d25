// tq_cache8_write / tq_cache8_read: an 8-bit paged KV cache with one
// power-of-two scale for each block of tokens and head.
//
// The work item is one (block a sequence touches, head, K or V): its rows are
// one contiguous piece of the cache, and its scale is theirs alone, so an item
// needs nothing from another and no atomics. The items follow from the prefix
// sums of the blocks each sequence touches, which every CTA forms for itself
// from the lengths in device memory (a call needs no host copy of them).
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

constexpr int kRowThreads = 256;

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

// One item of the walk: rows [r0, r1) of head `head` of a page, K or V; row r0 is row x0 of x.
struct Item {
  int kv, head, r0, r1;
  int page;
  int64_t x0;
};
__device__ __forceinline__ Item item_at(const RowsArgs& a, const Spans& s, int64_t item) {
  Item it;
  const bool both = a.x[0] && a.x[1];
  const unsigned per = static_cast<unsigned>(a.heads) * (both ? 2u : 1u);
  const int u = static_cast<int>(item / per);
  const unsigned rest = static_cast<unsigned>(item - static_cast<int64_t>(u) * per);
  it.kv = both ? rest >= static_cast<unsigned>(a.heads) : (a.x[0] ? 0 : 1);
  it.head = static_cast<int>(rest) - (both ? it.kv * a.heads : 0);
  const int b = find_seq(s.cum, a.batch, u);
  const int start = s.start[b];
  const int j = start / a.block + (u - s.cum[b]), p0 = j * a.block;
  it.r0 = max(start - p0, 0);
  it.r1 = min(s.end[b] - p0, a.block);
  it.x0 = static_cast<int64_t>(s.at[b]) + p0 + it.r0 - start;
  const int64_t page = a.table ? static_cast<int64_t>(a.table[b * a.table_stride + j]) : (a.first_seq + b) * a.table_stride + j;
  it.page = page >= 0 && page < a.n_blocks ? static_cast<int>(page) : -1;
  return it;
}

// Eight values of a row.
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
    w[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight values as loaded, kept in registers between the scale and the codes.
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
};

// Largest of `m` over the G threads of a group.
template <int G>
__device__ __forceinline__ float group_max(float m, float* red) {
  m = dev::warp_max(m);
  if (G == 32) return m;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < G / 32; ++k) m = fmaxf(m, red[k]);
  __syncthreads();
  return m;
}

// A group of G threads (the CTA, or a warp) takes an item. Each thread keeps up
// to kKeep pieces of eight values in registers from the pass that finds the
// block's largest magnitude to the pass that codes them (all of a 64 x 128
// block for a CTA); what lies beyond is read again, from L2.
constexpr int kKeep = 4;
template <typename T, bool INT8, int G>
__global__ void __launch_bounds__(kRowThreads) cache8_write_kernel(RowsArgs a) {
  __shared__ Spans spans;
  __shared__ float red[kRowThreads / 32];
  const int gt = threadIdx.x % G;                    // thread of the group
  scan_spans<kRowThreads>(a, spans);
  const int64_t items = static_cast<int64_t>(spans.cum[a.batch]) * 2 * a.heads;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kRowThreads / G);
  const int per_row = a.d / 8;
  int64_t item = static_cast<int64_t>(blockIdx.x) * (kRowThreads / G) + threadIdx.x / G;
  Item next = item < items ? item_at(a, spans, item) : Item();
  for (; item < items; item += step) {
    const Item it = next;
    if (item + step < items) next = item_at(a, spans, item + step);      // its page is on the way meanwhile
    if (it.page < 0) {
      if (gt == 0) report(a.d_status, TQ_DEV_BAD_BLOCK);
      continue;
    }
    const int kv = it.kv;
    const int64_t ts = a.ts[kv];
    const T* x = static_cast<const T*>(a.x[kv]) + it.x0 * ts + it.head * a.hs[kv];
    const int64_t ph = static_cast<int64_t>(it.page) * a.heads + it.head;
    uint8_t* dst = a.code[kv] + ph * a.block * a.d;
    const int chunks = (it.r1 - it.r0) * per_row;
    // c / per_row for c < 4096, per_row <= 32: exact, the error is at most c / 2^20 < 1 / 32.
    const auto where = [&](int c) {
      const int row = (c * a.row_magic) >> 20;
      return x + row * ts + (c - row * per_row) * 8;
    };
    const float old = it.r0 > 0 ? a.scale[kv][ph] : 0.f;
    Raw8<T> raw[kKeep];
#pragma unroll
    for (int k = 0; k < kKeep; ++k)
      if (gt + k * G < chunks) raw[k].load(where(gt + k * G));
    float m = 0.f;
    bool odd = false;
    const auto look = [&](const Raw8<T>& r) {
      float v[8];
      r.get(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float u = fabsf(v[e]);
        if (u <= kMost) m = fmaxf(m, u); else odd = true;
      }
    };
#pragma unroll
    for (int k = 0; k < kKeep; ++k)
      if (gt + k * G < chunks) look(raw[k]);
    for (int c = gt + kKeep * G; c < chunks; c += G) {
      Raw8<T> r;
      r.load(where(c));
      look(r);
    }
    if (odd) report(a.d_status, TQ_DEV_NONFINITE);
    m = group_max<G>(m, red);
    float scale = block_scale<INT8>(m);
    if (it.r0 > 0) {                                 // the block holds tokens: its scale may only grow
      if (old >= scale) {
        scale = old;
      } else {
        const float ratio = old * inv_pow2(scale);
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
    uint8_t* row0 = dst + static_cast<int64_t>(it.r0) * a.d;
    const auto put = [&](const Raw8<T>& r, int c) {
      float v[8];
      r.get(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= inv;
      *reinterpret_cast<uint2*>(row0 + c * 8) = make_uint2(encode4<INT8>(v), encode4<INT8>(v + 4));
    };
#pragma unroll
    for (int k = 0; k < kKeep; ++k)
      if (gt + k * G < chunks) put(raw[k], gt + k * G);
    for (int c = gt + kKeep * G; c < chunks; c += G) {
      Raw8<T> r;
      r.load(where(c));
      put(r, c);
    }
    // Every thread has read the old scale: group_max lies between.
    if (gt == 0) a.scale[kv][ph] = scale;
  }
}

// Reading back: a thread takes 16 codes at a time, four such pieces in flight.
template <typename T, bool INT8, int G>
__global__ void __launch_bounds__(kRowThreads) cache8_read_kernel(RowsArgs a) {
  __shared__ Spans spans;
  const int gt = threadIdx.x % G;
  scan_spans<kRowThreads>(a, spans);
  const int64_t items = static_cast<int64_t>(spans.cum[a.batch]) * (a.x[0] && a.x[1] ? 2 : 1) * a.heads;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kRowThreads / G);
  const int per_row = a.d / 16;
  int64_t item = static_cast<int64_t>(blockIdx.x) * (kRowThreads / G) + threadIdx.x / G;
  Item next = item < items ? item_at(a, spans, item) : Item();
  for (; item < items; item += step) {
    const Item it = next;
    if (item + step < items) next = item_at(a, spans, item + step);
    const bool ok = it.page >= 0;
    if (!ok && gt == 0) report(a.d_status, TQ_DEV_BAD_BLOCK);
    const int kv = it.kv;
    const int64_t ts = a.ts[kv];
    T* x = static_cast<T*>(a.x[kv]) + it.x0 * ts + it.head * a.hs[kv];
    const int64_t ph = static_cast<int64_t>(ok ? it.page : 0) * a.heads + it.head;
    const float scale = ok ? a.scale[kv][ph] : 0.f;
    const uint4* src = reinterpret_cast<const uint4*>(a.code[kv] + (ph * a.block + it.r0) * a.d);
    const int chunks = (it.r1 - it.r0) * per_row;
    for (int c0 = gt; c0 < chunks; c0 += kKeep * G) {
      uint4 raw[kKeep];
#pragma unroll
      for (int k = 0; k < kKeep; ++k)
        if (c0 + k * G < chunks) raw[k] = ok ? __ldg(src + c0 + k * G) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int k = 0; k < kKeep; ++k) {
        const int c = c0 + k * G;
        if (c >= chunks) break;
        const int row = (c * a.row_magic) >> 20;     // c / per_row, as above
        T* p = x + row * ts + (c - row * per_row) * 16;
        const uint32_t ws[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v[8];
          decode4<INT8>(ws[2 * h], v);
          decode4<INT8>(ws[2 * h + 1], v + 4);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= scale;
          store8(p + 8 * h, v);
        }
      }
    }
  }
}

template <bool WRITE, typename T, bool INT8>
void launch_group(bool warps, unsigned grid, const RowsArgs& a, cudaStream_t st) {
  if (WRITE) {
    if (warps) cache8_write_kernel<T, INT8, 32><<<grid, kRowThreads, 0, st>>>(a);
    else cache8_write_kernel<T, INT8, kRowThreads><<<grid, kRowThreads, 0, st>>>(a);
  } else {
    if (warps) cache8_read_kernel<T, INT8, 32><<<grid, kRowThreads, 0, st>>>(a);
    else cache8_read_kernel<T, INT8, kRowThreads><<<grid, kRowThreads, 0, st>>>(a);
  }
}

template <bool WRITE>
cudaError_t launch_rows(const tq_cache8* c, tq_dtype dtype, RowsArgs a, int64_t batch, cudaStream_t st) {
  const int32_t *cu = a.cu, *start = a.start, *table = a.table;
  const int per_row = a.d / (WRITE ? 8 : 16);
  a.row_magic = (1 << 20) / per_row + 1;
  // A warp per item where the call's sequences bring so few tokens that a warp
  // holds an item's new rows in registers; else a CTA per item.
  const bool warps = a.n / batch * (a.d / 8) <= 32 * kKeep;
  for (int64_t b0 = 0; b0 < batch; b0 += kC8Slice) {
    const int64_t nb = batch - b0 < kC8Slice ? batch - b0 : kC8Slice;
    a.batch = static_cast<int>(nb);
    a.first_seq = b0;
    a.cu = cu + b0;
    a.start = start + b0;
    a.table = table ? table + b0 * a.table_stride : nullptr;
    // Blocks touched: at most one per token, and two partial ones per sequence beside the full ones.
    const int64_t full = a.n / c->block + 2 * nb;
    const int64_t items = (a.n < full ? a.n : full) * c->heads * (a.x[0] && a.x[1] ? 2 : 1);
    const int64_t ctas = warps ? (items + kRowThreads / 32 - 1) / (kRowThreads / 32) : items;
    const int64_t most = 148 * 8;
    const unsigned grid = static_cast<unsigned>(ctas < most ? ctas : most);
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

tq_status check_cache8(const tq_cache8* c, const char* what) {
  if (!c) return fail(TQ_ERR_INVALID_ARG, "%s: cache is NULL", what);
  if (c->d < 16 || c->d > kMaxD || c->d % 16 != 0)
    return fail(TQ_ERR_INVALID_ARG, "%s: d must be a multiple of 16 in [16, %d] (got %d)", what, kMaxD, c->d);
  if (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128)
    return fail(TQ_ERR_INVALID_ARG, "%s: block must be 16, 32, 64 or 128 tokens (got %d)", what, c->block);
  if (c->code != TQ_E4M3 && c->code != TQ_INT8)
    return fail(TQ_ERR_INVALID_ARG, "%s: code must be TQ_E4M3 or TQ_INT8", what);
  if (c->heads < 1 || c->heads > 65536) return fail(TQ_ERR_INVALID_ARG, "%s: heads must be in [1, 65536]", what);
  if (c->n_blocks < 1 || c->n_blocks > 0x7fffffff)
    return fail(TQ_ERR_INVALID_ARG, "%s: n_blocks must be in [1, 2^31)", what);
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
  if (d < 16 || d > tq::kMaxD || d % 16 != 0 || heads < 1 || block < 1 || n_blocks < 0) return -1;
  return 2 * n_blocks * heads * (static_cast<int64_t>(block) * d + static_cast<int64_t>(sizeof(float)));
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
