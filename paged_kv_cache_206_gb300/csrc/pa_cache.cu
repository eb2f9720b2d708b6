// Norm and rotation of query and key heads, and the 8-bit cache written and
// read back (pa_cache.h).
#include <cuda_runtime.h>

#include <cmath>

#include "pa_cache.h"
#include "pa_device.cuh"
#include "pa_e4m3.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

enum RowMode { kRotate, kWrite, kStore };

struct RowParams {
  const __half *query, *key, *value, *q_weight, *k_weight;
  const float* cos_sin;
  const int32_t *positions, *block_tables, *context_lens, *q_seqlens;
  __half *q_out, *k_out;
  uint8_t *key_cache, *key_exps, *value_cache, *value_exps;
  uint32_t* status;
  int64_t tokens, query_stride, key_stride, value_stride;
  int batch, heads, kv_heads, hk, hv, rot, interleaved, max_positions;
  int block_size, num_blocks, max_blocks_per_seq, max_rows;
  int lanes;  // lanes of a row, a power of two
  float eps;
};

__device__ __forceinline__ void report(uint32_t* status, uint32_t bit) {
  if (status) atomicOr(status, bit);
}

// Sequence and index in it of token t: the last sequence whose tokens begin at
// or before t. Warp-collective; -1 past the last sequence.
__device__ __forceinline__ int find_sequence(const RowParams& P, int64_t t, int lane, int& index) {
  if (!P.q_seqlens) {
    index = 0;
    return t < P.batch ? int(t) : -1;
  }
  int64_t before = 0;
  for (int b0 = 0; b0 < P.batch; b0 += 32) {
    const int n = b0 + lane < P.batch ? min(max(P.q_seqlens[b0 + lane], 0), P.max_rows) : 0;
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    const bool mine = n > 0 && t >= before + sum - n && t < before + sum;
    const unsigned who = __ballot_sync(0xffffffffu, mine);
    if (who) {
      const int l = __ffs(who) - 1;
      index = int(t - before) - __shfl_sync(0xffffffffu, sum - n, l);
      return b0 + l;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  return -1;
}

// One warp per (token, slice of its head rows). A row's elements are 16-byte
// chunks of 8; a lane holds chunks p and p + rot / 16 of the rotated part (so
// that both members of every pair are its own, in either pairing), and two
// neighbouring chunks of the rest.
template <int MODE, int VPL>
__global__ void __launch_bounds__(256) rows_kernel(const RowParams P) {
  const int lane = threadIdx.x & 31;
  const int per_warp = 32 / P.lanes, group = lane / P.lanes, gl = lane % P.lanes;
  const int qrows = MODE == kWrite ? 0 : P.heads;
  const int rows = qrows + P.kv_heads * (MODE == kRotate ? 1 : 2);
  const int slices = (rows + per_warp - 1) / per_warp;
  const int64_t task = int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int64_t t = task / slices;
  if (t >= P.tokens) return;
  const int row = int(task % slices) * per_warp + group;

  // ---- where the token goes
  int64_t slot = -1;
  int block = 0, place = 0, pos = 0;
  if constexpr (MODE == kRotate) {
    pos = P.positions[t];
  } else {
    int i = 0;
    const int b = find_sequence(P, t, lane, i);
    if (b < 0) return;
    const int q = P.q_seqlens ? P.q_seqlens[b] : 1, L = P.context_lens[b];
    if (q > P.max_rows || L < q || int64_t(L) > int64_t(P.max_blocks_per_seq) * P.block_size) {
      report(P.status, PA_STATUS_BIT_PLAN);
      return;
    }
    pos = L - q + i;
    block = P.block_tables[int64_t(b) * P.max_blocks_per_seq + pos / P.block_size];
    place = pos % P.block_size;
    if (block >= 0 && block < P.num_blocks) slot = int64_t(block) * P.block_size + place;
    else report(P.status, PA_STATUS_BIT_BLOCK_INDEX);
    if (MODE == kStore && P.positions) pos = P.positions[t];
  }
  if (MODE != kWrite) {
    if (pos < -1 || pos >= P.max_positions) report(P.status, PA_STATUS_BIT_POSITION);
    if (pos < 0 || pos >= P.max_positions) return;
  }
  const bool is_q = row < qrows, is_k = !is_q && row < qrows + P.kv_heads;
  const bool is_v = !is_q && !is_k && row < rows;
  const int h = is_q ? row : is_k ? row - qrows : row - qrows - P.kv_heads;
  const int dims = is_v ? P.hv : P.hk;
  const __half* src = is_q   ? P.query + t * P.query_stride + int64_t(h) * P.hk
                      : is_k ? P.key + t * P.key_stride + int64_t(h) * P.hk
                      : is_v ? P.value + t * P.value_stride + int64_t(h) * P.hv
                             : nullptr;
  const __half* weight = is_q ? P.q_weight : is_k ? P.k_weight : nullptr;
  const int rot = is_v || MODE == kWrite ? 0 : P.rot, half = rot / 16;

  // ---- the row's elements
  float y[VPL][2][8];
  int at[VPL][2];
  float sq = 0.f;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int p = gl + v * P.lanes;
    at[v][0] = p < half ? p * 8 : (rot / 8 + 2 * (p - half)) * 8;
    at[v][1] = p < half ? (p + half) * 8 : at[v][0] + 8;
    const bool on = src && p < dims / 16;
    if (!on) at[v][0] = at[v][1] = -1;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (on) x = *reinterpret_cast<const uint4*>(src + at[v][c]);
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&x);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = h2f2(w[j]);
        y[v][c][2 * j] = f.x;
        y[v][c][2 * j + 1] = f.y;
        sq += f.x * f.x + f.y * f.y;
      }
    }
  }
  if constexpr (MODE != kWrite) {
    for (int o = P.lanes >> 1; o; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    const float inv = 1.0f / sqrtf(sq / float(P.hk) + P.eps);
    const float* table = P.cos_sin + int64_t(pos) * P.rot;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      if (at[v][0] < 0) continue;
      if (weight) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint4 x = *reinterpret_cast<const uint4*>(weight + at[v][c]);
          const uint32_t* w = reinterpret_cast<const uint32_t*>(&x);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = h2f2(w[j]);
            y[v][c][2 * j] *= inv * f.x;
            y[v][c][2 * j + 1] *= inv * f.y;
          }
        }
      }
      if (at[v][0] < rot) {
        if (P.interleaved) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float4 cs = *reinterpret_cast<const float4*>(table + at[v][c] / 2);
            const float4 sn = *reinterpret_cast<const float4*>(table + rot / 2 + at[v][c] / 2);
            const float* cc = reinterpret_cast<const float*>(&cs);
            const float* ss = reinterpret_cast<const float*>(&sn);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float a = y[v][c][2 * j], b = y[v][c][2 * j + 1];
              y[v][c][2 * j] = a * cc[j] - b * ss[j];
              y[v][c][2 * j + 1] = b * cc[j] + a * ss[j];
            }
          }
        } else {
#pragma unroll
          for (int j4 = 0; j4 < 2; ++j4) {
            const float4 cs = *reinterpret_cast<const float4*>(table + at[v][0] + 4 * j4);
            const float4 sn = *reinterpret_cast<const float4*>(table + rot / 2 + at[v][0] + 4 * j4);
            const float* cc = reinterpret_cast<const float*>(&cs);
            const float* ss = reinterpret_cast<const float*>(&sn);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float a = y[v][0][4 * j4 + j], b = y[v][1][4 * j4 + j];
              y[v][0][4 * j4 + j] = a * cc[j] - b * ss[j];
              y[v][1][4 * j4 + j] = b * cc[j] + a * ss[j];
            }
          }
        }
      }
    }
  }

  // ---- fp16 rows: the queries, and the keys of a plain rotation
  const bool dense = MODE != kWrite && (is_q || (MODE == kRotate && is_k));
  if (dense) {
    __half* dst = is_q ? P.q_out + (t * P.heads + h) * P.hk : P.k_out + (t * P.kv_heads + h) * P.hk;
#pragma unroll
    for (int v = 0; v < VPL; ++v)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (at[v][c] < 0) continue;
        const float* f = y[v][c];
        *reinterpret_cast<uint4*>(dst + at[v][c]) =
            make_uint4(pack_half2(f[0], f[1]), pack_half2(f[2], f[3]), pack_half2(f[4], f[5]),
                       pack_half2(f[6], f[7]));
      }
  }
  if constexpr (MODE != kRotate) {
    // ---- 8-bit rows: the exponent that the row's largest finite element
    // needs, then the codes (scaling by a power of two is exact)
    float top = 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          top = fmaxf(top, isfinite(y[v][c][j]) ? fabsf(y[v][c][j]) : 0.f);
    for (int o = P.lanes >> 1; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((is_k || is_v) && slot >= 0) {
      const int e = row_exponent(top);
      const float f = pow2(-e);
      uint8_t* dst = is_k ? P.key_cache + (slot * P.kv_heads + h) * P.hk
                          : P.value_cache + (slot * P.kv_heads + h) * P.hv;
#pragma unroll
      for (int v = 0; v < VPL; ++v)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (at[v][c] < 0) continue;
          const float* x = y[v][c];
          const uint32_t lo = e4m3x2(x[0] * f, x[1] * f) | e4m3x2(x[2] * f, x[3] * f) << 16;
          const uint32_t hi = e4m3x2(x[4] * f, x[5] * f) | e4m3x2(x[6] * f, x[7] * f) << 16;
          *reinterpret_cast<uint2*>(dst + at[v][c]) = make_uint2(lo, hi);
        }
      if (gl == 0) {
        uint8_t* exps = is_k ? P.key_exps : P.value_exps;
        exps[(int64_t(block) * P.kv_heads + h) * P.block_size + place] = uint8_t(e + kExpBias);
      }
    }
  }
}

template <int MODE>
pa_status launch_rows(RowParams P, cudaStream_t stream) {
  if (P.tokens == 0) return PA_OK;
  const int widest = (MODE == kRotate || P.hk > P.hv ? P.hk : P.hv) / 16;  // lanes' worth of chunk pairs
  P.lanes = 1;
  while (P.lanes < 32 && P.lanes < widest) P.lanes *= 2;
  const int rows = (MODE == kWrite ? 0 : P.heads) + P.kv_heads * (MODE == kRotate ? 1 : 2);
  const int64_t warps = P.tokens * cdiv(rows, 32 / P.lanes);
  const int64_t grid = cdiv(warps, 8);
  if (grid > INT32_MAX) return PA_ERR_INVALID_ARG;
  if (widest <= 32) rows_kernel<MODE, 1><<<unsigned(grid), 256, 0, stream>>>(P);
  else rows_kernel<MODE, 2><<<unsigned(grid), 256, 0, stream>>>(P);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// ---- reading back

struct ReadParams {
  const uint8_t *key_cache, *key_exps, *value_cache, *value_exps;
  const int32_t *block_tables, *starts, *context_lens, *out_starts;
  __half *k_out, *v_out;
  uint32_t* status;
  int64_t out_rows;
  int batch, kv_heads, hk, hv, block_size, num_blocks, max_blocks_per_seq, max_rows;
};

// A row's 16 codes to fp16: code * 2^e in fp32 (exact), rounded once.
__device__ __forceinline__ void widen(const uint4& codes, float f, uint4& lo, uint4& hi) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&codes);
  uint32_t o[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 a = h2f2(e4m3x2_half2(w[j])), b = h2f2(e4m3x2_half2(w[j] >> 16));
    o[2 * j] = pack_half2(a.x * f, a.y * f);
    o[2 * j + 1] = pack_half2(b.x * f, b.y * f);
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// One warp per cached token; its lanes stride over the token's key heads, then
// its value heads (each contiguous in the cache and in the output).
__global__ void __launch_bounds__(256) read_kernel(const ReadParams P) {
  const int lane = threadIdx.x & 31;
  const int64_t step = int64_t(gridDim.x) * (blockDim.x >> 5);
  const int64_t all = int64_t(P.batch) * P.max_rows;
  for (int64_t k = int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); k < all; k += step) {
    const int b = int(k / P.max_rows), i = int(k % P.max_rows);
    const int start = P.starts ? P.starts[b] : 0, L = P.context_lens[b];
    if (start < 0 || L < start || int64_t(L) > int64_t(P.max_blocks_per_seq) * P.block_size ||
        L - start > P.max_rows) {
      report(P.status, PA_STATUS_BIT_PLAN);
      continue;
    }
    const int pos = start + i;
    if (pos >= L) continue;
    const int64_t out = int64_t(P.out_starts[b]) + i;
    const int block = P.block_tables[int64_t(b) * P.max_blocks_per_seq + pos / P.block_size];
    const int place = pos % P.block_size;
    if (out < 0 || out >= P.out_rows) {
      report(P.status, PA_STATUS_BIT_WORKSPACE);
      continue;
    }
    if (block < 0 || block >= P.num_blocks) {
      report(P.status, PA_STATUS_BIT_BLOCK_INDEX);
      continue;
    }
    const int64_t slot = int64_t(block) * P.block_size + place;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const int hd = kv ? P.hv : P.hk, width = P.kv_heads * hd;
      const uint8_t* src = (kv ? P.value_cache : P.key_cache) + slot * width;
      const uint8_t* exps =
          (kv ? P.value_exps : P.key_exps) + int64_t(block) * P.kv_heads * P.block_size + place;
      __half* dst = (kv ? P.v_out : P.k_out) + out * width;
      for (int d = lane * 16; d < width; d += 512) {
        const uint4 codes = *reinterpret_cast<const uint4*>(src + d);
        const float f = pow2(int(exps[int64_t(d / hd) * P.block_size]) - kExpBias);
        uint4 lo, hi;
        widen(codes, f, lo, hi);
        *reinterpret_cast<uint4*>(dst + d) = lo;
        *reinterpret_cast<uint4*>(dst + d + 8) = hi;
      }
    }
  }
}

// ---- host checks

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

bool head_size_ok(int hs) { return hs > 0 && hs <= PA_MAX_HEAD_SIZE && hs % 16 == 0; }

pa_status check_cache(const pa_cache_config* c, const void* k, const void* ke, const void* v,
                      const void* ve, const int32_t* tables, const int32_t* lens) {
  if (!c || !k || !ke || !v || !ve || !tables || !lens) return PA_ERR_INVALID_ARG;
  if (c->batch <= 0 || c->batch > PA_MAX_BATCH || c->kv_heads <= 0) return PA_ERR_INVALID_ARG;
  if (!head_size_ok(c->head_size_k) || !head_size_ok(c->head_size_v)) return PA_ERR_INVALID_ARG;
  if (c->block_size <= 0 || c->block_size % 16 || c->num_blocks <= 0 || c->max_blocks_per_seq <= 0 ||
      c->max_rows < 0)
    return PA_ERR_INVALID_ARG;
  if (int64_t(c->num_blocks) * c->block_size > INT32_MAX) return PA_ERR_INVALID_ARG;
  if (int64_t(c->kv_heads) * PA_MAX_HEAD_SIZE > INT32_MAX) return PA_ERR_INVALID_ARG;
  if (k == v || ke == ve) return PA_ERR_INVALID_ARG;  // two caches, each with its own exponents
  if (!aligned16(k) || !aligned16(ke) || !aligned16(v) || !aligned16(ve)) return PA_ERR_INVALID_ARG;
  return PA_OK;
}

pa_status check_rotary(const pa_rotary* r, const void* q_weight, const void* k_weight,
                       const float* cos_sin) {
  if (!r || r->num_heads <= 0 || r->kv_heads <= 0 || !head_size_ok(r->head_size))
    return PA_ERR_INVALID_ARG;
  if (int64_t(r->num_heads) + 2 * int64_t(r->kv_heads) > INT32_MAX / PA_MAX_HEAD_SIZE)
    return PA_ERR_INVALID_ARG;
  if (r->rotary_dim < 0 || r->rotary_dim > r->head_size || r->rotary_dim % 16 ||
      r->max_positions <= 0)
    return PA_ERR_INVALID_ARG;
  if (!(r->eps >= 0.f) || std::isinf(r->eps)) return PA_ERR_INVALID_ARG;
  if (r->rotary_dim > 0 && !cos_sin) return PA_ERR_INVALID_ARG;
  if (!aligned16(q_weight) || !aligned16(k_weight) || !aligned16(cos_sin)) return PA_ERR_INVALID_ARG;
  return PA_OK;
}

// A row tensor: head h of token t at [t * stride + h * hs].
pa_status check_rows(const void* p, int64_t stride, int64_t width) {
  if (!p || !aligned16(p) || stride % 8 || stride < width) return PA_ERR_INVALID_ARG;
  return PA_OK;
}

void set_rotary(RowParams& P, const pa_rotary& r, const void* q_weight, const void* k_weight,
                const float* cos_sin, const int32_t* positions) {
  P.heads = r.num_heads;
  P.kv_heads = r.kv_heads;
  P.hk = r.head_size;
  P.rot = r.rotary_dim;
  P.interleaved = r.interleaved;
  P.max_positions = r.max_positions;
  P.eps = r.eps;
  P.q_weight = static_cast<const __half*>(q_weight);
  P.k_weight = static_cast<const __half*>(k_weight);
  P.cos_sin = cos_sin;
  P.positions = positions;
}

void set_cache(RowParams& P, const pa_cache_config& c, const int32_t* block_tables,
               const int32_t* context_lens, const int32_t* q_seqlens, void* key_cache,
               uint8_t* key_exps, void* value_cache, uint8_t* value_exps) {
  P.batch = c.batch;
  P.kv_heads = c.kv_heads;
  P.hk = c.head_size_k;
  P.hv = c.head_size_v;
  P.block_size = c.block_size;
  P.num_blocks = c.num_blocks;
  P.max_blocks_per_seq = c.max_blocks_per_seq;
  P.max_rows = q_seqlens ? c.max_rows : 1;
  P.block_tables = block_tables;
  P.context_lens = context_lens;
  P.q_seqlens = q_seqlens;
  P.key_cache = static_cast<uint8_t*>(key_cache);
  P.key_exps = key_exps;
  P.value_cache = static_cast<uint8_t*>(value_cache);
  P.value_exps = value_exps;
}

}  // namespace

}  // namespace pa

extern "C" pa_status pa_qk_norm_rope(const pa_rotary* rot, int64_t tokens, const void* query,
                                     int64_t query_stride, const void* key, int64_t key_stride,
                                     const void* q_weight, const void* k_weight,
                                     const float* cos_sin, const int32_t* positions, void* q_out,
                                     void* k_out, uint32_t* status, void* stream) {
  using namespace pa;
  pa_status st = check_rotary(rot, q_weight, k_weight, cos_sin);
  if (st != PA_OK) return st;
  const int64_t qw = int64_t(rot->num_heads) * rot->head_size;
  const int64_t kw = int64_t(rot->kv_heads) * rot->head_size;
  if (tokens < 0 || !positions || !q_out || !k_out || !aligned16(q_out) || !aligned16(k_out))
    return PA_ERR_INVALID_ARG;
  if ((st = check_rows(query, query_stride, qw)) != PA_OK) return st;
  if ((st = check_rows(key, key_stride, kw)) != PA_OK) return st;
  if ((q_out == query && query_stride != qw) || (k_out == key && key_stride != kw) || q_out == k_out)
    return PA_ERR_INVALID_ARG;
  RowParams P{};
  set_rotary(P, *rot, q_weight, k_weight, cos_sin, positions);
  P.tokens = tokens;
  P.query = static_cast<const __half*>(query);
  P.key = static_cast<const __half*>(key);
  P.query_stride = query_stride;
  P.key_stride = key_stride;
  P.q_out = static_cast<__half*>(q_out);
  P.k_out = static_cast<__half*>(k_out);
  P.status = status;
  return launch_rows<kRotate>(P, static_cast<cudaStream_t>(stream));
}

extern "C" pa_status pa_cache_write(const pa_cache_config* cfg, int64_t tokens, const void* key,
                                    int64_t key_stride, const void* value, int64_t value_stride,
                                    const int32_t* block_tables, const int32_t* context_lens,
                                    const int32_t* q_seqlens, void* key_cache, uint8_t* key_exps,
                                    void* value_cache, uint8_t* value_exps, uint32_t* status,
                                    void* stream) {
  using namespace pa;
  pa_status st = check_cache(cfg, key_cache, key_exps, value_cache, value_exps, block_tables, context_lens);
  if (st != PA_OK) return st;
  if (tokens < 0) return PA_ERR_INVALID_ARG;
  if ((st = check_rows(key, key_stride, int64_t(cfg->kv_heads) * cfg->head_size_k)) != PA_OK) return st;
  if ((st = check_rows(value, value_stride, int64_t(cfg->kv_heads) * cfg->head_size_v)) != PA_OK) return st;
  RowParams P{};
  set_cache(P, *cfg, block_tables, context_lens, q_seqlens, key_cache, key_exps, value_cache, value_exps);
  P.tokens = tokens;
  P.key = static_cast<const __half*>(key);
  P.value = static_cast<const __half*>(value);
  P.key_stride = key_stride;
  P.value_stride = value_stride;
  P.status = status;
  return launch_rows<kWrite>(P, static_cast<cudaStream_t>(stream));
}

extern "C" pa_status pa_cache_store(const pa_cache_config* cfg, const pa_rotary* rot, int64_t tokens,
                                    const void* query, int64_t query_stride, const void* key,
                                    int64_t key_stride, const void* value, int64_t value_stride,
                                    const void* q_weight, const void* k_weight,
                                    const float* cos_sin, const int32_t* positions,
                                    const int32_t* block_tables, const int32_t* context_lens,
                                    const int32_t* q_seqlens, void* key_cache, uint8_t* key_exps,
                                    void* value_cache, uint8_t* value_exps, void* q_out,
                                    uint32_t* status, void* stream) {
  using namespace pa;
  pa_status st = check_cache(cfg, key_cache, key_exps, value_cache, value_exps, block_tables, context_lens);
  if (st != PA_OK) return st;
  if ((st = check_rotary(rot, q_weight, k_weight, cos_sin)) != PA_OK) return st;
  if (rot->kv_heads != cfg->kv_heads || rot->head_size != cfg->head_size_k) return PA_ERR_INVALID_ARG;
  const int64_t qw = int64_t(rot->num_heads) * rot->head_size;
  if (tokens < 0 || !q_out || !aligned16(q_out) || (q_out == query && query_stride != qw))
    return PA_ERR_INVALID_ARG;
  if ((st = check_rows(query, query_stride, qw)) != PA_OK) return st;
  if ((st = check_rows(key, key_stride, int64_t(cfg->kv_heads) * cfg->head_size_k)) != PA_OK) return st;
  if ((st = check_rows(value, value_stride, int64_t(cfg->kv_heads) * cfg->head_size_v)) != PA_OK) return st;
  RowParams P{};
  set_rotary(P, *rot, q_weight, k_weight, cos_sin, positions);
  set_cache(P, *cfg, block_tables, context_lens, q_seqlens, key_cache, key_exps, value_cache, value_exps);
  P.tokens = tokens;
  P.query = static_cast<const __half*>(query);
  P.key = static_cast<const __half*>(key);
  P.value = static_cast<const __half*>(value);
  P.query_stride = query_stride;
  P.key_stride = key_stride;
  P.value_stride = value_stride;
  P.q_out = static_cast<__half*>(q_out);
  P.status = status;
  return launch_rows<kStore>(P, static_cast<cudaStream_t>(stream));
}

extern "C" pa_status pa_cache_read(const pa_cache_config* cfg, const void* key_cache,
                                   const uint8_t* key_exps, const void* value_cache,
                                   const uint8_t* value_exps, const int32_t* block_tables,
                                   const int32_t* starts, const int32_t* context_lens,
                                   const int32_t* out_starts, int64_t out_rows, void* k_out,
                                   void* v_out, uint32_t* status, void* stream) {
  using namespace pa;
  const pa_status st =
      check_cache(cfg, key_cache, key_exps, value_cache, value_exps, block_tables, context_lens);
  if (st != PA_OK) return st;
  if (!out_starts || out_rows < 0 || !k_out || !v_out || k_out == v_out || !aligned16(k_out) ||
      !aligned16(v_out))
    return PA_ERR_INVALID_ARG;
  if (cfg->max_rows == 0 || out_rows == 0) return PA_OK;
  ReadParams P{};
  P.key_cache = static_cast<const uint8_t*>(key_cache);
  P.key_exps = key_exps;
  P.value_cache = static_cast<const uint8_t*>(value_cache);
  P.value_exps = value_exps;
  P.block_tables = block_tables;
  P.starts = starts;
  P.context_lens = context_lens;
  P.out_starts = out_starts;
  P.k_out = static_cast<__half*>(k_out);
  P.v_out = static_cast<__half*>(v_out);
  P.status = status;
  P.out_rows = out_rows;
  P.batch = cfg->batch;
  P.kv_heads = cfg->kv_heads;
  P.hk = cfg->head_size_k;
  P.hv = cfg->head_size_v;
  P.block_size = cfg->block_size;
  P.num_blocks = cfg->num_blocks;
  P.max_blocks_per_seq = cfg->max_blocks_per_seq;
  P.max_rows = cfg->max_rows;
  const int64_t warps = int64_t(cfg->batch) * cfg->max_rows;
  const int64_t grid = cdiv(warps, 8) < 65536 ? cdiv(warps, 8) : 65536;
  read_kernel<<<unsigned(grid), 256, 0, static_cast<cudaStream_t>(stream)>>>(P);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
