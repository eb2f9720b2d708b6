// The pool of a paged cache's blocks (pa_blocks.h): one launch of one cluster, and a second one of a
// whole grid for the places of many tokens.
//
// Where every block and token goes follows from three running sums over the rows: of the
// blocks that they give back, of those that they need and of their tokens. Every CTA of the
// cluster makes all three (the rows are a few kilobytes of lengths), keeps them in shared
// memory and then takes its share of the blocks and tokens, each finding its row by
// bisection. Blocks that come back are written before the cluster's barrier and handed out
// behind it; what the sums are made of is read before it and changed behind it.
//
// Chains of a few loads are all it is: 256 decode steps take 4.4 us, in a cluster of 8 CTAs as in one CTA
// alone; the 8,000 blocks of 64 prompts are given back in 18 us by one CTA and in 6 by the cluster. The
// places of the prompts' 130,000 tokens took the cluster 18 us; a grid behind it, whose CTAs each
// sum the tokens again and whose threads take four at a time, takes 2 to 4 (its launch lies under the
// cluster's end, its work behind it).
#include <cuda_runtime.h>

#include <algorithm>

#include "pa_blocks.h"
#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_launch.h"

namespace pa {

namespace {

constexpr int kThreads = 512;
constexpr int kPer = PA_MAX_BATCH / kThreads;  // rows a thread sums, next to one another
constexpr int kCluster = 8;  // 4: 15.6 us for the prompts taken and given back, 8: 13.5
// Rows and tokens from which on the tokens have a grid of their own (a second launch, 2 us)
constexpr int64_t kAlone = 2048;
constexpr int kTokens = 4;  // next to one another, a thread's

struct BlocksParams {
  const int32_t *context_lens, *q_seqlens;
  int32_t *tables, *held, *gone, *free_blocks, *count, *positions;
  int64_t* slots;
  uint32_t* status;
  int batch, block_size, num_blocks, cols, window, kept, tokens;
  bool places;  // this kernel makes the tokens' places
};

__device__ __forceinline__ void report(uint32_t* status, uint32_t bit) {
  if (status) atomicOr(status, bit);
}

// What a row does in this step.
struct Row {
  int tokens;     // as stated, at most all that there are
  int back;       // blocks given back: `sinks` of the first ones, the others from entry `from` on
  int sinks, from;
  int held, more; // entries it has, blocks it needs
  int first_pos;  // of its tokens; -1: none of them has a place
  int new_gone;
  bool ends, ok;
};

__device__ __forceinline__ Row load_row(const BlocksParams& P, int b) {
  Row r{};
  const int L = P.context_lens[b], q = P.q_seqlens ? P.q_seqlens[b] : L > 0 ? 1 : 0;
  const int held = P.held[b], gone = P.gone[b];
  r.tokens = P.q_seqlens ? min(max(q, 0), P.tokens) : min(1, P.tokens);
  r.first_pos = -1;
  r.ok = q >= 0 && L >= q && int64_t(L) <= int64_t(P.cols) * P.block_size && held >= 0 && held <= P.cols &&
         gone >= 0 && (gone == 0 || gone <= held - P.kept);
  if (!r.ok) {
    report(P.status, PA_STATUS_BIT_PLAN);
    return r;
  }
  r.held = held;
  r.from = P.kept + gone;
  r.ends = L == 0;
  if (r.ends) {
    r.sinks = min(P.kept, held);
    r.back = r.sinks + max(held - r.from, 0);
  } else {
    const int lo = P.window ? L - q - P.window + 1 : 0;  // the first key that is still seen
    const int first = lo > 0 ? min(lo / P.block_size, held) : 0;
    r.back = max(first - r.from, 0);
    r.new_gone = gone + r.back;
    r.more = max((L - 1) / P.block_size + 1 - held, 0);
    r.first_pos = L - q;
  }
  return r;
}

struct Sums {
  int tokens, back, more;
};

__device__ __forceinline__ int add_tokens(const BlocksParams& P, int a, int b) {
  return int(min(uint32_t(a) + uint32_t(b), uint32_t(P.tokens)));
}

// The block as a slot's first position, or none.
__device__ __forceinline__ int checked(const BlocksParams& P, int block) {
  if (block >= 0 && block < P.num_blocks) return block;
  report(P.status, PA_STATUS_BIT_BLOCK_INDEX);
  return -1;
}

// The row that element k of a running sum (starts[0] = 0, .., starts[n]) belongs to: the last
// one that begins at or before it, k < starts[n].
__device__ __forceinline__ int row_of(const int* starts, int n, int k) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= k) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) blocks_kernel(const BlocksParams P) {
  extern __shared__ int shared[];
  const int n = P.batch;
  int* tok = shared;          // [n + 1] running sums
  int* back = tok + n + 1;    // [n + 1]
  int* more = back + n + 1;   // [n + 1]
  int* held = more + n + 1;   // [n]
  int* from = held + n;       // [n]
  int* sinks = from + n;      // [n]
  int* first_pos = sinks + n; // [n]
  __shared__ Sums of_warp[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int me = blockIdx.x * kThreads + tid, all = gridDim.x * kThreads;

  // ---- the rows and their running sums
  const int per = (n + kThreads - 1) / kThreads;  // at most kPer
  Row rows[kPer];
  Sums own{0, 0, 0};
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int b = tid * per + k;
    if (k >= per || b >= n) continue;
    rows[k] = load_row(P, b);
    own.tokens = min(own.tokens + rows[k].tokens, P.tokens);  // (below 2^30 each)
    own.back += rows[k].back;
    own.more += rows[k].more;
  }
  Sums upto = own;
  auto add = [&](Sums& a, int t, int x, int y) {
    a.tokens = add_tokens(P, a.tokens, t);
    a.back += x;
    a.more += y;
  };
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, upto.tokens, o), x = __shfl_up_sync(0xffffffffu, upto.back, o),
              y = __shfl_up_sync(0xffffffffu, upto.more, o);
    if (lane >= o) add(upto, t, x, y);
  }
  if (lane == 31) of_warp[warp] = upto;
  __syncthreads();
  Sums at{0, 0, 0};  // before this thread's rows
  for (int w = 0; w < warp; ++w) add(at, of_warp[w].tokens, of_warp[w].back, of_warp[w].more);
  {
    const int t = __shfl_up_sync(0xffffffffu, upto.tokens, 1), x = __shfl_up_sync(0xffffffffu, upto.back, 1),
              y = __shfl_up_sync(0xffffffffu, upto.more, 1);
    if (lane > 0) add(at, t, x, y);
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int b = tid * per + k;
    if (k >= per || b >= n) continue;
    tok[b] = at.tokens;
    back[b] = at.back;
    more[b] = at.more;
    held[b] = rows[k].held;
    from[b] = rows[k].from;
    sinks[b] = rows[k].sinks;
    first_pos[b] = rows[k].first_pos;
    // more tokens than there are, of this row or behind it
    if (P.places && me < kThreads &&
        max(P.q_seqlens ? P.q_seqlens[b] : 1, 0) > P.tokens - at.tokens)
      report(P.status, PA_STATUS_BIT_PLAN);
    add(at, rows[k].tokens, rows[k].back, rows[k].more);
    if (b == n - 1) {
      tok[n] = at.tokens;
      back[n] = at.back;
      more[n] = at.more;
    }
  }
  int free0 = *P.count;
  if (free0 < 0 || free0 > P.num_blocks) {
    if (me == 0) report(P.status, PA_STATUS_BIT_POOL);
    free0 = max(0, min(free0, P.num_blocks));
  }
  __syncthreads();
  const int n_back = back[n], n_more = more[n], n_tok = tok[n];
  const int top = int(min(int64_t(free0) + n_back, int64_t(P.num_blocks)));

  // ---- given back
  for (uint32_t i = me; i < uint32_t(n_back); i += all) {  // (up to 2^31 - 1, and a step of all threads past it)
    const int j = int(i);
    const int b = row_of(back, n, j), k = j - back[b];
    const int64_t entry = int64_t(b) * P.cols + (k < sinks[b] ? k : from[b] + k - sinks[b]);
    int block = P.tables[entry];
    P.tables[entry] = -1;
    if (block < 0 || block >= P.num_blocks) {
      report(P.status, PA_STATUS_BIT_BLOCK_INDEX);
      block = -1;
    }
    const int64_t to = int64_t(free0) + n_back - 1 - j;
    if (to < P.num_blocks) P.free_blocks[to] = block;
    else report(P.status, PA_STATUS_BIT_POOL);
  }
  launch_dependents();
  __syncwarp();  // (the barrier wants the warp converged, and the loop's last round may be some lanes' alone)
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");

  // ---- handed out, block k of all that are needed
  const auto taken = [&](int k) {
    if (k >= top) return -1;
    const int block = __ldcg(P.free_blocks + (top - 1 - k));
    return block < 0 || block >= P.num_blocks ? -1 : block;
  };
  for (int k = me; k < min(n_more, top); k += all) {
    const int b = row_of(more, n, k), block = taken(k);
    if (block < 0) report(P.status, PA_STATUS_BIT_BLOCK_INDEX);
    P.tables[int64_t(b) * P.cols + held[b] + (k - more[b])] = block;
  }
  if (me == 0) {
    *P.count = top - min(n_more, top);
    if (n_more > top) report(P.status, PA_STATUS_BIT_POOL);
  }
  if (me < kThreads) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int b = tid * per + k;
      if (k >= per || b >= n || !rows[k].ok) continue;
      P.held[b] = rows[k].ends ? 0 : rows[k].held + min(rows[k].more, max(top - more[b], 0));
      P.gone[b] = rows[k].new_gone;
    }
  }

  // ---- the tokens' places (none: they are slots_kernel's)
  for (int t = me; t < P.tokens; t += all) {
    int pos = -1;
    int64_t slot = -1;
    if (t < n_tok) {
      const int b = row_of(tok, n, t);
      if (first_pos[b] >= 0) {
        pos = first_pos[b] + (t - tok[b]);
        const int page = pos / P.block_size, place = pos - page * P.block_size;
        int block;
        if (page < held[b]) {
          block = checked(P, P.tables[int64_t(b) * P.cols + page]);
        } else {
          block = taken(more[b] + (page - held[b]));
        }
        if (block >= 0) slot = int64_t(block) * P.block_size + place;
      }
    }
    if (P.slots) P.slots[t] = slot;
    if (P.positions) P.positions[t] = pos;
  }
}

// The places of many tokens, behind blocks_kernel: the tables are as it leaves them, and so is what
// each row holds.
__global__ void __launch_bounds__(kThreads) slots_kernel(const BlocksParams P) {
  extern __shared__ int shared[];
  const int n = P.batch;
  int* tok = shared;        // [n + 1] running sum of the tokens
  int* first = tok + n + 1; // [n] the first one's position, -1: none of the row's has a place
  int* held = first + n;    // [n]
  __shared__ int of_warp[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (n + kThreads - 1) / kThreads;
  grid_dependency_wait();
  int tokens[kPer], own = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int b = tid * per + k;
    tokens[k] = 0;
    if (k >= per || b >= n) continue;
    const Row r = load_row(P, b);  // (a row that is not in order is as it was)
    tokens[k] = r.tokens;
    first[b] = r.first_pos;
    held[b] = r.held;
    own = add_tokens(P, own, r.tokens);
  }
  int upto = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto = add_tokens(P, upto, t);
  }
  if (lane == 31) of_warp[warp] = upto;
  __syncthreads();
  int at = __shfl_up_sync(0xffffffffu, upto, 1);
  if (lane == 0) at = 0;
  for (int w = 0; w < warp; ++w) at = add_tokens(P, at, of_warp[w]);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int b = tid * per + k;
    if (k >= per || b >= n) continue;
    tok[b] = at;
    // more tokens than there are, of this row or behind it
    if (blockIdx.x == 0 && max(P.q_seqlens ? P.q_seqlens[b] : 1, 0) > P.tokens - at)
      report(P.status, PA_STATUS_BIT_PLAN);
    at = add_tokens(P, at, tokens[k]);
    if (b == n - 1) tok[n] = at;
  }
  __syncthreads();
  const int n_tok = tok[n];
  for (int64_t t0 = (int64_t(blockIdx.x) * kThreads + tid) * kTokens; t0 < P.tokens;
       t0 += int64_t(gridDim.x) * kThreads * kTokens) {
    int b = t0 < n_tok ? row_of(tok, n, int(t0)) : n;
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
      const int t = int(t0) + k;
      if (t >= P.tokens) break;
      while (b < n && t >= tok[b + 1]) ++b;
      int pos = -1;
      int64_t slot = -1;
      if (b < n && first[b] >= 0) {
        pos = first[b] + (t - tok[b]);
        const int page = pos / P.block_size;
        const int block = page < held[b] ? checked(P, P.tables[int64_t(b) * P.cols + page]) : -1;
        if (block >= 0) slot = int64_t(block) * P.block_size + (pos - page * P.block_size);
      }
      if (P.slots) P.slots[t] = slot;
      if (P.positions) P.positions[t] = pos;
    }
  }
}

pa_status blocks_step(const pa_blocks_config* cfg, const int32_t* context_lens, const int32_t* q_seqlens,
                      int32_t* block_tables, int32_t* held, int32_t* gone, int32_t* free_blocks, int32_t* count,
                      int64_t tokens, int64_t* slots, int32_t* positions, uint32_t* status, void* stream) {
  if (!cfg || !context_lens || !block_tables || !held || !gone || !free_blocks || !count) return PA_ERR_INVALID_ARG;
  const pa_blocks_config& c = *cfg;
  if (c.batch <= 0 || c.batch > PA_MAX_BATCH || c.block_size <= 0 || c.block_size % 16 || c.num_blocks <= 0 ||
      c.max_blocks_per_seq <= 0 || c.window < 0 || c.sinks < 0)
    return PA_ERR_INVALID_ARG;
  if (int64_t(c.num_blocks) * c.block_size > INT32_MAX ||
      int64_t(c.batch) * c.max_blocks_per_seq > INT32_MAX || tokens < 0 || tokens > INT32_MAX / 2)
    return PA_ERR_INVALID_ARG;
  if (held == gone || held == count || gone == count || free_blocks == count || free_blocks == held ||
      free_blocks == gone || block_tables == held || block_tables == gone || block_tables == free_blocks ||
      block_tables == count)
    return PA_ERR_INVALID_ARG;
  const auto aligned = [](const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; };
  for (const void* p : {static_cast<const void*>(context_lens), static_cast<const void*>(q_seqlens),
                        static_cast<const void*>(block_tables), static_cast<const void*>(held),
                        static_cast<const void*>(gone), static_cast<const void*>(free_blocks),
                        static_cast<const void*>(count), static_cast<const void*>(positions),
                        static_cast<const void*>(status)})
    if (!aligned(p, 4)) return PA_ERR_INVALID_ARG;
  if (!aligned(slots, 8)) return PA_ERR_INVALID_ARG;
  BlocksParams P{};
  P.context_lens = context_lens;
  P.q_seqlens = q_seqlens;
  P.tables = block_tables;
  P.held = held;
  P.gone = gone;
  P.free_blocks = free_blocks;
  P.count = count;
  P.slots = slots;
  P.positions = positions;
  P.status = status;
  P.batch = c.batch;
  P.block_size = c.block_size;
  P.num_blocks = c.num_blocks;
  P.cols = c.max_blocks_per_seq;
  P.window = c.window;
  P.kept = int(std::min<int64_t>(cdiv(c.sinks, c.block_size), c.max_blocks_per_seq));
  P.tokens = slots || positions ? int(tokens) : 0;
  const bool many = P.tokens + int64_t(c.batch) > kAlone;
  const int bytes = (7 * c.batch + 3) * int(sizeof(int));
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(blocks_kernel), bytes);
  if (e != cudaSuccess) return PA_ERR_CUDA;
  cudaLaunchConfig_t launch = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  launch.gridDim = dim3(kCluster);
  launch.blockDim = dim3(kThreads);
  launch.dynamicSmemBytes = bytes;
  launch.stream = static_cast<cudaStream_t>(stream);
  launch.attrs = attr;
  launch.numAttrs = 1;
  BlocksParams A = P;
  A.places = (slots || positions) && !many;
  if (many) A.tokens = 0;  // they are slots_kernel's
  if (cudaLaunchKernelEx(&launch, blocks_kernel, A) != cudaSuccess) return PA_ERR_CUDA;
  if (!many || P.tokens == 0) return PA_OK;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  launch.gridDim = dim3(unsigned(std::min<int64_t>(cdiv(P.tokens, kThreads * kTokens), 304)));
  launch.dynamicSmemBytes = (3 * c.batch + 1) * int(sizeof(int));
  return cudaLaunchKernelEx(&launch, slots_kernel, P) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

}  // namespace pa

extern "C" pa_status pa_blocks_step(const pa_blocks_config* cfg, const int32_t* context_lens,
                                    const int32_t* q_seqlens, int32_t* block_tables, int32_t* held,
                                    int32_t* gone, int32_t* free_blocks, int32_t* count, int64_t tokens,
                                    int64_t* slots, int32_t* positions, uint32_t* status, void* stream) {
  try {
    return pa::blocks_step(cfg, context_lens, q_seqlens, block_tables, held, gone, free_blocks, count, tokens, slots,
                           positions, status, stream);
  } catch (...) {  // of the host's memory or locks
    return PA_ERR_CUDA;
  }
}
