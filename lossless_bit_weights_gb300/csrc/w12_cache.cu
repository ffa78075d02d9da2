// w12_cache.cu - upkeep of the paged K/V cache of a target's attention layers: block
// tables and slot maps built on the device, and rows copied into their slots.
#include <cstdint>

#include "w12_internal.cuh"
#include "w12_pdl.cuh"

namespace w12 {
namespace {

// ---------------------------------------------------------------- slots

constexpr int kSlotThreads = 256;
constexpr int kSlotMaxReq = 4096;
constexpr int64_t kMaxBlock = 1 << 24;  // block_size and table_width

constexpr int32_t kSlotBadRequest = 1, kSlotNoBlocks = 2, kSlotCapacity = 4, kSlotBadEntry = 8;

struct SlotArgs {
  const int32_t *cache_len, *add, *path_nodes, *req_offsets;
  int32_t *table, *pool, *src, *new_len, *status;
  const int64_t* pool_pos;
  int64_t *slot, *pool_pos_out, *total;
  int64_t table_stride, table_width, n_blocks, n_nodes, capacity;
  int32_t extra, n_req, block_size;
};

struct ReqPlan {
  int64_t append, fresh, freed;  // tokens appended, blocks taken, blocks returned
  int32_t have;                  // blocks held before
  bool ok;
};

__device__ __forceinline__ ReqPlan plan_request(const SlotArgs& a, int r) {
  ReqPlan p{0, 0, 0, 0, false};
  const int64_t len = a.cache_len[r], app = (int64_t)a.add[r] + a.extra;
  const int64_t bs = a.block_size;
  if (len < 0 || app < -1 || len + bs > 0x7FFFFFFF || (len + bs - 1) / bs > a.table_width) return p;
  p.have = (int32_t)((len + bs - 1) / bs);
  if (app < 0) {
    p.freed = p.have;
    p.ok = true;
    return p;
  }
  const int64_t end = (len + app + bs - 1) / bs;
  if (end > a.table_width || len + app + bs > 0x7FFFFFFF) return p;
  if (a.path_nodes) {
    const int64_t off = a.req_offsets ? a.req_offsets[r] : 0, stop = a.req_offsets ? a.req_offsets[r + 1] : a.n_nodes;
    if (off < 0 || stop < off || stop > a.n_nodes || app > stop - off) return p;
  }
  p.append = app;
  p.fresh = end - p.have;
  p.ok = true;
  return p;
}

// The largest r with pre[r] <= t (pre ascending, pre[0] = 0): the request that entry t
// belongs to, requests with no entries skipped.
__device__ __forceinline__ int owner(const int32_t* pre, int n, int32_t t) {
  int lo = 0, hi = n;  // pre[lo] <= t < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// Every block adds up all requests (sums of at most 4096 triples, in shared memory) and then
// fills its part of the slots, of the new table entries and of the returned blocks, so
// one launch does it all and nothing waits on another block: what a block reads (old table
// entries, the pool's front) no block writes (new entries, the pool behind its back).
// Bound by the chain of its loads, not by bytes: 4.8 us for the commit of 24 requests, 10 us for
// 448,507 new tokens of 500 requests (6 MB).
__global__ void __launch_bounds__(kSlotThreads) k_kv_slots(const __grid_constant__ SlotArgs a) {
  pdl_enter();
  extern __shared__ int32_t sm[];
  int32_t* pre_tok = sm;                       // n_req + 1 each
  int32_t* pre_new = pre_tok + a.n_req + 1;
  int32_t* pre_old = pre_new + a.n_req + 1;
  __shared__ int64_t warp_sum[3][kSlotThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.n_req + kSlotThreads - 1) / kSlotThreads;
  const int r0 = min(a.n_req, tid * per), r1 = min(a.n_req, r0 + per);

  int64_t s[3] = {0, 0, 0};
  bool ok = true;
  for (int r = r0; r < r1; ++r) {
    const ReqPlan p = plan_request(a, r);
    ok = ok && p.ok;
    s[0] += p.append;
    s[1] += p.fresh;
    s[2] += p.freed;
  }
  int64_t run[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    int64_t v = s[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += u;
    }
    run[i] = v - s[i];
    if (lane == 31) warp_sum[i][warp] = v;
  }
  ok = __syncthreads_and(ok) != 0;
  int64_t tot[3] = {0, 0, 0};
#pragma unroll
  for (int i = 0; i < 3; ++i)
#pragma unroll
    for (int w = 0; w < kSlotThreads / 32; ++w) {
      if (w < warp) run[i] += warp_sum[i][w];
      tot[i] += warp_sum[i][w];
    }

  const int64_t head = a.pool_pos[0], tail = a.pool_pos[1];
  int32_t bad = ok ? 0 : kSlotBadRequest;
  if (head < 0 || tail < head || tail - head > a.n_blocks || tail - head + tot[2] > a.n_blocks || tot[1] > tail - head)
    bad |= kSlotNoBlocks;
  if (tot[0] > a.capacity) bad |= kSlotCapacity;
  const int64_t t0 = (int64_t)blockIdx.x * kSlotThreads + tid, step = (int64_t)gridDim.x * kSlotThreads;
  if (bad) {
    for (int64_t t = t0; t < a.capacity; t += step) {
      a.slot[t] = -1;
      a.src[t] = -1;
    }
    if (blockIdx.x == 0) {
      for (int r = tid; r < a.n_req; r += kSlotThreads) a.new_len[r] = a.cache_len[r];
      if (tid == 0) {
        a.pool_pos_out[0] = head;
        a.pool_pos_out[1] = tail;
        *a.total = 0;
        atomicOr(a.status, bad);
      }
    }
    return;
  }
  for (int r = r0; r < r1; ++r) {
    const ReqPlan p = plan_request(a, r);
    pre_tok[r] = (int32_t)run[0];
    pre_new[r] = (int32_t)run[1];
    pre_old[r] = (int32_t)run[2];
    run[0] += p.append;
    run[1] += p.fresh;
    run[2] += p.freed;
    if (blockIdx.x == 0) a.new_len[r] = p.freed ? 0 : (int32_t)(a.cache_len[r] + p.append);
  }
  if (tid == 0) {
    pre_tok[a.n_req] = (int32_t)tot[0];
    pre_new[a.n_req] = (int32_t)tot[1];
    pre_old[a.n_req] = (int32_t)tot[2];
    if (blockIdx.x == 0) {
      a.pool_pos_out[0] = head + tot[1];
      a.pool_pos_out[1] = tail + tot[2];
      *a.total = tot[0];
    }
  }
  __syncthreads();

  const int32_t bs = a.block_size;
  for (int64_t t = t0; t < a.capacity; t += step) {
    int64_t slot = -1;
    int32_t src = -1;
    if (t < tot[0]) {
      const int r = owner(pre_tok, a.n_req, (int32_t)t);
      const int32_t j = (int32_t)t - pre_tok[r], len = a.cache_len[r], p = len + j;
      const int32_t have = (len + bs - 1) / bs, b = p / bs;
      const int32_t id = b < have ? a.table[r * a.table_stride + b]
                                  : a.pool[(head + pre_new[r] + (b - have)) % a.n_blocks];
      slot = id < 0 ? -2 : (int64_t)id * bs + (p - b * bs);  // (-1 would be passed over)
      if (id < 0) atomicOr(a.status, kSlotBadEntry);
      src = (int32_t)t;
      if (a.path_nodes) {
        const int32_t off = a.req_offsets ? a.req_offsets[r] : 0;
        const int64_t stop = a.req_offsets ? a.req_offsets[r + 1] : a.n_nodes;
        const int32_t node = a.path_nodes[off + j];
        const bool in = node >= 0 && node < stop - off;
        src = in ? off + node : -1;
        if (!in) atomicOr(a.status, kSlotBadEntry);
      }
    }
    a.slot[t] = slot;
    a.src[t] = src;
  }
  for (int64_t b = t0; b < tot[1]; b += step) {
    const int r = owner(pre_new, a.n_req, (int32_t)b);
    const int32_t have = (a.cache_len[r] + bs - 1) / bs;
    a.table[r * a.table_stride + have + ((int32_t)b - pre_new[r])] = a.pool[(head + b) % a.n_blocks];
  }
  for (int64_t b = t0; b < tot[2]; b += step) {
    const int r = owner(pre_old, a.n_req, (int32_t)b);
    const int32_t id = a.table[r * a.table_stride + ((int32_t)b - pre_old[r])];
    if (id < 0) atomicOr(a.status, kSlotBadEntry);
    a.pool[(tail + b) % a.n_blocks] = id;
  }
}

// ---------------------------------------------------------------- rows into slots

struct WriteArgs {
  uint16_t* cache[2];          // K, V at the first layer written
  const uint16_t* rows[2];
  int64_t layer_stride, block_stride, token_stride, head_stride;
  int64_t rows_layer[2], rows_row[2];
  const int64_t* slot;
  const int32_t* src;
  int32_t* status;
  int64_t n, n_rows, n_slots;
  int32_t block_size, chunks, head_chunks;  // 16-byte chunks of a row and of a head
};

constexpr int kWriteThreads = 128;
constexpr int kWriteTokens = 4;  // tokens of a block

// A block copies four tokens of one layer, a lane each for their slots and rows and four 16-byte
// pieces a thread on their way.  Bound by bytes, read once and written once: 12289 tokens of
// 8 heads of 128 (101 MB) in 17.6 us, 5.7 TB/s, 0.85 of the measured copy rate.  With every thread
// dividing for all four tokens 21.4; with 256 threads 18.7, with 64 18.5, 512 27; two or
// eight tokens a block 17.9 and 18.9.
__global__ void __launch_bounds__(kWriteThreads) k_kv_write(const __grid_constant__ WriteArgs a) {
  pdl_enter();
  const int64_t l = blockIdx.y;
  const int per_token = 2 * a.chunks;
  const int lane = threadIdx.x & 31;
  for (int64_t t0 = (int64_t)blockIdx.x * kWriteTokens; t0 < a.n; t0 += (int64_t)gridDim.x * kWriteTokens) {
    // A lane finds one token's row and place in the cache (the division is long), and the warp shares them.
    int64_t row = -1, place = -1;
    if (lane < kWriteTokens && t0 + lane < a.n) {
      place = a.slot[t0 + lane];
      row = a.src ? a.src[t0 + lane] : t0 + lane;
      if (place != -1) {
        if (place < 0 || place >= a.n_slots || row < 0 || row >= a.n_rows) {
          if (threadIdx.x < 32) atomicOr(a.status, 1);
          place = -1;
        } else {
          const int64_t block = place / a.block_size;
          place = l * a.layer_stride + block * a.block_stride + (place - block * a.block_size) * a.token_stride;
        }
      }
    }
    int64_t from[kWriteTokens], to[kWriteTokens];
#pragma unroll
    for (int k = 0; k < kWriteTokens; ++k) {
      from[k] = __shfl_sync(0xFFFFFFFFu, row, k);
      to[k] = __shfl_sync(0xFFFFFFFFu, place, k);
    }
    for (int e = threadIdx.x; e < per_token; e += kWriteThreads) {
      const int kv = e >= a.chunks, c = e - kv * a.chunks, h = c / a.head_chunks;
      const uint16_t* rows = a.rows[kv] + l * a.rows_layer[kv] + (int64_t)c * 8;
      uint16_t* cache = a.cache[kv] + h * a.head_stride + (int64_t)(c - h * a.head_chunks) * 8;
      uint4 x[kWriteTokens];
#pragma unroll
      for (int k = 0; k < kWriteTokens; ++k)
        if (to[k] >= 0) x[k] = *reinterpret_cast<const uint4*>(rows + from[k] * a.rows_row[kv]);
#pragma unroll
      for (int k = 0; k < kWriteTokens; ++k)
        if (to[k] >= 0) *reinterpret_cast<uint4*>(cache + to[k]) = x[k];
    }
  }
}

}  // namespace

// Shared by the calls that take a cache: its pointers, sizes and strides.
int check_cache(const kv_cache* c, const char* fn) {
  if (!c) return fail(W12_ERR_INVALID_ARG, "%s: null cache descriptor", fn);
  if (!c->k || !c->v) return fail(W12_ERR_INVALID_ARG, "%s: null cache pointer", fn);
  if (c->n_layers < 1 || c->n_blocks < 1 || c->n_blocks > 0x7FFFFFFF || c->block_size < 1 || c->block_size > kMaxBlock ||
      c->n_heads < 1 || c->n_heads > 65535 || c->head_dim < 1)
    return fail(W12_ERR_SHAPE, "%s: cache of %lld layers, %lld blocks of %d tokens, %d heads of %d out of range", fn,
                (long long)c->n_layers, (long long)c->n_blocks, c->block_size, c->n_heads, c->head_dim);
  if ((((uintptr_t)c->k | (uintptr_t)c->v) & 15u) ||
      ((c->layer_stride | c->block_stride | c->token_stride | c->head_stride) & 7) || c->layer_stride < 0 ||
      c->block_stride < 0 || c->token_stride < 0 || c->head_stride < 0)
    return fail(W12_ERR_INVALID_ARG, "%s: cache pointers must be 16-byte aligned and strides non-negative multiples of 8",
                fn);
  return W12_OK;
}

}  // namespace w12

using namespace w12;

extern "C" {

int kv_slots(const int32_t* cache_len, const int32_t* add, int32_t extra, int32_t n_req, int32_t* table,
             int64_t table_stride, int64_t table_width, int32_t* pool, int64_t n_blocks, const int64_t* pool_pos,
             int64_t block_size, const int32_t* path_nodes, const int32_t* req_offsets, int64_t n_nodes,
             int64_t capacity, int64_t* slot, int32_t* src, int32_t* new_len, int64_t* pool_pos_out, int64_t* total,
             int32_t* status, void* stream) {
  if (pool_pos_out == pool_pos || new_len == cache_len)
    return fail(W12_ERR_INVALID_ARG, "kv_slots: pool_pos_out and new_len must not be the inputs");
  if (n_req < 1 || n_req > kSlotMaxReq || block_size < 1 || block_size > kMaxBlock || table_width < 1 ||
      table_width > kMaxBlock || table_stride < table_width || n_blocks < 1 || n_blocks > 0x7FFFFFFF || capacity < 1 ||
      capacity > 0x7FFFFFFF)
    return fail(W12_ERR_SHAPE,
                "kv_slots: n_req=%d (1..%d), block_size=%lld, table_width=%lld (stride %lld), n_blocks=%lld, "
                "capacity=%lld out of range",
                n_req, kSlotMaxReq, (long long)block_size, (long long)table_width, (long long)table_stride,
                (long long)n_blocks, (long long)capacity);
  // (after the sizes: a tensor of no elements has a null pointer)
  if (!cache_len || !add || !table || !pool || !pool_pos || !slot || !src || !new_len || !pool_pos_out || !total ||
      !status)
    return fail(W12_ERR_INVALID_ARG, "kv_slots: null pointer");
  if (path_nodes && (n_nodes < 1 || n_nodes > 0x7FFFFFFF))
    return fail(W12_ERR_SHAPE, "kv_slots: n_nodes=%lld out of range", (long long)n_nodes);
  if (path_nodes && !req_offsets && n_req != 1)
    return fail(W12_ERR_INVALID_ARG, "kv_slots: req_offsets is null but n_req=%d", n_req);
  // Some blocks write their results while others still read.
  struct Range {
    uintptr_t from, bytes;
  };
  auto range = [](const void* p, int64_t n, int size) { return Range{(uintptr_t)p, p ? (uintptr_t)n * size : 0}; };
  const Range out[] = {range(slot, capacity, 8), range(src, capacity, 4), range(new_len, n_req, 4),
                       range(pool_pos_out, 2, 8), range(total, 1, 8), range(status, 1, 4)};
  const Range used[] = {range(cache_len, n_req, 4), range(add, n_req, 4),
                        range(table, (n_req - 1) * table_stride + table_width, 4), range(pool, n_blocks, 4),
                        range(pool_pos, 2, 8), range(path_nodes, n_nodes, 4),
                        range(path_nodes ? req_offsets : nullptr, n_req + 1, 4)};
  auto meet = [](const Range& x, const Range& y) { return x.from < y.from + y.bytes && y.from < x.from + x.bytes; };
  for (const Range& o : out) {
    bool bad = false;
    for (const Range& u : used) bad = bad || meet(o, u);
    for (const Range& x : out) bad = bad || (&x != &o && meet(o, x));
    if (bad) return fail(W12_ERR_INVALID_ARG, "kv_slots: results must not overlap one another or what the call reads");
  }
  SlotArgs a{};
  a.cache_len = cache_len;
  a.add = add;
  a.path_nodes = path_nodes;
  a.req_offsets = req_offsets;
  a.table = table;
  a.pool = pool;
  a.src = src;
  a.new_len = new_len;
  a.status = status;
  a.pool_pos = pool_pos;
  a.slot = slot;
  a.pool_pos_out = pool_pos_out;
  a.total = total;
  a.table_stride = table_stride;
  a.table_width = table_width;
  a.n_blocks = n_blocks;
  a.n_nodes = n_nodes;
  a.capacity = capacity;
  a.extra = extra;
  a.n_req = n_req;
  a.block_size = (int32_t)block_size;
  const size_t smem = (size_t)(n_req + 1) * 3 * 4;
  // (asked for whatever this call's size: the 48 KB that need no asking hold the kernel's static arrays too)
  static int configured[64] = {0};
  int dev = 0;
  W12_CUDA_TRY(cudaGetDevice(&dev));
  if (dev >= 64 || !configured[dev]) {
    W12_CUDA_TRY(cudaFuncSetAttribute(k_kv_slots, cudaFuncAttributeMaxDynamicSharedMemorySize, (kSlotMaxReq + 1) * 12));
    if (dev < 64) configured[dev] = 1;
  }
  const int64_t blocks = (capacity + kSlotThreads - 1) / kSlotThreads;
  W12_CUDA_TRY(launch_dependent(k_kv_slots, dim3((unsigned)(blocks < 608 ? blocks : 608)), kSlotThreads, smem, (cudaStream_t)stream, a));
  W12_LAUNCH_CHECK("kv_slots kernel");
  return W12_OK;
}

int kv_write(const kv_cache* cache, int64_t layer, int64_t n_layers, const uint16_t* k, int64_t k_layer_stride,
             int64_t k_row_stride, const uint16_t* v, int64_t v_layer_stride, int64_t v_row_stride, int64_t n_rows,
             const int64_t* slot, const int32_t* src, int64_t n, int32_t* status, void* stream) {
  int st = check_cache(cache, "kv_write");
  if (st) return st;
  if (!k || !v || !slot || !status) return fail(W12_ERR_INVALID_ARG, "kv_write: null pointer");
  if (cache->head_dim > 1024 || (cache->head_dim & 7))
    return fail(W12_ERR_SHAPE, "kv_write: head_dim=%d must be a multiple of 8 up to 1024", cache->head_dim);
  if (layer < 0 || n_layers < 1 || n_layers > 65535 || layer > cache->n_layers - n_layers || n < 1 || n > 0x7FFFFFFF ||
      n_rows < 1 || n_rows > 0x7FFFFFFF)
    return fail(W12_ERR_SHAPE, "kv_write: layers %lld..+%lld of %lld, n=%lld, n_rows=%lld out of range", (long long)layer,
                (long long)n_layers, (long long)cache->n_layers, (long long)n, (long long)n_rows);
  if ((((uintptr_t)k | (uintptr_t)v) & 15u) || ((k_layer_stride | k_row_stride | v_layer_stride | v_row_stride) & 7) ||
      k_layer_stride < 0 || k_row_stride < 0 || v_layer_stride < 0 || v_row_stride < 0)
    return fail(W12_ERR_INVALID_ARG, "kv_write: rows must be 16-byte aligned, their strides non-negative multiples of 8");
  WriteArgs a{};
  a.cache[0] = cache->k + layer * cache->layer_stride;
  a.cache[1] = cache->v + layer * cache->layer_stride;
  a.rows[0] = k;
  a.rows[1] = v;
  a.layer_stride = cache->layer_stride;
  a.block_stride = cache->block_stride;
  a.token_stride = cache->token_stride;
  a.head_stride = cache->head_stride;
  a.rows_layer[0] = k_layer_stride;
  a.rows_layer[1] = v_layer_stride;
  a.rows_row[0] = k_row_stride;
  a.rows_row[1] = v_row_stride;
  a.slot = slot;
  a.src = src;
  a.status = status;
  a.n = n;
  a.n_rows = n_rows;
  a.n_slots = cache->n_blocks * cache->block_size;
  a.block_size = cache->block_size;
  a.head_chunks = cache->head_dim / 8;
  a.chunks = cache->n_heads * a.head_chunks;
  const int64_t blocks = (n + kWriteTokens - 1) / kWriteTokens;
  W12_CUDA_TRY(launch_dependent(k_kv_write, dim3((unsigned)(blocks < 65536 ? blocks : 65536), (unsigned)n_layers), kWriteThreads, 0,
                                (cudaStream_t)stream, a));
  W12_LAUNCH_CHECK("kv_write kernel");
  return W12_OK;
}

}  // extern "C"
