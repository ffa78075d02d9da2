// w12_attn.cu - attention of draft-tree nodes over a paged cache and their ancestors.
//
// Plain form: one block per (node, query head), an online softmax in float over tiles of
// 128 keys, a key per thread for the scores and a column per thread for the sums.
#include <cstdint>

#include "w12_internal.cuh"

namespace w12 {

int check_cache(const kv_cache* c, const char* fn);

namespace {

constexpr int kAttnThreads = 128;
constexpr int kAttnMaxNodes = 256;
constexpr int32_t kAttnBadRequest = 1, kAttnBadBlock = 2;

struct AttnArgs {
  const uint16_t *q, *k, *v, *kc, *vc;
  int64_t q_stride, k_stride, v_stride, M;
  int64_t block_stride, token_stride, head_stride, n_blocks;
  const int32_t *table, *cache_len, *parent, *req_offsets;
  int64_t table_stride, table_width;
  int32_t n_req, block_size, group, n_q_heads;
  float scale;
  uint16_t* out;
  int32_t* status;
};

__device__ __forceinline__ float bf16_f(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

__device__ __forceinline__ uint16_t f_bf16(float f) {
  uint16_t h;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(f));
  return h;
}

template <int D>
__global__ void __launch_bounds__(kAttnThreads) k_tree_attn(AttnArgs a) {
  constexpr int kCols = (D + kAttnThreads - 1) / kAttnThreads;
  __shared__ float qs[D], ps[kAttnThreads], red[kAttnThreads / 32];
  __shared__ const uint16_t* vrow[kAttnThreads];
  __shared__ bool anc[kAttnMaxNodes];
  const int tid = threadIdx.x;
  const int64_t m = blockIdx.x;
  const int hq = blockIdx.y, h = hq / a.group;
  int r = 0;
  int64_t off = 0, end = a.M;
  if (a.req_offsets) {
    while (r < a.n_req && a.req_offsets[r + 1] <= m) ++r;
    if (r == a.n_req) return;
    off = a.req_offsets[r];
    end = a.req_offsets[r + 1];
    if (off > m) return;
  }
  const int64_t n64 = end - off, len = a.cache_len[r];
  bool ok = off >= 0 && end <= a.M && n64 <= kAttnMaxNodes && len >= 0 && len <= a.table_width * a.block_size;
  const int n = ok ? (int)n64 : 0;
  for (int i = tid; i < n; i += kAttnThreads) {
    const int32_t p = a.parent[off + i];
    ok = ok && (i == 0 ? p == -1 : p >= 0 && p < i);
    anc[i] = false;
  }
  if (!__syncthreads_and(ok)) {
    if (tid == 0) atomicOr(a.status, kAttnBadRequest);
    return;
  }
  const int32_t* table = a.table + r * a.table_stride;
  for (int64_t b = tid; b * a.block_size < len; b += kAttnThreads) ok = ok && table[b] >= 0 && table[b] < a.n_blocks;
  if (!__syncthreads_and(ok)) {
    if (tid == 0) atomicOr(a.status, kAttnBadBlock);
    return;
  }
  if (tid == 0)
    for (int32_t p = (int32_t)(m - off); p >= 0; p = a.parent[off + p]) anc[p] = true;
  for (int d = tid; d < D; d += kAttnThreads) qs[d] = bf16_f(a.q[m * a.q_stride + hq * D + d]) * a.scale;
  float acc[kCols] = {}, mx = -INFINITY, sum = 0.0f;
  for (int64_t j0 = 0; j0 < len + n; j0 += kAttnThreads) {
    __syncthreads();
    const int64_t j = j0 + tid;
    const uint16_t *kr = nullptr, *vr = nullptr;
    if (j < len) {
      const int64_t b = j / a.block_size, at = table[b] * a.block_stride + (j - b * a.block_size) * a.token_stride + h * a.head_stride;
      kr = a.kc + at;
      vr = a.vc + at;
    } else if (j < len + n && anc[j - len]) {
      kr = a.k + (off + j - len) * a.k_stride + h * D;
      vr = a.v + (off + j - len) * a.v_stride + h * D;
    }
    float s = -INFINITY;
    if (kr) {
      s = 0.0f;
      for (int d = 0; d < D; ++d) s = fmaf(qs[d], bf16_f(kr[d]), s);
    }
    float t = s;
    for (int o = 16; o; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, o));
    if ((tid & 31) == 0) red[tid >> 5] = t;
    __syncthreads();
    for (int w = 0; w < kAttnThreads / 32; ++w) t = fmaxf(t, red[w]);
    const float top = fmaxf(mx, t), ref = top == -INFINITY ? 0.0f : top, fix = mx == -INFINITY ? 0.0f : expf(mx - ref);
    mx = top;
    ps[tid] = kr ? expf(s - ref) : 0.0f;
    vrow[tid] = vr;
    __syncthreads();
    sum *= fix;
    for (int c = 0; c < kCols; ++c) acc[c] *= fix;
    for (int i = 0; i < kAttnThreads; ++i) {
      if (!vrow[i]) continue;
      sum += ps[i];
      for (int c = 0; c < kCols; ++c)
        if (tid + c * kAttnThreads < D) acc[c] = fmaf(ps[i], bf16_f(vrow[i][tid + c * kAttnThreads]), acc[c]);
    }
  }
  for (int c = 0; c < kCols; ++c)
    if (tid + c * kAttnThreads < D)
      a.out[(m * a.n_q_heads + hq) * D + tid + c * kAttnThreads] = f_bf16(acc[c] / sum);
}

}  // namespace
}  // namespace w12

using namespace w12;

extern "C" {

size_t tree_attn_workspace_size(int64_t M, int32_t n_req, int64_t n_q_heads, int64_t n_heads, int64_t head_dim) {
  return M >= 1 && n_req >= 1 && n_q_heads >= 1 && n_heads >= 1 && head_dim >= 1 ? 256 : 0;
}

int tree_attn(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride, const uint16_t* v,
              int64_t v_stride, int64_t M, int64_t n_q_heads, const kv_cache* cache, int64_t layer,
              const int32_t* table, int64_t table_stride, int64_t table_width, const int32_t* cache_len,
              const int32_t* parent, const int32_t* req_offsets, int32_t n_req, float scale, uint16_t* out,
              int32_t* status, void* ws, size_t ws_bytes, void* stream) {
  int st = check_cache(cache, "tree_attn");
  if (st) return st;
  if (!q || !k || !v || !table || !cache_len || !parent || !out || !status || !ws)
    return fail(W12_ERR_INVALID_ARG, "tree_attn: null pointer");
  const int64_t D = cache->head_dim, H = cache->n_heads;
  if (D != 64 && D != 128 && D != 256) return fail(W12_ERR_SHAPE, "tree_attn: head_dim=%lld (64, 128 or 256)", (long long)D);
  if (M < 1 || M > 0x7FFFFFFF || n_req < 1 || n_req > 65535 || n_q_heads < H || n_q_heads > 65535 || n_q_heads % H ||
      table_width < 1 || table_width > (1 << 24) || table_stride < table_width || layer < 0 || layer >= cache->n_layers)
    return fail(W12_ERR_SHAPE,
                "tree_attn: M=%lld, n_req=%d (1..65535), %lld query heads on %lld, table_width=%lld (stride %lld), layer %lld "
                "of %lld out of range",
                (long long)M, n_req, (long long)n_q_heads, (long long)H, (long long)table_width, (long long)table_stride,
                (long long)layer, (long long)cache->n_layers);
  if (!req_offsets && n_req != 1)
    return fail(W12_ERR_INVALID_ARG, "tree_attn: req_offsets is null but n_req=%d", n_req);
  if (!(scale > 0.0f) || scale > 3e38f) return fail(W12_ERR_INVALID_ARG, "tree_attn: scale must be positive and finite");
  if ((((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)out | (uintptr_t)ws) & 15u) ||
      ((q_stride | k_stride | v_stride) & 7) || q_stride < 0 || k_stride < 0 || v_stride < 0)
    return fail(W12_ERR_INVALID_ARG,
                "tree_attn: q, k, v, out and ws must be 16-byte aligned, strides non-negative multiples of 8");
  if (ws_bytes < tree_attn_workspace_size(M, n_req, n_q_heads, H, D))
    return fail(W12_ERR_BUFFER_TOO_SMALL, "tree_attn: workspace %zu < %zu", ws_bytes,
                tree_attn_workspace_size(M, n_req, n_q_heads, H, D));
  AttnArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.kc = cache->k + layer * cache->layer_stride;
  a.vc = cache->v + layer * cache->layer_stride;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.M = M;
  a.block_stride = cache->block_stride;
  a.token_stride = cache->token_stride;
  a.head_stride = cache->head_stride;
  a.n_blocks = cache->n_blocks;
  a.table = table;
  a.cache_len = cache_len;
  a.parent = parent;
  a.req_offsets = req_offsets;
  a.table_stride = table_stride;
  a.table_width = table_width;
  a.n_req = n_req;
  a.block_size = cache->block_size;
  a.group = (int32_t)(n_q_heads / H);
  a.n_q_heads = (int32_t)n_q_heads;
  a.scale = scale;
  a.out = out;
  a.status = status;
  const dim3 grid((unsigned)M, (unsigned)n_q_heads);
  if (D == 64) k_tree_attn<64><<<grid, kAttnThreads, 0, (cudaStream_t)stream>>>(a);
  else if (D == 128) k_tree_attn<128><<<grid, kAttnThreads, 0, (cudaStream_t)stream>>>(a);
  else k_tree_attn<256><<<grid, kAttnThreads, 0, (cudaStream_t)stream>>>(a);
  W12_LAUNCH_CHECK("tree_attn kernel");
  return W12_OK;
}

}  // extern "C"
