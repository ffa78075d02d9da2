// w12_logits.cu - rules on logits before the argmax: penalties for repeated tokens, a
// bias per token, a mask of allowed tokens; and the rows' argmax with greedy acceptance
// behind them.
//
// One block takes one request and one chunk of the vocabulary.  It builds the request's
// side of the rules for its chunk in shared memory: integer counts of the history, the
// prompt flag, the place of the last bias entry, and the list of the tokens that any rule of
// the request can touch.  Then each row's chunk is streamed once, 64 bytes a thread in
// flight: the untouched tokens (nearly all) go by with their mask bit alone.  The listed
// tokens follow, one a lane, with the count from the table plus the drafted tokens on the
// row's own path, so the table is never changed and rows need no barriers between them.
// (A test at every token instead sent almost every warp through the formula: with 2500
// distinct tokens in a history, 87 % of all runs of 128 tokens hold one.)
//
// Bound by bytes, the logits read once (and written once where they are asked for): 192 rows of
// 151936 tokens of 24 requests take 48 us with all rules (237 MB, 5.0 TB/s, 0.74 of the measured
// copy rate), 37.5 us with the argmax and acceptance instead of the rows (117 MB, 3.1 TB/s).  What is
// left is the making of the tables, during which a block streams nothing, the history and the
// listed tokens (about 13, 4 and 5 us of the 37).  Instructions count as much as bytes: bounds
// tests at every four tokens cost 12 and 8 us.
#include <cstdint>
#include <type_traits>

#include "w12_internal.cuh"
#include "w12_pdl.cuh"

namespace w12 {
namespace {

constexpr int kAcceptThreads = 512;
constexpr int kAcceptWarps = kAcceptThreads / 32;
constexpr int kRuleParts = 8;        // parts of a row's chunk, at most
constexpr int kRuleMaxNodes = 1024;  // nodes of one request
constexpr uint32_t kPromptFlag = 0x80000000u;
constexpr int32_t kRuleBadRequest = 1, kRuleClamped = 2;

struct RuleArgs {
  const float* logits;
  int64_t stride, M, V;
  logit_rules r;
  const int32_t *parent, *draft, *req_offsets;
  int32_t n_req;
  float* out;
  int64_t out_stride;
  int32_t* status;
  unsigned long long* key;  // [M][chunks] argmax keys, or null
  int32_t chunk, chunks, parts;
  bool vec;                 // rows allow 16-byte accesses
  bool hist_vec;            // so do the histories
};

// Nodes of request r, or false: its offsets are out of range or it has too many.
__device__ __forceinline__ bool request_rows(const int32_t* offsets, int64_t M, int r, int64_t& off, int& n) {
  off = offsets ? offsets[r] : 0;
  const int64_t end = offsets ? offsets[r + 1] : M;
  if (off < 0 || end < off || end > M || end - off > kRuleMaxNodes) return false;
  n = (int)(end - off);
  return true;
}

__device__ __forceinline__ unsigned long long arg_key(float x, int64_t v) {
  return ((unsigned long long)((uint32_t)order_key(x) ^ 0x80000000u) << 32) | (0xFFFFFFFFu - (uint32_t)v);
}

// The largest value so far and its token, in a thread that sees its tokens in rising order.
struct Best {
  int32_t key = INT32_MIN;  // NaN counts as the one above: below every number, above nothing
  int32_t at = -1;
  float value = -INFINITY;

  __device__ __forceinline__ void take(float f, int32_t i) {
    const int32_t k = max(order_key(f), INT32_MIN + 1);
    if (k > key || (k == key && i < at)) {
      key = k;
      at = i;
      value = f;
    }
  }
};

__device__ __forceinline__ float4 load4(const float* x, int i, int n, bool vec) {
  if (vec && i + 4 <= n) return __ldcs(reinterpret_cast<const float4*>(x + i));
  float4 f;
  f.x = i < n ? x[i] : 0.0f;
  f.y = i + 1 < n ? x[i + 1] : 0.0f;
  f.z = i + 2 < n ? x[i + 2] : 0.0f;
  f.w = i + 3 < n ? x[i + 3] : 0.0f;
  return f;
}

template <bool WRITE, int T>
__global__ void __launch_bounds__(T, (1024 + T / 2) / T) k_logit_rules(const __grid_constant__ RuleArgs a) {
  constexpr int kWarps = T / 32;
  pdl_enter();
  extern __shared__ __align__(16) uint32_t sm[];
  __shared__ int s_listed[kWarps], s_part[kRuleParts + 1];  // listed tokens: of a warp's words, before a part
  const int r = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t v0 = (int64_t)blockIdx.x * a.chunk;
  const int width = (int)min((int64_t)a.chunk, a.V - v0);
  int64_t off;
  int n;
  if (!request_rows(a.req_offsets, a.M, r, off, n)) {
    if (tid == 0) atomicOr(a.status, kRuleBadRequest);
    return;
  }
  if (n == 0) return;
  const bool count = a.r.rep || a.r.freq || a.r.pres, bias = a.r.bias_off != nullptr;
  const bool tree = a.parent != nullptr;
  const bool has_rep = a.r.rep != nullptr, has_freq = a.r.freq != nullptr, has_pres = a.r.pres != nullptr;
  // everything of the request that does not wait for anything else
  const float rep = has_rep ? a.r.rep[r] : 1.0f, freq = has_freq ? a.r.freq[r] : 0.0f, pres = has_pres ? a.r.pres[r] : 0.0f;
  const int64_t h_given = count && a.r.hist ? a.r.hist_len[r] : 0;
  const int64_t prompt = count && a.r.hist && a.r.prompt_len ? a.r.prompt_len[r] : 0;
  const int64_t b_given = bias ? a.r.bias_off[r] : 0, b_end = bias ? a.r.bias_off[r + 1] : 0;
  const int64_t len = min(max(h_given, (int64_t)0), a.r.hist_stride);
  const bool root_read = tree && prompt > len;  // the root, behind the history, ends the prompt (all rows have it)
  const int32_t* h = a.r.hist + r * a.r.hist_stride;
  // tokens of the history that a thread has on their way (four adjacent ones at a time where the rows
  // allow it), the first ones from here on
  constexpr int H = 8;
  int32_t told[H];
  auto place = [&](int64_t j0, int k) {  // of told[k]
    return a.hist_vec ? j0 + ((k >> 2) * T + tid) * 4 + (k & 3) : j0 + k * T + tid;
  };
  auto ask = [&](int64_t j0) {
    if (a.hist_vec) {
#pragma unroll
      for (int k = 0; k < H; k += 4) {
        const int64_t j = place(j0, k);
        int4 t = make_int4(-1, -1, -1, -1);
        if (j + 4 <= len) {
          t = *reinterpret_cast<const int4*>(h + j);
        } else if (j < len) {  // the last row may end with its history
          t.x = h[j];
          if (j + 1 < len) t.y = h[j + 1];
          if (j + 2 < len) t.z = h[j + 2];
        }
        told[k] = t.x, told[k + 1] = t.y, told[k + 2] = t.z, told[k + 3] = t.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < H; ++k) told[k] = place(j0, k) < len ? h[place(j0, k)] : -1;
    }
  };
  ask(0);
  // shared memory: the rows' best keys, bitmap, counts and bias places (chunk entries each), the
  // tree, the list of touched tokens
  unsigned long long* best = reinterpret_cast<unsigned long long*>(sm);
  uint32_t* bits = sm + (WRITE ? 0 : 2 * ((n + 1) & ~1));  // 16-byte aligned, as are the tables behind it
  uint32_t* cnt = bits + a.chunk / 32;
  int32_t* bias_at = reinterpret_cast<int32_t*>(cnt + (count ? a.chunk : 0));
  int32_t* parent = bias_at + (bias ? a.chunk : 0);
  int32_t* draft = parent + (tree ? n : 0);
  int32_t* up = draft + (tree ? n : 0);  // the nearest node on the path whose token is in the chunk
  uint16_t* list = reinterpret_cast<uint16_t*>(up + (tree ? n : 0));

  // the rows' chunk comes into L2 while the tables are made
  if (a.vec)
    for (int i = tid; i < n; i += T)
      if (width >= 4) prefetch_l2(a.logits + (off + i) * a.stride + v0, (uint32_t)(width & ~3) * 4);
  const int zeros = (a.chunk / 32 + (count ? a.chunk : 0) + (bias ? a.chunk : 0)) / 4;  // bitmap and tables, one run
  for (int i = tid; i < zeros; i += T) reinterpret_cast<uint4*>(bits)[i] = make_uint4(0, 0, 0, 0);
  if (!WRITE)
    for (int i = tid; i < n; i += T) best[i] = 0;
  bool ok = true;
  if (tree)
    for (int i = tid; i < n; i += T) {
      const int32_t p = a.parent[off + i];
      ok = ok && (i == 0 ? p == -1 : p >= 0 && p < i);
      parent[i] = p;
      draft[i] = i == 0 && root_read ? -1 : a.draft[off + i];
    }
  if (!__syncthreads_and(ok)) {
    if (tid == 0) atomicOr(a.status, kRuleBadRequest);
    if (!WRITE)  // no token: acceptance reports the tree as invalid
      for (int i = tid; i < n; i += T) a.key[(off + i) * a.chunks + blockIdx.x] = 0;
    return;
  }
  if (tid == 0 && (len != h_given || prompt < 0 || prompt > h_given + tree)) atomicOr(a.status, kRuleClamped);
  for (int64_t j0 = 0; j0 < len; j0 += H * T) {
#pragma unroll
    for (int k = 0; k < H; ++k) {
      // in 32 bits without a sign: a token below the chunk (or below zero) lands above its end
      const uint32_t i = (uint32_t)told[k] - (uint32_t)v0;
      const int64_t j = place(j0, k);
      if (i < (uint32_t)width && j < len) {
        if (j < prompt) atomicOr(&cnt[i], kPromptFlag);
        else atomicAdd(&cnt[i], 1u);
        atomicOr(&bits[i >> 5], 1u << (i & 31));
      }
    }
    ask(j0 + H * T);
  }
  if (root_read && tid == 0) {
    const uint32_t i = (uint32_t)a.draft[off] - (uint32_t)v0;
    if (i < (uint32_t)width) {
      atomicOr(&cnt[i], kPromptFlag);
      atomicOr(&bits[i >> 5], 1u << (i & 31));
    }
  }
  if (bias) {
    const int64_t b0 = min(max(b_given, (int64_t)0), a.r.n_bias), b1 = min(max(b_end, b0), a.r.n_bias);
    if (tid == 0 && (b0 != b_given || b1 != b_end)) atomicOr(a.status, kRuleClamped);
    for (int64_t j = b0 + tid; j < b1; j += T) {
      const uint32_t i = (uint32_t)a.r.bias_tok[j] - (uint32_t)v0;
      if (i < (uint32_t)width) {
        atomicMax(&bias_at[i], (int32_t)j + 1);
        atomicOr(&bits[i >> 5], 1u << (i & 31));
      }
    }
  }
  if (tree && count)
    for (int i = tid; i < n; i += T) {
      int32_t p = i;
      while (p >= 0 && !(draft[p] >= v0 && draft[p] < v0 + width)) p = parent[p];
      up[i] = p;
      if (p == i) {
        const int b = (int)(draft[i] - v0);
        atomicOr(&bits[b >> 5], 1u << (b & 31));
      }
    }
  __syncthreads();
  // ---- the touched tokens, listed in rising order (at most one word of the bitmap a thread:
  // chunk <= 32 * threads)
  const uint32_t mine = tid < a.chunk / 32 ? bits[tid] : 0u;
  int before = __popc(mine);
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xFFFFFFFFu, before, o);
    if (lane >= o) before += t;
  }
  if (lane == 31) s_listed[warp] = before;
  __syncthreads();
  int listed = 0;
  before -= __popc(mine);
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_listed[w];
    listed += s_listed[w];
  }
  const int part_len = a.chunk / a.parts;  // a multiple of 32
  if (tid * 32 < a.chunk && tid * 32 % part_len == 0) s_part[tid * 32 / part_len] = before;
  if (tid == 0) s_part[a.parts] = listed;
  for (uint32_t m = mine; m; m &= m - 1) list[before++] = (uint16_t)(tid * 32 + __ffs((int)m) - 1);
  __syncthreads();

  // ---- a warp takes one part of one row's chunk at a time
  for (int u = warp; u < n * a.parts; u += kWarps) {
    const int node = u / a.parts, part = u - node * a.parts, c0 = part * part_len, c1 = min(width, c0 + part_len);
    const int64_t m = off + node;
    const float* x = a.logits + m * a.stride + v0;
    float* y = WRITE ? a.out + m * a.out_stride + v0 : nullptr;
    const uint32_t* mask = a.r.mask ? a.r.mask + m * a.r.mask_stride + v0 / 32 : nullptr;
    // The untouched tokens: the largest value so far and the four tokens it was first seen among, kept
    // with their values; which of the four it is is asked once, at the end.
    float high = -INFINITY;
    int high_at = -1;
    float4 among = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    // listed tokens of the part: four a lane on their way, the first ones while the others stream
    float f4[4];
    uint32_t told4 = 0;
    auto ask_listed = [&](int j0) {
      told4 = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f4[k] = 0.0f;
        if (j0 + 32 * k >= s_part[part + 1]) continue;
        const int i = list[j0 + 32 * k];
        f4[k] = x[i];
        told4 |= (mask ? mask[i >> 5] >> (i & 31) & 1u : 1u) << k;
      }
    };
    ask_listed(s_part[part] + lane);
    constexpr int U = 4;
    auto stream = [&](int i0, auto whole) {  // U runs of four tokens a lane; whole: none of them passes c1
      float4 f[U];
      uint32_t hide[U];  // of the four tokens: not allowed, or listed (where nothing is written)
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int i = i0 + k * 128 + 4 * lane;
        f[k] = whole.value ? __ldcs(reinterpret_cast<const float4*>(x + i)) : load4(x, i, c1, a.vec);
        hide[k] = mask && (whole.value || i < c1) ? ~mask[i >> 5] >> (i & 31) : 0u;
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int i = i0 + k * 128 + 4 * lane;
        if (!whole.value && i >= c1) break;
        if (!WRITE) hide[k] |= bits[i >> 5] >> (i & 31);
        if (!whole.value && i + 4 > c1) hide[k] |= 15u << (c1 - i);
        if (hide[k] & 15u) {
          f[k].x = hide[k] & 1u ? -INFINITY : f[k].x;
          f[k].y = hide[k] & 2u ? -INFINITY : f[k].y;
          f[k].z = hide[k] & 4u ? -INFINITY : f[k].z;
          f[k].w = hide[k] & 8u ? -INFINITY : f[k].w;
        }
        if (WRITE) {
          if (whole.value || (a.vec && i + 4 <= c1)) {
            __stcs(reinterpret_cast<float4*>(y + i), f[k]);
          } else {
            y[i] = f[k].x;
            if (i + 1 < c1) y[i + 1] = f[k].y;
            if (i + 2 < c1) y[i + 2] = f[k].z;
            if (i + 3 < c1) y[i + 3] = f[k].w;
          }
        } else {
          const float t = fmaxf(fmaxf(f[k].x, f[k].y), fmaxf(f[k].z, f[k].w));
          if (t > high) {
            high = t;
            high_at = i;
            among = f[k];
          }
        }
      }
    };
    int at = c0;
    if (a.vec)
      for (; at + 128 * U <= c1; at += 128 * U) stream(at, std::true_type{});
    for (; at < c1; at += 128 * U) stream(at, std::false_type{});
    Best top;
    if (!WRITE) {
      float most = high;
      for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
      if (most > -INFINITY) {
        if (high == most)  // (tokens not allowed hold -inf; the lanes' candidates meet in the keys below)
          top.take(most, high_at + (among.x == most ? 0 : among.y == most ? 1 : among.z == most ? 2 : 3));
      } else {  // nothing above -inf: the first -inf, or else the first NaN
        for (int i = c0 + lane; i < c1; i += 32)
          if (!(bits[i >> 5] >> (i & 31) & 1u) && (!mask || (mask[i >> 5] >> (i & 31) & 1u))) top.take(x[i], i);
      }
    }
    if (WRITE) __syncwarp();  // a listed token is written again, by another lane
    for (int j0 = s_part[part] + lane; j0 < s_part[part + 1]; j0 += 128) {
      if (j0 >= s_part[part] + 128) ask_listed(j0);
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        if (!(told4 >> k & 1u)) continue;
        const int i = list[j0 + 32 * k];
        float f = k == 0 ? f4[0] : k == 1 ? f4[1] : k == 2 ? f4[2] : f4[3];
        uint32_t c = count ? cnt[i] : 0u;
        if (tree && count)
          for (int32_t p = up[node]; p >= 0;) {
            if (draft[p] == (int32_t)(v0 + i)) ++c;
            p = parent[p] >= 0 ? up[parent[p]] : -1;
          }
        const uint32_t times = c & ~kPromptFlag;
        if (c && has_rep) f = f > 0.0f ? __fdiv_rn(f, rep) : __fmul_rn(f, rep);
        if (times) {
          if (has_freq) f = __fsub_rn(f, __fmul_rn(freq, (float)times));
          if (has_pres) f = __fsub_rn(f, pres);
        }
        if (bias && bias_at[i] > 0) f = __fadd_rn(f, a.r.bias_val[bias_at[i] - 1]);
        if (WRITE) y[i] = f;
        else top.take(f, i);
      }
    }
    if (!WRITE) {
      unsigned long long k = top.at < 0 ? 0ull : arg_key(top.value, v0 + top.at);
      for (int o = 16; o; o >>= 1) {
        const unsigned long long t = __shfl_xor_sync(0xFFFFFFFFu, k, o);
        k = t > k ? t : k;
      }
      if (lane == 0 && k) atomicMax(&best[node], k);
    }
  }
  if (!WRITE) {
    __syncthreads();
    for (int i = tid; i < n; i += T) a.key[(off + i) * a.chunks + blockIdx.x] = best[i];
  }
}

// One block per request: the rows' tokens from their chunks' keys, then acceptance.
__global__ void __launch_bounds__(kAcceptThreads) k_rule_accept(const unsigned long long* __restrict__ key, int chunks,
                                                              const int32_t* __restrict__ parent_g,
                                                              const int32_t* __restrict__ draft_g,
                                                              const int32_t* __restrict__ offsets, int64_t M,
                                                              int32_t* __restrict__ tok_out, int32_t* path_len,
                                                              int32_t* __restrict__ path_nodes, int32_t* bonus) {
  __shared__ int32_t tok[kRuleMaxNodes], parent[kRuleMaxNodes], draft[kRuleMaxNodes];
  __shared__ unsigned long long s_best;
  pdl_enter();  // the keys are the previous kernel's
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t off;
  int n;
  const bool in = request_rows(offsets, M, r, off, n);
  if (!in || n == 0) {
    if (tid == 0) path_len[r] = bonus[r] = -1;
    return;
  }
  bool ok = true;
  for (int i = tid; i < n; i += kAcceptThreads) {
    const int32_t p = parent_g[off + i];
    ok = ok && (i == 0 ? p == -1 : p >= 0 && p < i);
    parent[i] = p;
    draft[i] = draft_g[off + i];
    path_nodes[off + i] = -1;
  }
  if (tid == 0) s_best = 0;
  ok = __syncthreads_and(ok) != 0;
  for (int i = warp; i < n; i += kAcceptWarps) {
    unsigned long long top = 0;
    const unsigned long long* k = key + (off + i) * chunks;
    for (int c = lane; c < chunks; c += 32) top = k[c] > top ? k[c] : top;
    for (int o = 16; o; o >>= 1) {
      const unsigned long long t = __shfl_xor_sync(0xFFFFFFFFu, top, o);
      top = t > top ? t : top;
    }
    if (lane == 0) tok[i] = tok_out[off + i] = top ? (int32_t)(0xFFFFFFFFu - (uint32_t)top) : -1;
  }
  if (!ok) {
    if (tid == 0) path_len[r] = bonus[r] = -1;
    return;
  }
  __syncthreads();
  // every node walks its own path; the deepest accepted one wins, the lowest index among equals
  for (int i = tid; i < n; i += kAcceptThreads) {
    int32_t depth = 0, p = i;
    bool taken = true;
    while (p > 0 && taken) {
      const int32_t t = tok[parent[p]];
      taken = t >= 0 && draft[p] == t;
      p = parent[p];
      ++depth;
    }
    if (taken) atomicMax(&s_best, ((unsigned long long)(depth + 1) << 32) | (0xFFFFFFFFu - (uint32_t)i));
  }
  __syncthreads();
  if (tid == 0) {
    const int32_t depth = (int32_t)(s_best >> 32) - 1, node = (int32_t)(0xFFFFFFFFu - (uint32_t)s_best);
    path_len[r] = depth;
    bonus[r] = tok[node];
    int32_t p = node;
    for (int32_t j = depth; j >= 0; --j) {
      path_nodes[off + j] = p;
      p = parent[p];
    }
  }
}

struct RulePlan {
  int chunk, chunks, parts, threads;
};

// Chunk of the vocabulary per block, a multiple of 256: the larger it is, the fewer blocks
// scan a request's history and the more rows share the table; the smaller, the more blocks
// there are.  The largest of 4096, 2048, 1024 with at least two blocks per SM: 192 rows took 47.8 us
// written and 37.5 verified at 4096, 51.3 and 49.8 at 2048; a 16-node tree 12.4 at 1024, 13.7 at 512.
// Parts of a row's chunk, one a warp at a time: smaller ones even out trees of unequal size, larger ones
// meet fewer loads' latencies (24 trees of 8 rows in the mean: 47.8 us at 1 part, 47.8 at 2, 49.7 at 4
// written, 34.3, 37.5 and 43.3 verified; a 16-node tree 12.4 at 1, 14.0 at 2).
// Threads: one row has eight parts, so eight warps (5.5 us, 5.9 at 384 threads, 5.9 at 512); where
// every block has an SM's half to itself, 512 make its tables and sixteen rows at once (a 16-node tree
// 12.4 us, 15.0 at 384, 15.5 at 256); else 384 (192 rows written 47.8 us, 49.4 at 256, 49.2 at 512;
// verified 37.5, 42.0, 46.3).
RulePlan rule_plan(int64_t M, int64_t V, int32_t n_req) {
  RulePlan p{};
  for (p.chunk = 4096; p.chunk > 1024; p.chunk /= 2)
    if ((V + p.chunk - 1) / p.chunk * n_req >= 304) break;
  p.chunks = (int)((V + p.chunk - 1) / p.chunk);
  const int64_t rows = (M + n_req - 1) / n_req;
  p.parts = rows >= 16 ? 1 : rows >= 8 ? 2 : rows >= 4 ? 4 : kRuleParts;
  p.threads = M <= n_req ? 256 : (int64_t)p.chunks * n_req <= 304 ? 512 : 384;
  return p;
}

int check_rules(const float* logits, int64_t stride, int64_t M, int64_t V, const logit_rules* rules,
                const int32_t* parent, const int32_t* draft, const int32_t* req_offsets, int32_t n_req,
                const int32_t* status, const char* fn) {
  if (!logits || !rules || !status) return fail(W12_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (M < 1 || M > 0x7FFFFFFF || V < 1 || V > 0x7FFFFFFF || stride < V || n_req < 1 || n_req > 65535)
    return fail(W12_ERR_SHAPE, "%s: M=%lld, V=%lld (stride %lld), n_req=%d (1..65535) out of range", fn, (long long)M,
                (long long)V, (long long)stride, n_req);
  if (!req_offsets && n_req != 1)
    return fail(W12_ERR_INVALID_ARG, "%s: req_offsets is null but n_req=%d", fn, n_req);
  if (!parent != !draft) return fail(W12_ERR_INVALID_ARG, "%s: parent and draft go together", fn);
  if (rules->hist && (!rules->hist_len || rules->hist_stride < 1))
    return fail(W12_ERR_INVALID_ARG, "%s: a history needs its lengths and a stride", fn);
  if ((rules->bias_off != nullptr) != (rules->bias_tok != nullptr) ||
      (rules->bias_off != nullptr) != (rules->bias_val != nullptr) || rules->n_bias < 0 || rules->n_bias > 0x7FFFFFFE)
    return fail(W12_ERR_INVALID_ARG, "%s: a bias needs offsets, tokens, values and a count", fn);
  if (rules->mask && rules->mask_stride < (V + 31) / 32)
    return fail(W12_ERR_SHAPE, "%s: mask_stride=%lld is less than a row's words", fn, (long long)rules->mask_stride);
  return W12_OK;
}

void (*const kRuleKernels[6])(RuleArgs) = {  // 256, 384 and 512 threads; verified, written
    k_logit_rules<false, 256>, k_logit_rules<false, 384>, k_logit_rules<false, 512>,
    k_logit_rules<true, 256>,  k_logit_rules<true, 384>,  k_logit_rules<true, 512>};

int launch_rules(const float* logits, int64_t stride, int64_t M, int64_t V, const logit_rules* rules,
                 const int32_t* parent, const int32_t* draft, const int32_t* req_offsets, int32_t n_req, float* out,
                 int64_t out_stride, int32_t* status, unsigned long long* key, cudaStream_t s, const char* what) {
  const RulePlan p = rule_plan(M, V, n_req);
  RuleArgs a{};
  a.logits = logits;
  a.stride = stride;
  a.M = M;
  a.V = V;
  a.r = *rules;
  a.parent = parent;
  a.draft = draft;
  a.req_offsets = req_offsets;
  a.n_req = n_req;
  a.out = out;
  a.out_stride = out_stride;
  a.status = status;
  a.key = key;
  a.chunk = p.chunk;
  a.chunks = p.chunks;
  a.parts = p.parts;
  const bool count = rules->rep || rules->freq || rules->pres;
  const int64_t nodes = M < kRuleMaxNodes ? M : kRuleMaxNodes;
  const size_t smem = (size_t)p.chunk / 8 + (count ? (size_t)p.chunk * 4 : 0) + (rules->bias_off ? (size_t)p.chunk * 4 : 0) +
                      (parent ? (size_t)nodes * 12 : 0) + (key ? (size_t)(nodes + 1) * 8 : 0) + (size_t)p.chunk * 2;
  constexpr size_t most = 4096 / 8 + 4096 * 10 + kRuleMaxNodes * 20 + 8;
  static int configured[64] = {0};
  int dev = 0;
  W12_CUDA_TRY(cudaGetDevice(&dev));
  if (dev >= 64 || !configured[dev]) {
    for (auto kernel : kRuleKernels)
      W12_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most));
    if (dev < 64) configured[dev] = 1;
  }
  a.vec = ((stride | (out ? out_stride : 0)) & 3) == 0 && (((uintptr_t)logits | (uintptr_t)out) & 15u) == 0;
  a.hist_vec = rules->hist && (rules->hist_stride & 3) == 0 && ((uintptr_t)rules->hist & 15u) == 0;
  const dim3 grid((unsigned)p.chunks, (unsigned)n_req);
  W12_CUDA_TRY(launch_dependent(kRuleKernels[(key ? 0 : 3) + p.threads / 128 - 2], grid, p.threads, smem, s, a));
  W12_LAUNCH_CHECK(what);
  return W12_OK;
}

}  // namespace
}  // namespace w12

using namespace w12;

extern "C" {

int logits_process(const float* logits, int64_t stride, int64_t M, int64_t V, const logit_rules* rules,
                   const int32_t* parent, const int32_t* draft, const int32_t* req_offsets, int32_t n_req, float* out,
                   int64_t out_stride, int32_t* status, void* stream) {
  int st = check_rules(logits, stride, M, V, rules, parent, draft, req_offsets, n_req, status, "logits_process");
  if (st) return st;
  if (!out) return fail(W12_ERR_INVALID_ARG, "logits_process: null pointer");
  if (out_stride < V) return fail(W12_ERR_SHAPE, "logits_process: out_stride=%lld is less than V", (long long)out_stride);
  // In place, apart, or side by side in the rows of one array.
  const uintptr_t l0 = (uintptr_t)logits, o0 = (uintptr_t)out, row = (uintptr_t)V * 4, pitch = (uintptr_t)stride * 4;
  const uintptr_t by = (o0 > l0 ? o0 - l0 : l0 - o0) % pitch;
  const bool alike = stride == out_stride || M == 1;
  const bool apart = o0 >= l0 + (M - 1) * pitch + row || l0 >= o0 + (uintptr_t)(M - 1) * out_stride * 4 + row;
  if (!apart && !(alike && (o0 == l0 || (M > 1 && by >= row && by + row <= pitch))))
    return fail(W12_ERR_INVALID_ARG, "logits_process: out must be logits or not overlap it");
  return launch_rules(logits, stride, M, V, rules, parent, draft, req_offsets, n_req, out, out_stride, status, nullptr,
                      (cudaStream_t)stream, "logits_process kernel");
}

size_t logits_verify_workspace_size(int64_t M, int64_t V, int32_t n_req) {
  if (M < 1 || V < 1 || n_req < 1) return 0;
  return (size_t)M * (size_t)rule_plan(M, V, n_req).chunks * 8;
}

int logits_verify(const float* logits, int64_t stride, int64_t M, int64_t V, const logit_rules* rules,
                  const int32_t* parent, const int32_t* draft, const int32_t* req_offsets, int32_t n_req, int32_t* tok,
                  int32_t* path_len, int32_t* path_nodes, int32_t* bonus, int32_t* status, void* ws, size_t ws_bytes,
                  void* stream) {
  int st = check_rules(logits, stride, M, V, rules, parent, draft, req_offsets, n_req, status, "logits_verify");
  if (st) return st;
  if (!parent || !tok || !path_len || !path_nodes || !bonus || !ws)
    return fail(W12_ERR_INVALID_ARG, "logits_verify: null pointer");
  if ((uintptr_t)ws & 7u) return fail(W12_ERR_INVALID_ARG, "logits_verify: the workspace must be 8-byte aligned");
  if (ws_bytes < logits_verify_workspace_size(M, V, n_req))
    return fail(W12_ERR_BUFFER_TOO_SMALL, "logits_verify: workspace %zu < %zu", ws_bytes,
                logits_verify_workspace_size(M, V, n_req));
  unsigned long long* key = static_cast<unsigned long long*>(ws);
  st = launch_rules(logits, stride, M, V, rules, parent, draft, req_offsets, n_req, nullptr, 0, status, key,
                    (cudaStream_t)stream, "logits_verify: rules kernel");
  if (st) return st;
  W12_CUDA_TRY(launch_dependent(k_rule_accept, dim3((unsigned)n_req), kAcceptThreads, 0, (cudaStream_t)stream, key,
                                rule_plan(M, V, n_req).chunks, parent, draft, req_offsets, M, tok, path_len, path_nodes, bonus));
  W12_LAUNCH_CHECK("logits_verify: acceptance kernel");
  return W12_OK;
}

}  // extern "C"
