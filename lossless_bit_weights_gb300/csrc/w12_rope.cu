// w12_rope.cu - from a fused projection's rows to the q, k and v of attention: positions of tree
// nodes, norms of each head and the position rotation in one pass, and the same with K and V going
// straight into their slots of a paged cache.
#include <cstdint>
#include <iterator>

#include "w12_internal.cuh"
#include "w12_pdl.cuh"

namespace w12 {

int check_cache(const kv_cache* c, const char* fn);

namespace {

// ---------------------------------------------------------------- positions

constexpr int kPosThreads = 256;
constexpr int kPosMaxNodes = 4096;  // nodes of one tree
constexpr int32_t kPosBadRequest = 1;

struct PosArgs {
  const int32_t *cache_len, *parent, *req_offsets;
  int32_t *pos, *status;
  int64_t rows;
  int32_t n_req;
};

// A request's rows [off, off + n), and whether its numbers are in range.
__device__ __forceinline__ bool pos_request(const PosArgs& a, int r, int64_t& off, int64_t& n) {
  const int64_t from = a.req_offsets ? a.req_offsets[r] : 0, to = a.req_offsets ? a.req_offsets[r + 1] : a.rows;
  const int64_t len = a.cache_len[r];
  off = min(max(from, (int64_t)0), a.rows);
  n = max(min(to, a.rows) - off, (int64_t)0);
  return from >= 0 && to >= from && to <= a.rows && len >= 0 && len + n <= 0x7FFFFFFF;
}

constexpr int kChainRows = 4;        // rows of a thread
constexpr int kChainRequests = 2048;  // offsets that fit in shared memory

// Chains (prompts, single tokens): a thread finds its first row's request by halving, in shared memory where the
// offsets fit, and goes on from there.  448,507 rows of 500 requests in 3.4 us (5.8 with a row a thread that halves in
// global memory): launch and two loads' latencies.
__global__ void __launch_bounds__(kPosThreads) k_chain_positions(const __grid_constant__ PosArgs a) {
  pdl_enter();
  __shared__ int32_t offsets[kChainRequests + 1];
  const int64_t t0 = (int64_t)blockIdx.x * kPosThreads + threadIdx.x, step = (int64_t)gridDim.x * kPosThreads;
  const bool here = a.req_offsets && a.n_req <= kChainRequests;
  if (here)
    for (int r = threadIdx.x; r <= a.n_req; r += kPosThreads) offsets[r] = a.req_offsets[r];
  __syncthreads();
  const int32_t* o = here ? offsets : a.req_offsets;
  for (int64_t r = t0; r < a.n_req; r += step) {
    int64_t off, n;
    if (!pos_request(a, (int)r, off, n)) atomicOr(a.status, kPosBadRequest);
  }
  for (int64_t i0 = t0 * kChainRows; i0 < a.rows; i0 += step * kChainRows) {
    int lo = 0, hi = a.n_req;  // the last request that starts at or before row i0
    while (o && hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (o[mid] <= i0) lo = mid; else hi = mid;
    }
    int64_t off, n;
    bool ok = pos_request(a, lo, off, n);
    int32_t len = a.cache_len[lo], pos[kChainRows];
#pragma unroll
    for (int k = 0; k < kChainRows; ++k) {
      const int64_t i = i0 + k;
      bool next = false;
      while (o && lo + 1 < a.n_req && o[lo + 1] <= i) {
        ++lo;
        next = true;
      }
      if (next) {
        ok = pos_request(a, lo, off, n);
        len = a.cache_len[lo];
      }
      pos[k] = ok && i >= off && i < off + n ? (int32_t)(len + (i - off)) : -1;
    }
    if (i0 + kChainRows <= a.rows && ((uintptr_t)a.pos & 15u) == 0) {
      *reinterpret_cast<int4*>(a.pos + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
      for (int k = 0; k < kChainRows && i0 + k < a.rows; ++k) a.pos[i0 + k] = pos[k];
    }
  }
}

// Trees: a block takes a request and doubles the step of every node's way up until all ways end at
// the root (3 rounds for 8 nodes, 12 for 4096), in shared memory.  Bound by its chain of loads
// (offsets, parents) and barriers, not by bytes: 24 trees of 192 nodes in 2.0 us.  The blocks behind the requests' fill the rows of none.
__global__ void __launch_bounds__(kPosThreads) k_tree_positions(const __grid_constant__ PosArgs a) {
  pdl_enter();
  __shared__ uint16_t up[2][kPosMaxNodes], depth[2][kPosMaxNodes];
  const int tid = threadIdx.x;
  if ((int)blockIdx.x >= a.n_req) {
    const int64_t first = a.req_offsets ? a.req_offsets[0] : 0, last = a.req_offsets ? a.req_offsets[a.n_req] : a.rows;
    const int64_t step = (int64_t)(gridDim.x - a.n_req) * kPosThreads;
    for (int64_t i = (int64_t)(blockIdx.x - a.n_req) * kPosThreads + tid; i < a.rows; i += step)
      if (i < first || i >= last) a.pos[i] = -1;
    return;
  }
  int64_t off, n64;
  bool ok = pos_request(a, blockIdx.x, off, n64) && n64 <= kPosMaxNodes;
  const int n = ok ? (int)n64 : 0;
  for (int i = tid; i < n; i += kPosThreads) {
    const int32_t p = a.parent[off + i];
    ok = ok && (i == 0 ? p == -1 : p >= 0 && p < i);
    up[0][i] = (uint16_t)(i == 0 ? 0 : p & (kPosMaxNodes - 1));
    depth[0][i] = i != 0;
  }
  if (!__syncthreads_and(ok)) {
    for (int64_t i = tid; i < n64; i += kPosThreads) a.pos[off + i] = -1;
    if (tid == 0) atomicOr(a.status, kPosBadRequest);
    return;
  }
  int b = 0;
  for (int reach = 1; reach < n; reach *= 2) {  // every way's first `reach` steps are counted
    bool more = false;
    for (int i = tid; i < n; i += kPosThreads) {
      const int u = up[b][i];
      depth[b ^ 1][i] = depth[b][i] + depth[b][u];
      up[b ^ 1][i] = up[b][u];
      more = more || up[b][u] != 0;
    }
    b ^= 1;
    if (!__syncthreads_or(more)) break;
  }
  const int32_t len = n ? a.cache_len[blockIdx.x] : 0;
  for (int i = tid; i < n; i += kPosThreads) a.pos[off + i] = len + depth[b][i];
}

// ---------------------------------------------------------------- norms and rotation

struct RopeArgs {
  const void* x;
  int64_t x_stride, M;
  const float *q_norm, *k_norm, *inv_freq;
  const int32_t* pos;
  uint16_t* out[3];        // q, k, v rows (null: not asked for)
  int64_t out_stride[3];
  uint16_t* cache[2];      // K, V at the layer, or null
  int64_t block_stride, token_stride, head_stride, n_slots;
  const int64_t* slot;
  int32_t* status;
  float eps, rot_scale;
  int32_t n_q, n_kv, d, half, block_size;
  bool stream;
};

constexpr int kRopeThreads = 128;

// Blocks on an SM, by the elements' size and the heads that a lane works on at once.
constexpr int rope_blocks(int size, int at_once) { return size == 4 || at_once == 4 ? 7 : 8; }

constexpr int kRopeMaxDim = 256;

__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {  // a in the low half, to nearest even
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// A lane's eight columns of a head, [lo, lo+4) and [hi, hi+4), eight adjacent ones where NEXT, as they were loaded.
template <typename T, bool NEXT>
struct Eight;

template <bool NEXT>
struct Eight<float, NEXT> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* x, int lo, int hi) {
    a = __ldcs(reinterpret_cast<const float4*>(x + lo));
    b = __ldcs(reinterpret_cast<const float4*>(x + hi));
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ __forceinline__ void get(float f[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
};

template <bool NEXT>
struct Eight<uint16_t, NEXT> {
  uint4 w;
  __device__ __forceinline__ void load(const uint16_t* x, int lo, int hi) {
    if constexpr (NEXT) {
      w = __ldcs(reinterpret_cast<const uint4*>(x + lo));
    } else {
      const uint2 a = __ldcs(reinterpret_cast<const uint2*>(x + lo)), b = __ldcs(reinterpret_cast<const uint2*>(x + hi));
      w = make_uint4(a.x, a.y, b.x, b.y);
    }
  }
  __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float f[8]) const {
    f[0] = bf16_low(w.x), f[1] = bf16_high(w.x), f[2] = bf16_low(w.y), f[3] = bf16_high(w.y);
    f[4] = bf16_low(w.z), f[5] = bf16_high(w.z), f[6] = bf16_low(w.w), f[7] = bf16_high(w.w);
  }
};

// (stream: more than L2 keeps, so that it should make room first)
template <bool NEXT>
__device__ __forceinline__ void store8(uint16_t* y, int lo, int hi, const uint32_t w[4], bool stream) {
  if constexpr (NEXT) {
    uint4* to = reinterpret_cast<uint4*>(y + lo);
    const uint4 v = make_uint4(w[0], w[1], w[2], w[3]);
    if (stream) __stcs(to, v);
    else *to = v;
  } else {
    uint2 *a = reinterpret_cast<uint2*>(y + lo), *b = reinterpret_cast<uint2*>(y + hi);
    const uint2 v = make_uint2(w[0], w[1]), z = make_uint2(w[2], w[3]);
    if (stream) {
      __stcs(a, v);
      __stcs(b, z);
    } else {
      *a = v;
      *b = z;
    }
  }
}

// Turns that a position moves a pair by, modulo 1, in units of 2^-64: inv_freq / (2 pi) = m R 2^(E - 278) with the
// float's mantissa m and exponent E and R = 2^128 / (2 pi).  A position times it, modulo 2^64, drops whole
// turns exactly and leaves an error below 1.5 * 2^-32 turns at 2^31 - 1 (the product's cut to 32 bits among it).  The float
// that sine and cosine are taken of rounds by 2^-26 turns at most.
__device__ __forceinline__ uint64_t turns_of(float inv_freq) {
  constexpr uint64_t kHigh = 0x28BE60DB9391054Aull, kLow = 0x7F09D5F47D4D3770ull;
  const uint32_t bits = __float_as_uint(inv_freq), e = bits >> 23 & 255u;
  const uint64_t m = (bits & 0x7FFFFFu) | (e ? 0x800000u : 0u);
  const uint64_t w0 = m * kLow, t = __umul64hi(m, kLow), w1 = m * kHigh + t;
  const uint64_t w2 = __umul64hi(m, kHigh) + (w1 < t);
  const int s = 214 - (int)max(e, 1u);  // m R shifted right by s
  uint64_t f = 0;
  if (s >= 128) f = w2 >> (s - 128);
  else if (s > 64) f = w1 >> (s - 64) | w2 << (128 - s);
  else if (s == 64) f = w1;
  else if (s > 0) f = w0 >> s | w1 << (64 - s);
  return bits >> 31 ? 0 - f : f;
}

// One row a block (and a share of its heads, gridDim.y), P lanes a head, eight columns a lane, U heads at a time:
//   y = x * rsqrt(mean(x^2) + eps) * w,   (a, b) -> s (a cos - b sin, b cos + a sin),
// with both columns of a pair in one lane, so that the rotation needs no exchange and the norm one sum
// over P lanes, the U heads' sums side by side.  The row's sines are found once, a thread each, while the first
// heads are on their way; the next heads are on theirs while U are worked on.
// Bound by bytes, the row read once and written once: 12289 float rows of 56 heads of 128, with norms, into a cache in
// 80.7 us (529 MB, 6.55 TB/s, 0.97 of the measured copy rate), 12289 bf16 rows of 32 heads of 256 without norms in 61.3
// (6.57 TB/s).  bf16 rows with norms are bound by instructions, 71 us for those heads, 67 for the 56 of 128.  Few rows are
// launch and latency: one 2.0 us, 192 3.8.
// What it took on the way (float, bf16): all heads' loads behind the position's 92, 99; the sums one by
// one 88, 79 with norms; rows that L2 cannot keep not streamed out 82, 62.
// U = 2 for float (4: 121 us) and for bf16 rows with norms (4: 82 for 67) or few rows (4: 4.9 us for 3.8 at 192 rows);
// 4 for the others (2: 66 us for 62).
template <typename T, int P, bool NEXT, int U>
__global__ void __launch_bounds__(kRopeThreads, rope_blocks(sizeof(T), U)) k_qkv_rope(const __grid_constant__ RopeArgs a) {
  constexpr int kGroups = kRopeThreads / P;  // heads of a block at a time
  __shared__ __align__(16) float s_cos[kRopeMaxDim / 2], s_sin[kRopeMaxDim / 2], s_norm[2][kRopeMaxDim];
  __shared__ int64_t s_place;
  pdl_enter();
  const int tid = threadIdx.x, g = tid / P, u = tid % P;
  const int64_t t = blockIdx.x;
  const int heads = a.n_q + 2 * a.n_kv, first = blockIdx.y * kGroups, step = gridDim.y * kGroups;
  const bool live = 8 * u < a.d, turned = 8 * u < 2 * a.half;
  const int lo = !NEXT && turned ? 4 * u : 8 * u, hi = !NEXT && turned ? a.half + 4 * u : 8 * u + 4;
  const T* x = static_cast<const T*>(a.x) + t * a.x_stride;
  const bool norm = a.q_norm || a.k_norm;
  Eight<T, NEXT> f[U];
  auto ask = [&](Eight<T, NEXT>& to, int h) {
    if (live && h < heads) to.load(x + h * a.d, lo, hi);
    else to.zero();
  };
  const int32_t pos = a.pos[t];
#pragma unroll
  for (int k = 0; k < U; ++k) ask(f[k], first + g + k * step);
  const float freq = tid < a.half ? a.inv_freq[tid] : 0.0f;
  int64_t place = a.cache[0] ? a.slot[t] : -1;
  if (norm)
    for (int c = tid; c < a.d; c += kRopeThreads) {
      s_norm[0][c] = a.q_norm ? a.q_norm[c] : 1.0f;
      s_norm[1][c] = a.k_norm ? a.k_norm[c] : 1.0f;
    }
  if (pos < 0) return;  // padding
  if (tid < a.half) {  // (half <= 128 threads)
    const int32_t turn = (int32_t)((uint64_t)(uint32_t)pos * turns_of(freq) >> 32);
    float sn, cs;
    sincospif((float)turn * 4.656612873077393e-10f, &sn, &cs);  // 2^-31: half turns
    s_cos[tid] = cs * a.rot_scale;
    s_sin[tid] = sn * a.rot_scale;
  }
  if (a.cache[0] && tid == kRopeThreads - 1) {
    if (place != -1) {
      if (place < 0 || place >= a.n_slots) {
        atomicOr(a.status, 1);
        place = -1;
      } else {
        const int64_t block = place / a.block_size;
        place = block * a.block_stride + (place - block * a.block_size) * a.token_stride;
      }
    }
    s_place = place;
  }
  __syncthreads();
  place = a.cache[0] ? s_place : -1;
  float c4[4] = {1.0f, 1.0f, 1.0f, 1.0f}, s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (turned) {
    const float4 cs = *reinterpret_cast<const float4*>(s_cos + 4 * u), sn = *reinterpret_cast<const float4*>(s_sin + 4 * u);
    c4[0] = cs.x, c4[1] = cs.y, c4[2] = cs.z, c4[3] = cs.w;
    s4[0] = sn.x, s4[1] = sn.y, s4[2] = sn.z, s4[3] = sn.w;
  }
  const float inv_d = 1.0f / (float)a.d;
  for (int h0 = first; h0 < heads; h0 += U * step) {  // the same for all lanes
    float y[U][8];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      f[k].get(y[k]);
      ask(f[k], h0 + g + (U + k) * step);  // the next head takes this one's place
    }
    if (norm) {
      float sum[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        sum[k] = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[k] = fmaf(y[k][i], y[k][i], sum[k]);
      }
#pragma unroll
      for (int o = P / 2; o; o >>= 1)
#pragma unroll
        for (int k = 0; k < U; ++k) sum[k] += __shfl_xor_sync(0xFFFFFFFFu, sum[k], o);
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int h = h0 + g + k * step, key = h >= a.n_q;
        if (live && (key ? a.k_norm && h < a.n_q + a.n_kv : a.q_norm != nullptr)) {
          const float r = rsqrtf(fmaf(sum[k], inv_d, a.eps));
          const float4 w0 = *reinterpret_cast<const float4*>(s_norm[key] + lo), w1 = *reinterpret_cast<const float4*>(s_norm[key] + hi);
          y[k][0] *= r * w0.x, y[k][1] *= r * w0.y, y[k][2] *= r * w0.z, y[k][3] *= r * w0.w;
          y[k][4] *= r * w1.x, y[k][5] *= r * w1.y, y[k][6] *= r * w1.z, y[k][7] *= r * w1.w;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int h = h0 + g + k * step;
      if (!live || h >= heads) continue;
      const int part = h < a.n_q ? 0 : h < a.n_q + a.n_kv ? 1 : 2;
      if (part < 2) {  // (a choice at the end: a branch that parts a warp costs 0.8 us of the bf16 rows' 61)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float &p = NEXT ? y[k][2 * i] : y[k][i], &q = NEXT ? y[k][2 * i + 1] : y[k][i + 4];
          const float p0 = p, q0 = q;
          p = turned ? fmaf(p0, c4[i], -(q0 * s4[i])) : p0;
          q = turned ? fmaf(q0, c4[i], p0 * s4[i]) : q0;
        }
      }
      const uint32_t b[4] = {pack_bf16(y[k][0], y[k][1]), pack_bf16(y[k][2], y[k][3]), pack_bf16(y[k][4], y[k][5]),
                             pack_bf16(y[k][6], y[k][7])};
      const int in = h - (part == 0 ? 0 : part == 1 ? a.n_q : a.n_q + a.n_kv);
      if (a.out[part]) store8<NEXT>(a.out[part] + t * a.out_stride[part] + in * a.d, lo, hi, b, a.stream);
      if (part && place >= 0) store8<NEXT>(a.cache[part - 1] + place + in * a.head_stride, lo, hi, b, a.stream);
    }
  }
}

template <typename T, int P, int U>
constexpr auto rope_kernel(bool next) {
  return next ? k_qkv_rope<T, P, true, U> : k_qkv_rope<T, P, false, U>;
}

// Rows of two strided arrays that share no element: apart, or side by side in the rows of one array.
bool rows_apart(uintptr_t a, uintptr_t a_row, uintptr_t a_pitch, uintptr_t b, uintptr_t b_row, uintptr_t b_pitch, int64_t n) {
  if (a + (n - 1) * a_pitch + a_row <= b || b + (n - 1) * b_pitch + b_row <= a) return true;
  if (n < 2 || a_pitch != b_pitch) return false;
  const uintptr_t by = (b > a ? b - a : a - b) % a_pitch;  // of the later one behind a row's start of the earlier
  return by >= (b > a ? a_row : b_row) && by + (b > a ? b_row : a_row) <= a_pitch;
}

// The checks that both calls share, and the kernel's arguments but for the cache's.
int rope_args(RopeArgs& a, const char* fn, const void* x, int32_t x_bf16, int64_t x_stride, int64_t M, const qkv_form* form,
              const int32_t* pos, uint16_t* q, int64_t q_stride, uint16_t* k, int64_t k_stride, uint16_t* v,
              int64_t v_stride) {
  if (!form) return fail(W12_ERR_INVALID_ARG, "%s: null form", fn);
  const int64_t nq = form->n_q_heads, nk = form->n_heads, d = form->head_dim;
  if (nq < 1 || nk < 1 || nq > 65535 || nk > 65535 || d < 8 || d > kRopeMaxDim || (d & 7) || form->rot_dim < 0 ||
      form->rot_dim > d || (form->rot_dim & 7))
    return fail(W12_ERR_SHAPE, "%s: %lld + 2 x %lld heads of %lld (a multiple of 8 up to %d), %d of them rotated (a multiple of 8)",
                fn, (long long)nq, (long long)nk, (long long)d, kRopeMaxDim, form->rot_dim);
  const int64_t width = (nq + 2 * nk) * d;
  if (M < 1 || M > 0x7FFFFFFF || (M > 1 && x_stride < width))
    return fail(W12_ERR_SHAPE, "%s: M=%lld rows of %lld (stride %lld) out of range", fn, (long long)M, (long long)width,
                (long long)x_stride);
  if (!x || !pos) return fail(W12_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (form->rot_dim && !form->inv_freq) return fail(W12_ERR_INVALID_ARG, "%s: a rotation needs its frequencies", fn);
  if (!(form->eps >= 0.0f) || !(form->eps <= 1e30f) || !(form->rot_scale >= -1e30f) || !(form->rot_scale <= 1e30f))
    return fail(W12_ERR_INVALID_ARG, "%s: eps=%g, rot_scale=%g out of range", fn, form->eps, form->rot_scale);
  uint16_t* out[3] = {q, k, v};
  const int64_t stride[3] = {q_stride, k_stride, v_stride}, wide[3] = {nq * d, nk * d, nk * d}, at[3] = {0, nq * d, (nq + nk) * d};
  uintptr_t bits = (uintptr_t)x;
  int64_t strides = x_stride;
  for (int i = 0; i < 3; ++i) {
    if (!out[i]) continue;
    bits |= (uintptr_t)out[i];
    strides |= stride[i];
    if (M > 1 && stride[i] < wide[i])
      return fail(W12_ERR_SHAPE, "%s: rows of %lld at a stride of %lld", fn, (long long)wide[i], (long long)stride[i]);
  }
  if ((bits & 15u) || (strides & 7))
    return fail(W12_ERR_INVALID_ARG, "%s: rows must be 16-byte aligned and their strides multiples of 8", fn);
  const int size = x_bf16 ? 2 : 4;
  // what all rows read: the norms' weights and the frequencies
  const float* const form_array[3] = {form->q_norm, form->k_norm, form->rot_dim ? form->inv_freq : nullptr};
  const uintptr_t form_bytes[3] = {(uintptr_t)d * 4, (uintptr_t)d * 4, (uintptr_t)form->rot_dim * 2};
  for (int i = 0; i < 3; ++i) {
    if (!out[i]) continue;
    const uintptr_t o = (uintptr_t)out[i], row = (uintptr_t)wide[i] * 2, pitch = (uintptr_t)stride[i] * 2;
    // in the place of the part of bf16 rows that it comes from, or nowhere in them
    const bool same = x_bf16 && o == (uintptr_t)x + (uintptr_t)at[i] * 2 && (stride[i] == x_stride || M == 1);
    bool ok = same || rows_apart(o, row, pitch, (uintptr_t)x, (uintptr_t)width * size, (uintptr_t)x_stride * size, M);
    ok = ok && rows_apart(o, row, pitch, (uintptr_t)pos, (uintptr_t)M * 4, 0, M);
    for (int j = 0; j < 3; ++j)
      ok = ok && (!form_array[j] || rows_apart(o, row, pitch, (uintptr_t)form_array[j], form_bytes[j], 0, M));
    for (int j = 0; j < i; ++j)
      ok = ok && (!out[j] || rows_apart(o, row, pitch, (uintptr_t)out[j], (uintptr_t)wide[j] * 2, (uintptr_t)stride[j] * 2, M));
    if (!ok) return fail(W12_ERR_INVALID_ARG, "%s: q, k and v must not overlap one another or what the call reads", fn);
    a.out[i] = out[i];
    a.out_stride[i] = stride[i];
  }
  a.x = x;
  a.x_stride = x_stride;
  a.M = M;
  a.q_norm = form->q_norm;
  a.k_norm = form->k_norm;
  a.inv_freq = form->inv_freq;
  a.pos = pos;
  a.eps = form->eps;
  a.rot_scale = form->rot_scale;
  a.n_q = (int32_t)nq;
  a.n_kv = (int32_t)nk;
  a.d = (int32_t)d;
  a.half = form->rot_dim / 2;
  a.stream = M * width * 2 > (int64_t)64 << 20;
  return W12_OK;
}

int launch_rope(const RopeArgs& a, int32_t x_bf16, int32_t interleaved, cudaStream_t s, const char* what) {
  const int lanes = a.d <= 64 ? 8 : a.d <= 128 ? 16 : 32;
  const bool next = interleaved || a.half == 0;  // (without a rotation the columns may as well be adjacent)
  const int groups = kRopeThreads / lanes, most = (a.n_q + 2 * a.n_kv + groups - 1) / groups;
  // few rows: their heads over more blocks, four an SM (256 rows took 3.8 us, 4.8 at three, 4.4 at six)
  int64_t split = 608 / a.M;
  split = split < 1 ? 1 : split > most ? most : split;
  using Kernel = void (*)(RopeArgs);
  const Kernel kernels[3][3] = {
      {rope_kernel<float, 8, 2>(next), rope_kernel<float, 16, 2>(next), rope_kernel<float, 32, 2>(next)},
      {rope_kernel<uint16_t, 8, 2>(next), rope_kernel<uint16_t, 16, 2>(next), rope_kernel<uint16_t, 32, 2>(next)},
      {rope_kernel<uint16_t, 8, 4>(next), rope_kernel<uint16_t, 16, 4>(next), rope_kernel<uint16_t, 32, 4>(next)}};
  const Kernel kernel = kernels[!x_bf16 ? 0 : split > 1 || a.q_norm || a.k_norm ? 1 : 2][lanes == 8 ? 0 : lanes == 16 ? 1 : 2];
  W12_CUDA_TRY(launch_dependent(kernel, dim3((unsigned)a.M, (unsigned)split), kRopeThreads, 0, s, a));
  W12_LAUNCH_CHECK(what);
  return W12_OK;
}

}  // namespace
}  // namespace w12

using namespace w12;

extern "C" {

int tree_positions(const int32_t* cache_len, const int32_t* parent, const int32_t* req_offsets, int32_t n_req, int64_t rows,
                   int32_t* pos, int32_t* status, void* stream) {
  if (n_req < 1 || n_req > 65535 || rows < 1 || rows > 0x7FFFFFFF)
    return fail(W12_ERR_SHAPE, "tree_positions: n_req=%d (1..65535), rows=%lld out of range", n_req, (long long)rows);
  if (!cache_len || !pos || !status) return fail(W12_ERR_INVALID_ARG, "tree_positions: null pointer");
  if (!req_offsets && n_req != 1)
    return fail(W12_ERR_INVALID_ARG, "tree_positions: req_offsets is null but n_req=%d", n_req);
  const uintptr_t o = (uintptr_t)pos, end = o + (uintptr_t)rows * 4;
  auto meets = [&](const void* p, int64_t n) { return p && (uintptr_t)p < end && o < (uintptr_t)p + (uintptr_t)n * 4; };
  if (meets(cache_len, n_req) || meets(parent, rows) || meets(req_offsets, n_req + 1) || meets(status, 1))
    return fail(W12_ERR_INVALID_ARG, "tree_positions: pos must not overlap what the call reads");
  PosArgs a{cache_len, parent, req_offsets, pos, status, rows, n_req};
  const int64_t blocks = (rows + kPosThreads - 1) / kPosThreads;
  if (parent) {
    const int fill = (int)(blocks < 16 ? blocks : 16);
    W12_CUDA_TRY(launch_dependent(k_tree_positions, dim3((unsigned)(n_req + fill)), kPosThreads, 0, (cudaStream_t)stream, a));
  } else {
    const int64_t fewer = (blocks + kChainRows - 1) / kChainRows;
    W12_CUDA_TRY(launch_dependent(k_chain_positions, dim3((unsigned)(fewer < 152 * 8 ? fewer : 152 * 8)), kPosThreads, 0,
                                  (cudaStream_t)stream, a));
  }
  W12_LAUNCH_CHECK("tree_positions kernel");
  return W12_OK;
}

int qkv_rope(const void* x, int32_t x_bf16, int64_t x_stride, int64_t M, const qkv_form* form, const int32_t* pos, uint16_t* q,
             int64_t q_stride, uint16_t* k, int64_t k_stride, uint16_t* v, int64_t v_stride, void* stream) {
  RopeArgs a{};
  const int st = rope_args(a, "qkv_rope", x, x_bf16, x_stride, M, form, pos, q, q_stride, k, k_stride, v, v_stride);
  if (st) return st;
  if (!q || !k || !v) return fail(W12_ERR_INVALID_ARG, "qkv_rope: null pointer");
  return launch_rope(a, x_bf16, form->interleaved, (cudaStream_t)stream, "qkv_rope kernel");
}

int kv_append(const void* x, int32_t x_bf16, int64_t x_stride, int64_t M, const qkv_form* form, const int32_t* pos,
              const kv_cache* cache, int64_t layer, const int64_t* slot, uint16_t* q, int64_t q_stride, uint16_t* k,
              int64_t k_stride, uint16_t* v, int64_t v_stride, int32_t* status, void* stream) {
  RopeArgs a{};
  int st = check_cache(cache, "kv_append");
  if (st) return st;
  st = rope_args(a, "kv_append", x, x_bf16, x_stride, M, form, pos, q, q_stride, k, k_stride, v, v_stride);
  if (st) return st;
  if (!slot || !status) return fail(W12_ERR_INVALID_ARG, "kv_append: null pointer");
  if (cache->n_heads != form->n_heads || cache->head_dim != form->head_dim)
    return fail(W12_ERR_SHAPE, "kv_append: a cache of %d heads of %d for rows with %d of %d", cache->n_heads, cache->head_dim,
                form->n_heads, form->head_dim);
  if (layer < 0 || layer >= cache->n_layers)
    return fail(W12_ERR_SHAPE, "kv_append: layer %lld of %lld", (long long)layer, (long long)cache->n_layers);
  // Rows, slots and the form's arrays stand outside the cache, and the status outside them all.
  const uintptr_t span = 2 * (uintptr_t)((cache->n_layers - 1) * cache->layer_stride + (cache->n_blocks - 1) * cache->block_stride +
                                         (cache->block_size - 1) * cache->token_stride +
                                         (cache->n_heads - 1) * cache->head_stride + cache->head_dim);
  struct Range {
    const void* p;
    int64_t bytes;
  };
  const int64_t nk = form->n_heads * (int64_t)form->head_dim, nq = form->n_q_heads * (int64_t)form->head_dim;
  const Range used[] = {{x, ((M - 1) * x_stride + nq + 2 * nk) * (x_bf16 ? 2 : 4)},
                        {q, ((M - 1) * q_stride + nq) * 2},
                        {k, ((M - 1) * k_stride + nk) * 2},
                        {v, ((M - 1) * v_stride + nk) * 2},
                        {pos, M * 4},
                        {slot, M * 8},
                        {form->q_norm, form->head_dim * 4},
                        {form->k_norm, form->head_dim * 4},
                        {form->rot_dim ? form->inv_freq : nullptr, form->rot_dim * 2},
                        {status, 4}};
  for (const Range& u : used)
    for (const uint16_t* c : {cache->k, cache->v})
      if (u.p && (uintptr_t)u.p < (uintptr_t)c + span && (uintptr_t)c < (uintptr_t)u.p + (uintptr_t)u.bytes)
        return fail(W12_ERR_INVALID_ARG, "kv_append: the cache must not overlap the call's other arrays");
  for (const Range& u : used)
    if (u.p && &u != std::end(used) - 1 && (uintptr_t)u.p < (uintptr_t)status + 4 &&
        (uintptr_t)status < (uintptr_t)u.p + (uintptr_t)u.bytes)
      return fail(W12_ERR_INVALID_ARG, "kv_append: status must not overlap the call's other arrays");
  for (int i = 1; i < 4; ++i)
    if (used[i].p && (uintptr_t)used[i].p < (uintptr_t)slot + (uintptr_t)M * 8 &&
        (uintptr_t)slot < (uintptr_t)used[i].p + (uintptr_t)used[i].bytes)
      return fail(W12_ERR_INVALID_ARG, "kv_append: q, k and v must not overlap the slots");
  a.cache[0] = cache->k + layer * cache->layer_stride;
  a.cache[1] = cache->v + layer * cache->layer_stride;
  a.block_stride = cache->block_stride;
  a.token_stride = cache->token_stride;
  a.head_stride = cache->head_stride;
  a.n_slots = cache->n_blocks * cache->block_size;
  a.block_size = cache->block_size;
  a.slot = slot;
  a.status = status;
  return launch_rope(a, x_bf16, form->interleaved, (cudaStream_t)stream, "kv_append kernel");
}

}  // extern "C"
