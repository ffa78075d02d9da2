// w12_sample.cu - acceptance of draft trees against the target's probabilities, from given random
// numbers: the text that comes out is distributed as if the target had been sampled token by token.
//
// At a node let p be the softmax of its logits over the temperature and q the drafter's probabilities, from
// which the children were drawn without replacement.  A child with token x is taken if
// u q_j(x) < p_j(x), where q_j is q off the refused tokens, divided by Q_j = 1 - sum of their q; a refusal
// leaves p_{j+1} = max(p_j - q_j, 0) / its sum.  Clamped subtractions of multiples of one q add
// up, so with e = 2^(log2(e) (l - max) / T), S its sum over the vocabulary and tau_0 = 0, M_0 = S,
//     p_j = max(e - tau_j q, 0) / M_j,   tau_{j+1} = tau_j + M_j / Q_j,   M_{j+1} = sum max(e - tau_{j+1} q, 0):
// a refusal costs one sum over the vocabulary, no row is ever stored, and the bonus token comes from the
// masses max(e - tau q, 0) of the last sum.  Without q, q is 1 at the child's own token.
//
// The bonus is the first token whose cumulative mass passes u M.  For large vocabularies the borders between
// tokens stand 2^-20 of the mass apart and closer, so the masses have to be good to far more than a float:
// each is a pair of floats (2^-28 of its value, from the exponent's 48-bit product on), summed without loss, and the
// sums meet in 64 bits.  (With plain floats one token in some hundreds would differ from the formula's.)
#include <cstdint>

#include "w12_internal.cuh"
#include "w12_pdl.cuh"

namespace w12 {
namespace {

constexpr int kSampleMaxNodes = 1024;  // nodes of one request
constexpr int kUnit = 1024;            // tokens of a row that a warp sums at once
constexpr int kStatThreads = 256;
constexpr int kWalkThreads = 512;
constexpr int kWalkWarps = kWalkThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int32_t kSampleBadRequest = 1;
constexpr float kGreedy = 1e-5f;       // temperatures below are the limit at zero

struct SampleArgs {
  const float *logits, *probs;
  int64_t stride, probs_stride, M, V;
  const int32_t *parent, *draft, *req_offsets;
  const float *u, *u_bonus, *temperature;
  int32_t *path_len, *path_nodes, *bonus, *status;
  struct UnitStat* stat;  // [M][units], of rows with children
  int64_t range;          // tokens of a warp in the walk, a multiple of 128
  int32_t n_req, units, parts;
  bool vec, probs_vec;    // rows allow 16-byte loads
};

struct UnitStat {
  float most;   // largest logit (-inf: none, NaN left out)
  int32_t at;   // its first token, of greedy requests
  double sum;   // of the masses, in units of 2^Ref::log of the largest
};

__device__ __forceinline__ bool sample_request(const SampleArgs& a, int r, int64_t& off, int& n) {
  off = a.req_offsets ? a.req_offsets[r] : 0;
  const int64_t end = a.req_offsets ? a.req_offsets[r + 1] : a.M;
  if (off < 0 || end < off || end > a.M || end - off > kSampleMaxNodes) return false;
  n = (int)(end - off);
  return true;
}

// ---------------------------------------------------------------- pairs of floats

__device__ __forceinline__ uint64_t both(float x) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %1};" : "=l"(d) : "f"(x));
  return d;
}
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 split2(uint64_t x) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(x));
  return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) { return fma2(b, both(-1.0f), a); }

// s + t = a + b exactly (no order of sizes needed)
__device__ __forceinline__ void two_sum(uint64_t a, uint64_t b, uint64_t& s, uint64_t& t) {
  s = add2(a, b);
  const uint64_t v = sub2(s, a);
  t = add2(sub2(a, sub2(s, v)), sub2(b, v));
}

// ---------------------------------------------------------------- masses

// What the masses of a row, or of a part of it, are measured in: 2^log, near the mass of the largest logit
// `most`.  Its exponent most * c is rounded to a whole number, so that rows' parts differ by powers of two
// alone; where it is past 2^21 (a tiny temperature), the float product would keep no fraction, and the logits
// are taken relative to `most` instead, which is exact for those that still have a mass.
struct Ref {
  float most, shift, whole;
  double log;
};

__device__ __forceinline__ Ref make_ref(float most, double c) {
  Ref r{most, 0.0f, 0.0f, 0.0};
  if (most == INFINITY || most == -INFINITY) {
    r.log = most;
  } else if (fabs(most * c) >= 2097152.0) {
    r.shift = most;
    r.log = most * c;
  } else {
    r.whole = rintf((float)(most * c));
    r.log = r.whole;
  }
  return r;
}

__device__ __forceinline__ double rescale(double from, double to) { return from == to ? 1.0 : exp2(from - to); }

// log2(e) / T as a pair of floats.
struct Slope {
  double c;
  float hi, lo;
};

__device__ __forceinline__ Slope make_slope(float T) {
  Slope s;
  s.c = 1.4426950408889634074 / (double)T;
  s.hi = (float)s.c;
  s.lo = (float)(s.c - (double)s.hi);
  return s;
}

// The masses of two logits, h + lo each: 2^(x - whole), x = (l - shift) c.  With n whole and |g| <= 1/2 (and
// a little) 2^x = 2^n 2^g, 2^g = 1 + g ln 2 + g^2 (Taylor's terms to the eighth; 2^-32 is left out), whose first
// two terms are pairs of floats.  Below 2^-125 (and for -inf and NaN) a mass is 0.
__device__ __forceinline__ void mass2(uint64_t l, const Ref& r, const Slope& c, uint64_t& h, uint64_t& lo) {
  constexpr float kLn2 = 0.6931471824645996f, kLn2Rest = -1.904654299957768e-9f;
  const float2 lf = split2(l);
  l = add2(l, both(-r.shift));
  const uint64_t p = mul2(l, both(c.hi));
  const uint64_t npl = fma2(l, both(-c.lo), fma2(l, both(-c.hi), p));  // minus the product's rest
  const float2 pf = split2(p);
  const float least = r.whole - 125.0f;
  const uint64_t q = pair2(fmaxf(pf.x, least), fmaxf(pf.y, least));
  const uint64_t magic = both(12582912.0f);  // 1.5 * 2^23: the sum's low bits are the rounded exponent
  const uint64_t t = add2(q, magic), f = sub2(q, sub2(t, magic));
  const uint64_t g = sub2(f, npl), gl = sub2(sub2(f, g), npl);
  uint64_t w = both(1.321548679014431e-6f);
  w = fma2(w, g, both(1.5252733804059841e-5f));
  w = fma2(w, g, both(1.540353039338161e-4f));
  w = fma2(w, g, both(1.3333558146428443e-3f));
  w = fma2(w, g, both(9.618129107628477e-3f));
  w = fma2(w, g, both(5.550410866482158e-2f));
  w = fma2(w, g, both(2.4022650695910072e-1f));
  w = mul2(w, mul2(g, g));
  const uint64_t tt = mul2(g, both(kLn2));
  const uint64_t ntl = fma2(gl, both(-kLn2), fma2(g, both(-kLn2Rest), fma2(g, both(-kLn2), tt)));
  const uint64_t s = add2(tt, w), sl = sub2(add2(sub2(tt, s), w), ntl);
  const uint64_t e = add2(both(1.0f), s), el = add2(add2(sub2(both(1.0f), e), s), sl);
  const float2 tf = split2(t);
  const uint32_t base = (127u - (uint32_t)(int32_t)r.whole - 0x4B400000u) << 23;  // 2^(n - whole) as a float
  const uint64_t two = pair2(__uint_as_float((__float_as_uint(tf.x) << 23) + base), __uint_as_float((__float_as_uint(tf.y) << 23) + base));
  const float2 hf = split2(mul2(e, two)), gf = split2(mul2(el, two));
  const bool x = pf.x > least, y = pf.y > least;
  h = pair2(x ? hf.x : 0.0f, y ? hf.y : 0.0f);
  lo = pair2(x ? gf.x : 0.0f, y ? gf.y : 0.0f);
  if (r.most == INFINITY) {  // the infinite ones alone, alike
    h = pair2(lf.x == INFINITY ? 1.0f : 0.0f, lf.y == INFINITY ? 1.0f : 0.0f);
    lo = both(0.0f);
  }
}

// One mass in 64 bits.
__device__ __forceinline__ double mass1(float l, const Ref& r, const Slope& c) {
  if (r.most == INFINITY) return l == INFINITY ? 1.0 : 0.0;
  return l > -INFINITY ? exp2(((double)l - (double)r.shift) * c.c - (double)r.whole) : 0.0;
}

// What a refusal leaves of a mass, max(e - tau q, 0), for two tokens.
__device__ __forceinline__ void left2(uint64_t& h, uint64_t& lo, uint64_t q, float tau_hi, float tau_lo) {
  const uint64_t p = mul2(q, both(-tau_hi)), rest = fma2(q, both(tau_hi), p);  // tau_hi q = rest - p
  uint64_t s, t;
  two_sum(h, p, s, t);
  t = add2(t, fma2(q, both(-tau_lo), sub2(lo, rest)));
  const float2 sf = split2(s), tf = split2(t);
  const bool x = sf.x + tf.x > 0.0f, y = sf.y + tf.y > 0.0f;
  h = pair2(x ? sf.x : 0.0f, y ? sf.y : 0.0f);
  lo = pair2(x ? tf.x : 0.0f, y ? tf.y : 0.0f);
}

// A running sum of pairs without loss but in its last part, two at a time.
struct Sum {
  uint64_t s = 0, rest = 0;
  __device__ __forceinline__ void add(uint64_t h, uint64_t lo) {
    uint64_t n, t;
    two_sum(s, h, n, t);
    s = n;
    rest = add2(rest, add2(t, lo));
  }
  __device__ __forceinline__ double value() const {
    const float2 a = split2(s), b = split2(rest);
    return ((double)a.x + (double)a.y) + ((double)b.x + (double)b.y);
  }
};

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
  return x;
}

// Four tokens from i on, `fill` behind the end.
__device__ __forceinline__ float4 four(const float* x, int64_t i, int64_t end, bool vec, float fill) {
  if (vec && i + 4 <= end) return *reinterpret_cast<const float4*>(x + i);
  float4 f = make_float4(fill, fill, fill, fill);
  if (i < end) f.x = x[i];
  if (i + 1 < end) f.y = x[i + 1];
  if (i + 2 < end) f.z = x[i + 2];
  if (i + 3 < end) f.w = x[i + 3];
  return f;
}

// The first place of `most` among a float4 of tokens from i on (least: none).
__device__ __forceinline__ void first_at(const float4& f, int64_t i, float most, int32_t& at) {
  const int k = f.x == most ? 0 : f.y == most ? 1 : f.z == most ? 2 : f.w == most ? 3 : 4;
  if (k < 4 && (int32_t)i + k < at) at = (int32_t)i + k;
}

// ---------------------------------------------------------------- rows with children

// Largest logit and mass of every 1024 tokens of the rows whose nodes have children (what the walk asks of a
// node it passes), a warp each, all 128 bytes a lane on their way at once.  Bound by the logits read once.
__global__ void __launch_bounds__(kStatThreads) k_sample_stats(const __grid_constant__ SampleArgs a) {
  pdl_enter();
  __shared__ uint32_t inner[kSampleMaxNodes / 32];
  const int r = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  const int unit = blockIdx.x * (kStatThreads / 32) + (tid >> 5);
  int64_t off;
  int n;
  if (!sample_request(a, r, off, n) || n < 2) return;
  if (tid < kSampleMaxNodes / 32) inner[tid] = 0;
  __syncthreads();
  for (int i = 1 + tid; i < n; i += kStatThreads) {
    const int32_t p = a.parent[off + i];
    if (p >= 0 && p < i) atomicOr(&inner[p >> 5], 1u << (p & 31));
  }
  __syncthreads();
  if (unit >= a.units) return;
  const float T = a.temperature ? a.temperature[r] : 1.0f;
  const bool greedy = T < kGreedy;
  const Slope c = make_slope(greedy ? 1.0f : T);
  const int64_t v0 = (int64_t)unit * kUnit, v1 = min(a.V, v0 + kUnit);
  int nth = 0;
  for (int w = 0; w * 32 < n; ++w)
    for (uint32_t m = inner[w]; m; m &= m - 1) {
      if (nth++ % a.parts != (int)blockIdx.z) continue;
      const int64_t row = off + w * 32 + __ffs((int)m) - 1;
      const float* x = a.logits + row * a.stride;
      float4 f[kUnit / 128];
#pragma unroll
      for (int k = 0; k < kUnit / 128; ++k) f[k] = four(x, v0 + k * 128 + 4 * lane, v1, a.vec, -INFINITY);
      float most = -INFINITY;
#pragma unroll
      for (int k = 0; k < kUnit / 128; ++k) most = fmaxf(most, fmaxf(fmaxf(f[k].x, f[k].y), fmaxf(f[k].z, f[k].w)));
      most = warp_max(most);
      UnitStat st{most, -1, 0.0};
      if (most > -INFINITY) {
        if (greedy) {
          int32_t at = 0x7FFFFFFF;
#pragma unroll
          for (int k = 0; k < kUnit / 128; ++k) first_at(f[k], v0 + k * 128 + 4 * lane, most, at);
          st.at = __reduce_min_sync(0xFFFFFFFFu, at);
          st.sum = 1.0;
        } else {
          const Ref ref = make_ref(most, c.c);
          Sum sum;
#pragma unroll
          for (int k = 0; k < kUnit / 128; ++k) {
            uint64_t h, lo;
            mass2(pair2(f[k].x, f[k].y), ref, c, h, lo);
            sum.add(h, lo);
            mass2(pair2(f[k].z, f[k].w), ref, c, h, lo);
            sum.add(h, lo);
          }
          st.sum = warp_sum(sum.value());
        }
      }
      if (lane == 0) a.stat[row * a.units + unit] = st;
    }
}

// ---------------------------------------------------------------- the walk

// What the first block of a cluster has all its blocks do next.
enum : int32_t { kOpDone, kOpSum, kOpFind };

struct Command {
  int32_t op;
  int32_t node;          // of the request
  int32_t known;         // kOpSum: `most` is the row's; else every warp finds its range's
  int32_t residual;      // tau q is taken off
  int32_t refused;       // the node's children are taken out (no q)
  int32_t owner;         // kOpFind: the block that holds the bonus token
  float most, tau_hi, tau_lo;
  double log, target;    // kOpFind: the mass before the bonus token in the owner's ranges, in units of 2^log
};

struct Total {
  float most;
  int32_t at;
  double log, sum;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  cluster_arrive();
  cluster_wait();
}

// 4-byte words of `from` (this block's shared memory) to the same place in block `rank` of the cluster.
template <typename S>
__device__ __forceinline__ void send(const S& from, S* to, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(to)), "r"(rank));
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&from);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(S) / 4); ++i)
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at + 4 * i), "r"(w[i]) : "memory");
}

struct WalkShared {
  int32_t parent[kSampleMaxNodes], draft[kSampleMaxNodes], refused[kSampleMaxNodes];
  float u[kSampleMaxNodes], l[kSampleMaxNodes], q[kSampleMaxNodes];  // of a node: its number, its token's logit and q at the parent
  float most[kSampleMaxNodes];                                       // of rows with children
  int32_t at[kSampleMaxNodes];
  double sum[kSampleMaxNodes];
  uint32_t inner[kSampleMaxNodes / 32];
  Command cmd;
  Total total[kMaxCluster];
  double warp_log[kWalkWarps], warp_sum[kWalkWarps], group[kWalkWarps];
  float warp_most[kWalkWarps];
  int32_t warp_at[kWalkWarps], n_refused, last;
};

// The masses of four tokens from i on.
struct Four {
  uint64_t h[2], lo[2];
};

__device__ __forceinline__ Four masses4(const float4& f, const float4& q, int64_t i, const Ref& ref, const Slope& c,
                                        const Command& cmd, const int32_t* refused, int n_refused) {
  Four m;
  mass2(pair2(f.x, f.y), ref, c, m.h[0], m.lo[0]);
  mass2(pair2(f.z, f.w), ref, c, m.h[1], m.lo[1]);
  if (cmd.residual) {
    left2(m.h[0], m.lo[0], pair2(q.x, q.y), cmd.tau_hi, cmd.tau_lo);
    left2(m.h[1], m.lo[1], pair2(q.z, q.w), cmd.tau_hi, cmd.tau_lo);
  }
  for (int k = 0; k < n_refused; ++k) {
    const int64_t at = refused[k] - i;
    if (at >= 0 && at < 4) {
      const uint64_t keep = at & 1 ? 0x00000000FFFFFFFFull : 0xFFFFFFFF00000000ull;
      m.h[at >> 1] &= keep;
      m.lo[at >> 1] &= keep;
    }
  }
  return m;
}

__device__ __forceinline__ float chance(float q) { return fminf(fmaxf(q, 0.0f), 1.0f); }  // (NaN: 0)

__device__ __forceinline__ float4 chance4(float4 q) { return make_float4(chance(q.x), chance(q.y), chance(q.z), chance(q.w)); }

// One warp's range of one row: its sum in units of 2^log, or its first largest token (greedy).
__device__ __forceinline__ void sum_range(const SampleArgs& a, const Command& cmd, const Slope& c, bool greedy, int64_t row,
                                          int64_t v0, int64_t v1, const int32_t* refused, int n_refused, float& most_out,
                                          int32_t& at_out, double& log_out, double& sum_out) {
  const int lane = threadIdx.x & 31;
  const float* x = a.logits + row * a.stride;
  const float* p = a.probs ? a.probs + row * a.probs_stride : nullptr;
  constexpr int U = 4;
  float most = cmd.most;
  if (!cmd.known) {
    most = -INFINITY;
    for (int64_t i0 = v0; i0 < v1; i0 += 128 * U) {
      float4 f[U];
#pragma unroll
      for (int k = 0; k < U; ++k) f[k] = four(x, i0 + k * 128 + 4 * lane, v1, a.vec, -INFINITY);
#pragma unroll
      for (int k = 0; k < U; ++k) most = fmaxf(most, fmaxf(fmaxf(f[k].x, f[k].y), fmaxf(f[k].z, f[k].w)));
    }
    most = warp_max(most);
  }
  most_out = most;
  at_out = 0x7FFFFFFF;
  log_out = -INFINITY;
  sum_out = 0.0;
  if (most == -INFINITY) return;
  if (greedy) {
    int32_t at = 0x7FFFFFFF;
    for (int64_t i = v0 + 4 * lane; i < v1 && at == 0x7FFFFFFF; i += 128) first_at(four(x, i, v1, a.vec, -INFINITY), i, most, at);
    at_out = __reduce_min_sync(0xFFFFFFFFu, at);
    return;
  }
  const Ref ref = make_ref(most, c.c);
  Sum sum;
  for (int64_t i0 = v0; i0 < v1; i0 += 128 * U) {
    float4 f[U], q[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      f[k] = four(x, i0 + k * 128 + 4 * lane, v1, a.vec, -INFINITY);
      q[k] = cmd.residual ? four(p, i0 + k * 128 + 4 * lane, v1, a.probs_vec, 0.0f) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const Four m = masses4(f[k], chance4(q[k]), i0 + k * 128 + 4 * lane, ref, c, cmd, refused, n_refused);
      sum.add(m.h[0], m.lo[0]);
      sum.add(m.h[1], m.lo[1]);
    }
  }
  log_out = ref.log;
  sum_out = warp_sum(sum.value());
}

// The bonus token, by the block that holds it: first the warp's range, then 128 tokens, then the token.  The
// sums of ranges, groups and lanes are rounded differently; where the last tokens do not pass the
// target by that, it is the last one with a mass.
__device__ __forceinline__ void find_token(const SampleArgs& a, WalkShared& s, const Slope& c, int64_t row, int64_t first,
                                           int32_t* bonus) {
  const Command& cmd = s.cmd;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  double before = 0.0, seen = 0.0;
  int range = 0;
  for (int w = 0; w < kWalkWarps; ++w) {
    const double m = s.warp_sum[w] > 0.0 ? s.warp_sum[w] * rescale(s.warp_log[w], cmd.log) : 0.0;
    if (!(m > 0.0)) continue;
    range = w;
    before = seen;
    seen += m;
    if (seen > cmd.target) break;
  }
  const double target = (cmd.target - before) * rescale(cmd.log, s.warp_log[range]);
  const Ref ref = make_ref(s.warp_most[range], c.c);
  const int64_t v0 = first + range * a.range, v1 = min(a.V, v0 + a.range);
  const float* x = a.logits + row * a.stride;
  const float* p = a.probs ? a.probs + row * a.probs_stride : nullptr;
  const int n_refused = cmd.refused ? s.n_refused : 0;
  if (tid == 0) s.last = -1;
  double run = 0.0;
  for (int64_t base = v0; base < v1; base += 128 * kWalkWarps) {
    const int64_t i = base + warp * 128 + 4 * lane;
    const float4 q = cmd.residual ? four(p, i, v1, a.probs_vec, 0.0f) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const Four f = masses4(four(x, i, v1, a.vec, -INFINITY), chance4(q), i, ref, c, cmd, s.refused, n_refused);
    double m[4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float2 h = split2(f.h[k]), lo = split2(f.lo[k]);
      m[2 * k] = (double)h.x + (double)lo.x;
      m[2 * k + 1] = (double)h.y + (double)lo.y;
    }
    const double mine = (m[0] + m[1]) + (m[2] + m[3]);
    double upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double t = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += t;
    }
    if (lane == 31) s.group[warp] = upto;
    __syncthreads();
    int hit = -1;
    for (int g = 0; g < kWalkWarps; ++g) {
      const double m_g = s.group[g];
      if (m_g > 0.0 && run + m_g > target) {
        hit = g;
        break;
      }
      run += m_g;
    }
    int last = -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) last = m[k] > 0.0 ? k : last;
    if (hit == warp) {
      double at = run + (upto - mine);
      int found = 4;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        at += m[k];
        if (found == 4 && m[k] > 0.0 && at > target) found = k;
      }
      const uint32_t passed = __ballot_sync(0xFFFFFFFFu, found < 4), some = __ballot_sync(0xFFFFFFFFu, last >= 0);
      if (passed ? lane == __ffs((int)passed) - 1 : some && lane == 31 - __clz((int)some))
        *bonus = (int32_t)i + (passed ? found : last);
    }
    if (hit >= 0) return;
    if (last >= 0) atomicMax(&s.last, (int32_t)i + last);
    __syncthreads();
  }
  if (tid == 0) *bonus = s.last;
}

// A cluster takes a request.  Its first block walks the tree (warp 0, all lanes alike) and has all blocks sum a
// row's masses, a range of tokens a warp, where a refusal or the bonus token asks for it; only that
// block decides what comes next, and the others do as they are told.
__global__ void __launch_bounds__(kWalkThreads) k_sample_walk(const __grid_constant__ SampleArgs a, int cluster) {
  __shared__ WalkShared s;
  cluster_arrive();  // a block's shared memory is written to only when the block runs
  pdl_enter();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  const int r = blockIdx.x / cluster;
  const int64_t first = (int64_t)rank * kWalkWarps * a.range;  // the block's tokens
  int64_t off;
  int n;
  bool ok = sample_request(a, r, off, n);
  if (!ok) n = 0;
  const float T = a.temperature ? a.temperature[r] : 1.0f;
  const bool greedy = T < kGreedy;
  const Slope c = make_slope(greedy ? 1.0f : T);

  // ---- the nodes, and the sums of the rows with children
  if (rank == 0) {
    if (tid < kSampleMaxNodes / 32) s.inner[tid] = 0;
    __syncthreads();
    ok = ok && T >= 0.0f;
    for (int i = tid; i < n; i += kWalkThreads) {
      const int32_t p = a.parent[off + i], x = a.draft[off + i];
      const bool fine = i == 0 ? p == -1 : p >= 0 && p < i;
      ok = ok && fine;
      s.parent[i] = p;
      s.draft[i] = i > 0 && x >= 0 && x < a.V ? x : -1;
      s.u[i] = fminf(fmaxf(a.u[off + i], 0.0f), 0.99999994f);
      a.path_nodes[off + i] = -1;
      if (i > 0 && fine) {
        atomicOr(&s.inner[p >> 5], 1u << (p & 31));
        s.l[i] = s.draft[i] >= 0 ? a.logits[(off + p) * a.stride + x] : 0.0f;
        s.q[i] = s.draft[i] >= 0 && a.probs ? chance(a.probs[(off + p) * a.probs_stride + x]) : 0.0f;
      }
    }
    ok = __syncthreads_and(ok);
    if (!ok && tid == 0) atomicOr(a.status, kSampleBadRequest);
    ok = ok && n > 0;
    if (!ok && tid == 0) a.path_len[r] = a.bonus[r] = -1;
    for (int i = warp; ok && i < n; i += kWalkWarps) {
      if (!(s.inner[i >> 5] >> (i & 31) & 1u)) continue;
      const UnitStat* st = a.stat + (off + i) * a.units;
      float most = -INFINITY;
      int32_t at = 0x7FFFFFFF;
      double log = -INFINITY, sum = 0.0;
      for (int k = lane; k < a.units; k += 32) {
        const UnitStat u = st[k];
        if (u.most == -INFINITY) continue;
        if (u.most > most || (u.most == most && u.at < at)) at = u.at;
        most = fmaxf(most, u.most);
        const double l = make_ref(u.most, c.c).log, top = fmax(l, log);
        sum = sum * rescale(log, top) + u.sum * rescale(l, top);
        log = top;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const float m = __shfl_xor_sync(0xFFFFFFFFu, most, o);
        const int32_t t = __shfl_xor_sync(0xFFFFFFFFu, at, o);
        if (m > most || (m == most && t < at)) at = t;
        most = fmaxf(most, m);
        const double l = __shfl_xor_sync(0xFFFFFFFFu, log, o), u = __shfl_xor_sync(0xFFFFFFFFu, sum, o), top = fmax(l, log);
        sum = sum * rescale(log, top) + u * rescale(l, top);
        log = top;
      }
      if (lane == 0) {
        s.most[i] = most;
        s.at[i] = at;
        s.sum[i] = sum;
      }
    }
    __syncthreads();
  }

  // ---- the walk's state (first block, warp 0)
  enum { kWalk, kRefused, kSummed } stage = kWalk;
  int cur = 0, last = 0, depth = 0;
  bool inner = false, summed = false, spent = false, refused = false;
  double tau = 0.0, Q = 1.0, M = 0.0, log = 0.0;
  Command cmd{};
  const double u_bonus = fminf(fmaxf(a.u_bonus[r], 0.0f), 0.99999994f);
  auto enter = [&](int node) {
    cur = last = node;
    inner = s.inner[node >> 5] >> (node & 31) & 1u;
    summed = spent = refused = false;
    tau = 0.0;
    Q = 1.0;
    M = inner ? s.sum[node] : 0.0;
    log = inner ? make_ref(s.most[node], c.c).log : 0.0;
  };
  auto ask = [&](bool residual) {
    cmd.op = kOpSum;
    cmd.node = cur;
    cmd.known = inner;
    cmd.most = inner ? s.most[cur] : 0.0f;
    cmd.residual = residual;
    cmd.refused = refused && !residual;
    cmd.tau_hi = (float)tau;
    cmd.tau_lo = (float)(tau - (double)cmd.tau_hi);
  };
  if (rank == 0 && warp == 0 && ok) {
    enter(0);
    if (lane == 0) a.path_nodes[off] = 0;
  }

  __syncwarp();
  cluster_wait();
  while (true) {
    if (rank == 0 && warp == 0) {
      cmd.op = kOpDone;
      if (ok) {
        if (stage != kWalk && !greedy) {  // the blocks' sums
          log = -INFINITY;
          for (int k = 0; k < cluster; ++k) log = fmax(log, s.total[k].log);
          M = 0.0;
          for (int k = 0; k < cluster; ++k)
            if (s.total[k].sum > 0.0) M += s.total[k].sum * rescale(s.total[k].log, log);
        }
        bool ends = stage == kSummed, asked = false;
        if (stage == kRefused) {
          summed = true;
          if (!(M > 0.0)) {  // nothing is left: the bonus comes from p as it was
            spent = true;
            summed = false;
          }
        }
        while (!ends && !asked) {
          int j = -1;  // the next child
          for (int i0 = last + 1; i0 < n && j < 0; i0 += 32) {
            const uint32_t b = __ballot_sync(0xFFFFFFFFu, i0 + lane < n && s.parent[i0 + lane] == cur);
            if (b) j = i0 + __ffs((int)b) - 1;
          }
          if (j < 0) {
            ends = true;
            break;
          }
          last = j;
          const int32_t x = s.draft[j];
          if (x < 0) continue;
          bool take;
          if (greedy) {
            take = s.most[cur] > -INFINITY && x == s.at[cur];
          } else {
            if (spent || !(s.sum[cur] > 0.0)) continue;
            bool twice = false;  // a sibling with this token was refused before
            for (int i0 = cur + 1; i0 < j && !twice; i0 += 32)
              twice = __any_sync(0xFFFFFFFFu, i0 + lane < j && s.parent[i0 + lane] == cur && s.draft[i0 + lane] == x);
            if (twice) continue;
            const double e = mass1(s.l[j], make_ref(s.most[cur], c.c), c), u = s.u[j], q = s.q[j];
            take = a.probs ? Q > 0.0 && u * (q / Q) * M < e - tau * q : u * M < e;
            if (!take) {
              if (!a.probs) {
                refused = true;
                M = fmax(M - e, 0.0);
              } else if (q > 0.0 && Q > 0.0) {
                tau += M / Q;
                Q -= q;
                ask(true);
                stage = kRefused;
                asked = true;
              }
              continue;
            }
          }
          if (take) {
            ++depth;
            if (lane == 0) a.path_nodes[off + depth] = j;
            enter(j);
          }
        }
        if (ends) {
          if (lane == 0 && stage != kSummed) a.path_len[r] = depth;
          if (greedy) {
            if (inner || stage == kSummed) {
              float most = inner ? s.most[cur] : -INFINITY;
              int32_t at = inner ? s.at[cur] : -1;
              if (!inner)
                for (int k = 0; k < cluster; ++k)
                  if (s.total[k].most > most) {  // the blocks' tokens rise
                    most = s.total[k].most;
                    at = s.total[k].at;
                  }
              if (lane == 0) a.bonus[r] = most > -INFINITY ? at : -1;
              cmd.op = kOpDone;
            } else {
              ask(false);
              stage = kSummed;
            }
          } else if (stage != kSummed && !summed) {
            ask(false);
            stage = kSummed;
          } else if (!(M > 0.0)) {
            if (cmd.refused) {  // all that had a mass was refused: p as it was
              refused = false;
              ask(false);
            } else {
              if (lane == 0) a.bonus[r] = -1;
              cmd.op = kOpDone;
            }
          } else {
            cmd.op = kOpFind;
            cmd.log = log;
            const double target = u_bonus * M;
            double before = 0.0, seen = 0.0;
            for (int k = 0; k < cluster; ++k) {
              const double m = s.total[k].sum > 0.0 ? s.total[k].sum * rescale(s.total[k].log, log) : 0.0;
              if (!(m > 0.0)) continue;
              cmd.owner = k;
              before = seen;
              seen += m;
              if (seen > target) break;
            }
            cmd.target = target - before;
          }
        }
      }
      if (lane < cluster) send(cmd, &s.cmd, (uint32_t)lane);
    }
    cluster_sync();
    if (s.cmd.op == kOpDone) break;
    const int64_t row = off + s.cmd.node;
    if (s.cmd.op == kOpFind) {
      if (s.cmd.owner == (int32_t)rank) find_token(a, s, c, row, first, a.bonus + r);
      break;
    }
    if (s.cmd.refused) {
      if (tid == 0) s.n_refused = 0;
      __syncthreads();
      for (int i = s.cmd.node + 1 + tid; i < n; i += kWalkThreads) {
        const int32_t x = a.draft[off + i];
        if (a.parent[off + i] == s.cmd.node && x >= 0 && x < a.V) s.refused[atomicAdd(&s.n_refused, 1)] = x;
      }
      __syncthreads();
    }
    {
      const int64_t v0 = first + warp * a.range, v1 = min(a.V, v0 + a.range);
      float most;
      int32_t at;
      double wlog, wsum;
      sum_range(a, s.cmd, c, greedy, row, v0, v1, s.refused, s.cmd.refused ? s.n_refused : 0, most, at, wlog, wsum);
      if (lane == 0) {
        s.warp_most[warp] = most;
        s.warp_at[warp] = at;
        s.warp_log[warp] = wlog;
        s.warp_sum[warp] = wsum;
      }
    }
    __syncthreads();
    if (tid == 0) {
      Total t{-INFINITY, -1, -INFINITY, 0.0};
      for (int w = 0; w < kWalkWarps; ++w) {
        if (s.warp_most[w] > t.most) {
          t.most = s.warp_most[w];
          t.at = s.warp_at[w];
        }
        t.log = fmax(t.log, s.warp_log[w]);
      }
      for (int w = 0; w < kWalkWarps; ++w)
        if (s.warp_sum[w] > 0.0) t.sum += s.warp_sum[w] * rescale(s.warp_log[w], t.log);
      send(t, &s.total[rank], 0);
    }
    cluster_sync();
  }
}

// Blocks of a request's cluster: as many as fill the SMs, up to the eight that every device takes.
int cluster_size(int32_t n_req, int64_t V) {
  int c = 1;
  while (c < kMaxCluster && 2 * c * (int64_t)n_req <= 152 && V > (int64_t)c * 8192) c *= 2;
  return c;
}

}  // namespace
}  // namespace w12

using namespace w12;

extern "C" {

size_t tree_verify_sampled_workspace_size(int64_t M, int64_t V) {
  if (M < 1 || V < 1) return 0;
  return (size_t)M * (size_t)((V + kUnit - 1) / kUnit) * sizeof(UnitStat);
}

int tree_verify_sampled(const float* logits, int64_t stride, int64_t M, int64_t V, const float* draft_probs,
                        int64_t probs_stride, const int32_t* parent, const int32_t* draft, const int32_t* req_offsets,
                        int32_t n_req, const float* u, const float* u_bonus, const float* temperature, int32_t* path_len,
                        int32_t* path_nodes, int32_t* bonus, int32_t* status, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "tree_verify_sampled";
  if (M < 1 || M > 0x7FFFFFFF || V < 1 || V > 0x7FFFFFFF || stride < V || (draft_probs && probs_stride < V) || n_req < 1 ||
      n_req > 65535)
    return fail(W12_ERR_SHAPE, "%s: M=%lld, V=%lld (strides %lld, %lld), n_req=%d (1..65535) out of range", fn, (long long)M,
                (long long)V, (long long)stride, (long long)probs_stride, n_req);
  if (!logits || !parent || !draft || !u || !u_bonus || !path_len || !path_nodes || !bonus || !status || !ws)
    return fail(W12_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!req_offsets && n_req != 1)
    return fail(W12_ERR_INVALID_ARG, "%s: req_offsets is null but n_req=%d", fn, n_req);
  if ((uintptr_t)ws & 15u) return fail(W12_ERR_INVALID_ARG, "%s: the workspace must be 16-byte aligned", fn);
  if (ws_bytes < tree_verify_sampled_workspace_size(M, V))
    return fail(W12_ERR_BUFFER_TOO_SMALL, "%s: workspace %zu < %zu", fn, ws_bytes, tree_verify_sampled_workspace_size(M, V));
  struct Range {
    const void* p;
    uintptr_t bytes;
  };
  const Range out[] = {{path_len, (uintptr_t)n_req * 4}, {path_nodes, (uintptr_t)M * 4}, {bonus, (uintptr_t)n_req * 4},
                       {status, 4}, {ws, tree_verify_sampled_workspace_size(M, V)}};
  const Range used[] = {{logits, (uintptr_t)((M - 1) * stride + V) * 4},
                        {draft_probs, draft_probs ? (uintptr_t)((M - 1) * probs_stride + V) * 4 : 0},
                        {parent, (uintptr_t)M * 4}, {draft, (uintptr_t)M * 4}, {u, (uintptr_t)M * 4},
                        {u_bonus, (uintptr_t)n_req * 4}, {temperature, temperature ? (uintptr_t)n_req * 4 : 0},
                        {req_offsets, req_offsets ? (uintptr_t)(n_req + 1) * 4 : 0}};
  auto meet = [](const Range& x, const Range& y) {
    return x.bytes && y.bytes && (uintptr_t)x.p < (uintptr_t)y.p + y.bytes && (uintptr_t)y.p < (uintptr_t)x.p + x.bytes;
  };
  for (const Range& o : out) {
    bool bad = false;
    for (const Range& x : used) bad = bad || meet(o, x);
    for (const Range& x : out) bad = bad || (&x != &o && meet(o, x));
    if (bad) return fail(W12_ERR_INVALID_ARG, "%s: results must not overlap one another or what the call reads", fn);
  }
  const int cluster = cluster_size(n_req, V);
  SampleArgs a{};
  a.logits = logits;
  a.probs = draft_probs;
  a.stride = stride;
  a.probs_stride = probs_stride;
  a.M = M;
  a.V = V;
  a.parent = parent;
  a.draft = draft;
  a.req_offsets = req_offsets;
  a.u = u;
  a.u_bonus = u_bonus;
  a.temperature = temperature;
  a.path_len = path_len;
  a.path_nodes = path_nodes;
  a.bonus = bonus;
  a.status = status;
  a.stat = static_cast<UnitStat*>(ws);
  a.units = (int32_t)((V + kUnit - 1) / kUnit);
  const int64_t warps = (int64_t)cluster * kWalkWarps;
  a.range = ((V + warps - 1) / warps + 127) / 128 * 128;
  a.n_req = n_req;
  a.vec = (stride & 3) == 0 && ((uintptr_t)logits & 15u) == 0;
  a.probs_vec = draft_probs && (probs_stride & 3) == 0 && ((uintptr_t)draft_probs & 15u) == 0;
  if (M > 1) {
    const int per = kStatThreads / 32;
    const int64_t blocks = (a.units + per - 1) / per * (int64_t)n_req, rows = (M + n_req - 1) / n_req;
    // few requests: their rows over more blocks
    a.parts = (int32_t)(blocks * 2 > 912 ? 1 : rows < 912 / blocks ? rows : 912 / blocks);
    W12_CUDA_TRY(launch_dependent(k_sample_stats, dim3((unsigned)((a.units + per - 1) / per), (unsigned)n_req, (unsigned)a.parts),
                                  kStatThreads, 0, (cudaStream_t)stream, a));
    W12_LAUNCH_CHECK("tree_verify_sampled: rows kernel");
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(cluster * n_req));
  cfg.blockDim = dim3(kWalkThreads);
  cfg.stream = (cudaStream_t)stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  W12_CUDA_TRY(cudaLaunchKernelEx(&cfg, k_sample_walk, a, cluster));
  W12_LAUNCH_CHECK("tree_verify_sampled: walk kernel");
  return W12_OK;
}

}  // extern "C"
