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
// sums stay pairs of floats.  (With plain floats one token in some hundreds would differ from the formula's.)
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
  float most;    // largest logit (-inf: none, NaN left out)
  int32_t at;    // its first token, of greedy requests
  float sum[2];  // of the masses, in the units of the largest
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

// A sum as an unevaluated pair of floats, |l| at most half of h's last place.
struct Pair {
  float h, l;
};

__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  const float s = a.h + b.h, v = s - a.h, e = ((a.h - (s - v)) + (b.h - v)) + (a.l + b.l);
  const float h = s + e;
  return {h, e - (h - s)};
}
__device__ __forceinline__ Pair operator-(Pair a, Pair b) { return a + Pair{-b.h, -b.l}; }
__device__ __forceinline__ Pair operator*(Pair a, float x) {
  const float p = __fmul_rn(a.h, x), e = fmaf(a.l, x, fmaf(a.h, x, -p));
  const float h = p + e;
  return {h, e - (h - p)};
}
__device__ __forceinline__ bool operator>(Pair a, Pair b) { return a.h > b.h || (a.h == b.h && a.l > b.l); }
__device__ __forceinline__ double wide(Pair a) { return (double)a.h + (double)a.l; }

__device__ __forceinline__ Pair shuffle_xor(Pair a, int o) {
  return {__shfl_xor_sync(0xFFFFFFFFu, a.h, o), __shfl_xor_sync(0xFFFFFFFFu, a.l, o)};
}
__device__ __forceinline__ Pair shuffle(Pair a, int lane) {
  return {__shfl_sync(0xFFFFFFFFu, a.h, lane), __shfl_sync(0xFFFFFFFFu, a.l, lane)};
}

__device__ __forceinline__ Pair warp_sum(Pair a) {
#pragma unroll
  for (int o = 16; o; o >>= 1) a = a + shuffle_xor(a, o);
  return a;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
  return x;
}

// The first lane at which the sum of the lanes' masses from lane 0 on passes the target, and the sum before it;
// where none does, the last lane with a mass (or -1) and passed = false.
struct Found {
  int lane;
  bool passed;
  Pair before, all;
};

__device__ __forceinline__ Found find_lane(Pair mine, Pair target) {
  const int lane = threadIdx.x & 31;
  Pair upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair t{__shfl_up_sync(0xFFFFFFFFu, upto.h, o), __shfl_up_sync(0xFFFFFFFFu, upto.l, o)};
    if (lane >= o) upto = t + upto;
  }
  const uint32_t some = __ballot_sync(0xFFFFFFFFu, mine.h > 0.0f);
  const uint32_t over = __ballot_sync(0xFFFFFFFFu, mine.h > 0.0f && upto > target);
  Found f;
  f.passed = over != 0;
  f.lane = over ? __ffs((int)over) - 1 : 31 - __clz((int)some);
  f.all = shuffle(upto, 31);
  f.before = f.lane > 0 ? shuffle(upto, f.lane - 1) : Pair{0.0f, 0.0f};
  return f;
}

// ---------------------------------------------------------------- masses

// log2(e) / T as a pair of floats.
struct Slope {
  float hi, lo;
};

__device__ __forceinline__ Slope make_slope(float T) {
  const double c = 1.4426950408889634074 / (double)T;
  Slope s;
  s.hi = (float)c;
  s.lo = (float)(c - (double)s.hi);
  return s;
}

// What the masses of a row, or of a part of it, are measured in: about the mass of its largest logit
// `most`.  The exponent most * c is rounded to a whole number, so that parts of rows differ by powers of two
// alone; where it is past 2^21 (a tiny temperature), the float product would keep no fraction, and the logits
// are taken relative to `most` instead, which is exact for those that still have a mass.
struct Ref {
  float most, shift, whole;
};

__device__ __forceinline__ Ref make_ref(float most, const Slope& c) {
  const float x = most * c.hi;
  const bool far = fabsf(x) >= 2097152.0f && fabsf(most) < INFINITY;
  return Ref{most, far ? most : 0.0f, far ? 0.0f : fabsf(most) == INFINITY ? most : rintf(x)};
}

__device__ __noinline__ float far_scale(Ref from, Ref to, Slope c) {
  const double k = (double)c.hi + (double)c.lo;
  const double a = from.shift != 0.0f ? (double)from.shift * k : (double)from.whole;
  const double b = to.shift != 0.0f ? (double)to.shift * k : (double)to.whole;
  return (float)exp2(a - b);
}

// One unit of `from` in units of `to`.
__device__ __forceinline__ float scale_of(const Ref& from, const Ref& to, const Slope& c) {
  if (from.most == to.most) return 1.0f;
  if (from.shift != 0.0f || to.shift != 0.0f) return far_scale(from, to, c);
  const float k = from.whole - to.whole;
  return k >= -126.0f ? __int_as_float((127 + (int)fminf(k, 127.0f)) << 23) : 0.0f;
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
  __device__ __forceinline__ Pair value() const {
    const float2 a = split2(s), b = split2(rest);
    return Pair{a.x, b.x} + Pair{a.y, b.y};
  }
};

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
      UnitStat st{most, -1, {0.0f, 0.0f}};
      if (most > -INFINITY) {
        if (greedy) {
          int32_t at = 0x7FFFFFFF;
#pragma unroll
          for (int k = 0; k < kUnit / 128; ++k) first_at(f[k], v0 + k * 128 + 4 * lane, most, at);
          st.at = __reduce_min_sync(0xFFFFFFFFu, at);
        } else {
          const Ref ref = make_ref(most, c);
          Sum sum;
#pragma unroll
          for (int k = 0; k < kUnit / 128; ++k) {
            uint64_t h, lo;
            mass2(pair2(f[k].x, f[k].y), ref, c, h, lo);
            sum.add(h, lo);
            mass2(pair2(f[k].z, f[k].w), ref, c, h, lo);
            sum.add(h, lo);
          }
          const Pair all = warp_sum(sum.value());
          st.sum[0] = all.h;
          st.sum[1] = all.l;
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
  Pair target;           // kOpFind: the mass before the bonus token in the owner's ranges, in the units of `most`
};

struct Total {
  float most;
  int32_t at;
  Pair sum;
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
  float u[kSampleMaxNodes], q[kSampleMaxNodes];  // of a node: its number, and q of its token at the parent
  Pair mass[kSampleMaxNodes];                    // its token's mass at the parent (the logit at first)
  float most[kSampleMaxNodes];                   // of rows with children
  int32_t at[kSampleMaxNodes];
  Pair sum[kSampleMaxNodes];
  uint32_t inner[kSampleMaxNodes / 32];
  Command cmd;
  Total total[kMaxCluster];
  Total range[kWalkWarps];
  Pair group[kWalkWarps];
  int32_t n_refused, last;
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

// One warp's range of one row: its sum, or its first largest token (greedy).
__device__ __forceinline__ Total sum_range(const SampleArgs& a, const Command& cmd, const Slope& c, bool greedy, int64_t row,
                                           int64_t v0, int64_t v1, const int32_t* refused, int n_refused) {
  const int lane = threadIdx.x & 31;
  const float* x = a.logits + row * a.stride;
  const float* p = a.probs ? a.probs + row * a.probs_stride : nullptr;
  constexpr int U = 4;
  Total t{cmd.most, 0x7FFFFFFF, {0.0f, 0.0f}};
  if (!cmd.known) {
    t.most = -INFINITY;
    for (int64_t i0 = v0; i0 < v1; i0 += 128 * U) {
      float4 f[U];
#pragma unroll
      for (int k = 0; k < U; ++k) f[k] = four(x, i0 + k * 128 + 4 * lane, v1, a.vec, -INFINITY);
#pragma unroll
      for (int k = 0; k < U; ++k) t.most = fmaxf(t.most, fmaxf(fmaxf(f[k].x, f[k].y), fmaxf(f[k].z, f[k].w)));
    }
    t.most = warp_max(t.most);
  }
  if (t.most == -INFINITY) return t;
  if (greedy) {
    int32_t at = 0x7FFFFFFF;
    for (int64_t i = v0 + 4 * lane; i < v1 && at == 0x7FFFFFFF; i += 128) first_at(four(x, i, v1, a.vec, -INFINITY), i, t.most, at);
    __syncwarp();
    t.at = __reduce_min_sync(0xFFFFFFFFu, at);
    return t;
  }
  const Ref ref = make_ref(t.most, c);
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
  t.sum = warp_sum(sum.value());
  return t;
}

// The parts' largest logit, their first token at it, and their sum in its units (a part a lane, 0 <= lane < n).
__device__ __forceinline__ Total join(const Total* part, int n, const Slope& c, Pair& mine) {
  const int lane = threadIdx.x & 31;
  Total t{-INFINITY, 0x7FFFFFFF, {0.0f, 0.0f}};
  if (lane < n) t = part[lane];
  const float most = warp_max(t.most);
  t.at = __reduce_min_sync(0xFFFFFFFFu, t.most == most ? t.at : 0x7FFFFFFF);
  mine = {0.0f, 0.0f};
  if (t.sum.h > 0.0f) {
    const float k = scale_of(make_ref(t.most, c), make_ref(most, c), c);
    mine = {t.sum.h * k, t.sum.l * k};
  }
  t.most = most;
  t.sum = warp_sum(mine);
  return t;
}

// The bonus token, by the block that holds it: first the warp's range, then 128 tokens, then the token.  The
// sums of ranges, groups and lanes are rounded differently; where the last tokens do not pass the
// target by that, it is the last one with a mass.
__device__ __forceinline__ void find_token(const SampleArgs& a, WalkShared& s, const Slope& c, int64_t row, int64_t first,
                                           int32_t* bonus) {
  const Command& cmd = s.cmd;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Ref whole = make_ref(cmd.most, c);
  Pair mine{0.0f, 0.0f};
  float k = 1.0f;
  if (lane < kWalkWarps && s.range[lane].sum.h > 0.0f) {
    const Ref part = make_ref(s.range[lane].most, c);
    k = scale_of(part, whole, c);
    mine = {s.range[lane].sum.h * k, s.range[lane].sum.l * k};
  }
  const Found in = find_lane(mine, cmd.target);
  const int range = max(in.lane, 0);
  const Ref ref = make_ref(s.range[range].most, c);
  Pair target = cmd.target - in.before;
  k = scale_of(whole, ref, c);
  target = {target.h * k, target.l * k};
  const int64_t v0 = first + range * a.range, v1 = min(a.V, v0 + a.range);
  const float* x = a.logits + row * a.stride;
  const float* p = a.probs ? a.probs + row * a.probs_stride : nullptr;
  const int n_refused = cmd.refused ? s.n_refused : 0;
  if (tid == 0) s.last = -1;
  for (int64_t base = v0; base < v1; base += 128 * kWalkWarps) {
    const int64_t i = base + warp * 128 + 4 * lane;
    const float4 q = cmd.residual ? four(p, i, v1, a.probs_vec, 0.0f) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const Four f = masses4(four(x, i, v1, a.vec, -INFINITY), chance4(q), i, ref, c, cmd, s.refused, n_refused);
    const float2 h0 = split2(f.h[0]), l0 = split2(f.lo[0]), h1 = split2(f.h[1]), l1 = split2(f.lo[1]);
    const Pair m[4] = {{h0.x, l0.x}, {h0.y, l0.y}, {h1.x, l1.x}, {h1.y, l1.y}};
    mine = (m[0] + m[1]) + (m[2] + m[3]);
    const Pair all = warp_sum(mine);
    if (lane == 0) s.group[warp] = all;
    __syncthreads();
    const Found at = find_lane(lane < kWalkWarps ? s.group[lane] : Pair{0.0f, 0.0f}, target);
    if (at.passed && at.lane == warp) {
      const Pair rest = target - at.before;
      const Found l = find_lane(mine, rest);
      if (lane == l.lane) {
        Pair sum = l.before;
        int found = -1, last = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sum = sum + m[e];
          if (m[e].h > 0.0f) last = e;
          if (found < 0 && m[e].h > 0.0f && sum > rest) found = e;
        }
        *bonus = (int32_t)i + (found >= 0 ? found : last);
      }
    }
    if (at.passed) return;
    target = target - at.all;
    int last = -1;
#pragma unroll
    for (int e = 0; e < 4; ++e) last = m[e].h > 0.0f ? e : last;
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
        s.mass[i].h = s.draft[i] >= 0 ? a.logits[(off + p) * a.stride + x] : 0.0f;
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
      for (int k = lane; k < a.units; k += 32) most = fmaxf(most, st[k].most);
      most = warp_max(most);
      const Ref ref = make_ref(most, c);
      int32_t at = 0x7FFFFFFF;
      Pair sum{0.0f, 0.0f};
      for (int k = lane; k < a.units; k += 32) {
        const UnitStat u = st[k];
        if (u.most == most) at = min(at, u.at);
        if (u.sum[0] > 0.0f) {
          const float scale = scale_of(make_ref(u.most, c), ref, c);
          sum = sum + Pair{u.sum[0] * scale, u.sum[1] * scale};
        }
      }
      at = __reduce_min_sync(0xFFFFFFFFu, at);
      sum = warp_sum(sum);
      if (lane == 0) {
        s.most[i] = most;
        s.at[i] = at;
        s.sum[i] = sum;
      }
    }
    __syncthreads();
    if (!greedy)
      for (int i = 1 + tid; ok && i < n; i += kWalkThreads) {
        uint64_t h, lo;
        mass2(both(s.mass[i].h), make_ref(s.most[s.parent[i]], c), c, h, lo);
        s.mass[i] = {split2(h).x, split2(lo).x};
      }
    __syncthreads();
  }

  // ---- the walk's state (first block, warp 0)
  enum { kWalk, kRefused, kSummed } stage = kWalk;
  int cur = 0, last = 0, depth = 0;
  bool inner = false, summed = false, spent = false, refused = false;
  double tau = 0.0, Q = 1.0, M = 0.0;
  Pair mine{0.0f, 0.0f};  // of a block, in its lane
  Total all{};
  Command cmd{};
  const float u_bonus = fminf(fmaxf(a.u_bonus[r], 0.0f), 0.99999994f);
  auto enter = [&](int node) {
    cur = last = node;
    inner = s.inner[node >> 5] >> (node & 31) & 1u;
    summed = spent = refused = false;
    tau = 0.0;
    Q = 1.0;
    M = inner ? wide(s.sum[node]) : 0.0;
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
        if (stage != kWalk) all = join(s.total, cluster, c, mine);  // the blocks' sums
        bool ends = stage == kSummed, asked = false;
        if (stage == kRefused) {
          M = wide(all.sum);
          summed = M > 0.0;
          spent = !summed;  // nothing is left: the bonus comes from p as it was
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
            if (spent || !(s.sum[cur].h > 0.0f)) continue;
            bool twice = false;  // a sibling with this token was refused before
            for (int i0 = cur + 1; i0 < j && !twice; i0 += 32)
              twice = __any_sync(0xFFFFFFFFu, i0 + lane < j && s.parent[i0 + lane] == cur && s.draft[i0 + lane] == x);
            if (twice) continue;
            const double e = wide(s.mass[j]), u = s.u[j], q = s.q[j];
            take = a.probs ? Q > 0.0 && u * q * M < (e - tau * q) * Q : u * M < e;
            if (!take) {
              if (!a.probs) {
                refused = true;
                M = fmax(M - e, 0.0);
              } else if (q > 0.0 && Q > 0.0) {
                tau += Q == 1.0 ? M : M / Q;
                Q -= q;
                ask(true);
                stage = kRefused;
                asked = true;
              }
            }
          }
          if (take) {
            ++depth;
            if (lane == 0) a.path_nodes[off + depth] = j;
            enter(j);
          }
        }
        if (ends) {
          if (stage != kSummed) {
            if (lane == 0) a.path_len[r] = depth;
            if (greedy && inner) {
              if (lane == 0) a.bonus[r] = s.most[cur] > -INFINITY ? s.at[cur] : -1;
            } else if (!summed) {
              ask(false);
              stage = kSummed;
            }
          } else if (greedy) {
            if (lane == 0) a.bonus[r] = all.most > -INFINITY ? all.at : -1;
          } else if (!(all.sum.h > 0.0f)) {
            if (cmd.refused) {  // all that had a mass was refused: p as it was
              refused = false;
              ask(false);
            } else if (lane == 0) {
              a.bonus[r] = -1;
            }
          } else {
            summed = true;
          }
          if (summed && !greedy) {
            const Pair target = all.sum * u_bonus;
            const Found f = find_lane(mine, target);
            cmd.op = kOpFind;
            cmd.most = all.most;
            cmd.owner = f.lane;
            cmd.target = target - f.before;
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
    const int64_t v0 = first + warp * a.range, v1 = min(a.V, v0 + a.range);
    const Total t = sum_range(a, s.cmd, c, greedy, row, v0, v1, s.refused, s.cmd.refused ? s.n_refused : 0);
    if (lane == 0) s.range[warp] = t;
    __syncthreads();
    if (warp == 0) {
      Pair part;
      const Total sum = join(s.range, kWalkWarps, c, part);
      if (lane == 0) send(sum, &s.total[rank], 0);
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
