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
// The bonus is the first token whose cumulative mass passes u M.  In a large vocabulary the borders between
// tokens stand 2^-20 of the mass apart and closer, so a mass has to be good to far more than a float: it
// is a pair of floats (2.8e-9 of its value), the sums stay pairs, and what adding rounds off is kept: a sum is good to
// 2^-28.  (With plain floats one token in some hundreds would differ from the formula's.)  tau takes its error from the
// sums before it: after j refusals a sum is off by j + 1 times 2^-27 of S at most, since what tau adds to one sum's error
// the next takes off again (sum of q over what is left: Q at most), and left2 rounds three times by 2^-30.5 of e.
//
// Two kernels: the rows that the walk may pass are summed by all SMs first, then a cluster of blocks per request
// walks its tree and sums a row again for every refusal.  192 nodes of 24 requests over 151936 tokens with q take
// 54 us (the rows' 70.5 MB and 24 rows of q are 13 us at the measured copy rate, the rows that these walks really
// need 7), a 16-node tree 23, 64 chains of five without q 57 (193 MB), one row of 32000 tokens 9.  What is left is
// the longest walk: a refusal is a round of the cluster, of which the sum over 15000 tokens a block is 4 to 6 us and a
// cluster barrier, the joining and the decision 2 to 3.
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "w12_internal.cuh"
#include "w12_pdl.cuh"

namespace w12 {
namespace {

constexpr int kSampleMaxNodes = 1024;  // nodes of one request
constexpr int kUnit = 1024;            // places of a row that make a unit of the rows' kernel
constexpr int kStatThreads = 256;
constexpr int kStatTile = 1024;       // nodes whose rows a column of blocks takes
constexpr int kStatRequests = 1024;   // offsets that fit in shared memory
constexpr int kWalkThreads = 512;
constexpr int kWalkWarps = kWalkThreads / 32;
constexpr int kMaxCluster = 16;
static_assert(kWalkWarps <= 16 && kMaxCluster <= 16, "join takes a part a lane of half a warp");
constexpr int32_t kSampleBadRequest = 1;
constexpr float kGreedy = 1e-5f;       // temperatures below are the limit at zero
constexpr float kMost = 3.402823466e38f;  // the largest float
constexpr float kLeast = 7.888609052210118e-31f;  // 2^-100: a smaller mass counts as none
constexpr float kSlow = 1e-36f;        // with slopes below, no two floats' masses differ by 2^-100

struct SampleArgs {
  const float *logits, *probs;
  int64_t stride, probs_stride, M, V;
  const int32_t *parent, *draft, *req_offsets;
  const float *u, *u_bonus, *temperature;
  int32_t *path_len, *path_nodes, *bonus, *status;
  struct UnitStat* stat;  // [M][units], of rows with children
  int32_t* falls;         // whether the offsets fall somewhere
  int64_t range;          // places of a warp in the walk, a multiple of 128
  int32_t n_req, units;
  bool rows_first;        // the rows' kernel stands before the walk (not for one node of one request)
};

struct alignas(16) UnitStat {
  float most;    // largest logit (-inf: none, NaN left out)
  int32_t at;    // its first token, of greedy requests
  float sum[2];  // of the masses, in the units of the largest (without q to 2^-15)
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
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
  const float p = __fmul_rn(a.h, b.h), e = fmaf(a.h, b.l, fmaf(a.l, b.h, fmaf(a.h, b.h, -p)));
  const float h = p + e;
  return {h, e - (h - p)};
}
__device__ __forceinline__ Pair operator/(Pair a, Pair b) {
  const float x = a.h / b.h;
  const Pair rest = a - b * x;
  const float y = rest.h / b.h, h = x + y;
  return {h, y - (h - x)};
}
__device__ __forceinline__ bool operator>(Pair a, Pair b) { return a.h > b.h || (a.h == b.h && a.l > b.l); }

__device__ __forceinline__ Pair shuffle_xor(Pair a, int o) {
  return {__shfl_xor_sync(0xFFFFFFFFu, a.h, o), __shfl_xor_sync(0xFFFFFFFFu, a.l, o)};
}
__device__ __forceinline__ Pair shuffle(Pair a, int lane) {
  return {__shfl_sync(0xFFFFFFFFu, a.h, lane), __shfl_sync(0xFFFFFFFFu, a.l, lane)};
}

__device__ __forceinline__ Pair warp_sum(Pair a) {
#pragma unroll 1
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

template <int N>  // lanes from N on hold nothing
__device__ __forceinline__ Found find_lane(Pair mine, Pair target) {
  const int lane = threadIdx.x & 31;
  Pair upto = mine;
#pragma unroll 1
  for (int o = 1; o < N; o <<= 1) {
    const Pair t{__shfl_up_sync(0xFFFFFFFFu, upto.h, o), __shfl_up_sync(0xFFFFFFFFu, upto.l, o)};
    if (lane >= o) upto = t + upto;
  }
  const uint32_t some = __ballot_sync(0xFFFFFFFFu, mine.h > 0.0f);
  const uint32_t over = __ballot_sync(0xFFFFFFFFu, mine.h > 0.0f && upto > target);
  Found f;
  f.passed = over != 0;
  f.lane = over ? __ffs((int)over) - 1 : 31 - __clz((int)some);
  f.all = shuffle(upto, N - 1);
  f.before = f.lane > 0 ? shuffle(upto, f.lane - 1) : Pair{0.0f, 0.0f};
  return f;
}

// ---------------------------------------------------------------- masses

// log2(e) / T as a pair of floats, and about one over it.
struct Slope {
  float hi, lo, over;
};

__device__ __forceinline__ Slope make_slope(float T) {
  const float x = __fdiv_rn(1.44269502162933349609375f, T);
  // (the first quotient's remainder is exact)
  const float rest = fmaf(-x, T, 1.44269502162933349609375f) + 1.925963033500011e-8f;
  return T < INFINITY ? Slope{x, __fdiv_rn(rest, T), T * 0.6931471805599453f} : Slope{0.0f, 0.0f, INFINITY};
}

// What the masses of a row, or of a part of it, are measured in: about the mass of its largest logit
// `most`.  The exponent most * c is rounded to a whole number, so that parts of rows differ by powers of two
// alone; where it is past 2^16 (a tiny temperature), the float product would keep too little of a fraction, and the
// logits are taken relative to `most` instead, which is exact for those that still have a mass.
struct Ref {
  float most, shift, whole;
};

__device__ __forceinline__ Ref make_ref(float most, const Slope& c) {
  const float x = most * c.hi;
  const bool far = fabsf(x) >= 65536.0f && fabsf(most) < INFINITY;
  return Ref{most, far ? most : 0.0f, far ? 0.0f : fabsf(most) == INFINITY ? most : rintf(x)};
}

// The smallest logit, less the shift, that is looked at: 2^-125 of a unit.
__device__ __forceinline__ float least_of(const Ref& r, const Slope& c) {
  return fmaxf((r.whole - 125.0f) * c.over, -kMost);
}

// (no power of two, so that the factor is a pair as well)
__device__ __noinline__ Pair far_scaled(Pair x, Ref from, Ref to, Slope c) {
  const double k = (double)c.hi + (double)c.lo;
  // (of two shifts the difference is exact)
  const double d = from.shift != 0.0f && to.shift != 0.0f ? ((double)from.shift - (double)to.shift) * k
                   : from.shift != 0.0f                   ? (double)from.shift * k - (double)to.whole
                                                          : (double)from.whole - (double)to.shift * k;
  const double e = exp2(d);
  const float h = (float)e;
  return x * Pair{h, h < INFINITY ? (float)(e - (double)h) : 0.0f};
}

// A mass, or a sum of them, in units of `to` instead of `from`.
__device__ __forceinline__ Pair scaled(Pair x, const Ref& from, const Ref& to, const Slope& c) {
  if (from.most == to.most) return x;
  if (from.shift != 0.0f || to.shift != 0.0f) return far_scaled(x, from, to, c);
  const float w = from.whole - to.whole;
  const float k = w >= -126.0f ? __int_as_float((127 + (int)fminf(w, 127.0f)) << 23) : 0.0f;
  return {x.h * k, x.l * k};
}

// 2^(j/32) as a float, and the rest of it as a part of that float.
__device__ const float2 kRoots[32] = {
    {1.0f, 0.0f}, {1.0218972f, -4.70845762e-08f}, {1.04427373f, 4.62854715e-08f}, {1.06714046f, -5.56042252e-08f},
    {1.09050775f, -1.19921575e-08f}, {1.1143868f, -4.87760623e-08f}, {1.13878858f, 4.72978243e-08f}, {1.1637249f, -3.48144269e-08f},
    {1.18920708f, 3.19341815e-08f}, {1.21524739f, -2.68866653e-08f}, {1.24185777f, 3.62105723e-08f}, {1.26905096f, 1.11842102e-09f},
    {1.29683959f, -3.09907193e-08f}, {1.32523668f, -2.63830096e-08f}, {1.35425556f, -7.47521334e-09f}, {1.38390994f, -4.24563567e-08f},
    {1.41421354f, 1.71142709e-08f}, {1.44518077f, 2.30019666e-08f}, {1.47682619f, -3.04768335e-08f}, {1.50916445f, -1.65385377e-08f},
    {1.54221082f, 5.23333421e-09f}, {1.5759809f, -3.5920646e-08f}, {1.61049032f, 6.10759177e-09f}, {1.64575553f, -3.11405444e-08f},
    {1.68179286f, -1.47196051e-08f}, {1.71861935f, -2.82181016e-08f}, {1.75625217f, -5.25879518e-09f}, {1.79470909f, -6.36038733e-09f},
    {1.8340081f, -6.12825968e-09f}, {1.87416768f, -2.48804088e-08f}, {1.91520655f, 5.14060927e-09f}, {1.95714414f, -8.69726691e-09f}};

// A row's constants of mass2; lane j keeps the j-th root, its exponent lowered by the unit's and by what the
// bits of t bring with them.
struct Scale {
  float shift, least, hi, lo;
  uint32_t root;
  float rest;
  bool endless;  // the largest logit is +inf: the infinite ones alone have a mass, alike
  bool plain;    // neither that nor a shift, nor a slope at which the clamp does not tell -inf
};

constexpr float kMagic = 393216.0f;  // 1.5 * 2^18: a float near it holds 32nds, its bits are kMagicBits + 32 x
constexpr uint32_t kMagicBits = 0x48C00000u;
constexpr float kExp1 = 0.6931471805599453f, kExp2 = 0.24022847f, kExp3 = 5.550410866482158e-2f;

// (float bits of t) * 2^18 + this is the mass's float: j's root at the exponent of the whole part
__device__ __forceinline__ uint32_t root_bits(float root, int j, float whole) {
  return __float_as_uint(root) - ((uint32_t)j << 18) - ((uint32_t)(int32_t)whole << 23) - (kMagicBits << 18);
}

__device__ __forceinline__ Scale make_scale(const Ref& r, const Slope& c, float2 root) {
  Scale s;
  s.shift = r.shift;
  s.hi = c.hi;
  s.lo = c.lo;
  s.endless = r.most == INFINITY;
  s.plain = !s.endless && r.shift == 0.0f && c.hi >= kSlow;
  s.least = s.endless ? 0.0f : least_of(r, c);
  s.root = root_bits(root.x, threadIdx.x & 31, s.endless ? 0.0f : r.whole);
  s.rest = root.y;
  return s;
}

// The masses of two logits, h + lo each: 2^(x - whole), x = (l - shift) c.  With 32 x rounded to n,
// 2^x = 2^(n / 32) 2^g, |g| <= 1/64; g comes from fused products without their rounding, and 2^g - 1 = g (ln 2 +
// g (a + g b)) to 2^-33 (Taylor's terms, the second raised by 0.83 of the fourth's most), with the root's rest.  The roundings
// are g's two (2^-31 each), w's last two (2^-30.5, 2^-31) and lo's (2^-30.5): a mass is good to 2.8e-9 of itself at worst
// (2^-28.6 was the most found).  What has none comes out as 2^-125 or so, which least2 and left2 take for nothing.
// All lanes of a warp take part.  Without ANY the scale is plain.
template <bool ANY>
__device__ __forceinline__ void mass2(uint64_t l, const Scale& c, uint64_t& h, uint64_t& lo) {
  const float2 given = split2(l);
  if (ANY) l = add2(l, both(-c.shift));
  const float2 lf = split2(l);
  l = pair2(fmaxf(lf.x, c.least), fmaxf(lf.y, c.least));
  const uint64_t t = fma2(l, both(c.hi), both(kMagic));
  const uint64_t g = fma2(l, both(c.lo), fma2(l, both(c.hi), sub2(both(kMagic), t)));
  const float2 tf = split2(t);
  const uint32_t tx = __float_as_uint(tf.x), ty = __float_as_uint(tf.y);
  const uint64_t rest = pair2(__shfl_sync(0xFFFFFFFFu, c.rest, tx), __shfl_sync(0xFFFFFFFFu, c.rest, ty));
  float x = __uint_as_float((tx << 18) + __shfl_sync(0xFFFFFFFFu, c.root, tx));
  float y = __uint_as_float((ty << 18) + __shfl_sync(0xFFFFFFFFu, c.root, ty));
  const uint64_t w = fma2(fma2(fma2(both(kExp3), g, both(kExp2)), g, both(kExp1)), g, rest);
  if (ANY) {  // (at an endless temperature the clamp does not tell -inf)
    x = given.x >= -kMost ? x : 0.0f;
    y = given.y >= -kMost ? y : 0.0f;
  }
  h = pair2(x, y);
  lo = mul2(h, w);
  if (ANY && c.endless) {
    h = pair2(given.x == INFINITY ? 1.0f : 0.0f, given.y == INFINITY ? 1.0f : 0.0f);
    lo = both(0.0f);
  }
}

// Masses below 2^-100 are left out.
__device__ __forceinline__ void least2(uint64_t& h, uint64_t& lo) {
  const float2 hf = split2(h), gf = split2(lo);
  const bool x = hf.x > kLeast, y = hf.y > kLeast;
  h = pair2(x ? hf.x : 0.0f, y ? hf.y : 0.0f);
  lo = pair2(x ? gf.x : 0.0f, y ? gf.y : 0.0f);
}

// What a refusal leaves of a mass, max(e - tau q, 0), for two tokens; less than 2^-100 is nothing.  (Where
// something is left, h is the larger or the difference exact, so its rounding comes back from three operations.)
__device__ __forceinline__ void left2(uint64_t& h, uint64_t& lo, uint64_t q, float tau_hi, float tau_lo) {
  const uint64_t p = mul2(q, both(-tau_hi)), rest = fma2(q, both(tau_hi), p);  // tau_hi q = rest - p
  const uint64_t s = add2(h, p);
  const uint64_t t = add2(sub2(p, sub2(s, h)), fma2(q, both(-tau_lo), sub2(lo, rest)));
  const float2 sf = split2(s), tf = split2(t), all = split2(add2(s, t));
  const bool x = all.x > kLeast, y = all.y > kLeast;
  h = pair2(x ? sf.x : 0.0f, y ? sf.y : 0.0f);
  lo = pair2(x ? tf.x : 0.0f, y ? tf.y : 0.0f);
}

// The masses of four tokens, unless LEFT will look at them those below 2^-100 left out.
struct Four {
  uint64_t h[2], lo[2];
};

template <bool ANY, bool LEFT = false>
__device__ __forceinline__ Four masses4(const float4& f, const Scale& c) {
  Four m;
  mass2<ANY>(pair2(f.x, f.y), c, m.h[0], m.lo[0]);
  mass2<ANY>(pair2(f.z, f.w), c, m.h[1], m.lo[1]);
  if (!LEFT) {
    least2(m.h[0], m.lo[0]);
    least2(m.h[1], m.lo[1]);
  }
  return m;
}

// 2^x and 2^((l - most) c) by plain floats, to 2^-20 or so.
__device__ __forceinline__ float rough_exp2(float x) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
  return e;
}

__device__ __forceinline__ float rough(float l, float most, float slope, float least) {
  const float d = l == most ? 0.0f : l - most;  // (equal infinities)
  return d >= least ? rough_exp2(d * slope) : 0.0f;
}

// A running sum of masses, two side by side, and what its additions round off (Knuth's six operations, since a mass
// may be larger than the sum so far).  Low parts are up to 1.1 % of their masses and often of one sign, so they are
// added like the masses, two as one: that sum's rounding, 2^-30.5 of the masses, is the only loss.  `rest` takes
// 2^-24 of the sum at a time, which a float adds up to 2^-30 of it at worst over kStretch places; longer ranges settle.
// With the low parts in `rest`, and sums that start above every mass for the sake of three operations, 9496 equal masses
// lost up to 2^-25.4 of their sum, 42752 2^-23.5; 192 nodes then took 50.4 us (53.4 now), 64 chains 55.3 (57.8).
// (Masses brought into order, lo the rounding of h, would lose nothing: 56.4 us.  The larger of sum and mass by comparison
// in place of three of the six operations 57.0.)
struct Sum {
  uint64_t s = both(0.0f), rest = both(0.0f);
  __device__ __forceinline__ uint64_t step(uint64_t x) {  // (what it leaves)
    const uint64_t n = add2(s, x), v = sub2(n, s), t = add2(sub2(s, sub2(n, v)), sub2(x, v));
    s = n;
    return t;
  }
  __device__ __forceinline__ void add(const Four& m) {
    const uint64_t x = add2(step(m.h[0]), step(m.h[1]));
    const uint64_t l = add2(m.lo[0], m.lo[1]), n = add2(s, l), y = sub2(l, sub2(n, s));  // (smaller than the sum)
    s = n;
    rest = add2(rest, add2(x, y));
  }
  __device__ __forceinline__ void settle() { rest = step(rest); }
  __device__ __forceinline__ Pair value() const {
    const float2 a = split2(s), b = split2(rest);
    return Pair{a.x, b.x} + Pair{a.y, b.y};
  }
};

constexpr int kStretch = 1 << 15;  // places of a warp

// A row of logits and its row of q.  Places are counted from the 16-byte boundary at or before the row's first logit,
// so that any row allows 16-byte loads: tokens stand at places lo .. hi - 1, token v at v + lo.
struct Row {
  const float *x, *p;
  int lo;
  int64_t hi;
  bool p_vec;  // q's row is aligned like the logits'
};

__device__ __forceinline__ int off_boundary(const float* x) { return (int)((uintptr_t)x >> 2 & 3u); }

__device__ __forceinline__ Row row_of(const SampleArgs& a, int64_t m) {
  Row r;
  r.x = a.logits + m * a.stride;
  r.lo = off_boundary(r.x);
  r.hi = a.V + r.lo;
  r.x -= r.lo;
  r.p = a.probs ? a.probs + m * a.probs_stride : nullptr;
  r.p_vec = a.probs && off_boundary(r.p) == r.lo;
  r.p = a.probs ? r.p - r.lo : nullptr;
  return r;
}

// Four places from i on (a multiple of four), `fill` outside lo .. hi - 1.
__device__ __forceinline__ float4 four(const float* x, int64_t i, int lo, int64_t hi, bool vec, float fill) {
  if (vec && i >= lo && i + 4 <= hi) return *reinterpret_cast<const float4*>(x + i);
  float4 f = make_float4(fill, fill, fill, fill);
  if (i >= lo && i < hi) f.x = x[i];
  if (i + 1 >= lo && i + 1 < hi) f.y = x[i + 1];
  if (i + 2 >= lo && i + 2 < hi) f.z = x[i + 2];
  if (i + 3 >= lo && i + 3 < hi) f.w = x[i + 3];
  return f;
}

// The first place of `most` among four from i on.
__device__ __forceinline__ void first_at(const float4& f, int64_t i, float most, int32_t& at) {
  const int k = f.x == most ? 0 : f.y == most ? 1 : f.z == most ? 2 : f.w == most ? 3 : 4;
  if (k < 4 && (int32_t)i + k < at) at = (int32_t)i + k;
}

// ---------------------------------------------------------------- ranges of a row

struct alignas(16) Total {
  float most;
  int32_t at;
  Pair sum;
};

// One warp's range of a row of a greedy request: its largest logit and the first token at it.
__device__ __forceinline__ Total first_of_range(const Row& row, int64_t v0, int64_t v1) {
  const int lane = threadIdx.x & 31;
  Total t{-INFINITY, 0x7FFFFFFF, {0.0f, 0.0f}};
  constexpr int W = 8;  // loads of a lane on their way
#pragma unroll 1
  for (int64_t i0 = v0; i0 < v1; i0 += 128 * W) {
    float4 f[W];
#pragma unroll
    for (int k = 0; k < W; ++k) f[k] = four(row.x, i0 + k * 128 + 4 * lane, row.lo, v1, true, -INFINITY);
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const float most = fmaxf(fmaxf(f[k].x, f[k].y), fmaxf(f[k].z, f[k].w));
      if (most > t.most) {
        t.most = most;
        t.at = 0x7FFFFFFF;
        first_at(f[k], i0 + k * 128 + 4 * lane, most, t.at);
      }
    }
  }
  const float most = warp_max(t.most);
  t.at = __reduce_min_sync(0xFFFFFFFFu, t.most == most ? t.at : 0x7FFFFFFF) - row.lo;
  t.most = most;
  return t;
}

// One warp's range of a row whose largest logit is not known (a node without children): the sum of its masses in
// one sweep, in units of the largest logit of the first tokens, and of larger ones where they come (the sum so far
// changes by a power of two then).  A mass may pass a unit by twice before that.
template <int U>  // loads of a lane on their way
__device__ __forceinline__ Total sum_unknown(const Row& row, const Slope& c, int64_t v0, int64_t v1, float2 root) {
  const int lane = threadIdx.x & 31;
  Total t{-INFINITY, 0x7FFFFFFF, {0.0f, 0.0f}};
  Scale scale{};
  Sum sum;
  float limit = -INFINITY;
#pragma unroll 1
  for (int64_t i0 = v0; i0 < v1; i0 += 128 * U) {
    float4 f[U];
#pragma unroll
    for (int k = 0; k < U; ++k) f[k] = four(row.x, i0 + k * 128 + 4 * lane, row.lo, v1, true, -INFINITY);
    float most = -INFINITY;
#pragma unroll
    for (int k = 0; k < U; ++k) most = fmaxf(most, fmaxf(fmaxf(f[k].x, f[k].y), fmaxf(f[k].z, f[k].w)));
    if (__any_sync(0xFFFFFFFFu, most > limit)) {
      most = warp_max(most);
      const Ref to = make_ref(most, c);
      if (t.most > -INFINITY) {
        t.sum = scaled(t.sum + sum.value(), make_ref(t.most, c), to, c);
        sum = Sum();
      }
      t.most = most;
      limit = fminf(most + c.over, kMost);  // (+inf passes it at any temperature)
      scale = make_scale(to, c, root);
    }
    if (t.most == -INFINITY) continue;
    if (scale.plain && v1 - v0 <= kStretch) {
#pragma unroll
      for (int k = 0; k < U; ++k) sum.add(masses4<false, true>(f[k], scale));
    } else {
#pragma unroll 1
      for (int k = 0; k < U; ++k) {
        const int64_t i = i0 + k * 128 + 4 * lane;
        sum.add(masses4<true>(four(row.x, i, row.lo, v1, true, -INFINITY), scale));
        sum.settle();
      }
    }
  }
  t.sum = warp_sum(t.sum + sum.value());
  if (!(t.sum.h > kLeast)) t.sum = {0.0f, 0.0f};  // (see sum_range)
  return t;
}

// The same by plain floats, a lane's sum in the mass of its own largest logit, which grows with it.  Over kStretch
// places that is good to 2^-15: 256 additions 2^-16 at worst, 32 changes of the largest logit 2^-16.7, the exponents'
// roundings 2^-18 where 2^-31 of the sum is a mass, less where it is more.  (They do not cancel: 4600 additions that round
// one way were seen to lose 6.8e-5 of the sum of 2^31 tokens.)
template <int U>
__device__ __forceinline__ Total rough_unknown(const Row& row, const Slope& c, int64_t v0, int64_t v1) {
  const int lane = threadIdx.x & 31;
  Total t{-INFINITY, 0x7FFFFFFF, {0.0f, 0.0f}};
  const float least = fmaxf(-125.0f * c.over, -kMost);
  float sum = 0.0f;
#pragma unroll 1
  for (int64_t i0 = v0; i0 < v1; i0 += 128 * U) {
    float4 f[U];
#pragma unroll
    for (int k = 0; k < U; ++k) f[k] = four(row.x, i0 + k * 128 + 4 * lane, row.lo, v1, true, -INFINITY);
    float most = t.most;
#pragma unroll
    for (int k = 0; k < U; ++k) most = fmaxf(most, fmaxf(fmaxf(f[k].x, f[k].y), fmaxf(f[k].z, f[k].w)));
    if (most > t.most) {
      sum *= rough(t.most, most, c.hi, least);
      t.most = most;
    }
#pragma unroll
    for (int k = 0; k < U; ++k)
      sum += (rough(f[k].x, most, c.hi, least) + rough(f[k].y, most, c.hi, least)) +
             (rough(f[k].z, most, c.hi, least) + rough(f[k].w, most, c.hi, least));
  }
  const float most = warp_max(t.most);
  sum *= rough(t.most, most, c.hi, least);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  t.most = most;
  if (most == -INFINITY) return t;  // (its -inf count as equal to the largest)
  const Ref r = make_ref(most, c);
  if (most < INFINITY && r.shift == 0.0f) sum *= rough_exp2(fmaf(most, c.lo, fmaf(most, c.hi, -r.whole)));
  t.sum = {sum, 0.0f};
  return t;
}

// ---------------------------------------------------------------- rows with children

// Largest logit and mass of the rows whose nodes have children (what the walk asks of a node it passes), in units of
// 1024 places.  Every block of a tile of nodes makes the list of its rows with children, and the tile's warps take
// equal shares of all units, 128 bytes a lane on their way.  Without q the sums only serve decisions, which plain floats
// (good to 2^-15 together) nearly always tell, and the walk sums again for the others.
// Bound by the logits read once, and with q by the pairs' arithmetic: 256 rows of 151936 (156 MB) in 30.7 us without q
// (5.1 TB/s, 0.75 of the measured copy rate; 2.8 of it to make the list), 116 rows (70.5 MB) in 23.4 with q, 16.6 if they
// were rough.  A form for each, since the pairs spill 28 bytes at 80 registers (loads of four steps in place of eight spill
// nothing and take 23.8).  Pairs for the chains too made their call 72 us for 59.  Bringing each warp's share into L2 ahead in bulk
// took 9 us more; two or four blocks an SM about 1; one row after another by a request's blocks twice the time.
template <bool PAIRS>
__global__ void __launch_bounds__(kStatThreads, 3) k_sample_stats(const __grid_constant__ SampleArgs a) {
  pdl_enter();
  __shared__ int32_t offsets[kStatRequests + 1];
  __shared__ uint32_t inner[kStatTile / 32];  // rows with children
  __shared__ uint16_t request[kStatTile], list[kStatTile];
  __shared__ float4 slopes[kStatTile];  // of the listed rows, and whether they are greedy
  __shared__ int rows;
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t m0 = (int64_t)blockIdx.y * kStatTile, m1 = min(a.M, m0 + kStatTile + kSampleMaxNodes);
  const bool here = a.req_offsets && a.n_req <= kStatRequests;
  const float2 root = kRoots[lane];
  int32_t p = m0 + tid < m1 ? a.parent[m0 + tid] : -1;
  if (tid < kStatTile / 32) inner[tid] = 0;
  if (here)
#pragma unroll 1
    for (int r = tid; r <= a.n_req; r += kStatThreads) offsets[r] = a.req_offsets[r];
  __syncthreads();
  const int32_t* o = here ? offsets : a.req_offsets;
  if (blockIdx.x == 0 && blockIdx.y == 0) {  // rows could then belong to two requests
    bool fall = false;
#pragma unroll 1
    for (int r = tid; o && r < a.n_req; r += kStatThreads) fall = fall || o[r + 1] < o[r];
    fall = __syncthreads_or(fall);
    if (tid == 0) *a.falls = fall;
  }
#pragma unroll 1
  for (int64_t m = m0 + tid; m < m1; m += kStatThreads) {
    if (m != m0 + tid) p = a.parent[m];
    int lo = 0, hi = a.n_req;  // the last request that starts at or before node m
#pragma unroll 1
    while (o && hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (o[mid] <= m) lo = mid; else hi = mid;
    }
    const int64_t off = o ? o[lo] : 0, end = o ? o[lo + 1] : a.M;
    if (off < 0 || off > m || end <= m || end > a.M || end - off > kSampleMaxNodes || p < 0 || p >= m - off) continue;
    const int64_t at = off + p - m0;
    if (at >= 0 && at < kStatTile) {
      request[at] = (uint16_t)lo;  // (all children write the same)
      atomicOr(&inner[at >> 5], 1u << (at & 31));
    }
  }
  __syncthreads();
  if (tid < 32) {
    int before = 0;
#pragma unroll 1
    for (int w = 0; w < kStatTile / 32 && m0 + w * 32 < a.M; ++w) {
      const uint32_t word = inner[w];
      if (word >> lane & 1u) list[before + __popc(word & ((1u << lane) - 1u))] = (uint16_t)(w * 32 + lane);
      before += __popc(word);
    }
    if (tid == 0) rows = before;
  }
  __syncthreads();
  if (tid < rows) {
#pragma unroll 1
    for (int k = tid; k < rows; k += kStatThreads) {
      const float T = a.temperature ? a.temperature[request[list[k]]] : 1.0f;
      const Slope c = make_slope(T < kGreedy ? 1.0f : T);
      slopes[k] = make_float4(c.hi, c.lo, c.over, T < kGreedy ? 1.0f : 0.0f);
    }
  }
  __syncthreads();
  // An equal share of all units for every warp, one stretch after another; a stretch in one row, of up to kStretch
  // places, has one sum, in the place of its first unit.  (At most 2^10 rows of 2^21 units.)
  const uint32_t units = a.units;
  const int64_t items = (int64_t)rows * units, warps = (int64_t)gridDim.x * (kStatThreads / 32);
  const int64_t mine = (int64_t)blockIdx.x * (kStatThreads / 32) + (tid >> 5), stop = items * (mine + 1) / warps;
#pragma unroll 1
  for (int64_t item = items * mine / warps; item < stop;) {
    const uint32_t nth = (uint32_t)item / units, unit = (uint32_t)item - nth * units;
    const uint32_t run = (uint32_t)min(stop - item, (int64_t)min(units - unit, kStretch / kUnit));
    const float4 slope = slopes[nth];
    const int64_t m = m0 + list[nth];
    const Row row = row_of(a, m);
    const int64_t v0 = (int64_t)unit * kUnit, v1 = min(row.hi, v0 + (int64_t)run * kUnit);
    const Slope c{slope.x, slope.y, slope.z};
    const Total t = slope.w != 0.0f ? first_of_range(row, v0, v1)
                    : PAIRS         ? sum_unknown<8>(row, c, v0, v1, root)
                                    : rough_unknown<8>(row, c, v0, v1);
    UnitStat* out = a.stat + m * units + unit;
#pragma unroll 1
    for (uint32_t k = lane; k < run; k += 32)
      out[k] = k ? UnitStat{-INFINITY, -1, {0.0f, 0.0f}} : UnitStat{t.most, t.at, {t.sum.h, t.sum.l}};
    item += run;
  }
}

// ---------------------------------------------------------------- the walk

// One lane's mass, by the arithmetic of mass2.
__device__ __forceinline__ Pair mass1(float l, const Ref& r, const Slope& c) {
  if (r.most == INFINITY) return {l == INFINITY ? 1.0f : 0.0f, 0.0f};
  const float d = fmaxf(l - r.shift, least_of(r, c));  // (NaN: the least)
  const float t = fmaf(d, c.hi, kMagic), g = fmaf(d, c.lo, fmaf(d, c.hi, kMagic - t));
  const uint32_t n = __float_as_uint(t);
  const float2 root = kRoots[n & 31u];
  const float w = fmaf(fmaf(fmaf(kExp3, g, kExp2), g, kExp1), g, root.y);
  const float h = __uint_as_float((n << 18) + root_bits(root.x, (int)(n & 31u), r.whole));
  return l >= -kMost && h > kLeast ? Pair{h, h * w} : Pair{0.0f, 0.0f};
}

// What a cluster's blocks do next.
enum : int32_t { kOpDone, kOpSum, kOpFind };

struct alignas(16) Command {
  int32_t op;
  int32_t node;          // of the request
  int32_t known;         // kOpSum: `most` is the row's; else every warp finds its range's
  int32_t residual;      // tau q is taken off
  int32_t refused;       // the node's children are taken out (no q)
  int32_t last;          // kOpSum: the bonus token comes from these masses, if there are any
  int32_t owner;         // kOpFind: the block that holds the bonus token
  float most, tau_hi, tau_lo;
  Pair target;           // kOpFind: the mass before the bonus token in the owner's ranges, in the units of `most`
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

// 16-byte words of `from` to the same place as `to` (this block's shared memory) in block `rank` of the cluster.
template <typename S>
__device__ __forceinline__ void send(const S& from, S* to, uint32_t rank) {
  static_assert(sizeof(S) % 16 == 0 && alignof(S) == 16, "sent in 16-byte words");
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(to)), "r"(rank));
  const uint4* w = reinterpret_cast<const uint4*>(&from);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(S) / 16); ++i)
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at + 16 * i), "r"(w[i].x), "r"(w[i].y), "r"(w[i].z),
                 "r"(w[i].w)
                 : "memory");
}

// Where the walk stands at a node: what it waits for, the children tried, and what refusals have left.
enum : int32_t { kStart, kRefused, kPrecise, kSummed };

struct Walk {
  int32_t stage, cur, last, depth;
  bool inner;    // the node has children
  bool rough;    // M is good to 2^-15 of p's sum only (no q)
  bool summed;   // the blocks hold the sums of what is left
  bool refused;  // a child was refused (no q)
  bool spent;    // nothing was left
  Pair tau, Q, M, out;  // out: the masses of the refused children (no q)
};

// What all blocks have from the first one, beside its tree: each then comes to the same decisions.
struct alignas(16) Given {
  int64_t off;
  int32_t n, ok;
  Slope slope;
  float u_bonus;
  int32_t greedy;
};

struct alignas(16) Tree {
  int32_t parent[kSampleMaxNodes], draft[kSampleMaxNodes];
  float u[kSampleMaxNodes], q[kSampleMaxNodes];  // of a node: its number, and q of its token at the parent
  float most[kSampleMaxNodes];                   // of rows with children
  int32_t at[kSampleMaxNodes];
  Pair mass[kSampleMaxNodes];                    // its token's mass at the parent (the logit at first)
  Pair sum[kSampleMaxNodes];                     // of rows with children
  uint32_t inner[kSampleMaxNodes / 32];

  // Where the 16-byte words of four nodes stand: kWords of them, the last for 128 nodes.
  static constexpr int kWords = 11;
  static __device__ __forceinline__ int place(int four, int word) {
    const int array = word < 6 ? word : word < 8 ? 6 : word < 10 ? 8 : 10;
    return array * 4 * kSampleMaxNodes + (word < 6 || word == 10 ? 16 * four : 32 * four + 16 * (word & 1));
  }
};
static_assert(sizeof(Tree) == (10 * 4 + 4 / 32.0) * kSampleMaxNodes, "arrays one behind another");

struct WalkShared : Tree {
  int32_t refused[kSampleMaxNodes];  // places
  Command cmd;
  Walk walk;
  Total total[2][kMaxCluster];  // the blocks', of every other round
  Given given;
  Total range[kWalkWarps];
  Pair group[kWalkWarps];
  int32_t n_refused, last;
};

// The refused ones of four tokens from i on have no mass.
__device__ __forceinline__ void without(Four& m, int64_t i, const int32_t* refused, int n_refused) {
  uint32_t out = 0;  // of the four
#pragma unroll 1
  for (int k = 0; k < n_refused; ++k) {
    const int64_t at = refused[k] - i;
    if (at >= 0 && at < 4) out |= 1u << at;
  }
  if (out) {
    const uint64_t low = 0x00000000FFFFFFFFull, high = 0xFFFFFFFF00000000ull;
    const uint64_t k0 = (out & 1u ? 0 : low) | (out & 2u ? 0 : high), k1 = (out & 4u ? 0 : low) | (out & 8u ? 0 : high);
    m.h[0] &= k0, m.lo[0] &= k0, m.h[1] &= k1, m.lo[1] &= k1;
  }
}

__device__ __forceinline__ void left4(Four& m, const float4& q, float tau_hi, float tau_lo) {
  left2(m.h[0], m.lo[0], pair2(q.x, q.y), tau_hi, tau_lo);
  left2(m.h[1], m.lo[1], pair2(q.z, q.w), tau_hi, tau_lo);
}

__device__ __forceinline__ float chance(float q) { return fmaxf(q, 0.0f); }  // (NaN: 0)

__device__ __forceinline__ float4 chance4(float4 q) { return make_float4(chance(q.x), chance(q.y), chance(q.z), chance(q.w)); }

// One warp's range of a row whose largest logit is known: the sum of its masses, or of what refusals leave of them.
__device__ __forceinline__ Total sum_range(const Row& row, const Command& cmd, const Slope& c, int64_t v0, int64_t v1,
                                           const int32_t* refused, int n_refused, float2 root) {
  const int lane = threadIdx.x & 31;
  const float *x = row.x, *p = row.p;
  constexpr int U = 2;
  Total t{cmd.most, 0x7FFFFFFF, {0.0f, 0.0f}};
  if (t.most == -INFINITY) return t;
  const Scale scale = make_scale(make_ref(t.most, c), c, root);
  Sum sum;
  bool mine = false;  // does the range hold a refused token
#pragma unroll 1
  for (int k = 0; k < n_refused; ++k) mine = mine || (refused[k] >= v0 && refused[k] < v1);
  const bool whole_steps = (!cmd.residual || row.p_vec) && scale.plain && v1 - v0 <= kStretch;
#pragma unroll 1
  for (int64_t i0 = v0; i0 < v1;) {
    bool plain = whole_steps && i0 >= row.lo && i0 + 128 * U <= v1;
    if (plain && mine)
#pragma unroll 1
      for (int k = 0; k < n_refused; ++k) plain = plain && !(refused[k] >= i0 && refused[k] < i0 + 128 * U);
    const int64_t i = i0 + 4 * lane;
    if (plain) {  // no branches inside, so that a warp's masses overlap one another
      float4 f[U], q[U];
      Four m[U];
#pragma unroll
      for (int k = 0; k < U; ++k) f[k] = *reinterpret_cast<const float4*>(x + i + k * 128);
      if (cmd.residual) {
#pragma unroll
        for (int k = 0; k < U; ++k) q[k] = *reinterpret_cast<const float4*>(p + i + k * 128);
#pragma unroll
        for (int k = 0; k < U; ++k) m[k] = masses4<false, true>(f[k], scale);
#pragma unroll
        for (int k = 0; k < U; ++k) left4(m[k], chance4(q[k]), cmd.tau_hi, cmd.tau_lo);
      } else {
#pragma unroll
        for (int k = 0; k < U; ++k) m[k] = masses4<false, true>(f[k], scale);
      }
#pragma unroll
      for (int k = 0; k < U; ++k) sum.add(m[k]);
      i0 += 128 * U;
    } else {
      Four m = masses4<true>(four(x, i, row.lo, v1, true, -INFINITY), scale);
      if (mine) without(m, i, refused, n_refused);
      if (cmd.residual) left4(m, chance4(four(p, i, row.lo, v1, row.p_vec, 0.0f)), cmd.tau_hi, cmd.tau_lo);
      sum.add(m);
      sum.settle();
      i0 += 128;
    }
  }
  t.sum = warp_sum(sum.value());
  // what has no mass stands in it with 2^-125 each, together less than 2^-101
  if (!(t.sum.h > kLeast)) t.sum = {0.0f, 0.0f};
  return t;
}

// The parts' largest logit, their first token at it (greedy), and their sum in its units (a part a lane, 0 <= lane <
// n <= 16).  All alike: the parts' largest logits are the row's.
__device__ __forceinline__ Total join(const Total* part, int n, const Slope& c, bool greedy, bool alike, Pair& mine) {
  const int lane = threadIdx.x & 31;
  Total t{-INFINITY, 0x7FFFFFFF, {0.0f, 0.0f}};
  if (lane < n) t = part[lane];
  mine = t.sum;
  float most = __shfl_sync(0xFFFFFFFFu, t.most, 0);
  if (!alike) {
    most = t.most;
#pragma unroll 1
    for (int o = 8; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
    most = __shfl_sync(0xFFFFFFFFu, most, 0);
    if (t.sum.h > 0.0f) mine = scaled(t.sum, make_ref(t.most, c), make_ref(most, c), c);
  }
  if (greedy) {
    t.at = __reduce_min_sync(0xFFFFFFFFu, t.most == most ? t.at : 0x7FFFFFFF);
  } else {
    t.sum = mine;
#pragma unroll 1
    for (int o = 8; o; o >>= 1) t.sum = t.sum + shuffle_xor(t.sum, o);
    t.sum = shuffle(t.sum, 0);
  }
  t.most = most;
  return t;
}

// The bonus token, by the block that holds it (`target` before it in the block's ranges, in units of `most`): first
// the warp's range, then 128 tokens, then the token.  The
// sums of ranges, groups and lanes are rounded differently; where the last tokens do not pass the
// target by that, it is the last one with a mass.
__device__ __forceinline__ void find_token(const SampleArgs& a, WalkShared& s, const Slope& c, const Row& row, int64_t first,
                                           float2 root, float most, Pair target, int32_t* bonus) {
  const Command& cmd = s.cmd;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Ref whole = make_ref(most, c);
  Pair mine{0.0f, 0.0f};
  if (lane < kWalkWarps && s.range[lane].sum.h > 0.0f)
    mine = scaled(s.range[lane].sum, make_ref(s.range[lane].most, c), whole, c);
  const Found in = find_lane<16>(mine, target);
  const int range = max(in.lane, 0);
  const Ref ref = make_ref(s.range[range].most, c);
  target = scaled(target - in.before, whole, ref, c);
  const Scale scale = make_scale(ref, c, root);
  const int64_t v0 = first + range * a.range, v1 = min(row.hi, v0 + a.range);
  const int n_refused = cmd.refused ? s.n_refused : 0;
  if (tid == 0) s.last = -1;
#pragma unroll 1
  for (int64_t base = v0; base < v1; base += 128 * kWalkWarps) {
    const int64_t i = base + warp * 128 + 4 * lane;
    Four f = masses4<true>(four(row.x, i, row.lo, v1, true, -INFINITY), scale);
    without(f, i, s.refused, n_refused);
    if (cmd.residual) left4(f, chance4(four(row.p, i, row.lo, v1, row.p_vec, 0.0f)), cmd.tau_hi, cmd.tau_lo);
    const float2 h0 = split2(f.h[0]), l0 = split2(f.lo[0]), h1 = split2(f.h[1]), l1 = split2(f.lo[1]);
    const Pair none{0.0f, 0.0f};  // (adding it brings a pair in order)
    const Pair m[4] = {none + Pair{h0.x, l0.x}, none + Pair{h0.y, l0.y}, none + Pair{h1.x, l1.x}, none + Pair{h1.y, l1.y}};
    mine = (m[0] + m[1]) + (m[2] + m[3]);
    const Pair all = warp_sum(mine);
    if (lane == 0) s.group[warp] = all;
    __syncthreads();
    const Found at = find_lane<16>(lane < kWalkWarps ? s.group[lane] : none, target);
    if (at.passed && at.lane == warp) {
      const Pair rest = target - at.before;
      const Found l = find_lane<32>(mine, rest);
      if (lane == l.lane) {
        Pair sum = l.before;
        int found = -1, last = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sum = sum + m[e];
          if (m[e].h > 0.0f) last = e;
          if (found < 0 && m[e].h > 0.0f && sum > rest) found = e;
        }
        *bonus = (int32_t)(i - row.lo) + (found >= 0 ? found : last);
      }
    }
    if (at.passed) return;
    target = target - at.all;
    int last = -1;
#pragma unroll
    for (int e = 0; e < 4; ++e) last = m[e].h > 0.0f ? e : last;
    if (last >= 0) atomicMax(&s.last, (int32_t)(i - row.lo) + last);
    __syncthreads();
  }
  if (tid == 0) *bonus = s.last;
}

// What comes next, by a block's first warp (all lanes alike, and all blocks): the walk goes on with the sums that it
// had asked for, until it needs others or ends.  The first block writes the results.
__device__ __forceinline__ Command decide(const SampleArgs& a, WalkShared& s, const Total* total, Slope c, bool greedy, int r,
                                          bool writes, int cluster) {
  const int lane = threadIdx.x & 31, n = s.given.n;
  const bool ok = s.given.ok;
  writes = writes && lane == 0;
  const Pair zero{0.0f, 0.0f}, one{1.0f, 0.0f};
  Walk w = s.walk;
  Command cmd = s.cmd;    // the last one
  Pair mine{0.0f, 0.0f};  // of a block, in its lane
  Total all{};
  auto enter = [&](int node) {
    w.cur = w.last = node;
    w.inner = s.inner[node >> 5] >> (node & 31) & 1u;
    w.summed = w.spent = w.refused = false;
    w.rough = !a.probs;
    w.tau = w.out = zero;
    w.Q = one;
    w.M = w.inner ? s.sum[node] : zero;
  };
  auto ask = [&](bool residual, bool off_refused, bool last) {
    cmd.op = kOpSum;
    cmd.node = w.cur;
    cmd.known = w.inner;
    cmd.most = w.inner ? s.most[w.cur] : 0.0f;
    cmd.residual = residual;
    cmd.refused = off_refused;
    cmd.last = last;
    cmd.tau_hi = w.tau.h;
    cmd.tau_lo = w.tau.l;
  };
  if (ok && w.stage == kStart) {
    enter(0);
    w.depth = 0;
    if (writes) a.path_nodes[s.given.off] = 0;
  }
  cmd.op = kOpDone;
  if (ok) {
    if (w.stage != kStart) all = join(total, cluster, c, greedy, cmd.known, mine);  // the blocks' sums
    bool ends = w.stage == kSummed, asked = false;
    if (w.stage == kRefused) {
      w.M = all.sum;
      w.summed = w.M > zero;
      w.spent = !w.summed;  // nothing is left: the bonus comes from p as it was
    } else if (w.stage == kPrecise) {
      w.M = all.sum - w.out;
      if (!(w.M > zero)) w.M = zero;
      w.rough = false;
      w.summed = !w.refused;
    }
#pragma unroll 1
    while (!ends && !asked) {
      int j = -1;  // the next child
#pragma unroll 1
      for (int i0 = w.last + 1; i0 < n && j < 0; i0 += 32) {
        const uint32_t b = __ballot_sync(0xFFFFFFFFu, i0 + lane < n && s.parent[i0 + lane] == w.cur);
        if (b) j = i0 + __ffs((int)b) - 1;
      }
      if (j < 0) {
        ends = true;
        break;
      }
      w.last = j;
      const int32_t x = s.draft[j];
      if (x < 0) continue;
      bool take = greedy && x == s.at[w.cur];
      if (greedy ? !(s.most[w.cur] > -INFINITY) : w.spent || !(s.sum[w.cur].h > 0.0f)) continue;
      if (!greedy || a.probs) {
        bool twice = false;  // a sibling with this token was refused before
#pragma unroll 1
        for (int i0 = w.cur + 1; i0 < j && !twice; i0 += 32)
          twice = __any_sync(0xFFFFFFFFu, i0 + lane < j && s.parent[i0 + lane] == w.cur && s.draft[i0 + lane] == x);
        if (twice) continue;
      }
      if (greedy && a.probs) {
        // p stays 1 at its token, unless q was all of what it had left there when a sibling was refused (tau: Q then)
        const Pair q{s.q[j], 0.0f};
        if (take) {
          take = w.Q > q * s.u[j] && w.Q > zero && (!(w.tau > zero) || w.tau > q);
        } else if (q > zero && w.Q > zero) {
          w.tau = w.Q;
          w.Q = w.Q - q;
        }
      } else if (!greedy) {
        const Pair e = zero + s.mass[j];
        const float u = s.u[j], q = a.probs ? s.q[j] : 1.0f;
        const Pair mine_u = w.M * u * q, limit = a.probs ? (e - w.tau * q) * w.Q : e;
        const bool moves = !a.probs || (q > 0.0f && w.Q > zero);  // a refusal would change p
        take = (!a.probs || w.Q > zero) && limit > mine_u;
        // (2^-14: a rough sum does not tell)
        if (w.rough && fabsf((mine_u - limit).h) <= 6.2e-5f * u * (w.M + w.out).h) {
          w.last = j - 1;
          ask(false, false, false);
          w.stage = kPrecise;
          asked = true;
          continue;
        }
        if (!take && moves) {
          w.summed = false;
          if (!a.probs) {
            w.refused = true;
            w.out = w.out + e;
            w.M = w.M - e;
            if (!(w.M > zero)) w.M = zero;
          } else {
            w.tau = w.tau + (w.Q.h == 1.0f && w.Q.l == 0.0f ? w.M : w.M / w.Q);
            w.Q = w.Q - Pair{q, 0.0f};
            bool more = false;  // children behind this one
#pragma unroll 1
            for (int i0 = j + 1; i0 < n && !more; i0 += 32)
              more = __any_sync(0xFFFFFFFFu, i0 + lane < n && s.parent[i0 + lane] == w.cur);
            if (!more && writes) a.path_len[r] = w.depth;
            ask(true, false, !more);
            w.stage = kRefused;
            asked = true;
          }
        }
      }
      if (take) {
        ++w.depth;
        if (writes) a.path_nodes[s.given.off + w.depth] = j;
        enter(j);
      }
    }
    if (ends) {
      if (w.stage != kSummed) {
        if (writes) a.path_len[r] = w.depth;
        if (greedy && w.inner) {
          if (writes) a.bonus[r] = s.most[w.cur] > -INFINITY ? s.at[w.cur] : -1;
        } else if (!w.summed) {
          ask(false, w.refused, !greedy);
          w.stage = kSummed;
        }
      } else if (greedy) {
        if (writes) a.bonus[r] = all.most > -INFINITY ? all.at : -1;
      } else if (!(all.sum.h > 0.0f)) {
        if (cmd.refused) {  // all that had a mass was refused: p as it was
          ask(false, false, true);
        } else if (writes) {
          a.bonus[r] = -1;
        }
      } else {
        w.summed = true;
      }
      if (w.summed && !greedy) {
        const Pair target = all.sum * s.given.u_bonus;
        const Found f = find_lane<16>(mine, target);
        cmd.op = kOpFind;
        cmd.most = all.most;
        cmd.owner = f.lane;
        cmd.target = target - f.before;
      }
    }
  }
  __syncwarp();
  if (lane == 0) s.walk = w;
  return cmd;
}

// A cluster takes a request.  Its first block reads the tree, the numbers and the sums of the rows with children and
// sends all of them to the others; then every block walks the tree (warp 0, all lanes alike), and where a refusal or
// the bonus token asks for a row's masses, each sums its part, a range of tokens a warp, and sends the sum to all. No
// block reads what decides from memory itself, so that all come to the same and no barrier can miss one.  Bound by
// the rounds' latencies (a single tree's round has 3 us of sums, as much for joining and deciding, 1 for the
// barrier), then by arithmetic (27 operations on pairs of floats a token and refusal).  With the first block alone
// deciding, and a second barrier a round for its command, 192 nodes took 52.5 us for 50 then, 64 chains 57.6 for 55.2.
// Asynchronous copies of a sum's next tokens to shared memory brought nothing.  Blocks of 512 threads, two an SM at
// 64 registers: an earlier form, 57 us for 192 nodes, took 64 with one an SM at 128, 61 with 1024 threads; four of
// 256 threads 55, but a single tree 27 for 23.  (72 bytes are spilled at 64 registers.)
__global__ void __launch_bounds__(kWalkThreads, 2) k_sample_walk(const __grid_constant__ SampleArgs a, int cluster) {
  __shared__ WalkShared s;
  cluster_arrive();  // a block's shared memory is written to only when the block runs
  // The rows' kernel has waited for all before it, so the tree and the numbers may be read while it runs.
  if (!a.rows_first) pdl_enter();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  const int r = blockIdx.x / cluster;
  const int64_t first = (int64_t)rank * kWalkWarps * a.range;  // the block's places
  const float2 root = kRoots[lane];

  // ---- the nodes, and the sums of the rows with children
  if (rank == 0) {
    int64_t off = 0;
    int n = 0;
    bool ok = sample_request(a, r, off, n);
    if (!ok) n = 0;
    const float T = a.temperature ? a.temperature[r] : 1.0f, u_bonus = fminf(fmaxf(a.u_bonus[r], 0.0f), 0.99999994f);
    const bool greedy = T < kGreedy;
    const Slope c = make_slope(greedy ? 1.0f : T);
    if (tid < kSampleMaxNodes / 32) s.inner[tid] = 0;
    __syncthreads();
    ok = ok && T >= 0.0f;
    // A row's largest logit and its sum.  (The first rows' are read with the tree; of those without children
    // nothing was written, and nothing is used.)
    auto row_sum = [&](int i) {
      const UnitStat* st = a.stat + (off + i) * a.units;
      constexpr int W = 6;  // loads of a lane on their way
      float most = -INFINITY;
      int32_t at = 0x7FFFFFFF;
      Pair sum{0.0f, 0.0f};
#pragma unroll 1
      for (int k0 = lane; k0 - lane < a.units; k0 += 32 * W) {
        UnitStat u[W];
        float top = most;
#pragma unroll
        for (int k = 0; k < W; ++k) {
          u[k] = k0 + 32 * k < a.units ? st[k0 + 32 * k] : UnitStat{-INFINITY, 0x7FFFFFFF, {0.0f, 0.0f}};
          top = fmaxf(top, u[k].most);
        }
        top = warp_max(top);
        const Ref ref = make_ref(top, c);
        if (top > most) {
          if (sum.h > 0.0f) sum = scaled(sum, make_ref(most, c), ref, c);
          most = top;
          at = 0x7FFFFFFF;
        }
#pragma unroll 1
        for (int k = 0; k < W; ++k) {
          const UnitStat v = u[0];
#pragma unroll
          for (int e = 1; e < W; ++e) u[e - 1] = u[e];  // (a loop's body once, with its registers named)
          if (v.most == most) at = min(at, v.at);
          if (v.sum[0] > 0.0f) sum = sum + scaled(Pair{v.sum[0], v.sum[1]}, make_ref(v.most, c), ref, c);
        }
      }
      at = __reduce_min_sync(0xFFFFFFFFu, at);
      sum = warp_sum(sum);
      if (lane == 0) {
        s.most[i] = most;
        s.at[i] = at;
        s.sum[i] = sum;
      }
    };
#pragma unroll 1
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
    if (a.rows_first) pdl_enter();
    if (warp < n && a.rows_first) row_sum(warp);
    if (a.rows_first) ok = ok && !*a.falls;
    ok = __syncthreads_and(ok);
    if (!ok && tid == 0) atomicOr(a.status, kSampleBadRequest);
    ok = ok && n > 0;
    if (!ok && tid == 0) a.path_len[r] = a.bonus[r] = -1;
#pragma unroll 1
    for (int i = warp + kWalkWarps; ok && i < n; i += kWalkWarps)
      if (s.inner[i >> 5] >> (i & 31) & 1u) row_sum(i);
    __syncthreads();
    if (ok && !greedy)
#pragma unroll 1
      for (int i0 = warp * 32; i0 < n; i0 += kWalkThreads) {
        // (a lane has a row of its own, so it takes the roots from memory)
        const int i = i0 + lane;
        if (i > 0 && i < n) s.mass[i] = mass1(s.mass[i].h, make_ref(s.most[s.parent[i]], c), c);
      }
    __syncthreads();
    cluster_wait();
    if (tid < cluster) send(Given{off, n, ok, c, u_bonus, greedy}, &s.given, (uint32_t)tid);
#pragma unroll 1
    for (int k = tid; ok && k < (n + 3) / 4 * Tree::kWords * (cluster - 1); k += kWalkThreads) {
      const int nth = k / (cluster - 1), four = nth / Tree::kWords, word = nth - four * Tree::kWords;
      if (word == 10 && four > (n - 1) / 128) continue;
      uint4* w = reinterpret_cast<uint4*>(reinterpret_cast<char*>(&s) + Tree::place(four, word));
      send(*w, w, (uint32_t)(1 + k - nth * (cluster - 1)));
    }
  } else {
    if (a.rows_first) pdl_enter();
    cluster_wait();
  }

  if (tid == 0) s.walk.stage = kStart;
  cluster_sync();
  const bool greedy = s.given.greedy;
  const Slope c = s.given.slope;
  int holder = -1;  // of the bonus token, and what find_token is told
  float most = 0.0f;
  Pair target{0.0f, 0.0f};
  int turn = 0;  // a block may send its next sums while another still reads the last ones
  while (true) {
    if (warp == 0) {
      const Command cmd = decide(a, s, s.total[turn], c, greedy, r, rank == 0, cluster);
      __syncwarp();
      if (lane == 0) s.cmd = cmd;
    }
    turn ^= 1;
    __syncthreads();
    if (s.cmd.op == kOpDone) break;
    const Row row = row_of(a, s.given.off + s.cmd.node);
    if (s.cmd.op == kOpFind) {
      holder = s.cmd.owner;
      most = s.cmd.most;
      target = s.cmd.target;
      break;
    }
    if (s.cmd.refused) {
      if (tid == 0) s.n_refused = 0;
      __syncthreads();
#pragma unroll 1
      for (int i = s.cmd.node + 1 + tid; i < s.given.n; i += kWalkThreads)
        if (s.parent[i] == s.cmd.node && s.draft[i] >= 0) s.refused[atomicAdd(&s.n_refused, 1)] = s.draft[i] + row.lo;
      __syncthreads();
    }
    const int64_t v0 = first + warp * a.range, v1 = min(row.hi, v0 + a.range);
    const int n_refused = s.cmd.refused ? s.n_refused : 0;
    const Total t = s.cmd.known ? sum_range(row, s.cmd, c, v0, v1, s.refused, n_refused, root)
                    : greedy    ? first_of_range(row, v0, v1)
                                : sum_unknown<4>(row, c, v0, v1, root);
    if (lane == 0) s.range[warp] = t;
    __syncthreads();
    const bool last = s.cmd.last, known = s.cmd.known;  // (behind the barrier the first warp goes on to the next command)
    if (warp == 0) {
      Pair part;
      const Total sum = join(s.range, kWalkWarps, c, greedy, known, part);
      if (lane < cluster) send(sum, &s.total[turn][rank], (uint32_t)lane);
    }
    cluster_sync();
    if (last) {  // every warp sees for itself which block holds the bonus token
      Pair mine;
      const Total all = join(s.total[turn], cluster, c, false, known, mine);
      if (all.sum.h > 0.0f) {
        target = all.sum * s.given.u_bonus;
        const Found f = find_lane<16>(mine, target);
        holder = f.lane;
        most = all.most;
        target = target - f.before;
        break;
      }
    }
  }
  if (holder == (int)rank) find_token(a, s, c, row_of(a, s.given.off + s.cmd.node), first, root, most, target, a.bonus + r);
}

int64_t sample_units(int64_t V) { return (V + 3 + kUnit - 1) / kUnit; }  // (a row's places start up to three early)

// Blocks of a request's cluster: as many as still leave all requests' clusters room at the same time, and 2048
// tokens or more a block.  (With room for a part of them the others start when those end: 24 requests at 16 blocks took
// 98 us where 4 took 80, both in an earlier form.  24 requests have room for clusters of 10: 52.5 us, 8 took 55.)
int cluster_size(int32_t n_req, int64_t V, int& size) {
  static std::mutex mu;  // (a host thread that saw a part of the table would take smaller clusters)
  static int room[64][kMaxCluster + 1] = {{0}};  // clusters of a size that a device holds at once
  int dev = 0;
  W12_CUDA_TRY(cudaGetDevice(&dev));
  size = 1;
  if (dev >= 64) return W12_OK;
  std::lock_guard<std::mutex> lk(mu);
  if (!room[dev][1]) {
    W12_CUDA_TRY(cudaFuncSetAttribute(k_sample_walk, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
    for (int blocks = kMaxCluster; blocks; --blocks) {
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = (unsigned)blocks;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)blocks);
      cfg.blockDim = dim3(kWalkThreads);
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int n = 0;
      W12_CUDA_TRY(cudaOccupancyMaxActiveClusters(&n, k_sample_walk, &cfg));
      room[dev][blocks] = n > 0 ? n : blocks == 1;
    }
  }
  for (size = kMaxCluster; size > 1 && (room[dev][size] < n_req || V <= size * (int64_t)2048);) --size;
  return W12_OK;
}

}  // namespace
}  // namespace w12

using namespace w12;

extern "C" {

size_t tree_verify_sampled_workspace_size(int64_t M, int64_t V) {
  if (M < 1 || V < 1) return 0;
  return 16 + (size_t)M * (size_t)sample_units(V) * sizeof(UnitStat);
}

int tree_verify_sampled(const float* logits, int64_t stride, int64_t M, int64_t V, const float* draft_probs,
                        int64_t probs_stride, const int32_t* parent, const int32_t* draft, const int32_t* req_offsets,
                        int32_t n_req, const float* u, const float* u_bonus, const float* temperature, int32_t* path_len,
                        int32_t* path_nodes, int32_t* bonus, int32_t* status, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "tree_verify_sampled";
  if (M < 1 || M > 65535 * (int64_t)kStatTile || V < 1 || V > 0x7FFFFFF0 || stride < V || (draft_probs && probs_stride < V) || n_req < 1 ||
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
  int cluster = 1;
  const int st = cluster_size(n_req, V, cluster);
  if (st) return st;
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
  a.falls = static_cast<int32_t*>(ws);
  a.stat = reinterpret_cast<UnitStat*>(static_cast<char*>(ws) + 16);
  a.units = (int32_t)sample_units(V);
  const int64_t warps = (int64_t)cluster * kWalkWarps;
  a.range = ((V + 3 + warps - 1) / warps + 127) / 128 * 128;
  a.n_req = n_req;
  a.rows_first = M > 1 || n_req > 1;
  if (a.rows_first) {
    // three blocks an SM, if there is that much (half of the nodes have children, or nearly all)
    const int64_t tiles = (M + kStatTile - 1) / kStatTile, most = (M < kStatTile ? M : kStatTile) * (int64_t)a.units;
    int64_t blocks = (most + kStatThreads / 32 - 1) / (kStatThreads / 32);
    blocks = blocks < 456 ? blocks : 456;
    W12_CUDA_TRY(launch_dependent(draft_probs ? k_sample_stats<true> : k_sample_stats<false>,
                                  dim3((unsigned)blocks, (unsigned)tiles), kStatThreads, 0, (cudaStream_t)stream, a));
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
