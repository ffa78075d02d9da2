// w12_attn.cu - attention of draft-tree nodes over a paged cache and their ancestors.
//
// For one cache head, the rows (node, query head of the group) of a request share every
// key: R = nodes * group rows, cut into units of 128 or 256, meet T = ceil((len + n) / BK)
// tiles of keys, the n drafted nodes standing behind the len cached tokens.  A CTA takes
// an equal, contiguous share of all units' tiles (one CTA per SM); a unit that falls
// into several shares leaves its parts (running reference, sum, unnormalised output) in
// the workspace, and a second kernel adds them in order, so the bits do not depend on
// who came first.
//
// Inside a CTA the score and output products run on the tensor core (tcgen05):
//   S = Q K^T   both operands in shared memory, 128 rows x BK keys, float in tensor memory;
//   P = exp2(S c - m) by one thread per row and half of the keys, over S in tensor memory;
//   O += P V    P from tensor memory, V as it lies in shared memory (keys x columns).
// The reference m follows the running maximum only when it has fallen more than 2^8
// behind, so O is rarely rescaled; any reference gives the same quotient.  Roles: eight
// softmax warps, four producer warps that keep a ring of K and V tiles filled across units, one warp
// that issues the scores and one that issues the outputs.
//
// Per 128 keys of a head with D = 128, an SM's share of the memory rate is about 2800 cycles
// (64 KB), its two products 1560 (24 of 65 cycles), its exponentials 1024, a step of the softmax
// 2200: the kernel is bound by the cache's bytes up to 128 rows, whose padding costs
// nothing, and a step takes about 3100 cycles.  Both softmax warpgroups work on the same
// tile, half of its keys each (they share the row's lanes of tensor memory and exchange the
// halves' maxima), so that scores computed ahead wait for no product.  Above 128 rows (D <=
// 128) a tile of keys meets two tiles of rows in turn, with an O each, so K and V are read
// once for 256 rows.  D = 256 has room for one O: 128 rows, tiles of 64 keys; more rows read
// K and V again, from L2 (the units of all heads follow one another for each 128 rows,
// so the shares of two 128-row halves run over the same keys at the same time).
//
// Measured on one GB300, kernel and join, back to back: 24 requests of 33 to 12001 tokens, 192
// nodes, 40 heads on 8 of 128: 119 us for 617 MB (5.2 TB/s, 0.77 of the measured copy rate); 16
// nodes over 65535 tokens 61 us (4.4 TB/s); 32 nodes over 131071 tokens, 24 heads on 4 of 256: 148
// us (0.70 PFLOP/s); 16 nodes over 8191 tokens 21 us, one node over 711 tokens 12 us, of which a
// launch, the chain length -> table -> keys -> scores, a last product and the join are
// about 10.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "w12_internal.cuh"
#include "w12_pdl.cuh"

namespace w12 {

int check_cache(const kv_cache* c, const char* fn);

namespace {

constexpr int kAttnMaxNodes = 256;
constexpr int32_t kAttnBadRequest = 1, kAttnBadBlock = 2, kAttnTimeout = 4;
constexpr int kAttnCtas = 152;  // one per SM of a GB300; fewer SMs only run them in turn
// What a unit costs beside its tiles (its last product, its outputs, the next one's first scores), in
// tiles; the shares count it in front of the unit.  24 requests of 33 to 12001 tokens took 143 us
// at 0, 130 at 1, 118 at 2 and 118 at 3.
constexpr int kUnitCost = 2;
constexpr int kMetaRing = 2;     // units whose tree shared memory holds
// P enters its product in two bf16 pieces, the upper one cut off, the lower one rounded: 2^-16
// of P is lost instead of 2^-8.  The lower piece is taken of P (1 + 2^-20), so that it is above
// zero wherever P is and an infinity in V stays one (no 0 * inf, no inf - inf).
constexpr float kUp = 1.0f + 1.0f / 1048576.0f;
constexpr float kRefSlack = 8.0f;  // log2 of the largest P before the reference moves

// Division of numbers below 2^31 by a divisor up to 2^24: floor(n * mul / 2^shift), mul =
// ceil(2^shift / d), shift = 31 + ceil(log2 d); the excess n (mul d - 2^shift) stays below 2^shift.
struct FastDiv {
  uint32_t mul, shift;
  __device__ __forceinline__ int32_t operator()(int32_t n) const { return (int32_t)(((uint64_t)(uint32_t)n * mul) >> shift); }
};

FastDiv fast_div(int64_t d) {
  FastDiv f{0, 31};
  while ((int64_t)1 << (f.shift - 31) < d) ++f.shift;
  f.mul = (uint32_t)((((uint64_t)1 << f.shift) + (uint64_t)d - 1) / (uint64_t)d);
  return f;
}

struct AttnArgs {
  const uint16_t *q, *k, *v, *kc, *vc;
  int64_t q_stride, k_stride, v_stride, M;
  int64_t block_stride, token_stride, head_stride, n_blocks;
  const int32_t *table, *cache_len, *parent, *req_offsets;
  int64_t table_stride, table_width;
  int32_t n_req, block_size, group, n_heads, n_q_heads, row_cap;
  FastDiv by_block, by_group;
  int32_t box_rows;  // tokens of a box of the tensor maps; 0: rows are copied by the threads
  uint32_t wait_cycles;  // bound of a wait
  float scale_log2;  // scale * log2(e)
  uint16_t* out;
  int32_t* status;
  float *part_o, *part_ml;  // [2 * CTAs][D / 4][row_cap][4], [2 * CTAs][row_cap][2]
  int32_t* part_bad;        // [2 * CTAs]
  struct JoinUnit* units;   // [CTAs]: the unit inside which a CTA's share begins
};

template <int D>
struct AttnPlan {
  static constexpr int kRowTiles = D <= 128 ? 2 : 1;
  static constexpr int kRows = 128 * kRowTiles;      // rows of a unit
  static constexpr int kBK = D <= 128 ? 128 : 64;    // keys of a tile
  static constexpr int kSlots = D == 64 ? 10 : 5;    // tiles of the ring
  static constexpr int kSB = D <= 128 ? 3 : 4;       // score buffers in tensor memory
  static constexpr int kSlotBytes = kBK * D * 2;
  static constexpr int kSoftmaxThreads = 256;
  static constexpr int kThreads = kSoftmaxThreads + 128 + 64;  // + producers + the two product warps
  static constexpr int kQ = 0;
  static constexpr int kQTile = 128 * D * 2;
  static constexpr int kRing = kQ + kRowTiles * kQTile;
  static constexpr int kX = kRing + kSlots * kSlotBytes;       // what the halves exchange: 2 x 2 x 128 floats
  static constexpr int kPar = kX + 2 * 2 * 128 * 4;            // parents, kMetaRing x 256 bytes
  static constexpr int kNf = kPar + kMetaRing * kAttnMaxNodes; // nodes with infinities or NaN in V, kMetaRing x 8 words
  static constexpr int kBad = kNf + kMetaRing * 32;            // kMetaRing words
  static constexpr int kMisc = kBad + kMetaRing * 4;           // tensor memory address, abort, schedule
  static constexpr int kBar = (kMisc + 16 + 7) & ~7;
  static constexpr int kBytes = kBar + 8 * (2 * kSlots + 3 * kSB + 6 + kMetaRing + 4);
  static_assert(kBytes <= 227 * 1024, "shared memory plan too large");
  static_assert(kThreads * 8 <= kSlots * kSlotBytes, "the ring holds the schedule's sums");
  // Tensor memory columns: O of the first tile of rows, then D <= 128: three score buffers, of
  // which the first gives way to the second O where a unit has two tiles of rows; D = 256:
  // four of 64 columns.
  static constexpr int kO1 = 128, kS0 = D <= 128 ? 128 : 256, kSCols = kBK;
};

// What the joining kernel has to know of a unit that several CTAs share.
struct JoinUnit {
  int64_t off;              // the request's first node
  int32_t h, row0, rows;    // rows = 0: the CTA's share begins with a unit
  int32_t first, last;      // the CTAs whose shares begin inside it
  int32_t pad;
};

// ---------------------------------------------------------------- schedule

struct Req {
  int64_t off;
  int32_t n, len, tiles, row_units;  // tiles: of a unit, its cost in front included
  bool ok;
};

template <int D>
__device__ __forceinline__ Req load_request(const AttnArgs& a, int r) {
  using P = AttnPlan<D>;
  Req q{0, 0, 0, 0, 0, true};
  q.off = a.req_offsets ? a.req_offsets[r] : 0;
  const int64_t end = a.req_offsets ? a.req_offsets[r + 1] : a.M, n = end - q.off;
  const int64_t len = a.cache_len[r], most = a.table_width * a.block_size;
  if (q.off < 0 || n < 0 || end > a.M || n > kAttnMaxNodes || len < 0 || len > most || len > 0x7FFFFFFF - 1024) {
    q.ok = false;
    return q;
  }
  q.n = (int32_t)n;
  q.len = (int32_t)len;
  if (n == 0) return q;
  q.tiles = (q.len + q.n + P::kBK - 1) / P::kBK + kUnitCost;
  q.row_units = (q.n * a.group + P::kRows - 1) / P::kRows;
  return q;
}

// Quotient of two non-negative numbers, in 32 bits where they allow it.
__device__ __forceinline__ int64_t quotient(int64_t n, int64_t d) {
  return ((n | d) >> 32) == 0 ? (int64_t)((uint32_t)n / (uint32_t)d) : n / d;
}
__device__ __forceinline__ int64_t share(int64_t total, int ctas, int c) { return quotient(total * c, ctas); }

struct Start {
  int64_t total, at;  // all tiles; the place of the wanted tile within its request
  int32_t r, ctas;
};

// Total number of tiles and, for CTA c of the grid, the request in which its share begins.  Every
// thread of the block calls this.  Up to 32 requests each warp finds it for itself, without a
// barrier; more take the whole block (scratch: 2 + threads / 32 int64 of shared memory).
template <int D>
__device__ __forceinline__ Start find_start(const AttnArgs& a, int c, int64_t* scratch) {
  constexpr int threads = AttnPlan<D>::kThreads, warps = threads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool small = a.n_req <= 32;
  int64_t mine = 0, sum = 0;
  for (int r = small ? lane : tid; r < a.n_req; r += threads) {
    const Req q = load_request<D>(a, r);
    if (!q.ok && c == 0) atomicOr(a.status, kAttnBadRequest);
    mine = (int64_t)q.tiles * q.row_units * a.n_heads;
    sum += mine;
  }
  Start s{0, 0, 0, 0};
  int64_t v = small ? mine : sum;
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += u;
  }
  if (small) {
    s.total = __shfl_sync(0xFFFFFFFFu, v, 31);
    s.ctas = (int32_t)(s.total < kAttnCtas ? s.total : kAttnCtas);
    if (c >= s.ctas) return s;
    const int64_t want = share(s.total, s.ctas, c);
    s.r = __ffs((int)__ballot_sync(0xFFFFFFFFu, want < v)) - 1;  // want < total: some lane says yes
    s.at = want - __shfl_sync(0xFFFFFFFFu, v - mine, s.r);
    return s;
  }
  if (lane == 31) scratch[2 + warp] = v;
  __syncthreads();
  for (int w = 0; w < warps; ++w) s.total += scratch[2 + w];
  s.ctas = (int32_t)(s.total < kAttnCtas ? s.total : kAttnCtas);
  if (c >= s.ctas) return s;
  const int64_t want = share(s.total, s.ctas, c);
  int64_t carry = 0;
  for (int r0 = 0; r0 < a.n_req; r0 += threads) {
    const int r = r0 + tid;
    int64_t w = 0;
    if (r < a.n_req) {
      const Req q = load_request<D>(a, r);
      w = (int64_t)q.tiles * q.row_units * a.n_heads;
    }
    v = w;
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += u;
    }
    __syncthreads();
    if (lane == 31) scratch[2 + warp] = v;
    __syncthreads();
    int64_t before = carry + v - w;
    for (int i = 0; i < warps; ++i) {
      if (i < warp) before += scratch[2 + i];
      carry += scratch[2 + i];
    }
    if (want >= before && want < before + w) {
      scratch[0] = r;
      scratch[1] = want - before;
    }
    if (want < carry) break;
  }
  __syncthreads();
  s.r = (int32_t)scratch[0];
  s.at = scratch[1];
  return s;
}

// The parts of a CTA's share, in order.  Every role of the CTA walks them for itself.
struct Part {
  Req q;
  int32_t r, h, row0, rows;  // rows row0 .. row0 + rows - 1 of the request's nodes * group
  int32_t ta, tb;            // tiles
  int64_t begin;             // place of the unit's first tile among its request's
};

template <int D>
struct Walk {
  int64_t at, left;
  int32_t r;
  bool fresh;
  Req q;

  __device__ __forceinline__ Walk(const Start& s, int c)
      : at(s.at), left(c < s.ctas ? share(s.total, s.ctas, c + 1) - share(s.total, s.ctas, c) : 0), r(s.r), fresh(true) {}

  // The next part with tiles; false at the share's end.
  __device__ __forceinline__ bool next(const AttnArgs& a, Part& p) {
    while (left > 0) {
      if (fresh) {
        while ((q = load_request<D>(a, r)).tiles == 0) ++r;  // left > 0: a request with tiles follows
        fresh = false;
      }
      const int64_t u = quotient(at, q.tiles), row_unit = quotient(u, a.n_heads);
      const int32_t ta = (int32_t)(at - u * q.tiles), take = (int32_t)min(left, (int64_t)(q.tiles - ta));
      p.q = q;
      p.r = r;
      p.ta = max(ta - kUnitCost, 0);
      p.tb = max(ta + take - kUnitCost, 0);
      p.begin = at - ta + kUnitCost;
      p.h = (int32_t)(u - row_unit * a.n_heads);
      p.row0 = (int32_t)row_unit * AttnPlan<D>::kRows;
      p.rows = min(AttnPlan<D>::kRows, q.n * a.group - p.row0);
      at += take;
      left -= take;
      if (at == (int64_t)q.tiles * q.row_units * a.n_heads) {
        ++r;
        at = 0;
        fresh = true;
      }
      if (p.tb > p.ta) return true;
    }
    return false;
  }
};

// ---------------------------------------------------------------- PTX

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void cp_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// 32 lanes x 32 columns, on their way; tmem_wait32 makes them readable (and waits for every
// load before it).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t r[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
      "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait32(uint32_t r[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t r[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Products issued by one elected thread of a converged warp: the operands are then the warp's and
// come from uniform registers.  64 back-to-back products of 128 x 64 x 16 took 32 cycles each this
// way and 62 from inside a branch to one thread.
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}
// A from tensor memory.
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void umma_commit_one(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar)
      : "memory");
}

// Shared-memory descriptor of V as the second operand of O = P V: rows are keys, 64 columns
// (128 bytes, swizzled) each; 8 keys are 1024 bytes apart, the next 64 columns `slab` bytes.
__device__ __forceinline__ uint64_t umma_desc_v(uint32_t saddr, uint32_t slab) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(slab >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
constexpr uint32_t kTransposeB = 1u << 16;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Pairs of floats, one instruction for both.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpair(uint64_t x, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// A box of the cache: 64 columns x box_rows tokens of one head of one block, swizzled as it lands.
__device__ __forceinline__ void box_load(uint32_t dst, const CUtensorMap* map, int col, int token, int head, int block,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(map), "r"(col), "r"(token), "r"(head), "r"(block), "r"(bar)
      : "memory");
}

// ---------------------------------------------------------------- the kernel

struct Shared {
  uint32_t base;         // shared-memory address of the block
  uint8_t* sm;
  volatile int32_t* abort;
  uint32_t limit;        // cycles of a wait
  uint32_t full, empty, q_full, q_free, s_full, p_full, o_done, unit_end, meta, reset, drain, pair;
};

// A bounded wait; one that runs out stops every role of the CTA.  The hardware suspends the thread
// in a try_wait for longer than a tile takes, so only waits that are stuck reach the slow path.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int32_t* abort, uint32_t limit) {
  const long long start = clock64();
  bool done;
  do {
    done = mbar_try_wait(bar, parity);
    if (*abort) return false;
    if (clock64() - start > limit) {  // also where the phase came, late
      *abort = 1;
      return false;
    }
  } while (!done);
  return true;
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, const Shared& s) {
  if (mbar_try_wait(bar, parity)) return true;
  return wait_slow(bar, parity, s.abort, s.limit);
}
// The same answer for the whole warp, whose next steps (tensor memory accesses, shuffles) take
// all of its threads.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const Shared& s) {
  return __all_sync(0xFFFFFFFFu, wait(bar, parity, s));
}
// The same with all of its time against the limit, the hardware's suspension too: for the wait that
// always takes some time, the one for a tile's probabilities.
__device__ __forceinline__ bool wait_warp_timed(uint32_t bar, uint32_t parity, const Shared& s) {
  return __all_sync(0xFFFFFFFFu, mbar_test_wait(bar, parity) || wait_slow(bar, parity, s.abort, s.limit));
}

// Which tile the item-th ring entry of a part holds, in the order in which they are
// taken.  Rows in two halves: K0 V0 K1 V1 ...; tiles in turn: K0 K1 V0 K2 V1 ... V(n-1).
__device__ __forceinline__ int ring_tile(int item, int cnt, bool two, bool& is_v) {
  if (two) {
    is_v = item & 1;
    return item >> 1;
  }
  if (item == 2 * cnt - 1) {
    is_v = true;
    return cnt - 1;
  }
  if (item < 2) {
    is_v = false;
    return item;
  }
  is_v = !(item & 1);
  return is_v ? (item - 2) >> 1 : (item + 1) >> 1;
}

template <int D>
__device__ bool produce(const AttnArgs& a, const CUtensorMap* k_map, const CUtensorMap* v_map, const Shared& s,
                        Walk<D> walk) {
  using P = AttnPlan<D>;
  constexpr int CPR = D / 8;              // 16-byte chunks of a row
  constexpr int RPW = 32 / CPR;           // rows a warp copies at once
  constexpr int IT = P::kBK / (4 * RPW);  // rounds of a tile
  const int pt = (int)threadIdx.x - P::kSoftmaxThreads, pw = pt >> 5, lane = pt & 31;
  const int chunk = lane % CPR, sub = lane / CPR;
  uint32_t entry = 0;  // ring entries so far
  Part p;
  for (int unit = 0; walk.next(a, p); ++unit) {
    const int ring = unit & 1, cnt = p.tb - p.ta;
    const bool two = P::kRowTiles == 2 && p.rows > 128;
    uint32_t* nf = reinterpret_cast<uint32_t*>(s.sm + P::kNf) + ring * 8;
    int32_t* bad = reinterpret_cast<int32_t*>(s.sm + P::kBad) + ring;
    bool bad_block = false;
    const int32_t* table = a.table + p.r * a.table_stride;
    const int64_t head_off = (int64_t)p.h * a.head_stride;
    // Lane L finds the row that the warp copies in round L / RPW as its (L % RPW)-th: its block (a
    // load that is on its way while the entries before are copied), then its place in the cache,
    // for K and V alike.  Where a tile can go by boxes of the tensor maps, lane L sends for the 4 L + warp-th.
    const int my_row = (lane / RPW) * 4 * RPW + pw * RPW + lane % RPW;
    const int boxes = a.box_rows ? P::kBK / a.box_rows : 1, my_box = (lane * 4 + pw) % boxes, my_slab = (lane * 4 + pw) / boxes;
    auto find_block = [&](int tile, int row) -> int32_t {
      const int32_t j = tile * P::kBK + row;
      return row < P::kBK && j < p.q.len ? table[a.by_block(j)] : 0;
    };
    auto is_tail = [&](int tile) { return (int64_t)(tile + 1) * P::kBK > p.q.len; };  // it holds drafted nodes
    auto asked_row = [&](int tile) { return a.box_rows && !is_tail(tile) ? my_box * a.box_rows : my_row; };
    auto find_place = [&](int tile, int32_t id) -> int64_t {  // -1: not in the cache
      const int32_t j = tile * P::kBK + my_row;
      if (my_row >= P::kBK) return 0;
      if (j >= p.q.len) return -1;
      if ((uint32_t)id >= (uint64_t)a.n_blocks) {
        bad_block = true;
        return -1;
      }
      return (int64_t)id * a.block_stride + (int64_t)(j - a.by_block(j) * a.block_size) * a.token_stride + head_off;
    };
    int64_t place0 = 0, place1 = 0;  // of the tiles whose K is under way and whose V is not, oldest first
    bool waiting = false;
    int32_t id = find_block(p.ta, asked_row(p.ta));
    for (int item = 0; item < 2 * cnt; ++item, ++entry) {
      bool is_v;
      const int i = ring_tile(item, cnt, two, is_v), tile = p.ta + i;
      const bool tail = is_tail(tile), by_box = a.box_rows && !tail;
      int64_t at;
      if (is_v) {
        at = place0;
        place0 = place1;
        waiting = !two && item < 2 * cnt - 1;  // K0 K1 V0 K2 V1 ...: one tile stays behind
      } else {
        if (by_box) {
          const bool in = (uint32_t)id < (uint64_t)a.n_blocks;
          bad_block = bad_block || !in;
          at = in ? id : 0;  // some block: the unit's outputs are dropped
        } else {
          at = find_place(tile, id);
        }
        const int next = p.ta + min(i + 1, cnt - 1);
        id = find_block(next, asked_row(next));
        if (waiting) place1 = at;
        else place0 = at;
        waiting = true;
      }
      const uint32_t slot = entry % P::kSlots, round = entry / P::kSlots;
      if (round > 0 && !wait_warp(s.empty + 8 * slot, (round - 1) & 1, s)) return false;
      const uint32_t dst = s.base + P::kRing + slot * P::kSlotBytes;
      // Before the arrivals of the part's last entry, behind which the softmax reads it.
      if (item == 2 * cnt - 1 && bad_block) {
        atomicOr(bad, kAttnBadBlock);
        __threadfence_block();
      }
      if (by_box) {
        const uint32_t bar = s.full + 8 * slot;
        if (my_slab < D / 64) {
          const int32_t j = tile * P::kBK + my_box * a.box_rows;
          mbar_arrive_expect_tx(bar, a.box_rows * 128);
          box_load(dst + my_slab * (P::kBK * 128) + my_box * a.box_rows * 128, is_v ? v_map : k_map, my_slab * 64,
                   j - a.by_block(j) * a.block_size, p.h, (int)at, bar);
        } else {
          mbar_arrive(bar);
        }
      } else {
        const uint16_t* mine = nullptr;  // the lane's row; none: zeros
        const int32_t node = tile * P::kBK + my_row - p.q.len;
        if (at >= 0) mine = (is_v ? a.vc : a.kc) + at;
        else if (node >= 0 && node < p.q.n)
          mine = (is_v ? a.v + (p.q.off + node) * a.v_stride : a.k + (p.q.off + node) * a.k_stride) + (int64_t)p.h * D;
#pragma unroll
        for (int i0 = 0; i0 < IT; i0 += 8) {
          unsigned long long o[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] = __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(mine), (i0 + k) * RPW + sub);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int row = (i0 + k) * 4 * RPW + pw * RPW + sub;
            cp16(dst + (chunk >> 3) * (P::kBK * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4),
                 o[k] ? reinterpret_cast<const uint16_t*>(o[k]) + chunk * 8 : a.kc, o[k] != 0);
          }
        }
      }
      if (item == 0) {
        // ---- the unit's query rows (past them shared memory stays as it is) and its tree, behind
        // the first keys.  The last unit's scores are there and the one before it is at its end:
        // the rows of the one and the tree of the other may go.
        if (unit > 0 && !wait_warp(s.q_free, (unit - 1) & 1, s)) return false;
        for (int row0 = 0; row0 < p.rows; row0 += P::kBK) {
          const int r = p.row0 + row0 + my_row, node = a.by_group(r);
          const int64_t o = (p.q.off + node) * a.q_stride + (int64_t)(p.h * a.group + r - node * a.group) * D;
          for (int it = 0; it < IT && row0 + it * 4 * RPW < p.rows; ++it) {
            const int row = row0 + it * 4 * RPW + pw * RPW + sub;
            const int64_t from = __shfl_sync(0xFFFFFFFFu, o, it * RPW + sub);
            if (row < p.rows)
              cp16(s.base + P::kQ + (row >> 7) * P::kQTile + (chunk >> 3) * 16384 + (row & 127) * 128 +
                       (((chunk & 7) ^ (row & 7)) << 4),
                   a.q + from + chunk * 8);
          }
        }
        if (pt < 8) nf[pt] = 0;
        if (pt == 8) *bad = 0;
        mbar_arrive(s.reset);
        if (!wait_warp(s.reset, unit & 1, s)) return false;
        if ((int64_t)p.tb * P::kBK > p.q.len) {
          uint8_t* par = s.sm + P::kPar + ring * kAttnMaxNodes;
          for (int n = pt; n < p.q.n; n += 128) {
            const int32_t x = a.parent[p.q.off + n];
            const bool in = n == 0 ? x == -1 : x >= 0 && x < n;
            par[n] = in && n ? (uint8_t)x : (uint8_t)255;  // 255: no parent
            if (!in) atomicOr(bad, kAttnBadRequest);
          }
        }
        mbar_arrive(s.meta + 8 * ring);
        cp_arrive(s.q_full);
      }
      if (by_box) {  // (its arrivals went with the boxes)
      } else if (tail && is_v) {
        // A tile with drafted nodes: an infinity or a NaN in a node's V would reach every row
        // (0 * inf), also those that do not attend to it.  It is taken out here, the node
        // marked, and the rows that do attend to it get it back at the end.
        cp_wait_all();
        const int32_t from = p.q.len - tile * P::kBK;  // the first node's row
        for (int it = max(from, 0) / (4 * RPW); it < IT && it * 4 * RPW < from + p.q.n; ++it) {
          const int row = it * 4 * RPW + pw * RPW + sub;
          const int32_t node = tile * P::kBK + row - p.q.len;
          if (node < 0 || node >= p.q.n) continue;
          const uint32_t at = dst + (chunk >> 3) * (P::kBK * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
          const uint4 x = lds128(at);
          uint32_t w[4] = {x.x, x.y, x.z, x.w};
          bool found = false;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if ((w[i] & 0x7F80u) == 0x7F80u) w[i] &= 0xFFFF0000u, found = true;
            if ((w[i] & 0x7F800000u) == 0x7F800000u) w[i] &= 0xFFFFu, found = true;
          }
          if (found) {
            sts128(at, w[0], w[1], w[2], w[3]);
            atomicOr(&nf[node >> 5], 1u << (node & 31));
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(s.full + 8 * slot);
      } else {
        cp_arrive(s.full + 8 * slot);
      }
    }
  }
  return true;
}

// A step of a unit is a tile of keys and a tile of rows: with one tile of rows, step x takes tile x
// and score buffer x % kSB; with two, tile x / 2 and buffer 1 + x % 2.  Two warps issue the products,
// the scores' and the outputs', each waiting only for what its own need (in one warp the two
// chains of waits and issues added up to 2900 cycles a step, more than the memory's 2800).
// A ring entry is waited for by the one warp that takes it.  The entry before it in the same slot may
// be the other warp's, and has then been taken: the scores of a buffer come after the output
// before them, and an output after its scores.
struct Steps {
  int b;
  bool two;
  __device__ __forceinline__ explicit Steps(bool two_) : b(two_ ? 1 : 0), two(two_) {}
  __device__ __forceinline__ void next(int buffers) { b = two ? 3 - b : b + 1 < buffers ? b + 1 : 0; }
};

// Place of a tile's K or V among a part's ring entries (the inverse of ring_tile).
__device__ __forceinline__ int ring_item(int tile, bool is_v, int cnt, bool two) {
  if (two) return 2 * tile + is_v;
  if (is_v) return tile == cnt - 1 ? 2 * cnt - 1 : 2 * tile + 2;
  return tile < 2 ? tile : 2 * tile - 1;
}

template <int D>
__device__ __forceinline__ bool take_entry(const Shared& s, uint32_t entry, uint32_t& addr, uint32_t& slot) {
  using P = AttnPlan<D>;
  slot = entry % P::kSlots;
  addr = s.base + P::kRing + slot * P::kSlotBytes;
  if (!wait_warp(s.full + 8 * slot, (entry / P::kSlots) & 1, s)) return false;
  fence_proxy_async_smem();  // the copies of other threads, before the tensor core reads them
  return true;
}

template <int D>
__device__ bool issue_scores(const AttnArgs& a, const Shared& s, Walk<D> walk, uint32_t tmem) {
  using P = AttnPlan<D>;
  constexpr uint32_t kId = umma_idesc_n(P::kBK);
  uint32_t entry = 0, slot = 0, k_addr = 0;
  uint32_t used = 0, o_par = 0;  // per score buffer: scores before, parity of the output after them
  bool had_two = false;
  Part p;
  for (int unit = 0; walk.next(a, p); ++unit) {
    const int cnt = p.tb - p.ta;
    const bool two = P::kRowTiles == 2 && p.rows > 128;
    const int steps = two ? 2 * cnt : cnt;
    if (!wait_warp(s.q_full, unit & 1, s)) return false;
    // the second O and score buffer 0 share their columns
    bool ended = unit == 0;
    if (had_two && !two && !(ended = wait_warp(s.unit_end, (unit - 1) & 1, s))) return false;
    had_two = two;
    Steps at(two);
    for (int x = 0; x < steps; ++x, at.next(P::kSB)) {
      const int row_tile = two ? x & 1 : 0;
      // The scores overwrite the P of an earlier product.  Products with different results are not
      // ordered among themselves, so that product has to have ended.
      if (used >> at.b & 1u) {
        if (!wait_warp(s.o_done + 8 * at.b, o_par >> at.b & 1u, s)) return false;
        o_par ^= 1u << at.b;
      }
      used |= 1u << at.b;
      if (!row_tile && !take_entry<D>(s, entry + ring_item(two ? x >> 1 : x, false, cnt, two), k_addr, slot)) return false;
      tc_fence_after();
      const uint32_t q_addr = s.base + P::kQ + row_tile * P::kQTile, d = tmem + P::kS0 + at.b * P::kSCols;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        umma_ss(d, umma_desc(q_addr + (ks >> 2) * 16384 + (ks & 3) * 32),
                umma_desc(k_addr + (ks >> 2) * (P::kBK * 128) + (ks & 3) * 32), kId, ks > 0);
      // The last unit's end is waited for before this unit's last scores are handed over: without them this
      // unit cannot end, so its end is never taken for the last one's.  (The products are on their way.)
      if (x == steps - 1 && !ended && !wait_warp(s.unit_end, (unit - 1) & 1, s)) return false;
      umma_commit_one(s.s_full + 8 * at.b);
      if (!two || row_tile) umma_commit_one(s.empty + 8 * slot);
    }
    umma_commit_one(s.q_free);  // (not before the last unit's end: its tree goes with the query rows)
    entry += 2 * cnt;
  }
  return true;
}

template <int D>
__device__ bool issue_outputs(const AttnArgs& a, const Shared& s, Walk<D> walk, uint32_t tmem) {
  using P = AttnPlan<D>;
  constexpr uint32_t kId = umma_idesc_n(D) | kTransposeB;
  uint32_t entry = 0, slot = 0, v_addr = 0, p_par = 0;
  Part p;
  for (int unit = 0; walk.next(a, p); ++unit) {
    const int cnt = p.tb - p.ta;
    const bool two = P::kRowTiles == 2 && p.rows > 128;
    const int steps = two ? 2 * cnt : cnt;
    if (unit > 0 && !wait_warp(s.unit_end, (unit - 1) & 1, s)) return false;  // the last unit's outputs have been read
    Steps at(two);
    for (int x = 0; x < steps; ++x, at.next(P::kSB)) {
      const int row_tile = two ? x & 1 : 0, tile = two ? x >> 1 : x;
      if (!wait_warp_timed(s.p_full + 8 * at.b, p_par >> at.b & 1u, s)) return false;
      p_par ^= 1u << at.b;
      if (!row_tile && !take_entry<D>(s, entry + ring_item(tile, true, cnt, two), v_addr, slot)) return false;
      tc_fence_after();
      const uint32_t d = tmem + row_tile * P::kO1, a0 = tmem + P::kS0 + at.b * P::kSCols;
#pragma unroll
      for (int ks = 0; ks < P::kBK / 16; ++ks) {  // 32 keys: 16 columns of upper pieces, 16 of lower ones
        const uint32_t p_addr = a0 + (ks >> 1) * 32 + (ks & 1) * 8;
        const uint64_t v_desc = umma_desc_v(v_addr + ks * 2048, P::kBK * 128);
        umma_ts(d, p_addr, v_desc, kId, tile > 0 || ks > 0);
        umma_ts(d, p_addr + 16, v_desc, kId, 1);
      }
      umma_commit_one(s.o_done + 8 * at.b);
      if (!two || row_tile) umma_commit_one(s.empty + 8 * slot);
    }
    entry += 2 * cnt;
  }
  return true;
}

template <int D>
__device__ bool softmax(const AttnArgs& a, const Shared& s, Walk<D> walk, uint32_t tmem, int c) {
  using P = AttnPlan<D>;
  constexpr int NC = P::kBK / 2, CH = NC / 32;  // keys of a thread in a tile, in chunks of 32
  constexpr int NW = P::kBK / 32;
  // warpgroup (the half of a tile's keys), tensor memory lane, and the quarter of the lanes
  const int g = threadIdx.x >> 7, lane_row = threadIdx.x & 127, quarter = lane_row >> 5;
  const uint32_t lane_base = tmem + ((uint32_t)quarter << 21);
  volatile float* xs = reinterpret_cast<volatile float*>(s.sm + P::kX);
  uint32_t x_count = 0, s_par = 0, o_par = 0;
  // The value that the thread of the other half has for the same row.
  auto exchange = [&](float mine, float& other) {
    volatile float* x = xs + (x_count & 1) * 256 + lane_row;
    x[g * 128] = mine;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(s.pair + 8 * quarter);
    if (!wait_warp(s.pair + 8 * quarter, x_count & 1, s)) return false;
    other = x[(g ^ 1) * 128];
    ++x_count;
    return true;
  };
  // Every product is waited for once and in order: a wait that skipped one could take its
  // end for the next one's.
  auto product_done = [&](int b) {
    if (!wait_warp(s.o_done + 8 * b, o_par >> b & 1u, s)) return false;
    o_par ^= 1u << b;
    tc_fence_after();
    return true;
  };
  Part p;
  for (int unit = 0; walk.next(a, p); ++unit) {
    const int ring = unit & 1, cnt = p.tb - p.ta;
    const bool two = P::kRowTiles == 2 && p.rows > 128;
    const uint8_t* par = s.sm + P::kPar + ring * kAttnMaxNodes;
    if (!wait_warp(s.meta + 8 * ring, (unit >> 1) & 1, s)) return false;
    // log2 reference of the row and sum of the half's probabilities, for the tile of rows in
    // turn and the other one
    float ref = -INFINITY, sum = 0.0f, ref2 = -INFINITY, sum2 = 0.0f;
    int b = two ? 1 : 0, b_last = 0;
    for (int step = 0; step < (two ? 2 * cnt : cnt); ++step) {
      const int i = two ? step >> 1 : step, row = (two ? (step & 1) * 128 : 0) + lane_row;
      if (two) b_last = b;
      const bool warp_live = (row & ~31) < p.rows;  // a warp of padding only keeps step
      const int32_t lim = p.q.len - (p.ta + i) * P::kBK;  // cached tokens from the tile's first key on
      const bool masked = lim < P::kBK;
      uint32_t may[CH];
      if (masked && warp_live) {
#pragma unroll
        for (int w = 0; w < CH; ++w) {
          const int l = lim - g * NC - 32 * w;
          may[w] = l >= 32 ? 0xFFFFFFFFu : l <= 0 ? 0u : (1u << l) - 1u;
        }
        for (int x = row < p.rows ? a.by_group(p.row0 + row) : -1; x >= 0;) {
          const int at = x + lim - g * NC;
          if (at < 0) break;
#pragma unroll
          for (int w = 0; w < CH; ++w)
            if ((at >> 5) == w) may[w] |= 1u << (at & 31);
          const int up = par[x];
          if (up == 255) break;
          x = up;
        }
      }
      if (!wait_warp(s.s_full + 8 * b, s_par >> b & 1u, s)) return false;
      s_par ^= 1u << b;
      bool waited = i == 0;
      if (warp_live) {
        tc_fence_after();
        const uint32_t st = lane_base + P::kS0 + b * P::kSCols + g * NC;
        uint32_t v[NC];
#pragma unroll
        for (int w = 0; w < CH; ++w) tmem_ld32(st + w * 32, v + w * 32);
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int w = 0; w < CH; ++w) tmem_wait32(v + w * 32);
        if (masked) {
#pragma unroll
          for (int e = 0; e < NC; ++e) v[e] = (may[e >> 5] >> (e & 31)) & 1u ? v[e] : 0xFF800000u;
        }
#pragma unroll
        for (int e = 0; e < NC; ++e) top[e & 3] = fmaxf(top[e & 3], __uint_as_float(v[e]));
        top[0] = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        if (!exchange(top[0], top[1])) return false;
        const float want = fmaxf(top[0], top[1]) * a.scale_log2;
        const bool move = row < p.rows && want - ref > kRefSlack;  // (rows past the unit's hold anything)
        if (__any_sync(0xFFFFFFFFu, move)) {
          const float next = move ? want : ref;
          if (i > 0) {
            const float fix = move ? ex2(ref - next) : 1.0f;
            sum *= fix;
            if (!product_done(b_last)) return false;
            waited = true;
            const uint32_t o = lane_base + (two ? (step & 1) * P::kO1 : 0) + g * (D / 2);
#pragma unroll 1
            for (int d = 0; d < D / 2; d += 16) {
              float x[16];
              tmem_ld16(o + d, x);
              uint32_t u[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(x[e] * fix);
              tmem_st16(o + d, u);
            }
          }
          ref = next;
        }
        const float m = ref == -INFINITY ? 0.0f : ref;
        const uint64_t scale2 = pair(a.scale_log2, a.scale_log2), m2 = pair(-m, -m), up2 = pair(kUp, kUp);
        uint64_t part[2] = {0, 0};
#pragma unroll
        for (int w = 0; w < CH; ++w) {
          uint32_t u[32];  // upper pieces, lower pieces
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float x0, x1;
            unpair(fma2(pair(__uint_as_float(v[w * 32 + 2 * e]), __uint_as_float(v[w * 32 + 2 * e + 1])), scale2, m2), x0, x1);
            x0 = ex2(x0);
            x1 = ex2(x1);
            const uint64_t x = pair(x0, x1);
            part[e & 1] = add2(part[e & 1], x);
            const uint32_t p0 = __float_as_uint(x0), p1 = __float_as_uint(x1);
            u[e] = __byte_perm(p0, p1, 0x7632);
            unpair(fma2(x, up2, pair(-__uint_as_float(p0 & 0xFFFF0000u), -__uint_as_float(p1 & 0xFFFF0000u))), x0, x1);
            u[16 + e] = pack2(x0, x1);
          }
          tmem_st16(st + w * 32, u);
          tmem_st16(st + w * 32 + 16, u + 16);
        }
        {
          float x0, x1, x2, x3;
          unpair(part[0], x0, x1);
          unpair(part[1], x2, x3);
          sum += (x0 + x1) + (x2 + x3);
        }
        tmem_st_wait();
      }
      if (!waited && !product_done(b_last)) return false;
      tc_fence_before();
      mbar_arrive(s.p_full + 8 * b);
      if (two) {
        float t = ref;
        ref = ref2, ref2 = t;
        t = sum;
        sum = sum2, sum2 = t;
        b = 3 - b;
      } else {
        b_last = b;
        b = b + 1 < P::kSB ? b + 1 : 0;
      }
    }
    // ---- the part's result, half of the columns each
    if (!product_done(two ? 1 : b_last) || (two && !product_done(2))) return false;
    const bool whole = p.ta == 0 && p.tb == p.q.tiles - kUnitCost;
    const int32_t bad = reinterpret_cast<volatile int32_t*>(s.sm + P::kBad)[ring];
    const uint32_t* nf = reinterpret_cast<const uint32_t*>(s.sm + P::kNf) + ring * 8;
    uint32_t any_nf = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) any_nf |= nf[w];
    const int part_slot = 2 * c + (p.ta > 0 ? 0 : 1);
    float* po = a.part_o + (int64_t)part_slot * D * a.row_cap;
    if (threadIdx.x == 0) {
      if (!whole) a.part_bad[part_slot] = bad;
      else if (bad) atomicOr(a.status, bad);
    }
    for (int t = 0; t < (two ? 2 : 1); ++t) {
      const int row = t * 128 + lane_row;
      if ((row & ~31) >= p.rows) break;
      float other;
      if (!exchange(t ? sum2 : sum, other)) return false;
      const float all = (t ? sum2 : sum) + other, inv = 1.0f / all;
      const bool live = row < p.rows;
      const int qrow = p.row0 + row, node = live ? a.by_group(qrow) : 0;
      uint16_t* out = a.out + ((p.q.off + node) * a.n_q_heads + p.h * a.group + (live ? qrow - node * a.group : 0)) * (int64_t)D;
      if (!whole && live && g == 0)
        *reinterpret_cast<float2*>(a.part_ml + 2 * ((int64_t)part_slot * a.row_cap + row)) = make_float2(t ? ref2 : ref, all);
#pragma unroll 1
      for (int d = g * (D / 2); d < (g + 1) * (D / 2); d += 16) {
        float v[16];
        tmem_ld16(lane_base + t * P::kO1 + d, v);
        if (!live) continue;
        if (any_nf) {
          for (int x = node;;) {
            if (nf[x >> 5] >> (x & 31) & 1u) {
              const uint16_t* vr = a.v + (p.q.off + x) * a.v_stride + (int64_t)p.h * D + d;
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if ((vr[e] & 0x7F80u) == 0x7F80u) v[e] += __uint_as_float((uint32_t)vr[e] << 16);
            }
            const int up = par[x];
            if (up == 255) break;
            x = up;
          }
        }
        if (!whole) {
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<float4*>(po + ((int64_t)(d + e) / 4 * a.row_cap + row) * 4) =
                make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        } else if (!bad) {
#pragma unroll
          for (int e = 0; e < 16; e += 8)
            *reinterpret_cast<uint4*>(out + d + e) =
                make_uint4(pack2(v[e] * inv, v[e + 1] * inv), pack2(v[e + 2] * inv, v[e + 3] * inv),
                           pack2(v[e + 4] * inv, v[e + 5] * inv), pack2(v[e + 6] * inv, v[e + 7] * inv));
        }
      }
    }
    tc_fence_before();
    mbar_arrive(s.unit_end);
  }
  return true;
}

template <int D>
__global__ void __launch_bounds__(AttnPlan<D>::kThreads, 1) k_tree_attn(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap k_map,
                const __grid_constant__ CUtensorMap v_map) {
  using P = AttnPlan<D>;
  extern __shared__ __align__(1024) uint8_t attn_sm[];
  const int tid = threadIdx.x, warp = tid >> 5, c = blockIdx.x;
  Shared s;
  s.sm = attn_sm;
  s.base = smem_u32(attn_sm);
  int32_t* misc = reinterpret_cast<int32_t*>(attn_sm + P::kMisc);
  s.abort = misc + 1;
  s.limit = a.wait_cycles;
  uint32_t bar = s.base + P::kBar;
  auto bars = [&](int n) {
    const uint32_t b = bar;
    bar += 8 * n;
    return b;
  };
  s.full = bars(P::kSlots);
  s.empty = bars(P::kSlots);
  s.s_full = bars(P::kSB);
  s.p_full = bars(P::kSB);
  s.o_done = bars(P::kSB);
  s.unit_end = bars(1);
  s.q_full = bars(1);
  s.q_free = bars(1);
  s.pair = bars(4);
  s.meta = bars(kMetaRing);
  s.reset = bars(1);
  s.drain = bars(2);
  if (tid == 0) {
    for (int i = 0; i < P::kSlots; ++i) {
      mbar_init(s.full + 8 * i, 128);
      mbar_init(s.empty + 8 * i, 1);
    }
    for (int i = 0; i < P::kSB; ++i) {
      mbar_init(s.s_full + 8 * i, 1);
      mbar_init(s.p_full + 8 * i, P::kSoftmaxThreads);
      mbar_init(s.o_done + 8 * i, 1);
    }
    mbar_init(s.q_full, 128);
    mbar_init(s.q_free, 1);
    for (int i = 0; i < 4; ++i) mbar_init(s.pair + 8 * i, 2);
    mbar_init(s.unit_end, P::kSoftmaxThreads);
    for (int i = 0; i < kMetaRing; ++i) mbar_init(s.meta + 8 * i, 128);
    mbar_init(s.reset, 128);
    mbar_init(s.drain, 1);
    mbar_init(s.drain + 8, 1);
    mbar_init_fence();
    misc[1] = 0;  // abort
  }
  pdl_enter();  // (the joining kernel may be set up from here on; it waits for this one's end)
  const Start start = find_start<D>(a, c, reinterpret_cast<int64_t*>(attn_sm + P::kRing));
  if (c >= start.ctas) {
    if (tid == 0) a.units[c].rows = 0;
    return;
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(s.base + P::kMisc) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (a.n_req > 32) fence_proxy_async_smem();  // the schedule's sums stood where boxes will land
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, (uint32_t)misc[0], 0);
  const Walk<D> walk(start, c);
  if (tid == P::kThreads - 1) {
    Part p;
    Walk<D> w = walk;
    JoinUnit u{};
    if (w.next(a, p) && p.ta > 0) {
      // shares first .. last begin behind the unit's first tile: begin < total * i / ctas < end
      const int64_t begin = share(start.total, start.ctas, c) - start.at + p.begin, end = begin + p.q.tiles - kUnitCost;
      u = JoinUnit{p.q.off, p.h, p.row0, p.rows, (int32_t)quotient((begin + 1) * start.ctas + start.total - 1, start.total),
                   (int32_t)quotient(end * start.ctas + start.total - 1, start.total) - 1, 0};
    }
    a.units[c] = u;
  }
  if (warp < P::kSoftmaxThreads / 32) {
    softmax<D>(a, s, walk, tmem, c);
  } else if (warp < P::kSoftmaxThreads / 32 + 4) {
    produce<D>(a, &k_map, &v_map, s, walk);
    cp_wait_all();
  } else {
    const int second = warp - (P::kSoftmaxThreads / 32 + 4);
    if (second) issue_outputs<D>(a, s, walk, tmem);
    else issue_scores<D>(a, s, walk, tmem);
    umma_commit_one(s.drain + 8 * second);  // nothing may be in flight when tensor memory goes back
    mbar_wait_bounded(s.drain + 8 * second, 0);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (misc[1] && a.box_rows) {  // given up: boxes that nobody waited for land before the block ends (9 ms)
    const long long began = clock64();
    while (clock64() - began < (1ll << 24)) {
    }
  }
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
  if (tid == 0 && misc[1]) atomicOr(a.status, kAttnTimeout);
}

// Adds the parts of the units that several CTAs worked on.  Block (c, y) takes, of the unit inside
// which CTA c + 1's share begins, every (n * gridDim.y)-th run of outputs, n such shares there being.
// Four threads share an output (four adjacent columns of a row): each adds every fourth part, eight
// of them loaded together, and the four sums meet in a fixed order.
constexpr int kJoinThreads = 256;
constexpr int kJoinOutputs = kJoinThreads / 4;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) k_tree_attn_join(const __grid_constant__ AttnArgs a) {
  const int c = blockIdx.x + 1, lane = threadIdx.x & 31, sub = lane >> 3;
  pdl_enter();  // the parts are the previous kernel's
  const JoinUnit u = a.units[c];
  if (u.rows <= 0) return;  // nothing to join here; the other fields say nothing then
  const int n = u.last - u.first + 1, outputs = u.rows * (D / 4);
  const int mine = (threadIdx.x >> 5) * 8 + (lane & 7);  // of the block's outputs
  for (int e0 = ((c - u.first) * gridDim.y + blockIdx.y) * kJoinOutputs; e0 < outputs; e0 += n * gridDim.y * kJoinOutputs) {
    const int e = min(e0 + mine, outputs - 1), c4 = e / u.rows, row = e - c4 * u.rows;
    // the parts are CTA first - 1's second slot and the first slots of first .. last
    float top = -INFINITY, sum = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    int32_t bad = 0;
    for (int i0 = u.first - 1 + sub; i0 <= u.last; i0 += 32) {
      float2 t[8];
      float4 x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = i0 + 4 * k;
        const int64_t slot = 2 * (int64_t)i + (i < u.first ? 1 : 0);
        t[k] = make_float2(-INFINITY, 0.0f);
        x[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (i <= u.last) {
          t[k] = *reinterpret_cast<const float2*>(a.part_ml + 2 * (slot * a.row_cap + row));
          x[k] = *reinterpret_cast<const float4*>(a.part_o + slot * D * a.row_cap + ((int64_t)c4 * a.row_cap + row) * 4);
          bad |= a.part_bad[slot];
        }
      }
      float next = top;
#pragma unroll
      for (int k = 0; k < 8; ++k) next = fmaxf(next, t[k].x);
      const float m = next == -INFINITY ? 0.0f : next, fix = ex2(top - m);
      sum *= fix;
      o.x *= fix, o.y *= fix, o.z *= fix, o.w *= fix;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float w = ex2(t[k].x - m);
        sum += w * t[k].y;
        o.x += w * x[k].x;
        o.y += w * x[k].y;
        o.z += w * x[k].z;
        o.w += w * x[k].w;
      }
      top = next;
    }
    float all = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 8));
    all = fmaxf(all, __shfl_xor_sync(0xFFFFFFFFu, all, 16));
    const float fix = ex2(top - (all == -INFINITY ? 0.0f : all));
    float v[5] = {sum * fix, o.x * fix, o.y * fix, o.z * fix, o.w * fix};
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], 8);
      v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], 16);
    }
    bad |= __shfl_xor_sync(0xFFFFFFFFu, bad, 8);
    bad |= __shfl_xor_sync(0xFFFFFFFFu, bad, 16);
    bad &= kAttnBadRequest | kAttnBadBlock;  // (a part that was given up holds anything)
    if (sub || e0 + mine >= outputs) continue;
    if (bad) {  // the same for every output of the unit
      if (e == 0) atomicOr(a.status, bad);
      continue;
    }
    const float inv = 1.0f / v[0];
    const int g = u.row0 + row, node = a.by_group(g);
    uint16_t* out = a.out + ((u.off + node) * a.n_q_heads + u.h * a.group + (g - node * a.group)) * (int64_t)D + c4 * 4;
    *reinterpret_cast<uint2*>(out) = make_uint2(pack2(v[1] * inv, v[2] * inv), pack2(v[3] * inv, v[4] * inv));
  }
}

std::atomic<uint32_t> g_wait_cycles{uint32_t(kWaitCycles)};

int64_t row_cap(int64_t M, int64_t group, int64_t D) {
  const int64_t rows = M * group, most = D == 256 ? 128 : 256;
  return rows >= most ? most : (rows + 31) / 32 * 32;
}

PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// The cache as a 4-D tensor (column, token of a block, head, block) in boxes of 64 columns x `rows`
// tokens, 128-byte swizzle.
bool make_cache_map(CUtensorMap* map, const uint16_t* base, const kv_cache* c, int rows) {
  auto enc = map_encoder();
  if (!enc) return false;
  cuuint64_t dims[4] = {(cuuint64_t)c->head_dim, (cuuint64_t)c->block_size, (cuuint64_t)c->n_heads, (cuuint64_t)c->n_blocks};
  cuuint64_t strides[3] = {(cuuint64_t)c->token_stride * 2, (cuuint64_t)c->head_stride * 2, (cuuint64_t)c->block_stride * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1}, one[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t*>(base), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tokens of a box: blocks of a power of two tokens, 8 or more, split a tile evenly or are split by
// it; other block sizes (and strides of zero) go row by row through the threads.  131071 tokens in
// blocks of 64 with 256-wide heads took 167 us by boxes and 193 row by row; 24 requests in blocks of 32
// took 127 either way.  A box costs its thread about 100 cycles, so the four warps send a quarter
// each (one warp alone took 141 us there).
int box_rows(const kv_cache* c, int bk) {
  const int64_t b = c->block_size, most = (int64_t)1 << 39;
  if (b < 8 || (b & (b - 1)) || c->token_stride < 1 || c->head_stride < 1 || c->block_stride < 1 ||
      c->token_stride >= most || c->head_stride >= most || c->block_stride >= most)
    return 0;
  return b < bk ? (int)b : bk;
}

template <int D>
int launch_attn(AttnArgs a, const kv_cache* c, cudaStream_t s) {
  using P = AttnPlan<D>;
  static int configured[64] = {0};
  int dev = 0;
  W12_CUDA_TRY(cudaGetDevice(&dev));
  if (dev >= 64 || !configured[dev]) {
    W12_CUDA_TRY(cudaFuncSetAttribute(k_tree_attn<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::kBytes));
    if (dev < 64) configured[dev] = 1;
  }
  CUtensorMap k_map{}, v_map{};
  a.box_rows = box_rows(c, P::kBK);
  if (a.box_rows && !(make_cache_map(&k_map, a.kc, c, a.box_rows) && make_cache_map(&v_map, a.vc, c, a.box_rows))) a.box_rows = 0;
  W12_CUDA_TRY(launch_dependent(k_tree_attn<D>, dim3(kAttnCtas), P::kThreads, P::kBytes, s, a, k_map, v_map));
  W12_LAUNCH_CHECK("tree_attn kernel");
  W12_CUDA_TRY(launch_dependent(k_tree_attn_join<D>, dim3(kAttnCtas - 1, a.row_cap * (D / 4) <= 16 * kJoinOutputs ? 2 : 8),
                                kJoinThreads, 0, s, a));
  W12_LAUNCH_CHECK("tree_attn: joining kernel");
  return W12_OK;
}

struct AttnWs {
  size_t o, ml, bad, units, total;
};

AttnWs attn_ws(int64_t M, int64_t group, int64_t D) {
  auto up = [](size_t b) { return (b + 255) & ~(size_t)255; };
  const size_t slots = 2 * (size_t)kAttnCtas, rows = (size_t)row_cap(M, group, D);
  AttnWs w{};
  w.o = 0;
  w.ml = up(slots * rows * (size_t)D * 4);
  w.bad = w.ml + up(slots * rows * 8);
  w.units = w.bad + up(slots * 4);
  w.total = w.units + up((size_t)kAttnCtas * sizeof(JoinUnit));
  return w;
}

}  // namespace
}  // namespace w12

using namespace w12;

extern "C" {

int tree_attn_set_wait_limit(int64_t cycles) {
  g_wait_cycles.store(uint32_t(cycles > 0 && cycles < kWaitCycles ? cycles : kWaitCycles), std::memory_order_relaxed);
  return W12_OK;
}

size_t tree_attn_workspace_size(int64_t M, int32_t n_req, int64_t n_q_heads, int64_t n_heads, int64_t head_dim) {
  if (M < 1 || n_req < 1 || n_heads < 1 || n_q_heads < n_heads || n_q_heads % n_heads || M > 0x7FFFFFFF ||
      (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return 0;
  return attn_ws(M, n_q_heads / n_heads, head_dim).total;
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
  const float scale_log2 = scale * 1.4426950408889634f;
  if (!(scale > 0.0f) || !std::isfinite(scale_log2))
    return fail(W12_ERR_INVALID_ARG, "tree_attn: scale and scale * log2(e) must be positive and finite");
  if ((((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)out | (uintptr_t)ws) & 15u) ||
      ((q_stride | k_stride | v_stride) & 7) || q_stride < 0 || k_stride < 0 || v_stride < 0)
    return fail(W12_ERR_INVALID_ARG,
                "tree_attn: q, k, v, out and ws must be 16-byte aligned, strides non-negative multiples of 8");
  const AttnWs w = attn_ws(M, n_q_heads / H, D);
  if (ws_bytes < w.total) return fail(W12_ERR_BUFFER_TOO_SMALL, "tree_attn: workspace %zu < %zu", ws_bytes, w.total);
  // Some blocks write their rows while others still read.
  const uintptr_t o0 = (uintptr_t)out, o1 = o0 + (uintptr_t)(M * n_q_heads * D) * 2;
  auto meets = [&](const uint16_t* p, int64_t stride, int64_t heads) {
    return (uintptr_t)p < o1 && o0 < (uintptr_t)p + (uintptr_t)((M - 1) * stride + heads * D) * 2;
  };
  if (meets(q, q_stride, n_q_heads) || meets(k, k_stride, H) || meets(v, v_stride, H))
    return fail(W12_ERR_INVALID_ARG, "tree_attn: out must not overlap q, k or v");
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
  a.n_heads = (int32_t)H;
  a.n_q_heads = (int32_t)n_q_heads;
  a.row_cap = (int32_t)row_cap(M, a.group, D);
  a.by_block = fast_div(a.block_size);
  a.by_group = fast_div(a.group);
  a.scale_log2 = scale_log2;
  a.wait_cycles = g_wait_cycles.load(std::memory_order_relaxed);
  a.out = out;
  a.status = status;
  uint8_t* base = static_cast<uint8_t*>(ws);
  a.part_o = reinterpret_cast<float*>(base + w.o);
  a.part_ml = reinterpret_cast<float*>(base + w.ml);
  a.part_bad = reinterpret_cast<int32_t*>(base + w.bad);
  a.units = reinterpret_cast<JoinUnit*>(base + w.units);
  cudaStream_t s = (cudaStream_t)stream;
  return D == 64 ? launch_attn<64>(a, cache, s) : D == 128 ? launch_attn<128>(a, cache, s) : launch_attn<256>(a, cache, s);
}

}  // extern "C"
