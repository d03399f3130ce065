// qe_attn.cu -- attention of one decode step over a paged cache, with a prefix
// that the whole batch shares.
//
//   out[b,i] = sum_j p_j v_j,   p = softmax_j(scale q[b,i] . k_j)
//
// over the prefix's keys, then row b's own.  The work is cut into tiles of 128
// keys of one key head for a block of query rows: the group's heads of one batch
// row (own keys), or rows of the whole batch (prefix keys, which are therefore
// read once for all of them).  A persistent CTA per SM takes an equal share of the
// tiles, whatever the lengths; a run of tiles of one block within a CTA is a
// segment.  A segment leaves, per query row, a reference m, the sum l of 2^(s - m)
// (scores s in log2 units) and the output sum o of 2^(s - m) v; the second kernel
// joins a row's segments in a fixed order:
//   out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i,   M = max m_i.
//
// Both products run on the tensor cores, accumulators in tensor memory.  Blocks of
// up to 64 rows (narrow) have the keys along M, so that a decode step's few rows
// are a small N and not a padded M:
//   S^T [128 keys x N] = K [128 x D] Q^T     (as they lie: K-major)
//   O^T [D x N]       += V^T [D x 128] P^T   (as they lie: MN-major; P in shared memory)
// Larger blocks (wide: up to 256 rows, 128 at head_dim 256) have 128 rows along M:
//   S [128 x 128 keys] = Q [128 x D] K^T
//   O [128 x D]       += P [128 x 128] V     (P over S in tensor memory)
// so that a softmax thread has a whole row and needs no other's.
// Roles of the 16 warps:
//   0-7   softmax, two groups of four: narrow segments alternate between them (the
//         end of one overlaps the start of the next), a wide one's rows 0-127 and
//         128-255 are one group's each;
//   8-11  producers, 32 keys of a tile each: K and V from their pages into a ring of
//         128-byte-swizzled tiles, by TMA in boxes of 64 dims x 8 to 32 rows of a page, or
//         row by row with cp.async where a page holds no such runs or some keys do not
//         exist (they become zeros: a V row of NaN would not vanish against a P of 0);
//   12    issues the products;
//   13    one thread deals out the CTA's segments, through a ring of descriptors
//         (each role working them out for itself made the code 160 KB and every
//         role wait for its instructions).
// Measured (device time of both kernels): 128 rows behind 32768 shared keys of 8 heads of
// 128 198 us, 353 TFLOP/s; 61 ragged rows of up to 8192 keys 47 us, 2.6 TB/s; two
// sequences of 65535 and 131071 keys of 2 heads of 256 82 us, 4.9 TB/s; one sequence of 4093 keys 16
// us.  Without the exponentials, with an eighth of the products or without most of the
// copies each of these stays within a tenth: none of them bounds a tile by itself.  What
// remains are the hand-overs from one role to the next (producers, scores, softmax,
// outputs), not timed by themselves: about 2.4 us a wide tile and 1.3 us a narrow one,
// and 8 us before the first.
// The reference m need not be the maximum (for fp16 it is set 7 below it): it is raised,
// and o and l rescaled, only when a score passes the maximum that it was set by by more
// than 2^8.  l is the sum of the fp32 numerators; their rounding to the cache's dtype is
// the one that the second product's operand type asks for.
#include <cuda.h>  // types of the tensor map
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "qe_attn.h"
#include "qe_device.cuh"
#include "qe_internal.h"

namespace qe {
namespace {

constexpr int kMaxBatch = 4096;  // B
constexpr int kTile = 128;       // keys per tile
constexpr int kNarrow = 64;      // most rows of a narrow block
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNoRef = 3.0e38f;  // -m before the first score
constexpr float kSlack = 8.f;      // a score may pass the one that set the reference by this (log2)
// The reference is this far below the largest score (log2).  fp16 numerators below 2^-25 become
// 0, and l counts them all the same: 60000 keys at 2^-25.5 of the largest are a thousandth of
// the mass.  Seven powers of two and the slack make 2^15, which fp16 still holds.  bf16 has
// fp32's exponents.
template <typename T>
constexpr float kLift = std::is_same<T, __half>::value ? 7.f : 0.f;
// A segment costs its CTA about one tile's time beside its tiles (queries, first
// reference, results): the deal counts that in.
constexpr int kSegmentCost = 1;

constexpr int kSoftWarps = 8, kProdWarps = 4;
constexpr int kAttnThreads = 512;  // 8 softmax, 4 producer, product and dealing warps; 2 fill up the register split
// registers a thread: 256 x 176 + 256 x 80 = 65536 = 512 x 128, the launch's
constexpr int kSoftRegs = 176, kOtherRegs = 80;
constexpr int kMaxStages = 10, kSegRing = 6;
// A wait's limit grows by this for each tile of a CTA: a tile takes 1.3 to 2.4 us.
constexpr uint64_t kTileNs = 10 * 1000;
// What a CTA waits at its end for its own copies and products, whatever the callers' limit:
// they take microseconds.
constexpr uint64_t kDrainNs = 50 * 1000 * 1000;
constexpr int kSegReaders = kSoftWarps + kProdWarps + 1;

template <int D>
struct Shape {
  static constexpr int kRows = D == 256 ? 128 : 256;  // query rows of a block at most
  static constexpr int kParts = D == 256 ? 2 : 1;     // a K or V tile is this many stages
  static constexpr int kDims = D / kParts;            // dims per stage
  static constexpr int kStage = kTile * kDims * 2;    // bytes
  static constexpr int kStages = D == 64 ? 10 : 5;
  // narrow queries: 128 (64) lines per 64 dims, two buffers of half of them each;
  // narrow P: two buffers of 128 keys x 64 rows; wide queries take both places
  static constexpr int kQLines = D == 256 ? 64 : 128;
  static constexpr int kQ = kQLines * D * 2;
  static constexpr int kP = kTile * kNarrow * 2;
  static constexpr int kSmem = 1024 + kStages * kStage + kQ + 2 * kP;
  static_assert(kSmem + 2048 <= 232448, "shared memory of a CTA");
  static_assert(kRows * D * 2 <= kQ + 2 * kP, "wide queries");
};

struct AttnArgs {
  const void* q;
  void* out;
  const void* kc;
  const void* vc;
  long long q_stride, out_stride, k_page_stride, v_page_stride;
  const int32_t* prefix_pages;
  const int32_t* table;
  const int32_t* kv_len;
  float* lse;
  int* err;
  long long* own_start;  // [grid + 1] where each CTA's share of the own line starts
  int2* own_ctas;        // [own block] first and last CTA that work on it
  int2* prefix_groups;   // [key head] first and last group
  float2* ml_prefix;     // [slot][B * G][4] {m, part of l}
  float2* ml_own;        // [slot][rows of a block][4]
  float* part_prefix;    // [slot][B * G][D]
  float* part_own;       // [slot][rows of a block][D]
  unsigned long long budget_ns;
  int B, n_q, n_kv, G, n_pages, table_stride, prefix_len;
  int prefix_tiles;       // per key head
  int prefix_cost;        // of a prefix tile, in narrow tiles
  int groups;             // groups of CTAs, one CTA per row block, that share the prefix
  int rb_prefix, rb_own;  // row blocks per key head
  int own_rows;           // rows of an own block: min(G, kRows)
  float scale_log2;
  float zero;             // 0, which the compiler does not know
  int run_bits;           // 2^run_bits keys lie behind one another: the power of two in page_size, at most 32; 0: no map
  FastDiv page, group;    // by the page size and by G
};

// ------------------------------------------------------------ tensor cores

// Shared-memory matrix descriptor, 128-byte swizzle, version 1, in two words: low =
// address and leading byte offset, high = stride byte offset and the constants.
// K-major: 1024 (the stride) bytes between groups of 8 rows, the leading offset is not used.
// MN-major: the leading offset is from one block of 64 elements along M or N to the
// next, the stride from one group of 8 along K to the next.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
QE_DEV uint32_t desc_low(uint32_t addr, uint32_t lbo) { return ((addr & 0x3ffffu) >> 4) | ((lbo >> 4) << 16); }
// Instruction descriptor, kind::f16: fp32 accumulator, both operands of T, M = 128.
template <typename T>
QE_DEV uint32_t mma_idesc(int N, bool a_mn, bool b_mn) {
  const uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
  return (1u << 4) | (type << 7) | (type << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
// The products are issued by the whole warp together, of which one lane is elected for each:
// their operands are then the same for the warp (61 ragged rows 45.6 us with a lane alone in
// a branch, 44.1 us this way, in one comparison).
QE_DEV void mma_issue(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 da, db;\n setp.ne.b32 p, %4, 0;\n mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
      " elect.sync _|e, 0xffffffff;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
      : "memory");
}
// the same with A in tensor memory
QE_DEV void mma_issue_ta(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 db;\n setp.ne.b32 p, %4, 0;\n mov.b64 db, {%2, %5};\n"
      " elect.sync _|e, 0xffffffff;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
      : "memory");
}
QE_DEV void mma_commit(uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar))
      : "memory");
}
// A value that is the same in all lanes, told so to the compiler.
template <typename V>
QE_DEV V uniform(V v) { return __shfl_sync(0xffffffffu, v, 0); }

QE_DEV void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
QE_DEV void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
QE_DEV void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 16 columns of the warp's 32 lanes
QE_DEV void tmem_ld16(uint32_t a, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(a));
}
template <typename U>
QE_DEV void tmem_st16(uint32_t a, const U (&v)[16]) {
  static_assert(sizeof(U) == 4, "32-bit columns");
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = *reinterpret_cast<const uint32_t*>(&v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Waits for the loads before it; the values are handed through, so that no use moves above it.
QE_DEV void tmem_wait_ld(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) asm volatile("" : "+f"(v[i]));
}
QE_DEV void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

typedef unsigned long long u64;
// two fp32 numbers in a register pair
QE_DEV u64 pair(float lo, float hi) {
  u64 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
QE_DEV float2 unpair(u64 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
QE_DEV u64 fma_pair(u64 a, u64 b, u64 c) {
  u64 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
QE_DEV u64 add_pair(u64 a, u64 b) {
  u64 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// s - m of two products of q and k.  Their product with the scale is rounded before the
// reference, a rounded product itself, is taken off: in one fma the largest score would keep
// its rounding, many powers of two from scores of 2^27 on, and its numerator be infinite.
// ptxas makes one fma of a packed product and sum, marked .rn or not, so that the product is
// an fma of its own with two zeros that the compiler does not know (narrow blocks), or two
// scalar products (wide ones).  128 rows behind 32768 shared keys: 196 us so, 199 us with the
// zeros, 193 us with one fma; narrow blocks take the same time with one fma and with two.
QE_DEV u64 exponents(u64 qk, u64 scale, u64 zero, u64 neg_ref) { return add_pair(fma_pair(qk, scale, zero), neg_ref); }
QE_DEV u64 exponents(float qk0, float qk1, float scale, u64 neg_ref) {
  return add_pair(pair(__fmul_rn(qk0, scale), __fmul_rn(qk1, scale)), neg_ref);
}
QE_DEV float exp2_approx(float x) {  // 2^-22 relative; below 2^-126: 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 bytes, or 16 zeros
QE_DEV void cp_async16z(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}

// A box of the cache's tensor map {dims, rows of a page, pages}; x is a multiple of 64 dims.
QE_DEV void tma_box(uint32_t dst, const CUtensorMap* map, int x, int row, int page, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(row), "r"(page), "r"(smem_u32(bar))
      : "memory");
}
// ------------------------------------------------------------------ shares

// x * num / den, with 32-bit arithmetic where the product has 32 bits (a 64-bit
// division takes about as long as a global load)
QE_DEV long long mul_div(long long x, int num, int den) {
  if (x < (1 << 20) && num < (1 << 11)) return (uint32_t)x * (uint32_t)num / (uint32_t)den;
  return x * num / den;
}

// How the work is dealt out.  Prefix: `groups` groups of one CTA per row block, so
// that a group reads the same keys at the same time; group g has the tiles
// [g S / groups, (g + 1) S / groups) of the line (key head, tile) of length S.  More
// row blocks than CTAs: one group, each CTA takes every grid-th block.  Own: a line
// (batch row, key head, row block, places), where a block has kSegmentCost places
// more than tiles, of which each CTA takes what brings its total to an equal share.
struct Deal {
  int grid, R, groups, grouped, cost;
  long long S, own;
  QE_DEV Deal(const AttnArgs& a, long long own_places)
      : grid(gridDim.x), R(a.rb_prefix), groups(a.groups), cost(a.prefix_cost), own(own_places) {
    S = (long long)a.prefix_tiles * a.n_kv;
    grouped = S == 0 ? 0 : R <= grid ? groups * R : grid;
  }
  QE_DEV long long group_start(int g) const { return mul_div(S, g, groups); }
  QE_DEV long long own_start(int c) const {
    if (c >= grid) return own;
    if (S == 0) return mul_div(own, c, grid);
    const long long total = own + S * R * cost, each = (S / groups + 1) * cost;
    if (R <= grid && total > each * grid) {  // every CTA has room for own tiles
      long long prefix = S * R;  // prefix tiles of the CTAs before c
      if (c < grouped) {
        const int g = c / R;
        const long long s = group_start(g);
        prefix = s * R + (group_start(g + 1) - s) * (c - g * R);
      }
      return mul_div(total, c, grid) - prefix * cost;
    }
    if (grouped < grid) return c <= grouped ? 0 : mul_div(own, c - grouped, grid - grouped);
    return mul_div(own, c, grid);
  }
};

// A run of tiles of one block: keys key0 + 128 i, i < n, up to kend.
struct Segment {
  const int32_t* list;  // pages
  int key0, kend, n;    // n = 0: no more segments
  int h, rows;          // key head, query rows
  int b, row0;          // own: batch row, first head of the group; prefix: -1, first row of B * G
  int slot;
};

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t s_full[2][2];                     // narrow, by softmax group and its tiles
  uint64_t p_full[2], p_free[2];             // narrow, by tile
  uint64_t ws_full[2], wp_full[2];           // wide, by group of rows
  uint64_t q_done[2], o_full[2], o_free[2];  // by segment
  uint64_t seg_full[kSegRing], seg_empty[kSegRing], drained;
  Segment seg[kSegRing];
  uint32_t tmem;
  int abort;
  alignas(16) uint32_t live[8][4];  // which keys of a tile exist, by tile number
  alignas(16) float neg_ref[2][kNarrow], factor[2][kNarrow];
  long long sum[16];
  int found, found_len;
  long long found_start;
};

static_assert(sizeof(Shared) <= 2048, "beside the dynamic shared memory");

// Bounded wait; false if it gave up.  Once one has, the error is recorded, `abort` is set and
// every later wait that is not over returns at once: the producers and the dealer write nothing
// any more, the roles walk to the end of their segment (within the same bounds of memory) and
// the CTA leaves in the ordinary way.
QE_DEV bool wait_for(uint64_t* bar, uint32_t parity, Shared& sh, const AttnArgs& a) {
  uint64_t deadline = 0;
  for (int i = 0; !mbar_try_wait(bar, parity); ++i) {
    if (*(volatile int*)&sh.abort) return false;
    if ((i & 15) != 15) continue;  // the timer is slow to read
    const uint64_t now = gtimer();
    if (deadline == 0) deadline = now + a.budget_ns;
    if (now > deadline) {
      *(volatile int*)&sh.abort = 1;
      set_error(a.err, QE_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}
// The k-th completion (from 0) of a barrier that is one of two used in turn.  A wait
// sees one bit of the phase: whoever waits for completion k has to know already that
// k - 2 has happened (it waited for it, or for something that comes after it), and k + 2
// must not happen before the wait is over.
QE_DEV void wait_turn(uint64_t* pair, int k, Shared& sh, const AttnArgs& a) { wait_for(&pair[k & 1], (k >> 1) & 1, sh, a); }

// The four softmax warps of a group.
QE_DEV bool group_vote(int group, bool x) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r) : "r"((uint32_t)x), "r"(1 + group) : "memory");
  return r != 0;
}
QE_DEV void group_sync(int group) {
  __syncwarp();
  asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
}

// ------------------------------------------------------------------- roles

// A role's place in the ring of segments.
struct Reader {
  int at = 0;
  uint32_t phase = 0;
  // Copies the next segment, by every lane of a warp.  The lanes agree on its end: one may have
  // seen a wait give up where another has not.
  QE_DEV void next(Segment& x, Shared& sh, const AttnArgs& a) {
    const bool there = wait_for(&sh.seg_full[at], phase, sh, a);
    x = sh.seg[at];
    if (!__all_sync(0xffffffffu, there && !*(volatile int*)&sh.abort)) x.n = 0;
    __syncwarp();  // all lanes have read it before its place is given back (a vote orders no memory)
    if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.seg_empty[at]);
    if (++at == kSegRing) {
      at = 0;
      phase ^= 1;
    }
  }
};

// One thread: the CTA's segments in order, prefix first.
template <int D>
QE_DEV void deal_out(const AttnArgs& a, const Deal& d, long long t, long long t1, int b, int len, long long b_start,
                     int cap, Shared& sh) {
  constexpr int max_rows = Shape<D>::kRows;
  const int c = blockIdx.x, per = a.n_kv * a.rb_own;
  int at = 0;
  uint32_t phase = 1;
  auto put = [&](const Segment& x) {
    if (!wait_for(&sh.seg_empty[at], phase, sh, a)) return;  // it may be being read still
    sh.seg[at] = x;
    mbar_arrive(&sh.seg_full[at]);
    if (++at == kSegRing) {
      at = 0;
      phase ^= 1;
    }
  };
  Segment x;
  if (c < d.grouped) {
    const bool many = d.R > d.grid;
    const int g = many ? 0 : c / d.R;
    const long long s0 = d.group_start(g), s1 = d.group_start(g + 1);
    x.list = a.prefix_pages;
    x.kend = a.prefix_len;
    x.b = -1;
    for (int rb = many ? c : c - g * d.R; rb < d.R; rb += many ? d.grid : d.R) {
      x.row0 = rb * max_rows;
      x.rows = min(max_rows, a.B * a.G - x.row0);
      long long s = s0;
      x.h = s < (1ll << 31) ? (int)((uint32_t)s / (uint32_t)a.prefix_tiles) : (int)(s / a.prefix_tiles);
      int i = (int)(s - (long long)x.h * a.prefix_tiles);
      while (s < s1) {
        x.n = (int)min((long long)(a.prefix_tiles - i), s1 - s);
        x.key0 = i * kTile;
        x.slot = g + x.h;
        if (rb == 0) {
          if (i == 0) a.prefix_groups[x.h].x = g;
          if (i + x.n == a.prefix_tiles) a.prefix_groups[x.h].y = g;
        }
        put(x);
        s += x.n;
        i = 0;
        ++x.h;
      }
    }
  }
  if (t < t1) {
    int nt = (len + kTile - 1) / kTile, places = nt + kSegmentCost;
    const long long in_row = t - b_start;
    int unit = in_row < (1ll << 31) ? (int)((uint32_t)in_row / (uint32_t)places) : (int)(in_row / places);
    int p = (int)(in_row - (long long)unit * places);
    for (;;) {
      const int p1 = (int)min((long long)places, p + (t1 - t));  // places [p, p1) of this block are this CTA's
      const int i = max(0, p - kSegmentCost), i1 = max(0, p1 - kSegmentCost);
      if (i < i1) {
        const int u = b * per + unit;
        x.n = i1 - i;
        x.h = unit / a.rb_own;
        x.list = a.table + (size_t)b * a.table_stride;
        x.key0 = i * kTile;
        x.kend = len;
        x.b = b;
        x.row0 = (unit - x.h * a.rb_own) * max_rows;
        x.rows = min(max_rows, a.G - x.row0);
        x.slot = c + u;
        if (i == 0) a.own_ctas[u].x = c;
        if (i1 == nt) a.own_ctas[u].y = c;
        put(x);
      }
      t += p1 - p;
      if (t >= t1) break;
      p = 0;
      if (++unit == per) {
        unit = 0;
        do {
          ++b;
          len = max(0, min(a.kv_len[b], cap));
        } while (len == 0 && b < a.B - 1);
        nt = (len + kTile - 1) / kTile;
        places = nt + kSegmentCost;
      }
    }
  }
  x.n = 0;
  put(x);
}

// The order of the stages.  Tile g's K comes right before tile g - 1's V, so that its
// scores can be computed while the softmax of g - 1 runs; only where narrow and wide
// segments meet (and after the last tile) V comes first.  This counts, for the
// consumer, the place of each K and V in that order.
struct Places {
  int k = 0, v = 0, next = 1;  // of the current K, of the V of the tile before it, and of what follows both
  QE_DEV void step(bool v_first) {  // to the next tile
    v = v_first ? next : next + 1;
    k = v_first ? next + 1 : next;
    next += 2;
  }
};

template <typename T, int D>
QE_DEV void produce(const AttnArgs& a, const CUtensorMap* k_map, const CUtensorMap* v_map, Shared& sh, unsigned char* ring,
                    unsigned char* qs) {
  using Sh = Shape<D>;
  constexpr int CH = Sh::kDims / 8;   // 16-byte pieces of a row of a stage
  constexpr int RPI = 32 / CH;        // rows a warp instruction copies
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - kSoftWarps;
  const int sub = lane % CH, sub_row = lane / CH;
  // this lane's place in a stage: of row 32 w + RPI k + sub_row, k < PERIOD; later rows are
  // whole swizzle periods of 1024 bytes further on
  constexpr int PERIOD = 8 / RPI;
  const uint32_t ring_u = smem_u32(ring) + (sub >> 3) * (kTile * 128) + 32 * w * 128;
  uint32_t place[PERIOD];
#pragma unroll
  for (int k = 0; k < PERIOD; ++k)
    place[k] = ring_u + (k * RPI + sub_row) * 128 + (((sub & 7) ^ ((k * RPI + sub_row) & 7)) << 4);
  const uint32_t q_u = smem_u32(qs);
  int stage = 0, phase = 1;  // fresh empty barriers count as free
  // this lane's row of the tile, of K and of the V that follows later: address, and place in the map
  unsigned long long k_row = 0, v_row = 0, v_next = 0;
  int k_page = 0, k_in_page = 0, v_page = 0, v_in_page = 0, issued = 0;
  uint32_t live = 0, v_live = 0;
  const uint32_t ring_at = smem_u32(ring);
  auto load = [&](bool is_v) {
#pragma unroll 1
    for (int p = 0; p < Sh::kParts; ++p) {
      const unsigned long long row = (is_v ? v_row : k_row) + 2 * p * Sh::kDims;
      const uint32_t lv = is_v ? v_live : live;
      // Once a wait has given up nothing more is copied: copies into a stage that is still being
      // filled would take its barrier's counts beyond their range.  The lanes go together.
      const bool given_up = *(volatile int*)&sh.abort;
      if (!__all_sync(0xffffffffu, wait_for(&sh.empty[stage], phase, sh, a) && !given_up)) return;
      const uint32_t at = stage * Sh::kStage;
      if (lv == 0xffffffffu && a.run_bits >= 3) {
        // lane l: run l mod (32 / run) of the warp's rows, 64 dims l / (32 / run)
        const int runs = 32 >> a.run_bits, from = (lane & (runs - 1)) << a.run_bits, block = lane >> (5 - a.run_bits);
        const int page = __shfl_sync(0xffffffffu, is_v ? v_page : k_page, from);
        const int in_page = __shfl_sync(0xffffffffu, is_v ? v_in_page : k_in_page, from);
        if (lane == 0) mbar_arrive_expect_tx(&sh.full[stage], 32 * Sh::kDims * 2);
        __syncwarp();
        if (block < Sh::kDims / 64)
          tma_box(ring_at + at + block * (kTile * 128) + (32 * w + from) * 128, is_v ? v_map : k_map,
                  p * Sh::kDims + block * 64, in_page, page, &sh.full[stage]);
        // Every lane (the barrier counts 33 a warp), once its cp.async have landed: on a segment's
        // first tile its queries are among them, and no other barrier says that they are there.
        cp_async_mbar_arrive_noinc(&sh.full[stage]);
      } else {
#pragma unroll
        for (int i = 0; i < 32 / RPI; ++i) {
          const int r = i * RPI + sub_row;
          const unsigned long long from = __shfl_sync(0xffffffffu, row, r);
          cp_async16z(place[i % PERIOD] + at + i / PERIOD * 1024, (const T*)from + sub * 8, (lv >> r) & 1);
        }
        // every lane's copies arrive when they land; lane 0 arrives for what it wrote itself
        cp_async_mbar_arrive_noinc(&sh.full[stage]);
        if (lane == 0) mbar_arrive(&sh.full[stage]);
      }
      ++issued;
      if (++stage == Sh::kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
  };
  Reader reader;
  Segment x;
  int left = 0, key0 = 0, n = 0, seg = -1, rows_before = 0, page_next = -1;
  auto page_at = [&](int key) { return key < x.kend ? __ldg(x.list + a.page.div((uint32_t)key)) : -1; };
  bool more = true;
  while (true) {
    bool first = false, v_first = false;
    if (left == 0) {
      reader.next(x, sh, a);
      left = x.n;
      key0 = x.key0;
      more = left > 0;
      first = more;
      v_first = n > 0 && (!more || (x.rows > kNarrow) != (rows_before > kNarrow));
    }
    // at most two loads: (V, K) or (K, V); one of them at either end
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      const bool is_v = (i == 0) == v_first;
      if (is_v) {
        if (n > 0) load(true);
        continue;
      }
      if (!more) continue;
      if (first) {
        // the block's queries, with its first tile's keys: two narrow buffers, or one place for all
        ++seg;
        const bool wide = x.rows > kNarrow, whole = x.rows > Sh::kQLines / 2, whole_before = rows_before > Sh::kQLines / 2;
        if (seg >= 2) wait_turn(sh.q_done, seg - 2, sh, a);
        if (seg >= 1 && (whole || whole_before)) wait_turn(sh.q_done, seg - 1, sh, a);
        if (seg >= 1 && wide && rows_before <= kNarrow) wait_turn(sh.o_full, seg - 1, sh, a);  // P is read no more
        __syncwarp();
        rows_before = x.rows;
        const int fill = wide ? (x.rows + 127) & ~127 : (x.rows + 15) & ~15;
        const uint32_t dst = q_u + (!whole && (seg & 1) ? Sh::kQLines / 2 * 128 : 0);
        // a thread keeps its 16-byte piece and steps through the rows, 128 / (D / 8) at a time
        constexpr int STEP = 32 * kProdWarps / (D / 8);
        const int tid = threadIdx.x - 32 * kSoftWarps, ch = tid % (D / 8), r0 = tid / (D / 8);
        const T* q_head = (const T*)a.q + (size_t)x.h * a.G * D + ch * 8 + (x.b >= 0 ? (size_t)x.b * a.q_stride : 0);
        const uint32_t col = dst + (ch >> 3) * ((wide ? 128 : Sh::kQLines) * 128);
#pragma unroll 4
        for (int r = r0; r < fill; r += STEP) {
          const int f = x.row0 + r, fb = x.b >= 0 ? 0 : (int)a.group.div((uint32_t)f);
          const T* src = q_head + (long long)fb * a.q_stride + (f - fb * a.G) * D;
          const uint32_t line = wide ? (r >> 7) * (D * 256) + (r & 127) * 128 : r * 128;
          cp_async16z(col + line + (((ch & 7) ^ (r & 7)) << 4), r < x.rows ? src : (const T*)a.q, r < x.rows);
        }
      }
      const int key = key0 + 32 * w + lane;
      const int page = first ? page_at(key) : page_next;  // asked for a tile ahead
      page_next = left > 1 ? page_at(key + kTile) : -1;
      const bool ok = page >= 0 && page < a.n_pages;
      if (key < x.kend && !ok) set_error(a.err, QE_ERR_INVALID_ARG);
      live = __ballot_sync(0xffffffffu, ok);
      k_page = page;
      k_in_page = x.h * (int)a.page.d + key - (int)a.page.div((uint32_t)key) * (int)a.page.d;
      const long long in_page = (long long)k_in_page * D;
      k_row = (unsigned long long)((const T*)a.kc + (ok ? page * a.k_page_stride + in_page : 0));
      v_next = (unsigned long long)((const T*)a.vc + (ok ? page * a.v_page_stride + in_page : 0));
      if (lane == 0) sh.live[n & 7][w] = live;
      load(false);
    }
    if (!more) break;
    v_row = v_next;
    v_page = k_page;
    v_in_page = k_in_page;
    v_live = live;
    key0 += kTile;
    --left;
    ++n;
  }
  cp_async_wait_all();
  // nothing may be in flight when the CTA leaves (after a wait that gave up, the last stages could be,
  // and one that not all warps have filled does not complete: it is given the time)
  const uint64_t deadline = gtimer() + kDrainNs;
  for (int i = max(0, issued - Sh::kStages); i < issued; ++i)
    while (!mbar_try_wait(&sh.full[i % Sh::kStages], (i / Sh::kStages) & 1))
      if (gtimer() > deadline) break;
}

// One warp, every value in it uniform.
template <typename T, int D>
QE_DEV void multiply(const AttnArgs& a, Shared& sh, unsigned char* ring, unsigned char* qs, unsigned char* ps,
                     uint32_t tmem) {
  using Sh = Shape<D>;
  const uint32_t ring_u = smem_u32(ring), q_u = smem_u32(qs), p_u = smem_u32(ps);
  // stage number `place * kParts + part` of the producers' order
  auto take = [&](int at) {
    wait_for(&sh.full[at % Sh::kStages], (at / Sh::kStages) & 1, sh, a);
    __syncwarp();
    fence_async_smem();  // the copies wrote through the generic proxy, the products read through the async one
    tc_after();
    return ring_u + at % Sh::kStages * Sh::kStage;
  };
  auto give = [&](int at) { mma_commit(&sh.empty[at % Sh::kStages]); };
  Places pl;
  int n = 0;  // narrow tiles so far
  int group_n[2] = {0, 0};  // of each softmax group
  auto narrow_scores = [&](const Segment& x, int seg) {
    const int n16 = (x.rows + 15) & ~15;
    const uint32_t idesc = mma_idesc<T>(n16, false, false), d = tmem + (n & 1) * 128;
    const uint32_t q_at = desc_low(q_u + (x.rows <= Sh::kQLines / 2 && (seg & 1) ? Sh::kQLines / 2 * 128 : 0), 16);
#pragma unroll 1
    for (int p = 0; p < Sh::kParts; ++p) {
      const uint32_t k_at = desc_low(take(pl.k * Sh::kParts + p), 16), qp = q_at + p * (Sh::kDims / 64) * (Sh::kQLines * 128 / 16);
#pragma unroll
      for (int k = 0; k < Sh::kDims / 16; ++k)
        mma_issue(d, k_at + (k >> 2) * (kTile * 128 / 16) + (k & 3) * 2, qp + (k >> 2) * (Sh::kQLines * 128 / 16) + (k & 3) * 2,
                  idesc, p > 0 || k > 0);
      give(pl.k * Sh::kParts + p);
    }
    mma_commit(&sh.s_full[seg & 1][group_n[seg & 1]++ & 1]);
  };
  auto narrow_outputs = [&](int m, int rows, int seg, bool first, int v_place) {
    wait_turn(sh.p_full, m, sh, a);
    __syncwarp();
    const uint32_t idesc = mma_idesc<T>((rows + 15) & ~15, true, true), d = tmem + 256 + (seg & 1) * 128;
    const uint32_t p_at = desc_low(p_u + (m & 1) * Sh::kP, kTile * 128);
#pragma unroll 1
    for (int p = 0; p < Sh::kParts; ++p) {
      // head_dim 64: the second 64 dims repeat the first (leading offset 0); they are not read
      const uint32_t v_at = desc_low(take(v_place * Sh::kParts + p), D == 64 ? 0 : kTile * 128);
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k)
        mma_issue(d + p * 64, v_at + k * (2048 / 16), p_at + k * (2048 / 16), idesc, !first || k > 0);
      give(v_place * Sh::kParts + p);
    }
    mma_commit(&sh.p_free[m & 1]);
  };
  auto wide_scores = [&](int blk, bool last_block) {
    const uint32_t idesc = mma_idesc<T>(kTile, false, false), d = tmem + blk * 128;
#pragma unroll 1
    for (int p = 0; p < Sh::kParts; ++p) {
      const uint32_t k_at = desc_low(take(pl.k * Sh::kParts + p), 16);
      const uint32_t q_at = desc_low(q_u + blk * (D * 256) + p * (Sh::kDims / 64) * (128 * 128), 16);
#pragma unroll
      for (int k = 0; k < Sh::kDims / 16; ++k)
        mma_issue(d, q_at + (k >> 2) * (128 * 128 / 16) + (k & 3) * 2, k_at + (k >> 2) * (kTile * 128 / 16) + (k & 3) * 2,
                  idesc, p > 0 || k > 0);
      if (last_block) give(pl.k * Sh::kParts + p);
    }
    mma_commit(&sh.ws_full[blk]);
  };
  auto wide_outputs = [&](int blk, bool last_block, bool first, int v_place) {
    const uint32_t idesc = mma_idesc<T>(Sh::kDims, false, true), p_at = tmem + blk * 128;
#pragma unroll 1
    for (int p = 0; p < Sh::kParts; ++p) {
      const uint32_t v_at = desc_low(take(v_place * Sh::kParts + p), kTile * 128), d = tmem + 256 + blk * 128 + p * 128;
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k) mma_issue_ta(d, p_at + k * 8, v_at + k * (2048 / 16), idesc, !first || k > 0);
      if (last_block) give(v_place * Sh::kParts + p);
    }
  };

  Reader reader;
  Segment x;
  auto next_segment = [&](Segment& y) {
    reader.next(y, sh, a);
    y.n = uniform(y.n);
    y.rows = uniform(y.rows);
  };
  next_segment(x);
  bool wide_before = false;
  int wide_n = 0;  // wide tiles so far, by which the phases of wp_full go (block 1 may have had fewer)
  int wide_n1 = 0;
  // the narrow tile whose outputs are still to be issued
  bool pending = false, pend_first = false;
  int pend_rows = 0, pend_seg = 0;
  for (int seg = 0; x.n > 0; ++seg) {
    const bool wide = x.rows > kNarrow;
    Segment y;
    if (!wide) {
      for (int i = 0; i < x.n; ++i) {
        // (the place of this tile's K was set when the tile before it was left)
        narrow_scores(x, seg);
        if (i == x.n - 1) mma_commit(&sh.q_done[seg & 1]);
        if (pending) {
          narrow_outputs(n - 1, pend_rows, pend_seg, pend_first, pl.v);
          if (pend_seg != seg) mma_commit(&sh.o_full[pend_seg & 1]);
        }
        pending = true;
        pend_rows = x.rows;
        pend_seg = seg;
        pend_first = i == 0;
        ++n;
        if (i == 0) {  // before the first outputs of this segment
          if (seg >= 2) wait_turn(sh.o_free, seg - 2, sh, a);
          if (wide_before) wait_turn(sh.o_free, seg - 1, sh, a);
        }
        bool v_first = false;
        if (i == x.n - 1) {
          next_segment(y);
          v_first = y.n == 0 || y.rows > kNarrow;
        }
        pl.step(v_first);
        if (v_first) {
          narrow_outputs(n - 1, pend_rows, pend_seg, pend_first, pl.v);
          mma_commit(&sh.o_full[seg & 1]);
          pending = false;
        }
      }
    } else {
      const int blocks = (x.rows + 127) >> 7;
      if (seg >= 2) wait_turn(sh.o_free, seg - 2, sh, a);
      if (seg >= 1) wait_turn(sh.o_free, seg - 1, sh, a);
      for (int blk = 0; blk < blocks; ++blk) wide_scores(blk, blk == blocks - 1);
      if (x.n == 1) mma_commit(&sh.q_done[seg & 1]);
      for (int i = 0; i < x.n; ++i) {
        bool v_first = false;
        if (i == x.n - 1) {
          next_segment(y);
          v_first = y.n == 0 || y.rows <= kNarrow;
        }
        pl.step(v_first);
        for (int blk = 0; blk < blocks; ++blk) {
          wait_for(&sh.wp_full[blk], (blk ? wide_n1 : wide_n) & 1, sh, a);
          __syncwarp();
          tc_after();
          wide_outputs(blk, blk == blocks - 1, i == 0, pl.v);
          if (i + 1 < x.n) wide_scores(blk, blk == blocks - 1);
        }
        ++wide_n;
        wide_n1 += blocks - 1;
        if (i + 2 == x.n) mma_commit(&sh.q_done[seg & 1]);
      }
      mma_commit(&sh.o_full[seg & 1]);
    }
    wide_before = wide;
    x = y;
  }
  // whatever happened, nothing is in flight when this returns
  __syncwarp();
  mma_commit(&sh.drained);
  const uint64_t deadline = gtimer() + kDrainNs;
  while (!mbar_try_wait_sleep(&sh.drained, 0, 10000u))
    if (gtimer() > deadline) {
      set_error(a.err, QE_ERR_TIMEOUT);
      break;
    }
}

// One narrow segment, by the group whose turn it is: a thread has one key (lane of
// S^T) and all columns.  n: number of its first tile among the narrow ones; own_n:
// among the group's; tile: among all.  The scores of tile n are issued after the
// outputs of tile n - 2, so that once they are there, that P has been read.
template <typename T, int D>
QE_DEV void soften_narrow(const AttnArgs& a, const Segment& x, int seg, int n, int own_n, int tile, Shared& sh,
                          unsigned char* ps, uint32_t tmem_base) {
  using Sh = Shape<D>;
  constexpr int J = kNarrow / 16;
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 3, group = threadIdx.x >> 7, key = threadIdx.x & 127;
  const uint32_t tmem = tmem_base + ((uint32_t)(32 * w) << 16), o_at = tmem + 256 + (seg & 1) * 128;
  const int nb = (x.rows + 15) >> 4;
  float l[J][16];
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int e = 0; e < 16; ++e) l[j][e] = 0.f;
  const u64 scale2 = pair(a.scale_log2, a.scale_log2), zero2 = pair(a.zero, a.zero);
  float* ref = sh.neg_ref[group];
  float* factor = sh.factor[group];
#pragma unroll 1
  for (int i = 0; i < x.n; ++i, ++n, ++own_n, ++tile) {
    const uint32_t s_at = tmem + (n & 1) * 128;
    wait_turn(sh.s_full[group], own_n, sh, a);
    __syncwarp();
    tc_after();
    const bool live = (sh.live[tile & 7][w] >> lane) & 1;
    float p[J][16];
#pragma unroll 1
    for (bool raise = i == 0;; raise = true) {
      if (raise) {
        // raise the references to the maxima so far; no product reads this P or writes o meanwhile
        if (i > 0) wait_turn(sh.p_free, n - 1, sh, a);
        __syncwarp();
        tc_after();
        float* scratch = reinterpret_cast<float*>(ps + (n & 1) * Sh::kP);
#pragma unroll 1
        for (int bb = 0; bb < nb; ++bb) {
          float v[16];
          __syncwarp();
          tmem_ld16(s_at + bb * 16, v);
          tmem_wait_ld(v);
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = live ? __fmul_rn(v[e], a.scale_log2) : -INFINITY;
          const float m = warp_reduce_rows_max<16>(v, lane);
          if ((lane & 1) == 0) scratch[w * kNarrow + bb * 16 + reduced_row_of_lane<16>(lane)] = m;
        }
        group_sync(group);
        if (key < nb * 16) {
          const float old = i == 0 ? -kNoRef : -ref[key];
          const float m = fmaxf(fmaxf(fmaxf(scratch[key], scratch[kNarrow + key]),
                                      fmaxf(scratch[2 * kNarrow + key], scratch[3 * kNarrow + key])) - kLift<T>, old);
          ref[key] = -m;
          factor[key] = exp2_approx(old - m);
        }
        group_sync(group);
        if (i > 0) {
#pragma unroll
          for (int j = 0; j < J; ++j)
            if (j < nb) {
#pragma unroll
              for (int e = 0; e < 16; e += 4) {
                const float4 r = *reinterpret_cast<const float4*>(factor + j * 16 + e);
                l[j][e] *= r.x;
                l[j][e + 1] *= r.y;
                l[j][e + 2] *= r.z;
                l[j][e + 3] *= r.w;
              }
            }
#pragma unroll 1
          for (int c = 0; c < nb * Sh::kParts; ++c) {
            const int bb = c % nb, d = c / nb;
            float o[16];
            const uint32_t at = o_at + d * 64 + bb * 16;
            __syncwarp();
            tmem_ld16(at, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] *= factor[bb * 16 + e];
            tmem_st16(at, o);
          }
          tmem_wait_st();
        }
        __syncwarp();
      }
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (j < nb) tmem_ld16(s_at + j * 16, p[j]);
#pragma unroll
      for (int j = 0; j < J; ++j) tmem_wait_ld(p[j]);
      float most = -INFINITY;
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (j < nb) {
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 r = *reinterpret_cast<const float4*>(ref + j * 16 + e);
            const float2 y0 = unpair(exponents(pair(p[j][e], p[j][e + 1]), scale2, zero2, pair(r.x, r.y)));
            const float2 y1 = unpair(exponents(pair(p[j][e + 2], p[j][e + 3]), scale2, zero2, pair(r.z, r.w)));
            p[j][e] = y0.x;
            p[j][e + 1] = y0.y;
            p[j][e + 2] = y1.x;
            p[j][e + 3] = y1.y;
          }
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            if (!live) p[j][e] = -INFINITY;
            top[e & 3] = fmaxf(top[e & 3], p[j][e]);
            p[j][e] = exp2_approx(p[j][e]);
          }
          most = fmaxf(most, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
        }
      if (raise || !group_vote(group, most > kSlack + kLift<T>)) break;
    }
    unsigned char* p_row = ps + (n & 1) * Sh::kP + key * 128;
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (j < nb) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float* v = p[j] + 8 * hf;
          *reinterpret_cast<uint4*>(p_row + (((2 * j + hf) ^ (key & 7)) << 4)) =
              make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) l[j][e] += p[j][e];
      }
    fence_async_smem();
    tc_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.p_full[n & 1]);
  }
  // the segment's results: each warp leaves its part of l
  const size_t row_at = x.b >= 0 ? (size_t)x.slot * a.own_rows : (size_t)x.slot * a.B * a.G + x.row0;
  float* po = (x.b >= 0 ? a.part_own : a.part_prefix) + row_at * D + key;
  float2* pml = (x.b >= 0 ? a.ml_own : a.ml_prefix) + row_at * 4 + w;
#pragma unroll
  for (int j = 0; j < J; ++j)
    if (j < nb) {
      const float sum = warp_reduce_rows<16>(l[j], lane);
      const int col = j * 16 + reduced_row_of_lane<16>(lane);
      if ((lane & 1) == 0 && col < x.rows) pml[col * 4] = make_float2(-ref[col], sum);
    }
  wait_turn(sh.o_full, seg, sh, a);
  __syncwarp();
  tc_after();
#pragma unroll 1
  for (int c = 0; c < nb * Sh::kParts; ++c) {
    const int bb = c % nb, d = c / nb;
    float o[16];
    __syncwarp();
    tmem_ld16(o_at + d * 64 + bb * 16, o);
    tmem_wait_ld(o);
    if (D >= 128 || key < D) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (bb * 16 + e < x.rows) po[(size_t)(bb * 16 + e) * D + d * 128] = o[e];
    }
  }
  tc_before();
  __syncwarp();
  if (lane < 2) mbar_arrive(&sh.o_free[seg & 1]);  // for the other group's four warps too
}

// One wide segment, one group's 128 rows: a thread has one row.  n: number of the
// first tile among the group's wide ones.
template <typename T, int D>
QE_DEV void soften_wide(const AttnArgs& a, const Segment& x, int seg, int n, int tile, Shared& sh, uint32_t tmem_base) {
  using Sh = Shape<D>;
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 3, group = threadIdx.x >> 7;
  const uint32_t tmem = tmem_base + ((uint32_t)(32 * w) << 16), s_at = tmem + group * 128, o_at = tmem + 256 + group * 128;
  const int row = threadIdx.x;  // of the block: group * 128 + lane of the accumulator
  float neg = kNoRef;
  u64 sum[2] = {0, 0};  // l in four parts
#pragma unroll 1
  for (int i = 0; i < x.n; ++i, ++n, ++tile) {
    wait_for(&sh.ws_full[group], n & 1, sh, a);  // the outputs of the tile before are complete then, too
    __syncwarp();
    tc_after();
    const uint4 live = *reinterpret_cast<const uint4*>(sh.live[tile & 7]);
    const bool all = (live.x & live.y & live.z & live.w) == 0xffffffffu;
    // half a row in registers at a time, read twice: the maximum, the exponentials and
    // the sums of its columns have no order among them, and a whole row would spill
    float v[4][16];
    auto half_row = [&](int c) {
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 4; ++k) tmem_ld16(s_at + c * 64 + k * 16, v[k]);
#pragma unroll
      for (int k = 0; k < 4; ++k) tmem_wait_ld(v[k]);
      if (!all) {
        const uint32_t w0 = c ? live.z : live.x, w1 = c ? live.w : live.y;
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (!(((k >> 1 ? w1 : w0) >> ((k & 1) * 16 + e)) & 1)) v[k][e] = -INFINITY;
      }
    };
    float top = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
      half_row(c);
      float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < 16; e += 2) t[(e >> 1) & 3] = fmaxf(t[(e >> 1) & 3], fmaxf(v[k][e], v[k][e + 1]));
      top = fmaxf(top, fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])));
    }
    top = __fmul_rn(top, a.scale_log2);  // scale > 0
    const bool raise = top + neg > kSlack + kLift<T>;
    top -= kLift<T>;
    if (__any_sync(0xffffffffu, raise)) {
      float f = 1.f;
      if (raise) {
        f = exp2_approx(-neg - top);
        neg = -top;
      }
      const u64 f2 = pair(f, f);
      sum[0] = fma_pair(sum[0], f2, 0);
      sum[1] = fma_pair(sum[1], f2, 0);
      if (i > 0) {
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          float o[16];
          __syncwarp();
          tmem_ld16(o_at + c * 16, o);
          tmem_wait_ld(o);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] *= f;
          tmem_st16(o_at + c * 16, o);
        }
      }
    }
    // (a masked score is -inf and its numerator 0, unless nothing was ever seen: neg is
    // 3e38 then, and -inf + 3e38 is -inf still)
    const u64 neg2 = pair(neg, neg);
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
      half_row(c);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float* x = &v[2 * k + (e >> 4)][e & 15];
          const float2 y = unpair(exponents(x[0], x[1], a.scale_log2, neg2));
          const float x0 = exp2_approx(y.x), x1 = exp2_approx(y.y);
          sum[(e >> 1) & 1] = add_pair(sum[(e >> 1) & 1], pair(x0, x1));
          pk[e >> 1] = pack2<T>(x0, x1);
        }
        tmem_st16(s_at + c * 32 + k * 16, pk);  // over scores that have been read
      }
    }
    tmem_wait_st();
    tc_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.wp_full[group]);
  }
  wait_turn(sh.o_full, seg, sh, a);
  __syncwarp();
  tc_after();
  const size_t row_at = x.b >= 0 ? (size_t)x.slot * a.own_rows : (size_t)x.slot * a.B * a.G + x.row0;
  float* po = (x.b >= 0 ? a.part_own : a.part_prefix) + (row_at + row) * D;
#pragma unroll 1
  for (int c = 0; c < D / 16; ++c) {
    float o[16];
    __syncwarp();
    tmem_ld16(o_at + c * 16, o);
    tmem_wait_ld(o);
    if (row < x.rows) {
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        *reinterpret_cast<float4*>(po + c * 16 + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
    }
  }
  if (row < x.rows) {
    float4* pml = reinterpret_cast<float4*>((x.b >= 0 ? a.ml_own : a.ml_prefix) + (row_at + row) * 4);
    const float2 l0 = unpair(sum[0]), l1 = unpair(sum[1]);
    pml[0] = make_float4(-neg, l0.x, -neg, l0.y);
    pml[1] = make_float4(-neg, l1.x, -neg, l1.y);
  }
  tc_before();
}

template <typename T, int D>
QE_DEV void soften(const AttnArgs& a, Shared& sh, unsigned char* ps, uint32_t tmem) {
  const int lane = threadIdx.x & 31, group = threadIdx.x >> 7;
  Reader reader;
  Segment x;
  int n = 0, own_n = 0, wide_n = 0, tile = 0;
#pragma unroll 1
  for (int seg = 0;; ++seg) {
    reader.next(x, sh, a);
    // a group's warps have to go through the same barriers: they end together
    if (group_vote(group, x.n == 0)) break;
    if (x.rows > kNarrow) {
      if (group * 128 < x.rows) {
        soften_wide<T, D>(a, x, seg, wide_n, tile, sh, tmem);
        wide_n += x.n;
        __syncwarp();
        if (lane < (x.rows > 128 ? 1 : 2)) mbar_arrive(&sh.o_free[seg & 1]);  // 2: for the group without rows, too
      }
    } else {
      if ((seg & 1) == group) {
        soften_narrow<T, D>(a, x, seg, n, own_n, tile, sh, ps, tmem);
        own_n += x.n;
      }
      n += x.n;
    }
    tile += x.n;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kAttnThreads, 1) qe_attn_part_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap k_map,
                        const __grid_constant__ CUtensorMap v_map) {
  using Sh = Shape<D>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(16) Shared sh;
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  unsigned char *ring = smem, *qs = smem + Sh::kStages * Sh::kStage, *ps = qs + Sh::kQ;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < Sh::kStages; ++i) {
      mbar_init(&sh.full[i], kProdWarps * 33);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[0][i], 1);
      mbar_init(&sh.s_full[1][i], 1);
      mbar_init(&sh.p_full[i], kSoftWarps / 2);
      mbar_init(&sh.p_free[i], 1);
      mbar_init(&sh.ws_full[i], 1);
      mbar_init(&sh.wp_full[i], kSoftWarps / 2);
      mbar_init(&sh.q_done[i], 1);
      mbar_init(&sh.o_full[i], 1);
      mbar_init(&sh.o_free[i], kSoftWarps);
    }
    for (int i = 0; i < kSegRing; ++i) {
      mbar_init(&sh.seg_full[i], 1);
      mbar_init(&sh.seg_empty[i], kSegReaders);
    }
    mbar_init(&sh.drained, 1);
    fence_mbar_init();
    sh.abort = 0;
  }
  if (warp == 12) {
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tc_before();
  }
  grid_dependency_wait();
  grid_launch_dependents();

  // where this CTA's share of the own line starts: one pass over the lengths for
  // up to 512 rows, a sum and a search for more
  const int cap = (int)min((long long)a.table_stride * a.page.d, 1ll << 30);
  const int per = a.n_kv * a.rb_own;
  auto len_of = [&](int b) {
    if (b >= a.B) return 0;
    const int n = a.kv_len[b];
    if (n > cap && blockIdx.x == 0) set_error(a.err, QE_ERR_INVALID_ARG);
    return max(0, min(n, cap));
  };
  auto places_of = [&](int len) { return len > 0 ? (len + kTile - 1) / kTile + kSegmentCost : 0; };
  auto block_scan = [&](long long v) {  // {inclusive sum, total} over the CTA
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += u;
    }
    __syncthreads();
    if (lane == 31) sh.sum[warp] = v;
    __syncthreads();
    long long all = 0;
#pragma unroll
    for (int i = 0; i < kAttnThreads / 32; ++i) {
      const long long s = sh.sum[i];
      if (i < warp) v += s;
      all += s;
    }
    return make_longlong2(v, all);
  };
  int len = len_of(threadIdx.x);
  long long mine = places_of(len);
  for (int b = threadIdx.x + kAttnThreads; b < a.B; b += kAttnThreads) mine += places_of(len_of(b));
  longlong2 scan = block_scan(mine);
  const Deal deal(a, scan.y * per);
  const long long t0 = deal.own_start(blockIdx.x), t1 = deal.own_start(blockIdx.x + 1);
  if (threadIdx.x == 0) {
    a.own_start[blockIdx.x] = t0;
    if (blockIdx.x == gridDim.x - 1) a.own_start[gridDim.x] = deal.own;
  }
  if (t0 < t1) {
    long long before = 0;  // places of the rows of earlier passes, per key head and row block
    for (int b0 = 0; b0 < a.B && before * per <= t0; b0 += kAttnThreads) {
      if (a.B > kAttnThreads) {
        len = len_of(b0 + threadIdx.x);
        scan = block_scan(places_of(len));
      }
      const long long end = (before + scan.x) * per, start = end - (long long)places_of(len) * per;
      if (start <= t0 && t0 < end) {
        sh.found = b0 + threadIdx.x;
        sh.found_len = len;
        sh.found_start = start;
      }
      before += scan.y;
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *(volatile uint32_t*)&sh.tmem;
  if (t0 < t1 || blockIdx.x < deal.grouped) {  // uniform over the CTA
    if (warp < kSoftWarps) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
      soften<T, D>(a, sh, ps, tmem);
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
      if (warp < kSoftWarps + kProdWarps) {
        produce<T, D>(a, &k_map, &v_map, sh, ring, qs);
      } else if (warp == 12) {
        multiply<T, D>(a, sh, ring, qs, ps, uniform(tmem));
        __syncwarp();
      } else if (warp == 13) {
        if (lane == 0) deal_out<D>(a, deal, t0, t1, sh.found, sh.found_len, sh.found_start, cap, sh);
        __syncwarp();
      }
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 12) {
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// Joins the segments of each row, prefix first, then own, in the order of their
// CTAs.  WPR warps take a row's segments in turn and are added up in order.
template <typename T, int D, int WPR>
__global__ void __launch_bounds__(128) qe_attn_join_kernel(const __grid_constant__ AttnArgs a) {
  __shared__ float sh_l[4];
  __shared__ float sh_o[4][D];
  constexpr int max_rows = Shape<D>::kRows;
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, share = warp % WPR;
  const int rows = a.B * a.n_q, row = blockIdx.x * (4 / WPR) + warp / WPR;
  const bool real = row < rows;
  const int at_row = real ? row : 0, b = at_row / a.n_q, hq = at_row - b * a.n_q, h = hq / a.G, g = hq - h * a.G;
  // what says where the row's segments are, in one round of loads
  const int unit = (b * a.n_kv + h) * a.rb_own + g / max_rows;
  const int kv = real ? a.kv_len[b] : -1;
  const int2 groups = a.prefix_tiles > 0 ? a.prefix_groups[h] : make_int2(0, -1);
  const int2 ctas = a.table_stride > 0 ? a.own_ctas[unit] : make_int2(0, -1);
  const int g0 = groups.x, np = kv >= 0 ? groups.y - groups.x + 1 : 0;
  const int c0 = ctas.x, no = kv > 0 ? ctas.y - ctas.x + 1 : 0;  // (a row of no keys: an old or no value, not used)
  // segment i of this row; false if that CTA had no own tiles (its slot holds anything then)
  auto where = [&](int i, const float2** ml, const float** o, bool* has) {
    const bool prefix = i < np;
    const int c = prefix ? 0 : c0 + i - np;
    const size_t at = prefix ? (size_t)(g0 + i + h) * a.B * a.G + (size_t)b * a.G + g : (size_t)(c + unit) * a.own_rows + g % max_rows;
    *ml = (prefix ? a.ml_prefix : a.ml_own) + at * 4;
    *o = (prefix ? a.part_prefix : a.part_own) + at * D;
    *has = a.own_start[c] < a.own_start[c + 1] || prefix;
  };
  constexpr int E = D / 32;
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  float m = -kNoRef, l = 0.f;
  // segments share, share + WPR, ... of this row, 32 in a pass: lane k has the k-th's m and l
#pragma unroll 1
  for (int i0 = share; i0 < np + no; i0 += 32 * WPR) {
    const int i = i0 + lane * WPR;
    float2 ml = make_float2(-kNoRef, 0.f);
    const float* o = nullptr;
    bool has = false;
    if (i < np + no) {
      const float2* p;
      where(i, &p, &o, &has);
      const float4 u = *reinterpret_cast<const float4*>(p), v = *reinterpret_cast<const float4*>(p + 2);
      if (has) ml = make_float2(u.x, (u.y + u.w) + (v.y + v.w));
    }
    const float top = fmaxf(m, warp_max(ml.x)), f0 = exp2_approx(m - top), f = has ? exp2_approx(ml.x - top) : 0.f;
    m = top;
    l = fmaf(f, ml.y, l * f0);  // per lane
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= f0;
    const int n = min(32, (np + no - i0 + WPR - 1) / WPR);
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const float w = __shfl_sync(0xffffffffu, f, k);
      const float* p = (const float*)__shfl_sync(0xffffffffu, (unsigned long long)(has ? o : nullptr), k);
      if (!p) continue;
      float v[E];
      if constexpr (E == 2) {
        *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(p + lane * E);
      } else {
#pragma unroll
        for (int e = 0; e < E; e += 4) *reinterpret_cast<float4*>(v + e) = *reinterpret_cast<const float4*>(p + lane * E + e);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(w, v[e], acc[e]);
    }
  }
  l = warp_sum(l);
  if constexpr (WPR > 1) {
    if (lane == 0) sh_l[warp] = m;
    __syncthreads();
    float top = m;
#pragma unroll
    for (int i = 0; i < WPR; ++i) top = fmaxf(top, sh_l[i]);
    const float f = exp2_approx(m - top);
    m = top;
    __syncthreads();
    if (lane == 0) sh_l[warp] = l * f;
#pragma unroll
    for (int e = 0; e < E; ++e) sh_o[warp][lane * E + e] = acc[e] * f;
    __syncthreads();
    if (share != 0) return;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
    for (int i = 0; i < WPR; ++i) {
      l += sh_l[i];
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += sh_o[i][lane * E + e];
    }
  }
  if (kv < 0) return;
  if (kv > 0 && a.table_stride == 0 && lane == 0) set_error(a.err, QE_ERR_INVALID_ARG);
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // a NaN sum stays one
  uint32_t* out = reinterpret_cast<uint32_t*>((T*)a.out + (size_t)b * a.out_stride + (size_t)hq * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) out[e / 2] = pack2<T>(acc[e] * inv, acc[e + 1] * inv);
  if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// Sizes that depend on the shape alone, whatever the lengths.
struct AttnPlan {
  int grid, max_rows, rb_own, rb_prefix, own_rows, groups;
  size_t off_cta, off_own, off_groups, off_mlp, off_mlo, off_pp, off_po, total;
};
AttnPlan attn_plan(int n_kv, int n_q, int D, int B, int sms) {
  AttnPlan p{};
  const int G = n_q / n_kv;
  p.grid = sms;
  p.max_rows = D == 256 ? Shape<256>::kRows : Shape<128>::kRows;
  p.rb_own = (G + p.max_rows - 1) / p.max_rows;
  p.rb_prefix = (B * G + p.max_rows - 1) / p.max_rows;
  p.own_rows = G < p.max_rows ? G : p.max_rows;
  // a segment's slot: its CTA (or group) plus its block's (or key head's) number
  p.groups = p.rb_prefix <= p.grid ? p.grid / p.rb_prefix : 1;
  const size_t rows_p = (size_t)(p.groups + n_kv) * B * G;
  const size_t rows_o = ((size_t)p.grid + (size_t)B * n_kv * p.rb_own) * p.own_rows;
  size_t off = sizeof(WsControl);
  auto take = [&](size_t bytes) { const size_t o = off; off = (off + bytes + 255) & ~(size_t)255; return o; };
  p.off_cta = take(8 * ((size_t)p.grid + 1));
  p.off_own = take(sizeof(int2) * (size_t)B * n_kv * p.rb_own);
  p.off_groups = take(sizeof(int2) * (size_t)n_kv);
  p.off_mlp = take(4 * sizeof(float2) * rows_p);
  p.off_mlo = take(4 * sizeof(float2) * rows_o);
  p.off_pp = take(4 * rows_p * D);
  p.off_po = take(4 * rows_o * D);
  p.total = off;
  return p;
}

// Tensor map of one half of the cache, {head_dim, n_kv * page_size, n_pages}, in boxes
// of 64 dims x `rows`.  False if there is none (the kernel then copies by rows).
bool cache_map(CUtensorMap* map, const qe_kv_cache* c, void* base, int64_t page_stride, int rows) {
  typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static std::atomic<void*> entry{nullptr};
  void* fn = entry;
  if (!fn) {
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess || !fn) {
      (void)cudaGetLastError();
      return false;
    }
    entry = fn;
  }
  const cuuint64_t dims[3] = {(cuuint64_t)c->head_dim, (cuuint64_t)c->n_kv * c->page_size, (cuuint64_t)c->n_pages};
  const cuuint64_t strides[2] = {(cuuint64_t)c->head_dim * 2, (cuuint64_t)page_stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)rows, 1}, step[3] = {1, 1, 1};
  return ((Encode)fn)(map, c->dtype == QE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, base,
                      dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct CacheMaps {
  CUtensorMap k, v;
};

template <typename T, int D>
cudaError_t launch_attn_t(const AttnArgs& a, const CacheMaps& m, int grid, cudaStream_t s) {
  static std::atomic<bool> set[64];  // per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!set[dev]) {
    e = cudaFuncSetAttribute(qe_attn_part_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D>::kSmem);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kAttnThreads);
  cfg.dynamicSmemBytes = Shape<D>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, qe_attn_part_kernel<T, D>, a, m.k, m.v);
  if (e != cudaSuccess) return e;
  const long long rows = (long long)a.B * a.n_q;
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  // few rows have many segments each: four warps a row; many rows have few
  if (rows < 8ll * grid) {
    cfg.gridDim = dim3((unsigned)rows);
    return cudaLaunchKernelEx(&cfg, qe_attn_join_kernel<T, D, 4>, a);
  }
  cfg.gridDim = dim3((unsigned)((rows + 3) / 4));
  return cudaLaunchKernelEx(&cfg, qe_attn_join_kernel<T, D, 1>, a);
}

template <typename T>
cudaError_t launch_attn(const AttnArgs& a, const CacheMaps& m, int D, int grid, cudaStream_t s) {
  if (D == 64) return launch_attn_t<T, 64>(a, m, grid, s);
  if (D == 128) return launch_attn_t<T, 128>(a, m, grid, s);
  return launch_attn_t<T, 256>(a, m, grid, s);
}

int check_attn_shape(const qe_kv_cache* c, int n_q, int B) {
  int rc = check_kv_cache(c);
  if (rc) return rc;
  if (n_q < 1 || n_q > kMaxHeads || n_q % c->n_kv)
    return fail(QE_ERR_INVALID_ARG, "n_q must be a positive multiple of n_kv <= %d (got %d, n_kv %d)", kMaxHeads, n_q, c->n_kv);
  if (B < 0 || B > kMaxBatch) return fail(QE_ERR_INVALID_ARG, "B must be in [0, %d] (got %d)", kMaxBatch, B);
  return QE_OK;
}

}  // namespace
}  // namespace qe

using namespace qe;

extern "C" QE_API size_t attn_workspace_bytes(const qe_kv_cache* c, int n_q, int B) {
  if (check_attn_shape(c, n_q, B) != QE_OK) return 0;
  const int sms = dev_info().sms;
  return attn_plan(c->n_kv, n_q, c->head_dim, B > 0 ? B : 1, sms > 0 ? sms : 148).total;
}

extern "C" QE_API int attn_decode_step(const qe_kv_cache* c, int B, int n_q, const void* q, int64_t q_stride,
                                       const int32_t* prefix_pages, int prefix_len, const int32_t* table,
                                       int table_stride, const int32_t* kv_len, float scale, void* out,
                                       int64_t out_stride, float* lse, void* ws, size_t ws_bytes, qe_stream_t stream) {
  int rc = check_attn_shape(c, n_q, B);
  if (rc) return rc;
  if (prefix_len < 0 || prefix_len >= 1 << 30) return fail(QE_ERR_INVALID_ARG, "prefix_len must be in [0, 2^30) (got %d)", prefix_len);
  if (table_stride < 0 || (int64_t)table_stride * c->page_size >= 1ll << 30)
    return fail(QE_ERR_INVALID_ARG, "table_stride * page_size must be in [0, 2^30)");
  // at 0x1p64 a scale times log2 e is far from the end of fp32
  if (!(scale >= 0.f && scale <= 0x1p64f)) return fail(QE_ERR_INVALID_ARG, "scale must be in [0, 2^64] (got %g)", scale);
  if (B == 0) return QE_OK;
  const int D = c->head_dim;
  if ((rc = check_ptr(q, "q", false, 16)) || (rc = check_ptr(out, "out", false, 16)) || (rc = check_ptr(kv_len, "kv_len")) ||
      (rc = check_ptr(table, "table", table_stride == 0)) || (rc = check_ptr(prefix_pages, "prefix_pages", prefix_len == 0)) ||
      (rc = check_ptr(lse, "lse", true)))
    return rc;
  if ((q_stride | out_stride) & 7) return fail(QE_ERR_INVALID_ARG, "row strides must be multiples of 8 elements");
  if (B > 1 && (q_stride < (int64_t)n_q * D || out_stride < (int64_t)n_q * D))
    return fail(QE_ERR_INVALID_ARG, "row strides must cover a row's heads");
  const size_t row = 2 * (size_t)n_q * D;
  if (rows_overlap({out, row, 2 * (size_t)out_stride, B}, {q, row, 2 * (size_t)q_stride, B}))
    return fail(QE_ERR_INVALID_ARG, "out overlaps q");
  if (!ws || ((uintptr_t)ws & 255)) return fail(QE_ERR_INVALID_ARG, "workspace must be a 256-byte aligned device pointer");
  const int sms = dev_info().sms;
  const AttnPlan p = attn_plan(c->n_kv, n_q, D, B, sms > 0 ? sms : 148);
  if (ws_bytes < p.total) return fail(QE_ERR_INVALID_ARG, "workspace too small: %zu < %zu bytes", ws_bytes, p.total);
  AttnArgs a{};
  char* w = (char*)ws;
  a.q = q; a.out = out; a.kc = c->k; a.vc = c->v;
  a.q_stride = q_stride; a.out_stride = out_stride;
  a.k_page_stride = c->k_page_stride; a.v_page_stride = c->v_page_stride;
  a.prefix_pages = prefix_pages; a.table = table; a.kv_len = kv_len; a.lse = lse;
  a.err = &((WsControl*)ws)->err;
  a.own_start = (long long*)(w + p.off_cta);
  a.own_ctas = (int2*)(w + p.off_own);
  a.prefix_groups = (int2*)(w + p.off_groups);
  a.ml_prefix = (float2*)(w + p.off_mlp); a.ml_own = (float2*)(w + p.off_mlo);
  a.part_prefix = (float*)(w + p.off_pp); a.part_own = (float*)(w + p.off_po);
  a.B = B; a.n_q = n_q; a.n_kv = c->n_kv; a.G = n_q / c->n_kv; a.n_pages = c->n_pages;
  a.table_stride = table_stride; a.prefix_len = prefix_len;
  a.prefix_tiles = (prefix_len + kTile - 1) / kTile;
  const long long line = (long long)a.prefix_tiles * c->n_kv;
  a.groups = line > 0 && line < p.groups ? (int)line : p.groups;
  a.rb_prefix = p.rb_prefix; a.rb_own = p.rb_own; a.own_rows = p.own_rows;
  // never 0: a masked score is -inf, which stays so times any other number.  The smallest one
  // turns scores below 2^64 into less than 2^-84, whose numerators are 1 as for a scale of 0.
  a.scale_log2 = fmaxf(scale * kLog2e, 0x1p-149f);
  a.page = fast_div((uint32_t)c->page_size);
  a.group = fast_div((uint32_t)a.G);
  // a wide tile of two blocks of 128 rows takes about twice a narrow one's time
  a.prefix_cost = (long long)B * a.G > 128 && p.max_rows > 128 ? 2 : 1;
  // A role may have to wait for as long as another's segment takes (a softmax group without rows
  // for a whole prefix), so the limit grows with the tiles that one CTA can have.
  const long long prefix_ctas = line == 0 ? 0 : p.rb_prefix <= p.grid ? (long long)a.groups * p.rb_prefix : p.grid;
  const long long cap = (long long)table_stride * c->page_size, own = (long long)B * c->n_kv * p.rb_own * (cap / kTile + 2);
  const long long tiles = (line == 0 ? 0 : p.rb_prefix <= p.grid ? line / a.groups + 1 : line * (p.rb_prefix / p.grid + 1)) +
                          own / (prefix_ctas < p.grid ? p.grid - prefix_ctas : p.grid) + 1;
  a.budget_ns = wait_budget_ns() + (unsigned long long)tiles * a.prefix_cost * kTileNs;
  CacheMaps m{};
  int bits = 0;
  while (bits < 5 && !((c->page_size >> bits) & 1)) ++bits;
  if (bits >= 3 && c->n_pages > 0 && cache_map(&m.k, c, c->k, c->k_page_stride, 1 << bits) &&
      cache_map(&m.v, c, c->v, c->v_page_stride, 1 << bits))
    a.run_bits = bits;
  const cudaError_t e = c->dtype == QE_BF16 ? launch_attn<__nv_bfloat16>(a, m, D, p.grid, (cudaStream_t)stream)
                                            : launch_attn<__half>(a, m, D, p.grid, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "attn_decode_step launch");
  return QE_OK;
}
