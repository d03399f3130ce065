// qe_sample.cu -- the next token of each row from its logits and a given
// uniform number: temperature, top-k, top-p and min-p.
//
// With x_max the row's largest logit, e_i = exp((x_i - x_max) / temperature).
// The candidates in descending order of x (ties: lower index first) are cut to
// the first top_k; of those to the shortest run whose mass reaches top_p of
// theirs; of those to e_i >= min_p.  The token is the first index i (ascending)
// at which the running sum of the kept e exceeds u times their total.
//
// A token is a whole number: it changes when a running sum crosses u times the
// total, so the sums have to be the same whoever adds them up in whichever
// order.  Each e_i is computed in fp64 and rounded to a multiple of 2^-S,
// S = 62 - ceil(log2 V) (at most 46), and the sums are exact 64-bit integers.
// The rounding moves a border by at most V 2^-(S+1) of the largest weight; a
// weight below 2^-(S+1) of it counts as 0.
//
// A cluster of CTAs shares a row.  Few rows: each CTA holds its run of the row as stored in its
// shared memory, so that the row is read once; a thread owns an odd number of
// consecutive 16-byte pieces, so that threads are in index order (which the
// running sums need) and their 16-byte reads fall on different banks.  Many rows
// (STREAM): the shared memory would leave few rows at work at a time (18 of 800 KB),
// so that four CTAs a row (eight for more than 262144 logits) read it from global memory,
// mostly the L2 cache, in every pass, each warp a run of its own, and 74 rows are at work.  Measured at 256 rows of
// 200000 fp32 logits: 443 us from shared memory (16 CTAs a row), streamed by 1, 2, 4
// and 8 CTAs a row 388, 268, 250 and 301 us; at 64 rows of 100003 bf16 logits 64 us and
// (by 4) 85 us.
//
// What costs time is the weights (a dozen fp64 operations each) and the
// cluster's barriers, so both are avoided:
//   - candidates: a bound on x_max - x that holds for every token that can be
//     kept comes from min_p, from a histogram of the threads' largest logits (the
//     k-th largest of them is at most the k-th largest logit), or from a histogram
//     of the weights over x_max - x.  Up to 2048 candidates are gathered, in index
//     order, by the first CTA, which sorts them and finishes alone;
//   - otherwise the cut is found without a sort: the histogram (2048 bins, 8
//     mantissa bits of 8 binades), summed over the cluster through distributed
//     shared memory, gives the bin in which the k-th token or the top_p mass
//     lies; further histograms over the bin's order-preserving keys, 11 bits at a
//     time, give the key itself.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
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

typedef unsigned long long u64;

constexpr int kSampleThreads = 512;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kBinBits = 11, kBins = 1 << kBinBits;
constexpr int kBinShift = 15;                // 8 mantissa bits of x_max - x
constexpr int kBinBias = (127 - 3) << 8;  // bin 0: below 2^-3 (1 + 2^-8); the last: from 2^5 on
constexpr int kMaxCand = 2048;
constexpr int kStreamCluster = 4;
constexpr int kAhead = 2;   // STREAM: 16-byte pieces a thread has on their way
constexpr int kGroups = 4;  // groups of a thread's logits of which the largest is kept
constexpr int kMaxVocab = 1 << 19;
constexpr int kMaxCluster = 16;
// Logits of one CTA.  The histogram adds 16-bit pieces of the weights in 32-bit words:
// 2^16 of them in one bin make less than 2^32.
constexpr int kMaxRun = 1 << 16;
constexpr int kRowBytes = 72 * 1024;  // of a CTA's run in shared memory, while more CTAs a row can be had
static_assert(kRowBytes / 2 <= kMaxRun && kMaxVocab / kMaxCluster <= kMaxRun, "runs on chip");

struct SampleArgs {
  const void* logits;
  long long stride;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int32_t* token;
  float* logprob;
  int B, V, shift, run;  // run: elements of the row per CTA
  int cluster;
  int smem_row;  // bytes of the row's run in shared memory
};

// 2^(i / 32): the table of a table-driven exponential (Tang, "Table-driven
// implementation of the exponential function in IEEE floating-point
// arithmetic", ACM TOMS 15, 1989), filled once per CTA; a copy for each pair of
// banks, so that the lanes of a half warp never meet.
constexpr int kExpTable = 32, kExpCopies = 16;

struct SampleShared {
  double exp2_table[kExpTable][kExpCopies];
  u64 xch[2][kMaxCluster];   // all-gather slots, two in turn
  u64 warp_sum[kSampleWarps];
  u64 found[2][3];           // crossing bin, the sum above it and its own
  union {
    unsigned piece[3][kBins];  // histogram: sums of 16-bit pieces of the weights,
    u64 sum[kBins];            // then put together in the same place
    struct {
      u64 cand[kMaxCand];   // {index, logit} in index order
      u64 order[kMaxCand];  // {key, ~place} to be sorted; the buffers of block_sort
    } few;
  };
};

QE_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
QE_DEV void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
QE_DEV void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
QE_DEV void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
QE_DEV uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
QE_DEV void st_peer64(uint32_t a, u64 v) { asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory"); }
QE_DEV u64 ld_peer64(uint32_t a) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}

// Order-preserving key of a logit: larger logit, larger key; -0 as +0; NaN as -inf.
QE_DEV uint32_t key_of(float x) {
  x = x == x ? x + 0.f : -INFINITY;
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

QE_DEV float logit_of(uint32_t key) { return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key); }

template <typename T>
struct Elems;
template <>
struct Elems<float> {
  static constexpr int N = 4, kKeyShift = 0;
  static QE_DEV void get(const uint4& w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y); x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
  }
  static QE_DEV float lowest() { return -INFINITY; }
};
template <typename T>
struct Elems {
  // a 16-bit logit as fp32 has this many low zero bits, and so has its key
  static constexpr int N = 8, kKeyShift = std::is_same<T, __half>::value ? 13 : 16;
  static QE_DEV void get(const uint4& w, float (&x)[8]) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<T>(v[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  static QE_DEV T lowest() { return (T)(-INFINITY); }
};

QE_DEV u64 warp_scan(u64 v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const u64 x = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += x;
  }
  return v;
}

// Descending, one value a thread: a bitonic sort, by shuffles within a warp and through
// two buffers of kSampleThreads in turn beyond it.
template <typename V>
QE_DEV V block_sort(V v, V* buf) {
  const int tid = threadIdx.x;
  int turn = 0;
  __syncthreads();
#pragma unroll 1
  for (int k = 2; k <= kSampleThreads; k *= 2)
#pragma unroll 1
    for (int j = k / 2; j > 0; j /= 2) {
      V o;
      if (j >= 32) {
        buf[turn + tid] = v;
        __syncthreads();
        o = buf[turn + (tid ^ j)];
        turn ^= kSampleThreads;
      } else {
        o = __shfl_xor_sync(0xffffffffu, v, j);
      }
      const bool larger = ((tid & j) == 0) == ((tid & k) == 0);
      v = (o > v) == larger ? o : v;
    }
  return v;
}

template <typename T, bool STREAM>
struct Row {
  static constexpr int N = Elems<T>::N;
  const SampleArgs& a;
  SampleShared& sh;
  const uint4* data;   // the run as stored; its first piece holds element `first` at 0
  int pieces, per;     // pieces of the run, and of a thread (STREAM: of a warp)
  u64 cta_before = 0, cta_sum = 0;  // of the CTA, as running() last found it
  int lo, hi;          // STREAM: elements [lo, hi) from `first` are the row's
  int first;           // index in the row of element 0 of piece 0 (may be below the run's start)
  uint32_t rank, size;
  int turn = 0, turn_found = 0;
  float x_max = 0.f;
  double inv_t = 1.0, scale = 1.0;
  float thr = -INFINITY;  // kept: x > thr, or x == thr and index < cut
  int cut = 0;

  QE_DEV Row(const SampleArgs& a_, SampleShared& s_) : a(a_), sh(s_) {}

  // Piece p of the row in global memory; what is not the row's counts as -inf.
  QE_DEV uint4 piece_at(int p) const {
    if (p * N >= lo && (p + 1) * N <= hi) return __ldg(data + p);
    uint4 w;
    T* t = reinterpret_cast<T*>(&w);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int i = p * N + e;
      t[e] = i >= lo && i < hi ? reinterpret_cast<const T*>(data)[i] : Elems<T>::lowest();
    }
    return w;
  }
  QE_DEV float element(int i) const { return (float)reinterpret_cast<const T*>(data)[i - first]; }  // of index i

  // f(x, index) over this thread's elements: consecutive ones in index order; STREAM: every
  // 32nd piece of the warp's run
  template <typename F>
  QE_DEV void each(F f) const {
    if constexpr (STREAM) {
      const int p0 = (threadIdx.x >> 5) * per, p1 = min(pieces, p0 + per);
      // The row's first and last piece may be partial: the lanes that have them take them
      // by elements, so that the loop's loads are plain ones, kAhead pieces on their way
      // while as many are worked on.
      const int lane = threadIdx.x & 31, head = lo > 0, tail = hi < pieces * N;
#pragma unroll 1
      for (int side = 0; side < 2; ++side) {
        const int p = side ? pieces - 1 : 0;
        if (!(side ? tail && (pieces > 1 || !head) : head) || p < p0 || p >= p1 || lane != 0) continue;
#pragma unroll 1
        for (int i = max(lo, p * N); i < min(hi, (p + 1) * N); ++i) f(element(first + i), first + i);
      }
      const int end = min(p1, pieces - tail);
      int p = max(p0, head) + lane;
      uint4 q[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (p + 32 * u < end) q[u] = __ldg(data + p + 32 * u);
#pragma unroll 1
      for (; p < end; p += 32 * kAhead) {
        uint4 n[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          if (p + 32 * (kAhead + u) < end) n[u] = __ldg(data + p + 32 * (kAhead + u));
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          if (p + 32 * u < end) {
            float x[N];
            Elems<T>::get(q[u], x);
#pragma unroll
            for (int e = 0; e < N; ++e) f(x[e], first + (p + 32 * u) * N + e);
          }
          q[u] = n[u];
        }
      }
    } else {
      const int p0 = threadIdx.x * per, p1 = min(pieces, p0 + per);
      for (int p = p0; p < p1; ++p) {
        float x[N];
        Elems<T>::get(data[p], x);
#pragma unroll
        for (int e = 0; e < N; ++e) f(x[e], first + p * N + e);
      }
    }
  }

  // All CTAs of the row, with what they wrote to each other.
  QE_DEV void sync_all() const { cluster_sync(); }
  // Every CTA's v, by rank, in the returned array (valid until the next but one call).
  QE_DEV const u64* all_gather(u64 v) {
    u64* slots = sh.xch[turn];
    turn ^= 1;
    if (threadIdx.x < size) st_peer64(peer_addr(slots + rank, threadIdx.x), v);
    sync_all();
    return slots;
  }
  // Weight of a logit as a multiple of 2^-S: e^y = 2^(k / 32) e^r with k the whole
  // number nearest to 32 y / ln 2 (left in the low bits by adding 1.5 2^52) and
  // |r| <= ln 2 / 64, where five terms after 1 leave r^6 / 720 = 2.3e-15.  The product
  // is below 2^52, so adding 2^52 rounds it to a whole number in the low bits.  No
  // branch: the elements of a piece are worked on side by side.  Below -45 (2^-64), and
  // for -inf and NaN, whatever comes out is dropped.
  // INF: the row's largest logit is +inf, and only its equals weigh.
  template <bool INF>
  QE_DEV u64 weight(float x) const {
    if constexpr (INF) return x == INFINITY ? (u64)1 << a.shift : 0;
    const double y = ((double)x - (double)x_max) * inv_t;
    const double km = fma(y, 46.166241308446828, 6755399441055744.0);
    const double r = fma(6755399441055744.0 - km, 0.021660849392498291, y);
    const int k = __double2loint(km);
    double p = fma(r, 1.0 / 120.0, 1.0 / 24.0);
    p = fma(p, r, 1.0 / 6.0);
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    p *= sh.exp2_table[k & (kExpTable - 1)][threadIdx.x % kExpCopies];
    const double two = __hiloint2double((1023 + a.shift + (k >> 5)) << 20, 0);
    const u64 w = (u64)__double_as_longlong(fma(p, two, 4503599627370496.0)) & 0xfffffffffffffull;
    return y > -45.0 ? w : 0;
  }
  QE_DEV bool kept(float x, int i) const { return x > thr || (x == thr && i < cut); }  // thr -inf: all

  QE_DEV int coarse_bin(float x) const {
    if (!(x < x_max)) return x == x_max ? 0 : kBins - 1;
    const int b = (int)(__float_as_uint(x_max - x) >> kBinShift) - kBinBias;
    return min(max(b, 0), kBins - 1);
  }
  // Upper end of a bin's x_max - x; infinity for the last.
  QE_DEV static float bin_end(int bin) {
    return bin == kBins - 1 ? INFINITY : __uint_as_float((uint32_t)(bin + 1 + kBinBias) << kBinShift);
  }

  // Zeroes the histogram; a barrier has to follow before the first add.
  QE_DEV void hist_clear() {
    for (int i = threadIdx.x; i < 3 * kBins; i += kSampleThreads) (&sh.piece[0][0])[i] = 0;
  }
  QE_DEV void hist_add(int bin, u64 w) {
    const unsigned lo = (unsigned)w & 0xffffu, mid = (unsigned)(w >> 16) & 0xffffu, hi = (unsigned)(w >> 32);
    if (lo) atomicAdd(&sh.piece[0][bin], lo);
    if (mid) atomicAdd(&sh.piece[1][bin], mid);
    if (hi) atomicAdd(&sh.piece[2][bin], hi);
  }
  // The cluster's histogram, in slices: thread t of CTA r gets the sums of the bins
  // first_bin() ..., their running sum before them and the total.
  struct Sums {
    u64 v[kBins / kSampleThreads], before, total;
  };
  QE_DEV int slice() const { return kBins / size; }  // size is a power of two
  QE_DEV int per_slot() const { return slice() >= kSampleThreads ? slice() / kSampleThreads : 1; }
  QE_DEV Sums hist_sums() {
    u64 put[kBins / kSampleThreads];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kBins / kSampleThreads; ++j) {
      const int i = threadIdx.x + j * kSampleThreads;
      put[j] = (u64)sh.piece[0][i] + ((u64)sh.piece[1][i] << 16) + ((u64)sh.piece[2][i] << 32);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kBins / kSampleThreads; ++j) sh.sum[threadIdx.x + j * kSampleThreads] = put[j];
    sync_all();  // every CTA's sums are there
    Sums s;
    const int m = per_slot();
    u64 sum = 0;
#pragma unroll
    for (int j = 0; j < kBins / kSampleThreads; ++j) {
      s.v[j] = 0;
      const int i = threadIdx.x * m + j;
      if (j < m && i < slice()) {
        u64 x[4] = {0, 0, 0, 0};
        for (uint32_t r = 0; r < size; r += 4)
#pragma unroll
          for (uint32_t k = 0; k < 4; ++k)
            if (r + k < size) x[k] += ld_peer64(peer_addr(&sh.sum[rank * slice() + i], r + k));
        s.v[j] = (x[0] + x[1]) + (x[2] + x[3]);
      }
      sum += s.v[j];
    }
    u64 scan = warp_scan(sum);
    __syncthreads();
    if ((threadIdx.x & 31) == 31) sh.warp_sum[threadIdx.x >> 5] = scan;
    __syncthreads();
    u64 all = 0;
#pragma unroll
    for (int w = 0; w < kSampleWarps; ++w) {
      if (w < (int)(threadIdx.x >> 5)) scan += sh.warp_sum[w];
      all += sh.warp_sum[w];
    }
    const u64* slices = all_gather(all);
    s.before = scan - sum;
    s.total = 0;
    for (uint32_t r = 0; r < size; ++r) {
      if (r < rank) s.before += slices[r];
      s.total += slices[r];
    }
    return s;
  }
  // The bin in which the sums, bin 0 first, reach `target` (1 <= target; at most the
  // total, the same in all CTAs, so that they agree whatever the logits are); above: the
  // sum before it; in_bin: its own.  All CTAs get it.
  QE_DEV int crossing(const Sums& s, u64 target, u64* above, u64* in_bin = nullptr) {
    *above = 0;
    if (in_bin) *in_bin = 0;
    if (s.total == 0) return kBins - 1;
    target = min(target, s.total);
    u64* out = sh.found[turn_found];
    turn_found ^= 1;
    u64 before = s.before;
#pragma unroll
    for (int j = 0; j < kBins / kSampleThreads; ++j) {
      if (before < target && target <= before + s.v[j])
        for (uint32_t r = 0; r < size; ++r) {
          st_peer64(peer_addr(out, r), (u64)(rank * slice() + threadIdx.x * per_slot() + j));
          st_peer64(peer_addr(out + 1, r), before);
          st_peer64(peer_addr(out + 2, r), s.v[j]);
        }
      before += s.v[j];
    }
    sync_all();
    *above = out[1];
    if (in_bin) *in_bin = out[2];
    return (int)out[0];
  }

  // Sum of w over the row; mine, before: this thread's (STREAM: warp's) part and what
  // comes before it.
  template <typename F>
  QE_DEV u64 running(F w, u64* mine, u64* before) {
    u64 m = 0;
    each([&](float x, int i) { m += w(x, i); });
    u64 scan = warp_scan(m);
    __syncthreads();
    if ((threadIdx.x & 31) == 31) sh.warp_sum[threadIdx.x >> 5] = scan;
    __syncthreads();
    if constexpr (STREAM) scan = m = sh.warp_sum[threadIdx.x >> 5];
    u64 all = 0;
#pragma unroll
    for (int k = 0; k < kSampleWarps; ++k) {
      if (k < (int)(threadIdx.x >> 5)) scan += sh.warp_sum[k];
      all += sh.warp_sum[k];
    }
    const u64* runs = all_gather(all);
    u64 total = 0;
    cta_before = 0;
    cta_sum = all;
    for (uint32_t r = 0; r < size; ++r) {
      if (r < rank) cta_before += runs[r];
      total += runs[r];
    }
    *mine = m;
    *before = cta_before + scan - m;
    return total;
  }
  // In the warp in whose part the running sum exceeds `target` (below the total): the
  // first such index; -1 in the others.  All threads call it, with what running() gave.
  // The part is shared out: among the lanes (STREAM: among all warps, then the lanes).
  template <typename F>
  QE_DEV int place_of(F w, u64 mine, u64 before, u64 target) {
    const int lane = threadIdx.x & 31;
    bool here = before <= target && target < before + mine;
    if constexpr (STREAM) {
      const int warp = threadIdx.x >> 5;
      u64* at = sh.found[turn_found];
      turn_found ^= 1;
      if (!(cta_before <= target && target < cta_before + cta_sum)) return -1;  // not in this CTA
      if (here && lane == 0) {
        at[0] = (u64)warp;
        at[1] = before;
      }
      __syncthreads();
      const int s0 = (int)at[0] * per, s1 = min(pieces, s0 + per), part = (s1 - s0 + kSampleWarps - 1) / kSampleWarps;
      const int p0 = min(s1, s0 + warp * part), p1 = min(s1, p0 + part);
      auto piece_sum = [&](int p) {
        float x[N];
        Elems<T>::get(piece_at(p), x);
        u64 m = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) m += w(x[e], first + p * N + e);
        return m;
      };
      u64 m = 0;
      for (int p = p0 + lane; p < p1; p += 32) m += piece_sum(p);
      m = warp_scan(m);
      if (lane == 31) sh.warp_sum[warp] = m;
      __syncthreads();
      u64 base = at[1];
      for (int k = 0; k < warp; ++k) base += sh.warp_sum[k];
      if (!(base <= target && target < base + sh.warp_sum[warp])) return -1;
      for (int p = p0; p < p1; p += 32) {
        const u64 own = p + lane < p1 ? piece_sum(p + lane) : 0, scan = base + warp_scan(own);
        const unsigned past = __ballot_sync(0xffffffffu, scan > target);
        if (past) {
          const int src = __ffs(past) - 1;
          int found = -1;
          if (lane == src) {
            u64 sum = scan - own;
            float x[N];
            Elems<T>::get(piece_at(p + lane), x);
#pragma unroll
            for (int e = 0; e < N; ++e) {
              sum += w(x[e], first + (p + lane) * N + e);
              if (found < 0 && sum > target) found = first + (p + lane) * N + e;
            }
          }
          return __shfl_sync(0xffffffffu, found, src);
        }
        base = __shfl_sync(0xffffffffu, scan, 31);
      }
      return -1;
    } else {
      const unsigned owner = __ballot_sync(0xffffffffu, here);
      if (!owner) return -1;
      const int src = __ffs(owner) - 1, p0 = ((threadIdx.x & ~31) + src) * per;
      const int end = min(pieces, p0 + per) * N;
      u64 base = __shfl_sync(0xffffffffu, before, src);
      for (int e0 = p0 * N; e0 < end; e0 += 32) {
        const int e = e0 + lane;
        const u64 scan = base + warp_scan(e < end ? w(element(first + e), first + e) : 0);
        const unsigned past = __ballot_sync(0xffffffffu, scan > target);
        if (past) return first + e0 + __ffs(past) - 1;
        base = __shfl_sync(0xffffffffu, scan, 31);
      }
      return -1;
    }
  }
  // {index, logit} of the elements that f(x) picks, in index order, to the first CTA's
  // list; before: as running() counted them.
  template <typename F>
  QE_DEV void gather(F f, u64 before) const {
    uint32_t to = peer_addr(sh.few.cand, 0) + (uint32_t)before * 8;
    if constexpr (STREAM) {
      const int lane = threadIdx.x & 31, p0 = (threadIdx.x >> 5) * per, p1 = min(pieces, p0 + per);
      for (int p = p0; p < p1; p += 32) {
        float x[N];
        int n = 0;
        if (p + lane < p1) {
          Elems<T>::get(piece_at(p + lane), x);
#pragma unroll
          for (int e = 0; e < N; ++e) n += f(x[e]);
        }
        if (!__any_sync(0xffffffffu, n)) continue;
        int scan = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, scan, d);
          if (lane >= d) scan += o;
        }
        uint32_t at = to + (scan - n) * 8;
        if (n) {
#pragma unroll
          for (int e = 0; e < N; ++e)
            if (f(x[e])) {
              st_peer64(at, ((u64)(uint32_t)(first + (p + lane) * N + e) << 32) | __float_as_uint(x[e]));
              at += 8;
            }
        }
        to += __shfl_sync(0xffffffffu, scan, 31) * 8;
      }
    } else {
      each([&](float x, int i) {
        if (!f(x)) return;
        st_peer64(to, ((u64)(uint32_t)i << 32) | __float_as_uint(x));
        to += 8;
      });
    }
  }

  // Cuts the kept elements, in descending order, to the shortest run whose sum
  // of w reaches target (1 <= target <= their sum).  w is 0 for what is not kept.
  template <typename F, typename U>
  QE_DEV void cut_at(F w, U unit, int bin, u64 target) {
    // bin: the coarse bin that the run ends in; target: what is to be reached within it.
    // unit(x): what w is for a kept logit x.
    // Keys that the bin can hold: its bounds on x_max - x, widened by two
    // units in the last place of that difference
    constexpr int KS = Elems<T>::kKeyShift;
    uint32_t k_hi = key_of(x_max), k_lo = key_of(-INFINITY);
    const double d_lo = (double)__uint_as_float((uint32_t)(bin + kBinBias) << kBinShift), d_hi = (double)bin_end(bin);
    if (bin > 0) k_hi = min(k_hi, key_of(__double2float_ru((double)x_max - d_lo * (1.0 - 2.4e-7))));
    if (bin < kBins - 1) k_lo = x_max < INFINITY ? key_of(__double2float_rd((double)x_max - d_hi * (1.0 + 2.4e-7))) : k_hi;
    k_hi >>= KS;
    k_lo >>= KS;
    u64 in_bin;
    for (;;) {
      const uint32_t range = k_hi - k_lo;
      const int bits = 32 - __clz(range | 1);
      const int sh_bits = bits > kBinBits ? bits - kBinBits : 0;
      hist_clear();  // crossing() ends well after the last peer's read
      __syncthreads();
      // (a key beyond an infinity's, from the missing bits, gives NaN: that infinity)
      const float x_lo = fmaxf(logit_of(k_lo << KS), -INFINITY), x_hi = fminf(logit_of((k_hi << KS) | ((1u << KS) - 1)), INFINITY);
      each([&](float x, int i) {
        if (!(x >= x_lo && x <= x_hi)) return;  // the cheapest test first: few pass
        const uint32_t k = key_of(x) >> KS;
        if (k < k_lo || k > k_hi || coarse_bin(x) != bin) return;
        const u64 v = w(x, i);
        if (v) hist_add((int)((k_hi - k) >> sh_bits), v);
      });
      u64 above;
      const Sums sums = hist_sums();
      const int b = crossing(sums, target, &above, &in_bin);
      target -= above;
      k_hi -= (uint32_t)b << sh_bits;
      if (sh_bits == 0) break;
      const uint32_t width = (1u << sh_bits) - 1;
      k_lo = k_hi - k_lo > width ? k_hi - width : k_lo;
    }
    k_hi = (k_hi << KS) | (k_hi >> (31 - KS) ? 0u : (1u << KS) - 1);  // a negative logit's key has ones there
    // of the elements with this key, each of the same weight, as many of the lowest
    // indices as it takes; all of them where one fewer would not reach the target
    const float x_cut = logit_of(k_hi);
    int at = thr == x_cut ? cut : 0x7fffffff;
    if (in_bin - unit(x_cut) >= target) {
      auto tie = [&](float x, int i) -> u64 { return x == x_cut ? w(x, i) : 0; };
      u64 mine, before;
      running(tie, &mine, &before);
      const int last = place_of(tie, mine, before, target - 1);  // the tie that reaches the target
      u64* out = sh.found[turn_found];
      turn_found ^= 1;
      if (last >= 0 && (threadIdx.x & 31) < size) st_peer64(peer_addr(out, threadIdx.x & 31), (u64)last);
      sync_all();
      at = min(at, (int)out[0] + 1);
    }
    thr = x_cut;
    cut = at;
  }
};

// floor(x total) for an fp32 0 < x < 1, exactly; rest: whether something was cut off.
QE_DEV u64 part_of(float x, u64 total, bool* rest) {
  int e;
  const u64 f = (u64)(frexpf(x, &e) * 16777216.f);  // x = f 2^-s
  const int s = 24 - e;
  const u64 hi = __umul64hi(f, total), lo = f * total;
  if (s < 64) {
    *rest = (lo & (((u64)1 << s) - 1)) != 0;
    return (hi << (64 - s)) | (lo >> s);
  }
  if (s < 128) {
    *rest = lo != 0 || (s > 64 && (hi & (((u64)1 << (s - 64)) - 1)) != 0);
    return s == 64 ? hi : hi >> (s - 64);
  }
  *rest = true;
  return 0;
}
// The least whole number that is at least top_p total, and at least 1.
QE_DEV u64 mass_target(float top_p, u64 total) {
  if (!(top_p > 0.f)) return 1;
  bool rest;
  u64 t = part_of(top_p, total, &rest);
  if (rest) ++t;
  return t < 1 ? 1 : t;
}
QE_DEV u64 choice_target(float u, u64 total) {
  if (u >= 1.f) return total - 1;
  if (!(u > 0.f)) return 0;
  bool rest;
  return part_of(u, total, &rest);
}

// The cuts and the choice among n <= kMaxCand candidates in index order, by one CTA.
// target_p: the mass that top_p keeps, where that is known already (no top_k).
template <bool INF, typename T, bool STREAM>
QE_DEV void finish_few(const Row<T, STREAM>& r, int n, int top_k, bool cut_p, float top_p, u64 target_p, u64 least, float u, int row) {
  SampleShared& sh = r.sh;
  const SampleArgs& a = r.a;
  constexpr int P = kMaxCand / kSampleThreads;  // places per thread
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // running sums over places, thread t having places P t ..
  auto block_running = [&](u64 (&v)[P], u64* total) {
#pragma unroll
    for (int j = 1; j < P; ++j) v[j] += v[j - 1];
    u64 scan = warp_scan(v[P - 1]);
    __syncthreads();
    if (lane == 31) sh.warp_sum[warp] = scan;
    __syncthreads();
    u64 before = scan - v[P - 1], all = 0;
#pragma unroll
    for (int w = 0; w < kSampleWarps; ++w) {
      if (w < warp) before += sh.warp_sum[w];
      all += sh.warp_sum[w];
    }
#pragma unroll
    for (int j = 0; j < P; ++j) v[j] += before;
    *total = all;
  };
  auto logit = [&](u64 c) { return __uint_as_float((uint32_t)c); };
  u64 last = 0;  // the last kept candidate's {key, ~place}; all from it on are kept
  if (top_k > 0 || cut_p) {
    // descending by key, ascending by place
    auto item = [&](int i) -> u64 { return i < n ? ((u64)key_of(logit(sh.few.cand[i])) << 32) | (uint32_t)~i : 0; };
    if (n <= kSampleThreads) {
      const u64 x = block_sort<u64>(item(tid), sh.few.order);
      __syncthreads();
      sh.few.order[tid] = x;
      __syncthreads();
    } else {
      for (int i = tid; i < kMaxCand; i += kSampleThreads) sh.few.order[i] = item(i);
      __syncthreads();
      for (int k = 2; k <= kMaxCand; k *= 2)
        for (int j = k / 2; j > 0; j /= 2) {
          for (int i = tid; i < kMaxCand / 2; i += kSampleThreads) {
            const int lo = 2 * i - (i & (j - 1)), hi = lo + j;
            const u64 x = sh.few.order[lo], y = sh.few.order[hi];
            if ((x < y) == ((lo & k) == 0)) {
              sh.few.order[lo] = y;
              sh.few.order[hi] = x;
            }
          }
          __syncthreads();
        }
    }
    int keep = top_k > 0 && top_k < n ? top_k : n;
    if (cut_p) {
      u64 v[P], w[P], total;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const int i = P * tid + j;
        w[j] = v[j] = i < keep ? r.template weight<INF>(logit(sh.few.cand[(uint32_t)~sh.few.order[i]])) : 0;
      }
      block_running(v, &total);
      const u64 target = top_k > 0 ? mass_target(top_p, total) : target_p;
#pragma unroll
      for (int j = 0; j < P; ++j)
        if (v[j] - w[j] < target && target <= v[j]) sh.found[0][0] = P * tid + j + 1;
      if (tid == 0 && target > total) sh.found[0][0] = keep;  // the mass is reached below min_p
      __syncthreads();
      keep = (int)sh.found[0][0];
    }
    last = sh.few.order[keep - 1];
  }
  u64 v[P], w[P], total;
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const int i = P * tid + j;
    u64 x = 0;
    if (i < n) {
      const float l = logit(sh.few.cand[i]);
      if ((((u64)key_of(l) << 32) | (uint32_t)~i) >= last) x = r.template weight<INF>(l);
      if (x < least) x = 0;
    }
    w[j] = v[j] = x;
  }
  block_running(v, &total);
  const u64 target = choice_target(u, total);
#pragma unroll
  for (int j = 0; j < P; ++j)
    if (v[j] - w[j] <= target && target < v[j]) {
      a.token[row] = (int)(sh.few.cand[P * tid + j] >> 32);
      if (a.logprob) a.logprob[row] = (float)log((double)w[j] / (double)total);
    }
}

// The cuts and the choice, once the row's largest logit is known.
template <bool INF, typename T, bool STREAM>
QE_DEV void choose(Row<T, STREAM>& r, float best, const float (&group)[kGroups], float t, int k, float tp, float mp, float u,
                   int row) {
  using R = Row<T, STREAM>;
  SampleShared& sh = r.sh;
  const SampleArgs& a = r.a;
  u64 mine, before;
  u64 least = 1;  // of a kept weight
  if (mp > 0.f) least = max((u64)1, (u64)ceil((double)fminf(mp, 1.f) * (double)((u64)1 << a.shift)));
  const bool cut_k = k > 0 && k < a.V, cut_p = tp < 1.f;

  // A bound on x_max - x for the candidates, all tokens that can be kept
  float far = INFINITY;
  int bin = kBins - 1;
  u64 target_p = 0, above = 0;
  if (cut_k) {
    // the k-th largest of the largest logits of disjoint groups is at most the k-th largest logit
    if constexpr (STREAM) {
      r.hist_clear();
      __syncthreads();
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
        if (group[g] > -INFINITY) atomicAdd(&sh.piece[0][r.coarse_bin(group[g])], 1u);
      const typename R::Sums sums = r.hist_sums();
      if (sums.total >= (u64)k) far = R::bin_end(r.crossing(sums, (u64)k, &above));
    } else {
      // if each CTA has ceil(k / CTAs) threads whose largest logit is at least L, there are k such logits
      const int j = (k + (int)r.size - 1) / (int)r.size;
      const uint32_t sorted = block_sort<uint32_t>(key_of(best), reinterpret_cast<uint32_t*>(sh.few.order));
      if ((int)threadIdx.x == min(j, kSampleThreads) - 1) sh.warp_sum[0] = j <= kSampleThreads ? sorted : 0;
      __syncthreads();
      const u64* bounds = r.all_gather(sh.warp_sum[0]);
      uint32_t k_min = (uint32_t)bounds[0];
      for (uint32_t c = 1; c < r.size; ++c) k_min = min(k_min, (uint32_t)bounds[c]);
      // a lowest logit as a bound on the difference (which rounds the same way for both)
      // (a difference beyond fp32 bounds nothing)
      const float d = r.x_max - logit_of(k_min);
      if (k_min > key_of(-INFINITY) && d < INFINITY) far = __uint_as_float(__float_as_uint(d) + 1);
    }
  } else if (cut_p) {
    r.hist_clear();
    __syncthreads();
    r.each([&](float x, int) {
      const u64 w = r.template weight<INF>(x);
      if (w) r.hist_add(r.coarse_bin(x), w);
    });
    const typename R::Sums sums = r.hist_sums();
    target_p = mass_target(tp, sums.total);
    bin = r.crossing(sums, target_p, &above);
    far = R::bin_end(bin);
  }
  // (with a top_k, top_p goes by the mass of all its tokens)
  if (mp > 0.f && !(cut_k && cut_p)) {
    // a kept weight is at least least - 1/2 before its rounding; 1e-6 covers the rounding of x_max - x
    const double d = -log(((double)least - 0.5) / (double)((u64)1 << a.shift)) * (double)t;
    far = fminf(far, __double2float_ru(d * (1.0 + 1e-6) + 1e-37));
  }
  if (INF) far = 0.f;  // only its equals, whose difference is no number
  // without a bound: all but -inf, by their differences, which are finite below 2^100 (the
  // others' may not be; a test of x itself costs every row 3%)
  if (far < INFINITY || (a.V <= kMaxCand && r.x_max < 0x1p100f)) {
    auto near = [&](float x) { return INF ? x == INFINITY : r.x_max - x < far; };
    const u64 n = r.running([&](float x, int) -> u64 { return near(x) ? 1 : 0; }, &mine, &before);
    if (n <= kMaxCand) {
      r.gather(near, before);
      r.sync_all();
      if (r.rank == 0) finish_few<INF>(r, (int)n, cut_k ? k : 0, cut_p, tp, target_p, least, u, row);
      return;
    }
  }

  if (cut_k) {
    auto one = [](float x, int) -> u64 { return x > -INFINITY; };  // tokens that can be chosen (NaN cannot)
    r.hist_clear();
    __syncthreads();
    r.each([&](float x, int i) {
      if (one(x, i)) atomicAdd(&sh.piece[0][r.coarse_bin(x)], 1u);
    });
    const typename R::Sums sums = r.hist_sums();
    if (sums.total > (u64)k) {
      bin = r.crossing(sums, (u64)k, &above);
      r.cut_at(one, [](float) -> u64 { return 1; }, bin, (u64)k - above);
    }
  }
  auto mass = [&](float x, int i) -> u64 { return r.kept(x, i) ? r.template weight<INF>(x) : 0; };
  if (cut_p) {
    if (cut_k) {
      r.hist_clear();
      __syncthreads();
      r.each([&](float x, int i) {
        const u64 w = mass(x, i);
        if (w) r.hist_add(r.coarse_bin(x), w);
      });
      const typename R::Sums sums = r.hist_sums();
      target_p = mass_target(tp, sums.total);
      bin = r.crossing(sums, target_p, &above);
    }
    r.cut_at(mass, [&](float x) { return r.template weight<INF>(x); }, bin, target_p - above);
  }
  auto pick = [&](auto w) {
    const u64 total = r.running(w, &mine, &before);
    const int at = r.place_of(w, mine, before, choice_target(u, total));
    if (at >= 0 && (threadIdx.x & 31) == 0) {
      a.token[row] = at;
      if (a.logprob) a.logprob[row] = (float)log((double)r.template weight<INF>(r.element(at)) / (double)total);
    }
  };
  // (nothing cut: no test for each logit)
  if (!cut_k && !cut_p && least == 1)
    pick([&](float x, int) { return r.template weight<INF>(x); });
  else
    pick([&](float x, int i) -> u64 {
      const u64 w = mass(x, i);
      return w >= least ? w : 0;
    });
  r.sync_all();
}

template <typename T, bool STREAM>
__global__ void __launch_bounds__(kSampleThreads, 2) qe_sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int N = Elems<T>::N;
  SampleShared& sh = *reinterpret_cast<SampleShared*>(smem + a.smem_row);
  const int row = blockIdx.x / a.cluster;
  using R = Row<T, STREAM>;
  R r(a, sh);
  r.size = a.cluster;
  r.rank = a.cluster == 1 ? 0 : cluster_rank();

  cluster_arrive();  // waited for before the first access to a peer: it has to be running
  static_assert(kExpTable * kExpCopies == kSampleThreads, "one entry a thread");
  sh.exp2_table[threadIdx.x / kExpCopies][threadIdx.x % kExpCopies] = exp2((double)(threadIdx.x / kExpCopies) / kExpTable);
  grid_dependency_wait();
  grid_launch_dependents();

  // this CTA's run of the row, element for element as stored, from the
  // 16-byte boundary at or before it
  const T* base = (const T*)a.logits + (size_t)row * a.stride;
  const int i0 = min(a.V, (int)r.rank * a.run), i1 = min(a.V, i0 + a.run);
  {
    const T* p0 = base + i0;
    const int skew = (int)(((uintptr_t)p0 & 15) / sizeof(T));
    const int n = i1 - i0;
    r.first = i0 - skew;
    r.pieces = n > 0 ? (skew + n + N - 1) / N : 0;
    const T* src = p0 - skew;
    if constexpr (STREAM) {
      r.data = reinterpret_cast<const uint4*>(src);
      r.lo = skew;
      r.hi = skew + n;
      r.per = ((r.pieces + kSampleWarps - 1) / kSampleWarps + 31) & ~31;
      __syncthreads();
    } else {
      r.per = ((r.pieces + kSampleThreads - 1) / kSampleThreads) | 1;
      r.data = reinterpret_cast<const uint4*>(smem);
      T* dst = reinterpret_cast<T*>(smem);
      for (int p = threadIdx.x; p < r.pieces; p += kSampleThreads) {
        if (p * N >= skew && (p + 1) * N <= skew + n) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst + p * N)), "l"(src + p * N) : "memory");
        } else {
          for (int e = p * N; e < (p + 1) * N; ++e)
            dst[e] = e >= skew && e < skew + n ? src[e] : Elems<T>::lowest();
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncthreads();
    }
  }

  // the largest logit
  float best = -INFINITY, group[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) group[g] = -INFINITY;
  if constexpr (STREAM) {
    r.each([&](float x, int i) {
      const int g = (i - r.first) & (kGroups - 1);  // known when the code is compiled
#pragma unroll
      for (int k = 0; k < kGroups; ++k)
        if (g == k) group[k] = fmaxf(group[k], x);
    });
#pragma unroll
    for (int g = 0; g < kGroups; ++g) best = fmaxf(best, group[g]);
  } else {
    r.each([&](float x, int) { best = fmaxf(best, x); });  // NaN loses
  }
  u64 top = key_of(best);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
  if ((threadIdx.x & 31) == 0) sh.warp_sum[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSampleWarps; ++w) top = max(top, sh.warp_sum[w]);
  cluster_wait();
  const u64* tops = r.all_gather(top);
  for (uint32_t k = 0; k < r.size; ++k) top = max(top, tops[k]);
  const uint32_t k_max = (uint32_t)top;
  r.x_max = logit_of(k_max);
  if (r.x_max == -INFINITY) {  // nothing to choose from
    if (r.rank == 0 && threadIdx.x == 0) {
      a.token[row] = -1;
      if (a.logprob) a.logprob[row] = -INFINITY;
    }
    r.sync_all();
    return;
  }
  const float t = a.temperature ? a.temperature[row] : 1.f;
  const int k = a.top_k ? a.top_k[row] : 0;
  const float tp = a.top_p ? a.top_p[row] : 1.f, mp = a.min_p ? a.min_p[row] : 0.f, u = a.u[row];
  u64 mine, before;
  if (!(t > 0.f)) {  // greedy: the first of the largest
    auto largest = [&](float x, int) -> u64 { return x == r.x_max; };
    r.running(largest, &mine, &before);
    const int at = r.place_of(largest, mine, before, 0);
    if (at >= 0 && (threadIdx.x & 31) == 0) {
      a.token[row] = at;
      if (a.logprob) a.logprob[row] = 0.f;
    }
    r.sync_all();
    return;
  }
  r.inv_t = 1.0 / (double)t;
  if (r.x_max == INFINITY) choose<true>(r, best, group, t, k, tp, mp, u, row);
  else choose<false>(r, best, group, t, k, tp, mp, u, row);
}

template <typename T, bool STREAM>
cudaError_t launch_sample_as(const SampleArgs& a, cudaStream_t s) {
  static std::atomic<bool> set[64];  // per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!set[dev]) {
    e = cudaFuncSetAttribute(qe_sample_kernel<T, STREAM>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(qe_sample_kernel<T, STREAM>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * a.cluster));
  cfg.blockDim = dim3(kSampleThreads);
  cfg.dynamicSmemBytes = a.smem_row + sizeof(SampleShared);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, qe_sample_kernel<T, STREAM>, a);
}

template <typename T>
cudaError_t launch_sample_t(SampleArgs a, cudaStream_t s) {
  // CTAs per row: so many that two CTAs (what the registers allow) fit into a
  // multiprocessor's memory, and more where that still leaves all of them running at once
  const int es = (int)sizeof(T);
  const int at_once = 2 * dev_info().sms;
  int cl = 1;
  while (cl < 16 && (long long)a.V * es / cl > kRowBytes) cl *= 2;
  while (cl < 16 && (long long)a.V * es / cl > 8 * 1024 && (long long)a.B * cl * 2 <= at_once) cl *= 2;
  const int n = 16 / es;
  if (cl > 1 && (long long)a.B * cl > 2ll * at_once) {  // clusters in more than two waves
    for (a.cluster = kStreamCluster;; a.cluster *= 2) {  // eight for more than 4 kMaxRun logits
      a.run = ((a.V + a.cluster - 1) / a.cluster + n - 1) / n * n;
      if (a.run <= kMaxRun) break;
    }
    a.smem_row = 0;
    return launch_sample_as<T, true>(a, s);
  }
  a.cluster = cl;
  a.run = ((a.V + cl - 1) / cl + n - 1) / n * n;
  a.smem_row = ((a.run + 2 * n) * es + 127) / 128 * 128;
  return launch_sample_as<T, false>(a, s);
}

}  // namespace
}  // namespace qe

using namespace qe;

extern "C" QE_API int token_sample(const void* logits, int dtype, int B, int V, int64_t stride, const float* temperature,
                                   const int32_t* top_k, const float* top_p, const float* min_p, const float* u,
                                   int32_t* token, float* logprob, qe_stream_t stream) {
  if (!(dtype == QE_F32 || dtype == QE_BF16 || dtype == QE_F16))
    return fail(QE_ERR_INVALID_ARG, "dtype must be QE_F32, QE_BF16 or QE_F16 (got %d)", dtype);
  if (B < 0 || B > 1 << 20) return fail(QE_ERR_INVALID_ARG, "B must be in [0, 2^20] (got %d)", B);
  if (V < 1 || V > kMaxVocab) return fail(QE_ERR_INVALID_ARG, "V must be in [1, %d] (got %d)", kMaxVocab, V);
  if (B > 1 && stride < V) return fail(QE_ERR_INVALID_ARG, "stride must be at least V");
  if (B == 0) return QE_OK;
  int rc;
  if ((rc = check_ptr(logits, "logits", false, dtype == QE_F32 ? 4 : 2)) || (rc = check_ptr(temperature, "temperature", true)) ||
      (rc = check_ptr(top_k, "top_k", true)) || (rc = check_ptr(top_p, "top_p", true)) || (rc = check_ptr(min_p, "min_p", true)) ||
      (rc = check_ptr(u, "u")) || (rc = check_ptr(token, "token")) || (rc = check_ptr(logprob, "logprob", true)))
    return rc;
  SampleArgs a{};
  a.logits = logits; a.stride = stride; a.temperature = temperature; a.top_k = top_k; a.top_p = top_p; a.min_p = min_p;
  a.u = u; a.token = token; a.logprob = logprob; a.B = B; a.V = V;
  int bits = 0;
  while ((1 << bits) < V) ++bits;
  a.shift = 62 - bits < 46 ? 62 - bits : 46;
  const cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = dtype == QE_F32 ? launch_sample_t<float>(a, s)
                        : dtype == QE_BF16 ? launch_sample_t<__nv_bfloat16>(a, s) : launch_sample_t<__half>(a, s);
  if (e != cudaSuccess) return cuda_fail(e, "token_sample launch");
  return QE_OK;
}
