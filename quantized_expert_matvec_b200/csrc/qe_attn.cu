// qe_attn.cu -- attention of one decode step over a paged cache, with a prefix
// that the whole batch shares.
//
//   out[b,i] = sum_j p_j v_j,   p = softmax_j(scale q[b,i] . k_j)
//
// over the prefix's keys, then row b's own.  The keys are cut into chunks; a
// CTA takes one chunk for 16 query rows of one key head and leaves, per row,
// the running maximum m and sum l of the softmax and the unnormalised output:
//   m' = max(m, s),  l' = l 2^(m - m') + 2^(s - m'),  o' = o 2^(m - m') + 2^(s - m') v
// (scores in log2 units).  A second kernel joins the chunks of a row in a fixed
// order.  Rows of the prefix are all rows of the batch, so its keys are read
// once for 16 rows and not once for each.
//
// Within a CTA four warps take 16-key tiles in turn, each with its own ring of
// tiles in shared memory (cp.async), its own m, l and o: no barrier until the
// four are joined at the end of the chunk.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "qe_attn.h"
#include "qe_device.cuh"
#include "qe_internal.h"

namespace qe {
namespace {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kTileKeys = 16;
constexpr int kMaxRows = 4096;  // B
constexpr float kLog2e = 1.4426950408889634f;

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
  float* part_prefix;   // [nsp][B * n_q][D]
  float2* ml_prefix;    // [nsp][B * n_q] {m, l}
  float* part_own;      // [chunk][n_q][D]
  float2* ml_own;
  int2* own_info;       // [B] {first chunk, chunks}
  int B, n_q, n_kv, G, n_pages, table_stride, prefix_len;
  int nsp, prefix_chunk;  // prefix splits and keys of each
  int rb_own, rb_prefix;  // blocks of 16 rows per key head
  int own_target;         // own chunks x key heads x row blocks aimed at
  float scale_log2;
  FastDiv page;
};

template <typename T>
QE_DEV void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
QE_DEV void mma16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
QE_DEV void mma16816<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
QE_DEV void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
QE_DEV void ldmatrix4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// 16 bytes, or 16 zeros
QE_DEV void cp_async16z(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}

template <int D>
constexpr int kAttnStages = D == 64 ? 6 : 3;
template <int D>
constexpr int kAttnTileBytes = kTileKeys * D * 2;  // K or V
template <int D>
constexpr int kAttnSmem = kAttnWarps * kAttnStages<D> * 2 * kAttnTileBytes<D>;

// One chunk [k0, k1) of the keys on pages list[0 ..] of key head h, for 16 rows
// of which `row_src(i)` gives row i's query (NULL: no such row); the result goes
// to po + row * D and pml[row] with row = row_dst(i).
template <typename T, int D, typename Src, typename Dst>
QE_DEV void attn_chunk(const AttnArgs& a, int h, const int32_t* list, int k0, int k1, Src row_src, Dst row_dst,
                       float* po, float2* pml, unsigned char* smem) {
  constexpr int S = kAttnStages<D>, TB = kAttnTileBytes<D>;
  constexpr int CH = D / 8;        // 16-byte pieces of a row
  constexpr int RPI = 32 / CH;     // rows one warp instruction copies (D = 256: one row)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned char* ring = smem + warp * S * 2 * TB;
  const uint32_t ring_u = smem_u32(ring);

  // fragments of the 16 query rows
  uint32_t qf[D / 16][4];
  {
    const T* r0 = (const T*)row_src(lane >> 2);
    const T* r1 = (const T*)row_src((lane >> 2) + 8);
    const int c = (lane & 3) * 2;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      qf[k][0] = r0 ? *reinterpret_cast<const uint32_t*>(r0 + 16 * k + c) : 0u;
      qf[k][1] = r1 ? *reinterpret_cast<const uint32_t*>(r1 + 16 * k + c) : 0u;
      qf[k][2] = r0 ? *reinterpret_cast<const uint32_t*>(r0 + 16 * k + c + 8) : 0u;
      qf[k][3] = r1 ? *reinterpret_cast<const uint32_t*>(r1 + 16 * k + c + 8) : 0u;
    }
  }

  const int tiles = (k1 - k0 + kTileKeys - 1) / kTileKeys;
  const int mine = tiles > warp ? (tiles - warp + kAttnWarps - 1) / kAttnWarps : 0;
  auto first_key = [&](int i) { return k0 + (warp + i * kAttnWarps) * kTileKeys; };
  // lanes 0..15: the page of key `lane` of my tile i, -1 if there is none
  auto page_of = [&](int i) {
    const int key = first_key(i) + (lane & 15);
    return (i < mine && key < k1) ? __ldg(list + a.page.div((uint32_t)key)) : -1;
  };
  int page_next = page_of(0);
  uint32_t ok_mask[S];  // which keys of the tile in slot s exist
#pragma unroll
  for (int s = 0; s < S; ++s) ok_mask[s] = 0;
  auto issue = [&](int i, int slot) -> uint32_t {
    uint32_t live = 0;
    if (i < mine) {
      const int key = first_key(i) + (lane & 15);
      const int page = page_next;
      const bool ok = page >= 0 && page < a.n_pages;
      if (key < k1 && !ok) set_error(a.err, QE_ERR_INVALID_ARG);
      live = __ballot_sync(0xffffffffu, ok) & 0xffffu;
      const int off = key - (int)a.page.div((uint32_t)key) * (int)a.page.d;
      const long long in_page = ((long long)h * a.page.d + off) * D;
      const long long ko = ok ? page * a.k_page_stride + in_page : 0, vo = ok ? page * a.v_page_stride + in_page : 0;
      const uint32_t kd = ring_u + slot * 2 * TB, vd = kd + TB;
#pragma unroll
      for (int r = 0; r < kTileKeys / RPI; ++r) {
        const int row = r * RPI + lane / CH, c = lane % CH;
        const long long k_at = __shfl_sync(0xffffffffu, ko, row), v_at = __shfl_sync(0xffffffffu, vo, row);
        const bool real = (live >> row) & 1;
        const uint32_t at = row * (D * 2) + ((c ^ (row & 7)) << 4);
        cp_async16z(kd + at, (const T*)a.kc + k_at + c * 8, real);
        cp_async16z(vd + at, (const T*)a.vc + v_at + c * 8, real);
      }
      page_next = page_of(i + 1);
    }
    cp_async_commit();
    return live;
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) ok_mask[s] = issue(s, s);

  float o[D / 8][4];
#pragma unroll
  for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

  for (int i0 = 0; i0 < mine; i0 += S) {
#pragma unroll
    for (int u = 0; u < S; ++u) {
      const int i = i0 + u;
      if (i >= mine) break;  // uniform over the warp
      __syncwarp();          // every lane is done with the tile whose slot is refilled now
      ok_mask[(u + S - 1) % S] = issue(i + S - 1, (u + S - 1) % S);
      cp_async_wait<S - 1>();
      __syncwarp();
      const uint32_t kb = ring_u + u * 2 * TB, vb = kb + TB;
      const uint32_t live = ok_mask[u];
      // scores of 16 rows x 16 keys
      float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        // matrices: keys 0-7 / 8-15 x dims 16k..+7 / +8..+15
        const int row = (lane & 7) + ((lane >> 4) << 3), c = 2 * k + ((lane >> 3) & 1);
        uint32_t b[4];
        ldmatrix4(b, kb + row * (D * 2) + ((c ^ (row & 7)) << 4));
        mma16816<T>(s0, qf[k], b[0], b[1]);
        mma16816<T>(s1, qf[k], b[2], b[3]);
      }
      // mask, then the running maximum
      const int c0 = (lane & 3) * 2;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s0[e] = (live >> (c0 + (e & 1))) & 1 ? s0[e] * a.scale_log2 : -INFINITY;
        s1[e] = (live >> (c0 + 8 + (e & 1))) & 1 ? s1[e] * a.scale_log2 : -INFINITY;
      }
      float n0 = fmaxf(fmaxf(s0[0], s0[1]), fmaxf(s1[0], s1[1]));
      float n1 = fmaxf(fmaxf(s0[2], s0[3]), fmaxf(s1[2], s1[3]));
      n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, 1));
      n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, 1));
      n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, 2));
      n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, 2));
      n0 = fmaxf(n0, m0);
      n1 = fmaxf(n1, m1);
      const float b0 = n0 == -INFINITY ? 0.f : n0, b1 = n1 == -INFINITY ? 0.f : n1;
      if (__any_sync(0xffffffffu, n0 > m0 || n1 > m1)) {
        const float f0 = exp2f(m0 - b0), f1 = exp2f(m1 - b1);
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          o[n][0] *= f0; o[n][1] *= f0;
          o[n][2] *= f1; o[n][3] *= f1;
        }
        m0 = n0;
        m1 = n1;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s0[e] = exp2f(s0[e] - (e < 2 ? b0 : b1));
        s1[e] = exp2f(s1[e] - (e < 2 ? b0 : b1));
      }
      l0 += (s0[0] + s0[1]) + (s1[0] + s1[1]);
      l1 += (s0[2] + s0[3]) + (s1[2] + s1[3]);
      const uint32_t p[4] = {pack2<T>(s0[0], s0[1]), pack2<T>(s0[2], s0[3]), pack2<T>(s1[0], s1[1]), pack2<T>(s1[2], s1[3])};
#pragma unroll
      for (int n = 0; n < D / 16; ++n) {
        // matrices (transposed): keys 0-7 / 8-15 x dims 16n..+7 / +8..+15
        const int row = lane & 15, c = 2 * n + (lane >> 4);
        uint32_t b[4];
        ldmatrix4t(b, vb + row * (D * 2) + ((c ^ (row & 7)) << 4));
        mma16816<T>(o[2 * n], p, b[0], b[1]);
        mma16816<T>(o[2 * n + 1], p, b[2], b[3]);
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
  l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 2);

  // join the four warps: their o go through the ring's memory (each warp's
  // ring holds its 16 x D floats), m and l through a small array
  __shared__ float2 ml[kAttnWarps][16];
  static_assert(kAttnStages<D> * 2 * kAttnTileBytes<D> >= 16 * D * 4, "ring holds a warp's output");
  float* mine_o = reinterpret_cast<float*>(ring);
  __syncwarp();
  const int r = lane >> 2;
#pragma unroll
  for (int n = 0; n < D / 8; ++n) {
    const int c = n * 8 + (lane & 3) * 2;
    *reinterpret_cast<float2*>(mine_o + r * D + c) = make_float2(o[n][0], o[n][1]);
    *reinterpret_cast<float2*>(mine_o + (r + 8) * D + c) = make_float2(o[n][2], o[n][3]);
  }
  if ((lane & 3) == 0) {
    ml[warp][r] = make_float2(m0, l0);
    ml[warp][r + 8] = make_float2(m1, l1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 16 * (D / 4); e += kAttnThreads) {
    const int row = e / (D / 4), c = (e % (D / 4)) * 4;
    const long long dst = row_dst(row);
    if (dst < 0) continue;
    float m = ml[0][row].x;
#pragma unroll
    for (int w = 1; w < kAttnWarps; ++w) m = fmaxf(m, ml[w][row].x);
    const float base = m == -INFINITY ? 0.f : m;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
      const float f = exp2f(ml[w][row].x - base);
      const float4 x = *reinterpret_cast<const float4*>(smem + w * S * 2 * TB + (row * D + c) * 4);
      acc.x = fmaf(f, x.x, acc.x);
      acc.y = fmaf(f, x.y, acc.y);
      acc.z = fmaf(f, x.z, acc.z);
      acc.w = fmaf(f, x.w, acc.w);
      l = fmaf(f, ml[w][row].y, l);
    }
    *reinterpret_cast<float4*>(po + dst * D + c) = acc;
    if (c == 0) pml[dst] = make_float2(m, l);
  }
}

QE_DEV int block_sum(int v, int* tmp) {  // over kAttnThreads threads; every thread gets the sum
  v = __reduce_add_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int w = 0; w < kAttnWarps; ++w) s += tmp[w];
  __syncthreads();
  return s;
}

template <typename T, int D>
__global__ void __launch_bounds__(kAttnThreads) qe_attn_part_kernel(const AttnArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int tmp[kAttnWarps];
  __shared__ int found[3];  // row, chunk within it, first chunk
  grid_dependency_wait();
  grid_launch_dependents();
  const int n_prefix = a.nsp * a.n_kv * a.rb_prefix;
  int item = blockIdx.x;
  if (item < n_prefix) {
    const int rb = item % a.rb_prefix;
    const int h = item / a.rb_prefix % a.n_kv;
    const int s = item / (a.rb_prefix * a.n_kv);
    const int k0 = s * a.prefix_chunk, k1 = min(a.prefix_len, k0 + a.prefix_chunk);
    const int rows = a.B * a.G;
    auto src = [&](int i) -> const void* {
      const int f = rb * 16 + i;
      return f < rows ? (const T*)a.q + (size_t)(f / a.G) * a.q_stride + (size_t)(h * a.G + f % a.G) * D : nullptr;
    };
    auto dst = [&](int i) -> long long {
      const int f = rb * 16 + i;
      return f < rows ? (long long)(f / a.G) * a.n_q + h * a.G + f % a.G : -1;
    };
    const size_t base = (size_t)s * a.B * a.n_q;
    attn_chunk<T, D>(a, h, a.prefix_pages, k0, k1, src, dst, a.part_prefix + base * D, a.ml_prefix + base, smem);
    return;
  }
  item -= n_prefix;
  // the rows' own keys: chunks of one length for the whole batch
  const int cap = (int)min((long long)a.table_stride * a.page.d, 1ll << 30);
  auto len_of = [&](int b) { return b < a.B ? max(0, min(a.kv_len[b], cap)) : 0; };
  long long total = 0;
  const int per = a.n_kv * a.rb_own;
  {
    // 64-bit total of lengths: sums of 16 bits each side of the word
    int lo = 0, hi = 0;
    for (int b = threadIdx.x; b < a.B; b += kAttnThreads) {
      const int n = len_of(b);
      lo += n & 0x7fff;
      hi += n >> 15;
    }
    total = (long long)block_sum(lo, tmp) + ((long long)block_sum(hi, tmp) << 15);
  }
  const long long want = (total * per + a.own_target - 1) / a.own_target;
  const int chunk = (int)(((want < 1 ? 1 : want) + 63) / 64 * 64);
  const int j = item / per, hr = item % per;
  // the row that chunk j belongs to
  int before = 0;
  bool have = false;
  for (int b0 = 0; b0 < a.B && !have; b0 += kAttnThreads) {
    const int b = b0 + threadIdx.x;
    const int n = (len_of(b) + chunk - 1) / chunk;
    int scan = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, scan, d);
      if ((threadIdx.x & 31) >= d) scan += x;
    }
    if ((threadIdx.x & 31) == 31) tmp[threadIdx.x >> 5] = scan;
    __syncthreads();
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
      if (w < (int)(threadIdx.x >> 5)) scan += tmp[w];
      sum += tmp[w];
    }
    const int first = before + scan - n;
    if (n > 0 && j >= first && j < first + n) {
      found[0] = b;
      found[1] = j - first;
      found[2] = first;
    }
    before += sum;
    have = j < before;
    __syncthreads();
  }
  if (!have) return;
  const int b = found[0], ci = found[1];
  const int len = len_of(b), h = hr / a.rb_own, rb = hr % a.rb_own;
  if (threadIdx.x == 0 && ci == 0 && hr == 0) {
    a.own_info[b] = make_int2(found[2], (len + chunk - 1) / chunk);
    if (a.kv_len[b] > cap) set_error(a.err, QE_ERR_INVALID_ARG);
  }
  const int k0 = ci * chunk, k1 = min(len, k0 + chunk);
  auto src = [&](int i) -> const void* {
    const int g = rb * 16 + i;
    return g < a.G ? (const T*)a.q + (size_t)b * a.q_stride + (size_t)(h * a.G + g) * D : nullptr;
  };
  auto dst = [&](int i) -> long long {
    const int g = rb * 16 + i;
    return g < a.G ? (long long)h * a.G + g : -1;
  };
  const size_t base = (size_t)j * a.n_q;
  attn_chunk<T, D>(a, h, a.table + (size_t)b * a.table_stride, k0, k1, src, dst, a.part_own + base * D,
                   a.ml_own + base, smem);
}

// Joins the chunks of each row: one warp a row, prefix chunks first, then own.
template <typename T, int D>
__global__ void __launch_bounds__(kAttnThreads) qe_attn_join_kernel(const AttnArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * kAttnWarps + (threadIdx.x >> 5);
  const long long rows = (long long)a.B * a.n_q;
  if (row >= rows) return;
  const int b = (int)(row / a.n_q), hq = (int)(row % a.n_q);
  const int kv = a.kv_len[b];
  if (kv < 0) return;
  const bool own = kv > 0 && a.table_stride > 0;
  if (kv > 0 && !own && lane == 0) set_error(a.err, QE_ERR_INVALID_ARG);
  const int2 info = own ? a.own_info[b] : make_int2(0, 0);
  const int n = a.nsp + info.y;
  auto at = [&](int i) { return i < a.nsp ? (size_t)i * rows + row : (size_t)(info.x + i - a.nsp) * a.n_q + hq; };
  float m = -INFINITY;
  for (int i = lane; i < n; i += 32) m = fmaxf(m, (i < a.nsp ? a.ml_prefix : a.ml_own)[at(i)].x);
  m = warp_max(m);
  const float base = m == -INFINITY ? 0.f : m;
  constexpr int E = D / 32;
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  float l = 0.f;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    float f = 0.f;
    if (i < n) {
      const float2 ml = (i < a.nsp ? a.ml_prefix : a.ml_own)[at(i)];
      f = exp2f(ml.x - base);
      l = fmaf(f, ml.y, l);
    }
    const int lim = min(32, n - i0);
#pragma unroll 4
    for (int k = 0; k < lim; ++k) {
      const float w = __shfl_sync(0xffffffffu, f, k);
      const int ik = i0 + k;
      const float* p = (ik < a.nsp ? a.part_prefix : a.part_own) + at(ik) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(w, p[e], acc[e]);
    }
  }
  l = warp_sum(l);
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // a NaN sum stays one
  uint32_t* out = reinterpret_cast<uint32_t*>((T*)a.out + (size_t)b * a.out_stride + (size_t)hq * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) out[e / 2] = pack2<T>(acc[e] * inv, acc[e + 1] * inv);
  if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (base + log2f(l)) * 0.69314718055994531f;
}

// Sizes that depend on the shape alone, whatever the lengths.
struct AttnPlan {
  int rb_own, rb_prefix, own_target, nsp_max, own_chunks_max;
  size_t off_info, off_mlp, off_mlo, off_pp, off_po, total;
};
AttnPlan attn_plan(int n_kv, int n_q, int D, int B, int sms) {
  AttnPlan p{};
  const int G = n_q / n_kv;
  p.rb_own = (G + 15) / 16;
  p.rb_prefix = (int)(((long long)B * G + 15) / 16);
  p.own_target = 4 * sms;
  p.nsp_max = 4 * sms / (n_kv * p.rb_prefix);
  if (p.nsp_max < 1) p.nsp_max = 1;
  p.own_chunks_max = p.own_target / (n_kv * p.rb_own) + 1 + B;
  size_t off = sizeof(WsControl);
  auto take = [&](size_t bytes) { const size_t o = off; off = (off + bytes + 255) & ~(size_t)255; return o; };
  const size_t rows = (size_t)B * n_q;
  p.off_info = take(sizeof(int2) * (size_t)B);
  p.off_mlp = take(sizeof(float2) * p.nsp_max * rows);
  p.off_mlo = take(sizeof(float2) * (size_t)p.own_chunks_max * n_q);
  p.off_pp = take(4 * (size_t)p.nsp_max * rows * D);
  p.off_po = take(4 * (size_t)p.own_chunks_max * n_q * D);
  p.total = off;
  return p;
}

template <typename T, int D>
cudaError_t launch_attn_t(const AttnArgs& a, int grid, cudaStream_t s) {
  static std::atomic<bool> set[64];  // per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!set[dev]) {
    e = cudaFuncSetAttribute(qe_attn_part_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kAttnSmem<D>);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kAttnThreads);
  cfg.dynamicSmemBytes = kAttnSmem<D>;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, qe_attn_part_kernel<T, D>, a);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)(((long long)a.B * a.n_q + kAttnWarps - 1) / kAttnWarps));
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, qe_attn_join_kernel<T, D>, a);
}

template <typename T>
cudaError_t launch_attn(const AttnArgs& a, int D, int grid, cudaStream_t s) {
  if (D == 64) return launch_attn_t<T, 64>(a, grid, s);
  if (D == 128) return launch_attn_t<T, 128>(a, grid, s);
  return launch_attn_t<T, 256>(a, grid, s);
}

int check_attn_shape(const qe_kv_cache* c, int n_q, int B) {
  int rc = check_kv_cache(c);
  if (rc) return rc;
  if (n_q < 1 || n_q > kMaxHeads || n_q % c->n_kv)
    return fail(QE_ERR_INVALID_ARG, "n_q must be a positive multiple of n_kv <= %d (got %d, n_kv %d)", kMaxHeads, n_q, c->n_kv);
  if (B < 0 || B > kMaxRows) return fail(QE_ERR_INVALID_ARG, "B must be in [0, %d] (got %d)", kMaxRows, B);
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
  if (B == 0) return QE_OK;
  const int D = c->head_dim;
  if ((rc = check_ptr(q, "q", false, 16)) || (rc = check_ptr(out, "out", false, 16)) || (rc = check_ptr(kv_len, "kv_len")) ||
      (rc = check_ptr(table, "table", table_stride == 0)) || (rc = check_ptr(prefix_pages, "prefix_pages", prefix_len == 0)) ||
      (rc = check_ptr(lse, "lse", true)))
    return rc;
  if ((q_stride | out_stride) & 7) return fail(QE_ERR_INVALID_ARG, "row strides must be multiples of 8 elements");
  if (B > 1 && (q_stride < (int64_t)n_q * D || out_stride < (int64_t)n_q * D))
    return fail(QE_ERR_INVALID_ARG, "row strides must cover a row's heads");
  const size_t last = (size_t)B - 1;
  if (ranges_overlap(out, 2 * (last * out_stride + (size_t)n_q * D), q, 2 * (last * q_stride + (size_t)n_q * D)))
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
  a.own_info = (int2*)(w + p.off_info);
  a.ml_prefix = (float2*)(w + p.off_mlp); a.ml_own = (float2*)(w + p.off_mlo);
  a.part_prefix = (float*)(w + p.off_pp); a.part_own = (float*)(w + p.off_po);
  a.B = B; a.n_q = n_q; a.n_kv = c->n_kv; a.G = n_q / c->n_kv; a.n_pages = c->n_pages;
  a.table_stride = table_stride; a.prefix_len = prefix_len;
  a.rb_own = p.rb_own; a.rb_prefix = p.rb_prefix; a.own_target = p.own_target;
  a.scale_log2 = scale * kLog2e;
  a.page = fast_div((uint32_t)c->page_size);
  if (prefix_len > 0) {
    int nsp = (prefix_len + 127) / 128;
    nsp = nsp > p.nsp_max ? p.nsp_max : nsp;
    a.prefix_chunk = ((prefix_len + nsp - 1) / nsp + 63) / 64 * 64;
    a.nsp = (prefix_len + a.prefix_chunk - 1) / a.prefix_chunk;
  }
  // own items: at most own_target plus one partial chunk for each row, key head and row block
  long long own = 0;
  if (table_stride > 0) {
    const long long per = (long long)a.n_kv * a.rb_own;
    const long long most = (long long)B * (((long long)table_stride * c->page_size + 63) / 64) * per;
    own = (long long)p.own_chunks_max * per;
    own = own < most ? own : most;
  }
  const long long grid = (long long)a.nsp * a.n_kv * a.rb_prefix + own;
  if (grid > 0x7fffffffLL) return fail(QE_ERR_UNSUPPORTED, "attn_decode_step: too many parts");
  const cudaError_t e = c->dtype == QE_BF16 ? launch_attn<__nv_bfloat16>(a, D, (int)grid, (cudaStream_t)stream)
                                            : launch_attn<__half>(a, D, (int)grid, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "attn_decode_step launch");
  return QE_OK;
}
