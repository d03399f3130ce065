// qe_kv.cu -- rotary positions on q and k, and the append of k and v to the
// paged cache: what precedes attn_decode_step in a full-attention layer.
//
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = pos[axis(i)] f_i
//
// The operator reads T (n_q + 2 n_kv) head_dim elements and writes as many: it is
// bound by HBM for prompts and by one launch's latency for a decode step.  The
// angles of a token's rotary_dim / 2 pairs are computed once, into shared memory, and
// used by all its heads.  A thread's item is 16 elements of a head in two runs of 8:
// two 16-byte loads (four for fp32) and two 16-byte stores, requested an item ahead.
// Measured: 1 token of 48 heads of 128 3.1 us, 256 tokens 3.7 us, 16384 tokens (403 MB)
// 71 us, 5.7 TB/s (with a thread's 16 elements in one run, which leaves its neighbours'
// requests half a sector each, 79 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "qe_attn.h"
#include "qe_device.cuh"
#include "qe_internal.h"

namespace qe {
namespace {

constexpr int kKvThreads = 256;
constexpr int kMaxPairs = 128;  // head_dim 256 / 2
constexpr int kKvTokens = 4;    // of one CTA at most

struct KvArgs {
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  void* kc;
  void* vc;
  long long q_stride, k_stride, v_stride, q_out_stride, k_page_stride, v_page_stride;
  const float* inv_freq;
  const int32_t* pos;
  const int32_t* kv_pos;
  const int32_t* seq;
  const int32_t* table;
  int* err;
  int T, n_q, n_kv, D, rd, n_pages, n_seq, table_stride, per_cta;
  FastDiv page;
  uint8_t axis[kMaxPairs];
};

// sin and cos of the angle pos * f.  The product of an integer below 2^31 and an fp32
// number has up to 55 bits: a is the nearest fp64 number and `rest` what it lacks, exactly.
// The nearest multiple of pi / 2 is taken off a in two parts (Cody and Waite's reduction,
// pi / 2 to 106 bits), which leaves |r| <= pi / 4 + 2^-8 to about 2^-52 for angles up to
// 2^45.  On that interval the Taylor polynomials to r^9 and r^10 are off by at most
// r^11 / 11! = 1.9e-9 and r^12 / 12! = 1.3e-10, below fp32's half step.
QE_DEV float2 cos_sin(int pos, float f) {
  const double a = (double)pos * (double)f, rest = fma((double)pos, (double)f, -a);
  const double n = rint(a * 0.63661977236758134308);
  double rd = fma(-n, 1.5707963267948965580, a);
  rd = fma(-n, 6.1232339957367660359e-17, rd) + rest;
  const int quadrant = (int)(__double2ll_rn(n) & 3);
  const float r = (float)rd, z = r * r;
  float s = fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
  s = fmaf(s, z, 1.f / 120.f);
  s = fmaf(s, z, -1.f / 6.f);
  s = fmaf(s * z, r, r);
  float c = fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
  c = fmaf(c, z, -1.f / 720.f);
  c = fmaf(c, z, 1.f / 24.f);
  c = fmaf(c, z, -0.5f);
  c = fmaf(c, z, 1.f);
  const float x = quadrant & 1 ? s : c, y = quadrant & 1 ? c : s;
  return make_float2((quadrant == 1 || quadrant == 2) ? -x : x, quadrant >= 2 ? -y : y);
}

template <typename TI>
struct Raw8;  // 8 elements as loaded
template <>
struct Raw8<float> {
  float4 a, b;
  QE_DEV void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  QE_DEV void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};
template <typename TI>
struct Raw8 {
  uint4 a;
  QE_DEV void load(const TI* p) { a = __ldcs(reinterpret_cast<const uint4*>(p)); }
  QE_DEV void get(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<TI>(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
};

template <typename TC>
QE_DEV void store8(TC* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2<TC>(x[0], x[1]), pack2<TC>(x[2], x[3]), pack2<TC>(x[4], x[5]),
                                            pack2<TC>(x[6], x[7]));
}

QE_DEV void turn_pair(float& a, float& b, float2 w) {
  const float x = fmaf(a, w.x, -b * w.y);
  b = fmaf(b, w.x, a * w.y);
  a = x;
}
QE_DEV void adjacent8(float (&x)[8], const float2* w) {
#pragma unroll
  for (int p = 0; p < 4; ++p) turn_pair(x[2 * p], x[2 * p + 1], w[p]);
}

// One CTA: `a.per_cta` consecutive tokens.  The angles of all of them first (the items' loads
// do not wait for them: each thread requests its first item before), then the items of
// one token after the other.
template <typename TI, typename TC, bool ADJ>
__global__ void __launch_bounds__(kKvThreads) qe_kv_append_kernel(const __grid_constant__ KvArgs a) {
  __shared__ float2 cs[kKvTokens * kMaxPairs];
  __shared__ int place[kKvTokens][2];  // page and offset in it; page -1: none, -2: a padding row
  grid_dependency_wait();
  grid_launch_dependents();
  const int t0 = blockIdx.x * a.per_cta, n = min(a.per_cta, a.T - t0);
  const int half = a.rd >> 1, per_head = a.D >> 4;
  const int items = (a.n_q + 2 * a.n_kv) * per_head;

  struct Item {
    Raw8<TI> r0, r1;
    int head, e0, e1;  // first elements of its two runs of 8
    bool turn;         // a pair's two halves (half pairs); some of it is turned (adjacent pairs)
  };
  // Item `it` of token t.  Its two runs of 8 lie apart, so that the runs of neighbouring
  // threads are neighbours: a pair's two halves, or halves of what is not split so.
  auto load = [&](int t, int it, Item& x) {
    x.head = it / per_head;
    const int i = it - x.head * per_head;
    const int rd = x.head < a.n_q + a.n_kv ? a.rd : 0;
    if (ADJ) {
      x.e0 = 8 * i;
      x.e1 = x.e0 + (a.D >> 1);
      x.turn = x.e0 < rd;
    } else {
      x.turn = 16 * i < rd;
      x.e0 = x.turn ? 8 * i : rd + 8 * i - (rd >> 1);
      x.e1 = x.e0 + ((x.turn ? rd : a.D - rd) >> 1);
    }
    const TI* src;
    if (x.head < a.n_q) src = (const TI*)a.q + (size_t)t * a.q_stride + (size_t)x.head * a.D;
    else if (x.head < a.n_q + a.n_kv) src = (const TI*)a.k + (size_t)t * a.k_stride + (size_t)(x.head - a.n_q) * a.D;
    else src = (const TI*)a.v + (size_t)t * a.v_stride + (size_t)(x.head - a.n_q - a.n_kv) * a.D;
    x.r0.load(src + x.e0);
    x.r1.load(src + x.e1);
  };
  auto finish = [&](int t, int i, const Item& x) {
    const int page = place[i][0], off = place[i][1];
    if (page == -2) return;
    TC* dst;
    if (x.head < a.n_q) {
      dst = (TC*)a.q_out + (size_t)t * a.q_out_stride + (size_t)x.head * a.D;
    } else {
      if (page < 0) return;
      const bool is_k = x.head < a.n_q + a.n_kv;
      const int h = x.head - a.n_q - (is_k ? 0 : a.n_kv);
      dst = (TC*)(is_k ? a.kc : a.vc) + (long long)page * (is_k ? a.k_page_stride : a.v_page_stride) +
            ((long long)h * a.page.d + off) * a.D;
    }
    bool second = true;
    if constexpr (sizeof(TI) == 2 && std::is_same<TI, TC>::value) {
      // what is not turned: the bits as they are (a NaN's too)
      if (!x.turn) *reinterpret_cast<uint4*>(dst + x.e0) = x.r0.a;
      second = x.turn && !(ADJ && x.e1 >= a.rd);
      if (!second) *reinterpret_cast<uint4*>(dst + x.e1) = x.r1.a;
      if (!x.turn) return;
    }
    float u[8], v[8];
    x.r0.get(u);
    x.r1.get(v);
    if (x.turn) {
      const float2* w = cs + i * half;
      if (ADJ) {
        adjacent8(u, w + (x.e0 >> 1));
        if (x.e1 < a.rd) adjacent8(v, w + (x.e1 >> 1));
      } else {
#pragma unroll
        for (int p = 0; p < 8; ++p) turn_pair(u[p], v[p], w[x.e0 + p]);
      }
    }
    store8(dst + x.e0, u);
    if (second) store8(dst + x.e1, v);
  };

  // The first items are on their way while places and angles are worked out.  Padding rows'
  // are read, too: to wait for kv_pos before costs 0.25 us of 1 token's 3.1 and 1.7 us of
  // 16384 tokens' 71.1.
  Item x;
  int i = 0, it = threadIdx.x;  // token of the CTA's, item of the token
  auto settle = [&](int& ti, int& k) {
    while (k >= items) {
      k -= items;
      ++ti;
    }
  };
  settle(i, it);
  if (i < n) load(t0 + i, it, x);
  if ((int)threadIdx.x < n) {
    const int t = t0 + threadIdx.x, p = a.kv_pos[t];
    int page = -2, off = 0;
    if (p >= 0) {
      const int s = a.seq ? a.seq[t] : t, col = (int)a.page.div((uint32_t)p);
      page = -1;
      if (s >= 0 && s < a.n_seq && col < a.table_stride) page = a.table[(size_t)s * a.table_stride + col];
      if (page < 0 || page >= a.n_pages) {
        page = -1;
        set_error(a.err, QE_ERR_INVALID_ARG);
      }
      off = p - col * (int)a.page.d;
    }
    place[threadIdx.x][0] = page;
    place[threadIdx.x][1] = off;
  }
  for (int c = threadIdx.x; c < n * half; c += blockDim.x) {
    const int j = c / half, pair = c - j * half;
    cs[c] = cos_sin(a.pos ? a.pos[(size_t)a.axis[pair] * a.T + t0 + j] : a.kv_pos[t0 + j], a.inv_freq[pair]);
  }
  __syncthreads();
  while (i < n) {
    int next = i, next_it = it + blockDim.x;
    settle(next, next_it);
    Item y;
    if (next < n) load(t0 + next, next_it, y);
    finish(t0 + i, i, x);
    x = y;
    i = next;
    it = next_it;
  }
}

template <typename TI, typename TC>
cudaError_t launch_kv_t(KvArgs a, bool adjacent, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  // one token a CTA until the GPU is full, then several, whose items follow one another
  // without a pause: 16384 tokens take 100 us by one, 88 by two, 79 by four and 82 by eight
  const int items = (a.n_q + 2 * a.n_kv) * (a.D >> 4);
  a.per_cta = a.T >= 16 * dev_info().sms ? kKvTokens : 1;
  int threads = (items + 31) / 32 * 32;
  threads = threads < 64 ? 64 : threads > kKvThreads ? kKvThreads : threads;
  cfg.gridDim = dim3((unsigned)((a.T + a.per_cta - 1) / a.per_cta));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return adjacent ? cudaLaunchKernelEx(&cfg, qe_kv_append_kernel<TI, TC, true>, a)
                  : cudaLaunchKernelEx(&cfg, qe_kv_append_kernel<TI, TC, false>, a);
}

template <typename TC>
cudaError_t launch_kv_in(const KvArgs& a, int in_dtype, bool adjacent, cudaStream_t s) {
  if (in_dtype == QE_F32) return launch_kv_t<float, TC>(a, adjacent, s);
  if (in_dtype == QE_BF16) return launch_kv_t<__nv_bfloat16, TC>(a, adjacent, s);
  return launch_kv_t<__half, TC>(a, adjacent, s);
}

}  // namespace

int check_kv_cache(const qe_kv_cache* c) {
  if (!c) return fail(QE_ERR_INVALID_ARG, "cache is NULL");
  if (!(c->dtype == QE_BF16 || c->dtype == QE_F16))
    return fail(QE_ERR_INVALID_ARG, "cache dtype must be QE_BF16 or QE_F16 (got %d)", c->dtype);
  if (!(c->head_dim == 64 || c->head_dim == 128 || c->head_dim == 256))
    return fail(QE_ERR_INVALID_ARG, "head_dim must be 64, 128 or 256 (got %d)", c->head_dim);
  if (c->page_size < 1 || c->page_size > kMaxPageSize)
    return fail(QE_ERR_INVALID_ARG, "page_size must be in [1, %d] (got %d)", kMaxPageSize, c->page_size);
  if (c->n_kv < 1 || c->n_kv > kMaxHeads) return fail(QE_ERR_INVALID_ARG, "n_kv must be in [1, %d] (got %d)", kMaxHeads, c->n_kv);
  if (c->n_pages < 0) return fail(QE_ERR_INVALID_ARG, "n_pages must be >= 0 (got %d)", c->n_pages);
  const int64_t page = (int64_t)c->n_kv * c->page_size * c->head_dim;
  if (c->k_page_stride < page || c->v_page_stride < page || (c->k_page_stride & 7) || (c->v_page_stride & 7))
    return fail(QE_ERR_INVALID_ARG, "page strides must be multiples of 8 elements, at least n_kv * page_size * head_dim");
  int rc;
  if (c->n_pages > 0 && ((rc = check_ptr(c->k, "cache k", false, 16)) || (rc = check_ptr(c->v, "cache v", false, 16)))) return rc;
  return QE_OK;
}

// Between the first and the last row of both, rows the same distance apart overlap where their
// places within that distance do; others, which may meet somewhere, count as overlapping.
bool rows_overlap(const Rows& a, const Rows& b) {
  const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
  const size_t last = (size_t)a.n - 1, a1 = a0 + last * a.stride + a.row, b1 = b0 + last * b.stride + b.row;
  if (a0 >= b1 || b0 >= a1) return false;
  if (a.n == 1 || a.stride != b.stride) return true;
  const size_t d = b0 >= a0 ? (b0 - a0) % a.stride : (a.stride - (a0 - b0) % a.stride) % a.stride;
  return d < a.row || d + b.row > a.stride;
}

}  // namespace qe

using namespace qe;

extern "C" QE_API int attn_kv_append(const qe_kv_cache* c, const qe_rope* rope, int T, int n_q, const void* q,
                                     const void* k, const void* v, int in_dtype, int64_t q_stride, int64_t k_stride,
                                     int64_t v_stride, void* q_out, int64_t q_out_stride, const int32_t* pos,
                                     const int32_t* kv_pos, const int32_t* seq, const int32_t* table, int n_seq,
                                     int table_stride, void* ws, size_t ws_bytes, qe_stream_t stream) {
  int rc = check_kv_cache(c);
  if (rc) return rc;
  if (T < 0) return fail(QE_ERR_INVALID_ARG, "T must be >= 0");
  if (n_q < 0 || n_q > kMaxHeads) return fail(QE_ERR_INVALID_ARG, "n_q must be in [0, %d] (got %d)", kMaxHeads, n_q);
  if (!(in_dtype == QE_F32 || in_dtype == QE_BF16 || in_dtype == QE_F16))
    return fail(QE_ERR_INVALID_ARG, "in_dtype must be QE_F32, QE_BF16 or QE_F16 (got %d)", in_dtype);
  const int D = c->head_dim;
  if (rope) {
    if (rope->rotary_dim < 0 || (rope->rotary_dim & 15) || rope->rotary_dim > D)
      return fail(QE_ERR_INVALID_ARG, "rotary_dim must be a multiple of 16 in [0, head_dim] (got %d)", rope->rotary_dim);
    if (rope->n_axes < 1 || rope->n_axes > 4) return fail(QE_ERR_INVALID_ARG, "n_axes must be in [1, 4] (got %d)", rope->n_axes);
    if (rope->rotary_dim > 0 && (rc = check_ptr(rope->inv_freq, "inv_freq"))) return rc;
    for (int i = 0; rope->pair_axis && i < rope->rotary_dim / 2; ++i)
      if (rope->pair_axis[i] >= rope->n_axes)
        return fail(QE_ERR_INVALID_ARG, "pair_axis[%d] = %d is not below n_axes = %d", i, rope->pair_axis[i], rope->n_axes);
  }
  if (T == 0) return QE_OK;
  if ((rc = check_ptr(k, "k", false, 16)) || (rc = check_ptr(v, "v", false, 16)) || (rc = check_ptr(q, "q", n_q == 0, 16)) ||
      (rc = check_ptr(q_out, "q_out", n_q == 0, 16)) || (rc = check_ptr(pos, "pos", true)) ||
      (rc = check_ptr(kv_pos, "kv_pos")) || (rc = check_ptr(seq, "seq", true)) || (rc = check_ptr(table, "table")))
    return rc;
  if (n_seq < 0 || table_stride < 0) return fail(QE_ERR_INVALID_ARG, "n_seq and table_stride must be >= 0");
  if ((q_stride | k_stride | v_stride | q_out_stride) & 7)
    return fail(QE_ERR_INVALID_ARG, "token strides must be multiples of 8 elements");
  if (T > 1 && (k_stride < (int64_t)c->n_kv * D || v_stride < (int64_t)c->n_kv * D ||
                (n_q > 0 && (q_stride < (int64_t)n_q * D || q_out_stride < (int64_t)n_q * D))))
    return fail(QE_ERR_INVALID_ARG, "token strides must cover a token's heads");
  if (!ws || ((uintptr_t)ws & 255) || ws_bytes < sizeof(WsControl))
    return fail(QE_ERR_INVALID_ARG, "workspace must be 256-byte aligned and hold its control block");
  if (n_q > 0) {
    const size_t es = in_dtype == QE_F32 ? 4 : 2, q_row = (size_t)n_q * D, kv_row = (size_t)c->n_kv * D;
    const bool in_place = q_out == q && (q_out_stride == q_stride || T == 1) && in_dtype == c->dtype;
    const Rows to{q_out, 2 * q_row, 2 * (size_t)q_out_stride, T};
    if ((!in_place && rows_overlap(to, {q, es * q_row, es * (size_t)q_stride, T})) ||
        rows_overlap(to, {k, es * kv_row, es * (size_t)k_stride, T}) || rows_overlap(to, {v, es * kv_row, es * (size_t)v_stride, T}))
      return fail(QE_ERR_INVALID_ARG, "q_out overlaps q, k or v");
  }
  KvArgs a{};
  a.q = q; a.k = k; a.v = v; a.q_out = q_out; a.kc = c->k; a.vc = c->v;
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride; a.q_out_stride = q_out_stride;
  a.k_page_stride = c->k_page_stride; a.v_page_stride = c->v_page_stride;
  a.pos = pos; a.kv_pos = kv_pos; a.seq = seq; a.table = table;
  a.err = &((WsControl*)ws)->err;
  a.T = T; a.n_q = n_q; a.n_kv = c->n_kv; a.D = D; a.n_pages = c->n_pages; a.n_seq = n_seq; a.table_stride = table_stride;
  a.page = fast_div((uint32_t)c->page_size);
  if (rope) {
    a.rd = rope->rotary_dim;
    a.inv_freq = rope->inv_freq;
    for (int i = 0; rope->pair_axis && i < a.rd / 2; ++i) a.axis[i] = rope->pair_axis[i];
  }
  const bool adj = rope && rope->adjacent;
  const cudaError_t e = c->dtype == QE_BF16 ? launch_kv_in<__nv_bfloat16>(a, in_dtype, adj, (cudaStream_t)stream)
                                            : launch_kv_in<__half>(a, in_dtype, adj, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "attn_kv_append launch");
  return QE_OK;
}
