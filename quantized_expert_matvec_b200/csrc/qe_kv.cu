// qe_kv.cu -- rotary positions on q and k, and the append of k and v to the
// paged cache: what precedes attn_decode_step in a full-attention layer.
//
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = pos[axis(i)] f_i
//
// The operator reads T (n_q + 2 n_kv) head_dim elements and writes as many:
// it is bound by HBM for prompts and by one launch's latency for a decode
// step.  One CTA serves one token: the angles of its rotary_dim / 2 pairs are
// computed once, into shared memory, and used by all its heads.  A thread's
// item is 16 elements of a head (8 pairs, or 16 elements that are copied): two
// 16-byte loads (four for fp32) and two 16-byte stores, requested before the
// angles are waited for.
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

constexpr int kKvThreads = 384;
constexpr int kMaxPairs = 128;  // head_dim 256 / 2

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
  int T, n_q, n_kv, D, rd, n_pages, n_seq, table_stride;
  FastDiv page;
  uint8_t axis[kMaxPairs];
};

// sin and cos of the angle a = pos * f.  The product of an integer below 2^31
// and an fp32 number is exact in fp64; the nearest multiple of pi / 2 is taken
// off in two parts (pi / 2 to 106 bits), which leaves |r| <= pi / 4 to about
// 2^-52 (n up to 2^31).  On that interval the Taylor polynomials to r^9 and r^10 are
// off by at most r^11 / 11! = 1.8e-9 and r^12 / 12! = 1.2e-10, below fp32's half step.
QE_DEV float2 cos_sin(int pos, float f) {
  const double a = (double)pos * (double)f;
  const double n = rint(a * 0.63661977236758134308);
  double rd = fma(-n, 1.5707963267948965580, a);
  rd = fma(-n, 6.1232339957367660359e-17, rd);
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

template <typename TI, typename TC, bool ADJ>
__global__ void __launch_bounds__(kKvThreads) qe_kv_append_kernel(const __grid_constant__ KvArgs a) {
  __shared__ float2 cs[kMaxPairs];
  grid_dependency_wait();
  grid_launch_dependents();
  const int t = blockIdx.x;
  const int p = a.kv_pos[t];
  if (p < 0) return;  // uniform over the CTA
  const int half = a.rd >> 1, per_head = a.D >> 4;
  const int items = (a.n_q + 2 * a.n_kv) * per_head;

  // where the token goes
  const int s = a.seq ? a.seq[t] : t;
  const int col = (int)a.page.div((uint32_t)p);
  int page = -1;
  if (s >= 0 && s < a.n_seq && col < a.table_stride) page = a.table[(size_t)s * a.table_stride + col];
  const bool ok = page >= 0 && page < a.n_pages;
  const int off = p - col * (int)a.page.d;
  if (!ok && threadIdx.x == 0) set_error(a.err, QE_ERR_INVALID_ARG);

  for (int i = threadIdx.x; i < half; i += blockDim.x)
    cs[i] = cos_sin(a.pos ? a.pos[(size_t)a.axis[i] * a.T + t] : p, a.inv_freq[i]);
  __syncthreads();

  for (int it = threadIdx.x; it < items; it += blockDim.x) {
    const int head = it / per_head, e = (it - head * per_head) << 4;  // first of 16 elements, in item order
    const TI* src;
    TC* dst;
    bool turn = true, write = true;
    if (head < a.n_q) {
      src = (const TI*)a.q + (size_t)t * a.q_stride + (size_t)head * a.D;
      dst = (TC*)a.q_out + (size_t)t * a.q_out_stride + (size_t)head * a.D;
    } else if (head < a.n_q + a.n_kv) {
      const int h = head - a.n_q;
      src = (const TI*)a.k + (size_t)t * a.k_stride + (size_t)h * a.D;
      dst = (TC*)a.kc + (long long)page * a.k_page_stride + ((long long)h * a.page.d + off) * a.D;
      write = ok;
    } else {
      const int h = head - a.n_q - a.n_kv;
      src = (const TI*)a.v + (size_t)t * a.v_stride + (size_t)h * a.D;
      dst = (TC*)a.vc + (long long)page * a.v_page_stride + ((long long)h * a.page.d + off) * a.D;
      turn = false;
      write = ok;
    }
    if (!write) continue;
    turn = turn && e < a.rd;
    // the two runs of 8: side by side, or a pair's two halves
    const bool split = turn && !ADJ;
    const int e0 = split ? e >> 1 : e, e1 = split ? e0 + half : e + 8;
    Raw8<TI> r0, r1;
    r0.load(src + e0);
    r1.load(src + e1);
    if constexpr (sizeof(TI) == 2 && std::is_same<TI, TC>::value) {
      if (!turn) {  // the bits as they are (a NaN's too)
        *reinterpret_cast<uint4*>(dst + e0) = r0.a;
        *reinterpret_cast<uint4*>(dst + e1) = r1.a;
        continue;
      }
    }
    float x[8], y[8];
    r0.get(x);
    r1.get(y);
    if (turn) {
      const int pair = e >> 1;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 w = cs[pair + j];
        float& u = ADJ ? (j < 4 ? x[2 * (j & 3)] : y[2 * (j & 3)]) : x[j];
        float& v = ADJ ? (j < 4 ? x[2 * (j & 3) + 1] : y[2 * (j & 3) + 1]) : y[j];
        const float u2 = fmaf(u, w.x, -v * w.y), v2 = fmaf(v, w.x, u * w.y);
        u = u2;
        v = v2;
      }
    }
    store8(dst + e0, x);
    store8(dst + e1, y);
  }
}

template <typename TI, typename TC>
cudaError_t launch_kv_t(const KvArgs& a, bool adjacent, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  const int items = (a.n_q + 2 * a.n_kv) * (a.D >> 4);
  int threads = (items + 31) / 32 * 32;
  threads = threads < 64 ? 64 : threads > kKvThreads ? kKvThreads : threads;
  cfg.gridDim = dim3((unsigned)a.T);
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

bool ranges_overlap(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a0 < b0 + b_bytes && b0 < a0 + a_bytes;
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
  if (n_q > 0 && !(q_out == q && q_out_stride == q_stride && in_dtype == c->dtype)) {
    const size_t es = in_dtype == QE_F32 ? 4 : 2, last = (size_t)T - 1;
    const size_t ob = 2 * (last * q_out_stride + (size_t)n_q * D);
    if (ranges_overlap(q_out, ob, q, es * (last * q_stride + (size_t)n_q * D)) ||
        ranges_overlap(q_out, ob, k, es * (last * k_stride + (size_t)c->n_kv * D)) ||
        ranges_overlap(q_out, ob, v, es * (last * v_stride + (size_t)c->n_kv * D)))
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
