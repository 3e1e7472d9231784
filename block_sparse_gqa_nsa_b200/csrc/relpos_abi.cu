// C entry points of the relative-position-bias attention and of the layer norm: argument checks,
// workspace carving, launches.  See include/lsrm_nsa.h for the contract of each call.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "relpos.cuh"

namespace lsrm {
lsrm_status launch_relpos_forward(const rp::Params& p, int D, int NA, const rp::FwdPlan& f, cudaStream_t s);
lsrm_status launch_relpos_backward(const rp::Params& p, int D, int NA, const rp::BwdPlan& b, cudaStream_t s);
lsrm_status launch_layer_norm_forward(long long rows, int C, int dtype, const void* x, const void* gamma,
                                      const void* beta, float eps, void* y, float* mean, float* rstd, cudaStream_t s);
lsrm_status launch_layer_norm_backward(long long rows, int C, int dtype, const void* dy, const void* x,
                                       const void* gamma, const float* mean, const float* rstd, void* dx, void* dgamma,
                                       void* dbeta, float* part, cudaStream_t s);
int ln_max_ctas(long long rows, int C);
}  // namespace lsrm

using namespace lsrm;

namespace {

bool on(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// the layer norm's column counters go a CTA past the row's end; more rows than this are more than 2^31 - 1 CTAs
constexpr int32_t kLnMostWidth = 1 << 30;
constexpr int64_t kLnMostRows = (int64_t)1 << 40;

lsrm_status check_relpos(const lsrm_relpos_desc* d) {
  if (d == nullptr) return LSRM_ERR_INVALID_ARG;
  if (d->n_q_tokens < 0 || d->n_k_tokens < 0 || d->n_segs < 1) return LSRM_ERR_INVALID_ARG;
  if (d->n_kv_heads < 1 || d->n_q_heads < d->n_kv_heads || d->n_q_heads % d->n_kv_heads) return LSRM_ERR_INVALID_ARG;
  if (d->n_axes < 1 || d->n_axes > rp::kMaxAxes) return LSRM_ERR_INVALID_ARG;
  if (d->n_buckets < 1 || d->n_buckets > rp::kMaxBuckets) return LSRM_ERR_INVALID_ARG;
  if (d->max_distance < 1 || d->max_distance > rp::kMaxDistance) return LSRM_ERR_INVALID_ARG;
  if (!(d->scale >= 0.0f) || isinf(d->scale)) return LSRM_ERR_INVALID_ARG;
  if (d->head_dim != 32 && d->head_dim != 64) return LSRM_ERR_UNSUPPORTED;
  if (d->n_q_tokens > (int64_t)INT32_MAX || d->n_k_tokens > (int64_t)INT32_MAX) return LSRM_ERR_UNSUPPORTED;
  if (d->n_q_heads > 65535) return LSRM_ERR_UNSUPPORTED;  // before the plans, which try splits of a group's heads
  // tiles of every kernel in one grid dimension (the finest: one query token a tile and a KV head)
  const rp::FwdPlan f = rp::fwd_plan(*d);
  const rp::BwdPlan b = rp::bwd_plan(*d);
  const long long most = INT32_MAX;
  if (f.ctas > most || b.short_ctas > most || b.dq_tiles * d->n_q_heads > most ||
      b.kv_tiles * d->n_kv_heads * b.splits > most || d->n_segs > most / 2 || d->n_q_tokens + d->n_segs > most ||
      d->n_k_tokens + d->n_segs > most)
    return LSRM_ERR_UNSUPPORTED;
  return LSRM_OK;
}

// the inputs that both calls have, by the alignment that the kernels read them with
bool inputs_aligned(const int32_t* off_q, const int32_t* off_k, const int32_t* pos_q, const int32_t* pos_k,
                    const int32_t* bucket_of, const void* table, const void* q, const void* k, const void* v) {
  for (const void* x : {(const void*)off_q, (const void*)off_k, (const void*)pos_q, (const void*)pos_k,
                        (const void*)bucket_of})
    if (!on(x, 4)) return false;
  return on(table, 2) && on(q, 16) && on(k, 16) && on(v, 16);
}

lsrm_status check_relpos_ws(const lsrm_relpos_desc& d, const void* ws, size_t bytes) {
  if (ws == nullptr || !on(ws, 256) || bytes < rp::ws_layout(d).total) return LSRM_ERR_WORKSPACE;
  return LSRM_OK;
}

rp::Params params_of(const lsrm_relpos_desc& d, const int32_t* off_q, const int32_t* off_k, const int32_t* pos_q,
                     const int32_t* pos_k, const int32_t* bucket_of, const void* table, const void* q, const void* k,
                     const void* v, void* ws) {
  rp::Params p;
  memset(&p, 0, sizeof(p));
  const rp::Ws w = rp::ws_layout(d);
  unsigned char* base = static_cast<unsigned char*>(ws);
  p.off_q = off_q, p.off_k = off_k, p.pos_q = pos_q, p.pos_k = pos_k, p.bucket_of = bucket_of;
  p.table = static_cast<const uint16_t*>(table);
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.o_part = reinterpret_cast<float*>(base + w.o_part);
  p.ml_part = reinterpret_cast<float2*>(base + w.ml_part);
  p.delta = reinterpret_cast<float*>(base + w.delta);
  p.corr = reinterpret_cast<float*>(base + w.corr);
  p.lse2 = reinterpret_cast<float*>(base + w.lse2);
  p.tab_part = reinterpret_cast<float*>(base + w.tab_part);
  p.kv_part = reinterpret_cast<float*>(base + w.kv_part);
  p.status = reinterpret_cast<uint32_t*>(base + w.status);
  p.Nq = (int)d.n_q_tokens, p.Nk = (int)d.n_k_tokens, p.S = d.n_segs;
  p.Hq = d.n_q_heads, p.Hkv = d.n_kv_heads, p.G = d.n_q_heads / d.n_kv_heads;
  p.NB = d.n_buckets, p.maxd = d.max_distance;
  p.scale = d.scale > 0 ? d.scale : 1.0f / sqrtf((float)d.head_dim);
  return p;
}

// n <= 1023 to a power of at most 32, times another: 640 bits hold every product below
struct Big {
  uint32_t w[20] = {1};
  void times(uint32_t x) {
    uint64_t carry = 0;
    for (uint32_t& v : w) {
      carry += (uint64_t)v * x;
      v = (uint32_t)carry;
      carry >>= 32;
    }
  }
  static Big power(uint32_t x, int n) {
    Big b;
    while (n-- > 0) b.times(x);
    return b;
  }
  bool below(const Big& o) const {
    for (int i = 19; i >= 0; --i)
      if (w[i] != o.w[i]) return w[i] < o.w[i];
    return false;
  }
};

}  // namespace

extern "C" {

size_t lsrm_relpos_workspace_size(const lsrm_relpos_desc* desc) {
  return check_relpos(desc) == LSRM_OK ? rp::ws_layout(*desc).total : 0;
}

lsrm_status lsrm_relpos_workspace_init(const lsrm_relpos_desc* desc, void* ws, size_t ws_bytes, void* stream) {
  lsrm_status st = check_relpos(desc);
  if (st != LSRM_OK || (st = check_relpos_ws(*desc, ws, ws_bytes)) != LSRM_OK) return st;
  // only the status word: nothing else is read before a call writes it
  return cudaMemsetAsync(ws, 0, 256, (cudaStream_t)stream) == cudaSuccess ? LSRM_OK : LSRM_ERR_CUDA;
}

lsrm_status lsrm_relpos_log_buckets(int32_t n_buckets, int32_t max_distance, int32_t* bucket_of_host) {
  if (n_buckets < 2 || n_buckets > rp::kMaxBuckets || (n_buckets & 1) || max_distance < 1 ||
      max_distance > rp::kMaxDistance || bucket_of_host == nullptr)
    return LSRM_ERR_INVALID_ARG;
  const int half = n_buckets / 2, e = half / 2 > 1 ? half / 2 : 1, m = half - e, D = max_distance;
  int b = 0;
  for (int n = 0; n <= D; ++n) {
    int bucket = n;
    if (n >= e) {
      const Big nm = Big::power(n, m);
      for (; b + 1 < m; ++b) {
        Big border = Big::power(e, m - b - 1);  // n^m >= e^(m-b-1) D^(b+1)
        for (int i = 0; i <= b; ++i) border.times(D);
        if (nm.below(border)) break;
      }
      bucket = e + b < half - 1 ? e + b : half - 1;
    }
    bucket_of_host[D - n] = bucket;
    if (n > 0) bucket_of_host[D + n] = half + bucket;
  }
  return LSRM_OK;
}

lsrm_status lsrm_relpos_forward(const lsrm_relpos_desc* desc, const int32_t* off_q, const int32_t* off_k,
                                const int32_t* pos_q, const int32_t* pos_k, const int32_t* bucket_of,
                                const void* table, const void* q, const void* k, const void* v, void* out,
                                float* lse_or_null, void* ws, size_t ws_bytes, void* stream) {
  lsrm_status st = check_relpos(desc);
  if (st != LSRM_OK || (st = check_relpos_ws(*desc, ws, ws_bytes)) != LSRM_OK) return st;
  if (off_q == nullptr || off_k == nullptr || bucket_of == nullptr || table == nullptr) return LSRM_ERR_INVALID_ARG;
  if (desc->n_q_tokens > 0 && (pos_q == nullptr || q == nullptr || out == nullptr)) return LSRM_ERR_INVALID_ARG;
  if (desc->n_k_tokens > 0 && (pos_k == nullptr || k == nullptr || v == nullptr)) return LSRM_ERR_INVALID_ARG;
  if (!inputs_aligned(off_q, off_k, pos_q, pos_k, bucket_of, table, q, k, v) || !on(out, 16) || !on(lse_or_null, 4))
    return LSRM_ERR_INVALID_ARG;
  if (desc->n_q_tokens == 0) return LSRM_OK;
  rp::Params p = params_of(*desc, off_q, off_k, pos_q, pos_k, bucket_of, table, q, k, v, ws);
  const rp::FwdPlan f = rp::fwd_plan(*desc);
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse_or_null;
  p.splits = f.splits;
  return launch_relpos_forward(p, desc->head_dim, desc->n_axes, f, (cudaStream_t)stream);
}

lsrm_status lsrm_relpos_backward(const lsrm_relpos_desc* desc, const int32_t* off_q, const int32_t* off_k,
                                 const int32_t* pos_q, const int32_t* pos_k, const int32_t* bucket_of,
                                 const void* table, const void* q, const void* k, const void* v, const void* out,
                                 const float* lse, const void* dout, void* dq, void* dk, void* dv, void* dtable,
                                 void* ws, size_t ws_bytes, void* stream) {
  lsrm_status st = check_relpos(desc);
  if (st != LSRM_OK || (st = check_relpos_ws(*desc, ws, ws_bytes)) != LSRM_OK) return st;
  if (off_q == nullptr || off_k == nullptr || bucket_of == nullptr || table == nullptr || dtable == nullptr)
    return LSRM_ERR_INVALID_ARG;
  if (desc->n_q_tokens > 0 && (pos_q == nullptr || q == nullptr || out == nullptr || lse == nullptr ||
                               dout == nullptr || dq == nullptr))
    return LSRM_ERR_INVALID_ARG;
  if (desc->n_k_tokens > 0 && (pos_k == nullptr || k == nullptr || v == nullptr || dk == nullptr || dv == nullptr))
    return LSRM_ERR_INVALID_ARG;
  if (!inputs_aligned(off_q, off_k, pos_q, pos_k, bucket_of, table, q, k, v) || !on(lse, 4) || !on(dtable, 2))
    return LSRM_ERR_INVALID_ARG;
  for (const void* x : {out, dout, (const void*)dq, (const void*)dk, (const void*)dv})
    if (!on(x, 16)) return LSRM_ERR_INVALID_ARG;
  rp::Params p = params_of(*desc, off_q, off_k, pos_q, pos_k, bucket_of, table, q, k, v, ws);
  const rp::BwdPlan b = rp::bwd_plan(*desc);
  p.o_in = static_cast<const uint16_t*>(out);
  p.lse_in = lse;
  p.dout = static_cast<const uint16_t*>(dout);
  p.dq = static_cast<uint16_t*>(dq);
  p.dk = static_cast<uint16_t*>(dk);
  p.dv = static_cast<uint16_t*>(dv);
  p.dtable = static_cast<uint16_t*>(dtable);
  p.splits = b.splits;
  return launch_relpos_backward(p, desc->head_dim, desc->n_axes, b, (cudaStream_t)stream);
}

lsrm_status lsrm_layer_norm_forward(int64_t rows, int32_t width, int32_t dtype, const void* x,
                                    const void* gamma_or_null, const void* beta_or_null, float eps, void* y,
                                    float* mean_or_null, float* rstd_or_null, void* stream) {
  if (rows < 0 || width < 1 || (dtype != LSRM_BF16 && dtype != LSRM_F32) || !(eps >= 0.0f) || isinf(eps))
    return LSRM_ERR_INVALID_ARG;
  if (width > kLnMostWidth || rows > kLnMostRows) return LSRM_ERR_UNSUPPORTED;
  if (rows == 0) return LSRM_OK;
  const size_t el = dtype == LSRM_BF16 ? 2 : 4;
  if (x == nullptr || y == nullptr) return LSRM_ERR_INVALID_ARG;
  if (!on(x, el) || !on(y, el) || !on(gamma_or_null, el) || !on(beta_or_null, el) || !on(mean_or_null, 4) ||
      !on(rstd_or_null, 4))
    return LSRM_ERR_INVALID_ARG;
  return launch_layer_norm_forward(rows, width, dtype, x, gamma_or_null, beta_or_null, eps, y, mean_or_null,
                                   rstd_or_null, (cudaStream_t)stream);
}

size_t lsrm_layer_norm_workspace_size(int64_t rows, int32_t width) {
  if (rows < 0 || width < 1 || width > kLnMostWidth || rows > kLnMostRows) return 0;
  return rp::up256((size_t)ln_max_ctas(rows, width) * 2 * (size_t)width * 4);
}

lsrm_status lsrm_layer_norm_backward(int64_t rows, int32_t width, int32_t dtype, const void* dy, const void* x,
                                     const void* gamma_or_null, const float* mean, const float* rstd, void* dx,
                                     void* dgamma_or_null, void* dbeta_or_null, void* ws, size_t ws_bytes,
                                     void* stream) {
  if (rows < 0 || width < 1 || (dtype != LSRM_BF16 && dtype != LSRM_F32)) return LSRM_ERR_INVALID_ARG;
  if (width > kLnMostWidth || rows > kLnMostRows) return LSRM_ERR_UNSUPPORTED;
  const size_t el = dtype == LSRM_BF16 ? 2 : 4;
  if (rows > 0 && (dy == nullptr || x == nullptr || mean == nullptr || rstd == nullptr || dx == nullptr))
    return LSRM_ERR_INVALID_ARG;
  for (const void* a : {dy, x, gamma_or_null, (const void*)dx, (const void*)dgamma_or_null, (const void*)dbeta_or_null})
    if (!on(a, el)) return LSRM_ERR_INVALID_ARG;
  if (!on(mean, 4) || !on(rstd, 4)) return LSRM_ERR_INVALID_ARG;
  if (ws == nullptr || !on(ws, 256) || ws_bytes < lsrm_layer_norm_workspace_size(rows, width))
    return LSRM_ERR_WORKSPACE;
  return launch_layer_norm_backward(rows, width, dtype, dy, x, gamma_or_null, mean, rstd, dx, dgamma_or_null,
                                    dbeta_or_null, static_cast<float*>(ws), (cudaStream_t)stream);
}

}  // extern "C"
