// Layer norm of rows, forward and backward, with the reduction of the weights' gradients.
//
//   mean = sum(x) / C,  rstd = 1 / sqrt(sum((x - mean)^2) / C + eps),  xh = (x - mean) rstd
//   y = xh gamma + beta
//   g = dy gamma,  dx = rstd (g - mean(g) - xh mean(g xh)),  dgamma = sum_rows dy xh,
//   dbeta = sum_rows dy
//
// Both directions are bound by HBM: the forward reads x and writes y, the backward reads x and dy
// and writes dx, once each.  So a row lives in the registers of the lanes that share it (a group of
// 1..32 lanes of a warp, or a whole CTA for wide rows) between its statistics and its output, and
// the variance is the two-pass one (deviations from the row's own mean), which needs no second read.
// Rows too wide for registers are read again: in the forward, from the caches, past 16384 columns (8192 where rows lie
// off 16 bytes); in the backward past 8192 columns of bf16 or 4096 of fp32 (512 off 16 bytes), where the weights' sums
// have a pass over x and dy of their own.  Rows off 16 bytes, taken element by element, are far from HBM's rate:
// 100000 rows of 509 bf16 103 us forward and 115 backward (floors 31 and 47), of 1001 612 and 1008 (62 and 93), 50000 rows
// of 1001 fp32 120 and 531 (62 and 93).
//
// The backward keeps the column sums of dgamma and dbeta in registers over all rows a thread meets
// (a grid of as many CTAs as are resident, each walking its rows), adds the CTA's partials in
// shared memory in a fixed order, and a second kernel adds the CTAs' partials in a fixed order: no
// float atomics, so the gradients are the same bit for bit on every run.  All sums are fp32.
#include <climits>
#include <type_traits>

#include "dependent.cuh"
#include "lsrm_common.cuh"

namespace lsrm {
namespace {

constexpr int kLnThreads = 256;
constexpr int kLnWarps = kLnThreads / 32;
constexpr int kLnSms = 148;
constexpr int kLnWidest = 8192;  // elements of a row that the backward keeps in registers, at most
constexpr int kLnWideSplits = 64;

// ---- element types ----
template <typename T>
__device__ __forceinline__ float ln_to_f32(T v);
template <>
__device__ __forceinline__ float ln_to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float ln_to_f32<uint16_t>(uint16_t v) { return bf16_to_f32(v); }
template <typename T>
__device__ __forceinline__ T ln_from_f32(float v);
template <>
__device__ __forceinline__ float ln_from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t ln_from_f32<uint16_t>(float v) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// VEC consecutive elements as loaded: 16 bytes, or one element where the rows are not aligned.
// Plain (coherent) loads: y may be x, and dx may be dy or x.
template <typename T, int VEC>
struct LnVec {
  static_assert(VEC == 1 || VEC * sizeof(T) == 16, "16-byte vectors or single elements");
  T v[VEC];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC == 1) {
      v[0] = *p;
    } else {
      *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p);
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (VEC == 1) {
      *p = v[0];
    } else {
      *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = T(0);
  }
  __device__ __forceinline__ float get(int e) const { return ln_to_f32<T>(v[e]); }
  __device__ __forceinline__ void set(int e, float f) { v[e] = ln_from_f32<T>(f); }
};

// ---- two fp32 values at once: packed f32x2 ----
// The forward issued 3.1 to 3.2 of 4 instructions a clock and SM without it (head rows of 32: 20.6 -> 18.6 us,
// hidden rows of 1024: 91 -> 87.7).  The backward waits for its loads (2.5 a clock) and stays scalar: packed, rows
// of 256 went 117 -> 135 us and rows of 4096 182 -> 202, others within 2%.
using P2 = uint64_t;
__device__ __forceinline__ P2 p2(float a, float b) {
  P2 r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ P2 p2_add(P2 a, P2 b) {
  P2 r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ P2 p2_mul(P2 a, P2 b) {
  P2 r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ P2 p2_fma(P2 a, P2 b, P2 c) {
  P2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ void p2_out(P2 a, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(x), "=f"(y) : "l"(a));
}
__device__ __forceinline__ float p2_sum(P2 a) {
  float x, y;
  p2_out(a, x, y);
  return x + y;
}

// As LnVec, in pairs (a single element's pair is the element and 0): two bf16 of a word are its shifted and
// its masked half, one instruction each, where an array of 16-bit elements costs two more to take apart.
template <typename T, int VEC>
struct LnPairs {
  static_assert(VEC * sizeof(T) == 16, "16-byte vectors or single elements");
  static constexpr int kPairs = VEC / 2;
  uint32_t w[4];
  __device__ __forceinline__ void load(const T* p) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  }
  __device__ __forceinline__ void store(T* p) const {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0; }
  __device__ __forceinline__ P2 get(int e) const {
    if constexpr (sizeof(T) == 2)
      return p2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
    else
      return p2(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1]));
  }
  __device__ __forceinline__ void set(int e, P2 a) {
    float x, y;
    p2_out(a, x, y);
    if constexpr (sizeof(T) == 2) {
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(w[e]) : "f"(y), "f"(x));
    } else {
      w[2 * e] = __float_as_uint(x);
      w[2 * e + 1] = __float_as_uint(y);
    }
  }
};
template <typename T>
struct LnPairs<T, 1> {
  static constexpr int kPairs = 1;
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ void store(T* p) const { *p = v; }
  __device__ __forceinline__ void zero() { v = T(0); }
  __device__ __forceinline__ P2 get(int) const { return p2(ln_to_f32<T>(v), 0.0f); }
  __device__ __forceinline__ void set(int, P2 a) {
    float x, y;
    p2_out(a, x, y);
    v = ln_from_f32<T>(x);
  }
};

// sum over the TPR threads that share a row: a lane group of a warp, or the whole CTA
template <int TPR>
__device__ __forceinline__ float ln_row_sum(float v, float* red) {
  constexpr int kLanes = TPR < 32 ? TPR : 32;
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (TPR > 32) {
    static_assert(TPR == kLnThreads, "a row belongs to a lane group or to the CTA");
    __syncthreads();  // the previous sum has been read
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < kLnWarps; ++w) v += red[w];
  }
  return v;
}

struct LnFwd {
  const void* x;
  const void* gamma;
  const void* beta;
  void* y;
  float* mean;
  float* rstd;
  long long rows;
  int C;
  float eps;
};

// Rows in registers: TPR threads a row, NV vectors of VEC elements a thread (C <= TPR * VEC * NV), R rows
// a thread group at once, all loaded before the first is used
template <typename T, int VEC, int TPR, int NV, int R>
__global__ void __launch_bounds__(kLnThreads) ln_fwd_kernel(const LnFwd p) {
  __shared__ float red[kLnWarps];
  constexpr int kGroups = kLnThreads / TPR;
  const int sub = threadIdx.x % TPR;
  const long long row0 = (long long)blockIdx.x * (kGroups * R) + threadIdx.x / TPR;
  using V = LnPairs<T, VEC>;
  V xv[R][NV];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const long long row = row0 + k * kGroups;
    const T* x = static_cast<const T*>(p.x) + (row < p.rows ? row : 0) * p.C;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + sub) * VEC;
      if (row < p.rows && c < p.C)
        xv[k][i].load(x + c);
      else
        xv[k][i].zero();
    }
  }
  float mean[R], rstd[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    P2 s = p2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < V::kPairs; ++e) s = p2_add(s, xv[k][i].get(e));
    mean[k] = ln_row_sum<TPR>(p2_sum(s), red) / (float)p.C;
  }
#pragma unroll
  for (int k = 0; k < R; ++k) {
    P2 s = p2(0.0f, 0.0f);
    const P2 less = p2(-mean[k], VEC == 1 ? 0.0f : -mean[k]);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if ((i * TPR + sub) * VEC < p.C) {
#pragma unroll
        for (int e = 0; e < V::kPairs; ++e) {
          const P2 d = p2_add(xv[k][i].get(e), less);
          s = p2_fma(d, d, s);
        }
      }
    }
    rstd[k] = rsqrtf(ln_row_sum<TPR>(p2_sum(s), red) / (float)p.C + p.eps);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + sub) * VEC;
    if (c >= p.C) continue;
    V gv, bv;
    if (p.gamma != nullptr) gv.load(static_cast<const T*>(p.gamma) + c);
    if (p.beta != nullptr) bv.load(static_cast<const T*>(p.beta) + c);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const long long row = row0 + k * kGroups;
      if (row >= p.rows) continue;
      const P2 less = p2(-mean[k], -mean[k]), by = p2(rstd[k], rstd[k]);
#pragma unroll
      for (int e = 0; e < V::kPairs; ++e) {
        P2 o = p2_mul(p2_add(xv[k][i].get(e), less), by);
        if (p.gamma != nullptr && p.beta != nullptr)
          o = p2_fma(o, gv.get(e), bv.get(e));
        else if (p.gamma != nullptr)
          o = p2_mul(o, gv.get(e));
        else if (p.beta != nullptr)
          o = p2_add(o, bv.get(e));
        xv[k][i].set(e, o);
      }
      xv[k][i].store(static_cast<T*>(p.y) + row * p.C + c);
    }
  }
  if (sub == 0) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const long long row = row0 + k * kGroups;
      if (row >= p.rows) continue;
      if (p.mean != nullptr) p.mean[row] = mean[k];
      if (p.rstd != nullptr) p.rstd[row] = rstd[k];
    }
  }
}

// Rows of any width, one CTA each, read three times (the later reads come from the caches)
template <typename T>
__global__ void __launch_bounds__(kLnThreads) ln_fwd_wide_kernel(const LnFwd p) {
  __shared__ float red[kLnWarps];
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.C;
  T* y = static_cast<T*>(p.y) + row * p.C;
  const T* gamma = static_cast<const T*>(p.gamma);
  const T* beta = static_cast<const T*>(p.beta);
  float s = 0.0f;
  for (int c = threadIdx.x; c < p.C; c += kLnThreads) s += ln_to_f32<T>(x[c]);
  const float mean = ln_row_sum<kLnThreads>(s, red) / (float)p.C;
  s = 0.0f;
  for (int c = threadIdx.x; c < p.C; c += kLnThreads) {
    const float d = ln_to_f32<T>(x[c]) - mean;
    s = fmaf(d, d, s);
  }
  const float rstd = rsqrtf(ln_row_sum<kLnThreads>(s, red) / (float)p.C + p.eps);
  for (int c = threadIdx.x; c < p.C; c += kLnThreads) {
    float o = (ln_to_f32<T>(x[c]) - mean) * rstd;
    if (gamma != nullptr) o *= ln_to_f32<T>(gamma[c]);
    if (beta != nullptr) o += ln_to_f32<T>(beta[c]);
    y[c] = ln_from_f32<T>(o);
  }
  if (threadIdx.x == 0) {
    if (p.mean != nullptr) p.mean[row] = mean;
    if (p.rstd != nullptr) p.rstd[row] = rstd;
  }
}

struct LnBwd {
  const void* dy;
  const void* x;
  const void* gamma;
  const float* mean;
  const float* rstd;
  void* dx;
  float* part;  // [CTAs][2][C]: the CTA's sums of dgamma and dbeta
  long long rows;
  int C;
};

// Rows shared by a lane group of a warp: TPR threads a row, R rows a group at once
template <typename T, int VEC, int TPR, int NV, int R>
__global__ void __launch_bounds__(kLnThreads) ln_bwd_kernel(const LnBwd p) {
  static_assert(TPR <= 32, "a lane group");
  __shared__ float cols[kLnWarps][2][32 * VEC];
  let_dependents();
  constexpr int kGroups = kLnThreads / TPR;
  const int sub = threadIdx.x % TPR;
  LnVec<T, VEC> gv[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + sub) * VEC;
    gv[i].zero();
    if (c < p.C) {
      if (p.gamma != nullptr)
        gv[i].load(static_cast<const T*>(p.gamma) + c);
      else
#pragma unroll
        for (int e = 0; e < VEC; ++e) gv[i].set(e, 1.0f);
    }
  }
  float dg[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) dg[i][e] = db[i][e] = 0.0f;

  const float inv_c = 1.0f / (float)p.C;
  const long long steps = (p.rows + kGroups * R - 1) / (kGroups * R);
  for (long long it = blockIdx.x; it < steps; it += gridDim.x) {
    const long long row0 = it * (kGroups * R) + threadIdx.x / TPR;
    LnVec<T, VEC> xv[R][NV], dv[R][NV];
    float mean[R], rstd[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const long long row = row0 + k * kGroups;
      const bool live = row < p.rows;
      const long long at = (live ? row : 0) * p.C;
      mean[k] = live ? p.mean[row] : 0.0f;
      rstd[k] = live ? p.rstd[row] : 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + sub) * VEC;
        if (live && c < p.C) {
          xv[k][i].load(static_cast<const T*>(p.x) + at + c);
          dv[k][i].load(static_cast<const T*>(p.dy) + at + c);
        } else {
          xv[k][i].zero();
          dv[k][i].zero();
        }
      }
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const long long row = row0 + k * kGroups;
      float sg = 0.0f, sgx = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float xh = (xv[k][i].get(e) - mean[k]) * rstd[k], d = dv[k][i].get(e), g = d * gv[i].get(e);
          sg += g;
          sgx = fmaf(g, xh, sgx);
          dg[i][e] = fmaf(d, xh, dg[i][e]);
          db[i][e] += d;
        }
      sg = ln_row_sum<TPR>(sg, nullptr) * inv_c;
      sgx = ln_row_sum<TPR>(sgx, nullptr) * inv_c;
      if (row >= p.rows) continue;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + sub) * VEC;
        if (c >= p.C) continue;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float xh = (xv[k][i].get(e) - mean[k]) * rstd[k], g = dv[k][i].get(e) * gv[i].get(e);
          xv[k][i].set(e, rstd[k] * (g - sg - xh * sgx));
        }
        xv[k][i].store(static_cast<T*>(p.dx) + row * p.C + c);
      }
    }
  }

  // the CTA's column sums, in a fixed order
  float* part = p.part + (long long)blockIdx.x * 2 * p.C;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      float a = dg[i][e], b = db[i][e];
#pragma unroll
      for (int o = TPR; o < 32; o <<= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
      }
      if (lane < TPR) {
        cols[warp][0][lane * VEC + e] = a;
        cols[warp][1][lane * VEC + e] = b;
      }
    }
    __syncthreads();
    for (int t = threadIdx.x; t < 2 * TPR * VEC; t += kLnThreads) {
      const int which = t / (TPR * VEC), c = t % (TPR * VEC), col = i * TPR * VEC + c;
      if (col >= p.C) continue;
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kLnWarps; ++w) s += cols[w][which][c];
      part[which * p.C + col] = s;
    }
  }
}

// Rows by whole CTAs of NT threads, one vector a thread (C <= NT * VEC), R rows at once.  A thread keeps
// the sums of only VEC columns, so several CTAs fit an SM (a warp a row would need 4 x the registers
// at 1024 columns and leave 8 warps an SM: 177 us against the floor of 115 at 121344 rows); the R rows'
// statistics cross the warps behind one barrier.
template <typename T, int VEC, int NT, int R>
__global__ void __launch_bounds__(NT, NT < 512 ? 512 / NT : 1) ln_bwd_cta_kernel(const LnBwd p) {
  constexpr int kWarps = NT / 32;
  static_assert(2 * R <= 32 && (2 * R & (2 * R - 1)) == 0, "the statistics are folded over the lanes");
  __shared__ float red[2][kWarps][2 * R];
  let_dependents();
  const int c = threadIdx.x * VEC, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool have = c < p.C;
  LnVec<T, VEC> gv;
  gv.zero();
  if (have) {
    if (p.gamma != nullptr)
      gv.load(static_cast<const T*>(p.gamma) + c);
    else
#pragma unroll
      for (int e = 0; e < VEC; ++e) gv.set(e, 1.0f);
  }
  float dg[VEC], db[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) dg[e] = db[e] = 0.0f;
  const float inv_c = 1.0f / (float)p.C;
  const long long steps = (p.rows + R - 1) / R;
  int buf = 0;
  for (long long it = blockIdx.x; it < steps; it += gridDim.x, buf ^= 1) {
    LnVec<T, VEC> xv[R], dv[R];
    float mean[R], rstd[R], s[2 * R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const long long row = it * R + k;
      const bool live = row < p.rows;
      mean[k] = live ? p.mean[row] : 0.0f;
      rstd[k] = live ? p.rstd[row] : 0.0f;
      if (live && have) {
        xv[k].load(static_cast<const T*>(p.x) + row * p.C + c);
        dv[k].load(static_cast<const T*>(p.dy) + row * p.C + c);
      } else {
        xv[k].zero();
        dv[k].zero();
      }
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      float sg = 0.0f, sgx = 0.0f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float xh = (xv[k].get(e) - mean[k]) * rstd[k], d = dv[k].get(e), g = d * gv.get(e);
        sg += g;
        sgx = fmaf(g, xh, sgx);
        dg[e] = fmaf(d, xh, dg[e]);
        db[e] += d;
      }
      s[2 * k] = sg;
      s[2 * k + 1] = sgx;
    }
    // 2 R sums over the warp: while there are several, the halves of the lanes swap the sums they give
    // up, so 2 R values cost 2 R - 1 + (5 - log2 2R) shuffles instead of 5 each
    int n = 2 * R, o = 16;
#pragma unroll
    for (int step = 0; step < 5; ++step, o >>= 1) {
      if (n > 1) {
        n >>= 1;
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          if (i >= n) break;
          const float give = up ? s[i] : s[i + n], keep = up ? s[i + n] : s[i];
          s[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
      } else {
        s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
      }
    }
    // lane bits from the top select the sum that the lane holds
    constexpr int kFold = 2 * R == 2 ? 1 : 2 * R == 4 ? 2 : 2 * R == 8 ? 3 : 4;
    if ((lane & ((1 << (5 - kFold)) - 1)) == 0) red[buf][warp][lane >> (5 - kFold)] = s[0];
    __syncthreads();  // the buffer's last readers are two barriers back
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const long long row = it * R + k;
      float sg = 0.0f, sgx = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        sg += red[buf][w][2 * k];
        sgx += red[buf][w][2 * k + 1];
      }
      sg *= inv_c;
      sgx *= inv_c;
      if (row >= p.rows || !have) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float xh = (xv[k].get(e) - mean[k]) * rstd[k], g = dv[k].get(e) * gv.get(e);
        xv[k].set(e, rstd[k] * (g - sg - xh * sgx));
      }
      xv[k].store(static_cast<T*>(p.dx) + row * p.C + c);
    }
  }
  if (!have) return;
  float* part = p.part + (long long)blockIdx.x * 2 * p.C;
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    part[c + e] = dg[e];
    part[p.C + c + e] = db[e];
  }
}

// dx of rows of any width (one CTA each, two reads); the weights' sums come from ln_bwd_cols_kernel
template <typename T>
__global__ void __launch_bounds__(kLnThreads) ln_bwd_wide_kernel(const LnBwd p) {
  __shared__ float red[kLnWarps];
  const long long row = blockIdx.x, at = row * p.C;
  const T* x = static_cast<const T*>(p.x) + at;
  const T* dy = static_cast<const T*>(p.dy) + at;
  const T* gamma = static_cast<const T*>(p.gamma);
  T* dx = static_cast<T*>(p.dx) + at;
  const float mean = p.mean[row], rstd = p.rstd[row];
  float sg = 0.0f, sgx = 0.0f;
  for (int c = threadIdx.x; c < p.C; c += kLnThreads) {
    const float g = ln_to_f32<T>(dy[c]) * (gamma != nullptr ? ln_to_f32<T>(gamma[c]) : 1.0f);
    sg += g;
    sgx = fmaf(g, (ln_to_f32<T>(x[c]) - mean) * rstd, sgx);
  }
  sg = ln_row_sum<kLnThreads>(sg, red) / (float)p.C;
  sgx = ln_row_sum<kLnThreads>(sgx, red) / (float)p.C;
  for (int c = threadIdx.x; c < p.C; c += kLnThreads) {
    const float g = ln_to_f32<T>(dy[c]) * (gamma != nullptr ? ln_to_f32<T>(gamma[c]) : 1.0f);
    dx[c] = ln_from_f32<T>(rstd * (g - sg - (ln_to_f32<T>(x[c]) - mean) * rstd * sgx));
  }
}

// column sums of a run of rows (grid: column tiles x row splits), before dx may overwrite x or dy
template <typename T>
__global__ void __launch_bounds__(kLnThreads) ln_bwd_cols_kernel(const LnBwd p) {
  const int c = blockIdx.x * kLnThreads + threadIdx.x;
  if (c >= p.C) return;
  const long long per = (p.rows + gridDim.y - 1) / gridDim.y;
  const long long r0 = blockIdx.y * per, r1 = min(r0 + per, p.rows);
  float a = 0.0f, b = 0.0f;
  for (long long r = r0; r < r1; ++r) {
    const float d = ln_to_f32<T>(static_cast<const T*>(p.dy)[r * p.C + c]);
    const float xh = (ln_to_f32<T>(static_cast<const T*>(p.x)[r * p.C + c]) - p.mean[r]) * p.rstd[r];
    a = fmaf(d, xh, a);
    b += d;
  }
  float* part = p.part + (long long)blockIdx.y * 2 * p.C;
  part[c] = a;
  part[p.C + c] = b;
}

// dgamma / dbeta = the sum of the CTAs' partials: 32 columns a CTA, its warps take every 32nd partial,
// and the warps' sums are added in order
template <typename T>
__global__ void __launch_bounds__(1024) ln_bwd_finish_kernel(const float* part, int n, int C, void* dgamma,
                                                             void* dbeta) {
  __shared__ float s[2][32][33];
  wait_for_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float a = 0.0f, b = 0.0f;
  if (c < C) {
#pragma unroll 4
    for (int i = warp; i < n; i += 32) {
      a += part[(long long)i * 2 * C + c];
      b += part[(long long)i * 2 * C + C + c];
    }
  }
  s[0][warp][lane] = a;
  s[1][warp][lane] = b;
  __syncthreads();
  if (warp >= 2 || c >= C) return;
  void* out = warp == 0 ? dgamma : dbeta;
  if (out == nullptr) return;
  float t = 0.0f;
#pragma unroll
  for (int w = 0; w < 32; ++w) t += s[warp][w][lane];
  static_cast<T*>(out)[c] = ln_from_f32<T>(t);
}

// ---- variants: by the row's width, the element type and alignment alone ----
//
// Aligned rows (C a multiple of the vector, pointers on 16 bytes): the fewest lanes that hold the row
// with one vector each up to a warp; then the forward takes up to 8 (bf16) or 16 (fp32) vectors a lane
// and a CTA a row past that, the backward whole CTAs of 64 to 1024 threads with one vector each.
// Others: single elements, coalesced across the lanes, up to 32 (backward 16) a lane.
struct LnShape {
  int vec, tpr, nv;  // nv = 0: the wide kernels; the backward's tpr > 32: CTAs of tpr threads
};

LnShape ln_shape(int C, int elem, bool vec_ok, bool backward) {
  const int vec = vec_ok ? 16 / elem : 1;
  const int n = (C + vec - 1) / vec;  // vectors a row
  const int most = vec_ok ? (backward ? 1 : 64 / vec) : (backward ? 16 : 32);
  int tpr = 1;
  while (tpr < 32 && tpr < n) tpr *= 2;
  int nv = 1;
  while (nv * tpr < n) nv *= 2;
  if (nv <= most) return {vec, tpr, nv};
  if (backward) {
    if (!vec_ok) return {1, kLnThreads, 0};
    while (tpr < n && tpr <= 1024) tpr *= 2;
    if (tpr <= 1024) return {vec, tpr, 1};
    return {1, kLnThreads, 0};
  }
  tpr = kLnThreads;
  nv = 1;
  while (nv * tpr < n) nv *= 2;
  if (nv <= most) return {vec, tpr, nv};
  return {1, kLnThreads, 0};
}

lsrm_status ln_launched() { return cudaGetLastError() == cudaSuccess ? LSRM_OK : LSRM_ERR_CUDA; }

// Rows a thread group takes at once: two where a thread holds 16 bytes of a row, as long as that still
// leaves every SM a few CTAs (head rows of 32, before the packed sums: one row 24.5 us, two or four 20.6, eight
// 25.7; four rows of 64 bytes a thread 159 us against 92 with one).
constexpr int kLnRows = 2;
// of the backward's CTAs (hidden rows of 1024: two rows 142 us, four 140, eight 183; at least 512 threads
// an SM: 640 cost spills, 148 -> 164 us)
constexpr int kLnCtaRows = 4;
template <typename T, int VEC, int TPR, int NV>
lsrm_status ln_run_fwd(const LnFwd& p, cudaStream_t s) {
  constexpr int kGroups = kLnThreads / TPR, R = NV * VEC * (int)sizeof(T) <= 16 ? kLnRows : 1;
  if (R > 1 && p.rows >= (long long)kGroups * R * 4 * kLnSms) {
    const long long ctas = (p.rows + kGroups * R - 1) / (kGroups * R);
    if (ctas > (long long)INT32_MAX) return LSRM_ERR_UNSUPPORTED;
    ln_fwd_kernel<T, VEC, TPR, NV, R><<<(unsigned)ctas, kLnThreads, 0, s>>>(p);
    return ln_launched();
  }
  const long long ctas = (p.rows + kGroups - 1) / kGroups;
  if (ctas > (long long)INT32_MAX) return LSRM_ERR_UNSUPPORTED;
  ln_fwd_kernel<T, VEC, TPR, NV, 1><<<(unsigned)ctas, kLnThreads, 0, s>>>(p);
  return ln_launched();
}

// CTAs of a persistent backward kernel: as many as are resident, or as there are steps
template <typename K>
lsrm_status ln_ctas(K kernel, int threads, long long steps, int max_ctas, int* ctas) {
  int per_sm = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, 0) != cudaSuccess) return LSRM_ERR_CUDA;
  const long long fit = (long long)kLnSms * (per_sm > 0 ? per_sm : 1);
  long long n = steps < fit ? steps : fit;
  if (n > max_ctas) n = max_ctas;
  *ctas = (int)n;
  return n < 1 ? LSRM_ERR_CUDA : LSRM_OK;
}

template <typename T, int VEC, int TPR, int NV>
lsrm_status ln_run_bwd(const LnBwd& p, int max_ctas, int* ctas, cudaStream_t s) {
  lsrm_status st;
  if constexpr (TPR > 32) {
    constexpr int R = TPR == 1024 ? 2 : kLnCtaRows;
    auto kernel = ln_bwd_cta_kernel<T, VEC, TPR, R>;
    if ((st = ln_ctas(kernel, TPR, (p.rows + R - 1) / R, max_ctas, ctas)) != LSRM_OK) return st;
    kernel<<<(unsigned)*ctas, TPR, 0, s>>>(p);
  } else {
    constexpr int kGroups = kLnThreads / TPR, R = VEC > 1 ? kLnRows : 1;
    auto kernel = ln_bwd_kernel<T, VEC, TPR, NV, R>;
    if ((st = ln_ctas(kernel, kLnThreads, (p.rows + kGroups * R - 1) / (kGroups * R), max_ctas, ctas)) != LSRM_OK)
      return st;
    kernel<<<(unsigned)*ctas, kLnThreads, 0, s>>>(p);
  }
  return ln_launched();
}

// f(vector width, vectors a thread, threads a row) with the shape as template arguments
template <int V, int N>
struct LnTag {
  static constexpr int vec = V, nv = N;
};
template <bool BWD, int TPR, typename T, typename F>
lsrm_status ln_nv(const LnShape& h, F f) {
  constexpr int V = 16 / sizeof(T);
  constexpr std::integral_constant<int, TPR> tpr{};
  if (h.vec == V) {
    if (h.nv == 1) return f(LnTag<V, 1>{}, tpr);
    if constexpr (!BWD && TPR >= 32) {
      switch (h.nv) {
        case 2: return f(LnTag<V, 2>{}, tpr);
        case 4: return f(LnTag<V, 4>{}, tpr);
        case 8: return f(LnTag<V, 8>{}, tpr);
        case 16: if constexpr (V == 4) return f(LnTag<V, 16>{}, tpr); break;
      }
    }
  } else if constexpr (!BWD || TPR <= 32) {
    if (h.nv == 1) return f(LnTag<1, 1>{}, tpr);
    if constexpr (TPR >= 32) {
      switch (h.nv) {
        case 2: return f(LnTag<1, 2>{}, tpr);
        case 4: return f(LnTag<1, 4>{}, tpr);
        case 8: return f(LnTag<1, 8>{}, tpr);
        case 16: return f(LnTag<1, 16>{}, tpr);
        case 32: if constexpr (!BWD) return f(LnTag<1, 32>{}, tpr); break;
      }
    }
  }
  return LSRM_ERR_UNSUPPORTED;
}
template <bool BWD, typename T, typename F>
lsrm_status ln_dispatch(const LnShape& h, F f) {
  switch (h.tpr) {
    case 1: return ln_nv<BWD, 1, T>(h, f);
    case 2: return ln_nv<BWD, 2, T>(h, f);
    case 4: return ln_nv<BWD, 4, T>(h, f);
    case 8: return ln_nv<BWD, 8, T>(h, f);
    case 16: return ln_nv<BWD, 16, T>(h, f);
    case 32: return ln_nv<BWD, 32, T>(h, f);
    case 64: if constexpr (BWD) return ln_nv<BWD, 64, T>(h, f); break;
    case 128: if constexpr (BWD) return ln_nv<BWD, 128, T>(h, f); break;
    case 256: return ln_nv<BWD, 256, T>(h, f);
    case 512: if constexpr (BWD) return ln_nv<BWD, 512, T>(h, f); break;
    case 1024: if constexpr (BWD) return ln_nv<BWD, 1024, T>(h, f); break;
  }
  return LSRM_ERR_UNSUPPORTED;
}

bool on16(const void* p) { return ((uintptr_t)p & 15) == 0; }

template <typename T>
lsrm_status ln_forward(const LnFwd& p, cudaStream_t s) {
  const bool vec_ok = (p.C * sizeof(T)) % 16 == 0 && on16(p.x) && on16(p.y) && on16(p.gamma) && on16(p.beta);
  const LnShape h = ln_shape(p.C, (int)sizeof(T), vec_ok, false);
  if (h.nv == 0) {
    if (p.rows > (long long)INT32_MAX) return LSRM_ERR_UNSUPPORTED;
    ln_fwd_wide_kernel<T><<<(unsigned)p.rows, kLnThreads, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? LSRM_OK : LSRM_ERR_CUDA;
  }
  return ln_dispatch<false, T>(h, [&](auto tag, auto tpr) {
    return ln_run_fwd<T, decltype(tag)::vec, decltype(tpr)::value, decltype(tag)::nv>(p, s);
  });
}

template <typename T>
lsrm_status ln_backward(const LnBwd& p, void* dgamma, void* dbeta, int max_ctas, cudaStream_t s) {
  const bool vec_ok = (p.C * sizeof(T)) % 16 == 0 && on16(p.x) && on16(p.dy) && on16(p.dx) && on16(p.gamma);
  const LnShape h = ln_shape(p.C, (int)sizeof(T), vec_ok, true);
  int n = 0;
  if (p.rows > 0) {
    if (h.nv == 0) {
      if (p.rows > (long long)INT32_MAX) return LSRM_ERR_UNSUPPORTED;
      n = (int)(p.rows < kLnWideSplits ? p.rows : kLnWideSplits);
      if (n > max_ctas) n = max_ctas;
      const dim3 grid((unsigned)((p.C + kLnThreads - 1) / kLnThreads), (unsigned)n);
      ln_bwd_cols_kernel<T><<<grid, kLnThreads, 0, s>>>(p);
      if (cudaGetLastError() != cudaSuccess) return LSRM_ERR_CUDA;
      ln_bwd_wide_kernel<T><<<(unsigned)p.rows, kLnThreads, 0, s>>>(p);
      if (cudaGetLastError() != cudaSuccess) return LSRM_ERR_CUDA;
    } else {
      const lsrm_status st = ln_dispatch<true, T>(h, [&](auto tag, auto tpr) {
        return ln_run_bwd<T, decltype(tag)::vec, decltype(tpr)::value, decltype(tag)::nv>(p, max_ctas, &n, s);
      });
      if (st != LSRM_OK) return st;
    }
  }
  if (dgamma == nullptr && dbeta == nullptr) return LSRM_OK;
  return launch_dependent(ln_bwd_finish_kernel<T>, dim3((unsigned)((p.C + 31) / 32)), 1024, s, (const float*)p.part, n,
                          p.C, dgamma, dbeta)
             ? LSRM_OK
             : LSRM_ERR_CUDA;
}

}  // namespace

// CTAs whose partial sums the workspace holds: as many as can be resident,
// or one a row where there are fewer rows.  Rows above kLnWidest never fit registers; their column
// sums are split kLnWideSplits ways.
int ln_max_ctas(long long rows, int C) {
  const long long most = C > kLnWidest ? kLnWideSplits : 16 * kLnSms;
  return (int)(rows < most ? (rows > 0 ? rows : 1) : most);
}

lsrm_status launch_layer_norm_forward(long long rows, int C, int dtype, const void* x, const void* gamma,
                                      const void* beta, float eps, void* y, float* mean, float* rstd,
                                      cudaStream_t s) {
  const LnFwd p{x, gamma, beta, y, mean, rstd, rows, C, eps};
  return dtype == LSRM_F32 ? ln_forward<float>(p, s) : ln_forward<uint16_t>(p, s);
}

lsrm_status launch_layer_norm_backward(long long rows, int C, int dtype, const void* dy, const void* x,
                                       const void* gamma, const float* mean, const float* rstd, void* dx,
                                       void* dgamma, void* dbeta, float* part, cudaStream_t s) {
  const LnBwd p{dy, x, gamma, mean, rstd, dx, part, rows, C};
  const int most = ln_max_ctas(rows, C);
  return dtype == LSRM_F32 ? ln_backward<float>(p, dgamma, dbeta, most, s)
                           : ln_backward<uint16_t>(p, dgamma, dbeta, most, s);
}

}  // namespace lsrm
