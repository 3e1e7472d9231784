// Shared pieces of the tensor-memory kernels of the relative-position attention (relpos_tc.cu: forward,
// relpos_bwd_tc.cu: backward).  A thread owns a row of a 128-row tile (a tensor-memory lane); the 64
// columns of a chunk are the same for all lanes, so a bias that is the same for a run of columns costs
// one look-up for the run, and branches on the columns' positions are uniform.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "relpos.cuh"
#include "tma_map.cuh"

namespace lsrm {
namespace rp {

using namespace tc;

constexpr int kTcThreads = 320;  // producer warp, MMA warp, eight warps on the scores
constexpr int kTcCols = 64;      // columns a chunk

template <int D>
struct TcTile {
  static constexpr int kRowBytes = D * 2;
  static constexpr uint32_t kLayout = D == 32 ? kLayoutSW64 : kLayoutSW128;
  static constexpr uint32_t kAtomBytes = 8 * kRowBytes;
  static constexpr int kRowsBytes = 128 * kRowBytes, kColsBytes = kTcCols * kRowBytes;
  static constexpr uint32_t kIdescScore = idesc_bf16(128, kTcCols, false);  // rows x columns
  static constexpr uint32_t kIdescHalf = idesc_bf16(128, kTcCols / 2, false);  // half of the columns
  static constexpr uint32_t kIdescSum = idesc_bf16(128, D, true);           // rows x D over the columns
};

// Wait for this thread's tensor-memory loads into r.  The registers are operands of the wait, so nothing
// that reads them can be moved above it; and every load here is followed by its wait at once, with no
// branch between the two.
__device__ __forceinline__ void tmem_wait16(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_wait32(uint32_t* r) {
  tmem_wait16(r);
  tmem_wait16(r + 16);
}

// Bounded waits as tc::mbar_wait, which look at the abort flag and the clock only every 32 tries: a
// waiting thread then issues little beside the tries themselves.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      *abort = 1;
      raise_status(status, LSRM_ERR_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_bar_w(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* status) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, abort, status));
}

// 64 rows of a [tokens][heads][D] tensor into a stage in the layout that TMA writes, zeros past n: what
// lies behind a segment may be anything, and a weight of 0 does not hide an infinity.  A whole warp;
// the caller makes it visible to the tensor cores (fence_async) before its arrive.
template <int D>
__device__ __forceinline__ void copy_tail(uint8_t* dst, const uint16_t* src, int r0, int n, int heads, int h,
                                          int lane) {
  constexpr int kPieces = D / 8;
  for (int i = lane; i < kTcCols * kPieces; i += 32) {
    const int r = i / kPieces, c = i % kPieces;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (r < n) u = *reinterpret_cast<const uint4*>(src + ((size_t)(r0 + r) * heads + h) * D + c * 8);
    const int sw = D == 32 ? c ^ ((r >> 1) & 3) : c ^ (r & 7);
    *reinterpret_cast<uint4*>(dst + r * (D * 2) + sw * 16) = u;
  }
  __syncwarp();
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }

// kTurn is for positions on three axes (volumes, in bricks: forward of 4096 tokens, 32 heads of 32, 453 -> 430 us);
// with two, the further branch costs frames by rows more than it can save (8 of 1370 patches 267 -> 291 us)
template <int NA>
constexpr bool kHasTurn = NA == 3;
// what a chunk's column positions have in common on each axis: their range, and in byte g of runs kLane,
// kFour, kTurn or kEach: columns 16 g .. 16 g + 15 have one position, one per aligned run of four, the same
// four in every such run, any
struct ChunkMeta {
  int lo[kMaxAxes], hi[kMaxAxes];
  uint32_t runs[kMaxAxes];
};
// the producer warp's part: lane i holds the positions of columns i and i + 32
template <int NA>
__device__ __forceinline__ void note_positions(const int (&x)[NA][2], int (*pos)[kTcCols], ChunkMeta& m, int lane,
                                               uint32_t* status) {
#pragma unroll
  for (int a = 0; a < NA; ++a) {
    const int lo = __reduce_min_sync(0xffffffffu, min(x[a][0], x[a][1]));
    const int hi = __reduce_max_sync(0xffffffffu, max(x[a][0], x[a][1]));
    if (lo < -kPosLimit || hi > kPosLimit) raise_status(status, LSRM_ERR_BOUNDS);
    const uint32_t e0 = __ballot_sync(0xffffffffu, x[a][0] == __shfl_down_sync(0xffffffffu, x[a][0], 1));
    const uint32_t e1 = __ballot_sync(0xffffffffu, x[a][1] == __shfl_down_sync(0xffffffffu, x[a][1], 1));
    const uint32_t f0 = __ballot_sync(0xffffffffu, x[a][0] == __shfl_down_sync(0xffffffffu, x[a][0], 4));
    const uint32_t f1 = __ballot_sync(0xffffffffu, x[a][1] == __shfl_down_sync(0xffffffffu, x[a][1], 4));
    pos[a][lane] = x[a][0];
    pos[a][lane + 32] = x[a][1];
    if (lane == 0) {
      uint32_t runs = 0;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint32_t e = (g < 2 ? e0 : e1) >> (16 * (g & 1)), f = (g < 2 ? f0 : f1) >> (16 * (g & 1));
        runs |= (uint32_t)((e & 0x7fffu) == 0x7fffu   ? kLane
                           : (e & 0x7777u) == 0x7777u ? kFour
                           : kHasTurn<NA> && (f & 0x0fffu) == 0x0fffu ? kTurn
                                                                      : kEach)
                << (8 * g);
      }
      m.lo[a] = lo, m.hi[a] = hi, m.runs[a] = runs;
    }
  }
}

// A chunk's biases for a warp's rows.  Per axis and run of 16 columns: kOne (the chunk has one clamped
// distance), kLane (one position in the run), kFour (one per four columns), kTurn (the same
// four), kEach.  Positions count so that columns less rows is the distance (the key pass, whose columns are
// queries, negates both).
// Told run by run, as rows of patches end anywhere (forward of 8 x 1370 patches, 16 heads of 64: 250 us; one
// kind for the chunk 272).
template <int NA>
struct ChunkBias {
  int one[NA];  // the chunk's only index into the table, or -1
  uint32_t runs[NA];  // as ChunkMeta's, or 0 (kOne) for all
  float ub;  // the bias common to the chunk
  __device__ __forceinline__ void set(const ChunkMeta& m, const int (&row_lo)[NA], const int (&row_hi)[NA], int maxd,
                                      const float* lut, int top) {
    ub = 0.0f;
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      const int lo = clamp_index(m.lo[a] - row_hi[a], maxd, top);
      const int hi = clamp_index(m.hi[a] - row_lo[a], maxd, top);
      one[a] = lo == hi ? lo : -1;
      runs[a] = m.runs[a];
      if (lo == hi) {
        runs[a] = kOne;
        ub += lut[a * (top + 1) + lo];
      }
    }
  }
  __device__ __forceinline__ int mode(int a, int g) const { return runs[a] >> (8 * g) & 7; }
  // whether run g has one bias per row
  __device__ __forceinline__ bool flat(int g) const {
    bool f = true;
#pragma unroll
    for (int a = 0; a < NA; ++a) f = f && mode(a, g) <= kLane;
    return f;
  }
  // the row's part of run g that is the same for its columns, on top of base
  __device__ __forceinline__ float row16(float base, int (*pos)[kTcCols], int g, const int (&rowc)[NA],
                                         const float* lut, int top) const {
#pragma unroll
    for (int a = 0; a < NA; ++a)
      if (mode(a, g) == kLane) base += lut[a * (top + 1) + clamp_index(pos[a][16 * g], rowc[a], top)];
    return base;
  }
  // axis a's biases of run g (kFour and up) added to its 16 scores
  __device__ __forceinline__ void axis16(float (&x)[16], int (*pos)[kTcCols], int a, int g, const int (&rowc)[NA],
                                         const float* lut, int top) const {
    const float* la = lut + a * (top + 1);
    const int4* xs = reinterpret_cast<const int4*>(&pos[a][16 * g]);
    const int m = mode(a, g);
    if (m == kFour) {
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const float y = la[clamp_index(xs[f].x, rowc[a], top)];
        fadd2_acc(x[4 * f], x[4 * f + 1], y, y);
        fadd2_acc(x[4 * f + 2], x[4 * f + 3], y, y);
      }
    } else if (kHasTurn<NA> && m == kTurn) {
      const int4 u = xs[0];
      const float y0 = la[clamp_index(u.x, rowc[a], top)], y1 = la[clamp_index(u.y, rowc[a], top)];
      const float y2 = la[clamp_index(u.z, rowc[a], top)], y3 = la[clamp_index(u.w, rowc[a], top)];
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        fadd2_acc(x[4 * f], x[4 * f + 1], y0, y1);
        fadd2_acc(x[4 * f + 2], x[4 * f + 3], y2, y3);
      }
    } else if (m == kEach) {
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int4 u = xs[f];
        // single adds: a pair of look-ups would first have to be moved into a pair of registers
        x[4 * f] += la[clamp_index(u.x, rowc[a], top)];
        x[4 * f + 1] += la[clamp_index(u.y, rowc[a], top)];
        x[4 * f + 2] += la[clamp_index(u.z, rowc[a], top)];
        x[4 * f + 3] += la[clamp_index(u.w, rowc[a], top)];
      }
    }
  }
  // the rest of run g's biases (what row16 leaves out) added to its 16 scores
  __device__ __forceinline__ void add16(float (&x)[16], int (*pos)[kTcCols], int g, const int (&rowc)[NA],
                                        const float* lut, int top) const {
#pragma unroll
    for (int a = 0; a < NA; ++a) axis16(x, pos, a, g, rowc, lut, top);
  }
  // x = s * mul + all of run g's biases in the formula's own order, whatever the run has in common
  __device__ __forceinline__ void exact16(float (&x)[16], const uint32_t (&s)[16], float mul, int (*pos)[kTcCols],
                                          int g, const int (&rowc)[NA], const float* lut, int top) const {
#pragma unroll
    for (int e = 0; e < 16; e += 2)
      ffma2(x[e], x[e + 1], __uint_as_float(s[e]), __uint_as_float(s[e + 1]), mul, 0.0f);
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      const int m = mode(a, g);
      if (m <= kLane) {
        const float y = lut[a * (top + 1) + (m == kOne ? one[a] : clamp_index(pos[a][16 * g], rowc[a], top))];
#pragma unroll
        for (int e = 0; e < 16; e += 2) fadd2_acc(x[e], x[e + 1], y, y);
      } else {
        axis16(x, pos, a, g, rowc, lut, top);
      }
    }
  }
};

}  // namespace rp
}  // namespace lsrm
