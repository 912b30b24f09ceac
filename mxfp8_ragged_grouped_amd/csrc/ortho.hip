// ortho.hip -- orthogonalising a stack of updates by Newton-Schulz products
// (mxw_orthogonalize, declared in include/mxfp8_wgrad.h), for gfx950.
//
// For every expert's matrix G [N, K], with n = min(N, K), X0 = G / (|G|_F + eps)
// and, for each step's (a, b, c),
//
//     S  = X X^T        (X^T X where N > K: always n x n)
//     P  = a I + b S + c S S
//     X <- P X          (X P where N > K)
//
// an odd polynomial of X's singular values that drives them towards 1 and
// leaves the singular vectors alone.  a X is folded into the product as a I.
//
// Cost of a step: S n^2 m flops and P n^3 (both symmetric: only the tiles on
// and below the diagonal are computed, each written to both places), P X
// 2 n^2 m.  Everything is matrix products of n, m >= 100s: bound by the MFMA.
//
// X, S and P are held in f16, times 2^10, with every sum in FP32.  Rounding to
// bf16 instead costs 1% of the result's norm after five steps (every step
// multiplies small singular values, and the rounding error beside them, by
// a = 3.4); f16 costs 0.13%, below the result's own rounding to bf16, at the
// same MFMA rate.  2^10 keeps the entries (at most |X|_2, about 1.2) clear of
// f16's subnormals and leaves a factor of 50 before its largest value.
//
// Measured, five steps: four 4096 x 7168 matrices 7.0 ms, 1,220 TFLOP/s of the flops
// above (the library's f16 product reaches 1,520 at its best size): at the board's
// power limit, 1.7 GHz.  Eight 1408 x 2048: 0.82 ms, 730 TFLOP/s: 168 tiles of S on
// 256 CUs, and a fixed 7 to 10 us a round of tiles.  Three 777 x 515: 125 us, 17 launches
// of 7 us.
//
// X stays [N, K] as the caller has it: for N > K the products read it by
// columns (gemm16.h's column form), so nothing is transposed.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.h"
#include "gemm16.h"
#include "mxfp8_wgrad.h"

namespace {

using namespace mxw;

constexpr float kOne = 1024.0f;             // 1.0 as stored
constexpr float kPerOne = 1.0f / 1024.0f;   // a product of two stored values -> stored
constexpr int kNormParts = 256;
constexpr int kMaxSteps = 32;

// ---- the norm, and X0 -------------------------------------------------------

struct LoadArgs {
  const void* G;
  int64_t strideE, strideN;  // elements
  int N, K, ldx;
  int parts;
  double* sums;   // [E][parts]
  uint16_t* X;    // [E][N][ldx]
  float eps;
};

template <bool F32>
__device__ __forceinline__ float element(const void* G, int64_t i) {
  if (F32) return ((const float*)G)[i];
  return __uint_as_float((uint32_t)((const uint16_t*)G)[i] << 16);
}
// Elements i .. i + 7.  Rows of any stride start at any element: the 16-byte loads
// need no alignment beyond the element's.
template <bool F32>
__device__ __forceinline__ void load8(const void* G, int64_t i, float (&v)[8]) {
  if (F32) {
    __builtin_memcpy(v, (const float*)G + i, 32);
  } else {
    uint16_t u[8];
    __builtin_memcpy(u, (const uint16_t*)G + i, 16);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float((uint32_t)u[j] << 16);
  }
}
// Sum of squares, in 64 bits, of this thread's share of `rows` rows of K elements,
// row_stride apart from `at` on: whole eights first, four in flight, then the rest.
template <bool F32>
__device__ __forceinline__ double squares(const void* G, int64_t at, int64_t row_stride, int rows, int K, int threads) {
  const int per = K >> 3, rest = K & 7;
  double sum = 0.0;
#pragma unroll 4
  for (int i = threadIdx.x; i < rows * per; i += threads) {
    const int row = i / per;
    float v[8];
    load8<F32>(G, at + row * row_stride + 8 * (i - row * per), v);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += (double)v[j] * (double)v[j];
  }
  for (int i = threadIdx.x; i < rows * rest; i += threads) {
    const int row = i / rest;
    const double v = element<F32>(G, at + row * row_stride + 8 * per + (i - row * rest));
    sum += v * v;
  }
  return sum;
}

__device__ __forceinline__ double block_sum(double v, double* lds) {
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  return lds[0] + lds[1] + lds[2] + lds[3];
}

// kOne / (|G| + eps) as a power of two and a factor of about kOne: as one float it
// would overflow for norms below 3e-36.  A zero matrix with eps = 0 stays zero; a
// NaN or infinite sum makes the factor NaN or 0, and NaN of what is infinite.
struct Scale {
  int exponent;
  float factor;
  __device__ __forceinline__ Scale(double total, float eps) {
    const double d = sqrt(total) + (double)eps;
    const bool plain = d > 0.0 && d < INFINITY;
    exponent = plain ? -ilogb(d) : 0;
    factor = d == 0.0 ? 0.0f : (float)((double)kOne / ldexp(d, exponent));
  }
  __device__ __forceinline__ float operator()(float v) const { return ldexpf(v, exponent) * factor; }
};

// sums of squares of one part of an expert's rows, in 64 bits: squares of any
// bf16 or FP32 gradient are in range, and the order is fixed
template <bool F32>
__global__ __launch_bounds__(256) void ortho_norm_kernel(LoadArgs a) {
  __shared__ double lds[4];
  const int e = blockIdx.y, part = blockIdx.x;
  const int r0 = (int)((int64_t)a.N * part / a.parts), r1 = (int)((int64_t)a.N * (part + 1) / a.parts);
  const double sum =
      block_sum(squares<F32>(a.G, e * a.strideE + r0 * a.strideN, a.strideN, r1 - r0, a.K, 256), lds);
  if (threadIdx.x == 0) a.sums[e * a.parts + part] = sum;
}

// X0 with its zero padding, 8 columns a thread
template <bool F32>
__global__ __launch_bounds__(256) void ortho_load_kernel(LoadArgs a) {
  __shared__ double lds[4];
  const int e = blockIdx.y;
  const double total = block_sum((int)threadIdx.x < a.parts ? a.sums[e * a.parts + threadIdx.x] : 0.0, lds);
  const Scale scale(total, a.eps);
  const int per = a.ldx >> 3, whole = a.K >> 3;
  uint16_t* X = a.X + (int64_t)e * a.N * a.ldx;
  const int64_t stride = (int64_t)gridDim.x * 256;
#pragma unroll 4
  for (int64_t i = blockIdx.x * 256 + threadIdx.x; i < (int64_t)a.N * whole; i += stride) {
    const int row = (int)(i / whole), col = 8 * (int)(i % whole);
    float v[8];
    load8<F32>(a.G, e * a.strideE + row * a.strideN + col, v);
    v4i w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = (int)pack2(scale(v[2 * j]), scale(v[2 * j + 1]), _Float16());
    *(v4i*)(X + (int64_t)row * a.ldx + col) = w;
  }
  // the row's rest and padding
  const int left = per - whole;
  for (int64_t i = blockIdx.x * 256 + threadIdx.x; i < (int64_t)a.N * left * 8; i += stride) {
    const int row = (int)(i / (8 * left)), col = 8 * whole + (int)(i % (8 * left));
    const float v = col < a.K ? element<F32>(a.G, e * a.strideE + row * a.strideN + col) : 0.0f;
    X[(int64_t)row * a.ldx + col] = (uint16_t)pack2(scale(v), 0.0f, _Float16());
  }
}

// ---- small matrices: all steps in one kernel --------------------------------

// One workgroup a matrix, which stays in LDS for all steps: X [np][mp + 8] and S,
// then P in its place, [np][np + 8] (np, mp: n, m rounded up to 32; the 8 spread
// the rows over the banks).  A wave owns 32 x 32 blocks: of S and P up to two,
// kept in registers until everyone has read; of X whole columns of blocks, which
// P X needs and replaces alone, so X is updated in place.  The same roundings and,
// element by element, the same sums as the products below.  Bound by latency
// (barriers, LDS reads of short products), 5.7 us a step at 128 x 256; against the
// general way's launches (kernel time alone, in a graph): four such matrices 38 us
// against 67, eight of 64 x 64 12 against 54, of 128 x 400 56 against 71.
constexpr int kSmallN = 128;
constexpr int kSmallLds = 155 * 1024;

struct SmallArgs {
  LoadArgs in;
  int tall, n, m, mp;
  int steps;
  uint16_t* out;
  float coeffs[3 * kMaxSteps];
};

size_t small_lds(int n, int m) {
  const size_t np = (n + 31) & ~31, mp = (m + 31) & ~31;
  return 2 * (np * (mp + 8) + np * (np + 8));
}

__device__ __forceinline__ v4f mfma_h(const v4i& a, const v4i& b, const v4f& c) { return mfma16(a, b, c, _Float16()); }

template <bool F32, int NB>  // NB: np / 32
__global__ __launch_bounds__(512, 2) void ortho_small_kernel(SmallArgs a) {
  extern __shared__ __align__(16) uint16_t dyn[];
  __shared__ double red[8];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g = lane >> 4;
  constexpr int np = 32 * NB, lds = np + 8, kOwn = NB * NB > 8 ? 2 : 1;  // blocks of S a wave owns
  const int e = blockIdx.x, ldx = a.mp + 8;
  uint16_t* X = dyn;
  uint16_t* S = dyn + np * ldx;
  const int64_t base = e * a.in.strideE;
  const int N = a.in.N, K = a.in.K;

  // the norm, then X0
  double sum = squares<F32>(a.in.G, base, a.in.strideN, N, K, 512);
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if (lane == 0) red[wave] = sum;
  if (a.n < np || a.m < a.mp)
    for (int i = tid; i < (np * ldx) >> 3; i += 512) ((v4i*)X)[i] = (v4i){0, 0, 0, 0};
  __syncthreads();
  sum = 0.0;
  for (int w = 0; w < 8; ++w) sum += red[w];
  const Scale scale(sum, a.in.eps);
  auto put = [&](int row, int col, float v) {
    X[a.tall ? col * ldx + row : row * ldx + col] = (uint16_t)pack2(scale(v), 0.0f, _Float16());
  };
  const int per = K >> 3, rest = K & 7;
#pragma unroll 4
  for (int i = tid; i < N * per; i += 512) {
    const int row = i / per, col = 8 * (i - row * per);
    float v[8];
    load8<F32>(a.in.G, base + row * a.in.strideN + col, v);
    if (a.tall) {
#pragma unroll
      for (int j = 0; j < 8; ++j) put(row, col + j, v[j]);
    } else {
      v4i w;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = (int)pack2(scale(v[2 * j]), scale(v[2 * j + 1]), _Float16());
      *(v4i*)(X + row * ldx + col) = w;
    }
  }
  for (int i = tid; i < N * rest; i += 512) {
    const int row = i / rest, col = 8 * per + (i - row * rest);
    put(row, col, element<F32>(a.in.G, base + row * a.in.strideN + col));
  }
  __syncthreads();

  const int mb = a.mp >> 5;
  // lane's fragment of 16 rows from r0 on, columns k .. k + 31 of a matrix of row
  // stride ld; and the same of its transpose (rows are columns, k the row)
  auto rows = [&](const uint16_t* M, int ld, int r0, int k) { return *(const v4i*)(M + (r0 + r) * ld + k + 8 * g); };
  auto cols = [&](const uint16_t* M, int ld, int c0, int k) {
    const uint8_t* at = (const uint8_t*)(M + (k + 8 * g + (r >> 2)) * ld + c0 + 4 * (r & 3));
    const v2i lo = lds_read_tr(at), hi = lds_read_tr(at + 8 * ld);
    return (v4i){lo.x, lo.y, hi.x, hi.y};
  };
  // the wave's blocks of S; one without any does block 0 and does not write it
  int m0[kOwn], n0[kOwn];
  bool own[kOwn];
#pragma unroll
  for (int u = 0; u < kOwn; ++u) {
    const int id = wave * kOwn + u;
    own[u] = id < NB * NB;
    m0[u] = own[u] ? id / NB * 32 : 0;
    n0[u] = own[u] ? id % NB * 32 : 0;
  }
  typedef _Float16 v4h __attribute__((ext_vector_type(4)));
  for (int s = 0; s < a.steps; ++s) {
    const float ca = a.coeffs[3 * s], cb = a.coeffs[3 * s + 1], cc = a.coeffs[3 * s + 2];
    v4f acc[kOwn][2][2];
    auto block = [&](const uint16_t* M, int ld, int k) {
#pragma unroll
      for (int u = 0; u < kOwn; ++u) {
        const v4i f0 = rows(M, ld, m0[u], k), f1 = rows(M, ld, m0[u] + 16, k);
        const v4i h0 = rows(M, ld, n0[u], k), h1 = rows(M, ld, n0[u] + 16, k);
        acc[u][0][0] = mfma_h(h0, f0, acc[u][0][0]);
        acc[u][0][1] = mfma_h(h1, f0, acc[u][0][1]);
        acc[u][1][0] = mfma_h(h0, f1, acc[u][1][0]);
        acc[u][1][1] = mfma_h(h1, f1, acc[u][1][1]);
      }
    };
    auto each = [&](auto f) {
#pragma unroll
      for (int u = 0; u < kOwn; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (own[u]) f(acc[u][i][j], m0[u] + 16 * i + r, n0[u] + 16 * j + 4 * g);
    };
    auto clear = [&]() {
#pragma unroll
      for (int u = 0; u < kOwn; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[u][i >> 1][i & 1] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
    };
    // S = X X^T
    clear();
#pragma unroll 4
    for (int k = 0; k < a.mp; k += 32) block(X, ldx, k);
    each([&](v4f& v, int m, int n) {
      v *= kPerOne;
      *(uint2*)(S + m * lds + n) = make_uint2(pack2(v[0], v[1], _Float16()), pack2(v[2], v[3], _Float16()));
    });
    __syncthreads();
    // P = a I + b S + c S S, over S once everyone has read it
    clear();
#pragma unroll
    for (int k = 0; k < np; k += 32) block(S, lds, k);
    each([&](v4f& v, int m, int n) {
      const v4h was = *(const v4h*)(S + m * lds + n);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = cc * kPerOne * v[q] + cb * (float)was[q] + (m == n + q ? ca * kOne : 0.0f);
    });
    __syncthreads();
    each([&](v4f& v, int m, int n) {
      *(uint2*)(S + m * lds + n) = make_uint2(pack2(v[0], v[1], _Float16()), pack2(v[2], v[3], _Float16()));
    });
    __syncthreads();
    // X <- P X, 32 columns at a time; after the last step the result's bf16
    const bool last = s + 1 == a.steps;
    for (int c = wave; c < mb; c += 8) {
      v4f x[2 * NB][2] = {};
#pragma unroll
      for (int k = 0; k < np; k += 32) {
        const v4i h0 = cols(X, ldx, 32 * c, k), h1 = cols(X, ldx, 32 * c + 16, k);
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i) {
          const v4i f = rows(S, lds, 16 * i, k);
          x[i][0] = mfma_h(h0, f, x[i][0]);
          x[i][1] = mfma_h(h1, f, x[i][1]);
        }
      }
#pragma unroll
      for (int i = 0; i < 2 * NB; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const v4f v = x[i][j] * (last ? kPerOne * kPerOne : kPerOne);
          *(uint2*)(X + (16 * i + r) * ldx + 32 * c + 16 * j + 4 * g) =
              last ? make_uint2(pack2(v[0], v[1], __bf16()), pack2(v[2], v[3], __bf16()))
                   : make_uint2(pack2(v[0], v[1], _Float16()), pack2(v[2], v[3], _Float16()));
        }
    }
    __syncthreads();
  }
  // out, rows as the caller has them
  uint16_t* out = a.out + (int64_t)e * N * K;
  auto at = [&](int row, int col) { return X[a.tall ? col * ldx + row : row * ldx + col]; };
  for (int i = tid; i < N * per; i += 512) {
    const int row = i / per, col = 8 * (i - row * per);
    uint16_t u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = at(row, col + j);
    __builtin_memcpy(out + row * K + col, u, 16);
  }
  for (int i = tid; i < N * rest; i += 512) {
    const int row = i / rest, col = 8 * per + (i - row * rest);
    out[row * K + col] = at(row, col);
  }
}

// ---- the products -----------------------------------------------------------

// S: stored and mirrored
struct EpiGram {
  static constexpr bool kStaged = true;
  struct Args {
    uint16_t* S;
    int64_t stride;
    int n, ld;
  };
  template <int BM, int BN, int WM, int WN, int MI, int NI>
  static __device__ void run(const GemmArgs&, const Args& a, const TileAt& at, v4f (&acc)[MI][NI], uint8_t* lds) {
    stage_part<_Float16, BN>(at, acc, lds, [&](int, int, int, float (&v)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= kPerOne;
    });
    __syncthreads();
    uint16_t* S = a.S + at.batch * a.stride;
    store_rows<BM, BN, WM * WN>(at, lds, S, a.ld, a.n, a.ld);
    if (at.mirror) store_cols<BM, BN, WM * WN>(at, lds, S, a.ld, a.n, a.ld);
  }
};

// FP32 partial sums of S over one part of m
struct EpiPart {
  static constexpr bool kStaged = false;
  struct Args {
    float* part;  // [splits][batch][n][ld]
    int n, ld, batch;
  };
  template <int BM, int BN, int WM, int WN, int MI, int NI>
  static __device__ void run(const GemmArgs&, const Args& a, const TileAt& at, v4f (&acc)[MI][NI], uint8_t*) {
    float* part = a.part + ((int64_t)at.split * a.batch + at.batch) * a.n * a.ld;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const int m = at.m0 + at.wm + 16 * i + (at.lane & 15), n = at.n0 + at.wn + 16 * j + 4 * (at.lane >> 4);
        if (m < a.n && n < a.ld) *(v4f*)(part + (int64_t)m * a.ld + n) = acc[i][j];
      }
  }
};

// S from its partial sums, in order
__global__ __launch_bounds__(256) void ortho_join_kernel(const float* part, int splits, int64_t count, uint16_t* S) {
  const int64_t i = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  if (i >= count) return;
  v4f v = *(const v4f*)(part + i);
#pragma unroll 8
  for (int k = 1; k < splits; ++k) v += *(const v4f*)(part + k * count + i);
  v *= kPerOne;
  *(uint2*)(S + i) = make_uint2(pack2(v[0], v[1], _Float16()), pack2(v[2], v[3], _Float16()));
}

// P = a I + b S + c S S.  S's tile comes to where P's is staged, by whole rows (from
// the accumulators' layout, 32 bytes a row, a product took 4 us more: eight 1408 x
// 2048 783 -> 762 us); every lane replaces what it reads.
struct EpiPoly {
  static constexpr bool kStaged = true;
  struct Args {
    const uint16_t* S;
    uint16_t* P;
    int64_t stride;
    int n, ld;
    float a, b, c;
  };
  template <int BM, int BN, int WM, int WN, int MI, int NI>
  static __device__ void run(const GemmArgs&, const Args& a, const TileAt& at, v4f (&acc)[MI][NI], uint8_t* lds) {
    load_tile<BM, BN, WM * WN>(at, lds, a.S + at.batch * a.stride, a.ld, a.n);
    stage_barrier<0>();
    stage_part<_Float16, BN>(at, acc, lds, [&](int, int m, int n, float (&v)[4]) {
      typedef _Float16 v4h __attribute__((ext_vector_type(4)));
      const v4h s = *(const v4h*)(lds + staged_at<BN>(m - at.m0, n - at.n0));
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = a.c * kPerOne * v[e] + a.b * (float)s[e] + (m == n + e ? a.a * kOne : 0.0f);
    });
    __syncthreads();
    uint16_t* P = a.P + at.batch * a.stride;
    store_rows<BM, BN, WM * WN>(at, lds, P, a.ld, a.n, a.ld);
    if (at.mirror) store_cols<BM, BN, WM * WN>(at, lds, P, a.ld, a.n, a.ld);
  }
};

// X of the next step (f16, times 2^10), or the result (bf16, unpadded rows)
template <bool LAST>
struct EpiNext {
  static constexpr bool kStaged = true;
  struct Args {
    uint16_t* X;
    int64_t stride;
    int rows, cols, ld;
  };
  template <int BM, int BN, int WM, int WN, int MI, int NI>
  static __device__ void run(const GemmArgs&, const Args& a, const TileAt& at, v4f (&acc)[MI][NI], uint8_t* lds) {
    constexpr float kScale = LAST ? kPerOne * kPerOne : kPerOne;
    auto scale = [&](int, int, int, float (&v)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= kScale;
    };
    uint16_t* X = a.X + at.batch * a.stride;
    if constexpr (LAST) {
      stage_part<__bf16, BN>(at, acc, lds, scale);
      __syncthreads();
    } else {
      stage_part<_Float16, BN>(at, acc, lds, scale);
      __syncthreads();
    }
    store_rows<BM, BN, WM * WN>(at, lds, X, a.ld, a.rows, a.cols);
  }
};

// `count` tiles of edge B 2^cut from the `first` of all on, each cut into tiles of edge B
template <int B, int WM, int WN, int DEEP, bool TA, bool TB, bool SYM, class Epi>
void launch_tiles(GemmArgs g, const typename Epi::Args& e, int64_t first, int64_t count, int cut, hipStream_t st) {
  const int edge = B << cut;
  g.tilesM = (g.M + edge - 1) / edge;
  g.tilesN = (g.N + edge - 1) / edge;
  g.tiles = SYM ? g.tilesM * (g.tilesM + 1) / 2 : g.tilesM * g.tilesN;
  g.first = (int)first;
  g.cut = cut;
  const int64_t grid = count << (2 * cut);
  hipLaunchKernelGGL((gemm16_kernel<_Float16, B, B, WM, WN, DEEP, TA, TB, SYM, Epi>), dim3((unsigned)grid),
                     dim3(WM * WN * 64), 0, st, g, e);
}

// The tile edge with the least estimated time.  For P X of 1408 x 2048 matrices, us
// with 64, 128 and 256: four 63, 39, 39; 32 of them 486, 294, 251; S of three 777 x 515
// 7.8, 12.2, 24.7; of two 2560 x 2560 80, 44, 57.  Last, 256-tiles for the whole rounds
// and the rest cut into 128- or 64-tiles, which costs a launch more (S of four 4096 x
// 7168, 544 tiles: 368 us and 81 for the rest with 128, 58 with 64; the whole of six
// 3998 x 2200 2,241 and 2,104).
template <bool TA, bool TB, bool SYM, class Epi>
void launch_product(GemmArgs g, const typename Epi::Args& e, int cus, hipStream_t st) {
  auto tiles = [&](int b) {
    const int64_t tm = (g.M + b - 1) / b, tn = (g.N + b - 1) / b;
    return (SYM ? tm * (tm + 1) / 2 : tm * tn) * g.batch;
  };
  g.splits = 1;
  g.ksplit = (g.K + kGemmStep - 1) / kGemmStep * kGemmStep;
  const int64_t s = g.ksplit / kGemmStep, t256 = tiles(256), t128 = tiles(128), t64 = tiles(64);
  const int64_t whole = t256 / cus * cus, rest = t256 - whole;
  const int64_t c256 = tiles_cost<256, 256>(t256, s, cus), c128 = tiles_cost<128, 128>(t128, s, cus);
  const int64_t c64 = tiles_cost<64, 64>(t64, s, cus);
  const int64_t r128 = tiles_cost<128, 128>(4 * rest, s, cus), r64 = tiles_cost<64, 64>(16 * rest, s, cus);
  const int64_t both =
      whole && rest ? tiles_cost<256, 256>(whole, s, cus) + (r128 < r64 ? r128 : r64) + 500 : INT64_MAX;
  if (c64 <= c128 && c64 <= c256 && c64 <= both) return launch_tiles<64, 2, 2, 5, TA, TB, SYM, Epi>(g, e, 0, t64, 0, st);
  if (c128 <= c256 && c128 <= both) return launch_tiles<128, 2, 2, 0, TA, TB, SYM, Epi>(g, e, 0, t128, 0, st);
  if (c256 <= both) return launch_tiles<256, 2, 4, 0, TA, TB, SYM, Epi>(g, e, 0, t256, 0, st);
  launch_tiles<256, 2, 4, 0, TA, TB, SYM, Epi>(g, e, 0, whole, 0, st);
  if (r128 < r64) return launch_tiles<128, 2, 2, 0, TA, TB, SYM, Epi>(g, e, whole, rest, 1, st);
  launch_tiles<64, 2, 2, 5, TA, TB, SYM, Epi>(g, e, whole, rest, 2, st);
}

// ---- host -------------------------------------------------------------------

template <int NB>
void launch_small_of(bool f32, const SmallArgs& a, int E, unsigned bytes, hipStream_t st) {
  if (f32) hipLaunchKernelGGL((ortho_small_kernel<true, NB>), dim3((unsigned)E), dim3(512), bytes, st, a);
  else hipLaunchKernelGGL((ortho_small_kernel<false, NB>), dim3((unsigned)E), dim3(512), bytes, st, a);
}

void launch_small(bool f32, const SmallArgs& a, int E, unsigned bytes, hipStream_t st) {
  switch ((a.n + 31) >> 5) {
    case 1: return launch_small_of<1>(f32, a, E, bytes, st);
    case 2: return launch_small_of<2>(f32, a, E, bytes, st);
    case 3: return launch_small_of<3>(f32, a, E, bytes, st);
    default: return launch_small_of<4>(f32, a, E, bytes, st);
  }
}

struct OrthoPlan {
  int n, m, ldx, lds;
  bool tall;
  int parts;
  int splits;  // of m in S, 1: none
  size_t sums, X[2], S, P, part, bytes;
};

int round64(int v) { return (v + 63) & ~63; }

OrthoPlan plan_of(int E, int N, int K) {
  OrthoPlan p = {};
  p.tall = N > K;
  p.n = p.tall ? K : N;
  p.m = p.tall ? N : K;
  p.ldx = round64(K);
  p.lds = round64(p.n);
  int64_t parts = ((int64_t)N * K + 8191) / 8192;  // 4 chunks a thread, until there are many
  if (parts > kNormParts) parts = kNormParts;
  if (parts > N) parts = N;
  p.parts = (int)parts;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at = (at + bytes + 255) & ~(size_t)255;
    return was;
  };
  p.sums = take((size_t)E * p.parts * 8);
  for (int i = 0; i < 2; ++i) p.X[i] = take((size_t)E * N * p.ldx * 2);
  p.S = take((size_t)E * p.n * p.lds * 2);
  p.P = take((size_t)E * p.n * p.lds * 2);
  // A long m over few 64-tiles of S (counting both triangles: the halves' saving
  // is small there) is split so that about 512 workgroups (two for each of the whole
  // device's 256 CUs: the size query runs without one) take 4 steps of it or more;
  // joining costs a launch, about 10 steps.  Two 177 x 6597 matrices: 236 us without,
  // 138 with.  So a matrix's bits depend on E here.
  const int64_t tiles = (int64_t)((p.n + 63) / 64) * ((p.n + 63) / 64) * E, steps = (p.m + 63) / 64;
  p.splits = (int)(512 / tiles < steps / 4 ? 512 / tiles : steps / 4);
  if (p.splits < 2 || steps - steps / p.splits < 16) p.splits = 1;
  if (p.splits > 1) p.part = take((size_t)p.splits * E * p.n * p.lds * 4);
  p.bytes = at;
  return p;
}

int check_sizes(int E, int N, int K) {
  if (E < 1 || E > MXW_MAX_EXPERTS || N < 1 || K < 1 || N > 65536 || K > 65536) return MXW_ERR_DIM;
  // launches of 64-tiles stay below 2^32 threads
  return (int64_t)E * ((N + 255) / 256) * ((K + 255) / 256) > (1 << 20) ? MXW_ERR_DIM : MXW_OK;
}

}  // namespace

extern "C" {

int64_t mxw_orthogonalize_workspace_size(int E, int N, int K) {
  if (check_sizes(E, N, K)) return MXW_ERR_DIM;
  return (int64_t)plan_of(E, N, K).bytes;
}

int mxw_orthogonalize(const void* G, int type, int64_t expert_stride, int64_t row_stride, int E, int N, int K,
                      const float* coeffs, int steps, float eps, uint16_t* out, void* workspace,
                      size_t workspace_bytes, void* stream) {
  if (!G || !coeffs || !out) return MXW_ERR_NULL;
  if (check_sizes(E, N, K) || (type != MXW_BF16 && type != MXW_F32) || steps < 1 || steps > kMaxSteps ||
      row_stride < K || expert_stride < 0 || !(eps >= 0.0f))
    return MXW_ERR_DIM;
  if (((uintptr_t)G & (type == MXW_F32 ? 3 : 1)) || ((uintptr_t)out & 1)) return MXW_ERR_ALIGN;
  const OrthoPlan p = plan_of(E, N, K);
  if (!workspace || workspace_bytes < p.bytes || ((uintptr_t)workspace & 255)) return MXW_ERR_WORKSPACE;
  int cus = 0;
  int rc = check_device(&cus);
  if (rc) return rc;
  hipStream_t st = (hipStream_t)stream;
  uint8_t* ws = (uint8_t*)workspace;

  LoadArgs la = {};
  la.G = G;
  la.strideE = expert_stride;
  la.strideN = row_stride;
  la.N = N;
  la.K = K;
  la.ldx = p.ldx;
  la.parts = p.parts;
  la.sums = (double*)(ws + p.sums);
  la.X = (uint16_t*)(ws + p.X[0]);
  la.eps = eps;
  const bool f32 = type == MXW_F32;
  if (p.n <= kSmallN && small_lds(p.n, p.m) <= kSmallLds) {
    SmallArgs sa = {};
    sa.in = la;
    sa.tall = p.tall;
    sa.n = p.n;
    sa.m = p.m;
    sa.mp = (p.m + 31) & ~31;
    sa.steps = steps;
    sa.out = out;
    for (int i = 0; i < 3 * steps; ++i) sa.coeffs[i] = coeffs[i];
    const unsigned bytes = (unsigned)small_lds(p.n, p.m);
    launch_small(f32, sa, E, bytes, st);
    return hipGetLastError() == hipSuccess ? MXW_OK : MXW_ERR_LAUNCH;
  }
  int64_t blocks = ((int64_t)N * (p.ldx / 8) + 1023) / 1024;  // about 4 chunks a thread
  if (blocks > 4096) blocks = 4096;
  const dim3 ng((unsigned)p.parts, (unsigned)E), lg((unsigned)blocks, (unsigned)E);
  if (f32) {
    hipLaunchKernelGGL((ortho_norm_kernel<true>), ng, dim3(256), 0, st, la);
    hipLaunchKernelGGL((ortho_load_kernel<true>), lg, dim3(256), 0, st, la);
  } else {
    hipLaunchKernelGGL((ortho_norm_kernel<false>), ng, dim3(256), 0, st, la);
    hipLaunchKernelGGL((ortho_load_kernel<false>), lg, dim3(256), 0, st, la);
  }

  const int64_t strideX = (int64_t)N * p.ldx, strideS = (int64_t)p.n * p.lds;
  uint16_t* S = (uint16_t*)(ws + p.S);
  uint16_t* P = (uint16_t*)(ws + p.P);
  for (int s = 0; s < steps; ++s) {
    const float a = coeffs[3 * s], b = coeffs[3 * s + 1], c = coeffs[3 * s + 2];
    const uint16_t* X = (const uint16_t*)(ws + p.X[s & 1]);
    uint16_t* next = (uint16_t*)(ws + p.X[(s + 1) & 1]);
    GemmArgs g = {};
    g.batch = E;
    // S
    g.A = g.B = X;
    g.strideA = g.strideB = strideX;
    g.lda = g.ldb = p.ldx;
    g.M = g.N = p.tall ? p.ldx : N;  // whole chunks by columns; their padding is zeros
    g.K = p.m;
    const EpiGram::Args eg = {S, strideS, p.n, p.lds};
    if (p.splits > 1) {
      float* part = (float*)(ws + p.part);
      const EpiPart::Args es = {part, p.n, p.lds, E};
      g.splits = p.splits;
      g.ksplit = ((p.m + kGemmStep - 1) / kGemmStep + p.splits - 1) / p.splits * kGemmStep;
      const int64_t edge = (p.n + 63) / 64, count = (int64_t)E * strideS;
      p.tall ? launch_tiles<64, 2, 2, 5, true, true, false, EpiPart>(g, es, 0, edge * edge * E * p.splits, 0, st)
                  : launch_tiles<64, 2, 2, 5, false, false, false, EpiPart>(g, es, 0, edge * edge * E * p.splits, 0, st);
      hipLaunchKernelGGL(ortho_join_kernel, dim3((unsigned)((count / 4 + 255) / 256)), dim3(256), 0, st,
                         (const float*)part, p.splits, count, S);
    } else {
      p.tall ? launch_product<true, true, true, EpiGram>(g, eg, cus, st)
             : launch_product<false, false, true, EpiGram>(g, eg, cus, st);
    }
    // P
    g.A = g.B = S;
    g.strideA = g.strideB = strideS;
    g.lda = g.ldb = p.lds;
    g.M = g.N = p.n;
    g.K = p.n;
    const EpiPoly::Args ep = {S, P, strideS, p.n, p.lds, a, b, c};
    launch_product<false, false, true, EpiPoly>(g, ep, cus, st);
    // X
    g.M = N;
    g.N = p.ldx;
    g.K = p.n;
    if (p.tall) {
      g.A = X;
      g.strideA = strideX;
      g.lda = p.ldx;
      g.B = P;
      g.strideB = strideS;
      g.ldb = p.lds;
      g.N = p.n;
    } else {
      g.A = P;
      g.strideA = strideS;
      g.lda = p.lds;
      g.B = X;
      g.strideB = strideX;
      g.ldb = p.ldx;
    }
    if (s + 1 < steps) {
      const EpiNext<false>::Args en = {next, strideX, N, p.ldx, p.ldx};
      p.tall ? launch_product<false, false, false, EpiNext<false>>(g, en, cus, st)
             : launch_product<false, true, false, EpiNext<false>>(g, en, cus, st);
    } else {
      const EpiNext<true>::Args en = {out, (int64_t)N * K, N, K, K};
      p.tall ? launch_product<false, false, false, EpiNext<true>>(g, en, cus, st)
             : launch_product<false, true, false, EpiNext<true>>(g, en, cus, st);
    }
  }
  if (hipGetLastError() != hipSuccess) return MXW_ERR_LAUNCH;
  return MXW_OK;
}

}  // extern "C"
