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

__device__ __forceinline__ double block_sum(double v, double* lds) {
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  return lds[0] + lds[1] + lds[2] + lds[3];
}

// sums of squares of one part of an expert's rows, in 64 bits: squares of any
// bf16 or FP32 gradient are in range, and the order is fixed
template <bool F32, bool VEC>
__global__ __launch_bounds__(256) void ortho_norm_kernel(LoadArgs a) {
  __shared__ double lds[4];
  const int e = blockIdx.y, part = blockIdx.x;
  const int r0 = (int)((int64_t)a.N * part / a.parts), r1 = (int)((int64_t)a.N * (part + 1) / a.parts);
  double sum = 0.0;
  if (VEC) {  // 8 elements a thread
    const int per = a.K >> 3;
    const int64_t count = (int64_t)(r1 - r0) * per;
    for (int64_t i = threadIdx.x; i < count; i += 256) {
      const int64_t at = e * a.strideE + (r0 + i / per) * a.strideN + 8 * (i % per);
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = element<F32>(a.G, at + j);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += (double)v[j] * (double)v[j];
    }
  } else {
    const int64_t count = (int64_t)(r1 - r0) * a.K;
    for (int64_t i = threadIdx.x; i < count; i += 256) {
      const double v = element<F32>(a.G, e * a.strideE + (r0 + i / a.K) * a.strideN + i % a.K);
      sum += v * v;
    }
  }
  sum = block_sum(sum, lds);
  if (threadIdx.x == 0) a.sums[e * a.parts + part] = sum;
}

// X0 with its zero padding, 8 columns a thread
template <bool F32, bool VEC>
__global__ __launch_bounds__(256) void ortho_load_kernel(LoadArgs a) {
  __shared__ double lds[4];
  const int e = blockIdx.y;
  const double total = block_sum((int)threadIdx.x < a.parts ? a.sums[e * a.parts + threadIdx.x] : 0.0, lds);
  const float scale = (float)(kOne / (sqrt(total) + (double)a.eps));
  const int per = a.ldx >> 3;
  const int64_t count = (int64_t)a.N * per;
  for (int64_t i = blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256) {
    const int row = (int)(i / per), col = 8 * (int)(i % per);
    const int64_t at = e * a.strideE + row * a.strideN + col;
    float v[8];
    if (VEC) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.0f;
      if (col < a.K) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = element<F32>(a.G, at + j);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = col + j < a.K ? element<F32>(a.G, at + j) : 0.0f;
    }
    v4i w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = (int)pack2(v[2 * j] * scale, v[2 * j + 1] * scale, _Float16());
    *(v4i*)(a.X + ((int64_t)e * a.N + row) * a.ldx + col) = w;
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

// P = a I + b S + c S S
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
    const uint16_t* S = a.S + at.batch * a.stride;
    stage_part<_Float16, BN>(at, acc, lds, [&](int, int m, int n, float (&v)[4]) {
      typedef _Float16 v4h __attribute__((ext_vector_type(4)));
      v4h s = {};
      if (m < a.n && n < a.ld) s = *(const v4h*)(S + (int64_t)m * a.ld + n);
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
      if ((a.ld & 7) == 0 && ((uintptr_t)a.X & 15) == 0)
        store_rows<BM, BN, WM * WN>(at, lds, X, a.ld, a.rows, a.cols);
      else
        store_rows_any<BM, BN, WM * WN>(at, lds, X, a.ld, a.rows, a.cols);
    } else {
      stage_part<_Float16, BN>(at, acc, lds, scale);
      __syncthreads();
      store_rows<BM, BN, WM * WN>(at, lds, X, a.ld, a.rows, a.cols);
    }
  }
};

template <int B, int WM, int WN, bool TA, bool TB, bool SYM, class Epi>
int launch_tiles(GemmArgs g, const typename Epi::Args& e, hipStream_t st) {
  g.tilesM = (g.M + B - 1) / B;
  g.tilesN = (g.N + B - 1) / B;
  g.tiles = SYM ? g.tilesM * (g.tilesM + 1) / 2 : g.tilesM * g.tilesN;
  const int64_t grid = (int64_t)g.tiles * g.batch;
  if (grid > 0x7FFFFFFF / 512) return MXW_ERR_DIM;
  hipLaunchKernelGGL((gemm16_kernel<_Float16, B, B, WM, WN, TA, TB, SYM, Epi>), dim3((unsigned)grid),
                     dim3(WM * WN * 64), 0, st, g, e);
  return MXW_OK;
}

template <bool TA, bool TB, bool SYM, class Epi>
int launch_product(GemmArgs g, const typename Epi::Args& e, int cus, hipStream_t st) {
  auto tiles = [&](int b) {
    const int64_t tm = (g.M + b - 1) / b, tn = (g.N + b - 1) / b;
    return (SYM ? tm * (tm + 1) / 2 : tm * tn) * g.batch;
  };
  g.splits = 1;
  g.ksplit = (g.K + kGemmStep - 1) / kGemmStep * kGemmStep;
  const int64_t big = (tiles(256) + cus - 1) / cus * 10, small = (tiles(128) + 2 * cus - 1) / (2 * cus) * 7;
  if (big <= small) return launch_tiles<256, 2, 4, TA, TB, SYM, Epi>(g, e, st);
  return launch_tiles<128, 2, 2, TA, TB, SYM, Epi>(g, e, st);
}

// ---- host -------------------------------------------------------------------

struct OrthoPlan {
  int n, m, ldx, lds;
  bool tall;
  int parts;
  size_t sums, X[2], S, P, bytes;
};

int round64(int v) { return (v + 63) & ~63; }

OrthoPlan plan_of(int E, int N, int K) {
  OrthoPlan p = {};
  p.tall = N > K;
  p.n = p.tall ? K : N;
  p.m = p.tall ? N : K;
  p.ldx = round64(K);
  p.lds = round64(p.n);
  int64_t parts = ((int64_t)N * K + 16383) / 16384;
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
  p.bytes = at;
  return p;
}

int check_sizes(int E, int N, int K) {
  return E < 1 || E > MXW_MAX_EXPERTS || N < 1 || K < 1 || N > 65536 || K > 65536 ? MXW_ERR_DIM : MXW_OK;
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
  // 8 elements at a time where rows keep them together and aligned
  const bool vec = (K & 7) == 0 && (row_stride & 7) == 0 && (expert_stride & 7) == 0 && ((uintptr_t)G & 15) == 0;
  int64_t blocks = ((int64_t)N * (p.ldx / 8) + 1023) / 1024;  // about 4 chunks a thread
  if (blocks > 4096) blocks = 4096;
  const dim3 ng((unsigned)p.parts, (unsigned)E), lg((unsigned)blocks, (unsigned)E);
  if (f32 && vec) {
    hipLaunchKernelGGL((ortho_norm_kernel<true, true>), ng, dim3(256), 0, st, la);
    hipLaunchKernelGGL((ortho_load_kernel<true, true>), lg, dim3(256), 0, st, la);
  } else if (f32) {
    hipLaunchKernelGGL((ortho_norm_kernel<true, false>), ng, dim3(256), 0, st, la);
    hipLaunchKernelGGL((ortho_load_kernel<true, false>), lg, dim3(256), 0, st, la);
  } else if (vec) {
    hipLaunchKernelGGL((ortho_norm_kernel<false, true>), ng, dim3(256), 0, st, la);
    hipLaunchKernelGGL((ortho_load_kernel<false, true>), lg, dim3(256), 0, st, la);
  } else {
    hipLaunchKernelGGL((ortho_norm_kernel<false, false>), ng, dim3(256), 0, st, la);
    hipLaunchKernelGGL((ortho_load_kernel<false, false>), lg, dim3(256), 0, st, la);
  }

  const int64_t strideX = (int64_t)N * p.ldx, strideS = (int64_t)p.n * p.lds;
  uint16_t* S = (uint16_t*)(ws + p.S);
  uint16_t* P = (uint16_t*)(ws + p.P);
  for (int s = 0; s < steps && rc == MXW_OK; ++s) {
    const float a = coeffs[3 * s], b = coeffs[3 * s + 1], c = coeffs[3 * s + 2];
    const uint16_t* X = (const uint16_t*)(ws + p.X[s & 1]);
    uint16_t* next = (uint16_t*)(ws + p.X[(s + 1) & 1]);
    GemmArgs g = {};
    g.batch = E;
    // S
    g.A = g.B = X;
    g.strideA = g.strideB = strideX;
    g.lda = g.ldb = p.ldx;
    g.M = g.N = p.tall ? p.ldx : N;
    g.K = p.m;
    const EpiGram::Args eg = {S, strideS, p.n, p.lds};
    rc = p.tall ? launch_product<true, true, true, EpiGram>(g, eg, cus, st)
                : launch_product<false, false, true, EpiGram>(g, eg, cus, st);
    if (rc) break;
    // P
    g.A = g.B = S;
    g.strideA = g.strideB = strideS;
    g.lda = g.ldb = p.lds;
    g.M = g.N = p.n;
    g.K = p.n;
    const EpiPoly::Args ep = {S, P, strideS, p.n, p.lds, a, b, c};
    rc = launch_product<false, false, true, EpiPoly>(g, ep, cus, st);
    if (rc) break;
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
      rc = p.tall ? launch_product<false, false, false, EpiNext<false>>(g, en, cus, st)
                  : launch_product<false, true, false, EpiNext<false>>(g, en, cus, st);
    } else {
      const EpiNext<true>::Args en = {out, (int64_t)N * K, N, K, K};
      rc = p.tall ? launch_product<false, false, false, EpiNext<true>>(g, en, cus, st)
                  : launch_product<false, true, false, EpiNext<true>>(g, en, cus, st);
    }
  }
  if (rc) return rc;
  if (hipGetLastError() != hipSuccess) return MXW_ERR_LAUNCH;
  return MXW_OK;
}

}  // extern "C"
