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

// elements i .. i + 7 of G, zeros from the `left`-th on.  Rows of any stride start
// at any element: the 16-byte loads need no alignment beyond the element's.
template <bool F32>
__device__ __forceinline__ void load8(const void* G, int64_t i, int left, float (&v)[8]) {
  if (F32) {
    const float* p = (const float*)G + i;
    if (left >= 8) {
      __builtin_memcpy(v, p, 32);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = j < left ? p[j] : 0.0f;
    }
  } else {
    const uint16_t* p = (const uint16_t*)G + i;
    uint16_t u[8];
    if (left >= 8) {
      __builtin_memcpy(u, p, 16);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = j < left ? p[j] : 0;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float((uint32_t)u[j] << 16);
  }
}

__device__ __forceinline__ double block_sum(double v, double* lds) {
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  return lds[0] + lds[1] + lds[2] + lds[3];
}

// sums of squares of one part of an expert's rows, in 64 bits: squares of any
// bf16 or FP32 gradient are in range, and the order is fixed
template <bool F32>
__global__ __launch_bounds__(256) void ortho_norm_kernel(LoadArgs a) {
  __shared__ double lds[4];
  const int e = blockIdx.y, part = blockIdx.x, per = (a.K + 7) >> 3;
  const int r0 = (int)((int64_t)a.N * part / a.parts), r1 = (int)((int64_t)a.N * (part + 1) / a.parts);
  const int count = (r1 - r0) * per;
  double sum = 0.0;
#pragma unroll 4
  for (int i = threadIdx.x; i < count; i += 256) {
    const int row = i / per, col = 8 * (i - row * per);
    float v[8];
    load8<F32>(a.G, e * a.strideE + (r0 + row) * a.strideN + col, a.K - col, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += (double)v[j] * (double)v[j];
  }
  sum = block_sum(sum, lds);
  if (threadIdx.x == 0) a.sums[e * a.parts + part] = sum;
}

// X0 with its zero padding, 8 columns a thread
template <bool F32>
__global__ __launch_bounds__(256) void ortho_load_kernel(LoadArgs a) {
  __shared__ double lds[4];
  const int e = blockIdx.y;
  const double total = block_sum((int)threadIdx.x < a.parts ? a.sums[e * a.parts + threadIdx.x] : 0.0, lds);
  const float scale = (float)(kOne / (sqrt(total) + (double)a.eps));
  const int per = a.ldx >> 3;
  const int64_t count = (int64_t)a.N * per;
#pragma unroll 4
  for (int64_t i = blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256) {
    const int row = (int)(i / per), col = 8 * (int)(i % per);
    float v[8];
    load8<F32>(a.G, e * a.strideE + row * a.strideN + col, a.K - col, v);
    v4i w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = (int)pack2(v[2 * j] * scale, v[2 * j + 1] * scale, _Float16());
    *(v4i*)(a.X + ((int64_t)e * a.N + row) * a.ldx + col) = w;
  }
}

// ---- small matrices: all steps in one kernel --------------------------------

// One workgroup a matrix, which stays in LDS for all steps: X [np][mp + 8] and S,
// then P in its place, [np][np + 8] (np, mp: n, m rounded up to 32; the 8 spread
// the rows over the banks).  A wave owns 32 x 32 blocks: of S and P up to two,
// kept in registers until everyone has read; of X whole columns of blocks, which
// P X needs and replaces alone, so X is updated in place.  The same roundings and,
// element by element, the same sums as the products below.  Bound by latency
// (barriers, LDS); against the launches of the general way: 128 x 256, four
// matrices, 96 us to 27 us.
constexpr int kSmallN = 128;
constexpr int kSmallLds = 155 * 1024;

struct SmallArgs {
  LoadArgs in;
  int tall, n, m, np, mp;
  int steps;
  uint16_t* out;
  float coeffs[3 * kMaxSteps];
};

size_t small_lds(int n, int m) {
  const size_t np = (n + 31) & ~31, mp = (m + 31) & ~31;
  return 2 * (np * (mp + 8) + np * (np + 8));
}

__device__ __forceinline__ v4f mfma_h(const v4i& a, const v4i& b, const v4f& c) { return mfma16(a, b, c, _Float16()); }

template <bool F32>
__global__ __launch_bounds__(512, 2) void ortho_small_kernel(SmallArgs a) {
  extern __shared__ __align__(16) uint16_t dyn[];
  __shared__ double red[8];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g = lane >> 4;
  const int e = blockIdx.x, ldx = a.mp + 8, lds = a.np + 8;
  uint16_t* X = dyn;
  uint16_t* S = dyn + a.np * ldx;
  const int64_t base = e * a.in.strideE;
  const int N = a.in.N, K = a.in.K;

  // the norm, summed in 64 bits in a fixed order, then X0
  const int per = (K + 7) >> 3, chunks = N * per;
  double sum = 0.0;
#pragma unroll 4
  for (int i = tid; i < chunks; i += 512) {
    const int row = i / per, col = 8 * (i - row * per);
    float v[8];
    load8<F32>(a.in.G, base + row * a.in.strideN + col, K - col, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += (double)v[j] * (double)v[j];
  }
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if (lane == 0) red[wave] = sum;
  for (int i = tid; i < (a.np * (ldx + lds)) >> 3; i += 512) ((v4i*)dyn)[i] = (v4i){0, 0, 0, 0};
  __syncthreads();
  sum = 0.0;
  for (int w = 0; w < 8; ++w) sum += red[w];
  const float scale = (float)(kOne / (sqrt(sum) + (double)a.in.eps));
#pragma unroll 4
  for (int i = tid; i < chunks; i += 512) {
    const int row = i / per, col = 8 * (i - row * per);
    float v[8];
    load8<F32>(a.in.G, base + row * a.in.strideN + col, K - col, v);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col + j < K)
        X[a.tall ? (col + j) * ldx + row : row * ldx + col + j] = (uint16_t)pack2(v[j] * scale, 0.0f, _Float16());
  }
  __syncthreads();

  const int nb = a.np >> 5, mb = a.mp >> 5;
  // lane's fragment of 16 rows from r0 on, columns k .. k + 31 of a matrix of row
  // stride ld; and the same of its transpose (rows are columns, k the row)
  auto rows = [&](const uint16_t* M, int ld, int r0, int k) { return *(const v4i*)(M + (r0 + r) * ld + k + 8 * g); };
  auto cols = [&](const uint16_t* M, int ld, int c0, int k) {
    const uint8_t* at = (const uint8_t*)(M + (k + 8 * g + (r >> 2)) * ld + c0 + 4 * (r & 3));
    const v2i lo = lds_read_tr(at), hi = lds_read_tr(at + 8 * ld);
    return (v4i){lo.x, lo.y, hi.x, hi.y};
  };
  for (int s = 0; s < a.steps; ++s) {
    const float ca = a.coeffs[3 * s], cb = a.coeffs[3 * s + 1], cc = a.coeffs[3 * s + 2];
    // S = X X^T, then P = a I + b S + c S S over it: blocks wave, wave + 8
    for (int pass = 0; pass < 2; ++pass) {
      v4f acc[2][2][2] = {};
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int id = wave + 8 * u;
        if (id >= nb * nb) continue;
        const int m0 = id / nb * 32, n0 = id % nb * 32;
        const uint16_t* M = pass ? S : X;
        const int ld = pass ? lds : ldx, depth = pass ? a.np : a.mp;
#pragma unroll 2
        for (int k = 0; k < depth; k += 32) {
          const v4i f0 = rows(M, ld, m0, k), f1 = rows(M, ld, m0 + 16, k);
          const v4i h0 = rows(M, ld, n0, k), h1 = rows(M, ld, n0 + 16, k);
          acc[u][0][0] = mfma_h(h0, f0, acc[u][0][0]);
          acc[u][0][1] = mfma_h(h1, f0, acc[u][0][1]);
          acc[u][1][0] = mfma_h(h0, f1, acc[u][1][0]);
          acc[u][1][1] = mfma_h(h1, f1, acc[u][1][1]);
        }
      }
      if (pass) __syncthreads();  // S has been read
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int id = wave + 8 * u;
        if (id >= nb * nb) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int m = id / nb * 32 + 16 * i + r, n = id % nb * 32 + 16 * j + 4 * g;
            typedef _Float16 v4h __attribute__((ext_vector_type(4)));
            v4h* to = (v4h*)(S + m * lds + n);
            float v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              v[q] = kPerOne * acc[u][i][j][q];
              if (pass) v[q] = cc * v[q] + cb * (float)(*to)[q] + (m == n + q ? ca * kOne : 0.0f);
            }
            *(uint2*)to = make_uint2(pack2(v[0], v[1], _Float16()), pack2(v[2], v[3], _Float16()));
          }
      }
      __syncthreads();
    }
    // X <- P X, 32 columns at a time
    for (int c = wave; c < mb; c += 8) {
      v4f acc[kSmallN / 16][2] = {};
      for (int k = 0; k < a.np; k += 32) {
        const v4i h0 = cols(X, ldx, 32 * c, k), h1 = cols(X, ldx, 32 * c + 16, k);
#pragma unroll
        for (int i = 0; i < kSmallN / 16; ++i) {
          if (16 * i >= a.np) break;
          const v4i f = rows(S, lds, 16 * i, k);
          acc[i][0] = mfma_h(h0, f, acc[i][0]);
          acc[i][1] = mfma_h(h1, f, acc[i][1]);
        }
      }
#pragma unroll
      for (int i = 0; i < kSmallN / 16; ++i) {
        if (16 * i >= a.np) break;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int m = 16 * i + r, n = 32 * c + 16 * j + 4 * g;
          if (s + 1 < a.steps) {
            const v4f v = acc[i][j] * kPerOne;
            *(uint2*)(X + m * ldx + n) = make_uint2(pack2(v[0], v[1], _Float16()), pack2(v[2], v[3], _Float16()));
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (m < a.n && n + q < a.m)
                a.out[(int64_t)e * N * K + (a.tall ? (int64_t)(n + q) * K + m : (int64_t)m * K + n + q)] =
                    (uint16_t)pack2(acc[i][j][q] * (kPerOne * kPerOne), 0.0f, __bf16());
          }
        }
      }
    }
    __syncthreads();
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
  if (p.n <= kSmallN && small_lds(p.n, p.m) <= kSmallLds) {
    SmallArgs sa = {};
    sa.in = la;
    sa.tall = p.tall;
    sa.n = p.n;
    sa.m = p.m;
    sa.np = (p.n + 31) & ~31;
    sa.mp = (p.m + 31) & ~31;
    sa.steps = steps;
    sa.out = out;
    for (int i = 0; i < 3 * steps; ++i) sa.coeffs[i] = coeffs[i];
    const unsigned bytes = (unsigned)small_lds(p.n, p.m);
    if (f32) hipLaunchKernelGGL((ortho_small_kernel<true>), dim3((unsigned)E), dim3(512), bytes, st, sa);
    else hipLaunchKernelGGL((ortho_small_kernel<false>), dim3((unsigned)E), dim3(512), bytes, st, sa);
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
