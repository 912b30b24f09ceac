// vocab_loss.hip -- softmax cross entropy over a large vocabulary with its
// gradients, in bounded memory (mxw_vocab_loss, declared in
// include/mxfp8_wgrad.h), for gfx950.
//
//     l = x w^T,  lse_t = log sum_v exp l_tv,  loss_t = lse_t - l_t,y(t)
//     g_tv = (exp(l_tv - lse_t) - [v = y(t)]) s,  dx = g w,  dw = g^T x
//
// with s = grad_scale (divided by the number of tokens that count, for the
// mean); tokens whose target is ignore_index have loss 0 and g = 0.
//
// A first product walks the whole vocabulary and leaves, per tile and token, the
// maximum and sum of exponentials of the tile's 256 (narrow tiles: 64) logits, 8 bytes
// for them; they are joined in a fixed order.  It also leaves the logits (FP32) if
// gradients are wanted and they take at most 4 GiB.  Then the vocabulary is walked in
// pieces, each small enough that g of the piece (bf16, unscaled: its entries lie in
// [-1, 1]) stays in the memory-side cache: g comes from the kept logits, or else a
// product makes them again and turns them into g in its epilogue (the same bits);
// one product adds g w to the FP32 sums of dx (split over the piece's vocabulary where
// T x H has few tiles; partial sums are joined in a fixed order at the end), one
// writes dw = g^T x of the piece's rows.
// 6 T H V flops with gradients (8 without room for the logits), 2 T H V without:
// bound by the MFMA except for few tokens, where reading w (twice with gradients)
// bounds it.
//
// Measured: 4,096 tokens, 128,000 words of 2,048: 5.6 ms, 1,150 TFLOP/s; 2,048 tokens,
// words of 7,168: 8.7 ms, 1,290; one token's loss against 32,000 words of 2,048 with
// cold caches: 31 us, 4.2 TB/s.
//
// All sums and statistics are FP32 (the mean's over tokens FP64); g is rounded
// to bf16 because the products that follow take 16-bit operands: at most
// 2^-8 of each term, about the gradients' own rounding to bf16.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.h"
#include "gemm16.h"
#include "mxfp8_wgrad.h"

namespace {

using namespace mxw;

// g of one piece: 4,096 tokens, 128,000 words of 2,048 take 6.83 ms with 64 MiB, 6.65
// with 128 or 256, 6.59 with 512, 6.64 with 1,024
constexpr int64_t kPieceBytes = 256LL << 20;
// The logits kept for g at most (of 288 GB): 4,096 tokens, 128,000 words of 2,048 5.83 ms
// against 6.74 with the logits made again, 2,048 tokens of 7,168 8.84 and 11.04, 32
// tokens 1.26 and 1.56.  Words of fewer than 1,024 values make them again in less time
// than a copy out of the caches takes: 2,048 tokens, 32,000 words of 256 291 us kept,
// 224 made again; 905 tokens, 4,629 of 896 (17 MB) 82 and 88.
constexpr int64_t kKeepBytes = 4LL << 30, kKeepShort = 64LL << 20;
// the padded copy of a piece's weights: one piece is copied once, more are copied for
// either pass (61 tokens, 49,036 words of 4,106: 140 us of 912)
constexpr int64_t kCopyBytes = 2LL << 30;
constexpr int kMaxTokens = 128 * 1024;
constexpr int kMaxVocab = 1 << 20;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Targets {
  const void* p;
  int wide;        // 64-bit
  int64_t ignore;
  int V;
  // the target's index, -1: ignored, -2: outside the vocabulary
  __device__ int at(int t) const {
    const int64_t y = wide ? ((const int64_t*)p)[t] : (int64_t)((const int32_t*)p)[t];
    return y == ignore ? -1 : (y < 0 || y >= V ? -2 : (int)y);
  }
};

// exp(l - m) with exp(-inf - m) = 0 for every m, NaN kept
__device__ __forceinline__ float exp_above(float l, float m) {
  return l == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((l - m) * kLog2e);
}
// (m, s) joined with (m2, s2)
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float top = fmaxf(m, m2);
  // a side without anything (m = -inf, s = 0, or a NaN sum) is kept as it is
  const float f = m == -INFINITY ? s : s * __builtin_amdgcn_exp2f((m - top) * kLog2e);
  const float f2 = m2 == -INFINITY ? s2 : s2 * __builtin_amdgcn_exp2f((m2 - top) * kLog2e);
  m = top;
  s = f + f2;
}

// ---- the logits' statistics -------------------------------------------------

// KEEP: the logits are written as well
template <bool KEEP>
struct EpiStats {
  static constexpr bool kStaged = false;
  struct Args {
    float2* part;      // [tiles of the vocabulary][T]
    float* hit;        // [T] the target's logit
    Targets y;
    int v0, V;         // the piece's first column; columns in all
    float* logits;     // KEEP: [T][ld], ld at least V rounded up to 4
    int ld;
  };
  template <int BM, int BN, int WM, int WN, int MI, int NI>
  static __device__ void run(const GemmArgs& p, const Args& a, const TileAt& at, v4f (&acc)[MI][NI], uint8_t* lds) {
    float2(*sh)[BM] = (float2(*)[BM])lds;  // [WN][BM]
    // columns of the wave's part from this lane's first on, and how many of
    // them the vocabulary has
    const int c0 = a.v0 + at.n0 + at.wn + 4 * (at.lane >> 4), left = a.V - c0;
    if (a.v0 + at.n0 + BN > a.V) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[i][j][q] = 16 * j + q < left ? acc[i][j][q] : -INFINITY;
    }
    if (KEEP) {
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int t = at.m0 + at.wm + 16 * i + (at.lane & 15);
#pragma unroll
        for (int j = 0; j < NI; ++j)
          if (t < p.M && 16 * j < left) *(v4f*)(a.logits + (int64_t)t * a.ld + c0 + 16 * j) = acc[i][j];
      }
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int r = at.wm + 16 * i + (at.lane & 15), t = at.m0 + r;
      const int y = (t < p.M ? a.y.at(t) : -1) - c0;  // the target among this lane's columns
      float m = -INFINITY, s = 0.0f, hit = 0.0f;
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          m = fmaxf(m, acc[i][j][q]);
          hit = y == 16 * j + q ? acc[i][j][q] : hit;
        }
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) s += exp_above(acc[i][j][q], m);
      if (y >= 0 && y < 16 * NI && (y & 12) == 0) a.hit[t] = hit;
      join(m, s, __shfl_xor(m, 16), __shfl_xor(s, 16));
      join(m, s, __shfl_xor(m, 32), __shfl_xor(s, 32));
      if (at.lane < 16) sh[at.wave % WN][r] = make_float2(m, s);
    }
    __syncthreads();
    const int tid = at.wave * 64 + at.lane;
    for (int r = tid; r < BM; r += WM * WN * 64) {
      float m = sh[0][r].x, s = sh[0][r].y;
#pragma unroll
      for (int w = 1; w < WN; ++w) join(m, s, sh[w][r].x, sh[w][r].y);
      if (at.m0 + r < p.M) a.part[(int64_t)((a.v0 + at.n0) / BN) * p.M + at.m0 + r] = make_float2(m, s);
    }
  }
};

// A token's lse and loss by one wave: its partial statistics joined (lane l: tiles l,
// l + 64, ...; then across lanes).  All lanes return the loss.
__device__ __forceinline__ float loss_row(const float2* part, const float* hit, const Targets& y, int T, int t, int tiles,
                                          float* lse, float* rows) {
  const int lane = threadIdx.x & 63;
  float m = -INFINITY, s = 0.0f;
#pragma unroll 4
  for (int i = lane; i < tiles; i += 64) {
    const float2 v = part[(int64_t)i * T + t];
    join(m, s, v.x, v.y);
  }
  for (int d = 1; d < 64; d <<= 1) join(m, s, __shfl_xor(m, d), __shfl_xor(s, d));
  const float l = m + __builtin_amdgcn_logf(s) * kLn2;
  const int at = y.at(t);
  const float loss = at == -1 ? 0.0f : at < 0 ? NAN : l - hit[t];
  if (lane == 0) {
    lse[t] = l;
    rows[t] = loss;
  }
  return loss;
}

__global__ __launch_bounds__(256) void loss_rows_kernel(const float2* part, const float* hit, Targets y, int T, int tiles,
                                                        float* lse, float* rows) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t < T) loss_row(part, hit, y, T, t, tiles, lse, rows);
}

// The reduced loss and the gradients' scale by one workgroup of 16 waves.  ROWS: it
// makes the tokens' losses as well, a wave each (at most 16 tokens: saves a launch,
// 4 us of 31 for one token against 32,000 words).
constexpr int kTotalWaves = 16;
template <bool ROWS>
__global__ __launch_bounds__(kTotalWaves * 64) void loss_total_kernel(const float2* part, const float* hit, Targets y, int T,
                                                                      int tiles, float* lse, float* rows, int mean,
                                                                      float grad_scale, float* loss, float* scale) {
  __shared__ double sums[kTotalWaves];
  __shared__ int counts[kTotalWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double s = 0.0;
  int n = 0;
  if (ROWS) {
    if (wave < T) {
      s = (double)loss_row(part, hit, y, T, wave, tiles, lse, rows);
      n = y.at(wave) != -1;
    }
  } else {
    for (int t = threadIdx.x; t < T; t += kTotalWaves * 64) {
      s += (double)rows[t];
      n += y.at(t) != -1;
    }
    for (int d = 1; d < 64; d <<= 1) {
      s += __shfl_xor(s, d);
      n += __shfl_xor(n, d);
    }
  }
  if (lane == 0) {
    sums[wave] = s;
    counts[wave] = n;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kTotalWaves; ++i) {
      s += sums[i];
      n += counts[i];
    }
    if (n < 1) n = 1;  // no token counts: loss 0, gradients 0
    if (loss) *loss = (float)(mean ? s / n : s);
    *scale = mean ? grad_scale / (float)n : grad_scale;
  }
}

// ---- the gradients ----------------------------------------------------------

// g of a piece, unscaled bf16
struct EpiGrad {
  static constexpr bool kStaged = true;
  struct Args {
    uint16_t* g;
    int64_t ld;
    const float* lse;
    Targets y;
    int v0, V, ncols;  // ncols: the piece's columns, rounded up to 64
  };
  template <int BM, int BN, int WM, int WN, int MI, int NI>
  static __device__ void run(const GemmArgs& p, const Args& a, const TileAt& at, v4f (&acc)[MI][NI], uint8_t* lds) {
    float lse[MI];
    int y[MI];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int t = at.m0 + at.wm + 16 * i + (at.lane & 15);
      y[i] = t < p.M ? a.y.at(t) : -1;
      lse[i] = t < p.M ? a.lse[t] : 0.0f;
    }
    stage_part<__bf16, BN>(at, acc, lds, [&](int i, int, int n, float (&v)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = a.v0 + n + e;
        const float pr = __builtin_amdgcn_exp2f((v[e] - lse[i]) * kLog2e) - (c == y[i] ? 1.0f : 0.0f);
        v[e] = y[i] < 0 || c >= a.V ? 0.0f : pr;
      }
    });
    __syncthreads();
    store_rows<BM, BN, WM * WN>(at, lds, a.g, a.ld, p.M, a.ncols);
  }
};

// the same from kept logits, 8 columns a thread, `per` workgroups a token
__global__ __launch_bounds__(256) void grad_kernel(const float* logits, int ldl, const float* lse, Targets y, int v0,
                                                   int ncols, int per, uint16_t* g, int64_t ld) {
  const int t = blockIdx.x / per, n = 8 * ((blockIdx.x - t * per) * 256 + threadIdx.x);
  if (n >= ncols) return;
  const int at = y.at(t), c = v0 + n;
  const float l = lse[t];
  const float* from = logits + (int64_t)t * ldl + c;
  uint32_t w[4] = {0, 0, 0, 0};
  if (at >= 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v4f v = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (c + 4 * h < y.V) v = *(const v4f*)(from + 4 * h);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = c + 4 * h + e < y.V
                   ? __builtin_amdgcn_exp2f((v[e] - l) * kLog2e) - (c + 4 * h + e == at ? 1.0f : 0.0f)
                   : 0.0f;
      w[2 * h] = pack2(v[0], v[1], __bf16());
      w[2 * h + 1] = pack2(v[2], v[3], __bf16());
    }
  }
  *(uint4*)(g + (int64_t)t * ld + n) = make_uint4(w[0], w[1], w[2], w[3]);
}

// FP32 partial sums of dx, per split: written, or added to
struct EpiSum {
  static constexpr bool kStaged = false;
  struct Args {
    float* sum;      // [splits][M][ld]
    int64_t stride;  // of a split
    int ld, add;
  };
  template <int BM, int BN, int WM, int WN, int MI, int NI>
  static __device__ void run(const GemmArgs& p, const Args& a, const TileAt& at, v4f (&acc)[MI][NI], uint8_t*) {
    float* sum = a.sum + at.split * a.stride;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int m = at.m0 + at.wm + 16 * i + (at.lane & 15);
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const int n = at.n0 + at.wn + 16 * j + 4 * (at.lane >> 4);
        if (m >= p.M || n >= a.ld) continue;
        v4f* to = (v4f*)(sum + (int64_t)m * a.ld + n);
        *to = a.add ? *to + acc[i][j] : acc[i][j];
      }
    }
  }
};

// dx: the splits' sums in order, scaled, to bf16
__global__ __launch_bounds__(256) void dx_kernel(const float* sum, int64_t stride, int splits, int ld, const float* scale,
                                                 uint16_t* dx, int T, int H) {
  const float s = *scale;
  const int per = ld >> 2;
  for (int64_t i = blockIdx.x * 256 + threadIdx.x; i < (int64_t)T * per; i += (int64_t)gridDim.x * 256) {
    const int t = (int)(i / per), c = 4 * (int)(i % per);
    float4 v = *(const float4*)(sum + (int64_t)t * ld + c);
#pragma unroll 8
    for (int k = 1; k < splits; ++k) {
      const float4 w = *(const float4*)(sum + k * stride + (int64_t)t * ld + c);
      v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
    }
    uint16_t* to = dx + (int64_t)t * H + c;
    const uint32_t lo = pack2(v.x * s, v.y * s, __bf16()), hi = pack2(v.z * s, v.w * s, __bf16());
    if ((H & 3) == 0 && ((uintptr_t)dx & 7) == 0) {
      if (c < H) *(uint2*)to = make_uint2(lo, hi);
    } else {
      if (c < H) to[0] = (uint16_t)lo;
      if (c + 1 < H) to[1] = (uint16_t)(lo >> 16);
      if (c + 2 < H) to[2] = (uint16_t)hi;
      if (c + 3 < H) to[3] = (uint16_t)(hi >> 16);
    }
  }
}

// dw of a piece, scaled, to bf16.  ONCE: rows of whole cache lines, stored past the
// caches, which keep g and w (129 tokens, 64,000 words of 2,048: 343 us with plain
// stores, 296; rows that share lines: 301 tokens, 32,003 of 1,001 171 plain, 174).
template <bool ONCE>
struct EpiWeight {
  static constexpr bool kStaged = true;
  struct Args {
    uint16_t* dw;  // the piece's first row
    const float* scale;
    int rows, H;
  };
  template <int BM, int BN, int WM, int WN, int MI, int NI>
  static __device__ void run(const GemmArgs&, const Args& a, const TileAt& at, v4f (&acc)[MI][NI], uint8_t* lds) {
    const float s = *a.scale;
    stage_part<__bf16, BN>(at, acc, lds, [&](int, int, int, float (&v)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= s;
    });
    __syncthreads();
    store_rows<BM, BN, WM * WN, ONCE>(at, lds, a.dw, a.H, a.rows, a.H);
  }
};

// rows copied to rows of ld (a multiple of 64) elements, zeros after H; rows may
// start at any element.  TOKENS: rows whose token does not count become zeros,
// whatever they hold: their g is 0, and 0 times a NaN would reach all of dw.
template <bool TOKENS>
__global__ __launch_bounds__(256) void pad_rows_kernel(const uint16_t* src, int64_t lds, int rows, int H, uint16_t* dst,
                                                       int ld, Targets y) {
  const int per = ld >> 3, whole = H >> 3;
  const int64_t stride = (int64_t)gridDim.x * 256, tid = blockIdx.x * 256 + threadIdx.x;
#pragma unroll 4
  for (int64_t i = tid; i < (int64_t)rows * whole; i += stride) {
    const int r = (int)(i / whole), c = 8 * (int)(i % whole);
    v4i w;
    __builtin_memcpy(&w, src + r * lds + c, 16);
    if (TOKENS && y.at(r) < 0) w = (v4i){0, 0, 0, 0};
    *(v4i*)(dst + (int64_t)r * ld + c) = w;
  }
  const int left = 8 * (per - whole);
  for (int64_t i = tid; i < (int64_t)rows * left; i += stride) {
    const int r = (int)(i / left), c = 8 * whole + (int)(i % left);
    dst[(int64_t)r * ld + c] = c < H && !(TOKENS && y.at(r) < 0) ? src[r * lds + c] : 0;
  }
}

// ---- host -------------------------------------------------------------------

struct LossPlan {
  bool packed;   // x and w are copied to padded rows
  bool copied;   // x is copied: packed, or for dw (0.1% of its time at 4,096 tokens and
                 // 128,000 words), which must not meet the rows that do not count
  int ld;        // H rounded up to 64
  int bm, bn;    // the logits' tile
  int bx, bw;    // rows of dx's tile; edge of dw's
  int tilesV, piece, splits;
  bool keep;     // the logits, for g
  int ldl;       // their rows
  size_t logits, part, hit, lse, rows, scale, xp, wp, g, sum, bytes;
};

// whether x and w are read in place (a tile of 256 rows stays below 2^31 bytes)
bool aligned(const void* x, int64_t ldx, const void* w, int64_t ldw, int H) {
  return (H & 63) == 0 && ldx <= 1 << 21 && ldw <= 1 << 21 && (ldx & 7) == 0 && (ldw & 7) == 0 && (((uintptr_t)x | (uintptr_t)w) & 15) == 0;
}

LossPlan plan_of(bool direct, int T, int H, int V, bool gx, bool gw, bool may_keep, int cus) {
  LossPlan p = {};
  p.packed = !direct;
  p.copied = p.packed || gw;
  p.ld = (H + 63) & ~63;
  auto up = [](int64_t n, int64_t d) { return (n + d - 1) / d; };
  const int64_t steps = p.ld / kGemmStep;
  // The logits' tile.  Few tokens: narrow tiles in deep rings, which bring w to all CUs
  // (one token against 32,000 words of 2,048: 31 us, with tiles of 128 x 256 34, of
  // 256 x 256 47; 43 tokens, 6,223 words of 4,992, the statistics alone: 21, 55, 84;
  // 200 tokens, 32,000 words of 2,048: 92, 38, 56; 365, 95,641 of 5,184: 1,194, 504, 412).
  const int64_t c32 = tiles_cost<32, 64>(up(T, 32) * up(V, 64), steps, cus);
  const int64_t c128 = tiles_cost<128, 256>(up(T, 128) * up(V, 256), steps, cus);
  const int64_t c256 = tiles_cost<256, 256>(up(T, 256) * up(V, 256), steps, cus);
  p.bm = c32 <= c128 && c32 <= c256 ? 32 : c128 <= c256 ? 128 : 256;
  p.bn = p.bm == 32 ? 64 : 256;
  p.tilesV = (V + p.bn - 1) / p.bn;
  const bool grads = gx || gw;
  // a piece of the vocabulary: all of it unless g (or the padded copy of its
  // weights) gets too large
  int64_t most = kPieceBytes / (2LL * (grads ? T : 1));
  if (p.packed && most > kCopyBytes / (2LL * p.ld)) most = kCopyBytes / (2LL * p.ld);
  if (most < 256) most = 256;
  p.piece = (int)(up(up(V, up(V, most)), 256) * 256);
  // dx: rows of its tile, and splits of a piece's vocabulary, so that the tiles fill
  // the device in whole rounds; a split's partial sums are written and read once, at
  // about 4 MB a us.  Without splits: 33 tokens, 32,000 words of 2,048 418 us against
  // 138; 1,000 tokens, 64,000 words 1,753 against 920.
  const int width = V < p.piece ? V : p.piece;
  p.splits = 1;
  if (gx) {
    const int64_t along = up(width, kGemmStep), sums = 8LL * T * p.ld / 40000;
    int64_t best = INT64_MAX;
    for (int n = 1; n <= 64 && n * 4 <= along + 3; ++n) {
      const int64_t s = up(along, n);
      const int64_t cost[3] = {tiles_cost<32, 64>(up(T, 32) * up(p.ld, 64) * n, s, cus),
                               tiles_cost<128, 256>(up(T, 128) * up(p.ld, 256) * n, s, cus),
                               tiles_cost<256, 256>(up(T, 256) * up(p.ld, 256) * n, s, cus)};
      for (int i = 0; i < 3; ++i)
        if (cost[i] + n * sums < best) {
          best = cost[i] + n * sums;
          p.splits = n;
          p.bx = i == 0 ? 32 : i == 1 ? 128 : 256;
        }
    }
  }
  // dw: 2,576 tokens, 1,073 words of 846: 15 us with tiles of 64, 25 with 128, 53 with
  // 256; 1,000, 4,096 of 2,048: 36, 22, 30; 600, 32,000 of 4,096: 383, 214, 183
  if (gw) {
    const int64_t s = up(T, kGemmStep);
    const int64_t w64 = tiles_cost<64, 64>(up(width, 64) * up(p.ld, 64), s, cus);
    const int64_t w128 = tiles_cost<128, 128>(up(width, 128) * up(p.ld, 128), s, cus);
    const int64_t w256 = tiles_cost<256, 256>(up(width, 256) * up(p.ld, 256), s, cus);
    p.bw = w64 <= w128 && w64 <= w256 ? 64 : w128 <= w256 ? 128 : 256;
  }
  p.ldl = (V + 63) & ~63;
  const int64_t kept = 4LL * T * p.ldl;
  p.keep = may_keep && grads && kept <= (H < 1024 ? kKeepShort : kKeepBytes);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at = (at + bytes + 255) & ~(size_t)255;
    return was;
  };
  p.part = take((size_t)p.tilesV * T * 8);
  p.hit = take((size_t)T * 4);
  p.lse = take((size_t)T * 4);
  p.rows = take((size_t)T * 4);
  p.scale = take(4);
  if (p.copied) p.xp = take((size_t)T * p.ld * 2);
  if (p.packed) {
    p.wp = take((size_t)(p.piece < V ? p.piece : V) * p.ld * 2);
  }
  if (p.keep) p.logits = take((size_t)T * p.ldl * 4);
  if (grads) p.g = take((size_t)T * p.piece * 2);
  if (gx) p.sum = take((size_t)p.splits * T * p.ld * 4);
  p.bytes = at;
  return p;
}

template <int BM, int BN, int WM, int WN, int DEEP, bool TA, bool TB, class Epi>
int launch(GemmArgs g, const typename Epi::Args& e, hipStream_t st) {
  g.batch = 1;
  g.tilesM = (g.M + BM - 1) / BM;
  g.tilesN = (g.N + BN - 1) / BN;
  g.tiles = g.tilesM * g.tilesN;
  const int64_t grid = (int64_t)g.tilesM * g.tilesN * g.splits;
  if (grid > 0xFFFFFFFFLL / (WM * WN * 64)) return MXW_ERR_DIM;
  hipLaunchKernelGGL((gemm16_kernel<__bf16, BM, BN, WM, WN, DEEP, TA, TB, false, Epi>), dim3((unsigned)grid),
                     dim3(WM * WN * 64), 0, st, g, e);
  return MXW_OK;
}

// products whose M axis is the tokens
template <bool TB, class Epi>
int launch_tokens(int bm, const GemmArgs& g, const typename Epi::Args& e, hipStream_t st) {
  if (bm == 32) return launch<32, 64, 1, 4, 6, false, TB, Epi>(g, e, st);
  if (bm == 128) return launch<128, 256, 2, 4, 0, false, TB, Epi>(g, e, st);
  return launch<256, 256, 2, 4, 0, false, TB, Epi>(g, e, st);
}

template <bool ONCE>
int launch_weight(int bw, const GemmArgs& g, const typename EpiWeight<ONCE>::Args& e, hipStream_t st) {
  if (bw == 64) return launch<64, 64, 2, 2, 5, true, true, EpiWeight<ONCE>>(g, e, st);
  if (bw == 128) return launch<128, 128, 2, 2, 0, true, true, EpiWeight<ONCE>>(g, e, st);
  return launch<256, 256, 2, 4, 0, true, true, EpiWeight<ONCE>>(g, e, st);
}

int check_loss(int T, int H, int V) {
  return T < 1 || T > kMaxTokens || H < 1 || H > 65536 || V < 1 || V > kMaxVocab ? MXW_ERR_DIM : MXW_OK;
}

unsigned copy_blocks(int64_t chunks) {
  const int64_t b = (chunks + 255) / 256;
  return (unsigned)(b < 1 ? 1 : b > 8192 ? 8192 : b);
}

}  // namespace

extern "C" {

int64_t mxw_vocab_loss_workspace_size(const uint16_t* x, int64_t ldx, const uint16_t* w, int64_t ldw, int T, int H,
                                      int V, int grads) {
  const int which = grads & ~MXW_LOSS_SMALL;
  if (check_loss(T, H, V) || ldx < H || ldw < H || which < 0 || which > 3) return MXW_ERR_DIM;
  int cus = 0;
  const int rc = check_device(&cus);
  if (rc) return rc;
  return (int64_t)plan_of(aligned(x, ldx, w, ldw, H), T, H, V, which & 1, which & 2, which == grads, cus).bytes;
}

int mxw_vocab_loss(const uint16_t* x, int64_t ldx, const uint16_t* w, int64_t ldw, const void* targets,
                   int target_bytes, int64_t ignore_index, int T, int H, int V, int reduction, float grad_scale,
                   float* loss, uint16_t* dx, uint16_t* dw, void* workspace, size_t workspace_bytes, void* stream) {
  if (!x || !w || !targets || !loss) return MXW_ERR_NULL;
  if (check_loss(T, H, V) || ldx < H || ldw < H || (target_bytes != 4 && target_bytes != 8) ||
      (reduction != MXW_NONE && reduction != MXW_MEAN && reduction != MXW_SUM))
    return MXW_ERR_DIM;
  if ((((uintptr_t)x | (uintptr_t)w | (uintptr_t)dx | (uintptr_t)dw) & 1) || ((uintptr_t)loss & 3) ||
      ((uintptr_t)targets & (target_bytes - 1)))
    return MXW_ERR_ALIGN;
  int cus = 0;
  int rc = check_device(&cus);
  if (rc) return rc;
  LossPlan p = plan_of(aligned(x, ldx, w, ldw, H), T, H, V, dx != nullptr, dw != nullptr, true, cus);
  if (workspace_bytes < p.bytes)
    p = plan_of(aligned(x, ldx, w, ldw, H), T, H, V, dx != nullptr, dw != nullptr, false, cus);
  if (!workspace || workspace_bytes < p.bytes || ((uintptr_t)workspace & 255)) return MXW_ERR_WORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  uint8_t* ws = (uint8_t*)workspace;
  const Targets y = {targets, target_bytes == 8, ignore_index, V};
  float* lse = (float*)(ws + p.lse);
  float* rows = reduction == MXW_NONE ? loss : (float*)(ws + p.rows);
  float* scale = (float*)(ws + p.scale);

  const uint16_t* xs = x;
  int64_t lx = ldx, lw = ldw;
  if (p.copied) {
    uint16_t* xp = (uint16_t*)(ws + p.xp);
    hipLaunchKernelGGL((pad_rows_kernel<true>), dim3(copy_blocks((int64_t)T * p.ld / 8)), dim3(256), 0, st, x, ldx, T,
                       H, xp, p.ld, y);
    xs = xp;
    lx = p.ld;
  }
  if (p.packed) lw = p.ld;
  // the piece's weights as the products read them
  auto weights = [&](int v0, int width) -> const uint16_t* {
    if (!p.packed) return w + v0 * ldw;
    uint16_t* wp = (uint16_t*)(ws + p.wp);
    hipLaunchKernelGGL((pad_rows_kernel<false>), dim3(copy_blocks((int64_t)width * p.ld / 8)), dim3(256), 0, st,
                       w + v0 * ldw, ldw, width, H, wp, p.ld, Targets{});
    return wp;
  };
  auto logits = [&](const uint16_t* wv, int width) {
    GemmArgs g = {};
    g.A = xs;
    g.lda = (int)lx;
    g.B = wv;
    g.ldb = (int)lw;
    g.M = T;
    g.N = width;
    g.K = p.ld;
    g.splits = 1;
    g.ksplit = p.ld;
    return g;
  };
  const bool grads = dx || dw;
  const uint16_t* kept = nullptr;  // one piece: its padded weights serve both passes
  for (int v0 = 0; v0 < V; v0 += p.piece) {
    const int width = V - v0 < p.piece ? V - v0 : p.piece;
    kept = weights(v0, width);
    float2* part = (float2*)(ws + p.part);
    float* hit = (float*)(ws + p.hit);
    rc = p.keep ? launch_tokens<false, EpiStats<true>>(p.bm, logits(kept, width),
                                                       {part, hit, y, v0, V, (float*)(ws + p.logits), p.ldl}, st)
                : launch_tokens<false, EpiStats<false>>(p.bm, logits(kept, width), {part, hit, y, v0, V, nullptr, 0}, st);
    if (rc) return rc;
  }
  {
    const float2* part = (const float2*)(ws + p.part);
    const float* hit = (const float*)(ws + p.hit);
    float* total = reduction == MXW_NONE ? nullptr : loss;
    const int mean = reduction == MXW_MEAN;
    if (T <= kTotalWaves) {
      hipLaunchKernelGGL((loss_total_kernel<true>), dim3(1), dim3(kTotalWaves * 64), 0, st, part, hit, y, T, p.tilesV, lse,
                         rows, mean, grad_scale, total, scale);
    } else {
      hipLaunchKernelGGL(loss_rows_kernel, dim3((unsigned)((T + 3) / 4)), dim3(256), 0, st, part, hit, y, T, p.tilesV, lse,
                         rows);
      if (total || grads)
        hipLaunchKernelGGL((loss_total_kernel<false>), dim3(1), dim3(kTotalWaves * 64), 0, st, part, hit, y, T, p.tilesV,
                           lse, rows, mean, grad_scale, total, scale);
    }
  }
  if (grads) {
    uint16_t* gp = (uint16_t*)(ws + p.g);
    const int64_t sumStride = (int64_t)T * p.ld;
    for (int v0 = 0; v0 < V; v0 += p.piece) {
      const int width = V - v0 < p.piece ? V - v0 : p.piece, padded = (width + 63) & ~63;
      const uint16_t* wv = V <= p.piece ? kept : weights(v0, width);
      if (p.keep) {
        const int per = (padded + 2047) / 2048;
        hipLaunchKernelGGL(grad_kernel, dim3((unsigned)(T * per)), dim3(256), 0, st, (const float*)(ws + p.logits), p.ldl,
                           (const float*)lse, y, v0, padded, per, gp, (int64_t)p.piece);
      } else {
        const EpiGrad::Args eg = {gp, p.piece, lse, y, v0, V, padded};
        rc = launch_tokens<false, EpiGrad>(p.bm, logits(wv, width), eg, st);
        if (rc) return rc;
      }
      GemmArgs g = {};
      if (dx) {
        g.A = gp;
        g.lda = p.piece;
        g.B = wv;
        g.ldb = (int)lw;
        g.M = T;
        g.N = p.ld;
        g.K = width;
        g.splits = p.splits;
        g.ksplit = ((width + kGemmStep - 1) / kGemmStep + p.splits - 1) / p.splits * kGemmStep;
        const EpiSum::Args e = {(float*)(ws + p.sum), sumStride, p.ld, v0 > 0};
        rc = launch_tokens<true, EpiSum>(p.bx, g, e, st);
        if (rc) return rc;
      }
      if (dw) {
        g.A = gp;
        g.lda = p.piece;
        g.B = xs;
        g.ldb = (int)lx;
        g.M = padded;
        g.N = p.ld;
        g.K = T;
        g.splits = 1;
        g.ksplit = (T + kGemmStep - 1) / kGemmStep * kGemmStep;
        uint16_t* to = dw + (int64_t)v0 * H;
        rc = (H & 63) == 0 && ((uintptr_t)dw & 127) == 0 ? launch_weight<true>(p.bw, g, {to, scale, width, H}, st)
                                                         : launch_weight<false>(p.bw, g, {to, scale, width, H}, st);
        if (rc) return rc;
      }
    }
    if (dx)
      hipLaunchKernelGGL(dx_kernel, dim3(copy_blocks((int64_t)T * p.ld / 4)), dim3(256), 0, st,
                         (const float*)(ws + p.sum), sumStride, p.splits, p.ld, (const float*)scale, dx, T, H);
  }
  if (hipGetLastError() != hipSuccess) return MXW_ERR_LAUNCH;
  return MXW_OK;
}

}  // extern "C"
