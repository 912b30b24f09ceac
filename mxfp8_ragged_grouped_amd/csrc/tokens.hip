// tokens.hip -- tokens to their experts' rows and back (mxw_sort_tokens,
// mxw_dispatch_tokens, mxw_combine_tokens, mxw_combine_tokens_grad) and the row-wise
// MX quantiser (mxw_quantize_rows), declared in include/mxfp8_wgrad.h, for gfx950.
//
//     xs[row[t][j]] = x[t];   out[t] = sum_j w[t][j] y[row[t][j]]
//     dy[row[t][j]] = w[t][j] dout[t],  dw[t][j] = <dout[t], y[row[t][j]]>
//
// All of it moves rows and computes next to nothing: bound by HBM, for few tokens by the
// launches.  Everything goes by tokens, not by rows: a token's own row is read (and quantised)
// once and stored to its experts' rows, or stored once after its experts' rows were read, so
// that every byte moves once (counters: 1.00 times what has to be read and written), and no
// row needs an index of where it came from.  A lane takes 8 neighbouring columns, on any
// alignment, and its k loads or stores are in flight together.
//
// Measured, bytes read and written once (one MI355X; a large copy 4.9 to 5.2 TB/s, reading or
// filling alone 6.9): 98,304 tokens of the 16B shape to 2 of 8 experts, bf16 and MXFP8 264 us
// (6.1 TB/s); 32,768 tokens joined from 8 rows of 2048 202 us (6.0); the gradient of 16,384
// tokens of the 671B shape, 8 rows each, 766 us (5.2, half of it stores); 65,536 x 7168 to
// MXFP8 216 us (6.6).  One token: 3 us a kernel and the host's call.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device.h"
#include "mx.h"
#include "mxfp8_wgrad.h"

namespace {

using namespace mxw;

// ---- the order --------------------------------------------------------------
//
// row[c] = first[e] + the number of choices before c of the same expert e: a stable
// counting sort.  A workgroup takes a piece of 1,024 to 16,384 choices, each of its 16 waves a
// consecutive run; it counts its waves' experts in LDS, turns the counts into first places, and a
// wave then walks its run 64 choices at a time: of each lane's choice, the lanes of the
// same expert (a ballot for each bit of the expert's number) before it give its rank.
// With more than one such piece, a kernel before leaves every piece's counts in the
// workspace, and each workgroup adds up what comes before its own.  Counting is in whole
// numbers: any order of the LDS atomics gives the same counts.
constexpr int kSortWaves = 16, kSortThreads = kSortWaves * 64;

struct SortArgs {
  const void* ids;
  int64_t ld;
  int n, k, E, align;   // n = T k choices
  int32_t *offs, *counts, *rows;
  int32_t* part;        // [pieces][E]
};

template <bool I64>
__device__ __forceinline__ int expert_of(const SortArgs& a, int c) {
  const int64_t at = (int64_t)(c / a.k) * a.ld + c % a.k;
  const int64_t e = I64 ? ((const int64_t*)a.ids)[at] : (int64_t)((const int32_t*)a.ids)[at];
  return e >= 0 && e < a.E ? (int)e : MXW_MAX_EXPERTS;
}

// LDS of one piece's counts, by wave
typedef int32_t WaveCounts[kSortWaves][MXW_MAX_EXPERTS];

// every wave's run of the piece into registers, and the counts of each
template <bool I64, int PER>
__device__ __forceinline__ void count_piece(const SortArgs& a, int (&e)[PER], WaveCounts& cnt) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = tid; i < kSortWaves * MXW_MAX_EXPERTS; i += kSortThreads) (&cnt[0][0])[i] = 0;
  const int first = blockIdx.x * (PER * kSortThreads), here = min(a.n - first, PER * kSortThreads);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = (wave * PER + i) * 64 + lane;
    e[i] = c < here ? expert_of<I64>(a, first + c) : MXW_MAX_EXPERTS;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (e[i] < MXW_MAX_EXPERTS) atomicAdd(&cnt[wave][e[i]], 1);
  __syncthreads();
}

template <bool I64, int PER>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortArgs a) {
  __shared__ WaveCounts cnt;
  int e[PER];
  count_piece<I64, PER>(a, e, cnt);
  for (int x = threadIdx.x; x < a.E; x += kSortThreads) {
    int sum = 0;
    for (int w = 0; w < kSortWaves; ++w) sum += cnt[w][x];
    a.part[(int64_t)blockIdx.x * a.E + x] = sum;
  }
}

template <bool I64, int PER>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortArgs a) {
  __shared__ WaveCounts cnt;
  __shared__ int32_t total[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int e[PER];
  count_piece<I64, PER>(a, e, cnt);
  int count = 0, before = 0, run = 0;  // of expert tid: its choices, those of earlier pieces, padded ends
  if (tid < MXW_MAX_EXPERTS) {
    if (tid < a.E) {
      if (gridDim.x == 1) {
        for (int w = 0; w < kSortWaves; ++w) count += cnt[w][tid];
      } else {
#pragma unroll 8
        for (int p = 0; p < (int)gridDim.x; ++p) {
          const int v = a.part[(int64_t)p * a.E + tid];
          count += v;
          before += p < (int)blockIdx.x ? v : 0;
        }
      }
    }
    const int padded = (count + a.align - 1) / a.align * a.align;
    run = padded;
    for (int d = 1; d < 64; d <<= 1) {
      const int u = __shfl_up(run, d);
      if (lane >= d) run += u;
    }
    if (lane == 63) total[wave] = run;
    before -= padded;
  }
  __syncthreads();
  if (tid < a.E) {
    for (int w = 0; w < wave; ++w) run += total[w];
    if (blockIdx.x == 0) {
      a.offs[tid] = run;
      a.counts[tid] = count;
    }
    int at = run + before;  // the expert's first row for this piece
    for (int w = 0; w < kSortWaves; ++w) {
      const int v = cnt[w][tid];
      cnt[w][tid] = at;
      at += v;
    }
  }
  __syncthreads();
  const int first = blockIdx.x * (PER * kSortThreads), here = min(a.n - first, PER * kSortThreads);
  volatile int32_t* place = cnt[wave];  // only this wave's from here on
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if ((wave * PER + i) * 64 >= here) break;
    uint64_t same = __ballot(e[i] < MXW_MAX_EXPERTS);
    for (int b = 0; (1 << b) < a.E; ++b) {
      const uint64_t vote = __ballot((e[i] >> b) & 1);
      same &= (e[i] >> b) & 1 ? vote : ~vote;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    const int c = (wave * PER + i) * 64 + lane;
    int row = -1;
    if (e[i] < MXW_MAX_EXPERTS) {
      const int at = place[e[i]];
      row = at + rank;
      __builtin_amdgcn_wave_barrier();  // every lane has read before the first of each expert writes
      if (rank == 0) place[e[i]] = at + __popcll(same);
      __builtin_amdgcn_wave_barrier();
    }
    if (c < here) a.rows[first + c] = row;
  }
}

// ---- rows -------------------------------------------------------------------

constexpr int kUnroll = 2;

struct RowArgs {
  const void* x;      // [T, H] the tokens: dispatch's x, the gradient's dout
  int64_t ldx;
  const void* y;      // [R, H] the experts' rows
  int64_t ldy;
  const int32_t *offs, *counts, *rows;
  const float* weights;
  const void* residual;
  int64_t ldr;
  int T, k, E, H, R;
  int pad_blocks, pad_split;
  void* out;          // [R, H], combine: [T, H]
  uint8_t *q, *s;     // [R, H], [R, H/32]
  float* dweights;
};

// Zeros in the padding rows of expert b / split: rows b % split, + split, ... of them.
template <bool F32, bool ROWS, bool MX>
__device__ __forceinline__ void pad_rows(const RowArgs& a, int b) {
  const int e = b / a.pad_split;
  const int64_t start = e ? min(max(a.offs[e - 1], 0), a.R) : 0;
  const int64_t end = min(max(a.offs[e], 0), a.R);
  for (int64_t r = start + max(a.counts[e], 0) + b % a.pad_split; r < end; r += a.pad_split) {
    const Raw8<F32> zero = {};
    for (int c = threadIdx.x * 8; c < a.H; c += 256 * 8) {
      if (ROWS) store_row<F32, false, false>(a.out, r * a.H, c, a.H, zero);
      if (MX) {
        *(i2*)(a.q + r * a.H + c) = (i2){0, 0};
        if (!(c & 31)) a.s[r * (a.H >> 5) + (c >> 5)] = 127;
      }
    }
  }
}

// xs[row[t][j]] = x[t]: a token is read once, by W waves, and stored to its k rows.
template <bool F32, bool ROWS, bool MX, int W, bool NT, bool SHARED>
__global__ __launch_bounds__(256) void dispatch_kernel(RowArgs a) {
  if ((int)blockIdx.x < a.pad_blocks) return pad_rows<F32, ROWS, MX>(a, blockIdx.x);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = (blockIdx.x - a.pad_blocks) * (4 / W) + wave / W;
  if (t >= a.T) return;
  const int32_t* rows = a.rows + (int64_t)t * a.k;
  const int64_t from = t * a.ldx;
  for (int c0 = ((wave % W) * 64 + (threadIdx.x & 63)) * 8; c0 < a.H; c0 += kUnroll * W * 512) {
    Raw8<F32> v[kUnroll];
    i2 q[kUnroll];
    int s[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int c = c0 + u * W * 512;
      if (c < a.H) v[u] = load_row<F32, NT, SHARED>(a.x, from, c, a.H);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (MX && c0 + u * W * 512 < a.H) {
        float f[8];
        values<F32>(v[u], f);
        s[u] = block_scale<8>(block_top(f));
        q[u] = encode_e4m3(f, s[u]);
      }
    for (int j = 0; j < a.k; ++j) {
      const int64_t r = rows[j];
      if (r < 0 || r >= a.R) continue;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int c = c0 + u * W * 512;
        if (ROWS && c < a.H) store_row<F32, NT, SHARED>(a.out, r * a.H, c, a.H, v[u]);
        if (MX && c < a.H) {
          store<NT>((i2*)(a.q + r * a.H + c), q[u]);
          if (!(c & 31)) a.s[r * (a.H >> 5) + (c >> 5)] = (uint8_t)s[u];
        }
      }
    }
  }
}

// a token's rows and weights, 8 choices at a time (-1: none)
template <bool WEIGHTS>
__device__ __forceinline__ void choices(const RowArgs& a, int t, int j0, int (&r)[8], float (&w)[8]) {
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const bool in = j0 + u < a.k;
    const int row = in ? a.rows[(int64_t)t * a.k + j0 + u] : -1;
    r[u] = row >= 0 && row < a.R ? row : -1;
    w[u] = WEIGHTS && r[u] >= 0 ? a.weights[(int64_t)t * a.k + j0 + u] : 1.0f;
  }
}

// out[t] = sum_j w[t][j] y[row[t][j]] (+ residual[t]), in the order of the choices
template <bool F32, bool WEIGHTS, int W, bool NT, bool SHARED>
__global__ __launch_bounds__(256) void combine_kernel(RowArgs a) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = blockIdx.x * (4 / W) + wave / W;
  if (t >= a.T) return;
  for (int c = ((wave % W) * 64 + (threadIdx.x & 63)) * 8; c < a.H; c += W * 512) {
    float sum[8] = {};
    for (int j0 = 0; j0 < a.k; j0 += 8) {
      int r[8];
      float w[8];
      choices<WEIGHTS>(a, t, j0, r, w);
      Raw8<F32> v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (r[u] >= 0) v[u] = load_row<F32, NT, SHARED>(a.y, r[u] * a.ldy, c, a.H);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (r[u] >= 0) {
          float f[8];
          values<F32>(v[u], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[i] = fmaf(w[u], f[i], sum[i]);
        }
    }
    if (a.residual) {
      float f[8];
      values<F32>(load_row<F32, false, SHARED>(a.residual, t * a.ldr, c, a.H), f);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += f[i];
    }
    store_row<F32, NT, SHARED>(a.out, (int64_t)t * a.H, c, a.H, rounded<F32>(sum));
  }
}

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float v) {   // lanes without a source add 0
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xF, false));
}
// the sum over a wave, in every lane
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<0x111, 0xF>(v);  // lane i takes from i - 1, 2, 4, 8 of its row of 16
  v += dpp<0x112, 0xF>(v);
  v += dpp<0x114, 0xF>(v);
  v += dpp<0x118, 0xF>(v);
  v += dpp<0x142, 0xA>(v);  // lane 15 of rows 0, 2 into rows 1, 3
  v += dpp<0x143, 0xC>(v);  // lane 31 into rows 2, 3
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// dy[row[t][j]] = w[t][j] dout[t], dw[t][j] = <dout[t], y[row[t][j]]>, by one wave a token or
// the workgroup's four
template <bool F32, bool ROWS, bool MX, int W, bool NT, bool SHARED>
__global__ __launch_bounds__(256) void combine_grad_kernel(RowArgs a) {
  __shared__ float red[4][8];
  if ((int)blockIdx.x < a.pad_blocks) return pad_rows<F32, ROWS, MX>(a, blockIdx.x);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = (blockIdx.x - a.pad_blocks) * (4 / W) + wave / W;
  if (W == 1 && t >= a.T) return;
  for (int j0 = 0; j0 < a.k; j0 += 8) {
    int r[8];
    float w[8], dot[8] = {};
    choices<true>(a, t, j0, r, w);
    for (int c = ((wave % W) * 64 + lane) * 8; c < a.H; c += W * 512) {
      const int n = min(a.H - c, 8);
      float d[8];
      values<F32>(load_row<F32, false, SHARED>(a.x, t * a.ldx, c, a.H), d);
      Raw8<F32> v[8];
      if (a.dweights) {
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (r[u] >= 0) v[u] = load_row<F32, NT, SHARED>(a.y, r[u] * a.ldy, c, a.H);
      }
      if (ROWS || MX) {
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (r[u] >= 0) {
            const int64_t row = (int64_t)r[u] * a.H, at = row + c;
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = w[u] * d[i];
            const Raw8<F32> o = rounded<F32>(f);
            if (ROWS) store_row<F32, NT, SHARED>(a.out, row, c, a.H, o);
            if (MX) {
              values<F32>(o, f);
              const int s = block_scale<8>(block_top(f));
              store<NT>((i2*)(a.q + at), encode_e4m3(f, s));
              if (!(c & 31)) a.s[at >> 5] = (uint8_t)s;
            }
          }
      }
      if (a.dweights) {
        if (SHARED && n < 8) {   // the lane before sums the first 8 - n
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] = i + n >= 8 ? d[i] : 0.0f;
#pragma unroll
          for (int i = 0; i < (F32 ? 8 : 4); ++i) {
            const int own = F32 ? (i + n >= 8 ? -1 : 0)
                                : (2 * i + n >= 8 ? 0xFFFF : 0) | (2 * i + 1 + n >= 8 ? (int)0xFFFF0000u : 0);
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u].v[i >> 2][i & 3] &= own;
          }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (r[u] >= 0) {
            float f[8];
            values<F32>(v[u], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot[u] = fmaf(d[i], f[i], dot[u]);
          }
      }
    }
    if (a.dweights) {
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (j0 + u < a.k) dot[u] = wave_sum(dot[u]);
      if (W == 4) {
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (lane == u) red[wave][u] = dot[u];
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 8; ++u) dot[u] = (red[0][u] + red[1][u]) + (red[2][u] + red[3][u]);
        __syncthreads();
      }
      if (wave % W == 0) {
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (lane == u && j0 + u < a.k) a.dweights[(int64_t)t * a.k + j0 + u] = dot[u];
      }
    }
  }
}

// ---- the row-wise quantiser -------------------------------------------------
//
// Blocks of 32 along the rows, 8 values a lane, 4 lanes a block, two such blocks a lane in
// flight (65,536 x 7168: 216 us; one 235, four 222).
struct QuantArgs {
  const void* x;
  int64_t ldx;
  int64_t chunks;   // R C / 8
  int per_row;      // C / 8
  uint8_t *q, *s;
};

template <bool F32, bool FP4, bool FLAT, bool NT>
__global__ __launch_bounds__(256) void quant_rows_kernel(QuantArgs a) {
  const int64_t i0 = (int64_t)blockIdx.x * (256 * kUnroll);
  // rows of another stride: the row and place of the workgroup's first chunk
  const int64_t row0 = FLAT ? 0 : i0 / a.per_row;
  const uint32_t in0 = FLAT ? 0 : (uint32_t)(i0 - row0 * a.per_row);
  Raw8<F32> v[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = i0 + u * 256 + threadIdx.x;
    if (i >= a.chunks) continue;
    if (FLAT) {
      v[u] = load8<F32, NT>(a.x, 8 * i);
    } else {
      const uint32_t in = in0 + u * 256 + threadIdx.x, down = in / (uint32_t)a.per_row;
      v[u] = load8<F32, NT>(a.x, (row0 + down) * a.ldx + 8 * (in - down * (uint32_t)a.per_row));
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = i0 + u * 256 + threadIdx.x;
    if (i >= a.chunks) continue;
    float f[8];
    values<F32>(v[u], f);
    const uint32_t top = block_top(f);
    const int s = block_scale<FP4 ? 2 : 8>(top);
    if (FP4)
      store<NT>((uint32_t*)(a.q + 4 * i), encode_e2m1(f, s));
    else
      store<NT>((i2*)(a.q + 8 * i), encode_e4m3(f, s));
    if (!(i & 3)) a.s[i >> 2] = (uint8_t)s;
  }
}

// ---- host -------------------------------------------------------------------

int64_t token_rows(int64_t T, int64_t k, int64_t E, int64_t align) {
  const int64_t n = T * k;
  return (n + (n < E ? n : E) * (align - 1)) / align * align;
}

// Choices of a lane of the sort: one workgroup alone up to 4,096 choices (6 us, two launches
// take 8), then the fewest that keep the pieces' counts, which every workgroup adds up, small
// next to the rest: 196,608 choices 11.2 us with 2 and 27.7 with 16, 800,000 over 256 experts
// 26.2 with 2, 19.5 with 4, 3.2 million 181, 73 and 40 with 2, 4 and 16.
int sort_per(int64_t n) {
  if (n <= 1024) return 1;
  if (n <= 2048) return 2;
  if (n <= 4096) return 4;
  if (n <= (1 << 19)) return 2;
  if (n <= (1 << 21)) return 4;
  return 16;
}

int check_plan(int T, int k, int E) {
  if (T < 0 || k < 1 || k > MXW_MAX_CHOICES || E < 1 || E > MXW_MAX_EXPERTS || (int64_t)T * k > MXW_MAX_ROWS)
    return MXW_ERR_DIM;
  return MXW_OK;
}

bool on(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

int launched() { return hipGetLastError() == hipSuccess ? MXW_OK : MXW_ERR_LAUNCH; }

// f(W, NT) with the waves of a token and the way past the caches as constants.  W waves take
// 512 W columns at a time; 4 leave few tokens spread over the device, and fewer have less idle
// lanes at a short row's end and, in the gradient, sums to join.  30,000 tokens joined from 4
// rows, with 1, 2 and 4 waves: 600 columns bf16 44, 41 and 46 us, 900 float32 115, 111 and 114,
// 1100 75, 68 and 68, 1500 95, 87 and 81; 32,768 from 8 of 2048 217, 208 and 202.  Dispatched to 2:
// 501 columns 28.6, 28.8 and 30.0, 1001 48, 47 and 51, 1284 to 8 76, 65 and 65.  Gradients, 1 and 4:
// 1024 columns 50 and 85, 1501 93 and 103, 1700 113 and 103.
template <int ONE, int TWO, class F>
void with_waves(int H, bool nt, F f) {
  auto w = [&](auto c) { nt ? f(c, std::true_type{}) : f(c, std::false_type{}); };
  if constexpr (TWO > ONE)
    if (H > ONE && H <= TWO) return w(std::integral_constant<int, 2>{});
  H <= ONE ? w(std::integral_constant<int, 1>{}) : w(std::integral_constant<int, 4>{});
}

// whether lanes may share columns (load_row): not where one stores over what another reads
bool may_share(int H, bool in_place) { return !(H & 7) || (H > 8 && !in_place); }

// Loads and stores past the caches where a call moves more than they hold (256 MB): 262,144
// rows of 2048 joined in 199 us, with cached ones 228; 65,536 rows of 7168 quantised in 221 and
// 239.  Below that whoever reads the result next finds it there: 4,096 tokens through 8 of 32
// experts, dispatched, joined and both gradients, 129 us, all past the caches 138.
bool past_caches(int64_t bytes) { return bytes > ((int64_t)256 << 20); }

// what dispatch and the gradient share: the padding rows' workgroups and the forms
int plan_pads(RowArgs& a) {
  a.pad_split = 4;
  a.pad_blocks = a.E * a.pad_split;
  return a.pad_blocks;
}

}  // namespace

extern "C" {

int64_t mxw_token_rows(int T, int k, int E, int align) {
  if (check_plan(T, k, E) != MXW_OK || align < 1 || align > 1024) return MXW_ERR_DIM;
  const int64_t R = token_rows(T, k, E, align);
  return R <= MXW_MAX_ROWS ? R : MXW_ERR_DIM;
}

int64_t mxw_sort_workspace_size(int T, int k, int E) {
  if (check_plan(T, k, E) != MXW_OK) return MXW_ERR_DIM;
  const int64_t n = (int64_t)T * k, piece = (int64_t)sort_per(n) * kSortThreads, pieces = (n + piece - 1) / piece;
  return pieces > 1 ? pieces * E * 4 : 0;
}

int mxw_sort_tokens(const void* ids, int id_bytes, int64_t ld, int T, int k, int E, int align, int32_t* offs,
                    int32_t* counts, int32_t* rows, void* workspace, size_t workspace_bytes, void* stream) {
  if (!offs || !counts || (T != 0 && (!ids || !rows))) return MXW_ERR_NULL;
  const int64_t R = mxw_token_rows(T, k, E, align);
  if (R < 0 || (id_bytes != 4 && id_bytes != 8) || ld < k) return MXW_ERR_DIM;
  if (!on(ids, id_bytes) || !on(offs, 4) || !on(counts, 4) || !on(rows, 4)) return MXW_ERR_ALIGN;
  const int64_t need = mxw_sort_workspace_size(T, k, E);
  if (need > 0 && (!workspace || !on(workspace, 256) || workspace_bytes < (size_t)need)) return MXW_ERR_WORKSPACE;
  const int64_t plan = (int64_t)T * k * 4;
  if (overlap<5>({{offs, 4 * E}, {counts, 4 * E}, {rows, plan}, {workspace, need}, {ids, T, ld, k, id_bytes}}, 4))
    return MXW_ERR_OVERLAP;
  if (const int rc = check_device()) return rc;
  SortArgs a = {ids, ld, T * k, k, E, align, offs, counts, rows, (int32_t*)workspace};
  hipStream_t st = (hipStream_t)stream;
  auto go = [&](auto i64, auto per) {
    constexpr bool I = decltype(i64)::value;
    constexpr int PER = decltype(per)::value;
    const int pieces = T ? (a.n + PER * kSortThreads - 1) / (PER * kSortThreads) : 1;
    if constexpr (PER > 1)   // 1: one piece
      if (pieces > 1) sort_count_kernel<I, PER><<<dim3(pieces), dim3(kSortThreads), 0, st>>>(a);
    sort_place_kernel<I, PER><<<dim3(pieces), dim3(kSortThreads), 0, st>>>(a);
  };
  auto pieces = [&](auto i64) {
    switch (sort_per(a.n)) {
      case 1: go(i64, std::integral_constant<int, 1>{}); break;
      case 2: go(i64, std::integral_constant<int, 2>{}); break;
      case 4: go(i64, std::integral_constant<int, 4>{}); break;
      default: go(i64, std::integral_constant<int, 16>{});
    }
  };
  if (id_bytes == 8)
    pieces(std::true_type{});
  else
    pieces(std::false_type{});
  return launched();
}

int mxw_dispatch_tokens(const void* x, int type, int64_t ldx, const int32_t* offs, const int32_t* counts,
                        const int32_t* rows, int T, int k, int E, int H, int R, void* xs, uint8_t* q, uint8_t* s,
                        void* stream) {
  if ((!xs && !q) || !q != !s) return MXW_ERR_NULL;
  if (check_plan(T, k, E) != MXW_OK || H < 1 || H > 65536 || R < 0 || R > MXW_MAX_ROWS || ldx < H ||
      (type != MXW_BF16 && type != MXW_F32) || (q && (H & 31)))
    return MXW_ERR_DIM;
  if (!offs || !counts || (T && (!x || !rows))) return MXW_ERR_NULL;
  const int size = type == MXW_F32 ? 4 : 2;
  if (!on(x, size) || !on(xs, size) || !on(offs, 4) || !on(counts, 4) || !on(rows, 4) || !on(q, 8)) return MXW_ERR_ALIGN;
  const int64_t RH = (int64_t)R * H, plan = (int64_t)T * k * 4;
  if (overlap<7>({{xs, RH * size}, {q, RH}, {s, RH / 32}, {x, T, ldx, H, size}, {offs, 4 * E}, {counts, 4 * E}, {rows, plan}}, 3))
    return MXW_ERR_OVERLAP;
  if (const int rc = check_device()) return rc;
  if (T == 0 || R == 0) return MXW_OK;
  RowArgs a = {};
  a.x = x, a.ldx = ldx, a.offs = offs, a.counts = counts, a.rows = rows;
  a.T = T, a.k = k, a.E = E, a.H = H, a.R = R, a.out = xs, a.q = q, a.s = s;
  // copied alone, FP32 rows go as rows of twice as many 16-bit elements: a lane's 16 bytes then
  // lie next to its neighbour's (30,000 tokens of 2048 to 2 rows each 139 us, with two times 16
  // bytes of 32 a lane 155; 5,000 of 3951 to 4 106 and 125)
  if (type == MXW_F32 && !q) a.H = 2 * H, a.ldx = 2 * ldx;
  const int pads = plan_pads(a);
  const bool nt = past_caches((int64_t)T * H * (size + k * ((xs ? size : 0) + (q ? 1 : 0))));
  hipStream_t st = (hipStream_t)stream;
  auto go = [&](auto f32, auto with_rows, auto mx) {
    constexpr bool F = decltype(f32)::value, RW = decltype(with_rows)::value, M = decltype(mx)::value;
    if constexpr (!M)   // MXFP8 rows are whole blocks
      if (!may_share(a.H, false)) {
        dispatch_kernel<F, RW, M, 1, false, false><<<dim3(pads + (T + 3) / 4), dim3(256), 0, st>>>(a);
        return;
      }
    with_waves<512, 1024>(a.H, nt, [&](auto w, auto past) {
      constexpr int W = decltype(w)::value, per = 4 / W;   // tokens of a workgroup
      dispatch_kernel<F, RW, M, W, decltype(past)::value, true><<<dim3(pads + (T + per - 1) / per), dim3(256), 0, st>>>(a);
    });
  };
  using Y = std::true_type;
  using N = std::false_type;
  auto forms = [&](auto f32) {
    if (!xs)
      go(f32, N{}, Y{});
    else
      go(f32, Y{}, Y{});
  };
  if (!q)
    go(N{}, Y{}, N{});
  else if (type == MXW_F32)
    forms(Y{});
  else
    forms(N{});
  return launched();
}

int mxw_combine_tokens(const void* y, int type, int64_t ldy, const int32_t* rows, const float* weights,
                       const void* residual, int64_t ldr, int T, int k, int H, int R, void* out, void* stream) {
  if (check_plan(T, k, 1) != MXW_OK || H < 1 || H > 65536 || R < 0 || R > MXW_MAX_ROWS || ldy < H ||
      (residual && ldr < H) || (type != MXW_BF16 && type != MXW_F32))
    return MXW_ERR_DIM;
  if (T && (!rows || !out || (R && !y))) return MXW_ERR_NULL;
  const int size = type == MXW_F32 ? 4 : 2;
  if (!on(y, size) || !on(residual, size) || !on(out, size) || !on(rows, 4) || !on(weights, 4)) return MXW_ERR_ALIGN;
  const int64_t plan = (int64_t)T * k * 4;
  const bool itself = residual == out && (ldr == H || T <= 1);
  if (overlap<5>({{out, (int64_t)T * H * size}, {y, R, ldy, H, size}, {rows, plan}, {weights, plan},
                  {itself ? nullptr : residual, T, ldr, H, size}}, 1))
    return MXW_ERR_OVERLAP;
  if (const int rc = check_device()) return rc;
  if (T == 0) return MXW_OK;
  RowArgs a = {};
  a.y = y, a.ldy = ldy, a.rows = rows, a.weights = weights, a.residual = residual, a.ldr = ldr;
  a.T = T, a.k = k, a.H = H, a.R = R, a.out = out;
  const bool nt = past_caches((int64_t)T * H * size * (k + 1));
  const bool shared = may_share(H, residual == out);
  hipStream_t st = (hipStream_t)stream;
  auto go = [&](auto f32, auto wt) {
    constexpr bool F = decltype(f32)::value, WT = decltype(wt)::value;
    with_waves<512, 1024>(H, nt, [&](auto w, auto past) {
      constexpr int W = decltype(w)::value, per = 4 / W;
      constexpr bool P = decltype(past)::value;
      const dim3 grid((T + per - 1) / per);
      if (shared)
        combine_kernel<F, WT, W, P, true><<<grid, dim3(256), 0, st>>>(a);
      else
        combine_kernel<F, WT, W, P, false><<<grid, dim3(256), 0, st>>>(a);
    });
  };
  using Y = std::true_type;
  using N = std::false_type;
  if (type == MXW_F32)
    weights ? go(Y{}, Y{}) : go(Y{}, N{});
  else
    weights ? go(N{}, Y{}) : go(N{}, N{});
  return launched();
}

int mxw_combine_tokens_grad(const void* dout, int type, int64_t ldo, const void* y, int64_t ldy, const int32_t* offs,
                            const int32_t* counts, const int32_t* rows, const float* weights, int T, int k, int E, int H,
                            int R, void* dy, uint8_t* q, uint8_t* s, float* dweights, void* stream) {
  if ((!dy && !q && !dweights) || !q != !s) return MXW_ERR_NULL;
  if (check_plan(T, k, E) != MXW_OK || H < 1 || H > 65536 || R < 0 || R > MXW_MAX_ROWS || ldo < H ||
      (dweights && ldy < H) || (type != MXW_BF16 && type != MXW_F32) || (q && (H & 31)))
    return MXW_ERR_DIM;
  if (((dy || q) && (!offs || !counts)) || (T && (!dout || !rows || !weights || (R && dweights && !y))))
    return MXW_ERR_NULL;
  const int size = type == MXW_F32 ? 4 : 2;
  if (!on(dout, size) || !on(y, size) || !on(dy, size) || !on(offs, 4) || !on(counts, 4) || !on(rows, 4) ||
      !on(weights, 4) || !on(dweights, 4) || !on(q, 8))
    return MXW_ERR_ALIGN;
  const int64_t RH = (int64_t)R * H, plan = (int64_t)T * k * 4;
  const Span yy(dweights ? y : nullptr, R, ldy, H, size);
  const bool itself = dy == y && (ldy == H || R <= 1);
  if (overlap<9>({{dy, RH * size}, {q, RH}, {s, RH / 32}, {dweights, plan}, {dout, T, ldo, H, size}, {weights, plan},
                  {rows, plan}, {offs, 4 * E}, {counts, 4 * E}}, 4) ||
      overlap<5>({{itself ? nullptr : dy, RH * size}, {q, RH}, {s, RH / 32}, {dweights, plan}, yy}, 4))
    return MXW_ERR_OVERLAP;
  if (const int rc = check_device()) return rc;
  if (T == 0) return MXW_OK;
  RowArgs a = {};
  a.x = dout, a.ldx = ldo, a.y = y, a.ldy = ldy, a.offs = offs, a.counts = counts, a.rows = rows, a.weights = weights;
  a.T = T, a.k = k, a.E = E, a.H = H, a.R = R, a.out = dy, a.q = q, a.s = s, a.dweights = dweights;
  const int pads = dy || q ? plan_pads(a) : 0;
  const bool shared = may_share(H, dweights && dy == y);
  const bool nt = past_caches((int64_t)T * H * (size + k * ((dweights ? size : 0) + (dy ? size : 0) + (q ? 1 : 0))));
  hipStream_t st = (hipStream_t)stream;
  auto go = [&](auto f32, auto with_rows, auto mx) {
    constexpr bool F = decltype(f32)::value, RW = decltype(with_rows)::value, M = decltype(mx)::value;
    with_waves<1536, 1536>(H, nt, [&](auto w, auto past) {
      constexpr int W = decltype(w)::value, per = 4 / W;
      constexpr bool P = decltype(past)::value;
      const dim3 grid(pads + (T + per - 1) / per);
      if (M || shared)
        combine_grad_kernel<F, RW, M, W, P, true><<<grid, dim3(256), 0, st>>>(a);
      else if constexpr (!M && (RW || W == 1))   // rows of under 8 columns, or dy over y
        combine_grad_kernel<F, RW, M, W, P, false><<<grid, dim3(256), 0, st>>>(a);
    });
  };
  using Y = std::true_type;
  using N = std::false_type;
  auto forms = [&](auto f32) {
    if (!q)
      dy ? go(f32, Y{}, N{}) : go(f32, N{}, N{});
    else
      dy ? go(f32, Y{}, Y{}) : go(f32, N{}, Y{});
  };
  if (type == MXW_F32)
    forms(Y{});
  else
    forms(N{});
  return launched();
}

int mxw_quantize_rows(const void* x, int type, int64_t ldx, int64_t R, int C, int format, uint8_t* q, uint8_t* s,
                      void* stream) {
  if (R < 0 || R > ((int64_t)1 << 31) || C < 32 || C > 65536 || (C & 31) || ldx < C ||
      (type != MXW_BF16 && type != MXW_F32) || (format != MXW_MXFP8 && format != MXW_MXFP4))
    return MXW_ERR_DIM;
  if (R && (!x || !q || !s)) return MXW_ERR_NULL;
  const int size = type == MXW_F32 ? 4 : 2;
  if (!on(x, size) || !on(q, 8)) return MXW_ERR_ALIGN;
  QuantArgs a = {x, ldx, R * (C >> 3), C >> 3, q, s};
  const int64_t blocks = (a.chunks + 256 * kUnroll - 1) / (256 * kUnroll);
  if (blocks > 0x7FFFFFFF / 256) return MXW_ERR_DIM;  // threads of a launch are counted in 32 bits
  if (overlap<3>({{q, R * C / (format == MXW_MXFP4 ? 2 : 1)}, {s, R * C / 32}, {x, R, ldx, C, size}}, 2)) return MXW_ERR_OVERLAP;
  if (const int rc = check_device()) return rc;
  if (R == 0) return MXW_OK;
  const bool nt = past_caches(R * C * (type == MXW_F32 ? 5 : 3));
  hipStream_t st = (hipStream_t)stream;
  auto go = [&](auto f32, auto fp4) {
    constexpr bool F = decltype(f32)::value, P = decltype(fp4)::value;
    if (ldx == C || R == 1)
      nt ? quant_rows_kernel<F, P, true, true><<<dim3((uint32_t)blocks), dim3(256), 0, st>>>(a)
         : quant_rows_kernel<F, P, true, false><<<dim3((uint32_t)blocks), dim3(256), 0, st>>>(a);
    else
      nt ? quant_rows_kernel<F, P, false, true><<<dim3((uint32_t)blocks), dim3(256), 0, st>>>(a)
         : quant_rows_kernel<F, P, false, false><<<dim3((uint32_t)blocks), dim3(256), 0, st>>>(a);
  };
  using Y = std::true_type;
  using N = std::false_type;
  if (type == MXW_F32)
    format == MXW_MXFP4 ? go(Y{}, Y{}) : go(Y{}, N{});
  else
    format == MXW_MXFP4 ? go(N{}, Y{}) : go(N{}, N{});
  return launched();
}

}  // extern "C"
