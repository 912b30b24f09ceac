// moe_layer.hip -- a whole mixture-of-experts layer for a few tokens on MXFP8
// weights (mxw_moe_layer, declared in include/mxfp8_wgrad.h), for gfx950.
//
//     r = x R^T; the k largest of each token's r (ties: the lower expert);
//     weights = softmax(r) at those, optionally divided by their sum
//     h_j = silu(x Wg[e_j]^T) * (x Wu[e_j]^T);  out = sum_j weight_j h_j Wd[e_j]^T
//
// Every weight of an expert that some token chose is read once, everything else
// is small: bound by reading HBM.  The kernels:
//
//   router  logits r [T, E], in parts of H that the reader adds (skipped when the
//           caller brings its own routing; a small router is left to gate/up)
//   route   for more than 4 tokens, the choice of each (for fewer every
//           workgroup of the next kernel makes it for itself, a wave a token)
//   gate/up items (expert, rows of Wg and Wu): h of those rows for the expert's
//           tokens, times the token's weight, to the workspace (bf16)
//   down    few experts: a workgroup owns 16 output columns of all tokens, its
//           waves split the chosen experts' rows of Wd in steps of 128 columns and
//           leave a partial sum of each step in LDS; many: items (expert, 64
//           columns) leave FP32 partial outputs per (token, expert).  Either way a
//           token's are added in the order of its own choices, so that its result
//           does not depend on what the other tokens chose
//
// The products run on the bf16 MFMA 16 x 16 x 32 with weight rows as the first
// operand and up to 16 of the expert's tokens as the second: with few tokens the
// matrix unit is idle most of the time, and its work is free next to the loads.
// A lane loads 32 consecutive codes of one row -- its 32 bytes share one E8M0
// scale, 4 lanes take a whole 128-byte line -- and converts them with the scaled
// conversion (exact: E4M3 has 4 significant bits and the scale is a power of
// two) to 4 MFMA operands.  The tokens' operand is loaded in the same order of k.
// No atomics on data: the result is bitwise reproducible.
//
// Measured: 64 tokens over 256 experts of the 16B shape (2.0 GB of weights) 361 us,
// 5.5 TB/s (reading alone reaches 7.0); one token through 8 of 32 experts of the 671B
// shape 85 us, 4.3 TB/s (gate/up 51 us, of them 6 before the first weight is asked
// for); through 2 of 8 of the 16B shape 19 us, launches and latency.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.h"
#include "gemm16.h"
#include "mxfp8_wgrad.h"

namespace {

using mxw::check_device;
using mxw::pack2;
using mxw::v4i;
using mxw::v8bf;

using mxw::v4f;

constexpr int kMaxTokens = MXW_MOE_MAX_TOKENS;  // a 64-bit mask of tokens per expert
constexpr int kMaxChoices = 16;
constexpr int kWaves = 8;  // of the router kernel
constexpr float kLog2e = 1.4426950408889634f;

static_assert(kMaxTokens == 64, "token masks are 64-bit, one token a lane");

struct MoeArgs {
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* router;  // NULL: ids and weights are inputs
  const uint8_t *wgu, *sgu, *wd, *sd;
  const uint8_t* active;   // NULL: every token
  int T, E, k, H, I;
  int normalize;
  float scale;
  int32_t* ids;
  float* weights;
  uint16_t* out;
  float* logits;       // [parts][T][E]
  int parts;
  // the routing by expert, written by workgroup 0 of the gate/up kernel
  int32_t* count;      // chosen experts
  int32_t* expert;     // [count], ascending
  int32_t* first;      // [count] the expert's first row of h
  uint64_t* tokens;    // [count] its tokens
  int32_t* row;        // [T][k] the choice's row of h, -1: none, or an expert's second mention
  uint16_t* h;         // [pairs][I]
  float* part;         // [pairs][H]
};

__device__ __forceinline__ v4f mfma(const v4i& a, const v4i& b, const v4f& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// 8 E4M3 codes times 2^(scale's exponent) to 8 bf16
__device__ __forceinline__ v4i decode8(int lo, int hi, float scale) {
  v4i r;
  r.x = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false));
  r.y = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true));
  r.z = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false));
  r.w = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true));
  return r;
}

// 32 codes of one row with their scale byte
struct Codes {
  v4i lo, hi;
  uint32_t s;
};
__device__ __forceinline__ Codes load_codes(const uint8_t* row, const uint8_t* srow, int block) {
  Codes c;
  c.lo = __builtin_nontemporal_load((const v4i*)(row + 32 * block));
  c.hi = __builtin_nontemporal_load((const v4i*)(row + 32 * block) + 1);
  c.s = srow[block];
  return c;
}
// operand q (k = 8 q .. 8 q + 7 of the lane's 32)
__device__ __forceinline__ v4i operand(const Codes& c, int q) {
  const float s = __uint_as_float(c.s << 23);
  const v4i& w = q < 2 ? c.lo : c.hi;
  return (q & 1) ? decode8(w.z, w.w, s) : decode8(w.x, w.y, s);
}

// 16 weight rows (`row` of this lane, scales srow) times up to 16 token rows (xt of
// this lane) over the 128-wide steps s0 .. s1 - 1 of `blocks` 32-blocks, the loads of
// D steps in flight; each step's sums go to sink(step, sums).
template <int D, class Sink>
__device__ __forceinline__ void stream(const uint8_t* row, const uint8_t* srow, const uint16_t* xt, int blocks, int s0,
                                       int s1, Sink sink) {
  const int b = (threadIdx.x & 63) >> 4;
  Codes c[D];
  v4i xv[D][4];
  auto load = [&](int d, int s) {
    const int at = 4 * s + b < blocks ? 4 * s + b : 0;
    c[d] = load_codes(row, srow, at);
#pragma unroll
    for (int q = 0; q < 4; ++q) xv[d][q] = *(const v4i*)(xt + 32 * at + 8 * q);
  };
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (s0 + d < s1) load(d, s0 + d);
  for (int s = s0; s < s1; s += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int now = s + d;
      if (now >= s1) break;
      if (4 * now + b >= blocks) {  // past the row's end: block 0 of both, made zeros
        c[d] = Codes{};
#pragma unroll
        for (int q = 0; q < 4; ++q) xv[d][q] = (v4i){0, 0, 0, 0};
      }
      v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int q = 0; q < 4; ++q) acc = mfma(operand(c[d], q), xv[d][q], acc);
      if (now + D < s1) load(d, now + D);
      sink(now, acc);
    }
  }
}

// ---- reductions over a wave by DPP ------------------------------------------

template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp(int old, int v) {
  return __builtin_amdgcn_update_dpp(old, v, CTRL, ROWS, 0xF, false);
}
template <class F>
__device__ __forceinline__ int wave_reduce(int v, int none, F f) {
  v = f(v, dpp<0x111, 0xF>(none, v));  // lane i takes from i - 1, 2, 4, 8 of its row of 16
  v = f(v, dpp<0x112, 0xF>(none, v));
  v = f(v, dpp<0x114, 0xF>(none, v));
  v = f(v, dpp<0x118, 0xF>(none, v));
  v = f(v, dpp<0x142, 0xA>(none, v));  // lane 15 of rows 0, 2 into rows 1, 3
  v = f(v, dpp<0x143, 0xC>(none, v));  // lane 31 into rows 2, 3
  return __builtin_amdgcn_readlane(v, 63);
}
__device__ __forceinline__ float wave_max(float v) {
  return __int_as_float(wave_reduce(__float_as_int(v), __float_as_int(-INFINITY),
                                    [](int a, int b) { return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b))); }));
}
__device__ __forceinline__ float wave_sum(float v) {
  return __int_as_float(
      wave_reduce(__float_as_int(v), 0, [](int a, int b) { return __float_as_int(__int_as_float(a) + __int_as_float(b)); }));
}
__device__ __forceinline__ int wave_min(int v) {
  return wave_reduce(v, 0x7FFFFFFF, [](int a, int b) { return a < b ? a : b; });
}

// ---- router -----------------------------------------------------------------

// Logits of 16 experts and 16 tokens over the steps first, first + stride, ... of
// 128 of H, split over the workgroup's waves; thread i < 256 gets token t0 + i % 16,
// expert e0 + 4 ((i % 64) / 16) + i / 64.
template <int WAVES>
__device__ __forceinline__ float router_tile(const MoeArgs& a, int e0, int t0, int first, int stride,
                                             float (*red)[256]) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, b = lane >> 4;
  const int e = e0 + r < a.E ? e0 + r : a.E - 1, t = t0 + r < a.T ? t0 + r : a.T - 1;
  const uint16_t* re = a.router + (int64_t)e * a.H;
  const uint16_t* xt = a.x + t * a.ldx;
  const int blocks = a.H >> 5;
  v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int s = first + wave; 4 * s < blocks; s += stride) {
    const bool in = 4 * s + b < blocks;
    const int at = 32 * (in ? 4 * s + b : 0);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v4i w = *(const v4i*)(re + at + 8 * q), xv = *(const v4i*)(xt + at + 8 * q);
      if (!in) w = xv = (v4i){0, 0, 0, 0};
      acc = mfma(w, xv, acc);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) red[wave][i * 64 + lane] = acc[i];
  __syncthreads();
  float v = 0.0f;
  if (tid < 256) {
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v += red[w][tid];
  }
  __syncthreads();
  return v;
}

// workgroup (experts, tokens, part of H)
__global__ __launch_bounds__(kWaves * 64) void moe_router_kernel(MoeArgs a) {
  __shared__ float red[kWaves][256];
  const int tid = threadIdx.x, e0 = blockIdx.x * 16, t0 = blockIdx.y * 16;
  const float v = router_tile<kWaves>(a, e0, t0, blockIdx.z * kWaves, gridDim.z * kWaves, red);
  const int e = e0 + 4 * ((tid & 63) >> 4) + (tid >> 6), t = t0 + (tid & 15);
  if (tid < 256 && e < a.E && t < a.T) a.logits[((int64_t)blockIdx.z * a.T + t) * a.E + e] = v;
}

// The routing of one token by one wave: lane l holds experts l, l + 64, ...
// Writes the token's choices and weights.  logits: [parts][T][E].
template <class Id>
__device__ __forceinline__ void route_token(const MoeArgs& a, const float* logits, int parts, int t, Id* ids,
                                            float* weights) {
  const int lane = threadIdx.x & 63;
  if (a.active && !a.active[t]) {
    if (lane < a.k) {
      ids[lane] = -1;
      weights[lane] = 0.0f;
    }
    return;
  }
  float v[4];
  uint32_t gone = 0;  // experts that are taken, or beyond E
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lane + 64 * i;
    v[i] = e < a.E ? 0.0f : -INFINITY;
    gone |= (uint32_t)(e >= a.E) << i;
  }
  // four parts' loads in flight, added in order
  for (int z0 = 0; z0 < parts; z0 += 4) {
    float u[4][4];
#pragma unroll
    for (int z = 0; z < 4; ++z) {
      const float* from = logits + ((int64_t)(z0 + z < parts ? z0 + z : z0) * a.T + t) * a.E;
#pragma unroll
      for (int i = 0; i < 4; ++i) u[z][i] = from[lane + 64 * i < a.E ? lane + 64 * i : 0];
    }
#pragma unroll
    for (int z = 0; z < 4; ++z)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += z0 + z < parts && lane + 64 * i < a.E ? u[z][i] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) top = fmaxf(top, v[i]);
  top = wave_max(top);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lane + 64 * i < a.E) sum += __builtin_amdgcn_exp2f((v[i] - top) * kLog2e);
  sum = wave_sum(sum);
  const bool broken = !(sum == sum);  // a NaN, or an infinity: no softmax
  if (a.E <= 64) {
    // an expert a lane: its rank is the number of experts that come before it
    const float u = v[0] == v[0] ? v[0] : -INFINITY;
    int rank = 0;
#pragma unroll 8
    for (int e = 0; e < a.E; ++e) {
      const float o = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(u), e));
      rank += o > u || (o == u && e < lane);
    }
    const bool mine = lane < a.E && rank < a.k;
    const float p = mine ? __builtin_amdgcn_exp2f((u - top) * kLog2e) : 0.0f;
    const float norm = a.normalize ? wave_sum(p) : sum;
    if (mine) {
      ids[rank] = (Id)lane;
      weights[rank] = broken ? NAN : p / norm * a.scale;
    }
    return;
  }
  int mine = 0;                       // lane j: the j-th choice and its logit
  float logit = 0.0f;
  for (int j = 0; j < a.k; ++j) {
    float best = -INFINITY;
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u = v[i] == v[i] ? v[i] : -INFINITY;  // NaN is chosen last, but never twice
      if (!((gone >> i) & 1) && (at == 0x7FFFFFFF || u > best)) {
        best = u;
        at = lane + 64 * i;
      }
    }
    const float m = wave_max(best);
    const int e = wave_min(best == m ? at : 0x7FFFFFFF);
    if ((e & 63) == lane) gone |= 1u << (e >> 6);
    if (lane == j) {
      mine = e;
      logit = m;
    }
  }
  float p = lane < a.k ? __builtin_amdgcn_exp2f((logit - top) * kLog2e) : 0.0f;
  const float norm = a.normalize ? wave_sum(p) : sum;
  p = broken ? NAN : p / norm * a.scale;
  if (lane < a.k) {
    ids[lane] = (Id)mine;
    weights[lane] = p;
  }
}

__global__ __launch_bounds__(256) void moe_route_kernel(MoeArgs a) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t < a.T) route_token(a, a.logits, a.parts, t, a.ids + t * a.k, a.weights + t * a.k);
}

// ---- gate/up ----------------------------------------------------------------

struct Routing {
  float weights[kMaxTokens * kMaxChoices];
  uint32_t mask[MXW_MAX_EXPERTS][2];   // by expert: its tokens
  int16_t ids[kMaxTokens * kMaxChoices];
  int16_t start[MXW_MAX_EXPERTS];      // by expert: its first row of h
  int16_t expert[MXW_MAX_EXPERTS];     // the chosen ones, ascending
  int32_t chosen[4], pairs[4];
};

// where a workgroup has the routing from
enum From { kGiven, kLogits, kRouter };  // ids and weights; the logits; x and the router
constexpr int kFusedLogits = 1024;       // T E at most, for kRouter

// The routing by expert into LDS, by every workgroup for itself; workgroup 0
// writes out what the down kernels and the caller need.  `scratch` (kRouter):
// kFusedLogits + 256 WAVES floats of LDS.  Returns the number of chosen experts.
template <From FROM, int WAVES>
__device__ __forceinline__ int make_routing(const MoeArgs& a, Routing& rt, float* scratch) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = a.T * a.k;
  if (FROM != kGiven) {
    const float* logits = a.logits;
    int parts = a.parts;
    if (FROM == kRouter) {
      logits = scratch;
      parts = 1;
      for (int e0 = 0; e0 < a.E; e0 += 16) {
        const float v = router_tile<WAVES>(a, e0, 0, 0, WAVES, (float(*)[256])(scratch + kFusedLogits));
        const int e = e0 + 4 * (lane >> 4) + wave, t = tid & 15;
        if (tid < 256 && e < a.E && t < a.T) scratch[t * a.E + e] = v;
      }
      __syncthreads();
    }
    for (int t = wave; t < a.T; t += WAVES) route_token(a, logits, parts, t, rt.ids + t * a.k, rt.weights + t * a.k);
  } else {
    for (int i = tid; i < n; i += WAVES * 64) {
      const int id = a.ids[i];
      const bool in = id >= 0 && id < a.E && !(a.active && !a.active[i / a.k]);
      rt.ids[i] = (int16_t)(in ? id : -1);
      rt.weights[i] = in ? a.weights[i] : 0.0f;
    }
  }
  for (int i = tid; i < 2 * MXW_MAX_EXPERTS; i += WAVES * 64) rt.mask[i >> 1][i & 1] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += WAVES * 64) {
    const int e = rt.ids[i], t = i / a.k;
    if (e >= 0) atomicOr(&rt.mask[e][t >> 5], 1u << (t & 31));
  }
  __syncthreads();
  // chosen experts in order and their first rows of h, a wave per 64 experts
  static_assert(WAVES >= 4, "64 experts a wave");
  int before = 0, rank = 0;
  bool chosen = false;
  if (wave < 4) {
    const int pairs = tid < a.E ? __popc(rt.mask[tid][0]) + __popc(rt.mask[tid][1]) : 0;
    chosen = pairs > 0;
    const uint64_t votes = __ballot(chosen);
    int run = pairs;  // inclusive sum over the wave
    for (int d = 1; d < 64; d <<= 1) {
      const int u = __shfl_up(run, d);
      if (lane >= d) run += u;
    }
    before = run - pairs;
    rank = __popcll(votes & ((1ull << lane) - 1));
    if (lane == 63) {
      rt.chosen[wave] = __popcll(votes);
      rt.pairs[wave] = run;
    }
  }
  __syncthreads();
  if (chosen) {
    for (int w = 0; w < wave; ++w) {
      rank += rt.chosen[w];
      before += rt.pairs[w];
    }
    rt.expert[rank] = (int16_t)tid;
    rt.start[tid] = (int16_t)before;
  }
  __syncthreads();
  const int count = rt.chosen[0] + rt.chosen[1] + rt.chosen[2] + rt.chosen[3];
  if (blockIdx.x == 0) {
    for (int i = tid; i < n; i += WAVES * 64) {
      const int e = rt.ids[i], t = i / a.k;
      if (FROM != kGiven) {
        a.ids[i] = e;
        a.weights[i] = rt.weights[i];
      }
      int row = -1;
      if (e >= 0) {
        const uint64_t mask = rt.mask[e][0] | (uint64_t)rt.mask[e][1] << 32;
        row = rt.start[e] + __popcll(mask & ((1ull << t) - 1));
        for (int j = t * a.k; j < i; ++j)
          if (rt.ids[j] == e) row = -1;
      }
      a.row[i] = row;
    }
    if (tid == 0) *a.count = count;
    for (int i = tid; i < count; i += WAVES * 64) {
      const int e = rt.expert[i];
      a.expert[i] = e;
      a.first[i] = rt.start[e];
      a.tokens[i] = rt.mask[e][0] | (uint64_t)rt.mask[e][1] << 32;
    }
  }
  return count;
}

// the n-th token of a mask (n below its count)
__device__ __forceinline__ int nth_token(uint64_t mask, int n) {
  int at = 0;
#pragma unroll
  for (int w = 32; w > 0; w >>= 1) {  // skip halves that hold no more than n tokens
    const int low = __popcll(mask & ((1ull << w) - 1));
    const bool skip = n >= low;
    n -= skip ? low : 0;
    mask = skip ? mask >> w : mask;
    at += skip ? w : 0;
  }
  return at;
}
__device__ __forceinline__ float share_of(const MoeArgs& a, const Routing& rt, int t, int e) {
  float share = 0.0f;
  for (int j = 0; j < a.k; ++j) share += rt.ids[t * a.k + j] == e ? rt.weights[t * a.k + j] : 0.0f;
  return share;
}
// silu(g) u w, rounded once to bf16, the down product's operand type
__device__ __forceinline__ uint16_t hidden(float g, float u, float w) {
  return (uint16_t)pack2(g / (1.0f + __builtin_amdgcn_exp2f(-g * kLog2e)) * u * w, 0.0f, __bf16());
}

// ---- streaming through LDS ---------------------------------------------------

// Loads straight to LDS: 16 bytes a lane from a 64-bit address, to lds + 16 l; a
// dword, or a byte, a lane from a 64-bit base and a 32-bit offset, to the dword at
// lds + 4 l.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void global_lds16(const void* from, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, off"
      :
      : "s"(lds), "v"(from)
      : "memory", "m0");
}
__device__ __forceinline__ void global_lds4(const void* base, uint32_t off, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dword %1, %2"
      :
      : "s"(lds), "v"(off), "s"(base)
      : "memory", "m0");
}
__device__ __forceinline__ void global_lds1(const void* base, uint32_t off, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_ubyte %1, %2"
      :
      : "s"(lds), "v"(off), "s"(base)
      : "memory", "m0");
}
#pragma clang diagnostic pop

constexpr int kRing = 68 * 1024;  // LDS of a workgroup's ring: two workgroups a CU, the routing included

// Weight rows of a workgroup of 4 waves: group g of wave w is 16 rows, the first 8
// from `first` on, the others from `second` on, `apart` rows after group g - 1's.
struct Rows {
  const uint8_t *first, *second;    // codes of row 0 of either
  int valid_first, valid_second;    // rows there (the rest reads as zeros)
  const uint8_t *sfirst, *ssecond;  // their scales
  int apart;
  int C;                            // row length, a multiple of 32
};

// acc[g][n] = the wave's group g of weight rows times token group n (16 tokens,
// source rows token[16 n ...] at src + row * ld elements).  One step is 128 columns:
// each wave brings its own rows' codes and scales and a quarter of the tokens'
// rows to the step's slot of the ring, D - 1 steps ahead; every load takes whole
// cache lines (read straight into the MFMA's operand layout, 16 lanes would touch
// 16 lines, which made the vector memory path the bound: 3.0 TB/s at 8 of 32
// experts of the 671B shape).  One barrier a step.  WORDS: C is a multiple of 128, so
// a row's 4 scales of a step are one aligned dword; else they come byte by byte
// (G - 1 more loads a step: 15% more time where both are possible).
template <int G, int N, bool WORDS>
__device__ __forceinline__ void stream_rows(const Rows& w, const uint16_t* src, int64_t ld, const int32_t* token,
                                            int ntok, uint8_t* ring, v4f (&acc)[G][N]) {
  constexpr int kScaleLoads = WORDS ? 1 : G;
  constexpr int kCodes = 4 * G * 2048, kTokens = N * 4096, kScales = 4 * kScaleLoads * 256;
  constexpr int kSlot = kCodes + kTokens + kScales;
  constexpr int D = kRing / kSlot < 6 ? kRing / kSlot : 6;
  constexpr int kLoads = 2 * G + N + kScaleLoads;  // a wave's loads a step
  static_assert(!WORDS || 16 * G <= 64, "a lane a row");
  static_assert(D >= 2, "two slots");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, b = lane >> 4;
  const int blocks = w.C >> 5, steps = (blocks + 3) >> 2;
  const uint32_t lds0 = (uint32_t)(uintptr_t)ring;

  // codes: 8 rows of 128 bytes a load, chunk c of row i at c ^ (i / 2) % 8
  uint32_t vo[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = 8 * h + (lane >> 3);
    vo[h] = (uint32_t)((wave * G * w.apart + (lane >> 3)) * w.C + (((lane & 7) ^ ((i >> 1) & 7)) << 4));
  }
  // scales: lane l brings the step's 4 of row l % 16 of group l / 16, or the one of
  // block l % 4 of row l / 4
  uint32_t so[kScaleLoads];
#pragma unroll
  for (int g = 0; g < kScaleLoads; ++g) {
    const int i = WORDS ? lane & 15 : lane >> 2, group = WORDS ? (lane >> 4) % G : g;
    const int h = i >> 3, last = (h ? w.valid_second : w.valid_first) - 1;
    int row = (wave * G + group) * w.apart + (i & 7);
    if (row > last) row = last > 0 ? last : 0;
    so[g] = (uint32_t)((h ? (uint32_t)(w.ssecond - w.sfirst) : 0u) + (uint32_t)row * (uint32_t)blocks);
  }
  // tokens: 4 rows of 256 bytes a load, chunk c of row t at c ^ t % 16
  const uint16_t* xa[N];
  const int xc = (r ^ (4 * wave + b)) << 3;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int t = 16 * n + 4 * wave + b;
    xa[n] = src + token[t < ntok ? t : 0] * ld;
  }
  auto load = [&](int s, uint32_t slot) {
    const int64_t done = (int64_t)s * 128;
    const bool in = s < steps;
    const int64_t left1 = in ? (int64_t)w.valid_first * w.C - done : 0;
    const int64_t left2 = in ? (int64_t)w.valid_second * w.C - done : 0;
    const auto first = mxw::buffer_of(w.first + done, mxw::range_of(left1));
    const auto second = mxw::buffer_of(w.second + done, mxw::range_of(left2));
    const uint32_t to = lds0 + slot * kSlot + wave * G * 2048;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      mxw::load_lds16(first, to + g * 2048, vo[0] + g * w.apart * w.C);
      mxw::load_lds16(second, to + g * 2048 + 1024, vo[1] + g * w.apart * w.C);
    }
    // past the end: the last step's again, not used; past a row's end in its last
    // step: the row's first values, made zeros below like the codes
    const int at = in ? s : steps - 1;
    const int col = WORDS || 128 * at + xc < w.C ? 128 * at + xc : 0;
#pragma unroll
    for (int n = 0; n < N; ++n)
      global_lds16(xa[n] + col, lds0 + slot * kSlot + kCodes + n * 4096 + wave * 1024);
    const uint32_t scales = lds0 + slot * kSlot + kCodes + kTokens + wave * kScaleLoads * 256;
    if (WORDS) {
      global_lds4(w.sfirst + 4 * at, so[0], scales);
    } else {
      const int block = 4 * at + (lane & 3) < blocks ? 4 * at + (lane & 3) : blocks - 1;
#pragma unroll
      for (int g = 0; g < kScaleLoads; ++g) global_lds1(w.sfirst, so[g] + block, scales + g * 256);
    }
  };
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int n = 0; n < N; ++n) acc[g][n] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
  mxw::stage_barrier<0>();  // the ring's last use is over
  for (int s = 0; s < D - 1; ++s) load(s, s);
  int slot = 0, next = D - 1;
  for (int s = 0; s < steps; ++s) {
    mxw::stage_barrier<(D - 2) * kLoads>();
    load(s + D - 1, next);
    const uint8_t* at = ring + slot * kSlot;
    const uint8_t* codes = at + wave * G * 2048 + r * 128;
    const int sw = (r >> 1) & 7;
    Codes c[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      c[g].lo = *(const v4i*)(codes + g * 2048 + (((2 * b) ^ sw) << 4));
      c[g].hi = *(const v4i*)(codes + g * 2048 + (((2 * b + 1) ^ sw) << 4));
      const uint8_t* scales = at + kCodes + kTokens + wave * kScaleLoads * 256;
      if (WORDS) {
        c[g].s = scales[(16 * g + r) * 4 + b];
      } else {
        c[g].s = *(const uint32_t*)(scales + g * 256 + (4 * r + b) * 4);
        if (4 * s + b >= blocks) c[g] = Codes{};  // past the row's end
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v4i xv[N];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        xv[n] = *(const v4i*)(at + kCodes + n * 4096 + r * 256 + (((4 * b + q) ^ r) << 4));
        if (!WORDS && 4 * s + b >= blocks) xv[n] = (v4i){0, 0, 0, 0};
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const v4i a = operand(c[g], q);
#pragma unroll
        for (int n = 0; n < N; ++n) acc[g][n] = mfma(a, xv[n], acc[g][n]);
      }
    }
    slot = slot + 1 == D ? 0 : slot + 1;
    next = next + 1 == D ? 0 : next + 1;
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): no load outlives the ring's use
}

// Items (expert, 32 G rows of Wg and of Wu) by workgroups of 4 waves: a wave's
// group is 8 rows of Wg and the same 8 of Wu.
template <int G, int N, bool WORDS>
__device__ __forceinline__ void gate_item(const MoeArgs& a, const Routing& rt, int e, int i0, const int32_t* token,
                                          int ntok, uint8_t* ring) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, b = lane >> 4, blocks = a.H >> 5;
  const int64_t at = (int64_t)e * 2 * a.I + i0;
  const Rows w = {a.wgu + at * a.H, a.wgu + (at + a.I) * a.H,   a.I - i0, a.I - i0,
                  a.sgu + at * blocks, a.sgu + (at + a.I) * blocks, 8, a.H};
  v4f acc[G][N];
  stream_rows<G, N, WORDS>(w, a.x, a.ldx, token, ntok, ring, acc);
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int tok = 16 * n + r;
    const float share = tok < ntok ? share_of(a, rt, token[tok], e) : 0.0f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      // lanes b < 2 hold rows 4 b .. of Wg, lanes b + 2 the same of Wu
      v4f up;
#pragma unroll
      for (int i = 0; i < 4; ++i) up[i] = __shfl_xor(acc[g][n][i], 32);
      const int i = i0 + 8 * (wave * G + g) + 4 * b;
      if (b < 2 && tok < ntok && i < a.I) {
        const v4f& ga = acc[g][n];
        *(uint2*)(a.h + (int64_t)(rt.start[e] + tok) * a.I + i) =
            make_uint2(hidden(ga.x, up.x, share) | (uint32_t)hidden(ga.y, up.y, share) << 16,
                       hidden(ga.z, up.z, share) | (uint32_t)hidden(ga.w, up.w, share) << 16);
      }
    }
  }
}

template <From FROM, int G, bool WORDS>
__global__ __launch_bounds__(256, 2) void moe_gate_kernel(MoeArgs a) {
  constexpr bool MANY = FROM == kGiven;  // the others come with at most 16 tokens
  __shared__ Routing rt;
  __shared__ int32_t token[kMaxTokens];
  __shared__ __align__(1024) uint8_t ring[kRing];
  static_assert(sizeof(Routing) + sizeof(token) + kRing <= 80 * 1024, "two workgroups a CU");
  const int count = make_routing<FROM, 4>(a, rt, (float*)ring);
  const int tiles = (a.I + 32 * G - 1) / (32 * G);
  for (int item = blockIdx.x; item < count * tiles; item += gridDim.x) {
    const int e = rt.expert[item / tiles], i0 = item % tiles * 32 * G;
    const uint64_t mask = rt.mask[e][0] | (uint64_t)rt.mask[e][1] << 32;
    const int ntok = __popcll(mask);
    __syncthreads();  // the last item is done with the list
    if ((int)threadIdx.x < ntok) token[threadIdx.x] = nth_token(mask, threadIdx.x);
    __syncthreads();
    if (!MANY || ntok <= 16) gate_item<G, 1, WORDS>(a, rt, e, i0, token, ntok, ring);
    else if (ntok <= 32) gate_item<G, MANY ? 2 : 1, WORDS>(a, rt, e, i0, token, ntok, ring);
    else gate_item<G, MANY ? 4 : 1, WORDS>(a, rt, e, i0, token, ntok, ring);
  }
}

// ---- down -------------------------------------------------------------------

// 16 output columns of all tokens: the waves split the (expert, 128 columns of
// I) units in order and leave every unit's sums in LDS.  Which wave takes a unit
// depends on how many experts the whole batch chose; the units do not, and a
// token's are added over its choices and their steps, by `lanes` lanes an output
// that take every lanes-th step and join in a fixed order.
constexpr int kDownWaves = 16;
constexpr int kDownLds = 144 << 10;  // of the sums, beside 8 KiB of lists
size_t down_lds(int T, int k, int I) { return (size_t)((I + 127) / 128) * T * k * 64; }

__global__ __launch_bounds__(kDownWaves * 64, 4) void moe_down_kernel(MoeArgs a) {
  extern __shared__ __align__(16) float sums[];  // [steps][T k][16]
  __shared__ int32_t expert[MXW_MAX_EXPERTS], first[MXW_MAX_EXPERTS], row[kMaxTokens * kMaxChoices];
  __shared__ uint64_t tokens[MXW_MAX_EXPERTS];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int count = *a.count, pairs = a.T * a.k;
  for (int i = tid; i < count; i += kDownWaves * 64) {
    expert[i] = a.expert[i];
    first[i] = a.first[i];
    tokens[i] = a.tokens[i];
  }
  for (int i = tid; i < pairs; i += kDownWaves * 64) row[i] = a.row[i];
  __syncthreads();
  const int h0 = blockIdx.x * 16, r = lane & 15, b = lane >> 4;
  const int blocks = a.I >> 5, steps = (blocks + 3) >> 2, units = count * steps;
  int u = (int)((int64_t)units * wave / kDownWaves);
  const int end = (int)((int64_t)units * (wave + 1) / kDownWaves);
  while (u < end) {
    const int which = u / steps, s0 = u - which * steps;
    const int s1 = end - which * steps < steps ? end - which * steps : steps;
    const int ntok = __popcll(tokens[which]);
    const int64_t at = (int64_t)expert[which] * a.H + h0 + r;
    for (int g0 = 0; g0 < ntok; g0 += 16) {
      const int p = first[which] + (g0 + r < ntok ? g0 + r : g0);
      stream<3>(a.wd + at * a.I, a.sd + at * blocks, a.h + (int64_t)p * a.I, blocks, s0, s1, [&](int s, const v4f& acc) {
        if (g0 + r < ntok) *(v4f*)(sums + (s * pairs + p) * 16 + 4 * b) = acc;
      });
    }
    u = which * steps + s1;
  }
  __syncthreads();
  const int shift = a.T <= 4 ? 4 : a.T <= 16 ? 2 : 0, lanes = 1 << shift;
  for (int i = tid; i < a.T * 16 << shift; i += kDownWaves * 64) {
    const int c = i >> shift & 15, t = i >> (shift + 4);
    float v = 0.0f;
    for (int j = 0; j < a.k; j += 4) {  // four choices' reads in flight
      int p[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) p[q] = j + q < a.k ? row[t * a.k + j + q] : -1;
      for (int s = i & (lanes - 1); s < steps; s += lanes) {
        float w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = sums[(s * pairs + (p[q] < 0 ? 0 : p[q])) * 16 + c];
#pragma unroll
        for (int q = 0; q < 4; ++q) v += p[q] < 0 ? 0.0f : w[q];
      }
    }
    for (int d = 1; d < lanes; d <<= 1) v += __shfl_xor(v, d);
    if ((i & (lanes - 1)) == 0) a.out[(int64_t)t * a.H + h0 + c] = (uint16_t)pack2(v, 0.0f, __bf16());
  }
}

// many experts: items (expert, 64 G columns), to FP32 partial outputs per
// (token, expert)
template <int G, int N, bool WORDS>
__device__ __forceinline__ void down_item(const MoeArgs& a, int e, int h0, int first, int ntok, const int32_t* order,
                                          uint8_t* ring) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, b = lane >> 4, blocks = a.I >> 5;
  const int64_t at = (int64_t)e * a.H + h0;
  const Rows w = {a.wd + at * a.I, a.wd + (at + 8) * a.I, a.H - h0, a.H - h0 - 8,
                  a.sd + at * blocks, a.sd + (at + 8) * blocks, 16, a.I};
  v4f acc[G][N];
  stream_rows<G, N, WORDS>(w, a.h + (int64_t)first * a.I, a.I, order, ntok, ring, acc);
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int h = h0 + 16 * (wave * G + g) + 4 * b;
      if (16 * n + r < ntok && h < a.H) *(v4f*)(a.part + (int64_t)(first + 16 * n + r) * a.H + h) = acc[g][n];
    }
}

template <int G, bool WORDS>
__global__ __launch_bounds__(256, 2) void moe_down_part_kernel(MoeArgs a) {
  __shared__ int32_t order[kMaxTokens];
  __shared__ __align__(1024) uint8_t ring[kRing];
  if (threadIdx.x < kMaxTokens) order[threadIdx.x] = threadIdx.x;
  __syncthreads();
  const int count = *a.count;
  const int tiles = (a.H + 64 * G - 1) / (64 * G);
  for (int item = blockIdx.x; item < count * tiles; item += gridDim.x) {
    const int which = item / tiles, h0 = (item - which * tiles) * 64 * G;
    const int e = a.expert[which], first = a.first[which], ntok = __popcll(a.tokens[which]);
    if (ntok <= 16) down_item<G, 1, WORDS>(a, e, h0, first, ntok, order, ring);
    else if (ntok <= 32) down_item<G, 2, WORDS>(a, e, h0, first, ntok, order, ring);
    else down_item<G, 4, WORDS>(a, e, h0, first, ntok, order, ring);
  }
}

// the partial outputs of each token's choices, added in their order
__global__ __launch_bounds__(256) void moe_combine_kernel(MoeArgs a) {
  const int t = blockIdx.y, c = 4 * (blockIdx.x * 256 + threadIdx.x);
  if (c >= a.H) return;
  v4f v = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j = 0; j < a.k; ++j) {
    const int row = a.row[t * a.k + j];
    if (row >= 0) v += *(const v4f*)(a.part + (int64_t)row * a.H + c);
  }
  uint16_t* to = a.out + (int64_t)t * a.H + c;
  const uint32_t lo = pack2(v.x, v.y, __bf16()), hi = pack2(v.z, v.w, __bf16());
  to[0] = (uint16_t)lo;
  to[1] = (uint16_t)(lo >> 16);
  to[2] = (uint16_t)hi;
  to[3] = (uint16_t)(hi >> 16);
}

// ---- host -------------------------------------------------------------------

struct MoePlan {
  int parts;     // of H in the router
  bool fused;    // the gate kernel makes the logits itself
  bool by_item;  // down: partial outputs per item
  size_t logits, count, expert, first, tokens, row, h, part, bytes;
};

// experts that can be chosen
int most_experts(int T, int E, int k) { return T * k < E ? T * k : E; }

MoePlan plan_of(int T, int E, int k, int H, int I) {
  MoePlan p = {};
  // a step of 128 a wave if there are few workgroups
  p.parts = (H + 128 * kWaves - 1) / (128 * kWaves);
  if (p.parts > 8) p.parts = 8;
  // A router of at most 64 KiB is read by every workgroup of the gate kernel (from
  // its XCD's L2) in about a us; a kernel of its own costs 3 us and a launch: 1 token,
  // router 8 x 2048, 18.8 us against 20.0; 16 x 2048 (16 tokens) 31.0 against 33.0,
  // but 32 x 2048 78.0 against 75.8 and 8 x 7168 100 against 95.
  p.fused = T <= 16 && T * E <= kFusedLogits && E * H <= (32 << 10);
  // A workgroup of the plain down kernel reads 16 rows of I of every chosen expert;
  // by items the same bytes spread over the device, for a launch and the FP32
  // partial outputs.  Plain against by items, us: 1 token, H 2048, 88 KiB of rows a
  // workgroup 22.8 and 23.7, 110 KiB 24.6 and 24.5, 176 KiB 32.7 and 30.5; from H 4096
  // on it has a workgroup for each of 256 CUs (the whole device's: the size query runs
  // without one): 4096 wide 192 KiB 46.3 and 48.1, 256 KiB 52.3 and 57.2, 7168 wide
  // 192 KiB 81.2 and 76.5, 256 KiB 93.4 and 85.3, so that one bound loses up to a
  // tenth on one side of it or the other.  More than 16 tokens an expert read its rows
  // again: 64 tokens, 64 KiB 29.4 and 26.3 (the bound's edge), 128 KiB 38.6 and 27.8,
  // 176 KiB 47.5 and 32.6.  And the plain kernel's sums have to fit in LDS.
  const int most = T > 16 ? 64 : H < 4096 ? 96 : 192;
  p.by_item = (int64_t)most_experts(T, E, k) * I * 16 > (most << 10) || down_lds(T, k, I) > kDownLds;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at = (at + bytes + 255) & ~(size_t)255;
    return was;
  };
  p.logits = take((size_t)p.parts * T * E * 4);
  p.count = take(4);
  p.expert = take(MXW_MAX_EXPERTS * 4);
  p.first = take(MXW_MAX_EXPERTS * 4);
  p.tokens = take(MXW_MAX_EXPERTS * 8);
  p.row = take((size_t)T * k * 4);
  p.h = take((size_t)T * k * I * 2);
  if (p.by_item) p.part = take((size_t)T * k * H * 4);
  p.bytes = at;
  return p;
}

int check_moe(int T, int E, int k, int H, int I) {
  return T < 1 || T > kMaxTokens || E < 1 || E > MXW_MAX_EXPERTS || k < 1 || k > kMaxChoices || k > E || H < 32 ||
                 H > 65536 || (H & 31) || I < 32 || I > 65536 || (I & 31)
             ? MXW_ERR_DIM
             : MXW_OK;
}

// Two groups a wave read a step's tokens half as often, one makes twice the items.
// Gate/up: two only where they fill two workgroups a CU (64 tokens, 256 experts of
// 2048 x 1408: 362 us against 392 with one; 16 tokens over 8 experts of 2048 x 512,
// where one fills half the device and two a quarter: 28.6 against 24.0).
template <From FROM, bool WORDS>
void launch_gate_of(const MoeArgs& a, int cus, hipStream_t st) {
  const int64_t most = most_experts(a.T, a.E, a.k);
  const int64_t slots = 2 * cus, one = most * ((a.I + 31) / 32), two = most * ((a.I + 63) / 64);
  if (two < slots)
    hipLaunchKernelGGL((moe_gate_kernel<FROM, 1, WORDS>), dim3((unsigned)(one < slots ? one : slots)),
                       dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((moe_gate_kernel<FROM, 2, WORDS>), dim3((unsigned)slots), dim3(256), 0, st, a);
}
template <From FROM>
void launch_gate(const MoeArgs& a, int cus, hipStream_t st) {
  if (a.H & 127) launch_gate_of<FROM, false>(a, cus, st);
  else launch_gate_of<FROM, true>(a, cus, st);
}

// Down, whose steps are few (I is short): two groups from a workgroup a CU on (one
// token through 8 of 32 experts of 7168 x 2048, the layer: 90.0 us against 93.0 with
// one; 64 tokens over 8 of 2048 x 1408, half the CUs idle with two: 41.4 against 37.1).
template <bool WORDS>
void launch_down_part(const MoeArgs& a, int cus, hipStream_t st) {
  const int64_t most = most_experts(a.T, a.E, a.k);
  const int64_t slots = 2 * cus, one = most * ((a.H + 63) / 64), two = most * ((a.H + 127) / 128);
  if (two < cus)
    hipLaunchKernelGGL((moe_down_part_kernel<1, WORDS>), dim3((unsigned)(one < slots ? one : slots)), dim3(256), 0,
                       st, a);
  else
    hipLaunchKernelGGL((moe_down_part_kernel<2, WORDS>), dim3((unsigned)(two < slots ? two : slots)), dim3(256),
                       0, st, a);
}

}  // namespace

extern "C" {

int64_t mxw_moe_workspace_size(int T, int E, int k, int H, int I) {
  if (check_moe(T, E, k, H, I)) return MXW_ERR_DIM;
  return (int64_t)plan_of(T, E, k, H, I).bytes;
}

int mxw_moe_layer(const uint16_t* x, int64_t ldx, const uint16_t* router, const uint8_t* wgu, const uint8_t* sgu,
                  const uint8_t* wd, const uint8_t* sd, const uint8_t* active, int T, int E, int k, int H, int I,
                  int normalize, float scale, int32_t* ids, float* weights, uint16_t* out, void* workspace,
                  size_t workspace_bytes, void* stream) {
  if (!x || !wgu || !sgu || !wd || !sd || !ids || !weights || !out) return MXW_ERR_NULL;
  if (check_moe(T, E, k, H, I) || ldx < H || (ldx & 7)) return MXW_ERR_DIM;
  if ((((uintptr_t)x | (uintptr_t)router | (uintptr_t)wgu | (uintptr_t)wd) & 15) || ((uintptr_t)out & 1) ||
      (((uintptr_t)ids | (uintptr_t)weights | (uintptr_t)sgu | (uintptr_t)sd) & 3))
    return MXW_ERR_ALIGN;
  const MoePlan p = plan_of(T, E, k, H, I);
  if (!workspace || workspace_bytes < p.bytes || ((uintptr_t)workspace & 255)) return MXW_ERR_WORKSPACE;
  int cus = 0;
  const int rc = check_device(&cus);
  if (rc) return rc;
  hipStream_t st = (hipStream_t)stream;
  uint8_t* ws = (uint8_t*)workspace;
  MoeArgs a = {};
  a.x = x;
  a.ldx = ldx;
  a.router = router;
  a.wgu = wgu;
  a.sgu = sgu;
  a.wd = wd;
  a.sd = sd;
  a.active = active;
  a.T = T;
  a.E = E;
  a.k = k;
  a.H = H;
  a.I = I;
  a.normalize = normalize;
  a.scale = scale;
  a.ids = ids;
  a.weights = weights;
  a.out = out;
  a.logits = (float*)(ws + p.logits);
  a.parts = p.parts;
  a.count = (int32_t*)(ws + p.count);
  a.expert = (int32_t*)(ws + p.expert);
  a.first = (int32_t*)(ws + p.first);
  a.tokens = (uint64_t*)(ws + p.tokens);
  a.row = (int32_t*)(ws + p.row);
  a.h = (uint16_t*)(ws + p.h);
  a.part = (float*)(ws + p.part);
  if (p.fused && router) {
    launch_gate<kRouter>(a, cus, st);
  } else {
    if (router)
      hipLaunchKernelGGL(moe_router_kernel, dim3((unsigned)((E + 15) / 16), (unsigned)((T + 15) / 16), (unsigned)p.parts),
                         dim3(kWaves * 64), 0, st, a);
    // 4 tokens over 32 experts: 43.2 us with the choices made in every workgroup,
    // 44.9 with a launch for them; 12 tokens 71.9 and 69.9; 16 tokens 77.7 and 73.3
    if (router && T <= 4) {
      launch_gate<kLogits>(a, cus, st);
    } else {
      if (router) hipLaunchKernelGGL(moe_route_kernel, dim3((unsigned)((T + 3) / 4)), dim3(256), 0, st, a);
      launch_gate<kGiven>(a, cus, st);
    }
  }
  if (p.by_item) {
    if (I & 127) launch_down_part<false>(a, cus, st);
    else launch_down_part<true>(a, cus, st);
    hipLaunchKernelGGL(moe_combine_kernel, dim3((unsigned)((H + 1023) / 1024), (unsigned)T), dim3(256), 0, st, a);
  } else {
    hipLaunchKernelGGL(moe_down_kernel, dim3((unsigned)(H / 16)), dim3(kDownWaves * 64), down_lds(T, k, I), st, a);
  }
  if (hipGetLastError() != hipSuccess) return MXW_ERR_LAUNCH;
  return MXW_OK;
}

}  // extern "C"
