// moe_layer.hip -- a whole mixture-of-experts layer for a few tokens on MXFP8
// weights (mxw_moe_layer, declared in include/mxfp8_wgrad.h), for gfx950.
//
//     r = x R^T; the k largest of each token's r (ties: the lower expert);
//     weights = softmax(r) at those, optionally divided by their sum
//     h_j = silu(x Wg[e_j]^T) * (x Wu[e_j]^T);  out = sum_j weight_j h_j Wd[e_j]^T
//
// Every weight of an expert that some token chose is read once, everything else
// is small: bound by reading HBM.  Three kernels:
//
//   router  logits r [T, E] (skipped when the caller brings its own routing,
//           and done by the next kernel where it is small)
//   gate/up every workgroup first makes the routing for itself from the logits
//           (a few us against a launch; workgroup 0 also writes it out), then
//           takes items (expert, rows of Wg and Wu): h of those rows for the
//           expert's tokens, times the token's weight, to the workspace (bf16)
//   down    a workgroup owns 16 output columns of all tokens; its waves walk the
//           chosen experts' rows of Wd and the sums are joined in a fixed order
//
// The products run on the bf16 MFMA 16 x 16 x 32 with weight rows as the first
// operand and up to 16 of the expert's tokens as the second: with few tokens the
// matrix unit is idle most of the time, and its work is free next to the loads.
// A lane loads 32 consecutive codes of one row -- its 32 bytes share one E8M0
// scale, 4 lanes take a whole 128-byte line -- and converts them with the scaled
// conversion (exact: E4M3 has 4 significant bits and the scale is a power of
// two) to 4 MFMA operands.  The tokens' operand is loaded in the same order of k.
// No atomics on data: the result is bitwise reproducible.
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
constexpr int kWaves = 8;  // of the router and gate/up kernels
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
  float* logits;       // [T][E]
  // the routing by expert, written by workgroup 0 of the gate/up kernel
  int32_t* count;      // chosen experts
  int32_t* expert;     // [count], ascending
  int32_t* first;      // [count] the expert's first row of h
  uint64_t* tokens;    // [count] its tokens
  uint16_t* h;         // [pairs][I]
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

// logits of 16 experts and 16 tokens by one workgroup of 8 waves, K split over
// the waves; thread i < 256 gets the sum for expert e0 + (i / 64) * 4 ... as the
// MFMA lays it out: token t0 + (i & 15), expert e0 + 4 ((i & 63) / 16) + i / 64
__device__ __forceinline__ float router_tile(const MoeArgs& a, int e0, int t0, float (&red)[kWaves][256]) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, b = lane >> 4;
  const int e = e0 + r < a.E ? e0 + r : a.E - 1, t = t0 + r < a.T ? t0 + r : a.T - 1;
  const uint16_t* re = a.router + (int64_t)e * a.H;
  const uint16_t* xt = a.x + t * a.ldx;
  const int blocks = a.H >> 5;
  v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
  for (int s = wave; 4 * s < blocks; s += kWaves) {
    const bool in = 4 * s + b < blocks;
    const int at = 32 * (in ? 4 * s + b : 0);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v4i w = *(const v4i*)(re + at + 8 * q);
      if (!in) w = (v4i){0, 0, 0, 0};
      acc = mfma(w, *(const v4i*)(xt + at + 8 * q), acc);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) red[wave][i * 64 + lane] = acc[i];
  __syncthreads();
  float v = 0.0f;
  if (tid < 256) {
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += red[w][tid];
  }
  __syncthreads();
  return v;
}

__global__ __launch_bounds__(kWaves * 64) void moe_router_kernel(MoeArgs a) {
  __shared__ float red[kWaves][256];
  const int e0 = blockIdx.x * 16, t0 = blockIdx.y * 16, tid = threadIdx.x;
  const float v = router_tile(a, e0, t0, red);
  const int e = e0 + 4 * ((tid & 63) >> 4) + (tid >> 6), t = t0 + (tid & 15);
  if (tid < 256 && e < a.E && t < a.T) a.logits[t * a.E + e] = v;
}

// The routing of one token by one wave: lane l holds experts l, l + 64, ...
// Writes the token's choices and weights to LDS.
__device__ __forceinline__ void route_token(const MoeArgs& a, const float* logits, int32_t* ids, float* weights) {
  const int lane = threadIdx.x & 63;
  float v[4];
  uint32_t gone = 0;  // experts that are taken, or beyond E
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lane + 64 * i;
    v[i] = e < a.E ? logits[e] : -INFINITY;
    gone |= (uint32_t)(e >= a.E) << i;
    top = fmaxf(top, v[i]);
  }
  top = wave_max(top);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lane + 64 * i < a.E) sum += __builtin_amdgcn_exp2f((v[i] - top) * kLog2e);
  sum = wave_sum(sum);
  const bool broken = !(sum == sum);  // a NaN, or an infinity: no softmax
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
    ids[lane] = mine;
    weights[lane] = p;
  }
}

// ---- gate/up ----------------------------------------------------------------

struct GateSmem {
  float red[kWaves][256];  // shared by the router, one token group's partial sums follow
  int32_t ids[kMaxTokens * kMaxChoices];
  float weights[kMaxTokens * kMaxChoices];
  uint32_t mask[MXW_MAX_EXPERTS][2];
  int32_t expert[MXW_MAX_EXPERTS];
  int32_t first[MXW_MAX_EXPERTS];
  int32_t wsum[4], wpairs[4];
  int32_t token[kMaxTokens];
  float share[kMaxTokens];
};

// routing for the whole batch into LDS: every workgroup for itself
template <bool FUSED>
__device__ __forceinline__ int make_routing(const MoeArgs& a, GateSmem& sm, float* logits) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = a.T * a.k;
  if (a.router) {
    const float* from = a.logits;
    if (FUSED) {
      for (int t0 = 0; t0 < a.T; t0 += 16)
        for (int e0 = 0; e0 < a.E; e0 += 16) {
          const float v = router_tile(a, e0, t0, sm.red);
          const int e = e0 + 4 * (lane >> 4) + wave, t = t0 + (tid & 15);
          if (tid < 256 && e < a.E && t < a.T) logits[t * a.E + e] = v;
        }
      __syncthreads();
      from = logits;
    }
    for (int t = wave; t < a.T; t += kWaves) {
      if (a.active && !a.active[t]) {
        if (lane < a.k) {
          sm.ids[t * a.k + lane] = -1;
          sm.weights[t * a.k + lane] = 0.0f;
        }
      } else {
        route_token(a, from + t * a.E, sm.ids + t * a.k, sm.weights + t * a.k);
      }
    }
  } else {
    for (int i = tid; i < n; i += kWaves * 64) {
      const int id = a.ids[i];
      const bool in = id >= 0 && id < a.E && !(a.active && !a.active[i / a.k]);
      sm.ids[i] = in ? id : -1;
      sm.weights[i] = in ? a.weights[i] : 0.0f;
    }
  }
  for (int i = tid; i < 2 * MXW_MAX_EXPERTS; i += kWaves * 64) sm.mask[i >> 1][i & 1] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += kWaves * 64) {
    const int e = sm.ids[i], t = i / a.k;
    if (e >= 0) atomicOr(&sm.mask[e][t >> 5], 1u << (t & 31));
  }
  __syncthreads();
  // chosen experts in order, and their first rows of h: ranks by ballot, sums
  // over 4 waves of 64 experts
  int before = 0, rank = 0;
  bool chosen = false;
  if (wave < 4) {
    const int pairs = tid < a.E ? __popc(sm.mask[tid][0]) + __popc(sm.mask[tid][1]) : 0;
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
      sm.wsum[wave] = __popcll(votes);
      sm.wpairs[wave] = run;
    }
  }
  __syncthreads();
  if (chosen) {
    for (int w = 0; w < wave; ++w) {
      rank += sm.wsum[w];
      before += sm.wpairs[w];
    }
    sm.expert[rank] = tid;
    sm.first[rank] = before;
  }
  __syncthreads();
  const int count = sm.wsum[0] + sm.wsum[1] + sm.wsum[2] + sm.wsum[3];
  if (blockIdx.x == 0) {
    if (a.router)
      for (int i = tid; i < n; i += kWaves * 64) {
        a.ids[i] = sm.ids[i];
        a.weights[i] = sm.weights[i];
      }
    if (tid == 0) *a.count = count;
    for (int i = tid; i < count; i += kWaves * 64) {
      const int e = sm.expert[i];
      a.expert[i] = e;
      a.first[i] = sm.first[i];
      a.tokens[i] = sm.mask[e][0] | (uint64_t)sm.mask[e][1] << 32;
    }
  }
  return count;
}

// Items (expert, RG * 16 rows of Wg and the same of Wu), workgroups striding
// over them.
template <int RG, bool FUSED>
__global__ __launch_bounds__(kWaves * 64, 2 * kWaves / 4) void moe_gate_kernel(MoeArgs a) {
  __shared__ GateSmem sm;
  __shared__ float part[kWaves][2 * RG][256];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int count = make_routing<FUSED>(a, sm, &part[0][0][0]);
  const int tiles = (a.I + 16 * RG - 1) / (16 * RG);
  const int blocks = a.H >> 5;
  const int r = lane & 15, b = lane >> 4;
  for (int item = blockIdx.x; item < count * tiles; item += gridDim.x) {
    const int which = item / tiles, i0 = (item - which * tiles) * 16 * RG;
    const int e = sm.expert[which], first = sm.first[which];
    const uint64_t mask = sm.mask[e][0] | (uint64_t)sm.mask[e][1] << 32;
    const int ntok = __popcll(mask);
    __syncthreads();  // the last item is done with the lists
    if (wave == 0 && ((mask >> lane) & 1)) {
      const int at = __popcll(mask & ((1ull << lane) - 1));
      float share = 0.0f;
      for (int j = 0; j < a.k; ++j)
        if (sm.ids[lane * a.k + j] == e) share += sm.weights[lane * a.k + j];
      sm.token[at] = lane;
      sm.share[at] = share;
    }
    __syncthreads();
    const uint8_t* row[2 * RG];
    const uint8_t* srow[2 * RG];
#pragma unroll
    for (int g = 0; g < RG; ++g) {
      int i = i0 + 16 * g + r;
      if (i >= a.I) i = a.I - 1;  // past the last rows: computed, not stored
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int64_t at = (int64_t)e * 2 * a.I + u * a.I + i;
        row[2 * g + u] = a.wgu + at * a.H;
        srow[2 * g + u] = a.sgu + at * blocks;
      }
    }
    for (int g0 = 0; g0 < ntok; g0 += 16) {
      const uint16_t* xt = a.x + sm.token[g0 + r < ntok ? g0 + r : g0] * a.ldx;
      v4f acc[2 * RG];
#pragma unroll
      for (int g = 0; g < 2 * RG; ++g) acc[g] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
      for (int s = wave; 4 * s < blocks; s += kWaves) {
        const bool in = 4 * s + b < blocks;
        const int at = in ? 4 * s + b : 0;
        Codes c[2 * RG];
        v4i xv[4];
#pragma unroll
        for (int g = 0; g < 2 * RG; ++g) c[g] = load_codes(row[g], srow[g], at);
#pragma unroll
        for (int q = 0; q < 4; ++q) xv[q] = *(const v4i*)(xt + 32 * at + 8 * q);
        if (!in) {
#pragma unroll
          for (int g = 0; g < 2 * RG; ++g) c[g] = Codes{};
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int g = 0; g < 2 * RG; ++g) acc[g] = mfma(operand(c[g], q), xv[q], acc[g]);
      }
#pragma unroll
      for (int g = 0; g < 2 * RG; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[wave][g][(4 * b + i) * 16 + r] = acc[g][i];  // [row][token]
      __syncthreads();
      for (int i = tid; i < RG * 256; i += kWaves * 64) {
        const int tok = i / (16 * RG), rr = i % (16 * RG), g = rr >> 4, at = (rr & 15) * 16 + tok;
        float gate = 0.0f, up = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          gate += part[w][2 * g][at];
          up += part[w][2 * g + 1][at];
        }
        // silu(g) u w, rounded once to bf16, the down product's operand type
        const float h = gate / (1.0f + __builtin_amdgcn_exp2f(-gate * kLog2e)) * up * sm.share[g0 + tok < ntok ? g0 + tok : 0];
        if (g0 + tok < ntok && i0 + rr < a.I)
          a.h[(int64_t)(first + g0 + tok) * a.I + i0 + rr] = (uint16_t)pack2(h, 0.0f, __bf16());
      }
      __syncthreads();
    }
  }
}

// ---- down -------------------------------------------------------------------

// 16 output columns of all tokens: the waves split the (expert, 128 columns of
// I) units in order, each keeps its own sums [token][16] in LDS.
template <int WAVES>
__global__ __launch_bounds__(WAVES * 64, 4) void moe_down_kernel(MoeArgs a) {
  extern __shared__ __align__(16) float sums[];  // [WAVES][T][16]
  __shared__ int32_t expert[MXW_MAX_EXPERTS], first[MXW_MAX_EXPERTS];
  __shared__ uint64_t tokens[MXW_MAX_EXPERTS];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int count = *a.count;
  for (int i = tid; i < count; i += WAVES * 64) {
    expert[i] = a.expert[i];
    first[i] = a.first[i];
    tokens[i] = a.tokens[i];
  }
  float* mine = sums + wave * a.T * 16;
  for (int i = lane; i < a.T * 16; i += 64) mine[i] = 0.0f;
  __syncthreads();
  const int h0 = blockIdx.x * 16, r = lane & 15, b = lane >> 4;
  const int blocks = a.I >> 5, steps = (blocks + 3) >> 2, units = count * steps;
  int u = (int)((int64_t)units * wave / WAVES);
  const int end = (int)((int64_t)units * (wave + 1) / WAVES);
  while (u < end) {
    const int which = u / steps, s0 = u - which * steps;
    const int s1 = end - which * steps < steps ? end - which * steps : steps;
    const int e = expert[which], p0 = first[which];
    const uint64_t mask = tokens[which];
    const int ntok = __popcll(mask);
    const int64_t at = (int64_t)e * a.H + h0 + r;
    const uint8_t* row = a.wd + at * a.I;
    const uint8_t* srow = a.sd + at * blocks;
    for (int g0 = 0; g0 < ntok; g0 += 16) {
      const int p = g0 + r < ntok ? g0 + r : g0;
      const uint16_t* hp = a.h + (int64_t)(p0 + p) * a.I;
      v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
      for (int s = s0; s < s1; ++s) {
        const bool in = 4 * s + b < blocks;
        const int k = in ? 4 * s + b : 0;
        Codes c = load_codes(row, srow, k);
        if (!in) c = Codes{};
#pragma unroll
        for (int q = 0; q < 4; ++q) acc = mfma(operand(c, q), *(const v4i*)(hp + 32 * k + 8 * q), acc);
      }
      // token of this lane's column: the (g0 + r)-th set bit
      uint64_t left = mask;
      for (int i = 0; i < g0 + r && left; ++i) left &= left - 1;
      if (g0 + r < ntok) {
        v4f* to = (v4f*)(mine + (__ffsll((unsigned long long)left) - 1) * 16 + 4 * b);
        *to = *to + acc;
      }
    }
    u = which * steps + s1;
  }
  __syncthreads();
  for (int i = tid; i < a.T * 16; i += WAVES * 64) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v += sums[w * a.T * 16 + i];
    a.out[(int64_t)(i >> 4) * a.H + h0 + (i & 15)] = (uint16_t)pack2(v, 0.0f, __bf16());
  }
}

// ---- host -------------------------------------------------------------------

struct MoePlan {
  size_t logits, count, expert, first, tokens, h, bytes;
};

MoePlan plan_of(int T, int E, int k, int I) {
  MoePlan p = {};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at = (at + bytes + 255) & ~(size_t)255;
    return was;
  };
  p.logits = take((size_t)T * E * 4);
  p.count = take(4);
  p.expert = take(MXW_MAX_EXPERTS * 4);
  p.first = take(MXW_MAX_EXPERTS * 4);
  p.tokens = take(MXW_MAX_EXPERTS * 8);
  p.h = take((size_t)T * k * I * 2);
  p.bytes = at;
  return p;
}

int check_moe(int T, int E, int k, int H, int I) {
  return T < 1 || T > kMaxTokens || E < 1 || E > MXW_MAX_EXPERTS || k < 1 || k > kMaxChoices || k > E || H < 32 ||
                 H > 65536 || (H & 31) || I < 32 || I > 65536 || (I & 31)
             ? MXW_ERR_DIM
             : MXW_OK;
}

template <bool FUSED>
void launch_gate(const MoeArgs& a, int cus, hipStream_t st) {
  const int most = a.T * a.k < a.E ? a.T * a.k : a.E;  // experts that can be chosen
  // 16 rows of each half an item while that gives few items, else 32: half the
  // token loads per weight
  const int64_t items = (int64_t)most * ((a.I + 31) / 32);
  const int64_t slots = 2LL * cus;
  if (items < slots) {
    const int64_t n = (int64_t)most * ((a.I + 15) / 16);
    hipLaunchKernelGGL((moe_gate_kernel<1, FUSED>), dim3((unsigned)(n < slots ? n : slots)), dim3(kWaves * 64), 0, st, a);
  } else {
    hipLaunchKernelGGL((moe_gate_kernel<2, FUSED>), dim3((unsigned)slots), dim3(kWaves * 64), 0, st, a);
  }
}

}  // namespace

extern "C" {

int64_t mxw_moe_workspace_size(int T, int E, int k, int H, int I) {
  if (check_moe(T, E, k, H, I)) return MXW_ERR_DIM;
  return (int64_t)plan_of(T, E, k, I).bytes;
}

int mxw_moe_layer(const uint16_t* x, int64_t ldx, const uint16_t* router, const uint8_t* wgu, const uint8_t* sgu,
                  const uint8_t* wd, const uint8_t* sd, const uint8_t* active, int T, int E, int k, int H, int I,
                  int normalize, float scale, int32_t* ids, float* weights, uint16_t* out, void* workspace,
                  size_t workspace_bytes, void* stream) {
  if (!x || !wgu || !sgu || !wd || !sd || !ids || !weights || !out) return MXW_ERR_NULL;
  if (check_moe(T, E, k, H, I) || ldx < H || (ldx & 7)) return MXW_ERR_DIM;
  if ((((uintptr_t)x | (uintptr_t)router | (uintptr_t)wgu | (uintptr_t)wd) & 15) || ((uintptr_t)out & 1) ||
      (((uintptr_t)ids | (uintptr_t)weights) & 3))
    return MXW_ERR_ALIGN;
  const MoePlan p = plan_of(T, E, k, I);
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
  a.count = (int32_t*)(ws + p.count);
  a.expert = (int32_t*)(ws + p.expert);
  a.first = (int32_t*)(ws + p.first);
  a.tokens = (uint64_t*)(ws + p.tokens);
  a.h = (uint16_t*)(ws + p.h);
  if (router)
    hipLaunchKernelGGL(moe_router_kernel, dim3((unsigned)((E + 15) / 16), (unsigned)((T + 15) / 16)), dim3(kWaves * 64), 0,
                       st, a);
  launch_gate<false>(a, cus, st);
  hipLaunchKernelGGL((moe_down_kernel<16>), dim3((unsigned)(H / 16)), dim3(16 * 64), 16 * T * 16 * 4, st, a);
  if (hipGetLastError() != hipSuccess) return MXW_ERR_LAUNCH;
  return MXW_OK;
}

}  // extern "C"
