// grad_norm.hip -- the norm of many gradients together, and their clipping to it
// (mxw_clip_grads, declared in include/mxfp8_wgrad.h), for gfx950.
//
//     n = (sum g^2)^(1/2)  or  max |g|;      out = g min(1, max_norm / (n + eps))
//
// Two passes, since the factor is known only after the last gradient is read: bound by
// reading HBM twice and writing it once.  The first leaves a partial result for each
// workgroup, whose share of the tiles depends on the sizes alone; every workgroup of the
// second adds all partials in one order, so no launch stands between them and the bits
// are the same run to run (with more tensors than one launch takes, a workgroup adds the
// partials of all launches first).  Squares are summed in 64 bits: a product of two FP32 values
// neither overflows nor vanishes there (FP32 sums would, beyond 1.8e19 and below 1e-23; the
// 64-bit ones cost nothing: the norm alone reads 6.9 TB/s, what reading alone reaches).
//
// Measured: 12 gradients of 1.09e9 elements, bf16 and FP32 (2.5 GB), clipped to other tensors or
// in place 1,320 us: in it the norm's kernel 366 (6.9 TB/s), the scaling's 952 (5.3 TB/s read and
// written); the norm alone 370; 20 small ones 28 us, the two kernels 4 and 6 of them.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <vector>

#include "device.h"
#include "mx.h"
#include "mxfp8_wgrad.h"

namespace {

using namespace mxw;

constexpr int kTileVecs = 4, kTileElems = 256 * 8 * kTileVecs;  // elements of a tile
constexpr int kMost = 96;                                       // tensors of a launch (its arguments: 4 KiB at most)
constexpr int kBlocks = 2048;                                   // workgroups of a launch
constexpr int kHead = 256;                                      // bytes before the partials, all of them as one

struct Item {
  const void* g;
  void* out;
  int64_t n;
  int32_t first;  // its first tile
  int32_t f32;
};
struct NormArgs {
  Item item[kMost];
  double max_norm, eps;
  float* norm;
  double* part;     // this launch's (first pass), all (second)
  int32_t items, tiles, parts;
};
static_assert(sizeof(NormArgs) <= 4096, "a kernel's arguments");

__device__ __forceinline__ int item_of(const NormArgs& a, int tile) {
  int lo = 0, hi = a.items - 1;  // the last with first <= tile
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.item[mid].first <= tile)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ double join(double x, double y, bool top) {
  // largest: NaN wins
  return top ? (x > y || x != x ? x : y) : x + y;
}

template <bool TOP>
__device__ __forceinline__ double block_join(double v) {
  __shared__ double red[4];
  for (int d = 32; d; d >>= 1) v = join(v, __shfl_xor(v, d), TOP);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return join(join(red[0], red[1], TOP), join(red[2], red[3], TOP), TOP);
}

template <bool TOP, bool F32, bool NT>
__device__ __forceinline__ double tile_norm(const Item& it, int64_t at) {
  double sum[2] = {0.0, 0.0};
  uint32_t top = 0;
  Raw8<F32> v[kTileVecs];
#pragma unroll
  for (int u = 0; u < kTileVecs; ++u) {
    const int64_t i = at + (u * 256 + (int)threadIdx.x) * 8;
    v[u] = Raw8<F32>{};
    if (i + 8 <= it.n)
      v[u] = load8<F32, NT>(it.g, i);
    else if (i < it.n)
      v[u] = load_some<F32>(it.g, i, (int)(it.n - i));
  }
#pragma unroll
  for (int u = 0; u < kTileVecs; ++u) {
    float f[8];
    values<F32>(v[u], f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (TOP)
        top = max(top, __float_as_uint(f[i]) & 0x7FFFFFFFu);
      else
        sum[i & 1] = fma((double)f[i], (double)f[i], sum[i & 1]);
    }
  }
  return TOP ? (double)__uint_as_float(top) : sum[0] + sum[1];
}

template <bool TOP, bool NT>
__global__ __launch_bounds__(256) void norm_kernel(NormArgs a) {
  double v = 0.0;
  for (int tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
    const Item& it = a.item[item_of(a, tile)];
    const int64_t at = (int64_t)(tile - it.first) * kTileElems;
    v = join(v, it.f32 ? tile_norm<TOP, true, NT>(it, at) : tile_norm<TOP, false, NT>(it, at), TOP);
  }
  v = block_join<TOP>(v);
  if (threadIdx.x == 0) a.part[blockIdx.x] = v;
}

template <bool F32, bool NT>
__device__ __forceinline__ void tile_scale(const Item& it, int64_t at, float power, float factor) {
  Raw8<F32> v[kTileVecs];
#pragma unroll
  for (int u = 0; u < kTileVecs; ++u) {
    const int64_t i = at + (u * 256 + (int)threadIdx.x) * 8;
    if (i + 8 <= it.n)
      v[u] = load8<F32, NT>(it.g, i);
    else if (i < it.n)
      v[u] = load_some<F32>(it.g, i, (int)(it.n - i));
  }
#pragma unroll
  for (int u = 0; u < kTileVecs; ++u) {
    const int64_t i = at + (u * 256 + (int)threadIdx.x) * 8;
    if (i >= it.n) continue;
    float f[8];
    values<F32>(v[u], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = f[j] * power * factor;
    if (i + 8 <= it.n)
      store8<F32, NT>(it.out, i, rounded<F32>(f));
    else
      store_some<F32>(it.out, i, rounded<F32>(f), (int)(it.n - i));
  }
}

// All partials as one.
template <bool TOP>
__global__ __launch_bounds__(256) void join_kernel(const double* part, int parts, double* to) {
  double v = 0.0;
  for (int i = threadIdx.x; i < parts; i += 256) v = join(v, part[i], TOP);
  v = block_join<TOP>(v);
  if (threadIdx.x == 0) *to = v;
}

// The norm from all partials, and this launch's tensors times the factor.
template <bool TOP, bool NT>
__global__ __launch_bounds__(256) void scale_kernel(NormArgs a) {
  double v = 0.0;
  for (int i = threadIdx.x; i < a.parts; i += 256) v = join(v, a.part[i], TOP);
  v = block_join<TOP>(v);
  const double norm = TOP ? v : sqrt(v);
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.norm) *a.norm = (float)norm;
  const double over = norm + a.eps;
  const double ratio = over == 0.0 ? 1.0 : a.max_norm / over;   // 0: zeros, which any factor keeps
  // a factor below FP32's normal range goes as two, so that it keeps its 24 bits
  const bool low = ratio < 0x1p-126;
  const float power = low ? 0x1p-126f : 1.0f;
  const float factor = ratio >= 1.0 ? 1.0f : (float)(low ? ratio * 0x1p126 : ratio);  // NaN: NaN
  for (int tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
    const Item& it = a.item[item_of(a, tile)];
    if (!low && factor == 1.0f && it.g == it.out) continue;  // low: a rest that rounds to 1 still stands beside 2^-126
    const int64_t at = (int64_t)(tile - it.first) * kTileElems;
    if (it.f32)
      tile_scale<true, NT>(it, at, power, factor);
    else
      tile_scale<false, NT>(it, at, power, factor);
  }
}

int64_t tiles_of(int64_t n) { return (n + kTileElems - 1) / kTileElems; }

}  // namespace

extern "C" {

int64_t mxw_clip_workspace_size(int count) {
  if (count < 0 || count > MXW_MAX_TENSORS) return MXW_ERR_DIM;
  return kHead + (int64_t)((count + kMost - 1) / kMost + (count == 0)) * kBlocks * 8;
}

int mxw_clip_grads(const void* const* grads, void* const* outs, const int64_t* sizes, const int32_t* types, int count,
                   int norm_type, double max_norm, double eps, float* norm, void* workspace, size_t workspace_bytes,
                   void* stream) {
  if (!norm || (count && (!grads || !sizes || !types))) return MXW_ERR_NULL;
  const int64_t need = mxw_clip_workspace_size(count);
  if (need < 0 || (norm_type != MXW_NORM_2 && norm_type != MXW_NORM_MAX)) return MXW_ERR_DIM;
  if (outs && (!(max_norm >= 0.0) || !(eps >= 0.0))) return MXW_ERR_DIM;
  if ((uintptr_t)norm & 3) return MXW_ERR_ALIGN;
  int64_t tiles = 0, bytes = 0;
  for (int i = 0; i < count; ++i) {
    if (sizes[i] < 0 || sizes[i] > ((int64_t)1 << 40) || (types[i] != MXW_BF16 && types[i] != MXW_F32)) return MXW_ERR_DIM;
    if (sizes[i] == 0) continue;
    if (!grads[i] || (outs && !outs[i])) return MXW_ERR_NULL;
    const uintptr_t mask = types[i] == MXW_F32 ? 3 : 1;
    if (((uintptr_t)grads[i] | (outs ? (uintptr_t)outs[i] : 0)) & mask) return MXW_ERR_ALIGN;
    tiles += tiles_of(sizes[i]);
    bytes += sizes[i] * (types[i] == MXW_F32 ? 4 : 2);
  }
  // Loads and stores past the caches where those (256 MB) do not keep the gradients from one
  // pass to the other: 2.5 GB clipped in 1.31 to 1.34 ms, with cached ones 1.38 (the norm alone
  // 366 us, 415); below that the scaled gradients stay for whoever reads them next.
  const bool nt = bytes > ((int64_t)256 << 20);
  if (tiles > 0x7FFFFFFF - kBlocks) return MXW_ERR_DIM;  // a workgroup counts up to kBlocks past them
  if (outs && count) {  // what is written overlaps nothing but the gradient it comes from, at the same place
    struct Range {
      uintptr_t lo, hi;
      bool written;
    };
    std::vector<Range> r;
    try {
      r.reserve(2 * (size_t)count);
    } catch (...) {
      return MXW_ERR_LAUNCH;
    }
    for (int i = 0; i < count; ++i) {
      const uintptr_t bytes = (uintptr_t)sizes[i] * (types[i] == MXW_F32 ? 4 : 2);
      if (!bytes) continue;
      r.push_back({(uintptr_t)outs[i], (uintptr_t)outs[i] + bytes, true});
      if (grads[i] != outs[i]) r.push_back({(uintptr_t)grads[i], (uintptr_t)grads[i] + bytes, false});
    }
    std::sort(r.begin(), r.end(), [](const Range& x, const Range& y) { return x.lo < y.lo; });
    uintptr_t written = 0, read = 0;  // where what began before ends
    for (const Range& x : r) {
      if (x.lo < written || (x.written && x.lo < read)) return MXW_ERR_OVERLAP;
      (x.written ? written : read) = std::max(x.written ? written : read, x.hi);
    }
  }
  if (!workspace || ((uintptr_t)workspace & 255) || workspace_bytes < (size_t)need) return MXW_ERR_WORKSPACE;
  // the norm and the workspace are written too, while the gradients are still read
  const Span writes[2] = {{norm, 4}, {workspace, need}};
  if (overlap<2>(writes, 2)) return MXW_ERR_OVERLAP;
  for (int i = 0; i < count; ++i) {
    const int64_t size = sizes[i] * (types[i] == MXW_F32 ? 4 : 2);
    if (overlap<4>({writes[0], writes[1], {grads[i], size}, {outs ? outs[i] : nullptr, size}}, 2)) return MXW_ERR_OVERLAP;
  }
  if (const int rc = check_device()) return rc;
  hipStream_t st = (hipStream_t)stream;
  const bool top = norm_type == MXW_NORM_MAX;
  double* const partials = (double*)((char*)workspace + kHead);
  int parts = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int i = 0;
    bool any = false;
    do {
      NormArgs a = {};
      a.max_norm = max_norm, a.eps = eps;
      for (; i < count && a.items < kMost; ++i) {
        if (sizes[i] == 0) continue;
        a.item[a.items++] = {grads[i], outs ? outs[i] : nullptr, sizes[i], a.tiles, types[i] == MXW_F32};
        a.tiles += (int32_t)tiles_of(sizes[i]);
      }
      const int blocks = std::min(a.tiles, kBlocks);
      if (pass == 0) {
        a.part = partials + parts;
        if (blocks) {
          if (top)
            nt ? norm_kernel<true, true><<<dim3(blocks), dim3(256), 0, st>>>(a)
               : norm_kernel<true, false><<<dim3(blocks), dim3(256), 0, st>>>(a);
          else
            nt ? norm_kernel<false, true><<<dim3(blocks), dim3(256), 0, st>>>(a)
               : norm_kernel<false, false><<<dim3(blocks), dim3(256), 0, st>>>(a);
        }
        parts += blocks;
      } else {
        const bool joined = count > kMost;
        if (joined && !any) {
          if (top)
            join_kernel<true><<<dim3(1), dim3(256), 0, st>>>(partials, parts, (double*)workspace);
          else
            join_kernel<false><<<dim3(1), dim3(256), 0, st>>>(partials, parts, (double*)workspace);
        }
        a.part = joined ? (double*)workspace : partials, a.parts = joined ? 1 : parts;
        a.norm = any ? nullptr : norm;
        if (!outs) a.tiles = 0, i = count;  // the norm alone
        const int run = outs ? std::max(blocks, 1) : 1;
        if (top)
          nt ? scale_kernel<true, true><<<dim3(run), dim3(256), 0, st>>>(a)
             : scale_kernel<true, false><<<dim3(run), dim3(256), 0, st>>>(a);
        else
          nt ? scale_kernel<false, true><<<dim3(run), dim3(256), 0, st>>>(a)
             : scale_kernel<false, false><<<dim3(run), dim3(256), 0, st>>>(a);
        any = true;
      }
    } while (i < count);
  }
  return hipGetLastError() == hipSuccess ? MXW_OK : MXW_ERR_LAUNCH;
}

}  // extern "C"
