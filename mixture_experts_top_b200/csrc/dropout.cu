// dropout.cu - dropout with a counter-based mask that is never stored, alone
// and in the combine's two directions.
//
//   dropout:  out = add + keep * x / (1 - p)            (its own gradient:
//             the same call on dout)
//   combine:  out[t] = residual[t] + keep[t] / (1 - p) * sum_j g_tj Y[dest[t,j]]
//   backward: D = keep * dy / (1 - p);  dY[dest[t,j]] = g_tj D[t],
//             dg_tj = <D[t], Y[dest[t,j]]>     (the residual's gradient is dy)
//
// The mask is dropout.cuh's; p counts in steps of 2^-16 and 1 / (1 - p) uses
// the rounded p.  A dropped element is selected away, never multiplied by 0,
// so Inf and NaN in dropped places do not spread.  The combine's sums and
// orders are those of combine.cu and backward.cu: "Mixture-of-Experts Routing
// - LLM Internals" (mlgrind.dev), Algorithm 3.  fp32 throughout, one rounding
// to the layer's dtype; all three are bound by HBM.
#include "dropout.cuh"
#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

// Block b of 8 elements: thread-strided, U blocks a thread with all their
// loads issued first.
template <typename T, int U, bool ADD>
__global__ void __launch_bounds__(256)
    dropout_kernel(const T* x, const T* add, T* out, long long nblk, DropArgs d) {
  pdl_wait_and_release();
  const uint64_t offset = drop_offset(d);
  const long long b0 = (long long)blockIdx.x * (256 * U) + threadIdx.x;
  float v[U][8], a[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long b = b0 + 256 * u;
    if (b < nblk) {
      load_row8(x + b * 8, v[u]);
      if (ADD) load_row8(add + b * 8, a[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long b = b0 + 256 * u;
    if (b >= nblk) break;
    const uint32_t keep = drop_keep8(d, offset, d.block0 + (uint64_t)b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float w = (keep >> i) & 1u ? v[u][i] * d.scale : 0.f;
      v[u][i] = ADD ? a[u][i] + w : w;
    }
    store_row8(out + b * 8, v[u]);
  }
}

// One warp per token, 8 columns a lane step; a dropped slot adds nothing.
template <typename T>
__global__ void __launch_bounds__(256)
    combine_dropout_kernel(const float* __restrict__ y_perm, const int32_t* __restrict__ dest,
                           const float* __restrict__ gates, const T* residual, T* out, int rows,
                           int k, int d_out, DropArgs d) {
  pdl_wait_and_release();
  const uint64_t offset = drop_offset(d);
  const int lane = threadIdx.x & 31;
  const int gw = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int nw = (gridDim.x * blockDim.x) >> 5;
  const int nvec = d_out / 8;
  for (int t = gw; t < rows; t += nw) {
    int dl = -1;
    float gl = 0.f;
    if (lane < k) {
      dl = dest[(size_t)t * k + lane];
      gl = gates[(size_t)t * k + lane];
    }
    int dj[8];
    float gj[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dj[j] = __shfl_sync(0xffffffffu, dl, j);
      gj[j] = __shfl_sync(0xffffffffu, gl, j);
    }
    const uint64_t blk = d.block0 + (uint64_t)t * nvec;
#pragma unroll 2
    for (int v = lane; v < nvec; v += 32) {
      float acc[8], r[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = r[i] = 0.f;
      if (residual != nullptr) load_row8(residual + ((size_t)t * nvec + v) * 8, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j < k && dj[j] >= 0) {
          const float4* src = reinterpret_cast<const float4*>(y_perm + (size_t)dj[j] * d_out) + 2 * v;
          const float4 a = __ldg(src), b = __ldg(src + 1);
          acc[0] = fmaf(gj[j], a.x, acc[0]);
          acc[1] = fmaf(gj[j], a.y, acc[1]);
          acc[2] = fmaf(gj[j], a.z, acc[2]);
          acc[3] = fmaf(gj[j], a.w, acc[3]);
          acc[4] = fmaf(gj[j], b.x, acc[4]);
          acc[5] = fmaf(gj[j], b.y, acc[5]);
          acc[6] = fmaf(gj[j], b.z, acc[6]);
          acc[7] = fmaf(gj[j], b.w, acc[7]);
        }
      }
      const uint32_t keep = drop_keep8(d, offset, blk + v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = r[i] + ((keep >> i) & 1u ? acc[i] * d.scale : 0.f);
      store_row8(out + ((size_t)t * nvec + v) * 8, acc);
    }
  }
}

// One warp per token; dgates as in backward.cu: per lane in column order,
// then a fixed butterfly over the warp.
template <typename T>
__global__ void __launch_bounds__(256)
    combine_dropout_backward_kernel(const T* __restrict__ dy, const float* __restrict__ y_perm,
                                    const int32_t* __restrict__ dest,
                                    const float* __restrict__ gates, float* __restrict__ dy_perm,
                                    float* __restrict__ dgates, int rows, int k, int d_out,
                                    DropArgs d) {
  pdl_wait_and_release();
  const uint64_t offset = drop_offset(d);
  const int lane = threadIdx.x & 31;
  const int gw = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int nw = (gridDim.x * blockDim.x) >> 5;
  const int nvec = d_out / 8;
  for (int t = gw; t < rows; t += nw) {
    int dl = -1;
    float gl = 0.f;
    if (lane < k) {
      dl = dest[(size_t)t * k + lane];
      gl = gates[(size_t)t * k + lane];
    }
    int dj[8];
    float gj[8], part[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dj[j] = __shfl_sync(0xffffffffu, dl, j);
      gj[j] = __shfl_sync(0xffffffffu, gl, j);
      part[j] = 0.f;
    }
    const uint64_t blk = d.block0 + (uint64_t)t * nvec;
    for (int v = lane; v < nvec; v += 32) {
      float g8[8];
      load_row8(dy + ((size_t)t * nvec + v) * 8, g8);
      const uint32_t keep = drop_keep8(d, offset, blk + v);
#pragma unroll
      for (int i = 0; i < 8; ++i) g8[i] = (keep >> i) & 1u ? g8[i] * d.scale : 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j < k && dj[j] >= 0) {
          float y8[8];
          load_row8(y_perm + (size_t)dj[j] * d_out + (size_t)v * 8, y8);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if ((keep >> i) & 1u) part[j] = fmaf(g8[i], y8[i], part[j]);
          float4* o = reinterpret_cast<float4*>(dy_perm + (size_t)dj[j] * d_out + (size_t)v * 8);
          o[0] = make_float4(gj[j] * g8[0], gj[j] * g8[1], gj[j] * g8[2], gj[j] * g8[3]);
          o[1] = make_float4(gj[j] * g8[4], gj[j] * g8[5], gj[j] * g8[6], gj[j] * g8[7]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) part[j] += __shfl_xor_sync(0xffffffffu, part[j], o);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < k && lane == j) dgates[(size_t)t * k + j] = dj[j] >= 0 ? part[j] : 0.f;
  }
}

template <typename T>
cudaError_t run_dropout(const void* x, const void* add, void* out, long long nblk,
                        const DropArgs& d, cudaStream_t s) {
  const T* xp = static_cast<const T*>(x);
  const T* ap = static_cast<const T*>(add);
  T* op = static_cast<T*>(out);
  const unsigned grid = (unsigned)((nblk + 255) / 256);
  if (add != nullptr)
    return launch_kernel(dropout_kernel<T, 1, true>, grid, 256, 0, s, 0, xp, ap, op, nblk, d);
  return launch_kernel(dropout_kernel<T, 1, false>, grid, 256, 0, s, 0, xp, ap, op, nblk, d);
}

}  // namespace

cudaError_t launch_dropout(long long rows, int width, bool bf16, const void* x, const void* add,
                           void* out, const DropArgs& d, cudaStream_t s) {
  const long long nblk = rows * (width / 8);
  if (nblk == 0) return cudaSuccess;
  return bf16 ? run_dropout<__nv_bfloat16>(x, add, out, nblk, d, s)
              : run_dropout<float>(x, add, out, nblk, d, s);
}

cudaError_t launch_combine_dropout(const moe_config_t& c, const float* y_perm, const int32_t* dest,
                                   const float* gates, const void* residual, void* out,
                                   const DropArgs& d, cudaStream_t s) {
  if (c.T == 0) return cudaSuccess;
  const int blocks = std::min(ceil_div(c.T, 8), device_sm_count() * 16);
  if (c.act_dtype == MOE_BF16)
    return launch_kernel(combine_dropout_kernel<__nv_bfloat16>, blocks, 256, 0, s, 0, y_perm, dest,
                         gates, static_cast<const __nv_bfloat16*>(residual),
                         static_cast<__nv_bfloat16*>(out), c.T, c.top_k, c.d_out, d);
  return launch_kernel(combine_dropout_kernel<float>, blocks, 256, 0, s, 0, y_perm, dest, gates,
                       static_cast<const float*>(residual), static_cast<float*>(out), c.T, c.top_k,
                       c.d_out, d);
}

cudaError_t launch_combine_dropout_backward(const moe_config_t& c, const void* dy,
                                            const float* y_perm, const int32_t* dest,
                                            const float* gates, float* dy_perm, float* dgates,
                                            const DropArgs& d, cudaStream_t s) {
  if (c.T == 0) return cudaSuccess;
  const int blocks = std::min(ceil_div(c.T, 8), device_sm_count() * 16);
  if (c.act_dtype == MOE_BF16)
    return launch_kernel(combine_dropout_backward_kernel<__nv_bfloat16>, blocks, 256, 0, s, 0,
                         static_cast<const __nv_bfloat16*>(dy), y_perm, dest, gates, dy_perm,
                         dgates, c.T, c.top_k, c.d_out, d);
  return launch_kernel(combine_dropout_backward_kernel<float>, blocks, 256, 0, s, 0,
                       static_cast<const float*>(dy), y_perm, dest, gates, dy_perm, dgates, c.T,
                       c.top_k, c.d_out, d);
}

}  // namespace moe
