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
#include <type_traits>

#include "dropout.cuh"
#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

// A block of 8 elements a thread.  At 8192 x 4096 fp32 with an addend 403 MB in 59
// us, the measured copy rate and a little more.
template <typename T, bool ADD>
__global__ void __launch_bounds__(256)
    dropout_kernel(const T* x, const T* add, T* out, long long nblk, DropArgs d) {
  pdl_wait_and_release();
  const uint64_t offset = drop_offset(d);
  const long long b = (long long)blockIdx.x * 256 + threadIdx.x;
  if (b >= nblk) return;
  float v[8], a[8];
  load_row8(x + b * 8, v);
  if (ADD) load_row8(add + b * 8, a);
  const uint32_t keep = drop_keep8(d, offset, d.block0 + (uint64_t)b);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float w = (keep >> i) & 1u ? v[i] * d.scale : 0.f;
    v[i] = ADD ? a[i] + w : w;
  }
  store_row8(out + b * 8, v);
}

// The combine's two directions.  W warps of a CTA share a token (8 / W tokens
// a CTA; W by d_out, so that a warp has about four steps of 32 x 8 columns and
// the grid has enough CTAs to end evenly).  K = top_k rounded up to 1, 2, 4 or
// 8.  Up to 4 a token's rows and gates take K registers; the kept slots are
// gathered first, and KB rows are loaded before the first is used: 2 forward,
// with four CTAs an SM, and 4 backward, with three for K > 2.  At 8192 x 4096
// top-2 the forward moves its 402 MB in 68 us and the backward its 604 MB in 94
// (0.90 and 0.98 of the measured copy rate).  Above 4 slots, see the rings below.

// The kept slots of token t in order, nk of them, one a lane: lane i < nk holds the
// i-th one's grouped row, gate and slot number.
__device__ __forceinline__ int lane_slots(const int32_t* __restrict__ dest,
                                          const float* __restrict__ gates, int t, int k, int& row,
                                          float& gate, int& slot) {
  const int lane = threadIdx.x & 31;
  int d = -1;
  float g = 0.f;
  if (lane < k) {
    d = __ldg(dest + (size_t)t * k + lane);
    g = __ldg(gates + (size_t)t * k + lane);
  }
  const unsigned kept = __ballot_sync(0xffffffffu, d >= 0);
  slot = (int)__fns(kept, 0, lane + 1) & 31;
  row = __shfl_sync(0xffffffffu, d, slot);
  gate = __shfl_sync(0xffffffffu, g, slot);
  return __popc(kept);
}

// The same with every slot's grouped row and gate in every lane.
template <int K>
__device__ __forceinline__ int load_slots(const int32_t* __restrict__ dest,
                                          const float* __restrict__ gates, int t, int k,
                                          int (&dj)[K], float (&gj)[K], int& slot) {
  int row;
  float gate;
  const int nk = lane_slots(dest, gates, t, k, row, gate, slot);
#pragma unroll
  for (int j = 0; j < K; ++j) {
    dj[j] = __shfl_sync(0xffffffffu, row, j);
    gj[j] = __shfl_sync(0xffffffffu, gate, j);
  }
  return nk;
}

template <typename T, int K>
__global__ void __launch_bounds__(256, 4)
    combine_dropout_kernel(const float* __restrict__ y_perm, const int32_t* __restrict__ dest,
                           const float* __restrict__ gates, const T* residual, T* out, int rows,
                           int k, int d_out, int W, DropArgs d) {
  pdl_wait_and_release();
  constexpr int KB = K < 2 ? K : 2;
  const uint64_t offset = drop_offset(d);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * (8 / W) + warp / W;
  if (t >= rows) return;
  const int nvec = d_out / 8;
  int dj[K];
  float gj[K];
  int slot;
  const int nk = load_slots<K>(dest, gates, t, k, dj, gj, slot);
  const size_t row = (size_t)t * nvec;
  for (int v = warp % W * 32 + lane; v < nvec; v += 32 * W) {
    float r[8], acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = r[i] = 0.f;
    if (residual != nullptr) load_row8(residual + (row + v) * 8, r);
    uint32_t keep = 0;
#pragma unroll
    for (int j0 = 0; j0 < K; j0 += KB) {
      if (j0 > 0 && j0 >= nk) break;
      float y[KB][8];
#pragma unroll
      for (int j = 0; j < KB; ++j)
        if (j0 + j < nk)
          load_row8_stream(y_perm + ((size_t)dj[j0 + j] * nvec + v) * 8, y[j]);
      if (j0 == 0) keep = drop_keep8(d, offset, d.block0 + row + v);
#pragma unroll
      for (int j = 0; j < KB; ++j)
        if (j0 + j < nk) {
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] = fmaf(gj[j0 + j], y[j][i], acc[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = r[i] + ((keep >> i) & 1u ? acc[i] * d.scale : 0.f);
    store_row8(out + (row + v) * 8, acc);
  }
}

// A token's dgates from its lanes' partial sums: a fixed butterfly over the warp, the
// token's W warps in order; 0 for dropped slots.  By the whole CTA.
template <int K>
__device__ __forceinline__ void store_dgates(float (&part)[K], float (&red)[8][K],
                                             float* __restrict__ dgates, bool in, int t, int k,
                                             int W, int nk, int slot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int j = 0; j < K; ++j) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) part[j] += __shfl_xor_sync(0xffffffffu, part[j], o);
    if (lane == 0) red[warp][j] = part[j];
  }
  if (W > 1) __syncthreads();
  else __syncwarp();
  if (in && warp % W == 0) {
    if (lane < nk) {
      float v = red[warp][lane];
      for (int w = 1; w < W; ++w) v += red[warp + w][lane];
      dgates[(size_t)t * k + slot] = v;
    }
    // dropped slots
    const unsigned kept = __reduce_or_sync(0xffffffffu, lane < nk ? 1u << slot : 0u);
    if (lane < k && !(kept >> lane & 1u)) dgates[(size_t)t * k + lane] = 0.f;
  }
}

template <typename T, int K>
__global__ void __launch_bounds__(256, K <= 2 ? 4 : 3)
    combine_dropout_backward_kernel(const T* __restrict__ dy, const float* __restrict__ y_perm,
                                    const int32_t* __restrict__ dest,
                                    const float* __restrict__ gates, float* __restrict__ dy_perm,
                                    float* __restrict__ dgates, int rows, int k, int d_out, int W,
                                    DropArgs d) {
  pdl_wait_and_release();
  constexpr int KB = K < 4 ? K : 4;
  __shared__ float red[8][K];
  const uint64_t offset = drop_offset(d);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * (8 / W) + warp / W;
  const bool in = t < rows;
  const int nvec = d_out / 8;
  int dj[K];
  float gj[K], part[K];
  int slot = 0;
  const int nk = in ? load_slots<K>(dest, gates, t, k, dj, gj, slot) : 0;
#pragma unroll
  for (int j = 0; j < K; ++j) part[j] = 0.f;
  const size_t row = (size_t)t * nvec;
  for (int v = warp % W * 32 + lane; in && v < nvec; v += 32 * W) {
    float g8[8];
    load_row8(dy + (row + v) * 8, g8);
    uint32_t keep = 0;
#pragma unroll
    for (int j0 = 0; j0 < K; j0 += KB) {
      if (j0 > 0 && j0 >= nk) break;
      float y[KB][8];
#pragma unroll
      for (int j = 0; j < KB; ++j)
        if (j0 + j < nk)
          load_row8_stream(y_perm + ((size_t)dj[j0 + j] * nvec + v) * 8, y[j]);
      if (j0 == 0) {
        keep = drop_keep8(d, offset, d.block0 + row + v);
#pragma unroll
        for (int i = 0; i < 8; ++i) g8[i] = (keep >> i) & 1u ? g8[i] * d.scale : 0.f;
      }
#pragma unroll
      for (int j = 0; j < KB; ++j)
        if (j0 + j < nk) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if ((keep >> i) & 1u) part[j0 + j] = fmaf(g8[i], y[j][i], part[j0 + j]);
            y[j][i] = gj[j0 + j] * g8[i];
          }
          store_row8_stream(dy_perm + ((size_t)dj[j0 + j] * nvec + v) * 8, y[j]);
        }
    }
  }
  store_dgates<K>(part, red, dgates, in, t, k, W, nk, slot);
}

// Above 4 slots: the same sums in the same order, but a warp copies its pieces to
// shared memory in the order it needs them, across rows and columns, and 5 are on
// their way while it works on one (rows in registers: 2 or 4, and none across
// columns).  Both directions on B200, us (rings against registers): 5003 x 2056
// top-6 with 43% of the slots kept (379 MB) 83 / 93, with all kept 152 / 170; 8192
// x 1024 top-8 152 / 158; 64 x 2048 top-6 19.6 / 18.6; but top-3 of 4096 x 1536 62
// / 59, and top-1 of 4096 x 768 14.4 / 12.3.  With 1 warp a token 92 at 5003 x
// 2056, with 4 88, with 8 105; 8 pieces deep 86, 4 deep 85.

// A warp's pieces of 32 x 8 columns, in the order: for each of its columns
// v, v + step, ... (in vectors of 8) the addend's (if there is one), then the nk
// kept rows'.  All calls by the whole warp.
template <typename T>
struct Pieces {
  static constexpr int DEPTH = 6;
  static constexpr int kBytes = 1024;
  const T* aux;              // the token's row, or null
  const float* y;
  int row, nk, nvec, step;   // row: of the lane's kept slot
  int v, j;                  // the next piece to copy: columns, -1 (aux) or kept slot
  uint32_t ring;
  const uint8_t* at;
  int put, get;
  __device__ Pieces(const T* aux_, const float* y_, int row_, int nk_, int nvec_, int v0,
                    int step_, uint8_t* smem)
      : aux(aux_), y(y_), row(row_), nk(nk_), nvec(nvec_), step(step_), v(v0), put(0), get(0) {
    j = aux != nullptr ? -1 : 0;
    if (j == nk) v = nvec;   // no pieces at all
    ring = smem_u32(smem);
    at = smem;
#pragma unroll
    for (int i = 0; i < DEPTH - 1; ++i) copy();
  }
  __device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  }
  __device__ __forceinline__ void copy() {
    const int lane = threadIdx.x & 31;
    if (v < nvec) {
      const uint32_t dst = ring + (uint32_t)(put * kBytes + lane * 16);
      const int left = nvec - v;   // vectors of 8 columns from here
      if (j < 0 && sizeof(T) == 2) {
        if (lane < left) copy16(dst, aux + (size_t)(v + lane) * 8);
      } else {
        const int r = __shfl_sync(0xffffffffu, row, max(j, 0));
        const float* src = j < 0 ? reinterpret_cast<const float*>(aux) + (size_t)v * 8
                                 : y + ((size_t)r * nvec + v) * 8;
        if (lane < 2 * left) copy16(dst, src + lane * 4);
        if (lane + 32 < 2 * left) copy16(dst + 512, src + 128 + lane * 4);
      }
      if (++j == nk) {
        j = aux != nullptr ? -1 : 0;
        v += step;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    put = put + 1 == DEPTH ? 0 : put + 1;
  }
  // The next piece: this lane's 8 columns.
  template <typename U>
  __device__ __forceinline__ void next(float (&x)[8]) {
    asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 2) : "memory");
    __syncwarp();   // all lanes' copies; and the last piece has been read
    copy();
    const int lane = threadIdx.x & 31;
    load_row8(reinterpret_cast<const U*>(at + get * kBytes) + lane * 8, x);
    get = get + 1 == DEPTH ? 0 : get + 1;
  }
};

template <typename T, int K>
__global__ void __launch_bounds__(256, 4)
    combine_dropout_ring_kernel(const float* __restrict__ y_perm, const int32_t* __restrict__ dest,
                           const float* __restrict__ gates, const T* residual, T* out, int rows,
                           int k, int d_out, int W, DropArgs d) {
  pdl_wait_and_release();
  extern __shared__ __align__(16) uint8_t smem[];
  const uint64_t offset = drop_offset(d);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * (8 / W) + warp / W;
  if (t >= rows) return;
  const int nvec = d_out / 8;
  int row, slot;
  float gate;
  const int nk = lane_slots(dest, gates, t, k, row, gate, slot);
  const size_t first = (size_t)t * nvec;
  Pieces<T> in(residual != nullptr ? residual + first * 8 : nullptr, y_perm, row, nk, nvec,
               warp % W * 32, 32 * W, smem + warp * Pieces<T>::DEPTH * Pieces<T>::kBytes);
  for (int vb = warp % W * 32; vb < nvec; vb += 32 * W) {
    const int v = vb + lane;
    float r[8], acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = r[i] = 0.f;
    if (residual != nullptr) in.template next<T>(r);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      if (j >= nk) break;
      float y[8];
      in.template next<float>(y);
      const float g = __shfl_sync(0xffffffffu, gate, j);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(g, y[i], acc[i]);
    }
    if (v < nvec) {
      const uint32_t keep = drop_keep8(d, offset, d.block0 + first + v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = r[i] + ((keep >> i) & 1u ? acc[i] * d.scale : 0.f);
      store_row8(out + (first + v) * 8, acc);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <typename T, int K>
__global__ void __launch_bounds__(256, 3)
    combine_dropout_backward_ring_kernel(const T* __restrict__ dy, const float* __restrict__ y_perm,
                                    const int32_t* __restrict__ dest,
                                    const float* __restrict__ gates, float* __restrict__ dy_perm,
                                    float* __restrict__ dgates, int rows, int k, int d_out, int W,
                                    DropArgs d) {
  pdl_wait_and_release();
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float red[8][K];
  const uint64_t offset = drop_offset(d);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * (8 / W) + warp / W;
  const bool in_rows = t < rows;
  const int nvec = in_rows ? d_out / 8 : 0;
  int row = 0, slot = 0;
  float gate = 0.f, part[K];
  const int nk = in_rows ? lane_slots(dest, gates, t, k, row, gate, slot) : 0;
#pragma unroll
  for (int j = 0; j < K; ++j) part[j] = 0.f;
  const size_t first = (size_t)t * nvec;
  Pieces<T> in(dy + first * 8, y_perm, row, nk, nvec, warp % W * 32, 32 * W,
               smem + warp * Pieces<T>::DEPTH * Pieces<T>::kBytes);
  for (int vb = warp % W * 32; vb < nvec; vb += 32 * W) {
    const int v = vb + lane;
    float g8[8];
    in.template next<T>(g8);
    const uint32_t keep = drop_keep8(d, offset, d.block0 + first + v);
#pragma unroll
    for (int i = 0; i < 8; ++i) g8[i] = (keep >> i) & 1u ? g8[i] * d.scale : 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j) {
      if (j >= nk) break;
      float y[8];
      in.template next<float>(y);
      const float g = __shfl_sync(0xffffffffu, gate, j);
      const int r = __shfl_sync(0xffffffffu, row, j);
      if (v < nvec) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if ((keep >> i) & 1u) part[j] = fmaf(g8[i], y[i], part[j]);
          y[i] = g * g8[i];
        }
        store_row8_stream(dy_perm + ((size_t)r * nvec + v) * 8, y);
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  store_dgates<K>(part, red, dgates, in_rows, t, k, W, nk, slot);
}

template <typename T>
cudaError_t run_dropout(const void* x, const void* add, void* out, long long nblk,
                        const DropArgs& d, cudaStream_t s) {
  const T* xp = static_cast<const T*>(x);
  const T* ap = static_cast<const T*>(add);
  T* op = static_cast<T*>(out);
  const unsigned grid = (unsigned)((nblk + 255) / 256);
  if (add != nullptr)
    return launch_kernel(dropout_kernel<T, true>, grid, 256, 0, s, 0, xp, ap, op, nblk, d);
  return launch_kernel(dropout_kernel<T, false>, grid, 256, 0, s, 0, xp, ap, op, nblk, d);
}

}  // namespace

cudaError_t launch_dropout(long long rows, int width, bool bf16, const void* x, const void* add,
                           void* out, const DropArgs& d, cudaStream_t s) {
  const long long nblk = rows * (width / 8);
  if (nblk == 0) return cudaSuccess;
  return bf16 ? run_dropout<__nv_bfloat16>(x, add, out, nblk, d, s)
              : run_dropout<float>(x, add, out, nblk, d, s);
}

namespace {

// Calls f(K) with top_k rounded up to 1, 2, 4 or 8.
template <typename F>
cudaError_t by_slots(int k, F&& f) {
  using std::integral_constant;
  if (k == 1) return f(integral_constant<int, 1>{});
  if (k == 2) return f(integral_constant<int, 2>{});
  if (k <= 4) return f(integral_constant<int, 4>{});
  return f(integral_constant<int, 8>{});
}

// Bytes of a CTA's rings.
constexpr int kRing = 8 * Pieces<float>::DEPTH * Pieces<float>::kBytes;

// The forms for K slots: rings above 4.
template <typename T, int K>
auto forward_kernel() {
  if constexpr (K > 4) return combine_dropout_ring_kernel<T, K>;
  else return combine_dropout_kernel<T, K>;
}
template <typename T, int K>
auto backward_kernel() {
  if constexpr (K > 4) return combine_dropout_backward_ring_kernel<T, K>;
  else return combine_dropout_backward_kernel<T, K>;
}

// Warps a token: four steps of 256 columns each, as far as d_out gives them.
int token_warps(int d_out) { return d_out >= 8192 ? 8 : d_out >= 4096 ? 4 : d_out >= 2048 ? 2 : 1; }

}  // namespace

cudaError_t launch_combine_dropout(const moe_config_t& c, const float* y_perm, const int32_t* dest,
                                   const float* gates, const void* residual, void* out,
                                   const DropArgs& d, cudaStream_t s) {
  if (c.T == 0) return cudaSuccess;
  auto run = [&](auto* o) {
    using T = std::remove_pointer_t<decltype(o)>;
    const int W = token_warps(c.d_out);
    const int smem = c.top_k > 4 ? kRing : 0;
    return by_slots(c.top_k, [&](auto K) {
      const auto kern = forward_kernel<T, decltype(K)::value>();
      if (smem != 0) {
        const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), smem);
        if (e != cudaSuccess) return e;
      }
      return launch_kernel(kern, ceil_div(c.T, 8 / W), 256, smem, s, 0, y_perm, dest, gates,
                           static_cast<const T*>(residual), o, c.T, c.top_k, c.d_out, W, d);
    });
  };
  return c.act_dtype == MOE_BF16 ? run(static_cast<__nv_bfloat16*>(out))
                                 : run(static_cast<float*>(out));
}

cudaError_t launch_combine_dropout_backward(const moe_config_t& c, const void* dy,
                                            const float* y_perm, const int32_t* dest,
                                            const float* gates, float* dy_perm, float* dgates,
                                            const DropArgs& d, cudaStream_t s) {
  if (c.T == 0) return cudaSuccess;
  auto run = [&](auto* g) {
    using T = std::remove_pointer_t<decltype(g)>;
    const int W = token_warps(c.d_out);
    const int smem = c.top_k > 4 ? kRing : 0;
    return by_slots(c.top_k, [&](auto K) {
      const auto kern = backward_kernel<std::remove_const_t<T>, decltype(K)::value>();
      if (smem != 0) {
        const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), smem);
        if (e != cudaSuccess) return e;
      }
      return launch_kernel(kern, ceil_div(c.T, 8 / W), 256, smem, s, 0, g, y_perm, dest, gates,
                           dy_perm, dgates, c.T, c.top_k, c.d_out, W, d);
    });
  };
  return c.act_dtype == MOE_BF16 ? run(static_cast<const __nv_bfloat16*>(dy))
                                 : run(static_cast<const float*>(dy));
}

}  // namespace moe
