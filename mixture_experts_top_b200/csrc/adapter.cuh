// adapter.cuh - what the adapters' kernels share: copies into swizzled tiles,
// the split of fp32 values into bf16 terms, and the low-rank products'
// arguments.
#pragma once

#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;   // 0: the 16 bytes are filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Arrives on `bar` when this thread's copies so far have landed (one of the
// barrier's counted arrivals).  The tensor core's reads (async proxy) of what
// they wrote come after the waiting thread's proxy fence: a fence in the
// copying thread would wait for all its copies in flight.
__device__ __forceinline__ void cp_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Byte offset of 16-byte piece c of row `row` in a tile of CPR pieces a row
// (a power of two): the 8 rows a matrix load reads fall on distinct banks.
template <int CPR>
__device__ __forceinline__ uint32_t tile_at(int row, int c) {
  constexpr int kPer = CPR >= 8 ? 1 : 8 / CPR;   // rows in 128 bytes
  const int sw = (row / kPer) & (CPR >= 8 ? 7 : CPR - 1);
  return (uint32_t)(row * CPR + (c ^ sw)) * 16u;
}

// Four values as a sum of N bf16 terms each: t[i] holds the four i-th terms.
template <int N>
__device__ __forceinline__ void split4(const float (&v)[4], uint2 (&t)[N]) {
  float a = v[0], b = v[1], c = v[2], d = v[3];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    t[i] = make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
    a -= __uint_as_float(t[i].x << 16);
    b -= __uint_as_float(t[i].x & 0xFFFF0000u);
    c -= __uint_as_float(t[i].y << 16);
    d -= __uint_as_float(t[i].y & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void st_cluster_v2(uint32_t addr, uint2 v) {
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(v.x), "r"(v.y)
               : "memory");
}

// tcgen05.mma and its commit, issued by one elected lane of a warp that runs
// its loop converged: the descriptors then stay in uniform registers.  With A
// in shared memory an MMA of M = 128, K = 16 takes 40 cycles for N = 16, 49 for
// 64, 65 for 128 and 129 for 256, measured: A's read is its floor.
__device__ __forceinline__ void umma_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// n of a barrier's counted arrivals.
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n)
               : "memory");
}
// 1 in one lane of a converged warp.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(e));
  return e;
}
// A in tensor memory: lane = row, a 32-bit column = two neighbouring k.  By one
// lane.
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// This warp's 32 lanes, 4 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_st_32x32b_x4(uint32_t taddr, uint32_t a, uint32_t b,
                                                  uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void umma_commit_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(
          smem_u32(bar))
      : "memory");
}

// The two products of every row tile (AdapterCall) as the kernels take them.
struct LowRankArgs {
  const __nv_bfloat16* in;    // (T, K)
  const __nv_bfloat16* W1;    // per adapter: forward A (K, r), backward B (r, K)
  const __nv_bfloat16* W2;    // per adapter: forward B (r, N), backward A (N, r)
  const float* scale;
  const void* base;           // (T, N), bf16 forward, fp32 backward; null (0) or out
  void* out;                  // (T, N)
  float* u;                   // forward: (T, r) out or null; backward: the forward's
  // backward: u's and v's three bf16 terms out, (tile slots x tile rows, 3, r),
  // zeros in a tile's rows behind its last
  __nv_bfloat16* up;
  __nv_bfloat16* vp;
  const int32_t* header;
  const int32_t* rows;
  const int2* tiles;
  int32_t* err;
  int T, n, r, K, N;
};

// A bf16 tensor (outer, rows, cols) as a tensor map with a box of box_rows x
// 64 columns (128 bytes: the swizzle's width); columns, rows and outer indices
// outside read as zeros.
inline bool encode_bf16(CUtensorMap* m, const void* ptr, uint64_t outer, uint64_t rows,
                        uint64_t cols, uint32_t box_rows) {
  if (tensor_map_encoder() == nullptr) return false;
  const cuuint64_t dims[3] = {cols, rows, outer};
  const cuuint64_t strides[2] = {cols * 2, rows * cols * 2};
  const cuuint32_t box[3] = {64, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return tensor_map_encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims,
                              strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Low-rank products on tcgen05 (adapter_tc.cu) for tiles of 64 rows.
cudaError_t launch_low_rank_tc(const LowRankArgs& g, bool backward, int tiles, cudaStream_t s);

}  // namespace moe
