// dropout.cuh - the counter-based dropout mask shared by the dropout kernel
// and the combine's two directions.
//
// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", SC 2011).  Block b of 8 consecutive elements of a
// row-major (rows, width) tensor, width a multiple of 8, takes the counter
// (b low, b high, offset low, offset high) under the key (seed low, seed
// high); element i of the block takes 16 of the 128 bits, the low half of
// word i / 2 for even i and the high half for odd i, and is kept where they
// are at least thr = round(65536 p).  16 bits an element make one generator
// call serve a 16-byte vector of bf16: about 6 integer instructions an
// element, which hide behind the HBM traffic; 32 bits would double that and
// lose the overlap.  The mask is a function of the position alone, so the
// backward draws it again and nothing is stored.
#pragma once

#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {

__device__ __forceinline__ uint4 philox4x32_10(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint32_t h0 = __umulhi(0xD2511F53u, c.x), l0 = 0xD2511F53u * c.x;
    const uint32_t h1 = __umulhi(0xCD9E8D57u, c.z), l1 = 0xCD9E8D57u * c.z;
    c = make_uint4(h1 ^ c.y ^ k0, l1, h0 ^ c.w ^ k1, l0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

// The stream offset: the value plus the device word, if one is given.
__device__ __forceinline__ uint64_t drop_offset(const DropArgs& d) {
  return d.offset + (d.offset_dev != nullptr ? __ldg(d.offset_dev) : 0ull);
}

// The 8 elements' keep bits of block b (bit i: element i).
__device__ __forceinline__ uint32_t drop_keep8(const DropArgs& d, uint64_t offset, uint64_t b) {
  if (d.thr == 0) return 0xFFu;
  const uint4 w = philox4x32_10(make_uint4((uint32_t)b, (uint32_t)(b >> 32), (uint32_t)offset,
                                           (uint32_t)(offset >> 32)),
                                (uint32_t)d.seed, (uint32_t)(d.seed >> 32));
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
  uint32_t keep = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    keep |= ((v[i] & 0xFFFFu) >= d.thr ? 1u : 0u) << (2 * i);
    keep |= ((v[i] >> 16) >= d.thr ? 1u : 0u) << (2 * i + 1);
  }
  return keep;
}

// 8 elements as fp32, and back with one rounding.  Plain loads: the output
// may be one of the inputs.
__device__ __forceinline__ void load_row8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 q = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load_row8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store_row8(__nv_bfloat16* p, const float (&a)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
                                            pack_bf16x2(a[4], a[5]), pack_bf16x2(a[6], a[7]));
}
__device__ __forceinline__ void store_row8(float* p, const float (&a)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(a[0], a[1], a[2], a[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(a[4], a[5], a[6], a[7]);
}

// fp32 rows read once and written once: past L1, and the first to leave L2.
__device__ __forceinline__ void load_row8_stream(const float* p, float (&v)[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
  const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store_row8_stream(float* p, const float (&a)[8]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(a[0], a[1], a[2], a[3]));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(a[4], a[5], a[6], a[7]));
}

}  // namespace moe
