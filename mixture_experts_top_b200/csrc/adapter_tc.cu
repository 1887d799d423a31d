// adapter_tc.cu - the adapters' two low-rank products on tcgen05, for batches
// of many rows (adapter.cu has the formulas, the plan and the other forms).
//
// One CTA per tile of 64 rows of one adapter, both products in one launch:
//   D1 (64, r)  = in[rows, :] W1         input columns 64 at a time
//   u           = scale D1, split into bf16 terms, written to shared memory
//   D2 (64, 64) = sum over the terms of u_w W2[:, 64 columns]; out = base + D2
// Warps 2, 3, 6, 7 gather the rows and load the weights by cp.async, input
// columns first and then base's, through ONE ring of stages: while u is formed
// the second product's loads are already in flight, so HBM never waits.  Warp
// 8 issues the MMAs (M = 128: the upper 64 rows read whatever follows in
// shared memory and are never looked at).  Warps 0, 1, 4, 5 own the tensor
// memory's lanes 0-63 (two halves of the columns each): they add D1's blocks
// of 512 input columns in round-to-nearest fp32 (the tensor core's own sums
// truncate), and write D2 through the stage's base tile, so that every global
// access of a warp covers whole sectors.
// Bound by HBM: 2 (K + 2 N) bytes a row forward, 2 K + 8 N backward.
// Every wait is bounded (moe_device.cuh) and recorded on the error word.
#include "adapter.cuh"
#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kTm = 64;             // rows of a tile
constexpr int kBlk = kTm * 128;     // 64 rows of 64 bf16 columns: 8 KiB
constexpr int kKc = 128;            // input columns a stage
// Warps: those with warp % 4 in {0, 1} (tensor memory's lanes 0-63) are the
// epilogue, four to a group: 12 of them.  Of the others 8 load rows, one issues
// the MMAs, one loads the weights and two idle.
constexpr int kGroups = 3;
constexpr int kThreads = 32 * 8 * kGroups;
constexpr int kProducers = 256;     // threads of the row producers
constexpr int kMmaWarp = 18, kWeightWarp = 19;
constexpr int kFlush = 4;           // input stages a block of D1's sum
constexpr int kAux = 1024;          // barriers, tmem address, rows
constexpr int kMaxStages = 8;

// Shared-memory descriptors, 128-byte swizzle, 8-row groups 1024 bytes apart.
// K-major: a k step of 16 is 32 bytes.  MN-major: boxes of 64 columns `box`
// bytes apart, a k step of 16 rows is 2048 bytes.
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, int box) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(box >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// D fp32, A and B bf16, A K-major, M = 128.
__device__ __forceinline__ uint32_t idesc(bool b_mn, int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(128 >> 4) << 24) | ((uint32_t)(n >> 3) << 17);
}

// Sizes that follow from the rank.
struct TcShape {
  int rp;          // rank rounded up to 16: the first MMA's N, the second's K
  int nb;          // blocks of 64 columns of u
  int w1, w2;      // bytes of a stage's W1, W2 part (multiples of 1024)
  int stage;       // bytes of a stage
  int stages;
  int u_bytes;     // the terms of u
  int smem;
  int groups;      // epilogue groups that take output stages, a D2 buffer each
};

template <bool BWD>
TcShape tc_shape(int r) {
  TcShape t;
  t.rp = ceil_div(r, 16) * 16;
  t.nb = ceil_div(t.rp, 64);
  // forward: W1 (128 k, r) and W2 (r k, 128) N-major; backward: W1 (r, 128 k)
  // and W2 (64, r k) K-major
  t.w1 = BWD ? 2 * t.rp * 128 : 2 * t.nb * kBlk;
  t.w2 = BWD ? t.nb * kBlk : 2 * t.rp * 128;
  t.stage = 2 * kBlk + std::max(t.w1, t.w2);
  t.u_bytes = (BWD ? 3 : 2) * t.nb * kBlk;
  // + kBlk: the MMA's upper rows of the last stage
  t.stages = std::min(kMaxStages, (224 * 1024 - 1024 - kAux - kBlk - t.u_bytes) / t.stage);
  t.smem = t.stages * t.stage + t.u_bytes + kBlk + kAux + 1024;
  t.groups = std::min(kGroups, (512 - 2 * t.nb * 64) / (BWD ? 64 : 128));
  return t;
}

template <bool BWD>
__global__ void __launch_bounds__(kThreads, 1) low_rank_tc_kernel(
    const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
    const LowRankArgs g, const TcShape sh) {
  constexpr int TERMS = BWD ? 3 : 2;
  constexpr int OB = BWD ? 4 : 2;               // bytes of an output element
  constexpr int PV = 16 / OB;                   // output elements of 16 bytes
  constexpr int NC = BWD ? 64 : 128;            // output columns a stage: 256 bytes a row
  constexpr int BC = 16;                        // 16-byte pieces of them
  pdl_wait_and_release();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* ring = smem + sh.u_bytes;            // u's terms stand first
  uint8_t* aux = ring + sh.stages * sh.stage + kBlk;
  uint64_t* full = reinterpret_cast<uint64_t*>(aux);
  uint64_t* empty = full + kMaxStages;
  uint64_t* d1_full = empty + kMaxStages;       // [2]
  uint64_t* d1_empty = d1_full + 2;
  uint64_t* d2_full = d1_empty + 2;             // [kGroups]
  uint64_t* d2_empty = d2_full + kGroups;
  uint64_t* u_full = d2_empty + kGroups;
  uint64_t* drained = u_full + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drained + 1);
  int32_t* left = reinterpret_cast<int32_t*>(aux + 384);   // epilogue warps done with a stage
  int32_t* s_rows = reinterpret_cast<int32_t*>(aux + 512);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hT = __ldg(g.header), hn = __ldg(g.header + 1);
  const int2 tl = __ldg(g.tiles + blockIdx.x);
  if (tid < kTm) s_rows[tid] = __ldg(g.rows + (size_t)blockIdx.x * kTm + tid);
  const int r = g.r, K = g.K, N = g.N, a = tl.x, nrows = tl.y;
  if (hT != g.T || hn != g.n) {
    if (tid == 0) report_error(g.err, kDevBadPlan);
    return;
  }
  if (nrows == 0) return;
  if (a == g.n) {   // rows without an adapter: out = base
    if (g.base == g.out) return;
    __syncthreads();
    const int pieces = N / PV;
    for (int row = warp; row < nrows; row += kThreads / 32) {
      const size_t at = (size_t)s_rows[row] * pieces;
      for (int c = lane; c < pieces; c += 32)
        static_cast<uint4*>(g.out)[at + c] = g.base != nullptr
                                                 ? static_cast<const uint4*>(g.base)[at + c]
                                                 : make_uint4(0, 0, 0, 0);
    }
    return;
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
    if (lane == 0) {
      for (int s = 0; s < sh.stages; ++s) {
        mbar_init(&full[s], kProducers + 1);   // each producer's copies, the weights' TMA
        mbar_init(&empty[s], 1);    // D1: the MMAs' completion; D2: the last epilogue warp
        left[s] = 0;
      }
      for (int b = 0; b < 2; ++b) {
        mbar_init(&d1_full[b], 1);
        mbar_init(&d1_empty[b], 4 * kGroups);   // the epilogue warps
      }
      for (int b = 0; b < kGroups; ++b) {
        mbar_init(&d2_full[b], 1);
        mbar_init(&d2_empty[b], 4);             // the group's warps
      }
      mbar_init(u_full, 4 * kGroups);
      mbar_init(drained, 1);
      fence_mbar_init();
      tma_prefetch_map(&mapA);
      tma_prefetch_map(&mapB);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_holder;
  const int nk = ceil_div_dev(K, kKc), nn = ceil_div_dev(N, NC);
  const int nf = ceil_div_dev(nk, kFlush);
  const int d1_col = sh.nb * 64, d2_col = 2 * d1_col;   // D1's second buffer, D2's first

  if (warp == kWeightWarp) {
    // ------------------------------------------------------ weight producer
    int slot = 0;
    uint32_t phase = 1;   // of the empty barriers; the first round waits for nothing
    for (int s = 0; lane == 0 && s < nk + nn; ++s) {
      if (s >= sh.stages && !mbar_wait(&empty[slot], phase)) {
        report_error(g.err, kDevTimeoutProducer);
        break;
      }
      uint8_t* ws = ring + slot * sh.stage + 2 * kBlk;
      const int n0 = (s - nk) * NC;
      mbar_arrive_expect_tx(&full[slot], (uint32_t)(s < nk ? sh.w1 : sh.w2));
      if ((s < nk) != BWD) {
        // A's rows, 64 at a time, in boxes of 64 of the rank's columns
        const int row0 = BWD ? n0 : s * kKc;
        for (int kb = 0; kb < (BWD ? 1 : 2); ++kb)
          for (int j = 0; j < sh.nb; ++j)
            tma_load_3d(ws + (kb * sh.nb + j) * kBlk, &mapA, &full[slot], j * 64, row0 + kb * 64,
                        a);
      } else {
        // B's columns, 128 at a time, in boxes of 64
        const int col0 = BWD ? s * kKc : n0;
        for (int kb = 0; kb < 2; ++kb)
          tma_load_3d(ws + kb * sh.rp * 128, &mapB, &full[slot], col0 + kb * 64, 0, a);
      }
      if (++slot == sh.stages) {
        slot = 0;
        phase ^= 1u;
      }
    }
  } else if ((warp & 2) != 0 && warp < 2 * kProducers / 32) {
    // -------------------------------------------------------- row producers
    const int p = ((warp >> 2) * 2 + (warp & 1)) * 32 + lane;   // 0 .. kProducers - 1
    constexpr int R = kTm * 16 / kProducers;   // rows of a thread in a stage, 16 apart
    int tok[R];
#pragma unroll
    for (int i = 0; i < R; ++i) tok[i] = s_rows[p / 16 + 16 * i];
    const int total = nk + nn;
    int slot = 0;
    uint32_t phase = 1;   // of the empty barriers; the first round waits for nothing
    for (int s = 0; s < total; ++s) {
      if (s >= sh.stages) {
        if (!__all_sync(0xffffffffu, mbar_wait(&empty[slot], phase))) {
          report_error(g.err, kDevTimeoutProducer);
          break;
        }
      }
      const uint32_t st = smem_u32(ring + slot * sh.stage);
      const int pc = p % 16;   // this thread's 16-byte piece of its rows' 256 bytes
      if (s < nk) {
        const int col = s * kKc + pc * 8;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const bool ok = tok[i] >= 0 && col < K;
          cp_async16(st + (pc >> 3) * kBlk + tile_at<8>(p / 16 + 16 * i, pc & 7),
                     ok ? g.in + (size_t)tok[i] * K + col : g.in, ok);
        }
      } else {
        const uint8_t* base = static_cast<const uint8_t*>(g.base);
        const int col = (s - nk) * NC + pc * PV;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const bool ok = tok[i] >= 0 && col < N && base != nullptr;
          cp_async16(st + tile_at<BC>(p / 16 + 16 * i, pc),
                     ok ? base + ((size_t)tok[i] * N + col) * OB
                        : reinterpret_cast<const uint8_t*>(g.in), ok);
        }
      }
      cp_arrive(&full[slot]);
      if (++slot == sh.stages) {
        slot = 0;
        phase ^= 1u;
      }
    }
    cp_wait_all();
  } else if ((warp & 2) == 0) {
    // ------------------------------------------------------------- epilogue
    // tensor-memory lane quarter, half of an output stage's columns, group
    const int q = warp & 1, half = (warp >> 2) & 1, grp = warp >> 3;
    const int row = q * 32 + lane, t = s_rows[row];
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
    // This thread's columns of u, 8 at a time: every (2 kGroups)-th piece.
    constexpr int PU = (kAdapterMaxRank / 8 + 2 * kGroups - 1) / (2 * kGroups);
    const int p0 = warp >> 2;
    const float sc = __ldg(g.scale + a);
    float acc[PU][8];
#pragma unroll
    for (int i = 0; i < PU; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
    bool alive = true;
    for (int f = 0; f < nf && alive; ++f) {
      alive = __all_sync(0xffffffffu, mbar_wait(&d1_full[f & 1], (uint32_t)(f >> 1) & 1u));
      if (!alive) break;
      tc_fence_after_sync();
#pragma unroll
      for (int i = 0; i < PU; ++i) {
        const int cg = p0 + i * 2 * kGroups;
        if (cg * 8 < r) {
          uint32_t d[8];
          tmem_ld_32x32b_x8(lanes + (uint32_t)((f & 1) * d1_col + cg * 8), d);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[i][j] += __uint_as_float(d[j]);
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&d1_empty[f & 1]);
    }
#pragma unroll
    for (int i = 0; i < PU; ++i) {
      const int cg = p0 + i * 2 * kGroups;   // 8 columns: a 16-byte piece of u's terms
      if (cg * 8 < r) {
        uint2 lo[TERMS], hi[TERMS];
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = acc[i][j] * sc;
        const float va[4] = {v[0], v[1], v[2], v[3]}, vb[4] = {v[4], v[5], v[6], v[7]};
        split4<TERMS>(va, lo);
        split4<TERMS>(vb, hi);
#pragma unroll
        for (int w = 0; w < TERMS; ++w)
          *reinterpret_cast<uint4*>(smem + (w * sh.nb + cg / 8) * kBlk + tile_at<8>(row, cg % 8)) =
              make_uint4(lo[w].x, lo[w].y, hi[w].x, hi[w].y);
        if (!BWD) {
          if (t >= 0 && g.u != nullptr) {
            float4* o = reinterpret_cast<float4*>(g.u + (size_t)t * r + cg * 8);
            o[0] = make_float4(v[0], v[1], v[2], v[3]);
            o[1] = make_float4(v[4], v[5], v[6], v[7]);
          }
        } else {
          // the gradient's operands: v's and u's terms
          float4 u0 = make_float4(0.f, 0.f, 0.f, 0.f), u1 = u0;
          if (t >= 0) {
            const float4* ui = reinterpret_cast<const float4*>(g.u + (size_t)t * r + cg * 8);
            u0 = __ldg(ui);
            u1 = __ldg(ui + 1);
          }
          const float ua[4] = {u0.x, u0.y, u0.z, u0.w}, ub[4] = {u1.x, u1.y, u1.z, u1.w};
          uint2 ulo[3], uhi[3];
          split4<3>(ua, ulo);
          split4<3>(ub, uhi);
#pragma unroll
          for (int w = 0; w < TERMS; ++w) {
            const size_t o = (((size_t)blockIdx.x * kTm + row) * 3 + w) * r + cg * 8;
            *reinterpret_cast<uint4*>(g.vp + o) = make_uint4(lo[w].x, lo[w].y, hi[w].x, hi[w].y);
            *reinterpret_cast<uint4*>(g.up + o) =
                make_uint4(ulo[w].x, ulo[w].y, uhi[w].x, uhi[w].y);
          }
        }
      } else if (cg * 8 < sh.rp) {   // columns behind an odd rank: zeros
#pragma unroll
        for (int w = 0; w < TERMS; ++w)
          *reinterpret_cast<uint4*>(smem + (w * sh.nb + cg / 8) * kBlk + tile_at<8>(row, cg % 8)) =
              make_uint4(0, 0, 0, 0);
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (alive && lane == 0) mbar_arrive(u_full);
    // The rows this lane stores: 4 at a time, 8 lanes (128 bytes) each.
    constexpr int HP = BC / 2;   // 16-byte pieces of this half's row
    uint8_t* orow[HP];
#pragma unroll
    for (int k = 0; k < HP; ++k) {
      const int tt = s_rows[q * 32 + k * 4 + lane / 8];
      orow[k] = tt >= 0 ? static_cast<uint8_t*>(g.out) + (size_t)tt * N * OB : nullptr;
    }
    const int ocol = half * (NC / 2) + lane % 8 * PV;   // this lane's first column in a stage
    const uint32_t acc2 = lanes + (uint32_t)(d2_col + grp * NC + half * (NC / 2));
    int use = 0;   // stages this group has taken
    for (int i = grp; grp < sh.groups && i < nn && alive; i += sh.groups, ++use) {
      const int slot = (nk + i) % sh.stages;
      const uint32_t fph = (uint32_t)((nk + i) / sh.stages) & 1u;
      alive = mbar_wait(&full[slot], fph) && mbar_wait(&d2_full[grp], (uint32_t)use & 1u);
      alive = __all_sync(0xffffffffu, alive);
      if (!alive) break;
      tc_fence_after_sync();
      uint8_t* bs = ring + slot * sh.stage;
#pragma unroll
      for (int c0 = 0; c0 < HP; c0 += 32 / PV) {   // 32 columns at a time
        uint32_t d[32];
        tmem_ld_32x32b_x32(acc2 + (uint32_t)(c0 * PV), d);
        tmem_ld_wait();
        if (c0 + 32 / PV >= HP) {
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&d2_empty[grp]);
        }
#pragma unroll
        for (int c = 0; c < 32 / PV; ++c) {
          uint4* x = reinterpret_cast<uint4*>(bs + tile_at<BC>(row, half * HP + c0 + c));
          uint4 v = *x;
          uint32_t* w = &v.x;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            w[j] = BWD ? __float_as_uint(__uint_as_float(w[j]) + __uint_as_float(d[c * 4 + j]))
                       : pack_bf16x2(__uint_as_float(w[j] << 16) +
                                         __uint_as_float(d[(c * 8 + 2 * j) & 31]),
                                     __uint_as_float(w[j] & 0xFFFF0000u) +
                                         __uint_as_float(d[(c * 8 + 2 * j + 1) & 31]));
          *x = v;
        }
      }
      __syncwarp();
      const int col = i * NC + ocol;
#pragma unroll
      for (int k = 0; k < HP; ++k)
        if (orow[k] != nullptr && col < N)
          *reinterpret_cast<uint4*>(orow[k] + (size_t)col * OB) = *reinterpret_cast<const uint4*>(
              bs + tile_at<BC>(q * 32 + k * 4 + lane / 8, half * HP + lane % 8));
      __syncwarp();
      if (lane == 0) {   // the last of the four warps frees the stage
        __threadfence_block();
        if (atomicAdd(&left[slot], 1) == 3) {
          left[slot] = 0;
          __threadfence_block();
          mbar_arrive(&empty[slot]);
        }
      }
    }
    if (!alive) report_error(g.err, kDevTimeoutEpilogue);
  } else if (warp == kMmaWarp) {
    // ----------------------------------------------------------- MMA issuer
    // the whole warp runs the loop; one lane issues
    auto wait = [](uint64_t* bar, uint32_t ph) {
      return (bool)__all_sync(0xffffffffu, mbar_wait(bar, ph));
    };
    int slot = 0;
    uint32_t fph = 0;
    bool alive = true;
    const uint32_t id1 = idesc(!BWD, sh.rp), id2 = idesc(!BWD, NC);
    for (int s = 0; s < nk && alive; ++s) {
      const int f = s / kFlush, b = f & 1;
      if (s % kFlush == 0 && f >= 2) alive = wait(&d1_empty[b], (uint32_t)(f / 2 - 1) & 1u);
      alive = alive && wait(&full[slot], fph);
      if (!alive) break;
      fence_proxy_async_smem();   // the copies' writes, before the tensor core reads them
      tc_fence_after_sync();
      const uint32_t xs = smem_u32(ring + slot * sh.stage), ws = xs + 2 * kBlk;
#pragma unroll
      for (int kk = 0; kk < kKc / 16; ++kk)
        umma_elect(tmem + (uint32_t)(b * d1_col), desc_k(xs + kk / 4 * kBlk + kk % 4 * 32),
                   BWD ? desc_k(ws + kk / 4 * sh.rp * 128 + kk % 4 * 32)
                       : desc_mn(ws + kk / 4 * sh.nb * kBlk + kk % 4 * 2048, kBlk),
                   id1, (s % kFlush | kk) != 0 ? 1u : 0u);
      umma_commit_elect(&empty[slot]);
      if (s % kFlush == kFlush - 1 || s == nk - 1) umma_commit_elect(&d1_full[b]);
      if (++slot == sh.stages) {
        slot = 0;
        fph ^= 1u;
      }
    }
    alive = alive && wait(u_full, 0);
    const uint32_t us = smem_u32(smem);
    int b = 0, use = 0;   // output stage i: group b, its use-th
    for (int i = 0; i < nn && alive; ++i) {
      if (use > 0) alive = wait(&d2_empty[b], (uint32_t)(use - 1) & 1u);
      alive = alive && wait(&full[slot], fph);
      if (!alive) break;
      fence_proxy_async_smem();
      tc_fence_after_sync();
      const uint32_t ws = smem_u32(ring + slot * sh.stage) + 2 * kBlk;
      uint32_t more = 0;
      for (int w = TERMS - 1; w >= 0; --w)   // the small terms first
        for (int kk = 0; kk < sh.rp / 16; ++kk) {
          umma_elect(tmem + (uint32_t)(d2_col + b * NC),
                       desc_k(us + (w * sh.nb + kk / 4) * kBlk + kk % 4 * 32),
                       BWD ? desc_k(ws + kk / 4 * kBlk + kk % 4 * 32)
                           : desc_mn(ws + kk * 2048, sh.rp * 128),
                       id2, more);
          more = 1;
        }
      umma_commit_elect(&d2_full[b]);
      if (++b == sh.groups) {
        b = 0;
        ++use;
      }
      if (++slot == sh.stages) {
        slot = 0;
        fph ^= 1u;
      }
    }
    if (!alive) report_error(g.err, kDevTimeoutMma);
    umma_commit_elect(drained);
    if (!wait(drained, 0)) report_error(g.err, kDevTimeoutDrain);
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

template <bool BWD>
cudaError_t run(const LowRankArgs& g, int tiles, cudaStream_t s) {
  const TcShape sh = tc_shape<BWD>(g.r);
  const auto kern = low_rank_tc_kernel<BWD>;
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), 227 * 1024);
  if (e != cudaSuccess) return e;
  CUtensorMap a, b;   // A (n, d, r) and B (n, r, d_out)
  if (!encode_bf16(&a, BWD ? g.W2 : g.W1, g.n, BWD ? g.N : g.K, g.r, 64) ||
      !encode_bf16(&b, BWD ? g.W1 : g.W2, g.n, g.r, BWD ? g.K : g.N, sh.rp))
    return cudaErrorNotSupported;
  return launch_kernel(kern, (unsigned)tiles, kThreads, sh.smem, s, 0, a, b, g, sh);
}

}  // namespace

cudaError_t launch_low_rank_tc(const LowRankArgs& g, bool backward, int tiles, cudaStream_t s) {
  return backward ? run<true>(g, tiles, s) : run<false>(g, tiles, s);
}

}  // namespace moe
