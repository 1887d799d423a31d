// adapter_tc.cu - the adapters' two low-rank products on tcgen05, for batches
// of many rows (adapter.cu has the formulas, the plan and the other forms).
//
// One CTA per tile of 64 rows of one adapter, both products in one launch:
//   D1 (64, r)  = in[rows, :] W1         input columns 128 at a time
//   u           = scale D1, split into bf16 terms, written to tensor memory
//   D2 (64, NC) = sum over the terms of u_w W2[:, NC columns]; out = base + D2
// with NC = 128 columns of bf16 forward, 64 of fp32 backward.  8 warps gather
// the rows by cp.async (input columns first and then base's) and one loads the
// weights by TMA, all through ONE ring of stages: while u is formed the second
// product's loads are already in flight, so HBM never waits.  One warp issues
// the MMAs (M = 128: the upper 64 rows read whatever follows in shared memory,
// or stands in tensor memory, and are never looked at).  The second product
// takes u's terms from tensor memory: an MMA of 128 x 64 x 16 takes 32 cycles
// so, 49 with A in shared memory.  The warps that own
// tensor memory's lanes 0-63 are the epilogue: three groups, an output stage and
// a D2 buffer each in turn.  They add D1's blocks in round-to-nearest fp32 (the
// tensor core's own sums truncate), and write D2 through the stage's base tile,
// so that every global access of a warp covers whole sectors.  u's terms reach
// the second product before what later launches need is written out.
// It moves 2 (K + 2 N) bytes a row forward, 2 K + 8 N backward, at two thirds of the
// measured copy rate: one CTA an SM, so that all read x together, wait while u is
// formed, and then read and write together.  B200, 8192 rows: forward, 4096 wide, rank
// 16, 44 us (4.6 TB/s); backward, 2048 wide, rank 64, 41 us (4.3 TB/s), where a
// stage's loads pace the second product.
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
constexpr int kProducers = 128;     // threads of the row producers
constexpr int kMmaWarp = 18, kWeightWarp = 19;
// Input stages a block of D1's sum: the truncation of 256 columns' sums leaves u
// and v within 2e-7 of exact, 512's within 4e-7, which u's and v's products, the
// gradients, would show.  (A forward pass that keeps no u could take blocks of 1024:
// 8192 x 4096, rank 16, 47.3 us against 47.4, but its output would have other bits
// than one that keeps it.)
constexpr int kFlush = 2;
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
  int smem;
  int u_col, d2_col;   // tensor-memory columns
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
  // + kBlk: the MMA's upper rows of the last stage
  t.stages = std::min(kMaxStages, (224 * 1024 - 1024 - kAux - kBlk) / t.stage);
  t.smem = t.stages * t.stage + kBlk + kAux + 1024;
  // tensor memory: D1, u's terms (two bf16 a column), a D2 for each group; D1's
  // second buffer is where the D2s come to stand
  t.u_col = t.nb * 64;
  t.d2_col = t.u_col + (BWD ? 3 : 2) * t.rp / 2;
  t.groups = std::min(kGroups, (512 - t.d2_col) / (BWD ? 64 : 128));
  return t;
}

// The three bf16 terms of 8 values, columns 8 cg on of this tile's row `row`.
__device__ __forceinline__ void store_terms(__nv_bfloat16* terms, int row, int cg, int r,
                                            const float4& a, const float4& b) {
  const float va[4] = {a.x, a.y, a.z, a.w}, vb[4] = {b.x, b.y, b.z, b.w};
  uint2 lo[3], hi[3];
  split4<3>(va, lo);
  split4<3>(vb, hi);
#pragma unroll
  for (int w = 0; w < 3; ++w)
    *reinterpret_cast<uint4*>(terms + (((size_t)blockIdx.x * kTm + row) * 3 + w) * r + cg * 8) =
        make_uint4(lo[w].x, lo[w].y, hi[w].x, hi[w].y);
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
  uint8_t* ring = smem;
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
        // D2: a group's epilogue warps; D1: the MMAs' completion, and three at once
        mbar_init(&empty[s], 4);
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
  } else if ((warp & 3) == 3 && warp < 4 * kProducers / 32) {
    // -------------------------------------------------------- row producers
    const int p = (warp >> 2) * 32 + lane;   // 0 .. kProducers - 1
    constexpr int R = kTm * 16 / kProducers;   // rows of a thread in a stage, 16 apart
    int tok[R];
#pragma unroll
    for (int i = 0; i < R; ++i) tok[i] = s_rows[p / 16 + kProducers / 16 * i];
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
          cp_async16(st + (pc >> 3) * kBlk + tile_at<8>(p / 16 + kProducers / 16 * i, pc & 7),
                     ok ? g.in + (size_t)tok[i] * K + col : g.in, ok);
        }
      } else {
        const uint8_t* base = static_cast<const uint8_t*>(g.base);
        const int col = (s - nk) * NC + pc * PV;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const bool ok = tok[i] >= 0 && col < N && base != nullptr;
          cp_async16(st + tile_at<BC>(p / 16 + kProducers / 16 * i, pc),
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
    if (BWD) {
      // one of the gradient's operands, u's terms, while D1 is formed
#pragma unroll
      for (int i = 0; i < PU; ++i) {
        const int cg = p0 + i * 2 * kGroups;
        if (cg * 8 >= r) continue;
        float4 u0 = make_float4(0.f, 0.f, 0.f, 0.f), u1 = u0;
        if (t >= 0) {
          const float4* ui = reinterpret_cast<const float4*>(g.u + (size_t)t * r + cg * 8);
          u0 = __ldg(ui);
          u1 = __ldg(ui + 1);
        }
        store_terms(g.up, row, cg, r, u0, u1);
      }
    }
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
      const uint32_t d1 = lanes + (uint32_t)((f & 1) * sh.d2_col);
      uint32_t d[PU][8];
#pragma unroll
      for (int i = 0; i < PU; ++i)
        if ((p0 + i * 2 * kGroups) * 8 < r)
          tmem_ld_32x32b_x8(d1 + (uint32_t)(p0 + i * 2 * kGroups) * 8, d[i]);
      tmem_ld_wait();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&d1_empty[f & 1]);
#pragma unroll
      for (int i = 0; i < PU; ++i)
        if ((p0 + i * 2 * kGroups) * 8 < r)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[i][j] += __uint_as_float(d[i][j]);
    }
#pragma unroll
    for (int i = 0; i < PU; ++i) {
      const int cg = p0 + i * 2 * kGroups;   // 8 columns: 4 of tensor memory's a term
      if (cg * 8 >= sh.rp) continue;         // (columns behind an odd rank: zeros)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i][j] = cg * 8 < r ? acc[i][j] * sc : 0.f;
      const float va[4] = {acc[i][0], acc[i][1], acc[i][2], acc[i][3]};
      const float vb[4] = {acc[i][4], acc[i][5], acc[i][6], acc[i][7]};
      uint2 lo[TERMS], hi[TERMS];
      split4<TERMS>(va, lo);
      split4<TERMS>(vb, hi);
#pragma unroll
      for (int w = 0; w < TERMS; ++w)
        tmem_st_32x32b_x4(lanes + (uint32_t)(sh.u_col + w * sh.rp / 2 + cg * 4), lo[w].x, lo[w].y,
                          hi[w].x, hi[w].y);
    }
    tmem_st_wait();
    tc_fence_before_sync();
    __syncwarp();
    if (alive && lane == 0) mbar_arrive(u_full);
    // u, or v's terms, for later launches, while the second product begins
#pragma unroll
    for (int i = 0; i < PU; ++i) {
      const int cg = p0 + i * 2 * kGroups;
      if (cg * 8 >= r) continue;
      const float4 v0 = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
      const float4 v1 = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
      if (BWD) {
        store_terms(g.vp, row, cg, r, v0, v1);
      } else if (t >= 0 && g.u != nullptr) {
        float4* o = reinterpret_cast<float4*>(g.u + (size_t)t * r + cg * 8);
        o[0] = v0;
        o[1] = v1;
      }
    }
    // The rows this lane stores: 4 at a time, 8 lanes (128 bytes) each.
    constexpr int HP = BC / 2;   // 16-byte pieces of this half's row
    uint8_t* orow[HP];
#pragma unroll
    for (int k = 0; k < HP; ++k) {
      const int tt = s_rows[q * 32 + k * 4 + lane / 8];
      orow[k] = tt >= 0 ? static_cast<uint8_t*>(g.out) + (size_t)tt * N * OB : nullptr;
    }
    const int ocol = half * (NC / 2) + lane % 8 * PV;   // this lane's first column in a stage
    const uint32_t acc2 = lanes + (uint32_t)(sh.d2_col + grp * NC + half * (NC / 2));
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
      if (lane == 0) mbar_arrive(&empty[slot]);
    }
    if (!alive) report_error(g.err, kDevTimeoutEpilogue);
  } else if (warp == kMmaWarp) {
    // ----------------------------------------------------------- MMA issuer
    // the whole warp runs the loop; one lane issues
    auto wait = [](uint64_t* bar, uint32_t ph) {
      return (bool)__all_sync(0xffffffffu, mbar_wait(bar, ph));
    };
    int slot = 0, block = 0, in_block = 0;
    uint32_t fph = 0;
    bool alive = true;
    const uint32_t id1 = idesc(!BWD, sh.rp), id2 = idesc(!BWD, NC);
    for (int s = 0; s < nk && alive; ++s) {
      if (in_block == 0 && block >= 2)
        alive = wait(&d1_empty[block & 1], (uint32_t)(block / 2 - 1) & 1u);
      alive = alive && wait(&full[slot], fph);
      if (!alive) break;
      fence_proxy_async_smem();   // the copies' writes, before the tensor core reads them
      tc_fence_after_sync();
      const uint32_t xs = smem_u32(ring + slot * sh.stage), ws = xs + 2 * kBlk;
      const uint32_t d1 = tmem + (uint32_t)((block & 1) * sh.d2_col);
      const uint64_t xd = desc_k(xs);
      const uint64_t wd0 = BWD ? desc_k(ws) : desc_mn(ws, kBlk);
      const uint64_t wd1 = wd0 + (uint32_t)(BWD ? sh.rp * 128 : sh.nb * kBlk) / 16;
#pragma unroll
      for (int kk = 0; kk < kKc / 16; ++kk)
        umma_elect(d1, xd + (kk / 4 * kBlk + kk % 4 * 32) / 16,
                   (kk < 4 ? wd0 : wd1) + kk % 4 * (BWD ? 32 : 2048) / 16, id1,
                   (in_block | kk) != 0 ? 1u : 0u);
      if (lane == 0) mbar_arrive_n(&empty[slot], 3);
      umma_commit_elect(&empty[slot]);
      if (++in_block == kFlush || s == nk - 1) {
        umma_commit_elect(&d1_full[block & 1]);
        ++block;
        in_block = 0;
      }
      if (++slot == sh.stages) {
        slot = 0;
        fph ^= 1u;
      }
    }
    alive = alive && wait(u_full, 0);
    // (Steps unrolled, their descriptors a constant apart, one election for all:
    // 40 cycles an MMA of 128 x 64 x 16 where a loop that elects for each took 66.)
    const int ks = sh.rp / 16;
    int b = 0, use = 0;   // output stage i: group b, its use-th
    for (int i = 0; i < nn && alive; ++i) {
      if (use > 0) alive = wait(&d2_empty[b], (uint32_t)(use - 1) & 1u);
      alive = alive && wait(&full[slot], fph);
      if (!alive) break;
      // (no proxy fence: these MMAs read tensor memory and the weights' TMA
      // alone, and the fence waits for the rows' copies in flight)
      tc_fence_after_sync();
      const uint32_t ws = smem_u32(ring + slot * sh.stage) + 2 * kBlk;
      const uint64_t wd = BWD ? desc_k(ws) : desc_mn(ws, sh.rp * 128);
      const uint32_t d2 = tmem + (uint32_t)(sh.d2_col + b * NC);
      if (elect_one()) {
#pragma unroll
        for (int w = TERMS - 1; w >= 0; --w) {   // the small terms first
          const uint32_t uw = tmem + (uint32_t)(sh.u_col + w * sh.rp / 2);
#pragma unroll
          for (int kk = 0; kk < kAdapterMaxRank / 16; ++kk) {
            if (kk == ks) break;
            umma_ts(d2, uw + kk * 8, wd + (BWD ? kk / 4 * kBlk + kk % 4 * 32 : kk * 2048) / 16,
                    id2, w != TERMS - 1 || kk != 0 ? 1u : 0u);
          }
        }
      }
      __syncwarp();
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
