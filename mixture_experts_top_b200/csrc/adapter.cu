// adapter.cu - low-rank adapters of many requests beside a projection that
// all requests share (the routed layer itself), and their gradients.
//
// Token t carries an adapter a = token_adapter[t] (none if negative):
//   u[t] = s_a x[t] A_a          output[t] = base[t] + u[t] B_a
//   v[t] = s_a dy[t] B_a^T       dx[t] = dx_add[t] + v[t] A_a^T
//   dA_a = sum_t x[t]^T v[t]     dB_a = sum_t u[t]^T dy[t]
// with A_a (d, r), B_a (r, d_out), r <= 128: 2 r (d + d_out) products a token
// against 2 (d + 2 d_out) bytes, so up to r = 64 or so HBM bounds it.
//
// plan     - the tokens grouped by adapter, in token order, and the row tiles
//            of the groups.  One CTA per adapter counts all tokens in shared
//            memory and writes its own rows: one launch, no global atomics, but
//            T n reads (8192 tokens on 8 adapters 5 us, 131072 on 64 36, on
//            1024 152).
// low rank - both products of a row tile in one launch.  A cluster of CTAs
//            shares a tile: each contracts its slice of the input's columns,
//            the r-wide partial sums meet through distributed shared memory
//            in CTA order, and each writes its slice of the output's columns;
//            u never makes a trip through HBM between the products.
//            (Many rows: adapter_tc.cu, one CTA per tile on tcgen05.)
// gradient - on tcgen05, rows of an adapter on the contraction, 128 columns of
//            x or dy a CTA; the rows are cut into equal chunks and the parts of
//            a cut adapter added in order by a last launch.  No floating-point
//            atomics anywhere.
//
// Precision: bf16 operands, fp32 sums.  The tensor core adds one staged block
// at a time and the blocks are added in round-to-nearest fp32.  u and v are
// fp32 values: where one is an operand it is split into bf16 terms, two
// (16 bits) for the bf16 output, three (all 24 bits) for the fp32 gradients.
#include "adapter.cuh"
#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

// ------------------------------------------------------------------- plan --

constexpr int kPlanThreads = 1024;

// CTA g writes group g: adapter g's rows, or (g = n) the rows without one.  Each
// warp owns a range of tokens and counts those of earlier groups and of its
// own; after one exchange it writes its rows in token order.  A group's tiles
// have the slots from offsets[g] / TM + g on, which no other group's have, so
// that nothing needs the other groups' counts; slots left over hold no rows.
// Rows stand by tile slot, -1 behind a tile's last, so that a kernel's CTA
// reads its tile and its rows at once.
__global__ void __launch_bounds__(kPlanThreads)
    adapter_plan_kernel(const int32_t* __restrict__ ids, int T, int n, int TM, int32_t* header,
                        int32_t* __restrict__ offsets, int32_t* __restrict__ rows,
                        int2* __restrict__ tiles, int32_t* err) {
  pdl_wait_and_release();
  __shared__ int32_t s_less[32], s_mine[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = blockIdx.x;
  const int per = ceil_div_dev(ceil_div_dev(T, 32), 32) * 32;   // T <= 2^30
  const int t0 = (int)min((long long)T, (long long)warp * per), t1 = min(T, t0 + per);
  auto group = [&](int t) {
    const int a = __ldg(ids + t);
    return (unsigned)a >= (unsigned)n ? n : a;
  };
  int less = 0, mine = 0;
  bool bad = false;
#pragma unroll 8
  for (int t = t0 + lane; t < t1; t += 32) {
    const int a = __ldg(ids + t);
    const int q = (unsigned)a >= (unsigned)n ? n : a;
    less += q < g;
    mine += q == g;
    bad |= a >= n;
  }
  if (bad && g == 0) report_error(err, kDevBadExpertIndex);
  less = __reduce_add_sync(0xffffffffu, less);
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) {
    s_less[warp] = less;
    s_mine[warp] = mine;
  }
  __syncthreads();
  const int row0 = __reduce_add_sync(0xffffffffu, s_less[lane]);
  const int cnt = __reduce_add_sync(0xffffffffu, s_mine[lane]);
  if (tid == 0) {
    offsets[g] = row0;
    if (g == n) {
      offsets[n + 1] = T;
      header[0] = T;
      header[1] = n;
    }
  }
  const int slot0 = row0 / TM + g, nslots = (row0 + cnt) / TM + g + 1 - slot0;
  rows += (size_t)slot0 * TM;
  for (int i = tid; i < nslots; i += kPlanThreads)
    tiles[slot0 + i] = make_int2(g, min(TM, max(0, cnt - i * TM)));
  for (int i = cnt + tid; i < nslots * TM; i += kPlanThreads) rows[i] = -1;
  if (mine == 0) return;
  int at = __reduce_add_sync(0xffffffffu, lane < warp ? s_mine[lane] : 0);
#pragma unroll 4
  for (int t = t0; t < t1; t += 32) {
    const bool in = t + lane < t1 && group(t + lane) == g;
    const unsigned b = __ballot_sync(0xffffffffu, in);
    if (in) rows[at + __popc(b & lanemask_lt())] = t + lane;
    at += __popc(b);
  }
}

// --------------------------------------------------------------- low rank --

// RP: the rank rounded up to 16, 32, 64 or 128; TM: rows of a tile.
template <int RP, int TM, bool BWD>
struct LowRank {
  static constexpr int KC = TM == 64 ? 64 : 128;      // input columns a stage
  static constexpr int NC = TM == 64 ? 64 : 128;      // output columns a stage
  static constexpr int WM = TM / 16;
  static constexpr int WK = TM == 16 ? 8 : (RP == 16 ? 2 : 1);   // warps along the contraction
  static constexpr int WN = 8 / (WM * WK);
  static constexpr int NT = RP / 8 / WN;              // 8-wide tiles a warp, first product
  static constexpr int W2 = 8 / WM;                   // warps along the output's columns
  static constexpr int NT2 = NC / W2 / 8;
  static constexpr int TERMS = BWD ? 3 : 2;
  static constexpr int OB = BWD ? 4 : 2;              // bytes of an output element
  static constexpr int S1 = TM * KC * 2 + KC * RP * 2;
  static constexpr int S2 = RP * NC * 2 + TM * NC * OB;
  static constexpr int ST1 = TM == 16 ? 3 : 4;
  static constexpr int ST2 = TM == 16 && RP > 32 ? 2 : 3;
  // Few rows (decode): both products' first stages are loaded at once, from
  // rings of their own.  Many rows: one ring, so that two to four CTAs fit an
  // SM and one's input overlaps another's output.
  static constexpr bool AHEAD = TM == 16;
  static constexpr int RED = WK > 1 ? WK * TM * RP * 4 : 0;
  static constexpr int R1 = ST1 * S1 > RED ? ST1 * S1 : RED;
  static constexpr int R2 = ST2 * S2;
  static constexpr int RING2 = AHEAD ? R1 : 0;        // where the second ring starts
  static constexpr int RING = AHEAD ? R1 + R2 : (R1 > R2 ? R1 : R2);
  static constexpr int US = TERMS * TM * RP * 2;
  static constexpr int PART = TM * RP * 4;
  static constexpr int SMEM = RING + US + PART;
  static constexpr int CTAS = 227 * 1024 / (SMEM + 1024 + TM * 4);   // an SM holds, by memory
};

template <int RP, int TM, bool BWD>
__global__ void __launch_bounds__(256) low_rank_kernel(LowRankArgs g) {
  using L = LowRank<RP, TM, BWD>;
  pdl_wait_and_release();
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t ring = smem_u32(smem), us = ring + L::RING;
  float* partp = reinterpret_cast<float*>(smem + L::RING + L::US);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t cs;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cs));
  const int CS = (int)cs, cr = (int)cluster_cta_rank();
  const int hT = __ldg(g.header), hn = __ldg(g.header + 1);
  const int tile = blockIdx.x / CS;
  const int2 tl = __ldg(g.tiles + tile);
  // The token of tile row i, -1 behind the last.
  auto token = [&](int i) { return __ldg(g.rows + (size_t)tile * TM + i); };
  constexpr int PV = 16 / L::OB;           // output elements of 16 bytes
  constexpr int BC = L::NC / PV;           // 16-byte pieces of a stage's output row
  constexpr int BR = TM * BC / 256;        // output rows of a thread in a stage
  constexpr int XC = L::KC / 8;            // 16-byte pieces of a stage's input row
  constexpr int XR = TM * XC / 256;        // input rows of a thread in a stage
  int bt[BR], xt[XR];
#pragma unroll
  for (int i = 0; i < BR; ++i) bt[i] = token(tid / BC + i * (256 / BC));
#pragma unroll
  for (int i = 0; i < XR; ++i) xt[i] = token(tid / XC + i * (256 / XC));
  const int r = g.r, K = g.K, N = g.N, a = tl.x;
  if (hT != g.T || hn != g.n) {   // the same for every CTA
    if (tid == 0) report_error(g.err, kDevBadPlan);
    return;
  }
  if (tl.y == 0) return;          // no rows: the same for the cluster
  const float sc = a < g.n ? __ldg(g.scale + a) : 0.f;
  const int nn = ceil_div_dev(N, L::NC);
  const int n0 = (int)((long long)nn * cr / CS), n1 = (int)((long long)nn * (cr + 1) / CS);
  if (a == g.n) {   // rows without an adapter: out = base
    if (g.base == g.out) return;
    for (int nc = n0; nc < n1; ++nc) {
      const int col = nc * L::NC + tid % BC * PV;
#pragma unroll
      for (int i = 0; i < BR; ++i)
        if (bt[i] >= 0 && col < N) {
          const size_t at = ((size_t)bt[i] * N + col) / PV;
          static_cast<uint4*>(g.out)[at] = g.base != nullptr
                                               ? static_cast<const uint4*>(g.base)[at]
                                               : make_uint4(0, 0, 0, 0);
        }
    }
    return;
  }
  const __nv_bfloat16* w1 = g.W1 + (size_t)a * K * r;
  const __nv_bfloat16* w2 = g.W2 + (size_t)a * N * r;

  // ---- loads ----
  const int nk = ceil_div_dev(K, L::KC);
  const int k0 = (int)((long long)nk * cr / CS), k1 = (int)((long long)nk * (cr + 1) / CS);
  const __nv_bfloat16* xrow[XR];
#pragma unroll
  for (int i = 0; i < XR; ++i) xrow[i] = xt[i] >= 0 ? g.in + (size_t)xt[i] * K : nullptr;
  auto load_w1 = [&](int kc) {
    const uint32_t ws = ring + (uint32_t)((kc - k0) % L::ST1) * L::S1 + TM * L::KC * 2;
    if (!BWD) {   // [k][j]
      constexpr int RC = RP / 8;
#pragma unroll
      for (int i = tid; i < L::KC * RC; i += 256) {
        const int row = i / RC, c = i % RC, col = kc * L::KC + row;
        const bool ok = col < K && c * 8 < r;
        cp_async16(ws + tile_at<RC>(row, c), ok ? w1 + (size_t)col * r + c * 8 : w1, ok);
      }
    } else {      // [j][k]
#pragma unroll
      for (int i = tid; i < RP * XC; i += 256) {
        const int row = i / XC, c = i % XC, col = kc * L::KC + c * 8;
        const bool ok = row < r && col < K;
        cp_async16(ws + tile_at<XC>(row, c), ok ? w1 + (size_t)row * K + col : w1, ok);
      }
    }
  };
  auto load_x = [&](int kc) {
    const uint32_t xs = ring + (uint32_t)((kc - k0) % L::ST1) * L::S1;
    const int col = kc * L::KC + tid % XC * 8;
#pragma unroll
    for (int i = 0; i < XR; ++i) {
      const bool ok = xrow[i] != nullptr && col < K;
      cp_async16(xs + tile_at<XC>(tid / XC + i * (256 / XC), tid % XC),
                 ok ? xrow[i] + col : g.in, ok);
    }
  };
  auto load2 = [&](int nc) {
    const uint32_t ws = ring + L::RING2 + (uint32_t)((nc - n0) % L::ST2) * L::S2;
    const uint32_t bs = ws + RP * L::NC * 2;
    if (!BWD) {   // [j][c]
      constexpr int CC = L::NC / 8;
#pragma unroll
      for (int i = tid; i < RP * CC; i += 256) {
        const int row = i / CC, c = i % CC, col = nc * L::NC + c * 8;
        const bool ok = row < r && col < N;
        cp_async16(ws + tile_at<CC>(row, c), ok ? w2 + (size_t)row * N + col : w2, ok);
      }
    } else {      // [c][j]
      constexpr int RC = RP / 8;
#pragma unroll
      for (int i = tid; i < L::NC * RC; i += 256) {
        const int row = i / RC, c = i % RC, col = nc * L::NC + row;
        const bool ok = col < N && c * 8 < r;
        cp_async16(ws + tile_at<RC>(row, c), ok ? w2 + (size_t)col * r + c * 8 : w2, ok);
      }
    }
    const int col = nc * L::NC + tid % BC * PV;
#pragma unroll
    for (int i = 0; i < BR; ++i) {
      const bool ok = bt[i] >= 0 && col < N && g.base != nullptr;
      const uint8_t* src =
          static_cast<const uint8_t*>(g.base) + ((size_t)(ok ? bt[i] : 0) * N + col) * L::OB;
      cp_async16(bs + tile_at<BC>(tid / BC + i * (256 / BC), tid % BC),
                 ok ? src : reinterpret_cast<const uint8_t*>(w2), ok);
    }
  };
  // The second product's first stages; AHEAD, they belong to the last group
  // that goes out before the first product.
  auto begin2 = [&]() {
#pragma unroll
    for (int i = 0; i < L::ST2 - 1; ++i) {
      if (n0 + i < n1) load2(n0 + i);
      if (!L::AHEAD) cp_commit();
    }
  };

  // ---- first product: part = in[rows, slice] W1[slice, :] ----
  const int wm = warp % L::WM, wk = (warp / L::WM) % L::WK, wn = warp / (L::WM * L::WK);
  float acc[L::NT][4];
#pragma unroll
  for (int i = 0; i < L::NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll
  for (int i = 0; i < L::ST1 - 1; ++i)
    if (k0 + i < k1) load_w1(k0 + i);   // (needs no row: out before the rows are known)
#pragma unroll
  for (int i = 0; i < L::ST1 - 1; ++i) {
    if (k0 + i < k1) load_x(k0 + i);
    if (L::AHEAD && i == L::ST1 - 2) begin2();
    cp_commit();
  }
  for (int kc = k0; kc < k1; ++kc) {
    cp_wait<L::ST1 - 2>();
    __syncthreads();
    if (kc + L::ST1 - 1 < k1) {
      load_w1(kc + L::ST1 - 1);
      load_x(kc + L::ST1 - 1);
    }
    cp_commit();
    const uint32_t xs = ring + (uint32_t)((kc - k0) % L::ST1) * L::S1;
    const uint32_t ws = xs + TM * L::KC * 2;
    float c[L::NT][4];
#pragma unroll
    for (int i = 0; i < L::NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) c[i][j] = 0.f;
#pragma unroll
    for (int ks = wk; ks < L::KC / 16; ks += L::WK) {
      uint32_t fa[4];
      ldsm4(xs + tile_at<XC>(wm * 16 + (lane & 15), ks * 2 + (lane >> 4)), fa);
#pragma unroll
      for (int p = 0; p < L::NT / 2; ++p) {
        const int j0 = wn * (RP / L::WN) + p * 16;
        uint32_t fb[4];
        if (!BWD)
          ldsm4_t(ws + tile_at<RP / 8>(ks * 16 + (lane & 15), j0 / 8 + (lane >> 4)), fb);
        else
          ldsm4(ws + tile_at<XC>(j0 + (lane & 7) + (lane >> 4) * 8, ks * 2 + ((lane >> 3) & 1)),
                fb);
        mma16816(c[2 * p], fa, fb[0], fb[1]);
        mma16816(c[2 * p + 1], fa, fb[2], fb[3]);
      }
    }
#pragma unroll
    for (int i = 0; i < L::NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] += c[i][j];
  }
  cp_wait<0>();
  __syncthreads();   // the first ring is free

  // ---- u (v): the warps' and then the CTAs' partial sums, in order ----
  if (!L::AHEAD && L::WK == 1) begin2();
  {
    const int row = wm * 16 + (lane >> 2), col0 = wn * (RP / L::WN) + (lane & 3) * 2;
    float* dst = L::WK > 1 ? reinterpret_cast<float*>(smem) + wk * TM * RP : partp;
#pragma unroll
    for (int i = 0; i < L::NT; ++i) {
      float* p = dst + row * RP + col0 + i * 8;
      *reinterpret_cast<float2*>(p) = make_float2(acc[i][0], acc[i][1]);
      *reinterpret_cast<float2*>(p + 8 * RP) = make_float2(acc[i][2], acc[i][3]);
    }
  }
  if (L::WK > 1) {
    __syncthreads();
    for (int i = tid * 4; i < TM * RP; i += 1024) {
      float4 v = *reinterpret_cast<const float4*>(smem + i * 4);
#pragma unroll
      for (int w = 1; w < L::WK; ++w) {
        const float4 q = *reinterpret_cast<const float4*>(smem + (w * TM * RP + i) * 4);
        v.x += q.x;
        v.y += q.y;
        v.z += q.z;
        v.w += q.w;
      }
      *reinterpret_cast<float4*>(partp + i) = v;
    }
    __syncthreads();
    if (!L::AHEAD) begin2();
  }
  if (CS > 1) cluster_sync_all();
  else __syncthreads();
  // Few rows: every CTA adds all of them over the cluster, which spares it a
  // second barrier.  Many: each adds its share and hands the bf16 terms to
  // every CTA's operand tile.
  const int own0 = TM * cr / CS, own1 = TM * (cr + 1) / CS;
  const int e0 = (L::AHEAD ? 0 : own0) * RP, e1 = (L::AHEAD ? TM : own1) * RP;
  for (int i = e0 + tid * 4; i < e1; i += 1024) {
    const int row = i / RP, j = i % RP;
    const int t = token(row);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int q = 0; q < CS; ++q) {
      const float4 p = CS > 1 ? ld_cluster_f4(cluster_smem_addr(partp + i, (uint32_t)q))
                              : *reinterpret_cast<const float4*>(partp + i);
      v[0] += p.x;
      v[1] += p.y;
      v[2] += p.z;
      v[3] += p.w;
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) v[m] *= sc;
    uint2 tm[L::TERMS];
    split4<L::TERMS>(v, tm);
    const uint32_t at = L::RING + tile_at<RP / 8>(row, j / 8) + (j % 8) * 2;
    if (L::AHEAD || CS == 1) {
#pragma unroll
      for (int w = 0; w < L::TERMS; ++w)
        *reinterpret_cast<uint2*>(smem + at + w * TM * RP * 2) = tm[w];
    } else {
      for (int q = 0; q < CS; ++q) {
        const uint32_t dst = cluster_smem_addr(smem + at, (uint32_t)q);
#pragma unroll
        for (int w = 0; w < L::TERMS; ++w) st_cluster_v2(dst + w * TM * RP * 2, tm[w]);
      }
    }
    if (j >= r || row < own0 || row >= own1) continue;
    if (!BWD) {
      if (t >= 0 && g.u != nullptr)
        *reinterpret_cast<float4*>(g.u + (size_t)t * r + j) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      // the gradient's operands: v's and u's terms
      float4 uq = make_float4(0.f, 0.f, 0.f, 0.f);
      if (t >= 0) uq = __ldg(reinterpret_cast<const float4*>(g.u + (size_t)t * r + j));
      const float uv[4] = {uq.x, uq.y, uq.z, uq.w};
      uint2 ut[3];
      split4<3>(uv, ut);
#pragma unroll
      for (int w = 0; w < 3; ++w) {
        const size_t o = (((size_t)tile * TM + row) * 3 + w) * r + j;
        *reinterpret_cast<uint2*>(g.vp + o) = tm[w < L::TERMS ? w : 0];
        *reinterpret_cast<uint2*>(g.up + o) = ut[w];
      }
    }
  }
  if (L::AHEAD || CS == 1) __syncthreads();
  else cluster_sync_all();

  // ---- second product: out[rows, slice] = base + u W2[:, slice] ----
  const int w2n = warp / L::WM;
  for (int nc = n0; nc < n1; ++nc) {
    cp_wait<L::ST2 - 2>();
    __syncthreads();
    if (nc + L::ST2 - 1 < n1) load2(nc + L::ST2 - 1);
    cp_commit();
    const uint32_t so = L::RING2 + (uint32_t)((nc - n0) % L::ST2) * L::S2;
    const uint32_t ws = ring + so;
    float c[L::NT2][4];
#pragma unroll
    for (int i = 0; i < L::NT2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) c[i][j] = 0.f;
#pragma unroll
    for (int ks = 0; ks < RP / 16; ++ks) {
      uint32_t fa[L::TERMS][4];
#pragma unroll
      for (int w = 0; w < L::TERMS; ++w)
        ldsm4(us + w * TM * RP * 2 +
                  tile_at<RP / 8>(wm * 16 + (lane & 15), ks * 2 + (lane >> 4)), fa[w]);
#pragma unroll
      for (int p = 0; p < L::NT2 / 2; ++p) {
        const int cc = w2n * (L::NC / L::W2) + p * 16;
        uint32_t fb[4];
        if (!BWD)
          ldsm4_t(ws + tile_at<L::NC / 8>(ks * 16 + (lane & 15), cc / 8 + (lane >> 4)), fb);
        else
          ldsm4(ws + tile_at<RP / 8>(cc + (lane & 7) + (lane >> 4) * 8,
                                     ks * 2 + ((lane >> 3) & 1)), fb);
#pragma unroll
        for (int w = L::TERMS - 1; w >= 0; --w) {   // the small terms first
          mma16816(c[2 * p], fa[w], fb[0], fb[1]);
          mma16816(c[2 * p + 1], fa[w], fb[2], fb[3]);
        }
      }
    }
    uint8_t* bs = smem + so + RP * L::NC * 2;
#pragma unroll
    for (int i = 0; i < L::NT2; ++i) {
      const int col = w2n * (L::NC / L::W2) + i * 8 + (lane & 3) * 2;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = wm * 16 + (lane >> 2) + h * 8, byte = col * L::OB;
        uint8_t* p = bs + tile_at<BC>(row, byte / 16) + byte % 16;
        if (!BWD) {
          uint32_t* q = reinterpret_cast<uint32_t*>(p);
          const uint32_t b = *q;
          *q = pack_bf16x2(__uint_as_float(b << 16) + c[i][2 * h],
                           __uint_as_float(b & 0xFFFF0000u) + c[i][2 * h + 1]);
        } else {
          float2* q = reinterpret_cast<float2*>(p);
          const float2 b = *q;
          *q = make_float2(b.x + c[i][2 * h], b.y + c[i][2 * h + 1]);
        }
      }
    }
    __syncthreads();
    const int col = nc * L::NC + tid % BC * PV;
#pragma unroll
    for (int i = 0; i < BR; ++i)
      if (bt[i] >= 0 && col < N)
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(g.out) +
                                  ((size_t)bt[i] * N + col) * L::OB) =
            *reinterpret_cast<const uint4*>(bs +
                                            tile_at<BC>(tid / BC + i * (256 / BC), tid % BC));
  }
  cp_wait<0>();
  if (L::AHEAD && CS > 1) cluster_sync_all();   // peers have read this CTA's partial sums
}

// --------------------------------------------------------------- gradient --

// On tcgen05: D (128 columns of x or dy, 3 r) = X^T [v0 | v1 | v2], the three
// terms side by side on the MMA's N, so that X is read from shared memory once
// for all of them; the epilogue adds a row's three column groups.  Both
// operands run down their rows on the contraction (MN-major, 128-byte swizzle:
// boxes of 64 columns x 32 rows).
// The rows, by tile slot, are cut into equal chunks, as many as give every SM
// two CTAs, whatever the adapters' sizes; a CTA walks the adapters that meet its
// chunk.  One that lies in it whole goes straight to the gradient; the part in
// chunk p of another, a, that starts in chunk p0 goes to the slot
// p + min(a, p0), and the last launch adds an adapter's parts in order.  (Of the
// cut adapters each starts in a chunk of its own and ends no later than the next one
// starts, so that both a and p0 grow from one to the next: no two parts share a
// slot, and there are fewer than chunks + min(n, chunks) of them.)  (One CTA per adapter and part
// instead ran in two uneven waves: 33 us against 25 at 8192 x 2048, rank 64.)
// Warps 0-3 read tensor memory, 4-7 gather x's rows into the stages by
// cp.async, 8 issues the MMAs, 9 loads the terms by TMA (its issue would hold
// up the rows' if they shared a warp).
constexpr int kGradCols = 128;   // columns of x (dA) or dy (dB) a CTA: the MMA's M
constexpr int kGradRows = 32;    // rows a stage
// Rows of a chunk, at most: the tensor core's fp32 sums of 1024 rows keep the
// gradients within 8e-7 of exact, normwise; the parts are added in
// round-to-nearest fp32.
constexpr int kGradMax = 1024;
constexpr int kGradBox = kGradRows * 128;           // 64 bf16 columns of a stage's rows
constexpr int kGradThreads = 320;
constexpr int kGradAux = 1024 + kGradMax * 4;       // barriers, tmem address, rows

// The MN-major descriptor: boxes along MN kGradBox apart, 8-row groups 1024
// bytes apart, 128-byte swizzle; a k step of 16 rows is 2048 bytes.
__device__ __forceinline__ uint64_t grad_desc(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(kGradBox >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// D fp32, A and B bf16, both MN-major, M = 128; N >> 3 at bit 17.
__device__ __forceinline__ uint32_t grad_idesc(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) |
         ((uint32_t)(kGradCols >> 4) << 24) | ((uint32_t)(n >> 3) << 17);
}

struct GradArgs {
  const __nv_bfloat16* x;   // (T, d)
  const __nv_bfloat16* dy;  // (T, d_out)
  float* dA;                // (n, d, r)
  float* dB;                // (n, r, d_out)
  float* part;              // (part_slots, r (d + d_out)): parts of cut adapters, dA's then dB's
  const int32_t* header;
  const int32_t* offsets;
  const int32_t* rows;
  int32_t* err;
  int T, n, r, d, d_out, TM, chunks;   // TM: the plan's tile rows
  int fold;   // no launch for the parts follows: adapters without rows are zeroed here
  int N, stage_bytes, tmem_cols;   // 3 r rounded up to 16; x's boxes and the terms'
};

// Adapter a's first row by tile slot.
__device__ __forceinline__ int first_row(const GradArgs& g, int a) {
  return (__ldg(g.offsets + a) / g.TM + a) * g.TM;
}
// Rows of a chunk: the adapters' tile slots in g.chunks equal parts, in whole
// stages.
__device__ __forceinline__ int chunk_rows(const GradArgs& g) {
  return ceil_div_dev(ceil_div_dev(first_row(g, g.n), g.chunks), kGradRows) * kGradRows;
}

// The parts of a chunk in order: rows [i0, i1) of adapter a, whose first row by
// tile slot is at `at`.
struct ChunkParts {
  const GradArgs& g;
  int lo, hi, len, a, at, i0, i1;
  bool whole;   // all of the adapter's rows
  // a0: the last adapter that starts at or before the chunk; len: rows of a chunk
  __device__ ChunkParts(const GradArgs& g_, int lo_, int hi_, int len_, int a0)
      : g(g_), lo(lo_), hi(hi_), len(len_), a(a0 - 1) {}
  // The part's slot.
  __device__ size_t slot(int chunk) const { return (size_t)(chunk + min(a, at / len)); }
  __device__ bool next() {
    while (++a < g.n) {
      const int o = __ldg(g.offsets + a), cnt = __ldg(g.offsets + a + 1) - o;
      at = (o / g.TM + a) * g.TM;
      if (at >= hi) return false;
      i0 = max(0, lo - at);
      i1 = min(cnt, hi - at);
      whole = i0 == 0 && i1 == cnt;
      if (i0 < i1) return true;
    }
    return false;
  }
};

// The last adapter a with first_row(a) <= row, or -1; by a converged warp.
__device__ __forceinline__ int find_adapter(const GradArgs& g, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = g.n;   // the answer + 1 is in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const bool le = i < hi && first_row(g, i) <= row;
    const int c = __popc(__ballot_sync(0xffffffffu, le));
    if (c == 0) break;
    hi = min(hi, lo + c * step);
    lo = lo + (c - 1) * step + 1;
  }
  return lo - 1;
}

template <int STAGES>
__global__ void __launch_bounds__(kGradThreads, 2)
    adapter_grad_kernel(const __grid_constant__ CUtensorMap mapU,
                        const __grid_constant__ CUtensorMap mapV,
                        const __grid_constant__ GradArgs g) {
  pdl_wait_and_release();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + STAGES * g.stage_bytes);
  uint64_t* empty_bar = full_bar + STAGES;
  uint64_t* d_full = empty_bar + STAGES;
  uint64_t* d_empty = d_full + 1;
  uint64_t* drained = d_empty + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drained + 1);
  int32_t* s_rows = reinterpret_cast<int32_t*>(smem + STAGES * g.stage_bytes + 256);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (__ldg(g.header) != g.T || __ldg(g.header + 1) != g.n) {
    if (tid == 0) report_error(g.err, kDevBadPlan);
    return;
  }
  const int mbx = ceil_div_dev(g.d, kGradCols), mbs = mbx + ceil_div_dev(g.d_out, kGradCols);
  const int chunk = blockIdx.x / mbs, mb = blockIdx.x - chunk * mbs;
  const int len = chunk_rows(g), lo = chunk * len;
  const int hi = min(lo + len, first_row(g, g.n));   // (T <= 2^30: no overflow)
  if (lo >= hi) return;
  // the chunk's rows are on their way while its first adapter is found
  constexpr int PRE = (kGradMax + kGradThreads - 1) / kGradThreads;
  int pre[PRE];
#pragma unroll
  for (int k = 0; k < PRE; ++k)
    pre[k] = tid + k * kGradThreads < hi - lo ? __ldg(g.rows + lo + tid + k * kGradThreads) : -1;
  const int a0 = max(0, find_adapter(g, lo));
  const bool isA = mb < mbx;
  const int m0 = (isA ? mb : mb - mbx) * kGradCols;
  const int M = isA ? g.d : g.d_out, r = g.r;
#pragma unroll
  for (int k = 0; k < PRE; ++k)
    if (tid + k * kGradThreads < kGradMax) s_rows[tid + k * kGradThreads] = pre[k];
  if (warp == 8) {
    tmem_alloc(tmem_holder, (uint32_t)g.tmem_cols);
    tmem_relinquish();
    if (lane == 0) {
      for (int s = 0; s < STAGES; ++s) {
        mbar_init(&full_bar[s], 129);  // each producer's copies, the terms' TMA
        mbar_init(&empty_bar[s], 1);   // the MMAs that read the stage
      }
      mbar_init(d_full, 1);
      mbar_init(d_empty, 4);           // the epilogue warps
      mbar_init(drained, 1);
      fence_mbar_init();
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_holder;
  ChunkParts part(g, lo, hi, len, a0);

  if (warp >= 4 && warp < 8) {
    // ---- producers
    const __nv_bfloat16* X = isA ? g.x : g.dy;
    const int p = tid - 128, c = p % 16, col = m0 + c * 8;
    // rows 8 apart: the swizzle is the same for all four
    const uint32_t dst = (uint32_t)(c / 8) * kGradBox + tile_at<8>(p / 16, c % 8);
    bool alive = true;
    for (int s = 0; alive && part.next();) {
      for (int i = part.i0; i < part.i1; i += kGradRows, ++s) {
        uint64_t* bar = &full_bar[s % STAGES];
        if (s >= STAGES) {
          alive = mbar_wait(&empty_bar[s % STAGES], (uint32_t)(s / STAGES - 1) & 1u);
          alive = __all_sync(0xffffffffu, alive);
          if (!alive) {
            report_error(g.err, kDevTimeoutProducer);
            break;
          }
        }
        uint8_t* stage = smem + (s % STAGES) * g.stage_bytes;
        const uint32_t xs = smem_u32(stage);
        const __nv_bfloat16* src[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int at = i + p / 16 + 8 * k;
          src[k] = at < part.i1 && col < M ? X + (size_t)s_rows[part.at + at - lo] * M + col
                                           : nullptr;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          cp_async16(dst + xs + k * 8 * 128, src[k] != nullptr ? src[k] : X, src[k] != nullptr);
        cp_arrive(bar);
      }
    }
    cp_wait_all();
  } else if (warp < 4) {
    // ---- epilogue: lane = column of x, tensor-memory columns = the three terms
    const size_t dsz = (size_t)g.d * r, bsz = (size_t)g.d_out * r;
    const int m = m0 + warp * 32 + lane;
    const uint32_t acc = tmem + ((uint32_t)(warp * 32) << 16);
    uint32_t ph = 0;
    while (part.next()) {
      if (!__all_sync(0xffffffffu, mbar_wait(d_full, ph))) {
        report_error(g.err, kDevTimeoutEpilogue);
        break;
      }
      ph ^= 1u;
      tc_fence_after_sync();
      const int a = part.a;
      float* out = part.whole
                       ? (isA ? g.dA + (size_t)a * dsz : g.dB + (size_t)a * bsz)
                       : g.part + part.slot(chunk) * (dsz + bsz) + (isA ? 0 : dsz);
      for (int j0 = 0; j0 < r; j0 += 16) {
        uint32_t t[2][3][8];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (j0 + 8 * h < r)
#pragma unroll
            for (int w = 0; w < 3; ++w)
              tmem_ld_32x32b_x8(acc + (uint32_t)(w * r + j0 + 8 * h), t[h][w]);
        tmem_ld_wait();
        if (j0 + 16 >= r) {
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(d_empty);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int j = j0 + 8 * h;
          if (j >= r || m >= M) continue;
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            v[i] = __uint_as_float(t[h][0][i]) +
                   (__uint_as_float(t[h][1][i]) + __uint_as_float(t[h][2][i]));
          if (isA) {
            float4* o = reinterpret_cast<float4*>(out + (size_t)m * r + j);
            o[0] = make_float4(v[0], v[1], v[2], v[3]);
            o[1] = make_float4(v[4], v[5], v[6], v[7]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) out[(size_t)(j + i) * M + m] = v[i];
          }
        }
      }
    }
    for (int a = 0; g.fold && a < g.n; ++a) {
      if (__ldg(g.offsets + a) != __ldg(g.offsets + a + 1)) continue;
      const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
      if (isA) {   // this CTA's rows of dA are one block
        float4* o = reinterpret_cast<float4*>(g.dA + (size_t)a * dsz + (size_t)m0 * r);
        for (int i = tid; i < min(kGradCols, M - m0) * r / 4; i += 128) o[i] = zero;
      } else if (m0 + lane * 4 < M) {
        float* o = g.dB + (size_t)a * bsz + m0 + lane * 4;
        for (int j = warp; j < r; j += 4) *reinterpret_cast<float4*>(o + (size_t)j * M) = zero;
      }
    }
  } else if (warp == 9) {
    // ---- the terms
    const CUtensorMap* terms = isA ? &mapV : &mapU;
    const int boxes = g.stage_bytes / kGradBox - 2;
    bool alive = lane == 0;
    for (int s = 0; alive && part.next();) {
      for (int i = part.i0; i < part.i1; i += kGradRows, ++s) {
        uint64_t* bar = &full_bar[s % STAGES];
        if (s >= STAGES) {
          alive = mbar_wait(&empty_bar[s % STAGES], (uint32_t)(s / STAGES - 1) & 1u);
          if (!alive) {
            report_error(g.err, kDevTimeoutProducer);
            break;
          }
        }
        uint8_t* stage = smem + (s % STAGES) * g.stage_bytes;
        mbar_arrive_expect_tx(bar, (uint32_t)(boxes * kGradBox));
        for (int b = 0; b < boxes; ++b)
          tma_load_3d(stage + (2 + b) * kGradBox, terms, bar, b * 64, part.at + i, 0);
      }
    }
  } else {
    // ---- MMA issuer: the whole warp runs the loop, one lane issues
    auto wait = [](uint64_t* bar, uint32_t ph) {
      return (bool)__all_sync(0xffffffffu, mbar_wait(bar, ph));
    };
    bool alive = true;
    int s = 0, q = 0;
    for (; alive && part.next(); ++q) {
      if (q > 0) alive = wait(d_empty, (uint32_t)(q - 1) & 1u);
      tc_fence_after_sync();
      uint32_t more = 0;
      for (int i = part.i0; alive && i < part.i1; i += kGradRows, ++s) {
        alive = wait(&full_bar[s % STAGES], (uint32_t)(s / STAGES) & 1u);
        if (!alive) break;
        fence_proxy_async_smem();   // the copies' writes, before the tensor core reads them
        tc_fence_after_sync();
        const uint32_t xs = smem_u32(smem + (s % STAGES) * g.stage_bytes), vs = xs + 2 * kGradBox;
        // (the terms' rows behind the adapter's last tile are not its own)
        const int steps = ceil_div_dev(min(kGradRows, part.i1 - i), 16);
        for (int kk = 0; kk < steps; ++kk) {
          const uint64_t ad = grad_desc(xs + kk * 2048);
          umma_elect(tmem, ad, grad_desc(vs + kk * 2048), grad_idesc(min(g.N, 256)), more);
          if (g.N > 256)
            umma_elect(tmem + 256, ad, grad_desc(vs + 4 * kGradBox + kk * 2048),
                       grad_idesc(g.N - 256), more);
          more = 1;
        }
        umma_commit_elect(&empty_bar[s % STAGES]);
      }
      umma_commit_elect(d_full);
    }
    if (!alive) report_error(g.err, kDevTimeoutMma);
    umma_commit_elect(drained);
    if (!wait(drained, 0)) report_error(g.err, kDevTimeoutDrain);
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, (uint32_t)g.tmem_cols);
  }
}

// Adapters in parts: the parts added in order; adapters without rows: zeros.
__global__ void __launch_bounds__(256) adapter_reduce_kernel(GradArgs g) {
  pdl_wait_and_release();
  if (__ldg(g.header) != g.T || __ldg(g.header + 1) != g.n) return;
  const int a = blockIdx.y;
  const int at = first_row(g, a), cnt = __ldg(g.offsets + a + 1) - __ldg(g.offsets + a);
  const int len = chunk_rows(g), p0 = len > 0 ? at / len : 0;
  const int parts = cnt > 0 ? (at + cnt - 1) / len - p0 + 1 : 0;
  if (parts == 1) return;
  const size_t dsz = (size_t)g.d * g.r, bsz = (size_t)g.d_out * g.r, all = dsz + bsz;
  const float* src = g.part + (size_t)(p0 + min(a, p0)) * all;
  for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4; i < all;
       i += (size_t)gridDim.x * 1024) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int b = 0; b < parts; ++b) {
      const float4 p = *reinterpret_cast<const float4*>(src + (size_t)b * all + i);
      s.x += p.x;
      s.y += p.y;
      s.z += p.z;
      s.w += p.w;
    }
    float* dst = i < dsz ? g.dA + (size_t)a * dsz + i : g.dB + (size_t)a * bsz + (i - dsz);
    *reinterpret_cast<float4*>(dst) = s;
  }
}

int rank_pad(int r) { return r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128; }

// Rows of a tile: 16 where there are few rows, in all or an adapter (decode; n counts
// the adapters loaded, since those in use are known on the device alone),
// so that they spread over the SMs and a tile is not mostly padding.  Forward and
// backward on B200, 2048 columns, us (16 against 64 rows): 1000 rows on 4
// adapters, rank 64, 47 / 52; 2000 on 100, rank 16, 75 / 87; but 1500 on 4, rank
// 64, 67 / 57, and 4000 on 100, rank 64, 180 / 145.
int tile_rows(int T, int n) { return T <= 1024 || T <= 32 * n ? 16 : 64; }

int max_tiles(int T, int n) { return T / tile_rows(T, n) + n + 1; }

// Whether the low-rank products run on tcgen05, a CTA (and an SM) to a tile of
// 64 rows, by the tiles (each adapter's last one in part): where they give work to
// more than half of the SMs; a quarter for ranks above 64, whose products weigh
// more, two thirds up to rank 16.  Fewer tiles are shared by clusters of CTAs on
// mma.sync instead.  Forward and backward on B200, 2048 columns, us (tcgen05
// against mma.sync): 8192 rows on 8 adapters, rank 64, 98 / 132; 4000 on 100, 145
// / 242; 4500 on 4, 83 / 112, but 3200 on 12, 83.4 / 82.7; rank 16: 6600 on 6, 86 /
// 93, but 5800 on 6, 81 / 75; rank 128, 4096 columns: 3200 on 8, 166 / 200.
bool use_tc(int T, int n, int r) {
  const int tiles = T / 64 + n, sms = device_sm_count();
  return tile_rows(T, n) == 64 && tiles > (r > 64 ? sms / 4 : r > 16 ? sms / 2 : sms * 2 / 3);
}

// Rows by tile slot (the plan's, and u's and v's terms): whole tiles.
size_t term_rows(int T, int n) { return (size_t)max_tiles(T, n) * tile_rows(T, n); }

// Chunks of the gradient's rows: two CTAs an SM, but 256 rows at least (a part's
// trip through memory costs more), unless adapters are so small that a chunk
// would walk more than about four of them, and kGradMax at most.  Forward and
// backward on B200, us: 1000 rows of 2048 on 4 adapters, rank 64, 47, with 128
// rows at least 49; 64 rows of 4096 on 64, rank 16, 53, with 512 at least 59; 32
// rows of 408 on 27, rank 40, 27, by rows alone 41.
int grad_chunks(const moe_config_t& c, int n) {
  const int mb = ceil_div(c.d, kGradCols) + ceil_div(c.d_out, kGradCols);
  const int64_t rows = (int64_t)term_rows(c.T, n);
  const int even = (int)std::min<int64_t>(2 * device_sm_count() / mb,
                                          std::max<int64_t>(rows / 256, n / 4));
  return std::max(std::max(1, even), (int)((rows + kGradMax - kGradRows - 1) /
                                           (kGradMax - kGradRows)));
}

// Slots of the parts (adapter_grad_kernel).
size_t part_slots(int chunks, int n) { return (size_t)chunks + std::min(n, chunks); }

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

AdapterPlanLayout adapter_plan_layout(const moe_config_t& c, int n) {
  AdapterPlanLayout L{};
  L.ctrl = 0;
  L.header = 64;   // cleared by moe_workspace_init: a plan not made fits no call
  L.offsets = 256;
  L.rows = L.offsets + up256((size_t)(n + 2) * 4);
  L.tiles = L.rows + up256(term_rows(c.T, n) * 4);
  L.total = L.tiles + up256((size_t)max_tiles(c.T, n) * 8);
  return L;
}

AdapterWsLayout adapter_ws_layout(const moe_config_t& c, int n, int r) {
  AdapterWsLayout L{};
  L.v = 0;
  L.u = up256(term_rows(c.T, n) * r * 6);
  L.part = 2 * L.u;
  L.total = L.part + up256(part_slots(grad_chunks(c, n), n) * r * ((size_t)c.d + c.d_out) * 4);
  return L;
}

cudaError_t launch_adapter_plan(const moe_config_t& c, int n, const int32_t* ids, void* plan,
                                cudaStream_t s) {
  const AdapterPlanLayout L = adapter_plan_layout(c, n);
  uint8_t* p = static_cast<uint8_t*>(plan);
  return launch_kernel(adapter_plan_kernel, n + 1, kPlanThreads, 0, s, 0, ids, c.T, n,
                       tile_rows(c.T, n), reinterpret_cast<int32_t*>(p + L.header),
                       reinterpret_cast<int32_t*>(p + L.offsets),
                       reinterpret_cast<int32_t*>(p + L.rows),
                       reinterpret_cast<int2*>(p + L.tiles), reinterpret_cast<int32_t*>(p));
}

namespace {

LowRankArgs low_rank_args(const AdapterCall& a) {
  const AdapterPlanLayout P = adapter_plan_layout(*a.c, a.n);
  uint8_t* p = static_cast<uint8_t*>(a.plan);
  return LowRankArgs{a.in, a.W1, a.W2, a.scale, a.base, a.out, a.u, a.up, a.vp,
                     reinterpret_cast<const int32_t*>(p + P.header),
                     reinterpret_cast<const int32_t*>(p + P.rows),
                     reinterpret_cast<const int2*>(p + P.tiles), reinterpret_cast<int32_t*>(p),
                     a.c->T, a.n, a.r, a.K, a.N};
}

template <int RP, int TM, bool BWD>
cudaError_t run_low_rank(const AdapterCall& a, cudaStream_t s) {
  using L = LowRank<RP, TM, BWD>;
  // CTAs of a tile's cluster: as many as the SMs hold at a time.  (Past that a
  // second wave starts: 4500 rows take 112 us where 4096 take 82.)
  const int tiles = max_tiles(a.c->T, a.n);
  const int most = std::min(ceil_div(a.K, L::KC), ceil_div(a.N, L::NC));
  const int64_t room = (int64_t)std::min(L::CTAS, 4) * device_sm_count();
  int cs = 1;
  while (cs < 8 && cs * 2 <= most && (int64_t)tiles * cs * 2 <= room) cs *= 2;
  const auto kern = low_rank_kernel<RP, TM, BWD>;
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), L::SMEM);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, (unsigned)tiles * cs, 256, L::SMEM, s, cs, low_rank_args(a));
}

template <int RP, bool BWD>
cudaError_t run_tm(const AdapterCall& a, cudaStream_t s) {
  return tile_rows(a.c->T, a.n) == 16 ? run_low_rank<RP, 16, BWD>(a, s)
                                      : run_low_rank<RP, 64, BWD>(a, s);
}

template <bool BWD>
cudaError_t run_rank(const AdapterCall& a, cudaStream_t s) {
  switch (rank_pad(a.r)) {
    case 16: return run_tm<16, BWD>(a, s);
    case 32: return run_tm<32, BWD>(a, s);
    case 64: return run_tm<64, BWD>(a, s);
    default: return run_tm<128, BWD>(a, s);
  }
}

template <int STAGES>
cudaError_t run_grad(const CUtensorMap& mapU, const CUtensorMap& mapV, const GradArgs& g,
                     cudaStream_t s) {
  const auto kern = adapter_grad_kernel<STAGES>;
  const int smem = STAGES * g.stage_bytes + 1024 + kGradAux;
  // the limit is set once per kernel: to the most any rank takes
  const int most = STAGES * (STAGES == 6 ? 8 : STAGES == 5 ? 5 : 6) * kGradBox + 1024 + kGradAux;
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), most);
  if (e != cudaSuccess) return e;
  const unsigned grid =
      (unsigned)(ceil_div(g.d, kGradCols) + ceil_div(g.d_out, kGradCols)) * (unsigned)g.chunks;
  return launch_kernel(kern, grid, kGradThreads, smem, s, 0, mapU, mapV, g);
}

}  // namespace

cudaError_t launch_adapter(const AdapterCall& a, bool backward, cudaStream_t s) {
  if (a.c->T == 0) return cudaSuccess;
  if (use_tc(a.c->T, a.n, a.r))
    return launch_low_rank_tc(low_rank_args(a), backward, max_tiles(a.c->T, a.n), s);
  return backward ? run_rank<true>(a, s) : run_rank<false>(a, s);
}

cudaError_t launch_adapter_grad(const moe_config_t& c, int n, int r, void* plan, const void* x,
                                const void* dy, float* dA, float* dB, void* ws, cudaStream_t s) {
  const size_t dsz = (size_t)c.d * r * n * 4, bsz = (size_t)c.d_out * r * n * 4;
  if (c.T == 0) {
    cudaError_t e = cudaMemsetAsync(dA, 0, dsz, s);
    return e == cudaSuccess ? cudaMemsetAsync(dB, 0, bsz, s) : e;
  }
  const AdapterPlanLayout P = adapter_plan_layout(c, n);
  const AdapterWsLayout W = adapter_ws_layout(c, n, r);
  uint8_t* p = static_cast<uint8_t*>(plan);
  uint8_t* w = static_cast<uint8_t*>(ws);
  // The terms' boxes of 64 columns; two CTAs an SM by shared and tensor memory
  // up to 256 columns (rank 80), one above.
  const int N = ceil_div(3 * r, 16) * 16, boxes = ceil_div(N, 64);
  int cols = 32;
  while (cols < N) cols *= 2;
  // One chunk of rows has no parts to add, and few adapters: their zeros, where
  // they have no rows, are written without a launch.  All of a step, us (without
  // that launch against with): 333 rows, 5 adapters 27.4 / 30.3; 300 rows, 4
  // adapters of 4096 41.3 / 44.0.
  const int chunks = grad_chunks(c, n);
  const int fold = chunks == 1;
  const GradArgs g{static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(dy),
                   dA, dB,
                   reinterpret_cast<float*>(w + W.part),
                   reinterpret_cast<const int32_t*>(p + P.header),
                   reinterpret_cast<const int32_t*>(p + P.offsets),
                   reinterpret_cast<const int32_t*>(p + P.rows), reinterpret_cast<int32_t*>(p),
                   c.T, n, r, c.d, c.d_out, tile_rows(c.T, n), chunks, fold, N,
                   (2 + boxes) * kGradBox, cols};
  CUtensorMap mapU, mapV;
  const uint64_t rows = term_rows(c.T, n);
  if (!encode_bf16(&mapU, w + W.u, 1, rows, 3 * (uint64_t)r, kGradRows) ||
      !encode_bf16(&mapV, w + W.v, 1, rows, 3 * (uint64_t)r, kGradRows))
    return cudaErrorNotSupported;
  cudaError_t e = boxes == 4   ? run_grad<4>(mapU, mapV, g, s)
                  : boxes == 3 ? run_grad<5>(mapU, mapV, g, s)
                               : run_grad<6>(mapU, mapV, g, s);
  if (e != cudaSuccess || fold != 0) return e;
  const int per = std::max(1, std::min(ceil_div((c.d + c.d_out) * r, 1024),
                                       ceil_div(8 * device_sm_count(), n)));
  return launch_kernel(adapter_reduce_kernel, dim3((unsigned)per, (unsigned)n), 256, 0, s, 0, g);
}

}  // namespace moe
