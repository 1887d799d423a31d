// balance.cu - the load-balancing loss and the router z-loss of packed, padded
// sequences, with per-expert counts and the gradient of the logits.
//
// The whole-batch form is "Mixture-of-Experts Routing - LLM Internals"
// (mlgrind.dev), Algorithm 4: aux = E * sum_e f_e P_e.  Here each sequence s
// of a packed batch has its own f and P over its n_s counted tokens (those
// whose mask byte is not 0), the S+ sequences with a counted token weigh the
// same, and z is the mean squared log-sum-exp over all N counted tokens:
//
//   f[s,e] = counts[s,e] / (n_s k)     P[s,e] = mean_t softmax(l_t)[e]
//   balance = 1/S+ sum_s E sum_e f[s,e] P[s,e]      z = 1/N sum_t lse(l_t)^2
//   dl[t,e] = p_te (a_se - sum_e' p_te' a_se' + dz 2 lse_t / N)
//             a_se = dbalance E f[s,e] / (S+ n_s)
//   (f counts slots and carries no gradient; rows not counted get 0)
//
// Both directions are one pass over the logits: bound by HBM for large T x E
// (B200, 131072 x 256: first launch 34 us, 4.1 TB/s, where load latency and issue
// slots count too; second 13; backward 46, 5.9 TB/s), by launch latency below
// about a million logits.  A token's E logits sit in
// the registers of G <= 16 lanes (32 where they cannot be read by 16-byte
// vectors), so a warp works on 32 / G tokens at once; maximum and sum are
// butterflies over the G lanes, in fp32.
//
// Summation order (no floating-point atomics, nothing depends on which CTA
// runs first): a warp owns C consecutive tokens and walks the sequences that
// meet them; each such piece gets the slot (warp + s) of the partial sums,
// which no other piece has (going to the next warp or the next sequence
// raises it by at least one), so no scan over the sequences is needed.  Where
// one sequence covers all 8 warps of a CTA, their sums are added and only the
// first warp's slot is written.  The second launch adds a sequence's slots in a
// fixed order in fp64.  A warp's fp32 sums cover at most 64 tokens, and a CTA's 8 of
// them are added in pairs; in batches whose warps own more (C > 64, above 303103
// tokens) both go on in fp64, blocks of 64 tokens in shared memory.
#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kLogWarps = 3, kWarps = 1 << kLogWarps;
constexpr int kLogSum = 6, kSumTokens = 1 << kLogSum;   // tokens of a warp's fp32 sums

// The number of i in [1, S] with off[i] <= t, for non-decreasing off: the
// sequence that holds token t if off[0] <= t < off[S].  32 samples a round.
__device__ __forceinline__ int warp_find_seq(const int32_t* __restrict__ off, int S, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = S;
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const long long i = lo + (long long)lane * step;
    const bool le = i < hi && __ldg(off + i + 1) <= t;
    const int c = __popc(__ballot_sync(0xffffffffu, le));
    if (c == 0) return lo;
    const long long nhi = lo + (long long)c * step;
    lo = lo + (c - 1) * step + 1;
    hi = nhi < hi ? (int)nhi : hi;
  }
  return lo;
}

// Bounds of sequence s inside [0, T] whatever the offsets hold; false if they
// had to be moved there.
__device__ __forceinline__ bool seq_bounds(const int32_t* __restrict__ off, int s, int T, int& lo,
                                           int& hi) {
  if (off == nullptr) {
    lo = 0;
    hi = T;
    return true;
  }
  const int a = __ldg(off + s), b = __ldg(off + s + 1);
  lo = min(max(a, 0), T);
  hi = min(max(b, lo), T);
  return lo == a && hi == b;
}

template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// How a token's experts lie in the G lanes of its group: NV a lane, by 16-byte
// vectors (VEC: E a multiple of 4, rows 16-byte aligned) or one by one.
template <int G_, int NV_, bool VEC_>
struct Lanes {
  static constexpr int G = G_, NV = NV_;
  static constexpr bool VEC = VEC_;
  static constexpr int W = 32 / G;   // tokens a warp works on at once
  // The expert of this lane's value i.
  static __device__ __forceinline__ int expert(int gl, int i) {
    return VEC ? 4 * (gl + G * (i / 4)) + i % 4 : gl + G * i;
  }
};

// This lane's logits of token t, -inf beyond the last expert; a token that is not
// in is not read: zeros, whose softmax is finite.
template <typename L>
__device__ __forceinline__ void load_logits(const float* __restrict__ logits, int t, bool in,
                                            int E, int gl, float (&v)[L::NV]) {
  const float* row = logits + (size_t)t * E;
  const float fill = in ? -INFINITY : 0.f;
  if constexpr (L::VEC) {
#pragma unroll
    for (int i = 0; i < L::NV; i += 4) {
      const int e = L::expert(gl, i);
      float4 q = make_float4(fill, fill, fill, fill);
      if (in && e < E) q = __ldg(reinterpret_cast<const float4*>(row + e));
      v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < L::NV; ++i) {
      const int e = L::expert(gl, i);
      v[i] = in && e < E ? __ldg(row + e) : fill;
    }
  }
}

// This lane's values of a row of E floats to memory.
template <typename L>
__device__ __forceinline__ void store_values(float* row, int E, int gl, const float (&v)[L::NV]) {
  if constexpr (L::VEC) {
#pragma unroll
    for (int i = 0; i < L::NV; i += 4) {
      const int e = L::expert(gl, i);
      if (e < E)
        *reinterpret_cast<float4*>(row + e) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < L::NV; ++i) {
      const int e = L::expert(gl, i);
      if (e < E) row[e] = v[i];
    }
  }
}

// This lane's values into a row of fp64 sums (first), or added to it.
template <typename L>
__device__ __forceinline__ void add_values(double* row, int E, int gl, bool first,
                                           const float (&v)[L::NV]) {
#pragma unroll
  for (int i = 0; i < L::NV; ++i) {
    const int e = L::expert(gl, i);
    if (e < E) row[e] = (first ? 0.0 : row[e]) + (double)v[i];
  }
}

// exp(l - max) of this lane's experts, their sum's inverse and the token's
// log-sum-exp, from the G lanes' logits.  Where act is false they are zeros, and
// so are inv and lse.
// exp(d), d = l - m <= 0, is 2^(d log2 e): one product and the hardware's 2^x,
// within 2.3 |d| + 4 half steps of fp32, and 0 below 2^-126.  Weighed by the shares
// |d| averages at most ln E <= 5.6, so that the sum, of 21 additions at most in a
// chain, is within 38 and p within 2.3 |d| + 44.  (One fused 2^(l log2e - m log2e) would
// overflow for logits at the type's lowest value.)  With expf the forward's first
// launch took 57 us, against 44, at 131072 x 256.
template <typename L>
__device__ __forceinline__ void softmax_terms(float (&v)[L::NV], bool act, float& inv,
                                              float& lse) {
  constexpr float kLog2e = 1.44269504f;
  float m = v[0];
#pragma unroll
  for (int i = 1; i < L::NV; ++i) m = fmaxf(m, v[i]);
  m = group_max<L::G>(m);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < L::NV; ++i) {
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(v[i]) : "f"((v[i] - m) * kLog2e));
    sum += v[i];
  }
  sum = group_sum<L::G>(sum);
  inv = act ? 1.f / sum : 0.f;
  lse = act ? m + logf(sum) : 0.f;
}

struct BalanceParts {
  float* p;        // (slots, E) sums of probabilities
  int32_t* c;      // (slots, E) routing slots per expert
  int32_t* n;      // (slots) counted tokens
  float* z;        // (slots) sums of lse^2
};

// The slots of a sequence [lo, hi) in order: the warps of a CTA it covers in
// part, one per CTA it covers whole, the warps of the last CTA in part.
struct SeqSlots {
  int s, first, nh, jm, nm, tail, nt;
  __device__ SeqSlots(int s_, int lo, int hi, int T, int lc) : s(s_) {
    first = nh = jm = nm = tail = nt = 0;
    if (lo >= hi) return;
    const int lcc = lc + kLogWarps;   // log2 of a CTA's tokens
    const int j0 = lo >> lcc, j1 = (hi - 1) >> lcc;
    const bool from = lo == j0 << lcc;
    const bool upto = hi >= (int)min((long long)T, (long long)(j1 + 1) << lcc);
    first = lo >> lc;
    if (j0 == j1 && !(from && upto)) {
      nh = ((hi - 1) >> lc) - first + 1;
      return;
    }
    jm = from ? j0 : j0 + 1;
    nh = from ? 0 : (j0 + 1) * kWarps - first;
    nm = (upto ? j1 + 1 : j1) - jm;
    tail = j1 * kWarps;
    nt = upto ? 0 : ((hi - 1) >> lc) - tail + 1;
  }
  __device__ int count() const { return nh + nm + nt; }
  __device__ size_t operator()(int i) const {
    const int w = i < nh ? first + i : i < nh + nm ? kWarps * (jm + i - nh) : tail + (i - nh - nm);
    return (size_t)w + s;
  }
};

struct BalanceOut {
  int32_t* counts;     // (S, E)
  float* prob_mean;    // (S, E)
  int32_t* tokens;     // (S + 2)
  float* losses;       // (2)
  double* terms;       // (S, 2): a sequence's share of both losses
};

// A CTA's shared memory for the sums below; EP threads (a power of two >= E)
// stand for the experts, NT / EP groups of them walk a sequence's slots.
template <int NT>
struct FinishSmem {
  double p[NT];
  int32_t c[NT];
  double d[2][NT / 32];
  int32_t i[2][NT / 32];
};

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Counts, P, n and the loss terms of sequence s, by the whole CTA.
template <int NT>
__device__ void finish_sequence(FinishSmem<NT>& sm, const BalanceParts& part,
                                const int32_t* __restrict__ off, int s, int T, int E, int k, int lc,
                                int EP, const BalanceOut& out, int32_t* err) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ng = NT / EP, e = tid & (EP - 1), gi = tid / EP;
  int lo, hi;
  if (!seq_bounds(off, s, T, lo, hi) && tid == 0) report_error(err, kDevBadOffsets);
  const SeqSlots slots(s, lo, hi, T, lc);
  const int ni = slots.count();
  double p = 0.0, z = 0.0;
  int c = 0, n = 0;
  if (e < E) {
    constexpr int U = 16;   // slots in flight
    for (int i = gi; i < ni; i += U * ng) {
      float pv[U];
      int cv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool in = i + u * ng < ni;
        const size_t at = in ? slots(i + u * ng) * E + e : 0;
        pv[u] = in ? __ldcg(part.p + at) : 0.f;
        cv[u] = in ? __ldcg(part.c + at) : 0;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        p += (double)pv[u];
        c += cv[u];
      }
    }
  }
  for (int i = tid; i < ni; i += NT) {
    const size_t at = slots(i);
    n += __ldcg(part.n + at);
    z += (double)__ldcg(part.z + at);
  }
  n = __reduce_add_sync(0xffffffffu, n);
  z = warp_sum(z);
  __syncthreads();   // the last sequence's sums have been read
  sm.p[tid] = p;
  sm.c[tid] = c;
  if (lane == 0) {
    sm.i[0][warp] = n;
    sm.d[0][warp] = z;
  }
  __syncthreads();
  n = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) n += sm.i[0][w];
  double term = 0.0;
  if (tid < E) {
    p = 0.0;
    c = 0;
    for (int j = 0; j < ng; ++j) {
      p += sm.p[j * EP + tid];
      c += sm.c[j * EP + tid];
    }
    const double inv = n > 0 ? 1.0 / (double)n : 0.0;
    const double P = p * inv;
    out.counts[(size_t)s * E + tid] = c;
    out.prob_mean[(size_t)s * E + tid] = (float)P;
    term = (double)c * inv * P;   // k f P
  }
  term = warp_sum(term);
  if (lane == 0) sm.d[1][warp] = term;
  __syncthreads();
  if (tid == 0) {
    z = term = 0.0;
    for (int w = 0; w < NT / 32; ++w) {
      z += sm.d[0][w];
      term += sm.d[1][w];
    }
    out.tokens[s] = n;
    out.terms[2 * (size_t)s] = term * E / k;
    out.terms[2 * (size_t)s + 1] = z;
  }
}

// The sequences' terms into the losses, N and S+, by the whole CTA.
template <int NT>
__device__ void finish_totals(FinishSmem<NT>& sm, int S, const BalanceOut& out) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  double b = 0.0, z = 0.0;
  int n = 0, live = 0;
  for (int s = tid; s < S; s += NT) {
    const int ns = __ldcg(out.tokens + s);
    b += __ldcg(out.terms + 2 * (size_t)s);
    z += __ldcg(out.terms + 2 * (size_t)s + 1);
    n += ns;
    live += ns > 0;
  }
  b = warp_sum(b);
  z = warp_sum(z);
  n = __reduce_add_sync(0xffffffffu, n);
  live = __reduce_add_sync(0xffffffffu, live);
  __syncthreads();
  if (lane == 0) {
    sm.d[0][warp] = b;
    sm.d[1][warp] = z;
    sm.i[0][warp] = n;
    sm.i[1][warp] = live;
  }
  __syncthreads();
  if (tid == 0) {
    b = z = 0.0;
    n = live = 0;
    for (int w = 0; w < NT / 32; ++w) {
      b += sm.d[0][w];
      z += sm.d[1][w];
      n += sm.i[0][w];
      live += sm.i[1][w];
    }
    out.losses[0] = live > 0 ? (float)(b / (double)live) : 0.f;
    out.losses[1] = n > 0 ? (float)(z / (double)n) : 0.f;
    out.tokens[S] = n;
    out.tokens[S + 1] = live;
  }
}

// True in every thread of the last CTA of the grid to get here; what the
// others wrote before is then visible through L2.
__device__ __forceinline__ bool last_cta(unsigned* done) {
  __shared__ bool last;
  __syncthreads();   // the release below covers the whole CTA's writes
  if (threadIdx.x == 0) {
    last = atom_add_acq_rel_gpu(done, 1u) == gridDim.x - 1;
    if (last) *done = 0;
  }
  __syncthreads();
  return last;
}

// kFused: the last CTA also adds up the sequences (few CTAs and sequences:
// the second launch would cost more than its work; 64 x 8 in both directions: 11.6
// us against 14.0).
// kLong: a warp owns more than kSumTokens tokens, and keeps fp64 sums of its blocks of
// that many in dynamic shared memory (fp64 for shorter batches too cost 16384 x 64
// in both directions 21.5 us against 20.5).
enum PartialForm { kFused, kPlain, kLong };
constexpr int kWideBytes = (kWarps * 256 + kWarps) * 8;   // kLong's p, then z

// a[0] + ... + a[kWarps - 1], `step` apart, in pairs.
__device__ __forceinline__ float pair_sum(const float* a, int step) {
  float v[kWarps];
#pragma unroll
  for (int w = 0; w < kWarps; ++w) v[w] = a[w * step];
#pragma unroll
  for (int o = 1; o < kWarps; o *= 2)
#pragma unroll
    for (int w = 0; w < kWarps; w += 2 * o) v[w] += v[w + o];
  return v[0];
}

__device__ __forceinline__ float wide_sum(const double* a, int step) {
  double v = 0.0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) v += a[w * step];
  return (float)v;
}

// This lane's values and z, summed over the warp's groups of G lanes.
template <int G, int NV>
__device__ __forceinline__ void warp_groups_sum(float (&v)[NV], float& z) {
#pragma unroll
  for (int o = 16; o >= G; o >>= 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    z += __shfl_xor_sync(0xffffffffu, z, o);
  }
}

template <typename L, PartialForm FORM>
__global__ void __launch_bounds__(256, 4)
    balance_partial_kernel(const float* __restrict__ logits, const int32_t* __restrict__ idx,
                           const int32_t* __restrict__ off, const uint8_t* __restrict__ mask,
                           int T, int E, int k, int S, int lc, BalanceParts part, int EP,
                           BalanceOut out, unsigned* done, int32_t* err) {
  pdl_wait_and_release();
  __shared__ int32_t hist[kWarps][256];
  __shared__ __align__(16) float red[kWarps][256];
  __shared__ int32_t red_n[kWarps];
  __shared__ float red_z[kWarps];
  __shared__ int first_seq[kWarps];
  extern __shared__ double wide[];   // kLong
  constexpr int G = L::G, W = L::W, NV = L::NV;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane / G, gl = lane % G;
  const int C = 1 << lc, gw = blockIdx.x * kWarps + warp;
  const int c0 = blockIdx.x * kWarps * C;
  const int c1 = (int)min((long long)T, (long long)c0 + kWarps * C);
  const int t0 = (int)min((long long)c1, (long long)c0 + warp * C);
  const int t1 = (int)min((long long)c1, (long long)t0 + C);
  // the first tokens' logits are on their way while their sequence is found
  float nxt[NV];
  load_logits<L>(logits, t0 + g, t0 + g < t1, E, gl, nxt);
  int lo, hi;
  int s = off == nullptr ? 0 : warp_find_seq(off, S, t0);
  if (lane == 0) first_seq[warp] = s;
  __syncthreads();
  const int s0 = first_seq[0];
  double* wide_p = wide + warp * 256;
  double* wide_z = wide + kWarps * 256 + warp;
  auto counted = [&](int t, int end) {
    return t < end && (mask == nullptr || __ldg(mask + t) != 0);
  };
  bool merged = false;   // one sequence holds the whole CTA's tokens
  if (s0 < S) {
    seq_bounds(off, s0, T, lo, hi);
    merged = lo <= c0 && hi >= c1;
  }
  if (merged) s = s0;    // (a warp without tokens may have found another)
  // the rest of the loop runs per warp; merged is the same for all of them
  for (; s < S; ++s) {
    seq_bounds(off, s, T, lo, hi);
    if (!merged && lo >= t1) break;
    const int b = max(lo, t0), e1 = min(hi, t1);
    if (!merged && b >= e1) continue;
    if (b != t0) load_logits<L>(logits, b + g, b + g < e1, E, gl, nxt);
    bool nact = counted(b + g, e1), nact2 = counted(b + W + g, e1);
    if (!nact) {   // read ahead: may hold anything
#pragma unroll
      for (int i = 0; i < NV; ++i) nxt[i] = 0.f;
    }
    for (int e = lane; e < E; e += 32) hist[warp][e] = 0;
    __syncwarp();
    for (int i0 = b * k + lane; i0 < e1 * k; i0 += 128) {
      int ev[4];
      bool in[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + 32 * u;
        in[u] = i < e1 * k;
        ev[u] = in[u] ? __ldg(idx + i) : 0;
        if (mask != nullptr && in[u]) in[u] = __ldg(mask + i / k) != 0;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (!in[u]) continue;
        if ((unsigned)ev[u] < (unsigned)E) atomicAdd(&hist[warp][ev[u]], 1);
        else report_error(err, kDevBadExpertIndex);
      }
    }
    if (FORM == kLong && b >= e1) {   // a warp of a merged CTA without tokens
      for (int e = lane; e < E; e += 32) wide_p[e] = 0.0;
      if (lane == 0) *wide_z = 0.0;
    }
    float acc[NV], z = 0.f;
    int n = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) acc[i] = 0.f;
    for (int tb = b; tb < e1; tb += W) {
      float v[NV], inv, lse;
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = nxt[i];
      const bool act = nact;
      nact = nact2;
      load_logits<L>(logits, tb + W + g, nact, E, gl, nxt);
      nact2 = counted(tb + 2 * W + g, e1);
      softmax_terms<L>(v, act, inv, lse);
#pragma unroll
      for (int i = 0; i < NV; ++i) acc[i] = fmaf(v[i], inv, acc[i]);
      if (gl == 0 && act) {
        z = fmaf(lse, lse, z);
        ++n;
      }
      if constexpr (FORM == kLong) {
        const int sofar = tb + W - b;
        if (sofar % kSumTokens != 0 && tb + W < e1) continue;
        warp_groups_sum<G, NV>(acc, z);
        const bool first = sofar <= kSumTokens;
        if (g == 0) add_values<L>(wide_p, E, gl, first, acc);
        if (lane == 0) *wide_z = (first ? 0.0 : *wide_z) + (double)z;
#pragma unroll
        for (int i = 0; i < NV; ++i) acc[i] = 0.f;
        z = 0.f;
      }
    }
    if constexpr (FORM != kLong) warp_groups_sum<G, NV>(acc, z);
#pragma unroll
    for (int o = 16; o >= G; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    __syncwarp();
    if (!merged) {
      const size_t slot = (size_t)gw + s;
      if constexpr (FORM == kLong) {
        for (int e = lane; e < E; e += 32) part.p[slot * E + e] = (float)wide_p[e];
        z = (float)*wide_z;
      } else {
        if (g == 0) store_values<L>(part.p + slot * E, E, gl, acc);
      }
      for (int e = lane; e < E; e += 32) part.c[slot * E + e] = hist[warp][e];
      if (lane == 0) {
        part.n[slot] = n;
        part.z[slot] = z;
      }
      __syncwarp();
      continue;
    }
    if (FORM != kLong && g == 0) store_values<L>(red[warp], E, gl, acc);
    if (lane == 0) {
      red_n[warp] = n;
      red_z[warp] = z;
    }
    __syncthreads();
    const size_t slot = (size_t)blockIdx.x * kWarps + s;
    for (int e = threadIdx.x; e < E; e += 256) {
      int c = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) c += hist[w][e];
      part.p[slot * E + e] =
          FORM == kLong ? wide_sum(wide + e, 256) : pair_sum(&red[0][e], 256);
      part.c[slot * E + e] = c;
    }
    if (threadIdx.x == 0) {
      int c = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) c += red_n[w];
      part.z[slot] = FORM == kLong ? wide_sum(wide + kWarps * 256, 1) : pair_sum(red_z, 1);
      part.n[slot] = c;
    }
    break;
  }
  if constexpr (FORM == kFused) {
    __shared__ FinishSmem<256> sm;
    if (!last_cta(done)) return;
    for (int s = 0; s < S; ++s) finish_sequence(sm, part, off, s, T, E, k, lc, EP, out, err);
    __threadfence_block();
    __syncthreads();
    finish_totals(sm, S, out);
  }
}

// One CTA per sequence (strided); the last CTA to finish adds the sequences.
// NT threads: 1024 where the sequences are fewer than the SMs (and so may be
// long, with a slot for every 64 tokens or more), else 256, several CTAs an SM.
// Both directions: 22002 x 256, 7 sequences, 40 us with 1024 and 64 with 256;
// 131072 x 256, 311 sequences, 100 and 96.
template <int NT>
__global__ void __launch_bounds__(NT)
    balance_finish_kernel(BalanceParts part, const int32_t* __restrict__ off, int T, int E, int k,
                          int S, int lc, int EP, BalanceOut out, unsigned* done, int32_t* err) {
  pdl_wait_and_release();
  __shared__ FinishSmem<NT> sm;
  for (int s = blockIdx.x; s < S; s += gridDim.x)
    finish_sequence(sm, part, off, s, T, E, k, lc, EP, out, err);
  if (last_cta(done)) finish_totals(sm, S, out);
}

template <typename L>
__global__ void __launch_bounds__(256, 4)
    balance_backward_kernel(const float* __restrict__ logits, const int32_t* __restrict__ off,
                            const uint8_t* __restrict__ mask, const int32_t* __restrict__ counts,
                            const int32_t* __restrict__ tokens, const float* __restrict__ dlosses,
                            int T, int E, int k, int S, int lc, float* __restrict__ dlogits,
                            int32_t* err) {
  pdl_wait_and_release();
  constexpr int G = L::G, W = L::W, NV = L::NV;
  const int lane = threadIdx.x & 31, g = lane / G, gl = lane % G;
  const int gw = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t0 = (int)min((long long)T, (long long)gw << lc);
  const int t1 = (int)min((long long)T, (long long)t0 + (1 << lc));
  if (t0 >= t1) return;
  float nxt[NV];
  load_logits<L>(logits, t0 + g, t0 + g < t1, E, gl, nxt);
  const int N = __ldg(tokens + S), live = __ldg(tokens + S + 1);
  const float dz = N > 0 ? (float)(2.0 * (double)__ldg(dlosses + 1) / (double)N) : 0.f;
  const double db = live > 0 ? (double)__ldg(dlosses) * E / (double)live : 0.0;
  auto counted = [&](int t, int end) {
    return t < end && (mask == nullptr || __ldg(mask + t) != 0);
  };
  auto zero_rows = [&](int b, int e) {
    for (size_t i = (size_t)b * E + lane; i < (size_t)e * E; i += 32) dlogits[i] = 0.f;
  };
  int s = 0, lo, hi;
  if (off != nullptr) {
    const int head = __ldg(off), tail = __ldg(off + S);
    if (head > t0) zero_rows(t0, min(t1, head));
    if (tail < t1) zero_rows(max(t0, tail), t1);
    s = warp_find_seq(off, S, t0);
    if (gw == 0 && lane == 0 && (head < 0 || tail > T)) report_error(err, kDevBadOffsets);
  }
  for (; s < S; ++s) {
    seq_bounds(off, s, T, lo, hi);
    if (lo >= t1) break;
    const int b = max(lo, t0), e1 = min(hi, t1);
    if (b >= e1) continue;
    const int n = __ldg(tokens + s);
    const double w = n > 0 ? db / ((double)n * (double)n * (double)k) : 0.0;
    float a[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = L::expert(gl, i);
      a[i] = e < E ? (float)(w * (double)__ldg(counts + (size_t)s * E + e)) : 0.f;
    }
    if (b != t0) load_logits<L>(logits, b + g, b + g < e1, E, gl, nxt);
    bool nact = counted(b + g, e1), nact2 = counted(b + W + g, e1);
    if (!nact) {   // read ahead: may hold anything
#pragma unroll
      for (int i = 0; i < NV; ++i) nxt[i] = 0.f;
    }
    for (int tb = b; tb < e1; tb += W) {
      float v[NV], inv, lse;
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = nxt[i];
      const bool act = nact;
      const int t = tb + g;
      nact = nact2;
      load_logits<L>(logits, t + W, nact, E, gl, nxt);
      nact2 = counted(t + 2 * W, e1);
      softmax_terms<L>(v, act, inv, lse);
      float pa = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) pa = fmaf(v[i], a[i], pa);
      pa = dz * lse - inv * group_sum<G>(pa);
      pa *= inv;
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = act ? v[i] * fmaf(a[i], inv, pa) : 0.f;
      if (t < e1) store_values<L>(dlogits + (size_t)t * E, E, gl, v);
    }
  }
}

// log2 of a warp's tokens C: the fewest (8, 16, ...) that give at most 32
// warps to each of 148 SMs.  Both directions at 131072 x 256, 311 sequences: 96
// us; with half the tokens a warp 99, with twice as many 107.
int chunk_log(int T) {
  int lc = 3;
  while ((T >> lc) >= 148 * 32 && lc < 20) ++lc;
  return lc;
}

// Calls f with the lane layout for E experts; vec: E a multiple of 4 and every
// row of fp32 values 16-byte aligned.  At most 16 values a lane: a token's, the next
// one's and the sums then stay in the 64 registers that four CTAs an SM leave, but
// for a few words of addresses and bounds (8 to 44 bytes spilled).  E = 256 by 32
// lanes of 8 spills nothing, yet the forward's first launch takes 40 us against 36 at
// 131072 tokens.
template <typename F>
cudaError_t by_width(int E, bool vec, F&& f) {
  if (vec) {
    if (E <= 4) return f(Lanes<1, 4, true>{});
    if (E <= 8) return f(Lanes<2, 4, true>{});
    if (E <= 16) return f(Lanes<4, 4, true>{});
    if (E <= 32) return f(Lanes<8, 4, true>{});
    if (E <= 64) return f(Lanes<8, 8, true>{});
    if (E <= 128) return f(Lanes<8, 16, true>{});
    return f(Lanes<16, 16, true>{});
  }
  if (E <= 4) return f(Lanes<4, 1, false>{});
  if (E <= 16) return f(Lanes<16, 1, false>{});
  if (E <= 64) return f(Lanes<32, 2, false>{});
  return f(Lanes<32, 8, false>{});
}

bool vector_rows(int E, const void* a, const void* b) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b);
  return E % 4 == 0 && (at & 15u) == 0;
}

}  // namespace

BalanceLayout balance_layout(const moe_config_t& c, int S) {
  BalanceLayout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) / 256 * 256;
    return o;
  };
  const size_t slots = (size_t)ceil_div(c.T, 1 << chunk_log(c.T)) + kWarps + (size_t)S;
  L.ctrl = take(256);
  L.p = take(slots * c.E * 4);
  L.c = take(slots * c.E * 4);
  L.n = take(slots * 4);
  L.z = take(slots * 4);
  L.terms = take((size_t)S * 16);
  L.total = off;
  return L;
}

cudaError_t launch_balance_loss(const moe_config_t& c, int S, const int32_t* off,
                                const uint8_t* mask, const float* logits, const int32_t* idx,
                                int32_t* counts, float* prob_mean, int32_t* tokens, float* losses,
                                void* ws, cudaStream_t s) {
  const BalanceLayout L = balance_layout(c, S);
  uint8_t* base = static_cast<uint8_t*>(ws);
  int32_t* err = reinterpret_cast<int32_t*>(base + L.ctrl);
  unsigned* done = reinterpret_cast<unsigned*>(base + L.ctrl + 64);
  const BalanceParts part{
      reinterpret_cast<float*>(base + L.p), reinterpret_cast<int32_t*>(base + L.c),
      reinterpret_cast<int32_t*>(base + L.n), reinterpret_cast<float*>(base + L.z)};
  const BalanceOut out{counts, prob_mean, tokens, losses,
                       reinterpret_cast<double*>(base + L.terms)};
  const int lc = chunk_log(c.T);
  int EP = 8;
  while (EP < c.E) EP *= 2;
  const int grid = ceil_div(c.T, kWarps << lc);
  const bool fused = grid > 0 && grid <= 16 && S <= 4;
  if (grid > 0) {
    const cudaError_t e = by_width(c.E, vector_rows(c.E, logits, nullptr), [&](auto lanes) {
      using W = decltype(lanes);
      const bool wide = lc > kLogSum;
      const auto kern = fused  ? balance_partial_kernel<W, kFused>
                        : wide ? balance_partial_kernel<W, kLong>
                               : balance_partial_kernel<W, kPlain>;
      return launch_kernel(kern, grid, 256, wide ? kWideBytes : 0, s, 0, logits, idx, off, mask,
                           c.T, c.E, c.top_k, S, lc, part, EP, out, done, err);
    });
    if (e != cudaSuccess || fused) return e;
  }
  const bool few = S < device_sm_count();
  return launch_kernel(few ? balance_finish_kernel<1024> : balance_finish_kernel<256>,
                       std::min(S, device_sm_count() * 4), few ? 1024 : 256, 0, s, 0, part, off,
                       c.T, c.E, c.top_k, S, lc, EP, out, done, err);
}

cudaError_t launch_balance_loss_backward(const moe_config_t& c, int S, const int32_t* off,
                                         const uint8_t* mask, const float* logits,
                                         const int32_t* counts, const int32_t* tokens,
                                         const float* dlosses, float* dlogits, void* ws,
                                         cudaStream_t s) {
  if (c.T == 0) return cudaSuccess;
  const int lc = chunk_log(c.T);
  int32_t* err = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + balance_layout(c, S).ctrl);
  return by_width(c.E, vector_rows(c.E, logits, dlogits), [&](auto lanes) {
    return launch_kernel(balance_backward_kernel<decltype(lanes)>, ceil_div(c.T, kWarps << lc), 256,
                         0, s, 0, logits, off, mask, counts, tokens, dlosses, c.T, c.E, c.top_k, S,
                         lc, dlogits, err);
  });
}

}  // namespace moe
