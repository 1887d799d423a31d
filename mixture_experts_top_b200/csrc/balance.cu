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
// Both directions are one pass over the logits: bound by HBM for large T x E,
// by launch latency below about a million logits.  A token's E logits sit in
// the registers of G = min(32, E rounded up to a power of 2) lanes, so a warp
// works on 32 / G tokens at once; maximum and sum are butterflies over the G
// lanes, in fp32.
//
// Summation order (no floating-point atomics, nothing depends on which CTA
// runs first): a warp owns C consecutive tokens and walks the sequences that
// meet them; each such piece gets the slot (warp + s) of the partial sums,
// which no other piece has (going to the next warp or the next sequence
// raises it by at least one), so no scan over the sequences is needed.  Where
// one sequence covers all 8 warps of a CTA, their sums are added in warp
// order and only the first warp's slot is written.  The second launch adds a
// sequence's slots in a fixed order in fp64.
#include <type_traits>

#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kWarps = 8;

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

// Bounds of sequence s inside [0, T] whatever the offsets hold.
__device__ __forceinline__ void seq_bounds(const int32_t* __restrict__ off, int s, int T, int& lo,
                                           int& hi) {
  if (off == nullptr) {
    lo = 0;
    hi = T;
    return;
  }
  lo = min(max(__ldg(off + s), 0), T);
  hi = min(max(__ldg(off + s + 1), lo), T);
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

// This lane's logits of token t: experts gl + G q.  Tokens not counted are
// not read (they may hold anything).
template <int G, int Q>
__device__ __forceinline__ void load_logits(const float* __restrict__ logits, int t, bool act,
                                            int E, int gl, float (&L)[Q]) {
  const float* row = logits + (size_t)t * E;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int e = gl + G * q;
    L[q] = act && e < E ? __ldg(row + e) : -INFINITY;
  }
}

// exp(l - max) of this lane's experts, their sum's inverse and the token's
// log-sum-exp, from the G lanes' logits; all 0 where act is false.
template <int G, int Q>
__device__ __forceinline__ void softmax_terms(float (&L)[Q], bool act, float& inv, float& lse) {
  float m = L[0];
#pragma unroll
  for (int q = 1; q < Q; ++q) m = fmaxf(m, L[q]);
  m = group_max<G>(m);
  float sum = 0.f;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    L[q] = act ? expf(L[q] - m) : 0.f;
    sum += L[q];
  }
  sum = group_sum<G>(sum);
  inv = act ? 1.f / sum : 0.f;
  lse = act ? m + logf(sum) : 0.f;
}

struct BalanceParts {
  float* p;        // (slots, E) sums of probabilities
  int32_t* c;      // (slots, E) routing slots per expert
  int32_t* n;      // (slots) counted tokens
  float* z;        // (slots) sums of lse^2
};

template <int G, int Q>
__global__ void __launch_bounds__(256)
    balance_partial_kernel(const float* __restrict__ logits, const int32_t* __restrict__ idx,
                           const int32_t* __restrict__ off, const uint8_t* __restrict__ mask,
                           int T, int E, int k, int S, int C, BalanceParts part, int32_t* err) {
  pdl_wait_and_release();
  __shared__ int32_t hist[kWarps][256];
  __shared__ float red[kWarps][256];
  __shared__ int32_t red_n[kWarps];
  __shared__ float red_z[kWarps];
  constexpr int W = 32 / G;   // tokens at once
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane / G, gl = lane % G;
  const int gw = blockIdx.x * kWarps + warp;
  const int c0 = blockIdx.x * kWarps * C;
  const int c1 = (int)min((long long)T, (long long)c0 + kWarps * C);
  const int t0 = (int)min((long long)c1, (long long)c0 + warp * C);
  const int t1 = (int)min((long long)c1, (long long)t0 + C);
  int lo, hi;
  const int s0 = off == nullptr ? 0 : warp_find_seq(off, S, c0);
  bool merged = false;
  if (s0 < S) {
    seq_bounds(off, s0, T, lo, hi);
    merged = lo <= c0 && hi >= c1;
  }
  // the rest of the loop runs per warp; merged is the same for all of them
  for (int s = merged || off == nullptr ? s0 : warp_find_seq(off, S, t0); s < S; ++s) {
    seq_bounds(off, s, T, lo, hi);
    if (!merged && lo >= t1) break;
    const int b = max(lo, t0), e1 = min(hi, t1);
    if (!merged && b >= e1) continue;
    for (int e = lane; e < E; e += 32) hist[warp][e] = 0;
    __syncwarp();
    for (int i = b * k + lane; i < e1 * k; i += 32) {
      if (mask != nullptr && mask[i / k] == 0) continue;
      const int e = __ldg(idx + i);
      if ((unsigned)e < (unsigned)E) atomicAdd(&hist[warp][e], 1);
      else report_error(err, kDevBadExpertIndex);
    }
    float acc[Q], z = 0.f;
    int n = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q) acc[q] = 0.f;
    float nxt[Q];
    bool nact = b + g < e1 && (mask == nullptr || mask[b + g] != 0);
    load_logits<G, Q>(logits, b + g, nact, E, gl, nxt);
    for (int tb = b; tb < e1; tb += W) {
      float L[Q], inv, lse;
#pragma unroll
      for (int q = 0; q < Q; ++q) L[q] = nxt[q];
      const bool act = nact;
      const int tn = tb + W + g;
      nact = tn < e1 && (mask == nullptr || mask[tn] != 0);
      load_logits<G, Q>(logits, tn, nact, E, gl, nxt);
      softmax_terms<G, Q>(L, act, inv, lse);
#pragma unroll
      for (int q = 0; q < Q; ++q) acc[q] = fmaf(L[q], inv, acc[q]);
      if (gl == 0 && act) {
        z = fmaf(lse, lse, z);
        ++n;
      }
    }
#pragma unroll
    for (int o = 16; o >= G; o >>= 1) {
#pragma unroll
      for (int q = 0; q < Q; ++q) acc[q] += __shfl_xor_sync(0xffffffffu, acc[q], o);
      z += __shfl_xor_sync(0xffffffffu, z, o);
      n += __shfl_xor_sync(0xffffffffu, n, o);
    }
    __syncwarp();
    if (!merged) {
      const size_t slot = (size_t)gw + s;
      if (g == 0) {
#pragma unroll
        for (int q = 0; q < Q; ++q)
          if (gl + G * q < E) part.p[slot * E + gl + G * q] = acc[q];
      }
      for (int e = lane; e < E; e += 32) part.c[slot * E + e] = hist[warp][e];
      if (lane == 0) {
        part.n[slot] = n;
        part.z[slot] = z;
      }
      __syncwarp();
      continue;
    }
    if (g == 0) {
#pragma unroll
      for (int q = 0; q < Q; ++q) red[warp][gl + G * q] = acc[q];
    }
    if (lane == 0) {
      red_n[warp] = n;
      red_z[warp] = z;
    }
    __syncthreads();
    const size_t slot = (size_t)blockIdx.x * kWarps + s;
    for (int e = threadIdx.x; e < E; e += 256) {
      float v = 0.f;
      int c = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        v += red[w][e];
        c += hist[w][e];
      }
      part.p[slot * E + e] = v;
      part.c[slot * E + e] = c;
    }
    if (threadIdx.x == 0) {
      float v = 0.f;
      int c = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        v += red_z[w];
        c += red_n[w];
      }
      part.z[slot] = v;
      part.n[slot] = c;
    }
    break;
  }
}

// The slots of a sequence [lo, hi) in order: the warps of a CTA it covers in
// part, one per CTA it covers whole, the warps of the last CTA in part.
struct SeqSlots {
  int s, first, nh, jm, nm, tail, nt;
  __device__ SeqSlots(int s_, int lo, int hi, int T, int C) : s(s_) {
    first = nh = jm = nm = tail = nt = 0;
    if (lo >= hi) return;
    const int CC = kWarps * C;
    const int j0 = lo / CC, j1 = (hi - 1) / CC;
    const bool from = lo == j0 * CC;
    const bool upto = hi >= (int)min((long long)T, (long long)(j1 + 1) * CC);
    first = lo / C;
    if (j0 == j1 && !(from && upto)) {
      nh = (hi - 1) / C - first + 1;
      return;
    }
    jm = from ? j0 : j0 + 1;
    nh = from ? 0 : (j0 + 1) * kWarps - first;
    nm = (upto ? j1 + 1 : j1) - jm;
    tail = j1 * kWarps;
    nt = upto ? 0 : (hi - 1) / C - tail + 1;
  }
  __device__ int count() const { return nh + nm + nt; }
  __device__ size_t operator()(int i) const {
    const int w = i < nh ? first + i : i < nh + nm ? kWarps * (jm + i - nh) : tail + (i - nh - nm);
    return (size_t)w + s;
  }
};

// Sum over the CTA's 256 threads in a fixed order; every thread gets it.
template <typename V>
__device__ __forceinline__ V block_sum(V v, V* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  V r = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) r += buf[w];
  __syncthreads();
  return r;
}

// One CTA per sequence (strided): counts, P, n and the sequence's terms of
// both losses; the last CTA to finish adds the sequences.
__global__ void __launch_bounds__(256)
    balance_finish_kernel(BalanceParts part, const int32_t* __restrict__ off, int T, int E, int k,
                          int S, int C, int EP, int32_t* __restrict__ counts,
                          float* __restrict__ prob_mean, int32_t* tokens, float* losses,
                          double* seq_terms, unsigned* done, int32_t* err) {
  pdl_wait_and_release();
  __shared__ double sp[256];
  __shared__ int32_t sc[256];
  __shared__ double bufd[8];
  __shared__ int32_t bufi[8];
  __shared__ bool last;
  const int tid = threadIdx.x;
  const int ng = 256 / EP, e = tid % EP, gi = tid / EP;   // ng groups walk the slots
  for (int s = blockIdx.x; s < S; s += gridDim.x) {
    if (off != nullptr && tid == 0 &&
        (off[s] < 0 || off[s + 1] < off[s] || off[s + 1] > T))
      report_error(err, kDevBadOffsets);
    int lo, hi;
    seq_bounds(off, s, T, lo, hi);
    const SeqSlots slots(s, lo, hi, T, C);
    const int ni = slots.count();
    double p = 0.0, z = 0.0;
    int c = 0, n = 0;
    if (e < E) {
      for (int i = gi; i < ni; i += 4 * ng) {
        float pv[4];
        int cv[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const bool in = i + u * ng < ni;
          const size_t at = in ? slots(i + u * ng) * E + e : 0;
          pv[u] = in ? part.p[at] : 0.f;
          cv[u] = in ? part.c[at] : 0;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          p += (double)pv[u];
          c += cv[u];
        }
      }
    }
    for (int i = tid; i < ni; i += 256) {
      const size_t at = slots(i);
      n += part.n[at];
      z += (double)part.z[at];
    }
    sp[tid] = p;
    sc[tid] = c;
    n = block_sum(n, bufi);   // (also orders sp and sc)
    z = block_sum(z, bufd);
    double term = 0.0;
    if (tid < E) {
      p = 0.0;
      c = 0;
      for (int j = 0; j < ng; ++j) {
        p += sp[j * EP + tid];
        c += sc[j * EP + tid];
      }
      const double P = n > 0 ? p / (double)n : 0.0;
      counts[(size_t)s * E + tid] = c;
      prob_mean[(size_t)s * E + tid] = (float)P;
      if (n > 0) term = (double)c / ((double)n * k) * P;
    }
    term = block_sum(term, bufd);
    if (tid == 0) {
      tokens[s] = n;
      seq_terms[2 * (size_t)s] = term * E;
      seq_terms[2 * (size_t)s + 1] = z;
    }
  }
  __threadfence();
  __syncthreads();
  if (tid == 0) last = atom_add_acq_rel_gpu(done, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  double b = 0.0, z = 0.0;
  int n = 0, live = 0;
  for (int s = tid; s < S; s += 256) {
    const int ns = __ldcg(tokens + s);
    b += __ldcg(seq_terms + 2 * (size_t)s);
    z += __ldcg(seq_terms + 2 * (size_t)s + 1);
    n += ns;
    live += ns > 0;
  }
  b = block_sum(b, bufd);
  z = block_sum(z, bufd);
  n = block_sum(n, bufi);
  live = block_sum(live, bufi);
  if (tid == 0) {
    losses[0] = live > 0 ? (float)(b / (double)live) : 0.f;
    losses[1] = n > 0 ? (float)(z / (double)n) : 0.f;
    tokens[S] = n;
    tokens[S + 1] = live;
    *done = 0;
  }
}

// The gradient: each warp owns C tokens and walks the sequences that meet
// them; a sequence's a_se are in the lanes' registers.
template <int G, int Q>
__global__ void __launch_bounds__(256)
    balance_backward_kernel(const float* __restrict__ logits, const int32_t* __restrict__ off,
                            const uint8_t* __restrict__ mask, const int32_t* __restrict__ counts,
                            const int32_t* __restrict__ tokens, const float* __restrict__ dlosses,
                            int T, int E, int k, int S, int C, float* __restrict__ dlogits,
                            int32_t* err) {
  pdl_wait_and_release();
  constexpr int W = 32 / G;
  const int lane = threadIdx.x & 31, g = lane / G, gl = lane % G;
  const int gw = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t0 = (int)min((long long)T, (long long)gw * C);
  const int t1 = (int)min((long long)T, (long long)t0 + C);
  if (t0 >= t1) return;
  const int N = __ldg(tokens + S), live = __ldg(tokens + S + 1);
  const float dz = N > 0 ? (float)(2.0 * (double)__ldg(dlosses + 1) / (double)N) : 0.f;
  const double db = live > 0 ? (double)__ldg(dlosses) * E / (double)live : 0.0;
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
    float a[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int e = gl + G * q;
      a[q] = e < E ? (float)(w * (double)__ldg(counts + (size_t)s * E + e)) : 0.f;
    }
    float nxt[Q];
    bool nact = b + g < e1 && (mask == nullptr || mask[b + g] != 0);
    load_logits<G, Q>(logits, b + g, nact, E, gl, nxt);
    for (int tb = b; tb < e1; tb += W) {
      float L[Q], inv, lse;
#pragma unroll
      for (int q = 0; q < Q; ++q) L[q] = nxt[q];
      const bool act = nact;
      const int t = tb + g, tn = t + W;
      nact = tn < e1 && (mask == nullptr || mask[tn] != 0);
      load_logits<G, Q>(logits, tn, nact, E, gl, nxt);
      softmax_terms<G, Q>(L, act, inv, lse);
      float pa = 0.f;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        L[q] *= inv;
        pa = fmaf(L[q], a[q], pa);
      }
      pa = group_sum<G>(pa);
      if (t < e1) {
        float* out = dlogits + (size_t)t * E;
#pragma unroll
        for (int q = 0; q < Q; ++q)
          if (gl + G * q < E) out[gl + G * q] = act ? L[q] * (a[q] - pa + dz * lse) : 0.f;
      }
    }
  }
}

// Tokens of a warp: the fewest (8, 16, ...) that give at most 32 warps to
// each of 148 SMs.
int chunk_tokens(int T) {
  int C = 8;
  while (ceil_div(T, C) > 148 * 32 && C < (1 << 20)) C *= 2;
  return C;
}

// Calls f<G, Q>() for E experts.
template <typename F>
cudaError_t by_width(int E, F&& f) {
  using std::integral_constant;
#define MOE_WIDTH(G, Q) f(integral_constant<int, G>{}, integral_constant<int, Q>{})
  if (E <= 4) return MOE_WIDTH(4, 1);
  if (E <= 8) return MOE_WIDTH(8, 1);
  if (E <= 16) return MOE_WIDTH(16, 1);
  if (E <= 32) return MOE_WIDTH(32, 1);
  if (E <= 64) return MOE_WIDTH(32, 2);
  if (E <= 128) return MOE_WIDTH(32, 4);
  return MOE_WIDTH(32, 8);
#undef MOE_WIDTH
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
  const size_t slots = (size_t)ceil_div(c.T, chunk_tokens(c.T)) + kWarps + (size_t)S;
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
  const int C = chunk_tokens(c.T);
  if (c.T > 0) {
    const cudaError_t e = by_width(c.E, [&](auto G, auto Q) {
      return launch_kernel(balance_partial_kernel<decltype(G)::value, decltype(Q)::value>,
                           ceil_div(c.T, kWarps * C), 256, 0, s, 0, logits, idx, off, mask, c.T,
                           c.E, c.top_k, S, C, part, err);
    });
    if (e != cudaSuccess) return e;
  }
  int EP = 8;
  while (EP < c.E) EP *= 2;
  return launch_kernel(balance_finish_kernel, std::min(S, device_sm_count() * 8), 256, 0, s, 0,
                       part, off, c.T, c.E, c.top_k, S, C, EP, counts, prob_mean, tokens, losses,
                       reinterpret_cast<double*>(base + L.terms), done, err);
}

cudaError_t launch_balance_loss_backward(const moe_config_t& c, int S, const int32_t* off,
                                         const uint8_t* mask, const float* logits,
                                         const int32_t* counts, const int32_t* tokens,
                                         const float* dlosses, float* dlogits, void* ws,
                                         cudaStream_t s) {
  if (c.T == 0) return cudaSuccess;
  const int C = chunk_tokens(c.T);
  int32_t* err = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + balance_layout(c, S).ctrl);
  return by_width(c.E, [&](auto G, auto Q) {
    return launch_kernel(balance_backward_kernel<decltype(G)::value, decltype(Q)::value>,
                         ceil_div(c.T, kWarps * C), 256, 0, s, 0, logits, off, mask, counts,
                         tokens, dlosses, c.T, c.E, c.top_k, S, C, dlogits, err);
  });
}

}  // namespace moe
