// Next token by sampling: one token per row of logits, from one given uniform number.
//
// With x the row's logits, m their maximum and T the temperature, token v has the weight
// w_v = exp((x_v - m) / T).  The tokens are ordered by logit, ties by the lower index.
//   top-k: the first k of the order stay;
//   top-p: of these, those whose preceding tokens hold less than top_p of their total weight;
//   min-p: of these, those with w_v >= min_p.
// The first of the order always stays.  The token drawn is the first v, in the vocabulary's
// order, at which the running sum of the kept weights exceeds u times their total.
// NaN logits take no part.  T <= 0, or a row with no weight: the most likely token.
//
// Weights are rounded to whole numbers of 2^-44, so every sum is exact
// whatever its order, the same on every run, and a border cannot be missed between two passes.
// The exponent (x - m) log2(e) / T is formed in two fp32 words, so a weight is off by about
// one rounding of its 24 bits wherever it lies.
#include "common.cuh"
#include "kernels.h"

namespace rdt {

namespace {
constexpr int NT = 1024, NW = NT / 32;
typedef unsigned long long u64;

// order of floats as unsigned integers; NaN below everything
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);   // -0 and 0 are the same logit
  if (x != x) return 0u;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k); }

struct Weigh {
  float m, chi, clo;   // maximum; log2(e) / T in two words
  __device__ Weigh(float mx, float T) : m(mx) {
    const double c = 1.4426950408889634074 / (double)T;
    chi = (float)c;
    clo = isinf(chi) ? 0.f : (float)(c - (double)chi);
  }
  // weight of x in units of 2^-44
  __device__ __forceinline__ u64 operator()(float x) const {
    if (x == m) return 1ull << 44;
    const float d = m - x, t = d * chi;
    if (!(t < 46.f)) return 0;                                   // also NaN and -inf
    const float bb = d - m;
    const float dlo = (m - (d - bb)) + (-x - bb);                // d + dlo = m - x
    const float e = fmaf(d, chi, -t) + fmaf(d, clo, dlo * chi);  // t + e = (m - x) log2(e) / T
    const int i = __float2int_rn(t);
    const float w = exp2f(-((t - (float)i) + e));                // 2^-1/2 .. 2^1/2
    return (((u64)(uint32_t)(w * 16777216.f) << 21 >> i) + 1) >> 1;
  }
};

__device__ u64 block_sum64(u64 v, u64* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[threadIdx.x & 31];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct Cut {
  uint32_t key;   // the last key that stays
  u64 ties;       // of the tokens at that key, how many stay (from the lowest index)
  u64 before;     // measure (count or weight) of the tokens above the key
};

// The key at which the running measure of the order (count, or weight) reaches `want` >= 1:
// four passes, 8 bits of the key each.
template <bool MASS>
__device__ Cut select(const float* row, int V, const Weigh& wt, u64 want, u64* hist, u64* sh) {
  uint32_t prefix = 0;
  u64 before = 0;
  for (int level = 3; level >= 0; --level) {
    const int sft = level * 8;
    for (int i = threadIdx.x; i < 256; i += NT) hist[i] = 0;
    __syncthreads();
    for (int v = threadIdx.x; v < V; v += NT) {
      const uint32_t k = key_of(row[v]);
      if (level < 3 && (k >> (sft + 8)) != (prefix >> (sft + 8))) continue;
      const u64 q = MASS ? wt(row[v]) : 1ull;
      if (q) atomicAdd(&hist[(k >> sft) & 255], q);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      u64 c = before;
      int bin = 255;
      for (; bin > 0; --bin) {
        if (c + hist[bin] >= want) break;
        c += hist[bin];
      }
      sh[0] = c;
      sh[1] = (u64)bin;
    }
    __syncthreads();
    before = sh[0];
    prefix |= (uint32_t)sh[1] << sft;
    __syncthreads();
  }
  Cut r;
  r.key = prefix;
  r.before = before;
  const u64 unit = MASS ? wt(of_key(prefix)) : 1ull;
  r.ties = unit ? (want - before + unit - 1) / unit : ~0ull;
  return r;
}
}  // namespace

__global__ void __launch_bounds__(NT) k_sample(SampleParams p) {
  __shared__ u64 hist[256], red[NW], sh[2], wsum[NW];
  __shared__ float fmx[NW];
  __shared__ int found;
  const int r = blockIdx.x, V = p.vocab, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float* row = p.logits + (long long)r * p.ld;
  const float T = p.temperature_row ? p.temperature_row[r] : p.temperature;
  const int k = p.top_k_row ? p.top_k_row[r] : p.top_k;
  const float top_p = p.top_p_row ? p.top_p_row[r] : p.top_p;
  const float min_p = p.min_p_row ? p.min_p_row[r] : p.min_p;
  float mx = -INFINITY;
  for (int v = tid; v < V; v += NT) mx = fmaxf(mx, row[v]);      // fmaxf drops NaN
  mx = warp_max(mx);
  if (lane == 0) fmx[warp] = mx;
  __syncthreads();
  mx = warp_max(fmx[lane]);
  if (tid == 0) found = 0x7fffffff;
  __syncthreads();
  if (!(T > 0.f) || mx == -INFINITY) {                           // the most likely token
    int best = 0x7fffffff;
    for (int v = tid; v < V && best == 0x7fffffff; v += NT)
      if (row[v] == mx) best = v;
    atomicMin(&found, best);
    __syncthreads();
    if (tid == 0) {
      p.tokens[(long long)r * p.out_ld] = found == 0x7fffffff ? 0 : found;
      if (p.logprob) p.logprob[r] = 0.f;
    }
    return;
  }
  const Weigh wt(mx, T);
  Cut cut{0u, ~0ull, 0};
  if (k > 0 && k < V) cut = select<false>(row, V, wt, (u64)k, hist, sh);
  if (top_p < 1.f) {
    u64 above = 0, ties = 0;
    for (int v = tid; v < V; v += NT) {
      const uint32_t q = key_of(row[v]);
      if (q > cut.key) above += wt(row[v]);
      else if (q == cut.key) ++ties;
    }
    above = block_sum64(above, red);
    ties = block_sum64(ties, red);
    const u64 mass = above + min(ties, cut.ties) * wt(of_key(cut.key));
    const u64 want = (u64)max(1.0, ceil((double)max(top_p, 0.f) * (double)mass));
    cut = select<true>(row, V, wt, want, hist, sh);
  }
  // min-p: (x - m) / T >= ln(min_p)
  double xmin = -INFINITY;
  if (min_p > 0.f) xmin = (double)mx + (double)T * log((double)fminf(min_p, 1.f));
  // the kept weight of each warp's piece of the row; where a tie straddles the cut, its last index
  const int piece = ((V + NW - 1) / NW + 31) / 32 * 32;
  const int v0 = warp * piece, v1 = min(V, v0 + piece);
  u64 ties = 0;
  for (int v = v0 + lane; v < v1; v += 32) ties += key_of(row[v]) == cut.key;
  const u64 all_ties = block_sum64(ties, red);
  int last_tie = V - 1;
  if (cut.ties < all_ties) {
    if (tid == 0) {
      u64 n = 0;
      for (int v = 0; v < V; ++v)
        if (key_of(row[v]) == cut.key && ++n == cut.ties) {
          found = v;
          break;
        }
    }
    __syncthreads();
    last_tie = found;
  }
  auto kept = [&](float x, int v) -> u64 {
    const uint32_t q = key_of(x);
    if (q < cut.key || (q == cut.key && v > last_tie) || (double)x < xmin) return 0;
    return wt(x);
  };
  u64 mine = 0;
  for (int v = v0 + lane; v < v1; v += 32) mine += kept(row[v], v);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) wsum[warp] = mine;
  __syncthreads();
  u64 total = 0;
  for (int w = 0; w < NW; ++w) total += wsum[w];
  const float u = p.u[r];
  const double uc = u > 0.f ? fmin((double)u, 1.0 - 0x1p-24) : 0.0;   // NaN: 0
  const u64 target = (u64)(uc * (double)total);
  u64 base = 0;
  int w = 0;
  for (; w < NW - 1 && base + wsum[w] <= target; ++w) base += wsum[w];
  if (warp != w) return;
  for (int v = v0; v < v1; v += 32) {
    const u64 q = v + lane < v1 ? kept(row[v + lane], v + lane) : 0;
    u64 c = q;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 t = __shfl_up_sync(0xffffffffu, c, o);
      if (lane >= o) c += t;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + c > target);
    if (hit) {
      const int l = __ffs(hit) - 1;
      if (lane == l) {
        p.tokens[(long long)r * p.out_ld] = v + lane;
        if (p.logprob) {
          const double x = row[v + lane];
          const double z = x == (double)mx ? 0.0 : (x - (double)mx) / (double)T;
          p.logprob[r] = (float)(z - log((double)total * 0x1p-44));
        }
      }
      return;
    }
    base += __shfl_sync(0xffffffffu, c, 31);
  }
}

void launch_sample(const SampleParams& p, cudaStream_t s) {
  k_sample<<<p.n, NT, 0, s>>>(p);
  note_launch();
}

}  // namespace rdt
