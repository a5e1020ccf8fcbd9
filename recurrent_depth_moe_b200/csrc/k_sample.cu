// Next token by sampling: one token per row of logits, from one given uniform number.
//
// With x the row's logits, m their maximum and T the temperature, token v has the weight
// w_v = exp((x_v - m) / T).  The tokens are ordered by logit, ties by the lower index.
//   top-k: the first k of the order stay;
//   top-p: of these, those whose preceding tokens hold less than top_p of their total weight;
//   min-p: of these, those with w_v >= min_p.
// The first of the order always stays.  The token drawn is the first v, in the vocabulary's
// order, at which the running sum of the kept weights exceeds u times their total.
// NaN logits take no part.  T below 2^-127 (log2(e) / T is past fp32's range), or a row with no
// weight: the most likely token; an infinite T: every logit above -inf weighs 1.
//
// The exponent (x - m) log2(e) / T is formed in two fp32 words, so a weight is off by about one
// rounding of its 24 bits wherever it lies.  A thread sums its weights in two fp32 words, in a
// fixed order; beyond a thread weights and sums are whole numbers of 2^-44 in 64 bits, so the
// result does not depend on the order in which threads arrive.  A sum is off by about 2^-33
// of itself, a border by as much.
//
// A cluster of up to 8 CTAs holds one row in its shared memory, so the logits are read from
// HBM once; sums, histograms and candidates travel through distributed shared memory and no
// workspace is needed.  Without the row on chip each of the up to four passes would read it
// again.  The order is never sorted: a histogram over the exponent (1/16 of a power of two per
// bin) brackets the border of top-k or top-p, the few tokens of the bracket become candidates,
// and histograms over their (logit, index) order narrow the border to at most 32 of them, which
// one warp ranks.  The kept tokens are then those at or before one (logit, index) pair.
//
// Measured on one B200, us: a row of 201,088 logits with top-p 30; 64 such rows with mixed
// parameters 67; 256 with top-p 305 (the logits at the copy rate: 31).  Each row passes up to seven
// cluster barriers, each about 2 us with the remote reads behind it, and that chain bounds it: of
// 44 us that a wave of 37 clusters takes, 7 are the load, 15 the passes and 20 the barriers and
// exchanges.
#include "common.cuh"
#include "kernels.h"

#include <cooperative_groups.h>

#include <float.h>

#include <algorithm>
#include <type_traits>

namespace cg = cooperative_groups;

namespace rdt {

namespace {
constexpr int NWMAX = 16;        // warps of a CTA
constexpr int BINS = 46 * 16;    // of the exponent: a weight below 2^-45 is nothing
constexpr int RB = 256;          // bins of one refinement
constexpr int HB = BINS / 4;     // threads that sum the cluster's histograms, four bins each
constexpr int LCAP = 1000;       // candidates one CTA lists (below 2^10: sums of their weights' halves stay in 32
                                 // bits); more are found by passes over the row
constexpr int IDX_BITS = 20;
constexpr int CMAX = 8;          // CTAs of a cluster
typedef unsigned long long u64;

// order of floats as unsigned integers
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);   // -0 and 0 are the same logit
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k); }
// place in the order: larger comes first, and no two tokens share one
__device__ __forceinline__ u64 place_of(float x, int v) {
  return ((u64)key_of(x) << IDX_BITS) | (uint32_t)((1 << IDX_BITS) - 1 - v);
}

// Two fp32 values handled by one instruction.
struct F2 {
  u64 v;
  __device__ __forceinline__ F2() {}
  __device__ __forceinline__ F2(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
  __device__ __forceinline__ explicit F2(float a) : F2(a, a) {}
  __device__ __forceinline__ void get(float& a, float& b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 operator-(F2 a, F2 b) { return fma2(b, F2(-1.f), a); }

// z = x log2(e) / T as zh + e, in two fp32 words; the weight is 2^(z - M), M that of the maximum.
struct Weigh {
  float m, chi, clo, nfM, c16;   // log2(e) / T in two words; minus M's fraction; bins per logit
  float magic;                   // MAGIC minus M's whole part
  float floor;                   // the smallest logit with a weight: 2^-45 of the maximum's
  bool wide;                     // |M| so large that z has no fraction left: the difference m - x is formed first
  static constexpr float MAGIC = 12582912.f;   // 1.5 * 2^23: x + MAGIC rounds x to a whole number
  __device__ Weigh(float mx, float T) : m(mx) {
    const double c = 1.4426950408889634074 / (double)T;
    chi = (float)c;
    clo = isinf(chi) ? 0.f : (float)(c - (double)chi);
    c16 = fminf(16.f * chi, 3.0e38f);
    const float Mh = mx * chi;
    wide = !(fabsf(Mh) <= 65536.f);
    const float i0 = (Mh + MAGIC) - MAGIC;
    magic = MAGIC - i0;
    nfM = -((Mh - i0) + (fmaf(mx, chi, -Mh) + mx * clo));
    // 45 / log2(e); finite, so that -inf has no weight, and within fp32's range of the maximum, so
    // that m - x is finite from floor on (either only matters for T above 10^37)
    floor = fmaxf(__double2float_ru((double)mx - 31.191623125218536 * (double)T), fmaxf(-FLT_MAX, mx - FLT_MAX));
  }
  // MAGIC plus the bin, 16 times the exponent rounded to a whole number; monotone in x, NaN for NaN
  __device__ __forceinline__ float bin(float x) const { return fmaf(m - x, c16, MAGIC); }
  // the weight, to 24 bits (that of floor for what is below it, NaN too)
  template <bool WIDE> __device__ __forceinline__ float weight(float x) const {
    float s, e;
    int k;                                                           // minus the whole part of the exponent
    x = fmaxf(x, floor);
    if (!WIDE) {
      const float zh = x * chi, r = zh + magic;                      // MAGIC - k
      s = ((zh - (r - magic)) + fmaf(x, clo, nfM)) + fmaf(x, chi, -zh);
      k = -__float_as_int(r);                                        // (MAGIC's bits leave the word below)
    } else {
      const float d = m - x, t = d * chi, bb = d - m;
      const float dlo = (m - (d - bb)) + (-x - bb);                  // d + dlo = m - x
      const float r = t + MAGIC;
      s = x == m ? 0.f : -((t - (r - MAGIC)) + (fmaf(d, chi, -t) + fmaf(d, clo, dlo * chi)));
      k = x == m ? 0 : min(47, __float_as_int(r) - __float_as_int(MAGIC));
    }
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(s));            // -1 <= s <= 1
    return __int_as_float(__float_as_int(e) - (k << 23));
  }
  // the same of two
  template <bool WIDE> __device__ __forceinline__ F2 weight2(float x0, float x1) const {
    if (WIDE) return F2(weight<true>(x0), weight<true>(x1));
    const F2 x(fmaxf(x0, floor), fmaxf(x1, floor)), c(chi), mg(magic);
    const F2 zh = x * c, r = zh + mg;
    const F2 s = ((zh - (r - mg)) + fma2(x, F2(clo), F2(nfM))) + fma2(x, c, zh * F2(-1.f));
    float s0, s1, r0, r1, e0, e1;
    s.get(s0, s1);
    r.get(r0, r1);
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(s0));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(s1));
    return F2(__int_as_float(__float_as_int(e0) + (__float_as_int(r0) << 23)),
              __int_as_float(__float_as_int(e1) + (__float_as_int(r1) << 23)));
  }
  // 16 times the exponent of two: MAGIC plus the bins, and by how much it is above them
  __device__ __forceinline__ void bin2(float x0, float x1, float& b0, float& b1, F2& f) const {
    const F2 d = F2(m) - F2(x0, x1), c(c16), b = fma2(d, c, F2(MAGIC));
    f = fma2(d, c, F2(MAGIC) - b);
    b.get(b0, b1);
  }
  // In whole units of 2^-44, one at least from floor on: wherever sums of weights say that there is
  // something, a token with a weight is found (the sums cut at floor too, by the same comparison).
  __device__ __forceinline__ u64 operator()(float x) const {
    const float w = wide ? weight<true>(x) : weight<false>(x);
    return x >= floor ? max(1ull, __float2ull_rn(w * 0x1p44f)) : 0;
  }
};

// Sum of up to 512 weights of at most 1, two at a time: each half of `a` stays between 2^8 and
// 2^9, so a + w rounds w to a multiple of 2^-15 exactly and `lo` takes up what that leaves.
struct Sum {
  F2 a, lo;
  __device__ __forceinline__ Sum() : a(256.f), lo(0.f) {}
  __device__ __forceinline__ void add(F2 w) {
    const F2 s = a + w;
    lo = lo + (w - (s - a));
    a = s;
  }
  __device__ __forceinline__ u64 units() const {   // of 2^-44
    float a0, a1, l0, l1;
    a.get(a0, a1);
    lo.get(l0, l1);
    return (u64)__double2ll_rn((((double)a0 + (double)a1 - 512.0) + ((double)l0 + (double)l1)) * 0x1p44);
  }
};

struct __align__(16) Shared {
  u64 mass[2][RB];       // refinements: weight, and number, of the candidates by bin
  u64 wsum[NWMAX];       // kept weight of each warp's piece of the row
  u64 glist[2][32];      // [top-k, top-p] the last candidates
  u64 ranked[32];
  u64 red[NWMAX];
  u64 bc[3];
  u64 total, above;
  __align__(16) uint32_t hist[BINS];
  __align__(16) uint32_t cnt[2][RB];
  uint32_t list[LCAP];
  uint32_t fcnt[2], gcnt[2], kmin[2], kmax[2];
  uint32_t add[NWMAX][2], nranked;
  uint32_t idx;
  int ib[4];
  float fred[NWMAX];
  float mx;
};

template <typename V> __device__ __forceinline__ V warp_scan(V v) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V t = __shfl_up_sync(0xffffffffu, v, o);
    if ((int)(threadIdx.x & 31) >= o) v += t;
  }
  return v;
}
// A barrier of the cluster, with its shared memory visible across it; of one CTA, the CTA's.
__device__ __forceinline__ void cluster_sync(const cg::cluster_group& cl, int C) {
  if (C > 1) cl.sync();
  else __syncthreads();
}
// Inclusive sum over the block's NW warps; `red` holds NW values, `total` the block's.
template <int NW, typename V> __device__ __forceinline__ V block_scan(V v, V* red, V& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_scan(v);
  __syncthreads();
  if (lane == 31) red[warp] = v;
  __syncthreads();
  const V w = warp_scan(lane < NW ? red[lane] : (V)0);
  total = __shfl_sync(0xffffffffu, w, NW - 1);
  const V before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  return warp ? v + before : v;
}
__device__ __forceinline__ u64 warp_sum64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// RES: the CTA's piece of the row lives in shared memory; else (a row too long for the cluster)
// every pass reads it again.
template <bool RES> struct Row {
  const float* row;
  const float4* chunk;   // RES: the piece
  int V, a, q0, nq;      // the row starts a floats past a 16-byte boundary; quads q0 .. q0 + nq - 1 are this CTA's
  int jb, je;            // this warp's quads, contiguous
  bool inf_row;          // the maximum is +inf: the infinities weigh 1, the rest nothing
  __device__ __forceinline__ bool full(int j) const {   // the quad lies inside the row
    const int i = 4 * (q0 + j) - a;
    return i >= 0 && i + 4 <= V;
  }
  __device__ __forceinline__ float4 load(int j) const {
    const int i = 4 * (q0 + j) - a;
    if (full(j)) return __ldg(reinterpret_cast<const float4*>(row + i));
    const float none = __int_as_float(0x7fffffff);   // past the row's ends: NaN, which takes no part
    float4 v;
    v.x = i >= 0 && i < V ? row[i] : none;
    v.y = i + 1 >= 0 && i + 1 < V ? row[i + 1] : none;
    v.z = i + 2 >= 0 && i + 2 < V ? row[i + 2] : none;
    v.w = i + 3 >= 0 && i + 3 < V ? row[i + 3] : none;
    return v;
  }
  __device__ __forceinline__ float fix(float x) const { return !inf_row ? x : x == INFINITY ? 0.f : -INFINITY; }
  __device__ __forceinline__ float4 quad(int j) const {
    if (RES) return chunk[j];
    const float4 v = load(j);
    return make_float4(fix(v.x), fix(v.y), fix(v.z), fix(v.w));
  }
  __device__ __forceinline__ int index(int local) const { return 4 * q0 + local - a; }
  __device__ __forceinline__ float at(int local) const {
    return RES ? reinterpret_cast<const float*>(chunk)[local] : fix(row[index(local)]);
  }
  // f(four elements, local index of the first) over the warp's piece, in no order across lanes
  template <typename F> __device__ __forceinline__ void each4(F f) const {
#pragma unroll 2
    for (int j = jb + (threadIdx.x & 31); j < je; j += 32) {
      const float4 v = quad(j);
      const float x[4] = {v.x, v.y, v.z, v.w};
      f(x, 4 * j);
    }
  }
  // f(x, local index) for every element of the warp's piece
  template <typename F> __device__ __forceinline__ void each(F f) const {
    each4([&](const float* x, int l) {
#pragma unroll
      for (int e = 0; e < 4; ++e) f(x[e], l + e);
    });
  }
};

// Which tokens are in play: bins below L, and of bin L (none: L is BINS) those at or before `place`.
struct Cut {
  float L;     // MAGIC + bin
  u64 place;
  __device__ __forceinline__ bool holds(float b, float x, int v) const {
    return b < L || (b == L && L < Weigh::MAGIC + BINS && place_of(x, v) >= place);
  }
};
__device__ __forceinline__ int bin_index(float b) { return __float_as_int(b) - __float_as_int(Weigh::MAGIC); }

template <bool RES, int NT> struct Sampler {
  static constexpr int NW = NT / 32;
  cg::cluster_group cl;
  Shared& sh;
  const Row<RES>& row;
  const Weigh& wt;
  int C, level;
  __device__ __forceinline__ Sampler(Shared& s, const Row<RES>& r, const Weigh& w)
      : cl(cg::this_cluster()), sh(s), row(r), wt(w), C((int)cl.num_blocks()), level(0) {}

  // Sum of the cluster's histograms: bins 4 * thread + i (remote reads, all in flight; few and
  // wide, since they cost by the request).
  __device__ __forceinline__ void counts(uint32_t (&c)[4]) {
    uint4 h[CMAX];
#pragma unroll
    for (int r = 0; r < CMAX; ++r)
      h[r] = r < C && threadIdx.x < HB ? reinterpret_cast<const uint4*>(cl.map_shared_rank(sh.hist, r))[threadIdx.x]
                                       : make_uint4(0, 0, 0, 0);
    c[0] = c[1] = c[2] = c[3] = 0;
#pragma unroll
    for (int r = 0; r < CMAX; ++r) c[0] += h[r].x, c[1] += h[r].y, c[2] += h[r].z, c[3] += h[r].w;
  }
  // Candidates' bins of a refinement: RB equal steps of the exponent over bins blo .. bhi.
  struct Steps {
    float lo, per;
    __device__ __forceinline__ Steps(float blo, float bhi)
        : lo(blo - Weigh::MAGIC - 0.5f), per((float)RB / (bhi - blo + 1.f)) {}
    __device__ __forceinline__ int operator()(const Weigh& wt, float x) const {
      // (no contraction: the same bin wherever this is inlined)
      const float t = __fmul_rn(__fsub_rn(__fmul_rn(__fsub_rn(wt.m, x), wt.c16), lo), per);
      return min(RB - 1, max(0, __float2int_rd(t)));
    }
  };
  __device__ __forceinline__ void clear_level(int par) {
    for (int i = threadIdx.x; i < RB; i += NT) sh.mass[par][i] = 0, sh.cnt[par][i] = 0;
  }
  // One pass over the warp's piece: f(four elements, local index of the first) returns a bit
  // for each that is a candidate of phase ph.  A lane's bits of eight quads are kept in a
  // register and listed together; each candidate also counts (with MASS its weight too) in the
  // refinement `par`.
  template <bool MASS, typename F>
  __device__ __forceinline__ void list_each4(int ph, int par, const Steps& steps, F f) {
    const int lane = threadIdx.x & 31;
    uint32_t klo = ~0u, khi = 0;
    for (int j0 = row.jb; j0 < row.je; j0 += 256) {
      uint32_t bits = 0;
      const int end = min(row.je, j0 + 256);
      int e = 0;
#pragma unroll 2
      for (int j = j0 + lane; j < end; j += 32, e += 4) {
        const float4 v = row.quad(j);
        const float x[4] = {v.x, v.y, v.z, v.w};
        bits |= f(x, 4 * j) << e;
      }
      __syncwarp();
      const int c = __popc(bits), incl = warp_scan(c), n = __shfl_sync(0xffffffffu, incl, 31);
      if (n == 0) continue;
      uint32_t at = 0;
      if (lane == 31) at = atomicAdd(&sh.fcnt[ph], (uint32_t)n);
      at = __shfl_sync(0xffffffffu, at, 31) + incl - c;
      for (; bits; bits &= bits - 1, ++at) {
        const int e = __ffs(bits) - 1, l = 4 * (j0 + 32 * (e >> 2) + lane) + (e & 3);
        const float x = row.at(l);
        const uint32_t k = key_of(x);
        const int b = steps(wt, x);
        klo = min(klo, k);
        khi = max(khi, k);
        if (at < LCAP) sh.list[at] = l;
        atomicAdd(&sh.cnt[par][b], 1u);
        if (MASS) atomicAdd(&sh.mass[par][b], wt(x));
      }
      __syncwarp();
    }
    klo = __reduce_min_sync(0xffffffffu, klo);
    khi = __reduce_max_sync(0xffffffffu, khi);
    if (lane == 0 && klo <= khi) {
      atomicMin(&sh.kmin[ph], klo);
      atomicMax(&sh.kmax[ph], khi);
    }
  }
  // The cluster's candidates of phase ph: how many, the range of their places, and whether one
  // CTA has more than its list holds.
  __device__ __forceinline__ void range(int ph, u64& n, u64& lo, u64& hi, bool& all) {
    const int lane = threadIdx.x & 31;
    uint32_t f = 0, klo = ~0u, khi = 0;
    if (lane < C) {
      f = *cl.map_shared_rank(&sh.fcnt[ph], lane);
      klo = *cl.map_shared_rank(&sh.kmin[ph], lane);
      khi = *cl.map_shared_rank(&sh.kmax[ph], lane);
    }
    n = __reduce_add_sync(0xffffffffu, f);
    all = __any_sync(0xffffffffu, f > LCAP);
    lo = (u64)__reduce_min_sync(0xffffffffu, klo) << IDX_BITS;
    hi = ((u64)__reduce_max_sync(0xffffffffu, khi) << IDX_BITS) | ((1 << IDX_BITS) - 1);
  }
  // f(x, token) for the CTA's candidates of phase ph with places lo .. hi: its list, or
  // (`all`) every element that `in` holds.
  template <typename F> __device__ __forceinline__ void candidates(int ph, bool all, const Cut& in, u64 lo, u64 hi, F f) {
    if (!all) {
      for (uint32_t i = threadIdx.x; i < sh.fcnt[ph]; i += NT) {
        const int l = sh.list[i], v = row.index(l);
        const float x = row.at(l);
        const u64 pl = place_of(x, v);
        if (pl >= lo && pl <= hi) f(x, pl);
      }
    } else {
      const float xlo = of_key((uint32_t)(lo >> IDX_BITS));
      row.each([&](float x, int l) {
        if (!(x >= xlo)) return;
        const int v = row.index(l);
        const u64 pl = place_of(x, v);
        if (pl >= lo && pl <= hi && in.holds(wt.bin(x), x, v)) f(x, pl);
      });
    }
  }
  // The bin of refinement `par` in which the running measure (number, or with MASS weight; `base`
  // before the first bin) reaches `want`, into sh.ib[0], with the measure before it and the number
  // of candidates in it in sh.bc.  False: it is not reached.
  struct Level {
    u64 c[2], m[2];   // bins 2 * thread, + 1
  };
  template <bool MASS> __device__ __forceinline__ Level level_sums(int par) {
    Level v = {{0, 0}, {0, 0}};
    if (threadIdx.x < RB / 2) {
      uint2 hc[CMAX];
      ulonglong2 hm[CMAX];
#pragma unroll
      for (int r = 0; r < CMAX; ++r) {
        hc[r] = r < C ? reinterpret_cast<const uint2*>(cl.map_shared_rank(&sh.cnt[par][0], r))[threadIdx.x] : make_uint2(0, 0);
        hm[r] = MASS && r < C ? reinterpret_cast<const ulonglong2*>(cl.map_shared_rank(&sh.mass[par][0], r))[threadIdx.x]
                              : make_ulonglong2(0, 0);
      }
#pragma unroll
      for (int r = 0; r < CMAX; ++r) v.c[0] += hc[r].x, v.c[1] += hc[r].y, v.m[0] += hm[r].x, v.m[1] += hm[r].y;
    }
    if (!MASS) v.m[0] = v.c[0], v.m[1] = v.c[1];
    return v;
  }
  __device__ __forceinline__ bool reach(const Level& v, u64 base, u64 want) {
    u64 total;
    u64 at = base + block_scan<NW>(v.m[0] + v.m[1], sh.red, total) - (v.m[0] + v.m[1]);
    if (base + total < want) return false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (at < want && want <= at + v.m[i]) {
        sh.ib[0] = 2 * threadIdx.x + i;
        sh.bc[0] = at;
        sh.bc[1] = v.c[i];
      }
      at += v.m[i];
    }
    __syncthreads();
    return true;
  }
  // The last place that stays among at most 32 candidates, those of phase ph that `is` holds:
  // the one at which the running measure, `base` before them, reaches `want`.
  template <bool MASS, typename F>
  __device__ __forceinline__ bool rank_last(int ph, bool all, const Cut& in, u64 lo, u64 hi, F is, u64 base, u64 want,
                                            u64& place) {
    candidates(ph, all, in, lo, hi, [&](float x, u64 pl) {
      if (!is(x)) return;
      const uint32_t i = atomicAdd(&sh.gcnt[ph], 1u);
      if (i < 32) sh.glist[ph][i] = pl;
    });
    cluster_sync(cl, C);
    if (threadIdx.x < 32) {
      // (places are not 0: the unused entries)
      const int lane = threadIdx.x;
      if (lane == 0) sh.nranked = 0;
      sh.ranked[lane] = 0;
      u64 got[CMAX];
#pragma unroll
      for (int r = 0; r < CMAX; ++r) got[r] = r < C ? cl.map_shared_rank(&sh.glist[ph][0], r)[lane] : 0;
      __syncwarp();
#pragma unroll
      for (int r = 0; r < CMAX; ++r)
        if (got[r]) {
          const uint32_t i = atomicAdd(&sh.nranked, 1u);
          if (i < 32) sh.ranked[i] = got[r];
        }
      __syncwarp();
      const u64 pl = sh.ranked[lane];
      u64 w = 0, before = base;
      if (pl) w = MASS ? wt(of_key((uint32_t)(pl >> IDX_BITS))) : 1;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const u64 opl = __shfl_sync(0xffffffffu, pl, j), ow = __shfl_sync(0xffffffffu, w, j);
        if (opl > pl) before += ow;
      }
      u64 mine = pl && before < want ? pl : ~0ull;
      u64 far = pl ? before + w : 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        mine = min(mine, __shfl_xor_sync(0xffffffffu, mine, o));
        far = max(far, __shfl_xor_sync(0xffffffffu, far, o));
      }
      if (threadIdx.x == 0) sh.bc[2] = far >= want ? mine : 0;
    }
    __syncthreads();
    place = sh.bc[2];
    return place != 0;
  }
  // The last place that stays: in the order of the candidates lo .. hi (n of them), with `base`
  // of the measure before them, the one at which the running measure reaches `want`.  False: it
  // is not reached.  The candidates are narrowed by RB at a time.
  template <bool MASS>
  __device__ bool resolve(int ph, bool all, const Cut& in, u64 lo, u64 hi, u64 n, u64 base, u64 want, u64& place) {
    while (n > 32 || all) {
      const int par = level++ & 1;   // the other half may still be read by the cluster
      clear_level(par);
      __syncthreads();
      const int s = max(0, 64 - __clzll((long long)(hi - lo)) - 8);
      candidates(ph, all, in, lo, hi, [&](float x, u64 pl) {
        const int b = (int)((hi - pl) >> s);
        atomicAdd(&sh.cnt[par][b], 1u);
        if (MASS) atomicAdd(&sh.mass[par][b], wt(x));
      });
      cluster_sync(cl, C);
      if (!reach(level_sums<MASS>(par), base, want)) return false;
      const u64 b = sh.ib[0];
      base = sh.bc[0];
      n = sh.bc[1];
      hi -= b << s;
      const u64 span = (1ull << s) - 1;
      if (hi - lo > span) lo = hi - span;
      __syncthreads();
      if (n <= 32) break;
    }
    return rank_last<MASS>(ph, all, in, lo, hi, [](float) { return true; }, base, want, place);
  }
  // The same for the candidates that list_each4 has counted in a refinement, whose sums are v (taken
  // after a cluster barrier): with at most 32 in the bin that reaches `want` they are ranked at once,
  // else (many equal logits, a list that is full) narrowed by their places.
  template <bool MASS>
  __device__ bool settle(int ph, const Level& v, const Steps& steps, const Cut& in, u64 base, u64 want, u64& place) {
    u64 n, lo, hi;
    bool all;
    range(ph, n, lo, hi, all);
    if (n == 0) return false;
    if (!all) {
      if (!reach(v, base, want)) return false;
      const int bin = sh.ib[0];
      const u64 before = sh.bc[0], here = sh.bc[1];
      __syncthreads();
      if (here <= 32)
        return rank_last<MASS>(ph, false, in, lo, hi, [&](float x) { return steps(wt, x) == bin; }, before, want,
                               place);
    }
    return resolve<MASS>(ph, all, in, lo, hi, n, base, want, place);
  }
};
}  // namespace

template <bool RES, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) k_sample(SampleParams p, int chunk_quads) {
  constexpr int NW = NT / 32;
  typedef typename Sampler<RES, NT>::Steps Steps;
  extern __shared__ __align__(16) float4 chunk[];
  __shared__ Shared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int r = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float T = p.temperature_row ? p.temperature_row[r] : p.temperature;
  const int k = p.top_k_row ? p.top_k_row[r] : p.top_k;
  const float top_p = p.top_p_row ? p.top_p_row[r] : p.top_p;
  const float min_p = p.min_p_row ? p.min_p_row[r] : p.min_p;
  Row<RES> row;
  row.row = p.logits + (long long)r * p.ld;
  row.chunk = chunk;
  row.V = p.vocab;
  row.a = (int)((reinterpret_cast<uintptr_t>(row.row) >> 2) & 3);
  row.nq = max(0, min(chunk_quads, (p.vocab + row.a + 3) / 4 - rank * chunk_quads));
  row.q0 = rank * chunk_quads;
  const int piece = (chunk_quads + NW - 1) / NW;   // quads of a warp
  row.jb = min(row.nq, warp * piece);
  row.je = min(row.nq, row.jb + piece);
  row.inf_row = false;
  for (int i = tid; i < BINS; i += NT) sh.hist[i] = 0;
  if (tid < 2) sh.fcnt[tid] = sh.gcnt[tid] = sh.kmax[tid] = 0, sh.kmin[tid] = ~0u;
  if (tid == 0) sh.idx = 0x7fffffff;
  if (tid < 2 * NWMAX) sh.add[tid >> 1][tid & 1] = 0;
  if (tid < 64) sh.glist[tid >> 5][tid & 31] = 0;
  float mx = -INFINITY;
  if (RES) {                                                     // the whole piece is in flight at once
    const int jf = row.q0 == 0 && row.a ? 1 : 0, jl = (p.vocab + row.a) / 4 - row.q0;   // whole quads: jf .. jl - 1
    uint32_t to = (uint32_t)__cvta_generic_to_shared(chunk + row.jb + lane);
    const float* from = row.row + row.index(4 * (row.jb + lane));
#pragma unroll 4
    for (int j = row.jb + lane; j < row.je; j += 32, to += 512, from += 128) {
      if (j >= jf && j < jl) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from));
      else chunk[j] = row.load(j);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");             // each lane reads its own quads back
  }
  row.each([&](float x, int) { mx = fmaxf(mx, x); });            // fmaxf drops NaN
  float own_mx = mx;                                             // of this thread's elements
  mx = warp_max(mx);
  if (lane == 0) sh.fred[warp] = mx;
  __syncthreads();
  if (warp == 0) {
    mx = warp_max(lane < NW ? sh.fred[lane] : -INFINITY);
    if (lane == 0) sh.mx = mx;
  }
  cluster_sync(cl, C);
  mx = warp_max(lane < C ? *cl.map_shared_rank(&sh.mx, lane) : -INFINITY);
  if (!(T >= 0x1p-127f) || mx == -INFINITY) {                    // the most likely token
    uint32_t best = 0x7fffffff;
    row.each4([&](const float* x, int l) {
      if (x[0] == mx || x[1] == mx || x[2] == mx || x[3] == mx)
        best = min(best, (uint32_t)row.index(l + (x[0] == mx ? 0 : x[1] == mx ? 1 : x[2] == mx ? 2 : 3)));
    });
    if (best != 0x7fffffff) atomicMin(&sh.idx, best);
    cluster_sync(cl, C);
    if (rank == 0 && tid == 0) {
      for (int i = 0; i < C; ++i) best = min(best, *cl.map_shared_rank(&sh.idx, i));
      p.tokens[(long long)r * p.out_ld] = best == 0x7fffffff ? 0 : (int)best;
      if (p.logprob) p.logprob[r] = 0.f;
    }
    cluster_sync(cl, C);                                         // remote shared memory is read until here
    return;
  }
  if (mx == INFINITY) {
    row.inf_row = true;
    if (RES)
      for (int j = row.jb + lane; j < row.je; j += 32) {
        const float4 v = chunk[j];
        chunk[j] = make_float4(row.fix(v.x), row.fix(v.y), row.fix(v.z), row.fix(v.w));
      }
    own_mx = row.fix(own_mx);
    mx = 0.f;
  }
  const Weigh wt(mx, T);
  Sampler<RES, NT> sm(sh, row, wt);
  constexpr float MAGIC = Weigh::MAGIC;
  Cut cut{MAGIC + BINS, 0};
  bool listed = false;                                           // every token in play is in a list, in these steps:
  Steps listed_steps(MAGIC, MAGIC);
  if (k > 0 && k < p.vocab) {
    // The largest element of each thread is a subset of the row, so where k of those are reached
    // the row's k-th token is at least as likely: the candidates are the bins down to there.
    // With fewer than k threads' worth, or that bin too full, a histogram of the whole row is
    // taken and the candidates are the one bin in which it reaches k.
    uint32_t c[4], total;
    u64 before = 0;
    bool all = true;                                             // (a list is full)
    float blo = MAGIC, bhi = MAGIC;
    int par = 0;
    if (float b = wt.bin(own_mx); b < MAGIC + BINS) atomicAdd(&sh.hist[bin_index(b)], 1u);
    cluster_sync(cl, C);
    // the bin in which the histogram reaches k, and how many are before it
    auto reach_k = [&] {
      sm.counts(c);
      const uint32_t own = c[0] + c[1] + c[2] + c[3];
      uint32_t n0 = block_scan<NW>(own, reinterpret_cast<uint32_t*>(sh.red), total) - own;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (n0 < (uint32_t)k && (uint32_t)k <= n0 + c[i]) sh.ib[0] = 4 * tid + i, sh.bc[0] = n0;
        n0 += c[i];
      }
      __syncthreads();
    };
    auto list = [&] {
      par = sm.level++ & 1;
      sm.clear_level(par);
      __syncthreads();
      sm.template list_each4<false>(0, par, Steps(blo, bhi), [&](const float* x, int) {
        uint32_t bits = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float b = wt.bin(x[e]);
          bits |= (uint32_t)(b >= blo && b <= bhi) << e;
        }
        return bits;
      });
      cluster_sync(cl, C);
      all = __any_sync(0xffffffffu, lane < C && *cl.map_shared_rank(&sh.fcnt[0], min(lane, C - 1)) > LCAP);
    };
    reach_k();
    if (total >= (uint32_t)k) {
      bhi = MAGIC + (float)sh.ib[0];
      list();
    }
    bool border = true;
    if (all) {
      cluster_sync(cl, C);
      for (int i = tid; i < BINS; i += NT) sh.hist[i] = 0;
      if (tid == 0) sh.fcnt[0] = sh.kmax[0] = 0, sh.kmin[0] = ~0u;
      __syncthreads();
      row.each([&](float x, int) {
        const float b = wt.bin(x);
        if (b < MAGIC + BINS) atomicAdd(&sh.hist[bin_index(b)], 1u);
      });
      cluster_sync(cl, C);
      reach_k();
      border = total > (uint32_t)k;                              // else every token that weighs something stays
      if (border) {
        blo = bhi = MAGIC + (float)sh.ib[0];
        before = sh.bc[0];
        list();
      } else {
        cluster_sync(cl, C);
      }
    }
    if (border) {
      const Cut in{bhi, 0};                                      // (the places leave only the candidates)
      listed_steps = Steps(blo, bhi);
      const auto level = sm.template level_sums<false>(par);
      listed = sm.template settle<false>(0, level, listed_steps, in, before, (u64)k, cut.place) && blo == MAGIC && !all;
      cut.L = wt.bin(of_key((uint32_t)(cut.place >> IDX_BITS)));
    }
    if (top_p < 1.f && !listed) {
      for (int i = tid; i < BINS; i += NT) sh.hist[i] = 0;
      __syncthreads();
    }
  }
  bool summed = false;                                           // sh.wsum holds the kept weight
  if (top_p < 1.f && listed) {
    // what top-k left is few: its weights are counted from the lists
    const int par = sm.level++ & 1;
    sm.clear_level(par);
    if (tid == 0) sh.fcnt[1] = sh.fcnt[0];
    __syncthreads();
    const u64 top = (1ull << (32 + IDX_BITS)) - 1;
    u64 total = 0;
    sm.candidates(1, false, cut, cut.place, top, [&](float x, u64) {
      const u64 w = wt(x);
      const int b = listed_steps(wt, x);
      atomicAdd(&sh.cnt[par][b], 1u);
      atomicAdd(&sh.mass[par][b], w);
      total += w;
    });
    total = warp_sum64(total);
    if (lane == 0) sh.red[warp] = total;
    __syncthreads();
    if (warp == 0) {
      total = warp_sum64(lane < NW ? sh.red[lane] : 0);
      if (lane == 0) sh.total = total;
    }
    cluster_sync(cl, C);
    const auto level = sm.template level_sums<true>(par);
    total = warp_sum64(lane < C ? *cl.map_shared_rank(&sh.total, lane) : 0);
    const u64 want = (u64)max(1.0, ceil((double)fmaxf(top_p, 0.f) * (double)total));
    sm.reach(level, 0, want);                                    // (the total is the bins' own)
    const int bin = sh.ib[0];
    const u64 before = sh.bc[0], here = sh.bc[1];
    __syncthreads();
    u64 place = 0;
    const bool ok = here <= 32 ? sm.template rank_last<true>(1, false, cut, cut.place, top,
                                                             [&](float x) { return listed_steps(wt, x) == bin; }, before,
                                                             want, place)
                               : sm.template resolve<true>(1, false, cut, cut.place, top, (u64)p.vocab, 0, want, place);
    if (ok) cut.place = place;
  } else if (top_p < 1.f) {
    // A weight is counted as 11 bits of 2^-(bin / 16) (2^20 of them fit 32 bits), interpolated
    // linearly in the bin (up to half a bin to each side): off by less than 5e-4 of it, so bins
    // whose running weight is within 6e-4 of the border bracket it.  (Tokens below 1e-4 / V of the largest weight hold
    // less than 1e-4 of the total: they are not counted.)
    const float lim = fminf(MAGIC + (BINS - 1), cut.L);
    const bool cut_any = cut.L < MAGIC + BINS;
    const float far = fminf(lim, MAGIC + ceilf(16.f * log2f(1e4f * (float)p.vocab)));
    const uint32_t hist0 = (uint32_t)__cvta_generic_to_shared(sh.hist) - 4 * __float_as_uint(MAGIC);
    auto count = [&](auto with_cut) {
      row.each4([&](const float* x, int l) {
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          float b[2], v[2];
          F2 f;
          wt.bin2(x[e], x[e + 1], b[0], b[1], f);
          fma2(f, F2(-88.72f), F2(2048.f + 8388608.f)).get(v[0], v[1]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (decltype(with_cut)::value && !cut.holds(b[i], x[e + i], row.index(l + e + i))) b[i] = MAGIC + BINS;
            // (a predicate instead of a branch round each)
            asm volatile("{\n .reg .pred p;\n setp.le.f32 p, %0, %1;\n @p red.shared.add.u32 [%2], %3;\n}" ::"f"(b[i]),
                         "f"(far), "r"(hist0 + 4 * __float_as_uint(b[i])), "r"(__float_as_uint(v[i]) & 0x3fffu) : "memory");
          }
        }
      });
    };
    if (cut_any) count(std::true_type());
    else count(std::false_type());
    if (tid < 2) sh.ib[2 + tid] = tid ? BINS - 1 : 0;
    cluster_sync(cl, C);
    int par;
    {
      // the bins in which the running weight reaches the border less, and plus, the margin
      uint32_t c[4];
      u64 w[4], own = 0, all;
      sm.counts(c);
#pragma unroll
      for (int i = 0; i < 4; ++i) own += w[i] = (u64)((float)c[i] * exp2f(20.f - (float)(4 * tid + i) / 16.f));
      u64 at = block_scan<NW>(own, sh.red, all) - own;
      const u64 b0 = (u64)fmax(0.0, ((double)top_p - 6e-4) * (double)all), b1 = (u64)(((double)top_p + 6e-4) * (double)all);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (at < b0 && b0 <= at + w[i]) sh.ib[2] = 4 * tid + i;
        if (at < b1 && b1 <= at + w[i]) sh.ib[3] = 4 * tid + i;
        at += w[i];
      }
      par = sm.level++ & 1;
      sm.clear_level(par);
      __syncthreads();
    }
    const float blo = MAGIC + (float)sh.ib[2], bhi = MAGIC + (float)sh.ib[3];
    const Steps steps(blo, bhi);
    Sum sum_total, sum_above;
    auto weigh = [&](auto wide, auto with_cut) {
      sm.template list_each4<true>(1, par, steps, [&](const float* x, int l) {
        float b[4];
        uint32_t bits = 0;
        F2 f;
        wt.bin2(x[0], x[1], b[0], b[1], f);
        wt.bin2(x[2], x[3], b[2], b[3], f);
        if (decltype(with_cut)::value) {
          if (!(b[0] <= lim || b[1] <= lim || b[2] <= lim || b[3] <= lim)) return bits;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!cut.holds(b[e], x[e], row.index(l + e))) b[e] = MAGIC + BINS;
        }
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          float w0, w1;
          wt.template weight2<decltype(wide)::value>(x[e], x[e + 1]).get(w0, w1);
          w0 = x[e] >= wt.floor && !(decltype(with_cut)::value && b[e] == MAGIC + BINS) ? w0 : 0.f;
          w1 = x[e + 1] >= wt.floor && !(decltype(with_cut)::value && b[e + 1] == MAGIC + BINS) ? w1 : 0.f;
          sum_total.add(F2(w0, w1));
          sum_above.add(F2(b[e] < blo ? w0 : 0.f, b[e + 1] < blo ? w1 : 0.f));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (b[e] >= blo && b[e] <= bhi) bits |= 1u << e;
        return bits;
      });
    };
    if (wt.wide) cut_any ? weigh(std::true_type(), std::true_type()) : weigh(std::true_type(), std::false_type());
    else cut_any ? weigh(std::false_type(), std::true_type()) : weigh(std::false_type(), std::false_type());
    u64 total = warp_sum64(sum_total.units()), above = warp_sum64(sum_above.units());
    if (lane == 0) sh.wsum[warp] = above, sh.red[warp] = total;
    __syncthreads();
    if (warp == 0) {
      const u64 t = warp_sum64(lane < NW ? sh.red[lane] : 0), a = warp_sum64(lane < NW ? sh.wsum[lane] : 0);
      if (lane == 0) sh.total = t, sh.above = a;
    }
    cluster_sync(cl, C);
    const auto level = sm.template level_sums<true>(par);        // (with the other remote reads)
    total = warp_sum64(lane < C ? *cl.map_shared_rank(&sh.total, lane) : 0);
    above = warp_sum64(lane < C ? *cl.map_shared_rank(&sh.above, lane) : 0);
    const u64 want = (u64)max(1.0, ceil((double)fmaxf(top_p, 0.f) * (double)total));
    u64 place = 0;
    const bool full = __any_sync(0xffffffffu, lane < C && *cl.map_shared_rank(&sh.fcnt[1], min(lane, C - 1)) > LCAP);
    summed = above < want && !full;
    bool ok = above < want && sm.template settle<true>(1, level, steps, cut, above, want, place);
    // The bracket missed the border, as where 16 bins per power of two pass fp32's range (T below
    // 7.7e-38): the whole order of what weighs something.
    if (!ok) {
      cluster_sync(cl, C);
      if (tid == 0) sh.gcnt[1] = 0;
      if (tid < 32) sh.glist[1][tid] = 0;
      summed = false;
      __syncthreads();
      ok = sm.template resolve<true>(1, true, cut, (u64)key_of(wt.floor) << IDX_BITS, (1ull << (32 + IDX_BITS)) - 1,
                                     (u64)p.vocab, 0, want, place);
    }
    cut.L = -1.f;                                                // the place alone decides
    // (not reached: the weights rounded one by one sum to less than top_p of their sum, which then is
    // within a rounding of 1, and top-k's border stays)
    if (ok) cut.place = place;
  }
  // min-p: (x - m) / T >= ln(min_p)
  float xmin = -INFINITY;
  if (min_p > 0.f) {
    // (an infinite temperature: every weight is 1)
    xmin = isinf(T) ? -INFINITY : fminf(mx, __double2float_ru((double)mx + (double)T * log((double)fminf(min_p, 1.f))));
  }
  const bool by_place = cut.place != 0;
  const float xcut = by_place ? of_key((uint32_t)(cut.place >> IDX_BITS)) : -INFINITY;
  const float xlim = fmaxf(fmaxf(xmin, xcut), wt.floor);
  // beyond x >= xlim: a token level with the border
  auto drops = [&](float x, int l) { return by_place && x == xcut && place_of(x, row.index(l)) < cut.place; };
  auto kept = [&](float x, int l) -> u64 { return x >= xlim && !drops(x, l) ? wt(x) : 0; };
  if (listed || (summed && xmin <= xcut)) {
    // the weight before the bracket is known (with a list of all: none): the kept candidates
    // join their pieces (22 bits to a word: up to LCAP of them fit)
    if (listed && tid < NW) sh.wsum[tid] = 0;
    const uint32_t n = listed ? sh.fcnt[0] : sh.fcnt[1];
    for (uint32_t i = tid; i < n; i += NT) {
      const int l = sh.list[i], w = (l >> 2) / piece;
      const u64 q = kept(row.at(l), l);
      if (q) atomicAdd(&sh.add[w][0], (uint32_t)q & 0x3fffffu), atomicAdd(&sh.add[w][1], (uint32_t)(q >> 22));
    }
    __syncthreads();
    if (tid < NW) sh.wsum[tid] += sh.add[tid][0] + ((u64)sh.add[tid][1] << 22);
  } else {
    Sum sum;
    auto weigh = [&](auto wide) {
      row.each4([&](const float* x, int l) {
        if (!(x[0] >= xlim || x[1] >= xlim || x[2] >= xlim || x[3] >= xlim)) return;
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          wt.template weight2<decltype(wide)::value>(x[e], x[e + 1]).get(w[e], w[e + 1]);
          if (!(x[e] >= xlim)) w[e] = 0.f;
          if (!(x[e + 1] >= xlim)) w[e + 1] = 0.f;
        }
        if (x[0] == xcut || x[1] == xcut || x[2] == xcut || x[3] == xcut) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (drops(x[e], l + e)) w[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 4; e += 2) sum.add(F2(w[e], w[e + 1]));
      });
    };
    if (wt.wide) weigh(std::true_type());
    else weigh(std::false_type());
    const u64 mine = warp_sum64(sum.units());
    __syncthreads();
    if (lane == 0) sh.wsum[warp] = mine;
  }
  cluster_sync(cl, C);
  const u64 mine = tid < C * NW ? cl.map_shared_rank(&sh.wsum[0], tid / NW)[tid % NW] : 0;
  u64 total;
  const u64 incl = block_scan<NW>(mine, sh.red, total);
  if (C > 1) cl.barrier_arrive();                                // the last read of remote shared memory is done
  const float u = p.u[r];
  const double uc = u > 0.f ? fmin((double)u, 1.0 - 0x1p-24) : 0.0;   // NaN: 0
  const u64 target = (u64)(uc * (double)total);
  if (mine && incl - mine <= target && target < incl) {
    sh.ib[0] = tid;
    sh.bc[0] = incl - mine;
  }
  __syncthreads();
  if (sh.ib[0] == rank * NW + warp) {
    u64 base = sh.bc[0];
    int tok = -1;                                                // the last kept token so far
    float tok_x = 0.f;
    bool found = false;
    for (int j0 = row.jb; j0 < row.je; j0 += 32) {
      const int j = j0 + lane;
      u64 w[4] = {0, 0, 0, 0};
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (j < row.je) {
        v = row.quad(j);
        w[0] = kept(v.x, 4 * j); w[1] = kept(v.y, 4 * j + 1); w[2] = kept(v.z, 4 * j + 2); w[3] = kept(v.w, 4 * j + 3);
      }
      const u64 c = warp_scan(w[0] + w[1] + w[2] + w[3]);
      const unsigned hit = __ballot_sync(0xffffffffu, base + c > target);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          u64 s = base + c - (w[0] + w[1] + w[2] + w[3]);
          int e = 0;
          for (; e < 3; ++e) {
            s += w[e];
            if (s > target) break;
          }
          tok_x = e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w;
          tok = row.index(4 * j + e);
          found = true;
        }
        break;
      }
      if (w[0] | w[1] | w[2] | w[3]) {
        const int e = w[3] ? 3 : w[2] ? 2 : w[1] ? 1 : 0;
        tok_x = e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w;
        tok = row.index(4 * j + e);
      }
      base += __shfl_sync(0xffffffffu, c, 31);
    }
    // the warp's sum was off by a rounding and the target lies in it: the last kept token
    const int top = __reduce_max_sync(0xffffffffu, tok);
    const bool any = __any_sync(0xffffffffu, found);
    if (any ? found : tok == top && tok >= 0) {
      p.tokens[(long long)r * p.out_ld] = tok;
      if (p.logprob) {
        const double z = tok_x == mx ? 0.0 : ((double)tok_x - (double)mx) / (double)T;
        p.logprob[r] = (float)(z - log((double)total * 0x1p-44));
      }
    }
  }
  if (C > 1) cl.barrier_wait();
}

// Cluster size: two CTAs on an SM can hold 100 KB of a row each, so that one's passes run while
// the other loads; with few rows the cluster grows, down to 4096 logits a CTA.
// Threads: with 256 a CTA issues fewer instructions (what it does beside the passes costs every
// warp the same) but waits longer for each.  More short rows than SMs run better with them (512
// rows of 8000 logits with top-p: 31 us, with 512 threads 43); others do not (33 rows of 4000
// without it: 10.8 us, with 512 threads 8.7; 256 rows of 201,088 with it, in an earlier state:
// 432 us, with 512 threads 358).
int launch_sample(const SampleParams& p, cudaStream_t s) {
  const int quads = p.vocab / 4 + 2;                             // whatever the row's alignment
  const int sms = device_sm_count();
  int C = 1;
  while (C < CMAX && ((quads + C - 1) / C > 25200 / 4 || ((long long)p.n * C < sms && quads > C * 2048))) C *= 2;
  const int chunk = (quads + C - 1) / C, most = 227 * 1024 - 1024 - (int)sizeof(Shared);
  const bool res = (long long)chunk * 16 <= most;
  const bool small = p.vocab <= 8192 && p.n > sms;
  void (*kernel)(SampleParams, int) = small ? k_sample<true, 256> : res ? k_sample<true, 512> : k_sample<false, 512>;
  if (!ensure_smem_limit((const void*)kernel, res ? most : 0)) return -1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.n * (long long)C));
  cfg.blockDim = dim3(small ? 256 : 512);
  cfg.dynamicSmemBytes = res ? (size_t)chunk * 16 : 0;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, p, chunk) != cudaSuccess) return -1;
  note_launch();
  return 0;
}

}  // namespace rdt
