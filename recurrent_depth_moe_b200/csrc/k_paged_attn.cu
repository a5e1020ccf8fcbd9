// One-token attention over the paged key / value cache (GQA): for query head h of sequence b
//   o = sum_j softmax_j(q . k_j / sqrt(hd)) v_j,   j < the sequence's visible keys,
// zero where nothing is visible.  The keys of a sequence are split into n_split ranges of its
// own length, each with a running maximum m and sum l (base-2 logarithms); the ranges are
// joined by  o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s.
//
// k_paged_attn_any: any head width up to 256, any page size, fp32 or bf16, both storage forms.
// CTA = (range, kv head and tile of 8 of its query heads, sequence); 32-key K and V tiles are
// widened to fp32 in shared memory, a warp scores its heads with a key per lane, and a thread
// sums its output channels.  Everything is held in fp32.
#include "paged.cuh"

#include <algorithm>

namespace rdt {

namespace {
constexpr int TK = 32, GT = 8;   // keys and query heads per tile
inline size_t any_smem(int hd) { return sizeof(float) * ((size_t)GT * hd + 2 * (size_t)TK * (hd + 1) + GT * TK + GT) + 2 * TK * sizeof(long long); }
}  // namespace

template <typename T, bool Q>
__global__ void __launch_bounds__(128) k_paged_attn_any(PagedAttnParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int hd = p.c.hd, Hkv = p.c.Hkv, G = p.H / Hkv, ldk = hd + 1;
  long long* off = reinterpret_cast<long long*>(smem);          // [TK] slot of each key (-1: masked)
  float* qs = reinterpret_cast<float*>(off + TK);               // [GT][hd]
  float* Ks = qs + GT * hd;                                     // [TK][hd + 1]
  float* Vs = Ks + TK * ldk;
  float* ps = Vs + TK * ldk;                                    // [GT][TK]
  float* corr = ps + GT * TK;                                   // [GT]
  const int split = blockIdx.x, n_split = gridDim.x, n_ht = (G + GT - 1) / GT;
  const int g = blockIdx.y / n_ht, h0 = (blockIdx.y % n_ht) * GT, nh = min(GT, G - h0), b = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int len = visible_keys(p.c, p.lens, b, p.len_add, p.st, 221);
  const int chunk = ((len + n_split - 1) / n_split + TK - 1) / TK * TK;
  const long long j0 = (long long)split * chunk;
  const int j1 = (int)min((long long)len, j0 + chunk);
  const float sl2 = p.scale * 1.4426950408889634f;
  for (int i = tid; i < nh * hd; i += 128)
    qs[i] = to_f(((const T*)p.q)[(long long)b * p.q_row + (long long)(g * G + h0) * hd + i]) * sl2;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};       // heads warp and warp + 4
  float acc[GT][2];                                             // channels tid and tid + 128
#pragma unroll
  for (int h = 0; h < GT; ++h) acc[h][0] = acc[h][1] = 0.f;
  for (long long j = j0; j < j1; j += TK) {
    const int nk = (int)min((long long)TK, j1 - j);
    __syncthreads();
    if (tid < TK) {
      long long o = -1;
      if (tid < nk) {
        const int page = page_of(p.c, b, (int)j + tid, p.st, 222);
        if (page >= 0) o = ((long long)page * Hkv + g) * p.c.page_size + ((int)j + tid) % p.c.page_size;
      }
      off[tid] = o;
    }
    __syncthreads();
    for (int i = tid; i < TK * hd; i += 128) {
      const int r = i / hd, d = i - r * hd;
      const long long o = off[r];
      float kx = 0.f, vx = 0.f;                                 // masked rows hold zeros: 0 * v is 0 whatever the slot holds
      if (o >= 0) {
        if (Q) {
          kx = e4m3_f(((const uint8_t*)p.c.k)[o * hd + d]) * exp_byte_scale(p.c.ke[o]);
          vx = e4m3_f(((const uint8_t*)p.c.v)[o * hd + d]) * exp_byte_scale(p.c.ve[o]);
        } else {
          kx = to_f(((const T*)p.c.k)[o * hd + d]);
          vx = to_f(((const T*)p.c.v)[o * hd + d]);
        }
      }
      Ks[r * ldk + d] = kx;
      Vs[r * ldk + d] = vx;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int h = warp + 4 * u;
      if (h < nh) {
        float s = 0.f;
        for (int d = 0; d < hd; ++d) s = fmaf(qs[h * hd + d], Ks[lane * ldk + d], s);
        if (off[lane] < 0) s = -INFINITY;
        const float mx = fmaxf(m[u], warp_max(s));
        const float base = mx == -INFINITY ? 0.f : mx;
        const float e = exp2f(s - base), c = exp2f(m[u] - base);
        m[u] = mx;
        l[u] = l[u] * c + warp_sum(e);
        ps[h * TK + lane] = e;
        if (lane == 0) corr[h] = c;
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int d = tid + 128 * u;
      if (d < hd) {
#pragma unroll
        for (int h = 0; h < GT; ++h)
          if (h < nh) acc[h][u] *= corr[h];
        for (int r = 0; r < TK; ++r) {
          const float v = Vs[r * ldk + d];
#pragma unroll
          for (int h = 0; h < GT; ++h)
            if (h < nh) acc[h][u] = fmaf(ps[h * TK + r], v, acc[h][u]);
        }
      }
    }
  }
  // joined here (one range) or by k_paged_attn_join
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int h = warp + 4 * u;
    if (h < nh && lane == 0) {
      if (n_split == 1) {
        corr[h] = l[u];
      } else {
        const long long s = ((long long)b * p.H + g * G + h0 + h) * n_split + split;
        p.part_ml[2 * s] = m[u];
        p.part_ml[2 * s + 1] = l[u];
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int d = tid + 128 * u;
    if (d >= hd) continue;
#pragma unroll
    for (int h = 0; h < GT; ++h) {
      if (h >= nh) continue;
      const int head = g * G + h0 + h;
      if (n_split == 1) {
        ((T*)p.o)[(long long)b * p.o_row + (long long)head * hd + d] = from_f<T>(corr[h] != 0.f ? acc[h][u] / corr[h] : 0.f);
      } else {
        p.part_o[(((long long)b * p.H + head) * n_split + split) * hd + d] = acc[h][u];
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(128) k_paged_attn_join(PagedAttnParams p, int n_split) {
  const long long bh = blockIdx.x;
  const int b = (int)(bh / p.H), h = (int)(bh % p.H), hd = p.c.hd;
  const float* ml = p.part_ml + bh * n_split * 2;
  float M = -INFINITY;
  for (int s = 0; s < n_split; ++s) M = fmaxf(M, ml[2 * s]);
  const float base = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  for (int s = 0; s < n_split; ++s) L += exp2f(ml[2 * s] - base) * ml[2 * s + 1];
  for (int d = threadIdx.x; d < hd; d += 128) {
    float o = 0.f;
    for (int s = 0; s < n_split; ++s) o += exp2f(ml[2 * s] - base) * p.part_o[(bh * n_split + s) * hd + d];
    ((T*)p.o)[(long long)b * p.o_row + (long long)h * hd + d] = from_f<T>(L != 0.f ? o / L : 0.f);
  }
}

// Ranges per sequence: enough CTAs for four on each SM, at most one per 128 positions the
// table can hold.
static int any_splits(const PagedView& c, int B, int H) {
  const long long ctas = (long long)B * c.Hkv * ((H / c.Hkv + GT - 1) / GT);
  const long long cap = (long long)c.max_pages * c.page_size;
  const long long want = (4LL * device_sm_count() + ctas - 1) / ctas;
  return (int)std::max<long long>(1, std::min<long long>(std::min<long long>(want, (cap + 127) / 128), 1024));
}

size_t paged_attn_scratch(int dtype, const PagedView& c, int B, int H) {
  (void)dtype;
  const int n = any_splits(c, B, H);
  return n > 1 ? (size_t)B * H * n * (c.hd + 2) * sizeof(float) : 0;
}

int launch_paged_attn(int dtype, const PagedAttnParams& p0, cudaStream_t s) {
  PagedAttnParams p = p0;
  const int G = p.H / p.c.Hkv, n_ht = (G + GT - 1) / GT, n_split = any_splits(p.c, p.B, p.H);
  p.part_o = (float*)p.scratch;
  p.part_ml = p.part_o + (size_t)p.B * p.H * n_split * p.c.hd;
  const dim3 grid((unsigned)n_split, (unsigned)(p.c.Hkv * n_ht), (unsigned)p.B);
  const int smem = (int)any_smem(p.c.hd), most = (int)any_smem(256);
#define RDT_ANY(TT, QQ)                                                                     \
  do {                                                                                      \
    if (!ensure_smem_limit((const void*)k_paged_attn_any<TT, QQ>, most)) return -1;         \
    k_paged_attn_any<TT, QQ><<<grid, 128, smem, s>>>(p);                                    \
    note_launch();                                                                          \
    if (n_split > 1) {                                                                      \
      k_paged_attn_join<TT><<<(unsigned)(p.B * p.H), 128, 0, s>>>(p, n_split);              \
      note_launch();                                                                        \
    }                                                                                       \
  } while (0)
  if (dtype == 0) {
    if (p.c.e4m3) RDT_ANY(float, true);
    else RDT_ANY(float, false);
  } else {
    if (p.c.e4m3) RDT_ANY(bf16, true);
    else RDT_ANY(bf16, false);
  }
#undef RDT_ANY
  return 0;
}

}  // namespace rdt
