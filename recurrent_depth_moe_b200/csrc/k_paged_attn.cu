// One-token attention over the paged key / value cache (GQA): for query head h of sequence b
//   o = sum_j softmax_j(q . k_j / sqrt(hd)) v_j,   j < the sequence's visible keys,
// zero where nothing is visible.  Every cached byte is read once (per 8 query heads of a kv
// head), so the floor is the cache's bytes at HBM rate.
//
// The work is one line of tiles: (sequence, kv head and group of 8 query heads, keys).  The
// grid is what the GPU holds at once (up to 128 channels), and its i-th worker takes the i-th
// equal piece of the line, so ragged lengths and any batch keep every worker busy to the end; the
// lengths stay on the device.  A worker walks its piece with the running maximum m and sum l of a
// softmax (base-2 logarithms).  A (sequence, head group) that one worker walks whole is written at
// once; where it is spread over several, k_paged_attn_join joins their parts,
//   o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s.
//
// k_paged_attn_mma (bf16 model, either storage, head width a multiple of 8 (16 for e4m3) up to
// 256): both products on mma.m16n8k16 with the query heads as the 16 rows.  The cache moves by
// 16-byte cp.async into a ring that each warp keeps for itself, so no warp waits for another.
// Fragments are read with 16-byte loads under a permutation of the channels (scores) and of the
// keys (values), the same on both operands, and a xor of the 16-byte pieces by row keeps those
// loads free of bank conflicts.  A weight p enters the second product in two 16-bit words: rows
// 0-7 hold its upper, rows 8-15 its lower word, which the 8 heads leave free, so p has 16 (bf16)
// or 22 (fp16) bits at no cost.  e4m3 values become fp16, exactly; a row's exponent of K scales
// its score, of V its weight.  fp16 ends at 2^-24, so what enters there is p 2^(e - top + 15), e
// the row's exponent and top the largest so far, under a reference m that is the largest score
// only while the rows' exponents lie close together: else a row far above the others that no
// head attends would push the weights of the rest below fp16's range.  Then m is the largest of
// score + e - top, each head's own, so that what counts most in the sum stands at 2^15 (the
// weights themselves are fp32 and may pass 1).
//
// Measured on one B200 (128 channels; share of the measured copy rate, 6548.5 GB/s): one sequence
// of 131,071 keys, 32 heads on 8, bf16 98 us (84%); 64 sequences of 1 to 4224 keys, 24 heads on 8,
// bf16 106 us (80%), bound by HBM with a quarter of the issue slots used; 128 sequences of 4097 to
// 8191 keys in e4m3 324 us (77%), bound by issue (48% active with 12 warps on an SM).
//
// k_paged_attn_simt (fp32 model, other widths): a lane per key and per channel in fp32; 64
// sequences of 1000 to 2000 keys, 24 heads on 8, in fp32 171 us (70%), in e4m3 281 us (11%).
#include "paged.cuh"

#include <algorithm>

namespace rdt {

namespace {
constexpr int GT = 8;               // query heads of a group
constexpr int WARPS = 4;            // of a CTA
constexpr float LOG2E = 1.4426950408889634f;

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// ------------------------------------------------------------------------------------------
// the line of work
// ------------------------------------------------------------------------------------------
// Units per sequence: ceil(keys / tile) tiles, and START for what a group costs beside them, for
// each of `segs` (kv head, head group) pairs; tile t is unit START + t of its group.
constexpr int START = 2;
constexpr int LENS = 512;           // lengths kept in shared memory (of a longer batch: none)
struct Lens {
  const PagedAttnParams& p;
  const int* kept;                  // shared memory, or null
  __device__ __forceinline__ int keys(int b) const {
    return kept ? kept[b] : visible_keys(p.c, p.lens, b, p.len_add, nullptr, 0);
  }
  __device__ __forceinline__ int tiles(int b, int tile) const { return (keys(b) + tile - 1) / tile; }
  __device__ __forceinline__ int units(int b, int tile) const {
    const int n = tiles(b, tile);
    return n ? n + START : 0;
  }
};
// Length of the line (all 128 threads of the CTA; keep: LENS ints, red: 4 words of shared memory).
__device__ long long line_length(const PagedAttnParams& p, int segs, int tile, int* keep, long long* red) {
  long long n = 0;
  for (int b = threadIdx.x; b < p.B; b += 128) {
    const int len = visible_keys(p.c, p.lens, b, p.len_add, p.st, 221);
    if (p.B <= LENS) keep[b] = len;
    if (len > 0) n += (long long)((len + tile - 1) / tile + START) * segs;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = n;
  __syncthreads();
  return red[0] + red[1] + red[2] + red[3];
}
// The sequence that holds unit x, and x's place in it, by one warp: 32 sequences at a time.
struct Place {
  int b;
  long long at;
};
__device__ __forceinline__ Place line_find(const Lens& lens, int segs, int tile, long long x) {
  const int lane = threadIdx.x & 31;
  long long base = 0;
  for (int b0 = 0; b0 < lens.p.B; b0 += 32) {
    const int b = b0 + lane;
    const long long n = b < lens.p.B ? (long long)lens.units(b, tile) * segs : 0;
    long long c = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, c, o);
      if (lane >= o) c += t;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + c > x);
    if (hit) {
      const int l = __ffs(hit) - 1;
      return Place{b0 + l, x - base - __shfl_sync(0xffffffffu, c - n, l)};
    }
    base += __shfl_sync(0xffffffffu, c, 31);
  }
  return Place{lens.p.B, 0};
}
// Units of a worker: an equal share, but no less than `least` (a short line is not spread thin).
__device__ __forceinline__ long long piece_of(long long length, int workers, int least) {
  const long long q = (length + workers - 1) / workers;
  return q > least ? q : least;
}

// ------------------------------------------------------------------------------------------
// parts of a head group: m, l per head and o per head and channel, fp32
// ------------------------------------------------------------------------------------------
// CTA i leaves part 0 of the group it enters in the middle and part 1 of the one it begins and
// does not finish, and in desc[i] the group it enters in the middle and finishes: it is the
// last of the CTAs first .. i that share it.  (Behind the CTAs' parts lie those of their warps.)
struct Desc {
  int b, seg, first, pad;
};
__device__ __forceinline__ float* part_ml(const PagedAttnParams& p, int at, int which) {
  return p.part_ml + ((long long)at * 2 + which) * GT * 2;
}
__device__ __forceinline__ float* part_o(const PagedAttnParams& p, int at, int which) {
  return p.part_o + ((long long)at * 2 + which) * GT * p.c.hd;
}
__device__ __forceinline__ Desc* desc_of(const PagedAttnParams& p) { return reinterpret_cast<Desc*>(p.scratch); }
__device__ __forceinline__ void zero_rows(const PagedAttnParams& p, const Lens& lens, int es) {
  const int n = p.H * p.c.hd * es / 2;   // 16-bit words of a row
  for (int b = blockIdx.x; b < p.B; b += gridDim.x)
    if (lens.keys(b) == 0)
      for (int i = threadIdx.x; i < n; i += 128) ((uint16_t*)p.o)[(long long)b * p.o_row * es / 2 + i] = 0;
}
__device__ __forceinline__ void let_join_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
}  // namespace

// ------------------------------------------------------------------------------------------
// tensor-core kernel
// ------------------------------------------------------------------------------------------
namespace {
// Keys of a tile (K and V are 8 KB at 128 channels), ring stages and CTAs on an SM.  bf16 waits
// for memory, so it takes the deeper ring (105 us against 110 with 2 and 3, one sequence of
// 131,071 keys); e4m3 issues twice the instructions a byte and takes more warps (313 us against
// 342, 128 sequences of 4097 to 8191 keys).
template <int HD, bool Q> struct Tile {
  static constexpr int KEYS = Q || HD == 64 ? 32 : 16, STAGES = Q ? 2 : 3, CTAS = Q ? 3 : 2;
};

template <int HD, bool Q> struct Ring {    // HD: the head width rounded up to 64, 128 or 256
  static constexpr int ROW = HD * (Q ? 1 : 2);                  // bytes of a row
  static constexpr int STAGE = 2 * Tile<HD, Q>::KEYS * ROW;         // K then V
  static constexpr int BYTES = Tile<HD, Q>::STAGES * STAGE;         // of a warp
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src));
}
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;                                 // 0: zeros are written, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n));
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
template <bool Q>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if (Q)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t e4m3x2_h2(uint32_t two) {   // two e4m3 bytes to fp16, exactly
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)two));
  return r;
}
// Two weights as 16-bit words: the upper ones packed, and what they leave.
template <bool Q> __device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  if (Q) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    const float2 f = __bfloat1622float2(h);
    const __nv_bfloat162 l = __floats2bfloat162_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
  }
}
// 16-byte piece c of row r of a K tile: the 8 lanes of one 16-byte load phase hold rows 2i,
// 2i + 1 and 4 neighbouring pieces; of a V tile: rows 2i (+ const), i < 4, and pieces 2j, 2j + 1.
// Rows of 4 pieces (64 e4m3 channels) lie two to a 128-byte line: K needs no xor, and half the
// conflicts of V remain.
template <int PIECES> __device__ __forceinline__ int swz_k(int r, int c) {
  return PIECES < 8 ? c : c ^ ((r & 1) << 2 | (r >> 1 & 3));
}
template <int PIECES> __device__ __forceinline__ int swz_v(int r, int c) {
  return c ^ (PIECES < 8 ? (r >> 1 & 1) << 1 : (r >> 1 & 3) << 1);
}
}  // namespace

// The sum over the weights' upper words and over their lower ones, which may be 0 or negative: an
// infinite value is in the upper words' sum as it should be (those are above 0), in the lower
// words' as a NaN or with the wrong sign.
__device__ __forceinline__ float both_words(float hi, float lo) { return fabsf(hi) <= 3.402823466e38f ? hi + lo : hi; }
// 2^d, d <= 127; below the smallest normal value: nothing
__device__ __forceinline__ float pow2_down(int d) { return d < -126 ? 0.f : __int_as_float((127 + d) << 23); }
// e4m3: a row's weight carries 2^UP, for fp16's upper range (65504).  A tile whose rows' exponents
// are at most SPREAD below the largest so far, and none above, keeps the score as the reference
// (its largest weight stands at 2^(UP - SPREAD) or more) and pays one vote for this; 128 sequences
// of 4097 to 8191 keys 324 us, without 322.  The reference is at most LAG powers of two below the
// largest score, so that the sum of the weights stays inside fp32.
constexpr int UP = 15, SPREAD = 8;
constexpr float LAG = 90.f;

template <int HD, bool Q, bool UNI>
__global__ void __launch_bounds__(32 * WARPS, HD <= 128 ? Tile<HD, Q>::CTAS : 1) k_paged_attn_mma(PagedAttnParams p, int least) {
  constexpr int KEYS = Tile<HD, Q>::KEYS, STAGES = Tile<HD, Q>::STAGES, ROW = Ring<HD, Q>::ROW, STAGE = Ring<HD, Q>::STAGE;
  constexpr int NG = KEYS / 8;                        // groups of 8 keys
  constexpr unsigned ALL = KEYS == 32 ? 0xffffffffu : (1u << KEYS % 32) - 1;
  constexpr int PIECES = ROW / 16, EPP = Q ? 16 : 8;  // 16-byte pieces of a row, elements of a piece
  constexpr int QR = HD / 16;                         // k16 steps of a score
  constexpr int VH = (PIECES + 7) / 8;                // pieces of a value row that one lane reads
  constexpr int NC = VH * EPP;                        // groups of 8 channels
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long red[WARPS];
  __shared__ int kept[LENS];
  __shared__ long long run_id[2 * WARPS];             // the groups of the warps' parts, -1: none
  __shared__ int run_end[WARPS], run_first[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j4 = lane & 3, n8 = lane >> 2;
  const int hd = p.c.hd, Hkv = p.c.Hkv, G = p.H / Hkv, n_ht = (G + GT - 1) / GT, segs = Hkv * n_ht;
  const int ps = p.c.page_size, row_bytes = hd * (Q ? 1 : 2), pieces = row_bytes / 16;
  const bool vec_o = !(((uintptr_t)p.o | (uintptr_t)(p.o_row * 2)) & 15) && hd % 8 == 0;
  const long long length = line_length(p, segs, KEYS, kept, red);
  const Lens lens{p, p.B <= LENS ? kept : nullptr};
  zero_rows(p, lens, 2);
  const int worker = blockIdx.x * WARPS + warp;
  const long long piece = piece_of(length, gridDim.x * WARPS, least);
  const long long w0 = worker * piece, w1 = w0 + piece < length ? w0 + piece : length;
  unsigned char* ring = smem + warp * Ring<HD, Q>::BYTES;
  const uint32_t ring_a = smem_addr(ring);
  // the pieces past the head's width hold zeros
  if (pieces < PIECES)
    for (int i = lane; i < Ring<HD, Q>::BYTES / 16; i += 32) reinterpret_cast<uint4*>(ring)[i] = make_uint4(0, 0, 0, 0);
  __syncwarp();
  if (lane < 2) run_id[2 * warp + lane] = -1;
  const Place start = w0 < w1 ? line_find(lens, segs, KEYS, w0) : Place{0, 0};

  // ---- loading: the tiles of w0 .. w1 - 1 one after another, whatever group they belong to,
  // STAGES - 1 ahead of the products.  Lane r holds the slot of key r of the tile to issue.
  // UNI: pages hold whole groups of 16 keys, so a group's rows lie one after another.
  int left = (int)(w1 - w0), ib = start.b, ilen = 0, int_ = 0, iseg = 0, it = 0, ig = 0, ist = 0;   // left: units of the line
  if (w0 < w1) {
    ilen = lens.keys(ib);
    int_ = (ilen + KEYS - 1) / KEYS;
    iseg = (int)(start.at / (int_ + START));
    it = (int)(start.at % (int_ + START)) - START;
    left += min(it, 0);
    it = max(it, 0);
    ig = iseg / n_ht;
  }
  const int* table = p.c.table + (long long)ib * p.c.max_pages;
  auto slot_of = [&]() -> long long {
    const int key = it * KEYS + lane;
    if (left <= 0 || lane >= KEYS || key >= ilen) return -1;   // (lengths are within the table)
    const int pi = page_index(p.c, key);
    const int page = __ldg(table + pi);
    if ((unsigned)page >= (unsigned)p.c.n_pages) {
      record_bad(p.c, p.st, 222, page);
      return -1;
    }
    return ((long long)page * Hkv + ig) * ps + (key - pi * ps);
  };
  long long slot_n = slot_of();
  int ke_r[STAGES], ve_r[STAGES];                     // e4m3: exponent bytes of the lane's key; [0]: of the tile in hand
  unsigned ok_r[STAGES];                              // keys that take part
#pragma unroll
  for (int i = 0; i < STAGES; ++i) ke_r[i] = ve_r[i] = 0, ok_r[i] = 0;
  auto issue = [&](int& ke, int& ve, unsigned& ok) {
    const long long slot = slot_n;
    ok = __ballot_sync(0xffffffffu, slot >= 0);
    if (left > 0) {
      const uint32_t ka = ring_a + ist * STAGE, va = ka + KEYS * ROW;
      const long long mine = slot * row_bytes;
      // each row's pieces by neighbouring lanes
      if (UNI && ok == ALL) {
        constexpr int RPI = 32 / PIECES;              // rows of one round
        const int r0 = lane / PIECES, c = lane % PIECES;
#pragma unroll
        for (int gr = 0; gr < KEYS; gr += 16) {
          const long long off = __shfl_sync(0xffffffffu, mine, gr) + r0 * row_bytes + c * 16;
          const char *kp = (const char*)p.c.k + off, *vp = (const char*)p.c.v + off;
          if (pieces == PIECES) {                     // (known strides)
#pragma unroll
            for (int i = 0; i < 16 / RPI; ++i) {
              const int r = gr + i * RPI + r0;
              cp16(ka + r * ROW + swz_k<PIECES>(r, c) * 16, kp + i * RPI * ROW);
              cp16(va + r * ROW + swz_v<PIECES>(r, c) * 16, vp + i * RPI * ROW);
            }
          } else if (c < pieces) {
#pragma unroll
            for (int i = 0; i < 16 / RPI; ++i) {
              const int r = gr + i * RPI + r0;
              cp16(ka + r * ROW + swz_k<PIECES>(r, c) * 16, kp + i * RPI * row_bytes);
              cp16(va + r * ROW + swz_v<PIECES>(r, c) * 16, vp + i * RPI * row_bytes);
            }
          }
        }
      } else {
#pragma unroll
        for (int i0 = 0; i0 < KEYS * PIECES; i0 += 32) {
          const int i = i0 + lane, r = i / PIECES, c = i % PIECES;
          const long long s = __shfl_sync(0xffffffffu, mine, r);
          if (c < pieces) {
            const long long off = s >= 0 ? s + c * 16 : 0;
            cp16_or_zero(ka + r * ROW + swz_k<PIECES>(r, c) * 16, (const char*)p.c.k + off, s >= 0);
            cp16_or_zero(va + r * ROW + swz_v<PIECES>(r, c) * 16, (const char*)p.c.v + off, s >= 0);
          }
        }
      }
      if (Q && slot >= 0) {
        ke = __ldg(p.c.ke + slot);
        ve = __ldg(p.c.ve + slot);
      }
      ist = ist + 1 == STAGES ? 0 : ist + 1;
      --left;
      if (++it == int_ && left > 0) {                 // the next group
        it = 0;
        left -= START;
        if (++iseg == segs) {
          iseg = 0;
          do ilen = lens.keys(++ib);
          while (ilen == 0 && ib + 1 < p.B);
          int_ = (ilen + KEYS - 1) / KEYS;
          table = p.c.table + (long long)ib * p.c.max_pages;
        }
        ig = iseg / n_ht;
      }
    }
    cp_commit();
    slot_n = slot_of();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) issue(ke_r[i], ve_r[i], ok_r[i]);

  Place at = start;
  int st = 0;
  for (long long x = w0; x < w1;) {
    // ---- one (sequence, head group): tiles t0 .. t1 - 1 of its nt
    const int b = at.b, nt = lens.tiles(b, KEYS), nu = lens.units(b, KEYS);
    if (at.at >= (long long)nu * segs) {
      at = Place{b + 1, 0};
      continue;
    }
    const int seg = (int)(at.at / nu), u0 = (int)(at.at % nu), u1 = nu - u0 < w1 - x ? nu : u0 + (int)(w1 - x);
    const int t0 = max(u0 - START, 0), t1 = max(u1 - START, 0);
    const long long begin = x - u0;                   // the group's first unit
    x += u1 - u0;
    at.at += u1 - u0;
    if (t0 == t1) continue;
    const int g = seg / n_ht, h0 = seg % n_ht * GT, nh = min(GT, G - h0);
    float m = -INFINITY, l = 0.f;                     // of head n8: reference, sum of this lane's keys
    float smax = -INFINITY;                           // e4m3: the largest score up to the last tile that was not close
    float acc[NC][4];                                 // [channel group]: rows n8 (upper words), n8 + 8 (lower)
    uint32_t qf[QR][2];                               // the query's fragments: row n8, columns of the two k8 halves
    int vexp = -128;                                  // e4m3: acc is in units of 2^(vexp - UP)
    float sl2;                                        // scores to base-2 logarithms (and the query's own scale)
    // the query
    {
      const bf16* q = (const bf16*)p.q + (long long)b * p.q_row + (long long)(g * G + h0 + n8) * hd;
      float qmax = 0.f;
      if (Q) {
        if (n8 < nh)
          for (int d = j4; d < hd; d += 4) qmax = fmaxf(qmax, finite_abs(to_f(q[d])));
        qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, 1));
        qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, 2));
      }
      // e4m3: the query becomes fp16 with its largest magnitude in [2^14, 2^15), which leaves
      // out only what is 2^39 smaller
      int qe = 0;
      if (Q && qmax > 0.f) {
        frexpf(qmax, &qe);
        qe = 15 - qe;
      }
      const float qs = Q ? ldexpf(1.f, min(qe, 126)) : 1.f;
      sl2 = p.scale * LOG2E / qs;
      // channel of (piece round i, k16 step u, half, pair): lane j4 of a row holds piece 4 i + j4
#pragma unroll
      for (int s = 0; s < QR; ++s)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int per = EPP / 4;                    // k16 steps of a round
          const int d = ((s / per) * 4 + j4) * EPP + (s % per) * 4 + hf * 2;
          float x = 0.f, y = 0.f;
          if (n8 < nh && d < hd) x = to_f(q[d]), y = to_f(q[d + 1]);
          if (Q) {
            const __half2 h = __floats2half2_rn(x * qs, y * qs);
            qf[s][hf] = *reinterpret_cast<const uint32_t*>(&h);
          } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
            qf[s][hf] = *reinterpret_cast<const uint32_t*>(&h);
          }
        }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;

    for (int t = t0; t < t1; ++t) {
        issue(ke_r[STAGES - 1], ve_r[STAGES - 1], ok_r[STAGES - 1]);
        cp_wait<STAGES - 1>();
        __syncwarp();
        const uint32_t ka = ring_a + st * STAGE, va = ka + KEYS * ROW;
        const unsigned ok = ok_r[0];
        st = st + 1 == STAGES ? 0 : st + 1;
        // scores of head n8, keys 8 g + 2 j4, + 1
        float sc[NG][4];
#pragma unroll
        for (int kg = 0; kg < NG; ++kg) {
          sc[kg][0] = sc[kg][1] = sc[kg][2] = sc[kg][3] = 0.f;
          const int r = kg * 8 + n8;
#pragma unroll
          for (int i = 0; i < (PIECES + 3) / 4; ++i) {
            const uint4 v = lds16(ka + r * ROW + swz_k<PIECES>(r, 4 * i + j4) * 16);
            if (!Q) {
              mma<Q>(sc[kg], qf[2 * i][0], 0u, qf[2 * i][1], 0u, v.x, v.y);
              mma<Q>(sc[kg], qf[2 * i + 1][0], 0u, qf[2 * i + 1][1], 0u, v.z, v.w);
            } else {
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int u = 0; u < 4; ++u)
                mma<Q>(sc[kg], qf[4 * i + u][0], 0u, qf[4 * i + u][1], 0u, e4m3x2_h2(w[u] & 0xffff), e4m3x2_h2(w[u] >> 16));
            }
          }
        }
        // e4m3: lane r turns its key's exponents into the factors of the score and of the weight
        float kf = 0.f, vf = 0.f;
        float drop = 0.f, lv = 0.f;
        bool close = true;                              // the exponents are within SPREAD below the largest before
        if (Q) {
          const bool mine = ok >> lane & 1;
          const int ve = mine ? ve_r[0] - 127 : -128;
          kf = exp_byte_scale(ke_r[0]);
          close = !__any_sync(0xffffffffu, mine && (unsigned)(vexp - ve) > (unsigned)SPREAD);
          if (!close) {
            const int top = max(vexp, (int)__reduce_max_sync(0xffffffffu, ve));
            drop = (float)(vexp - top);                 // by how much acc's unit grows
            vexp = top;
            lv = (float)(ve - top);
          }
          vf = mine ? pow2_down(ve - vexp + UP) : 0.f;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int kg = 0; kg < NG; ++kg)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            sc[kg][e] *= Q ? sl2 * __shfl_sync(0xffffffffu, kf, kg * 8 + 2 * j4 + e) : sl2;
            mx = fmaxf(mx, sc[kg][e]);
          }
        if (ok != ALL) {                                // the last tile, or a bad page
          mx = -INFINITY;
#pragma unroll
          for (int kg = 0; kg < NG; ++kg)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (!(ok >> (kg * 8 + 2 * j4 + e) & 1)) sc[kg][e] = -INFINITY;
              mx = fmaxf(mx, sc[kg][e]);
            }
        }
        // (a NaN score drops out of the maximum, and its weight makes the sums NaN)
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        float mn = fmaxf(m, mx);
        if (Q && !close) {
          smax = fmaxf(fmaxf(smax, m), mx);             // (m: of the tiles since)
          float mu = -INFINITY;
#pragma unroll
          for (int kg = 0; kg < NG; ++kg)
#pragma unroll
            for (int e = 0; e < 2; ++e) mu = fmaxf(mu, sc[kg][e] + __shfl_sync(0xffffffffu, lv, kg * 8 + 2 * j4 + e));
          mu = fmaxf(mu, __shfl_xor_sync(0xffffffffu, mu, 1));
          mu = fmaxf(mu, __shfl_xor_sync(0xffffffffu, mu, 2));
          mn = fmaxf(fmaxf(m + drop, mu), smax - LAG);
        }
        const float base = mn == -INFINITY ? 0.f : mn;
        const float corr = ex2(m - base);
        if (__any_sync(0xffffffffu, corr != 1.f) || (Q && !close)) {
          const float f = Q && !close ? ex2(m + drop - base) : corr;
          l *= corr;
#pragma unroll
          for (int i = 0; i < NC; ++i) acc[i][0] *= f, acc[i][1] *= f, acc[i][2] *= f, acc[i][3] *= f;
        }
        m = mn;
        uint32_t ph[NG], pl[NG];                        // weights of keys 8 g + 2 j4, + 1
#pragma unroll
        for (int kg = 0; kg < NG; ++kg) {
          float w[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            w[e] = ex2(sc[kg][e] - base);
            l += w[e];                                  // this lane's keys; the 4 lanes are summed at the end
            if (Q) w[e] *= __shfl_sync(0xffffffffu, vf, kg * 8 + 2 * j4 + e);
          }
          split2<Q>(w[0], w[1], ph[kg], pl[kg]);
        }
        // values: lane holds keys 2 j4, + 1 of two groups, pieces n8 (+ 8) of their rows
#pragma unroll
        for (int kk = 0; kk < NG; kk += 2)
#pragma unroll
          for (int h = 0; h < VH; ++h) {
            // (e4m3 rows of 64 have 4 pieces: the upper lanes' channels do not exist)
            const int cc = PIECES % 8 ? (h * 8 + n8) % PIECES : h * 8 + n8, r = kk * 8 + 2 * j4;
            uint32_t x[4][4];                           // keys r, r + 1, r + 8, r + 9
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int ri = r + (i & 1) + 8 * (i >> 1);
              const uint4 v = lds16(va + ri * ROW + swz_v<PIECES>(ri, cc) * 16);
              x[i][0] = v.x, x[i][1] = v.y, x[i][2] = v.z, x[i][3] = v.w;
            }
            auto add = [&](float(&o)[4], uint32_t b0, uint32_t b1) {
              mma<Q>(o, ph[kk], pl[kk], ph[kk + 1], pl[kk + 1], b0, b1);
            };
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              if (!Q) {                                 // channels 2 u, 2 u + 1 of the piece
                add(acc[h * 8 + 2 * u], __byte_perm(x[0][u], x[1][u], 0x5410), __byte_perm(x[2][u], x[3][u], 0x5410));
                add(acc[h * 8 + 2 * u + 1], __byte_perm(x[0][u], x[1][u], 0x7632), __byte_perm(x[2][u], x[3][u], 0x7632));
              } else {                                  // channels 4 u .. 4 u + 3
                const uint32_t a0 = __byte_perm(x[0][u], x[1][u], 0x5140), a1 = __byte_perm(x[0][u], x[1][u], 0x7362);
                const uint32_t b0 = __byte_perm(x[2][u], x[3][u], 0x5140), b1 = __byte_perm(x[2][u], x[3][u], 0x7362);
                float(*o)[4] = acc + h * EPP + EPP / 4 * u;
                add(o[0], e4m3x2_h2(a0 & 0xffff), e4m3x2_h2(b0 & 0xffff));
                add(o[1], e4m3x2_h2(a0 >> 16), e4m3x2_h2(b0 >> 16));
                add(o[2 % (EPP / 4)], e4m3x2_h2(a1 & 0xffff), e4m3x2_h2(b1 & 0xffff));
                add(o[3 % (EPP / 4)], e4m3x2_h2(a1 >> 16), e4m3x2_h2(b1 >> 16));
              }
            }
          }
        __syncwarp();                                   // the stage is free to be written
#pragma unroll
        for (int i = 0; i + 1 < STAGES; ++i) ke_r[i] = ke_r[i + 1], ve_r[i] = ve_r[i + 1], ok_r[i] = ok_r[i + 1];
    }
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    const float back = Q ? ldexpf(1.f, vexp) : 1.f, down = Q ? pow2_down(-UP) : 1.f;
    // column n of channel group c is element c % EPP of the piece c / EPP * 8 + n, and this
    // lane has columns 2 j4, + 1 of row n8: whole pieces
    if (t0 == 0 && t1 == nt) {
      const float inv = l != 0.f ? 1.f / l : 0.f;
      bf16* o = (bf16*)p.o + (long long)b * p.o_row + (long long)(g * G + h0 + n8) * hd;
      if (n8 < nh)
#pragma unroll
        for (int h = 0; h < VH; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int ch = (h * 8 + 2 * j4 + e) * EPP;
            if (ch >= hd) continue;
            bf16 y[EPP];
#pragma unroll
            for (int i = 0; i < EPP; ++i) y[i] = from_f<bf16>(both_words(acc[h * EPP + i][e], acc[h * EPP + i][2 + e]) * down * inv * back);
#pragma unroll
            for (int i = 0; i < EPP; i += 8) {
              uint32_t w[4];
#pragma unroll
              for (int u = 0; u < 4; ++u)
                w[u] = (uint32_t)__bfloat16_as_ushort(y[i + 2 * u]) | (uint32_t)__bfloat16_as_ushort(y[i + 2 * u + 1]) << 16;
              if (vec_o) *reinterpret_cast<uint4*>(o + ch + i) = make_uint4(w[0], w[1], w[2], w[3]);
              else
#pragma unroll
                for (int u = 0; u < 8; ++u) o[ch + i + u] = y[i + u];
            }
          }
    } else {
      const int which = t0 == 0;
      if (lane == 0) {
        run_id[2 * warp + which] = (long long)b * segs + seg;
        if (which == 0) run_end[warp] = t1 == nt, run_first[warp] = (int)((begin + START) / (piece * WARPS));
      }
      float* ml = part_ml(p, gridDim.x + worker, which);
      float* po = part_o(p, gridDim.x + worker, which) + n8 * hd;
      if (j4 == 0) {
        ml[n8 * 2] = m;
        ml[n8 * 2 + 1] = l;
      }
      if (n8 < nh)
#pragma unroll
        for (int h = 0; h < VH; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int ch = (h * 8 + 2 * j4 + e) * EPP;
            if (ch >= hd) continue;
#pragma unroll
            for (int i = 0; i < EPP; i += 4) {
              float4 y;
              y.x = both_words(acc[h * EPP + i][e], acc[h * EPP + i][2 + e]) * down * back;
              y.y = both_words(acc[h * EPP + i + 1][e], acc[h * EPP + i + 1][2 + e]) * down * back;
              y.z = both_words(acc[h * EPP + i + 2][e], acc[h * EPP + i + 2][2 + e]) * down * back;
              y.w = both_words(acc[h * EPP + i + 3][e], acc[h * EPP + i + 3][2 + e]) * down * back;
              *reinterpret_cast<float4*>(po + ch + i) = y;
            }
          }
    }
  }
  // ---- the warps' parts of one group, neighbours in the order (entered, left) of the warps,
  // become the output if the group lies within the CTA, else the CTA's part
  __syncthreads();
  Desc joins{-1, 0, 0, 0};
  const int first = gridDim.x + blockIdx.x * WARPS;   // of the warps' parts
  int item = 0;
  for (int i = 0; i < 2 * WARPS;) {
    const long long id = run_id[i];
    if (id < 0) {
      ++i;
      continue;
    }
    int last = i, j = i + 1;
    for (; j < 2 * WARPS && (run_id[j] < 0 || run_id[j] == id); ++j)
      if (run_id[j] == id) last = j;
    const bool begun = i & 1, ended = !(last & 1) && run_end[last >> 1];   // within this CTA
    const int b = (int)(id / segs), seg = (int)(id % segs), g = seg / n_ht, h0 = seg % n_ht * GT, nh = min(GT, G - h0);
    if (!begun && ended) joins = Desc{b, seg, run_first[last >> 1], 0};
    for (int h = 0; h < nh; ++h) {
      if ((item++ & (WARPS - 1)) != warp) continue;   // a warp per (group, head)
      const int part = lane < 2 * WARPS && lane >= i && lane <= last && run_id[lane] == id ? lane : -1;
      const float2 ml = part >= 0 ? *reinterpret_cast<const float2*>(part_ml(p, first + (part >> 1), part & 1) + h * 2)
                                  : make_float2(-INFINITY, 0.f);
      const unsigned parts = __ballot_sync(0xffffffffu, part >= 0);
      float4 v[2 * WARPS];
      auto load = [&](int ch) {                       // (the first before m and l are in)
#pragma unroll
        for (int k = 0; k < 2 * WARPS; ++k)
          if ((parts >> k & 1) && ch < hd)
            v[k] = *reinterpret_cast<const float4*>(part_o(p, first + (k >> 1), k & 1) + h * hd + ch);
      };
      load(4 * lane);
      const float M = warp_max(ml.x), base = M == -INFINITY ? 0.f : M;
      const float w = ex2(ml.x - base), L = warp_sum(w * ml.y), inv = begun && ended ? (L != 0.f ? 1.f / L : 0.f) : 1.f;
      for (int ch = 4 * lane; ch < (hd + 127) / 128 * 128; ch += 128) {
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (ch >= 128) load(ch);
#pragma unroll
        for (int k = 0; k < 2 * WARPS; ++k) {
          const float wk = __shfl_sync(0xffffffffu, w, k);
          if (!(parts >> k & 1)) continue;
          o.x = fmaf(wk, v[k].x, o.x), o.y = fmaf(wk, v[k].y, o.y);
          o.z = fmaf(wk, v[k].z, o.z), o.w = fmaf(wk, v[k].w, o.w);
        }
        if (ch >= hd) continue;
        if (begun && ended) {
          bf16* y = (bf16*)p.o + (long long)b * p.o_row + (long long)(g * G + h0 + h) * hd + ch;
          y[0] = from_f<bf16>(o.x * inv), y[1] = from_f<bf16>(o.y * inv);
          y[2] = from_f<bf16>(o.z * inv), y[3] = from_f<bf16>(o.w * inv);
        } else {
          *reinterpret_cast<float4*>(part_o(p, blockIdx.x, begun) + h * hd + ch) = o;
        }
      }
      if (lane == 0 && !(begun && ended))
        *reinterpret_cast<float2*>(part_ml(p, blockIdx.x, begun) + h * 2) = make_float2(M, L);
    }
    i = j;
  }
  if (threadIdx.x == 0) desc_of(p)[blockIdx.x] = joins;
  let_join_start();
}

// ------------------------------------------------------------------------------------------
// plain kernel: any width and page size, fp32 or bf16, both storage forms; a worker is a CTA
// ------------------------------------------------------------------------------------------
// 32-key tiles of K and V in fp32 in shared memory, NH (1, 2, 4 or 8) query heads at a time.
// Scores: a lane per key, each warp a quarter of the channels for all heads, so a K element
// serves NH products; values: a thread per channel, so a V element serves NH.  An fp32 cache is
// copied by cp.async one tile ahead; the other forms are widened on the way.
namespace {
constexpr int TK = 32;
struct PlainSm {
  __host__ __device__ static int stride(int hd) { return (hd + 3) / 4 * 4 + 4; }   // 4 mod 32 words: no conflicts
  __host__ __device__ static size_t tile(int hd) { return 2 * (size_t)TK * stride(hd); }   // floats: K then V
  __host__ __device__ static size_t bytes(int hd, int nh, int buffers) {
    return buffers * TK * 8 + sizeof(float) * ((size_t)nh * ((hd + 3) / 4 * 4) + buffers * tile(hd) + WARPS * nh * TK + TK * nh + GT);
  }
};
template <int NH> struct Heads { float x[NH]; };
template <int NH> __device__ __forceinline__ Heads<NH> heads_at(const float* p) {   // aligned to NH floats
  Heads<NH> r;
  if (NH == 8) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    r.x[0] = a.x; r.x[1 % NH] = a.y; r.x[2 % NH] = a.z; r.x[3 % NH] = a.w;
    r.x[4 % NH] = b.x; r.x[5 % NH] = b.y; r.x[6 % NH] = b.z; r.x[7 % NH] = b.w;
  } else if (NH == 4) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    r.x[0] = a.x; r.x[1 % NH] = a.y; r.x[2 % NH] = a.z; r.x[3 % NH] = a.w;
  } else if (NH == 2) {
    const float2 a = *reinterpret_cast<const float2*>(p);
    r.x[0] = a.x; r.x[1 % NH] = a.y;
  } else {
    r.x[0] = *p;
  }
  return r;
}
}  // namespace

template <typename T, bool Q, int NH, bool VEC>
__global__ void __launch_bounds__(128, 5) k_paged_attn_simt(PagedAttnParams p, int least) {
  constexpr bool AHEAD = VEC && !Q && sizeof(T) == 4;   // copied as it is, a tile ahead
  constexpr int BUF = AHEAD ? 2 : 1, HW = (NH + WARPS - 1) / WARPS;   // heads of a warp
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long red[WARPS];
  __shared__ int kept[LENS];
  const int hd = p.c.hd, hd4 = (hd + 3) / 4 * 4, Hkv = p.c.Hkv, G = p.H / Hkv, n_ht = (G + GT - 1) / GT, segs = Hkv * n_ht;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ld = PlainSm::stride(hd);
  long long* slot_s = reinterpret_cast<long long*>(smem);       // [BUF][TK] slot of each key, -1: takes no part
  float* qs = reinterpret_cast<float*>(slot_s + BUF * TK);      // [hd4][NH]
  float* kv = qs + NH * hd4;                                    // [BUF][2][TK][ld]
  float* part = kv + BUF * 2 * TK * ld;                         // [WARPS][NH][TK]
  float* ws = part + WARPS * NH * TK;                           // [TK][NH]
  float* corr_s = ws + TK * NH;                                 // [GT]
  const long long length = line_length(p, segs, TK, kept, red);
  const Lens lens{p, p.B <= LENS ? kept : nullptr};
  zero_rows(p, lens, (int)sizeof(T));
  const long long piece = piece_of(length, gridDim.x, least);
  const long long w0 = blockIdx.x * piece, w1 = w0 + piece < length ? w0 + piece : length;
  // channels past the width (up to a multiple of 4) are zeros in q and K
  for (int i = tid; i < NH * hd4; i += 128) qs[i] = 0.f;
  for (int i = tid; i < BUF * 2 * TK * ld; i += 128) kv[i] = 0.f;
  Desc joins{-1, 0, 0, 0};
  Place at = w0 < w1 ? line_find(lens, segs, TK, w0) : Place{0, 0};
  for (long long x = w0; x < w1;) {
    const int b = at.b, len = lens.keys(b), nt = lens.tiles(b, TK), nu = lens.units(b, TK);
    if (at.at >= (long long)nu * segs) {
      at = Place{b + 1, 0};
      continue;
    }
    const int seg = (int)(at.at / nu), u0 = (int)(at.at % nu), u1 = nu - u0 < w1 - x ? nu : u0 + (int)(w1 - x);
    const int t0 = max(u0 - START, 0), t1 = max(u1 - START, 0);
    const long long begin = x - u0;                   // the group's first unit
    x += u1 - u0;
    at.at += u1 - u0;
    if (t0 == t1) continue;
    const int g = seg / n_ht, h0 = seg % n_ht * GT, nh = min(GT, G - h0);   // nh <= NH
    const bool whole = t0 == 0 && t1 == nt;
    const int which = t0 == 0;
    if (t0 > 0 && t1 == nt) joins = Desc{b, seg, (int)((begin + START) / piece), 0};
    const float sl2 = p.scale * LOG2E;
    __syncthreads();
    for (int i = tid; i < nh * hd; i += 128) {
      const int h = i / hd, d = i - h * hd;
      qs[d * NH + h] = to_f(((const T*)p.q)[(long long)b * p.q_row + (long long)(g * G + h0) * hd + i]) * sl2;
    }
    if (nh < NH)
      for (int i = tid; i < (NH - nh) * hd; i += 128) qs[i / (NH - nh) * NH + nh + i % (NH - nh)] = 0.f;
    float m[HW], l[HW], acc[NH][2];                           // heads warp + 4 u; channels tid and tid + 128
#pragma unroll
    for (int u = 0; u < HW; ++u) m[u] = -INFINITY, l[u] = 0.f;
#pragma unroll
    for (int h = 0; h < NH; ++h) acc[h][0] = acc[h][1] = 0.f;
    auto find_slots = [&](int t) {
      if (tid < TK) {
        const int key = t * TK + tid;
        long long s = -1;
        if (key < len) {
          const int page = page_of(p.c, b, key, p.st, 222);
          if (page >= 0) s = ((long long)page * Hkv + g) * p.c.page_size + (key - page_index(p.c, key) * p.c.page_size);
        }
        slot_s[(t & (BUF - 1)) * TK + tid] = s;
      }
    };
    // masked rows hold zeros: 0 * v is 0 whatever the slot holds
    auto copy = [&](int t) {
      const long long* slots = slot_s + (t & (BUF - 1)) * TK;
      float *k = kv + (t & (BUF - 1)) * 2 * TK * ld, *v = k + TK * ld;
      if (VEC) {
        const int q4 = hd / 4;
        for (int i = tid; i < TK * q4; i += 128) {
          const int r = i / q4, c = i - r * q4;
          const long long s = slots[r];
          if (AHEAD) {
            const long long off = s >= 0 ? s * q4 + c : 0;
            cp16_or_zero(smem_addr(k + r * ld + 4 * c), (const float4*)p.c.k + off, s >= 0);
            cp16_or_zero(smem_addr(v + r * ld + 4 * c), (const float4*)p.c.v + off, s >= 0);
            continue;
          }
          float4 kx = make_float4(0.f, 0.f, 0.f, 0.f), vx = kx;
          if (s >= 0) {
            if (Q) {
              const uint32_t kw = __ldg((const uint32_t*)p.c.k + s * q4 + c), vw = __ldg((const uint32_t*)p.c.v + s * q4 + c);
              const float ks = exp_byte_scale(p.c.ke[s]), vs = exp_byte_scale(p.c.ve[s]);
              kx = make_float4(e4m3_f(kw & 255) * ks, e4m3_f(kw >> 8 & 255) * ks, e4m3_f(kw >> 16 & 255) * ks, e4m3_f(kw >> 24) * ks);
              vx = make_float4(e4m3_f(vw & 255) * vs, e4m3_f(vw >> 8 & 255) * vs, e4m3_f(vw >> 16 & 255) * vs, e4m3_f(vw >> 24) * vs);
            } else {
              const uint2 kw = __ldg((const uint2*)p.c.k + s * q4 + c), vw = __ldg((const uint2*)p.c.v + s * q4 + c);
              kx = make_float4(__uint_as_float(kw.x << 16), __uint_as_float(kw.x & 0xffff0000u), __uint_as_float(kw.y << 16),
                               __uint_as_float(kw.y & 0xffff0000u));
              vx = make_float4(__uint_as_float(vw.x << 16), __uint_as_float(vw.x & 0xffff0000u), __uint_as_float(vw.y << 16),
                               __uint_as_float(vw.y & 0xffff0000u));
            }
          }
          *reinterpret_cast<float4*>(k + r * ld + 4 * c) = kx;
          *reinterpret_cast<float4*>(v + r * ld + 4 * c) = vx;
        }
      } else {
        for (int i = tid; i < TK * hd; i += 128) {
          const int r = i / hd, d = i - r * hd;
          const long long s = slots[r];
          float kx = 0.f, vx = 0.f;
          if (s >= 0) {
            if (Q) {
              kx = e4m3_f(((const uint8_t*)p.c.k)[s * hd + d]) * exp_byte_scale(p.c.ke[s]);
              vx = e4m3_f(((const uint8_t*)p.c.v)[s * hd + d]) * exp_byte_scale(p.c.ve[s]);
            } else {
              kx = to_f(((const T*)p.c.k)[s * hd + d]);
              vx = to_f(((const T*)p.c.v)[s * hd + d]);
            }
          }
          k[r * ld + d] = kx;
          v[r * ld + d] = vx;
        }
      }
      if (AHEAD) cp_commit();
    };
    if (AHEAD) {
      find_slots(t0);
      __syncthreads();
      copy(t0);
    }
    for (int t = t0; t < t1; ++t) {
      if (!AHEAD) __syncthreads();                            // the tile before is done with
      const int tn = AHEAD ? t + 1 : t;
      if (tn < t1) find_slots(tn);
      __syncthreads();
      if (tn < t1) copy(tn);
      else if (AHEAD) cp_commit();
      if (AHEAD) cp_wait<1>();
      __syncthreads();
      const float *k = kv + (t & (BUF - 1)) * 2 * TK * ld, *v = k + TK * ld;
      {
        const int n4 = hd4 / 4, c0 = n4 * warp / WARPS, c1 = n4 * (warp + 1) / WARPS;
        float s[NH] = {};
#pragma unroll 2
        for (int c = c0; c < c1; ++c) {
          const float4 k4 = *reinterpret_cast<const float4*>(k + lane * ld + 4 * c);
          const float kk[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const Heads<NH> q = heads_at<NH>(qs + (4 * c + e) * NH);
#pragma unroll
            for (int h = 0; h < NH; ++h) s[h] = fmaf(q.x[h], kk[e], s[h]);
          }
        }
#pragma unroll
        for (int h = 0; h < NH; ++h) part[(warp * NH + h) * TK + lane] = s[h];
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < HW; ++u) {
        const int h = warp + WARPS * u;
        if (h < NH) {
          float s = 0.f;
#pragma unroll
          for (int w = 0; w < WARPS; ++w) s += part[(w * NH + h) * TK + lane];
          if (slot_s[(t & (BUF - 1)) * TK + lane] < 0) s = -INFINITY;
          const float mx = fmaxf(m[u], warp_max(s));
          const float base = mx == -INFINITY ? 0.f : mx;
          const float e = exp2f(s - base), c = exp2f(m[u] - base);
          m[u] = mx;
          l[u] = l[u] * c + warp_sum(e);
          ws[lane * NH + h] = e;
          if (lane == 0) corr_s[h] = c;
        }
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int d = tid + 128 * u;
        if (d < hd) {
#pragma unroll
          for (int h = 0; h < NH; ++h) acc[h][u] *= corr_s[h];
#pragma unroll 8
          for (int r = 0; r < TK; ++r) {
            const float vx = v[r * ld + d];
            const Heads<NH> w = heads_at<NH>(ws + r * NH);
#pragma unroll
            for (int h = 0; h < NH; ++h) acc[h][u] = fmaf(w.x[h], vx, acc[h][u]);
          }
        }
      }
    }
    if (AHEAD) cp_wait<0>();
    __syncthreads();
    if (lane == 0) {
#pragma unroll
      for (int u = 0; u < HW; ++u) {
        const int h = warp + WARPS * u;
        if (h < NH) {
          corr_s[h] = l[u];
          if (!whole && h < nh) {
            float* ml = part_ml(p, blockIdx.x, which);
            ml[h * 2] = m[u];
            ml[h * 2 + 1] = l[u];
          }
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int d = tid + 128 * u;
      if (d >= hd) continue;
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        if (h >= nh) continue;
        if (whole)
          ((T*)p.o)[(long long)b * p.o_row + (long long)(g * G + h0 + h) * hd + d] =
              from_f<T>(corr_s[h] != 0.f ? acc[h][u] / corr_s[h] : 0.f);
        else
          part_o(p, blockIdx.x, which)[h * hd + d] = acc[h][u];
      }
    }
  }
  if (tid == 0) desc_of(p)[blockIdx.x] = joins;
  let_join_start();
}

// ------------------------------------------------------------------------------------------
// join: the parts of the group that CTA i finished
// ------------------------------------------------------------------------------------------
// CTA (i, head): 4 warps take slices of the parts, a lane four channels (of each 128).
template <typename T>
__global__ void __launch_bounds__(128) k_paged_attn_join(PagedAttnParams p) {
  extern __shared__ float wj[];                       // [parts] 2^(m - M)
  __shared__ float red[WARPS];
  __shared__ __align__(16) float4 sum[WARPS][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Desc d = desc_of(p)[blockIdx.x];
  if (d.b < 0) return;
  const int hd = p.c.hd, G = p.H / p.c.Hkv, n_ht = (G + GT - 1) / GT, h = blockIdx.y;
  const int g = d.seg / n_ht, h0 = d.seg % n_ht * GT, n = (int)blockIdx.x - d.first + 1;
  if (h >= min(GT, G - h0)) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // part 1 of the first CTA, part 0 of the others
  const bool by4 = hd % 4 == 0;
  float4 ahead[8];                                    // a warp's first parts, loaded before their weights are known
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int s = warp + i * WARPS;
    ahead[i] = by4 && s < n && 4 * lane < hd
                   ? *reinterpret_cast<const float4*>(part_o(p, d.first + s, s == 0) + h * hd + 4 * lane)
                   : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const float2 none = make_float2(-INFINITY, 0.f);
  const float2 ml0 = tid < n ? *reinterpret_cast<const float2*>(part_ml(p, d.first + tid, tid == 0) + h * 2) : none;
  float M = ml0.x, L = 0.f;
  for (int s = tid + 128; s < n; s += 128) M = fmaxf(M, part_ml(p, d.first + s, 0)[h * 2]);
  M = warp_max(M);
  if (lane == 0) red[warp] = M;
  __syncthreads();
  M = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float base = M == -INFINITY ? 0.f : M;
  for (int s = tid; s < n; s += 128) {
    const float2 ml = s == tid ? ml0 : *reinterpret_cast<const float2*>(part_ml(p, d.first + s, 0) + h * 2);
    const float w = exp2f(ml.x - base);
    wj[s] = w;
    L += w * ml.y;
  }
  __syncthreads();
  L = block_sum(L, red);
  const float inv = L != 0.f ? 1.f / L : 0.f;
  T* o = (T*)p.o + (long long)d.b * p.o_row + (long long)(g * G + h0 + h) * hd;
  if (by4) {
    for (int ch0 = 0; ch0 < hd; ch0 += 128) {
      const int ch = ch0 + 4 * lane;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      if (ch < hd) {
        int s = warp;
        if (ch0 == 0)
#pragma unroll
          for (int i = 0; i < 8; ++i, s += WARPS) {
            const float w = s < n ? wj[s] : 0.f;
            a.x = fmaf(w, ahead[i].x, a.x); a.y = fmaf(w, ahead[i].y, a.y);
            a.z = fmaf(w, ahead[i].z, a.z); a.w = fmaf(w, ahead[i].w, a.w);
          }
#pragma unroll 8
        for (; s < n; s += WARPS) {
          const float4 x = *reinterpret_cast<const float4*>(part_o(p, d.first + s, s == 0) + h * hd + ch);
          const float w = wj[s];
          a.x = fmaf(w, x.x, a.x); a.y = fmaf(w, x.y, a.y); a.z = fmaf(w, x.z, a.z); a.w = fmaf(w, x.w, a.w);
        }
      }
      sum[warp][lane] = a;
      __syncthreads();
      if (ch0 + tid < hd) {
        const float* f = reinterpret_cast<const float*>(&sum[0][0]);
        o[ch0 + tid] = from_f<T>(((f[tid] + f[128 + tid]) + (f[256 + tid] + f[384 + tid])) * inv);
      }
      __syncthreads();
    }
  } else {
    for (int ch = tid; ch < hd; ch += 128) {
      float a = 0.f;
      for (int s = 0; s < n; ++s) a = fmaf(wj[s], part_o(p, d.first + s, s == 0)[h * hd + ch], a);
      o[ch] = from_f<T>(a * inv);
    }
  }
}

// ------------------------------------------------------------------------------------------
// launch
// ------------------------------------------------------------------------------------------
namespace {
// 16-byte copies need rows and bases on 16 bytes
bool mma_takes(int dtype, const PagedView& c) {
  const int rb = c.hd * (c.e4m3 ? 1 : 2);
  return dtype == 1 && c.hd % 8 == 0 && rb % 16 == 0 && !(((uintptr_t)c.k | (uintptr_t)c.v) & 15);
}
// Above 128 channels an SM holds one CTA, and the same grid runs in two (bf16) or three waves.  A grid
// of one wave takes, us at 256 channels, 16 heads on 4: 32 sequences of 4097 to 8191 keys in bf16 160
// (170), in e4m3 150 (166); 64 of 1 to 4224 76 (70), 57 (76); 4 of 37 29 (22), 27 (22): less for long
// lines, more for short ones.
int ctas_mma(bool e4m3) { return device_sm_count() * (e4m3 ? Tile<128, true>::CTAS : Tile<128, false>::CTAS); }
constexpr int SIMT_CTAS = 5;   // on an SM at most (an fp32 tile of 128 channels, twice, is 68 KB: three)
int ctas_simt(int smem) { return device_sm_count() * std::max(1, std::min(SIMT_CTAS, 227 * 1024 / (smem + 4096))); }
// descriptors, then the parts of `ctas` CTAs and, on tensor cores, of their warps
size_t scratch_bytes(int ctas, int parts, int hd) {
  return (size_t)ctas * sizeof(Desc) + (size_t)parts * 2 * GT * (hd + 2) * sizeof(float);
}

template <typename T> int launch_join(const PagedAttnParams& p, int ctas, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, (unsigned)std::min(GT, p.H / p.c.Hkv));
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = (size_t)ctas * sizeof(float);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // launched while the workers finish
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, k_paged_attn_join<T>, p) != cudaSuccess) return -1;
  note_launch();
  return 0;
}
}  // namespace

// The same for every batch and head count: the parts belong to the CTAs.
size_t paged_attn_scratch(const PagedView& c) {
  const int n = ctas_mma(c.e4m3);
  return std::max(scratch_bytes(n, n * (1 + WARPS), c.hd), scratch_bytes(ctas_simt(0), ctas_simt(0), c.hd));
}

int launch_paged_attn(int dtype, const PagedAttnParams& p0, cudaStream_t s) {
  PagedAttnParams p = p0;
  const bool tc = mma_takes(dtype, p.c);
  const int eb = p.c.e4m3 ? 1 : dtype == 0 ? 4 : 2, G = p.H / p.c.Hkv;
  const bool vec = p.c.hd % 4 == 0 && !(((uintptr_t)p.c.k | (uintptr_t)p.c.v) & (4 * eb - 1));
  const int nh = G >= 5 ? 8 : G >= 3 ? 4 : G, buffers = vec && dtype == 0 && !p.c.e4m3 ? 2 : 1;
  const int simt_smem = (int)PlainSm::bytes(p.c.hd, nh, buffers), ctas = tc ? ctas_mma(p.c.e4m3) : ctas_simt(simt_smem);
  p.part_ml = reinterpret_cast<float*>((char*)p.scratch + (size_t)ctas * sizeof(Desc));
  p.part_o = p.part_ml + (size_t)(tc ? ctas * (1 + WARPS) : ctas) * 2 * GT * 2;
  if (tc) {
#define RDT_MMA(HD, QQ)                                                                                     \
  do {                                                                                                      \
    constexpr int smem = WARPS * Ring<HD, QQ>::BYTES;                                                       \
    auto kernel = p.c.page_size % 16 ? k_paged_attn_mma<HD, QQ, false> : k_paged_attn_mma<HD, QQ, true>;    \
    if (!ensure_smem_limit((const void*)kernel, smem)) return -1;                                           \
    kernel<<<ctas, 32 * WARPS, smem, s>>>(p, 4);                                                              \
  } while (0)
    if (p.c.e4m3) {
      if (p.c.hd <= 64) RDT_MMA(64, true);
      else if (p.c.hd <= 128) RDT_MMA(128, true);
      else RDT_MMA(256, true);
    } else {
      if (p.c.hd <= 64) RDT_MMA(64, false);
      else if (p.c.hd <= 128) RDT_MMA(128, false);
      else RDT_MMA(256, false);
    }
#undef RDT_MMA
    note_launch();
    return launch_join<bf16>(p, ctas, s);
  }
  const int most = (int)PlainSm::bytes(256, 8, 2);
  void (*kernel)(PagedAttnParams, int) = nullptr;
#define RDT_SIMT(TT, QQ, NN) kernel = vec ? k_paged_attn_simt<TT, QQ, NN, true> : k_paged_attn_simt<TT, QQ, NN, false>
#define RDT_SIMT_H(TT, QQ)              \
  do {                                  \
    if (nh == 1) RDT_SIMT(TT, QQ, 1);   \
    else if (nh == 2) RDT_SIMT(TT, QQ, 2); \
    else if (nh == 4) RDT_SIMT(TT, QQ, 4); \
    else RDT_SIMT(TT, QQ, 8);           \
  } while (0)
  if (dtype == 0) {
    if (p.c.e4m3) RDT_SIMT_H(float, true);
    else RDT_SIMT_H(float, false);
  } else {
    if (p.c.e4m3) RDT_SIMT_H(bf16, true);
    else RDT_SIMT_H(bf16, false);
  }
#undef RDT_SIMT_H
#undef RDT_SIMT
  if (!ensure_smem_limit((const void*)kernel, most)) return -1;
  kernel<<<ctas, 128, simt_smem, s>>>(p, 3);
  note_launch();
  return dtype == 0 ? launch_join<float>(p, ctas, s) : launch_join<bf16>(p, ctas, s);
}

}  // namespace rdt
