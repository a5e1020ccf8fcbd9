// Writing the paged key / value cache and reading it back.
//
// write: row i = b * seq + t of k and v goes to slot pos % page_size of page
//   table[b][pos / page_size], every kv head as one row of head_dim values, in the model dtype
//   or as e4m3 with one exponent byte (paged.cuh).  pos < 0: a padding row, nothing written.
// read: positions 0 .. lens[b] - 1 of every sequence, contiguous, in the model dtype; a position
//   whose page is out of range stays as it was, or (for a caller that reads all rows) becomes zeros.
// Both move each byte once, so they are HBM-bound: a lane moves 16 bytes of the wider side at a
// time, and a thread has several rows of K and V in flight.  Widths or addresses that 16-byte
// pieces do not divide go value by value.  Measured on one B200: 16,384 rows of 8 heads of 128
// quantised in 23 us (4.4 TB/s; issue: conversion, maxima, addresses), copied in 20.5 (6.5 TB/s); 64
// sequences of 37 to 4224 positions read back from e4m3 in 140 us (6.0 TB/s, 91% of the copy rate).
#include "paged.cuh"

#include <algorithm>

namespace rdt {

namespace {
template <typename T> struct Vec { static constexpr int N = 16 / (int)sizeof(T); };   // values of a 16-byte piece
template <typename T> __device__ __forceinline__ void unpack(const uint4& w, float (&x)[Vec<T>::N]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (sizeof(T) == 4) {
      x[i] = __uint_as_float(u[i]);
    } else {
      x[(2 * i) % Vec<T>::N] = __uint_as_float(u[i] << 16);
      x[(2 * i + 1) % Vec<T>::N] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
}
template <typename T> __device__ __forceinline__ uint4 pack(const float (&x)[Vec<T>::N]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (sizeof(T) == 4) {
      u[i] = __float_as_uint(x[i]);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[(2 * i) % Vec<T>::N], x[(2 * i + 1) % Vec<T>::N]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}
constexpr int NT = 128;
__device__ __forceinline__ int slot_of(const PagedView& c, int pos) { return pos - page_index(c, pos) * c.page_size; }
}  // namespace

// One warp per (row, kv head): K, then V, value by value.
template <typename T, bool Q>
__global__ void __launch_bounds__(NT) k_paged_write(PagedWriteParams p) {
  const long long wid = (long long)blockIdx.x * (NT / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, Hkv = p.c.Hkv, hd = p.c.hd;
  if (wid >= (long long)p.n_rows * Hkv) return;
  const int row = (int)(wid / Hkv), g = (int)(wid % Hkv);
  const int pos = p.pos[row];
  if (pos < 0) return;
  const int page = page_of(p.c, p.seq == 1 ? row : row / p.seq, pos, p.st, 201);
  if (page < 0) return;
  const long long slot = ((long long)page * Hkv + g) * p.c.page_size + slot_of(p.c, pos);
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const T* src = (const T*)(kv ? p.v : p.k) + (long long)row * p.ld + (long long)g * hd;
    if (!Q) {
      T* dst = (T*)(kv ? p.c.v : p.c.k) + slot * hd;
      for (int d = lane; d < hd; d += 32) dst[d] = src[d];
    } else {
      float a = 0.f;
      for (int d = lane; d < hd; d += 32) a = fmaxf(a, finite_abs(to_f(src[d])));
      const int E = row_exponent(warp_max(a));
      const float inv = pow2_neg(E);
      uint8_t* dst = (uint8_t*)(kv ? p.c.v : p.c.k) + slot * hd;
      for (int d = lane; d < hd; d += 32) dst[d] = to_e4m3(to_f(src[d]), inv);
      if (lane == 0) (kv ? p.c.ve : p.c.ke)[slot] = (uint8_t)(E + 127);
    }
  }
}

// GL lanes (a power of two with GL pieces of 16 bytes covering a row; a row of 512 bytes or more
// takes the warp several times) per (row, kv head), K and V in flight together.
template <typename T, bool Q, int GL>
__global__ void __launch_bounds__(NT) k_paged_write_vec(PagedWriteParams p) {
  constexpr int N = Vec<T>::N, RPT = GL == 32 && sizeof(T) == 4 ? 2 : 1;   // pieces of a lane
  const int gl = threadIdx.x % GL, Hkv = p.c.Hkv, hd = p.c.hd;
  const unsigned id = blockIdx.x * (unsigned)(NT / GL) + threadIdx.x / GL;   // (rows x heads fit 31 bits)
  if (id >= (unsigned)p.n_rows * (unsigned)Hkv) return;    // (whole groups leave: shuffles stay inside one)
  const int row = (int)(id / (unsigned)Hkv), g = (int)(id - (unsigned)row * (unsigned)Hkv);
  const int pos = __ldg(p.pos + row);
  if (pos < 0) return;
  const long long src = (long long)row * p.ld + (long long)g * hd;
  uint4 w[2][RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int d = (i * GL + gl) * N;
    w[0][i] = d < hd ? __ldcs(reinterpret_cast<const uint4*>((const T*)p.k + src + d)) : make_uint4(0, 0, 0, 0);
    w[1][i] = d < hd ? __ldcs(reinterpret_cast<const uint4*>((const T*)p.v + src + d)) : make_uint4(0, 0, 0, 0);
  }
  const int page = page_of(p.c, p.seq == 1 ? row : row / p.seq, pos, p.st, 201);
  if (page < 0) return;
  const long long slot = ((long long)page * Hkv + g) * p.c.page_size + slot_of(p.c, pos);
  const unsigned group = GL == 32 ? 0xffffffffu : ((1u << GL) - 1) << ((threadIdx.x & 31) / GL * GL);
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    if (!Q) {
      T* dst = (T*)(kv ? p.c.v : p.c.k) + slot * hd;
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const int d = (i * GL + gl) * N;
        if (d < hd) *reinterpret_cast<uint4*>(dst + d) = w[kv][i];
      }
    } else {
      float x[RPT][N], a = 0.f;
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        unpack<T>(w[kv][i], x[i]);
#pragma unroll
        for (int e = 0; e < N; ++e) a = fmaxf(a, fabsf(x[i][e]));   // (fmaxf drops NaN)
      }
#pragma unroll
      for (int o = GL / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(group, a, o));
      if (a == INFINITY) {                                 // infinities leave the scale alone
        a = 0.f;
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
          for (int e = 0; e < N; ++e) {
            a = fmaxf(a, finite_abs(x[i][e]));
            x[i][e] = inf_to_nan(x[i][e]);
          }
#pragma unroll
        for (int o = GL / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(group, a, o));
      }
      const int E = row_exponent(a);
      const float inv = pow2_neg(E);
      uint8_t* dst = (uint8_t*)(kv ? p.c.v : p.c.k) + slot * hd;
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const int d = (i * GL + gl) * N;
        if (d >= hd) continue;
        if (N == 8)
          *reinterpret_cast<uint2*>(dst + d) = make_uint2(to_e4m3x4(x[i][0], x[i][1], x[i][2], x[i][3], inv),
                                                          to_e4m3x4(x[i][4 % N], x[i][5 % N], x[i][6 % N], x[i][7 % N], inv));
        else
          *reinterpret_cast<uint32_t*>(dst + d) = to_e4m3x4(x[i][0], x[i][1], x[i][2], x[i][3], inv);
      }
      if (gl == 0) (kv ? p.c.ve : p.c.ke)[slot] = (uint8_t)(E + 127);
    }
  }
}

// One warp per (sequence, kv head, position): K, then V, value by value.
template <typename T, bool Q>
__global__ void __launch_bounds__(NT) k_paged_read(PagedReadParams p) {
  const int lane = threadIdx.x & 31, Hkv = p.c.Hkv, hd = p.c.hd;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5), g = blockIdx.y, b = blockIdx.z;
  const int n = min(visible_keys(p.c, p.lens, b, p.len_add, p.st, 211), p.t_out);
  if (t >= n) return;
  const int page = page_of(p.c, b, t, p.st, 212);
  if (page < 0 && !p.zero_bad) return;
  const long long slot = ((long long)page * Hkv + g) * p.c.page_size + slot_of(p.c, t);
  const long long out = (((long long)b * Hkv + g) * p.t_out + t) * hd;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    T* dst = (T*)(kv ? p.v_out : p.k_out) + out;
    if (page < 0) {
      for (int d = lane; d < hd; d += 32) dst[d] = from_f<T>(0.f);
    } else if (!Q) {
      const T* src = (const T*)(kv ? p.c.v : p.c.k) + slot * hd;
      for (int d = lane; d < hd; d += 32) dst[d] = src[d];
    } else {
      const uint8_t* src = (const uint8_t*)(kv ? p.c.v : p.c.k) + slot * hd;
      const float sc = exp_byte_scale((kv ? p.c.ve : p.c.ke)[slot]);
      for (int d = lane; d < hd; d += 32) dst[d] = from_f<T>(e4m3_f(src[d]) * sc);
    }
  }
}

// RT positions per CTA of one (sequence, kv head).  The threads first look the positions' slots
// up together; then the CTA's pieces (16 bytes of the output) go to neighbouring threads, UN of
// K and UN of V in flight each.
template <typename T, bool Q>
__global__ void __launch_bounds__(NT) k_paged_read_vec(PagedReadParams p, int rt) {
  constexpr int N = Vec<T>::N, UN = 4;
  __shared__ long long slot_s[NT];
  __shared__ float sc[2][NT];
  const int Hkv = p.c.Hkv, hd = p.c.hd, g = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int n = min(visible_keys(p.c, p.lens, b, p.len_add, p.st, 211), p.t_out), t0 = blockIdx.x * rt;
  if (t0 >= n) return;
  if (tid < rt) {
    const int t = t0 + tid;
    long long s = -1;
    if (t < n) {
      const int page = page_of(p.c, b, t, p.st, 212);
      if (page >= 0) s = ((long long)page * Hkv + g) * p.c.page_size + slot_of(p.c, t);
      else if (p.zero_bad) s = -2;
    }
    slot_s[tid] = s;
    if (Q && s >= 0) sc[0][tid] = exp_byte_scale(__ldg(p.c.ke + s)), sc[1][tid] = exp_byte_scale(__ldg(p.c.ve + s));
  }
  __syncthreads();
  const int per = hd / N, pieces = rt * per;                 // pieces of a row, of the CTA
  const long long out = (((long long)b * Hkv + g) * p.t_out + t0) * hd;
  for (int i0 = tid; i0 < pieces; i0 += NT * UN) {
    uint4 w[2][UN];
    int at[UN];                                              // row of the piece, -1: nothing to copy, -2: zeros
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int i = i0 + u * NT, r = i / per, d = (i - r * per) * N;
      at[u] = i >= pieces ? -1 : slot_s[r] >= 0 ? r : (int)slot_s[r];
      if (at[u] < 0) continue;
      const long long s = slot_s[r] * hd + d;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const void* src = kv ? p.c.v : p.c.k;
        if (!Q) w[kv][u] = __ldcs(reinterpret_cast<const uint4*>((const T*)src + s));
        else if (N == 8) {
          const uint2 q = __ldcs(reinterpret_cast<const uint2*>((const uint8_t*)src + s));
          w[kv][u].x = q.x, w[kv][u].y = q.y;
        } else w[kv][u].x = __ldcs(reinterpret_cast<const unsigned int*>((const uint8_t*)src + s));
      }
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      if (at[u] == -1) continue;
      const int i = i0 + u * NT;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        uint4 y = at[u] < 0 ? make_uint4(0, 0, 0, 0) : w[kv][u];
        if (Q && at[u] >= 0) {
          const float f = sc[kv][at[u]];
          const uint32_t q[2] = {y.x, y.y};
          float x[N];
#pragma unroll
          for (int e = 0; e < N; ++e) x[e] = e4m3_f((uint8_t)(q[e / 4] >> (8 * (e % 4)))) * f;
          y = pack<T>(x);
        }
        __stcs(reinterpret_cast<uint4*>((T*)(kv ? p.v_out : p.k_out) + out) + i, y);
      }
    }
  }
}

namespace {
bool on16(const void* a, const void* b) { return !(((uintptr_t)a | (uintptr_t)b) & 15); }

template <typename T, bool Q> void write_t(const PagedWriteParams& p, cudaStream_t s) {
  const int n = Vec<T>::N, pieces = p.c.hd / n;
  const long long ids = (long long)p.n_rows * p.c.Hkv;
  note_launch();
  // the stored rows are aligned like their base: hd is a multiple of a piece's values
  if (p.c.hd % n || p.ld % n || !on16(p.k, p.v) || !on16(p.c.k, p.c.v)) {
    k_paged_write<T, Q><<<(unsigned)((ids + 3) / 4), NT, 0, s>>>(p);
    return;
  }
#define RDT_W(GL) k_paged_write_vec<T, Q, GL><<<(unsigned)((ids * GL + NT - 1) / NT), NT, 0, s>>>(p)
  if (pieces <= 8) RDT_W(8);
  else if (pieces <= 16) RDT_W(16);
  else RDT_W(32);
#undef RDT_W
}
template <typename T, bool Q> void read_t(const PagedReadParams& p, cudaStream_t s) {
  const int n = Vec<T>::N, most = std::min(p.t_out, p.c.max_pages * p.c.page_size);   // (a table holds 2^30 positions at most)
  note_launch();
  if (p.c.hd % n || !on16(p.c.k, p.c.v) || !on16(p.k_out, p.v_out)) {
    k_paged_read<T, Q><<<dim3((unsigned)((most + 3) / 4), (unsigned)p.c.Hkv, (unsigned)p.B), NT, 0, s>>>(p);
    return;
  }
  // two rounds of the threads' pieces
  const int rt = std::max(1, std::min(NT, 2 * 4 * NT / (p.c.hd / n)));
  k_paged_read_vec<T, Q><<<dim3((unsigned)((most + rt - 1) / rt), (unsigned)p.c.Hkv, (unsigned)p.B), NT, 0, s>>>(p, rt);
}
}  // namespace

void launch_paged_write(int dtype, const PagedWriteParams& p, cudaStream_t s) {
  if (dtype == 0) p.c.e4m3 ? write_t<float, true>(p, s) : write_t<float, false>(p, s);
  else p.c.e4m3 ? write_t<bf16, true>(p, s) : write_t<bf16, false>(p, s);
}

void launch_paged_read(int dtype, const PagedReadParams& p, cudaStream_t s) {
  if (dtype == 0) p.c.e4m3 ? read_t<float, true>(p, s) : read_t<float, false>(p, s);
  else p.c.e4m3 ? read_t<bf16, true>(p, s) : read_t<bf16, false>(p, s);
}

}  // namespace rdt
