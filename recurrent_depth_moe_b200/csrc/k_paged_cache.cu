// Writing the paged key / value cache and reading it back.
//
// write: row i = b * seq + t of k and v goes to slot pos % page_size of page
//   table[b][pos / page_size], every kv head as one row of head_dim values, in the model dtype
//   or as e4m3 with one exponent byte (paged.cuh).  pos < 0: a padding row, nothing written.
// read: positions 0 .. lens[b] - 1 of every sequence, contiguous, in the model dtype.
// Both move each byte once, so they are HBM-bound.
#include "paged.cuh"

namespace rdt {

// One warp per (row, kv head): K, then V.
template <typename T, bool Q>
__global__ void __launch_bounds__(128) k_paged_write(PagedWriteParams p) {
  const long long wid = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, Hkv = p.c.Hkv, hd = p.c.hd;
  if (wid >= (long long)p.n_rows * Hkv) return;
  const int row = (int)(wid / Hkv), g = (int)(wid % Hkv);
  const int pos = p.pos[row];
  if (pos < 0) return;
  const int page = page_of(p.c, row / p.seq, pos, p.st, 201);
  if (page < 0) return;
  const long long slot = ((long long)page * Hkv + g) * p.c.page_size + pos % p.c.page_size;
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

// One warp per (sequence, kv head, position): K, then V.
template <typename T, bool Q>
__global__ void __launch_bounds__(128) k_paged_read(PagedReadParams p) {
  const int lane = threadIdx.x & 31, Hkv = p.c.Hkv, hd = p.c.hd;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5), g = blockIdx.y, b = blockIdx.z;
  const int n = min(visible_keys(p.c, p.lens, b, p.len_add, p.st, 211), p.t_out);
  if (t >= n) return;
  const int page = page_of(p.c, b, t, p.st, 212);
  if (page < 0) return;
  const long long slot = ((long long)page * Hkv + g) * p.c.page_size + t % p.c.page_size;
  const long long out = (((long long)b * Hkv + g) * p.t_out + t) * hd;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    T* dst = (T*)(kv ? p.v_out : p.k_out) + out;
    if (!Q) {
      const T* src = (const T*)(kv ? p.c.v : p.c.k) + slot * hd;
      for (int d = lane; d < hd; d += 32) dst[d] = src[d];
    } else {
      const uint8_t* src = (const uint8_t*)(kv ? p.c.v : p.c.k) + slot * hd;
      const float sc = exp_byte_scale((kv ? p.c.ve : p.c.ke)[slot]);
      for (int d = lane; d < hd; d += 32) dst[d] = from_f<T>(e4m3_f(src[d]) * sc);
    }
  }
}

#define RDT_PAGED_DISPATCH(KERNEL, GRID, P)                                                      \
  do {                                                                                           \
    if (dtype == 0 && !P.c.e4m3) KERNEL<float, false><<<GRID, 128, 0, s>>>(P);                   \
    else if (dtype == 0) KERNEL<float, true><<<GRID, 128, 0, s>>>(P);                            \
    else if (!P.c.e4m3) KERNEL<bf16, false><<<GRID, 128, 0, s>>>(P);                             \
    else KERNEL<bf16, true><<<GRID, 128, 0, s>>>(P);                                             \
    note_launch();                                                                               \
  } while (0)

void launch_paged_write(int dtype, const PagedWriteParams& p, cudaStream_t s) {
  const long long warps = (long long)p.n_rows * p.c.Hkv;
  const dim3 grid((unsigned)((warps + 3) / 4));
  RDT_PAGED_DISPATCH(k_paged_write, grid, p);
}

void launch_paged_read(int dtype, const PagedReadParams& p, cudaStream_t s) {
  const dim3 grid((unsigned)((p.t_out + 3) / 4), (unsigned)p.c.Hkv, (unsigned)p.B);
  RDT_PAGED_DISPATCH(k_paged_read, grid, p);
}
#undef RDT_PAGED_DISPATCH

}  // namespace rdt
