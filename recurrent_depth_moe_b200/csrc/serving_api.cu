// C ABI of the serving operators: the paged key / value cache and the sampled next token.
// Host validation only; the kernels are in k_paged_cache.cu, k_paged_attn.cu and k_sample.cu.
#include "../../include/rdt.h"
#include "common.cuh"
#include "kernels.h"
#include "paged_host.h"

#include <math.h>
#include <string.h>

using namespace rdt;

namespace rdt {

rdt_status check_paged_cache(const rdt_paged_cache* c) {
  if (!c || !c->k || !c->v || !c->page_table) return RDT_ERR_INVALID_ARG;
  if ((c->dtype != 0 && c->dtype != 1) || (c->kv_type != 0 && c->kv_type != 1)) return RDT_ERR_INVALID_ARG;
  if (c->kv_type == 1 && (!c->k_exp || !c->v_exp)) return RDT_ERR_INVALID_ARG;
  if (c->n_loops <= 0 || c->n_pages <= 0 || c->page_size <= 0 || c->n_kv_heads <= 0 || c->head_dim <= 0 ||
      c->batch <= 0 || c->max_pages <= 0)
    return RDT_ERR_INVALID_ARG;
  // positions are 32-bit; the grids put sequences and kv heads on their short axes
  if (c->head_dim > 256 || c->n_kv_heads > 4096 || c->batch > 65535) return RDT_ERR_UNSUPPORTED;
  if ((long long)c->max_pages * c->page_size > (1LL << 30)) return RDT_ERR_UNSUPPORTED;
  return RDT_OK;
}

PagedView paged_view(const rdt_paged_cache* c, int loop) {
  PagedView v;
  const size_t rows = (size_t)c->n_pages * c->n_kv_heads * c->page_size;
  const size_t es = c->kv_type ? 1 : c->dtype == 0 ? 4 : 2;
  v.k = (char*)c->k + loop * rows * c->head_dim * es;
  v.v = (char*)c->v + loop * rows * c->head_dim * es;
  v.ke = c->kv_type ? c->k_exp + loop * rows : nullptr;
  v.ve = c->kv_type ? c->v_exp + loop * rows : nullptr;
  v.table = c->page_table;
  v.e4m3 = c->kv_type;
  v.n_pages = c->n_pages; v.page_size = c->page_size; v.Hkv = c->n_kv_heads; v.hd = c->head_dim;
  v.max_pages = c->max_pages;
  v.also = (DevStatus*)c->status;
  v.ps_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (c->page_size == 1 << i) v.ps_shift = i;
  return v;
}

}  // namespace rdt

extern "C" {

rdt_status rdt_paged_kv_write(const rdt_paged_cache* cache, int loop, const void* k, const void* v, long long row_ld,
                              const int32_t* positions, int n_rows, int seq, void* status, void* stream) {
  rdt_status st = check_paged_cache(cache);
  if (st != RDT_OK) return st;
  if (loop < 0 || loop >= cache->n_loops || n_rows < 0 || seq <= 0 || n_rows % seq || n_rows / seq > cache->batch)
    return RDT_ERR_INVALID_ARG;
  if (n_rows == 0) return RDT_OK;
  if (!k || !v || !positions || row_ld < (long long)cache->n_kv_heads * cache->head_dim) return RDT_ERR_INVALID_ARG;
  if ((long long)n_rows * cache->n_kv_heads > (1LL << 31)) return RDT_ERR_UNSUPPORTED;
  cudaStream_t s = (cudaStream_t)stream;
  ProfScope ps(PC_OTHER, s);
  PagedWriteParams p;
  memset(&p, 0, sizeof(p));
  p.c = paged_view(cache, loop);
  p.k = k; p.v = v; p.ld = row_ld; p.pos = positions; p.n_rows = n_rows; p.seq = seq; p.st = (DevStatus*)status;
  launch_paged_write(cache->dtype, p, s);
  return cudaGetLastError() == cudaSuccess ? RDT_OK : RDT_ERR_CUDA;
}

rdt_status rdt_paged_kv_read(const rdt_paged_cache* cache, int loop, const int32_t* lens, int batch, int t_out,
                             void* k_out, void* v_out, void* status, void* stream) {
  rdt_status st = check_paged_cache(cache);
  if (st != RDT_OK) return st;
  if (loop < 0 || loop >= cache->n_loops || batch < 0 || batch > cache->batch || t_out < 0) return RDT_ERR_INVALID_ARG;
  if (batch == 0 || t_out == 0) return RDT_OK;
  if (!lens || !k_out || !v_out) return RDT_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  ProfScope ps(PC_OTHER, s);
  PagedReadParams p;
  memset(&p, 0, sizeof(p));
  p.c = paged_view(cache, loop);
  p.lens = lens; p.B = batch; p.t_out = t_out; p.k_out = k_out; p.v_out = v_out; p.st = (DevStatus*)status;
  launch_paged_read(cache->dtype, p, s);
  return cudaGetLastError() == cudaSuccess ? RDT_OK : RDT_ERR_CUDA;
}

size_t rdt_paged_attention_workspace_size(const rdt_paged_cache* cache, int batch, int n_heads) {
  if (check_paged_cache(cache) != RDT_OK || batch <= 0 || batch > cache->batch || n_heads <= 0 ||
      n_heads % cache->n_kv_heads)
    return 0;
  return 256 + (paged_attn_scratch(paged_view(cache, 0)) + 255) / 256 * 256;
}

rdt_status rdt_paged_attention(const rdt_paged_cache* cache, int loop, const void* q, long long q_ld,
                               const int32_t* lens, int batch, int n_heads, float scale, void* o, long long o_ld,
                               void* ws, size_t ws_bytes, void* status, void* stream) {
  rdt_status st = check_paged_cache(cache);
  if (st != RDT_OK) return st;
  if (loop < 0 || loop >= cache->n_loops || batch < 0 || batch > cache->batch || n_heads <= 0 ||
      n_heads % cache->n_kv_heads || !isfinite(scale))
    return RDT_ERR_INVALID_ARG;
  if (batch == 0) return RDT_OK;
  const long long w = (long long)n_heads * cache->head_dim;
  if (!q || !o || !lens || q == o || q_ld < w || o_ld < w) return RDT_ERR_INVALID_ARG;
  if (n_heads > 4096 || (long long)batch * n_heads > (1LL << 30)) return RDT_ERR_UNSUPPORTED;
  // a worker's share of the tiles (16 keys of up to 8 heads, some hundred workers) is counted in 32 bits
  if ((double)batch * cache->max_pages * cache->page_size * n_heads > 1e12) return RDT_ERR_UNSUPPORTED;
  if (!ws || ((uintptr_t)ws & 255) || ws_bytes < rdt_paged_attention_workspace_size(cache, batch, n_heads))
    return RDT_ERR_WORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  ProfScope ps(PC_ATTN, s);
  PagedAttnParams p;
  memset(&p, 0, sizeof(p));
  p.c = paged_view(cache, loop);
  p.q = q; p.q_row = q_ld; p.o = o; p.o_row = o_ld; p.lens = lens; p.B = batch; p.H = n_heads; p.scale = scale;
  p.scratch = ws; p.st = (DevStatus*)status;
  if (launch_paged_attn(cache->dtype, p, s) != 0) return RDT_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? RDT_OK : RDT_ERR_CUDA;
}

rdt_status rdt_sample_tokens(const float* logits, long long ld, int n, int vocab, const float* u,
                             const rdt_sampling* params, int32_t* tokens, int out_ld, float* logprob, void* stream) {
  if (!params || n < 0 || vocab <= 0 || ld < vocab || out_ld < 1) return RDT_ERR_INVALID_ARG;
  const rdt_sampling& a = *params;
  if (!a.temperature_rows && !(a.temperature >= 0.f && isfinite(a.temperature))) return RDT_ERR_INVALID_ARG;
  if (!a.top_k_rows && a.top_k < 0) return RDT_ERR_INVALID_ARG;
  if (!a.top_p_rows && !(a.top_p > 0.f && a.top_p <= 1.f)) return RDT_ERR_INVALID_ARG;
  if (!a.min_p_rows && !(a.min_p >= 0.f && a.min_p <= 1.f)) return RDT_ERR_INVALID_ARG;
  if (n == 0) return RDT_OK;
  if (!logits || !u || !tokens) return RDT_ERR_INVALID_ARG;
  if (vocab >= (1 << 20) || n > (1 << 27)) return RDT_ERR_UNSUPPORTED;   // the 64-bit weight sums hold 2^20 tokens
  cudaStream_t s = (cudaStream_t)stream;
  ProfScope ps(PC_TOKENS, s);
  SampleParams p;
  memset(&p, 0, sizeof(p));
  p.logits = logits; p.ld = ld; p.n = n; p.vocab = vocab; p.u = u;
  p.temperature = a.temperature; p.top_k = a.top_k; p.top_p = a.top_p; p.min_p = a.min_p;
  p.temperature_row = a.temperature_rows; p.top_k_row = a.top_k_rows;
  p.top_p_row = a.top_p_rows; p.min_p_row = a.min_p_rows;
  p.tokens = tokens; p.out_ld = out_ld; p.logprob = logprob;
  if (launch_sample(p, s) != 0) return RDT_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? RDT_OK : RDT_ERR_CUDA;
}

}  // extern "C"
