// C ABI of the paged cache: validation, sizes, launches.
// Declarations and contracts: include/kvq.h, "Paged cache".
#include "kvq_paged.cuh"

namespace kvq {

int resolve_paged(const kvq_paged_config *cfg, Paged *p) {
  if (!cfg || !p) return KVQ_EINVAL;
  const kvq_paged_config &c = *cfg;
  if (c.n_kv_heads < 1 || c.n_q_heads < 1 || c.n_pages < 1) return KVQ_EINVAL;
  if (c.n_q_heads % c.n_kv_heads != 0) return KVQ_EINVAL;
  if (c.dtype != KVQ_F16 && c.dtype != KVQ_BF16) return KVQ_EINVAL;
  if (c.head_dim != 64 && c.head_dim != 128) return KVQ_EUNSUPPORTED;
  if (c.bits != 2 && c.bits != 4 && c.bits != 8) return KVQ_EUNSUPPORTED;
  if (c.page_size != 16 && c.page_size != 32 && c.page_size != 64 && c.page_size != 128 &&
      c.page_size != 256)
    return KVQ_EUNSUPPORTED;
  if (c.n_q_heads / c.n_kv_heads > 128 || c.n_kv_heads > 1024) return KVQ_EUNSUPPORTED;
  // page ids are int32; the pool's bytes stay far below 2^63
  if (c.n_pages > (1LL << 31)) return KVQ_EUNSUPPORTED;
  *p = Paged{};
  p->H = c.n_kv_heads;
  p->Hq = c.n_q_heads;
  p->rg = c.n_q_heads / c.n_kv_heads;
  p->d = c.head_dim;
  p->bits = c.bits;
  p->page = c.page_size;
  p->bf16 = c.dtype == KVQ_BF16;
  p->rb = c.head_dim * c.bits / 8;
  p->atom_bytes = 2 * kAtom * (p->rb + 4 * c.head_dim / kPagedGroup);
  p->head_bytes = (int64_t)(c.page_size / kAtom) * p->atom_bytes;
  p->page_bytes = p->head_bytes * c.n_kv_heads;
  p->n_pages = c.n_pages;
  return KVQ_OK;
}

static bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// Resolves a call's configuration, cache and batch.
static int resolve_call(const kvq_paged_config *cfg, const kvq_paged_cache *cache,
                        const kvq_paged_batch *batch, Paged *p) {
  const int r = resolve_paged(cfg, p);
  if (r != KVQ_OK) return r;
  if (!cache || !batch || !cache->pages || !cache->dev_status) return KVQ_EINVAL;
  if (!batch->block_table || !batch->seq_lens || !batch->cu_tokens) return KVQ_EINVAL;
  if (batch->n_seqs < 1 || batch->table_width < 1 || batch->n_tokens < 0 || batch->max_tokens < 0)
    return KVQ_EINVAL;
  if (batch->n_seqs > kMaxSeqs) return KVQ_EUNSUPPORTED;
  // positions and row counts are int32 on the device
  if (batch->table_width > (1LL << 30) / p->page || batch->n_tokens > (1LL << 30) ||
      batch->n_tokens * p->Hq > (1LL << 34))
    return KVQ_EUNSUPPORTED;
  if (!aligned(cache->pages, 16) || !aligned(cache->dev_status, 4) ||
      !aligned(batch->block_table, 4) || !aligned(batch->seq_lens, 4) ||
      !aligned(batch->cu_tokens, 4))
    return KVQ_EALIGN;
  p->pages = static_cast<uint8_t *>(cache->pages);
  p->status = cache->dev_status;
  p->table = batch->block_table;
  p->lens = batch->seq_lens;
  p->cu = batch->cu_tokens;
  p->width = batch->table_width;
  p->B = batch->n_seqs;
  p->max_tokens = batch->max_tokens;
  p->T = batch->n_tokens;
  return KVQ_OK;
}

// A packed row array with its own stride between rows of `heads` heads.
static int check_rows(const Paged &p, const void *x, int64_t stride, int heads) {
  if (!x) return KVQ_EINVAL;
  if (stride < (int64_t)heads * p.d || stride > (1LL << 31)) return KVQ_EINVAL;
  if (!aligned(x, 16) || stride % 8 != 0) return KVQ_EALIGN;
  return KVQ_OK;
}

// Whether two packed row arrays overlap (16-bit elements).
static bool overlap(const Paged &p, const void *a, int64_t sa, const void *b, int64_t sb,
                    int heads) {
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  const uintptr_t row = (uintptr_t)heads * p.d * 2;
  return a0 < b0 + (uintptr_t)(p.T - 1) * sb * 2 + row && b0 < a0 + (uintptr_t)(p.T - 1) * sa * 2 + row;
}

static int done(cudaError_t e, int launches) {
  if (e != cudaSuccess) return KVQ_ECUDA;
  note_launch(launches);
  return KVQ_OK;
}

}  // namespace kvq

using namespace kvq;

extern "C" {

int kvq_paged_cache_bytes(const kvq_paged_config *cfg, size_t *pool, size_t *page) {
  Paged p;
  const int r = resolve_paged(cfg, &p);
  if (r != KVQ_OK) return r;
  if (pool) *pool = (size_t)p.page_bytes * (size_t)p.n_pages;
  if (page) *page = (size_t)p.page_bytes;
  return KVQ_OK;
}

int kvq_paged_workspace_bytes(const kvq_paged_config *cfg, size_t *bytes) {
  if (!bytes) return KVQ_EINVAL;
  Paged p;
  const int r = resolve_paged(cfg, &p);
  if (r != KVQ_OK) return r;
  *bytes = paged_workspace_bytes();
  return KVQ_OK;
}

int kvq_paged_write(const kvq_paged_config *cfg, kvq_paged_cache *cache,
                    const kvq_paged_batch *batch, const void *k, int64_t k_stride, const void *v,
                    int64_t v_stride, void *stream) {
  Paged p;
  int r = resolve_call(cfg, cache, batch, &p);
  if (r != KVQ_OK) return r;
  if (p.T == 0) return done(cudaSuccess, 0);
  if ((r = check_rows(p, k, k_stride, p.H)) != KVQ_OK) return r;
  if ((r = check_rows(p, v, v_stride, p.H)) != KVQ_OK) return r;
  return done(launch_paged_write(p, k, k_stride, v, v_stride, static_cast<cudaStream_t>(stream)),
              1);
}

int kvq_paged_read(const kvq_paged_config *cfg, const kvq_paged_cache *cache,
                   const kvq_paged_batch *batch, void *k_out, void *v_out, void *stream) {
  Paged p;
  int r = resolve_call(cfg, cache, batch, &p);
  if (r != KVQ_OK) return r;
  if (p.T == 0) return done(cudaSuccess, 0);
  const int64_t stride = (int64_t)p.H * p.d;
  if ((r = check_rows(p, k_out, stride, p.H)) != KVQ_OK) return r;
  if ((r = check_rows(p, v_out, stride, p.H)) != KVQ_OK) return r;
  if (overlap(p, k_out, stride, v_out, stride, p.H)) return KVQ_EINVAL;
  return done(launch_paged_read(p, k_out, v_out, static_cast<cudaStream_t>(stream)), 1);
}

int kvq_paged_attention(const kvq_paged_config *cfg, const kvq_paged_cache *cache,
                        const kvq_paged_batch *batch, const void *q, int64_t q_stride, void *out,
                        float softmax_scale, void *ws, size_t ws_bytes, void *stream) {
  Paged p;
  int r = resolve_call(cfg, cache, batch, &p);
  if (r != KVQ_OK) return r;
  if (!(softmax_scale == softmax_scale) || softmax_scale - softmax_scale != 0.0f)
    return KVQ_EINVAL;
  if (!ws) return KVQ_EINVAL;
  if (!aligned(ws, 16)) return KVQ_EALIGN;
  if (ws_bytes < paged_workspace_bytes()) return KVQ_ECAPACITY;
  if (p.T == 0) return done(cudaSuccess, 0);
  if ((r = check_rows(p, q, q_stride, p.Hq)) != KVQ_OK) return r;
  const int64_t stride = (int64_t)p.Hq * p.d;
  if ((r = check_rows(p, out, stride, p.Hq)) != KVQ_OK) return r;
  if (overlap(p, q, q_stride, out, stride, p.Hq)) return KVQ_EINVAL;
  int n = 0;
  const cudaError_t e = launch_paged_attention(p, q, q_stride, out, softmax_scale, ws,
                                               static_cast<cudaStream_t>(stream), &n);
  return done(e, n);
}

int kvq_paged_status(kvq_paged_cache *cache, void *stream) {
  if (!cache || !cache->dev_status) return KVQ_EINVAL;
  kvq_cache c = {};
  c.dev_status = cache->dev_status;
  return kvq_get_device_status(&c, stream);
}

}  // extern "C"
