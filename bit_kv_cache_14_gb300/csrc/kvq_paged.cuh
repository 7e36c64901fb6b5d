// Paged cache (include/kvq.h, "Paged cache"): what its translation units share.
#pragma once

#include <cuda_bf16.h>

#include "kvq_internal.cuh"

namespace kvq {

constexpr int kAtom = 16;         // tokens stored together inside a page
constexpr int kPagedGroup = 32;   // channels that share a scale and a zero point
constexpr int kMaxSeqs = 2048;  // (running sums over the sequences fit shared memory)
constexpr float kPagedLimit = 32768.0f;  // stored magnitudes saturate here
constexpr float kMostScale = 3.4028235e38f;  // factors of the scores stay finite: 0 times one is 0

// One paged call, resolved on the host and copied by value into every kernel.
struct Paged {
  int H, Hq, rg, d, bits, page, bf16;
  int rb;             // bytes of one row of codes
  int atom_bytes;
  int64_t head_bytes;  // one head of one page
  int64_t page_bytes;
  int64_t n_pages;
  uint8_t *pages;
  int32_t *status;
  const int32_t *table, *lens, *cu;
  int64_t width;      // block table entries per sequence
  int B;
  int max_tokens;
  int64_t T;          // rows of the packed arrays
};

// Attention of sequences with at most this many query rows (tokens x query
// heads) per KV head goes to the split kernel (kvq_paged_rows.cu).
constexpr int kPagedFewRows = 16;
constexpr int kPagedRowBlocks = 320;  // its most blocks

int resolve_paged(const kvq_paged_config *cfg, Paged *p);

// Calls on the packed rows (cudaError_t of the launch).
cudaError_t launch_paged_write(const Paged &p, const void *k, int64_t ks, const void *v,
                               int64_t vs, cudaStream_t st);
cudaError_t launch_paged_read(const Paged &p, void *k, void *v, cudaStream_t st);
cudaError_t launch_paged_attention(const Paged &p, const void *q, int64_t qs, void *out,
                                   float scale, void *ws, cudaStream_t st, int *launches);
size_t paged_workspace_bytes();
cudaError_t launch_paged_rows(const Paged &p, const void *q, int64_t qs, void *out, float scale,
                              int few, bool beside, void *ws, int num_sms, cudaStream_t st);
size_t paged_rows_workspace();
cudaError_t launch_paged_chunk(const Paged &p, const void *q, int64_t qs, void *out, float scale,
                               int few, void *ws, int num_sms, cudaStream_t st);
size_t paged_chunk_workspace();
int num_sms_cached();

// Launch with or without leave to start while the previous kernel on the stream
// ends (programmatic dependent launch; the kernel waits itself where it has to).
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kern)(P...), unsigned grid, unsigned threads, int smem,
                             cudaStream_t st, bool early, A &&...args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(grid);
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = (size_t)smem;
  c.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = attr;
  c.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&c, kern, static_cast<A &&>(args)...);
}

namespace {

// ---- device helpers ------------------------------------------------------
// The first error stays in the status word until it is read, but for a wait that
// ran out: that one takes the word over, since the scratch has to be cleared.
__device__ __forceinline__ void paged_error(const Paged &p, int code) {
  if (code == KVQ_ETIMEOUT) atomicExch(p.status, code);
  else atomicCAS(p.status, 0, code);
}

// Whether sequence b's rows are none of the call's: out of order (their
// difference could wrap), outside the packed arrays, or more than allowed.
__device__ __forceinline__ bool bad_rows(const Paged &p, int b) {
  const int r0 = p.cu[b], r1 = p.cu[b + 1];
  return r0 < 0 || r1 < r0 || r1 > p.T || r1 - r0 > p.max_tokens;
}

// Position of row t of sequence b (negative: the row precedes its sequence).
__device__ __forceinline__ int64_t row_position(const Paged &p, int b, int64_t t) {
  return (int64_t)p.lens[b] - p.cu[b + 1] + t;
}

// Address of the atom that holds position `pos` (>= 0) of sequence b and head
// 0, or null with KVQ_EPAGE recorded.
__device__ __forceinline__ uint8_t *atom_of(const Paged &p, int b, int64_t pos) {
  const int64_t i = pos / p.page;
  int64_t id = -1;
  if (i < p.width) id = p.table[b * p.width + i];
  if (id < 0 || id >= p.n_pages) {
    paged_error(p, KVQ_EPAGE);
    return nullptr;
  }
  return p.pages + id * p.page_bytes + (int64_t)((int)(pos % p.page) / kAtom) * p.atom_bytes;
}

}  // namespace
}  // namespace kvq
