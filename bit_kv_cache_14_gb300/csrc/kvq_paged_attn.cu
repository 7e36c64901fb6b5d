// Paged cache: attention of packed query rows over the pages, causal or (cross) over
// all of a sequence -- which kernel takes which sequence.
//
// Both forms run the same kernels: a row sees the tokens up to a position of its own,
// and a cross row's is the last.  Cross attention on a GB300: 32 encoders of 1515 to
// 4096 tokens, four beams of four heads each, 4 bits: 68 us (118 MB); one row of four
// heads each over 64 of 8192 tokens, 4 bits: 155 us = 64 % of the copy rate; 2 x 2048 rows
// over 16384 tokens, 32 and 8 heads, 4 bits: 762 us = 1443 TFLOP/s, 77 % of the measured
// rate (809 us back to back for seconds, at a lower clock: 80 % of the sustained rate).
//
// Its errors are the causal call's, from operands rounded to fp16: against 64 bits, as a
// share of the output's norm, fp16 with 122 to 219 rows at 2 bits 7.1e-4, of which 6.2e-4
// are the keys' rounding and 2.1e-4 the output's; few rows 2.3e-4; bf16 1.7e-3, the
// output's rounding.  Keys in two parts would take that away, for half as many matrix
// operations again and 64 KB of shared memory that the operand tiles do not leave.
//
// (For 9 to 32 rows a tcgen05 kernel with tokens and channels as the MMA rows was
// built: 96 us for 16 rows where the split kernel takes 77, 130 to 138 for 20 to 32 where
// the chunk kernel took 120, 186 for 146 at 8 bits; not kept.)
//
// A sequence's rows are its new tokens times the query heads of one KV head.
// Up to 16 rows the cache's bytes bound the time and the split kernel
// (kvq_paged_rows.cu) reads them once, at 8 or 16 rows an MMA tile; from there
// on the tcgen05 kernel (kvq_paged_chunk.cu) takes the sequence (32 sequences of
// 8192 tokens, 4 new ones of 4 heads each, 4 bits: 129 us split, 223 us tcgen05;
// 8 new ones: 203 us there).  Lengths are on the device, so a call whose
// max_tokens allows both launches both, and each kernel passes over the other's
// sequences.
#include "kvq_paged.cuh"

namespace kvq {

size_t paged_workspace_bytes() { return paged_rows_workspace() + paged_chunk_workspace(); }

cudaError_t launch_paged_attention(const Paged &p, const void *q, int64_t qs, void *out,
                                   float scale, void *ws, cudaStream_t st, int *launches) {
  const int sms = num_sms_cached();
  // (a call without rows, only padding, still looks whether that is so)
  const int64_t most = (int64_t)(p.max_tokens > 0 ? p.max_tokens : 1) * p.rg;
  // a mixed call's small sequences are decode steps: the 8-row form of the
  // split kernel, where the heads of one token fit it (a chunk of 512 with 63
  // decodes of up to 8000 tokens: 190 us, 248 us with the 16-row form)
  const int few = (most <= 8 || (most > kPagedFewRows && p.rg <= 8)) ? 8 : kPagedFewRows;
  const bool rows = p.rg <= few, chunks = most > few;
  cudaError_t e = cudaSuccess;
  // The split kernel may start its blocks while the kernel before it ends: alone
  // it waits there before it reads; behind the chunk kernel, which starts when
  // everything before the call is done, it takes the room that one leaves.
  if (chunks)
    e = launch_paged_chunk(p, q, qs, out, scale, few,
                           static_cast<uint8_t *>(ws) + paged_rows_workspace(), sms, st);
  if (e == cudaSuccess && rows)
    e = launch_paged_rows(p, q, qs, out, scale, few, chunks, ws, sms, st);
  *launches = (int)rows + (int)chunks;
  return e;
}

}  // namespace kvq
