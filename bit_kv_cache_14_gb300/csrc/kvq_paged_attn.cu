// Paged cache: causal attention of packed query rows over the pages.
//
// The plain kernel: one warp per (row, query head) walks its sequence token by
// token, the running maximum and sum of the softmax and the output row in
// fp32 registers.  Bound by its own instructions.
#include "kvq_paged.cuh"

namespace kvq {
namespace {

constexpr int kAttnThreads = 256;

// Code of channel c of a row (the layout of include/kvq.h, slot by slot).
template <int D, int BITS>
__device__ __forceinline__ float code_of(const uint8_t *row, int c, bool value) {
  const int g = c / kPagedGroup, r = c % kPagedGroup;
  int bit;
  if (value) {
    constexpr int W = (D == 64 && BITS == 2) ? 8 : 16;
    const int pair = (g >> 1) * 4 + (r & 3), at = pair * BITS;
    bit = (r >> 2) * (D * BITS / 8) + at / W * 2 * W + at % W + W * (g & 1);
  } else {
    const int pair = g * 4 + (r & 7) / 2, at = pair * BITS;
    bit = (r >> 3) * (D * BITS / 4) + at / 16 * 32 + at % 16 + 16 * (r & 1);
  }
  return (float)((row[bit >> 3] >> (bit & 7)) & ((1 << BITS) - 1));
}

template <int D, int BITS>
__global__ void __launch_bounds__(kAttnThreads)
paged_attention_kernel(Paged p, const uint16_t *q, int64_t qs, uint16_t *out, float scale) {
  constexpr int RB = D * BITS / 8, SB = 4 * D / kPagedGroup, NG = D / kPagedGroup;
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * (kAttnThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = item / p.Hq;
  if (t >= p.T) return;
  const int hq = (int)(item % p.Hq), h = hq / p.rg;
  const int b = seq_of_row(p, t);
  if (b < 0) return;
  if (p.cu[b + 1] - p.cu[b] > p.max_tokens) {
    paged_error(p, KVQ_EINVAL);
    return;
  }
  const int64_t pos = row_position(p, b, t);
  // lane's channels: lane + 32 g, one of every group
  float qf[NG], o[NG] = {};
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const uint16_t w = q[t * qs + (int64_t)hq * D + lane + 32 * g];
    qf[g] = p.bf16 ? __uint_as_float((uint32_t)w << 16) : __half2float(__ushort_as_half(w));
  }
  float m = -INFINITY, l = 0.0f;
  for (int64_t s = 0; s <= pos; ++s) {
    const uint8_t *atom = atom_of(p, b, s);
    if (!atom) continue;
    atom += h * p.head_bytes;
    const int row = (int)(s % kAtom);
    const __half *ks = reinterpret_cast<const __half *>(atom + 2 * kAtom * RB + row * SB);
    const __half *vs = reinterpret_cast<const __half *>(atom + 2 * kAtom * RB + kAtom * SB + row * SB);
    float x = 0.0f;
#pragma unroll
    for (int g = 0; g < NG; ++g)
      x += qf[g] * (code_of<D, BITS>(atom + row * RB, lane + 32 * g, false) * __half2float(ks[g]) +
                    __half2float(ks[NG + g]));
#pragma unroll
    for (int i = 16; i; i >>= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
    x *= scale;
    const float mn = fmaxf(m, x), f = __expf(m - mn), w = __expf(x - mn);
    m = mn;
    l = l * f + w;
#pragma unroll
    for (int g = 0; g < NG; ++g)
      o[g] = o[g] * f + w * (code_of<D, BITS>(atom + kAtom * RB + row * RB, lane + 32 * g, true) *
                                 __half2float(vs[g]) +
                             __half2float(vs[NG + g]));
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const float r = o[g] * inv;
    out[(t * p.Hq + hq) * D + lane + 32 * g] =
        p.bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(r)) : __half_as_ushort(__float2half_rn(r));
  }
}

}  // namespace

size_t paged_workspace_bytes() { return paged_rows_workspace(); }

cudaError_t launch_paged_attention(const Paged &p, const void *q, int64_t qs, void *out,
                                   float scale, void *ws, cudaStream_t st, int *launches) {
  if ((int64_t)p.max_tokens * p.rg <= kPagedFewRows) {
    *launches = 1;
    return launch_paged_rows(p, q, qs, out, scale, ws, num_sms_cached(), st);
  }
  const unsigned grid = (unsigned)((p.T * p.Hq + kAttnThreads / 32 - 1) / (kAttnThreads / 32));
  auto kern = p.d == 128 ? (p.bits == 2   ? paged_attention_kernel<128, 2>
                            : p.bits == 4 ? paged_attention_kernel<128, 4>
                                          : paged_attention_kernel<128, 8>)
                         : (p.bits == 2   ? paged_attention_kernel<64, 2>
                            : p.bits == 4 ? paged_attention_kernel<64, 4>
                                          : paged_attention_kernel<64, 8>);
  kern<<<grid, kAttnThreads, 0, st>>>(p, static_cast<const uint16_t *>(q), qs,
                                      static_cast<uint16_t *>(out), scale);
  *launches = 1;
  return cudaGetLastError();
}

}  // namespace kvq
