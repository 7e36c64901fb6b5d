// Verification of drafted tokens (include/kvq.h, kvq_verify_drafts).
//
// Row t of a sequence holds the target's logits x for the token after row t's, and
// the draft model's y.  With p = softmax(x / T), q = softmax(y / T), the drafted
// token c of the next row stays while u q(c) < p(c); at the first that does not,
// the next token is the largest max(p - q, 0)_i / e_i, behind the last draft the
// largest p_i / e_i, with the caller's exponential e (the smallest of exponentials
// of rates p_i is at i with probability p_i).
//
// Two launches.  Rows: every (row, part of the vocabulary) leaves its maximum m
// and s = sum 2^((x - m) c), c = log2(e) / T, so each logit is read once; all rows
// are taken, since which draft is the first refused is known only afterwards.
// Draw: the blocks of a sequence each join its rows' parts (a few hundred bytes),
// decide, and race their share of the one row that is drawn from; shares are joined
// by a maximum over (score, lowest index), which has no order.
#include <algorithm>

#include "kvq_paged.cuh"
#include "kvq_tc_common.cuh"

namespace kvq {
namespace {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int64_t kMaxRows = 65535;      // (rows are a grid dimension)
constexpr int64_t kMaxVocab = 1 << 24;
// Logits are held to +-2^126, so that differences of two are finite; a logit down
// there is masked (probability 0), and NaN is taken as masked.
constexpr float kMasked = -8.507059e37f;
constexpr double kLog2e = 1.4426950408889634;

struct VerifyArgs {
  const int32_t *cu, *tokens;
  const void *logits, *draft;
  int64_t stride, dstride, nstride;
  const float *temperature, *uniform, *noise;
  int32_t *out, *accepted, *dropped;
  float *logprobs;
  int32_t *status;
  unsigned long long *keys;  // [B][2], zero between calls
  int *tickets;              // [B], zero between calls
  float4 *parts;             // [2][T][parts]: maximum, sum, lowest index of the maximum
  int64_t T;
  int B, V, n_parts, splits;
};

__device__ __forceinline__ void verify_error(const VerifyArgs &a, int code) {
  atomicCAS(a.status, 0, code);
}
__device__ __forceinline__ bool bad_range(const VerifyArgs &a, int r0, int r1) {
  return r0 < 0 || r1 < r0 || r1 > a.T;
}

// The sequence of row t, found by the whole warp (32 candidates a round), or -1.
__device__ __forceinline__ int sequence_of(const VerifyArgs &a, int64_t t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = a.B;  // the largest b with cu[b] <= t
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, b = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, b < hi && a.cu[b] <= t);
    if (le == 0) return -1;
    lo += (31 - __clz(le)) * step;
    hi = min(lo + step, hi);
  }
  const int r0 = a.cu[lo], r1 = a.cu[lo + 1];
  return t >= r0 && t < r1 && !bad_range(a, r0, r1) ? lo : -1;
}

// The temperature of sequence b; 0: greedy (also for what is no temperature).
__device__ __forceinline__ float temperature_of(const VerifyArgs &a, int b) {
  const float t = a.temperature ? a.temperature[b] : 0.0f;
  return t > 0.0f ? t : 0.0f;
}
// log2(e) / T in 64 bits, held where its product with any difference of logits and
// that product's low part stay numbers.  Greedy rows: T = 1.
__device__ __forceinline__ double factor_of(float temperature) {
  const double c = temperature > 0.0f ? kLog2e / (double)temperature : kLog2e;
  return fmin(fmax(c, 0x1p-100), 0x1p25);
}

// Types: 0 fp16, 1 bf16, 2 fp32.
template <int TYPE>
struct Logit {
  static constexpr int kSize = TYPE == 2 ? 4 : 2;
  static constexpr int kVec = 16 / kSize;  // of a 16-byte vector
};
__device__ __forceinline__ float tame(float x) { return fminf(fmaxf(x, kMasked), -kMasked); }
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
template <int TYPE>
__device__ __forceinline__ float load_logit(const void *row, int64_t i) {
  float x;
  if (TYPE == 2) {
    x = __ldg(static_cast<const float *>(row) + i);
  } else {
    const uint32_t h = __ldg(static_cast<const uint16_t *>(row) + i);
    x = TYPE == 1 ? __uint_as_float(h << 16) : __half2float(__ushort_as_half((uint16_t)h));
  }
  return tame(x);
}
// Elements of a 16-byte vector.
template <int TYPE>
__device__ __forceinline__ void unpack(uint4 v, float (&x)[Logit<TYPE>::kVec]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (TYPE == 2) {
      x[i] = __uint_as_float(w[i]);
    } else if constexpr (TYPE == 1) {
      x[2 * i] = bf16_lo(w[i]);
      x[2 * i + 1] = bf16_hi(w[i]);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}
// How many elements before the row's first its first 16-byte vector begins.
template <int TYPE>
__device__ __forceinline__ int lead_of(const void *row) {
  return (int)((uintptr_t)row & 15) / Logit<TYPE>::kSize;
}

// 2^((x - m) c), c in two parts: a difference is exact or nearly so, and its
// product keeps what one rounded factor would lose for every element alike.
__device__ __forceinline__ float weight(float x, float m, float ch, float cl) {
  const float d = x - m;
  return exp2_approx(fmaf(d, ch, d * cl));
}

// ---- rows -------------------------------------------------------------------
// Block (part, row, model): NV vectors a thread, vector i of thread t the part's
// vector i * threads + t.
template <int TYPE, int NV>
__global__ void __launch_bounds__(kVerifyThreads)
verify_rows_kernel(const __grid_constant__ VerifyArgs a) {
  using L = Logit<TYPE>;
  constexpr int N = L::kVec;
  __shared__ float sm[kVerifyWarps], ss[kVerifyWarps];
  __shared__ int first;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int part = blockIdx.x, model = blockIdx.z;
  const int64_t t = blockIdx.y;
  grid_dep_trigger();
  grid_dep_wait();
  const char *row = static_cast<const char *>(model ? a.draft : a.logits) +
                    t * (model ? a.dstride : a.stride) * L::kSize;
  const int lead = lead_of<TYPE>(row);
  // vector v holds elements v * N - lead .. + N - 1
  float x[NV][N];
  const int64_t v0 = (int64_t)part * NV * kVerifyThreads + tid;
  const uint4 *vec = reinterpret_cast<const uint4 *>(row - lead * L::kSize);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t e0 = (v0 + i * kVerifyThreads) * N - lead;
    if (e0 >= 0 && e0 + N <= a.V) {
      unpack<TYPE>(__ldg(vec + v0 + i * kVerifyThreads), x[i]);
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k)
        x[i][k] = e0 + k >= 0 && e0 + k < a.V ? load_logit<TYPE>(row, e0 + k) : kMasked;
    }
  }
  const int b = sequence_of(a, t);
  if (b < 0) return;
  const float temperature = temperature_of(a, b);
  if (model && (temperature == 0.0f || t + 1 == a.cu[b + 1])) return;  // not looked at
  float m = kMasked;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < N; ++k) {
      x[i][k] = tame(x[i][k]);
      m = fmaxf(m, x[i][k]);
    }
  const double c = factor_of(temperature);
  const float ch = (float)c, cl = (float)(c - (double)ch);
  float s = 0.0f;
  const float mine = m;
  if (m > kMasked) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < N; ++k) s += weight(x[i][k], m, ch, cl);
  }
  float top = m;
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) sm[warp] = top;
  if (tid == 0) first = 0x7fffffff;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kVerifyWarps; ++w) top = fmaxf(top, sm[w]);
  s = mine > kMasked ? s * weight(mine, top, ch, cl) : 0.0f;
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) ss[warp] = s;
  // the lowest index of the maximum, for greedy rows
  if (temperature == 0.0f && mine == top && top > kMasked) {
    int at = 0x7fffffff;
#pragma unroll
    for (int i = NV - 1; i >= 0; --i)
#pragma unroll
      for (int k = N - 1; k >= 0; --k)
        if (x[i][k] == top) at = (int)((v0 + i * kVerifyThreads) * N - lead + k);
    atomicMin(&first, at);
  }
  __syncthreads();
  if (tid == 0) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kVerifyWarps; ++w) sum += ss[w];
    a.parts[((int64_t)model * a.T + t) * a.n_parts + part] =
        make_float4(top, sum, __int_as_float(first), 0.0f);
  }
}

// ---- draw -------------------------------------------------------------------
// Maximum, sum and lowest index of the maximum of a row, by the whole warp, in a
// fixed order.
struct Row {
  float m, s;
  int at;
};
__device__ __forceinline__ Row join_row(const VerifyArgs &a, int model, int64_t t, double c) {
  const int lane = threadIdx.x & 31;
  const float4 *p = a.parts + ((int64_t)model * a.T + t) * a.n_parts;
  const float ch = (float)c, cl = (float)(c - (double)ch);
  Row r = {kMasked, 0.0f, 0x7fffffff};
  for (int i = lane; i < a.n_parts; i += 32) r.m = fmaxf(r.m, __ldcg(p + i).x);
#pragma unroll
  for (int o = 16; o; o >>= 1) r.m = fmaxf(r.m, __shfl_xor_sync(0xffffffffu, r.m, o));
  if (r.m == kMasked) return r;
  for (int i = lane; i < a.n_parts; i += 32) {
    const float4 v = __ldcg(p + i);
    if (v.x > kMasked) r.s += v.y * weight(v.x, r.m, ch, cl);
    if (v.x == r.m) r.at = min(r.at, __float_as_int(v.z));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    r.s += __shfl_xor_sync(0xffffffffu, r.s, o);
    r.at = min(r.at, __shfl_xor_sync(0xffffffffu, r.at, o));
  }
  return r;
}

// Natural logarithm of a token's probability: logit x in a row of maximum m, sum s.
__device__ __forceinline__ float log_probability(float x, const Row &r, double c) {
  return (float)(((double)(x - r.m) * c) * 0.6931471805599453) - logf(r.s);
}

// u q(c) < p(c): 2^(tp - tq) s_q / s_p against u, the exponent in 64 bits.
__device__ __forceinline__ bool stays(float u, float x, const Row &p, float y, const Row &q,
                                      bool model, double c) {
  if (!(x > kMasked)) return false;  // p(c) = 0
  double t = (double)(x - p.m) * c;
  float sq = 1.0f;
  if (model) {
    if (!(y > kMasked)) return true;  // q(c) = 0 < p(c)
    t -= (double)(y - q.m) * c;
    sq = q.s;
  }
  t = fmin(fmax(t, -1000.0), 1000.0);
  const double k = rint(t);
  const float f = exp2f((float)(t - k));
  return (double)u * (double)p.s < ldexp((double)(f * sq), (int)k);
}

__device__ __forceinline__ unsigned long long key_of(float score, int64_t i) {
  return score > 0.0f ? (unsigned long long)__float_as_uint(score) << 32 | (0xffffffffu - (uint32_t)i)
                      : 0ull;
}
__device__ __forceinline__ unsigned long long max64(unsigned long long a, unsigned long long b) {
  return a > b ? a : b;
}

// Block (share, sequence).
template <int TYPE>
__global__ void __launch_bounds__(kVerifyThreads)
verify_draw_kernel(const __grid_constant__ VerifyArgs a) {
  using L = Logit<TYPE>;
  __shared__ int stop, last;
  __shared__ Row row_p, row_q;  // of the row that is drawn from
  __shared__ unsigned long long best[2][kVerifyWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.y, share = blockIdx.x;
  grid_dep_trigger();
  grid_dep_wait();
  const int r0 = a.cu[b], r1 = a.cu[b + 1], n = r1 - r0;
  if (bad_range(a, r0, r1) || n == 0) {
    if (share == 0 && tid == 0) {
      if (n != 0 || bad_range(a, r0, r1)) verify_error(a, KVQ_EINVAL);
      a.accepted[b] = 0;
      a.dropped[b] = 0;
    }
    return;
  }
  const float temperature = temperature_of(a, b);
  const bool greedy = temperature == 0.0f, model = a.draft != nullptr && !greedy;
  const double c = factor_of(temperature);
  auto row_of = [&](int which, int64_t t) {
    return static_cast<const char *>(which ? a.draft : a.logits) +
           t * (which ? a.dstride : a.stride) * L::kSize;
  };
  if (tid == 0) stop = n - 1;
  __syncthreads();
  // ---- the drafts that stay; the block of share 0 writes their outputs below
  for (int i = warp; i < n - 1; i += kVerifyWarps) {
    const int64_t t = r0 + i;
    const int token = a.tokens[t + 1];
    const Row p = join_row(a, 0, t, c);
    bool ok = token >= 0 && token < a.V;
    if (!ok && share == 0 && lane == 0) verify_error(a, KVQ_EINVAL);
    if (ok && greedy) {
      ok = p.at == token;
    } else if (ok) {
      Row q = {0.0f, 1.0f, 0};
      float y = 0.0f;
      if (model) {
        q = join_row(a, 1, t, c);
        y = load_logit<TYPE>(row_of(1, t), token);
      }
      ok = stays(a.uniform[t], load_logit<TYPE>(row_of(0, t), token), p, y, q, model, c);
    }
    if (!ok && lane == 0) atomicMin(&stop, i);
  }
  __syncthreads();
  const int kept = stop;
  const int64_t t = r0 + kept;
  const bool refused = kept < n - 1;
  if (warp == 0) {
    const Row p = join_row(a, 0, t, c);
    if (lane == 0) row_p = p;
  } else if (warp == 1 && refused && model) {
    const Row q = join_row(a, 1, t, c);
    if (lane == 0) row_q = q;
  }
  __syncthreads();
  const Row p = row_p;
  if (greedy) {
    if (share != 0) return;
  } else {
    // ---- the race over this share of the vocabulary
    const bool rest = refused && model;
    const int gone = refused && !model ? a.tokens[t + 1] : -1;  // all of q
    const float ch = (float)c, cl = (float)(c - (double)ch);
    const Row q = rest ? row_q : Row{0.0f, 1.0f, 0};
    // (a draft row without a finite logit takes nothing off)
    const float ip = 1.0f / p.s, iq = rest && q.s > 0.0f ? 1.0f / q.s : 0.0f;
    const char *xr = row_of(0, t), *yr = rest ? row_of(1, t) : xr;
    const float *er = a.noise + b * a.nstride;
    unsigned long long k0 = 0, k1 = 0;  // by what is left of p; by p
    auto race = [&](int64_t i, float x, float y, float e) {
      // (products rounded by themselves: equal p and q leave exactly nothing)
      const float wp = __fmul_rn(weight(x, p.m, ch, cl), ip);
      const float r = 1.0f / fmaxf(e, 1.1754944e-38f);
      float w = wp;
      if (rest) w = __fsub_rn(wp, __fmul_rn(weight(y, q.m, ch, cl), iq));
      if (i == gone) w = 0.0f;
      if (e == e) k0 = max64(k0, key_of(w * r, i)), k1 = max64(k1, key_of(wp * r, i));
    };
    if (p.m > kMasked) {
      const int64_t per = (a.V + a.splits - 1) / a.splits;
      const int64_t i0 = share * per, i1 = min(i0 + per, (int64_t)a.V);
      for (int64_t i = i0 + tid; i < i1; i += kVerifyThreads)
        race(i, load_logit<TYPE>(xr, i), rest ? load_logit<TYPE>(yr, i) : 0.0f, __ldg(er + i));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      k0 = max64(k0, __shfl_xor_sync(0xffffffffu, k0, o));
      k1 = max64(k1, __shfl_xor_sync(0xffffffffu, k1, o));
    }
    if (lane == 0) best[0][warp] = k0, best[1][warp] = k1;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
      for (int w = 1; w < kVerifyWarps; ++w) k0 = max64(k0, best[0][w]), k1 = max64(k1, best[1][w]);
      if (k0) atomicMax(&a.keys[2 * b], k0);
      if (k1) atomicMax(&a.keys[2 * b + 1], k1);
      __threadfence();
      last = atomicAdd(&a.tickets[b], 1) == a.splits - 1;
    }
    __syncthreads();
    if (!last) return;
  }
  // ---- outputs
  __shared__ int next;
  if (tid == 0) {
    int token = greedy && p.m > kMasked ? p.at : -1;
    if (!greedy) {
      __threadfence();
      const unsigned long long k0 = atomicExch(&a.keys[2 * b], 0ull);
      const unsigned long long k1 = atomicExch(&a.keys[2 * b + 1], 0ull);
      const unsigned long long k = k0 ? k0 : k1;
      if (k) token = (int)(0xffffffffu - (uint32_t)k);
      a.tickets[b] = 0;
    }
    next = token;
    a.accepted[b] = kept;
    a.dropped[b] = n - 1 - kept;
  }
  __syncthreads();
  for (int i = warp; i < n; i += kVerifyWarps) {
    const int token = i < kept ? a.tokens[r0 + i + 1] : i == kept ? next : -1;
    float lp = 0.0f;
    if (token >= 0) {
      const Row r = i == kept ? p : join_row(a, 0, r0 + i, c);
      lp = log_probability(load_logit<TYPE>(row_of(0, r0 + i), token), r, c);
    }
    if (lane == 0) {
      a.out[r0 + i] = token;
      a.logprobs[r0 + i] = lp;
    }
  }
}

// Vectors a thread of the rows' kernel.
constexpr int kVectors = 4;
int parts_of(int64_t vocab, int type) {
  const int64_t per = (int64_t)kVectors * kVerifyThreads * (type == 2 ? 4 : 8);
  return (int)((vocab + (type == 2 ? 3 : 7) + per - 1) / per);
}

// What must stay zero lies in front, whatever the call's sizes.
constexpr size_t kTicketsAt = (size_t)kMaxSeqs * 16, kPartsAt = kTicketsAt + (size_t)kMaxSeqs * 4;
size_t verify_bytes(int64_t T, int64_t V, int type) {
  return kPartsAt + (size_t)2 * T * parts_of(V, type) * sizeof(float4);
}

template <int TYPE>
cudaError_t verify_as(const VerifyArgs &a, cudaStream_t st, int *launches) {
  *launches = 0;
  if (a.T > 0) {
    const dim3 grid((unsigned)a.n_parts, (unsigned)a.T, a.draft ? 2 : 1);
    const cudaError_t e = launch_dependent(verify_rows_kernel<TYPE, kVectors>, grid,
                                           kVerifyThreads, 0, st, true, a);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  ++*launches;
  const dim3 grid((unsigned)a.splits, (unsigned)a.B);
  return launch_dependent(verify_draw_kernel<TYPE>, grid, kVerifyThreads, 0, st, true, a);
}

int check_drafts(const kvq_draft_batch *d) {
  if (!d || !d->cu_tokens || !d->dev_status) return KVQ_EINVAL;
  if (d->n_seqs < 1 || d->vocab < 1 || d->n_tokens < 0) return KVQ_EINVAL;
  if (d->dtype != KVQ_F16 && d->dtype != KVQ_BF16 && d->dtype != KVQ_F32) return KVQ_EINVAL;
  if (d->n_tokens > 0 && !d->tokens) return KVQ_EINVAL;
  if (d->n_seqs > kMaxSeqs || d->n_tokens > kMaxRows || d->vocab > kMaxVocab)
    return KVQ_EUNSUPPORTED;
  if (((uintptr_t)d->cu_tokens & 3) || ((uintptr_t)d->tokens & 3) || ((uintptr_t)d->dev_status & 3))
    return KVQ_EALIGN;
  return KVQ_OK;
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" {

int kvq_verify_workspace_bytes(const kvq_draft_batch *batch, size_t *bytes) {
  if (!bytes || !batch) return KVQ_EINVAL;
  if (batch->n_seqs < 1 || batch->vocab < 1 || batch->n_tokens < 0) return KVQ_EINVAL;
  if (batch->dtype != KVQ_F16 && batch->dtype != KVQ_BF16 && batch->dtype != KVQ_F32)
    return KVQ_EINVAL;
  if (batch->n_seqs > kMaxSeqs || batch->n_tokens > kMaxRows || batch->vocab > kMaxVocab)
    return KVQ_EUNSUPPORTED;
  *bytes = verify_bytes(batch->n_tokens, batch->vocab, batch->dtype);
  return KVQ_OK;
}

int kvq_verify_drafts(const kvq_draft_batch *batch, const void *logits, int64_t stride,
                      const void *draft_logits, int64_t draft_stride, const float *temperature,
                      const float *uniform, const float *noise, int64_t noise_stride,
                      int32_t *out_tokens, int32_t *accepted, int32_t *dropped, float *logprobs,
                      void *ws, size_t ws_bytes, void *stream) {
  const int r = check_drafts(batch);
  if (r != KVQ_OK) return r;
  if (!accepted || !dropped || !ws) return KVQ_EINVAL;
  const int64_t T = batch->n_tokens, V = batch->vocab;
  const uintptr_t word = batch->dtype == KVQ_F32 ? 3 : 1;
  if (T > 0) {
    if (!logits || !out_tokens || !logprobs || stride < V) return KVQ_EINVAL;
    if (draft_logits && draft_stride < V) return KVQ_EINVAL;
    if (temperature && (!uniform || !noise || noise_stride < V)) return KVQ_EINVAL;
    if (((uintptr_t)logits & word) || ((uintptr_t)draft_logits & word)) return KVQ_EALIGN;
    for (const void *p : {(const void *)temperature, (const void *)uniform, (const void *)noise,
                          (const void *)out_tokens, (const void *)logprobs})
      if ((uintptr_t)p & 3) return KVQ_EALIGN;
  }
  if (((uintptr_t)accepted & 3) || ((uintptr_t)dropped & 3) || ((uintptr_t)ws & 15))
    return KVQ_EALIGN;
  if (ws_bytes < verify_bytes(T, V, batch->dtype)) return KVQ_ECAPACITY;
  VerifyArgs a = {};
  a.cu = batch->cu_tokens;
  a.tokens = batch->tokens;
  a.logits = logits;
  a.draft = temperature ? draft_logits : nullptr;
  a.stride = stride;
  a.dstride = draft_stride;
  a.nstride = noise_stride;
  a.temperature = temperature;
  a.uniform = uniform;
  a.noise = noise;
  a.out = out_tokens;
  a.accepted = accepted;
  a.dropped = dropped;
  a.logprobs = logprobs;
  a.status = batch->dev_status;
  a.T = T;
  a.B = batch->n_seqs;
  a.V = (int)V;
  a.n_parts = parts_of(V, batch->dtype);
  uint8_t *w = static_cast<uint8_t *>(ws);
  a.keys = reinterpret_cast<unsigned long long *>(w);
  a.tickets = reinterpret_cast<int *>(w + kTicketsAt);
  a.parts = reinterpret_cast<float4 *>(w + kPartsAt);
  // shares of 2048 tokens, fewer where the sequences alone fill the GPU
  int64_t splits = (V + 2047) / 2048;
  const int64_t most = std::max<int64_t>(1, (int64_t)num_sms_cached() * 16 / a.B);
  a.splits = temperature ? (int)std::min(splits, most) : 1;
  int n = 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = batch->dtype == KVQ_F16    ? verify_as<0>(a, st, &n)
                        : batch->dtype == KVQ_BF16 ? verify_as<1>(a, st, &n)
                                                   : verify_as<2>(a, st, &n);
  if (e != cudaSuccess) return KVQ_ECUDA;
  note_launch(n);
  return KVQ_OK;
}

}  // extern "C"
