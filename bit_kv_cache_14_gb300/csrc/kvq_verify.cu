// Verification of drafted tokens (include/kvq.h, kvq_verify_drafts).
//
// Row t of a sequence holds the target's logits x for the token after row t's, and
// the draft model's y.  With p = softmax(x / T), q = softmax(y / T), the drafted
// token c of the next row stays while u q(c) < p(c); at the first that does not,
// the next token is the largest max(p - q, 0)_i / e_i, behind the last draft the
// largest p_i / e_i, with the caller's exponential e (the smallest of exponentials
// of rates p_i is at i with probability p_i).
//
// Two launches.  Rows: a warp reads up to four pieces of 4 KB of a row (one where there
// are few) and leaves their maximum m and s = sum 2^((x - m) c), c = log2(e) / T, so each
// logit is read once; all rows are taken, since which draft is the first refused is known
// only afterwards.  Draw: the blocks of a sequence each join its rows' parts (16 bytes
// each: 256 bytes of a bf16 row of 131072 in parts of four pieces), decide, and race their
// share of the one row that is drawn from; shares are joined by a maximum over (score,
// lowest index), which has no order.  The draw's blocks come in as the rows' leave, look
// up their drafts' logits and call their noise into L2 before they wait for the parts.
//
// Large calls are bound by HBM, the draw also by its chain of loads.  Measured on a GB300
// (graph replay): 64 sequences of 4 drafts, bf16 logits of 131072 tokens and a draft
// model's, 185 MB: 43.7 us = 4.2 TB/s, 62 % of the copy rate (the draw reads 61 MB in 15
// us, 6 to 11 of them the race, the rest its chain and the join); 128 x 3 greedy, fp32,
// 65537 tokens: 26.9 us = 5.0 TB/s, 73 %.  Small ones by latency: 24 sequences, 50001
// tokens, no draft model: 13.2 us; one sequence, 32000 tokens: 8.6.  With one block a
// part, factors in 64 bits (which this GPU divides slowly) and single loads the first
// took 173 us.
#include <algorithm>

#include "kvq_paged.cuh"
#include "kvq_tc_common.cuh"

namespace kvq {
namespace {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int64_t kMaxRows = 65535;
constexpr int64_t kMaxVocab = 1 << 24;
constexpr float kMasked = -INFINITY;  // logits of probability 0; NaN is taken as one

struct VerifyArgs {
  const int32_t *cu, *tokens;
  const void *logits, *draft;
  int64_t stride, dstride, nstride;
  const float *temperature, *uniform, *noise;
  int32_t *out, *accepted, *dropped;
  float *logprobs;
  int32_t *status;
  unsigned long long *keys;  // [B], zero between calls
  int *tickets;              // [B], zero between calls
  float4 *parts;             // [2][T][parts]: maximum, sum, lowest index of the maximum
  int64_t T;
  int B, V, splits;
  int row_pieces, pieces, n_parts;  // pieces of a row, of a part; parts of a row
  int padded;  // rows that no sequence owns are written, too
};

__device__ __forceinline__ void verify_error(const VerifyArgs &a, int code) {
  atomicCAS(a.status, 0, code);
}

// The sequence of row t, found by the whole warp (32 candidates a round), or -1: exact
// where cu_tokens is in order, and nothing is made of it where it is not (the draw).
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
  return t >= a.cu[lo] && t < a.cu[lo + 1] ? lo : -1;
}

// The temperature of sequence b; 0: greedy (also for NaN).
__device__ __forceinline__ float temperature_of(const VerifyArgs &a, int b) {
  const float t = a.temperature ? a.temperature[b] : 0.0f;
  return t > 0.0f ? fminf(fmaxf(t, 0x1p-100f), 0x1p100f) : 0.0f;
}
// log2(e) / T in two parts (greedy rows: T = 1): a difference of logits is exact or
// nearly so, and its product keeps what one rounded factor would lose for every
// element alike.  Both are positive, so minus infinity times them stays that.
struct Factor {
  float hi, lo;
};
__device__ __forceinline__ Factor factor_of(float temperature) {
  constexpr float kHi = 1.4426950408889634f;
  constexpr float kLo = (float)(1.4426950408889634 - (double)kHi);
  static_assert(kLo > 0.0f, "the first part is rounded down");
  const float t = temperature > 0.0f ? temperature : 1.0f, hi = __fdiv_rz(kHi, t);
  return {hi, (fmaf(-hi, t, kHi) + kLo) / t};
}
// 2^((x - m) c)
__device__ __forceinline__ float weight(float x, float m, Factor c) {
  const float d = x - m;
  return exp2_approx(fmaf(d, c.hi, d * c.lo));
}

// Types: 0 fp16, 1 bf16, 2 fp32.
template <int TYPE>
struct Logit {
  static constexpr int kSize = TYPE == 2 ? 4 : 2;
  static constexpr int kVec = 16 / kSize;  // of a 16-byte vector
  static constexpr float kMost = TYPE == 0 ? 65504.0f : TYPE == 1 ? 3.3895314e38f : 3.4028235e38f;
};
// A logit as the operator takes it: NaN masked, plus infinity the largest number.
template <int TYPE>
__device__ __forceinline__ float tame(float x) {
  return fminf(fmaxf(x, kMasked), Logit<TYPE>::kMost);
}
// ... and a word of them.
template <int TYPE>
__device__ __forceinline__ uint32_t tame_word(uint32_t w) {
  if (TYPE == 0) {
    asm("max.f16x2 %0, %0, %1;" : "+r"(w) : "r"(0xfc00fc00u));
    asm("min.f16x2 %0, %0, %1;" : "+r"(w) : "r"(0x7bff7bffu));
  } else if (TYPE == 1) {
    asm("max.bf16x2 %0, %0, %1;" : "+r"(w) : "r"(0xff80ff80u));
    asm("min.bf16x2 %0, %0, %1;" : "+r"(w) : "r"(0x7f7f7f7fu));
  } else {
    w = __float_as_uint(tame<2>(__uint_as_float(w)));
  }
  return w;
}
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
  return tame<TYPE>(x);
}
// How many elements before the row's first its first 16-byte vector begins.
template <int TYPE>
__device__ __forceinline__ int lead_of(const void *row) {
  return (int)((uintptr_t)row & 15) / Logit<TYPE>::kSize;
}

// The larger elements of two words.
template <int TYPE>
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
  if (TYPE == 0) asm("max.f16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
  else if (TYPE == 1) asm("max.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
  else a = __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  return a;
}
// The word's two elements (fp32: the word twice).
template <int TYPE>
__device__ __forceinline__ float2 both(uint32_t w) {
  if (TYPE == 0) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
  if (TYPE == 1) return make_float2(bf16_lo(w), bf16_hi(w));
  return make_float2(__uint_as_float(w), __uint_as_float(w));
}

// ---- rows -------------------------------------------------------------------
// A warp a unit: `pieces` pieces of a row of one model, a piece being kVectors 16-byte
// vectors a lane, vector i of lane l its vector 32 * i + l.  What bounds it is HBM, if
// the instructions a logit stay few: packed pairs for taming and the maximum, pairs of
// fp32 for differences, products and sums, one exponential a logit.  Vectors that the
// row's ends cut are left out there; their up to seven logits are taken one by one.
constexpr int kVectors = 8;
template <int TYPE>
__global__ void __launch_bounds__(kVerifyThreads, 4)
verify_rows_kernel(const __grid_constant__ VerifyArgs a) {
  using L = Logit<TYPE>;
  constexpr int N = L::kVec, kPiece = kVectors * 32;  // vectors
  const int lane = threadIdx.x & 31;
  // (in this order: where the draw's blocks start, everything before the call is done)
  grid_dep_wait();
  grid_dep_trigger();
  const uint32_t unit = blockIdx.x * kVerifyWarps + (threadIdx.x >> 5);
  const uint32_t line = unit / (uint32_t)a.n_parts;
  const int part = (int)(unit - line * (uint32_t)a.n_parts);
  const bool model = line >= a.T;
  const int64_t t = model ? line - a.T : line;
  if (line >= (a.draft ? 2 : 1) * a.T) return;
  const int b = sequence_of(a, t);
  if (b < 0) return;
  const float temperature = temperature_of(a, b);
  // a draft row is looked at where there is a draft to sample against
  if (model && (temperature == 0.0f || t + 1 == a.cu[b + 1])) return;
  const Factor c = factor_of(temperature);
  const uint64_t chi = pair64(c.hi, c.hi), clo = pair64(c.lo, c.lo);
  const char *row = static_cast<const char *>(model ? a.draft : a.logits) +
                    t * (model ? a.dstride : a.stride) * L::kSize;
  const int lead = lead_of<TYPE>(row);
  // vector v holds elements v * N - lead .. + N - 1
  const uint4 *vec = reinterpret_cast<const uint4 *>(row - lead * L::kSize);
  constexpr uint32_t kNone = TYPE == 0 ? 0xfc00fc00u : TYPE == 1 ? 0xff80ff80u : 0xff800000u;

  float m = kMasked, s = 0.0f;
  int first = 0x7fffffff;  // greedy rows: the lane's lowest index of its maximum
  auto take = [&](int v0, auto whole) {
    uint32_t w[kVectors][4];
#pragma unroll
    for (int i = 0; i < kVectors; ++i) {
      const int e0 = (v0 + i * 32) * N - lead;
      if (decltype(whole)::value || (e0 >= 0 && e0 + N <= a.V)) {
        const uint4 v = __ldg(vec + v0 + i * 32);
        w[i][0] = v.x, w[i][1] = v.y, w[i][2] = v.z, w[i][3] = v.w;
      } else {
        w[i][0] = w[i][1] = w[i][2] = w[i][3] = kNone;
      }
    }
    uint32_t most = kNone;
#pragma unroll
    for (int i = 0; i < kVectors; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        w[i][k] = tame_word<TYPE>(w[i][k]);
        most = larger<TYPE>(most, w[i][k]);
      }
    const float2 ends = both<TYPE>(most);
    const float top = fmaxf(m, fmaxf(ends.x, ends.y));
    if (temperature == 0.0f && top > m) {
      first = 0x7fffffff;
#pragma unroll
      for (int i = kVectors - 1; i >= 0; --i)
#pragma unroll
        for (int k = 3; k >= 0; --k) {
          const float2 x = both<TYPE>(w[i][k]);
          const int e = (v0 + i * 32) * N - lead + k * (4 / L::kSize);
          if (TYPE != 2 && x.y == top) first = e + 1;
          if (x.x == top) first = e;
        }
    }
    const float ref = top > kMasked ? top : 0.0f;
    const uint64_t nm = pair64(-ref, -ref);
    uint64_t s2 = 0;
    auto add = [&](uint64_t x) {
      const uint64_t d = add2(x, nm);
      const float2 e = unpair64(fma2(d, chi, mul2(d, clo)));
      s2 = add2(s2, pair64(exp2_approx(e.x), exp2_approx(e.y)));
    };
#pragma unroll
    for (int i = 0; i < kVectors; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (TYPE == 2) {
          if (k & 1) add(pair64(__uint_as_float(w[i][k - 1]), __uint_as_float(w[i][k])));
        } else {
          const float2 x = both<TYPE>(w[i][k]);
          add(pair64(x.x, x.y));
        }
      }
    const float2 e = unpair64(s2);
    s = (m > kMasked ? s * weight(m, top, c) : 0.0f) + (e.x + e.y);
    m = top;
  };
  const int p1 = min((part + 1) * a.pieces, a.row_pieces);
  for (int piece = part * a.pieces; piece < p1; ++piece) {
    const int v0 = piece * kPiece;
    if (v0 * N >= lead && (v0 + kPiece) * N - lead <= a.V)
      take(v0 + lane, std::true_type());
    else
      take(v0 + lane, std::false_type());
  }
  // the row's ends: what the last vector holds of it, where that is cut, and (by
  // another lane) what vector 0 does, where that begins before the row
  const int last = (a.V - 1 + lead) / N;
  const bool cut = (a.V + lead) % N != 0;
  int e0 = 0, e1 = 0;
  if (cut && part == last / kPiece / a.pieces && lane == last % 32)
    e0 = max(last * N - lead, 0), e1 = a.V;
  else if (lead > 0 && part == 0 && lane == (last + 1) % 32 && !(cut && last == 0))
    e1 = min(N - lead, a.V);
  for (int e = e0; e < e1; ++e) {
    const float x = load_logit<TYPE>(row, e);
    if (x > m) {
      s = s * weight(m, x, c) + 1.0f;
      m = x;
      first = e;
    } else if (x > kMasked) {
      s += weight(x, m, c);
      if (x == m) first = min(first, e);
    }
  }
  float top = m;
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  s = m > kMasked ? s * weight(m, top, c) : 0.0f;
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  first = __reduce_min_sync(0xffffffffu, m == top ? first : 0x7fffffff);
  if (lane == 0)
    a.parts[((int64_t)model * a.T + t) * a.n_parts + part] =
        make_float4(top, s, __int_as_float(first), 0.0f);
}

// ---- draw -------------------------------------------------------------------
// Maximum, sum and lowest index of the maximum of a row, by the whole warp, in a
// fixed order.
struct Row {
  float m, s;
  int at;
};
__device__ __forceinline__ Row join_row(const VerifyArgs &a, int model, int64_t t, Factor c) {
  const int lane = threadIdx.x & 31;
  const float4 *p = a.parts + ((int64_t)model * a.T + t) * a.n_parts;
  Row r = {kMasked, 0.0f, 0x7fffffff};
#pragma unroll 2
  for (int i = lane; i < a.n_parts; i += 32) {
    const float4 v = __ldcg(p + i);
    if (v.x > r.m) {
      r.s = r.s * weight(r.m, v.x, c) + v.y;
      r.m = v.x;
      r.at = __float_as_int(v.z);
    } else if (v.x > kMasked) {
      r.s += v.y * weight(v.x, r.m, c);
    }
  }
  float m = r.m;
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float s = r.m > kMasked ? r.s * weight(r.m, m, c) : 0.0f;
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int at = __reduce_min_sync(0xffffffffu, r.m == m ? r.at : 0x7fffffff);
  return {m, s, at};
}

// Natural logarithm of a token's probability: logit x in a row of maximum m, sum s.
__device__ __forceinline__ float log_probability(float x, const Row &r, float temperature) {
  return (x - r.m) / (temperature > 0.0f ? temperature : 1.0f) - logf(r.s);
}

// u q(c) < p(c), as u s_p < 2^(tp - tq) s_q with the exponent in two parts.
__device__ __forceinline__ bool stays(float u, float x, const Row &p, float y, const Row &q,
                                      bool model, Factor c) {
  if (!(x > kMasked)) return false;  // p(c) = 0
  if (model && !(y > kMasked)) return true;  // q(c) = 0 < p(c)
  if (u == 0.0f) return true;
  const float dp = x - p.m, dq = model ? y - q.m : 0.0f;
  const float hp = dp * c.hi, hq = dq * c.hi;
  const float lp = fmaf(dp, c.hi, -hp) + dp * c.lo, lq = fmaf(dq, c.hi, -hq) + dq * c.lo;
  // hp - hq and what its rounding loses
  const float h = hp - hq, back = h - hp, lost = (hp - (h - back)) + (-hq - back);
  // a clamped exponent decides: the sums lie in [1, 2^24]
  const float k = rintf(fminf(fmaxf(h, -400.0f), 400.0f));
  const float f = exp2f(fabsf(h) < 400.0f ? (h - k) + (lost + (lp - lq)) : 0.0f);
  // both sides times 2^100, so that small numbers stay normal ones
  return u * 0x1p100f * p.s < ldexpf(f * (model ? q.s : 1.0f), (int)k + 100);
}

// 1 / e of the race: e below 2^-126 counts as that, NaN stays.
__device__ __forceinline__ float rate(float e) {
  float r;
  asm("max.NaN.f32 %0, %1, 0f00800000;\n rcp.approx.ftz.f32 %0, %0;" : "=&f"(r) : "f"(e));
  return r;
}

// Block (share, sequence).
constexpr int kSaved = 64;  // rows whose joined parts a block keeps
template <int TYPE>
__global__ void __launch_bounds__(kVerifyThreads, 4)
verify_draw_kernel(const __grid_constant__ VerifyArgs a) {
  using L = Logit<TYPE>;
  constexpr int N = L::kVec;
  __shared__ int stop, last, next;
  __shared__ Row saved[2][kSaved], row_p, row_q;
  __shared__ unsigned long long best[kVerifyWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.y, share = blockIdx.x;
  if (tid == 0) stop = 0x7fffffff;
  grid_dep_trigger();
  // Until the wait only the call's inputs are looked at (the rows' kernel passes its
  // own wait before this one starts), and nothing is written.
  const int r0 = a.cu[b], r1 = a.cu[b + 1], n = r1 - r0;
  // rows out of order anywhere, or outside the packed arrays: which sums belong to which
  // sequence is not known, and none is judged
  bool bad = a.cu[0] < 0 || a.cu[a.B] > a.T;
  for (int i = tid; i < a.B; i += kVerifyThreads) bad |= a.cu[i + 1] < a.cu[i];
  bad = __syncthreads_or(bad);
  // after the wait: rows that no sequence owns (where bad, all of them)
  auto unowned = [&]() {
    if (!a.padded || share != 0) return;
    const int64_t from = bad ? a.T : a.cu[0], to = bad ? 0 : a.cu[a.B];
    for (int64_t t = b * kVerifyThreads + tid; t < a.T; t += a.B * kVerifyThreads)
      if (t < from || t >= to) a.out[t] = -1, a.logprobs[t] = 0.0f;
  };
  if (bad || n == 0) {
    grid_dep_wait();
    unowned();
    if (share == 0 && tid == 0) {
      if (bad) verify_error(a, KVQ_EINVAL);
      a.accepted[b] = 0;
      a.dropped[b] = 0;
    }
    return;
  }
  const float temperature = temperature_of(a, b);
  const bool greedy = temperature == 0.0f, model = a.draft != nullptr && !greedy;
  const Factor c = factor_of(temperature);
  // the share's tokens
  const int per = ((a.V + a.splits - 1) / a.splits + 7) & ~7;
  const int i0 = min(share * per, a.V), i1 = min(i0 + per, a.V);
  const float *er = a.noise + b * a.nstride;
  if (!greedy)  // its noise comes into L2 meanwhile
    for (int i = i0 + tid * 32; i < i1; i += kVerifyThreads * 32)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(er + i));
  auto row_of = [&](int which, int64_t t) {
    return static_cast<const char *>(which ? a.draft : a.logits) +
           t * (which ? a.dstride : a.stride) * L::kSize;
  };
  // ---- the drafts that stay, a warp a draft
  bool waited = false;
  for (int i = warp; i < n; i += kVerifyWarps) {
    const int64_t t = r0 + i;
    const bool drafted = i < n - 1;
    const int token = drafted ? a.tokens[t + 1] : -1;
    const bool valid = token >= 0 && token < a.V;
    const bool test = valid && !greedy;
    const float x = test ? load_logit<TYPE>(row_of(0, t), token) : 0.0f;
    const float y = test && model ? load_logit<TYPE>(row_of(1, t), token) : 0.0f;
    const float u = test ? a.uniform[t] : 0.0f;
    if (!waited) grid_dep_wait();
    waited = true;
    const Row p = join_row(a, 0, t, c);
    Row q = {kMasked, 0.0f, 0};
    if (drafted && model) q = join_row(a, 1, t, c);
    if (lane == 0) {
      if (i < kSaved) saved[0][i] = p, saved[1][i] = q;
      if (drafted && !valid && share == 0) verify_error(a, KVQ_EINVAL);
      const bool ok = valid && (greedy ? p.at == token : stays(u, x, p, y, q, model, c));
      if (!ok) atomicMin(&stop, i);  // (the last row is the end anyway)
    }
  }
  if (!waited) grid_dep_wait();
  unowned();
  __syncthreads();
  const int kept = stop;
  const int64_t t = r0 + kept;
  const bool refused = kept < n - 1;
  if (kept >= kSaved && warp < 2) {
    const Row r = warp == 0 || (refused && model) ? join_row(a, warp, t, c)
                                                  : Row{kMasked, 0.0f, 0};
    if (lane == 0) *(warp == 0 ? &row_p : &row_q) = r;
  }
  if (kept >= kSaved) __syncthreads();
  const Row p = kept < kSaved ? saved[0][kept] : row_p;
  if (greedy && share != 0) return;
  // ---- the race over tokens [from, to) of the row.  Scores are taken times the sum
  // of p, so what is left of p is w_x - w_y s_p / s_q (equal rows leave exactly
  // nothing).  A thread's i only grows: of equal scores its lowest index stays.
  auto race = [&](int from, int to, bool rest) {
    const Row q = kept < kSaved ? saved[1][kept] : row_q;
    const int gone = refused && !model && rest ? a.tokens[t + 1] : -1;  // all of q
    rest = rest && refused && model && q.s > 0.0f;  // (a masked draft row takes nothing off)
    const float ratio = rest ? p.s / q.s : 0.0f;
    const char *xr = row_of(0, t), *yr = rest ? row_of(1, t) : xr;
    float score = 0.0f;
    uint32_t at = 0;
    auto single = [&](int i) {
      float w = weight(load_logit<TYPE>(xr, i), p.m, c);
      if (rest) w = fmaf(-weight(load_logit<TYPE>(yr, i), q.m, c), ratio, w);
      const float r = w * rate(__ldg(er + i));
      if (r > score && i != gone) score = r, at = (uint32_t)i;
    };
    // 16-byte vectors where the rows and the noise agree on where those begin
    const int lead = lead_of<TYPE>(xr), skip = (N - lead) % N;
    if (lead_of<TYPE>(yr) == lead && (((uintptr_t)(er + from + skip)) & 15) == 0) {
      // (from is a multiple of eight)
      const int v0 = min(from + skip, to), v1 = v0 + (to - v0) / N * N;
      if (tid < v0 - from) single(from + tid);
      const uint64_t chi = pair64(c.hi, c.hi), clo = pair64(c.lo, c.lo);
      const uint64_t np = pair64(-p.m, -p.m), nq = pair64(-q.m, -q.m);
      auto pairs = [&](uint4 v, uint64_t nm, float (&out)[N]) {  // weights of a vector
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < N; k += 2) {
          float2 x;
          if (TYPE == 2)
            x = make_float2(__uint_as_float(tame_word<TYPE>(w[k % 4])),
                            __uint_as_float(tame_word<TYPE>(w[(k + 1) % 4])));
          else
            x = both<TYPE>(tame_word<TYPE>(w[k / 2]));
          const uint64_t d = add2(pair64(x.x, x.y), nm);
          const float2 e = unpair64(fma2(d, chi, mul2(d, clo)));
          out[k] = exp2_approx(e.x);
          out[k + 1] = exp2_approx(e.y);
        }
      };
      // (the next vectors are on their way while these are worked on)
      uint4 x, y = make_uint4(0, 0, 0, 0);
      float4 f[N / 4];
      auto fetch = [&](int i) {
        if (i >= v1) return;
        x = __ldg(reinterpret_cast<const uint4 *>(xr + (int64_t)i * L::kSize));
        if (rest) y = __ldg(reinterpret_cast<const uint4 *>(yr + (int64_t)i * L::kSize));
#pragma unroll
        for (int k = 0; k < N / 4; ++k) f[k] = __ldg(reinterpret_cast<const float4 *>(er + i) + k);
      };
      fetch(v0 + tid * N);
#pragma unroll 1
      for (int i = v0 + tid * N; i < v1; i += kVerifyThreads * N) {
        float w[N], e[N];
#pragma unroll
        for (int k = 0; k < N; k += 4)
          e[k] = f[k / 4].x, e[k + 1] = f[k / 4].y, e[k + 2] = f[k / 4].z, e[k + 3] = f[k / 4].w;
        const uint4 cx = x, cy = y;
        fetch(i + kVerifyThreads * N);
        pairs(cx, np, w);
        if (rest) {
          float wy[N];
          pairs(cy, nq, wy);
#pragma unroll
          for (int k = 0; k < N; ++k) w[k] = fmaf(-wy[k], ratio, w[k]);
        }
        float top = score;
#pragma unroll
        for (int k = 0; k < N; ++k) {
          w[k] *= rate(e[k]);
          top = fmaxf(top, w[k]);  // (NaN is dropped)
        }
        if (top > score) {  // rare after the first few
#pragma unroll
          for (int k = 0; k < N; ++k)
            if (w[k] > score && i + k != gone) score = w[k], at = (uint32_t)(i + k);
        }
      }
      if (tid < to - v1) single(v1 + tid);
    } else {
#pragma unroll 4
      for (int i = from + tid; i < to; i += kVerifyThreads) single(i);
    }
    unsigned long long key =
        score > 0.0f ? (unsigned long long)__float_as_uint(score) << 32 | (0xffffffffu - at) : 0ull;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const unsigned long long other = __shfl_xor_sync(0xffffffffu, key, o);
      key = other > key ? other : key;
    }
    if (lane == 0) best[warp] = key;
    __syncthreads();
    if (tid == 0)
#pragma unroll
      for (int w = 1; w < kVerifyWarps; ++w) key = best[w] > key ? best[w] : key;
    return key;  // of thread 0: the block's
  };
  int token = greedy && p.m > kMasked ? p.at : -1;
  if (!greedy) {
    unsigned long long key = p.m > kMasked ? race(i0, i1, true) : 0;
    if (tid == 0) {
      if (key) atomicMax(&a.keys[b], key);
      __threadfence();
      last = atomicAdd(&a.tickets[b], 1) == a.splits - 1;
    }
    __syncthreads();
    if (!last) return;
    __shared__ unsigned long long won;
    if (tid == 0) {
      __threadfence();
      won = atomicExch(&a.keys[b], 0ull);
      a.tickets[b] = 0;
    }
    __syncthreads();
    key = won;
    // nothing was left of p (or only where the noise is NaN or infinite): p itself
    if (key == 0 && refused && p.m > kMasked) key = race(0, a.V, false);
    if (key) token = (int)(0xffffffffu - (uint32_t)key);
  }
  // ---- outputs
  if (tid == 0) {
    next = token;
    a.accepted[b] = kept;
    a.dropped[b] = n - 1 - kept;
  }
  __syncthreads();
  for (int i = warp; i < n; i += kVerifyWarps) {
    const int out = i < kept ? a.tokens[r0 + i + 1] : i == kept ? next : -1;
    float lp = 0.0f;
    if (out >= 0) {
      const Row r = i == kept ? p : i < kSaved ? saved[0][i] : join_row(a, 0, r0 + i, c);
      lp = log_probability(load_logit<TYPE>(row_of(0, r0 + i), out), r, temperature);
    }
    if (lane == 0) {
      a.out[r0 + i] = out;
      a.logprobs[r0 + i] = lp;
    }
  }
}

// Pieces of a row that begins `lead` elements into a 16-byte vector.
int pieces_of(int64_t vocab, int type, int lead) {
  const int64_t per = (int64_t)kVectors * 32 * (type == 2 ? 4 : 8);
  return (int)((vocab + lead + per - 1) / per);
}
int most_pieces(int64_t vocab, int type) { return pieces_of(vocab, type, type == 2 ? 3 : 7); }

// What must stay zero lies in front, whatever the call's sizes.
constexpr size_t kTicketsAt = (size_t)kMaxSeqs * 8, kPartsAt = kTicketsAt + (size_t)kMaxSeqs * 4;
size_t verify_bytes(int64_t T, int64_t V, int type) {
  return kPartsAt + (size_t)2 * T * most_pieces(V, type) * sizeof(float4);
}

template <int TYPE>
cudaError_t verify_as(const VerifyArgs &a, cudaStream_t st, int *launches) {
  *launches = 0;
  if (a.T > 0) {
    const int64_t units = (a.draft ? 2 : 1) * a.T * a.n_parts;  // (below 2^32)
    const unsigned grid = (unsigned)((units + kVerifyWarps - 1) / kVerifyWarps);
    const cudaError_t e = launch_dependent(verify_rows_kernel<TYPE>, grid,
                                           kVerifyThreads, 0, st, true, a);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  ++*launches;
  const dim3 grid((unsigned)a.splits, (unsigned)a.B);
  return launch_dependent(verify_draw_kernel<TYPE>, grid, kVerifyThreads, 0, st, a.T > 0, a);
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

int verify_drafts(bool padded, const kvq_draft_batch *batch, const void *logits, int64_t stride,
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
    if (out_tokens < batch->tokens + T && batch->tokens < out_tokens + T) return KVQ_EINVAL;
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
  a.padded = padded;
  a.B = batch->n_seqs;
  a.V = (int)V;
  // rows that all begin on a 16-byte vector have no lead
  const int size = batch->dtype == KVQ_F32 ? 4 : 2;
  const bool even = ((uintptr_t)logits & 15) == 0 && stride * size % 16 == 0 &&
                    (!a.draft || (((uintptr_t)draft_logits & 15) == 0 && draft_stride * size % 16 == 0));
  a.row_pieces = even ? pieces_of(V, batch->dtype, 0) : most_pieces(V, batch->dtype);
  // Four pieces a unit, whose start and end take as long as one, or as few as give each
  // of the 32 warps an SM holds a unit (64 x 5 rows of 131072 in units of 2, 4, 8: 45.1,
  // 43.4, 43.3 us; 128 x 4 fp32 rows of 65537: 29.3, 26.6, 28.1).
  const int64_t all = (a.draft ? 2 : 1) * T * a.row_pieces, warps = (int64_t)num_sms_cached() * 32;
  a.pieces = (int)std::min<int64_t>(std::max<int64_t>(all / warps, 1), 4);
  a.n_parts = (a.row_pieces + a.pieces - 1) / a.pieces;
  uint8_t *w = static_cast<uint8_t *>(ws);
  a.keys = reinterpret_cast<unsigned long long *>(w);
  a.tickets = reinterpret_cast<int *>(w + kTicketsAt);
  a.parts = reinterpret_cast<float4 *>(w + kPartsAt);
  // shares of 2048 tokens (a vector a thread), or larger ones, since every block of a
  // sequence decides about its drafts by itself
  const int64_t splits = (V + 2047) / 2048;
  const int64_t most = std::max<int64_t>(1, (int64_t)num_sms_cached() * 4 / a.B);
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
  return verify_drafts(false, batch, logits, stride, draft_logits, draft_stride, temperature,
                       uniform, noise, noise_stride, out_tokens, accepted, dropped, logprobs, ws,
                       ws_bytes, stream);
}

int kvq_verify_drafts_padded(const kvq_draft_batch *batch, const void *logits, int64_t stride,
                             const void *draft_logits, int64_t draft_stride,
                             const float *temperature, const float *uniform, const float *noise,
                             int64_t noise_stride, int32_t *out_tokens, int32_t *accepted,
                             int32_t *dropped, float *logprobs, void *ws, size_t ws_bytes,
                             void *stream) {
  return verify_drafts(true, batch, logits, stride, draft_logits, draft_stride, temperature,
                       uniform, noise, noise_stride, out_tokens, accepted, dropped, logprobs, ws,
                       ws_bytes, stream);
}

}  // extern "C"
