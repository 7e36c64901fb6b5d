// Paged cache: quantizing rows into their pages, and reading them back.
//
// Both move bytes: per token and head a write reads 4*d bytes and stores
// d*b/4 + d/4, a read the reverse; a handful of operations per element, so
// HBM should bound them.  Measured on a GB300, 32768 tokens of 8 heads of 128 at 4
// bits (176 MB): write 53 us = 3.3 TB/s, 49 % of the copy rate, with 3 of 4
// instructions issued a clock (54 us at 2 bits, 49 at 8); read 33 us = 5.3 TB/s,
// 78 % (29 us, 81 %, at 2 bits, 34 at 8); 48930 tokens at 8 bits, 50 us = 93 %.
#include "kvq_paged.cuh"

namespace kvq {
namespace {

constexpr int kIoThreads = 256;
constexpr int kManyRows = 8192;
constexpr int kIoBatch = 2;  // pairs of loads of a warp in flight

// The sequence of row t, found by the whole warp (32 candidates a round), or -1
// for padding (also for a cu_tokens array that does not increase around t).
__device__ __forceinline__ int warp_seq_of_row(const Paged &p, int64_t t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = p.B;  // the largest b with cu[b] <= t
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, b = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, b < hi && p.cu[b] <= t);
    if (le == 0) return -1;
    lo += (31 - __clz(le)) * step;
    hi = min(lo + step, hi);
  }
  return (t >= p.cu[lo] && t < p.cu[lo + 1]) ? lo : -1;
}

// The two halves of a word as fp32.
template <int BF16>
__device__ __forceinline__ float2 unpack2(uint32_t u) {
  if (BF16) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}
// Two values rounded once to the 16-bit type, x0 in the low half.
template <int BF16>
__device__ __forceinline__ uint32_t pack2(float x0, float x1) {
  if (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  const __half2 h = __floats2half2_rn(x0, x1);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Packed minimum and maximum; NaN where either side is.
template <int BF16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t d;
  if (BF16) asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <int BF16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t d;
  if (BF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// One 16-bit input as the stored form takes it: saturated, NaN as 0.
__device__ __forceinline__ float tame(float x) {
  return x == x ? fminf(fmaxf(x, -kPagedLimit), kPagedLimit) : 0.0f;
}

// x / (2^BITS - 1), rounded to nearest even as the IEEE division does: the
// product with the rounded reciprocal, corrected once by its remainder
// (Markstein's quotient; compared with the division for every mantissa of x and
// the three divisors).  For quotients in the normal range; a smaller one may
// differ in its last bit, far below what the fp16 scale keeps.
template <int BITS>
__device__ __forceinline__ float over_top(float x) {
  constexpr float kTop = (float)((1 << BITS) - 1), kInv = 1.0f / kTop;
  const float q = __fmul_rn(x, kInv);
  return fmaf(fmaf(-kTop, q, x), kInv, q);
}

// clamp(rint((x - zero) / scale)) by the IEEE division.
template <int BITS>
__device__ __forceinline__ float careful_code(float x, float zero, float scale) {
  const float r = scale == 0.0f ? 0.0f : rintf(__fdiv_rn(__fsub_rn(x, zero), scale));
  return fminf(fmaxf(r, 0.0f), (float)((1 << BITS) - 1));
}

// A half warp (d = 128) or quarter warp (d = 64) holds the row of one head,
// lane l its channels 8*l .. 8*l + 7 (w): group l / 4, quarter j = l % 4 of the
// key layout, eighths 2*j and 2*j + 1 of the value layout.
//
// What bounds it is the instructions per element (22 lane operations, where HBM
// would leave time for about 14), so: minima and maxima on packed pairs; one reciprocal
// per group; rint by adding 1.5 * 2^23 in the fma that forms the quotient; codes
// put together as integer sums.  The hardware reciprocal is within 2^-23 of
// 1 / scale and the IEEE quotient within 2^-24 of the true one, so for quotients
// below 2^8 + 1 the two are less than 2^-14 apart (2^-18 below 2^4 + 1), and the
// integer is the same for both unless the quotient lies within kGuard = 2^-12
// (2^-16 for 2 and 4 bits, so that one warp in a hundred sees one) of a
// half-integer.
// Threads that see such a quotient, or a scale under 2^-13 (where its own
// rounding could pass the code range), go through the division; groups with
// inputs to tame are tamed first.
template <int D, int BITS, int BF16, bool VALUE>
__device__ __forceinline__ void quantize_row(uint4 w4, int l, uint8_t *codes, __half *stats) {
  constexpr int NG = D / kPagedGroup;
  constexpr unsigned kAll = 0xffffffffu;
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23 = 0x4b400000
  constexpr float kGuard = BITS == 8 ? kTieGuard : kTieGuard / 16.0f;
  constexpr uint32_t kMagicBits = 0x4b400000u, kSign = 0x80008000u;
  uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
  float mn, mx;
  auto ends = [&]() {  // (-min, max) of the group, packed
    const uint32_t hi = max2<BF16>(max2<BF16>(w[0], w[1]), max2<BF16>(w[2], w[3]));
    const uint32_t lo = min2<BF16>(min2<BF16>(w[0], w[1]), min2<BF16>(w[2], w[3])) ^ kSign;
    uint32_t mm = max2<BF16>(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
    mm = max2<BF16>(mm, __shfl_xor_sync(kAll, mm, 1));
    mm = max2<BF16>(mm, __shfl_xor_sync(kAll, mm, 2));
    const float2 e = unpack2<BF16>(mm);
    mn = -e.x, mx = e.y;
  };
  ends();
  if (__any_sync(kAll, !(mx <= kPagedLimit && mn >= -kPagedLimit))) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = unpack2<BF16>(w[i]);
      w[i] = pack2<BF16>(tame(x.x), tame(x.y));
    }
    ends();
  }
  const __half s16 = __float2half_rn(over_top<BITS>(__fsub_rn(mx, mn)));
  const __half z16 = __float2half_rn(canon_zero(mn));
  const float s = __half2float(s16), z = __half2float(z16);
  float inv;  // (a scale of 0 takes the careful way below)
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  // keys: even channels then odd ones; values: in order
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = VALUE ? w[i] : __byte_perm(w[2 * (i & 1)], w[2 * (i & 1) + 1], i < 2 ? 0x5410 : 0x7632);
  uint32_t y[8];  // kMagicBits + code
  float far = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack2<BF16>(v[i]);
    const float d0 = __fsub_rn(x.x, z), d1 = __fsub_rn(x.y, z);
    const float y0 = fmaf(d0, inv, kMagic), y1 = fmaf(d1, inv, kMagic);
    far = fmaxf(far, fmaxf(fabsf(fmaf(d0, inv, kMagic - y0)), fabsf(fmaf(d1, inv, kMagic - y1))));
    y[2 * i] = __float_as_uint(y0);
    y[2 * i + 1] = __float_as_uint(y1);
  }
  if (far > 0.5f - kGuard || s < 1.0f / 8192.0f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = unpack2<BF16>(v[i]);
      y[2 * i] = __float_as_uint(careful_code<BITS>(x.x, z, s) + kMagic);
      y[2 * i + 1] = __float_as_uint(careful_code<BITS>(x.y, z, s) + kMagic);
    }
  }
  // four codes of BITS bits in a word (the magic numbers taken out again)
  constexpr uint32_t kFour =
      kMagicBits * (1u + (1u << BITS) + (1u << 2 * BITS) + (1u << 3 * BITS));
  auto four = [&](int k) {
    return y[k] + (y[k + 1] << BITS) + (y[k + 2] << 2 * BITS) + (y[k + 3] << 3 * BITS) - kFour;
  };
  const uint32_t lo = four(0), hi = four(4);

  const int grp = l >> 2, j = l & 3, e = grp & 1, h = grp >> 1;
  // Key words: pair k (channels 2k, 2k+1) at bit k*BITS of each 16-bit half.
  // Value words: this group's channels at bits i*BITS of half e, so the two
  // lanes of a pair of groups swap one eighth each and hold a full word.
  uint32_t a = lo, b = hi;  // what goes to the low halves and to the high halves
  if (VALUE) {
    const uint32_t got = __shfl_xor_sync(kAll, e ? lo : hi, 4);
    a = e ? got : lo;
    b = e ? hi : got;
  }
  if (BITS == 8) {
    const uint2 word = make_uint2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
    uint8_t *dst = VALUE ? codes + (2 * j + e) * (D / 8) + h * 8 : codes + j * (D / 4) + grp * 8;
    *reinterpret_cast<uint2 *>(dst) = word;
  } else if (BITS == 4) {
    uint8_t *dst = VALUE ? codes + (2 * j + e) * (D / 16) + h * 4 : codes + j * (D / 8) + grp * 4;
    *reinterpret_cast<uint32_t *>(dst) = a | (b << 16);
  } else if (VALUE && D == 64) {
    // one pair of groups: the eighth is two bytes
    *reinterpret_cast<uint16_t *>(codes + (2 * j + e) * 2) = (uint16_t)(a | (b << 8));
  } else {
    // 2 bits: a word holds two groups (keys) or two pairs of groups (values)
    const int part = VALUE ? h : e;
    const uint32_t word = (a | (b << 16)) << (8 * part);
    const uint32_t other = __shfl_xor_sync(kAll, word, VALUE ? 8 : 4);
    uint8_t *dst = VALUE ? codes + (2 * j + e) * (D / 32) : codes + j * (D / 16) + h * 4;
    if (part == 0) *reinterpret_cast<uint32_t *>(dst) = word | other;
  }
  if (j < 2) stats[grp + NG * j] = j ? z16 : s16;
}

// One warp per row and group of heads: a warp instruction covers the keys, and
// the next the values, of two heads (d = 128) or of four (d = 64); kIoBatch of
// those pairs in flight.
template <int D, int BITS, int BF16>
__global__ void __launch_bounds__(kIoThreads)
paged_write_kernel(const __grid_constant__ Paged p, const uint16_t *k, int64_t ks,
                   const uint16_t *v, int64_t vs) {
  constexpr int LR = D / 8;      // lanes of one row
  constexpr int HW = 32 / LR;    // heads per warp instruction
  constexpr int RB = D * BITS / 8, SB = 4 * D / kPagedGroup;
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * (kIoThreads / 32) + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const int l = lane % LR;
  const int b = warp_seq_of_row(p, t);
  if (b < 0) return;
  const int64_t pos = row_position(p, b, t);
  if (pos < 0) return;
  k += t * ks + 8 * l;
  v += t * vs + 8 * l;
  // (lanes past the last head repeat it and store the same bytes as the lanes
  // that hold it; every exit is the whole warp's)
  const int row = (int)(pos & (kAtom - 1)), head_bytes = (int)p.head_bytes;
  const int stat_at = 2 * kAtom * RB + row * (SB - RB);
  uint8_t *atom = nullptr;
  for (int h0 = blockIdx.y * kIoBatch * HW; h0 < p.H; h0 += gridDim.y * kIoBatch * HW) {
    const int hl = h0 + lane / LR;
    uint4 wk[kIoBatch], wv[kIoBatch];
#pragma unroll
    for (int i = 0; i < kIoBatch; ++i)
      if (h0 + i * HW < p.H) {
        const int h = min(hl + i * HW, p.H - 1);
        wk[i] = __ldg(reinterpret_cast<const uint4 *>(k + h * D));
        wv[i] = __ldg(reinterpret_cast<const uint4 *>(v + h * D));
      }
    if (!atom) {
      atom = atom_of(p, b, pos);
      if (!atom) return;
      atom += row * RB;
    }
#pragma unroll
    for (int i = 0; i < kIoBatch; ++i) {
      if (h0 + i * HW >= p.H) break;
      uint8_t *at = atom + (int64_t)min(hl + i * HW, p.H - 1) * head_bytes;
      quantize_row<D, BITS, BF16, false>(wk[i], l, at, reinterpret_cast<__half *>(at + stat_at));
      quantize_row<D, BITS, BF16, true>(wv[i], l, at + kAtom * RB,
                                        reinterpret_cast<__half *>(at + stat_at + kAtom * SB));
    }
  }
}

// One warp per row and group of heads: eight lanes to a head, four for the
// quarters of the key row, four for pairs of eighths of the value row, 32 or 16
// channels each; four heads per warp instruction, kReadBatch of those in
// flight.
constexpr int kReadBatch = 2;
template <int D, int BITS, int BF16>
__global__ void __launch_bounds__(kIoThreads)
paged_read_kernel(const __grid_constant__ Paged p, uint16_t *k, uint16_t *v) {
  constexpr int RB = D * BITS / 8, SB = 4 * D / kPagedGroup, NG = D / kPagedGroup;
  constexpr int QB = RB / 4, QW = QB / 4;  // bytes, words of a quarter
  const int lane = threadIdx.x & 31, part = lane & 7, j = part & 3;
  const bool value = part >= 4;
  const int64_t t = (int64_t)blockIdx.x * (kIoThreads / 32) + (threadIdx.x >> 5);
  const int h0 = blockIdx.y * kReadBatch * 4;
  if (t >= p.T) return;
  const int b = warp_seq_of_row(p, t);
  if (b < 0) return;
  const int64_t pos = row_position(p, b, t);
  const uint8_t *atom = pos >= 0 ? atom_of(p, b, pos) : nullptr;
  const int row = (int)(pos & (kAtom - 1));
  const int code_at = (value ? kAtom * RB : 0) + row * RB + j * QB;
  const int stat_at = 2 * kAtom * RB + (value ? kAtom * SB : 0) + row * SB;
  uint16_t *out = (value ? v : k) + t * p.H * D + 8 * j;
  uint32_t w[kReadBatch][QW], st[kReadBatch][NG];
#pragma unroll
  for (int i = 0; i < kReadBatch; ++i) {
    const int h = h0 + 4 * i + (lane >> 3);
#pragma unroll
    for (int n = 0; n < NG; ++n) st[i][n] = 0;
#pragma unroll
    for (int n = 0; n < QW; ++n) w[i][n] = 0;
    if (h < p.H && atom) {
      const uint8_t *at = atom + h * p.head_bytes;
      if constexpr (QW % 4 == 0) {
#pragma unroll
        for (int n = 0; n < QW; n += 4) {
          const uint4 x = __ldg(reinterpret_cast<const uint4 *>(at + code_at + 4 * n));
          w[i][n] = x.x, w[i][n + 1] = x.y, w[i][n + 2] = x.z, w[i][n + 3] = x.w;
        }
      } else if constexpr (QW == 2) {
        const uint2 x = __ldg(reinterpret_cast<const uint2 *>(at + code_at));
        w[i][0] = x.x, w[i][1] = x.y;
      } else {
        w[i][0] = __ldg(reinterpret_cast<const uint32_t *>(at + code_at));
      }
      if constexpr (NG == 4) {
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(at + stat_at));
        st[i][0] = x.x, st[i][1] = x.y, st[i][2 % NG] = x.z, st[i][3 % NG] = x.w;
      } else {
        const uint2 x = __ldg(reinterpret_cast<const uint2 *>(at + stat_at));
        st[i][0] = x.x, st[i][1] = x.y;
      }
    }
  }
  // Codes of channels 8j + m, m = 0 .. 7, of group G: a key's are pairs (2k,
  // 2k + 1) at bit k*BITS of the two halves, a value's are bits i*BITS of half
  // G & 1 of its eighth.
  constexpr uint32_t kOne = (1u << BITS) - 1;
  constexpr float kBase = 8388608.0f;  // 2^23: a code in the low bits of this is itself
#pragma unroll
  for (int i = 0; i < kReadBatch; ++i) {
    const int h = h0 + 4 * i + (lane >> 3);
    if (h >= p.H) break;
#pragma unroll
    for (int G = 0; G < NG; ++G) {
      const float2 s2 = __half22float2(*reinterpret_cast<const __half2 *>(&st[i][G / 2]));
      const float2 z2 = __half22float2(*reinterpret_cast<const __half2 *>(&st[i][NG / 2 + G / 2]));
      const float s = G & 1 ? s2.y : s2.x, z = G & 1 ? z2.y : z2.x;
      uint32_t o[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        float x[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int c8 = 2 * m + u;
          const int kbit = (G * 4 + m) * BITS;
          uint32_t kw = w[i][kbit / 16] >> (kbit % 16 + 16 * u), vw;
          if (RB / 8 == 2) {
            vw = w[i][0] >> (16 * (c8 >> 2) + 8 * (G & 1) + (c8 & 3) * BITS);
          } else {
            const int vbit = ((G >> 1) * 4 + (c8 & 3)) * BITS;
            vw = w[i][((c8 >> 2) * (QW / 2) + vbit / 16) % QW] >> (vbit % 16 + 16 * (G & 1));
          }
          const uint32_t code = (value ? vw : kw) & kOne;
          x[u] = fmaf(__uint_as_float(code | 0x4b000000u) - kBase, s, z);
        }
        o[m] = pack2<BF16>(x[0], x[1]);
      }
      *reinterpret_cast<uint4 *>(out + (int64_t)h * D + G * 32) =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// A warp copies 4 KB of a page at a time, its lanes eight 16-byte vectors each, and
// reads the next piece's page numbers meanwhile.  HBM bounds it: 3400 pages of 80 KB,
// 557 MB in and out, 87.6 us = 6.4 TB/s, 94 % of the copy rate; 40000 pages 984 us = 6.7.
//
// The list ends at its first negative pair, which may stand anywhere and with any pairs
// behind it, so each block looks at every pair up to those it is copying, 2048 a turn,
// while its loads are on their way; what is stored is decided after that.  Blocks of 16
// warps, so that few read the list (pages of 768 bytes, 200000 of them: 101 us, 125 with
// 8 warps, 60 without a look); eight neighbouring pieces to a block, so that a short list
// is on all SMs (60 pages 3.1 us, 2.9 without a look).
constexpr int kCopyVecs = 8, kCopyBytes = 32 * 16 * kCopyVecs;
constexpr int kCopyThreads = 512, kCopyLook = 4, kCopyGroup = 8, kCopyGroups = 2;
static_assert(kCopyGroup * kCopyGroups * 32 == kCopyThreads, "a warp a piece");
__global__ void __launch_bounds__(kCopyThreads, 2)
paged_copy_kernel(const __grid_constant__ Paged p, const int2 *copies, uint32_t n) {
  __shared__ uint32_t found;  // the least negative pair's number
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t pieces = (uint32_t)((p.page_bytes + kCopyBytes - 1) / kCopyBytes);
  // the warp's piece, as pair k and place `off` in its page, and the block's first one
  const uint32_t first = blockIdx.x * kCopyGroup, row = gridDim.x * kCopyGroup;
  const uint32_t u = first + warp / kCopyGroup * row + warp % kCopyGroup;
  uint32_t k = u / pieces, off = u % pieces, k0 = first / pieces, off0 = first % pieces;
  const uint32_t step = row * kCopyGroups, step_k = step / pieces, step_off = step % pieces;
  auto advance = [&](uint32_t &kk, uint32_t &oo) {
    kk += step_k;
    oo += step_off;
    if (oo >= pieces) oo -= pieces, ++kk;
  };
  if (tid == 0) found = n;
  auto pair_at = [&](uint32_t i) { return i < n ? __ldg(copies + i) : make_int2(-1, -1); };
  uint32_t seen = 0, end = n;  // pairs looked at; where the list ends, as far as is known
  int2 c = pair_at(k);
  do {
    const bool pages = c.x >= 0 && c.x < p.n_pages && c.y >= 0 && c.y < p.n_pages;
    const int64_t at = (int64_t)off * kCopyBytes + lane * 16;
    const uint8_t *src = p.pages + c.x * p.page_bytes + at;
    uint8_t *dst = p.pages + c.y * p.page_bytes + at;
    int left = pages && c.x != c.y ? (int)min(p.page_bytes - at, (int64_t)kCopyBytes) : 0;
    uint4 v[kCopyVecs];
#pragma unroll
    for (int i = 0; i < kCopyVecs; ++i)
      if (i * 512 < left) v[i] = *reinterpret_cast<const uint4 *>(src + i * 512);
    const uint32_t mine = k;
    advance(k, off);
    const int2 next = pair_at(k);
    // (the same for the whole block; no warp's pair is behind k0 + step_k + 1)
    const uint32_t need = min(k0 + step_k + 2, n);
    while (seen < need && end == n) {
      uint32_t least = n;
#pragma unroll
      for (int i = kCopyLook - 1; i >= 0; --i) {
        const uint32_t j = seen + i * kCopyThreads + tid;
        if (j < n && __ldg(&copies[j].x) < 0) least = j;
      }
      if (__syncthreads_or(least < n)) {
        if (least < n) atomicMin(&found, least);
        __syncthreads();
        end = found;
      }
      seen += kCopyLook * kCopyThreads;
    }
    if (mine < end) {
      if (!pages && lane == 0) paged_error(p, KVQ_EPAGE);
#pragma unroll
      for (int i = 0; i < kCopyVecs; ++i)
        if (i * 512 < left) *reinterpret_cast<uint4 *>(dst + i * 512) = v[i];
    }
    c = next;
    advance(k0, off0);
  } while (k0 < end);
}

// Warps of a call: rows x groups of `per` heads.
dim3 io_grid(const Paged &p, int per) {
  return dim3((unsigned)((p.T + kIoThreads / 32 - 1) / (kIoThreads / 32)),
              (unsigned)((p.H + per - 1) / per));
}

template <int D, int BITS>
cudaError_t write_as(const Paged &p, const void *k, int64_t ks, const void *v, int64_t vs,
                     cudaStream_t st) {
  dim3 grid = io_grid(p, kIoBatch * (32 / (D / 8)));
  // where the rows alone fill the GPU a warp takes all heads of its row, which
  // is found once then (8 heads, 4 bits: 32768 rows 53 us for 59, 2400 rows 7.4
  // for 6.8)
  if (p.T >= kManyRows) grid.y = 1;
  auto kern = p.bf16 ? paged_write_kernel<D, BITS, 1> : paged_write_kernel<D, BITS, 0>;
  kern<<<grid, kIoThreads, 0, st>>>(p, static_cast<const uint16_t *>(k), ks,
                                    static_cast<const uint16_t *>(v), vs);
  return cudaGetLastError();
}

template <int D, int BITS>
cudaError_t read_as(const Paged &p, void *k, void *v, cudaStream_t st) {
  const dim3 grid = io_grid(p, kReadBatch * 4);
  auto kern = p.bf16 ? paged_read_kernel<D, BITS, 1> : paged_read_kernel<D, BITS, 0>;
  kern<<<grid, kIoThreads, 0, st>>>(p, static_cast<uint16_t *>(k), static_cast<uint16_t *>(v));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_write(const Paged &p, const void *k, int64_t ks, const void *v,
                               int64_t vs, cudaStream_t st) {
  if (p.d == 128)
    return p.bits == 2   ? write_as<128, 2>(p, k, ks, v, vs, st)
           : p.bits == 4 ? write_as<128, 4>(p, k, ks, v, vs, st)
                         : write_as<128, 8>(p, k, ks, v, vs, st);
  return p.bits == 2   ? write_as<64, 2>(p, k, ks, v, vs, st)
         : p.bits == 4 ? write_as<64, 4>(p, k, ks, v, vs, st)
                       : write_as<64, 8>(p, k, ks, v, vs, st);
}

cudaError_t launch_paged_read(const Paged &p, void *k, void *v, cudaStream_t st) {
  if (p.d == 128)
    return p.bits == 2   ? read_as<128, 2>(p, k, v, st)
           : p.bits == 4 ? read_as<128, 4>(p, k, v, st)
                         : read_as<128, 8>(p, k, v, st);
  return p.bits == 2   ? read_as<64, 2>(p, k, v, st)
         : p.bits == 4 ? read_as<64, 4>(p, k, v, st)
                       : read_as<64, 8>(p, k, v, st);
}

cudaError_t launch_paged_copy(const Paged &p, const int32_t *copies, int64_t n, int num_sms,
                              cudaStream_t st) {
  // Two blocks an SM at a time.  Twice as many are faster where a block copies long for
  // each pair it looks at (3400 pages of 80 KB: 87.6 us, 91.5 with two), slower where it
  // does not (100000 pages of 5 KB: 162 us with two, 221 with four).
  const int64_t pieces = (p.page_bytes + kCopyBytes - 1) / kCopyBytes;
  const int64_t blocks = (n * pieces + kCopyGroup - 1) / kCopyGroup;
  const int64_t most = (int64_t)num_sms * (pieces >= 8 ? 4 : 2);
  paged_copy_kernel<<<(unsigned)(blocks < most ? blocks : most), kCopyThreads, 0, st>>>(
      p, reinterpret_cast<const int2 *>(copies), (uint32_t)n);
  return cudaGetLastError();
}

}  // namespace kvq
