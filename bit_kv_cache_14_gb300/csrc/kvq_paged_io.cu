// Paged cache: quantizing rows into their pages, and reading them back.
//
// Both move bytes: per token and head a write reads 4*d bytes and stores
// d*b/4 + d/4, a read the reverse; a handful of operations per element, so
// HBM is what bounds them.
#include "kvq_paged.cuh"

namespace kvq {
namespace {

constexpr int kIoThreads = 256;

template <int BF16>
__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
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

// clamp(rint((x - zero) / scale)), with one reciprocal per group.  The hardware
// reciprocal is within 2^-23 of 1 / scale and each product or quotient is
// rounded within 2^-24, so for quotients up to 2^9 the product differs from
// the IEEE quotient by less than 2^-12 = kTieGuard: rint gives the same
// integer for both unless the product lies that close to a half-integer,
// where (and beyond 2^9, which the statistics exclude) the division decides.
template <int BITS>
__device__ __forceinline__ uint32_t paged_code(float x, float zero, float scale, float inv) {
  const float d = __fsub_rn(x, zero);
  float r = __fmul_rn(d, inv);
  const float f = __fsub_rn(r, floorf(r));
  if (!(fabsf(r) < 512.0f) || fabsf(__fsub_rn(f, 0.5f)) < kTieGuard)
    r = scale == 0.0f ? 0.0f : __fdiv_rn(d, scale);
  r = fminf(fmaxf(rintf(r), 0.0f), (float)((1 << BITS) - 1));
  return (uint32_t)r;
}

// A half warp (d = 128) or quarter warp (d = 64) holds the row of one head,
// lane l its channels 8*l .. 8*l + 7: group l / 4, quarter j = l % 4 of the
// key layout, eighths 2*j and 2*j + 1 of the value layout.
template <int D, int BITS>
__device__ __forceinline__ void quantize_row(const float (&xin)[8], int l, bool value,
                                             uint8_t *codes, __half *stats) {
  constexpr int NG = D / kPagedGroup;
  constexpr unsigned kAll = 0xffffffffu;
  float x[8], mn, mx;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // NaN -> 0; fminf / fmaxf return their other operand for a NaN
    const float c = xin[i] == xin[i] ? xin[i] : 0.0f;
    x[i] = fminf(fmaxf(c, -kPagedLimit), kPagedLimit);
    mn = i ? fminf(mn, x[i]) : x[i];
    mx = i ? fmaxf(mx, x[i]) : x[i];
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(kAll, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, o));
  }
  const __half s16 = __float2half_rn(
      __fdiv_rn(__fsub_rn(mx, mn), (float)((1 << BITS) - 1)));
  const __half z16 = __float2half_rn(canon_zero(mn));
  const float s = __half2float(s16), z = __half2float(z16);
  const float inv = recip_or_zero(s);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = paged_code<BITS>(x[i], z, s, inv);

  const int grp = l >> 2, j = l & 3, e = grp & 1, h = grp >> 1;
  // Key words: pair k (channels 2k, 2k+1) at bit k*BITS of each 16-bit half.
  // Value words: this group's channels at bits i*BITS of half e, so the two
  // lanes of a pair of groups swap one eighth each and hold a full word.
  uint32_t lo = 0, hi = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    lo |= (value ? c[k] : c[2 * k]) << (k * BITS);           // values: eighth 2j
    hi |= (value ? c[4 + k] : c[2 * k + 1]) << (k * BITS);   // values: eighth 2j + 1
  }
  // keys keep (lo, hi) = (even, odd channels); values trade with the lane of
  // the other group of the pair
  const uint32_t got = __shfl_xor_sync(kAll, e ? lo : hi, 4);
  const uint32_t a = value ? (e ? got : lo) : lo;  // what goes to the low halves
  const uint32_t b = value ? (e ? hi : got) : hi;  // and to the high halves
  if (BITS == 8) {
    const uint2 w = make_uint2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
    // 8 channels: two words
    uint8_t *dst = value ? codes + (2 * j + e) * (D / 8) + h * 8 : codes + j * (D / 4) + grp * 8;
    *reinterpret_cast<uint2 *>(dst) = w;
  } else if (BITS == 4) {
    uint8_t *dst = value ? codes + (2 * j + e) * (D / 16) + h * 4 : codes + j * (D / 8) + grp * 4;
    *reinterpret_cast<uint32_t *>(dst) = a | (b << 16);
  } else {
    // 2 bits: a word holds two groups (keys) or two pairs of groups (values)
    const int part = value ? h : e;
    uint32_t w = (a | (b << 16)) << (8 * part);
    const uint32_t other = __shfl_xor_sync(kAll, w, value ? 8 : 4);
    if (value && D == 64) {
      // one pair of groups: the eighth is two bytes
      *reinterpret_cast<uint16_t *>(codes + (2 * j + e) * 2) = (uint16_t)(a | (b << 8));
    } else if (part == 0) {
      uint8_t *dst = value ? codes + (2 * j + e) * (D / 32) : codes + j * (D / 16) + h * 4;
      *reinterpret_cast<uint32_t *>(dst) = w | other;
    }
  }
  if (j == 0) {
    stats[grp] = s16;
    stats[NG + grp] = z16;
  }
}

// One warp per (row, group of heads): a warp instruction covers the key and
// the value of one head (d = 128) or of two (d = 64).
template <int D, int BITS, int BF16>
__global__ void __launch_bounds__(kIoThreads)
paged_write_kernel(Paged p, const uint16_t *k, int64_t ks, const uint16_t *v, int64_t vs,
                   int head_groups) {
  constexpr int LR = D / 8;            // lanes of one row
  constexpr int HW = 32 / (2 * LR);    // heads per warp instruction
  constexpr int RB = D * BITS / 8, SB = 4 * D / kPagedGroup;
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * (kIoThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = item / head_groups;
  if (t >= p.T) return;
  const int h = (int)(item % head_groups) * HW + (lane / (2 * LR)) % HW;
  const bool value = (lane / LR) & 1;
  const int l = lane % LR;
  const int b = seq_of_row(p, t);
  if (b < 0) return;
  const int64_t pos = row_position(p, b, t);
  if (pos < 0) return;
  uint8_t *atom = atom_of(p, b, pos);
  if (!atom) return;
  // (every exit above is the whole warp's; lanes past the last head repeat it
  // and store the same bytes as the lanes that hold it)
  const int hh = h < p.H ? h : p.H - 1;
  const uint16_t *src = value ? v + t * vs : k + t * ks;
  const uint4 w = __ldg(reinterpret_cast<const uint4 *>(src + (int64_t)hh * D) + l);
  float x[8];
  unpack8<BF16>(w, x);
  atom += hh * p.head_bytes;
  const int row = (int)(pos % kAtom);
  uint8_t *codes = atom + (value ? kAtom * RB : 0) + row * RB;
  __half *stats = reinterpret_cast<__half *>(atom + 2 * kAtom * RB + (value ? kAtom * SB : 0) +
                                             row * SB);
  quantize_row<D, BITS>(x, l, value, codes, stats);
}

// Codes of 8 (keys: channels 32G + 8j ..; values: 4 channels of a pair of
// groups) at pair offset p0 of a segment, as bytes of `BITS`-bit values.
template <int BITS, int W>
__device__ __forceinline__ uint32_t code_at(const uint32_t *words, int pair, int e) {
  // W: bits of a half; units of 2W bits
  const int bit = pair * BITS;
  const int unit = bit / W, off = bit % W + W * e;
  if (W == 8) return (words[0] >> (16 * unit + off)) & ((1u << BITS) - 1);
  return (words[unit] >> off) & ((1u << BITS) - 1);
}

// Eight threads per token and head: four for the quarters of the key row, four
// for pairs of eighths of the value row, 32 or 16 channels each.
template <int D, int BITS, int BF16>
__global__ void __launch_bounds__(kIoThreads)
paged_read_kernel(Paged p, uint16_t *k, uint16_t *v) {
  constexpr int RB = D * BITS / 8, SB = 4 * D / kPagedGroup, NG = D / kPagedGroup;
  constexpr int QB = RB / 4;  // bytes of a quarter
  const int64_t i = (int64_t)blockIdx.x * kIoThreads + threadIdx.x;
  const int64_t th = i >> 3;
  const int64_t t = th / p.H;
  if (t >= p.T) return;
  const int h = (int)(th % p.H), part = (int)(i & 7), j = part & 3;
  const bool value = part >= 4;
  const int b = seq_of_row(p, t);
  if (b < 0) return;
  const int64_t pos = row_position(p, b, t);
  const uint8_t *atom = pos >= 0 ? atom_of(p, b, pos) : nullptr;
  uint16_t *dst = (value ? v : k) + (t * p.H + h) * D;
  if (!atom) {
    for (int g = 0; g < NG; ++g)
      *reinterpret_cast<uint4 *>(dst + g * 32 + j * 8) = make_uint4(0, 0, 0, 0);
    return;
  }
  atom += h * p.head_bytes;
  const int row = (int)(pos % kAtom);
  uint32_t w[QB / 4];
  const uint8_t *src = atom + (value ? kAtom * RB : 0) + row * RB + j * QB;
#pragma unroll
  for (int n = 0; n < QB / 4; ++n) w[n] = __ldg(reinterpret_cast<const uint32_t *>(src) + n);
  const __half *st = reinterpret_cast<const __half *>(atom + 2 * kAtom * RB +
                                                      (value ? kAtom * SB : 0) + row * SB);
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const float s = __half2float(st[g]), z = __half2float(st[NG + g]);
    uint32_t o[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      float x[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t c;
        if (value) {
          // channels 8j + 2m + u of group g: eighth 2j + m / 2
          constexpr int W = (D == 64 && BITS == 2) ? 8 : 16;
          const int c8 = 2 * m + u;
          if (W == 8) {
            const uint32_t half = (w[0] >> (16 * (c8 >> 2))) & 0xffffu;
            c = (half >> ((c8 & 3) * BITS + 8 * (g & 1))) & ((1u << BITS) - 1);
          } else {
            c = code_at<BITS, 16>(w + (c8 >> 2) * (QB / 8), (g >> 1) * 4 + (c8 & 3), g & 1);
          }
        } else {
          c = code_at<BITS, 16>(w, g * 4 + m, u);
        }
        x[u] = __fadd_rn(__fmul_rn((float)c, s), z);
      }
      o[m] = pack2<BF16>(x[0], x[1]);
    }
    *reinterpret_cast<uint4 *>(dst + g * 32 + j * 8) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

template <int D, int BITS>
cudaError_t write_as(const Paged &p, const void *k, int64_t ks, const void *v, int64_t vs,
                     cudaStream_t st) {
  const int hw = 32 / (2 * D / 8), groups = (p.H + hw - 1) / hw;
  const int64_t warps = p.T * groups;
  const unsigned grid = (unsigned)((warps + kIoThreads / 32 - 1) / (kIoThreads / 32));
  auto kern = p.bf16 ? paged_write_kernel<D, BITS, 1> : paged_write_kernel<D, BITS, 0>;
  kern<<<grid, kIoThreads, 0, st>>>(p, static_cast<const uint16_t *>(k), ks,
                                    static_cast<const uint16_t *>(v), vs, groups);
  return cudaGetLastError();
}

template <int D, int BITS>
cudaError_t read_as(const Paged &p, void *k, void *v, cudaStream_t st) {
  const int64_t threads = p.T * p.H * 8;
  const unsigned grid = (unsigned)((threads + kIoThreads - 1) / kIoThreads);
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

}  // namespace kvq
