// Paged cache: attention of sequences with few query rows (decode steps, a few
// speculated tokens): at most 16 rows per KV head, a row being one query token
// and head.
//
// What bounds it: the cache is read once, 2*(d*b/8 + d/8) bytes per token and
// head against 4*d operations per row, so HBM, if the instructions per code stay
// few enough (at 4 bits about 3.4 lane instructions per element keep up).
// Measured on a GB300: 64 sequences of 5500 to 16384 tokens, 32 query and 8 KV
// heads of 128, 4 bits: 200 us = 4.47 TB/s, 66 % of the copy rate; 8 bits, 16
// sequences of 8192: 64 us = 4.7 TB/s; 2 bits, 32 heads of their own, 8 x 4096:
// 48 us = 2.1 TB/s (twice the instructions a byte, and 11 us of fixed cost).
//
//  * Split: the tiles (two 16-token atoms, one at 8 bits) of all (sequence,
//    head) pairs form one list, cut into equal contiguous ranges, one per block;
//    inside a block the six or eight warps share each pair's tiles evenly.  Pairs that
//    end up in several blocks leave partials (m, l, o), and the block that
//    finishes a pair last joins them in block order, so results do not depend
//    on timing.
//  * A warp streams its tiles through a ring of shared-memory slots, one
//    cp.async.bulk per tile (contiguous by layout; one per atom where pages hold
//    one), 32 tiles' page numbers read at a time, ahead of their use.
//  * Keys: S^T[token][row] on mma.sync m16n8k16 with the raw codes as the A
//    operand: a masked code in the low ten bits of a half is the fp16
//    subnormal code * 2^(bit position) * 2^-24, exactly; the query operand
//    divides the position out.  The row permutation of the layout makes a
//    lane's share of a row one aligned vector.  Each group's sum is multiplied
//    by the token's scale in fp32; the zero points enter through one
//    m16n8k8 with the query's group sums in fp16 hi + lo.
//  * Values: O^T[channel][row] with the codes of two tokens joined by a PRMT as
//    the A operand and w = p * scale (fp16, one per group) as the B operand;
//    movmatrix turns the score fragment into it.  Zero points: sum p * zero in
//    fp32.
//    (Measured without the 17 products per atom: 139 us where the whole takes
//    199 and the copies alone 137.  No pipe is full meanwhile (2.2 of 4
//    instructions a clock, ALU 48 %, tensor 19 %): a tile is one chain of scores,
//    vote, exponentials, turns and products, and three warps a scheduler do not
//    cover its waits.)
//  * Softmax: a lazy reference per row, moved only when a score passes it by
//    more than 2 (log2 units), decided by one vote.  The reference also carries
//    E, the exponent of the largest value scale seen, and lies kRoom = 12 below,
//    so that w <= 2^14: where score and scale are the largest so far w is 2^11 or
//    more, and a w down to 2^-25 of that is a normal fp16 number; a smaller one
//    keeps an absolute 2^-36 of it.  (Without the room a warp's 1000 weights of
//    2^-26.5 beside one of 1 went to zero, and one saturated group of values cost
//    the others up to 2^-6 of their size.)
#include "kvq_paged.cuh"
#include "kvq_tc_common.cuh"

namespace kvq {

int debug_stall_limit();

namespace {

constexpr int kRowWaitLimit = 1 << 24;
constexpr float kNoRef = -1e30f;
constexpr int kRoom = 12;  // log2 units between the reference and the largest weight

struct RowsArgs {
  Paged p;
  const uint16_t *q;
  int64_t qs;
  uint16_t *out;
  float scale_log2;
  float *ws_ml;    // [2 * blocks][rows][2]
  float *ws_o;     // [2 * blocks][rows][d]
  int *ws_count;   // [blocks], zero between calls
  int few;         // sequences with more rows are not this kernel's
  int stall_limit;
  // Launched beside the chunk kernel of the same call: that kernel started after
  // everything before the call was done, and the two write different rows, so
  // this one does not wait for it to begin, only to end, and its completion
  // stands for both.
  bool beside;
};

template <int D, int BITS, int NT>
struct RowsCfg {
  // two blocks of 6 warps at 168 registers (8 warps at 128 spill: 217 us for 199),
  // or one of 8 at 255 for two row tiles (6 warps: 159 us for 127)
  static constexpr int kRowWarps = NT == 1 ? 6 : 8, kRowThreads = 32 * kRowWarps;
  static constexpr int RB = D * BITS / 8, SB = 4 * D / kPagedGroup, NG = D / kPagedGroup;
  static constexpr int AB = 2 * kAtom * (RB + SB);
  static constexpr int kBlocks = NT == 1 ? 2 : 1;  // per SM
  static constexpr int TA = AB > 4000 ? 1 : 2;  // atoms per tile
  static constexpr int TB = TA * AB;
  // ring slots per warp: about 150 KB in flight per SM
  static constexpr int S = NT == 1 ? (TB > 4000 ? 2 : TB > 3000 ? 3 : TB > 2000 ? 4 : 6)
                                   : (TB > 4000 ? 4 : TB > 3000 ? 6 : 8);
  static constexpr int ROWB = D * 4 + 16;  // padded row of the merge buffer
  static constexpr int off_merge = kRowWarps * S * TB;
  static constexpr int off_ml = off_merge + kRowWarps / 2 * 8 * NT * ROWB;
  static constexpr int off_bar = off_ml + kRowWarps / 2 * 8 * NT * 8;
  static constexpr int off_prefix = off_bar + kRowWarps * (S + 1) * 8;
  static constexpr int smem(int seqs) { return off_prefix + (seqs + 1) * 12; }
};

__device__ __forceinline__ uint32_t movm(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Products that start from zero.
__device__ __forceinline__ void mma1688(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, "
      "{%7,%7,%7,%7};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(b0), "f"(0.0f));
}
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// Codes at bit `off` of both halves of w: code * 2^(off % 8) * 2^-24 as fp16.
template <int BITS>
__device__ __forceinline__ uint32_t codes_at(uint32_t w, uint32_t w8, int off) {
  constexpr uint32_t kOne = (1u << BITS) - 1;
  return (off & 8 ? w8 : w) & ((kOne | kOne << 16) << (off & 7));
}

template <int N>
__device__ __forceinline__ void lds_words(const uint8_t *src, uint32_t (&w)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4 *>(src + 4 * i);
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2 *>(src);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t *>(src);
  }
}


// 64-bit quotients of numbers that are small almost always.
__device__ __forceinline__ int64_t div64(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}
// Where a unit index lies: sequence, head, offset inside the pair.
struct Place {
  int b, h, off, tiles;
};
__device__ __forceinline__ Place locate(const int64_t *prefix, int H, int64_t x, int b) {
  while (H * prefix[b + 1] <= x) ++b;
  Place u;
  u.b = b;
  u.tiles = (int)(prefix[b + 1] - prefix[b]);
  const int64_t r = x - H * prefix[b];
  u.h = (int)div64(r, u.tiles);
  u.off = (int)(r - (int64_t)u.h * u.tiles);
  return u;
}
__device__ __forceinline__ int seq_of_unit(const int64_t *prefix, int B, int H, int64_t x) {
  int lo = 0, hi = B;  // the last b with H * prefix[b] <= x and units of its own
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (H * prefix[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// The list is cut in one of two ways.  Joining a pair's parts costs about as
// much time as kPiece tiles take a block, so when every pair in pieces of about
// kPiece tiles gives no more pieces than there are blocks, each block takes one
// piece.  A longer list is cut evenly into ranges of U tiles, though not within
// kSnap tiles of a pair's border.
constexpr int kPiece = 16, kSnap = 4;
__device__ __forceinline__ int pieces_of(int64_t tiles) {
  return tiles == 0 ? 0 : max(1, (int)((tiles + kPiece / 2) / kPiece));
}
// First unit of block c under the even cut.
__device__ __forceinline__ int64_t border(const int64_t *prefix, int B, int H, int64_t total,
                                          int64_t U, int64_t c) {
  const int64_t x = c * U;
  if (x >= total) return total;
  if (x == 0) return 0;
  const Place u = locate(prefix, H, x, seq_of_unit(prefix, B, H, x));
  const int rest = u.tiles - u.off;
  if (u.off <= kSnap && u.off <= rest) return x - u.off;
  return rest <= kSnap ? x + rest : x;
}

template <int D, int BITS, int NT>
__global__ void __launch_bounds__(RowsCfg<D, BITS, NT>::kRowThreads, RowsCfg<D, BITS, NT>::kBlocks)
paged_rows_kernel(const __grid_constant__ RowsArgs a) {
  using C = RowsCfg<D, BITS, NT>;
  constexpr int RB = C::RB, SB = C::SB, NG = C::NG, S = C::S;
  constexpr int kRowWarps = C::kRowWarps, kRowThreads = C::kRowThreads;
  constexpr int TA = C::TA, TB = C::TB, kTile = TA * kAtom;
  constexpr int KW = RB / 16, VW = (RB / 8 + 3) / 4;  // words of a key quarter, a value eighth
  constexpr int kRows = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  // pairs this block shares with others: 0 one that began before it, 1 one that
  // goes on behind it
  struct Shared {
    int64_t pair0, pair1;
    int row0, rows, h, first, last, join;
  };
  __shared__ Shared shared_pair[2];
  int n_shared = 0;  // bit per entry
  const Paged &p = a.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, j = lane & 3;
  uint8_t *ring = smem + warp * S * TB;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::off_bar) + warp * (S + 1);
  int64_t *prefix = reinterpret_cast<int64_t *>(smem + C::off_prefix);
  int *pieces = reinterpret_cast<int *>(prefix + p.B + 1);

  grid_dep_trigger();
  if (lane <= S) bar_init(&bars[lane], 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");

  if (!a.beside) grid_dep_wait();
  // ---- the list of work: prefix[b] = tiles of one head of the sequences
  // before b that have between 1 and a.few rows
  {
    __shared__ int64_t warp_sum[kRowWarps];
    __shared__ int warp_pieces[kRowWarps];
    const int per = (p.B + kRowThreads - 1) / kRowThreads;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    int64_t sum = 0;
    int psum = 0;
    for (int b = b0; b < b1; ++b) {
      const int n = (int)((unsigned)p.cu[b + 1] - (unsigned)p.cu[b]);
      int64_t tiles = 0;
      if (bad_rows(p, b)) {
        if (blockIdx.x == 0) paged_error(p, KVQ_EINVAL);
      } else if (n > 0 && (int64_t)n * p.rg <= a.few) {
        const int64_t cap = p.width * p.page, len = p.lens[b];
        if (len > cap && blockIdx.x == 0) paged_error(p, KVQ_EPAGE);
        tiles = (min(len, cap) + kTile - 1) / kTile;
        if (tiles < 1) tiles = 1;  // rows that see nothing are written too
      }
      sum += tiles;
      psum = min(psum + pieces_of(tiles), 1 << 20);  // (beyond any grid)
      prefix[b + 1] = sum;
      pieces[b + 1] = psum;
    }
    int64_t inc = sum;
    int pinc = psum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
      const int pup = __shfl_up_sync(0xffffffffu, pinc, o);
      if (lane >= o) inc += up, pinc = min(pinc + pup, 1 << 20);
    }
    if (lane == 31) warp_sum[warp] = inc, warp_pieces[warp] = pinc;
    __syncthreads();
    int64_t before = inc - sum;
    int pbefore = pinc - psum;
    for (int w = 0; w < warp; ++w) before += warp_sum[w], pbefore += warp_pieces[w];
    for (int b = b0; b < b1; ++b) {
      prefix[b + 1] += before;
      pieces[b + 1] = min(pieces[b + 1] + pbefore, 1 << 20);
    }
    if (tid == 0) prefix[0] = 0, pieces[0] = 0;
    __syncthreads();
  }
  const int H = p.H;
  const int64_t total = H * prefix[p.B];
  const int64_t U = max(div64(total + gridDim.x - 1, gridDim.x), (int64_t)(2 * kSnap + 1));
  const bool by_piece = (int64_t)H * pieces[p.B] <= gridDim.x;
  int64_t x0, x1;
  int first_b, c_first = blockIdx.x, c_last = blockIdx.x;  // by_piece: the blocks of the pair
  if (by_piece) {
    const int c = blockIdx.x;
    if (c >= H * pieces[p.B]) {
      if (a.beside) grid_dep_wait();
      return;
    }
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (H * pieces[mid] <= c) lo = mid; else hi = mid;
    }
    first_b = lo;
    const int n = pieces[lo + 1] - pieces[lo], r = c - H * pieces[lo], k = r % n;
    const int64_t tiles = prefix[lo + 1] - prefix[lo];
    const int64_t pair = H * prefix[lo] + r / n * tiles;
    x0 = pair + (int64_t)k * kPiece;
    x1 = k == n - 1 ? pair + tiles : x0 + kPiece;
    c_first = c - k;
    c_last = c_first + n - 1;
  } else {
    x0 = border(prefix, p.B, H, total, U, blockIdx.x);
    x1 = border(prefix, p.B, H, total, U, blockIdx.x + 1);
    if (x0 >= x1) {
      if (a.beside) grid_dep_wait();
      return;
    }
    first_b = seq_of_unit(prefix, p.B, H, x0);
  }

  const uint64_t policy = l2_evict_first();
  bool dead = false;
  if (a.stall_limit > 0 && !bar_wait(&bars[S], 0, a.stall_limit)) {
    if (lane == 0) paged_error(p, KVQ_ETIMEOUT);
    dead = true;
  }

  // ---- queries of a pair: lane (g, j) holds, of row 8*nt + g, channels 32*G +
  // 8*j .. + 7.  Loaded ahead: the first pair's before its tiles, the next
  // pair's before this one's join.
  uint4 qraw[NT][NG];
  auto load_queries = [&](int64_t x, int b) {
    const Place u = locate(prefix, H, x, b);
    const int row0 = p.cu[u.b], rows = (p.cu[u.b + 1] - row0) * p.rg;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = 8 * nt + g;
      const uint16_t *src = a.q + (int64_t)(row0 + r / p.rg) * a.qs +
                            (int64_t)(u.h * p.rg + r % p.rg) * D + 8 * j;
#pragma unroll
      for (int G = 0; G < NG; ++G) {
        qraw[nt][G] = make_uint4(0, 0, 0, 0);
        if (r < rows) qraw[nt][G] = __ldg(reinterpret_cast<const uint4 *>(src + 32 * G));
      }
    }
  };
  load_queries(x0, first_b);

  // ---- fetch side: this warp's tiles of every segment of [x0, x1) in turn.
  // (fb, fh): the pair being fetched; [f0, f1): its tiles to come
  int64_t fx = x0;
  int fb = first_b, fh = 0, f0 = 0, f1 = 0, flen = 0;
  const int page_log = __ffs(p.page) - 1;
  // Page numbers: lane k holds those of tile pbase + k, the next 32 tiles' are
  // on their way.  (A pair that holds no tokens has one tile without a page: any
  // entry.)
  int pids[TA], pnext[TA], pbase = 0;
  auto read_pids = [&](int first, int (&to)[TA]) {
    const int t = (first + lane) * kTile;
    const int32_t *row = p.table + fb * p.width;
#pragma unroll
    for (int i = 0; i < TA; ++i) to[i] = -1;
    if (first + lane < f1) {
      to[0] = __ldg(row + (t >> page_log));
      if (TA == 2) {
        to[TA - 1] = to[0];
        if (p.page == kAtom) to[TA - 1] = t + kAtom < flen ? __ldg(row + (t >> page_log) + 1) : -1;
      }
    }
  };
  auto fetch_next = [&]() {  // moves to the next tile; false at the end
    if (f0 == f1) {
      do {
        if (fx >= x1) return false;
        const Place u = locate(prefix, H, fx, fb);
        const int n = (int)min((int64_t)(u.tiles - u.off), x1 - fx);
        fb = u.b, fh = u.h;
        f0 = u.off + n * warp / kRowWarps;
        f1 = u.off + n * (warp + 1) / kRowWarps;
        fx += n;
      } while (f0 == f1);
      flen = (int)min((int64_t)max(p.lens[fb], 0), p.width * p.page);
      pbase = f0;
      read_pids(f0, pids);
      read_pids(f0 + 32, pnext);
    } else if (f0 - pbase == 32) {
      pbase = f0;
#pragma unroll
      for (int i = 0; i < TA; ++i) pids[i] = pnext[i];
      read_pids(f0 + 32, pnext);
    }
    return true;
  };
  int issue_slot = 0, in_flight = 0, slot = 0;
  uint32_t phase = 0, skip = 0;  // skip: TA bits per slot, the atom's page does not exist
  bool more = fetch_next();
  auto issue = [&]() {
    const uint8_t *src[TA];
    uint32_t gone = 0;
    const int64_t in_page = fh * p.head_bytes +
                            (int64_t)(((f0 * kTile) & (p.page - 1)) / kAtom) * C::AB;
#pragma unroll
    for (int i = 0; i < TA; ++i) {
      const int64_t id = __shfl_sync(0xffffffffu, pids[i], f0 - pbase);
      if (id < 0 || id >= p.n_pages) gone |= 1u << i;
      src[i] = p.pages + id * p.page_bytes + in_page;
    }
    const bool paired = TA == 1 || p.page > kAtom;  // one copy for the tile
    ++f0;
    more = fetch_next();
    skip = (skip & ~(((1u << TA) - 1) << (TA * issue_slot))) | gone << (TA * issue_slot);
    if (lane == 0) {
      uint64_t *bar = &bars[issue_slot];
      const uint32_t dst = smem_u32(ring + issue_slot * TB);
      if (paired && !gone) {
        bulk_g2s_pred(true, smem_u32(bar), TB, dst, src[0], TB, policy);
      } else if (paired || gone == (1u << TA) - 1) {
        bar_expect_tx(bar, 0);
      } else {
        // pages of one atom: the copies that exist, one arrival
        const uint32_t both = gone ? C::AB : TB;
        if (!(gone & 1)) bulk_g2s_pred(true, smem_u32(bar), both, dst, src[0], C::AB, policy);
        if (!(gone & 2)) {
          if (gone & 1)
            bulk_g2s_pred(true, smem_u32(bar), both, dst + C::AB, src[TA - 1], C::AB, policy);
          else
            bulk_g2s(ring + issue_slot * TB + C::AB, src[TA - 1], C::AB, bar);
        }
      }
    }
    issue_slot = issue_slot + 1 == S ? 0 : issue_slot + 1;
    ++in_flight;
  };
  if (!dead)
    for (int i = 0; i < S && more; ++i) issue();

  auto store = [&](int first_row, int h, int r, int quad, float4 v, float sum) {
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint2 w2;
    if (p.bf16) {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * inv, v.y * inv);
      const __nv_bfloat162 hi = __floats2bfloat162_rn(v.z * inv, v.w * inv);
      w2 = make_uint2(*reinterpret_cast<const uint32_t *>(&lo),
                      *reinterpret_cast<const uint32_t *>(&hi));
    } else {
      w2 = make_uint2(h2u(__floats2half2_rn(v.x * inv, v.y * inv)),
                      h2u(__floats2half2_rn(v.z * inv, v.w * inv)));
    }
    const int64_t t = first_row + r / p.rg;
    if (t < p.T)
      *reinterpret_cast<uint2 *>(a.out + (t * p.Hq + h * p.rg + r % p.rg) * D + 4 * quad) = w2;
  };
  constexpr int kQuads = D / 4;

  // ---- consume side, segment by segment
  int b = first_b;
  for (int64_t x = x0; x < x1;) {
    const Place u = locate(prefix, H, x, b);
    b = u.b;
    const int n = (int)min((int64_t)(u.tiles - u.off), x1 - x);
    const int a0 = u.off + n * warp / kRowWarps;
    const int a1 = u.off + n * (warp + 1) / kRowWarps;
    const int row0 = p.cu[b], tokens = p.cu[b + 1] - row0, rows = tokens * p.rg;
    const int64_t cap = p.width * p.page;
    const int len = (int)min((int64_t)max(p.lens[b], 0), cap);
    // newest position row r may see; every row's is below len
    const int64_t pos0 = (int64_t)p.lens[b] - tokens;

    // queries scaled so that the row's largest is in [2^8, 2^9)
    uint32_t qf[NT][NG][4], qsum[NT];
    float F[NT][2];
    int limit[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float f[NG][8], big = 0.0f;
#pragma unroll
      for (int G = 0; G < NG; ++G) {
        const uint4 w = qraw[nt][G];
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (p.bf16) {
            f[G][2 * i] = __uint_as_float(ww[i] << 16);
            f[G][2 * i + 1] = __uint_as_float(ww[i] & 0xffff0000u);
          } else {
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&ww[i]));
            f[G][2 * i] = v.x;
            f[G][2 * i + 1] = v.y;
          }
          big = fmaxf(big, fmaxf(fabsf(f[G][2 * i]), fabsf(f[G][2 * i + 1])));
        }
      }
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      int ex = ((__float_as_int(big) >> 23) & 255) - 127;
      ex = big == 0.0f ? 0 : max(min(ex, 90), -90);
      const float mul = __int_as_float((127 + 8 - ex) << 23);
      float gs[NG];
#pragma unroll
      for (int G = 0; G < NG; ++G) {
        gs[G] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int o = ((G * 4 + i) * BITS) % 8;  // position of this pair's codes
          const float pos = __int_as_float((127 - o) << 23);
          // (bf16 queries round here, to fp16 relative to the row's largest)
          const __half2 v = __floats2half2_rn(f[G][2 * i] * mul, f[G][2 * i + 1] * mul);
          const float2 vf = __half22float2(v);
          gs[G] += vf.x + vf.y;
          qf[nt][G][i] = h2u(__floats2half2_rn(vf.x * pos, vf.y * pos));
        }
        gs[G] += __shfl_xor_sync(0xffffffffu, gs[G], 1);
        gs[G] += __shfl_xor_sync(0xffffffffu, gs[G], 2);
      }
      // zero-point operand: k = group for the hi parts, then for the lo parts
      uint32_t hi, lo;
      if (NG == 4) {
        const bool up = j & 1;
        split2(up ? gs[2 % NG] : gs[0], up ? gs[3 % NG] : gs[1], hi, lo);
        qsum[nt] = j < 2 ? hi : lo;
      } else {
        split2(gs[0], gs[1], hi, lo);
        qsum[nt] = j == 0 ? hi : j == 1 ? lo : 0u;
      }
      // per-row factors move to the lanes that hold the row's scores
      const float mine = fmaxf(
          fminf(a.scale_log2 * __int_as_float((127 + 24 + ex - 8) << 23), kMostScale), -kMostScale);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int rr = 8 * nt + 2 * j + s;
        F[nt][s] = __shfl_sync(0xffffffffu, mine, (2 * j + s) * 4);
        const int64_t see = pos0 + rr / p.rg;
        limit[nt][s] = rr < rows ? (int)min(see, (int64_t)len - 1) : len - 1;
      }
    }
    const int least = (int)min(pos0, (int64_t)len - 1);  // newest position every row sees

    float o[NG][2][NT][4] = {}, za[NG][NT][2] = {}, l[NT][2] = {}, rf[NT][2];
    uint32_t e2 = 0;  // largest value scale covered by the reference, in both halves
    int E = -24 - kRoom;  // the exponent of that, less the room above the reference
    float slack = kSlack - (float)E;  // how far a score may pass the reference
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int s = 0; s < 2; ++s) rf[nt][s] = 0.0f;
    uint32_t fresh = (1u << (2 * NT)) - 1;  // rows that have seen no score: no reference yet

    for (int at = a0; at < a1; ++at) {
      if (dead) break;
      if (!bar_wait(&bars[slot], phase, kRowWaitLimit)) {
        if (lane == 0) paged_error(p, KVQ_ETIMEOUT);
        dead = true;
        break;
      }
      const uint8_t *at_s = ring + slot * TB;
      const uint32_t gone = skip >> (TA * slot) & ((1u << TA) - 1);
      const int pos = at * kTile;
      // token of fragment row r < 8 of an atom: (r >> 1) + 4 * (r & 1); rows 8..
      // 8 more
      const int t0 = (g >> 1) + 4 * (g & 1);
      // masked: some token is hidden from some row, or is not there at all
      const bool masked = pos + kTile - 1 > least || gone != 0;
      if (gone != 0 && pos < len && lane == 0) {
#pragma unroll
        for (int u = 0; u < TA; ++u)
          if ((gone >> u & 1) && pos + u * kAtom < len) paged_error(p, KVQ_EPAGE);
      }
      auto absent = [&](int u, int i) {  // token t0 + 8 * i of atom u
        return pos + u * kAtom + t0 + 8 * i >= len || (gone >> u & 1);
      };
      // statistics of a token: NG scales then NG zeros, as pairs; 0 where there
      // is no token (such slots hold anything)
      auto load_stats = [&](int u, int which, uint32_t (&st)[2][NG]) {
        const uint8_t *at = at_s + u * C::AB + 2 * kAtom * RB + which * kAtom * SB + t0 * SB;
        lds_words(at, st[0]);
        lds_words(at + 8 * SB, st[1]);
        if (masked) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (absent(u, i)) {
#pragma unroll
              for (int k = 0; k < NG; ++k) st[i][k] = 0u;
            }
        }
      };
      // ---- scores, relative to the reference
      float t[TA][NT][4];
      bool over = fresh != 0;
      __half2 smax = __float2half2_rn(0.0f);
#pragma unroll
      for (int u = 0; u < TA; ++u) {
        uint32_t k0[KW], k1[KW], ks[2][NG];
        lds_words(at_s + u * C::AB + t0 * RB + j * (RB / 4), k0);
        lds_words(at_s + u * C::AB + (t0 + 8) * RB + j * (RB / 4), k1);
        load_stats(u, 0, ks);
        {
          const uint32_t z0 = NG == 4 ? (j & 1 ? ks[0][3 % NG] : ks[0][2 % NG]) : ks[0][1];
          const uint32_t z1 = NG == 4 ? (j & 1 ? ks[1][3 % NG] : ks[1][2 % NG]) : ks[1][1];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma1688(t[u][nt], z0, z1, qsum[nt]);
#pragma unroll
            for (int i = 0; i < 4; ++i) t[u][nt][i] *= 1.0f / kSub;
          }
        }
        uint32_t k08[KW], k18[KW];
#pragma unroll
        for (int i = 0; i < KW; ++i) k08[i] = k0[i] >> 8, k18[i] = k1[i] >> 8;
#pragma unroll
        for (int G = 0; G < NG; ++G) {
          float c[NT][4];
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const int pa = (G * 4 + 2 * m) * BITS, pb = pa + BITS;  // bit offsets of two pairs
            const uint32_t x0_ = codes_at<BITS>(k0[pa / 16], k08[pa / 16], pa % 16);
            const uint32_t x1_ = codes_at<BITS>(k1[pa / 16], k18[pa / 16], pa % 16);
            const uint32_t x2_ = codes_at<BITS>(k0[pb / 16], k08[pb / 16], pb % 16);
            const uint32_t x3_ = codes_at<BITS>(k1[pb / 16], k18[pb / 16], pb % 16);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              if (m == 0)
                mma16816_first(c[nt], x0_, x1_, x2_, x3_, qf[nt][G][0], qf[nt][G][1]);
              else
                mma16816(c[nt], x0_, x1_, x2_, x3_, qf[nt][G][2], qf[nt][G][3]);
          }
          const float2 s0 = __half22float2(*reinterpret_cast<const __half2 *>(&ks[0][G / 2]));
          const float2 s1 = __half22float2(*reinterpret_cast<const __half2 *>(&ks[1][G / 2]));
          const float fa = G & 1 ? s0.y : s0.x, fb_ = G & 1 ? s1.y : s1.x;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            t[u][nt][0] = fmaf(fa, c[nt][0], t[u][nt][0]);
            t[u][nt][1] = fmaf(fa, c[nt][1], t[u][nt][1]);
            t[u][nt][2] = fmaf(fb_, c[nt][2], t[u][nt][2]);
            t[u][nt][3] = fmaf(fb_, c[nt][3], t[u][nt][3]);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            t[u][nt][i] = fmaf(t[u][nt][i], F[nt][i & 1], -rf[nt][i & 1]);
        if (masked) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (absent(u, i >> 1) || pos + u * kAtom + t0 + 8 * (i >> 1) > limit[nt][i & 1])
                t[u][nt][i] = -INFINITY;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          over |= fmaxf(fmaxf(t[u][nt][0], t[u][nt][1]), fmaxf(t[u][nt][2], t[u][nt][3])) > slack;
        // the largest value scale
        uint32_t vs[2][NG];
        load_stats(u, 1, vs);
#pragma unroll
        for (int k = 0; k < NG / 2; ++k)
          smax = __hmax2(smax, __hmax2(*reinterpret_cast<const __half2 *>(&vs[0][k]),
                                       *reinterpret_cast<const __half2 *>(&vs[1][k])));
      }
      over |= !__hble2(smax, *reinterpret_cast<const __half2 *>(&e2));
      if (__any_sync(0xffffffffu, over)) {
        // move the reference: to the largest score, and E to the scales
        float sm = fmaxf(__low2float(smax), __high2float(smax));
#pragma unroll
        for (int s = 16; s; s >>= 1) sm = fmaxf(sm, __shfl_xor_sync(0xffffffffu, sm, s));
        const int En = sm > 0.0f ? max(E, ((__float_as_int(sm) >> 23) & 255) - 126 - kRoom) : E;
        const uint32_t top = h2u(__float2half2_rn(__int_as_float((127 + En + kRoom) << 23)));
        e2 = En + kRoom > 15 ? 0x7bff7bffu : top;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            float mx = fmaxf(t[0][nt][s], t[0][nt][2 + s]);
            if (TA == 2) mx = fmaxf(mx, fmaxf(t[TA - 1][nt][s], t[TA - 1][nt][2 + s]));
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
            // from the reference to the larger of itself and the scores, and
            // from the old E to the new; a row without scores stays
            const bool first = fresh >> (2 * nt + s) & 1;
            float by = fmaxf(mx + (float)E, 0.0f) + (float)(En - E);
            if (first) by = mx == -INFINITY ? 0.0f : mx + (float)En;
            if (mx != -INFINITY) fresh &= ~(1u << (2 * nt + s));
            const float f = first ? 0.0f : exp2_approx(-by);
            rf[nt][s] += by;
#pragma unroll
            for (int u = 0; u < TA; ++u) {
              t[u][nt][s] -= by;
              t[u][nt][2 + s] -= by;
            }
            l[nt][s] *= f;
#pragma unroll
            for (int G = 0; G < NG; ++G) {
              za[G][nt][s] *= f;
              o[G][0][nt][s] *= f;
              o[G][0][nt][2 + s] *= f;
              o[G][1][nt][s] *= f;
              o[G][1][nt][2 + s] *= f;
            }
          }
        E = En;
        slack = kSlack - (float)E;
      }
#pragma unroll
      for (int u = 0; u < TA; ++u) {
        // ---- weights
        uint32_t vs[2][NG];
        load_stats(u, 1, vs);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int i = 0; i < 4; ++i) t[u][nt][i] = exp2_approx(t[u][nt][i]);
          l[nt][0] += t[u][nt][0] + t[u][nt][2];
          l[nt][1] += t[u][nt][1] + t[u][nt][3];
        }
        uint32_t w[NG][NT][2];
#pragma unroll
        for (int G = 0; G < NG; ++G) {
          const float2 s0 = __half22float2(*reinterpret_cast<const __half2 *>(&vs[0][G / 2]));
          const float2 s1 = __half22float2(*reinterpret_cast<const __half2 *>(&vs[1][G / 2]));
          const float2 z0 =
              __half22float2(*reinterpret_cast<const __half2 *>(&vs[0][NG / 2 + G / 2]));
          const float2 z1 =
              __half22float2(*reinterpret_cast<const __half2 *>(&vs[1][NG / 2 + G / 2]));
          const float sa = G & 1 ? s0.y : s0.x, sb = G & 1 ? s1.y : s1.x;
          const float ya = G & 1 ? z0.y : z0.x, yb = G & 1 ? z1.y : z1.x;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float(&q4)[4] = t[u][nt];
            w[G][nt][0] = movm(h2u(__floats2half2_rn(q4[0] * sa, q4[1] * sa)));
            w[G][nt][1] = movm(h2u(__floats2half2_rn(q4[2] * sb, q4[3] * sb)));
            za[G][nt][0] = fmaf(q4[0], ya, fmaf(q4[2], yb, za[G][nt][0]));
            za[G][nt][1] = fmaf(q4[1], ya, fmaf(q4[3], yb, za[G][nt][1]));
          }
        }
        // ---- values: tokens (j, j + 4) and (j + 8, j + 12), eighth g
        const uint8_t *vc = at_s + u * C::AB + kAtom * RB + g * (RB / 8);
        uint32_t v[4][VW];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (RB / 8 == 2)
            v[i][0] = *reinterpret_cast<const uint16_t *>(vc + (j + 4 * i) * RB);
          else
            lds_words(vc + (j + 4 * i) * RB, v[i]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t xa[VW], xb[VW], xa8[VW], xb8[VW];
#pragma unroll
          for (int i = 0; i < VW; ++i) {
            // (the two-byte eighths of d = 64, 2 bits: both halves in one)
            const uint32_t sel = RB / 8 == 2 ? 0x5410u : e ? 0x7632u : 0x5410u;
            xa[i] = __byte_perm(v[0][i], v[1][i], sel);
            xb[i] = __byte_perm(v[2][i], v[3][i], sel);
            xa8[i] = xa[i] >> 8;
            xb8[i] = xb[i] >> 8;
          }
#pragma unroll
          for (int h2 = 0; h2 < NG / 2; ++h2) {
            const int G = 2 * h2 + e;
#pragma unroll
            for (int ii = 0; ii < 2; ++ii) {
              const int pa = (h2 * 4 + 2 * ii) * BITS + (RB / 8 == 2 ? 8 * e : 0), pb = pa + BITS;
              const uint32_t y0 = codes_at<BITS>(xa[pa / 16], xa8[pa / 16], pa % 16);
              const uint32_t y1 = codes_at<BITS>(xa[pb / 16], xa8[pb / 16], pb % 16);
              const uint32_t y2 = codes_at<BITS>(xb[pa / 16], xb8[pa / 16], pa % 16);
              const uint32_t y3 = codes_at<BITS>(xb[pb / 16], xb8[pb / 16], pb % 16);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816(o[G][ii][nt], y0, y1, y2, y3, w[G][nt][0], w[G][nt][1]);
            }
          }
        }
      }
      // the slot is free once every lane has read it
      __syncwarp();
      --in_flight;
      if (++slot == S) slot = 0, phase ^= 1;
      if (more) issue();
    }

    if (x + n < x1) load_queries(x + n, b);
    // ---- the block's state of this segment: half the warps leave (reference,
    // l, o) in shared memory, the others join theirs to it, and those are then
    // joined slice by slice
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) l[nt][s] += __shfl_xor_sync(0xffffffffu, l[nt][s], k);
        if (fresh >> (2 * nt + s) & 1) rf[nt][s] = kNoRef;
#pragma unroll
        for (int G = 0; G < NG; ++G) {
          float z = za[G][nt][s];
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) z += __shfl_xor_sync(0xffffffffu, z, k);
          // the accumulators hold code sums at their codes' positions
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int off = (((G >> 1) * 4 + i) * BITS + (RB / 8 == 2 ? 8 * (G & 1) : 0)) % 8;
            float &v = o[G][i >> 1][nt][2 * (i & 1) + s];
            v = fmaf(v, __int_as_float((127 + 24 - off) << 23), z);
          }
        }
      }
    constexpr int kHalf = kRowWarps / 2;
#pragma unroll
    for (int round = 0; round < 2; ++round) {
      if ((warp >= kHalf) == (round == 0)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int r = (warp % kHalf) * kRows + 8 * nt + 2 * j + s;
            uint8_t *row = smem + C::off_merge + r * C::ROWB;
            float2 *ml = reinterpret_cast<float2 *>(smem + C::off_ml + r * 8);
            float f = 1.0f, fy = 0.0f;
            if (round == 1) {
              const float2 y = *ml;
              const float m = fmaxf(rf[nt][s], y.x);
              f = exp2_approx(rf[nt][s] - m), fy = exp2_approx(y.x - m);
              rf[nt][s] = m;
              l[nt][s] = l[nt][s] * f + y.y * fy;
            }
#pragma unroll
            for (int G = 0; G < NG; ++G) {
              float4 *at = reinterpret_cast<float4 *>(row + (G * 8 + g) * 16);
              float4 v = make_float4(o[G][0][nt][s], o[G][0][nt][2 + s], o[G][1][nt][s],
                                     o[G][1][nt][2 + s]);
              if (round == 1) {
                const float4 y = *at;
                v = make_float4(v.x * f + y.x * fy, v.y * f + y.y * fy, v.z * f + y.z * fy,
                                v.w * f + y.w * fy);
              }
              *at = v;
            }
            if (round == 1) __syncwarp();
            if (g == 0) *ml = make_float2(rf[nt][s], l[nt][s]);
          }
      }
      __syncthreads();
    }
    const int64_t pair0 = x - u.off, pair1 = pair0 + u.tiles;
    const bool whole = pair0 >= x0 && pair1 <= x1;
    const int my_slot = 2 * blockIdx.x + (pair0 >= x0 ? 1 : 0);
    for (int i = tid; i < rows * kQuads; i += kRowThreads) {
      const int r = i / kQuads, quad = i % kQuads;
      float m = kNoRef;
      float2 ml[kHalf];
#pragma unroll
      for (int w = 0; w < kHalf; ++w) {
        ml[w] = *reinterpret_cast<const float2 *>(smem + C::off_ml + (w * kRows + r) * 8);
        m = fmaxf(m, ml[w].x);
      }
      float sum = 0.0f;
      float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int w = 0; w < kHalf; ++w) {
        const float f = exp2_approx(ml[w].x - m);
        const float4 y = *reinterpret_cast<const float4 *>(
            smem + C::off_merge + (w * kRows + r) * C::ROWB + quad * 16);
        sum += f * ml[w].y;
        v.x += f * y.x;
        v.y += f * y.y;
        v.z += f * y.z;
        v.w += f * y.w;
      }
      if (whole) {
        store(row0, u.h, r, quad, v, sum);
      } else {
        *reinterpret_cast<float4 *>(a.ws_o + ((int64_t)my_slot * kRows + r) * D + 4 * quad) = v;
        if (quad == 0)
          *reinterpret_cast<float2 *>(a.ws_ml + ((int64_t)my_slot * kRows + r) * 2) =
              make_float2(m, sum);
      }
    }
    if (!whole) {
      const int e = pair0 >= x0;
      n_shared |= 1 << e;
      if (tid == 0) {
        Shared &sp = shared_pair[e];
        sp.pair0 = pair0, sp.pair1 = pair1;
        sp.row0 = row0, sp.rows = rows, sp.h = u.h;
      }
    }
    __syncthreads();  // the merge buffer is free for the next segment
    x += n;
  }

  // ---- shared pairs, once all of the block's work is done: the block that
  // arrives last joins the parts, in block order
  if (n_shared) {
    __threadfence();
    __syncthreads();
    const int e = tid >> 5;
    if (e < 2 && lane == 0 && (n_shared >> e & 1)) {
      Shared &sp = shared_pair[e];
      int first = c_first, last = c_last;
      if (!by_piece) {
        // a pair that began here, or ends here, has its first or last part here
        if (sp.pair0 < x0) {
          first = (int)div64(sp.pair0, U);
          while (border(prefix, p.B, H, total, U, first) > sp.pair0) --first;
          while (border(prefix, p.B, H, total, U, first + 1) <= sp.pair0) ++first;
        }
        if (sp.pair1 > x1) {
          last = (int)div64(sp.pair1 - 1, U);
          while (border(prefix, p.B, H, total, U, last) >= sp.pair1) --last;
          while (border(prefix, p.B, H, total, U, last + 1) < sp.pair1) ++last;
        }
      }
      sp.first = first, sp.last = last;
      sp.join = atomicAdd(&a.ws_count[first], 1) == last - first;
      if (sp.join) a.ws_count[first] = 0;
    }
    __syncthreads();
    for (int e2 = 0; e2 < 2; ++e2) {
      if (!(n_shared >> e2 & 1) || !shared_pair[e2].join) continue;
      const Shared sp = shared_pair[e2];
      __threadfence();
      for (int i = tid; i < sp.rows * kQuads; i += kRowThreads) {
        const int r = i / kQuads, quad = i % kQuads;
        float m = kNoRef, sum = 0.0f;
        float4 v = make_float4(0, 0, 0, 0);
#pragma unroll 4
        for (int c = sp.first; c <= sp.last; ++c) {
          const int64_t at = (int64_t)(2 * c + (c == sp.first)) * kRows + r;
          const float2 ml = __ldcg(reinterpret_cast<const float2 *>(a.ws_ml + at * 2));
          const float4 y = __ldcg(reinterpret_cast<const float4 *>(a.ws_o + at * D + 4 * quad));
          const float nm = fmaxf(m, ml.x), f = exp2_approx(m - nm), f2 = exp2_approx(ml.x - nm);
          m = nm;
          sum = sum * f + f2 * ml.y;
          v.x = v.x * f + f2 * y.x;
          v.y = v.y * f + f2 * y.y;
          v.z = v.z * f + f2 * y.z;
          v.w = v.w * f + f2 * y.w;
        }
        store(sp.row0, sp.h, r, quad, v, sum);
      }
    }
  }
  // a warp that gave up leaves no copy of its own in flight
  if (dead)
    for (; in_flight > 0; --in_flight) {
      bar_wait(&bars[slot], phase, kDrainLimit);
      if (++slot == S) slot = 0, phase ^= 1;
    }
  if (a.beside) grid_dep_wait();
}

template <int D, int BITS, int NT>
cudaError_t launch_as(RowsArgs &a, int num_sms, cudaStream_t st) {
  using C = RowsCfg<D, BITS, NT>;
  static KernelSetup setup;
  const int smem = C::smem(a.p.B);
  int occ = 0;
  auto kern = paged_rows_kernel<D, BITS, NT>;
  cudaError_t e = kernel_setup(setup, kern, C::kRowThreads, smem, &occ);
  if (e != cudaSuccess) return e;
  int blocks = num_sms * occ;
  if (blocks > kPagedRowBlocks) blocks = kPagedRowBlocks;
  return launch_dependent(kern, (unsigned)blocks, C::kRowThreads, smem, st, true, a);
}

}  // namespace

cudaError_t launch_paged_rows(const Paged &p, const void *q, int64_t qs, void *out, float scale,
                              int few, bool beside, void *ws, int num_sms, cudaStream_t st) {
  RowsArgs a;
  a.p = p;
  a.q = static_cast<const uint16_t *>(q);
  a.qs = qs;
  a.out = static_cast<uint16_t *>(out);
  a.scale_log2 = fmaxf(fminf(scale * 1.4426950408889634f, kMostScale), -kMostScale);
  uint8_t *w = static_cast<uint8_t *>(ws);
  a.ws_count = reinterpret_cast<int *>(w);
  a.ws_ml = reinterpret_cast<float *>(w + kPagedRowBlocks * 4);
  a.ws_o = reinterpret_cast<float *>(w + kPagedRowBlocks * 4 +
                                     2 * kPagedRowBlocks * kPagedFewRows * 8);
  a.stall_limit = debug_stall_limit();
  a.few = few;
  a.beside = beside;
  const int64_t most = few;
  // one tile of 8 rows when no sequence has more, two otherwise
  if (p.d == 128) {
    if (most <= 8)
      return p.bits == 2   ? launch_as<128, 2, 1>(a, num_sms, st)
             : p.bits == 4 ? launch_as<128, 4, 1>(a, num_sms, st)
                           : launch_as<128, 8, 1>(a, num_sms, st);
    return p.bits == 2   ? launch_as<128, 2, 2>(a, num_sms, st)
           : p.bits == 4 ? launch_as<128, 4, 2>(a, num_sms, st)
                         : launch_as<128, 8, 2>(a, num_sms, st);
  }
  if (most <= 8)
    return p.bits == 2   ? launch_as<64, 2, 1>(a, num_sms, st)
           : p.bits == 4 ? launch_as<64, 4, 1>(a, num_sms, st)
                         : launch_as<64, 8, 1>(a, num_sms, st);
  return p.bits == 2   ? launch_as<64, 2, 2>(a, num_sms, st)
         : p.bits == 4 ? launch_as<64, 4, 2>(a, num_sms, st)
                       : launch_as<64, 8, 2>(a, num_sms, st);
}

size_t paged_rows_workspace() {
  return kPagedRowBlocks * 4 + 2 * kPagedRowBlocks * kPagedFewRows * (8 + 4 * kMaxHeadDim);
}

}  // namespace kvq
