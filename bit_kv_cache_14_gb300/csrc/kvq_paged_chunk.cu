// Paged cache: attention of chunks of new tokens, on tcgen05.
//
// Rows: the query tokens of a sequence times the query heads of one KV head,
// token-major, so that grouped heads share the keys and values read for them.
// A block works on 256 of them (two MMA tiles of 128) against 128 cached tokens
// at a time:
//   S_i = Q_i K^T                      tcgen05.mma, both operands in shared memory
//   P_i = 2^(S_i F - ref)              one thread per row; fp16, back into tensor memory
//   O_i (+)= P_i V                     tcgen05.mma, P from tensor memory
// S, P and O stay in tensor memory (S and P share columns).  The reference of
// a row lies 4 (log2 units) below the maximum of earlier steps and moves only
// when a score passes that by more than 9, so the weights need no pass over the
// scores for the maximum first, and O is rescaled a few times per row at most, by
// the row's own thread.  The 4 are fp16's room above 1: the largest weight is held
// at 2^4 or more, so weights down to 2^-18 of it are normal fp16 numbers and
// smaller ones keep an absolute 2^-29 of it (held at 1, weights of 2^-26.5 went to
// zero, and with them the output of rows that thousands of those make up).  More
// room costs moves: 4096 tokens of 32768 at 2 bits in 1502, 1549, 1585 and 1611
// us at 0, 3, 4 and 5; at 4 bits 1410, 1419, 1425 and 1437 (before the queries came
// asynchronously, which took 60 us off either).
//
// Bound: 4*128*256*d operations per step on the tensor core against 128*256
// exponentials and the dequantization of 128 keys and values: eight producer
// warps read codes and statistics into registers one step ahead, turn codes
// into fp16 (1024 + code by one LOP3, the code by one HFMA2, code * scale +
// zero by a second: exact but for one rounding) and store the swizzled operand
// tiles, which both query tiles use.  Measured on a GB300, 32 query and 8 KV heads
// of 128, 4 bits: the last 4096 tokens of 32768, 1357 us = 1520 TFLOP/s, 81 % of the
// measured matrix rate (1471 us back to back for seconds, at a lower clock: 82 % of the
// sustained rate; 1524 at 2 bits, 1665 at 8, 1239 with heads of 64); the last 512 of 8192
// four times, 226 us = 1180 TFLOP/s; 64 tokens alone, 20 us.  Cross attention of 2 x 2048
// rows over 16384 tokens: 762 us = 1443 TFLOP/s, 77 %.
//
// What made the difference: no role may spill (a spilled MMA thread needed 200
// clocks an instruction instead of 64), role code has to be small or rolled (five
// roles share the instruction caches), and waiting warps have to sleep between
// polls.
//
//   warps 0-3, 4-7: softmax and output of query tiles 0 and 1
//   warps 8-15: producers    warp 16: MMA issue    warp 17: lists of items and
//   of steps (the addresses of their pages)
//   (warps 18, 19 only give up registers)
//
// Split: every (sequence, head, 256-row tile) is a list of its visible 128-token
// steps.  Where all tiles in pieces of about 6, 8 or 12 steps (the smallest that
// does) give no more pieces than there are blocks, each block takes a piece; a
// longer list, kOver units added to each tile for its start and end, is cut into
// equal ranges, one per block.  A tile that several blocks share leaves partials,
// joined in block order by the block that finishes last.
#include "kvq_paged.cuh"
#include "kvq_tc_common.cuh"

namespace kvq {

int debug_stall_limit();

namespace {

constexpr int kChunkThreads = 640;
// Registers a thread, of the 640 * 96 at launch: softmax, producers (which hold
// a step's codes), the others.  256 * 136 + 256 * 88 + 128 * 32 = 61440.
constexpr int kSoftRegs = 136, kProducerRegs = 88, kOtherRegs = 32;
static_assert(256 * kSoftRegs + 256 * kProducerRegs + 128 * kOtherRegs <= 640 * 96, "registers");
constexpr int kProducerWarp = 8, kMmaWarp = 16, kItemWarp = 17;
constexpr int kItems = 4;   // items on their way to the roles
constexpr int kSteps = 16;  // steps known to the producers and the softmax warps
constexpr int kAhead = 8;   // steps the list runs ahead of the producers' loads
constexpr int kPWarps = kMmaWarp - kProducerWarp;
constexpr int kStep = 128;       // cached tokens per step
constexpr int kTileRows = 256;   // query rows per block
constexpr int kOver = 6;         // units of a tile's start and end, which take about as long
constexpr int kMinUnits = 16;    // (borders move by up to kOver + 1 units)
// Steps worth a block of their own: joining the parts of a tile costs about four
// steps' time (a 512-token chunk in pieces of 4, 6 and 10 steps: all within 1 %,
// 128 tokens over 4096: 50.5, 47.7, 50.4 us).
constexpr int kPieceSizes = 3;
__host__ __device__ constexpr int piece_size(int k) { return k == 0 ? 6 : k == 1 ? 8 : 12; }
constexpr int kMaxChunkBlocks = 160;
constexpr int kChunkWait = 1 << 25;
constexpr float kChunkBase = 4.0f;    // log2 of the weight a reference is set to give
constexpr float kChunkSlack = 13.0f;  // ... above which it moves before the next step
constexpr float kChunkTop = 15.0f;    // ... within a step: weights up to 2^15 fit fp16
constexpr float kNoRef = -1e30f;

struct ChunkArgs {
  Paged p;
  const uint16_t *q;
  int64_t qs;
  uint16_t *out;
  float scale_log2;  // >= 0
  float sign;        // of the softmax scale, folded into the queries
  int few;           // sequences with at most this many rows are not this kernel's
  float *ws_ml;      // [2 * blocks][2 tiles][128][2]
  float *ws_o;       // [2 * blocks][2 tiles][d / 4][128] float4
  int *ws_count;     // [blocks][2 tiles], zero between calls
  int stall_limit;
};

template <int D>
struct ChunkCfg {
  static constexpr int kTile = kStep * D * 2;  // bytes of a 128-row operand tile
  static constexpr int off_q = 0;
  static constexpr int off_k = 2 * kTile;
  static constexpr int off_v = off_k + 2 * kTile;
  static constexpr int off_f = off_v + 2 * kTile;          // float [256] row factors
  static constexpr int off_step = off_f + kTileRows * 4;   // Step [kSteps]
  static constexpr int off_bar = off_step + kSteps * 80;
  static constexpr int kBars = 19 + 2 * kItems + 2 * kAhead;
  static constexpr int off_item = (off_bar + kBars * 8 + 15) / 16 * 16;
  static constexpr int off_misc = off_item + kItems * 64;  // tensor memory base, dead flag, flags
  static constexpr int smem = off_misc + 64 + 1024;
  // the running sums of the plan lie where the operands come later
  static_assert((1 + kPieceSizes) * (kMaxSeqs + 1) * 8 <= 6 * kTile, "room for the plan");
};

// ---- PTX ------------------------------------------------------------------
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(ok));
  return ok != 0;
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
               : "memory");
}
// One arrival for the warp, after every lane's earlier work.
__device__ __forceinline__ void bar_arrive_warp(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0)
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void async_fence() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// 32 consecutive 32-bit columns of the warp's lanes.
__device__ __forceinline__ void tc_ld32(uint32_t addr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tc_ld16(uint32_t addr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31, %32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Shared-memory matrix descriptor: 128-byte swizzle, strides in bytes.  Adding
// n to it moves the address by 16 * n bytes.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(lbo >> 4) << 16 |
         (uint64_t)(sbo >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// Instruction descriptor: fp16 operands, fp32 accumulator, M = 128.
__host__ __device__ constexpr uint32_t mma_desc(int n, bool b_mn_major) {
  return 1u << 4 | (b_mn_major ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (128u >> 4) << 24;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((int)acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((int)acc)
      : "memory");
}

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__host__ __device__ constexpr uint32_t dup16(uint32_t h) { return h | h << 16; }

// Codes at bit `off` (0 .. 7) of both halves of w, as exact fp16 numbers:
// (code << off) | 1024.0, times 2^-off, minus 1024 * 2^-off.
template <int BITS>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int off) {
  const uint32_t mask = dup16(((1u << BITS) - 1) << off);
  const uint32_t h = and_or(w, mask, 0x64006400u);
  // 2^-off and -1024 * 2^-off as fp16
  const uint32_t mul = dup16((uint32_t)(15 - off) << 10);
  const uint32_t sub = dup16(0x8000u | (uint32_t)(25 - off) << 10);
  return hfma2(h, mul, sub);
}

// ---- the list of work -------------------------------------------------------
// Tokens, rows and visible length of sequence b; rows = 0 when it is not this
// kernel's.
struct Seq {
  int row0, tokens, rows, len;
  int64_t pos0;
};
__device__ __forceinline__ Seq seq_of(const ChunkArgs &a, int b) {
  const Paged &p = a.p;
  Seq s;
  s.row0 = p.cu[b];
  s.tokens = (int)((unsigned)p.cu[b + 1] - (unsigned)s.row0);
  const int64_t cap = p.width * p.page;
  s.len = (int)min((int64_t)max(p.lens[b], 0), cap);
  s.pos0 = first_seen(p, b, s.tokens);
  const int64_t rows = (int64_t)s.tokens * p.rg;
  s.rows = !bad_rows(p, b) && rows > a.few ? (int)rows : 0;
  return s;
}
// Visible steps of 256-row tile t.
__device__ __forceinline__ int steps_of(const ChunkArgs &a, const Seq &s, int t) {
  const int last = min((t + 1) * kTileRows, s.rows) - 1;
  const int64_t see = min(s.pos0 + last / a.p.rg, (int64_t)s.len - 1) + 1;
  return see < 1 ? 1 : (int)((see + kStep - 1) / kStep);
}

__device__ __forceinline__ int pieces_of(int steps, int size) {
  return max(1, (steps + size / 2) / size);
}

// One block's share of one tile, as the roles read it from shared memory.
struct __align__(16) Item {
  int b, h;             // sequence (-1: no more items), KV head
  int j0, j1;           // steps [j0, j1) of the tile
  int row0, row_first;  // the sequence's first packed row; the tile's first row in it
  int rows, len;        // rows and visible length of the sequence
  int64_t pos0;         // newest position the sequence's first row sees
  int steps;            // of the whole tile
  int c0, c1;           // first and last block with a share
  int pad[3];
};
static_assert(sizeof(Item) == 64, "layout of the item ring");

// One step, as the producers read it: where its eight atoms are (0: nowhere),
// how many of its tokens exist (-1: no more steps), and which atoms belong to
// the sequence but have no page.
struct __align__(16) Step {
  uint64_t atom[kStep / kAtom];
  int tokens;
  uint32_t bad;
  int pad[2];
};
static_assert(sizeof(Step) == 80, "layout of the step ring");

template <int D, int BITS>
__global__ void __launch_bounds__(kChunkThreads, 1)
paged_chunk_kernel(const __grid_constant__ ChunkArgs a) {
  using C = ChunkCfg<D>;
  constexpr int RB = D * BITS / 8, SB = 4 * D / kPagedGroup, NG = D / kPagedGroup;
  constexpr int AB = 2 * kAtom * (RB + SB);
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t smem_s = smem_u32(smem);
  const Paged &p = a.p;
  // (through a shuffle, so that the compiler knows it to be uniform)
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  // the split kernel of the same call may run where this one leaves room
  grid_dep_trigger();

  // barriers
  const uint32_t bars = smem_s + C::off_bar;
  auto bar_q = [&](int i) { return bars + 8u * i; };             // queries of tile i are in
  auto bar_s = [&](int i) { return bars + 8u * (2 + i); };       // scores of tile i are in
  auto bar_p = [&](int i) { return bars + 8u * (4 + i); };       // weights of tile i are in
  auto bar_o = [&](int i) { return bars + 8u * (6 + i); };       // output of tile i complete
  auto bar_kf = [&](int s) { return bars + 8u * (8 + s); };      // key stage full / empty
  auto bar_ke = [&](int s) { return bars + 8u * (10 + s); };
  auto bar_vf = [&](int s) { return bars + 8u * (12 + s); };
  auto bar_ve = [&](int s) { return bars + 8u * (14 + s); };
  const uint32_t bar_end = bars + 8u * 16;                       // everything issued is done
  auto bar_g = [&](int i) { return bars + 8u * (17 + i); };      // the 128 threads of tile i
  uint32_t *misc = reinterpret_cast<uint32_t *>(smem + C::off_misc);
  volatile uint32_t *dead = misc + 1;
  int64_t *units = reinterpret_cast<int64_t *>(smem);  // running sums over the sequences
  // and kPieceSizes times those of the pieces
  int64_t *sh_x = reinterpret_cast<int64_t *>(misc + 4);  // borders of the block's range
  int *sh_at = reinterpret_cast<int *>(misc + 8);         // b, h, t, off of its first unit

  if (tid == 0) {
    for (int i = 0; i < kItems; ++i) {
      bar_init(reinterpret_cast<uint64_t *>(smem + C::off_bar) + 19 + i, 1);
      bar_init(reinterpret_cast<uint64_t *>(smem + C::off_bar) + 19 + kItems + i, kProducerWarp + 1);
    }
    for (int i = 0; i < kAhead; ++i) {
      bar_init(reinterpret_cast<uint64_t *>(smem + C::off_bar) + 19 + 2 * kItems + i, 1);
      bar_init(reinterpret_cast<uint64_t *>(smem + C::off_bar) + 19 + 2 * kItems + kAhead + i,
               kPWarps);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(reinterpret_cast<uint64_t *>(smem + C::off_bar) + i, 4);
      bar_init(reinterpret_cast<uint64_t *>(smem + C::off_bar) + 2 + i, 1);
      bar_init(reinterpret_cast<uint64_t *>(smem + C::off_bar) + 4 + i, 4);
      bar_init(reinterpret_cast<uint64_t *>(smem + C::off_bar) + 6 + i, 1);
      bar_init(reinterpret_cast<uint64_t *>(smem + C::off_bar) + 8 + i, kPWarps);
      bar_init(reinterpret_cast<uint64_t *>(smem + C::off_bar) + 10 + i, 1);
      bar_init(reinterpret_cast<uint64_t *>(smem + C::off_bar) + 12 + i, kPWarps);
      bar_init(reinterpret_cast<uint64_t *>(smem + C::off_bar) + 14 + i, 1);
      bar_init(reinterpret_cast<uint64_t *>(smem + C::off_bar) + 17 + i, 4);
    }
    bar_init(reinterpret_cast<uint64_t *>(smem + C::off_bar) + 16, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    misc[1] = 0;
    for (int i = 0; i <= kPieceSizes; ++i) units[i * (kMaxSeqs + 1)] = 0;
  }

  // ---- units (and pieces) of one head of sequences 0 .. b at [b + 1]
  for (int b = warp; b < p.B; b += kChunkThreads / 32) {
    const Seq s = seq_of(a, b);
    if (lane == 0 && blockIdx.x == 0) {
      if (bad_rows(p, b)) paged_error(p, KVQ_EINVAL);
      if (s.rows > 0 && p.lens[b] > p.width * p.page) paged_error(p, KVQ_EPAGE);
    }
    const int tiles = (s.rows + kTileRows - 1) / kTileRows;
    int64_t sum[1 + kPieceSizes] = {};
    for (int t = lane; t < tiles; t += 32) {
      const int steps = steps_of(a, s, t);
      sum[0] += steps + kOver;
#pragma unroll
      for (int i = 0; i < kPieceSizes; ++i) sum[1 + i] += pieces_of(steps, piece_size(i));
    }
#pragma unroll
    for (int i = 0; i <= kPieceSizes; ++i) {
#pragma unroll
      for (int o = 16; o; o >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
      if (lane == 0) units[i * (kMaxSeqs + 1) + b + 1] = sum[i];
    }
  }
  __syncthreads();
  if (warp <= kPieceSizes) {  // running sums, 32 sequences at a time
    int64_t *sums = units + warp * (kMaxSeqs + 1), before = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      int64_t v = b0 + lane < p.B ? sums[b0 + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += up;
      }
      v += before;
      if (b0 + lane < p.B) sums[b0 + lane + 1] = v;
      before = __shfl_sync(0xffffffffu, v, 31);
    }
  }
  __syncthreads();
  int size = 0;  // of the pieces, or 0
  const int64_t *prefix = units;
#pragma unroll
  for (int i = kPieceSizes - 1; i >= 0; --i) {
    const int64_t *sums = units + (1 + i) * (kMaxSeqs + 1);
    if (p.H * sums[p.B] <= gridDim.x) size = piece_size(i), prefix = sums;
  }
  const bool by_piece = size > 0;
  const int64_t total = p.H * prefix[p.B];
  const int64_t U =
      by_piece ? 1 : max((total + gridDim.x - 1) / (int64_t)gridDim.x, (int64_t)kMinUnits);
  auto cost_of = [&](const Seq &s, int t) {
    const int steps = steps_of(a, s, t);
    return by_piece ? pieces_of(steps, size) : steps + kOver;
  };
  // ---- the block's borders: warp 0 its first unit, warp 1 the next block's.
  // A border inside a tile's first units moves to its start, one at its last
  // step to its end, so every item has steps of its own.
  if (warp < 2) {
    int64_t x = (blockIdx.x + warp) * U;
    int b = 0, h = 0, t = 0, off = 0;
    if (x >= total) {
      x = total;
    } else {
      int lo = 0, hi = p.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.H * prefix[mid] <= x) lo = mid; else hi = mid;
      }
      b = lo;
      const Seq s = seq_of(a, b);
      const int64_t per = prefix[b + 1] - prefix[b], r = x - p.H * prefix[b];
      h = (int)(r / per);
      int64_t y = r - h * per;  // unit inside the head
      const int tiles = (s.rows + kTileRows - 1) / kTileRows;
      for (int t0 = 0;; t0 += 32) {
        int64_t cost = t0 + lane < tiles ? cost_of(s, t0 + lane) : 0, run = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t up = __shfl_up_sync(0xffffffffu, run, o);
          if (lane >= o) run += up;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, run > y);
        if (hit) {
          const int w = __ffs(hit) - 1;
          t = t0 + w;
          const int64_t end = __shfl_sync(0xffffffffu, run, w);
          cost = __shfl_sync(0xffffffffu, cost, w);
          off = (int)(y - (end - cost));
          if (by_piece) {
          } else if (off <= kOver + 1) {
            x -= off;
            off = 0;
          } else if (cost - off <= 1) {
            x += cost - off;
            ++t;
            off = 0;
          }
          break;
        }
        y -= __shfl_sync(0xffffffffu, run, 31);
        if (t0 + 32 >= tiles) break;  // (not reached: y is inside the head)
      }
    }
    if (lane == 0) {
      sh_x[warp] = x;
      if (warp == 0) sh_at[0] = b, sh_at[1] = h, sh_at[2] = t, sh_at[3] = off;
    }
  }
  __syncthreads();
  const int64_t x0 = sh_x[0], x1 = sh_x[1];
  if (x0 >= x1) return;

  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_s + C::off_misc)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  auto tm_s = [&](int i) { return tmem + 128u * i; };
  auto tm_o = [&](int i) { return tmem + 256u + 128u * i; };

  // Bounded waits: one that runs out records KVQ_ETIMEOUT and ends every role.
  // (Between polls a warp sleeps a little: waiting warps share their schedulers
  // with working ones.)
  auto wait = [&](uint32_t bar, uint32_t parity, int ns = 20) {
    for (int i = 0; i < kChunkWait; ++i) {
      if (bar_try_wait(bar, parity)) return true;
      __nanosleep(ns);
      if ((i & 63) == 63 && *dead) return false;
    }
    *dead = 1;
    paged_error(p, KVQ_ETIMEOUT);
    return false;
  };
  // item n of the block (b < 0: there are no more, or a wait ran out), and its
  // release once the warp has taken what it needs
  const Item *items = reinterpret_cast<const Item *>(smem + C::off_item);
  const Step *steps = reinterpret_cast<const Step *>(smem + C::off_step);
  auto bar_sf = [&](uint32_t n) { return bars + 8u * (19 + 2 * kItems + (n % kAhead)); };
  auto bar_se = [&](uint32_t n) { return bars + 8u * (19 + 2 * kItems + kAhead + (n % kAhead)); };
  auto bar_if = [&](uint32_t n) { return bars + 8u * (19 + (n % kItems)); };
  auto bar_ie = [&](uint32_t n) { return bars + 8u * (19 + kItems + (n % kItems)); };
  // the same for a whole warp, with one answer (tcgen05.ld / st need it whole)
  auto wait_warp = [&](uint32_t bar, uint32_t parity, int ns = 20) {
    return (bool)__all_sync(0xffffffffu, wait(bar, parity, ns));
  };
  auto take_item = [&](uint32_t n) -> const Item * {
    if (!wait_warp(bar_if(n), n / kItems & 1)) return nullptr;
    const Item *it = items + n % kItems;
    return it->b < 0 ? nullptr : it;
  };
  if (a.stall_limit > 0 && tid == 0) {
    bool ok = false;
    for (int i = 0; i < a.stall_limit && !ok; ++i) ok = bar_try_wait(bar_end, 0);
    if (!ok) {
      *dead = 1;
      paged_error(p, KVQ_ETIMEOUT);
    }
  }

  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kMmaWarp) {
      // ---- MMA issue: the whole warp keeps step, one lane issues
      constexpr uint32_t kQK = mma_desc(kStep, false), kPV = mma_desc(D, true);
      const uint64_t q_desc = smem_desc(smem_s + C::off_q, 16, 1024);
      const uint64_t k_desc = smem_desc(smem_s + C::off_k, 16, 1024);
      const uint64_t v_desc = smem_desc(smem_s + C::off_v, kStep * 128, 1024);
      const bool leader = elect_one();
      auto scores = [&](int i, uint32_t stage) {
        if (leader) {
          const uint64_t qd = q_desc + i * (C::kTile / 16), kd = k_desc + stage * (C::kTile / 16);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            // 16 channels: 32 bytes inside a 128-byte row, 64 channels a subtile
            const uint32_t o = ((k / 4) * (kStep * 128) + (k % 4) * 32) / 16;
            mma_ss(tm_s(i), qd + o, kd + o, kQK, k > 0);
          }
          tc_commit(bar_s(i));
        }
        __syncwarp();
      };
      auto outputs = [&](int i, uint32_t stage, bool first, bool last) {
        if (leader) {
          const uint64_t vd = v_desc + stage * (C::kTile / 16);
          mma_ts(tm_o(i), tm_s(i), vd, kPV, !first);
#pragma unroll
          for (int k = 1; k < kStep / 16; ++k)
            mma_ts(tm_o(i), tm_s(i) + 8 * k, vd + k * (2048 / 16), kPV, true);
          if (last) tc_commit(bar_o(i));
        }
        __syncwarp();
      };
      auto commit = [&](uint32_t bar) {
        if (leader) tc_commit(bar);
        __syncwarp();
      };
      uint32_t kn = 0, vn = 0;  // key / value steps taken
      uint32_t qn = 0, pn = 0;  // parities: bit i for tile i
      bool ok = true;
      for (uint32_t in = 0; ok; ++in) {
        const Item *it = take_item(in);
        if (!it) break;
        const bool two = __shfl_sync(0xffffffffu, it->rows - it->row_first, 0) > 128;
        const int n = __shfl_sync(0xffffffffu, it->j1 - it->j0, 0);
        bar_arrive_warp(bar_ie(in));
        ok = wait_warp(bar_q(0), qn & 1);
        if (ok && two) ok = wait_warp(bar_q(1), qn >> 1);
        qn ^= two ? 3u : 1u;
        ok = ok && wait_warp(bar_kf(kn & 1), kn >> 1 & 1);
        if (!ok) break;
        tc_fence_after();
        scores(0, kn & 1);
        if (two) scores(1, kn & 1);
        commit(bar_ke(kn & 1));
        ++kn;
        for (int j = 0; j < n; ++j, ++vn) {
          const bool more = j + 1 < n;
          ok = wait_warp(bar_vf(vn & 1), vn >> 1 & 1) && wait_warp(bar_p(0), pn & 1);
          if (!ok) break;
          tc_fence_after();
          outputs(0, vn & 1, j == 0, !more);
          if (!two) commit(bar_ve(vn & 1));
          if (more) {
            if (!(ok = wait_warp(bar_kf(kn & 1), kn >> 1 & 1))) break;
            tc_fence_after();
            scores(0, kn & 1);
          }
          if (two) {
            if (!(ok = wait_warp(bar_p(1), pn >> 1))) break;
            tc_fence_after();
            outputs(1, vn & 1, j == 0, !more);
            commit(bar_ve(vn & 1));
            if (more) scores(1, kn & 1);
          }
          pn ^= two ? 3u : 1u;
          if (more) {
            commit(bar_ke(kn & 1));
            ++kn;
          }
        }
      }
      // whatever was issued ends before tensor memory is freed
      commit(bar_end);
      bool done = false;
      for (int i = 0; i < kChunkWait && !done; ++i) done = bar_try_wait(bar_end, 0);
      __syncwarp();
    } else if (warp == kItemWarp) {
      // ---- the items of [x0, x1), in turn, and their steps
      int b = sh_at[0], h = sh_at[1], t = sh_at[2], off = sh_at[3];
      int64_t x = x0;
      Seq s = seq_of(a, b);
      int tiles = (s.rows + kTileRows - 1) / kTileRows;
      const int apage_log = __ffs(p.page / kAtom) - 1;
      uint32_t sn = 0;  // steps listed
      for (uint32_t in = 0;; ++in) {
        if (in >= kItems && !wait_warp(bar_ie(in), (in / kItems - 1) & 1, 200)) break;
        Item *it = const_cast<Item *>(items) + in % kItems;
        const bool end = x >= x1;
        int j0 = 0, j1 = 0;
        if (end) {
          if (lane == 0) it->b = -1;
        } else {
          while (t >= tiles) {
            t = 0;
            if (tiles > 0 && ++h < p.H) break;
            h = 0;
            do {
              ++b;
              s = seq_of(a, b);
            } while (s.rows == 0);
            tiles = (s.rows + kTileRows - 1) / kTileRows;
          }
          const int nsteps = steps_of(a, s, t), cost = cost_of(s, t);
          const int n = (int)min((int64_t)(cost - off), x1 - x);
          const int64_t first = x - off, last = first + cost;
          int c0, c1;  // the blocks that share the tile
          if (by_piece) {
            j0 = (int)((int64_t)nsteps * off / cost);
            j1 = (int)((int64_t)nsteps * (off + 1) / cost);
            c0 = (int)first, c1 = (int)last - 1;
          } else {
            j0 = off > kOver ? off - kOver : 0;
            j1 = off + n - kOver;
            // (the borders as they were moved, above)
            c0 = (int)(first / U), c1 = (int)((last - 1) / U);
            if ((c0 + 1) * U - first <= kOver + 1) ++c0;
            if (last - c1 * U <= 1) --c1;
          }
          if (lane == 0) {
            it->b = b, it->h = h;
            it->j0 = j0, it->j1 = j1;
            it->row0 = s.row0, it->row_first = t * kTileRows;
            it->rows = s.rows, it->len = s.len;
            it->pos0 = s.pos0;
            it->steps = nsteps;
            it->c0 = c0, it->c1 = c1;
          }
          x += n;
          off = 0;
          ++t;
        }
        bar_arrive_warp(bar_if(in));
        // its steps (at the end: one that says so)
        bool ok = true;
        const int64_t head_at = (int64_t)h * p.head_bytes;
        for (int j = j0; j < j1 + (end ? 1 : 0); ++j, ++sn) {
          if (sn >= kAhead && !(ok = wait_warp(bar_se(sn), (sn / kAhead - 1) & 1, 200))) break;
          Step *st = const_cast<Step *>(steps) + sn % kSteps;
          bool bad = false;
          if (lane < kStep / kAtom && !end) {
            const int atom = j * (kStep / kAtom) + lane;
            uint64_t at = 0;
            if (atom * kAtom < s.len) {
              const int64_t id = __ldg(p.table + (int64_t)b * p.width + (atom >> apage_log));
              bad = id < 0 || id >= p.n_pages;
              if (!bad)
                at = reinterpret_cast<uint64_t>(p.pages) + id * p.page_bytes + head_at +
                     (atom & ((1 << apage_log) - 1)) * AB;
            }
            st->atom[lane] = at;
          }
          const uint32_t all_bad = __ballot_sync(0xffffffffu, bad);
          if (lane == 0) {
            st->tokens = end ? -1 : s.len - j * kStep;
            st->bad = all_bad;
            if (all_bad) paged_error(p, KVQ_EPAGE);
          }
          bar_arrive_warp(bar_sf(sn));
        }
        if (end || !ok) break;
      }
    }
  } else if (warp >= kProducerWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    // ---- producers: thread (quarter jq, token t8 of eight), two tokens a step
    constexpr int QW = RB / 16;        // words of a quarter row
    constexpr int kUnits = kStep / (8 * kPWarps);  // tokens of a thread
    const int pw = warp - kProducerWarp, t8 = lane & 7, jq = lane >> 3;
    uint32_t kraw[kUnits][QW], kst[kUnits][NG], vraw[kUnits][QW], vst[kUnits][NG];
    // the thread's tokens of a step are row 8 * (pw & 1) + t8 of atoms
    // 4 * u + pw / 2
    const uint32_t row = 8 * (pw & 1) + t8;
    const uint32_t code_at = row * RB + jq * (RB / 4), stat_at = 2 * kAtom * RB + row * SB;
    // codes and statistics of the keys (or values) of a step; statistics 0 where
    // there is no token: nothing there may reach an output
    auto fetch = [&](const Step *st, bool value, uint32_t (&raw)[kUnits][QW],
                     uint32_t (&stat)[kUnits][NG]) {
      const int tokens = st->tokens;
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const uint64_t at = st->atom[kPWarps / 2 * u + (pw >> 1)];
        const bool ok = at != 0 && 8 * (kPWarps * u + pw) + t8 < tokens;
        const uint8_t *base = ok ? reinterpret_cast<const uint8_t *>(at) : p.pages;
        const uint8_t *src = base + code_at + (value ? kAtom * RB : 0);
        if constexpr (QW % 4 == 0) {
#pragma unroll
          for (int i = 0; i < QW; i += 4) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src + 4 * i));
            raw[u][i] = v.x, raw[u][i + 1] = v.y, raw[u][i + 2] = v.z, raw[u][i + 3] = v.w;
          }
        } else if constexpr (QW == 2) {
          const uint2 v = __ldg(reinterpret_cast<const uint2 *>(src));
          raw[u][0] = v.x, raw[u][1] = v.y;
        } else {
          raw[u][0] = __ldg(reinterpret_cast<const uint32_t *>(src));
        }
        const uint8_t *ss = base + stat_at + (value ? kAtom * SB : 0);
        if constexpr (NG == 4) {
          const uint4 v = __ldg(reinterpret_cast<const uint4 *>(ss));
          stat[u][0] = v.x, stat[u][1] = v.y, stat[u][2 % NG] = v.z, stat[u][3 % NG] = v.w;
        } else {
          const uint2 v = __ldg(reinterpret_cast<const uint2 *>(ss));
          stat[u][0] = v.x, stat[u][1] = v.y;
        }
      }
    };
    // which of the thread's tokens a step has
    auto present = [&](const Step *st) {
      uint32_t m = 0;
#pragma unroll
      for (int u = 0; u < kUnits; ++u)
        if (st->atom[kPWarps / 2 * u + (pw >> 1)] != 0 &&
            8 * (kPWarps * u + pw) + t8 < st->tokens)
          m |= 1u << u;
      return m;
    };
    auto clear = [&](uint32_t m, uint32_t (&stat)[kUnits][NG]) {
      if (__all_sync(0xffffffffu, m == (1u << kUnits) - 1)) return;
#pragma unroll
      for (int u = 0; u < kUnits; ++u)
        if (!(m >> u & 1)) {
#pragma unroll
          for (int i = 0; i < NG; ++i) stat[u][i] = 0;
        }
    };
    auto store_keys = [&](uint32_t tile) {
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const int trow = 8 * (kPWarps * u + pw) + t8;
#pragma unroll
        for (int G = 0; G < NG; ++G) {
          const uint32_t sel = G & 1 ? 0x3232u : 0x1010u;
          const uint32_t s = __byte_perm(kst[u][G / 2], 0, sel);
          const uint32_t z = __byte_perm(kst[u][NG / 2 + G / 2], 0, sel);
          uint32_t x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int bit = (4 * G + i) * BITS, w = bit / 16, off = bit % 16;
            x[i] = hfma2(code_pair<BITS>(off & 8 ? kraw[u][w] >> 8 : kraw[u][w], off & 7), s, z);
          }
          // channels 32G + 8jq .. + 7
          const int unit = (G & 1) * 4 + jq;
          const uint32_t at = tile + (G / 2) * (kStep * 128) + trow * 128 + ((unit ^ t8) << 4);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x[0]), "r"(x[1]),
                       "r"(x[2]), "r"(x[3])
                       : "memory");
        }
      }
    };
    auto store_values = [&](uint32_t tile) {
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const int trow = 8 * (kPWarps * u + pw) + t8;
#pragma unroll
        for (int e8 = 0; e8 < 2; ++e8) {  // eighths 2jq, 2jq + 1
#pragma unroll
          for (int h = 0; h < NG / 2; ++h) {
            uint32_t x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w;
              int off;
              if (RB / 8 == 2) {  // two bytes an eighth: spread them over two halves
                w = __byte_perm(vraw[u][0], 0, e8 ? 0x4342u : 0x4140u);
                off = i * BITS;
              } else {
                const int bit = (4 * h + i) * BITS;
                w = vraw[u][(e8 * (RB / 8) / 4 + bit / 16) % QW];
                off = bit % 16;
              }
              x[i] = hfma2(code_pair<BITS>(off & 8 ? w >> 8 : w, off & 7), vst[u][h],
                           vst[u][NG / 2 + h]);
            }
            // columns ((eighth * NG/2 + h) * 4 + i) * 2 + e hold channel
            // 32 * (2h + e) + 4 * eighth + i
            const int unit = (2 * jq + e8) * (NG / 2) + h;
            const uint32_t at =
                tile + (unit >> 3) * (kStep * 128) + trow * 128 + (((unit & 7) ^ t8) << 4);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x[0]),
                         "r"(x[1]), "r"(x[2]), "r"(x[3])
                         : "memory");
          }
        }
      }
    };
    auto step_at = [&](uint32_t k) { return steps + k % kSteps; };
    bool go = wait_warp(bar_sf(0), 0) && step_at(0)->tokens >= 0;
    uint32_t have = 0;
    if (go) {
      fetch(step_at(0), false, kraw, kst);
      fetch(step_at(0), true, vraw, vst);
      have = present(step_at(0));
      bar_arrive_warp(bar_se(0));
    }
    for (uint32_t n = 0; go; ++n) {
      const uint32_t stage = n & 1, now = have;
      clear(now, kst);
      // (a stage's first use waits for nothing)
      if (n >= 2 && !wait_warp(bar_ke(stage), ((n >> 1) - 1) & 1, 60)) break;
      store_keys(smem_s + C::off_k + stage * C::kTile);
      async_fence();
      bar_arrive_warp(bar_kf(stage));
      const Step *next = step_at(n + 1);
      if (!wait_warp(bar_sf(n + 1), (n + 1) / kAhead & 1)) break;
      go = next->tokens >= 0;
      if (go) {
        fetch(next, false, kraw, kst);
        have = present(next);
      }
      clear(now, vst);
      if (n >= 2 && !wait_warp(bar_ve(stage), ((n >> 1) - 1) & 1, 60)) break;
      store_values(smem_s + C::off_v + stage * C::kTile);
      async_fence();
      bar_arrive_warp(bar_vf(stage));
      if (go) {
        fetch(next, true, vraw, vst);
        bar_arrive_warp(bar_se(n + 1));
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ---- softmax and output: one thread per row
    const int i = warp >> 2, r = tid & 127;
    const uint32_t lane_base = (uint32_t)(warp & 3) * 32u << 16;
    const uint32_t ts = tm_s(i) + lane_base, to = tm_o(i) + lane_base;
    float *fs = reinterpret_cast<float *>(smem + C::off_f) + i * 128;
    uint32_t sn = 0, step = 0;  // score tiles taken; steps of the block (for the bad-page bytes)
    uint32_t on = 0, gn = 0;    // tiles finished; meetings of the tile's threads
    bool ok = true;
    // queries: LR lanes to a row, LR rows a lane, copied to their places in the operand
    // tile and scaled there so that a row's largest is in [2^8, 2^9), which bf16 queries
    // need to fit fp16.  (In rolled loops: unrolled code that runs once an item spent 14 us
    // on instructions that were in no cache, all of a small call's start.)
    constexpr int LR = D / 8;
    const int ql = lane % LR, qr = (warp & 3) * 32 + lane / LR;
    auto query_at = [&](int rr) {
      return smem_s + C::off_q + i * C::kTile + (ql >> 3) * (kStep * 128) + rr * 128 +
             (((ql & 7) ^ (rr & 7)) << 4);
    };
    const uint32_t rg_inv = (65535 + p.rg) / p.rg;  // n / rg = n * this >> 16 for n < 512
    auto load_queries = [&](const Item *it) {
      const int first = it->row_first + i * 128 + qr, t0 = first / p.rg, r0 = first - t0 * p.rg;
#pragma unroll 1
      for (int k = 0; k < LR; ++k) {
        const int rr = qr + k * (32 / LR), n = r0 + k * (32 / LR);
        const int dt = (int)(n * rg_inv >> 16);
        const bool there = first + k * (32 / LR) < it->rows;
        const uint16_t *src = a.q + (int64_t)(it->row0 + t0 + dt) * a.qs +
                              (int64_t)(it->h * p.rg + n - dt * p.rg) * D + 8 * ql;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(query_at(rr)),
                     "l"(there ? src : a.q), "r"(there ? 16 : 0)
                     : "memory");
      }
    };
    auto scale_queries = [&]() {  // (each lane what it copied itself)
      asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 2
      for (int k = 0; k < LR; ++k) {
        const int rr = qr + k * (32 / LR);
        uint32_t ww[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(ww[0]), "=r"(ww[1]), "=r"(ww[2]), "=r"(ww[3])
                     : "r"(query_at(rr))
                     : "memory");
        float f[8], big = 0.0f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (p.bf16) {
            f[2 * c] = __uint_as_float(ww[c] << 16);
            f[2 * c + 1] = __uint_as_float(ww[c] & 0xffff0000u);
          } else {
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&ww[c]));
            f[2 * c] = v.x;
            f[2 * c + 1] = v.y;
          }
          big = fmaxf(big, fmaxf(fabsf(f[2 * c]), fabsf(f[2 * c + 1])));
        }
#pragma unroll
        for (int o = 1; o < LR; o <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
        int ex = ((__float_as_int(big) >> 23) & 255) - 127;
        ex = big == 0.0f ? 0 : max(min(ex, 90), -90);
        const float mul = a.sign * __int_as_float((127 + 8 - ex) << 23);
        uint32_t o4[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          o4[c] = h2u(__floats2half2_rn(f[2 * c] * mul, f[2 * c + 1] * mul));
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(query_at(rr)), "r"(o4[0]),
                     "r"(o4[1]), "r"(o4[2]), "r"(o4[3])
                     : "memory");
        // (never 0: a hidden column's -inf stays -inf)
        if (ql == 0)
          fs[rr] = fminf(fmaxf(a.scale_log2 * __int_as_float((127 + ex - 8) << 23), 1e-30f),
                         kMostScale);
      }
    };
    auto queries_in = [&]() {
      async_fence();
      tc_fence_before();
      bar_arrive_warp(bar_q(i));
    };
    auto has_rows = [&](const Item *it) { return it->row_first + i * 128 < it->rows; };
    uint32_t item = 0;
    const Item *it = nullptr;  // the item at hand, if its queries are in already
    for (;;) {
      if (!it) {
        // the block's next item with rows for this tile
        for (;; ++item) {
          it = take_item(item);
          if (!it || has_rows(it)) break;
          step += it->j1 - it->j0;
          bar_arrive_warp(bar_ie(item));
        }
        if (!it) break;
        load_queries(it);
        scale_queries();
        queries_in();
      }
      const int row_first = it->row_first + i * 128, rows = it->rows;
      const int j0 = it->j0, j1 = it->j1;
      const float F = fs[r];  // (rows of this warp: written by this warp)
      const int row = row_first + r;
      const bool in = row < rows;
      // (rows behind the last have queries of 0 and no output: nothing to hide)
      const int limit = (int)min(in ? it->pos0 + row / p.rg : (int64_t)it->len, (int64_t)it->len - 1);
      // newest position every row of the tile sees (its first row's)
      const int least = (int)min(it->pos0 + row_first / p.rg, (int64_t)it->len - 1);
      float ref = kNoRef, l = 0.0f;  // reference and sum of the row's weights
      float over = 0.0f;             // by how much the last step's scores passed it
      for (int j = j0; j < j1; ++j, ++step) {
        if (!(ok = wait_warp(bar_s(i), sn & 1))) break;
        tc_fence_after();
        const uint32_t bad = steps[step % kSteps].bad;  // a bit per 16 tokens
        const bool masked = j * kStep + kStep - 1 > least || bad != 0;
        // these scores were issued after the sums of the earlier steps and are
        // here, so those are complete and O may be scaled
        auto rescale = [&](float f) {
          l *= f;
          if (j > j0) {
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t y[16];
              tc_ld16(to + c, y);
              tc_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * f);
              tc_st16(to + c, y);
            }
            tc_wait_st();
          }
        };
        // the reference moves where the last step's scores passed it by more
        // than the slack, back to kChunkBase below them
        if (__any_sync(0xffffffffu, over > kChunkSlack)) {
          const float by = over > kChunkSlack ? over - kChunkBase : 0.0f;
          rescale(exp2_approx(-by));
          ref += by;
        }
        over = 0.0f;
        auto hide = [&](uint32_t (&y)[32], int c) {
          const int seen = limit - j * kStep - 32 * c;  // columns 0 .. seen
          const uint32_t b2 = bad >> (2 * c);
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (k > seen || (b2 >> (k / 16) & 1)) y[k] = 0xff800000u;
        };
        float sum0 = 0.0f, sum1 = 0.0f;
        // The usual step: nothing to hide.  Straight code without a branch, the
        // weights kept in registers until the maximum is known.  Where fp16 could
        // not hold one, or the row has no reference yet, that moves to
        // kChunkBase below the maximum and the step is taken once more.
        if (!masked) {
          uint32_t w[64];
          float top;
#pragma unroll 1
          for (int again = 0;; ++again) {
            uint32_t x[2][16];
            float m0 = -INFINITY, m1 = -INFINITY;
            const uint64_t F2 = pair64(F, F), R2 = pair64(-ref, -ref);
            uint64_t sa = 0, sb = 0;
            tc_ld16(ts, x[0]);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              uint32_t (&y)[16] = x[c & 1];
              tc_wait_ld();
              if (c < 7) tc_ld16(ts + 16 * (c + 1), x[(c + 1) & 1]);
#pragma unroll
              for (int k = 0; k < 16; k += 4) {
                m0 = max3(m0, __uint_as_float(y[k]), __uint_as_float(y[k + 1]));
                m1 = max3(m1, __uint_as_float(y[k + 2]), __uint_as_float(y[k + 3]));
                const float2 a0 = unpair64(fma2(pair64u(y[k], y[k + 1]), F2, R2));
                const float2 a1 = unpair64(fma2(pair64u(y[k + 2], y[k + 3]), F2, R2));
                const float p0 = exp2_approx(a0.x), p1 = exp2_approx(a0.y);
                const float p2 = exp2_approx(a1.x), p3 = exp2_approx(a1.y);
                sa = add2(sa, pair64(p0, p1));
                sb = add2(sb, pair64(p2, p3));
                w[8 * c + k / 2] = h2u(__floats2half2_rn(p0, p1));
                w[8 * c + k / 2 + 1] = h2u(__floats2half2_rn(p2, p3));
              }
            }
            const float m = fmaxf(m0, m1);
            top = fmaf(m, F, -ref);
            const float2 s0 = unpair64(sa), s1 = unpair64(sb);
            sum0 = s0.x + s0.y, sum1 = s1.x + s1.y;
            if (again || !__any_sync(0xffffffffu, top > kChunkTop)) break;
            const bool first = ref == kNoRef, jump = top > kChunkTop;
            const float by = jump && !first ? top - kChunkBase : 0.0f;
            rescale(exp2_approx(-by));
            if (jump) ref = first ? fmaf(m, F, -kChunkBase) : ref + by;
          }
          over = fmaxf(top, 0.0f);
          tc_st32(ts, w);
          tc_st32(ts + 32, w + 32);
        } else {
        uint32_t x[2][32];
        tc_ld32(ts, x[0]);
        // (rolled: straight-line code for a whole row runs out of the
        // instruction caches that the roles share)
#pragma unroll 1
        for (int c2 = 0; c2 < 4; c2 += 2) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int c = c2 + e;
            uint32_t (&y)[32] = x[e];
            tc_wait_ld();
            if (c < 3) tc_ld32(ts + 32 * (c + 1), x[e ^ 1]);
            if (masked) hide(y, c);
            float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              m0 = max3(m0, __uint_as_float(y[k]), __uint_as_float(y[k + 1]));
              m1 = max3(m1, __uint_as_float(y[k + 2]), __uint_as_float(y[k + 3]));
            }
            const float m = fmaxf(m0, m1);
            float top = fmaf(m, F, -ref);
            if (__any_sync(0xffffffffu, top > kChunkTop)) {
              // A weight that fp16 could not hold, or a row's first scores: the
              // reference moves now, and with it the weights stored before (by a
              // power of two: exact for those that stay normal).
              const bool first = ref == kNoRef, jump = top > kChunkTop;
              const float by = jump && !first ? floorf(top) - kChunkBase : 0.0f;
              const float f = jump && first ? 0.0f : exp2_approx(-by);
              sum0 *= f, sum1 *= f;
              const uint32_t f2 = h2u(__float2half2_rn(f));
              tc_wait_st();
#pragma unroll 1
              for (int b8 = 0; b8 < 16 * c; b8 += 16) {
                uint32_t v[16];
                tc_ld16(ts + b8, v);
                tc_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; ++k)
                  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(v[k]) : "r"(v[k]), "r"(f2));
                tc_st16(ts + b8, v);
              }
              rescale(f);
              if (jump) {
                ref = first ? fmaf(m, F, -kChunkBase) : ref + by;
                over = 0.0f;
              }
              top = fmaf(m, F, -ref);
            }
            over = fmaxf(over, top);
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              const float p0 = exp2_approx(fmaf(__uint_as_float(y[k]), F, -ref));
              const float p1 = exp2_approx(fmaf(__uint_as_float(y[k + 1]), F, -ref));
              const float p2 = exp2_approx(fmaf(__uint_as_float(y[k + 2]), F, -ref));
              const float p3 = exp2_approx(fmaf(__uint_as_float(y[k + 3]), F, -ref));
              sum0 += p0 + p1;
              sum1 += p2 + p3;
              w[k / 2] = h2u(__floats2half2_rn(p0, p1));
              w[k / 2 + 1] = h2u(__floats2half2_rn(p2, p3));
            }
            // columns 16c .. 16c + 15: read already, 32c + 32 and up are not touched
            tc_st16(ts + 16 * c, w);
          }
        }
        }
        l += sum0 + sum1;
        tc_wait_st();
        tc_fence_before();
        bar_arrive_warp(bar_p(i));
        ++sn;
      }
      if (!ok) break;

      // the next item's queries come in while the last sums are added (this item's scores
      // are all there, so its own are not needed any more), and its first scores are
      // computed during this item's output.  Only the next item, though: this one still
      // holds its entry of the ring, which the list refills once all have let go, so a
      // tile that skipped on from here past items without rows for it could wait for
      // itself.
      const uint32_t this_item = item++;
      const Item *next = take_item(item);
      if (next && !has_rows(next)) next = nullptr;  // taken up after the release
      if (next) {
        load_queries(next);
        scale_queries();
        queries_in();
      }
      if (!(ok = wait_warp(bar_o(i), on++ & 1))) break;
      tc_fence_after();
      // ---- output of the tile's steps [j0, j1)
      const bool whole = j0 == 0 && j1 == it->steps;
      const int64_t t = it->row0 + (in ? row / p.rg : 0);
      uint16_t *dst = a.out + (t * p.Hq + it->h * p.rg + row % p.rg) * D;
      // 32 columns of the output row, scaled, to their channels
      auto put = [&](int c32, const float (&v)[32], float inv) {
#pragma unroll
        for (int G = 0; G < NG; ++G) {
          // column ((g * NG/2 + h) * 4 + i) * 2 + e, channel 32 * (2h + e) + 4 * g + i
          constexpr int kG = 16 / NG * 2;   // channels of one group in 32 columns
          uint32_t w[kG / 2];
#pragma unroll
          for (int c = 0; c < kG; c += 2) {
            const int n0 = ((c / 4 * (NG / 2) + G / 2) * 4 + c % 4) * 2 + (G & 1);
            if (p.bf16) {
              const __nv_bfloat162 h = __floats2bfloat162_rn(v[n0] * inv, v[n0 + 2] * inv);
              w[c / 2] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
              w[c / 2] = h2u(__floats2half2_rn(v[n0] * inv, v[n0 + 2] * inv));
            }
          }
#pragma unroll
          for (int c = 0; c < kG / 2; c += 4)
            *reinterpret_cast<uint4 *>(dst + 32 * G + c32 / 32 * kG + 2 * c) =
                make_uint4(w[c], w[c + 1], w[c + 2], w[c + 3]);
        }
      };
      if (whole) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t y[32];
          __syncwarp();
          tc_ld32(to + c, y);
          tc_wait_ld();
          float v[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(y[k]);
          if (in) put(c, v, inv);
        }
      } else {
        const int c0 = it->c0, c1 = it->c1;
        const int slot = 2 * blockIdx.x + (j0 == 0 ? 1 : 0);
        float4 *wo = reinterpret_cast<float4 *>(a.ws_o) + (int64_t)(slot * 2 + i) * (D / 4) * 128 + r;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t y[32];
          __syncwarp();
          tc_ld32(to + c, y);
          tc_wait_ld();
          if (in) {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              wo[(c + k) / 4 * 128] = make_float4(__uint_as_float(y[k]), __uint_as_float(y[k + 1]),
                                                  __uint_as_float(y[k + 2]),
                                                  __uint_as_float(y[k + 3]));
          }
        }
        float2 *wm = reinterpret_cast<float2 *>(a.ws_ml) + (slot * 2 + i) * 128 + r;
        *wm = make_float2(ref, l);
        __threadfence();
        bar_arrive_warp(bar_g(i));
        if (!(ok = wait_warp(bar_g(i), gn++ & 1))) break;
        volatile uint32_t *flag = misc + 12 + i;
        if (r == 0) {
          int *count = a.ws_count + c0 * 2 + i;
          const int last = atomicAdd(count, 1) == c1 - c0;
          if (last) *count = 0;
          *flag = last;
        }
        bar_arrive_warp(bar_g(i));
        if (!(ok = wait_warp(bar_g(i), gn++ & 1))) break;
        if (*flag) {
          __threadfence();
          const float2 *ml = reinterpret_cast<const float2 *>(a.ws_ml);
          float m = kNoRef, sum = 0.0f;
#pragma unroll 4
          for (int c = c0; c <= c1; ++c) {
            const float2 y = __ldcg(ml + ((2 * c + (c == c0)) * 2 + i) * 128 + r);
            const float nm = fmaxf(m, y.x);
            sum = sum * exp2_approx(m - nm) + y.y * exp2_approx(y.x - nm);
            m = nm;
          }
          const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
          if (in) {
#pragma unroll 1
            for (int c32 = 0; c32 < D; c32 += 32) {
              // (two parts' loads in flight; a part without visible tokens is 0)
              float v[32] = {};
#pragma unroll 2
              for (int c = c0; c <= c1; ++c) {
                const int at = (2 * c + (c == c0)) * 2 + i;
                const float4 *src = reinterpret_cast<const float4 *>(a.ws_o) +
                                    (int64_t)at * (D / 4) * 128 + c32 / 4 * 128 + r;
                float4 w[8];
                const float2 y = __ldcg(ml + at * 128 + r);
#pragma unroll
                for (int k = 0; k < 8; ++k) w[k] = __ldcg(src + k * 128);
                const float f = exp2_approx(y.x - m);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  v[4 * k] += f * w[k].x;
                  v[4 * k + 1] += f * w[k].y;
                  v[4 * k + 2] += f * w[k].z;
                  v[4 * k + 3] += f * w[k].w;
                }
              }
              put(c32, v, inv);
            }
          }
        }
      }
      bar_arrive_warp(bar_ie(this_item));
      it = next;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

template <int D, int BITS>
cudaError_t chunk_as(const ChunkArgs &a, int num_sms, cudaStream_t st) {
  static KernelSetup setup;
  constexpr int smem = ChunkCfg<D>::smem;
  // the register split draws on what the block is launched with: a kernel built
  // with fewer registers a thread would wait for the rest forever
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, paged_chunk_kernel<D, BITS>);
    if (e != cudaSuccess) return e;
    regs.store(fa.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) * kChunkThreads <
      256 * kSoftRegs + 256 * kProducerRegs + 128 * kOtherRegs)
    return cudaErrorInvalidConfiguration;
  auto kern = paged_chunk_kernel<D, BITS>;
  const cudaError_t e = kernel_setup(setup, kern, kChunkThreads, smem, nullptr);
  if (e != cudaSuccess) return e;
  const int blocks = num_sms < kMaxChunkBlocks ? num_sms : kMaxChunkBlocks;
  return launch_dependent(kern, (unsigned)blocks, kChunkThreads, smem, st, false, a);
}

constexpr size_t kCountBytes = 2 * kMaxChunkBlocks * 4;
constexpr size_t kMlBytes = (size_t)2 * kMaxChunkBlocks * kTileRows * 8;

}  // namespace

cudaError_t launch_paged_chunk(const Paged &p, const void *q, int64_t qs, void *out, float scale,
                               int few, void *ws, int num_sms, cudaStream_t st) {
  ChunkArgs a;
  a.p = p;
  a.q = static_cast<const uint16_t *>(q);
  a.qs = qs;
  a.out = static_cast<uint16_t *>(out);
  a.scale_log2 = fminf(fabsf(scale) * 1.4426950408889634f, kMostScale);
  a.sign = scale < 0.0f ? -1.0f : 1.0f;
  a.few = few;
  uint8_t *w = static_cast<uint8_t *>(ws);
  a.ws_count = reinterpret_cast<int *>(w);
  a.ws_ml = reinterpret_cast<float *>(w + kCountBytes);
  a.ws_o = reinterpret_cast<float *>(w + kCountBytes + kMlBytes);
  a.stall_limit = debug_stall_limit();
  if (p.d == 128)
    return p.bits == 2   ? chunk_as<128, 2>(a, num_sms, st)
           : p.bits == 4 ? chunk_as<128, 4>(a, num_sms, st)
                         : chunk_as<128, 8>(a, num_sms, st);
  return p.bits == 2   ? chunk_as<64, 2>(a, num_sms, st)
         : p.bits == 4 ? chunk_as<64, 4>(a, num_sms, st)
                       : chunk_as<64, 8>(a, num_sms, st);
}

size_t paged_chunk_workspace() {
  return kCountBytes + kMlBytes + (size_t)2 * kMaxChunkBlocks * kTileRows * kMaxHeadDim * 4;
}

}  // namespace kvq
