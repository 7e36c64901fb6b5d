// Paged cache: cross attention of 9 to 32 query rows per KV head (a few beams or
// samples of grouped heads), on tcgen05 with the operands' roles turned: cached tokens
// and channels are the 128 MMA rows, query rows the columns.
//   S^T = K Q^T        128 tokens x NR rows      both operands in shared memory
//   P^T = 2^(S^T F - ref)   a thread a token; fp16, to shared memory
//   O^T (+)= V^T P^T   128 channels x NR rows    V read as it lies, P as the N operand
// so a step of 128 tokens costs the tensor core 2 * NR / 128 of what a tile of 128 rows
// does, and an exponential a token and row that exists.
//
// What bounds it: the cache is read once, as by the split kernel (kvq_paged_rows.cu),
// and each code becomes an fp16 operand element by about 1.7 lane instructions, shared by
// all rows; the exponentials are NR a token.
//
//  * Split: the 128-token steps of all (sequence, head) pairs form one list, cut into
//    equal ranges, one per block (one a SM).  Pairs that several blocks share leave
//    partials, joined in block order by the block that finishes last.
//  * Two softmax groups of four warps (0-3, 4-7) take every other step, each with an
//    accumulator and reference of its own, joined at a pair's end, so that one group's
//    exponentials cover the other's waits.  Warps 8-15 turn codes into swizzled operand
//    tiles, warp 16 issues the products, warp 17 copies atoms into a ring of 64-token
//    slots (cp.async.bulk); 18 and 19 only give up registers.
//  * A row's reference moves only when a score passes it by 15 (log2 units), back to 4
//    below the largest: as in the chunk kernel weights down to 2^-18 of the largest are
//    normal fp16 numbers.  Whether any does is one vote a step.
//  * Every role walks the block's range by itself; only bytes and their presence go
//    through rings.
#include "kvq_paged.cuh"
#include "kvq_umma.cuh"

namespace kvq {

int debug_stall_limit();

namespace {

constexpr int kD128 = 128;
constexpr int kStep = 128;         // cached tokens per step
constexpr int kSlot = 64;          // ... per slot of the ring
constexpr int kTileBytes = kStep * kD128 * 2;
constexpr int kProducer0 = 8, kProducers = 8, kMmaWarp = 16, kLoadWarp = 17;
constexpr int kCrossThreads = 640;
// Registers a thread, of the 640 * 96 at launch: softmax, producers, the others.
// 256 * 136 + 256 * 80 + 128 * 48 = 61440.
constexpr int kSoftRegs = 136, kProducerRegs = 80, kOtherRegs = 48;
constexpr int kRegSum = 256 * kSoftRegs + 256 * kProducerRegs + 128 * kOtherRegs;
static_assert(kRegSum <= kCrossThreads * 96, "registers");
constexpr int kBad = 16;           // steps whose missing atoms are known
constexpr int kMaxCrossBlocks = 160;
constexpr int kMinSteps = 4;       // a block's least
constexpr int kCrossWait = 1 << 25;
constexpr float kCrossBase = 4.0f, kCrossTop = 15.0f;
constexpr float kNoRef = -1e30f;

struct CrossArgs {
  Paged p;
  const uint16_t *q;
  int64_t qs;
  uint16_t *out;
  float scale_log2;  // >= 0
  float sign;        // of the softmax scale, folded into the queries
  int *ws_count;     // [blocks], zero between calls
  float *ws_ml;      // [2 * blocks][NR][2]
  float *ws_o;       // [2 * blocks][NR][128]
  int stall_limit;
};

template <int BITS, int NR>
struct CrossCfg {
  static constexpr int RB = kD128 * BITS / 8, SB = 16, AB = 2 * kAtom * (RB + SB);
  static constexpr int kSlotBytes = kSlot / kAtom * AB;
  // about 50 to 60 KB on their way
  static constexpr int R = BITS == 2 ? 8 : BITS == 4 ? (NR == 16 ? 6 : 5) : 3;
  static constexpr int off_k = 0;
  static constexpr int off_v = off_k + 2 * kTileBytes;
  static constexpr int off_q = off_v + 2 * kTileBytes;
  static constexpr int off_p = off_q + NR * kD128 * 2;          // two tiles [NR][128 tokens]
  static constexpr int off_raw = off_p + 2 * NR * kStep * 2;
  static constexpr int off_f = off_raw + R * kSlotBytes;         // [2 items][NR]
  static constexpr int off_ref = off_f + 2 * NR * 4;             // [2 groups][NR]
  static constexpr int off_max = off_ref + 2 * NR * 4;           // [2 groups][4 warps][NR]
  static constexpr int off_l = off_max + 8 * NR * 4;             // the same
  static constexpr int off_bad = off_l + 8 * NR * 4;
  static constexpr int kBars = 2 * R + 17;
  static constexpr int off_bar = off_bad + kBad * 4;
  static constexpr int off_misc = off_bar + kBars * 8 + 8;
  static constexpr int off_prefix = off_misc + 32;
  static int smem(int seqs) { return off_prefix + (seqs + 1) * 8 + 1024; }
  static_assert(off_p % 1024 == 0 && off_q % 1024 == 0, "swizzled tiles");
  static_assert(off_prefix + (kMaxSeqs + 1) * 8 + 1024 <= 227 * 1024, "shared memory");
  // the groups' outputs are joined where their weights were
  static_assert(2 * NR * kStep * 2 >= NR * kD128 * 4, "room for one group's output");
};

// The block's share of one pair, found by every role alike.
struct Item {
  int b, h, j0, j1, steps;
  int64_t first;  // the pair's first unit in the list
};

template <int BITS, int NR>
__global__ void __launch_bounds__(kCrossThreads, 1)
paged_cross_kernel(const __grid_constant__ CrossArgs a) {
  using C = CrossCfg<BITS, NR>;
  constexpr int RB = C::RB, SB = C::SB, AB = C::AB, R = C::R, NG = 4;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t smem_s = smem_u32(smem);
  const Paged &p = a.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t bars = smem_s + C::off_bar;
  auto bar_rf = [&](uint32_t s) { return bars + 8u * s; };        // raw slot full / empty
  auto bar_re = [&](uint32_t s) { return bars + 8u * (R + s); };
  auto bar_kf = [&](uint32_t s) { return bars + 8u * (2 * R + s); };      // key stage
  auto bar_ke = [&](uint32_t s) { return bars + 8u * (2 * R + 2 + s); };
  auto bar_vf = [&](uint32_t s) { return bars + 8u * (2 * R + 4 + s); };  // value stage
  auto bar_ve = [&](uint32_t s) { return bars + 8u * (2 * R + 6 + s); };
  auto bar_s = [&](uint32_t g) { return bars + 8u * (2 * R + 8 + g); };   // scores of group g
  auto bar_p = [&](uint32_t g) { return bars + 8u * (2 * R + 10 + g); };  // its weights
  auto bar_o = [&](uint32_t g) { return bars + 8u * (2 * R + 12 + g); };  // its output
  const uint32_t bar_qf = bars + 8u * (2 * R + 14), bar_qe = bars + 8u * (2 * R + 15);
  const uint32_t bar_end = bars + 8u * (2 * R + 16);
  uint32_t *misc = reinterpret_cast<uint32_t *>(smem + C::off_misc);
  volatile uint32_t *dead = misc + 1;
  int64_t *prefix = reinterpret_cast<int64_t *>(smem + C::off_prefix);
  volatile uint32_t *missing = reinterpret_cast<uint32_t *>(smem + C::off_bad);

  grid_dep_trigger();
  if (tid == 0) {
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::off_bar);
    for (int i = 0; i < R; ++i) bar_init(bar + i, 1), bar_init(bar + R + i, kProducers);
    for (int i = 0; i < 2; ++i) {
      bar_init(bar + 2 * R + i, kProducers);
      bar_init(bar + 2 * R + 2 + i, 1);
      bar_init(bar + 2 * R + 4 + i, kProducers);
      bar_init(bar + 2 * R + 6 + i, 1);
      bar_init(bar + 2 * R + 8 + i, 1);
      bar_init(bar + 2 * R + 10 + i, 4);
      bar_init(bar + 2 * R + 12 + i, 1);
    }
    bar_init(bar + 2 * R + 14, 4);
    bar_init(bar + 2 * R + 15, 1 + 4);
    bar_init(bar + 2 * R + 16, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    misc[1] = 0;
  }
  grid_dep_wait();

  // ---- the list: steps of one head of sequences 0 .. b at [b + 1]
  const int64_t cap = p.width * p.page;
  for (int b = tid; b < p.B; b += kCrossThreads) {
    const int64_t n = (int64_t)p.cu[b + 1] - p.cu[b], len = p.lens[b];
    int64_t v = 0;
    if (bad_rows(p, b)) {
      if (blockIdx.x == 0) paged_error(p, KVQ_EINVAL);
    } else if (n > 0) {
      if (len > cap && blockIdx.x == 0) paged_error(p, KVQ_EPAGE);
      v = (min(len, cap) + kStep - 1) / kStep;
      if (v < 1) v = 1;  // rows that see nothing are written too
    }
    prefix[b + 1] = v;
  }
  __syncthreads();
  if (warp == 0) {  // running sums
    int64_t before = 0;
    if (lane == 0) prefix[0] = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      int64_t v = b0 + lane < p.B ? prefix[b0 + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += up;
      }
      v += before;
      if (b0 + lane < p.B) prefix[b0 + lane + 1] = v;
      before = __shfl_sync(0xffffffffu, v, 31);
    }
  } else if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_s + C::off_misc),
                 "n"(4 * NR)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  auto tm_s = [&](uint32_t g) { return tmem + NR * g; };
  auto tm_o = [&](uint32_t g) { return tmem + NR * (2 + g); };
  const int H = p.H;
  const int64_t total = H * prefix[p.B];
  const int64_t U = max((total + gridDim.x - 1) / (int64_t)gridDim.x, (int64_t)kMinSteps);
  const int64_t x0 = min(blockIdx.x * U, total), x1 = min(x0 + U, total);

  auto wait = [&](uint32_t bar, uint32_t parity, int ns = 20) {
    for (int i = 0; i < kCrossWait; ++i) {
      if (bar_try_wait(bar, parity)) return true;
      __nanosleep(ns);
      if ((i & 63) == 63 && *dead) return false;
    }
    *dead = 1;
    paged_error(p, KVQ_ETIMEOUT);
    return false;
  };
  auto wait_warp = [&](uint32_t bar, uint32_t parity, int ns = 20) {
    return (bool)__all_sync(0xffffffffu, wait(bar, parity, ns));
  };
  if (a.stall_limit > 0 && tid == 0) {
    bool ok = false;
    for (int i = 0; i < a.stall_limit && !ok; ++i) ok = bar_try_wait(bar_end, 0);
    if (!ok) {
      *dead = 1;
      paged_error(p, KVQ_ETIMEOUT);
    }
  }
  // the item that begins at unit x (< x1); b: a sequence at or before its own
  auto item_at = [&](int64_t x, int b) {
    Item it;
    while (H * prefix[b + 1] <= x) ++b;
    it.b = b;
    it.steps = (int)(prefix[b + 1] - prefix[b]);
    const int64_t r = x - H * prefix[b];
    it.h = (int)(r / it.steps);
    it.j0 = (int)(r - (int64_t)it.h * it.steps);
    it.first = x - it.j0;
    it.j1 = (int)min((int64_t)it.steps, it.j0 + (x1 - x));
    return it;
  };
  int start_b = 0;
  if (x0 < x1) {
    int lo = 0, hi = p.B;  // the last b with H * prefix[b] <= x0
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (H * prefix[mid] <= x0) lo = mid; else hi = mid;
    }
    start_b = lo;
  }
  auto length = [&](int b) { return (int)min((int64_t)max(p.lens[b], 0), cap); };

  if (warp >= kMmaWarp) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == kLoadWarp) {
    // ---- atoms into the ring, 64 tokens a slot, two slots a step
    const int apage_log = __ffs(p.page / kAtom) - 1;
    uint32_t sn = 0, step = 0;  // slots filled, steps
    bool ok = true;
    int b = start_b;
    for (int64_t x = x0; ok && x < x1;) {
      const Item it = item_at(x, b);
      b = it.b;
      x += it.j1 - it.j0;
      const int len = length(b), atoms = (len + kAtom - 1) / kAtom;
      const int32_t *row = p.table + (int64_t)b * p.width;
      // page numbers of 32 atoms, and of the next 32 on their way
      auto ids_of = [&](int atom) {
        return atom + lane < atoms ? __ldg(row + ((atom + lane) >> apage_log)) : -1;
      };
      int base = it.j0 * (kStep / kAtom);
      int ids = ids_of(base), next = ids_of(base + 32);
      uint32_t lost = 0;  // of the step: atoms that belong to the sequence but have no page
      for (int s = 2 * it.j0; ok && s < 2 * it.j1; ++s, ++sn) {
        const int atom0 = s * (kSlot / kAtom);
        if (atom0 - base == 32) {
          base = atom0;
          ids = next;
          next = ids_of(base + 32);
        }
        const int64_t id = __shfl_sync(0xffffffffu, ids, (atom0 - base + lane) & 31);
        const int atom = atom0 + lane;
        const bool mine = lane < kSlot / kAtom && atom < atoms;
        const bool there = mine && id >= 0 && id < p.n_pages;
        const uint32_t have = __ballot_sync(0xffffffffu, there);
        const uint32_t gone = __ballot_sync(0xffffffffu, mine && !there);
        lost = (s & 1) ? lost | gone << 4 : gone;
        const uint32_t slot = sn % R;
        if (sn >= R && !(ok = wait_warp(bar_re(slot), (sn / R - 1) & 1))) break;
        if (lane == 0) {
          if (gone) paged_error(p, KVQ_EPAGE);
          if (s & 1) missing[step % kBad] = lost;
          // (the arrival also hands over what was written above)
          bar_expect_tx(reinterpret_cast<uint64_t *>(smem + C::off_bar) + slot,
                        (uint32_t)__popc(have) * AB);
        }
        __syncwarp();
        if (there)
          bulk_g2s(smem + C::off_raw + slot * C::kSlotBytes + lane * AB,
                   p.pages + id * p.page_bytes + it.h * p.head_bytes +
                       (int64_t)(atom & ((1 << apage_log) - 1)) * AB,
                   AB, reinterpret_cast<uint64_t *>(smem + C::off_bar) + slot);
        if (s & 1) ++step;
      }
    }
    if (*dead) {
      // copies on their way end before the block does
      const uint32_t n = min(sn, (uint32_t)R);
      for (uint32_t i = sn - n; i < sn; ++i)
        bar_wait(bar_rf(i % R), (i / R) & 1, kDrainLimit);
    }
  } else if (warp == kMmaWarp) {
    // ---- products: scores of a step, then the weighted values of the one before
    constexpr uint32_t kQK = mma_desc(NR, false);
    constexpr uint32_t kPV = mma_desc(NR, false, true);
    const uint64_t k_desc = smem_desc(smem_s + C::off_k, 16, 1024);
    const uint64_t v_desc = smem_desc(smem_s + C::off_v, kStep * 128, 1024);
    const uint64_t q_desc = smem_desc(smem_s + C::off_q, 16, 1024);
    const uint64_t p_desc = smem_desc(smem_s + C::off_p, 16, 1024);
    const bool leader = elect_one();
    auto commit = [&](uint32_t bar) {
      if (leader) tc_commit(bar);
      __syncwarp();
    };
    auto outputs = [&](uint32_t s, bool first) {
      if (leader) {
        const uint64_t vd = v_desc + (s & 1) * (kTileBytes / 16);
        const uint64_t pd = p_desc + (s & 1) * (NR * kStep * 2 / 16);
#pragma unroll
        for (int k = 0; k < kStep / 16; ++k)
          mma_ss(tm_o(s & 1), vd + k * (2048 / 16),
                 pd + ((k / 4) * (NR * 128) + (k % 4) * 32) / 16, kPV, !(first && k == 0));
        tc_commit(bar_ve(s & 1));
      }
      __syncwarp();
    };
    uint32_t s = 0, items = 0;
    bool ok = true;
    int b = start_b;
    for (int64_t x = x0; ok && x < x1; ++items) {
      const Item it = item_at(x, b);
      b = it.b;
      const int n = it.j1 - it.j0;
      x += n;
      if (!(ok = wait_warp(bar_qf, items & 1))) break;
      for (int j = 0; j <= n; ++j) {
        if (j < n) {
          const uint32_t g = (s + j) & 1;
          if (!(ok = wait_warp(bar_kf(g), ((s + j) >> 1) & 1))) break;
          tc_fence_after();
          if (leader) {
            const uint64_t kd = k_desc + g * (kTileBytes / 16);
#pragma unroll
            for (int k = 0; k < kD128 / 16; ++k)
              mma_ss(tm_s(g), kd + ((k / 4) * (kStep * 128) + (k % 4) * 32) / 16,
                     q_desc + ((k / 4) * (NR * 128) + (k % 4) * 32) / 16, kQK, k > 0);
            tc_commit(bar_s(g));
            tc_commit(bar_ke(g));
            if (j == n - 1) tc_commit(bar_qe);
          }
          __syncwarp();
        }
        if (j > 0) {
          const uint32_t t = s + j - 1, g = t & 1;
          ok = wait_warp(bar_vf(g), (t >> 1) & 1) && wait_warp(bar_p(g), (t >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          outputs(t, j <= 2);
          if (j >= n - 1) commit(bar_o(g));
        }
      }
      s += n;
    }
    commit(bar_end);
    bool done = false;
    for (int i = 0; i < kCrossWait && !done; ++i) done = bar_try_wait(bar_end, 0);
    __syncwarp();
  }
  } else if (warp >= kProducer0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    // ---- producers: thread (quarter jq, token t8 of eight), a token of each slot
    constexpr int QW = RB / 16;  // words of a quarter row
    const int pw = warp - kProducer0, t8 = lane & 7, jq = lane >> 3;
    const uint32_t row = 8 * (pw & 1) + t8;  // in the atom pw / 2 of the slot
    const uint32_t code_at = (pw >> 1) * AB + row * RB + jq * (RB / 4);
    const uint32_t stat_at = (pw >> 1) * AB + 2 * kAtom * RB + row * SB;
    uint32_t s = 0;
    bool ok = true;
    int b = start_b;
    for (int64_t x = x0; ok && x < x1;) {
      const Item it = item_at(x, b);
      b = it.b;
      x += it.j1 - it.j0;
      const int len = length(b);
      for (int j = it.j0; ok && j < it.j1; ++j, ++s) {
        uint32_t kraw[2][QW], kst[2][4], vraw[2][QW], vst[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t n = 2 * s + u, slot = n % R;
          if (!(ok = wait_warp(bar_rf(slot), (n / R) & 1))) break;
          const uint8_t *src = smem + C::off_raw + slot * C::kSlotBytes;
          auto words = [&](const uint8_t *at, uint32_t (&w)[QW]) {
            if constexpr (QW % 4 == 0) {
#pragma unroll
              for (int i = 0; i < QW; i += 4) {
                const uint4 v = *reinterpret_cast<const uint4 *>(at + 4 * i);
                w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
              }
            } else {
              const uint2 v = *reinterpret_cast<const uint2 *>(at);
              w[0] = v.x, w[1] = v.y;
            }
          };
          words(src + code_at, kraw[u]);
          words(src + code_at + kAtom * RB, vraw[u]);
          const uint4 ks = *reinterpret_cast<const uint4 *>(src + stat_at);
          const uint4 vs = *reinterpret_cast<const uint4 *>(src + stat_at + kAtom * SB);
          // (a step's lost atoms are known once its second slot is)
          kst[u][0] = ks.x, kst[u][1] = ks.y, kst[u][2] = ks.z, kst[u][3] = ks.w;
          vst[u][0] = vs.x, vst[u][1] = vs.y, vst[u][2] = vs.z, vst[u][3] = vs.w;
        }
        if (!ok) break;
        // statistics 0 where there is no token: nothing there may reach an output
        const uint32_t lost = missing[s % kBad];
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (j * kStep + kSlot * u + 8 * pw + t8 >= len || (lost >> (4 * u + (pw >> 1)) & 1)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) kst[u][i] = vst[u][i] = 0;
          }
        // (the reads are done: their values are looked at above)
        bar_arrive_warp(bar_re((2 * s) % R));
        bar_arrive_warp(bar_re((2 * s + 1) % R));
        const uint32_t stage = s & 1;
        if (s >= 2 && !(ok = wait_warp(bar_ke(stage), ((s >> 1) - 1) & 1))) break;
        const uint32_t k_tile = smem_s + C::off_k + stage * kTileBytes;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int trow = kSlot * u + 8 * pw + t8;
#pragma unroll
          for (int G = 0; G < NG; ++G) {
            const uint32_t sel = G & 1 ? 0x3232u : 0x1010u;
            const uint32_t sc = __byte_perm(kst[u][G / 2], 0, sel);
            const uint32_t z = __byte_perm(kst[u][2 + G / 2], 0, sel);
            uint32_t y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int bit = (4 * G + i) * BITS, w = bit / 16, off = bit % 16;
              y[i] = hfma2(code_pair<BITS>(off & 8 ? kraw[u][w] >> 8 : kraw[u][w], off & 7), sc, z);
            }
            const int unit = (G & 1) * 4 + jq;  // channels 32G + 8jq .. + 7
            sts128(k_tile + (G / 2) * (kStep * 128) + trow * 128 + ((unit ^ t8) << 4), y);
          }
        }
        async_fence();
        bar_arrive_warp(bar_kf(stage));
        if (s >= 2 && !(ok = wait_warp(bar_ve(stage), ((s >> 1) - 1) & 1))) break;
        const uint32_t v_tile = smem_s + C::off_v + stage * kTileBytes;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int trow = kSlot * u + 8 * pw + t8;
#pragma unroll
          for (int e8 = 0; e8 < 2; ++e8) {  // eighths 2jq, 2jq + 1
#pragma unroll
            for (int h = 0; h < NG / 2; ++h) {
              uint32_t y[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int bit = (4 * h + i) * BITS, off = bit % 16;
                const uint32_t w = vraw[u][(e8 * (RB / 8) / 4 + bit / 16) % QW];
                y[i] = hfma2(code_pair<BITS>(off & 8 ? w >> 8 : w, off & 7), vst[u][h],
                             vst[u][2 + h]);
              }
              // columns ((eighth * 2 + h) * 4 + i) * 2 + e hold channel
              // 32 * (2h + e) + 4 * eighth + i
              const int unit = (2 * jq + e8) * 2 + h;
              sts128(v_tile + (unit >> 3) * (kStep * 128) + trow * 128 + (((unit & 7) ^ t8) << 4),
                     y);
            }
          }
        }
        async_fence();
        bar_arrive_warp(bar_vf(stage));
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ---- softmax and output: group g takes the steps of its parity, a thread a token
    // (scores) or a channel (output)
    const uint32_t g = warp >> 2;
    const int w4 = warp & 3, r = 32 * w4 + lane, gt = tid;
    const uint32_t lane_base = (uint32_t)w4 * 32u << 16;
    const uint32_t ts = tm_s(g) + lane_base, to = tm_o(g) + lane_base;
    float *fs = reinterpret_cast<float *>(smem + C::off_f);
    float *refs = reinterpret_cast<float *>(smem + C::off_ref);
    float *maxima = reinterpret_cast<float *>(smem + C::off_max) + g * 4 * NR;
    float *sums = reinterpret_cast<float *>(smem + C::off_l);
    float *myref = refs + g * NR;
    // the weights of token r of row n lie at pt + n * 128 + ((n & 7) << 4 ^ px)
    const uint32_t pt = smem_s + C::off_p + g * (NR * kStep * 2) + (r >> 6) * (NR * 128) +
                        (r & 7) * 2;
    const uint32_t px = (uint32_t)((r & 63) >> 3) << 4;
    // meetings of a group, and of both
    auto meet = [&]() { asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + g) : "memory"); };
    auto meet_all = [&]() { asm volatile("barrier.cta.sync 3, 256;" ::: "memory"); };
    auto any_of_group = [&](bool x) {
      uint32_t y;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n"
          " barrier.cta.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
          : "=r"(y)
          : "r"((uint32_t)x), "r"(1 + g)
          : "memory");
      return y != 0;
    };

    // queries: group 0, 16 lanes to a row, 8 rows a round; scaled so that a row's largest
    // is in [2^8, 2^9), which bf16 queries need to fit fp16
    constexpr int kRounds = NR / 8;
    const int ql = gt & 15, qr = (gt & 127) >> 4;
    uint4 qw[kRounds];
    auto load_queries = [&](const Item &it) {
      const int row0 = p.cu[it.b], rows = (p.cu[it.b + 1] - row0) * p.rg;
#pragma unroll
      for (int k = 0; k < kRounds; ++k) {
        const int n = qr + 8 * k;
        qw[k] = make_uint4(0, 0, 0, 0);
        if (n < rows)
          qw[k] = __ldg(reinterpret_cast<const uint4 *>(a.q + (int64_t)(row0 + n / p.rg) * a.qs +
                                                        (int64_t)(it.h * p.rg + n % p.rg) * kD128) +
                        ql);
      }
    };
    auto store_queries = [&](uint32_t item) {
#pragma unroll
      for (int k = 0; k < kRounds; ++k) {
        const int n = qr + 8 * k;
        const uint32_t ww[4] = {qw[k].x, qw[k].y, qw[k].z, qw[k].w};
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
        for (int o = 1; o < 16; o <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
        int ex = ((__float_as_int(big) >> 23) & 255) - 127;
        ex = big == 0.0f ? 0 : max(min(ex, 90), -90);
        const float mul = a.sign * __int_as_float((127 + 8 - ex) << 23);
        uint32_t y[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          y[c] = h2u(__floats2half2_rn(f[2 * c] * mul, f[2 * c + 1] * mul));
        sts128(smem_s + C::off_q + (ql >> 3) * (NR * 128) + n * 128 +
                   (((ql & 7) ^ (n & 7)) << 4),
               y);
        if (ql == 0)
          fs[(item & 1) * NR + n] = fminf(
              fmaxf(a.scale_log2 * __int_as_float((127 + ex - 8) << 23), 1e-30f), kMostScale);
      }
      async_fence();
      bar_arrive_warp(bar_qf);
    };

    // (No warp leaves these loops early: the groups' meetings have no limit, so after a
    // wait that ran out all go on, on what is there; every later wait ends at once.)
    uint32_t s = 0, items = 0, seen = 0, outs = 0;  // steps, items; this group's steps, outputs
    int b = start_b;
    if (g == 0 && x0 < x1) {
      load_queries(item_at(x0, b));
      store_queries(0);
    }
    for (int64_t x = x0; x < x1; ++items) {
      const Item it = item_at(x, b);
      b = it.b;
      const int n = it.j1 - it.j0;
      x += n;
      const int len = length(b);
      float l[NR];
#pragma unroll
      for (int i = 0; i < NR; ++i) l[i] = 0.0f;
      if (gt % 128 < NR) myref[gt % 128] = kNoRef;
      wait_warp(bar_qf, items & 1);
      if (g == 1) bar_arrive_warp(bar_qe);
      meet();
      const float *F = fs + (items & 1) * NR;
      const int mine0 = (int)((s ^ g) & 1);  // this group's first step of the item
      for (int j = mine0; j < n; j += 2, ++seen) {
        wait_warp(bar_s(g), seen & 1);
        tc_fence_after();
        const int at = (it.j0 + j) * kStep + r;
        const uint32_t lost = missing[(s + j) % kBad];
        const bool alive = at < len && !(lost >> (r / kAtom) & 1);
        uint32_t y[NR];
        if constexpr (NR == 32) tc_ld32(ts, y); else tc_ld16(ts, y);
        tc_wait_ld();
        // the largest score, against its row's reference (a row without one yet lies far
        // above it)
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < NR; i += 4) {
          const float4 f = *reinterpret_cast<const float4 *>(F + i);
          const float4 o = *reinterpret_cast<const float4 *>(myref + i);
          top = max3(top, fmaf(__uint_as_float(y[i]), f.x, -o.x),
                     fmaf(__uint_as_float(y[i + 1]), f.y, -o.y));
          top = max3(top, fmaf(__uint_as_float(y[i + 2]), f.z, -o.z),
                     fmaf(__uint_as_float(y[i + 3]), f.w, -o.w));
        }
        if (any_of_group(alive && top > kCrossTop)) {
          // references move: to kCrossBase below the step's largest score
#pragma unroll
          for (int i = 0; i < NR; ++i) {
            float m = alive ? __uint_as_float(y[i]) : -INFINITY;
#pragma unroll
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (lane == i) maxima[w4 * NR + i] = m;
          }
          meet();
          if (r < NR) {  // (the only one to look at row r's maxima)
            const float m = fmaxf(fmaxf(maxima[r], maxima[NR + r]),
                                  fmaxf(maxima[2 * NR + r], maxima[3 * NR + r]));
            const float old = myref[r], now = fmaf(m, F[r], -kCrossBase);
            // one that is passed by no more than the slack stays
            const bool move = m > -INFINITY && fmaf(m, F[r], -old) > kCrossTop;
            maxima[r] = move ? exp2_approx(old - now) : 1.0f;
            if (move) myref[r] = now;
          }
          meet();
#pragma unroll
          for (int i = 0; i < NR; ++i) l[i] *= maxima[i];
          if (j > mine0) {
            // the group's earlier products are done: these scores came after them
#pragma unroll
            for (int c = 0; c < NR; c += 16) {
              uint32_t o[16];
              tc_ld16(to + c, o);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i)
                o[i] = __float_as_uint(__uint_as_float(o[i]) * maxima[c + i]);
              tc_st16(to + c, o);
            }
            tc_wait_st();
          }
        }
#pragma unroll
        for (int i = 0; i < NR; i += 4) {
          const float4 f = *reinterpret_cast<const float4 *>(F + i);
          const float4 o = *reinterpret_cast<const float4 *>(myref + i);
          const float ff[4] = {f.x, f.y, f.z, f.w}, oo[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float w =
                alive ? exp2_approx(fmaf(__uint_as_float(y[i + e]), ff[e], -oo[e])) : 0.0f;
            l[i + e] += w;
            const uint16_t h = __half_as_ushort(__float2half_rn(w));
            asm volatile("st.shared.b16 [%0], %1;" ::"r"(pt + (i + e) * 128 +
                                                         (px ^ (((i + e) & 7) << 4))),
                         "h"(h)
                         : "memory");
          }
        }
        async_fence();
        tc_fence_before();
        bar_arrive_warp(bar_p(g));
      }
      s += n;
      // the next item's queries go in once all of this one's scores are done (and group
      // 1 has seen these)
      if (g == 0 && x < x1) {
        load_queries(item_at(x, b));
        wait_warp(bar_qe, items & 1);
        store_queries(items + 1);
      }
      // ---- sums over the tokens, then both groups' parts
#pragma unroll
      for (int i = 0; i < NR; ++i) {
#pragma unroll
        for (int o = 16; o; o >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
        if (lane == i) sums[(g * 4 + w4) * NR + i] = l[i];
      }
      const bool any_step = mine0 < n;
      if (any_step) wait_warp(bar_o(g), outs++ & 1);
      tc_fence_after();
      meet_all();
      // group 1 leaves its output where the weights were, group 0 adds its own
      float *joined = reinterpret_cast<float *>(smem + C::off_p);
      uint32_t o[NR];
#pragma unroll
      for (int i = 0; i < NR; ++i) o[i] = 0;
      if (any_step) {
        if constexpr (NR == 32) tc_ld32(to, o); else tc_ld16(to, o);
        tc_wait_ld();
      }
      if (g == 1) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const float f = exp2_approx(refs[NR + i] - fmaxf(refs[i], refs[NR + i]));
          joined[i * kD128 + r] = __uint_as_float(o[i]) * f;
        }
      }
      meet_all();
      const int row0 = p.cu[b], rows = (p.cu[b + 1] - row0) * p.rg;
      const bool whole = it.j0 == 0 && it.j1 == it.steps;
      const int slot = 2 * blockIdx.x + (it.j0 == 0 ? 1 : 0);
      const int c0 = (int)(it.first / U), c1 = (int)((it.first + it.steps - 1) / U);
      // column r of V holds this channel
      const int channel = 32 * (((r >> 3) & 1) * 2 + (r & 1)) + 4 * (r >> 4) + ((r >> 1) & 3);
      auto put = [&](int i, float v) {
        const int64_t t = row0 + i / p.rg;
        uint16_t *dst = a.out + (t * p.Hq + it.h * p.rg + i % p.rg) * kD128 + channel;
        *dst = p.bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v))
                      : __half_as_ushort(__float2half_rn(v));
      };
      if (g == 0) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const float r0 = refs[i], r1 = refs[NR + i], m = fmaxf(r0, r1);
          const float f0 = exp2_approx(r0 - m), f1 = exp2_approx(r1 - m);
          const float v = fmaf(__uint_as_float(o[i]), f0, joined[i * kD128 + r]);
          float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
          for (int w = 0; w < 4; ++w) sum0 += sums[w * NR + i], sum1 += sums[(4 + w) * NR + i];
          const float sum = sum0 * f0 + sum1 * f1;
          if (i >= rows) continue;
          if (whole) {
            put(i, sum == 0.0f ? 0.0f : v / sum);
          } else {
            a.ws_o[((int64_t)slot * NR + i) * kD128 + r] = v;
            if (r == 0)
              *reinterpret_cast<float2 *>(a.ws_ml + ((int64_t)slot * NR + i) * 2) =
                  make_float2(m, sum);
          }
        }
      }
      if (!whole) {
        // the block that arrives last joins the parts, in block order
        __threadfence();
        meet_all();
        volatile uint32_t *flag = misc + 2;
        if (gt == 0) {
          const int last = atomicAdd(&a.ws_count[c0], 1) == c1 - c0;
          if (last) a.ws_count[c0] = 0;
          *flag = last;
        }
        meet_all();
        if (*flag) {
          __threadfence();
#pragma unroll 1
          for (int i = (int)g; i < rows; i += 2) {
            float m = kNoRef, sum = 0.0f, v = 0.0f;
#pragma unroll 4
            for (int c = c0; c <= c1; ++c) {
              const int64_t at = (int64_t)(2 * c + (c == c0)) * NR + i;
              const float2 ml = __ldcg(reinterpret_cast<const float2 *>(a.ws_ml + at * 2));
              const float w = __ldcg(a.ws_o + at * kD128 + r);
              const float nm = fmaxf(m, ml.x), f = exp2_approx(m - nm), f2 = exp2_approx(ml.x - nm);
              m = nm;
              sum = sum * f + f2 * ml.y;
              v = v * f + f2 * w;
            }
            put(i, sum == 0.0f ? 0.0f : v / sum);
          }
        }
      }
      tc_fence_before();
      meet_all();  // the weights' room, sums and references are free
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(4 * NR));
  }
}

template <int BITS, int NR>
cudaError_t cross_as(const CrossArgs &a, int num_sms, cudaStream_t st) {
  static KernelSetup setup;
  const int smem = CrossCfg<BITS, NR>::smem(a.p.B);
  auto kern = paged_cross_kernel<BITS, NR>;
  // the register split draws on what the block is launched with: a kernel built
  // with fewer registers a thread would wait for the rest forever
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    regs.store(fa.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) * kCrossThreads < kRegSum)
    return cudaErrorInvalidConfiguration;
  const cudaError_t e = kernel_setup(setup, kern, kCrossThreads, smem, nullptr);
  if (e != cudaSuccess) return e;
  const int blocks = num_sms < kMaxCrossBlocks ? num_sms : kMaxCrossBlocks;
  return launch_dependent(kern, (unsigned)blocks, kCrossThreads, smem, st, true, a);
}

}  // namespace

cudaError_t launch_paged_cross(const Paged &p, const void *q, int64_t qs, void *out, float scale,
                               int rows, void *ws, int num_sms, cudaStream_t st) {
  // (the split kernel's room: 2 * 320 partials of 16 rows are 2 * 160 of 32)
  static_assert(kMaxCrossBlocks * 32 <= kPagedRowBlocks * kPagedFewRows, "workspace");
  CrossArgs a;
  a.p = p;
  a.q = static_cast<const uint16_t *>(q);
  a.qs = qs;
  a.out = static_cast<uint16_t *>(out);
  a.scale_log2 = fminf(fabsf(scale) * 1.4426950408889634f, kMostScale);
  a.sign = scale < 0.0f ? -1.0f : 1.0f;
  uint8_t *w = static_cast<uint8_t *>(ws);
  a.ws_count = reinterpret_cast<int *>(w);
  a.ws_ml = reinterpret_cast<float *>(w + kPagedRowBlocks * 4);
  a.ws_o = reinterpret_cast<float *>(w + kPagedRowBlocks * 4 +
                                     2 * kPagedRowBlocks * kPagedFewRows * 8);
  a.stall_limit = debug_stall_limit();
  if (rows <= 16)
    return p.bits == 2   ? cross_as<2, 16>(a, num_sms, st)
           : p.bits == 4 ? cross_as<4, 16>(a, num_sms, st)
                         : cross_as<8, 16>(a, num_sms, st);
  return p.bits == 2   ? cross_as<2, 32>(a, num_sms, st)
         : p.bits == 4 ? cross_as<4, 32>(a, num_sms, st)
                       : cross_as<8, 32>(a, num_sms, st);
}

}  // namespace kvq
