// Page tables (include/kvq.h, "Page tables"): which pages each sequence holds, and
// how many hold each page.  Whole numbers only, and small: what bounds these calls
// is the latency of a launch and of a chain of dependent loads, so each is one or
// two launches, and what one block can do without waiting for others is one block's.
//
// A free page is a set bit of the free map; pages go out lowest first, so low
// numbers stay in use, and `hint` (no word before it has a free page) is where the
// search begins.  Holder counts change by atomics, whose order does not matter: who
// takes the last holder away sets the page's bit.
//
// Measured on a GB300 (graph replay): drop and reserve of 16 sequences 6.8 us, of 2048
// over a pool of 431000 pages 10.3 (25 when one warp walked 32 neighbouring words of the
// map); select, reserve and the copy of 60 forks' pages 14.3; recount, compact and the
// copy of 278 MB in a pool of 14000 pages 101, 83 of them the copy.
#include <algorithm>

#include "kvq_paged.cuh"
#include "kvq_tc_common.cuh"

namespace kvq {
namespace {

constexpr int64_t kMostPages = 1LL << 26;
constexpr unsigned kAll = 0xffffffffu;
constexpr int kReserveThreads = 1024;
constexpr int kReserveWarps = kReserveThreads / 32;
constexpr int kRowThreads = 256;             // kernels over the tables' rows: a warp a stretch
constexpr int kStretch = 128;                // entries of a stretch
constexpr int kMoveThreads = 256;
constexpr int kMoveWords = 64;               // compaction: words of the map a block

// The head of kvq_page_table.state.
struct Head {
  int free, hint;
  int moves, front;  // of the last compaction: pages moved, pages live
};

struct Table {
  int32_t *table, *lens, *refs, *status;
  Head *head;
  uint32_t *map;     // [words] free pages
  int32_t *tickets;  // [B], zero between calls
  int32_t *held;     // [2][B]: entries of the old row, of the new one; [B] new lengths
  int32_t *rows;     // [B][width] rows to come (select); {word, free pages before} (compact)
  int64_t width;
  int n_pages, words, page_log, page, B, stretches;
};

__device__ __forceinline__ void table_error(const Table &t, int code) {
  atomicCAS(t.status, 0, code);
}
// Table entries that hold n tokens, of the `width` there are.
__device__ __forceinline__ int entries_of(const Table &t, int64_t n) {
  return n <= 0 ? 0 : (int)min((n + t.page - 1) >> t.page_log, t.width);
}
// What is wrong with a sequence of len tokens, recorded by `one` thread: nothing is made
// of such a length, and its row stays as it is.
__device__ __forceinline__ bool bad_length(const Table &t, int len, bool one) {
  const bool bad = len < 0 || len > t.width * t.page;
  if (bad && one) table_error(t, len < 0 ? KVQ_EINVAL : KVQ_EPAGE);
  return bad;
}

// Takes a holder off page id; the last one frees it.  Called by whole warps, with
// `on` the lanes that do.
__device__ __forceinline__ void release(const Table &t, bool on, int id) {
  if (on && (id < 0 || id >= t.n_pages)) {
    table_error(t, KVQ_EPAGE);
    on = false;
  }
  int before = 0;
  if (on) {
    before = atomicSub(&t.refs[id], 1);
    if (before <= 0) {  // had none: the tables and the counts do not agree
      atomicAdd(&t.refs[id], 1);
      table_error(t, KVQ_EINVAL);
    }
  }
  const bool last = on && before == 1;
  if (last) atomicOr(&t.map[id >> 5], 1u << (id & 31));
  const unsigned who = __ballot_sync(kAll, last);
  if (who == 0) return;
  const int low = __reduce_min_sync(kAll, last ? id >> 5 : 0x7fffffff);
  if ((threadIdx.x & 31) == 0) {
    atomicAdd(&t.head->free, __popc(who));
    atomicMin(&t.head->hint, low);
  }
}

// Inclusive running sums over the block, and the total.  sums: one per warp.
template <int WARPS>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *sums, int64_t &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(kAll, v, o);
    if (lane >= o) v += up;
  }
  __syncthreads();  // (sums of an earlier scan have been read)
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int64_t s = lane < WARPS ? sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < WARPS; o <<= 1) {
      const int64_t up = __shfl_up_sync(kAll, s, o);
      if (lane >= o) s += up;
    }
    if (lane < WARPS) sums[lane] = s;
  }
  __syncthreads();
  total = sums[WARPS - 1];
  return v + (warp ? sums[warp - 1] : 0);
}

// ---- reserve ------------------------------------------------------------------
// One block: a sequence (or two) a thread counts the pages it needs, running sums
// number them, and the warps walk the free map a bit a lane (neighbouring words in
// different warps) and hand the r-th free page to the sequence whose numbers hold r.
__global__ void __launch_bounds__(kReserveThreads, 1)
pages_reserve_kernel(const __grid_constant__ Table t, const int32_t *cu, int2 *copies,
                     int32_t *cu_call) {
  constexpr int kPer = kMaxSeqs / kReserveThreads;
  __shared__ int64_t sums[kReserveWarps];
  __shared__ int first[kMaxSeqs + 1];   // number of the first page of each sequence
  __shared__ int entry[kMaxSeqs];       // its table entry
  __shared__ int from[kMaxSeqs];        // the page it copies, or -1
  __shared__ int pair[kMaxSeqs];        // ... and that copy's place in the list
  __shared__ uint32_t map_bits[kReserveThreads];  // a stretch of the map, and the number
  __shared__ int map_before[kReserveThreads];     // of each word's first free page
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_trigger();
  grid_dep_wait();
  const int per = t.B > kReserveThreads ? kPer : 1;
  const int b0 = tid * per;
  const int64_t cap = t.width * t.page;
  const int free = t.head->free;
  int hint = max(t.head->hint, 0);

  // ---- what each sequence needs
  int rows[kPer], held[kPer], id[kPer];
  int64_t len[kPer], need[kPer];
  bool claim[kPer], keep[kPer];
  int bad = KVQ_OK, any = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = b0 + i;
    rows[i] = held[i] = 0, id[i] = -1, len[i] = need[i] = 0, claim[i] = keep[i] = false;
    if (i >= per || b >= t.B) continue;
    const int c0 = cu[b], c1 = cu[b + 1];
    len[i] = t.lens[b];
    if (c0 < 0 || c1 < c0 || len[i] < 0 || (b == 0 && c0 != 0)) {
      bad = KVQ_EINVAL;
      continue;
    }
    rows[i] = c1 - c0;
    if (rows[i] == 0) continue;
    if (len[i] + rows[i] > cap) {
      if (bad == KVQ_OK) bad = KVQ_ECAPACITY;
      continue;
    }
    held[i] = entries_of(t, len[i]);
    need[i] = entries_of(t, len[i] + rows[i]) - held[i];
    if ((len[i] & (t.page - 1)) != 0) {  // the first new token lies in a page that is begun
      id[i] = t.table[b * t.width + held[i] - 1];
      const int holders = id[i] >= 0 && id[i] < t.n_pages ? __ldcg(&t.refs[id[i]]) : -1;
      if (holders < 1) bad = holders < 0 ? KVQ_EPAGE : KVQ_EINVAL;
      claim[i] = holders > 1;
      any |= claim[i];
    }
  }
  if (bad != KVQ_OK) table_error(t, bad);
  bool fail = __syncthreads_or(bad != KVQ_OK);
  any = __syncthreads_or(any);
  // ---- pages to copy.  Each writer of a shared page gives up its hold; where that
  // leaves no holder all of them write, and the first keeps the page.
  if (!fail && any) {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (claim[i]) atomicSub(&t.refs[id[i]], 1);
    __syncthreads();
    constexpr int kBelow = 1 << 30;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (claim[i] && __ldcg(&t.refs[id[i]]) <= 0) atomicMin(&t.refs[id[i]], b0 + i - kBelow);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      keep[i] = claim[i] && __ldcg(&t.refs[id[i]]) == b0 + i - kBelow;
      if (claim[i] && !keep[i]) ++need[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (keep[i]) t.refs[id[i]] = 1;
  }
  // ---- numbers of the pages, and of the copies
  int64_t total = 0, n_copies = 0;
  const int64_t mine = need[0] + need[1];
  int64_t at = block_scan<kReserveWarps>(mine, sums, total) - mine;
  const bool c0 = claim[0] && !keep[0], c1 = claim[1] && !keep[1];
  int place = 0;
  if (any) {
    const int64_t pairs = (int64_t)c0 + c1;
    place = (int)(block_scan<kReserveWarps>(pairs, sums, n_copies) - pairs);
  }
  // the holds go back, and the call hands out nothing
  auto give_back = [&]() {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (keep[i]) t.refs[id[i]] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (claim[i]) atomicAdd(&t.refs[id[i]], 1);
  };
  auto outputs = [&]() {
    for (int i = tid; i <= t.B; i += kReserveThreads) cu_call[i] = fail ? 0 : cu[i];
    for (int i = tid; i < t.B; i += kReserveThreads)
      if (fail || i >= n_copies) copies[i] = make_int2(-1, -1);
  };
  if (!fail && total > free) {  // not enough
    if (tid == 0) table_error(t, KVQ_ECAPACITY);
    give_back();
    fail = true;
  }
  outputs();
  if (fail) return;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = b0 + i;
    if (i >= per || b >= t.B) break;
    const bool copy = claim[i] && !keep[i];
    first[b] = (int)at;
    entry[b] = held[i] - (copy ? 1 : 0);
    from[b] = copy ? id[i] : -1;
    pair[b] = place;
    at += need[i];
    place += copy;
    if (rows[i] > 0) t.lens[b] = (int)(len[i] + rows[i]);
  }
  if (total == 0) return;
  if (tid == 0) first[t.B] = (int)total, t.head->free = free - (int)total;
  __syncthreads();
  // ---- the free map, 1024 words at a time
  const int n = (int)total;
  int64_t done = 0;
  for (int w0 = hint; w0 < t.words && done < n; w0 += kReserveThreads) {
    const int w = w0 + tid;
    const uint32_t bits = w < t.words ? t.map[w] : 0u;
    if (!__syncthreads_or(bits != 0)) continue;
    const int64_t count = __popc(bits);
    int64_t found = 0;
    map_bits[tid] = bits;
    map_before[tid] = (int)(done + block_scan<kReserveWarps>(count, sums, found) - count);
    __syncthreads();
    // a warp takes every 32nd word, a lane a bit of it
    for (int j = warp; j < kReserveThreads && map_before[j] < n; j += kReserveWarps) {
      const uint32_t word = map_bits[j];
      const int r = map_before[j] + __popc(word & ((1u << lane) - 1));
      const int page = (w0 + j) * 32 + lane;
      const bool take = (word >> lane & 1) && r < n && page < t.n_pages;
      if (take) {
        int lo = 0, hi = t.B;  // the last b with first[b] <= r that needs a page
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (first[mid] <= r) lo = mid; else hi = mid;
        }
        t.table[lo * t.width + entry[lo] + (r - first[lo])] = page;
        t.refs[page] = 1;
        if (from[lo] >= 0 && r == first[lo]) copies[pair[lo]] = make_int2(from[lo], page);
      }
      const unsigned gone = __ballot_sync(kAll, take);
      if (lane == 0 && gone) t.map[w0 + j] = word & ~gone;
    }
    done += found;
    hint = w0;
  }
  if (done >= n) {
    if (tid == 0) t.head->hint = hint;
    return;
  }
  // the map holds fewer free pages than the head says: those handed out go back
  if (tid == 0) table_error(t, KVQ_EINVAL), t.head->free = free;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = b0 + i;
    if (i >= per || b >= t.B) break;
    int32_t *row = t.table + b * t.width + entry[b];
    const int64_t got = min(need[i], done - first[b]);
    for (int64_t k = 0; k < got; ++k) {
      const int page = row[k];
      row[k] = k == 0 ? from[b] : -1;
      if (page < 0 || page >= t.n_pages) continue;  // (a bit behind the last page's)
      t.refs[page] = 0;
      atomicOr(&t.map[page >> 5], 1u << (page & 31));
    }
    if (rows[i] > 0) t.lens[b] = (int)len[i];
  }
  give_back();
  fail = true;
  outputs();
}

// ---- kernels over the rows: a warp takes every `stretches`-th stretch of a row ----
struct Stretch {
  int b, s;
};
__device__ __forceinline__ Stretch row_of_warp(const Table &t) {
  const int64_t w = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  return {(int)min(w / t.stretches, (int64_t)t.B), (int)(w % t.stretches)};
}

__global__ void __launch_bounds__(kRowThreads)
pages_drop_kernel(const __grid_constant__ Table t, const int32_t *tokens) {
  const int lane = threadIdx.x & 31;
  grid_dep_trigger();
  grid_dep_wait();
  const Stretch p = row_of_warp(t);
  if (p.b >= t.B) return;
  const int drop = tokens[p.b], len = t.lens[p.b];
  if (bad_length(t, len, p.s == 0 && lane == 0) || drop <= 0 || len == 0) return;
  const int left = max(len - drop, 0);
  const int e0 = entries_of(t, left), e1 = entries_of(t, len);
  int32_t *row = t.table + p.b * t.width;
  for (int e = e0 + p.s * 32; e < e1; e += t.stretches * 32) {
    const bool on = e + lane < e1;
    release(t, on, on ? row[e + lane] : 0);
    if (on) row[e + lane] = -1;
  }
  // the length changes once every warp of the row has read it
  if (lane == 0) {
    bool last = true;
    if (t.stretches > 1) {
      __threadfence();
      last = atomicAdd(&t.tickets[p.b], 1) == t.stretches - 1;
      if (last) t.tickets[p.b] = 0;
    }
    if (last) t.lens[p.b] = left;
  }
}

// Rows to come are gathered and their pages held before any hold is given up, so no
// page is freed in between; an entry that stays what it was changes no count.
__global__ void __launch_bounds__(kRowThreads)
pages_gather_kernel(const __grid_constant__ Table t, const int32_t *parents) {
  const int lane = threadIdx.x & 31;
  grid_dep_trigger();
  grid_dep_wait();
  const Stretch p = row_of_warp(t);
  if (p.b >= t.B) return;
  const int parent = parents[p.b], len = t.lens[p.b];
  const bool one = p.s == 0 && lane == 0, known = parent >= -1 && parent < t.B;
  if (!known && one) table_error(t, KVQ_EINVAL);
  const int to = known && parent >= 0 ? t.lens[parent] : 0;
  if (bad_length(t, len, one) || !known || parent == p.b || bad_length(t, to, one)) {
    if (one) t.held[p.b] = -1;  // stays as it is
    return;
  }
  const int old = entries_of(t, len), now = entries_of(t, to);
  const int32_t *src = t.table + max(parent, 0) * t.width, *row = t.table + p.b * t.width;
  for (int e = p.s * 32 + lane; e < now; e += t.stretches * 32) {
    const int id = src[e];
    t.rows[p.b * t.width + e] = id;
    if (e < old && row[e] == id) continue;
    if (id >= 0 && id < t.n_pages)
      atomicAdd(&t.refs[id], 1);
    else
      table_error(t, KVQ_EPAGE);
  }
  if (one) t.held[p.b] = old, t.held[t.B + p.b] = now, t.held[2 * t.B + p.b] = to;
}
__global__ void __launch_bounds__(kRowThreads)
pages_replace_kernel(const __grid_constant__ Table t) {
  const int lane = threadIdx.x & 31;
  grid_dep_trigger();
  grid_dep_wait();
  const Stretch p = row_of_warp(t);
  if (p.b >= t.B) return;
  const int old = t.held[p.b];
  if (old < 0) return;
  const int now = t.held[t.B + p.b];
  int32_t *row = t.table + p.b * t.width;
  const int32_t *to = t.rows + p.b * t.width;
  for (int e = p.s * 32; e < max(old, now); e += t.stretches * 32) {
    const int at = e + lane;
    const int was = at < old ? row[at] : -1, is = at < now ? to[at] : -1;
    release(t, at < old && !(at < now && was == is), was);
    if (at < max(old, now)) row[at] = is;
  }
  if (p.s == 0 && lane == 0) t.lens[p.b] = t.held[2 * t.B + p.b];
}

// ---- recount --------------------------------------------------------------------
__global__ void __launch_bounds__(kRowThreads)
pages_clear_kernel(const __grid_constant__ Table t) {
  grid_dep_trigger();
  grid_dep_wait();
  const int64_t i = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
  if (i < t.n_pages) t.refs[i] = 0;
  if (i < t.B) t.tickets[i] = 0;
  if (i == 0) *t.head = Head{0, 0x7fffffff, 0, 0};
}
__global__ void __launch_bounds__(kRowThreads)
pages_count_kernel(const __grid_constant__ Table t) {
  const int lane = threadIdx.x & 31;
  grid_dep_trigger();
  grid_dep_wait();
  const Stretch p = row_of_warp(t);
  if (p.b >= t.B) return;
  const int len = t.lens[p.b];
  bad_length(t, len, p.s == 0 && lane == 0);
  const int held = entries_of(t, len);
  int32_t *row = t.table + p.b * t.width;
  for (int64_t e = p.s * 32 + lane; e < t.width; e += t.stretches * 32) {
    if (e >= held) {
      row[e] = -1;
      continue;
    }
    const int id = row[e];
    if (id >= 0 && id < t.n_pages)
      atomicAdd(&t.refs[id], 1);
    else
      table_error(t, KVQ_EPAGE);
  }
}
__global__ void __launch_bounds__(kRowThreads)
pages_map_kernel(const __grid_constant__ Table t) {
  grid_dep_trigger();
  grid_dep_wait();
  const int64_t i = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
  const unsigned bits = __ballot_sync(kAll, i < t.n_pages && t.refs[i] == 0);
  if ((threadIdx.x & 31) == 0 && i < (int64_t)t.words * 32) t.map[i >> 5] = bits;
  // one addition a block: of single ones the head's word is the bound
  const int n = __syncthreads_count(i < t.n_pages && (bits >> (threadIdx.x & 31) & 1));
  if (threadIdx.x == 0 && n) {
    atomicAdd(&t.head->free, n);
    atomicMin(&t.head->hint, (int)(i >> 5));
  }
}

// ---- compact ---------------------------------------------------------------------
// n live pages go to [0, n): the k-th live page from n on moves to the k-th free page
// before n.  Each block counts the free pages before its words by itself (the map is
// a bit a page), so blocks wait for nothing.  That is work with the square of the pool:
// both launches take 20 us for 2^20 pages, 107 for 2^22, 1190 for 2^24 and by that some
// 20 ms for the 2^26 that a table may have.
__global__ void __launch_bounds__(kMoveThreads)
pages_moves_kernel(const __grid_constant__ Table t, int2 *copies, int64_t n_copies) {
  __shared__ int64_t sums[kMoveThreads / 32];
  __shared__ uint32_t word_bits[kMoveWords];
  __shared__ int word_before[kMoveWords];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_trigger();
  grid_dep_wait();
  // (a count that is none leaves a front in range; the last block finds it out)
  const int64_t live = (int64_t)t.n_pages - t.head->free;
  const int front = (int)min(max(live, (int64_t)0), (int64_t)t.n_pages), front_word = front >> 5;
  const uint32_t front_bits = (1u << (front & 31)) - 1;  // of that word: before the front
  const int w0 = blockIdx.x * kMoveWords;
  // free pages before the block's words, and before the front, four words a load
  const int ends = min(max(w0, front_word + 1), t.words);
  int64_t before = 0, holes = 0, total;
  auto count = [&](int w, uint32_t bits) {
    if (w < w0) before += __popc(bits);
    if (w < front_word) holes += __popc(bits);
    if (w == front_word) holes += __popc(bits & front_bits);
  };
#pragma unroll 4
  for (int w = 4 * tid; w < ends; w += 4 * kMoveThreads) {
    // (the map's room is a multiple of four words)
    const uint4 v = *reinterpret_cast<const uint4 *>(t.map + w);
    count(w, v.x);
    count(w + 1, v.y);
    count(w + 2, v.z);
    count(w + 3, v.w);
  }
  block_scan<kMoveThreads / 32>(before, sums, total);
  before = total;
  block_scan<kMoveThreads / 32>(holes, sums, total);
  const int moves = (int)total;
  const int w = w0 + tid;
  const bool mine = tid < kMoveWords && w < t.words;
  const uint32_t bits = mine ? t.map[w] : 0u;
  const int64_t free = __popc(bits);
  const int here = (int)(before + block_scan<kMoveThreads / 32>(free, sums, total) - free);
  if (tid < kMoveWords) word_bits[tid] = bits, word_before[tid] = here;
  if (mine) reinterpret_cast<uint2 *>(t.rows)[w] = make_uint2(bits, (uint32_t)here);
  if (blockIdx.x == gridDim.x - 1 && tid == 0) {
    const bool agree = before + total == t.head->free;
    t.head->moves = moves, t.head->front = agree ? front : -1;
    if (!agree) table_error(t, KVQ_EINVAL);
  }
  __syncthreads();
  // a warp a word, a lane a page: a free one before the front, a live one behind
  for (int j = warp; j < kMoveWords && w0 + j < t.words; j += kMoveThreads / 32) {
    const uint32_t word = word_bits[j];
    const int f = word_before[j] + __popc(word & ((1u << lane) - 1));
    const int id = (w0 + j) * 32 + lane;
    const bool is_free = word >> lane & 1;
    const int64_t k = id < front ? f : (int64_t)id - f - (front - moves);
    // (in range wherever the head's count is the map's)
    if (k < 0 || k >= n_copies || id >= t.n_pages) continue;
    if (id < front && is_free) copies[k].y = id;
    if (id >= front && !is_free) copies[k].x = id;
  }
  for (int64_t k = moves + (int64_t)blockIdx.x * kMoveThreads + tid; k < n_copies;
       k += (int64_t)gridDim.x * kMoveThreads)
    copies[k] = make_int2(-1, -1);
}
// Blocks [0, row_blocks): table entries; behind them: pages and the free map.
__global__ void __launch_bounds__(kRowThreads)
pages_rename_kernel(const __grid_constant__ Table t, int2 *copies, int64_t n_copies,
                    int row_blocks) {
  const int lane = threadIdx.x & 31;
  grid_dep_trigger();
  grid_dep_wait();
  const int front = t.head->front, moves = t.head->moves;
  if (front < 0) {  // the count and the map do not agree: nothing moves
    for (int64_t k = (int64_t)blockIdx.x * kRowThreads + threadIdx.x; k < n_copies;
         k += (int64_t)gridDim.x * kRowThreads)
      copies[k] = make_int2(-1, -1);
    return;
  }
  const uint2 *snap = reinterpret_cast<const uint2 *>(t.rows);
  auto moved_to = [&](int id) {  // of a live page behind the front
    const uint2 s = snap[id >> 5];
    const int f = (int)s.y + __popc(s.x & ((1u << (id & 31)) - 1));
    const int64_t k = (int64_t)id - f - (front - moves);
    const int to = k >= 0 && k < n_copies ? copies[k].y : -1;
    return to >= 0 && to < t.n_pages ? to : id;
  };
  if (blockIdx.x < row_blocks) {
    const Stretch p = row_of_warp(t);
    if (p.b >= t.B) return;
    // (of a length that is none, what entries are pages follow them all the same)
    const int len = t.lens[p.b];
    const bool bad = bad_length(t, len, p.s == 0 && lane == 0);
    const int held = bad ? (int)t.width : entries_of(t, len);
    int32_t *row = t.table + p.b * t.width;
    for (int e = p.s * 32 + lane; e < held; e += t.stretches * 32) {
      const int id = row[e];
      if (id < 0 || id >= t.n_pages || (snap[id >> 5].x >> (id & 31) & 1)) {
        if (!bad) table_error(t, id < 0 || id >= t.n_pages ? KVQ_EPAGE : KVQ_EINVAL);
      } else if (id >= front) {
        row[e] = moved_to(id);
      }
    }
    return;
  }
  const int64_t i = (int64_t)(blockIdx.x - row_blocks) * kRowThreads + threadIdx.x;
  if (i < t.n_pages && i >= front && !(snap[i >> 5].x >> (i & 31) & 1)) {
    const int holders = t.refs[i];
    t.refs[i] = 0;
    t.refs[moved_to((int)i)] = holders;
  }
  const unsigned bits = __ballot_sync(kAll, i < t.n_pages && i >= front);
  if (lane == 0 && i < (int64_t)t.words * 32) t.map[i >> 5] = bits;
  if (i == 0) t.head->hint = front >> 5;
}

// ---- host -------------------------------------------------------------------------
struct Layout {
  size_t map, tickets, held, rows, end;
};
Layout layout_of(const kvq_page_table &t) {
  auto up = [](size_t n) { return (n + 15) / 16 * 16; };
  const size_t words = ((size_t)t.n_pages + 31) / 32;
  Layout l;
  l.map = up(sizeof(Head));
  l.tickets = l.map + up(words * 4);
  l.held = l.tickets + up((size_t)t.n_seqs * 4);
  l.rows = l.held + up((size_t)t.n_seqs * 12);
  l.end = l.rows + up(std::max((size_t)t.n_seqs * (size_t)t.table_width * 4, words * 8));
  return l;
}

int check_sizes(const kvq_page_table *t) {
  if (!t) return KVQ_EINVAL;
  if (t->n_seqs < 1 || t->table_width < 1 || t->n_pages < 1) return KVQ_EINVAL;
  if (t->page_size != 16 && t->page_size != 32 && t->page_size != 64 && t->page_size != 128 &&
      t->page_size != 256)
    return KVQ_EUNSUPPORTED;
  if (t->n_seqs > kMaxSeqs || t->n_pages > kMostPages ||
      t->table_width > (1LL << 30) / t->page_size)
    return KVQ_EUNSUPPORTED;
  return KVQ_OK;
}

int resolve_table(const kvq_page_table *p, Table *t) {
  const int r = check_sizes(p);
  if (r != KVQ_OK) return r;
  if (!p->block_table || !p->seq_lens || !p->page_refs || !p->state || !p->dev_status)
    return KVQ_EINVAL;
  if (((uintptr_t)p->block_table | (uintptr_t)p->seq_lens | (uintptr_t)p->page_refs |
       (uintptr_t)p->dev_status) & 3)
    return KVQ_EALIGN;
  if ((uintptr_t)p->state & 15) return KVQ_EALIGN;
  const Layout l = layout_of(*p);
  uint8_t *s = static_cast<uint8_t *>(p->state);
  *t = Table{};
  t->table = p->block_table;
  t->lens = p->seq_lens;
  t->refs = p->page_refs;
  t->status = p->dev_status;
  t->head = reinterpret_cast<Head *>(s);
  t->map = reinterpret_cast<uint32_t *>(s + l.map);
  t->tickets = reinterpret_cast<int32_t *>(s + l.tickets);
  t->held = reinterpret_cast<int32_t *>(s + l.held);
  t->rows = reinterpret_cast<int32_t *>(s + l.rows);
  t->width = p->table_width;
  t->n_pages = (int)p->n_pages;
  t->words = (int)((p->n_pages + 31) / 32);
  t->page = p->page_size;
  t->page_log = __builtin_ctz((unsigned)p->page_size);
  t->B = p->n_seqs;
  // a long row is shared by up to 64 warps
  t->stretches = (int)std::min<int64_t>(64, (p->table_width + kStretch - 1) / kStretch);
  return KVQ_OK;
}

unsigned row_blocks(const Table &t) {
  return (unsigned)(((int64_t)t.B * t.stretches + kRowThreads / 32 - 1) / (kRowThreads / 32));
}
unsigned blocks_of(int64_t n, int per) { return (unsigned)((n + per - 1) / per); }

int done(cudaError_t e, int launches) {
  if (e != cudaSuccess) return KVQ_ECUDA;
  note_launch(launches);
  return KVQ_OK;
}
bool misaligned(const void *p, uintptr_t mask) { return ((uintptr_t)p & mask) != 0; }

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" {

int kvq_pages_state_bytes(const kvq_page_table *table, size_t *bytes) {
  if (!bytes) return KVQ_EINVAL;
  const int r = check_sizes(table);
  if (r != KVQ_OK) return r;
  *bytes = layout_of(*table).end;
  return KVQ_OK;
}

int kvq_pages_recount(const kvq_page_table *table, void *stream) {
  Table t;
  const int r = resolve_table(table, &t);
  if (r != KVQ_OK) return r;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_dependent(pages_clear_kernel,
                                   blocks_of(std::max<int64_t>(t.n_pages, t.B), kRowThreads),
                                   kRowThreads, 0, st, true, t);
  if (e == cudaSuccess)
    e = launch_dependent(pages_count_kernel, row_blocks(t), kRowThreads, 0, st, true, t);
  if (e == cudaSuccess)
    e = launch_dependent(pages_map_kernel, blocks_of((int64_t)t.words * 32, kRowThreads),
                         kRowThreads, 0, st, true, t);
  return done(e, 3);
}

int kvq_pages_reserve(const kvq_page_table *table, const int32_t *cu_tokens, int32_t *copies,
                      int32_t *cu_call, void *stream) {
  Table t;
  const int r = resolve_table(table, &t);
  if (r != KVQ_OK) return r;
  if (!cu_tokens || !copies || !cu_call || cu_call == cu_tokens) return KVQ_EINVAL;
  if (misaligned(cu_tokens, 3) || misaligned(copies, 7) || misaligned(cu_call, 3))
    return KVQ_EALIGN;
  return done(launch_dependent(pages_reserve_kernel, 1u, kReserveThreads, 0,
                               static_cast<cudaStream_t>(stream), true, t, cu_tokens,
                               reinterpret_cast<int2 *>(copies), cu_call),
              1);
}

int kvq_pages_drop(const kvq_page_table *table, const int32_t *tokens, void *stream) {
  Table t;
  const int r = resolve_table(table, &t);
  if (r != KVQ_OK) return r;
  if (!tokens) return KVQ_EINVAL;
  if (misaligned(tokens, 3)) return KVQ_EALIGN;
  return done(launch_dependent(pages_drop_kernel, row_blocks(t), kRowThreads, 0,
                               static_cast<cudaStream_t>(stream), true, t, tokens),
              1);
}

int kvq_pages_select(const kvq_page_table *table, const int32_t *parents, void *stream) {
  Table t;
  const int r = resolve_table(table, &t);
  if (r != KVQ_OK) return r;
  if (!parents) return KVQ_EINVAL;
  if (misaligned(parents, 3)) return KVQ_EALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e =
      launch_dependent(pages_gather_kernel, row_blocks(t), kRowThreads, 0, st, true, t, parents);
  if (e == cudaSuccess)
    e = launch_dependent(pages_replace_kernel, row_blocks(t), kRowThreads, 0, st, true, t);
  return done(e, 2);
}

int kvq_pages_compact(const kvq_page_table *table, int32_t *copies, int64_t n_copies,
                      void *stream) {
  Table t;
  const int r = resolve_table(table, &t);
  if (r != KVQ_OK) return r;
  if (!copies) return KVQ_EINVAL;
  if (misaligned(copies, 7)) return KVQ_EALIGN;
  if (n_copies < t.n_pages / 2) return KVQ_ECAPACITY;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int2 *pairs = reinterpret_cast<int2 *>(copies);
  cudaError_t e = launch_dependent(pages_moves_kernel, blocks_of(t.words, kMoveWords),
                                   kMoveThreads, 0, st, true, t, pairs, n_copies);
  const int rows = (int)row_blocks(t);
  if (e == cudaSuccess)
    e = launch_dependent(pages_rename_kernel,
                         rows + blocks_of((int64_t)t.words * 32, kRowThreads), kRowThreads, 0, st,
                         true, t, pairs, n_copies, rows);
  return done(e, 2);
}

}  // extern "C"
