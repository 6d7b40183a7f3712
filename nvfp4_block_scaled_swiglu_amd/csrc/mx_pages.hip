// mx_pages.hip - which pages of a paged cache the sequences hold, kept on the device, and
// copies of whole pages (gfx950).
//
// The bookkeeping is integers: a few loads that depend on one another, so its time is their
// latency and the launches. Its results do not depend on the order in which threads run:
// counts change by integer atomics, a slot that is listed twice is settled by the lower
// place in the list, and free pages are given out lowest first in the list's order. Copies are
// bound by memory, every byte read and written once.
//
// Measured, 48 slots of 130 pages: free 3.3 us, fork 4.9, reserve 10.6 with the entries; 1,024 slots of 515, 37,000
// pages: free 6.6, fork 7.0, reserve 19.4 + 4.1. Compaction of 14,500 pages, 256 slots: 13 + 4.8. Copies of 3,200 pages
// of 70 KB: 88 us, 5.1 TB/s.
#include "mx_pages.hpp"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kPlan = 1024;           // threads of the one workgroup that scans the counts
constexpr int kWords = 4096;          // 64-page words of its bitmap, in LDS
constexpr int64_t kSegment = (int64_t)kWords * 64;
constexpr int kEach = kWords / kPlan;

__device__ __forceinline__ int pages_of(const MxPages& p, int len) {
  const int n = len <= 0 ? 0 : (int)(((int64_t)len + (1 << p.page_shift) - 1) >> p.page_shift);
  return n < p.max_pages ? n : p.max_pages;
}

// the tokens of a slot, which its row has room for (below 2^30)
__device__ __forceinline__ int length_of(const MxPages& p, int slot) {
  const int len = p.lens[slot], most = p.max_pages << p.page_shift;
  return len < 0 ? 0 : len < most ? len : most;
}

__device__ __forceinline__ bool is_page(const MxPages& p, int page) { return page >= 0 && page < p.num_pages; }

constexpr int kTogether = 8;  // list entries of a workgroup

// The entries of a workgroup of the list, and what the whole list says about them.
struct Listed {
  int slot[kTogether], other[kTogether];
  int begin[kTogether], end[kTogether];  // entries of their rows to go through; end 0: none
};

// A page in as many consecutive rows gets one atomic for all of them: forks of one sequence,
// which stand next to each other in lists, share most of their pages. (64 x 16 forks of 513 pages: 7 us,
// with an atomic each 20.)
__device__ __forceinline__ void count_runs(const MxPages& p, const int (&page)[kTogether], int by) {
  int run = 0;
#pragma unroll
  for (int k = 0; k < kTogether; ++k) {
    ++run;
    if (k + 1 < kTogether && page[k + 1] == page[k]) continue;
    if (is_page(p, page[k])) atomicAdd(p.refs + page[k], by * run);
    run = 0;
  }
}

// ---- free ----
// Of entries with the same slot the first does the work, down to the smallest number that one of them
// keeps; nobody else looks at the slot.
__global__ __launch_bounds__(1024) void mx_pages_free_kernel(MxPages p, const int32_t* slots, const int32_t* keep, int n) {
  __shared__ Listed at;
  const int first = blockIdx.x * kTogether;
  if (threadIdx.x < kTogether) {
    const int i = first + threadIdx.x, slot = i < n ? slots[i] : -1;
    at.slot[threadIdx.x] = slot >= 0 && slot < p.slots ? slot : -1;
    at.other[threadIdx.x] = i < n && keep && keep[i] > 0 ? keep[i] : 0;
  }
  __syncthreads();
  int slot[kTogether];
#pragma unroll
  for (int k = 0; k < kTogether; ++k) slot[k] = at.slot[k];
  __syncthreads();
  for (int j = threadIdx.x; j < n; j += blockDim.x) {
    const int other = slots[j];
#pragma unroll
    for (int k = 0; k < kTogether; ++k) {
      if (other != slot[k] || j == first + k || slot[k] < 0) continue;
      if (j < first + k) at.slot[k] = -1;
      else atomicMin(at.other + k, keep && keep[j] > 0 ? keep[j] : 0);
    }
  }
  __syncthreads();
  if (threadIdx.x < kTogether) {
    const int mine = at.slot[threadIdx.x], left = at.other[threadIdx.x];
    const int len = mine >= 0 ? length_of(p, mine) : 0;
    at.begin[threadIdx.x] = pages_of(p, left);
    at.end[threadIdx.x] = left < len ? pages_of(p, len) : 0;
    if (left < len) p.lens[mine] = left;
  }
  __syncthreads();
  int last = 0;
#pragma unroll
  for (int k = 0; k < kTogether; ++k) last = at.end[k] > last ? at.end[k] : last;
  for (int e = threadIdx.x; e < last; e += blockDim.x) {
    int page[kTogether];
#pragma unroll
    for (int k = 0; k < kTogether; ++k)
      page[k] = e >= at.begin[k] && e < at.end[k] ? p.table[(int64_t)at.slot[k] * p.stride + e] : -1;
#pragma unroll
    for (int k = 0; k < kTogether; ++k)
      if (e >= at.begin[k] && e < at.end[k]) p.table[(int64_t)at.slot[k] * p.stride + e] = -1;
    count_runs(p, page, -1);
  }
}

// ---- fork ----
// Whether a pair counts depends on the lists, and on lengths that no pair that counts writes but
// its own.
__global__ __launch_bounds__(1024) void mx_pages_fork_kernel(MxPages p, const int32_t* parents, const int32_t* children,
                                                             int n, int32_t* done) {
  __shared__ Listed at;  // slot: the child, other: the parent
  __shared__ int bad[kTogether];
  const int first = blockIdx.x * kTogether;
  if (threadIdx.x < kTogether) {
    const int i = first + threadIdx.x, child = i < n ? children[i] : -1, parent = i < n ? parents[i] : -1;
    at.slot[threadIdx.x] = child;
    at.other[threadIdx.x] = parent;
    bad[threadIdx.x] = child < 0 || child >= p.slots || parent < 0 || parent >= p.slots || p.lens[child] > 0;
  }
  __syncthreads();
  int child[kTogether], parent[kTogether];
#pragma unroll
  for (int k = 0; k < kTogether; ++k) {
    child[k] = at.slot[k];
    parent[k] = at.other[k];
  }
  for (int j = threadIdx.x; j < n; j += blockDim.x) {
    const int other = children[j];
#pragma unroll
    for (int k = 0; k < kTogether; ++k)
      if ((other == child[k] && j < first + k) || other == parent[k]) bad[k] = 1;
  }
  __syncthreads();
  if (threadIdx.x < kTogether) {
    const int i = first + threadIdx.x, no = bad[threadIdx.x];
    const int len = no ? 0 : length_of(p, at.other[threadIdx.x]);
    at.end[threadIdx.x] = pages_of(p, len);
    if (!no) p.lens[at.slot[threadIdx.x]] = len;
    if (i < n) done[i] = !no;
  }
  __syncthreads();
  int last = 0;
#pragma unroll
  for (int k = 0; k < kTogether; ++k) last = at.end[k] > last ? at.end[k] : last;
  for (int e = threadIdx.x; e < last; e += blockDim.x) {
    int page[kTogether];
#pragma unroll
    for (int k = 0; k < kTogether; ++k) page[k] = e < at.end[k] ? p.table[(int64_t)parent[k] * p.stride + e] : -1;
#pragma unroll
    for (int k = 0; k < kTogether; ++k)
      if (e < at.end[k]) p.table[(int64_t)child[k] * p.stride + e] = page[k];
    count_runs(p, page, 1);
  }
}

// ---- scans over the counts ----

// exclusive sums over the workgroup's threads; all: the total
template <typename T>
__device__ __forceinline__ T scan(T x, T* sums /* [kPlan / 64] in LDS */, T& all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  T s = x;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const T y = __shfl_up(s, off, 64);
    if (lane >= off) s += y;
  }
  __syncthreads();
  if (lane == 63) sums[wave] = s;
  __syncthreads();
  T before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < kPlan / 64; ++w) {
    if (w < wave) before += sums[w];
    all += sums[w];
  }
  return before + s - x;
}

__device__ __forceinline__ uint64_t below(int64_t n) {  // the lowest n bits
  return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1;
}

// Bit b of word w: page 64 w + b has a count above 0. Up to kOneScan pages the planning workgroup
// reads the counts itself (131,072: some 5 us at a CU's rate), beyond that a launch over all CUs
// leaves it the words, an eighth of a byte a page.
constexpr int64_t kOneScan = 1 << 17;

__device__ __forceinline__ uint64_t used_word(const MxPages& p, int64_t word) {
  const int64_t page = word * 64 + (threadIdx.x & 63);
  return __ballot(page < p.num_pages && p.refs[page] > 0);
}

__global__ __launch_bounds__(kThreads) void mx_pages_words_kernel(MxPages p, uint64_t* words) {
  const int64_t word = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  const uint64_t b = used_word(p, word);
  if ((threadIdx.x & 63) == 0 && word * 64 < p.num_pages) words[word] = b;
}

// the words of a segment in LDS, 0 behind the last page
__device__ __forceinline__ void fill_bits(const MxPages& p, int64_t base, const uint64_t* ready, uint64_t* bits) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t left = p.num_pages - base;
  const int words = left >= kSegment ? kWords : (int)((left + 63) >> 6);
  if (ready) {
    for (int w = threadIdx.x; w < kWords; w += kPlan) bits[w] = w < words ? ready[base / 64 + w] : 0;
    return;
  }
  constexpr int kStep = kPlan / 64, kAhead = 8;
  for (int w = wave; w < words; w += kStep * kAhead) {
    int v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t page = base + (int64_t)(w + i * kStep) * 64 + lane;
      v[i] = p.refs[page < p.num_pages ? page : p.num_pages - 1];  // (a load under a condition waits for the one before)
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const uint64_t b = __ballot(v[i] > 0) & below(left - (int64_t)(w + i * kStep) * 64);
      if (lane == 0 && w + i * kStep < words) bits[w + i * kStep] = b;
    }
  }
  for (int w = words + threadIdx.x; w < kWords; w += kPlan) bits[w] = 0;
}

// ---- reserve ----
// One workgroup finds what each listed slot needs, where its share of the new pages starts, and
// the lowest free pages. A wave for each slot then enters them: for short lists a wave of the same
// workgroup, otherwise of a launch of its own.
constexpr int kOneLaunch = 128;

// every access of the thread has been performed, atomics and stores in the L2
__device__ __forceinline__ void drained() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0);
  asm volatile("" ::: "memory");
}

// by the wave, for list entry i
__device__ __forceinline__ void enter(const MxPages& p, int i, int2 plan, int found, int slot, int target, int len, int32_t* done,
                                      int32_t* src, int32_t* dst, const int32_t* fresh) {
  const int lane = threadIdx.x & 63, need = plan.y >> 1;
  const bool served = plan.y >= 0 && (need == 0 || (int64_t)plan.x + need <= found);
  int from = -1, to = -1;
  if (served) {
    int32_t* row = p.table + (int64_t)slot * p.stride;
    int have = pages_of(p, len);
    if (plan.y & 1) {
      --have;  // the last one too is new
      from = row[have];
      to = fresh[plan.x];
    }
    for (int k = lane; k < need; k += 64) {
      const int page = fresh[plan.x + k];
      row[have + k] = page;
      p.refs[page] = 1;
    }
    if (lane == 0) {
      if (from >= 0) atomicSub(p.refs + from, 1);
      if (target > len) p.lens[slot] = target;
    }
  }
  if (lane == 0) {
    done[i] = served ? 1 : 0;
    src[i] = from;
    dst[i] = to;
  }
}

__global__ __launch_bounds__(kPlan) void mx_pages_plan_kernel(MxPages p, const int32_t* slots, const int32_t* lens, int n,
                                                              int32_t* done, int32_t* src, int32_t* dst, MxReserveWork work,
                                                              const uint64_t* ready) {
  __shared__ uint64_t bits[kWords];
  __shared__ int before[kWords];
  __shared__ int64_t sums[kPlan / 64];
  __shared__ int2 plans[kOneLaunch];
  __shared__ int4 asked[kOneLaunch];  // slot, length to be, length
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // The first place in the list of each slot, by atomics: a store to be seen by them has to be in
  // the L2, which waiting for it ensures; a fence would write back all of the L2 (2 us each).
  for (int i = threadIdx.x; i < n; i += kPlan)
    if (slots[i] >= 0 && slots[i] < p.slots)
      __hip_atomic_store(work.mark + slots[i], n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  drained();
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlan)
    if (slots[i] >= 0 && slots[i] < p.slots) atomicMin(work.mark + slots[i], i);
  fill_bits(p, 0, ready, bits);
  drained();
  __syncthreads();
  int64_t total = 0;
  for (int i0 = 0; i0 < n; i0 += kPlan) {
    const int i = i0 + threadIdx.x;
    int need = -1;  // not to be served
    bool copies = false;
    int slot = -1, to = 0, len = 0;
    if (i < n) {
      slot = slots[i];
      to = lens[i];
      if (slot >= 0 && slot < p.slots) {
        const int first = __hip_atomic_load(work.mark + slot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        len = length_of(p, slot);
        const int have = pages_of(p, len);
        if (first == i && to >= len && (int64_t)to <= (int64_t)p.max_pages << p.page_shift) {
          if (to > len && (len & ((1 << p.page_shift) - 1)) != 0) {
            const int last = p.table[(int64_t)slot * p.stride + have - 1];
            copies = is_page(p, last) && p.refs[last] > 1;
          }
          need = pages_of(p, to) - have + (copies ? 1 : 0);
        }
      }
    }
    int64_t all;
    const int64_t start = total + scan<int64_t>(need > 0 ? need : 0, sums, all);
    const int2 plan = make_int2(start < p.num_pages ? (int)start : (int)p.num_pages, need < 0 ? -1 : 2 * need + copies);
    if (n <= kOneLaunch && i < n) {
      plans[i] = plan;
      asked[i] = make_int4(slot, to, len, 0);
    } else if (i < n) {
      work.plan[i] = plan;
    }
    total += all;
  }
  const int64_t most = total < p.num_pages ? total : p.num_pages;
  int64_t found = 0;
  for (int64_t base = 0; found < most && base < p.num_pages; base += kSegment) {
    if (base > 0) {
      __syncthreads();
      fill_bits(p, base, ready, bits);
      __syncthreads();
    }
    const int64_t left = p.num_pages - base;
    const int words = left >= kSegment ? kWords : (int)((left + 63) >> 6);
    int count = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int w = threadIdx.x * kEach + j;
      count += __popcll(~bits[w] & below(left - (int64_t)w * 64));
    }
    int all;
    int at = scan<int>(count, (int*)sums, all);
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int w = threadIdx.x * kEach + j;
      before[w] = at;
      at += __popcll(~bits[w] & below(left - (int64_t)w * 64));
    }
    __syncthreads();
    for (int w = wave; w < words; w += kPlan / 64) {
      const uint64_t b = ~bits[w] & below(left - (int64_t)w * 64);
      const int64_t k = found + before[w] + __popcll(b & below(lane));
      if (found + before[w] >= most) break;
      if ((b >> lane & 1) != 0 && k < most) work.fresh[k] = (int)(base + (int64_t)w * 64 + lane);
    }
    found += all;
  }
  found = found < most ? found : most;
  if (threadIdx.x == 0) *work.found = (int)found;
  if (n > kOneLaunch) return;
  __syncthreads();
  for (int i = wave; i < n; i += kPlan / 64)
    enter(p, i, plans[i], (int)found, asked[i].x, asked[i].y, asked[i].z, done, src, dst, work.fresh);
}

__global__ __launch_bounds__(kThreads) void mx_pages_enter_kernel(MxPages p, const int32_t* slots, const int32_t* lens, int n,
                                                                  int32_t* done, int32_t* src, int32_t* dst,
                                                                  MxReserveWork work) {
  const int i = blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (i >= n) return;
  const int slot = slots[i];
  const int2 plan = work.plan[i];
  const int len = plan.y >= 0 ? length_of(p, slot) : 0;
  enter(p, i, plan, *work.found, slot, lens[i], len, done, src, dst, work.fresh);
}

// ---- compact ----
// With u pages in use, those at u and above move into the free ones below it, k-th to k-th.
// One workgroup numbers both; then the tables are rewritten.
__global__ __launch_bounds__(kPlan) void mx_pages_moves_kernel(MxPages p, int32_t* src, int32_t* dst, int32_t* used,
                                                               int32_t* rank, int32_t* counts, const uint64_t* ready) {
  __shared__ uint64_t bits[kWords];
  __shared__ int before[kWords];
  __shared__ int64_t sums[kPlan / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t u = 0, all;
  for (int64_t base = 0; base < p.num_pages; base += kSegment) {
    __syncthreads();
    fill_bits(p, base, ready, bits);
    __syncthreads();
    int count = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) count += __popcll(bits[threadIdx.x * kEach + j]);
    scan<int64_t>(count, sums, all);
    u += all;
  }
  if (threadIdx.x == 0) *used = (int)u;
  // A word below u has free pages to number, one above it used ones, the one that u lies in
  // both, whose used ones are the first.
  int64_t holes = 0, movers = 0;
  for (int64_t base = 0; base < p.num_pages; base += kSegment) {
    if (p.num_pages > kSegment) {  // else they are there
      __syncthreads();
      fill_bits(p, base, ready, bits);
      __syncthreads();
    }
    int nh[kEach], nm[kEach], h = 0, m = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const uint64_t w = bits[threadIdx.x * kEach + j];
      const uint64_t low = below(u - base - (int64_t)(threadIdx.x * kEach + j) * 64);
      nh[j] = __popcll(~w & low);
      nm[j] = __popcll(w & ~low);
      h += nh[j];
      m += nm[j];
    }
    const int64_t both = scan<int64_t>((int64_t)h << 32 | m, sums, all);  // each below 2^31
    h = (int)(both >> 32);
    m = (int)(both & 0xFFFFFFFF);
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      before[threadIdx.x * kEach + j] = u > base + (int64_t)(threadIdx.x * kEach + j) * 64 ? h : m;
      h += nh[j];
      m += nm[j];
    }
    __syncthreads();
    const int64_t left = p.num_pages - base;
    const int words = left >= kSegment ? kWords : (int)((left + 63) >> 6);
    for (int i = wave; i < words; i += kPlan / 64) {
      const uint64_t w = bits[i], low = below(u - base - (int64_t)i * 64), upto = below(lane);
      const int64_t page = base + (int64_t)i * 64 + lane;
      if ((~w & low) >> lane & 1) dst[holes + before[i] + __popcll(~w & low & upto)] = (int)page;
      if ((w & ~low) >> lane & 1) {
        const int64_t k = movers + (low == 0 ? before[i] : 0) + __popcll(w & ~low & upto);
        src[k] = (int)page;
        rank[page] = (int)k;
      }
    }
    holes += all >> 32;
    movers += all & 0xFFFFFFFF;
  }
  for (int64_t k = movers + threadIdx.x; k < p.num_pages / 2; k += kPlan) src[k] = dst[k] = -1;
  __syncthreads();
  constexpr int kAhead = 4;  // the movers' counts: two loads each, of four at a time
  for (int64_t k0 = threadIdx.x; k0 < movers; k0 += kPlan * kAhead) {
    int c[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) c[i] = k0 + i * kPlan < movers ? src[k0 + i * kPlan] : 0;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) c[i] = p.refs[c[i]];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (k0 + i * kPlan < movers) counts[k0 + i * kPlan] = c[i];
  }
}

// One thread for each count and each entry. A count is read where it is written, or from the
// movers' list, and so may be rewritten in place.
__global__ __launch_bounds__(kThreads) void mx_pages_rewrite_kernel(MxPages p, int32_t* table, int64_t stride, int32_t* refs,
                                                                    const int32_t* src, const int32_t* dst,
                                                                    const int32_t* used,
                                                                    const int32_t* rank, const int32_t* counts,
                                                                    int64_t count_groups, int64_t row_groups) {
  const int u = *used;
  if (blockIdx.x < count_groups) {
    const int64_t page = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (page < p.num_pages) {
      const int c = p.refs[page];
      if (page >= u) refs[page] = 0;
      else if (c > 0) refs[page] = c;
    }
    if (page < p.num_pages / 2 && dst[page] >= 0) refs[dst[page]] = counts[page];
    return;
  }
  const int64_t group = blockIdx.x - count_groups, slot = group / row_groups;
  const int64_t e = (group - slot * row_groups) * kThreads + threadIdx.x;
  if (e >= p.max_pages) return;
  int page = p.table[slot * p.stride + e];
  if (e < pages_of(p, p.lens[slot]) && is_page(p, page) && page >= u) {
    const int k = rank[page];  // anything if the page is held without a count: then it is not the k-th mover
    if (k >= 0 && k < p.num_pages / 2 && src[k] == page) page = dst[k];
  }
  table[slot * stride + e] = page;
}

// ---- copies of pages ----
struct CopyArgs {
  const uint8_t* from[4];  // codes and scales of keys, of values
  uint8_t* to[4];
  int64_t codes, scales;   // 16-byte pieces of a page
  int64_t from_pages, to_pages, items;
  int chunks;              // items of a pair
  const int32_t* src;
  const int32_t* dst;
};

constexpr int kPieces = 4;  // of a thread in an item, all in flight

// Workgroups of a fixed number take items (a pair and a part of its page) in turn and look at 64
// of theirs at once, so that a list of few pairs among many entries costs little.
__global__ __launch_bounds__(kThreads) void mx_cache_copy_kernel(CopyArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t each = 2 * (a.codes + a.scales);
  for (int64_t first = blockIdx.x; first < a.items; first += (int64_t)gridDim.x * 64) {
    const int64_t mine = first + (int64_t)lane * gridDim.x;
    int from = -1, to = -1, part = 0;
    if (mine < a.items) {
      const int64_t pair = mine / a.chunks;
      part = (int)(mine - pair * a.chunks);
      from = a.src[pair];
      to = a.dst[pair];
    }
    uint64_t live = __ballot(from >= 0 && from < a.from_pages && to >= 0 && to < a.to_pages);
    for (; live != 0; live &= live - 1) {
      const int l = __builtin_ctzll(live);
      const int64_t s = __builtin_amdgcn_readlane(from, l), d = __builtin_amdgcn_readlane(to, l);
      const int64_t at = (int64_t)__builtin_amdgcn_readlane(part, l) * (kThreads * kPieces) + threadIdx.x;
      u32x4_t x[kPieces];
      u32x4_t* out[kPieces];
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        int64_t piece = at + i * kThreads;
        out[i] = nullptr;
        if (piece >= each) continue;
        int which = 0;
        if (piece >= a.codes + a.scales) {
          piece -= a.codes + a.scales;
          which = 2;
        }
        if (piece >= a.codes) {
          piece -= a.codes;
          which += 1;
        }
        const int64_t n = which & 1 ? a.scales : a.codes;
        const uint8_t* const from_at = which == 0 ? a.from[0] : which == 1 ? a.from[1] : which == 2 ? a.from[2] : a.from[3];
        uint8_t* const to_at = which == 0 ? a.to[0] : which == 1 ? a.to[1] : which == 2 ? a.to[2] : a.to[3];
        x[i] = *((const u32x4_t*)from_at + s * n + piece);
        out[i] = (u32x4_t*)to_at + d * n + piece;
      }
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        if (out[i]) *out[i] = x[i];
    }
  }
}

}  // namespace

// threads for rows of so many entries
static int row_threads(const MxPages& p) { return p.max_pages > 512 ? 1024 : kThreads; }

static unsigned list_groups(int n) { return (unsigned)((n + kTogether - 1) / kTogether); }

// the words, for many pages; null: the planning workgroup reads the counts
static hipError_t launch_words(const MxPages& p, uint64_t* words, const uint64_t** ready, hipStream_t stream) {
  *ready = nullptr;
  if (p.num_pages <= kOneScan) return hipSuccess;
  *ready = words;
  const int64_t n = (p.num_pages + 63) / 64;
  constexpr int per = kThreads / 64;
  mx_pages_words_kernel<<<(unsigned)((n + per - 1) / per), kThreads, 0, stream>>>(p, words);
  return hipGetLastError();
}

static int64_t words_bytes(int64_t num_pages) { return num_pages <= kOneScan ? 0 : (num_pages + 63) / 64 * 8; }

int64_t mx_reserve_bytes(int64_t n, int64_t slots, int64_t max_pages, int64_t num_pages) {
  const int64_t most = n * (max_pages + 1), fresh = most < num_pages ? most : num_pages;
  return (words_bytes(num_pages) + 8 * n + 16 + 4 * slots + 4 * fresh + 15) / 16 * 16;
}

int64_t mx_compact_bytes(int64_t num_pages) {
  return (words_bytes(num_pages) + 4 * num_pages + 4 * (num_pages / 2) + 15) / 16 * 16;
}

hipError_t launch_mx_pages_free(const MxPages& p, const int32_t* slots, const int32_t* keep, int n, hipStream_t stream) {
  mx_pages_free_kernel<<<list_groups(n), row_threads(p), 0, stream>>>(p, slots, keep, n);
  return hipGetLastError();
}

hipError_t launch_mx_pages_fork(const MxPages& p, const int32_t* parents, const int32_t* children, int n, int32_t* done,
                                hipStream_t stream) {
  mx_pages_fork_kernel<<<list_groups(n), row_threads(p), 0, stream>>>(p, parents, children, n, done);
  return hipGetLastError();
}

hipError_t launch_mx_pages_reserve(const MxPages& p, const int32_t* slots, const int32_t* lens, int n, int32_t* done,
                                   int32_t* src, int32_t* dst, void* workspace, hipStream_t stream) {
  const uint64_t* ready;
  hipError_t e = launch_words(p, (uint64_t*)workspace, &ready, stream);
  if (e != hipSuccess) return e;
  MxReserveWork w;
  w.plan = (int2*)((uint8_t*)workspace + words_bytes(p.num_pages));
  w.found = (int32_t*)(w.plan + n);
  w.mark = w.found + 4;
  w.fresh = w.mark + p.slots;
  mx_pages_plan_kernel<<<1, kPlan, 0, stream>>>(p, slots, lens, n, done, src, dst, w, ready);
  e = hipGetLastError();
  if (e != hipSuccess || n <= kOneLaunch) return e;
  constexpr int per = kThreads / 64;
  mx_pages_enter_kernel<<<(n + per - 1) / per, kThreads, 0, stream>>>(p, slots, lens, n, done, src, dst, w);
  return hipGetLastError();
}

hipError_t launch_mx_pages_compact(const MxPages& p, int32_t* table_out, int64_t stride_out, int32_t* refs_out,
                                   int32_t* src, int32_t* dst, int32_t* used, void* workspace, hipStream_t stream) {
  const uint64_t* ready;
  hipError_t e = launch_words(p, (uint64_t*)workspace, &ready, stream);
  if (e != hipSuccess) return e;
  int32_t* rank = (int32_t*)((uint8_t*)workspace + words_bytes(p.num_pages));
  int32_t* counts = rank + p.num_pages;
  mx_pages_moves_kernel<<<1, kPlan, 0, stream>>>(p, src, dst, used, rank, counts, ready);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t count_groups = (p.num_pages + kThreads - 1) / kThreads, row_groups = (p.max_pages + kThreads - 1) / kThreads;
  mx_pages_rewrite_kernel<<<(unsigned)(count_groups + p.slots * row_groups), kThreads, 0, stream>>>(
      p, table_out, stride_out, refs_out, src, dst, used, rank, counts, count_groups, row_groups);
  return hipGetLastError();
}

hipError_t launch_mx_cache_copy(const MxCache& from, int64_t from_pages, const MxCache& to, int64_t to_pages,
                                int page_size, const int32_t* src, const int32_t* dst, int64_t n, hipStream_t stream) {
  CopyArgs a;
  const int64_t rows = (int64_t)from.kv_heads * page_size;
  a.codes = rows * (from.head_dim / 2) / 16;
  a.scales = rows * (from.head_dim / 32) / 16;
  const uint8_t* f[4] = {from.k_codes, from.k_scales, from.v_codes, from.v_scales};
  uint8_t* t[4] = {to.k_codes, to.k_scales, to.v_codes, to.v_scales};
  for (int i = 0; i < 4; ++i) {
    a.from[i] = f[i];
    a.to[i] = t[i];
  }
  a.from_pages = from_pages;
  a.to_pages = to_pages;
  a.chunks = (int)((2 * (a.codes + a.scales) + kThreads * kPieces - 1) / (kThreads * kPieces));
  a.items = n * a.chunks;
  a.src = src;
  a.dst = dst;
  const int64_t groups = a.items < 2048 ? a.items : 2048;
  mx_cache_copy_kernel<<<(unsigned)groups, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace nvfp4
