// mx_pages.hip - which pages of a paged cache the sequences hold, kept on the device, and
// copies of whole pages (gfx950).
//
// The bookkeeping is integers: a few loads that depend on one another, so its time is their
// latency and the launches. Its results do not depend on the order in which threads run:
// counts change by integer atomics, a slot that is listed twice is settled by the lower
// place in the list, and free pages are given out lowest first in the list's order. Copies are
// bound by memory, every byte read and written once.
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

__device__ __forceinline__ bool is_page(const MxPages& p, int page) { return page >= 0 && page < p.num_pages; }

// ---- free ----
// A workgroup per listed slot. Entries are taken out by exchange, so that of two workgroups
// with the same slot one lowers a page's count; either finds the slot's length as it was or
// cut by the other, and what the other cut, the other takes out.
__global__ __launch_bounds__(kThreads) void mx_pages_free_kernel(MxPages p, const int32_t* slots, const int32_t* keep) {
  const int slot = slots[blockIdx.x];
  if (slot < 0 || slot >= p.slots) return;
  __shared__ int len_was;
  if (threadIdx.x == 0) len_was = __hip_atomic_load(p.lens + slot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  const int len = len_was, left = keep && keep[blockIdx.x] > 0 ? keep[blockIdx.x] : 0;
  if (left >= len) return;
  int32_t* row = p.table + (int64_t)slot * p.stride;
  const int end = pages_of(p, len);
#pragma unroll 4
  for (int e = pages_of(p, left) + threadIdx.x; e < end; e += kThreads) {
    const int page = atomicExch(row + e, -1);
    if (is_page(p, page)) atomicSub(p.refs + page, 1);
  }
  if (threadIdx.x == 0) atomicMin(p.lens + slot, left);
}

// ---- fork ----
// A workgroup per pair. Whether a pair counts depends on the lists and on lengths that no
// pair that counts writes.
__global__ __launch_bounds__(kThreads) void mx_pages_fork_kernel(MxPages p, const int32_t* parents, const int32_t* children,
                                                                 int n, int32_t* done) {
  const int i = blockIdx.x, parent = parents[i], child = children[i];
  bool bad = parent < 0 || parent >= p.slots || child < 0 || child >= p.slots;
  for (int j = threadIdx.x; j < n; j += kThreads) {
    const int other = children[j];
    bad |= (j < i && other == child) || other == parent;
  }
  if (!__syncthreads_or(bad)) bad = p.lens[child] > 0;
  else bad = true;
  // every thread has read the length before it is written
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) done[i] = 0;
    return;
  }
  const int len = p.lens[parent], held = pages_of(p, len);
  const int32_t* from = p.table + (int64_t)parent * p.stride;
  int32_t* to = p.table + (int64_t)child * p.stride;
#pragma unroll 4
  for (int e = threadIdx.x; e < held; e += kThreads) {
    const int page = from[e];
    to[e] = page;
    if (is_page(p, page)) atomicAdd(p.refs + page, 1);
  }
  if (threadIdx.x == 0) {
    p.lens[child] = len;
    done[i] = 1;
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

// bit b of word w: page base + 64 w + b has a count above 0 (used) or not (free)
__device__ __forceinline__ void fill_bits(const MxPages& p, int64_t base, bool used, uint64_t* bits) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t left = p.num_pages - base;
  const int words = left >= kSegment ? kWords : (int)((left + 63) >> 6);
  constexpr int kStep = kPlan / 64, kAhead = 8;
  for (int w = wave; w < words; w += kStep * kAhead) {
    int v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t page = base + (int64_t)(w + i * kStep) * 64 + lane;
      v[i] = page < p.num_pages ? p.refs[page] : (used ? 0 : 1);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const uint64_t b = __ballot((v[i] > 0) == used);
      if (lane == 0 && w + i * kStep < words) bits[w + i * kStep] = b;
    }
  }
  for (int w = words + threadIdx.x; w < kWords; w += kPlan) bits[w] = 0;
}

// ---- reserve ----
// Two launches: one workgroup finds what each listed slot needs, where its share of the new
// pages starts, and the lowest free pages; then a wave for each slot enters them.
__global__ __launch_bounds__(kPlan) void mx_pages_plan_kernel(MxPages p, const int32_t* slots, const int32_t* lens, int n,
                                                              MxReserveWork work) {
  __shared__ uint64_t bits[kWords];
  __shared__ int before[kWords];
  __shared__ int64_t sums[kPlan / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  fill_bits(p, 0, false, bits);
  // the first place in the list of each slot
  for (int i = threadIdx.x; i < n; i += kPlan)
    if (slots[i] >= 0 && slots[i] < p.slots) work.mark[slots[i]] = n;
  __threadfence();
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlan)
    if (slots[i] >= 0 && slots[i] < p.slots) atomicMin(work.mark + slots[i], i);
  __threadfence();
  __syncthreads();
  int64_t total = 0;
  for (int i0 = 0; i0 < n; i0 += kPlan) {
    const int i = i0 + threadIdx.x;
    int need = -1;  // not to be served
    bool copies = false;
    if (i < n) {
      const int slot = slots[i], to = lens[i];
      if (slot >= 0 && slot < p.slots &&
          __hip_atomic_load(work.mark + slot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == i) {
        const int len = p.lens[slot] > 0 ? p.lens[slot] : 0, have = pages_of(p, len);
        if (to >= len && (int64_t)to <= (int64_t)p.max_pages << p.page_shift) {
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
    if (i < n) work.plan[i] = make_int2(start < p.num_pages ? (int)start : (int)p.num_pages, need < 0 ? -1 : 2 * need + copies);
    total += all;
  }
  const int64_t most = total < p.num_pages ? total : p.num_pages;
  int64_t found = 0;
  for (int64_t base = 0; found < most && base < p.num_pages; base += kSegment) {
    if (base > 0) {
      __syncthreads();
      fill_bits(p, base, false, bits);
    }
    __syncthreads();
    int count = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) count += __popcll(bits[threadIdx.x * kEach + j]);
    int64_t all;
    int at = (int)scan<int64_t>(count, sums, all);
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      before[threadIdx.x * kEach + j] = at;
      at += __popcll(bits[threadIdx.x * kEach + j]);
    }
    __syncthreads();
    const int64_t left = p.num_pages - base;
    const int words = left >= kSegment ? kWords : (int)((left + 63) >> 6);
    for (int w = wave; w < words; w += kPlan / 64) {
      const uint64_t b = bits[w];
      const int64_t k = found + before[w] + __popcll(b & ((1ull << lane) - 1));
      if ((b >> lane & 1) != 0 && k < most) work.fresh[k] = (int)(base + (int64_t)w * 64 + lane);
    }
    found += all;
  }
  if (threadIdx.x == 0) *work.found = (int)(found < most ? found : most);
}

__global__ __launch_bounds__(kThreads) void mx_pages_enter_kernel(MxPages p, const int32_t* slots, const int32_t* lens, int n,
                                                                  int32_t* done, int32_t* src, int32_t* dst,
                                                                  MxReserveWork work) {
  const int lane = threadIdx.x & 63;
  const int i = blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (i >= n) return;
  const int2 plan = work.plan[i];
  const int need = plan.y >> 1;
  const bool served = plan.y >= 0 && (need == 0 || (int64_t)plan.x + need <= *work.found);
  int from = -1, to = -1;
  if (served) {
    const int slot = slots[i], target = lens[i];
    const int len = p.lens[slot] > 0 ? p.lens[slot] : 0;
    int32_t* row = p.table + (int64_t)slot * p.stride;
    int have = pages_of(p, len);
    if (plan.y & 1) {
      --have;  // the last one too is new
      from = row[have];
      to = work.fresh[plan.x];
    }
    for (int k = lane; k < need; k += 64) {
      const int page = work.fresh[plan.x + k];
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

// ---- compact ----
__device__ __forceinline__ uint64_t below(int64_t n) {  // the lowest n bits
  return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1;
}

// With u pages in use, those at u and above move into the free ones below it, k-th to k-th.
// One workgroup numbers both; then the tables are rewritten.
__global__ __launch_bounds__(kPlan) void mx_pages_moves_kernel(MxPages p, int32_t* src, int32_t* dst, int32_t* used,
                                                               int32_t* rank, int32_t* counts) {
  __shared__ uint64_t bits[kWords];
  __shared__ int before[kWords];
  __shared__ int64_t sums[kPlan / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t u = 0, all;
  for (int64_t base = 0; base < p.num_pages; base += kSegment) {
    __syncthreads();
    fill_bits(p, base, true, bits);
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
      fill_bits(p, base, true, bits);
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
      const uint64_t w = bits[i], low = below(u - base - (int64_t)i * 64), upto = (1ull << lane) - 1;
      const int64_t page = base + (int64_t)i * 64 + lane;
      if ((~w & low) >> lane & 1) dst[holes + before[i] + __popcll(~w & low & upto)] = (int)page;
      if ((w & ~low) >> lane & 1) {
        const int64_t k = movers + (low == 0 ? before[i] : 0) + __popcll(w & ~low & upto);
        src[k] = (int)page;
        counts[k] = p.refs[page];
        rank[page] = (int)k;
      }
    }
    holes += all >> 32;
    movers += all & 0xFFFFFFFF;
  }
  for (int64_t k = movers + threadIdx.x; k < p.num_pages / 2; k += kPlan) src[k] = dst[k] = -1;
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

hipError_t launch_mx_pages_free(const MxPages& p, const int32_t* slots, const int32_t* keep, int n, hipStream_t stream) {
  mx_pages_free_kernel<<<n, kThreads, 0, stream>>>(p, slots, keep);
  return hipGetLastError();
}

hipError_t launch_mx_pages_fork(const MxPages& p, const int32_t* parents, const int32_t* children, int n, int32_t* done,
                                hipStream_t stream) {
  mx_pages_fork_kernel<<<n, kThreads, 0, stream>>>(p, parents, children, n, done);
  return hipGetLastError();
}

hipError_t launch_mx_pages_reserve(const MxPages& p, const int32_t* slots, const int32_t* lens, int n, int32_t* done,
                                   int32_t* src, int32_t* dst, void* workspace, hipStream_t stream) {
  MxReserveWork w;
  w.plan = (int2*)workspace;
  w.found = (int32_t*)(w.plan + n);
  w.mark = w.found + 4;
  w.fresh = w.mark + p.slots;
  mx_pages_plan_kernel<<<1, kPlan, 0, stream>>>(p, slots, lens, n, w);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  constexpr int per = kThreads / 64;
  mx_pages_enter_kernel<<<(n + per - 1) / per, kThreads, 0, stream>>>(p, slots, lens, n, done, src, dst, w);
  return hipGetLastError();
}

hipError_t launch_mx_pages_compact(const MxPages& p, int32_t* table_out, int64_t stride_out, int32_t* refs_out,
                                   int32_t* src, int32_t* dst, int32_t* used, void* workspace, hipStream_t stream) {
  int32_t* rank = (int32_t*)workspace;
  int32_t* counts = rank + p.num_pages;
  mx_pages_moves_kernel<<<1, kPlan, 0, stream>>>(p, src, dst, used, rank, counts);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t count_groups = (p.num_pages + kThreads - 1) / kThreads, row_groups = (p.max_pages + kThreads - 1) / kThreads;
  mx_pages_rewrite_kernel<<<(unsigned)(count_groups + p.slots * row_groups), kThreads, 0, stream>>>(
      p, table_out, stride_out, refs_out, src, dst, used, rank, counts, count_groups, row_groups > 0 ? row_groups : 1);
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
