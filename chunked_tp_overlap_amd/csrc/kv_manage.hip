// The pages of a paged key-value cache: sequences that share pages, pages given and taken back,
// copies of pages, and tokens moved to the places after their sequence's kept ones.
//
// What holds a page is counted: refs[page] rows of the table have it, and a page of count 0 is
// free.  There is no list of free pages: giving pages takes the free ones of the lowest numbers,
// so that the same calls give the same pages on every run, whatever order counts changed in.
// Counts and tables are a few integers per page; what bounds these calls is their chains of
// loads and launches.  In kv_resize one workgroup gives pages, as a row's pages depend on all rows
// before it; then a wave for each row takes back what it gives up, in a launch of its own where
// rows are many.
// kv_copy_pages and kv_compact move tokens, 16 bytes to a lane.
//
// Measured on MI355X: 64 prompts of up to 8192 tokens forked into 8 samples each, which grow by up to 200
// tokens and end, 4 heads on 4, pages of 64: 29 us for the four calls, of which 3.7, 10, 3.6, 9 and 3.7
// are their kernels' (the copies 63 MB, 7 TB/s).
#include <hip/hip_runtime.h>

#include "attn_internal.h"
#include "gemm_common.h"
#include "kv_pages.h"

namespace ubx {
namespace {

__device__ inline int pages_of(int len, int page) { return len / page + (len % page != 0); }
__device__ inline int row_len(const Table& t, int len, int page) { return clamp_len(len, table_cap(t.per, page)); }

// ---- fork -----------------------------------------------------------------------------------
// A workgroup for each row of `in`, whose pages' counts change by its uses less one, then one
// for each row of `out`.
__global__ __launch_bounds__(256) void kv_fork(ForkArgs a) {
  const int r = blockIdx.x;
  if (r < a.in.n) {
    __shared__ int uses;
    if (threadIdx.x == 0) uses = -1;
    __syncthreads();
    int mine = 0;
    for (int i = threadIdx.x; i < a.out.n; i += 256) mine += a.parents[i] == r;
    if (mine) atomicAdd(&uses, mine);
    __syncthreads();
    const int change = uses, n = pages_of(row_len(a.in, a.lens[r], a.page), a.page);
    if (change == 0) return;
    const int32_t* row = a.in.p + (int64_t)r * a.in.ld;
    for (int e = threadIdx.x; e < n; e += 256) {
      const int id = row[e];
      if (id >= 0 && id < a.n_pages) atomicAdd(a.refs + id, change);
    }
    return;
  }
  const int i = r - a.in.n, of = a.parents[i];
  const bool some = of >= 0 && of < a.in.n;
  const int len = some ? row_len(a.in, a.lens[of], a.page) : 0, n = pages_of(len, a.page);
  const int32_t* from = a.in.p + (int64_t)(some ? of : 0) * a.in.ld;
  int32_t* to = a.out.p + (int64_t)i * a.out.ld;
  for (int e = threadIdx.x; e < a.out.per; e += 256) to[e] = e < n ? from[e] : -1;
  if (threadIdx.x == 0) a.lens_out[i] = len;
}

// ---- resize ---------------------------------------------------------------------------------
constexpr int GIVERS = 1024, GIVE_WAVES = GIVERS / 64;
constexpr int PER = 8;  // counts a thread looks at at a time

// What a row asks for: table entries `begin` and on, the last of which would be page number
// `end` (less one) of those that all rows up to it ask for.
struct Ask {
  int64_t end;
  int32_t begin, had;
  int32_t part, src;  // tokens of a shared last page, which goes to another row's holders; its id
};
// The workspace: free pages, or at least as many as are asked for, then the rows' asks.
constexpr int ASKS_AT = 16;
__device__ inline int64_t* free_of(void* ws) { return static_cast<int64_t*>(ws); }
__device__ inline Ask* asks_of(void* ws) {
  return reinterpret_cast<Ask*>(static_cast<unsigned char*>(ws) + ASKS_AT);
}

// Sum over the workgroup's threads before this one; all: over all of them.
__device__ inline int64_t scan_before(int64_t v, int64_t* sums, int64_t& all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t incl = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int64_t o = __shfl_up(incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 63) sums[wave] = incl;
  __syncthreads();
  int64_t before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < GIVE_WAVES; ++w) {
    if (w < wave) before += sums[w];
    all += sums[w];
  }
  __syncthreads();
  return before + incl - v;
}

// The lengths that a row has and is to have, within its table; a new length past it is none.
struct Lens {
  int has, wants;
  bool fits;
};
__device__ inline Lens lens_of(const ResizeArgs& a, int i) {
  const int cap = table_cap(a.table.per, a.page), len = a.lens[i], want = a.new_lens[i];
  Lens l;
  l.has = clamp_len(len, cap);
  l.fits = want <= cap;
  l.wants = l.fits ? max(want, 0) : l.has;
  return l;
}

// A row's end of the call, by one wave: what it gives up, its copy and its length; k: its ask,
// given: it gets what it asks for.
__device__ inline void take_row(const ResizeArgs& a, int i, const Ask& k, bool given) {
  const int lane = threadIdx.x & 63;
  const Lens l = lens_of(a, i);
  const int len = given ? l.wants : l.has, has = pages_of(len, a.page);
  int32_t* row = a.table.p + (int64_t)i * a.table.ld;
  const int to = given && k.part > 0 ? row[k.had - 1] : -1;
  auto take = [&](int e) {
    const int id = row[e];
    if (id >= 0 && id < a.n_pages) atomicAdd(a.refs + id, -1);
    row[e] = -1;
  };
  for (int e = has + lane; e < k.had; e += 64) take(e);
  bool hidden = false;  // all of the page that would be copied to
  if (a.win.size > 0 && len > a.win.size) {
    // pages of hidden tokens alone
    const int begin = pages_of(a.win.sinks, a.page), end = min((len - a.win.size) / a.page, has);
    hidden = k.had - 1 >= begin && k.had - 1 < end;
    for (int e = begin + lane; e < end; e += 64) take(e);
  }
  if (lane == 0) {
    const bool copy = given && k.part > 0 && !hidden;
    int32_t* c = a.copies + 3 * (int64_t)i;
    c[0] = copy ? k.src : -1;
    c[1] = copy ? to : -1;
    c[2] = copy ? k.part : 0;
    if (given && k.part > 0) atomicAdd(a.refs + k.src, -1);
    a.lens_out[i] = len;
  }
}

// One workgroup.  The rows' asks, the free pages counted as far as they are asked for, and then
// turn by turn a list of free pages in LDS, from which each goes to its row: the first whose `end`
// lies past the page's rank, found in LDS too (ROWS_IN_LDS rows and fewer).  576 rows that grow by
// 2000 pages together take 10.2 us; with the search in the workspace, and a page's place from the
// counts that its thread read, 19.6.  64 rows that get 500 pages each take some 50 us: one workgroup
// searches for the row of each of 32000 pages.
// ALL: and then what kv_take does for every row.
constexpr int ROWS_IN_LDS = 4096;
template <bool ALL>
__global__ __launch_bounds__(GIVERS) void kv_give(ResizeArgs a) {
  __shared__ int64_t sums[GIVE_WAVES];
  __shared__ int32_t ids[GIVERS * PER], ends[ROWS_IN_LDS];
  Ask* ask = asks_of(a.ws);
  const int n = a.table.n;
  const bool in_lds = n <= ROWS_IN_LDS;
  int64_t total = 0;
  for (int c = 0; c < n; c += GIVERS) {
    const int i = c + threadIdx.x;
    Ask k{0, 0, 0, 0, -1};
    int need = 0;
    if (i < n) {
      const Lens l = lens_of(a, i);
      k.had = pages_of(l.has, a.page);
      k.begin = k.had;
      if (l.wants > l.has) {
        const int part = l.has % a.page;
        if (part) {
          const int id = a.table.p[(int64_t)i * a.table.ld + k.had - 1];
          if (id >= 0 && id < a.n_pages && a.refs[id] > 1) {
            k.src = id;
            k.part = part;
            --k.begin;
          }
        }
        need = pages_of(l.wants, a.page) - k.begin;
      }
    }
    int64_t all;
    const int64_t before = scan_before(need, sums, all);
    if (i < n) {
      k.end = total + before + need;
      ask[i] = k;
      if (in_lds) ends[i] = (int32_t)min(k.end, (int64_t)0x7FFFFFFF);  // ranks stay below it
    }
    total += all;
  }
  // the first row whose end lies past `rank`, below n
  auto row_of = [&](int64_t rank) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if ((in_lds ? (int64_t)ends[mid] : ask[mid].end) > rank) hi = mid;
      else lo = mid + 1;
    }
    return lo;
  };
  int32_t r[PER];
  auto read = [&](int64_t id0) {
    if (id0 + PER <= a.n_pages) {
      const i32x4 lo = *GLOBAL_PTR(const i32x4, a.refs + id0), hi = *GLOBAL_PTR(const i32x4, a.refs + id0 + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r[j] = lo[j];
        r[4 + j] = hi[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j) r[j] = id0 + j < a.n_pages ? a.refs[id0 + j] : 1;
    }
    int mine = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) mine += r[j] == 0;
    return mine;
  };
  constexpr int TURN = GIVERS * PER;
  int64_t free = 0;
  bool first = true;  // r holds the first turn's counts
  for (int64_t c = 0; c < a.n_pages && free < total; c += TURN) {
    int64_t all;
    first = c == 0;
    scan_before(read(c + (int64_t)threadIdx.x * PER), sums, all);
    free += all;
  }
  if (threadIdx.x == 0) *free_of(a.ws) = free;
  // as many as go to rows that get all they ask for
  int64_t limit = total;
  if (free < total) {
    const int row = row_of(free);
    limit = row > 0 ? (in_lds ? ends[row - 1] : ask[row - 1].end) : 0;
  }
  int64_t found = 0;
  for (int64_t c = 0; c < a.n_pages && found < limit; c += TURN) {
    const int64_t id0 = c + (int64_t)threadIdx.x * PER;
    int mine = 0;
    if (c == 0 && first) {
#pragma unroll
      for (int j = 0; j < PER; ++j) mine += r[j] == 0;
    } else {
      mine = read(id0);
    }
    int64_t all;
    int at = (int)scan_before(mine, sums, all);  // and the last turn's list is read
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (r[j] == 0) ids[at++] = (int32_t)(id0 + j);
    __syncthreads();
    const int give = (int)min(all, limit - found);
    for (int i = threadIdx.x; i < give; i += GIVERS) {
      const int64_t rank = found + i;
      const int row = row_of(rank);
      const int64_t before = row == 0 ? 0 : in_lds ? (int64_t)ends[row - 1] : ask[row - 1].end;
      a.table.p[(int64_t)row * a.table.ld + ask[row].begin + (rank - before)] = ids[i];
      a.refs[ids[i]] = 1;
    }
    found += all;
    __syncthreads();
  }
  if (!ALL) return;
  __syncthreads();
  for (int i = threadIdx.x >> 6; i < n; i += GIVE_WAVES) {
    const Ask k = ask[i];
    take_row(a, i, k, k.end == (i > 0 ? ask[i - 1].end : 0) || k.end <= free);
  }
}

__global__ __launch_bounds__(64) void kv_take(ResizeArgs a) {
  const Ask* ask = asks_of(a.ws);
  const int i = blockIdx.x;
  const Ask k = ask[i];
  take_row(a, i, k, k.end == (i > 0 ? ask[i - 1].end : 0) || k.end <= *free_of(a.ws));
}

// ---- copies ---------------------------------------------------------------------------------
// A workgroup for each record, head, and keys or values.
__global__ __launch_bounds__(256) void kv_copy_pages(KvCache c, int G, int vec, const int32_t* copies) {
  const int kv = blockIdx.x & 1, head = (blockIdx.x >> 1) % G, i = (blockIdx.x >> 1) / G;
  const int src = copies[3 * (int64_t)i], dst = copies[3 * (int64_t)i + 1];
  const int tokens = min(copies[3 * (int64_t)i + 2], c.page_size);
  if (src < 0 || src >= c.n_pages || dst < 0 || dst >= c.n_pages || src == dst) return;
  const int eb = c.e4m3 ? 1 : 2;
  unsigned char* base = static_cast<unsigned char*>(kv ? c.v : c.k) + head * c.hs * eb;
  const unsigned char* from = base + src * c.ps * eb;
  unsigned char* to = base + dst * c.ps * eb;
  const int at_once = 256 / vec, piece = threadIdx.x % vec, first = threadIdx.x / vec;
  if (first >= at_once) return;
  for (int64_t t = first; t < tokens; t += at_once) {
    const int64_t at = t * c.ts * eb + piece * 16;
    *GLOBAL_PTR(u32x4, to + at) = *GLOBAL_PTR(const u32x4, from + at);
  }
}

// ---- compaction -----------------------------------------------------------------------------
// A workgroup for each sequence and `planes` of its planes, the heads' keys and values.  A thread
// moves AHEAD pieces of 16 bytes at a time.  As the kept places rise, token d comes from place d or
// a later one: with all loads of a turn before its stores, and turn after turn, no place is
// written before it is read.  A turn holds whole planes if the list is short enough for one;
// otherwise it is some tokens of one plane.
constexpr int AHEAD = 4, MOVERS = 256;
__global__ __launch_bounds__(MOVERS) void kv_compact(CompactArgs a, int vec, int planes) {
  __shared__ int count;
  const int groups = (2 * a.G + planes - 1) / planes;
  const int i = blockIdx.x / groups, plane0 = (blockIdx.x - i * groups) * planes;
  const int plane1 = min(plane0 + planes, 2 * a.G);
  const int cap = table_cap(a.pages_per_seq, a.cache.page_size);
  const int len = clamp_len(a.lens[i], cap);
  const int32_t* kept = a.kept + (int64_t)i * a.kept_ld;
  // the list's first entries are loaded beside its length
  const int own = (int)threadIdx.x < a.most ? kept[threadIdx.x] : 0;
  const int prev = threadIdx.x > 0 && (int)threadIdx.x < a.most ? kept[threadIdx.x - 1] : -1;
  const int given = min(max(a.kept_lens[i], 0), a.most);
  if (threadIdx.x == 0) count = given;
  __syncthreads();
  for (int d = threadIdx.x; d < given; d += MOVERS) {
    const int x = d < MOVERS ? own : kept[d];
    if (x <= (d < MOVERS ? prev : kept[d - 1]) || x >= cap - len) {
      atomicMin(&count, d);
      break;
    }
  }
  __syncthreads();
  const int n = count;
  if (plane0 == 0 && threadIdx.x == 0) a.lens_out[i] = len + n;
  if (n == 0) return;
  const int eb = a.cache.e4m3 ? 1 : 2;
  const int32_t* pages = a.pages + (int64_t)i * a.pages_ld;
  auto place = [&](int t) {
    return token_offset(t, pages[page_entry(t, a.cache.page_size, a.pages_per_seq)], a.cache.n_pages, a.cache.page_size,
                        a.cache.ps, a.cache.ts);
  };
  const int slots = MOVERS / vec, piece = threadIdx.x % vec, first = threadIdx.x / vec;  // of a turn's AHEAD shares
  const int at_once = max(slots * AHEAD / n, 1), tokens = min(n, slots * AHEAD);         // planes and tokens of a turn
  for (int p0 = plane0; p0 < plane1; p0 += at_once)
    for (int d0 = 0; d0 < n; d0 += tokens) {
      u32x4 x[AHEAD];
      unsigned char* to[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const int s = j * slots + first, dp = s / tokens;  // the turn's plane and token
        const int d = d0 + s - dp * tokens, plane = p0 + dp;
        to[j] = nullptr;
        if (first < slots && dp < at_once && plane < plane1 && d < n && kept[d] != d) {
          const int64_t from = place(len + kept[d]), into = place(len + d);
          if (from < 0 || into < 0) continue;
          unsigned char* base = static_cast<unsigned char*>(plane & 1 ? a.cache.v : a.cache.k) +
                                (plane >> 1) * a.cache.hs * eb + piece * 16;
          to[j] = base + into * eb;
          x[j] = *GLOBAL_PTR(const u32x4, base + from * eb);
        }
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < AHEAD; ++j)
        if (to[j]) *GLOBAL_PTR(u32x4, to[j]) = x[j];
    }
}

}  // namespace

hipError_t launch_kv_fork(const ForkArgs& a, hipStream_t s) {
  const int64_t blocks = (int64_t)a.in.n + a.out.n;
  if (blocks == 0) return hipSuccess;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  return launch_k(&kv_fork, dim3((unsigned)blocks), dim3(256), 0, s, a);
}

size_t kv_resize_bytes(int32_t n) { return n > 0 ? ASKS_AT + sizeof(Ask) * (size_t)n : 0; }

constexpr int ONE_LAUNCH = 64, ONE_LAUNCH_WINDOW = 16;
hipError_t launch_kv_resize(const ResizeArgs& a, hipStream_t s) {
  if (a.table.n == 0) return hipSuccess;
  // Few rows are done by the one workgroup's waves, a launch less (of a call's 7 us on the host, 2).  On
  // the device, in a graph, 64 rows that grow take 8.5 us with one launch, 65 take 7.8 with two;
  // under a window, whose pages left behind each wave looks for, 14.4 and 9.2, and 16 rows 7.9.
  if (a.table.n <= (a.win.size > 0 ? ONE_LAUNCH_WINDOW : ONE_LAUNCH)) return launch_k(&kv_give<true>, dim3(1), dim3(GIVERS), 0, s, a);
  const hipError_t e = launch_k(&kv_give<false>, dim3(1), dim3(GIVERS), 0, s, a);
  return e == hipSuccess ? launch_k(&kv_take, dim3((unsigned)a.table.n), dim3(64), 0, s, a) : e;
}

hipError_t launch_kv_copy_pages(const KvCache& c, int32_t G, int32_t D, const int32_t* copies, int32_t n,
                                hipStream_t s) {
  const int64_t blocks = 2 * (int64_t)G * n;
  if (blocks == 0) return hipSuccess;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  return launch_k(&kv_copy_pages, dim3((unsigned)blocks), dim3(256), 0, s, c, G, D / (c.e4m3 ? 16 : 8), copies);
}

hipError_t launch_kv_compact(const CompactArgs& a, hipStream_t s) {
  if (a.n == 0) return hipSuccess;
  // a workgroup for each plane of a long list, for two of a short one, which takes a turn or two.
  // Measured with 1, 2, 4 and all 8 planes, the append of 256 drafts of up to 60 nodes, 4 heads,
  // and the move of their accepted paths: 26.3, 25.1, 27.9 and 29 us
  const int planes = a.most <= 256 ? 2 : 1;
  const int64_t blocks = (int64_t)a.n * (2 * a.G / planes);
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  return launch_k(&kv_compact, dim3((unsigned)blocks), dim3(MOVERS), 0, s, a, a.D / (a.cache.e4m3 ? 16 : 8), planes);
}

}  // namespace ubx
