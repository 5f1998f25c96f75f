// Rows and pages of the paged cache moved as they are (compaction of accepted drafts, page copies), and the page pool:
// counts of the rows that hold each page, pages taken and given back, all on the device.
//
// The moves are bound by memory: bytes in, bytes out, in the widest unit that a plane's tokens are aligned to, with all planes'
// units dealt to all threads at once, since small moves are bound by their dependent trips (path, pages, tokens).  250 trees
// of 64 drafts, NVFP4: 9.7 us (a plane after the other took 25), 16 trees of 8, MXFP8: 7.0 us; 336 page copies of 19 MB:
// 9.3 us, 4.0 TB/s in and out (17.8 a plane after the other).
// The pool's two launches are bound by their dependent trips to memory: one wave a row gives pages back and sees what is
// missing, then one workgroup numbers the missing pages in row order, finds as many free ones in page order, and hands
// them out: 4 and 5 us for 64 rows of 130 pages.  Sums and ranks of whole numbers: no result depends on the order of the atomics.
#include <hip/hip_runtime.h>

#include "drafts.h"

#define MX_DEV __device__ __forceinline__

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 8;        // units on their way in each thread

typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));

// Units of a token in the planes before plane p.
MX_DEV int64_t units_before(const MoveArgs& a, int p) { return p == 0 ? 0 : p == 1 ? a.ends[0] : p == 2 ? a.ends[1] : p == 3 ? a.ends[2] : a.ends[3]; }

MX_DEV int64_t slot_at(const MoveArgs& a, const int32_t* row, int64_t pos) {
  if (pos < 0) return -1;
  const uint32_t p = (uint32_t)pos / (uint32_t)a.page_size;  // start and place in the path: below 2^32
  if (p >= (uint32_t)a.max_pages) return -1;
  const int64_t page = row[p];
  if (page < 0 || page >= a.num_pages) return -1;
  return page * a.page_size + ((uint32_t)pos - p * (uint32_t)a.page_size);
}

// A unit of `unit` bytes at the head of 16; WIDE: all planes' are 16 bytes.
template <bool WIDE>
MX_DEV u32x4_t get_unit(const uint8_t* p, int unit) {
  u32x4_t v = {0, 0, 0, 0};
  if (WIDE || unit == 16) return *(const u32x4_t*)p;
  if (unit == 8) {
    const uint64_t x = *(const uint64_t*)p;
    v[0] = (uint32_t)x;
    v[1] = (uint32_t)(x >> 32);
  } else {
    v[0] = unit == 4 ? *(const uint32_t*)p : unit == 2 ? *(const uint16_t*)p : *p;
  }
  return v;
}
template <bool WIDE>
MX_DEV void put_unit(uint8_t* p, int unit, u32x4_t v) {
  if (WIDE || unit == 16) *(u32x4_t*)p = v;
  else if (unit == 8) *(uint64_t*)p = (uint64_t)v[1] << 32 | v[0];
  else if (unit == 4) *(uint32_t*)p = v[0];
  else if (unit == 2) *(uint16_t*)p = (uint16_t)v[0];
  else *p = (uint8_t)v[0];
}

// blockIdx.x: sequence, blockIdx.y: a stripe of each token's units, those of all planes in a row.  The moved tokens' units
// are dealt to the threads in path order, kBatch each a round, and all of a round are read before any is written.  Where an
// earlier token goes, no later one comes from (the path increases, and is never behind its place), so nothing is read
// that another round has written.
template <bool WIDE>
__global__ __launch_bounds__(kThreads) void compact_kernel(MoveArgs a) {
  __shared__ int64_t from[kThreads], to[kThreads];
  __shared__ int32_t in_wave[kThreads / 64], stop;
  const int t = threadIdx.x, wave = t >> 6;
  for (int b = blockIdx.x; b < a.n_seqs; b += gridDim.x) {
    const int32_t* path = a.path + (int64_t)b * a.ld_path;
    const int32_t* row = a.table + (int64_t)b * a.ld_table;
    const int64_t first = a.start ? a.start[b] : 0;
    int64_t accepted = 0;
    for (int64_t c = 0; c < a.path_cols; c += kThreads) {
      if (t == 0) stop = kThreads;
      __syncthreads();
      const int64_t i = c + t;
      int32_t e = -1;
      if (i < a.path_cols) {
        const int32_t before = i ? path[i - 1] : -1;
        e = path[i];
        if (e <= before) e = -1;
      }
      if (e < 0) atomicMin(&stop, t);
      __syncthreads();
      const int n = stop;
      int64_t src = -1, dst = -1;
      if (t < n && e != i) {
        src = slot_at(a, row, first + e);
        dst = slot_at(a, row, first + i);
      }
      // the moves, in path order and without gaps
      const bool moves = src >= 0 && dst >= 0;
      const uint64_t mine = __ballot(moves);
      if ((t & 63) == 0) in_wave[wave] = __popcll(mine);
      __syncthreads();
      int at = __popcll(mine & ((1ull << (t & 63)) - 1)), total = 0;
      for (int w = 0; w < kThreads / 64; w++) {
        if (w < wave) at += in_wave[w];
        total += in_wave[w];
      }
      if (moves) {
        from[at] = src;
        to[at] = dst;
      }
      __syncthreads();
      const int64_t u0 = units_before(a, 4) * blockIdx.y / gridDim.y;
      const uint32_t units = (uint32_t)(units_before(a, 4) * (blockIdx.y + 1) / gridDim.y - u0), count = units * (uint32_t)total;
      // a thread's unit of a token, and what a step of all threads adds to them
      uint32_t token = t / units, u = t - token * units;
      const uint32_t step_token = kThreads / units, step_u = kThreads - step_token * units;
      const auto step = [&](uint32_t& token, uint32_t& u) {
        token += step_token;
        u += step_u;
        if (u >= units) u -= units, token++;
      };
      const auto place = [&](const int64_t* slots, uint32_t token, uint32_t u, int& unit) {
        int64_t at = u0 + u;
        const int p = (at >= units_before(a, 1)) + (at >= units_before(a, 2)) + (at >= units_before(a, 3));
        at -= units_before(a, p);
        unit = a.plane[p].unit;
        return a.plane[p].base + slots[token] * a.plane[p].row + at * unit;
      };
      for (uint32_t first = 0; first < count; first += kBatch * kThreads) {
        u32x4_t v[kBatch];
        uint32_t to_token = token, to_u = u;
        int unit;
#pragma unroll
        for (int k = 0; k < kBatch; k++) {
          if (first + k * kThreads + t < count) v[k] = get_unit<WIDE>(place(from, token, u, unit), unit);
          step(token, u);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kBatch; k++) {
          if (first + k * kThreads + t < count) {
            uint8_t* const at = place(to, to_token, to_u, unit);
            put_unit<WIDE>(at, unit, v[k]);
          }
          step(to_token, to_u);
        }
      }
      accepted += n;
      __syncthreads();
      if (n < kThreads) break;
    }
    if (a.lengths && blockIdx.y == 0 && t == 0) a.lengths[b] = (int32_t)(first + accepted);
  }
}

struct Stripes {
  int64_t ends[4];  // up to and with each plane
};

// blockIdx.x: pair, blockIdx.y: a stripe of a page's units, kBatch a thread; those of all planes in a row.
template <bool WIDE>
__global__ __launch_bounds__(kThreads) void copy_pages_kernel(MoveArgs a, Stripes stripes) {
  const int64_t* const e = stripes.ends;
  for (int64_t y = blockIdx.y; y < e[3]; y += gridDim.y) {
    const int p = (y >= e[0]) + (y >= e[1]) + (y >= e[2]);
    const BytePlane plane = a.plane[p];
    const int64_t first = p == 0 ? 0 : p == 1 ? e[0] : p == 2 ? e[1] : e[2];
    const int64_t per = plane.row / plane.unit, u = (y - first) * kThreads * kBatch + threadIdx.x;
    for (int i = blockIdx.x; i < a.n; i += gridDim.x) {
      const int64_t src = a.src[i], dst = a.dst[i];
      if (src < 0 || src >= a.num_pages || dst < 0 || dst >= a.num_pages || src == dst) continue;
      const int64_t units = (a.rows ? min(a.rows[i], a.page_size) : a.page_size) * per;
      const uint8_t* from = plane.base + src * a.page_size * plane.row + u * plane.unit;
      uint8_t* to = plane.base + dst * a.page_size * plane.row + u * plane.unit;
      u32x4_t v[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; k++)
        if (u + k * kThreads < units) v[k] = get_unit<WIDE>(from + (int64_t)k * kThreads * plane.unit, plane.unit);
#pragma unroll
      for (int k = 0; k < kBatch; k++)
        if (u + k * kThreads < units) put_unit<WIDE>(to + (int64_t)k * kThreads * plane.unit, plane.unit, v[k]);
    }
  }
}

// ---------------------------------------------------------------------------------------------
// The pool.

// What the first launch found about each row (resize) or pair (fork).
struct Items {
  int32_t *need;    // pages to take
  int32_t *first;   // column of the first of them
  int32_t *from;    // page that the row's last page is a copy of, -1: none; resize: where it is shared
  int32_t *offset;  // pages to take before this item's
  int32_t *list;    // free pages
};

// Gives the row's pages from column `keep` on back, sets these columns to -1, and returns how many pages the row held.
MX_DEV int give_back(const PoolArgs& a, int32_t* row, int64_t keep, int lane) {
  int held = 0;
  bool run = true;
  for (int c = 0; c < a.max_pages; c += 64) {
    const int i = c + lane;
    const int32_t e = i < a.max_pages ? row[i] : -1;
    const uint64_t bad = ~__ballot(e >= 0 && e < a.num_pages);
    const int good = run ? (bad ? __ffsll((unsigned long long)bad) - 1 : 64) : 0;
    held += good;
    run = run && good == 64;
    if (i < a.max_pages && i >= keep) {
      if (lane < good) atomicSub(&a.refs[e], 1);
      if (e != -1) row[i] = -1;
    }
  }
  return held;
}

MX_DEV void resize_row(const PoolArgs& a, const Items& it, int b, int lane) {
  int32_t* row = a.table + (int64_t)b * a.ld_table;
  const int32_t len = a.lengths[b];
  int32_t need = 0, first = 0, from = -1, tail = 0;
  if (len >= 0) {
    const int64_t whole = len / a.page_size;
    tail = len - (int32_t)(whole * a.page_size);
    int64_t want = whole + (tail > 0);
    if (want > a.max_pages) {
      want = a.max_pages;
      tail = 0;
    }
    const int held = give_back(a, row, want, lane);
    if (held < want) {
      need = (int32_t)want - held;
      first = held;
    } else if (tail > 0) {
      first = (int32_t)want - 1;
      from = row[first];
    }
  }
  if (lane == 0) {
    it.need[b] = need;
    it.first[b] = first;
    it.from[b] = from;
    a.copies[b] = -1;
    a.copies[a.n + b] = -1;
    a.copies[2 * (int64_t)a.n + b] = from >= 0 ? tail : 0;
  }
}

MX_DEV void fork_pair(const PoolArgs& a, const Items& it, int i, int lane) {
  const int32_t s = a.src[i], d = a.dst[i], len = a.lengths[i];
  bool good = s >= 0 && s < a.n_rows && d >= 0 && d < a.n_rows && len >= 0;
  if (good) {
    bool clash = false;
    for (int j = lane; j < a.n; j += 64) clash = clash || a.src[j] == d || (j < i && a.dst[j] == d);
    good = !__any(clash);
  }
  int32_t need = 0, first = 0, from = -1, tail = 0;
  if (good) {
    int32_t* row = a.table + (int64_t)d * a.ld_table;
    const int32_t* other = a.table + (int64_t)s * a.ld_table;
    give_back(a, row, 0, lane);
    const int64_t whole = len / a.page_size;
    tail = len - (int32_t)(whole * a.page_size);
    // the pages that the source holds, as far as they are wanted
    for (int64_t c = 0; c < a.max_pages && c <= whole; c += 64) {
      const int64_t k = c + lane;
      const int32_t e = k < a.max_pages && k <= whole ? other[k] : -1;
      const uint64_t bad = ~__ballot(e >= 0 && e < a.num_pages);
      const int run = bad ? __ffsll((unsigned long long)bad) - 1 : 64;
      if (lane < run && k < whole) {
        atomicAdd(&a.refs[e], 1);
        row[k] = e;
      }
      if (whole >= c && whole < c + run && tail > 0) {
        need = 1;
        first = (int32_t)whole;
        from = __shfl(e, (int)(whole - c));
      }
      if (run < 64) break;
    }
  }
  if (lane == 0) {
    it.need[i] = need;
    it.first[i] = first;
    it.from[i] = from;
    a.copies[i] = -1;
    a.copies[a.n + i] = -1;
    a.copies[2 * (int64_t)a.n + i] = from >= 0 ? tail : 0;
  }
}

template <bool FORK>
__global__ __launch_bounds__(kThreads) void pool_rows_kernel(PoolArgs a, Items it) {
  const int lane = threadIdx.x & 63, waves = gridDim.x * (kThreads / 64);
  for (int i = blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6); i < a.n; i += waves) {
    if (FORK)
      fork_pair(a, it, i, lane);
    else
      resize_row(a, it, i, lane);
  }
}

constexpr int kPool = 1024;     // threads of the second launch
constexpr int kPoolScan = 8;    // counts of a thread at a time

// The sum of v over the threads before this one, and over all of them; part: kPool / 64 values.
MX_DEV int32_t scan(int32_t v, int32_t* part, int32_t& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int32_t s = v;
#pragma unroll
  for (int h = 1; h < 64; h <<= 1) {
    const int32_t o = __shfl_up(s, h);
    if (lane >= h) s += o;
  }
  __syncthreads();  // the values of the scan before have been read
  if (lane == 63) part[wave] = s;
  __syncthreads();
  int32_t before = 0;
  total = 0;
  for (int w = 0; w < kPool / 64; w++) {
    if (w < wave) before += part[w];
    total += part[w];
  }
  return before + s - v;
}

template <bool FORK>
__global__ __launch_bounds__(kPool) void pool_take_kernel(PoolArgs a, Items it) {
  __shared__ int32_t part[kPool / 64], kept;
  const int t = threadIdx.x;
  int32_t wanted = 0, all;
  for (int c = 0; c < a.n; c += kPool) {
    const int i = c + t;
    int32_t need = 0;
    if (i < a.n) {
      need = it.need[i];
      if (!FORK && it.from[i] >= 0) {
        if (a.refs[it.from[i]] > 1) {
          need = 1;
          it.need[i] = 1;
        } else {
          it.from[i] = -1;
          a.copies[2 * (int64_t)a.n + i] = 0;
        }
      }
    }
    const int32_t before = scan(need, part, all);
    if (i < a.n) it.offset[i] = wanted + before;
    wanted += all;
  }
  // the first `wanted` free pages
  int32_t found = 0;
  for (int64_t c = 0; c < a.num_pages && found < wanted; c += kPool * kPoolScan) {
    const int64_t p0 = c + t * kPoolScan;
    uint32_t free_bits = 0;
#pragma unroll
    for (int k = 0; k < kPoolScan; k++)
      if (p0 + k < a.num_pages && a.refs[p0 + k] <= 0) free_bits |= 1u << k;
    int32_t at = found + scan(__popc(free_bits), part, all);
    for (int k = 0; k < kPoolScan; k++)
      if (free_bits >> k & 1) {
        if (at < wanted) it.list[at] = (int32_t)(p0 + k);
        at++;
      }
    found += all;
  }
  if (found > wanted) found = wanted;
  if (t == 0) kept = 0;
  __syncthreads();
  // hand them out: page r of the list goes to the last item whose offset is at most r
  const auto item_of = [&](int32_t r) {
    int lo = 0, hi = a.n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (it.offset[mid] <= r) lo = mid; else hi = mid - 1;
    }
    return lo;
  };
  for (int32_t r = t; r < wanted; r += kPool) {
    const int lo = item_of(r);
    const int32_t page = r < found ? it.list[r] : -1, from = it.from[lo];
    const int32_t row = FORK ? a.dst[lo] : lo;
    int32_t* entry = a.table + (int64_t)row * a.ld_table + it.first[lo] + (r - it.offset[lo]);
    if (page >= 0) {
      a.refs[page] = 1;
      *entry = page;
      if (from >= 0) {
        if (!FORK) atomicSub(&a.refs[from], 1);
        a.copies[lo] = from;
        a.copies[a.n + lo] = page;
      }
    } else if (from >= 0) {
      a.copies[2 * (int64_t)a.n + lo] = 0;
      if (!FORK) atomicSub(&a.refs[from], 1);  // (fork: its entry is -1 already)
    } else {
      *entry = -1;
    }
  }
  // Rows whose shared page could not be replaced have let go of it, so that none writes where another reads.  A page that
  // nobody holds any more stays with the last of its rows: the highest, whatever the order of the atomics.
  if (!FORK && found < wanted) {
    const auto refs_of = [&](int32_t page) { return __hip_atomic_load(&a.refs[page], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
    __threadfence();
    __syncthreads();
    for (int32_t r = found + t; r < wanted; r += kPool) {
      const int lo = item_of(r);
      const int32_t from = it.from[lo];
      if (from >= 0 && refs_of(from) <= 0) atomicMin(&a.refs[from], -1 - lo);
    }
    __threadfence();
    __syncthreads();
    for (int32_t r = found + t; r < wanted; r += kPool) {
      const int lo = item_of(r);
      const int32_t from = it.from[lo];
      if (from < 0) continue;
      if (refs_of(from) == -1 - lo) {
        atomicExch(&a.refs[from], 1);
        atomicAdd(&kept, 1);
      } else {
        a.table[(int64_t)lo * a.ld_table + it.first[lo]] = -1;
      }
    }
    __syncthreads();
  }
  if (t == 0) *a.missing = wanted - found - kept;
}

int status() { return hipGetLastError() == hipSuccess ? MXFP4_OK : MXFP4_ERR_DEVICE; }

bool wide(const MoveArgs& a) {
  for (int p = 0; p < a.planes; p++)
    if (a.plane[p].unit != 16) return false;
  return true;
}

}  // namespace

int launch_compact(const MoveArgs& a, hipStream_t stream) {
  // stripes that take one round if the whole path moves, as long as the sequences leave room for more workgroups
  const int64_t units = a.ends[3], round = kThreads * kBatch, moves = min(a.path_cols, kThreads);
  const int64_t n = max(min(min((units * moves + round - 1) / round, units), int64_t(4096 / a.n_seqs)), int64_t(1));
  const dim3 grid((unsigned)min(a.n_seqs, 65536), (unsigned)n);
  if (wide(a))
    hipLaunchKernelGGL(compact_kernel<true>, grid, dim3(kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL(compact_kernel<false>, grid, dim3(kThreads), 0, stream, a);
  return status();
}

int launch_copy_pages(const MoveArgs& a, hipStream_t stream) {
  Stripes stripes;
  int64_t n = 0;
  for (int p = 0; p < 4; p++) {
    if (p < a.planes) n += ((int64_t)a.page_size * (a.plane[p].row / a.plane[p].unit) + kThreads * kBatch - 1) / (kThreads * kBatch);
    stripes.ends[p] = n;
  }
  const dim3 grid((unsigned)min(a.n, 65536), (unsigned)min(n, int64_t(65535)));
  if (wide(a))
    hipLaunchKernelGGL(copy_pages_kernel<true>, grid, dim3(kThreads), 0, stream, a, stripes);
  else
    hipLaunchKernelGGL(copy_pages_kernel<false>, grid, dim3(kThreads), 0, stream, a, stripes);
  return status();
}

int launch_pool(bool fork, const PoolArgs& a, const PoolWs& w, uint8_t* ws, hipStream_t stream) {
  const Items it = {(int32_t*)(ws + w.need), (int32_t*)(ws + w.first), (int32_t*)(ws + w.from), (int32_t*)(ws + w.offset),
                    (int32_t*)(ws + w.list)};
  if (a.n > 0) {
    const int n = (a.n + kThreads / 64 - 1) / (kThreads / 64);
    const dim3 grid((unsigned)(n < 65536 ? n : 65536));
    if (fork)
      hipLaunchKernelGGL(pool_rows_kernel<true>, grid, dim3(kThreads), 0, stream, a, it);
    else
      hipLaunchKernelGGL(pool_rows_kernel<false>, grid, dim3(kThreads), 0, stream, a, it);
    const int st = status();
    if (st) return st;
  }
  if (fork)
    hipLaunchKernelGGL(pool_take_kernel<true>, dim3(1), dim3(kPool), 0, stream, a, it);
  else
    hipLaunchKernelGGL(pool_take_kernel<false>, dim3(1), dim3(kPool), 0, stream, a, it);
  return status();
}
