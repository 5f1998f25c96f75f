// Rows and pages of the paged cache moved as they are (compaction of accepted drafts, page copies), and the page pool:
// counts of the rows that hold each page, pages taken and given back, all on the device.
//
// The moves are bound by memory: bytes in, bytes out, in the widest unit that a plane's tokens are aligned to.
// The pool's two launches are bound by their dependent trips to memory: one wave a row gives pages back and sees what is
// missing, then one workgroup numbers the missing pages in row order, finds as many free ones in page order, and hands
// them out.  Sums and ranks of whole numbers: no result depends on the order of the atomics.
#include <hip/hip_runtime.h>

#include "drafts.h"

#define MX_DEV __device__ __forceinline__

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 8;        // units on their way in each thread

typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));

// A unit of 1 to 16 bytes.
template <typename F>
MX_DEV void with_unit(int unit, F f) {
  if (unit == 16) f(u32x4_t{});
  else if (unit == 8) f((uint64_t)0);
  else if (unit == 4) f((uint32_t)0);
  else if (unit == 2) f((uint16_t)0);
  else f((uint8_t)0);
}

MX_DEV int64_t slot_at(const MoveArgs& a, const int32_t* row, int64_t pos) {
  if (pos < 0) return -1;
  const int64_t p = pos / a.page_size;
  if (p >= a.max_pages) return -1;
  const int64_t page = row[p];
  if (page < 0 || page >= a.num_pages) return -1;
  return page * a.page_size + (pos - p * a.page_size);
}

// blockIdx.x: sequence, blockIdx.y: a stripe of each token's units.  A thread owns its units of all moved tokens and goes
// through them in path order: the path increases, so a token's source never lies where an earlier token went, and
// each batch is read before it is written.
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
      for (int p = 0; p < a.planes; p++) {
        with_unit(a.plane[p].unit, [&](auto zero) {
          using U = decltype(zero);
          const int64_t units = a.plane[p].row / (int)sizeof(U);
          for (int64_t u = (int64_t)blockIdx.y * kThreads + t; u < units; u += (int64_t)gridDim.y * kThreads) {
            U* base = (U*)a.plane[p].base + u;
            for (int j = 0; j < total; j += kBatch) {
              U v[kBatch];
#pragma unroll
              for (int k = 0; k < kBatch; k++)
                if (j + k < total) v[k] = base[from[j + k] * units];
#pragma unroll
              for (int k = 0; k < kBatch; k++)
                if (j + k < total) base[to[j + k] * units] = v[k];
            }
          }
        });
      }
      accepted += n;
      __syncthreads();
      if (n < kThreads) break;
    }
    if (a.lengths && blockIdx.y == 0 && t == 0) a.lengths[b] = (int32_t)(first + accepted);
  }
}

// blockIdx.x: pair, blockIdx.y: a stripe of the pages' units.
__global__ __launch_bounds__(kThreads) void copy_pages_kernel(MoveArgs a) {
  for (int i = blockIdx.x; i < a.n; i += gridDim.x) {
    const int64_t src = a.src[i], dst = a.dst[i];
    if (src < 0 || src >= a.num_pages || dst < 0 || dst >= a.num_pages || src == dst) continue;
    const int64_t rows = a.rows ? min(a.rows[i], a.page_size) : a.page_size;
    for (int p = 0; p < a.planes; p++) {
      with_unit(a.plane[p].unit, [&](auto zero) {
        using U = decltype(zero);
        const int64_t per = a.plane[p].row / (int)sizeof(U), units = rows * per, page = a.page_size * per;
        const U* from = (const U*)a.plane[p].base + src * page;
        U* to = (U*)a.plane[p].base + dst * page;
        const int64_t step = (int64_t)gridDim.y * kThreads;
        for (int64_t u = (int64_t)blockIdx.y * kThreads + threadIdx.x; u < units; u += kBatch * step) {
          U v[kBatch];
#pragma unroll
          for (int k = 0; k < kBatch; k++)
            if (u + k * step < units) v[k] = from[u + k * step];
#pragma unroll
          for (int k = 0; k < kBatch; k++)
            if (u + k * step < units) to[u + k * step] = v[k];
        }
      });
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
  __shared__ int32_t part[kPool / 64];
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
  if (t == 0) *a.missing = wanted - found;
  __syncthreads();
  // hand them out: page r of the list goes to the last item whose offset is at most r
  for (int32_t r = t; r < wanted; r += kPool) {
    int lo = 0, hi = a.n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (it.offset[mid] <= r) lo = mid; else hi = mid - 1;
    }
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
      a.copies[2 * (int64_t)a.n + lo] = 0;  // resize: the shared page stays; fork: its entry is -1 already
    } else {
      *entry = -1;
    }
  }
}

int status() { return hipGetLastError() == hipSuccess ? MXFP4_OK : MXFP4_ERR_DEVICE; }

// Workgroups along each token or page: enough of them for the plane with the most units, at most `most`.
unsigned stripes(const MoveArgs& a, int64_t tokens, int64_t most) {
  int64_t units = 1;
  for (int p = 0; p < a.planes; p++) units = max(units, tokens * (a.plane[p].row / a.plane[p].unit));
  const int64_t n = (units + kThreads - 1) / kThreads;
  return (unsigned)(n < most ? n : most);
}

}  // namespace

int launch_compact(const MoveArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)min(a.n_seqs, 65536), stripes(a, 1, 64));
  hipLaunchKernelGGL(compact_kernel, grid, dim3(kThreads), 0, stream, a);
  return status();
}

int launch_copy_pages(const MoveArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)min(a.n, 65536), stripes(a, a.page_size, 16));
  hipLaunchKernelGGL(copy_pages_kernel, grid, dim3(kThreads), 0, stream, a);
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
