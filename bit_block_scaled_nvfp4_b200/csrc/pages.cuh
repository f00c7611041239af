// Page pool: allocation, forking, freeing and compaction of a paged cache's pages, and the copying
// of page contents (rules in include/qk4v8.h). The state is refs[page] alone, the number of
// sequences holding each page; free pages are taken lowest number first, so every result is a
// function of the state and the arguments, whatever order the threads run in.
//
// The planning steps need one consistent view of refs and lens, so each is one CTA: a pass over
// refs (4 bytes a page, 128 pages a warp-wide 16-byte load) and block scans; a fork's table rows are
// checked and copied by that CTA too, so its time grows with forks times the table's width. Page contents and the
// tables of freed and compacted sequences are spread over the device.
//
// Measured as graphs: 64 sequences of 200 to 4000 tokens freed and forked again, their last pages copied:
// 17 us, three launches and the one CTA's passes (the bytes alone: 1.3 us); 48 sequences of 500 to 5000 tokens
// compacted among three times as many pages, contents of 8 heads copied: 55 us, four launches, of which the copies'
// bytes are 32 (52 us before the rows were checked in a launch of their own).
#pragma once
#include "ptx.cuh"

namespace qk4v8 {

constexpr int kPoolThreads = 1024;

__host__ __device__ constexpr int pool_pages_of(int n) { return (n >> 6) + ((n & 63) != 0); }

// Exclusive prefix sum of v over the CTA; `total` gets the sum. `sh`: 33 ints of shared memory.
__device__ __forceinline__ int block_scan(int v, int* sh, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();                                     // the last call's readers are done with sh
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int t = lane < kPoolThreads / 32 ? sh[lane] : 0, s = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    sh[lane] = s - t;
    if (lane == 31) sh[32] = s;
  }
  __syncthreads();
  total = sh[32];
  return sh[warp] + x - v;
}

// Four refs from page p on; pages past the end read as `past`.
__device__ __forceinline__ int4 load_refs(const int32_t* refs, int P, int p, int past) {
  if (p + 3 < P && (reinterpret_cast<uintptr_t>(refs) & 15) == 0) return *reinterpret_cast<const int4*>(refs + p);
  return make_int4(p < P ? refs[p] : past, p + 1 < P ? refs[p + 1] : past, p + 2 < P ? refs[p + 2] : past,
                   p + 3 < P ? refs[p + 3] : past);
}

// The lowest `want` pages with refs <= 0, ascending, into ids[]; returns how many there were
// (stops at `want`). ids is visible to the whole CTA on return.
__device__ __forceinline__ int find_free(const int32_t* refs, int P, int want, int32_t* ids, int* sh) {
  int found = 0;
  for (int base = 0; base < P && found < want; base += kPoolThreads * 4) {
    const int p = base + threadIdx.x * 4;
    const int4 r = p < P ? load_refs(refs, P, p, 1) : make_int4(1, 1, 1, 1);
    const int f0 = r.x <= 0, f1 = r.y <= 0, f2 = r.z <= 0, f3 = r.w <= 0;
    int total, at = found + block_scan(f0 + f1 + f2 + f3, sh, total);
    if (f0) { if (at < want) ids[at] = p; ++at; }
    if (f1) { if (at < want) ids[at] = p + 1; ++at; }
    if (f2) { if (at < want) ids[at] = p + 2; ++at; }
    if (f3) { if (at < want) ids[at] = p + 3; ++at; }
    found += total;
  }
  __syncthreads();
  return min(found, want);
}

// ws: off [S + 1], ids [P]
__global__ void __launch_bounds__(kPoolThreads)
pages_alloc_kernel(int32_t* refs, int P, int32_t* table, int S, int max_pages,
                   const int32_t* lens, const int32_t* new_lens, int32_t* off, int32_t* ids) {
  __shared__ int sh[33];
  long long want = 0;
  bool bad = false;
  for (int s0 = 0; s0 < S; s0 += kPoolThreads) {
    const int s = s0 + threadIdx.x;
    int need = 0;
    if (s < S) {
      const int n0 = lens[s], n1 = new_lens[s];
      if (n0 < 0 || n1 < n0 || pool_pages_of(n1) > max_pages) bad = true;
      else need = pool_pages_of(n1) - pool_pages_of(n0);
      if (!bad && n1 > n0 && (n0 & 63) != 0) {           // tokens will be stored into its last page: it has to be its own
        const int id = table[static_cast<int64_t>(s) * max_pages + (n0 >> 6)];
        if (id >= 0 && id < P && refs[id] > 1) bad = true;
      }
    }
    // 2^20 pages more for one sequence are refused as well: 1024 of them would pass 32 bits
    if (need > P || need >= 1 << 20) { bad = true; need = 0; }
    if (__syncthreads_or(bad)) { bad = true; break; }
    int total;
    const int at = block_scan(need, sh, total);
    if (s < S) off[s] = static_cast<int>(want) + at;
    want += total;
    if (want > P) { bad = true; break; }
  }
  if (!bad && find_free(refs, P, static_cast<int>(want), ids, sh) < want) bad = true;
  if (bad) {
    if (threadIdx.x == 0) flag_error(kStatusBounds);
    return;
  }
  for (int k = threadIdx.x; k < want; k += kPoolThreads) {
    int lo = 0, hi = S - 1;                            // the last s with off[s] <= k
    while (lo < hi) {
      const int m = (lo + hi + 1) >> 1;
      if (off[m] <= k) lo = m; else hi = m - 1;
    }
    table[static_cast<int64_t>(lo) * max_pages + pool_pages_of(lens[lo]) + k - off[lo]] = ids[k];
    refs[ids[k]] = 1;
  }
}

// ws: claim [S], ids [P]
__global__ void __launch_bounds__(kPoolThreads)
pages_fork_kernel(int32_t* refs, int P, int32_t* table, int S, int max_pages, int32_t* lens,
                  const int32_t* src, const int32_t* dst, int n, int32_t* move_src,
                  int32_t* move_dst, int32_t* seq_src, int32_t* seq_dst, int32_t* claim,
                  int32_t* ids) {
  __shared__ int sh[33];
  bool bad = false;
  for (int i = threadIdx.x; i < n; i += kPoolThreads) {
    const int s = src[i], d = dst[i];
    if (s < 0 || s >= S || d < 0 || d >= S || s == d || lens[d] != 0 || lens[s] < 0 ||
        pool_pages_of(lens[s]) > max_pages)
      bad = true;
    else
      claim[d] = n;
  }
  bad = __syncthreads_or(bad);
  if (!bad) {                                          // each dst belongs to its lowest pair
    for (int i = threadIdx.x; i < n; i += kPoolThreads) atomicMin(&claim[dst[i]], i);
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPoolThreads) bad |= claim[dst[i]] != i;
    bad = __syncthreads_or(bad);
  }
  // pages that are not full, in the order of the pairs
  int want = 0;
  for (int i0 = 0; i0 < n && !bad; i0 += kPoolThreads) {
    const int i = i0 + threadIdx.x;
    const int part = i < n && (lens[src[i]] & 63) != 0;
    int total;
    const int at = want + block_scan(part, sh, total);
    if (i < n) move_dst[i] = part ? at : -1;            // rank for now
    want += total;
  }
  if (!bad && find_free(refs, P, want, ids, sh) < want) bad = true;
  // every page that is to be shared or copied has to exist and be held
  for (int64_t k = threadIdx.x; k < static_cast<int64_t>(n) * max_pages && !bad; k += kPoolThreads) {
    const int i = static_cast<int>(k / max_pages), p = static_cast<int>(k % max_pages);
    if (p >= pool_pages_of(lens[src[i]])) continue;
    const int id = table[static_cast<int64_t>(src[i]) * max_pages + p];
    if (id < 0 || id >= P || refs[id] <= 0) bad = true;
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    for (int i = threadIdx.x; i < n; i += kPoolThreads)
      move_src[i] = move_dst[i] = seq_src[i] = seq_dst[i] = -1;
    if (threadIdx.x == 0) flag_error(kStatusBounds);
    return;
  }
  for (int64_t k = threadIdx.x; k < static_cast<int64_t>(n) * max_pages; k += kPoolThreads) {
    const int i = static_cast<int>(k / max_pages), p = static_cast<int>(k % max_pages);
    const int64_t from = static_cast<int64_t>(src[i]) * max_pages, to = static_cast<int64_t>(dst[i]) * max_pages;
    if (p >= lens[src[i]] >> 6) continue;
    const int id = table[from + p];
    table[to + p] = id;
    atomicAdd(&refs[id], 1);
  }
  for (int i = threadIdx.x; i < n; i += kPoolThreads) {
    const int len = lens[src[i]], full = len >> 6, rank = move_dst[i];
    move_src[i] = rank < 0 ? -1 : table[static_cast<int64_t>(src[i]) * max_pages + full];
    move_dst[i] = rank < 0 ? -1 : ids[rank];
    seq_src[i] = src[i];
    seq_dst[i] = dst[i];
    if (rank >= 0) {
      table[static_cast<int64_t>(dst[i]) * max_pages + full] = ids[rank];
      refs[ids[rank]] = 1;
    }
  }
  __syncthreads();                                     // every pair has read its source's length
  for (int i = threadIdx.x; i < n; i += kPoolThreads) claim[dst[i]] = lens[src[i]];
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPoolThreads) lens[dst[i]] = claim[dst[i]];
}

// One CTA per listed sequence. Taking the length out by an exchange makes a sequence that is
// named twice empty for the second one.
__global__ void __launch_bounds__(128)
pages_free_kernel(int32_t* refs, int P, int32_t* table, int S, int max_pages, int32_t* lens,
                  const int32_t* seqs) {
  __shared__ int len_sh;
  const int s = seqs[blockIdx.x];
  if (s < 0 || s >= S) {
    if (threadIdx.x == 0) flag_error(kStatusBounds);
    return;
  }
  if (threadIdx.x == 0) len_sh = atomicExch(&lens[s], 0);
  __syncthreads();
  const int len = len_sh;
  if (len < 0 || pool_pages_of(len) > max_pages) {
    if (threadIdx.x == 0) flag_error(kStatusBounds);
    if (len < 0) return;
  }
  const int np = min(pool_pages_of(len), max_pages);
  for (int p = threadIdx.x; p < np; p += blockDim.x) {
    const int64_t e = static_cast<int64_t>(s) * max_pages + p;
    const int id = table[e];
    table[e] = -1;
    if (id < 0 || id >= P) flag_error(kStatusBounds);
    else if (atomicSub(&refs[id], 1) <= 0) {
      atomicAdd(&refs[id], 1);
      flag_error(kStatusBounds);
    }
  }
}

// Whether each sequence's length fits its row and its pages exist and are held, for the compaction that
// follows: bad [S]. One CTA per sequence.
__global__ void __launch_bounds__(128)
pages_check_kernel(const int32_t* refs, int P, const int32_t* table, int max_pages, const int32_t* lens,
                   int32_t* bad) {
  const int s = blockIdx.x, len = lens[s];
  bool wrong = len < 0 || pool_pages_of(len) > max_pages;
  const int np = wrong ? 0 : pool_pages_of(len);
  for (int p = threadIdx.x; p < np; p += blockDim.x) {
    const int id = table[static_cast<int64_t>(s) * max_pages + p];
    if (id < 0 || id >= P || refs[id] <= 0) wrong = true;
  }
  wrong = __syncthreads_or(wrong);
  if (threadIdx.x == 0) bad[s] = wrong;
}

// ws: n_live [1] (-1: refused), bad [S], holes [P], map [P]. move_src / move_dst have P / 2 + 1 entries: a move fills a
// hole, so there are no more moves than live pages and no more than holes.
__global__ void __launch_bounds__(kPoolThreads)
pages_compact_kernel(int32_t* refs, int P, int S, int32_t* move_src, int32_t* move_dst, int32_t* move_count,
                     int32_t* n_live_out, const int32_t* bad, int32_t* holes, int32_t* map) {
  __shared__ int sh[33];
  bool wrong = false;
  for (int s = threadIdx.x; s < S; s += kPoolThreads) wrong |= bad[s] != 0;
  if (__syncthreads_or(wrong)) {
    for (int i = threadIdx.x; i < P / 2 + 1; i += kPoolThreads) move_src[i] = move_dst[i] = -1;
    if (threadIdx.x == 0) {
      *move_count = 0;
      *n_live_out = -1;
      flag_error(kStatusBounds);
    }
    return;
  }
  int live = 0;
  for (int base = 0; base < P; base += kPoolThreads * 4) {
    const int p = base + threadIdx.x * 4;
    if (p < P) {
      const int4 r = load_refs(refs, P, p, 0);
      live += (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0);
    }
  }
  int n_live;
  block_scan(live, sh, n_live);
  // holes before n_live (free pages, ascending)
  const int n_holes = find_free(refs, n_live, n_live, holes, sh);
  // live pages from n_live on, ascending: as many as there are holes
  int at0 = 0;
  for (int base = n_live & ~3; base < P; base += kPoolThreads * 4) {
    const int p = base + threadIdx.x * 4;
    const int4 r = p < P ? load_refs(refs, P, p, 0) : make_int4(0, 0, 0, 0);
    const int rv[4] = {r.x, r.y, r.z, r.w};
    int mine = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) mine += p + k >= n_live && rv[k] > 0;
    int total, at = at0 + block_scan(mine, sh, total);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (p + k < n_live || p + k >= P) continue;
      map[p + k] = -1;
      if (rv[k] <= 0) continue;
      const int to = holes[at];
      move_src[at] = p + k;
      move_dst[at] = to;
      map[p + k] = to;
      refs[to] = rv[k];
      refs[p + k] = 0;
      ++at;
    }
    at0 += total;
  }
  for (int i = n_holes + threadIdx.x; i < P / 2 + 1; i += kPoolThreads) move_src[i] = move_dst[i] = -1;
  if (threadIdx.x == 0) {
    *move_count = n_holes;
    *n_live_out = n_live;
  }
}

// Page-table entries of moved pages (all checked before anything moved). One CTA per sequence.
__global__ void __launch_bounds__(128)
pages_remap_kernel(int P, int32_t* table, int max_pages, const int32_t* lens, const int32_t* n_live,
                   const int32_t* map) {
  const int s = blockIdx.x, live = *n_live;
  if (live < 0) return;
  const int np = min(pool_pages_of(lens[s]), max_pages);
  for (int p = threadIdx.x; p < np; p += blockDim.x) {
    const int64_t e = static_cast<int64_t>(s) * max_pages + p;
    const int id = table[e];
    if (id >= live && id < P) table[e] = map[id];
  }
}

// ---------------------------------------------------------------------------------------
// Page contents. A page of all arrays together is a run of 16-byte words; a CTA copies 1024
// words of it (four loads in flight a thread) and walks over the moves.
// ---------------------------------------------------------------------------------------
constexpr int kMaxPageArrays = 8;
struct PageCopyArgs {
  uint4* base[kMaxPageArrays];
  int64_t end[kMaxPageArrays];     // words of a page up to and with this array
  int64_t words[kMaxPageArrays];   // words of a page of this array
  int32_t n_arrays, num_pages, n;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* count;
};

__global__ void __launch_bounds__(256) pages_copy_kernel(PageCopyArgs a) {
  const int64_t total = a.end[a.n_arrays - 1];
  int n = a.n;
  if (a.count != nullptr) n = min(n, max(*a.count, 0));
  // where this thread's words lie: the same in every page
  uint4* base[4];
  int64_t stride[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 1024 + k * 256 + threadIdx.x;
    base[k] = nullptr;
    stride[k] = 0;
    if (w < total) {
      int i = 0;
      while (w >= a.end[i]) ++i;
      base[k] = a.base[i] + (w - (a.end[i] - a.words[i]));
      stride[k] = a.words[i];
    }
  }
  for (int m = blockIdx.y; m < n; m += gridDim.y) {
    const int s = a.src[m], d = a.dst[m];
    if (s == -1 && d == -1) continue;
    if (s < 0 || s >= a.num_pages || d < 0 || d >= a.num_pages) {
      if (threadIdx.x == 0) flag_error(kStatusBounds);
      continue;
    }
    uint4 u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (base[k] != nullptr) u[k] = base[k][s * stride[k]];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (base[k] != nullptr) base[k][d * stride[k]] = u[k];
  }
}

}  // namespace qk4v8
