// ws_kv_pages.cu -- the upkeep of a paged key-value cache on the device, with
// nothing read back: tokens' rows into their pages; rows of the table grown,
// shortened and ended; rows forked; the cache brought together at its low end.
//
// A page is free where its reference count is 0.  Which pages a call takes is a
// function of what it finds, whatever the order of its threads: the lowest free
// ones, in the order of the rows (or pairs) that need them.  One CTA decides
// that, with its block's sums (k_pages_resize, k_pages_fork, k_pages_compact);
// the pages' contents, and what the table's other rows need, follow in a second
// kernel over the whole device (k_pages_move).
//
// Bound by latency: the plan reads every count (four bytes a page) through one
// SM, 16 a thread at a time, until it has enough; then by DRAM: the moved pages.  64 rows
// resized, 16384 pages: 9.5 us; 256 rows, 300000 pages: 24.5; 16 rows, 1024 pages: 6.3.  64
// children forked, 28 layers: 31.5 us.  A cache of 2048 pages, 8 layers compacted: the plan 8 us,
// 528 MB read and as much written in 157, 6.7 TB/s, 0.99 of the copy rate.
#include "ws_kv_q4.cuh"
#include "ws_paged.cuh"

#include "wsgemv.h"

namespace ws {

// ---------------------------------------------------------------- rows into pages

struct PageStoreParams {
  const void* k;  // [T] tokens of [nkv][128], strides in elements
  const void* v;
  const int* cu;     // [n + 1] token bounds of the sequences; null: token i is sequence i
  const int* rows;   // [n] table row of each sequence; null: row i
  const int* start;  // [n] slot of its first token, negative: none
  const int* table;
  uint16_t* kp;
  uint16_t* vp;
  long long ks, vs;
  int T, n, n_rows, max_pages, n_pages, ps, nkv;
  int per;  // tokens a warp
  int* err;
};

// The place of token t: slot `at` of the cache's rows of head 0, or -1 (none), -2 (none,
// but there should be one).  No access is made outside the table or the cache,
// whatever the bounds.
__host__ __device__ __forceinline__ long long page_place(const PageStoreParams& a, int t) {
  int i = t;
  long long in = 0;
  if (a.cu) {
    if (a.cu[0] > t) return -1;
    int lo = 0, hi = a.n;  // the last bound at or before t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.cu[mid] <= t) lo = mid; else hi = mid - 1;
    }
    if (lo >= a.n || a.cu[lo + 1] <= t) return -1;
    i = lo;
    in = (long long)t - a.cu[lo];
  }
  if (a.start[i] < 0) return -1;
  const long long slot = a.start[i] + in;
  const int row = a.rows ? a.rows[i] : i;
  if (row < 0 || row >= a.n_rows || slot >= (long long)a.max_pages * a.ps) return -2;
  const int j = (int)slot / a.ps, page = a.table[(size_t)row * a.max_pages + j];
  if (page < 0 || page >= a.n_pages) return -2;
  return (long long)page * a.nkv * a.ps + ((int)slot - j * a.ps);
}

// A warp takes `per` tokens, whose places its lanes find side by side: lanes 0..15 store
// a key row, 16..31 the value row.  56195 tokens x 8 heads in bf16: 72-73 us, 6.3 TB/s,
// 0.94 of the copy rate (78 with four rows in flight a lane); fp32 102, 1.00.
template <int SRC, int DST>
__global__ void __launch_bounds__(128) k_kv_store_paged(const __grid_constant__ PageStoreParams a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, c = (lane & 15) * 8;
  const bool keys = lane < 16;
  const long long t0 = ((long long)blockIdx.x * 4 + (threadIdx.x >> 5)) * a.per;
  if (t0 >= a.T) return;
  const int n = (int)min((long long)a.per, a.T - t0);
  long long place = -1;
  if (lane < n) {
    place = page_place(a, (int)t0 + lane);
    if (place == -2) atomicExch(a.err, kDerrBadSlot);
  }
  constexpr int kBytes = SRC == DT_F32 ? 4 : 2;
  const char* src = static_cast<const char*>(keys ? a.k : a.v) + ((keys ? a.ks : a.vs) * t0 + c) * kBytes;
  const size_t step = (size_t)(keys ? a.ks : a.vs) * kBytes;
  uint16_t* dst = (keys ? a.kp : a.vp) + c;
  // (rows of all tokens in one loop: 18.1 us for 56195 tokens of one head with one for
  // each, 13.8 so)
  int i = 0, h = 0;
#pragma unroll 2
  for (int j = 0; j < n * a.nkv; ++j) {
    const long long at = __shfl_sync(0xffffffffu, place, i);
    const char* s = src + i * step + (size_t)h * kKvDim * kBytes;
    uint16_t* d = dst + (at + (long long)h * a.ps) * kKvDim;
    if (++h == a.nkv) h = 0, ++i;
    if (at < 0) continue;
    if constexpr (SRC == DST) {
      *reinterpret_cast<uint4*>(d) = *reinterpret_cast<const uint4*>(s);
    } else {
      float x[8];
      load8<SRC>(s, x);
      store8<DST>(d, x);
    }
  }
}

// ---------------------------------------------------------------- plans

constexpr int kPlanThreads = 1024;

struct PagesParams {
  int* table;   // [n_rows][max_pages]
  int* refs;    // [n_pages]
  int* tokens;  // [n_rows]
  const int* want;  // resize: [n_rows]
  const int* src;   // fork: [n]
  const int* dst;
  int n, n_rows, max_pages, n_pages, ps;
  unsigned char* k;  // [layers][n_pages] pages
  unsigned char* v;
  int layers;
  long long page_bytes;
  // workspace
  int* head;    // [16]: moves, live pages
  int* claim;   // [n_rows], zero after a call; what lies behind it depends on n_rows
  int4* rec;    // fork: [n] source row, new row, tokens (-1: skipped), fresh page (-1: none)
  int* list;    // [n_pages] free pages, or the pages that move
  int* to;      // [n_pages] compact: where they go
  int* map;     // [n_pages] compact: new number of each page from the live count on
  int* err;
};

__device__ __forceinline__ int pages_of(int tokens, int ps) { return (tokens + ps - 1) / ps; }
__device__ __forceinline__ bool tokens_ok(const PagesParams& a, int n) {
  return n >= 0 && n <= a.max_pages * a.ps;
}

struct BlockSum {
  long long warp[32];
};
// Sum of x over the threads before this one; `total` over all.  Two barriers.
template <typename N>
__device__ __forceinline__ N block_before(N x, N& total, BlockSum& sh) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  N s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const N u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) sh.warp[w] = s;
  __syncthreads();
  N v = (N)sh.warp[lane];
  __syncthreads();
  const N mine = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const N u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  total = __shfl_sync(0xffffffffu, v, 31);
  return __shfl_sync(0xffffffffu, v - mine, w) + s - x;
}

// Bit i: page p + i (of 16, p a multiple of 16) has a count above 0; past the
// last page 0.  The counts are read where the atomics left them.
__device__ __forceinline__ uint32_t live16(const PagesParams& a, int p) {
  uint32_t m = 0;
  if (p + 16 <= a.n_pages) {
    int4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __ldcg(reinterpret_cast<const int4*>(a.refs + p) + i);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m |= (uint32_t)((x[i].x > 0) | (x[i].y > 0) << 1 | (x[i].z > 0) << 2 | (x[i].w > 0) << 3) << 4 * i;
  } else {
    for (int i = 0; p + i < a.n_pages; ++i) m |= (uint32_t)(__ldcg(a.refs + p + i) > 0) << i;
  }
  return m;
}
__device__ __forceinline__ uint32_t in16(const PagesParams& a, int p) {  // bits of pages that exist
  return p + 16 <= a.n_pages ? 0xffffu : p < a.n_pages ? (1u << (a.n_pages - p)) - 1 : 0u;
}

// The lowest `need` free pages to a.list, in rising order; returns how many
// there are of them (all threads).
__device__ __forceinline__ int take_free(const PagesParams& a, int need, BlockSum& sh) {
  int found = 0;
  for (long long base = 0; base < a.n_pages && found < need; base += 16 * kPlanThreads) {
    const long long p = base + 16 * threadIdx.x;
    uint32_t m = p < a.n_pages ? ~live16(a, (int)p) & in16(a, (int)p) : 0u;
    int total;
    int i = found + block_before(__popc(m), total, sh);
    for (; m && i < need; m &= m - 1) a.list[i++] = (int)p + __ffs(m) - 1;
    found += total;
  }
  __syncthreads();
  return min(found, need);
}

// Rows to want[r] tokens (negative: as it is).  What is given back first, by
// all rows, may be taken again.
__global__ void __launch_bounds__(kPlanThreads) k_pages_resize(const __grid_constant__ PagesParams a) {
  __shared__ BlockSum sh;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  pdl_launch_dependents();
  pdl_wait();
  // rows that may change: claim 1.  A row is not shortened to inside a page that
  // others hold too: its next token there would be theirs.
  for (int r = t; r < a.n_rows; r += kPlanThreads) {
    const int w = a.want[r], n = a.tokens[r];
    int ok = 0;
    if (w >= 0) {
      ok = tokens_ok(a, w) && tokens_ok(a, n);
      if (!ok) atomicExch(a.err, kDerrBadSlot);
      else if (w < n && w % a.ps) {
        const int page = a.table[(size_t)r * a.max_pages + w / a.ps];
        if (page >= 0 && page < a.n_pages && a.refs[page] > 1) {
          ok = 0;
          atomicExch(a.err, kDerrPageUse);
        }
      }
    }
    a.claim[r] = ok;
  }
  __syncthreads();
  for (int r = warp; r < a.n_rows; r += kPlanThreads / 32) {
    if (!a.claim[r]) continue;
    const int w = a.want[r], n = a.tokens[r];
    if (w >= n) continue;
    for (int j = pages_of(w, a.ps) + lane; j < pages_of(n, a.ps); j += 32) {
      int* e = a.table + (size_t)r * a.max_pages + j;
      const int page = *e;
      if (page >= 0 && page < a.n_pages) atomicSub(a.refs + page, 1);
      else atomicExch(a.err, kDerrBadSlot);
      *e = -1;
    }
  }
  __syncthreads();
  long long need = 0;  // of the rows before
  for (int r0 = 0; r0 < a.n_rows; r0 += kPlanThreads) {
    const int r = r0 + t;
    int more = 0, w = 0, n = 0;
    const bool ok = r < a.n_rows && a.claim[r];
    if (ok) {
      w = a.want[r];
      n = a.tokens[r];
      more = max(0, pages_of(w, a.ps) - pages_of(n, a.ps));
    }
    long long total;
    const long long before = need + block_before((long long)more, total, sh);
    // the row's first place in the list of free pages, from 1 on
    if (r < a.n_rows) a.claim[r] = more ? (int)min(before, (long long)a.n_pages) + 1 : 0;
    if (ok && !more) a.tokens[r] = w;
    need += total;
  }
  const int found = need ? take_free(a, (int)min(need, (long long)a.n_pages), sh) : 0;
  __syncthreads();
  for (int r = warp; r < a.n_rows; r += kPlanThreads / 32) {
    const int at = a.claim[r] - 1;
    if (at < 0) continue;
    const int w = a.want[r], first = pages_of(a.tokens[r], a.ps), more = pages_of(w, a.ps) - first;
    const bool served = at <= found && more <= found - at;
    if (served) {
      for (int j = lane; j < more; j += 32) {
        const int page = a.list[at + j];
        a.table[(size_t)r * a.max_pages + first + j] = page;
        a.refs[page] = 1;
      }
    } else if (lane == 0) {
      atomicExch(a.err, kDerrNoPage);
    }
    __syncwarp();
    if (lane == 0) {
      if (served) a.tokens[r] = w;
      a.claim[r] = 0;
    }
  }
}

// Which pairs fork, their fresh pages, and the new rows' tokens; the table's rows
// and the pages follow in k_pages_move.
__global__ void __launch_bounds__(kPlanThreads) k_pages_fork(const __grid_constant__ PagesParams a) {
  __shared__ BlockSum sh;
  const int t = threadIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  auto usable = [&](int i) {
    const int s = a.src[i], d = a.dst[i];
    return s >= 0 && s < a.n_rows && d >= 0 && d < a.n_rows && tokens_ok(a, a.tokens[s]) &&
           a.tokens[d] == 0 && s != d;
  };
  // a row named twice goes to the first pair that names it.  (The claims may hold what a call
  // for a cache of fewer rows left there.)
  for (int i = t; i < a.n; i += kPlanThreads) {
    const int d = a.dst[i];
    if (d >= 0 && d < a.n_rows) a.claim[d] = 0;
  }
  __syncthreads();
  for (int i = t; i < a.n; i += kPlanThreads)
    if (usable(i)) atomicMax(a.claim + a.dst[i], a.n - i);
  __syncthreads();
  int need = 0;
  for (int i0 = 0; i0 < a.n; i0 += kPlanThreads) {
    const int i = i0 + t;
    int4 r = make_int4(0, 0, -1, -1);
    if (i < a.n) {
      if (usable(i) && __ldcg(a.claim + a.dst[i]) == a.n - i)
        r = make_int4(a.src[i], a.dst[i], a.tokens[a.src[i]], -1);
      else atomicExch(a.err, kDerrPageUse);
    }
    int total;
    const int more = r.z > 0 && r.z % a.ps != 0;
    const int before = need + block_before(more, total, sh);
    if (more) r.w = before;
    if (i < a.n) a.rec[i] = r;
    need += total;
  }
  const int found = need ? take_free(a, min(need, a.n_pages), sh) : 0;
  __syncthreads();
  for (int i = t; i < a.n; i += kPlanThreads) {
    const int s = a.src[i], d = a.dst[i];
    if (s >= 0 && s < a.n_rows && d >= 0 && d < a.n_rows) a.claim[d] = 0;
    int4 r = a.rec[i];
    if (r.z < 0) continue;
    if (r.w >= found) {
      r.z = -1;
      atomicExch(a.err, kDerrNoPage);
    } else {
      if (r.w >= 0) {
        r.w = a.list[r.w];
        a.refs[r.w] = 1;
      }
      a.tokens[r.y] = r.z;
    }
    a.rec[i] = r;
  }
}

// The live pages at or above their number L and the free ones below it, each in
// rising order: list[i] goes to to[i].
__global__ void __launch_bounds__(kPlanThreads) k_pages_compact(const __grid_constant__ PagesParams a) {
  __shared__ BlockSum sh;
  const int t = threadIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  int live = 0;
  for (long long p = 16 * t; p < a.n_pages; p += 16 * kPlanThreads) live += __popc(live16(a, (int)p));
  int L;
  block_before(live, L, sh);
  int movers = 0, holes = 0;
  for (long long base = 0; base < a.n_pages; base += 16 * kPlanThreads) {
    const long long p = base + 16 * t;
    uint32_t up = 0, down = 0;
    if (p < a.n_pages) {
      const uint32_t m = live16(a, (int)p), in = in16(a, (int)p);
      const uint32_t low = p >= L ? 0u : p + 16 <= L ? 0xffffu : (1u << (L - (int)p)) - 1;
      up = m & ~low;
      down = ~m & in & low;
      for (uint32_t f = ~m & in & ~low; f; f &= f - 1) a.map[p + __ffs(f) - 1] = (int)p + __ffs(f) - 1;
    }
    int total;
    int i = movers + block_before(__popc(up), total, sh);
    for (; up; up &= up - 1) a.list[i++] = (int)p + __ffs(up) - 1;
    movers += total;
    i = holes + block_before(__popc(down), total, sh);
    for (; down; down &= down - 1) a.to[i++] = (int)p + __ffs(down) - 1;
    holes += total;
  }
  __syncthreads();
  for (int i = t; i < movers; i += kPlanThreads) {
    const int p = a.list[i], q = a.to[i];
    a.map[p] = q;
    a.refs[q] = a.refs[p];
    a.refs[p] = 0;
  }
  if (t == 0) a.head[0] = movers, a.head[1] = L;
}

// ---------------------------------------------------------------- the pages themselves

constexpr int kMoveThreads = 256;
constexpr int kMoveVecs = 8;                                  // of 16 bytes a thread
constexpr int kMoveChunk = kMoveThreads * kMoveVecs * 16;     // bytes of a page at a time

__device__ __forceinline__ void move_chunk(const PagesParams& a, int from, int to, int plane, long long at) {
  unsigned char* base = (plane & 1 ? a.v : a.k) + (size_t)(plane >> 1) * a.n_pages * a.page_bytes;
  const uint4* s = reinterpret_cast<const uint4*>(base + (size_t)from * a.page_bytes + at);
  uint4* d = reinterpret_cast<uint4*>(base + (size_t)to * a.page_bytes + at);
  const int n = (int)((a.page_bytes - at < kMoveChunk ? a.page_bytes - at : kMoveChunk) >> 4);
  uint4 x[kMoveVecs];
#pragma unroll
  for (int i = 0; i < kMoveVecs; ++i) {
    const int e = i * kMoveThreads + threadIdx.x;
    if (e < n) x[i] = __ldcs(s + e);
  }
#pragma unroll
  for (int i = 0; i < kMoveVecs; ++i) {
    const int e = i * kMoveThreads + threadIdx.x;
    if (e < n) __stcs(d + e, x[i]);
  }
}

template <bool FORK>
__global__ void __launch_bounds__(kMoveThreads) k_pages_move(const __grid_constant__ PagesParams a) {
  pdl_launch_dependents();
  pdl_wait();
  const long long chunks = (a.page_bytes + kMoveChunk - 1) / kMoveChunk, planes = 2ll * a.layers;
  const long long step = (long long)gridDim.x * kMoveThreads;
  if constexpr (FORK) {
    for (long long x = (long long)blockIdx.x * kMoveThreads + threadIdx.x; x < (long long)a.n * a.max_pages;
         x += step) {
      const int i = (int)(x / a.max_pages), j = (int)(x - (long long)i * a.max_pages);
      const int4 r = a.rec[i];
      if (r.z < 0) continue;
      const int full = r.z / a.ps;
      int* e = a.table + (size_t)r.y * a.max_pages + j;
      if (j < full) {
        const int page = a.table[(size_t)r.x * a.max_pages + j];
        *e = page;
        if (page >= 0 && page < a.n_pages) atomicAdd(a.refs + page, 1);
        else atomicExch(a.err, kDerrBadSlot);
      } else if (j == full && r.w >= 0) {
        *e = r.w;
      }
    }
  } else {
    const int L = a.head[1];
    for (long long x = (long long)blockIdx.x * kMoveThreads + threadIdx.x;
         x < (long long)a.n_rows * a.max_pages; x += step) {
      const int page = a.table[x];
      if (page >= L && page < a.n_pages) a.table[x] = a.map[page];
    }
  }
  const int moves = FORK ? a.n : a.head[0];
  for (long long x = blockIdx.x; x < moves * planes * chunks; x += gridDim.x) {
    const long long y = x / chunks, at = (x - y * chunks) * kMoveChunk;
    const int i = (int)(y / planes), plane = (int)(y - i * planes);
    int from, to;
    if constexpr (FORK) {
      const int4 r = a.rec[i];
      if (r.z < 0 || r.w < 0) continue;
      from = a.table[(size_t)r.x * a.max_pages + r.z / a.ps];
      to = r.w;
      if (from < 0 || from >= a.n_pages) {
        if (threadIdx.x == 0) atomicExch(a.err, kDerrBadSlot);
        continue;
      }
    } else {
      from = a.list[i];
      to = a.to[i];
    }
    move_chunk(a, from, to, plane, at);
  }
}

static size_t pages_workspace(int n_rows, int n_pages) {
  return 64 + ((size_t)n_rows * 4 + 15) / 16 * 16 + (size_t)n_rows * 16 + 3 * (((size_t)n_pages * 4 + 15) / 16 * 16);
}

static ws_status pages_bind(PagesParams& a, void* ws, size_t bytes) {
  if (!paged_table_ok(a.n_rows, a.max_pages, a.n_pages, a.ps)) {
    set_error("pages: n_rows, max_pages and n_pages at least 1, page_size a multiple of 16 to 1024, "
              "max_pages * page_size at most 2^30");
    return WS_ERR_SHAPE;
  }
  const void* al[] = {a.refs, a.k, a.v, ws};
  for (const void* p : al)
    if ((uintptr_t)p & 15u) {
      set_error("pages: refs, pages and workspace must be 16-byte aligned");
      return WS_ERR_ALIGN;
    }
  const size_t need = pages_workspace(a.n_rows, a.n_pages);
  if (bytes < need) {
    set_error("workspace too small: need %zu bytes, got %zu", need, bytes);
    return WS_ERR_ARG;
  }
  unsigned char* p = static_cast<unsigned char*>(ws);
  auto cut = [&](size_t n) {
    void* r = p;
    p += (n + 15) / 16 * 16;
    return r;
  };
  a.head = static_cast<int*>(cut(64));
  a.claim = static_cast<int*>(cut((size_t)a.n_rows * 4));
  a.rec = static_cast<int4*>(cut((size_t)a.n_rows * 16));
  a.list = static_cast<int*>(cut((size_t)a.n_pages * 4));
  a.to = static_cast<int*>(cut((size_t)a.n_pages * 4));
  a.map = static_cast<int*>(cut((size_t)a.n_pages * 4));
  a.err = device_error_ptr();
  if (!a.err) {
    set_error("device error flag unavailable");
    return WS_ERR_CUDA;
  }
  return WS_OK;
}

static bool pages_data_ok(const PagesParams& a) {
  if (a.layers >= 1 && a.layers <= 65535 && a.page_bytes >= 16 && a.page_bytes % 16 == 0 &&
      a.page_bytes <= (1ll << 30))
    return true;
  set_error("pages: layers 1..65535, page_bytes a multiple of 16 to 2^30");
  return false;
}

static ws_status pages_done(cudaError_t e) {
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) return WS_OK;
  set_error("launch failed: %s", cudaGetErrorString(e));
  return WS_ERR_CUDA;
}

// CTAs of k_pages_move: as many as are resident, no more than `most` pieces of work.
static int move_grid(long long most) {
  const long long g = (long long)device_sm_count() * 8;
  return (int)(most < 1 ? 1 : most < g ? most : g);
}

template <int SRC, int DST>
static cudaError_t store_launch(const PageStoreParams& a, cudaStream_t s) {
  return launch_serving(k_kv_store_paged<SRC, DST>, dim3((unsigned)((a.T + 4ll * a.per - 1) / (4 * a.per))), 128, 0,
                        s, a);
}

}  // namespace ws

using namespace ws;

extern "C" {

ws_status ws_kv_store_paged(const void *k, const void *v, int src_dtype, const int32_t *cu_seqlens,
                            const int32_t *rows, const int32_t *start, const int32_t *table,
                            void *k_pages, void *v_pages, int dtype, int T, int n_seqs, int n_rows,
                            int max_pages, int n_pages, int page_size, int n_kv_heads, int head_dim,
                            long long k_stride, long long v_stride, ws_stream_t stream) {
  if (!k || !v || !start || !table || !k_pages || !v_pages) {
    set_error("null argument");
    return WS_ERR_ARG;
  }
  if ((dtype != WS_DTYPE_BF16 && dtype != WS_DTYPE_F16) ||
      (src_dtype != WS_DTYPE_F32 && src_dtype != dtype)) {
    set_error("paged store: pages in bf16 or fp16, k and v in fp32 or the pages' type");
    return WS_ERR_ARG;
  }
  if (T < 1 || T > (1 << 30) || n_seqs < 1 || (!cu_seqlens && T != n_seqs) || head_dim != kKvDim ||
      !paged_shape_ok(n_rows, max_pages, n_pages, page_size, n_kv_heads) ||
      (!rows && n_rows < n_seqs) || k_stride % 8 || v_stride % 8 ||
      k_stride < (long long)n_kv_heads * kKvDim || v_stride < (long long)n_kv_heads * kKvDim) {
    set_error("paged store: T (to 2^30) and n_seqs at least 1 (equal without cu_seqlens, n_seqs at "
              "most n_rows without rows), head_dim %d, page_size a multiple of 16 to 1024, "
              "max_pages * page_size at most 2^30, n_pages * n_kv_heads * page_size below 2^31, "
              "token strides a multiple of 8 and at least the heads' dimensions", kKvDim);
    return WS_ERR_SHAPE;
  }
  if (((uintptr_t)k | (uintptr_t)v | (uintptr_t)k_pages | (uintptr_t)v_pages) & 15u) {
    set_error("paged store: k, v and the pages must be 16-byte aligned");
    return WS_ERR_ALIGN;
  }
  PageStoreParams a = {};
  a.k = k;
  a.v = v;
  a.cu = cu_seqlens;
  a.rows = rows;
  a.start = start;
  a.table = table;
  a.kp = static_cast<uint16_t*>(k_pages);
  a.vp = static_cast<uint16_t*>(v_pages);
  a.ks = k_stride;
  a.vs = v_stride;
  a.T = T;
  a.n = n_seqs;
  a.n_rows = n_rows;
  a.max_pages = max_pages;
  a.n_pages = n_pages;
  a.ps = page_size;
  a.nkv = n_kv_heads;
  // 8 rows of keys and of values a warp, one token's where that leaves SMs idle
  a.per = (long long)T * n_kv_heads > 16384 && n_kv_heads < 8 ? 8 / n_kv_heads : 1;
  a.err = device_error_ptr();
  if (!a.err) {
    set_error("device error flag unavailable");
    return WS_ERR_CUDA;
  }
  const cudaStream_t s = (cudaStream_t)stream;
  if (dtype == WS_DTYPE_F16)
    return pages_done(src_dtype == WS_DTYPE_F32 ? store_launch<DT_F32, DT_F16>(a, s)
                                                : store_launch<DT_F16, DT_F16>(a, s));
  return pages_done(src_dtype == WS_DTYPE_F32 ? store_launch<DT_F32, DT_BF16>(a, s)
                                              : store_launch<DT_BF16, DT_BF16>(a, s));
}

long ws_debug_page_places(const int32_t *cu_seqlens, const int32_t *rows, const int32_t *start,
                          const int32_t *table, int T, int n_seqs, int n_rows, int max_pages,
                          int n_pages, int page_size, long long *places) {
  if (!start || !table || !places || T < 1 || n_seqs < 1 || (!cu_seqlens && T != n_seqs) ||
      !paged_shape_ok(n_rows, max_pages, n_pages, page_size, 1) || (!rows && n_rows < n_seqs))
    return -1;
  PageStoreParams a = {};
  a.cu = cu_seqlens;
  a.rows = rows;
  a.start = start;
  a.table = table;
  a.n = n_seqs;
  a.n_rows = n_rows;
  a.max_pages = max_pages;
  a.n_pages = n_pages;
  a.ps = page_size;
  a.nkv = 1;
  long found = 0;
  for (int t = 0; t < T; ++t) found += (places[t] = page_place(a, t)) >= 0;
  return found;
}

size_t ws_kv_pages_workspace_bytes(int n_rows, int n_pages) {
  return n_rows < 1 || n_pages < 1 ? 0 : pages_workspace(n_rows, n_pages);
}

ws_status ws_kv_pages_resize(int32_t *table, int32_t *refs, int32_t *tokens, const int32_t *want,
                             int n_rows, int max_pages, int n_pages, int page_size,
                             void *workspace, size_t workspace_bytes, ws_stream_t stream) {
  if (!table || !refs || !tokens || !want || !workspace) {
    set_error("null argument");
    return WS_ERR_ARG;
  }
  PagesParams a = {};
  a.table = table;
  a.refs = refs;
  a.tokens = tokens;
  a.want = want;
  a.n_rows = n_rows;
  a.max_pages = max_pages;
  a.n_pages = n_pages;
  a.ps = page_size;
  const ws_status st = pages_bind(a, workspace, workspace_bytes);
  if (st != WS_OK) return st;
  return pages_done(launch_serving(k_pages_resize, dim3(1), kPlanThreads, 0, (cudaStream_t)stream, a));
}

ws_status ws_kv_pages_fork(int32_t *table, int32_t *refs, int32_t *tokens, const int32_t *src,
                           const int32_t *dst, int n, void *k_pages, void *v_pages, int layers,
                           long long page_bytes, int n_rows, int max_pages, int n_pages,
                           int page_size, void *workspace, size_t workspace_bytes,
                           ws_stream_t stream) {
  if (!table || !refs || !tokens || !src || !dst || !k_pages || !v_pages || !workspace) {
    set_error("null argument");
    return WS_ERR_ARG;
  }
  PagesParams a = {};
  a.table = table;
  a.refs = refs;
  a.tokens = tokens;
  a.src = src;
  a.dst = dst;
  a.n = n;
  a.k = static_cast<unsigned char*>(k_pages);
  a.v = static_cast<unsigned char*>(v_pages);
  a.layers = layers;
  a.page_bytes = page_bytes;
  a.n_rows = n_rows;
  a.max_pages = max_pages;
  a.n_pages = n_pages;
  a.ps = page_size;
  if (n < 1 || n > n_rows) {
    set_error("fork: 1 to n_rows pairs");
    return WS_ERR_SHAPE;
  }
  if (!pages_data_ok(a)) return WS_ERR_SHAPE;
  const ws_status st = pages_bind(a, workspace, workspace_bytes);
  if (st != WS_OK) return st;
  cudaError_t e = launch_serving(k_pages_fork, dim3(1), kPlanThreads, 0, (cudaStream_t)stream, a);
  if (e != cudaSuccess) return pages_done(e);
  const long long work = (long long)n * (2ll * layers * ((page_bytes + kMoveChunk - 1) / kMoveChunk) +
                                         max_pages / kMoveThreads + 1);
  return pages_done(launch_serving(k_pages_move<true>, dim3(move_grid(work)), kMoveThreads, 0,
                                   (cudaStream_t)stream, a));
}

ws_status ws_kv_pages_compact(int32_t *table, int32_t *refs, void *k_pages, void *v_pages,
                              int layers, long long page_bytes, int n_rows, int max_pages,
                              int n_pages, int page_size, void *workspace, size_t workspace_bytes,
                              ws_stream_t stream) {
  if (!table || !refs || !k_pages || !v_pages || !workspace) {
    set_error("null argument");
    return WS_ERR_ARG;
  }
  PagesParams a = {};
  a.table = table;
  a.refs = refs;
  a.k = static_cast<unsigned char*>(k_pages);
  a.v = static_cast<unsigned char*>(v_pages);
  a.layers = layers;
  a.page_bytes = page_bytes;
  a.n_rows = n_rows;
  a.max_pages = max_pages;
  a.n_pages = n_pages;
  a.ps = page_size;
  if (!pages_data_ok(a)) return WS_ERR_SHAPE;
  const ws_status st = pages_bind(a, workspace, workspace_bytes);
  if (st != WS_OK) return st;
  cudaError_t e = launch_serving(k_pages_compact, dim3(1), kPlanThreads, 0, (cudaStream_t)stream, a);
  if (e != cudaSuccess) return pages_done(e);
  const long long work = (long long)n_pages * (2ll * layers * ((page_bytes + kMoveChunk - 1) / kMoveChunk)) +
                         (long long)n_rows * max_pages / kMoveThreads + 1;
  return pages_done(launch_serving(k_pages_move<false>, dim3(move_grid(work)), kMoveThreads, 0,
                                   (cudaStream_t)stream, a));
}

}  // extern "C"
