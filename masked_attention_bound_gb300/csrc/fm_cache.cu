// The paged K/V cache: writing new tokens, moving accepted nodes together,
// and the page bookkeeping (fork, reserve, compact).
//
// All of it moves bytes and counts integers; nothing rounds.  The copies are
// bound by HBM (2 bytes of traffic per byte moved), the bookkeeping by the
// latency of a launch and of a few dependent passes over the reference
// counts.  Results do not depend on the order in which threads run: pages
// are ranked by prefix sums, and counts change by atomic additions only.
#include <cooperative_groups.h>

#include "fm_cache.h"
#include "fm_ptx.cuh"

namespace cg = cooperative_groups;

namespace fm {

fm_status check_cache(const fm_cache* c, bool pools) {
  if (!c) return FM_ERR_INVALID;
  if (c->B < 1 || c->n_pages < 1 || c->max_pages < 1) return FM_ERR_INVALID;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return FM_ERR_UNSUPPORTED;
  if (c->n_pages > kMaxPoolPages ||
      static_cast<int64_t>(c->max_pages) * c->page_size > kMaxTokenIndex)
    return FM_ERR_UNSUPPORTED;
  // sums of pages over the rows are counted in 31 bits
  if (static_cast<int64_t>(c->B) * c->max_pages > 0x7fffffff) return FM_ERR_UNSUPPORTED;
  if (!pools) return FM_OK;
  if (c->Hkv < 1 || c->layers < 1) return FM_ERR_INVALID;
  if ((c->d != 64 && c->d != 128) || c->Hkv > kMaxHeads) return FM_ERR_UNSUPPORTED;
  for (const int64_t* st : {c->k_stride, c->v_stride})
    for (int i = 0; i < 4; ++i)
      if (st[i] <= 0 || st[i] % 8 != 0 || st[i] >= (int64_t(1) << 36)) return FM_ERR_INVALID;
  return FM_OK;
}

namespace {

// The pools of a cache as the copy kernels see them, in 16-byte vectors.
struct Pools {
  uint4* p[2];          // K, V
  int64_t layer[2], page[2], slot[2], head[2];
  int chunk_shift;      // vectors per head (d / 8, of codes d / 16) as a power of two
  int row;              // vectors of one token, K or V
  int page_shift;       // page_size as a power of two
  FastDiv by_row;
  bool linear[2];       // a page's tokens lie one after the other without gaps
  float* scale[2];      // of a cache of codes, [layers][pages][Hkv][blocks of a page]; null: bf16
  int64_t scale_layer;  // scales of a layer
  int scale_page, block_shift;   // of a page; log2 of its blocks
  __device__ __forceinline__ int page_size() const { return 1 << page_shift; }
  // place of vector r of a token: head r >> chunk_shift
  __device__ __forceinline__ int64_t in_token(int kv, int r) const {
    return (r >> chunk_shift) * head[kv] + (r & ((1 << chunk_shift) - 1));
  }
};

// k_scale, v_scale: of a cache of e4m3 codes
Pools pools_of(const fm_cache& c, void* k, void* v, float* k_scale = nullptr, float* v_scale = nullptr) {
  Pools P;
  const int unit = k_scale ? 16 : 8;     // elements of a vector
  P.scale[0] = k_scale;
  P.scale[1] = v_scale;
  P.block_shift = page_shift(c.page_size) - 4;
  P.scale_page = c.Hkv << P.block_shift;
  P.scale_layer = static_cast<int64_t>(c.n_pages) * P.scale_page;
  P.p[0] = static_cast<uint4*>(k);
  P.p[1] = static_cast<uint4*>(v);
  const int64_t* st[2] = {c.k_stride, c.v_stride};
  for (int t = 0; t < 2; ++t) {
    P.layer[t] = st[t][0] / unit;
    P.page[t] = st[t][1] / unit;
    P.slot[t] = st[t][2] / unit;
    P.head[t] = st[t][3] / unit;
    P.linear[t] = (c.Hkv == 1 || P.head[t] == c.d / unit) && P.slot[t] == c.Hkv * (c.d / unit);
  }
  P.chunk_shift = (c.d == 64 ? 3 : 4) - (k_scale ? 1 : 0);
  P.row = c.Hkv << P.chunk_shift;
  P.by_row = FastDiv::of(P.row);
  P.page_shift = page_shift(c.page_size);
  return P;
}

// ------------------------------------------------------------------ append
// Each block takes a few consecutive packed tokens.  All threads first load
// its 16-byte vectors, K and V, which needs no lookup; meanwhile a warp (or, of
// more than eight tokens a block, a thread) per token finds its sequence (a
// search over cu), page and slot.  128 single tokens took 3.2 us by threads and
// 2.6 by warps, 20000 tokens of 512 bytes 4.2 by threads and 6.9 by warps.
constexpr int kAppendThreads = 256, kAppendVecs = 4;

struct AppendArgs {
  const uint4* src[2];
  int64_t tok[2], head[2];     // source strides in vectors
  const int32_t *cu, *table, *lens;
  int* status;
  int B, total, max_pages, n_pages, tokens;  // tokens: per block
};

__global__ void __launch_bounds__(kAppendThreads)
    append_kernel(const __grid_constant__ AppendArgs A, const __grid_constant__ Pools P) {
  extern __shared__ int64_t where[];   // per token of the block: page << 8 | slot, -1: skip
  grid_launch_dependents();
  grid_dependency_wait();
  const int t0 = blockIdx.x * A.tokens;
  const int per = 2 * P.row;           // vectors of one token, K then V
  const int all = min(A.tokens, A.total - t0) * per;
  uint4 x[kAppendVecs];
  // vector v of the block: token, K or V, vector of the token
  struct At {
    int i, kv, r;
  };
  auto at = [&](int v) -> At {
    const int half = P.by_row(v);      // 2 i + kv
    return At{half >> 1, half & 1, v - half * P.row};
  };
  auto load = [&](int v0) {
#pragma unroll
    for (int u = 0; u < kAppendVecs; ++u) {
      const int v = v0 + u * kAppendThreads;
      if (v < all) {
        const At w = at(v);
        const int64_t head = (w.r >> P.chunk_shift) * A.head[w.kv];
        x[u] = __ldg(A.src[w.kv] + (t0 + w.i) * A.tok[w.kv] + head +
                     (w.r & ((1 << P.chunk_shift) - 1)));
      }
    }
  };
  load(threadIdx.x);
  // token t of sequence b, the last one with cu[b] <= t: page << 8 | slot
  auto place = [&](int t, int b) -> int64_t {
    int n;
    const int base = context_of(A.lens, A.cu, b, A.total, A.max_pages << P.page_shift, n);
    const int node = t - A.cu[b], pos = base + node;
    if (base >= 0 && node >= 0 && node < n) {
      const int pg = A.table[static_cast<int64_t>(b) * A.max_pages + (pos >> P.page_shift)];
      if (pg >= 0 && pg < A.n_pages) return (static_cast<int64_t>(pg) << 8) | (pos & (P.page_size() - 1));
    }
    flag(A.status, DEV_CACHE);
    return -1;
  };
  const int behind = A.cu[A.B];          // tokens from here on belong to no sequence
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (A.tokens <= kAppendThreads / 32) {
    // a warp per token: 32 of the offsets a step
    const int t = t0 + warp;
    if (warp < A.tokens && t < A.total) {
      int lo = 0;
      for (int n = A.B; n > 1;) {
        const int step = (n + 31) >> 5;
        const unsigned below = __ballot_sync(0xffffffffu, lane * step < n && A.cu[lo + lane * step] <= t);
        const int k = 31 - __clz(below | 1u);
        lo += k * step;
        n = min(step, n - k * step);
      }
      const int64_t to = t < behind ? place(t, lo) : -1;
      if (lane == 0) where[warp] = to;
    }
  } else {
    for (int i = threadIdx.x; i < A.tokens; i += kAppendThreads) {
      const int t = t0 + i;
      int lo = 0, hi = A.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (A.cu[mid] <= t) lo = mid; else hi = mid;
      }
      where[i] = t < A.total && t < behind ? place(t, lo) : -1;
    }
  }
  __syncthreads();
  for (int v0 = threadIdx.x; v0 < all; v0 += kAppendVecs * kAppendThreads) {
    if (v0 != threadIdx.x) load(v0);
#pragma unroll
    for (int u = 0; u < kAppendVecs; ++u) {
      const int v = v0 + u * kAppendThreads;
      if (v < all) {
        const At w = at(v);
        const int64_t to = where[w.i];
        if (to >= 0)
          P.p[w.kv][(to >> 8) * P.page[w.kv] + (to & 255) * P.slot[w.kv] + P.in_token(w.kv, w.r)] = x[u];
      }
    }
  }
}

// ------------------------------------------------------------------ accept
// A block moves the accepted nodes of one sequence in one layer; its first
// warp looks their places up, 32 at a time.  Each thread keeps one 16-byte
// vector of a token (of K or V) and walks the nodes in ascending order.  The
// node moved i-th comes from a place at or past base + i and goes to base +
// i, so a thread that loads node i before it stores node i never overwrites
// a source that it still needs; threads share no bytes.  Bound by the latency
// of the lookups, so what counts is how many blocks an SM holds: 64 trees of 8
// accepted nodes in 16 layers took 5.7 us with 4 nodes in flight a thread and
// 40 registers, 7.8 us with 8 and 72.
constexpr int kAcceptThreads = 128;

struct AcceptArgs {
  const int32_t *accept, *n_accept, *cu, *table, *lens;
  int32_t *lens_out, *ref;
  int* status;
  int max_accept, max_pages, n_pages;
};

__global__ void __launch_bounds__(kAcceptThreads, 12)
    accept_kernel(const __grid_constant__ AcceptArgs A, const __grid_constant__ Pools P) {
  __shared__ int2 place[32];           // from, to: page << 8 | slot
  __shared__ int good;
  grid_launch_dependents();
  grid_dependency_wait();
  const int b = blockIdx.y, layer = blockIdx.z, lane = threadIdx.x & 31;
  const int32_t* acc = A.accept + static_cast<int64_t>(b) * A.max_accept;
  const int32_t* row = A.table + static_cast<int64_t>(b) * A.max_pages;
  const int m = A.n_accept[b];
  int n;
  const int base = context_of(A.lens, A.cu, b, 0x7fffffff, A.max_pages << P.page_shift, n);
  const bool sized = base >= 0 && m >= 0 && m <= n && m <= A.max_accept;
  // page << 8 | slot of a position, -1 if its page is out of range
  auto at = [&](int pos) -> int {
    const int pg = row[pos >> P.page_shift];
    return pg >= 0 && pg < A.n_pages ? (pg << 8) | (pos & (P.page_size() - 1)) : -1;
  };
  // the first page past the context and x more tokens
  auto first_free = [&](int x) { return (base + x + P.page_size() - 1) >> P.page_shift; };
  // entry i of the list, valid or not
  auto look = [&](int i, int2& p) -> bool {
    const int a = acc[i], before = i ? acc[i - 1] : -1;
    if (a <= before || a >= n) return false;
    p = make_int2(at(base + a), at(base + i));
    return p.x >= 0 && p.y >= 0;
  };
  if (threadIdx.x < 32) {
    bool ok = sized;
    int2 p = make_int2(0, 0);
    for (int i = lane; sized && i < m; i += 32) {
      int2 q;
      ok = look(i, q) && ok;
      if (i < 32) p = q;
    }
    // the pages past the new length, which the first block of the sequence
    // lets go of: looked at by all, since one that is out of range leaves the
    // whole sequence as it is
    if (sized && A.ref)
      for (int j = first_free(m) + lane; j < first_free(n); j += 32) ok = at(j << P.page_shift) >= 0 && ok;
    ok = __all_sync(0xffffffffu, ok);
    place[lane] = p;
    if (lane == 0) good = ok;
  }
  __syncthreads();
  const bool ok = good != 0;
  if (blockIdx.x == 0 && layer == 0) {
    if (threadIdx.x == 0) {
      A.lens_out[b] = ok ? base + m : A.lens[b];
      if (!ok) flag(A.status, DEV_CACHE);
    }
    if (ok && A.ref)
      for (int j = first_free(m) + threadIdx.x; j < first_free(n); j += blockDim.x) atomicSub(A.ref + row[j], 1);
  }
  if (!ok) return;
  const int v = blockIdx.x * kAcceptThreads + threadIdx.x;
  const int kv = v >= P.row;
  uint4* pool = P.p[kv] + layer * P.layer[kv] + P.in_token(kv, v - kv * P.row);
  constexpr int U = 4;
  for (int i0 = 0; i0 < m; i0 += 32) {
    if (i0 > 0) {                      // the next 32 places
      __syncthreads();
      int2 q;
      if (threadIdx.x < 32 && i0 + lane < m && look(i0 + lane, q)) place[lane] = q;
      __syncthreads();
    }
    if (v >= 2 * P.row) continue;
    const int end = min(m - i0, 32);
    for (int j0 = 0; j0 < end; j0 += U) {
      uint4 x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int2 p = place[(j0 + u) & 31];
        if (j0 + u < end && p.x != p.y) x[u] = pool[(p.x >> 8) * P.page[kv] + (p.x & 255) * P.slot[kv]];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int2 p = place[(j0 + u) & 31];
        if (j0 + u < end && p.x != p.y) pool[(p.y >> 8) * P.page[kv] + (p.y & 255) * P.slot[kv]] = x[u];
      }
    }
  }
}

// ------------------------------------------------------------------ fork
struct PageArgs {
  const int32_t *table, *lens, *ref;
  int32_t *table_out, *lens_out, *ref_out;
  int* status;
  int B, page_size, n_pages, max_pages;
};

// Pages of a row, 0 (and the status) if its length is out of range.
__device__ __forceinline__ int pages_of(const PageArgs& A, int b, int& len, bool& ok) {
  len = A.lens[b];
  ok = len >= 0 && len <= A.max_pages * A.page_size;
  if (!ok) len = 0;
  return (len + A.page_size - 1) / A.page_size;
}

// One warp per row: the new row's pages gain a hold, the old row's lose one.
__device__ __forceinline__ void fork_row(const PageArgs& A, const int32_t* parent, int b) {
  const int lane = threadIdx.x & 31;
  int p = parent[b];
  bool ok = p >= -1 && p < A.B;
  if (!ok) p = -1;
  int len_old, len = 0, used = 0;
  bool ok_old, ok_new = true;
  const int used_old = pages_of(A, b, len_old, ok_old);
  if (p >= 0) used = pages_of(A, p, len, ok_new);
  ok = ok && ok_old && ok_new;
  for (int j = lane; j < used; j += 32) {
    const int pg = A.table[static_cast<int64_t>(p) * A.max_pages + j];
    A.table_out[static_cast<int64_t>(b) * A.max_pages + j] = pg;
    const bool in = pg >= 0 && pg < A.n_pages;
    if (in && p != b) atomicAdd(A.ref_out + pg, 1);
    ok = ok && in;
  }
  if (p != b)
    for (int j = lane; j < used_old; j += 32) {
      const int pg = A.table[static_cast<int64_t>(b) * A.max_pages + j];
      const bool in = pg >= 0 && pg < A.n_pages;
      if (in) atomicSub(A.ref_out + pg, 1);
      ok = ok && in;
    }
  if (lane == 0) A.lens_out[b] = len;
  if (!ok) flag(A.status, DEV_CACHE);
}

// ref_out has the old counts already: it is ref itself, or ref_copy_kernel ran.
__global__ void __launch_bounds__(128) fork_kernel(const __grid_constant__ PageArgs A, const int32_t* parent) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int b = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (b < A.B) fork_row(A, parent, b);
}
// Both by one block, for few pages and rows.
__global__ void __launch_bounds__(1024)
    fork_copy_kernel(const __grid_constant__ PageArgs A, const int32_t* parent) {
  grid_launch_dependents();
  grid_dependency_wait();
#pragma unroll 4
  for (int i = threadIdx.x; i < A.n_pages; i += 1024) A.ref_out[i] = A.ref[i];
  __syncthreads();
  for (int b = threadIdx.x >> 5; b < A.B; b += 32) fork_row(A, parent, b);
}
__global__ void __launch_bounds__(256) ref_copy_kernel(const int32_t* from, int32_t* to, int n) {
  grid_launch_dependents();
  grid_dependency_wait();
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) to[i] = from[i];
}

// ------------------------------------------------------------------ page plans
// Reserve and compact rank the pages of the pool by prefix sums of the
// reference counts.  One cluster of N blocks does it in a single launch: each
// block owns an N-th of the pages (and of the rows), the blocks exchange their
// sums through distributed shared memory, and the cluster barrier separates
// the passes.  N is 8, or 1 where a block has few pages and rows to a thread:
// its barriers are cheaper.
constexpr int kPlanThreads = 1024;

template <int N>
__device__ __forceinline__ void plan_sync(cg::cluster_group& cl) {
  if constexpr (N == 1) __syncthreads();
  else cl.sync();
}


// Regions of the pages workspace (int32 words).
struct PlanWs {
  int32_t* info;     // [8] numbers handed to the copy kernel
  int32_t* row;      // [B] per row: pages it asks for, bit 30: its last page is replaced
  int32_t* copy;     // [B][3] source, destination (-1: none), tokens
  int32_t* list;     // [n_pages] free pages in the order they are taken (holes)
  int32_t* mover;    // [n_pages] pages that move
  int32_t* to;       // [n_pages] where a page that moves goes
  size_t bytes;
};

PlanWs plan_ws(const fm_cache& c, void* ws) {
  PlanWs W;
  size_t off = 0;
  char* base = static_cast<char*>(ws);
  auto take = [&](size_t words) {
    int32_t* p = reinterpret_cast<int32_t*>(base + off);
    off = (off + words * 4 + 255) & ~static_cast<size_t>(255);
    return p;
  };
  W.info = take(8);
  W.row = take(c.B);
  W.copy = take(3 * static_cast<size_t>(c.B));
  W.list = take(c.n_pages);
  W.mover = take(c.n_pages);
  W.to = take(c.n_pages);
  W.bytes = off;
  return W;
}

// Exclusive prefix sum of one value per thread over the block; total: the sum.
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();                       // the sums of an earlier call have been read
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  int before = 0, all = 0;
  const int n = blockDim.x >> 5;
  if (lane < n) all = warp_sums[lane];
  int w = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, n - 1);
  before = __shfl_sync(0xffffffffu, w - all, warp);
  return before + inc - x;
}

// What the blocks of a plan tell each other.
struct PlanShared {
  int warp_sums[32];
  int said[4];       // this block's numbers, read by the others
  int before[4], all[4];
  int parts[3][32];  // see block_sums
};

// Sums of n values per thread over the block (kPlanThreads), into sh.said.
template <int n>
__device__ __forceinline__ void block_sums(const int (&x)[n], PlanShared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < n; ++i) {
    const int s = __reduce_add_sync(0xffffffffu, x[i]);
    if (lane == 0) sh.parts[i][warp] = s;
  }
  __syncthreads();
  if (warp < n) {
    const int s = __reduce_add_sync(0xffffffffu, sh.parts[warp][lane]);
    if (lane == 0) sh.said[warp] = s;
  }
}

// Exchange: sums over the blocks before this one, and over all, of `said`.
template <int N>
__device__ __forceinline__ void exchange(cg::cluster_group& cl, PlanShared& sh, int n) {
  plan_sync<N>(cl);
  if (threadIdx.x < n) {
    int before = 0, all = 0;
    for (int r = 0; r < N; ++r) {
      const int x = *cl.map_shared_rank(&sh.said[threadIdx.x], r);
      if (r < static_cast<int>(cl.block_rank())) before += x;
      all += x;
    }
    sh.before[threadIdx.x] = before;
    sh.all[threadIdx.x] = all;
  }
  plan_sync<N>(cl);                      // nobody's numbers change before all have read them
}

// info (the caller's): free pages after the call, pages asked for.
template <int N>
__global__ void __cluster_dims__(N, 1, 1) __launch_bounds__(kPlanThreads, 1)
    reserve_kernel(const __grid_constant__ PageArgs A, const int32_t* grow,
                   const __grid_constant__ PlanWs W, int32_t* info) {
  cg::cluster_group cl = cg::this_cluster();
  __shared__ PlanShared sh;
  __shared__ int3 rows_of[kPlanThreads];   // asked for, pages, first of the taken ones
  const int rank = cl.block_rank();
  grid_launch_dependents();
  grid_dependency_wait();
  const int rows = (A.B + N - 1) / N;
  const int b0 = min(rank * rows, A.B), b1 = min(b0 + rows, A.B);
  const int span = (A.n_pages + N - 1) / N;
  const int p0 = min(rank * span, A.n_pages), p1 = min(p0 + span, A.n_pages);
  constexpr int kReplace = 1 << 30;

  // what the rows ask for; anything out of range refuses the call
  int asked = 0, bad = 0;
  for (int b = b0 + threadIdx.x; b < b1; b += kPlanThreads) {
    int len;
    bool ok;
    const int have = pages_of(A, b, len, ok);
    const int g = grow[b];
    const int32_t* row = A.table + static_cast<int64_t>(b) * A.max_pages;
    int need = 0;
    if (!ok || g < 0 || g > A.max_pages * A.page_size - len) {
      bad = 1;
    } else {
      need = (len + g + A.page_size - 1) / A.page_size - have;
      if (g > 0 && len % A.page_size != 0) {
        const int last = row[have - 1];
        if (last < 0 || last >= A.n_pages) bad = 1;
        else if (A.ref[last] > 1) need |= kReplace;
      }
    }
    W.row[b] = need;
    asked += (need & ~kReplace) + (need >= kReplace);
  }
  int free_pages = 0;
#pragma unroll 4
  for (int p = p0 + threadIdx.x; p < p1; p += kPlanThreads) {
    const int r = A.ref[p];
    free_pages += r == 0;
    bad |= r < 0;
  }
  block_sums<3>({asked, free_pages, bad}, sh);
  exchange<N>(cl, sh, 3);
  const int total = sh.all[0], n_free = sh.all[1];
  const bool refused = sh.all[2] != 0;
  const bool full = total > n_free;
  const bool go = !refused && !full;

  // the taken pages: the first `total` free ones
  int rank0 = sh.before[1];
  for (int p = p0; p < p1; p += kPlanThreads) {
    if (rank0 >= (go ? total : 0) && A.ref_out == A.ref) break;   // nothing more to write
    const int q = p + threadIdx.x;
    const int r = q < p1 ? A.ref[q] : -1;
    int n;
    const int k = rank0 + block_scan(r == 0, sh.warp_sums, n);
    rank0 += n;
    if (q < p1) {
      const bool taken = go && r == 0 && k < total;
      if (taken) W.list[k] = q;
      if (taken || A.ref_out != A.ref) A.ref_out[q] = taken ? 1 : r;
    }
  }
  if (rank == 0 && threadIdx.x == 0) {
    info[1] = total;
    if (refused) flag(A.status, DEV_CACHE);
    if (full) flag(A.status, DEV_PAGES);
  }
  plan_sync<N>(cl);                      // the list is complete, and ref_out

  // the rows, 1024 at a time: a thread each for the counts, then a warp each
  // for the entries
  int first = sh.before[0], released = 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int c0 = b0; c0 < b1; c0 += kPlanThreads) {
    const int b = c0 + threadIdx.x;
    const int word = b < b1 && go ? W.row[b] : 0;
    const int mine = (word & ~kReplace) + (word >= kReplace);
    int n;
    const int at = first + block_scan(mine, sh.warp_sums, n);
    first += n;
    if (b < b1) {
      int len;
      bool ok;
      const int have = pages_of(A, b, len, ok);
      A.lens_out[b] = go ? len + grow[b] : A.lens[b];
      int32_t* copy = W.copy + 3 * static_cast<int64_t>(b);
      copy[1] = -1;
      if (word >= kReplace) {
        const int old = A.table[static_cast<int64_t>(b) * A.max_pages + have - 1];
        copy[0] = old;
        copy[1] = W.list[at];
        copy[2] = len % A.page_size;
        released += atomicSub(A.ref_out + old, 1) == 1;
      }
      rows_of[threadIdx.x] = make_int3(word, have, at);
    }
    __syncthreads();
    for (int i = warp; i < min(b1 - c0, kPlanThreads); i += kPlanThreads / 32) {
      const int3 r = rows_of[i];
      const int swap = r.x >= kReplace;
      const int32_t* row = A.table + static_cast<int64_t>(c0 + i) * A.max_pages;
      int32_t* out = A.table_out + static_cast<int64_t>(c0 + i) * A.max_pages;
      if (A.table_out != A.table)
        for (int j = lane; j < r.y - swap; j += 32) out[j] = row[j];
      for (int j = lane; j < (r.x & ~kReplace) + swap; j += 32) out[r.y - swap + j] = W.list[r.z + j];
    }
  }
  block_sums<1>({released}, sh);
  exchange<N>(cl, sh, 1);
  if (rank == 0 && threadIdx.x == 0) info[0] = n_free - (go ? total : 0) + sh.all[0];
}

// info of the workspace: [0] moves, [1] held pages
template <int N>
__global__ void __cluster_dims__(N, 1, 1) __launch_bounds__(kPlanThreads, 1)
    compact_kernel(const __grid_constant__ PageArgs A, const __grid_constant__ PlanWs W,
                   int32_t* n_live_out) {
  cg::cluster_group cl = cg::this_cluster();
  __shared__ PlanShared sh;
  const int rank = cl.block_rank();
  grid_launch_dependents();
  grid_dependency_wait();
  const int span = (A.n_pages + N - 1) / N;
  const int p0 = min(rank * span, A.n_pages), p1 = min(p0 + span, A.n_pages);
  int live = 0;
#pragma unroll 4
  for (int p = p0 + threadIdx.x; p < p1; p += kPlanThreads) live += A.ref[p] != 0;
  block_sums<1>({live}, sh);
  exchange<N>(cl, sh, 1);
  const int n_live = sh.all[0];

  int holes = 0, movers = 0;
#pragma unroll 4
  for (int p = p0 + threadIdx.x; p < p1; p += kPlanThreads) {
    const bool held = A.ref[p] != 0;
    holes += !held && p < n_live;
    movers += held && p >= n_live;
  }
  block_sums<2>({holes, movers}, sh);
  exchange<N>(cl, sh, 2);
  const int moves = sh.all[1];           // as many holes as movers
  int h0 = sh.before[0], m0 = sh.before[1];
  for (int p = p0; p < p1; p += kPlanThreads) {
    const int q = p + threadIdx.x;
    const int r = q < p1 ? A.ref[q] : 0;
    const bool hole = q < p1 && r == 0 && q < n_live, mover = q < p1 && r != 0 && q >= n_live;
    int n, m;
    // holes lie below n_live and movers at or past it: one scan serves both
    const int kh = block_scan(static_cast<int>(hole) | (static_cast<int>(mover) << 16), sh.warp_sums, n);
    m = n >> 16;
    n &= 0xffff;
    if (hole) W.list[h0 + (kh & 0xffff)] = q;
    if (mover) W.mover[m0 + (kh >> 16)] = q;
    if (q < p1 && !hole && !mover && A.ref_out != A.ref) A.ref_out[q] = r;
    if (q < p1 && q >= n_live) W.to[q] = q;   // movers get their place below
    if (r < 0) flag(A.status, DEV_CACHE);
    h0 += n;
    m0 += m;
  }
  if (rank == 0 && threadIdx.x == 0) {
    W.info[0] = moves;
    W.info[1] = n_live;
    *n_live_out = n_live;
  }
  plan_sync<N>(cl);
  for (int k = rank * kPlanThreads + threadIdx.x; k < moves; k += N * kPlanThreads) {
    const int src = W.mover[k], dst = W.list[k];
    W.to[src] = dst;
    A.ref_out[dst] = A.ref[src];
    A.ref_out[src] = 0;
  }
}

// ------------------------------------------------------------------ page copies
// n tokens of one page of one layer, K or V, from page src to page dst, by
// one block: vectors of 16 bytes, four in flight per thread, neither side
// kept in L1.  Small pages (4 KB of K or V at 16 tokens of 2 heads of 64) are
// bound by the latency of finding them, large ones by HBM: 256 sequences of
// 8000 tokens, half of the pages free, took 335 us by blocks of 128 threads and
// 622 by blocks of 256 with eight in flight, and 64 KB pages 254 and 255.
constexpr int kCopyThreads = 128;

// (SCALES, a kernel of its own: with the scales' copy behind a branch the pages of
// bf16 took 260 us instead of 250)
template <bool SCALES>
__device__ __forceinline__ void copy_page(const Pools& P, int kv, int layer, int src, int dst, int n) {
  const uint4* from = P.p[kv] + layer * P.layer[kv] + src * P.page[kv];
  uint4* to = P.p[kv] + layer * P.layer[kv] + dst * P.page[kv];
  const int all = n * P.row;
  const bool linear = P.linear[kv];
  constexpr int U = 4;
  for (int v0 = threadIdx.x; v0 < all; v0 += U * kCopyThreads) {
    uint4 x[U];
    int64_t at[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = v0 + u * kCopyThreads;
      at[u] = v;
      if (!linear) {
        const int s = P.by_row(v);
        at[u] = s * P.slot[kv] + P.in_token(kv, v - s * P.row);
      }
      if (v < all) x[u] = __ldcs(from + at[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (v0 + u * kCopyThreads < all) __stcs(to + at[u], x[u]);
  }
  if constexpr (SCALES) {
    // the scales of the blocks that hold these tokens
    float* s = P.scale[kv] + layer * P.scale_layer;
    for (int i = threadIdx.x; i < P.scale_page; i += kCopyThreads)
      if ((i & ((1 << P.block_shift) - 1)) * 16 < n)
        s[static_cast<int64_t>(dst) * P.scale_page + i] = s[static_cast<int64_t>(src) * P.scale_page + i];
  }
}

template <bool SCALES>
__global__ void __launch_bounds__(kCopyThreads)
    reserve_copy_kernel(const __grid_constant__ Pools P, const int32_t* copy, int B, int layers) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t items = static_cast<int64_t>(B) * layers * 2;
  for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
    const int b = static_cast<int>(i / (layers * 2)), r = static_cast<int>(i % (layers * 2));
    const int32_t* c = copy + 3 * static_cast<int64_t>(b);
    if (c[1] < 0) continue;
    copy_page<SCALES>(P, r & 1, r >> 1, c[0], c[1], c[2]);
  }
}

template <bool SCALES>
__global__ void __launch_bounds__(kCopyThreads)
    compact_copy_kernel(const __grid_constant__ Pools P, const __grid_constant__ PageArgs A,
                        const __grid_constant__ PlanWs W, int layers) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int moves = W.info[0], n_live = W.info[1];
  const int64_t items = static_cast<int64_t>(moves) * layers * 2;
  for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
    const int k = static_cast<int>(i / (layers * 2)), r = static_cast<int>(i % (layers * 2));
    copy_page<SCALES>(P, r & 1, r >> 1, W.mover[k], W.list[k], P.page_size());
  }
  for (int b = blockIdx.x; b < A.B; b += gridDim.x) {
    int len;
    bool ok;
    const int used = pages_of(A, b, len, ok);
    for (int j = threadIdx.x; j < used; j += kCopyThreads) {
      const int64_t at = static_cast<int64_t>(b) * A.max_pages + j;
      const int pg = A.table[at];
      const bool in = pg >= 0 && pg < A.n_pages;
      A.table_out[at] = in && pg >= n_live ? W.to[pg] : pg;
      ok = ok && in;
    }
    if (!ok) flag(A.status, DEV_CACHE);
  }
}

// Each output is its input itself or does not overlap it.
bool outputs_apart(const fm_cache& c, const PageArgs& A) {
  const size_t nt = static_cast<size_t>(c.B) * c.max_pages * 4, nl = static_cast<size_t>(c.B) * 4,
               nr = static_cast<size_t>(c.n_pages) * 4;
  if (A.table_out != A.table && overlaps(A.table_out, nt, A.table, nt)) return false;
  if (A.lens_out && A.lens_out != A.lens && overlaps(A.lens_out, nl, A.lens, nl)) return false;
  if (A.ref_out != A.ref && overlaps(A.ref_out, nr, A.ref, nr)) return false;
  return true;
}

// Few enough pages (four a thread) and rows (two a warp) that the page
// bookkeeping is faster by one block: a fork and a reserve of 8 rows took 9.0
// us so and 12.6 by clusters, of 64 rows 12.5 and 13.2, of 128 rows 17.6 and
// 14.6; a compaction of 250 pages 6.3 and 8.6.
bool few_pages(const fm_cache& c) { return c.n_pages <= 4096 && c.B <= 64; }

int copy_grid() { return num_sms() * 16; }

// k_scale, v_scale: of a cache of e4m3 codes; both null with a cache of bf16.
fm_status reserve_pages(const fm_cache* c, const int32_t* grow, void* k_pool, void* v_pool, float* k_scale,
                        float* v_scale, const int32_t* table, const int32_t* lens, const int32_t* ref,
                        int32_t* table_out, int32_t* lens_out, int32_t* ref_out, int32_t* info, void* ws,
                        size_t ws_bytes, int32_t* status, void* stream) {
  fm_status st = check_cache(c, true);
  if (st != FM_OK) return st;
  if (!grow || !table || !lens || !ref || !table_out || !lens_out || !ref_out || !info)
    return FM_ERR_INVALID;
  if (!aligned_to(k_pool, 16) || !aligned_to(v_pool, 16)) return FM_ERR_INVALID;
  PageArgs A{table, lens, ref, table_out, lens_out, ref_out, status, c->B, c->page_size, c->n_pages,
             c->max_pages};
  if (!outputs_apart(*c, A)) return FM_ERR_INVALID;
  if (!aligned_to(ws, 256)) return FM_ERR_WORKSPACE;
  const PlanWs W = plan_ws(*c, ws);
  if (ws_bytes < W.bytes) return FM_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  prof_begin(K_PAGES_PLAN, s);
  cudaError_t e = few_pages(*c)
                      ? launch_dependent(reserve_kernel<1>, dim3(1), kPlanThreads, 0, s, A, grow, W, info)
                      : launch_dependent(reserve_kernel<8>, dim3(8), kPlanThreads, 0, s, A, grow, W, info);
  prof_end(K_PAGES_PLAN, s);
  if (e != cudaSuccess) return FM_ERR_CUDA;
  const int64_t items = static_cast<int64_t>(c->B) * c->layers * 2;
  prof_begin(K_PAGES_COPY, s);
  const dim3 grid(items < copy_grid() ? static_cast<int>(items) : copy_grid());
  const Pools pools = pools_of(*c, k_pool, v_pool, k_scale, v_scale);
  e = k_scale ? launch_dependent(reserve_copy_kernel<true>, grid, kCopyThreads, 0, s, pools, W.copy, c->B, c->layers)
              : launch_dependent(reserve_copy_kernel<false>, grid, kCopyThreads, 0, s, pools, W.copy, c->B, c->layers);
  prof_end(K_PAGES_COPY, s);
  return done(e);
}

fm_status compact_pages(const fm_cache* c, void* k_pool, void* v_pool, float* k_scale, float* v_scale,
                        const int32_t* table, const int32_t* lens, const int32_t* ref, int32_t* table_out,
                        int32_t* ref_out, int32_t* n_live, void* ws, size_t ws_bytes, int32_t* status,
                        void* stream) {
  fm_status st = check_cache(c, true);
  if (st != FM_OK) return st;
  if (!table || !lens || !ref || !table_out || !ref_out || !n_live) return FM_ERR_INVALID;
  if (!aligned_to(k_pool, 16) || !aligned_to(v_pool, 16)) return FM_ERR_INVALID;
  PageArgs A{table, lens, ref, table_out, nullptr, ref_out, status, c->B, c->page_size, c->n_pages,
             c->max_pages};
  if (!outputs_apart(*c, A)) return FM_ERR_INVALID;
  if (!aligned_to(ws, 256)) return FM_ERR_WORKSPACE;
  const PlanWs W = plan_ws(*c, ws);
  if (ws_bytes < W.bytes) return FM_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  prof_begin(K_PAGES_PLAN, s);
  cudaError_t e = few_pages(*c)
                      ? launch_dependent(compact_kernel<1>, dim3(1), kPlanThreads, 0, s, A, W, n_live)
                      : launch_dependent(compact_kernel<8>, dim3(8), kPlanThreads, 0, s, A, W, n_live);
  prof_end(K_PAGES_PLAN, s);
  if (e != cudaSuccess) return FM_ERR_CUDA;
  prof_begin(K_PAGES_COPY, s);
  const Pools pools = pools_of(*c, k_pool, v_pool, k_scale, v_scale);
  e = k_scale ? launch_dependent(compact_copy_kernel<true>, dim3(copy_grid()), kCopyThreads, 0, s, pools, A, W, c->layers)
              : launch_dependent(compact_copy_kernel<false>, dim3(copy_grid()), kCopyThreads, 0, s, pools, A, W, c->layers);
  prof_end(K_PAGES_COPY, s);
  return done(e);
}

}  // namespace
}  // namespace fm

using namespace fm;

extern "C" {

fm_status fm_cache_append(const fm_cache* c, const void* k, const void* v, const int64_t* k_stride,
                          const int64_t* v_stride, const int32_t* cu, int total, void* k_pool,
                          void* v_pool, const int32_t* table, const int32_t* lens, int32_t* status,
                          void* stream) {
  fm_status st = check_cache(c, true);
  if (st != FM_OK) return st;
  if (!k_stride || !v_stride || !cu || !table || !lens || total < 1) return FM_ERR_INVALID;
  if (!aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(k_pool, 16) || !aligned_to(v_pool, 16))
    return FM_ERR_INVALID;
  for (const int64_t* s : {k_stride, v_stride})
    for (int i = 0; i < 2; ++i)
      if (s[i] <= 0 || s[i] % 8 != 0 || s[i] >= (int64_t(1) << 36)) return FM_ERR_INVALID;
  Pools P = pools_of(*c, k_pool, v_pool);
  AppendArgs A;
  A.src[0] = static_cast<const uint4*>(k);
  A.src[1] = static_cast<const uint4*>(v);
  A.tok[0] = k_stride[0] / 8; A.head[0] = k_stride[1] / 8;
  A.tok[1] = v_stride[0] / 8; A.head[1] = v_stride[1] / 8;
  A.cu = cu; A.table = table; A.lens = lens; A.status = status;
  A.B = c->B; A.total = total; A.max_pages = c->max_pages; A.n_pages = c->n_pages;
  // the vectors that a block's threads hold, in more blocks where there are few
  int tokens = kAppendVecs * kAppendThreads / (2 * P.row);
  if (tokens < 1) tokens = 1;
  while (tokens > 1 && ceil_div(total, tokens) < 2 * num_sms()) tokens = (tokens + 1) / 2;
  A.tokens = tokens;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  prof_begin(K_CACHE_APPEND, s);
  const cudaError_t e = launch_dependent(append_kernel, dim3(ceil_div(total, tokens)), kAppendThreads,
                                         tokens * sizeof(int64_t), s, A, P);
  prof_end(K_CACHE_APPEND, s);
  return done(e);
}

fm_status fm_cache_accept(const fm_cache* c, const int32_t* accept, int max_accept,
                          const int32_t* n_accept, const int32_t* cu, void* k_pool, void* v_pool,
                          const int32_t* table, const int32_t* lens, int32_t* lens_out, int32_t* ref,
                          int32_t* status, void* stream) {
  fm_status st = check_cache(c, true);
  if (st != FM_OK) return st;
  if (!accept || max_accept < 1 || !n_accept || !cu || !table || !lens || !lens_out)
    return FM_ERR_INVALID;
  if (!aligned_to(k_pool, 16) || !aligned_to(v_pool, 16)) return FM_ERR_INVALID;
  if (overlaps(lens, c->B * 4ull, lens_out, c->B * 4ull)) return FM_ERR_INVALID;
  if (c->B > 65535 || c->layers > 65535) return FM_ERR_UNSUPPORTED;
  Pools P = pools_of(*c, k_pool, v_pool);
  AcceptArgs A{accept, n_accept, cu, table, lens, lens_out, ref, status, max_accept, c->max_pages,
               c->n_pages};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  prof_begin(K_CACHE_ACCEPT, s);
  const cudaError_t e =
      launch_dependent(accept_kernel, dim3(ceil_div(2 * P.row, kAcceptThreads), c->B, c->layers),
                       kAcceptThreads, 0, s, A, P);
  prof_end(K_CACHE_ACCEPT, s);
  return done(e);
}

fm_status fm_pages_fork(const fm_cache* c, const int32_t* parent, const int32_t* table,
                        const int32_t* lens, const int32_t* ref, int32_t* table_out,
                        int32_t* lens_out, int32_t* ref_out, int32_t* status, void* stream) {
  fm_status st = check_cache(c, false);
  if (st != FM_OK) return st;
  if (!parent || !table || !lens || !ref || !table_out || !lens_out || !ref_out) return FM_ERR_INVALID;
  PageArgs A{table, lens, ref, table_out, lens_out, ref_out, status, c->B, c->page_size, c->n_pages,
             c->max_pages};
  if (table_out == table || lens_out == lens || !outputs_apart(*c, A)) return FM_ERR_INVALID;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  prof_begin(K_PAGES_FORK, s);
  cudaError_t e = cudaSuccess;
  if (ref_out != ref && few_pages(*c)) {
    e = launch_dependent(fork_copy_kernel, dim3(1), 1024, 0, s, A, parent);
    prof_end(K_PAGES_FORK, s);
    return done(e);
  }
  if (ref_out != ref) {
    const int blocks = ceil_div(c->n_pages, 1024);
    e = launch_dependent(ref_copy_kernel, dim3(blocks < 1024 ? blocks : 1024), 256, 0, s, ref, ref_out,
                         c->n_pages);
  }
  if (e == cudaSuccess) e = launch_dependent(fork_kernel, dim3(ceil_div(c->B, 4)), 128, 0, s, A, parent);
  prof_end(K_PAGES_FORK, s);
  return done(e);
}

size_t fm_pages_workspace_size(const fm_cache* c) {
  if (check_cache(c, false) != FM_OK) return 0;
  return plan_ws(*c, nullptr).bytes;
}

fm_status fm_pages_reserve(const fm_cache* c, const int32_t* grow, void* k_pool, void* v_pool,
                           const int32_t* table, const int32_t* lens, const int32_t* ref,
                           int32_t* table_out, int32_t* lens_out, int32_t* ref_out, int32_t* info,
                           void* ws, size_t ws_bytes, int32_t* status, void* stream) {
  return reserve_pages(c, grow, k_pool, v_pool, nullptr, nullptr, table, lens, ref, table_out, lens_out,
                       ref_out, info, ws, ws_bytes, status, stream);
}

fm_status fm_pages_reserve_fp8(const fm_cache* c, const int32_t* grow, void* k_pool, void* v_pool,
                               float* k_scale, float* v_scale, const int32_t* table, const int32_t* lens,
                               const int32_t* ref, int32_t* table_out, int32_t* lens_out, int32_t* ref_out,
                               int32_t* info, void* ws, size_t ws_bytes, int32_t* status, void* stream) {
  const fm_status st = check_cache8(c, k_pool, v_pool, k_scale, v_scale);
  if (st != FM_OK) return st;
  return reserve_pages(c, grow, k_pool, v_pool, k_scale, v_scale, table, lens, ref, table_out, lens_out,
                       ref_out, info, ws, ws_bytes, status, stream);
}

fm_status fm_pages_compact(const fm_cache* c, void* k_pool, void* v_pool, const int32_t* table,
                           const int32_t* lens, const int32_t* ref, int32_t* table_out,
                           int32_t* ref_out, int32_t* n_live, void* ws, size_t ws_bytes,
                           int32_t* status, void* stream) {
  return compact_pages(c, k_pool, v_pool, nullptr, nullptr, table, lens, ref, table_out, ref_out, n_live, ws,
                       ws_bytes, status, stream);
}

fm_status fm_pages_compact_fp8(const fm_cache* c, void* k_pool, void* v_pool, float* k_scale,
                               float* v_scale, const int32_t* table, const int32_t* lens,
                               const int32_t* ref, int32_t* table_out, int32_t* ref_out, int32_t* n_live,
                               void* ws, size_t ws_bytes, int32_t* status, void* stream) {
  const fm_status st = check_cache8(c, k_pool, v_pool, k_scale, v_scale);
  if (st != FM_OK) return st;
  return compact_pages(c, k_pool, v_pool, k_scale, v_scale, table, lens, ref, table_out, ref_out, n_live, ws,
                       ws_bytes, status, stream);
}

}  // extern "C"
