// Appending with the position rotation, to a cache of bf16 or of e4m3 codes,
// and keeping the accepted nodes of a tree in a cache of e4m3 codes.
//
// A cache of codes holds, for every 16 tokens of a head (a block), 16 * d
// codes and one scale; a value is code * scale.
#include <cuda_bf16.h>

#include "fm_cache.h"
#include "fm_fp8.cuh"

namespace fm {
namespace {

// K or V: its new tokens, its pool (16-byte vectors' units: elements) and scales.
struct Side {
  const __nv_bfloat16* src;
  int64_t tok, head;                     // of src, in elements
  void* pool;
  int64_t page, slot, phead;             // of the pool, in elements
  float* scale;                          // null: the pool holds bf16
};

// ------------------------------------------------------------------ angles
// The angle of position p at frequency f (radians a position) is p f mod 2
// pi.  It is kept as a 64-bit fraction of a turn: f / 2 pi is cut off to 64
// bits once, and the product with p wraps around like the angle does, exactly
// (2^30 positions on, 2^-34 of a turn is left).  cos and sin come from their
// Taylor series on an eighth of a turn to either side of a quarter's multiple,
// as sums of two floats (off by 2^-27), and are rounded to one float each.
struct Turn {
  float c, s;
};

// f / 2 pi as a fraction of a turn, cut off to 64 bits: f is m 2^e with 24 bits of m,
// and 2^128 / 2 pi times m has the bits that are wanted from 64 - e on.  (In
// integers: with doubles, of which an SM does two a cycle, 16 trees of 64 nodes took
// 8.25 us instead of 7.37.)
__device__ __forceinline__ uint64_t turn_step(float f) {
  const uint32_t bits = __float_as_uint(f), top = (bits >> 23) & 0xff;
  const uint32_t m = (bits & 0x7fffff) | (top ? 0x800000 : 0);
  const int e = static_cast<int>(top ? top : 1) - 150;
  const uint64_t p0 = 0x7d4d3770ull * m, p1 = 0x7f09d5f4ull * m + (p0 >> 32);
  const uint64_t p2 = 0x9391054aull * m + (p1 >> 32), p3 = 0x28be60dbull * m + (p2 >> 32);
  uint64_t step;
  if (e > -32) {                             // f of 2^-8 and more
    const uint64_t high = (p3 << 32) | (p2 & 0xffffffffu), low = (p1 << 32) | (p0 & 0xffffffffu);
    if (e < 0) step = (high >> -e) | ((p3 >> 32) << (64 + e));
    else if (e == 0) step = high;
    else step = e < 64 ? (high << e) | (low >> (64 - e)) : low << (e - 64);
  } else {
    step = e > -96 ? p3 >> (-32 - e) : 0;
  }
  return bits >> 31 ? 0 - step : step;
}

__device__ __forceinline__ Turn turn_of(int64_t pos, uint64_t step) {
  const uint64_t x = static_cast<uint64_t>(pos) * step + (1ull << 61);
  const int quarter = static_cast<int>(x >> 62);
  const int64_t r = static_cast<int64_t>(x & ((1ull << 62) - 1)) - (1ll << 61);   // of 2^64: +- 1/8
  // angle th + tl from the first 24 bits and the next 24
  constexpr float k1 = 9.36267597e-08f, k2 = -2.60540187e-15f;                    // 2 pi / 2^26
  const float a = static_cast<float>(static_cast<int>(r >> 38));
  const float b = static_cast<float>(static_cast<int>((r >> 14) & 0xffffff)) * 0x1p-24f;
  const float u = a * k1, v = b * k1, uv = u + v, low = (u - uv) + v + fmaf(a, k1, -u) + a * k2;
  const float th = uv + low, tl = (uv - th) + low;
  const float zz = th * th, zt = fmaf(th, th, -zz) + 2.f * th * tl, z = zz + zt, zl = (zz - z) + zt;
  // cos = 1 - z / 2 + z^2 / 24 - ...
  float y = fmaf(z, 2.08767559e-9f, -2.755732e-7f);
  y = fmaf(z, y, 2.48015876e-5f);
  y = fmaf(z, y, -1.38888892e-3f);
  y = fmaf(z, y, 4.16666679e-2f) * z * z;
  const float ch = fmaf(-0.5f, z, 1.f);
  const float cl = fmaf(-0.5f, z, 1.f - ch) + fmaf(-0.5f, zl, y);
  // sin = t - t z / 6 + t z^2 / 120 - ...
  y = fmaf(z, -2.50521079e-8f, 2.75573188e-6f);
  y = fmaf(z, y, -1.98412701e-4f);
  y = fmaf(z, y, 8.33333377e-3f) * z * z;
  constexpr float k6 = -0.166666672f, k6l = 4.96705373e-9f;                        // -1/6
  const float m = z * k6, ml = fmaf(z, k6, -m) + fmaf(z, k6l, zl * k6);
  const float p = th * m, pl = fmaf(th, m, -p);
  const float sh = th + p;
  const float sl = (th - sh) + p + pl + fmaf(th, ml + y, tl * fmaf(-0.5f, z, 1.f));
  float c = ch + cl, s = sh + sl;
  if (quarter & 1) {
    const float y = c;
    c = -s;
    s = y;
  }
  return quarter & 2 ? Turn{-c, -s} : Turn{c, s};
}

__device__ __forceinline__ void turn_pair(float& a, float& b, const Turn& t) {
  const float x = fmaf(a, t.c, -b * t.s);
  b = fmaf(b, t.c, a * t.s);
  a = x;
}

// ------------------------------------------------------------------ append
// The unit of work is a block: 16 tokens of the cache that share a scale, all
// heads.  Sequence b's blocks are numbered from cu[b] / 16 + 2 b on, which
// leaves each sequence room enough wherever its first token lies in a block;
// a thread block finds its sequence by a search over cu.  With n new tokens in
// the block, a group of n d / 16 threads (rounded up to a power of two) holds a
// head's new tokens, 16 elements (two vectors of 8) a thread, so that a block's
// largest value is known before any is rounded and K and V are read once.  The
// groups take the heads of q, K and V in turn, each with the next three's loads
// under way; a thread has the same token and elements throughout, and so its
// eight angles in registers.
// Bound by HBM for prompts, by the latency of the lookups for single tokens.  (A
// warp for all of a head's 16 tokens needed 159 registers: one thread block per
// SM, 174 us for 16K tokens of 32 + 2 * 8 heads to codes.)
constexpr int kRotThreads = 256;
// Heads under way, in shared memory: in registers there was room for one (codes)
// or two ahead (16K prompt tokens 93 us and 79 us instead of 75 and 71).  Two
// stages 83 and 74; five 73 and 71, but a batch of single tokens 5.74 us instead
// of 5.62.  Three thread blocks an SM (four without codes): two (three) 76 and 72,
// four (five) with three stages 92 and 90.
constexpr int kRotStages = 4;

__device__ __forceinline__ void copy_async16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

struct RotArgs {
  Side kv[2];
  const __nv_bfloat16* q;
  __nv_bfloat16* q_out;
  int64_t q_stride[2], o_stride[2];
  const float* freqs;
  const int32_t *positions, *cu, *table, *lens;
  int* status;
  int B, total, max_pages, n_pages, page_shift;
  int Hkv, H;                // H: query heads, or 0
  int nrot;                  // rot / 16
  int inter;
};

__device__ __forceinline__ void unpack8(const uint4& x, float* f) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

template <int D, bool CODES>
__global__ void __launch_bounds__(kRotThreads, CODES ? 3 : 4)
    append_rotary_kernel(const __grid_constant__ RotArgs A) {
  constexpr int CH = D / 16;               // chunks of 16 elements of a head
  __shared__ Turn turns[16][8][CH];        // [token][element of the chunk's eight angles][chunk]
  __shared__ uint32_t tops[2][kRotThreads / 32];
  __shared__ uint4 ring[kRotStages][2][kRotThreads];
  grid_launch_dependents();
  grid_dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int max_tokens = A.max_pages << A.page_shift;
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    for (int b = tid; b < A.B; b += kRotThreads) {
      int n;
      if (context_of(A.lens, A.cu, b, A.total, max_tokens, n) < 0) flag(A.status, DEV_CACHE);
    }
  }
  // the last sequence whose first block is at or before this one
  const int me = blockIdx.x;
  int lo = 0;
  for (int n = A.B; n > 1;) {
    const int step = (n + 31) >> 5;
    const int b = lo + lane * step;
    const unsigned below = __ballot_sync(0xffffffffu, lane * step < n && (A.cu[b] >> 4) + 2 * b <= me);
    const int k = 31 - __clz(below | 1u);
    lo += k * step;
    n = min(step, n - k * step);
  }
  int n_new;
  const int base = context_of(A.lens, A.cu, lo, A.total, max_tokens, n_new);
  const int at = me - ((A.cu[lo] >> 4) + 2 * lo);
  if (base < 0 || at < 0 || at > (n_new >> 4) + 1) return;
  const int block = (base >> kScaleShift) + at;              // of the sequence
  const int p0 = max(base, block << kScaleShift);            // its new tokens' places
  const int n = min(base + n_new, (block + 1) << kScaleShift) - p0;
  if (n <= 0) return;
  const int t0 = A.cu[lo] + p0 - base;                       // their packed rows
  const int first = p0 & (kScaleBlock - 1);
  const int pg = A.table[static_cast<int64_t>(lo) * A.max_pages + (p0 >> A.page_shift)];
  const bool in = pg >= 0 && pg < A.n_pages;
  if (!in && tid == 0) flag(A.status, DEV_CACHE);
  const int slot0 = p0 & ((1 << A.page_shift) - 1);

  // groups of threads: token i and chunk c of one head after another
  int size_shift = CH == 8 ? 3 : 2;
  while ((1 << size_shift) < n * CH) ++size_shift;
  const int size = 1 << size_shift, group = tid >> size_shift, member = tid & (size - 1);
  const int i = member / CH, c = member % CH;
  const bool active = i < n;
  const int nrot = A.nrot;
  const bool inter = A.inter != 0, turned = c < nrot;
  // the chunk's two vectors
  const int va = 8 * (inter || !turned ? 2 * c : c), vb = inter || !turned ? va + 8 : va + 8 * nrot;
  // The jobs, a head each: those of K, of V, of q.  The thread blocks of this
  // place and their groups take them in turn.
  const int Hkv = A.Hkv, jobs = 2 * Hkv + A.H;
  const int first_job = blockIdx.y + gridDim.y * group, next_job = gridDim.y * (kRotThreads >> size_shift);
  // This thread's elements of head 0, so that a job multiplies by its head only
  // (a batch of single tokens 5.45 us so, 5.60 with the whole address each time)
  const __nv_bfloat16* k_row = A.kv[0].src + (t0 + i) * A.kv[0].tok + va;
  const __nv_bfloat16* v_row = A.kv[1].src + (t0 + i) * A.kv[1].tok + va;
  const __nv_bfloat16* q_row = A.q + (t0 + i) * A.q_stride[0] + va;
  __nv_bfloat16* o_row = A.q_out + (t0 + i) * A.o_stride[0] + va;
  const int second = vb - va;
  // A thread's own elements, of this head and the next ones, in shared memory:
  // nobody waits for another thread's.
  auto fetch = [&](int job, int stage) {
    if (active && job < jobs) {
      const __nv_bfloat16* src = job >= 2 * Hkv ? q_row + (job - 2 * Hkv) * A.q_stride[1]
                                 : job < Hkv    ? k_row + job * A.kv[0].head
                                                : v_row + (job - Hkv) * A.kv[1].head;
      copy_async16(&ring[stage][0][tid], src);
      copy_async16(&ring[stage][1][tid], src + second);
    }
    copy_async_commit();
  };
  int ahead = first_job;
#pragma unroll
  for (int k = 0; k < kRotStages - 1; ++k) {
    fetch(ahead, k);
    ahead += next_job;
  }

  // the angles
  if (nrot > 0) {
    const int half = 8 * nrot, row = half <= 8 ? 8 : half <= 16 ? 16 : half <= 32 ? 32 : 64;
    const int p = tid & (row - 1);
    if (p < half) {
      const float f = A.freqs[p];
      const float poison = f - f;          // NaN where f is not finite
      const uint64_t turn = turn_step(f);
      for (int k = tid / row; k < n; k += kRotThreads / row) {
        const Turn w = turn_of(A.positions ? A.positions[t0 + k] : p0 + k, turn);
        turns[k][p & 7][p >> 3] = Turn{w.c + poison, w.s + poison};
      }
    }
    __syncthreads();
  }
  Turn w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = active && turned ? turns[i][e][c] : Turn{0.f, 0.f};

  int stage = 0;
  int which = 0;             // of tops: a group's threads are one barrier apart at most
#pragma unroll 1
  for (int job = first_job; job < jobs; job += next_job, ahead += next_job) {
    const int x = job < Hkv ? 0 : job < 2 * Hkv ? 1 : 2;        // K, V, q
    const int head = job - x * Hkv;
    // (into the stage that the head before has been read from)
    fetch(ahead, (stage + kRotStages - 1) % kRotStages);
    copy_async_wait<kRotStages - 1>();
    uint4 a = ring[stage][0][tid], b = ring[stage][1][tid];
    stage = (stage + 1) % kRotStages;
    float f[16];
    const bool rotates = turned && x != 1;
    if (rotates || (CODES && x < 2)) {
      unpack8(a, f);
      unpack8(b, f + 8);
    }
    if (rotates) {
      if (inter) {
#pragma unroll
        for (int e = 0; e < 8; ++e) turn_pair(f[2 * e], f[2 * e + 1], w[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) turn_pair(f[e], f[8 + e], w[e]);
      }
    }
    if (!CODES || x == 2) {
      if (rotates) {
        a = pack8(f);
        b = pack8(f + 8);
      }
      __nv_bfloat16* dst = x == 2 ? o_row + head * A.o_stride[1]
                                  : static_cast<__nv_bfloat16*>(A.kv[x].pool) + pg * A.kv[x].page +
                                        (slot0 + i) * A.kv[x].slot + head * A.kv[x].phead + va;
      if (active && (x == 2 || in)) {
        *reinterpret_cast<uint4*>(dst) = a;
        *reinterpret_cast<uint4*>(dst + second) = b;
      }
    } else {
      const Side& S = A.kv[x];
      float* sp = S.scale + ((static_cast<int64_t>(pg) * Hkv + head) << (A.page_shift - kScaleShift)) +
                  (slot0 >> kScaleShift);
      // (only where the block has tokens is its scale read)
      const float raw = in && first > 0 ? *sp : 0.f;
      uint32_t top = 0;
      if (active) {
        float t4[4];                                         // (a NaN is passed over)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          t4[e] = fmaxf(fmaxf(fabsf(f[e]), fabsf(f[4 + e])), fmaxf(fabsf(f[8 + e]), fabsf(f[12 + e])));
        top = __float_as_uint(fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])));
        if (top >= 0x7f800000u) {                            // the finite ones
          top = 0;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const uint32_t z = __float_as_uint(f[e]) & 0x7fffffffu;
            top = max(top, z < 0x7f800000u ? z : 0u);
          }
        }
      }
      // over the group, all of which has read the scale when its first thread writes
      // the new one
      if (size >= 32) {
        top = __reduce_max_sync(0xffffffffu, top);
        __syncwarp();
        if (size > 32) {
          which ^= 1;
          if (lane == 0) tops[which][warp] = top;
          asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(size) : "memory");
          const int w0 = group << (size_shift - 5);
          for (int o = 0; o < size / 32; ++o) top = max(top, tops[which][w0 + o]);
        }
      } else {
        const unsigned peers = ((1u << size) - 1u) << (lane & ~(size - 1));
        for (int o = 1; o < size; o <<= 1) top = max(top, __shfl_xor_sync(peers, top, o));
        __syncwarp(peers);
      }
      float s = scale_for(__uint_as_float(top));
      uint8_t* pool = static_cast<uint8_t*>(S.pool) + pg * S.page + head * S.phead +
                      static_cast<int64_t>(slot0 - first) * S.slot;      // the block's first token
      if (first > 0) {
        // tokens of the block keep their values: all 16 places but the new
        // ones, which are written below
        const float old = clamp_scale(raw);
        s = fmaxf(s, old);
        if (in && s > old) {
          for (int row = i; row < kScaleBlock; row += size / CH) {
            uint4* at16 = reinterpret_cast<uint4*>(pool + row * S.slot + c * 16);
            if (row < first || row >= first + n) *at16 = rescale_e4m3x16(*at16, old / s);
          }
        }
      }
      if (in && active) {
        if (member == 0) *sp = s;
        const float inv = 1.f / s;         // exact: a power of two, or the caller's own
        uint8_t* dst = pool + (first + i) * S.slot;
#pragma unroll
        for (int e = 0; e < 16; ++e) f[e] *= inv;
        *reinterpret_cast<uint2*>(dst + va) =
            make_uint2(pack_e4m3x4(f[0], f[1], f[2], f[3]), pack_e4m3x4(f[4], f[5], f[6], f[7]));
        *reinterpret_cast<uint2*>(dst + vb) =
            make_uint2(pack_e4m3x4(f[8], f[9], f[10], f[11]), pack_e4m3x4(f[12], f[13], f[14], f[15]));
      }
    }
  }
}

// ------------------------------------------------------------------ accept
// A warp keeps the accepted nodes of one sequence, head and run of layers, K or V: it
// walks the blocks that they go to in ascending order.  Into a block D go
// at most 16 tokens, from D itself or from later blocks; all are loaded before
// one is stored, so a block may be overwritten once it has been done.  D's new
// scale is the largest of its own and those of the blocks that its tokens come
// from: no value grows out of range, and where the scales are equal (most
// trees lie in a few blocks written together) the codes are copied as they
// are.
constexpr int kAccept8Warps = 4;

struct Accept8Args {
  Side kv[2];                  // without sources
  int64_t layer[2];            // of the pools, in elements
  int64_t scale_layer;
  const int32_t *accept, *n_accept, *cu, *table, *lens;
  int32_t *lens_out, *ref;
  int* status;
  int max_accept, max_pages, n_pages, page_shift, Hkv;
  int layers, per_block;       // layers of a thread block
};

template <int D>
__global__ void __launch_bounds__(kAccept8Warps * 32, 8)
    accept8_kernel(const __grid_constant__ Accept8Args A) {
  __shared__ int place[32];            // by place within two blocks: source (page << 8 | slot), -1: none
  __shared__ int dest[2];              // the two blocks' own first tokens
  __shared__ int good;
  grid_launch_dependents();
  grid_dependency_wait();
  const int b = blockIdx.y, layer0 = blockIdx.z * A.per_block, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t* acc = A.accept + static_cast<int64_t>(b) * A.max_accept;
  const int32_t* row = A.table + static_cast<int64_t>(b) * A.max_pages;
  const int m = A.n_accept[b], page = 1 << A.page_shift;
  int n;
  const int base = context_of(A.lens, A.cu, b, 0x7fffffff, A.max_pages << A.page_shift, n);
  const bool sized = base >= 0 && m >= 0 && m <= n && m <= A.max_accept;
  // page << 8 | slot of a position, -1 if its page is out of range
  auto at = [&](int pos) -> int {
    const int pg = row[pos >> A.page_shift];
    return pg >= 0 && pg < A.n_pages ? (pg << 8) | (pos & (page - 1)) : -1;
  };
  auto first_free = [&](int x) { return (base + x + page - 1) >> A.page_shift; };
  // source of entry i, -1: the entry is not valid
  auto look = [&](int i) -> int {
    const int a = acc[i], before = i ? acc[i - 1] : -1;
    if (a <= before || a >= n || at(base + i) < 0) return -1;
    return at(base + a);
  };
  const int skew = base & (kScaleBlock - 1);   // entry i goes to place skew + i of the first block on
  if (threadIdx.x < 32) {
    bool ok = sized;
    place[lane] = -1;
    __syncwarp();
    for (int i = lane; sized && i < m; i += 32) {
      const int from = look(i);
      ok = from >= 0 && ok;
      if (skew + i < 32) {
        place[skew + i] = from;
        if (i == 0 || skew + i == 16) dest[(skew + i) >> 4] = at(base + i) & ~(kScaleBlock - 1);
      }
    }
    // the pages past the new length, as in the accept of a bf16 cache
    if (sized && A.ref)
      for (int j = first_free(m) + lane; j < first_free(n); j += 32) ok = at(j << A.page_shift) >= 0 && ok;
    ok = __all_sync(0xffffffffu, ok);
    if (lane == 0) good = ok;
  }
  __syncthreads();
  const bool ok = good != 0;
  if (blockIdx.x == 0 && layer0 == 0) {
    if (threadIdx.x == 0) {
      A.lens_out[b] = ok ? base + m : A.lens[b];
      if (!ok) flag(A.status, DEV_CACHE);
    }
    if (ok && A.ref)
      for (int j = first_free(m) + threadIdx.x; j < first_free(n); j += blockDim.x) atomicSub(A.ref + row[j], 1);
  }
  if (!ok || m == 0) return;
  const int unit = blockIdx.x * kAccept8Warps + warp, hk = unit >> 1;
  const Side& S = A.kv[unit & 1];
  const bool mine = hk < A.Hkv;
  const int nb_shift = A.page_shift - kScaleShift;
  constexpr int LPR = D / 16, ROWS = 32 / LPR, PASSES = 16 / ROWS;
  const int r = lane / LPR, c = lane % LPR;
  const int layer1 = min(layer0 + A.per_block, A.layers);
  for (int d0 = 0; d0 < skew + m; d0 += kScaleBlock) {       // destination blocks
    if (d0 >= 32 && (d0 & 31) == 0) {                        // the next two blocks' places
      __syncthreads();
      if (threadIdx.x < 32) {
        const int i = d0 + lane - skew;
        place[lane] = i < m ? look(i) : -1;
        if ((lane & 15) == 0 && i < m) dest[lane >> 4] = at(base + i);
      }
      __syncthreads();
    }
    if (!mine) continue;
    const int* from = place + (d0 & 31);
    const int to = dest[(d0 >> 4) & 1];
    const int src = lane < 16 ? from[lane] : -1;
#pragma unroll 1
    for (int layer = layer0; layer < layer1; ++layer) {
      float* scales = S.scale + layer * A.scale_layer;
      auto scale_at = [&](int where) -> float* {
        return scales + (((static_cast<int64_t>(where >> 8) * A.Hkv + hk) << nb_shift) + ((where & 255) >> kScaleShift));
      };
      uint8_t* pool = static_cast<uint8_t*>(S.pool) + layer * A.layer[unit & 1] + hk * S.phead + c * 16;
      auto codes_at = [&](int where) -> uint4* {
        return reinterpret_cast<uint4*>(pool + (where >> 8) * S.page + static_cast<int64_t>(where & 255) * S.slot);
      };
      // the codes that move, and at the same time the scales: lane t < 16 that of
      // token t's source, the others the block's own
      uint4 x[PASSES];
#pragma unroll
      for (int k = 0; k < PASSES; ++k) {
        const int t = k * ROWS + r, w = from[t];
        if (w >= 0 && w != to + t) x[k] = *codes_at(w);
      }
      const float own_raw = *scale_at(to), old = clamp_scale(own_raw);
      const float mine_s = src >= 0 ? clamp_scale(*scale_at(src)) : old;
      const float s = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(mine_s, old))));
      __syncwarp();                                          // all loads before the stores
#pragma unroll
      for (int k = 0; k < PASSES; ++k) {
        const int t = k * ROWS + r, w = from[t];
        const float have = __shfl_sync(0xffffffffu, mine_s, t);
        const bool moves = w >= 0 && w != to + t;
        if (!moves && have == s) continue;
        uint4* here = codes_at(to + t);
        uint4 y = moves ? x[k] : *here;
        if (have != s) y = rescale_e4m3x16(y, have / s);
        *here = y;
      }
      if (lane == 0 && s != own_raw) *scale_at(to) = s;
      __syncwarp();
    }
  }
}

Side side_of(const fm_cache& c, int which, void* pool, float* scale) {
  const int64_t* st = which ? c.v_stride : c.k_stride;
  Side S{};
  S.pool = pool;
  S.page = st[1];
  S.slot = st[2];
  S.phead = st[3];
  S.scale = scale;
  return S;
}

// Heads of packed tokens, [total][heads][d] with the strides of a call (elements of bf16).
struct Rows {
  const void* p;
  int64_t tok, head, heads;
  int64_t in_token(int d) const { return (heads - 1) * head + d; }
  int64_t span(int total, int d) const { return (total - 1) * tok + in_token(d); }
};
Rows rows_of(const void* p, const int64_t* stride, int total, int heads) {
  // what is never stepped along has no stride
  return Rows{p, total > 1 ? stride[0] : 0, heads > 1 ? stride[1] : 0, heads};
}

// a and b share no element, as far as that is found out: where their spans cross
// their token strides must be the same, and their head strides too unless they lie
// side by side in each token (slices of one buffer do).
bool rows_apart(const Rows& a, const Rows& b, int total, int d) {
  if (!overlaps(a.p, 2 * a.span(total, d), b.p, 2 * b.span(total, d))) return true;
  if (a.tok != b.tok) return false;
  const int64_t bytes = static_cast<const char*>(b.p) - static_cast<const char*>(a.p);
  if (bytes % 2 != 0) return false;
  const int64_t delta = bytes / 2, s = a.tok;
  if (s > 0) {           // side by side within a token
    const int64_t off = ((delta % s) + s) % s;
    if (off >= a.in_token(d) && off + b.in_token(d) <= s) return true;
  }
  const int64_t head = a.heads > 1 ? a.head : b.head;
  if (b.heads > 1 && b.head != head) return false;
  // element t s + i head + c of a is element t' s + i' head + c' of b at delta: for each
  // i' - i the nearest t - t'
  for (int64_t i = 1 - a.heads; i < b.heads; ++i) {
    const int64_t x = delta + i * head;
    int64_t t = s > 0 ? (2 * x + (x < 0 ? -s : s)) / (2 * s) : 0;
    t = t < 1 - total ? 1 - total : t > total - 1 ? total - 1 : t;
    const int64_t left = x - t * s;
    if (left < d && left > -d) return false;
  }
  return true;
}

bool stride_ok(const int64_t* s, int n, int unit) {
  for (int i = 0; i < n; ++i)
    if (s[i] <= 0 || s[i] % unit != 0 || s[i] >= (int64_t(1) << 36)) return false;
  return true;
}

}  // namespace

fm_status check_cache8(const fm_cache* c, const void* k_pool, const void* v_pool, const void* k_scale,
                       const void* v_scale) {
  const fm_status st = check_cache(c, true);
  if (st != FM_OK) return st;
  if (!stride_ok(c->k_stride, 4, 16) || !stride_ok(c->v_stride, 4, 16)) return FM_ERR_INVALID;
  if (!aligned_to(k_pool, 16) || !aligned_to(v_pool, 16) || !aligned_to(k_scale, 4) || !aligned_to(v_scale, 4))
    return FM_ERR_INVALID;
  return FM_OK;
}

}  // namespace fm

using namespace fm;

extern "C" {

fm_status fm_cache_append_rotary(const fm_cache* c, const fm_rotary* t, const void* k, const void* v,
                                 const int64_t* k_stride, const int64_t* v_stride, const int32_t* cu,
                                 int total, void* k_pool, void* v_pool, float* k_scale, float* v_scale,
                                 const int32_t* table, const int32_t* lens, int32_t* status,
                                 void* stream) {
  const bool codes = k_scale || v_scale;
  fm_status st = codes ? check_cache8(c, k_pool, v_pool, k_scale, v_scale) : check_cache(c, true);
  if (st != FM_OK) return st;
  if (!t || !k_stride || !v_stride || !cu || !table || !lens || total < 1) return FM_ERR_INVALID;
  if (!aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(k_pool, 16) || !aligned_to(v_pool, 16))
    return FM_ERR_INVALID;
  if (!stride_ok(k_stride, 2, 8) || !stride_ok(v_stride, 2, 8)) return FM_ERR_INVALID;
  if (t->rot < 0 || t->rot > c->d || t->rot % 16 != 0 || (t->rot > 0 && !aligned_to(t->freqs, 4)))
    return FM_ERR_INVALID;
  if (t->H < 0 || t->H % c->Hkv != 0) return FM_ERR_INVALID;
  if (t->H > 0 && (!aligned_to(t->q, 16) || !aligned_to(t->q_out, 16) || !stride_ok(t->q_stride, 2, 8) ||
                   !stride_ok(t->o_stride, 2, 8)))
    return FM_ERR_INVALID;
  if (static_cast<int64_t>(total) * (t->H > c->Hkv ? t->H : c->Hkv) > kMaxTokenIndex) return FM_ERR_UNSUPPORTED;
  const int64_t blocks = total / kScaleBlock + 2 * static_cast<int64_t>(c->B);
  if (blocks > 0x7fffffff) return FM_ERR_UNSUPPORTED;
  if (t->H > 0) {        // other thread blocks read K, V and the queries while one writes its own
    const Rows q = rows_of(t->q, t->q_stride, total, t->H), o = rows_of(t->q_out, t->o_stride, total, t->H);
    const bool in_place = q.p == o.p && q.tok == o.tok && q.head == o.head;
    if ((!in_place && !rows_apart(q, o, total, c->d)) ||
        !rows_apart(rows_of(k, k_stride, total, c->Hkv), o, total, c->d) ||
        !rows_apart(rows_of(v, v_stride, total, c->Hkv), o, total, c->d))
      return FM_ERR_INVALID;
  }
  RotArgs A{};
  A.kv[0] = side_of(*c, 0, k_pool, k_scale);
  A.kv[1] = side_of(*c, 1, v_pool, v_scale);
  A.kv[0].src = static_cast<const __nv_bfloat16*>(k);
  A.kv[1].src = static_cast<const __nv_bfloat16*>(v);
  A.kv[0].tok = k_stride[0]; A.kv[0].head = k_stride[1];
  A.kv[1].tok = v_stride[0]; A.kv[1].head = v_stride[1];
  A.q = static_cast<const __nv_bfloat16*>(t->q);
  A.q_out = static_cast<__nv_bfloat16*>(t->q_out);
  for (int i = 0; i < 2; ++i) {
    A.q_stride[i] = t->q_stride[i];
    A.o_stride[i] = t->o_stride[i];
  }
  A.freqs = t->freqs;
  A.positions = t->positions;
  A.cu = cu; A.table = table; A.lens = lens; A.status = status;
  A.B = c->B; A.total = total; A.max_pages = c->max_pages; A.n_pages = c->n_pages;
  A.page_shift = page_shift(c->page_size);
  A.Hkv = c->Hkv; A.H = t->H;
  A.nrot = t->rot / 16;
  A.inter = t->interleaved != 0;
  // few blocks: the heads are spread over more of them
  int64_t y = (4 * static_cast<int64_t>(num_sms()) + blocks - 1) / blocks;
  if (y > c->Hkv) y = c->Hkv;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(y));
  prof_begin(K_CACHE_APPEND_ROTARY, s);
  auto go = [&](auto kern) { return launch_dependent(kern, grid, kRotThreads, 0, s, A); };
  const cudaError_t e = c->d == 64 ? (codes ? go(append_rotary_kernel<64, true>) : go(append_rotary_kernel<64, false>))
                                   : (codes ? go(append_rotary_kernel<128, true>) : go(append_rotary_kernel<128, false>));
  prof_end(K_CACHE_APPEND_ROTARY, s);
  return done(e);
}

fm_status fm_cache_accept_fp8(const fm_cache* c, const int32_t* accept, int max_accept,
                              const int32_t* n_accept, const int32_t* cu, void* k_pool, void* v_pool,
                              float* k_scale, float* v_scale, const int32_t* table, const int32_t* lens,
                              int32_t* lens_out, int32_t* ref, int32_t* status, void* stream) {
  const fm_status st = check_cache8(c, k_pool, v_pool, k_scale, v_scale);
  if (st != FM_OK) return st;
  if (!accept || max_accept < 1 || !n_accept || !cu || !table || !lens || !lens_out) return FM_ERR_INVALID;
  if (overlaps(lens, c->B * 4ull, lens_out, c->B * 4ull)) return FM_ERR_INVALID;
  if (c->B > 65535 || c->layers > 65535) return FM_ERR_UNSUPPORTED;
  Accept8Args A{};
  A.kv[0] = side_of(*c, 0, k_pool, k_scale);
  A.kv[1] = side_of(*c, 1, v_pool, v_scale);
  A.layer[0] = c->k_stride[0];
  A.layer[1] = c->v_stride[0];
  A.scale_layer = static_cast<int64_t>(c->n_pages) * c->Hkv * (c->page_size / kScaleBlock);
  A.accept = accept; A.n_accept = n_accept; A.cu = cu; A.table = table; A.lens = lens;
  A.lens_out = lens_out; A.ref = ref; A.status = status;
  A.max_accept = max_accept; A.max_pages = c->max_pages; A.n_pages = c->n_pages;
  A.page_shift = page_shift(c->page_size);
  A.Hkv = c->Hkv;
  A.layers = c->layers;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // as many layers a thread block, whose lookups are the same for all, as leave
  // some two rounds of them (64 trees of 8 accepted nodes in 16 layers of 8 heads:
  // 9.3 us so, 9.7 us by a layer each, 14.5 us by eight.  Most of that is blocks
  // whose scale grows and which are written again, 4 KB of traffic each.)
  const int x = ceil_div(2 * c->Hkv, kAccept8Warps);
  const int64_t blocks = static_cast<int64_t>(x) * c->B * c->layers, round = 16ll * num_sms();
  A.per_block = static_cast<int>((blocks + round - 1) / round < c->layers ? (blocks + round - 1) / round : c->layers);
  const dim3 grid(x, c->B, ceil_div(c->layers, A.per_block));
  prof_begin(K_CACHE_ACCEPT, s);
  const cudaError_t e = c->d == 64 ? launch_dependent(accept8_kernel<64>, grid, kAccept8Warps * 32, 0, s, A)
                                   : launch_dependent(accept8_kernel<128>, grid, kAccept8Warps * 32, 0, s, A);
  prof_end(K_CACHE_ACCEPT, s);
  return done(e);
}

}  // extern "C"
