// Attention of drafted trees and single tokens over the paged cache: the
// entry point, the kernel for units of up to 16 rows, and the join of units
// that several blocks worked on.
#include <cfloat>
#include <cmath>

#include "fm_tree8.cuh"

namespace fm {

// ---------------------------------------------------------------- narrow kernel
// Units of up to 16 rows (one token of up to 16 query heads per K/V head, or
// a few nodes).  Bound by reading K and V once: 512 bytes per key and head at
// d = 128 against 8 KFLOP.  Two warps load K and V tiles by TMA through
// rings of tiles; four warps each take 16 keys of every 64-key tile and keep
// their own running maximum, sum and O in registers, so no warp waits for
// another inside a unit.  S and O come from mma.sync (16 x 8 x 16, bf16): its
// fragments leave P in registers as the A operand of the second product, and
// 16 rows fill its M, where a tcgen05.mma would pad them to 128.
// Two blocks share an SM: one's fetching of rows, merging and writing at the
// ends of units runs while the other's tiles stream (one block of twice the
// size took 56 us for 1024 units of three 128-key tiles).
template <int D>
struct NarrowCfg {
  using Geo = NarrowGeo;
  static constexpr int R = Geo::R, KT = Geo::KT;
  static constexpr int WARPS = 4;                  // consumers
  static constexpr int THREADS = 32 * (WARPS + 2);
  static constexpr int TILE = KT * D * 2;          // bytes of a K or V tile
  static constexpr int KS = D == 128 ? 3 : 5, VS = D == 128 ? 2 : 5;   // rings of tiles
  static constexpr int PITCH = D + 8;              // floats of a row of the merge buffer
  static constexpr int OFF_V = KS * TILE;
  static constexpr int OFF_MERGE = OFF_V + VS * TILE;            // [WARPS][R / 2][PITCH]
  static constexpr int OFF_ML = OFF_MERGE + WARPS * R / 2 * PITCH * 4;   // float2 [R][WARPS] max and sum
  static constexpr int OFF_SEEN = OFF_ML + WARPS * R * 8;        // [R] see bits
  static constexpr int OFF_NF = OFF_SEEN + R * 4;                // [2][8] keys with values not finite
  static constexpr int OFF_BAR = OFF_NF + 64;
  static constexpr int OFF_ABORT = OFF_BAR + 2 * (KS + VS) * 8;
  static constexpr int SMEM = OFF_ABORT + 8;
  static_assert(2 * (SMEM + 1024) <= 228 * 1024, "two blocks per SM");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
__global__ void __launch_bounds__(NarrowCfg<D>::THREADS, 2)
    tree_narrow_kernel(const __grid_constant__ TreeParams P, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV) {
  using C = NarrowCfg<D>;
  using Load = TileLoad<D, C::KT>;
  constexpr int R = C::R, KT = C::KT;
  extern __shared__ __align__(1024) uint8_t smem[];
  volatile int& abort_flag = *reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0 && P.status) atomicOr(P.status, DEV_LAYOUT);
    return;
  }
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::OFF_BAR;
  auto full = [&](int i) { return bar0 + 8u * i; };                      // K stages, then V's
  auto empty = [&](int i) { return bar0 + 8u * (C::KS + C::VS + i); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 2) touch_memory<D>(P, lane, blockIdx.x);
  if (tid == 0) {
    for (int i = 0; i < C::KS + C::VS; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), C::WARPS);
    }
    abort_flag = 0;
    fence_barrier_init();
  }
  if (tid < 16) reinterpret_cast<uint32_t*>(smem + C::OFF_NF)[tid] = 0;
  if (warp == C::WARPS && lane == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  grid_launch_dependents();
  grid_dependency_wait();
  TreeWalk<typename C::Geo> u(tree_run<typename C::Geo>(P, blockIdx.x));
  __syncthreads();

  // every lane gets the same answer
  auto wait_all = [&](uint32_t bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, tree_wait(bar, parity, P, &abort_flag));
  };

  if (warp >= C::WARPS) {
    // ------------------------------------------------------------ loads
    // one warp for K, one for V
    const bool isk = warp == C::WARPS;
    const CUtensorMap* tm = isk ? &tmK : &tmV;
    const int stages = isk ? C::KS : C::VS, first = isk ? 0 : C::KS;
    const uint32_t buf = sbase + (isk ? 0 : C::OFF_V);
    const uint64_t policy = policy_evict_first();
    int st = 0, issued = 0;
    uint32_t use = 0;
    bool ok = true;
    while (ok && u.next(P)) {
      if (u.keys == 0) continue;
      int page = Load::lane_page(P, u, u.t0, lane);
#pragma unroll 1
      for (int t = u.t0; t < u.t1; ++t) {
        const int next = t + 1 < u.t1 ? Load::lane_page(P, u, t + 1, lane) : 0;
        if (use > 0) ok = wait_all(empty(first + st), (use - 1) & 1);
        if (!ok) break;
        Load::issue(P, u, t, lane, page, tm, buf + st * C::TILE, full(first + st), policy);
        ++issued;
        if (++st == stages) {
          st = 0;
          ++use;
        }
        page = next;
      }
    }
    // every issued copy has landed before the block may exit
    if (lane == 0)
#pragma unroll 1
      for (int x = max(issued - stages, 0); x < issued; ++x)
        mbar_wait(full(first + x % stages), (x / stages) & 1, P.status, P.wait_ns);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ attention
    // A warp whose wait gave up goes on without waiting or computing: the
    // block-wide merges of every piece still find all four warps.
    bool ok = true;
    uint32_t e = 0;                              // tiles so far
    const int g = lane >> 2, tq = lane & 3;      // fragment row and column pair
    uint32_t* seen = reinterpret_cast<uint32_t*>(smem + C::OFF_SEEN);
    uint32_t* nf_all = reinterpret_cast<uint32_t*>(smem + C::OFF_NF);
    float* merge = reinterpret_cast<float*>(smem + C::OFF_MERGE);
    float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
    uint32_t pieces = 0;
    if (tid == 0) P.rec[blockIdx.x] = make_int4(-1, 0, 0, 0);
    for (; u.next(P); ++pieces) {
      // tiles from this one on hold keys that not every row sees
      const int part0 = u.origin / KT;
      // the next piece's flags, read by nobody now
      uint32_t* nf = nf_all + 8 * (pieces & 1);
      if (tid == 0) nf_all[8 * ((pieces + 1) & 1)] = 0;
      // Q of rows g and g + 8 as A fragments, straight from memory
      uint32_t qf[D / 16][4];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int r = g + 8 * hh;
        const int rr = u.row_first + r;
        const int node = P.by_G(rr);
        const __nv_bfloat16* src = P.q + (u.s.row0 + node) * P.q_stride[0] +
                                   (u.hk * P.G + rr - node * P.G) * P.q_stride[1] + 2 * tq;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          qf[kk][hh] = r < u.rows ? *reinterpret_cast<const uint32_t*>(src + kk * 16) : 0u;
          qf[kk][hh + 2] = r < u.rows ? *reinterpret_cast<const uint32_t*>(src + kk * 16 + 8) : 0u;
        }
      }
      // which keys from origin on row lane & 15 sees: bit i is key origin + i
      // (16 rows are of 16 nodes at most)
      uint32_t bits = 0;
      {
        const int node = P.by_G(u.row_first + min(lane & 15, u.rows - 1));
        if (P.tree) {
          // lane l knows the parent of node l
          const int mine = lane < u.s.n && u.s.base >= 0 ? tree_parent(P, u.s, lane) : -1;
          int a = u.s.base >= 0 ? node : -1;
          while (__any_sync(0xffffffffu, a >= 0)) {
            const int p = __shfl_sync(0xffffffffu, mine, a & 31);
            if (a >= 0 && p != -2) bits |= 1u << a;
            a = a < 0 || p == -2 ? -1 : p;   // a node drafted after a padding node is a root
          }
        } else {
          bits = (2u << (u.s.base + node - u.origin)) - 1u;
        }
      }
      if (tid < R) seen[tid] = bits;    // for values that are not finite
      const uint32_t bits_of[2] = {__shfl_sync(0xffffffffu, bits, g), __shfl_sync(0xffffffffu, bits, g + 8)};
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
      float acc[D / 8][4];
#pragma unroll
      for (int x = 0; x < D / 8; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) acc[x][y] = 0.f;

#pragma unroll 1
      for (int t = u.t0; u.keys > 0 && t < u.t1; ++t) {
        const int ks = e % C::KS, vs = e % C::VS;
        const uint32_t kp = (e / C::KS) & 1, vp = (e / C::VS) & 1;
        ++e;
        const int k0 = t * KT + warp * 16;          // first key of this warp
        const uint32_t sk = sbase + ks * C::TILE, sv = sbase + C::OFF_V + vs * C::TILE;
        const bool mine = k0 < u.keys;                 // any keys at all
        if (ok) ok = wait_all(full(ks), kp);
        float s[2][4];
        if (ok && mine) {
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) s[x][y] = 0.f;
          // matrices of one ldmatrix: keys 0-7 d 0-7, keys 0-7 d 8-15, keys
          // 8-15 d 0-7, keys 8-15 d 8-15
          const int key = warp * 16 + (lane & 7) + ((lane >> 4) << 3);
          const int chunk0 = (lane >> 3) & 1;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t b[4];
            const int ch = kk * 2 + chunk0;
            ldsm4(sk + (ch >> 3) * (KT * 128) + key * 128 + (((ch & 7) ^ (key & 7)) << 4), b);
            mma16816(s[0], qf[kk], b[0], b[1]);
            mma16816(s[1], qf[kk], b[2], b[3]);
          }
        }
        // (a test of the wait limit withholds the first one: the K loader's
        // wait for the stage then runs out)
        if (!(P.withhold == 8 && e == 1)) mbar_arrive_warp(empty(ks));
        uint32_t pf[4], pl[4];
        if (ok && mine) {
          if (t >= part0 || k0 + 16 > u.keys) {
            // keys past origin: only what the row sees; bit i of vis is key k0 + i
            const int j0 = k0 - u.origin;
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const uint32_t vis = j0 >= 16 ? 0u
                                   : j0 >= 0 ? bits_of[hh] >> j0
                                   : j0 > -16 ? bits_of[hh] << -j0 | ((1u << -j0) - 1u)
                                              : 0xffffu;
#pragma unroll
              for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y)
                  if (!((vis >> (x * 8 + 2 * tq + y)) & 1u)) s[x][2 * hh + y] = -INFINITY;
            }
          }
          bool grow = false;
          float alpha[2], ref[2];
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            float mx = fmaxf(fmaxf(s[0][2 * hh], s[0][2 * hh + 1]),
                             fmaxf(s[1][2 * hh], s[1][2 * hh + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            mx *= P.scale_log2;
            // the reference moves only when the maximum grows by more than
            // 2^8: until then P stays in range and nothing is rescaled
            const bool up = mx > m[hh] + 8.f;
            alpha[hh] = up ? ex2(m[hh] - mx) : 1.f;
            m[hh] = up ? mx : m[hh];
            ref[hh] = m[hh] == -INFINITY ? 0.f : m[hh];
            grow |= up;
          }
          if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int x = 0; x < D / 8; ++x)
#pragma unroll
              for (int y = 0; y < 4; ++y) acc[x][y] *= alpha[y >> 1];
            l[0] *= alpha[0];
            l[1] *= alpha[1];
          }
          float p[2][4];
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              p[x][y] = ex2(fmaf(s[x][y], P.scale_log2, -ref[y >> 1]));
              l[y >> 1] += p[x][y];
            }
          // P as the sum of two bf16 numbers (16 bits of mantissa): with one,
          // its rounding is as large an error of O as the rounding of the
          // output, and the tensor cores have the time here.  Both are
          // positive wherever P is, so that an infinity of V in the context
          // stays one: the first is P cut off, never rounded up, and the
          // second at least the smallest bf16 number.
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              float lo[2];
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const float w = p[x][2 * hh + y];
                const float cut = __uint_as_float(__float_as_uint(w) & 0xffff0000u);
                lo[y] = fminf(w, fmaxf(w - cut, __uint_as_float(0x00010000u)));
              }
              pf[2 * x + hh] =
                  __byte_perm(__float_as_uint(p[x][2 * hh]), __float_as_uint(p[x][2 * hh + 1]), 0x7632);
              pl[2 * x + hh] = pack_bf16(lo[0], lo[1]);
            }
        }
        if (ok) ok = wait_all(full(C::KS + vs), vp);
        if (ok && mine) {
          if (t >= part0 || k0 + 16 > u.keys) {
            // this warp's 16 rows of V: zeros past the unit's keys, and clean
            // where not every row sees the key
            const int row = warp * 16 + (lane >> 1);
            const int key = k0 + (lane >> 1), j = key - u.origin;
            auto word = [&](int c) {
              const int ch = (lane & 1) * (D / 16) + c;
              return reinterpret_cast<uint4*>(smem + C::OFF_V + vs * C::TILE + (ch >> 3) * (KT * 128) +
                                              row * 128 + (((ch & 7) ^ (row & 7)) << 4));
            };
            bool dirty = false;
            if (key >= u.keys) {
#pragma unroll
              for (int c = 0; c < D / 16; ++c) *word(c) = make_uint4(0u, 0u, 0u, 0u);
            } else if (j >= 0) {
              uint32_t zero = 0;               // 0, or NaN once a value was not finite
#pragma unroll
              for (int c = 0; c < D / 16; ++c) {
                const uint4 x = *word(c);
                zero = bf16x2_times_zero(x.x, zero);
                zero = bf16x2_times_zero(x.y, zero);
                zero = bf16x2_times_zero(x.z, zero);
                zero = bf16x2_times_zero(x.w, zero);
              }
              dirty = bf16x2_not_finite(zero);
            }
            if (dirty) {
              atomicOr(nf, 1u << j);
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint4* x = word(c);
                *x = make_uint4(bf16x2_clean(x->x), bf16x2_clean(x->y), bf16x2_clean(x->z), bf16x2_clean(x->w));
              }
            }
            fence_proxy_async_smem();   // before the next copy into this slot
            __syncwarp();
          }
          // matrices: keys 0-7 d 0-7, keys 8-15 d 0-7, keys 0-7 d 8-15, keys 8-15 d 8-15
          const int row = warp * 16 + (lane & 15);
          const int chunk0 = lane >> 4;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t b[4];
            const int ch = kk * 2 + chunk0;
            ldsm4_t(sv + (ch >> 3) * (KT * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4), b);
            mma16816(acc[2 * kk], pf, b[0], b[1]);
            mma16816(acc[2 * kk + 1], pf, b[2], b[3]);
            mma16816(acc[2 * kk], pl, b[0], b[1]);
            mma16816(acc[2 * kk + 1], pl, b[2], b[3]);
          }
        }
        mbar_arrive_warp(empty(C::KS + vs));
      }

      // ---------------------------------------------------------- merge the four warps
      // Each warp's maxima, sums and O as they are to shared memory, eight rows
      // at a time; then a thread adds four columns of a row.
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 1);
        l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 2);
        // a padding node's row sees nothing, the context included
        const bool dead = P.tree && bits_of[hh] == 0;
        if (tq == 0)
          ml[(g + 8 * hh) * C::WARPS + warp] =
              dead ? make_float2(-INFINITY, 0.f) : make_float2(m[hh], l[hh]);
      }
#pragma unroll 1
      for (int r0 = 0; r0 < u.rows; r0 += 8) {
        if (r0 > 0) named_sync(1, 32 * C::WARPS);       // the first eight rows have been read
#pragma unroll
        for (int x = 0; x < D / 8; ++x)
          *reinterpret_cast<float2*>(merge + (warp * 8 + g) * C::PITCH + x * 8 + 2 * tq) =
              r0 ? make_float2(acc[x][2], acc[x][3]) : make_float2(acc[x][0], acc[x][1]);
        named_sync(1, 32 * C::WARPS);
        const bool any = *nf != 0;
#pragma unroll 1
        for (int i = tid; i < min(u.rows - r0, 8) * (D / 4); i += 32 * C::WARPS) {
          const int rl = i / (D / 4), c = i % (D / 4) * 4, r = r0 + rl;
          float2 w[C::WARPS];
          float mm = -INFINITY, ll = 0.f;
#pragma unroll
          for (int k = 0; k < C::WARPS; ++k) {
            w[k] = ml[r * C::WARPS + k];
            mm = fmaxf(mm, w[k].x);
          }
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < C::WARPS; ++k) {
            const float4 y = *reinterpret_cast<const float4*>(merge + (k * 8 + rl) * C::PITCH + c);
            if (w[k].y != 0.f) {        // 0: that warp's keys were not seen
              const float f = ex2(w[k].x - mm);
              ll += w[k].y * f;
              v.x += y.x * f;
              v.y += y.y * f;
              v.z += y.z * f;
              v.w += y.w * f;
            }
          }
          const uint4 none = make_uint4(0u, 0u, 0u, 0u);
          if (u.whole()) {
            const int rr = u.row_first + r, node = P.by_G(rr), h = u.hk * P.G + rr - node * P.G;
            const float inv = ll > 0.f ? 1.f / ll : ll;     // 0 or NaN as it is
            __nv_bfloat16* dst = P.o + (u.s.row0 + node) * P.o_stride[0] + h * P.o_stride[1] + c;
            *reinterpret_cast<uint2*>(dst) =
                make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
            if (any) fix_row(P, u.b, u.hk, u.origin, nf, make_uint4(seen[r], 0u, 0u, 0u), none, c, 4, dst);
            if (c == 0)
              P.lse[static_cast<int64_t>(h) * P.total + u.s.row0 + node] =
                  ll > 0.f || ll != ll ? (mm + __log2f(ll)) * 0.69314718055994530942f : -INFINITY;
          } else {
            const int64_t at = static_cast<int64_t>(2 * blockIdx.x + (u.t0 == 0 ? 1 : 0)) * P.part_rows + r;
            float* dst = P.part_o + at * D + c;
            *reinterpret_cast<float4*>(dst) = v;
            if (any) fix_row(P, u.b, u.hk, u.origin, nf, make_uint4(seen[r], 0u, 0u, 0u), none, c, 4, dst);
            if (c == 0) P.part_ml[at] = make_float2(mm, ll);
          }
        }
      }
      if (tid == 0) leave_record(P, u, blockIdx.x);
      named_sync(1, 32 * C::WARPS);     // ml, merge, seen and nf have been read
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------- join
// A unit that block c starts and does not finish has parts in slot 2 c + 1
// and in slot 2 x of the blocks x after it up to the one that finishes it
// (rec.w == 1).  For each row: the maximum of the parts' maxima, then their
// sums and O weighted by 2^(m - maximum).  The blocks of a unit (one column of
// the grid for every block that it runs through but the last) share its rows;
// where there are more warps than rows, 2, 4 or 8 warps share a row, each
// taking every second, fourth or eighth part (76 parts of two units took 33 us
// with a warp a row).  The order of the sums depends on the cuts only.
constexpr int kJoinThreads = 256, kMaxJoin = 4096;   // blocks of the first kernel

template <int R, int D>
__global__ void __launch_bounds__(kJoinThreads)
    tree_join_kernel(const __grid_constant__ TreeParams P, int blocks) {
  constexpr int NW = kJoinThreads / 32, CPT = D / 32, RPW = R == NarrowGeo::R ? 2 : 4;
  __shared__ float sums[NW][D + 2];
  __shared__ unsigned middle[kMaxJoin / 32];
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // bit x: block x is in the middle of a unit
#pragma unroll 1
  for (int i = warp; i * 32 < blocks; i += NW) {
    const int x = i * 32 + lane;
    const unsigned mid = __ballot_sync(0xffffffffu, x < blocks && P.rec[x].w == 2);
    if (lane == 0) middle[i] = mid;
  }
  __syncthreads();
  // the unit: opened by the nearest block c at or before this one that is not
  // in the middle of one, and finished by the next such block
  int c = blockIdx.x, last = blockIdx.x + 1;
#pragma unroll 1
  while (c > 0 && ((middle[c >> 5] >> (c & 31)) & 1u)) {
    const unsigned below = ~middle[c >> 5] & ((1u << (c & 31)) - 1u);
    c = below ? (c & ~31) + 31 - __clz(below) : (c & ~31) - 1;
  }
#pragma unroll 1
  while (last < blocks - 1 && ((middle[last >> 5] >> (last & 31)) & 1u)) {
    const unsigned above = ~middle[last >> 5] & ~((2u << (last & 31)) - 1u);
    last = above ? (last & ~31) + __ffs(above) - 1 : (last & ~31) + 32;
  }
  last = min(last, blocks - 1);
  const int4 rec = P.rec[c];
  if (rec.x < 0) return;
  const TreeSeq s = tree_seq(P, rec.x);
  const int row_first = rec.z * R, rows = min(R, s.n * P.G - row_first), parts = last - c + 1;
  // the blocks in the middle of the unit (in [c, last)) take rows of it too
  const int first = blockIdx.y * (last - c) + blockIdx.x - c, step = (last - c) * gridDim.y;
  // part i of the unit is in slot 2 (c + i), the first in slot 2 c + 1
  const float* po = P.part_o + static_cast<int64_t>(2 * c) * P.part_rows * D + lane * CPT;
  const float2* pm = P.part_ml + 2 * c * P.part_rows;
  auto at = [&](int i, int r) -> int { return (i ? 2 * i : 1) * P.part_rows + r; };
  auto load = [&](int i, int r, float (&y)[CPT]) {
    const float* src = po + at(i, r) * D;
    if constexpr (CPT == 4) {
      const float4 z = *reinterpret_cast<const float4*>(src);
      y[0] = z.x; y[1] = z.y; y[2] = z.z; y[3] = z.w;
    } else {
      const float2 z = *reinterpret_cast<const float2*>(src);
      y[0] = z.x; y[1] = z.y;
    }
  };
  auto write = [&](int r, float mm, float ll, const float (&v)[CPT]) {
    const int rr = row_first + r, node = P.by_G(rr), h = rec.y * P.G + rr - node * P.G;
    const float inv = ll > 0.f ? 1.f / ll : 0.f;
    uint32_t w[CPT / 2];
#pragma unroll
    for (int i = 0; i < CPT / 2; ++i)
      w[i] = ll == 0.f ? 0u : pack_bf16(v[2 * i] * inv, v[2 * i + 1] * inv);
    __nv_bfloat16* dst = P.o + (s.row0 + node) * P.o_stride[0] + h * P.o_stride[1] + lane * CPT;
    if constexpr (CPT == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(dst) = w[0];
    if (lane == 0)
      P.lse[static_cast<int64_t>(h) * P.total + s.row0 + node] =
          ll > 0.f || ll != ll ? (mm + __log2f(ll)) * 0.69314718055994530942f : -INFINITY;
  };

  // warps per row
  int wpr = 1;
#pragma unroll 1
  while (wpr < NW && 2 * wpr <= parts &&
         (parts > 32 * wpr || rows * 2 * wpr <= (last - c) * static_cast<int>(gridDim.y) * NW))
    wpr *= 2;
  if (wpr == 1) {
    // a warp joins RPW rows at a time, to have their loads in flight together
    // (one row at a time left the parts of 150 units at 3 TB/s)
#pragma unroll 1
    for (int r0 = (first * NW + warp) * RPW; r0 < rows; r0 += step * NW * RPW) {
      float mm[RPW], f[RPW], ll[RPW], v[RPW][CPT];
      unsigned seen[RPW];
      // lane i: maximum and sum of part i; a sum of 0 says that its keys were
      // not seen
      float2 p[RPW];
#pragma unroll
      for (int k = 0; k < RPW; ++k)
        p[k] = lane < parts && r0 + k < rows ? pm[at(lane, r0 + k)] : make_float2(-INFINITY, 0.f);
      // and, at the same time, the first two parts' rows (there are two at least)
      float y0[RPW][CPT], y1[RPW][CPT];
#pragma unroll
      for (int k = 0; k < RPW; ++k)
        if (r0 + k < rows) {
          load(0, r0 + k, y0[k]);
          load(1, r0 + k, y1[k]);
        }
#pragma unroll
      for (int k = 0; k < RPW; ++k) {
        mm[k] = p[k].x;
#pragma unroll
        for (int o = 16; o; o >>= 1) mm[k] = fmaxf(mm[k], __shfl_xor_sync(0xffffffffu, mm[k], o));
        f[k] = p[k].y != 0.f ? ex2(p[k].x - mm[k]) : 0.f;
        seen[k] = __ballot_sync(0xffffffffu, p[k].y != 0.f);
        ll[k] = p[k].y != 0.f ? p[k].y * f[k] : 0.f;
#pragma unroll
        for (int o = 16; o; o >>= 1) ll[k] += __shfl_xor_sync(0xffffffffu, ll[k], o);
#pragma unroll
        for (int x = 0; x < CPT; ++x) v[k][x] = 0.f;
      }
      auto add = [&](int i, const float (&y)[RPW][CPT]) {
#pragma unroll
        for (int k = 0; k < RPW; ++k) {
          const float w = __shfl_sync(0xffffffffu, f[k], i);
          if ((seen[k] >> i) & 1u)
#pragma unroll
            for (int x = 0; x < CPT; ++x) v[k][x] += y[k][x] * w;
        }
      };
      add(0, y0);
      add(1, y1);
#pragma unroll 1
      for (int i = 2; i < parts; ++i) {
#pragma unroll
        for (int k = 0; k < RPW; ++k)
          if (r0 + k < rows) load(i, r0 + k, y0[k]);
        add(i, y0);
      }
#pragma unroll
      for (int k = 0; k < RPW; ++k)
        if (r0 + k < rows) write(r0 + k, mm[k], ll[k], v[k]);
    }
    return;
  }

  const int team = warp / wpr, sub = warp % wpr, teams = NW / wpr;
#pragma unroll 1
  for (int r0 = first * teams; r0 < rows; r0 += step * teams) {
    const int r = r0 + team;
    float mm = -INFINITY, ll = 0.f, v[CPT];
#pragma unroll
    for (int i = 0; i < CPT; ++i) v[i] = 0.f;
    if (r < rows) {
#pragma unroll 1
      for (int i0 = sub; i0 < parts; i0 += 32 * wpr) {
        // lane j: maximum and sum of part i0 + j * wpr; a sum of 0 says that
        // its keys were not seen
        const int mine = i0 + lane * wpr;
        const float2 p = mine < parts ? pm[at(mine, r)] : make_float2(-INFINITY, 0.f);
        float m = p.x;
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        m = fmaxf(m, mm);
        const float old = mm == -INFINITY ? (ll == 0.f ? 0.f : 1.f) : ex2(mm - m);
        mm = m;
        const float f = p.y != 0.f ? ex2(p.x - m) : 0.f;
        const unsigned seen = __ballot_sync(0xffffffffu, p.y != 0.f);
        float l = p.y != 0.f ? p.y * f : 0.f;
#pragma unroll
        for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        ll = ll * old + l;
#pragma unroll
        for (int x = 0; x < CPT; ++x) v[x] *= old;
        const int n = min(32, (parts - i0 + wpr - 1) / wpr);
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
          float y[CPT];
          load(i0 + j * wpr, r, y);
          const float w = __shfl_sync(0xffffffffu, f, j);
          if ((seen >> j) & 1u)
#pragma unroll
            for (int x = 0; x < CPT; ++x) v[x] += y[x] * w;
        }
      }
    }
    __syncthreads();                   // the rows before have been read
#pragma unroll
    for (int x = 0; x < CPT; ++x) sums[warp][lane * CPT + x] = v[x];
    if (lane == 0) {
      sums[warp][D] = ll;
      sums[warp][D + 1] = mm;
    }
    __syncthreads();
    if (sub > 0 || r >= rows) continue;
    float top = mm;
#pragma unroll 1
    for (int w = 1; w < wpr; ++w) top = fmaxf(top, sums[warp + w][D + 1]);
    float total = 0.f;
#pragma unroll
    for (int x = 0; x < CPT; ++x) v[x] = 0.f;
#pragma unroll 1
    for (int w = 0; w < wpr; ++w) {
      const float* from = sums[warp + w];
      if (from[D] == 0.f) continue;    // nothing seen
      const float f = ex2(from[D + 1] - top);
      total += from[D] * f;
#pragma unroll
      for (int x = 0; x < CPT; ++x) v[x] += from[lane * CPT + x] * f;
    }
    write(r, top, total, v);
  }
}

template <int R, int D>
static fm_status launch_join(const TreeParams& P, int grid, cudaStream_t s) {
  if (grid < 2 || P.whole) return FM_OK;
  if (grid > kMaxJoin) return FM_ERR_UNSUPPORTED;
  // Columns of the grid, for as many units as there can be: one group of rows
  // a warp, or a warp a row where units are in 32 parts or more, which then
  // take eight warps a row.  (Columns for units of two parts throughout left
  // 3 us more between the kernel and the end of the join of two units of 131072
  // keys: their blocks start in turn.)
  const int64_t units = P.B * P.Hkv * ((static_cast<int64_t>(P.max_nodes) * P.G + R - 1) / R);
  const int64_t rows = (units < grid ? units : grid) * P.part_rows;
  const int64_t per_block = units * 32 <= grid ? 1 : kJoinThreads / 32 * (R == NarrowGeo::R ? 2 : 4);
  const int y = static_cast<int>((rows + grid * per_block - 1) / (grid * per_block));
  prof_begin(K_TREE_JOIN, s);
  const cudaError_t e = launch_dependent(
      tree_join_kernel<R, D>, dim3(grid - 1, y), kJoinThreads,
      0, s, P, grid);
  prof_end(K_TREE_JOIN, s);
  return e == cudaSuccess ? FM_OK : FM_ERR_CUDA;
}

fm_status launch_tree_join(const TreeParams& P, int d, int rows, int grid, cudaStream_t s) {
  const bool d64 = d == 64;
  if (rows == NarrowGeo::R)
    return d64 ? launch_join<NarrowGeo::R, 64>(P, grid, s) : launch_join<NarrowGeo::R, 128>(P, grid, s);
  if (rows == MidGeo::R)
    return d64 ? launch_join<MidGeo::R, 64>(P, grid, s) : launch_join<MidGeo::R, 128>(P, grid, s);
  return launch_join<WideGeo::R, 128>(P, grid, s);
}

template <int D>
static fm_status launch_narrow(const TreeParams& P, const CUtensorMap& tk, const CUtensorMap& tv,
                               int grid, cudaStream_t s) {
  using C = NarrowCfg<D>;
  auto kern = tree_narrow_kernel<D>;
  static std::atomic<uint64_t> ready{0};
  const fm_status st = prepare_kernel(kern, C::SMEM, 0, ready);
  if (st != FM_OK) return st;
  prof_begin(K_TREE, s);
  const cudaError_t e = launch_dependent(kern, dim3(grid), C::THREADS, C::SMEM, s, P, tk, tv);
  prof_end(K_TREE, s);
  return e == cudaSuccess ? FM_OK : FM_ERR_CUDA;
}

namespace {

fm_status check_tree(const fm_cache* c, const fm_tree_desc* t) {
  fm_status st = check_cache(c, true);
  if (st != FM_OK) return st;
  if (!t || t->H < 1 || t->H % c->Hkv != 0 || t->total < 1 || t->max_nodes < 1) return FM_ERR_INVALID;
  if (static_cast<int64_t>(t->total) * t->H > kMaxTokenIndex) return FM_ERR_UNSUPPORTED;
  for (const int64_t* s : {t->q_stride, t->o_stride})
    for (int i = 0; i < 2; ++i)
      if (s[i] <= 0 || s[i] % 8 != 0 || s[i] >= (int64_t(1) << 36)) return FM_ERR_INVALID;
  return FM_OK;
}

// Workspace: the blocks' records, then their parts (two each).
enum TreeKind { NARROW, MID, WIDE };
int unit_rows(TreeKind k) { return k == NARROW ? NarrowGeo::R : k == MID ? MidGeo::R : WideGeo::R; }
struct TreeWs {
  TreeKind kind;
  int rows;    // of a part: the largest unit's
  int grid;
  size_t rec, ml, o, bytes;
};
void tree_ws_places(TreeWs& W, int d) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  W.rec = 0;
  W.ml = up(static_cast<size_t>(W.grid) * sizeof(int4));
  W.o = W.ml + up(2ull * W.grid * W.rows * sizeof(float2));
  W.bytes = W.o + 2ull * W.grid * W.rows * d * sizeof(float);
}
TreeWs tree_ws(const fm_cache& c, const fm_tree_desc& t, int sms) {
  const int64_t nodes = t.max_nodes < t.total ? t.max_nodes : t.total, rows = nodes * (t.H / c.Hkv);
  TreeWs W;
  W.rows = rows <= NarrowGeo::R ? NarrowGeo::R
           : rows >= WideGeo::R ? WideGeo::R
                                : (static_cast<int>(rows) + 31) / 32 * 32;
  // The kernel: tiles of 128 rows side by side beat pairs of them with d = 64
  // (64 sequences of 1000 tokens with 150 rows: 70 us against 81), and where
  // the rows of the table hold at most 640 tokens, so that a unit's ends are
  // most of it (512 units of 256 rows and 164 keys: 46 us against 56, 544 keys
  // 75 and 76, 1064 keys 103 and 92)
  const int64_t tokens = static_cast<int64_t>(c.max_pages) * c.page_size;
  const bool pairs = c.d == 128 && tokens > 640;
  // More rows than 16 on the kernel for 16, which reads K and V again for each
  // 16 but starts sooner, where it is little: one tree of 8 nodes of 4 heads
  // over 2000 tokens took 12.3 us so and 18.4 by 128 rows, 16 over 250 11.4
  // and 12.4, 32 over 250 18.4 and 13.5, 8 over 2000 23.8 and 22.4.  (Up to 16
  // nodes: what a row sees is held in 16 bits.  Not where units of up to 512
  // tokens are left whole: 13.8 and 12.7 over 450.)
  const int64_t units = static_cast<int64_t>(c.B) * c.Hkv * ((rows + NarrowGeo::R - 1) / NarrowGeo::R);
  const bool little = nodes <= 16 && units <= 2 * sms && units * tokens <= 80000 && (tokens <= 320 || tokens > 512);
  W.kind = W.rows <= NarrowGeo::R || little ? NARROW : (W.rows <= MidGeo::R || !pairs ? MID : WIDE);
  if (W.kind == NARROW) W.rows = NarrowGeo::R;
  if (W.kind == MID && W.rows > MidGeo::R) W.rows = MidGeo::R;   // of a part
  W.grid = W.kind == WIDE ? sms : 2 * sms;       // by the kernel's blocks per SM
  tree_ws_places(W, c.d);
  return W;
}

// Bytes that suffice for every call of up to these nodes and tokens, whatever
// kernel the other sizes choose: a part for each of two blocks per SM, of the
// rows of a unit, at most 128.  (The kernel for 256 rows has half the blocks.)
size_t tree_ws_bound(const fm_cache& c, const fm_tree_desc& t, int sms) {
  const int64_t nodes = t.max_nodes < t.total ? t.max_nodes : t.total, rows = nodes * (t.H / c.Hkv);
  TreeWs W;
  W.rows = rows <= NarrowGeo::R ? NarrowGeo::R
           : rows >= MidGeo::R  ? MidGeo::R
                                : (static_cast<int>(rows) + 31) / 32 * 32;
  W.grid = 2 * sms;
  tree_ws_places(W, c.d);
  return W.bytes;
}

// The same for a cache of e4m3 codes.
TreeWs tree_ws8(const fm_cache& c, const fm_tree_desc& t, int sms) {
  const int64_t nodes = t.max_nodes < t.total ? t.max_nodes : t.total, rows = nodes * (t.H / c.Hkv);
  TreeWs W;
  const int64_t tokens = static_cast<int64_t>(c.max_pages) * c.page_size;
  // More than 16 rows on the kernel for 16 where it is little: a tree of 32 rows
  // over 16000 tokens 16.7 us so and 18.6 by 128 rows, over 40000 21.0 and 20.8;
  // 64 rows of 2 heads over 10000 18.0 and 19.4, over 20000 22.6 and 20.1; 128
  // rows of 8 heads over 1200 17.3 and 19.7, over 300 (units left whole) 12.1 and
  // 11.6; 42 sequences of 18 rows of 4 heads over 318 22.3 and 16.0.
  const int64_t units = static_cast<int64_t>(c.B) * c.Hkv * ((rows + NarrowGeo::R - 1) / NarrowGeo::R);
  const bool little = units <= 2 * sms && units * tokens <= 80000 && tokens > 512;
  // Pairs of tiles of 128 rows (d = 128) beat tiles side by side at every length:
  // 512 units of 256 rows and 100, 560 and 980 tokens of context 53, 84 and 101 us
  // against 56, 112 and 142; causal runs of 1920 rows after 100 and 1500 tokens 46
  // and 81 against 56 and 98.
  W.kind = rows <= NarrowGeo::R || little ? NARROW : rows <= MidGeo::R || c.d == 64 ? MID : WIDE;
  W.rows = W.kind == NARROW ? NarrowGeo::R
           : W.kind == WIDE ? (rows >= WideGeo::R ? WideGeo::R : (static_cast<int>(rows) + 31) / 32 * 32)
           : rows >= MidGeo::R ? MidGeo::R
                               : (static_cast<int>(rows) + 31) / 32 * 32;
  W.grid = W.kind == WIDE ? sms : 2 * sms;
  tree_ws_places(W, c.d);
  return W;
}

// k_scale, v_scale: of a cache of e4m3 codes; both null with a cache of bf16.
fm_status tree_fwd(const fm_cache* c, const fm_tree_desc* t, const void* q, const void* k_pool,
                   const void* v_pool, const float* k_scale, const float* v_scale,
                   const int32_t* table, const int32_t* lens, const int32_t* cu, const int32_t* parents,
                   float scale, void* o, float* lse, void* ws, size_t ws_bytes, int32_t* status,
                   void* stream) {
  const bool codes = k_scale != nullptr;
  fm_status st = check_tree(c, t);
  if (st != FM_OK) return st;
  if (parents && t->max_nodes > FM_TREE_MAX_NODES) return FM_ERR_UNSUPPORTED;
  if (!aligned_to(q, 16) || !aligned_to(k_pool, 16) || !aligned_to(v_pool, 16) || !aligned_to(o, 16))
    return FM_ERR_INVALID;
  if (!table || !lens || !cu || !lse) return FM_ERR_INVALID;
  // masked scores are -inf, the largest score is the largest product, and a
  // masked score times the scale is -inf again
  const float scale_log2 = scale * 1.4426950408889634f;
  if (!(scale_log2 >= FLT_MIN && scale_log2 < INFINITY)) return FM_ERR_INVALID;
  const TreeWs W = codes ? tree_ws8(*c, *t, num_sms()) : tree_ws(*c, *t, num_sms());
  const int grid = W.grid;
  if (!aligned_to(ws, 256) || ws_bytes < W.bytes) return FM_ERR_WORKSPACE;
  // the length of the line of units (an upper bound) is counted in 31 bits
  const double units = static_cast<double>(c->Hkv) *
                       (static_cast<double>(t->total) * (t->H / c->Hkv) / NarrowGeo::R + c->B);
  if (units * (static_cast<double>(c->max_pages) * c->page_size / MidGeo::KT + 10) >= 2147483647.0)
    return FM_ERR_UNSUPPORTED;
  char* w = static_cast<char*>(ws);
  TreeParams P{};
  P.B = c->B; P.H = t->H; P.Hkv = c->Hkv; P.G = t->H / c->Hkv;
  P.total = t->total; P.max_nodes = t->max_nodes;
  P.page_shift = page_shift(c->page_size);
  P.n_pages = c->n_pages; P.max_pages = c->max_pages;
  P.by_G = FastDiv::of(P.G);
  P.by_grid = FastDiv::of(grid);
  P.tree = parents != nullptr;
  // Units are not cut, and the join (3 us after the first kernel) is spared,
  // where the rows of the table hold at most 320 tokens (512 units of 100 keys
  // 11.7 us, cut 15.0; 4096 of 250 keys 116, cut 113), or at most 512 as long as
  // no block has more than two pairs of a sequence and a K/V head (512 units of
  // 64 rows and 400 keys 31.3 us, cut 36.4; 1024 units of 480 keys 48, cut 43).
  // Row tiles are not counted: causal runs of 480 tokens of 32 heads over 8,
  // 15 units a pair, took 28.6, 88 and 284 us for 4, 16 and 64 of them left
  // whole, and 35, 89 and 290 cut.  What the host knows of the lengths is the
  // table's width: one token of 256 keys takes 6.7 us with a table of 272
  // tokens a row and 7.9 with one of 1024 or more.
  const int64_t tokens = static_cast<int64_t>(c->max_pages) * c->page_size;
  P.whole = tokens <= 320 || (tokens <= 512 && static_cast<int64_t>(c->B) * c->Hkv <= 2 * grid);
  P.scale_log2 = scale_log2;
  P.q = static_cast<const __nv_bfloat16*>(q);
  P.o = static_cast<__nv_bfloat16*>(o);
  for (int i = 0; i < 2; ++i) {
    P.q_stride[i] = t->q_stride[i];
    P.o_stride[i] = t->o_stride[i];
  }
  P.lse = lse;
  P.v_pool = static_cast<const __nv_bfloat16*>(v_pool);
  for (int i = 0; i < 3; ++i) P.v_stride[i] = c->v_stride[i + 1];
  P.table = table; P.lens = lens; P.cu = cu; P.parents = parents;
  P.rec = reinterpret_cast<int4*>(w + W.rec);
  P.part_rows = W.rows;
  P.part_ml = reinterpret_cast<float2*>(w + W.ml);
  P.part_o = reinterpret_cast<float*>(w + W.o);
  P.status = status;
  const TestHooks th = test_hooks();
  P.wait_ns = th.wait_ns < 4000000000ull ? static_cast<uint32_t>(th.wait_ns) : 4000000000u;
  P.withhold = th.withhold;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (codes) {
    // a page, or a tile's part of it
    const int box = W.kind != NARROW && c->page_size > MidGeo::KT ? MidGeo::KT : c->page_size;
    P.box_shift = page_shift(box);
    Tree8Params A{P, k_scale, v_scale, static_cast<const uint8_t*>(v_pool)};
    CUtensorMap tk, tv;
    // (tcgen05's V: 64 columns a box, see VTile8)
    if (!make_tmap_pool8(&tk, k_pool, c->n_pages, c->page_size, c->Hkv, c->d, c->k_stride + 1, box, c->d) ||
        !make_tmap_pool8(&tv, v_pool, c->n_pages, c->page_size, c->Hkv, c->d, c->v_stride + 1, box,
                         W.kind == NARROW ? c->d : 64))
      return FM_ERR_CUDA;
    const int64_t rows = static_cast<int64_t>(t->max_nodes < t->total ? t->max_nodes : t->total) * P.G;
    if (W.kind == MID) st = launch_tree8_mid(A, c->d, tk, tv, grid, s);
    else if (W.kind == WIDE) st = launch_tree8_wide(A, tk, tv, grid, s);
    else st = launch_tree8_narrow(A, c->d, static_cast<int>(rows), tk, tv, grid, s);
    return st != FM_OK ? st : launch_tree_join(P, c->d, unit_rows(W.kind), grid, s);
  }
  // one page of one head, or a tile's part of it, is a box of 64 columns
  const int box = W.kind == WIDE || c->page_size < MidGeo::KT ? c->page_size : MidGeo::KT;
  P.box_shift = page_shift(box);
  // A row of 64 elements is 128 bytes, and the next 128 are mostly another
  // head's: fetched along, they are read twice (64 sequences of 8192 tokens, 8
  // heads, 16 nodes of 4 query heads: 197 us, 148 without; one token 199 and
  // 156).
  const CUtensorMapL2promotion fetch =
      c->d == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  CUtensorMap tk, tv;
  if (!make_tmap_bshd(&tk, k_pool, c->n_pages, c->page_size, c->Hkv, c->d, c->k_stride + 1, box, 1, fetch) ||
      !make_tmap_bshd(&tv, v_pool, c->n_pages, c->page_size, c->Hkv, c->d, c->v_stride + 1, box, 1, fetch))
    return FM_ERR_CUDA;
  // Q of 128 rows of a unit: the G heads of 128 / G nodes
  CUtensorMap tq = tk;
  P.q_tma = W.kind == WIDE && 128 % P.G == 0;
  if (P.q_tma) {
    const int64_t st[3] = {8, t->q_stride[0], t->q_stride[1]};
    if (!make_tmap_bshd(&tq, q, 1, t->total, t->H, c->d, st, 128 / P.G, P.G)) return FM_ERR_CUDA;
  }
  if (W.kind == NARROW) st = c->d == 64 ? launch_narrow<64>(P, tk, tv, grid, s) : launch_narrow<128>(P, tk, tv, grid, s);
  else if (W.kind == MID) st = launch_tree_mid(P, c->d, tq, tk, tv, grid, s);
  else st = launch_tree_wide(P, tq, tk, tv, grid, s);
  if (st != FM_OK) return st;
  return launch_tree_join(P, c->d, unit_rows(W.kind), grid, s);
}

}  // namespace
}  // namespace fm

using namespace fm;

extern "C" {

size_t fm_tree_workspace_size(const fm_cache* c, const fm_tree_desc* t) {
  if (check_tree(c, t) != FM_OK) return 0;
  return tree_ws_bound(*c, *t, num_sms());
}

fm_status fm_tree_fwd(const fm_cache* c, const fm_tree_desc* t, const void* q, const void* k_pool,
                      const void* v_pool, const int32_t* table, const int32_t* lens,
                      const int32_t* cu, const int32_t* parents, float scale, void* o, float* lse,
                      void* ws, size_t ws_bytes, int32_t* status, void* stream) {
  return tree_fwd(c, t, q, k_pool, v_pool, nullptr, nullptr, table, lens, cu, parents, scale, o, lse, ws,
                  ws_bytes, status, stream);
}

fm_status fm_tree_fwd_fp8(const fm_cache* c, const fm_tree_desc* t, const void* q, const void* k_pool,
                          const void* v_pool, const float* k_scale, const float* v_scale,
                          const int32_t* table, const int32_t* lens, const int32_t* cu,
                          const int32_t* parents, float scale, void* o, float* lse, void* ws,
                          size_t ws_bytes, int32_t* status, void* stream) {
  const fm_status st = check_cache8(c, k_pool, v_pool, k_scale, v_scale);
  if (st != FM_OK) return st;
  return tree_fwd(c, t, q, k_pool, v_pool, k_scale, v_scale, table, lens, cu, parents, scale, o, lse, ws,
                  ws_bytes, status, stream);
}

}  // extern "C"
