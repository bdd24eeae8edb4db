// Attention over a paged cache of e4m3 codes: the kernel for units of up to 16
// rows.
//
// Bound by reading K and V once, 2 d bytes a key and head.  The products run
// transposed: S^T = K Q^T and O^T = V^T P^T, mma.sync 16 x 8 x 16 with 16 keys
// (or 16 elements of V) as M and 8 rows as N, so that one token of up to 8
// query heads per K/V head wastes nothing on rows that are not there, and O
// takes half the registers.  The codes never become a tile of f16: a lane
// turns them into f16 as it loads its operands.
//  - K: the order of the d elements in S's sum is free, so lane (g, t) of a
//    fragment takes bytes [t d/4, (t + 1) d/4) of keys g and g + 8, whole
//    16-byte words, and Q is loaded in the same order.
//  - V: ldmatrix.trans on pairs of bytes brings a lane the pairs (2g, 2g + 1)
//    of keys 2t and 2t + 1; a byte permutation makes of them two operands, for
//    elements 2g and 2g + 1.
// Two warps load by TMA through rings of 128-key tiles; four warps each take
// two blocks of 16 keys of every tile and keep their own maximum, sum and O,
// so no warp waits for another inside a unit.  Two thread blocks share an SM.
#include "fm_tree8.cuh"

namespace fm {

// HEADS_FIRST: with the blocks numbered as below, the heads of a sequence are
// read at about the same time.  A token's codes of a head are 128 bytes (64),
// and the next heads' follow: a step of 128 sequences of up to 8192 tokens
// (d = 128) takes 270 us so, 279 with a sequence's heads one after another.
struct Narrow8Geo {
  static constexpr bool HEADS_FIRST = true;
  static constexpr int R = 16, KT = 128, LEAST = 2;
  __device__ static __forceinline__ int end(int) { return 2; }
};

template <int D, int NT>
struct Narrow8Cfg {
  using Geo = Narrow8Geo;
  static constexpr int R = Geo::R, KT = Geo::KT;
  static constexpr int WARPS = 4;                  // consumers
  static constexpr int THREADS = 32 * (WARPS + 2);
  static constexpr int TILE = KT * D;              // bytes of a K or V tile
  static constexpr int KS = D == 128 ? 3 : 5, VS = D == 128 ? 2 : 5;   // rings of tiles
  static constexpr int BLOCKS = KT / kScaleBlock;
  static constexpr int PITCH = D + 4;              // floats of a row of the merge buffer
  static constexpr int OFF_V = KS * TILE;
  static constexpr int OFF_MERGE = OFF_V + VS * TILE;            // [WARPS][8][PITCH]
  static constexpr int OFF_ML = OFF_MERGE + WARPS * 8 * PITCH * 4;       // float2 [R][WARPS] max and sum
  static constexpr int OFF_SCALE = OFF_ML + WARPS * R * 8;       // [KS + VS][BLOCKS]
  static constexpr int OFF_SEEN = OFF_SCALE + (KS + VS) * BLOCKS * 4;    // [R][8] see bits
  static constexpr int OFF_NF = OFF_SEEN + R * 32;               // [2][8] keys with a NaN
  static constexpr int OFF_PAR = OFF_NF + 64;                    // int16 [256] parents
  static constexpr int OFF_BAR = OFF_PAR + 512;
  static constexpr int OFF_ABORT = OFF_BAR + 2 * (KS + VS) * 8;
  static constexpr int SMEM = OFF_ABORT + 8;
  static_assert(2 * (SMEM + 1024) <= 228 * 1024, "two blocks per SM");
};

namespace {

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 x;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(addr) : "memory");
  return x;
}

}  // namespace

// NT: groups of 8 rows of a unit.
template <int D, int NT>
__global__ void __launch_bounds__(Narrow8Cfg<D, NT>::THREADS, 2)
    tree8_narrow_kernel(const __grid_constant__ Tree8Params A, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV) {
  using C = Narrow8Cfg<D, NT>;
  using Load = TileLoad8<D, C::KT>;
  constexpr int KT = C::KT;
  const TreeParams& P = A.P;
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
  // Blocks next to each other have one head each of the same stretch: the line
  // is cut into as many runs as blocks, and block x has run x / Hkv of head x %
  // Hkv (where the heads divide the blocks).
  int block = blockIdx.x;
  if (P.Hkv > 1 && gridDim.x % P.Hkv == 0)
    block = blockIdx.x % P.Hkv * (gridDim.x / P.Hkv) + blockIdx.x / P.Hkv;
  if (warp == 2) touch_memory<D>(P, lane, block);
  if (tid == 0) {
    for (int i = 0; i < C::KS + C::VS; ++i) {
      mbar_init(full(i), Load::ARRIVALS);
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
  TreeWalk<typename C::Geo> u(tree_run<typename C::Geo>(P, block));
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
    const float* scales = isk ? A.k_scale : A.v_scale;
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
        Load::copy_scales(P, u, t, lane, page, scales, sbase + C::OFF_SCALE + (first + st) * C::BLOCKS * 4);
        Load::landed(full(first + st), lane);
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
    int16_t* par = reinterpret_cast<int16_t*>(smem + C::OFF_PAR);
    float* merge = reinterpret_cast<float*>(smem + C::OFF_MERGE);
    float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
    const float* scale_ring = reinterpret_cast<const float*>(smem + C::OFF_SCALE);
    uint32_t pieces = 0;
    int par_of = -1;                             // the sequence whose parents are in shared memory
    if (tid == 0) P.rec[block] = make_int4(-1, 0, 0, 0);
    for (; u.next(P); ++pieces) {
      // tiles from this one on hold keys that not every row sees
      const int part0 = u.origin / KT;
      // the next piece's flags, read by nobody now
      uint32_t* nf = nf_all + 8 * (pieces & 1);
      if (tid < 8) nf_all[8 * ((pieces + 1) & 1) + tid] = 0;
      // Q of rows g (and g + 8) as B fragments, in K's order: step kk takes
      // elements D/4 tq + 4 kk + 0..3.  Multiplied by a power of two per row;
      // back holds what undoes it, times the scale, of the rows of S^T's
      // columns 2 tq and 2 tq + 1
      uint32_t qf[NT][D / 16][2];
      float back[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = g + 8 * nt;
        const int rr = u.row_first + r;
        const int node = P.by_G(rr);
        const __nv_bfloat16* src = P.q + (u.s.row0 + node) * P.q_stride[0] +
                                   (u.hk * P.G + rr - node * P.G) * P.q_stride[1] + tq * (D / 4);
        uint32_t w[D / 8];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint4 x = r < u.rows ? *reinterpret_cast<const uint4*>(src + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
          w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
        }
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int up = row_shift(top);
        const float mul = pow2(up);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) qf[nt][i >> 1][i & 1] = f16x2_of_bf16x2(w[i], mul);
        // (an infinity in a row makes it NaN, also where all its scores would be -inf)
        const float undo = top < 0x7f80u ? pow2(-up) * P.scale_log2 : __int_as_float(0x7fc00000);
        back[nt][0] = __shfl_sync(0xffffffffu, undo, 8 * tq);
        back[nt][1] = __shfl_sync(0xffffffffu, undo, 8 * tq + 4);
      }
      // which keys from origin on a row sees: bit i is key origin + i
      if (P.tree && par_of != u.b) {
#pragma unroll 1
        for (int i = tid; i < u.s.n && i < FM_TREE_MAX_NODES && u.s.base >= 0; i += 32 * C::WARPS)
          par[i] = static_cast<int16_t>(tree_parent(P, u.s, i));
        named_sync(1, 32 * C::WARPS);
        par_of = u.b;
      }
      if (tid < C::R) {
        uint32_t bits[8];
        const int node = P.by_G(u.row_first + min(tid, u.rows - 1));
        if (P.tree) {
          tree_ancestors(u.s.base >= 0 ? node : -1, [&](int a) -> int { return par[a]; }, bits);
        } else {
          // (16 rows are of 16 nodes at most)
#pragma unroll
          for (int i = 1; i < 8; ++i) bits[i] = 0;
          bits[0] = u.s.base >= 0 ? (2u << (u.s.base + node - u.origin)) - 1u : 0u;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) seen[tid * 8 + i] = bits[i];
      }
      named_sync(1, 32 * C::WARPS);
      float m[NT][2], l[NT][2];
      float acc[D / 16][NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) acc[x][nt][y] = 0.f;
      }

#pragma unroll 1
      for (int t = u.t0; u.keys > 0 && t < u.t1; ++t) {
        const int ks = e % C::KS, vs = e % C::VS;
        const uint32_t kp = (e / C::KS) & 1, vp = (e / C::VS) & 1;
        ++e;
        const uint32_t sk = sbase + ks * C::TILE, sv = sbase + C::OFF_V + vs * C::TILE;
        // This warp's blocks: warp and warp + 4 of the tile, both always (what is
        // past the unit's keys is masked, in its last tile only): without
        // branches between them their loads and products overlap.
        if (ok) ok = wait_all(full(ks), kp);
        float s[2][NT][4];
        float fk[2];
        if (ok) {
          // two accumulators a block and row group: a product waits for the one
          // before into the same
          float s2[2][NT][4];
          uint4 ka[2][D / 64], kb[2][D / 64];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int r0 = (warp + 4 * x) * 16 + g;
            fk[x] = scale_ring[ks * C::BLOCKS + warp + 4 * x];
#pragma unroll
            for (int w = 0; w < D / 64; ++w) {
              ka[x][w] = lds128(sk + Load::word16(r0, tq * (D / 64) + w));
              kb[x][w] = lds128(sk + Load::word16(r0 + 8, tq * (D / 64) + w));
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int y = 0; y < 4; ++y) s[x][nt][y] = s2[x][nt][y] = 0.f;
          }
#pragma unroll
          for (int w = 0; w < D / 64; ++w)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint4 &a = ka[x][w], &b = kb[x][w];
                const uint32_t wa = i == 0 ? a.x : i == 1 ? a.y : i == 2 ? a.z : a.w;
                const uint32_t wb = i == 0 ? b.x : i == 1 ? b.y : i == 2 ? b.z : b.w;
                const uint32_t f[4] = {f16x2_of_e4m3x2(wa), f16x2_of_e4m3x2(wb), f16x2_of_e4m3x2(wa >> 16),
                                       f16x2_of_e4m3x2(wb >> 16)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma_f16(i & 1 ? s2[x][nt] : s[x][nt], f, qf[nt][4 * w + i][0], qf[nt][4 * w + i][1]);
              }
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int y = 0; y < 4; ++y) s[x][nt][y] += s2[x][nt][y];
        }
        // (a test of the wait limit withholds the first one: the K loader's
        // wait for the stage then runs out)
        if (!(P.withhold == 8 && e == 1)) mbar_arrive_warp(empty(ks));
        if (ok) ok = wait_all(full(C::KS + vs), vp);
        uint32_t pf[2][NT][2];
        if (ok) {
          float4 f[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            f[x] = block_factors(fk[x], scale_ring[(C::KS + vs) * C::BLOCKS + warp + 4 * x]);
          }
          // z = x + log2 sv, in place
#pragma unroll
          for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int y = 0; y < 4; ++y)
                s[x][nt][y] = fmaf(s[x][nt][y], finite(back[nt][y & 1] * f[x].x), f[x].y);
          }
          if (t >= part0 || (t + 1) * KT > u.keys) {
            // keys past origin: only what the row sees
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int key0 = t * KT + (warp + 4 * x) * 16 + g;
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const int key = key0 + 8 * (y >> 1), j = key - u.origin;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  const int r = 8 * nt + 2 * tq + (y & 1);
                  const bool sees = key < u.keys && (j < 0 || ((seen[r * 8 + ((j >> 5) & 7)] >> (j & 31)) & 1u));
                  if (!sees) s[x][nt][y] = -INFINITY;
                }
              }
            }
          }
          bool grow = false;
          float alpha[NT][2], ref[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              float mx = fmaxf(fmaxf(s[0][nt][y], s[0][nt][y + 2]), fmaxf(s[1][nt][y], s[1][nt][y + 2]));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
              // the reference moves only when the maximum grows by more than
              // 2^8: until then P stays in range and nothing is rescaled
              const bool up = mx > m[nt][y] + 8.f;
              alpha[nt][y] = up ? ex2(m[nt][y] - mx) : 1.f;
              m[nt][y] = up ? mx : m[nt][y];
              ref[nt][y] = (m[nt][y] == -INFINITY ? 0.f : m[nt][y]) - kPOffset;
              grow |= up;
            }
          if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
              for (int x = 0; x < D / 16; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) acc[x][nt][y] *= alpha[nt][y & 1];
              l[nt][0] *= alpha[nt][0];
              l[nt][1] *= alpha[nt][1];
            }
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float p[4];
#pragma unroll
              for (int y = 0; y < 4; ++y) p[y] = ex2(s[x][nt][y] - ref[nt][y & 1]);
              l[nt][0] = fmaf(p[0] + p[2], f[x].z, l[nt][0]);
              l[nt][1] = fmaf(p[1] + p[3], f[x].z, l[nt][1]);
              pf[x][nt][0] = transpose8(pack_f16(p[0], p[1]));
              pf[x][nt][1] = transpose8(pack_f16(p[2], p[3]));
            }
          }
          if (t >= part0 || (t + 1) * KT > u.keys) {
            // this warp's rows of V: zeros past the unit's keys, and clean
            // where not every row sees the key
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
              const int row = (warp + 4 * x) * 16 + (lane >> 1);
              const int key = t * KT + row, j = key - u.origin;
              auto word = [&](int c) {
                return reinterpret_cast<uint4*>(smem + C::OFF_V + vs * C::TILE +
                                                Load::word16(row, (lane & 1) * (D / 32) + c));
              };
              if (key >= u.keys) {
#pragma unroll
                for (int c = 0; c < D / 32; ++c) *word(c) = make_uint4(0u, 0u, 0u, 0u);
              } else if (j >= 0) {
                uint32_t any = 0;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                  const uint4 y = *word(c);
                  any |= e4m3x4_nan(y.x) | e4m3x4_nan(y.y) | e4m3x4_nan(y.z) | e4m3x4_nan(y.w);
                }
                if (any) {
                  atomicOr(nf + (j >> 5), 1u << (j & 31));
#pragma unroll 1
                  for (int c = 0; c < D / 32; ++c) {
                    uint4* y = word(c);
                    *y = make_uint4(y->x & ~e4m3x4_nan(y->x), y->y & ~e4m3x4_nan(y->y), y->z & ~e4m3x4_nan(y->z),
                                    y->w & ~e4m3x4_nan(y->w));
                  }
                }
              }
            }
            fence_proxy_async_smem();   // before the next copy into this slot
            __syncwarp();
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            // matrices: keys 0-7 bytes 0-15, keys 8-15 bytes 0-15, keys 0-7
            // bytes 16-31, keys 8-15 bytes 16-31
            const int row = (warp + 4 * x) * 16 + (lane & 15);
#pragma unroll
            for (int dd = 0; dd < D / 32; ++dd) {
              uint32_t b[4];
              ldsm4_t(sv + Load::word16(row, dd * 2 + (lane >> 4)), b);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t lo = __byte_perm(b[2 * i], 0, 0x3120), hi = __byte_perm(b[2 * i + 1], 0, 0x3120);
                const uint32_t f[4] = {f16x2_of_e4m3x2(lo), f16x2_of_e4m3x2(lo >> 16), f16x2_of_e4m3x2(hi),
                                       f16x2_of_e4m3x2(hi >> 16)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16(acc[2 * dd + i][nt], f, pf[x][nt][0], pf[x][nt][1]);
              }
            }
          }
        }
        mbar_arrive_warp(empty(C::KS + vs));
      }

      // ---------------------------------------------------------- merge the four warps
      // Each warp's maxima, sums and O as they are to shared memory, eight rows
      // at a time; then a thread adds four columns of a row.
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int r = 8 * nt + 2 * tq + y;
          float mm = -INFINITY, ll = 0.f;
          if (nt < NT) {
            mm = m[nt % NT][y];
            ll = l[nt % NT][y];
            ll += __shfl_xor_sync(0xffffffffu, ll, 4);
            ll += __shfl_xor_sync(0xffffffffu, ll, 8);
            ll += __shfl_xor_sync(0xffffffffu, ll, 16);
            // a padding node's row sees nothing, the context included
            if (P.tree) {
              uint32_t any = 0;
#pragma unroll
              for (int i = 0; i < 8; ++i) any |= seen[r * 8 + i];
              if (!any) {
                mm = -INFINITY;
                ll = 0.f;
              }
            }
          }
          if (g == 0) ml[r * C::WARPS + warp] = make_float2(mm, ll);
        }
#pragma unroll 1
      for (int r0 = 0; r0 < u.rows; r0 += 8) {
        if (r0 > 0) named_sync(1, 32 * C::WARPS);       // the first eight rows have been read
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            // row 2 tq + y, elements 16 x + 2 g and the next one
            const float a0 = (NT > 1 && r0 ? acc[x][NT - 1][y] : acc[x][0][y]) * kPUndo;
            const float a1 = (NT > 1 && r0 ? acc[x][NT - 1][y + 2] : acc[x][0][y + 2]) * kPUndo;
            *reinterpret_cast<float2*>(merge + (warp * 8 + 2 * tq + y) * C::PITCH + x * 16 + 2 * g) = make_float2(a0, a1);
          }
        named_sync(1, 32 * C::WARPS);
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) any |= nf[i];
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
          if (u.whole()) {
            const int rr = u.row_first + r, node = P.by_G(rr), h = u.hk * P.G + rr - node * P.G;
            const float inv = ll > 0.f ? 1.f / ll : ll;     // 0 or NaN as it is
            __nv_bfloat16* dst = P.o + (u.s.row0 + node) * P.o_stride[0] + h * P.o_stride[1] + c;
            *reinterpret_cast<uint2*>(dst) =
                make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
            if (any)
              fix_row8(A, u.b, u.hk, u.origin, nf, *reinterpret_cast<const uint4*>(seen + r * 8),
                       *reinterpret_cast<const uint4*>(seen + r * 8 + 4), c, 4, dst);
            if (c == 0)
              P.lse[static_cast<int64_t>(h) * P.total + u.s.row0 + node] =
                  ll > 0.f || ll != ll ? (mm + __log2f(ll)) * 0.69314718055994530942f : -INFINITY;
          } else {
            const int64_t at = static_cast<int64_t>(2 * block + (u.t0 == 0 ? 1 : 0)) * P.part_rows + r;
            float* dst = P.part_o + at * D + c;
            *reinterpret_cast<float4*>(dst) = v;
            if (any)
              fix_row8(A, u.b, u.hk, u.origin, nf, *reinterpret_cast<const uint4*>(seen + r * 8),
                       *reinterpret_cast<const uint4*>(seen + r * 8 + 4), c, 4, dst);
            if (c == 0) P.part_ml[at] = make_float2(mm, ll);
          }
        }
      }
      if (tid == 0) leave_record(P, u, block);
      named_sync(1, 32 * C::WARPS);     // ml, merge, seen and nf have been read
    }
  }
  __syncthreads();
}

template <int D, int NT>
static fm_status launch_narrow8(const Tree8Params& A, const CUtensorMap& tk, const CUtensorMap& tv, int grid,
                                cudaStream_t s) {
  using C = Narrow8Cfg<D, NT>;
  auto kern = tree8_narrow_kernel<D, NT>;
  static std::atomic<uint64_t> ready{0};
  const fm_status st = prepare_kernel(kern, C::SMEM, 0, ready);
  if (st != FM_OK) return st;
  prof_begin(K_TREE, s);
  const cudaError_t e = launch_dependent(kern, dim3(grid), C::THREADS, C::SMEM, s, A, tk, tv);
  prof_end(K_TREE, s);
  return e == cudaSuccess ? FM_OK : FM_ERR_CUDA;
}

fm_status launch_tree8_narrow(const Tree8Params& A, int d, int rows, const CUtensorMap& tk, const CUtensorMap& tv,
                              int grid, cudaStream_t s) {
  if (d == 64) return rows <= 8 ? launch_narrow8<64, 1>(A, tk, tv, grid, s) : launch_narrow8<64, 2>(A, tk, tv, grid, s);
  return rows <= 8 ? launch_narrow8<128, 1>(A, tk, tv, grid, s) : launch_narrow8<128, 2>(A, tk, tv, grid, s);
}

}  // namespace fm
