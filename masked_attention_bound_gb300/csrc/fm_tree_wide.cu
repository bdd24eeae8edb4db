// Attention over the paged cache for units of up to 128 or 256 rows (drafted
// trees, causal runs, many query heads per K/V head), on the 5th-generation
// tensor cores.
//
// A unit's rows fill one or two 128-row tiles of tcgen05.mma.  A slot is an
// S/P and an O in tensor memory, a warpgroup of softmax threads (thread = row
// = TMEM lane) and an MMA warp.
//
// SLOTS = 1 (up to 128 rows, bound by reading K and V): 64-key tiles and two
// blocks per SM, so that one's fetching and writing at the ends of units run
// while the other's tiles stream.  S has two buffers: S of a tile is computed
// while the softmax of the one before runs, and its PV while that of the next.
//
// SLOTS = 2 (some unit has more than 128 rows): 128-key tiles, one block per
// SM, one slot's softmax running while the other's products do:
//  - more than 128 rows: slot s holds rows [128 s, 128 s + 128) and both walk
//    every tile, so a tile is loaded once for 256 rows; such units are bound
//    by the softmax and the tensor pipe;
//  - up to 128 rows: both slots hold the same rows and take the key tiles in
//    turn; their O, maximum and sum are merged at the end of the piece.
//
// Warps: 4 per slot for the softmax, then one that loads K, slot 0's MMAs, one
// that loads V, slot 1's MMAs.  Rows of a unit are nodes times query heads: Q
// comes by TMA (SLOTS = 2, a group size that divides 128) or by the softmax
// warps' copies.  The softmax warps also clean the V tiles that hold drafted
// nodes.
//
// P is rounded to bf16, the type of V, for its product (the operands of
// tcgen05.mma have one type), as in the prompt forward; its sum, the maximum, S
// and O are fp32.  That is at most 2^-8 of a weight, and O is off by 0.0023 of
// its norm against float64 where an fp32 computation rounded once is off by
// 0.0017.  P as two bf16 numbers, as in the kernel for 16 rows, would bring
// 0.0017 and cost a second product: 64 sequences of 1000 tokens with 64 rows
// took 55.7 us so and 50.7 with one number, with d = 64 and 150 rows 74.7 and
// 64.5.
//
// CODES: the cache holds e4m3 codes (see fm_tree8.cuh for the arithmetic).  S
// multiplies K's codes as they are.  V's go to stages of their own and become f16
// tiles in front of the MMAs, laid out as the bf16 tiles are, by warps that do
// nothing else.  Tiles have 64 keys and S two buffers a slot with SLOTS = 2 as
// well: the slots take no turns, and always hold rows [128 s, 128 s + 128).  A tile
// of 256 rows takes 2200 cycles, which is its softmax's chain of tensor memory
// loads, maximum, weights and barriers in two warps a scheduler: without the second
// part of Q, half of PV or exp2, each left out by itself, 16 trees of 64 nodes over
// 16384 tokens took 199, 200 and 206 us instead of 204.
//
// TMEM: S/P of slot s at column 128 s (SLOTS = 1: of every second tile at
// column 64), the O's after the S's.
#include <type_traits>

#include "fm_tree8.cuh"

namespace fm {

template <int D, int SLOTS_, bool CODES_>
struct WideCfg {
  static constexpr int SLOTS = SLOTS_;
  static constexpr bool CODES = CODES_;
  static constexpr int DIM = D;
  static_assert(D == 128 || SLOTS == 1, "d = 64 runs with tiles of 128 rows side by side");
  // Two S buffers of 64 columns a slot: S of a tile is computed while the
  // softmax of the one before runs, and slots do not take turns.
  static constexpr bool BUFS = SLOTS == 1 || CODES;
  using Geo = std::conditional_t<SLOTS == 1, MidGeo, std::conditional_t<CODES, Wide8Geo, WideGeo>>;
  static constexpr int KT = Geo::KT;
  static constexpr int TILE = KT * D * 2;               // bytes of a V tile in front of the MMAs
  static constexpr int KTILE = CODES ? KT * D : TILE;   // of a K tile
  static constexpr int QTILE = 128 * D * 2;             // of a slot's Q (CODES: two parts of one byte)
  static constexpr int KSTAGES = CODES ? (D == 64 || SLOTS == 2 ? 5 : 3) : D == 64 ? 4 : 2;
  static constexpr int VSTAGES = CODES ? (SLOTS == 2 ? 3 : 2) : D == 64 ? 5 : 3;
  static constexpr int VCODES = !CODES ? 0 : D == 64 || SLOTS == 2 ? 4 : 2;   // stages of V's codes
  static constexpr int BLOCKS = KT / kScaleBlock;
  static constexpr int SM_WARPS = 4 * SLOTS;            // softmax
  // CODES: warps that turn V's codes into f16: a warpgroup of their own, or with
  // SLOTS = 1, where registers are short, the places of the V loader (K's loads
  // both) and of a second slot's MMAs.
  static constexpr int CV_WARPS = !CODES ? 0 : SLOTS == 2 ? 4 : 2;
  static constexpr int THREADS = 32 * (SM_WARPS + 4 + (SLOTS == 2 ? CV_WARPS : 0));
  static constexpr bool LOADS_BOTH = CODES && SLOTS == 1;
  // S of a tile is issued once its V tile and factors are there, which saves the
  // softmax a wait.  (Not with V's two stages of SLOTS = 1: 32 nodes over 131072
  // keys 37.8 us so and 34.5 us with that wait.)
  static constexpr bool V_FIRST = CODES && SLOTS == 2;
  static constexpr int BLOCKS_PER_SM = SLOTS == 2 ? 1 : 2;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = SLOTS * QTILE;
  static constexpr int OFF_V = OFF_K + KSTAGES * KTILE;
  static constexpr int OFF_VC = OFF_V + VSTAGES * TILE;                      // V's codes
  static constexpr int OFF_FACT = OFF_VC + VCODES * KTILE;        // CODES: [VSTAGES][BLOCKS] of float4, then of float
  static constexpr int OFF_SCALE = OFF_FACT + (CODES ? VSTAGES * BLOCKS * 20 : 0);     // float [VCODES][K, V][BLOCKS]
  static constexpr int OFF_ML = OFF_SCALE + VCODES * 2 * BLOCKS * 4;         // BUFS false: float2 [slot][128]
  static constexpr int OFF_NF = OFF_ML + (BUFS ? 0 : 2 * 128 * 8);   // [4][8] keys with values not finite
  static constexpr int OFF_BAR = OFF_NF + 128;
  static constexpr int NBAR = CODES ? 48 : 34;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;   // abort flag, TMEM address
  static constexpr int OFF_PAR = OFF_MISC + 16;         // int16 [256] parents of the unit's nodes
  static constexpr int USED = OFF_PAR + 512;
  static constexpr int SMEM = USED;
  static_assert(BLOCKS_PER_SM * (SMEM + 1024) <= 228 * 1024, "blocks per SM");
  static_assert(KSTAGES <= 5 && VSTAGES <= 5 && VCODES <= 4, "barriers of the stages");
  // O is written through 4 KB per softmax warp, in its slot's Q tile: that
  // slot's S have all been read by then
  static_assert(4 * 4096 <= QTILE, "room for the output's staging");
  static constexpr uint32_t T_COLS = 256 * SLOTS, T_O = 128 * SLOTS;
  // register split: the softmax warpgroups' and the others' budgets add up to
  // what the block is launched with (384 x 168, 256 x 128; CODES: 512 x 128)
  static constexpr uint32_t REGS_SOFTMAX = CODES ? 152 : SLOTS == 2 ? 216 : 184;
  static constexpr uint32_t REGS_PRODUCER = CODES ? 104 : 72;
  static constexpr int MIN_LAUNCH_REGS =
      (32 * SM_WARPS * REGS_SOFTMAX + (THREADS - 32 * SM_WARPS) * REGS_PRODUCER + THREADS - 1) / THREADS;
};

enum {
  W_QFULL = 0, W_SFULL = 2, W_PFULL = 4, W_PVDONE = 6, W_OEMPTY = 8, W_KFULL = 10, W_KEMPTY = 15,
  W_VFULL = 20, W_VEMPTY = 25, W_DRAIN = 30, W_TURN = 31, W_QEMPTY = 33,
  W_VCODES = 34, W_VCEMPTY = 38,   // CODES: stages of V's codes
  W_PVTILE = W_PVDONE + 1,  // SLOTS 1: the PV of each tile (the SFULL and PFULL are its two buffers')
  // BUFS of two slots: the second slot's SFULL and PFULL, the slots' PVTILE
  W_SFULL_B = 42, W_PFULL_B = 44, W_PVTILE_2 = 46
};

// How the slots share a piece.
struct WideSplit {
  bool rows;     // slots split the rows (else the key tiles)
  int n;         // key tiles of the piece
  // slot s takes part at all
  __device__ __forceinline__ bool active(int s) const { return s == 0 || rows || n > 1; }
};
template <bool BUFS>
__device__ __forceinline__ WideSplit wide_split(const TreePiece& u) {
  return WideSplit{BUFS || u.rows > 128, u.keys > 0 ? u.t1 - u.t0 : 0};
}

// 16 bytes from global to shared memory without a register or a line of L1;
// `bytes` 0 reads nothing and writes zeros.
__device__ __forceinline__ void copy_async16(uint32_t dst, uint64_t src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// All softmax warps.
template <int SLOTS>
__device__ __forceinline__ void slots_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(128 * SLOTS) : "memory");
}

template <bool CODES>
using WideParams = std::conditional_t<CODES, Tree8Params, TreeParams>;
__device__ __forceinline__ const TreeParams& tree_params(const TreeParams& A) { return A; }
__device__ __forceinline__ const TreeParams& tree_params(const Tree8Params& A) { return A.P; }

// CODES: rows [part * rows, (part + 1) * rows) of V tile `e` of the block, clean
// of what not every row sees (see fix_row8), and what the scales of its blocks
// bring to the softmax.  (The stage's last PV has ended, so the softmax of that
// tile has read its factors.)
template <typename C, typename W>
__device__ __forceinline__ bool convert_v(const TreeParams& P, const TreePiece& u, int t, uint32_t e, int part,
                                          int rows, int lane, const uint8_t* smem, uint32_t sbase,
                                          uint32_t* nf, W wait_all) {
  using V = VTile8<C::DIM, C::KT>;
  const uint32_t cs = e % C::VCODES, st = e % C::VSTAGES;
  bool ok = wait_all(W_VCODES + cs, (e / C::VCODES) & 1);
  if (ok && e >= C::VSTAGES) ok = wait_all(W_VEMPTY + st, (e / C::VSTAGES - 1) & 1);
  if (!ok) return false;
  const float* scales = reinterpret_cast<const float*>(smem + C::OFF_SCALE) + cs * 2 * C::BLOCKS;
  const int b = part * (rows / kScaleBlock) + lane;
  if (lane < rows / kScaleBlock) {
    const float4 f = block_factors(scales[b], scales[C::BLOCKS + b]);
    // in pairs, as the packed arithmetic takes them
    asm volatile("st.shared.v4.f32 [%0], {%1, %1, %2, %2};" ::"r"(sbase + C::OFF_FACT + (st * C::BLOCKS + b) * 16),
                 "f"(f.x), "f"(f.y)
                 : "memory");
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(sbase + C::OFF_FACT + C::VSTAGES * C::BLOCKS * 16 +
                                                 (st * C::BLOCKS + b) * 4),
                 "f"(f.z)
                 : "memory");
  }
  const uint32_t from = sbase + C::OFF_VC + cs * C::KTILE, to = sbase + C::OFF_V + st * C::TILE;
  const bool partial = t >= u.origin / C::KT;
#pragma unroll 1
  for (int r0 = part * rows; r0 < (part + 1) * rows; r0 += 16) {
    if (partial) {
      V::to_f16(from, to, r0, lane, [&](int row, uint4& y) {
        const int key = t * C::KT + row, i = key - u.origin;
        if (key >= u.keys) {
          y = make_uint4(0u, 0u, 0u, 0u);
        } else if (i >= 0) {
          const uint4 nan = make_uint4(e4m3x4_nan(y.x), e4m3x4_nan(y.y), e4m3x4_nan(y.z), e4m3x4_nan(y.w));
          if (nan.x | nan.y | nan.z | nan.w) {
            atomicOr(nf + (i >> 5), 1u << (i & 31));
            y = make_uint4(y.x & ~nan.x, y.y & ~nan.y, y.z & ~nan.z, y.w & ~nan.w);
          }
        }
      });
    } else {
      V::to_f16(from, to, r0, lane, [](int, uint4&) {});
    }
  }
  fence_proxy_async_smem();
  mbar_arrive_warp(sbase + C::OFF_BAR + 8u * (W_VCEMPTY + cs));
  if (lane == 0) mbar_arrive(sbase + C::OFF_BAR + 8u * (W_VFULL + st));
  return true;
}

template <int D, int SLOTS, bool CODES>
__global__ void __launch_bounds__(WideCfg<D, SLOTS, CODES>::THREADS, WideCfg<D, SLOTS, CODES>::BLOCKS_PER_SM)
    tree_wide_kernel(const __grid_constant__ WideParams<CODES> A, const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
  using C = WideCfg<D, SLOTS, CODES>;
  using Load = std::conditional_t<CODES, TileLoad8<D, C::KT>, TileLoad<D, C::KT>>;
  constexpr int KT = C::KT;
  const TreeParams& P = tree_params(A);
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0 && P.status) atomicOr(P.status, DEV_LAYOUT);
    return;
  }
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + C::OFF_BAR + 8u * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC + 4);
  uint32_t* nf_all = reinterpret_cast<uint32_t*>(smem + C::OFF_NF);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int K_WARP = C::SM_WARPS, MMA_WARP = K_WARP + 1, V_WARP = K_WARP + 2, MMA_WARP_B = K_WARP + 3;

  // Q by TMA as soon as the piece before has left its tiles, while the softmax
  // warps find out what their rows see: 512 units of 544 keys took 76 us so
  // and 82 us with these warps' copies.  (With two blocks per SM the other
  // block has the time: 50 us by their copies, 53 by TMA.)
  const bool q_tma = SLOTS == 2 && !CODES && P.q_tma;

  if (warp == 2) touch_memory<D>(P, lane, blockIdx.x);
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(W_QFULL + s), q_tma ? 1 : 4);   // else one arrival per softmax warp of the slot
      mbar_init(bar(W_SFULL + s), C::V_FIRST ? 2 : 1);
      mbar_init(bar(W_PFULL + s), 4);
      mbar_init(bar(W_PVDONE + s), 1);
      mbar_init(bar(W_OEMPTY + s), C::SM_WARPS);   // every slot's warps may read O of either
      mbar_init(bar(W_TURN + s), 1);
    }
    // a stage is free after a commit per slot: one by each MMA warp, or both
    // by the one whose slot took the tile
    for (int i = 0; i < C::KSTAGES; ++i) {
      mbar_init(bar(W_KFULL + i), 1);
      mbar_init(bar(W_KEMPTY + i), SLOTS);
    }
    for (int i = 0; i < C::VSTAGES; ++i) {
      mbar_init(bar(W_VFULL + i), CODES ? C::CV_WARPS : 1);
      mbar_init(bar(W_VEMPTY + i), SLOTS);
    }
    if constexpr (CODES) {
      for (int i = 0; i < C::VCODES; ++i) {
        mbar_init(bar(W_VCODES + i), Load::ARRIVALS);
        mbar_init(bar(W_VCEMPTY + i), C::CV_WARPS);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(bar(W_SFULL_B + i), 2);
        mbar_init(bar(W_PFULL_B + i), 4);
        mbar_init(bar(W_PVTILE_2 + i), 1);
      }
    }
    mbar_init(bar(W_DRAIN), SLOTS);
    mbar_init(bar(W_QEMPTY), C::SM_WARPS);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (tid < 32) nf_all[tid] = 0;
  if (warp == MMA_WARP) {
    tmem_alloc(smem_u32(tmem_slot), C::T_COLS);
    tmem_relinquish();
  }
  if (warp == K_WARP && lane == 0) tma_prefetch_desc(&tmK);
  if (warp == V_WARP && lane == 0) tma_prefetch_desc(&tmV);
  if (q_tma && warp == MMA_WARP && lane == 0) tma_prefetch_desc(&tmQ);
  grid_launch_dependents();
  grid_dependency_wait();
  tc_fence_before();
  TreeWalk<typename C::Geo> u(tree_run<typename C::Geo>(P, blockIdx.x));
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;

  // BUFS: the barriers of a slot's buffer
  auto s_full = [](int slot, int buf) { return (SLOTS == 2 && slot ? W_SFULL_B : W_SFULL) + buf; };
  auto p_full = [](int slot, int buf) { return (SLOTS == 2 && slot ? W_PFULL_B : W_PFULL) + buf; };
  auto pv_tile = [](int slot) { return SLOTS == 2 ? W_PVTILE_2 + slot : static_cast<int>(W_PVTILE); };
  auto wait = [&](int b, uint32_t parity) -> bool { return tree_wait(bar(b), parity, P, abort_flag); };
  // every lane gets the same answer
  auto wait_all = [&](int b, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, wait(b, parity));
  };

  if (warp >= C::SM_WARPS) {
    regs_decrease<C::REGS_PRODUCER>();
    if (warp == K_WARP || (warp == V_WARP && !C::LOADS_BOTH)) {
      // ---------------------------------------------------------- K / V loads
      const bool isk = warp == K_WARP;
      constexpr bool BOTH = C::LOADS_BOTH;
      uint32_t vst = 0, vuse = 0;
      auto load_v_codes = [&](const TreePiece& u, int t, int page, uint32_t st, uint64_t policy) {
        if constexpr (CODES) {                         // and the scales of both
          const uint32_t to = sbase + C::OFF_SCALE + st * (2 * C::BLOCKS * 4);
          VTile8<D, KT>::issue(P, u, t, lane, page, &tmV, sbase + C::OFF_VC + st * C::KTILE, bar(W_VCODES + st), policy);
          Load::copy_scales(P, u, t, lane, page, A.k_scale, to);
          Load::copy_scales(P, u, t, lane, page, A.v_scale, to + C::BLOCKS * 4);
          Load::landed(bar(W_VCODES + st), lane);
        }
      };
      const int stages = isk ? C::KSTAGES : CODES ? C::VCODES : C::VSTAGES;
      const int b_full = isk ? W_KFULL : CODES ? W_VCODES : W_VFULL;
      const int b_empty = isk ? W_KEMPTY : CODES ? W_VCEMPTY : W_VEMPTY;
      const uint32_t buf = sbase + (isk ? C::OFF_K : CODES ? C::OFF_VC : C::OFF_V);
      const CUtensorMap* tm = isk ? &tmK : &tmV;
      const uint64_t policy = policy_evict_first();
      uint32_t st = 0, use = 0, issued = 0;    // stage, its uses so far, tiles issued
      bool ok = true;
      while (ok && u.next(P)) {
        if (u.keys == 0) continue;
        int page = Load::lane_page(P, u, u.t0, lane);
#pragma unroll 1
        for (int t = u.t0; t < u.t1; ++t) {
          const int next = t + 1 < u.t1 ? Load::lane_page(P, u, t + 1, lane) : 0;
          if (use > 0) ok = wait_all(b_empty + st, (use - 1) & 1);
          if (!ok) break;
          if (CODES && !isk) load_v_codes(u, t, page, st, policy);
          else Load::issue(P, u, t, lane, page, tm, buf + st * C::KTILE, bar(b_full + st), policy);
          if constexpr (BOTH) {
            if (vuse > 0) ok = wait_all(W_VCEMPTY + vst, (vuse - 1) & 1);
            if (ok) load_v_codes(u, t, page, vst, policy);
            if (ok && ++vst == C::VCODES) {
              vst = 0;
              ++vuse;
            }
          }
          ++issued;
          if (++st == stages) {
            st = 0;
            ++use;
          }
          if (!ok) break;
          page = next;
        }
      }
      // every issued copy has landed before the block may exit
      if (lane == 0)
#pragma unroll 1
        for (uint32_t x = issued > stages ? issued - stages : 0; x < issued; ++x)
          mbar_wait(bar(b_full + x % stages), (x / stages) & 1, P.status, P.wait_ns);
      if constexpr (BOTH) {
        const uint32_t vs = vuse * C::VCODES + vst;
        if (lane == 0)
#pragma unroll 1
          for (uint32_t x = vs > C::VCODES ? vs - C::VCODES : 0; x < vs; ++x)
            mbar_wait(bar(W_VCODES + x % C::VCODES), (x / C::VCODES) & 1, P.status, P.wait_ns);
      }
      __syncwarp();
    } else if (warp == MMA_WARP || (SLOTS == 2 && warp == MMA_WARP_B)) {
      // ---------------------------------------------------------- MMA issuers
      // The whole warp walks and waits, and one elected lane issues: the
      // descriptors are then uniform, and an MMA costs its issue only.
      const int s = warp == MMA_WARP ? 0 : 1;
      constexpr uint32_t idS = CODES ? idesc_e4m3(128, KT) : idesc_bf16(128, KT, false, false);
      constexpr uint32_t idPV = CODES ? idesc_f16(128, D, false, true) : idesc_bf16(128, D, false, true);
      const uint32_t dQ = sdesc_lo(sbase + C::OFF_Q + s * C::QTILE, 16);
      const uint32_t dK0 = sdesc_lo(sbase + C::OFF_K, 16);
      const uint32_t dV0 = sdesc_lo(sbase + C::OFF_V, KT * 128);
      const uint32_t tS = tbase + 128 * s, tO = tbase + C::T_O + 128 * s;
      // Step i of SSTEPS of S (CODES: of Q's first part, then of its second)
      constexpr int SSTEPS = D / 16;
      auto s_step = [&](uint32_t to, uint32_t dK, int i) {
        if constexpr (CODES) {
          const int part = i / (D / 32), kk = i % (D / 32);
          const uint32_t id = part ? idesc_e5m2_e4m3(128, KT) : idS;
          if constexpr (D == 128)
            mma_ss_f8(to, sdesc_at(dQ, part * (128 * D) + kk * 32), sdesc_at(dK, kk * 32), id, i > 0 ? 1u : 0u);
          else
            mma_ss_f8(to, sdesc64_at(dQ, part * (128 * D) + kk * 32), sdesc64_at(dK, kk * 32), id, i > 0 ? 1u : 0u);
        } else {
          mma_ss(to, sdesc_at(dQ, (i >> 2) * (128 * 128) + (i & 3) * 32),
                 sdesc_at(dK, (i >> 2) * (KT * 128) + (i & 3) * 32), idS, i > 0 ? 1u : 0u);
        }
      };
      uint32_t kst = 0, kph = 0, vst = 0, vph = 0;   // stages and phases of the next tile of the block
      uint32_t pieces = 0;      // pieces with keys before this one
      uint32_t qn = 0, np = 0;  // Q tiles, P tiles of this slot so far
      uint32_t turn = 0;        // turns taken
      bool ok = true;
      while (ok && u.next(P)) {
        const WideSplit w = wide_split<C::BUFS>(u);
        if (w.n == 0) continue;
        // The two MMA warps take turns: a turn is one tile's PV and the next
        // one's S.  Without it the slots fall into step (both wait for the
        // same K, then both softmaxes run, then both slots' MMAs share the
        // tensor pipe: 4900 cycles a pair of tiles); with turns one slot's
        // MMAs run while the other's softmax does.
        auto my_turn = [&]() -> bool {
          if constexpr (SLOTS == 1) return true;
          return s == 0 ? (turn == 0 || wait_all(W_TURN + 1, (turn - 1) & 1)) : wait_all(W_TURN, turn & 1);
        };
        auto end_turn = [&]() {
          if (SLOTS == 2 && elect_one()) mbar_arrive(bar(W_TURN + s));
          ++turn;
        };
        // stages advance by the piece's tiles; the slot's own tiles are every
        // first or every second one
        const int step = w.rows ? 1 : 2, x0 = w.rows ? 0 : s;
        const int turns = (w.rows ? w.n : (w.n + 1) / 2) + 1;   // of either slot
        auto advance = [](uint32_t& st, uint32_t& ph, int by, int stages) {
          st += by;
          while (st >= stages) {
            st -= stages;
            ph ^= 1;
          }
        };
        uint32_t ks = kst, kp = kph, vs = vst, vp = vph;        // of tiles x (K) and x - step (V)
        advance(ks, kp, x0, C::KSTAGES);
        advance(vs, vp, x0, C::VSTAGES);
        if (w.active(s)) {
          if (q_tma) {
            // the rows of the piece before have left through the Q tiles
            if (pieces > 0) ok = wait_all(W_QEMPTY, (pieces - 1) & 1);
            if (!ok) break;
            if (elect_one()) {
              const int node0 = u.s.row0 + P.by_G(u.row_first + (w.rows ? 128 * s : 0));
              mbar_arrive_expect_tx(bar(W_QFULL + s), C::QTILE);
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                tma_load_4d(sbase + C::OFF_Q + s * C::QTILE + c * (128 * 128), &tmQ, bar(W_QFULL + s), c * 64,
                            u.hk * P.G, node0, 0);
            }
            __syncwarp();
          }
          ok = wait_all(W_QFULL + s, qn & 1);
          ++qn;
        }
        if constexpr (C::BUFS) {
          // S of tile x + 1 overwrites P of tile x - 1, whose PV this warp has
          // issued before; then PV of tile x.  (Two slots have a warp each: one
          // for both spent 2700 cycles a tile on its waits and issues, 291 us.)
          uint32_t fs = vst, fp = vph;             // V's stage of the next S
          auto issue_s = [&](uint32_t tile) -> bool {
            if (!wait_all(W_KFULL + ks, kp)) return false;
            if constexpr (C::V_FIRST) {
              if (!wait_all(W_VFULL + fs, fp)) return false;
              advance(fs, fp, 1, C::VSTAGES);
            }
            const uint32_t dK = dK0 + ks * (C::KTILE >> 4);
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < SSTEPS; ++kk) s_step(tS + 64 * (tile & 1), dK, kk);
              mma_commit(bar(s_full(s, tile & 1)));
              mma_commit(bar(W_KEMPTY + ks));
              // (what this thread knows of the factors goes on with its own arrival)
              if constexpr (C::V_FIRST) mbar_arrive(bar(s_full(s, tile & 1)));
            }
            __syncwarp();
            advance(ks, kp, 1, C::KSTAGES);
            return true;
          };
          if (ok) ok = issue_s(np);
#pragma unroll 1
          for (int x = 0; ok && x < w.n; ++x, ++np) {
            if (x + 1 < w.n) ok = issue_s(np + 1);
            if (ok && !C::V_FIRST) ok = wait_all(W_VFULL + vs, vp);
            // O is overwritten: the last piece's must have been read
            if (ok && x == 0 && pieces > 0) ok = wait_all(W_OEMPTY + s, (pieces - 1) & 1);
            if (ok) ok = wait_all(p_full(s, np & 1), (np >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t dV = dV0 + vs * (C::TILE >> 4), tP = tS + 64 * (np & 1);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < KT / 16; ++kk)
                mma_ts(tO, tP + kk * 8, sdesc_at(dV, kk * 2048), idPV, (x > 0 || kk > 0) ? 1u : 0u);
              mma_commit(bar(pv_tile(s)));
              if (x + 1 == w.n) mma_commit(bar(W_PVDONE + s));
              mma_commit(bar(W_VEMPTY + vs));
            }
            __syncwarp();
            advance(vs, vp, 1, C::VSTAGES);
          }
          kst = ks; kph = kp; vst = vs; vph = vp;
          ++pieces;
          continue;
        }
        int x = x0;
#pragma unroll 1
        for (int i = 0; ok && i < turns; ++i) {
          // PV of the slot's tile x - step, then S of its tile x, which
          // overwrites that P: MMAs run in the order in which a thread issues them
          const bool pv = i > 0 && x - step < w.n, sn = x < w.n;
          // P comes last: what else the turn needs is known by then, and the
          // product starts as soon as P is there
          bool kready = true;
          if (pv) {
            ok = wait_all(W_VFULL + vs, vp);
            // O of the slot is overwritten: the last piece's must have been read
            if (ok && i == 1 && pieces > 0) ok = wait_all(W_OEMPTY + s, (pieces - 1) & 1);
            if (ok) ok = my_turn();
            if (sn) kready = __all_sync(0xffffffffu, mbar_try_wait(bar(W_KFULL + ks), kp));
            if (ok) ok = wait_all(W_PFULL + s, np & 1);
            ++np;
          } else {
            if (sn) ok = wait_all(W_KFULL + ks, kp);
            if (ok) ok = my_turn();
          }
          if (!ok) break;
          tc_fence_after();
          if (pv) {
            const uint32_t dV = dV0 + vs * (C::TILE >> 4);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < KT / 16; ++kk)
                mma_ts(tO, tS + kk * 8, sdesc_at(dV, kk * 2048), idPV, (i > 1 || kk > 0) ? 1u : 0u);
              if (!sn) mma_commit(bar(W_PVDONE + s));
              mma_commit(bar(W_VEMPTY + vs));
              if (!w.rows) mma_commit(bar(W_VEMPTY + vs));
            }
            __syncwarp();
            advance(vs, vp, step, C::VSTAGES);
          }
          bool given = false;
          if (sn) {
            if (!kready) kready = __all_sync(0xffffffffu, mbar_try_wait(bar(W_KFULL + ks), kp));
            if (!kready) {
              end_turn();        // K has not landed: the other slot need not wait for it
              given = true;
              ok = wait_all(W_KFULL + ks, kp);
              if (!ok) break;
              tc_fence_after();
            }
            const uint32_t dK = dK0 + ks * (C::KTILE >> 4);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < SSTEPS; ++kk) {
                s_step(tS, dK, kk);
                // the turn passes a little early: the other warp needs some
                // 250 cycles to notice
                if (SLOTS == 2 && kk == SSTEPS - 4 && !given) mbar_arrive(bar(W_TURN + s));
              }
              mma_commit(bar(W_SFULL + s));
              mma_commit(bar(W_KEMPTY + ks));
              if (!w.rows) mma_commit(bar(W_KEMPTY + ks));
            }
            __syncwarp();
            advance(ks, kp, step, C::KSTAGES);
            if (!given) ++turn;
          } else {
            end_turn();
          }
          x += step;
        }
        advance(kst, kph, w.n % (2 * C::KSTAGES), C::KSTAGES);
        advance(vst, vph, w.n % (2 * C::VSTAGES), C::VSTAGES);
        ++pieces;
      }
      if (elect_one()) {
        if (q_tma && qn > 0) mbar_wait(bar(W_QFULL + s), (qn - 1) & 1, P.status, P.wait_ns);   // the last Q has landed
        mma_commit(bar(W_DRAIN));
        mbar_wait(bar(W_DRAIN), 0, P.status, P.wait_ns);
      }
    } else if (CODES) {
      // ---------------------------------------------------------- V's codes to f16
      if constexpr (CODES) {
        const int part = SLOTS == 2 ? warp - (K_WARP + 4) : warp == V_WARP ? 0 : 1;
        uint32_t e = 0, pieces = 0;
        bool ok = true;
        while (ok && u.next(P)) {
          if (u.keys == 0) continue;
#pragma unroll 1
          for (int t = u.t0; ok && t < u.t1; ++t, ++e)
            ok = convert_v<C>(P, u, t, e, part, KT / C::CV_WARPS, lane, smem, sbase, nf_all + 8 * (pieces % 4),
                              wait_all);
          ++pieces;
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    regs_increase<C::REGS_SOFTMAX>();
    const int slot = warp >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;                 // row within the slot = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tbase + lane_off + 128 * slot;
    const uint32_t tO = tbase + lane_off + C::T_O + 128 * slot;
    float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
    // A warp whose wait gave up goes on without waiting or touching tensor
    // memory: the slots' barriers of every piece still find all eight warps.
    bool ok = true;
    uint32_t e0 = 0, pieces = 0, j = 0;                // j: tiles of this slot so far
    uint32_t pd0 = 0, pd1 = 0;                         // pieces in which slot 0 / 1 took part
    int par_of = -1;                                   // the sequence whose parents are in shared memory
    if (tid == 0) P.rec[blockIdx.x] = make_int4(-1, 0, 0, 0);
    while (u.next(P)) {
      const WideSplit w = wide_split<C::BUFS>(u);
      const int ur = w.rows ? slot * 128 + r : r;      // row of the unit
      const bool mine = ur < u.rows;
      const int rr = u.row_first + ur;
      const int node = ur < u.rows ? P.by_G(rr) : 0;
      const int h = u.hk * P.G + (ur < u.rows ? rr - node * P.G : 0);
      auto out_row = [&]() { return P.o + (u.s.row0 + node) * P.o_stride[0] + h * P.o_stride[1]; };
      auto out_lse = [&]() { return P.lse + static_cast<int64_t>(h) * P.total + u.s.row0 + node; };
      if (w.n == 0) {                                  // no keys: zeros in all its rows
        const int z = slot * 128 + r, zr = u.row_first + z, zn = P.by_G(zr), zh = u.hk * P.G + zr - zn * P.G;
        if (z < u.rows) {
          uint4* dst = reinterpret_cast<uint4*>(P.o + (u.s.row0 + zn) * P.o_stride[0] + zh * P.o_stride[1]);
#pragma unroll 1
          for (int c = 0; c < D / 8; ++c) dst[c] = make_uint4(0u, 0u, 0u, 0u);
          P.lse[static_cast<int64_t>(zh) * P.total + u.s.row0 + zn] = -INFINITY;
        }
        continue;
      }
      const bool active = w.active(slot);
      // This piece's flags, and the next piece's, read by nobody now, cleared.
      // (CODES: the warps that set them may be as many tiles ahead as V has
      // stages, and so as many pieces.)
      constexpr int AHEAD = CODES ? C::VSTAGES : 1, SETS = CODES ? 4 : 2;
      static_assert(AHEAD < SETS, "sets of flags");
      uint32_t* nf = nf_all + 8 * (pieces % SETS);
      if (tid < 8) nf_all[8 * ((pieces + AHEAD) % SETS) + tid] = 0;
      const int part0 = u.origin / KT;                 // tiles from here on are not seen by all
      bool live = mine;
      if (P.tree) {
        // the sequence's parents, in shared memory for all its units: from L2
        // a step up the tree took 700 cycles
        int16_t* par = reinterpret_cast<int16_t*>(smem + C::OFF_PAR);
        if (par_of != u.b) {
#pragma unroll 1
          for (int i = tid; i < u.s.n; i += 128 * SLOTS) par[i] = static_cast<int16_t>(tree_parent(P, u.s, i));
          slots_sync<SLOTS>();
          par_of = u.b;
        }
        if (mine) live = par[node] != -2;
      }
      // which keys from origin on the row sees: bit i is key origin + i.
      // Found again for each of the unit's few tiles that need it, which
      // leaves eight registers to the loop.
      auto row_sees = [&](uint32_t (&seen)[8]) {
        if (P.tree) {
          const int16_t* par = reinterpret_cast<const int16_t*>(smem + C::OFF_PAR);
          tree_ancestors(live ? node : -1, [&](int a) -> int { return par[a]; }, seen);
        } else {
          const int upto = u.s.base + node - u.origin;   // last visible bit
#pragma unroll
          for (int x = 0; x < 8; ++x)
            seen[x] = upto >= 32 * x + 31 ? 0xffffffffu
                                          : (upto < 32 * x ? 0u : (2u << (upto - 32 * x)) - 1u);
        }
      };
      const bool warp_live = __any_sync(0xffffffffu, live);
      float m_used = -INFINITY, l = 0.f;
      [[maybe_unused]] float back = 0.f;               // CODES: the scale, and what undoes the row's shift
      if (active) {
        // Q, where the MMA warps do not fetch it (S of the slots' earlier
        // pieces has been read): a row is copied by D / 8 lanes, so that a
        // warp's copy covers whole rows, and asynchronously past L1: the few
        // KB that shared memory leaves of it hold up plain loads of 64 KB for
        // 7000 cycles
        if (!q_tma) {
          const __nv_bfloat16* src =
              P.q + (u.s.row0 + node) * P.q_stride[0] + static_cast<int64_t>(h) * P.q_stride[1];
          constexpr int LPR = D / 8, RPI = 32 / LPR;     // lanes a row, rows an instruction
          const unsigned in_rows = __ballot_sync(0xffffffffu, mine);
          if constexpr (CODES) {
            // to two parts (see split_q), times a power of two per row; lane l keeps what undoes
            // row l's.  All loads first: behind the stream of K and V each takes some
            // 3000 cycles (four at a time 13000 of a unit's 20000 for its ends).
            uint4 x[32 / RPI];
#pragma unroll
            for (int i = 0; i < 32 / RPI; ++i) {
              const int from = i * RPI + lane / LPR;
              const uint64_t row = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(src), from);
              x[i] = make_uint4(0u, 0u, 0u, 0u);
              if ((in_rows >> from) & 1u) x[i] = *reinterpret_cast<const uint4*>(row + (lane % LPR) * 16);
            }
            // a row's largest magnitude: over the words of a lane, then over its
            // LPR lanes by halves, after which lane l of them has row l RPI's
            uint32_t top[LPR];
#pragma unroll
            for (int i = 0; i < LPR; ++i)
              top[i] = __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu));
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
              for (int i = 0; i < o; ++i) {
                const uint32_t give = lane & o ? top[i] : top[i + o], keep = lane & o ? top[i + o] : top[i];
                top[i] = __vmaxu2(keep, __shfl_xor_sync(0xffffffffu, give, o));
              }
            const uint32_t most = max(top[0] & 0xffffu, top[0] >> 16);
            const int up = row_shift(most) - 6;        // the largest at [2^7, 2^8)
            const float mul = pow2(up);
            // (an infinity has no code: its row becomes NaN, as its scores are)
            back = __shfl_sync(0xffffffffu, most < 0x7f80u ? pow2(-up) * P.scale_log2 : __int_as_float(0x7fc00000),
                               (lane % RPI) * LPR + lane / RPI);
#pragma unroll
            for (int i = 0; i < LPR; ++i) {
              const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
              uint2 hi, lo;
              split_q(w, __shfl_sync(0xffffffffu, mul, (lane & ~(LPR - 1)) + i), hi, lo);
              uint8_t* to = smem + C::OFF_Q + slot * C::QTILE +
                            Load::word16(quarter * 32 + i * RPI + lane / LPR, (lane % LPR) >> 1) + (lane & 1) * 8;
              *reinterpret_cast<uint2*>(to) = hi;
              *reinterpret_cast<uint2*>(to + 128 * D) = lo;
            }
          } else {
#pragma unroll 2
            for (int i = 0; i < 32 / RPI; ++i) {
              const int from = i * RPI + lane / LPR;
              const uint64_t row = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(src), from);
              copy_async16(sbase + C::OFF_Q + slot * C::QTILE +
                               sw128_offset(quarter * 32 + from, (lane % LPR) * 8, 128),
                           row + (lane % LPR) * 16, (in_rows >> from) & 1u ? 16 : 0);
            }
            copy_async_wait();
          }
          fence_proxy_async_smem();
          mbar_arrive_warp(bar(W_QFULL + slot));
        }
        int done = 0;
#pragma unroll 1
        for (int x0 = w.rows ? 0 : slot; x0 < w.n; x0 += w.rows ? 1 : 2) {
          const int t = u.t0 + x0;
          const bool partial = t >= part0;
          // BUFS: they alternate
          const int b_s = C::BUFS ? s_full(slot, j & 1) : W_SFULL + slot, b_p = C::BUFS ? p_full(slot, j & 1) : W_PFULL + slot;
          const uint32_t tSj = C::BUFS ? tS + 64 * (j & 1) : tS;
          const uint32_t vt = e0 + x0;
          // the tile's factors
          if (CODES && !C::V_FIRST && ok) ok = wait_all(W_VFULL + vt % C::VSTAGES, (vt / C::VSTAGES) & 1);
          if (ok) ok = wait_all(b_s, C::BUFS ? (j >> 1) & 1 : j & 1);
          tc_fence_after();
          if (ok && warp_live) {
            if (partial) {
              // what the row does not see becomes -inf, 32 columns at a time
              // and back to tensor memory: a few tiles of a unit at most, and
              // the loop below stays free of it
              uint32_t seen[8];
              row_sees(seen);
#pragma unroll 1
              for (int y = 0; y < KT / 32; ++y) {
                const int j0 = t * KT + 32 * y - u.origin;      // bit 0 is key origin + j0
                if (j0 <= -32) continue;                        // seen by all
                // the 64 bits from word (j0 >> 5) on, ones before bit 0
                const int i0 = j0 >> 5;
                uint32_t lo = i0 < 0 ? 0xffffffffu : 0u, hi = i0 + 1 < 0 ? 0xffffffffu : 0u;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  lo = i == i0 ? seen[i] : lo;
                  hi = i == i0 + 1 ? seen[i] : hi;
                }
                const uint32_t vis = __funnelshift_r(lo, hi, j0 & 31);
                uint32_t q[32];
                tmem_ld32(tSj + 32 * y, q);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 32; ++c) q[c] = (vis >> c) & 1u ? q[c] : 0xff800000u;
                tmem_st32(tSj + 32 * y, q);
              }
              tmem_wait_st();
            }
            float alpha = 1.f;                       // what the earlier tiles' O takes
            float sum4[4] = {0.f, 0.f, 0.f, 0.f};
            if constexpr (CODES) {
              // (In tiles of 128 keys with one S a slot, as the bf16 pairs, a row of
              // S spilled registers in this loop or was loaded twice, and its
              // softmax and its MMAs came one after the other: 198 us.  32 columns
              // at a time in one pass, with what had been done scaled where the
              // maximum grew: 259 us.)
              float sv[KT];
#pragma unroll
              for (int y = 0; y < KT / 32; ++y) tmem_ld32(tSj + 32 * y, reinterpret_cast<uint32_t*>(sv) + 32 * y);
              tmem_wait_ld();
              // block b's factor and log2 sv, twice each, and what the sum takes of P
              uint32_t facts = sbase + C::OFF_FACT + vt % C::VSTAGES * (C::BLOCKS * 16);
              uint32_t takes = sbase + C::OFF_FACT + (C::VSTAGES * 16 + vt % C::VSTAGES * 4) * C::BLOCKS;
              // (the addresses only from here on, after the wait for S: the loads
              // themselves may be moved)
              asm volatile("" : "+r"(facts), "+r"(takes)::"memory");
              auto factors = [&](int b, uint64_t& k, uint64_t& v) {
                asm("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(k), "=l"(v) : "r"(facts + b * 16));
              };
              float m_tile = -INFINITY;
#pragma unroll
              for (int b = 0; b < C::BLOCKS; ++b) {
                const float* s = sv + 16 * b;
                uint64_t k, v;
                factors(b, k, v);
                float a[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) a[y] = fmax3(s[y], s[y + 4], s[y + 8]);
                const float top = fmax3(fmax3(a[0], s[12], a[1]), fmax3(s[13], a[2], s[14]), fmaxf(a[3], s[15]));
                m_tile = fmaxf(m_tile, fmaf(top, score_factor(__uint_as_float(static_cast<uint32_t>(k)), back),
                                            __uint_as_float(static_cast<uint32_t>(v))));
              }
              // the reference moves only when the maximum grows by more than
              // 2^8 (as in the prompt forward): few tiles rescale O
              const bool grow = m_tile > m_used + 8.f;
              const float m_new = grow ? m_tile : m_used;
              alpha = grow ? ex2(m_used - m_new) : 1.f;
              l *= alpha;
              m_used = m_new;
              const uint64_t shift2 = splat2(kPOffset - (m_used == -INFINITY ? 0.f : m_used));
#pragma unroll
              for (int b = 0; b < C::BLOCKS; ++b) {
                uint64_t k, v;
                float take;
                factors(b, k, v);
                asm("ld.shared.f32 %0, [%1];" : "=f"(take) : "r"(takes + b * 4));
                const uint64_t sc2 = splat2(score_factor(__uint_as_float(static_cast<uint32_t>(k)), back));
                const uint64_t nm2 = add2(v, shift2);
                uint32_t pk[8];
                float s0 = 0.f, s1 = 0.f;
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                  float a0, a1;
                  fma2_bc(a0, a1, sv[b * 16 + 2 * y], sv[b * 16 + 2 * y + 1], sc2, nm2);
                  const float p0 = ex2(a0), p1 = ex2(a1);
                  add2_acc(s0, s1, p0, p1);
                  pk[y] = pack_f16(p0, p1);
                }
                sum4[b & 3] = fmaf(s0 + s1, take, sum4[b & 3]);
                tmem_st8(tSj + b * 8, pk);
              }
            } else {
              float sv[KT];
              uint32_t* raw = reinterpret_cast<uint32_t*>(sv);
#pragma unroll
              for (int y = 0; y < KT / 32; ++y) tmem_ld32(tSj + 32 * y, raw + 32 * y);
              tmem_wait_ld();
              float mx8[8];
#pragma unroll
              for (int y = 0; y < 8; ++y) mx8[y] = fmax3(sv[y], sv[y + 8], sv[y + 16]);
#pragma unroll
              for (int c = 24; c < KT - 8; c += 16)
#pragma unroll
                for (int y = 0; y < 8; ++y) mx8[y] = fmax3(mx8[y], sv[c + y], sv[c + 8 + y]);
#pragma unroll
              for (int y = 0; y < 8; ++y) mx8[y] = fmaxf(mx8[y], sv[KT - 8 + y]);
              const float mx = fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]),
                                     fmaxf(mx8[6], mx8[7]));
              // the reference moves only when the maximum grows by more than
              // 2^8 (as in the prompt forward): few tiles rescale O
              const float m_tile = mx * P.scale_log2;
              const bool grow = m_tile > m_used + 8.f;
              const float m_new = grow ? m_tile : m_used;
              alpha = grow ? ex2(m_used - m_new) : 1.f;
              l *= alpha;
              m_used = m_new;
              const float m_ref = m_used == -INFINITY ? 0.f : m_used;
              const uint64_t sc2 = splat2(P.scale_log2), nm2 = splat2(-m_ref);
#pragma unroll
              for (int c4 = 0; c4 < KT / 32; ++c4) {
                uint32_t pk[16];
#pragma unroll
                for (int y = 0; y < 16; ++y) {
                  float a0, a1;
                  fma2_bc(a0, a1, sv[c4 * 32 + 2 * y], sv[c4 * 32 + 2 * y + 1], sc2, nm2);
                  const float p0 = ex2(a0), p1 = ex2(a1);
                  if (y & 1) add2_acc(sum4[2], sum4[3], p0, p1);
                  else add2_acc(sum4[0], sum4[1], p0, p1);
                  pk[y] = pack_bf16(p0, p1);   // P in bf16 for the product; the sum keeps 32 bits
                }
                tmem_st16(tSj + c4 * 16, pk);
              }
            }
            if (done > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
              // O holds the PVs of the earlier tiles; with two S buffers the
              // last one may still run
              if (C::BUFS) {
                ok = wait_all(pv_tile(slot), (j - 1) & 1);
                tc_fence_after();
              }
#pragma unroll 1
              for (int y = 0; y < D / 32; ++y) {
                uint32_t ro[32];
                tmem_ld32(tO + 32 * y, ro);
                tmem_wait_ld();
#pragma unroll
                for (int z = 0; z < 32; ++z) ro[z] = __float_as_uint(__uint_as_float(ro[z]) * alpha);
                tmem_st32(tO + 32 * y, ro);
              }
            }
            l += (sum4[0] + sum4[1]) + (sum4[2] + sum4[3]);
            tmem_wait_st();
          }
          if (!CODES && partial && ok) {
            // clean row r of the V tile (see fix_row) before the product
            const uint32_t e = e0 + x0, st = e % C::VSTAGES;
            ok = wait_all(W_VFULL + st, (e / C::VSTAGES) & 1);
            if (ok) {
              const int key = t * KT + r, i = key - u.origin;
              // 16-byte words of the row, the slabs KT * 128 bytes apart; the
              // lanes start at different words (bank conflicts)
              uint8_t* v = smem + C::OFF_V + st * C::TILE + r * 128;
              auto word = [&](int c) {
                return reinterpret_cast<uint4*>(v + (c >> 3) * (KT * 128) + ((c ^ r) & 7) * 16);
              };
              bool dirty = false;
              if (r >= KT) {
                // the tile has no row for this thread
              } else if (key >= u.keys) {
#pragma unroll 1
                for (int c = 0; c < D / 8; ++c) *word(c) = make_uint4(0u, 0u, 0u, 0u);
              } else if (i >= 0) {
                uint32_t zero = 0;             // 0, or NaN once a value was not finite
#pragma unroll 4
                for (int c = 0; c < D / 8; ++c) {
                  const uint4 y = *word(c);
                  zero = bf16x2_times_zero(y.x, zero);
                  zero = bf16x2_times_zero(y.y, zero);
                  zero = bf16x2_times_zero(y.z, zero);
                  zero = bf16x2_times_zero(y.w, zero);
                }
                dirty = bf16x2_not_finite(zero);
              }
              if (dirty) {
                // the flag first: whoever finds the row clean finds the flag
                atomicOr(nf + (i >> 5), 1u << (i & 31));
                __threadfence_block();
#pragma unroll 1
                for (int c = 0; c < D / 8; ++c) {
                  uint4* y = word(c);
                  *y = make_uint4(bf16x2_clean(y->x), bf16x2_clean(y->y), bf16x2_clean(y->z),
                                  bf16x2_clean(y->w));
                }
              }
              fence_proxy_async_smem();
            }
          }
          tc_fence_before();
          // (a test of the wait limit withholds the first one of slot 0: its
          // MMA warp's wait then runs out)
          if (!(P.withhold == 8 && slot == 0 && j == 0)) mbar_arrive_warp(bar(b_p));
          ++j;
          ++done;
        }
      }
      if (!live) {                // a padding node's row sees nothing, the context included
        m_used = -INFINITY;
        l = 0.f;
      }

      // ---------------------------------------------------------- the piece's end
      const bool two = !C::BUFS && !w.rows && w.n > 1; // O is in both slots
      int c0 = 0, c1 = D;                              // columns that this thread writes
      float m_out = m_used, l_out = l, f0 = 1.f, f1 = 0.f;
      if (!C::BUFS && !w.rows) {
        ml[slot * 128 + r] = make_float2(m_used, l);
        slots_sync<SLOTS>();
        const float2 a = ml[r], b = two ? ml[128 + r] : make_float2(-INFINITY, 0.f);
        m_out = fmaxf(a.x, b.x);
        // negative: that slot's keys were not seen.  A weight of 0 is no such
        // sign: a NaN under it counts
        f0 = a.y != 0.f ? ex2(a.x - m_out) : -1.f;
        f1 = b.y != 0.f ? ex2(b.x - m_out) : -1.f;
        l_out = (a.y != 0.f ? a.y * f0 : 0.f) + (b.y != 0.f ? b.y * f1 : 0.f);
        c0 = slot * (D / 2);
        c1 = c0 + D / 2;
      }
      if (ok && (!w.rows || slot == 0)) ok = wait_all(W_PVDONE, pd0 & 1);
      if (ok && (w.rows ? slot == 1 : two)) ok = wait_all(W_PVDONE + 1, pd1 & 1);
      pd0 += w.active(0);
      pd1 += w.active(1);
      tc_fence_after();
      const bool whole = u.whole();
      const bool writes = mine && ok;
      constexpr float undo = CODES ? kPUndo : 1.f;     // P's offset
      const float inv = whole ? (l_out > 0.f ? undo / l_out : (l_out == 0.f ? 0.f : l_out)) : undo;
      const int slot_part = 2 * blockIdx.x + (u.t0 == 0 ? 1 : 0);
      const int64_t at = static_cast<int64_t>(slot_part) * P.part_rows + ur;
      float* const prow = P.part_o + at * D;
      __nv_bfloat16* const orow = out_row();
      // O by blocks of 32 columns; each passes through the warp's part of the
      // slot's Q buffer (no longer needed), so that the stores cover whole
      // runs of a row: 64 bytes (bf16) or 128 bytes (fp32 parts)
      uint8_t* stage = smem + C::OFF_Q + slot * C::QTILE + quarter * 4096;
      const unsigned out_rows = __ballot_sync(0xffffffffu, writes);
#pragma unroll 1
      for (int cb = c0 / 32; cb < c1 / 32; ++cb) {
        float v[32];
        uint32_t* raw = reinterpret_cast<uint32_t*>(v);
        if (ok) {
          tmem_ld32(w.rows ? tO + cb * 32 : tbase + lane_off + C::T_O + cb * 32, raw);
          if (two) {
            uint32_t rb[32];
            tmem_ld32(tbase + lane_off + C::T_O + 128 + cb * 32, rb);
            tmem_wait_ld();
#pragma unroll
            for (int y = 0; y < 32; ++y)
              v[y] = (f0 < 0.f ? 0.f : v[y] * f0) + (f1 < 0.f ? 0.f : __uint_as_float(rb[y]) * f1);
          } else {
            tmem_wait_ld();
          }
        }
#pragma unroll
        for (int y = 0; y < 32; ++y) v[y] = l_out == 0.f ? 0.f : v[y] * inv;
        // 16-byte words of a row's 32 columns: 4 (bf16) or 8 (fp32), stored
        // at their number xor the row's
        if (whole) {
          uint4* own = reinterpret_cast<uint4*>(stage) + lane * 4;
#pragma unroll
          for (int y = 0; y < 4; ++y)
            own[y ^ ((lane >> 1) & 3)] =
                make_uint4(pack_bf16(v[8 * y], v[8 * y + 1]), pack_bf16(v[8 * y + 2], v[8 * y + 3]),
                           pack_bf16(v[8 * y + 4], v[8 * y + 5]), pack_bf16(v[8 * y + 6], v[8 * y + 7]));
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = i * 8 + lane / 4, word = lane % 4;
            const uint64_t dst = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(orow), row);
            if ((out_rows >> row) & 1u)
              reinterpret_cast<uint4*>(dst)[cb * 4 + word] =
                  reinterpret_cast<const uint4*>(stage)[row * 4 + (word ^ ((row >> 1) & 3))];
          }
        } else {
          uint4* own = reinterpret_cast<uint4*>(stage) + lane * 8;
#pragma unroll
          for (int y = 0; y < 8; ++y)
            own[y ^ (lane & 7)] = make_uint4(raw[4 * y], raw[4 * y + 1], raw[4 * y + 2], raw[4 * y + 3]);
          __syncwarp();
          // a part's rows lie one after the other
          uint4* dst = reinterpret_cast<uint4*>(prow - static_cast<int64_t>(lane) * D) + cb * 8;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int row = i * 4 + lane / 8, word = lane % 8;
            if ((out_rows >> row) & 1u)
              dst[row * (D / 4) + word] = reinterpret_cast<const uint4*>(stage)[row * 8 + (word ^ (row & 7))];
          }
        }
        __syncwarp();
      }
      if (q_tma) {
        fence_proxy_async_smem();
        mbar_arrive_warp(bar(W_QEMPTY));
      }
      tc_fence_before();
      if (w.rows) {
        // for each of this slot's warps, and those of the other
        __syncwarp();
        if (lane == 0) mbar_arrive_count(bar(W_OEMPTY + slot), SLOTS);
      } else {
        mbar_arrive_warp(bar(W_OEMPTY));
        mbar_arrive_warp(bar(W_OEMPTY + 1));
      }
      if (writes) {
        if (c0 == 0) {
          if (whole) {
            const float m_ref = m_out == -INFINITY ? 0.f : m_out;
            *out_lse() = l_out == 0.f ? -INFINITY : (m_ref + __log2f(l_out)) * 0.69314718055994530942f;
          } else {
            P.part_ml[at] = make_float2(m_out, l_out);
          }
        }
        uint32_t any = 0;
#pragma unroll
        for (int x = 0; x < 8; ++x) any |= nf[x];
        if (any) {
          uint32_t seen[8];
          row_sees(seen);
          const uint4 s0 = make_uint4(seen[0], seen[1], seen[2], seen[3]);
          const uint4 s1 = make_uint4(seen[4], seen[5], seen[6], seen[7]);
          if constexpr (CODES) {
            if (whole) fix_row8(A, u.b, u.hk, u.origin, nf, s0, s1, c0, c1 - c0, orow + c0);
            else fix_row8(A, u.b, u.hk, u.origin, nf, s0, s1, c0, c1 - c0, prow + c0);
          } else {
            if (whole) fix_row(P, u.b, u.hk, u.origin, nf, s0, s1, c0, c1 - c0, orow + c0);
            else fix_row(P, u.b, u.hk, u.origin, nf, s0, s1, c0, c1 - c0, prow + c0);
          }
        }
      }
      if (tid == 0) leave_record(P, u, blockIdx.x);
      e0 += w.n;
      ++pieces;
      slots_sync<SLOTS>();        // ml and nf have been read, and S of both slots
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tbase, C::T_COLS);
  }
}

template <int D, int SLOTS, bool CODES>
static fm_status launch_wide_d(const WideParams<CODES>& P, const CUtensorMap& tq, const CUtensorMap& tk,
                               const CUtensorMap& tv, int grid, cudaStream_t s) {
  using C = WideCfg<D, SLOTS, CODES>;
  auto kern = tree_wide_kernel<D, SLOTS, CODES>;
  // the setmaxnreg split must fit in the registers the block launches with
  static std::atomic<uint64_t> ready{0};
  const fm_status st = prepare_kernel(kern, C::SMEM, C::MIN_LAUNCH_REGS, ready);
  if (st != FM_OK) return st;
  prof_begin(K_TREE, s);
  const cudaError_t e = launch_dependent(kern, dim3(grid), C::THREADS, C::SMEM, s, P, tq, tk, tv);
  prof_end(K_TREE, s);
  return e == cudaSuccess ? FM_OK : FM_ERR_CUDA;
}

fm_status launch_tree_mid(const TreeParams& P, int d, const CUtensorMap& tq, const CUtensorMap& tk,
                          const CUtensorMap& tv, int grid, cudaStream_t s) {
  return d == 64 ? launch_wide_d<64, 1, false>(P, tq, tk, tv, grid, s)
                 : launch_wide_d<128, 1, false>(P, tq, tk, tv, grid, s);
}

fm_status launch_tree_wide(const TreeParams& P, const CUtensorMap& tq, const CUtensorMap& tk,
                           const CUtensorMap& tv, int grid, cudaStream_t s) {
  return launch_wide_d<128, 2, false>(P, tq, tk, tv, grid, s);
}

fm_status launch_tree8_wide(const Tree8Params& A, const CUtensorMap& tk, const CUtensorMap& tv, int grid,
                            cudaStream_t s) {
  return launch_wide_d<128, 2, true>(A, tk, tk, tv, grid, s);
}

fm_status launch_tree8_mid(const Tree8Params& A, int d, const CUtensorMap& tk, const CUtensorMap& tv, int grid,
                           cudaStream_t s) {
  return d == 64 ? launch_wide_d<64, 1, true>(A, tk, tk, tv, grid, s)
                 : launch_wide_d<128, 1, true>(A, tk, tk, tv, grid, s);
}

}  // namespace fm
