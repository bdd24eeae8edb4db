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
// TMEM: S/P of slot s at column 128 s (SLOTS = 1: of every second tile at
// column 64), the O's after the S's.
#include <type_traits>

#include "fm_tree.h"

namespace fm {

template <int D, int SLOTS_>
struct WideCfg {
  static constexpr int SLOTS = SLOTS_;
  static_assert(D == 128 || SLOTS == 1, "d = 64 runs with tiles of 128 rows side by side");
  using Geo = std::conditional_t<SLOTS == 2, WideGeo, MidGeo>;
  static constexpr int KT = Geo::KT;
  static constexpr int TILE = KT * D * 2;               // bytes of a K or V tile
  static constexpr int QTILE = 128 * D * 2;             // of a slot's Q
  static constexpr int KSTAGES = D == 64 ? 4 : 2, VSTAGES = D == 64 ? 5 : 3;
  static constexpr int SM_WARPS = 4 * SLOTS;            // softmax
  static constexpr int THREADS = 32 * (SM_WARPS + 4);
  static constexpr int BLOCKS = SLOTS == 2 ? 1 : 2;     // per SM
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = SLOTS * QTILE;
  static constexpr int OFF_V = OFF_K + KSTAGES * TILE;
  static constexpr int OFF_ML = OFF_V + VSTAGES * TILE; // SLOTS 2: float2 [slot][128]
  static constexpr int OFF_NF = OFF_ML + (SLOTS == 2 ? 2 * 128 * 8 : 0);   // [2][8] keys with values not finite
  static constexpr int OFF_BAR = OFF_NF + 64;
  static constexpr int NBAR = 34;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;   // abort flag, TMEM address
  static constexpr int OFF_PAR = OFF_MISC + 16;         // int16 [256] parents of the unit's nodes
  static constexpr int USED = OFF_PAR + 512;
  static constexpr int SMEM = USED;
  static_assert(BLOCKS * (SMEM + 1024) <= 228 * 1024, "blocks per SM");
  // O is written through 4 KB per softmax warp, in its slot's Q tile: that
  // slot's S have all been read by then
  static_assert(4 * 4096 <= QTILE, "room for the output's staging");
  static constexpr uint32_t T_COLS = 256 * SLOTS, T_O = 128 * SLOTS;
  // register split: the softmax warpgroups' and the others' budgets add up to
  // what the block is launched with (384 x 168, 256 x 128)
  static constexpr uint32_t REGS_SOFTMAX = SLOTS == 2 ? 216 : 184, REGS_PRODUCER = 72;
  static constexpr int MIN_LAUNCH_REGS =
      (32 * SM_WARPS * REGS_SOFTMAX + 128 * REGS_PRODUCER + THREADS - 1) / THREADS;
};

enum {
  W_QFULL = 0, W_SFULL = 2, W_PFULL = 4, W_PVDONE = 6, W_OEMPTY = 8, W_KFULL = 10, W_KEMPTY = 15,
  W_VFULL = 20, W_VEMPTY = 25, W_DRAIN = 30, W_TURN = 31, W_QEMPTY = 33,
  W_PVTILE = W_PVDONE + 1   // SLOTS 1: the PV of each tile (the SFULL and PFULL are its two buffers')
};

// How the slots share a piece.
struct WideSplit {
  bool rows;     // slots split the rows (else the key tiles)
  int n;         // key tiles of the piece
  // slot s takes part at all
  __device__ __forceinline__ bool active(int s) const { return s == 0 || rows || n > 1; }
};
template <int SLOTS>
__device__ __forceinline__ WideSplit wide_split(const TreePiece& u) {
  return WideSplit{SLOTS == 1 || u.rows > 128, u.keys > 0 ? u.t1 - u.t0 : 0};
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

template <int D, int SLOTS>
__global__ void __launch_bounds__(WideCfg<D, SLOTS>::THREADS, WideCfg<D, SLOTS>::BLOCKS)
    tree_wide_kernel(const __grid_constant__ TreeParams P, const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
  using C = WideCfg<D, SLOTS>;
  using Load = TileLoad<D, C::KT>;
  constexpr int KT = C::KT;
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
  const bool q_tma = SLOTS == 2 && P.q_tma;

  if (warp == 2) touch_memory<D>(P, lane);
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(W_QFULL + s), q_tma ? 1 : 4);   // else one arrival per softmax warp of the slot
      mbar_init(bar(W_SFULL + s), 1);
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
      mbar_init(bar(W_VFULL + i), 1);
      mbar_init(bar(W_VEMPTY + i), SLOTS);
    }
    mbar_init(bar(W_DRAIN), SLOTS);
    mbar_init(bar(W_QEMPTY), C::SM_WARPS);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (tid < 16) nf_all[tid] = 0;
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
  TreeWalk<typename C::Geo> u(tree_run<typename C::Geo>(P));
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;

  auto wait = [&](int b, uint32_t parity) -> bool { return tree_wait(bar(b), parity, P, abort_flag); };
  // every lane gets the same answer
  auto wait_all = [&](int b, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, wait(b, parity));
  };

  if (warp >= C::SM_WARPS) {
    regs_decrease<C::REGS_PRODUCER>();
    if (warp == K_WARP || warp == V_WARP) {
      // ---------------------------------------------------------- K / V loads
      const bool isk = warp == K_WARP;
      const int stages = isk ? C::KSTAGES : C::VSTAGES;
      const int b_full = isk ? W_KFULL : W_VFULL, b_empty = isk ? W_KEMPTY : W_VEMPTY;
      const uint32_t buf = sbase + (isk ? C::OFF_K : C::OFF_V);
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
          Load::issue(P, u, t, lane, page, tm, buf + st * C::TILE, bar(b_full + st), policy);
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
        for (uint32_t x = issued > stages ? issued - stages : 0; x < issued; ++x)
          mbar_wait(bar(b_full + x % stages), (x / stages) & 1, P.status, P.wait_ns);
      __syncwarp();
    } else if (warp == MMA_WARP || (SLOTS == 2 && warp == MMA_WARP_B)) {
      // ---------------------------------------------------------- MMA issuers
      // The whole warp walks and waits, and one elected lane issues: the
      // descriptors are then uniform, and an MMA costs its issue only.
      const int s = warp == MMA_WARP ? 0 : 1;
      constexpr uint32_t idS = idesc_bf16(128, KT, false, false);
      constexpr uint32_t idPV = idesc_bf16(128, D, false, true);
      const uint32_t dQ = sdesc_lo(sbase + C::OFF_Q + s * C::QTILE, 16);
      const uint32_t dK0 = sdesc_lo(sbase + C::OFF_K, 16);
      const uint32_t dV0 = sdesc_lo(sbase + C::OFF_V, KT * 128);
      const uint32_t tS = tbase + 128 * s, tO = tbase + C::T_O + 128 * s;
      uint32_t kst = 0, kph = 0, vst = 0, vph = 0;   // stages and phases of the next tile of the block
      uint32_t pieces = 0;      // pieces with keys before this one
      uint32_t qn = 0, np = 0;  // Q tiles, P tiles of this slot so far
      uint32_t turn = 0;        // turns taken
      bool ok = true;
      while (ok && u.next(P)) {
        const WideSplit w = wide_split<SLOTS>(u);
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
        if constexpr (SLOTS == 1) {
          // S of tile x + 1 overwrites P of tile x - 1, whose PV this warp has
          // issued before; then PV of tile x
          auto issue_s = [&](uint32_t tile) {
            const uint32_t dK = dK0 + ks * (C::TILE >> 4);
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                mma_ss(tS + 64 * (tile & 1), sdesc_at(dQ, (kk >> 2) * (128 * 128) + (kk & 3) * 32),
                       sdesc_at(dK, (kk >> 2) * (KT * 128) + (kk & 3) * 32), idS, kk > 0 ? 1u : 0u);
              mma_commit(bar(W_SFULL + (tile & 1)));
              mma_commit(bar(W_KEMPTY + ks));
            }
            __syncwarp();
            advance(ks, kp, 1, C::KSTAGES);
          };
          if (ok) ok = wait_all(W_KFULL + ks, kp);
          if (ok) issue_s(np);
#pragma unroll 1
          for (int x = 0; ok && x < w.n; ++x, ++np) {
            if (x + 1 < w.n) {
              ok = wait_all(W_KFULL + ks, kp);
              if (!ok) break;
              issue_s(np + 1);
            }
            ok = wait_all(W_VFULL + vs, vp);
            // O is overwritten: the last piece's must have been read
            if (ok && x == 0 && pieces > 0) ok = wait_all(W_OEMPTY, (pieces - 1) & 1);
            if (ok) ok = wait_all(W_PFULL + (np & 1), (np >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t dV = dV0 + vs * (C::TILE >> 4), tP = tS + 64 * (np & 1);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < KT / 16; ++kk)
                mma_ts(tO, tP + kk * 8, sdesc_at(dV, kk * 2048), idPV, (x > 0 || kk > 0) ? 1u : 0u);
              mma_commit(bar(W_PVTILE));
              if (x + 1 == w.n) mma_commit(bar(W_PVDONE));
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
            const uint32_t dK = dK0 + ks * (C::TILE >> 4);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                mma_ss(tS, sdesc_at(dQ, (kk >> 2) * (128 * 128) + (kk & 3) * 32),
                       sdesc_at(dK, (kk >> 2) * (KT * 128) + (kk & 3) * 32), idS, kk > 0 ? 1u : 0u);
                // the turn passes a little early: the other warp needs some
                // 250 cycles to notice
                if (SLOTS == 2 && kk == D / 16 - 4 && !given) mbar_arrive(bar(W_TURN + s));
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
      const WideSplit w = wide_split<SLOTS>(u);
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
      uint32_t* nf = nf_all + 8 * (pieces & 1);
      if (tid < 8) nf_all[8 * ((pieces + 1) & 1) + tid] = 0;   // the next piece's, read by nobody now
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
#pragma unroll 2
          for (int i = 0; i < 32 / RPI; ++i) {
            const int from = i * RPI + lane / LPR;
            const uint64_t row = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(src), from);
            copy_async16(sbase + C::OFF_Q + slot * C::QTILE +
                             sw128_offset(quarter * 32 + from, (lane % LPR) * 8, 128),
                         row + (lane % LPR) * 16, (in_rows >> from) & 1u ? 16 : 0);
          }
          copy_async_wait();
          fence_proxy_async_smem();
          mbar_arrive_warp(bar(W_QFULL + slot));
        }
        int done = 0;
#pragma unroll 1
        for (int x0 = w.rows ? 0 : slot; x0 < w.n; x0 += w.rows ? 1 : 2) {
          const int t = u.t0 + x0;
          const bool partial = t >= part0;
          // SLOTS 1: the buffers alternate
          const int buf = SLOTS == 1 ? j & 1 : slot;
          const uint32_t tSj = SLOTS == 1 ? tS + 64 * (j & 1) : tS;
          if (ok) ok = wait_all(W_SFULL + buf, SLOTS == 1 ? (j >> 1) & 1 : j & 1);
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
            const float alpha = grow ? ex2(m_used - m_new) : 1.f;
            l *= alpha;
            m_used = m_new;
            const float m_ref = m_used == -INFINITY ? 0.f : m_used;
            const uint64_t sc2 = splat2(P.scale_log2), nm2 = splat2(-m_ref);
            float sum4[4] = {0.f, 0.f, 0.f, 0.f};
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
            if (done > 0 && __any_sync(0xffffffffu, grow)) {
              // O holds the PVs of the earlier tiles; with two S buffers the
              // last one may still run
              if (SLOTS == 1) {
                ok = wait_all(W_PVTILE, (j - 1) & 1);
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
          if (partial && ok) {
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
          if (!(P.withhold == 8 && slot == 0 && j == 0)) mbar_arrive_warp(bar(W_PFULL + buf));
          ++j;
          ++done;
        }
      }
      if (!live) {                // a padding node's row sees nothing, the context included
        m_used = -INFINITY;
        l = 0.f;
      }

      // ---------------------------------------------------------- the piece's end
      const bool two = !w.rows && w.n > 1;             // O is in both slots
      int c0 = 0, c1 = D;                              // columns that this thread writes
      float m_out = m_used, l_out = l, f0 = 1.f, f1 = 0.f;
      if (!w.rows) {
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
      const float inv = whole ? (l_out > 0.f ? 1.f / l_out : (l_out == 0.f ? 0.f : l_out)) : 1.f;
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
          if (whole) fix_row(P, u.b, u.hk, u.origin, nf, s0, s1, c0, c1 - c0, orow + c0);
          else fix_row(P, u.b, u.hk, u.origin, nf, s0, s1, c0, c1 - c0, prow + c0);
        }
      }
      if (tid == 0) leave_record(P, u);
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

template <int D, int SLOTS>
static fm_status launch_wide_d(const TreeParams& P, const CUtensorMap& tq, const CUtensorMap& tk,
                               const CUtensorMap& tv, int grid, cudaStream_t s) {
  using C = WideCfg<D, SLOTS>;
  auto kern = tree_wide_kernel<D, SLOTS>;
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
  return d == 64 ? launch_wide_d<64, 1>(P, tq, tk, tv, grid, s) : launch_wide_d<128, 1>(P, tq, tk, tv, grid, s);
}

fm_status launch_tree_wide(const TreeParams& P, const CUtensorMap& tq, const CUtensorMap& tk,
                           const CUtensorMap& tv, int grid, cudaStream_t s) {
  return launch_wide_d<128, 2>(P, tq, tk, tv, grid, s);
}

}  // namespace fm
