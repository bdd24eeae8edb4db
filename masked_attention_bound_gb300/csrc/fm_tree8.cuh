// Attention over a paged cache of e4m3 codes: what its kernels share.
//
// With sk and sv the scales of a key's block, the score of key j is x_j =
// scale log2(e) (sk q . k8_j) and O = sum_j 2^x_j sv v8_j / sum_j 2^x_j.  sv
// goes into the exponent: P_j = 2^(x_j + log2 sv - R), with R the running
// maximum of x_j + log2 sv, is what multiplies the codes of V, and the sum of
// the weights takes P_j / sv, a factor per block of 16 keys.  So no element is
// multiplied by its scale, and neither are K's: a factor per block and row
// goes into the exponent's multiply-add.
//
// The products' operands are f16, which holds every code exactly.  Q is
// multiplied by a power of two per row that brings its largest element to
// 2^13 at least: every element within 2^-27 of that one then has all its bits
// in f16, and what is below is off by 2^-38 of it at most.  P is offset by
// 2^7 (R moves when the maximum has grown by more than 2^8), so that f16 holds
// it with 11 bits down to 2^-21 of the largest and with an error of 2^-32 of
// that below; its rounding, 2^-11 at most of a weight, is an eighth of the
// output's.  Sums, maxima, scores and O are fp32.
#pragma once
#include "fm_fp8.cuh"
#include "fm_tree.h"

namespace fm {

struct Tree8Params {
  TreeParams P;                  // v_stride in elements of the codes
  const float *k_scale, *v_scale;
  const uint8_t* v_pool;
};

constexpr float kPOffset = 7.f, kPUndo = 0x1p-7f;

// ---------------------------------------------------------------- loads
// One KT-key tile of codes of K or V into shared memory by TMA: boxes of
// min(page_size, KT) rows of D bytes, swizzled by 16-byte words as wide as
// the row (word16), and the scales of its KT / 16 blocks by asynchronous
// copies.  A stage's barrier counts 1 + KT / 16 arrivals.  Boxes past the
// unit's keys are not loaded, their blocks' scales are 0 (read as the least).
template <int D, int KT>
struct TileLoad8 {
  static constexpr int BLOCKS = KT / kScaleBlock;
  static constexpr int ARRIVALS = 1 + BLOCKS;
  // the lanes' pages: lane l has box l's, as TileLoad's
  __device__ static __forceinline__ int boxes(const TreeParams& P, const TreePiece& u, int tile) {
    const int keys = min(u.keys - tile * KT, KT);
    return keys <= 0 ? 0 : (keys + (1 << P.box_shift) - 1) >> P.box_shift;
  }
  __device__ static __forceinline__ int lane_page(const TreeParams& P, const TreePiece& u, int tile, int lane) {
    if (lane >= boxes(P, u, tile)) return P.n_pages;
    const int pg = P.table[static_cast<int64_t>(u.b) * P.max_pages + ((tile * KT + (lane << P.box_shift)) >> P.page_shift)];
    if (pg >= 0 && pg < P.n_pages) return pg;
    if (P.status) atomicOr(P.status, DEV_CACHE);
    return P.n_pages;
  }
  __device__ static __forceinline__ void issue(const TreeParams& P, const TreePiece& u, int tile, int lane,
                                               int page, const CUtensorMap* tm, const float* scales,
                                               uint32_t dst, uint32_t dst_scales, uint32_t bar, uint64_t policy) {
    const int n = boxes(P, u, tile);
    if (lane == 0) mbar_arrive_expect_tx(bar, (n << P.box_shift) * D);
    __syncwarp();
    const int in_page = (1 << P.page_shift) - 1;
    if (lane < n)
      tma_load_4d_hint(dst + (lane << P.box_shift) * D, tm, bar, 0, u.hk, (tile * KT + (lane << P.box_shift)) & in_page,
                       page, policy);
    // block i of the tile lies in box i * 16 >> box_shift
    const int key = tile * KT + lane * kScaleBlock;
    const int pg = __shfl_sync(0xffffffffu, page, (lane * kScaleBlock) >> P.box_shift);
    if (lane < BLOCKS) {
      const bool there = pg < P.n_pages;
      const float* src = there ? scales + (((static_cast<int64_t>(pg) * P.Hkv + u.hk) << (P.page_shift - kScaleShift)) +
                                           ((key & in_page) >> kScaleShift))
                               : scales;
      asm volatile(
          "cp.async.ca.shared.global [%0], [%1], 4, %2;\n\t"
          "cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%3];" ::"r"(dst_scales + lane * 4),
          "l"(src), "r"(there ? 4 : 0), "r"(bar)
          : "memory");
    }
  }
  // place of the 16-byte word c of row r of the tile
  __device__ static __forceinline__ uint32_t word16(int r, int c) {
    return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  }
};

// ---------------------------------------------------------------- NaN of V
// As fix_row of a bf16 cache: keys at or past `origin` are cleaned of NaN (the
// one code that is not finite) in shared memory, and the rows that do see such
// a key get it here.
template <typename T>
static __device__ __noinline__ void fix_row8(const Tree8Params& A, int b, int hk, int origin, const uint32_t* nf,
                                             const uint32_t* seen, int c0, int n, T* row) {
  const TreeParams& P = A.P;
#pragma unroll 1
  for (int w = 0; w < 8; ++w) {
    uint32_t bits = nf[w] & seen[w];
#pragma unroll 1
    while (bits) {
      const int pos = origin + w * 32 + __ffs(bits) - 1;
      bits &= bits - 1;
      const int pg = P.table[static_cast<int64_t>(b) * P.max_pages + (pos >> P.page_shift)];
      if (pg < 0 || pg >= P.n_pages) continue;
      const uint8_t* v = A.v_pool + pg * P.v_stride[0] + (pos & ((1 << P.page_shift) - 1)) * P.v_stride[1] +
                         hk * P.v_stride[2] + c0;
#pragma unroll 1
      for (int i = 0; i < n; ++i)
        if ((v[i] & 0x7f) == 0x7f) row[i] = static_cast<T>(__int_as_float(0x7fc00000));
    }
  }
}

fm_status launch_tree8_narrow(const Tree8Params& A, int d, int rows, const CUtensorMap& tk, const CUtensorMap& tv,
                              int grid, cudaStream_t s);
// Joins the parts that the first kernel left (fm_tree.cu); rows: of its units.
fm_status launch_tree_join(const TreeParams& P, int d, int rows, int grid, cudaStream_t s);

}  // namespace fm
