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
// The codes are exact operands: as they are for tcgen05.mma's S = Q K^T, as
// f16 otherwise.  Q is multiplied by a power of two per row.  For the kernel of
// few rows that brings its largest element to 2^13 at least, and it becomes
// f16: every element within 2^-27 of the largest has all its bits, and what is
// below is off by 2^-38 of it at most.  For tcgen05, whose operands have one
// width, Q is the sum of two 8-bit numbers, with the largest element at 2^7 or
// more: the nearest e4m3 one (4 of its 8 bits) and the rest, which is at most 8
// of the bf16's last steps and so has the 3 bits of e5m2, whose range goes on
// to 2^-16 where e4m3's ends at 2^-9.  Elements within 2^-13 of the largest are
// exact, and what is below is off by 2^-21 of it at most.  (Two products at the
// 8-bit rate take as long as one of f16, and K needs no conversion: with
// f16 tiles of K too, 16 trees of 64 nodes took 373 us.)  P is f16 and offset by
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
// copies.  Boxes past the unit's keys are not loaded, their blocks' scales are
// 0 (read as the least).
template <int D, int KT>
struct TileLoad8 {
  static constexpr int BLOCKS = KT / kScaleBlock;
  static constexpr int ARRIVALS = 1 + BLOCKS;    // of a barrier for codes and scales
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
  __device__ static __forceinline__ void issue(const TreeParams& P, const TreePiece& u, int tile, int lane, int page,
                                               const CUtensorMap* tm, uint32_t dst, uint32_t bar, uint64_t policy) {
    const int n = boxes(P, u, tile);
    if (lane == 0) mbar_arrive_expect_tx(bar, (n << P.box_shift) * D);
    __syncwarp();
    if (lane < n)
      tma_load_4d_hint(dst + (lane << P.box_shift) * D, tm, bar, 0, u.hk,
                       (tile * KT + (lane << P.box_shift)) & ((1 << P.page_shift) - 1), page, policy);
  }
  // The tile's scales, block i's to dst + 4 i; landed() makes the barrier wait
  // for all of them that were copied before.
  __device__ static __forceinline__ void copy_scales(const TreeParams& P, const TreePiece& u, int tile, int lane,
                                                     int page, const float* scales, uint32_t dst) {
    // block i of the tile lies in box i * 16 >> box_shift
    const int key = tile * KT + lane * kScaleBlock;
    const int pg = __shfl_sync(0xffffffffu, page, (lane * kScaleBlock) >> P.box_shift);
    if (lane < BLOCKS) {
      const bool there = pg < P.n_pages;
      const float* src = there ? scales + (((static_cast<int64_t>(pg) * P.Hkv + u.hk) << (P.page_shift - kScaleShift)) +
                                           ((key & ((1 << P.page_shift) - 1)) >> kScaleShift))
                               : scales;
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + lane * 4), "l"(src), "r"(there ? 4 : 0)
                   : "memory");
    }
  }
  __device__ static __forceinline__ void landed(uint32_t bar, int lane) {
    if (lane < BLOCKS) asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
  }
  // place of the 16-byte word c of row r of the tile
  __device__ static __forceinline__ uint32_t word16(int r, int c) {
    return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  }
};

// V for tcgen05: a tile of codes as slabs of 64 columns, KT rows of 64 bytes
// with the 64-byte swizzle (a box each), and rows [r0, r0 + 16) of it at src to a
// tile of f16 at dst (slabs of 64 columns of KT * 128 bytes with the 128-byte
// swizzle), by a warp: 8 rows of 4 words of 16 codes an instruction, which are
// loaded and stored without bank conflicts.  `clean`(row, word): called for each
// word.
template <int D, int KT>
struct VTile8 {
  static constexpr int SLABS = D / 64;
  __device__ static __forceinline__ void issue(const TreeParams& P, const TreePiece& u, int tile, int lane, int page,
                                               const CUtensorMap* tm, uint32_t dst, uint32_t bar, uint64_t policy) {
    const int n = TileLoad8<D, KT>::boxes(P, u, tile);
    if (lane == 0) mbar_arrive_expect_tx(bar, (n << P.box_shift) * D);
    __syncwarp();
    const int j = lane / SLABS, slab = lane % SLABS, pg = __shfl_sync(0xffffffffu, page, j);
    if (j < n)
      tma_load_4d_hint(dst + slab * (KT * 64) + (j << P.box_shift) * 64, tm, bar, slab * 64, u.hk,
                       (tile * KT + (j << P.box_shift)) & ((1 << P.page_shift) - 1), pg, policy);
  }
  template <typename F>
  __device__ static __forceinline__ void to_f16(uint32_t src, uint32_t dst, int r0, int lane, F clean) {
    const int w = lane & 3, row0 = r0 + (lane >> 2);   // and row0 + 8: the same place of the swizzles
    const uint32_t from = src + row0 * 64 + ((w ^ ((row0 >> 1) & 3)) << 4);
    const uint32_t to = dst + row0 * 128, c = ((2 * w) ^ (row0 & 7)) << 4;
    uint4 x[2 * SLABS];
#pragma unroll
    for (int i = 0; i < 2 * SLABS; ++i)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(x[i].x), "=r"(x[i].y), "=r"(x[i].z), "=r"(x[i].w)
                   : "r"(from + (i >> 1) * (KT * 64) + (i & 1) * 512)
                   : "memory");
#pragma unroll
    for (int i = 0; i < 2 * SLABS; ++i) {
      clean(row0 + (i & 1) * 8, x[i]);
      const uint32_t at = to + (i >> 1) * (KT * 128) + (i & 1) * 1024;
      st_shared_v4(at + c, f16x2_of_e4m3x2(x[i].x), f16x2_of_e4m3x2(x[i].x >> 16), f16x2_of_e4m3x2(x[i].y),
                   f16x2_of_e4m3x2(x[i].y >> 16));
      st_shared_v4(at + (c ^ 16), f16x2_of_e4m3x2(x[i].z), f16x2_of_e4m3x2(x[i].z >> 16), f16x2_of_e4m3x2(x[i].w),
                   f16x2_of_e4m3x2(x[i].w >> 16));
    }
  }
};

// What a tile's blocks bring to the softmax: sk, log2 sv, and what the sum of
// the weights takes of P.
__device__ __forceinline__ float4 block_factors(float sk, float sv) {
  const float lv = __log2f(clamp_scale(sv));
  return make_float4(clamp_scale(sk), lv, kPUndo * ex2(-lv), 0.f);
}

// The power of two that brings a row's largest element to [2^13, 2^14), top
// being its bf16 bits without the sign (0: a row of zeros).
__device__ __forceinline__ int row_shift(uint32_t top) {
  return top ? min(13 - (static_cast<int>(top >> 7) - 127), 126) : 0;
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }
// What takes S to a score, a block's scale times a row's factor, kept within the
// normal numbers: a masked -inf stays one (times 0 it would be NaN, and sk is
// 2^-60 where nothing was loaded), a score of 0 stays 0.  NaN stays NaN.
__device__ __forceinline__ float score_factor(float sk, float back) {
  float f;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(f) : "f"(sk * back), "f"(0x1p-126f));
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(f) : "f"(f), "f"(0x1.fffffep127f));
  return f;
}
// A factor kept finite, so that a score of 0 stays 0 (NaN stays NaN).
__device__ __forceinline__ float finite(float x) { return x > 0x1.fffffep127f ? 0x1.fffffep127f : x; }
// Two bf16 times a factor, as f16.
__device__ __forceinline__ uint32_t f16x2_of_bf16x2(uint32_t x, float mul) {
  return pack_f16(__uint_as_float(x << 16) * mul, __uint_as_float(x & 0xffff0000u) * mul);
}
// Eight bf16 times a factor that brings them below 2^8, as two parts whose sum
// they are: `hi` the nearest e4m3 code, `lo` the rest's nearest e5m2 code.  f16
// has all their bits from 2^-17 on, where e5m2 ends too, and the difference is
// exact in it.  From 2^-6 on, where e4m3 has its 4 bits, so is `lo`.
__device__ __forceinline__ uint32_t e4m3x2_of_f16x2(uint32_t x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t e5m2x2_of_f16x2(uint32_t x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ void split_q(const uint32_t (&w)[4], float mul, uint2& hi, uint2& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = f16x2_of_bf16x2(w[i], mul);
    h[i] = e4m3x2_of_f16x2(x);
    l[i] = e5m2x2_of_f16x2(sub_f16x2(x, f16x2_of_e4m3x2(h[i])));
  }
  hi = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
  lo = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
}

// ---------------------------------------------------------------- NaN of V
// As fix_row of a bf16 cache: keys at or past `origin` are cleaned of NaN (the
// one code that is not finite) in shared memory, and the rows that do see such
// a key get it here.
template <typename T>
static __device__ __noinline__ void fix_row8(const Tree8Params& A, int b, int hk, int origin, const uint32_t* nf,
                                             uint4 s0, uint4 s1, int c0, int n, T* row) {
  const TreeParams& P = A.P;
#pragma unroll 1
  for (int w = 0; w < 8; ++w) {
    const uint4 s = w < 4 ? s0 : s1;
    uint32_t bits = nf[w] & ((w & 3) == 0 ? s.x : (w & 3) == 1 ? s.y : (w & 3) == 2 ? s.z : s.w);
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

// Instruction descriptor of an MMA whose A is the second part (e5m2: format 1) and
// whose B is codes (e4m3: format 0).
__host__ __device__ constexpr uint32_t idesc_e5m2_e4m3(int M, int N) { return idesc_e4m3(M, N) | (1u << 7); }

fm_status launch_tree8_mid(const Tree8Params& A, int d, const CUtensorMap& tk, const CUtensorMap& tv, int grid,
                           cudaStream_t s);        // up to 128 rows
fm_status launch_tree8_wide(const Tree8Params& A, const CUtensorMap& tk, const CUtensorMap& tv, int grid,
                            cudaStream_t s);       // d = 128
fm_status launch_tree8_narrow(const Tree8Params& A, int d, int rows, const CUtensorMap& tk, const CUtensorMap& tv,
                              int grid, cudaStream_t s);
// Joins the parts that the first kernel left (fm_tree.cu); rows: of its units.
fm_status launch_tree_join(const TreeParams& P, int d, int rows, int grid, cudaStream_t s);

}  // namespace fm
