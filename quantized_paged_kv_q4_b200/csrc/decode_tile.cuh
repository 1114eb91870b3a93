// One 16-token tile of split-KV decode: the format traits of a (key, value) pair and the tile's
// arithmetic, which the single-sequence and the ragged-batch decode share.
#pragma once

#include "common.cuh"

namespace kvattn {

constexpr int kTileBlocks = kBlocks;  // 32-channel blocks of a row

// The regions of a K and a V page of a format pair.  Every region (codes, fifth bits, scales,
// minima) is ordered by 16-token tile first, so tiles [g0, g1) of a page are one contiguous range
// of each region: (offset of the region, bytes per tile).
template <int KF, int VF>
struct TileFormat {
  static constexpr bool kK5 = KF == kKeyQ51 || KF == kKeyQ50;  // 5-bit key codes
  static constexpr bool kKMin = KF == kKeyQ51;                 // keys with a zero point
  static constexpr bool kVMin = VF == kValQ41;                 // values with a zero point
  static constexpr int kKBytes =
      KF == kKeyQ4 ? kK4PageBytes : KF == kKeyQ51 ? kK5PageBytes : KF == kKeyQ50 ? kK50PageBytes : kKPageBytes;
  static constexpr int kKScaleOff = KF == kKeyQ4 ? kK4ScaleOffset : kK5 ? kK5ScaleOffset : kKScaleOffset;
  static constexpr int kVBytes = VF == kValQ8 ? kV8PageBytes : VF == kValQ41 ? kV41PageBytes : kV4PageBytes;
  static constexpr int kVScaleOff = VF == kValQ8 ? kV8ScaleOffset : kV4ScaleOffset;
  static constexpr int kKRegions = KF == kKeyQ51 ? 4 : KF == kKeyQ50 ? 3 : 2;
  static constexpr int kVRegions = VF == kValQ41 ? 3 : 2;
  __host__ __device__ static constexpr int k_reg_off(int r) {
    return r == 0 ? 0 : r == 1 ? (kK5 ? kK5HighOffset : kKScaleOff) : r == 2 ? kK5ScaleOffset : kK5MinOffset;
  }
  __host__ __device__ static constexpr int k_reg_tile(int r) {
    return r == 0 ? (KF == kKeyQ8 ? 4096 : 2048) : r == 1 && kK5 ? 512 : 256;
  }
  __host__ __device__ static constexpr int v_reg_off(int r) { return r == 0 ? 0 : r == 1 ? kVScaleOff : kV41MinOffset; }
  __host__ __device__ static constexpr int v_reg_tile(int r) { return r == 0 ? (VF == kValQ8 ? 4096 : 2048) : 256; }
  static_assert(8 * (k_reg_tile(0) + k_reg_tile(1) + (kKRegions > 2 ? k_reg_tile(2) : 0) +
                     (kKRegions > 3 ? k_reg_tile(3) : 0)) == kKBytes, "K regions");
  static_assert(8 * (v_reg_tile(0) + v_reg_tile(1) + (kVRegions > 2 ? v_reg_tile(2) : 0)) == kVBytes, "V regions");
  static_assert(k_reg_off(1) == 8 * k_reg_tile(0) && (kKRegions < 3 || k_reg_off(2) == k_reg_off(1) + 8 * k_reg_tile(1)) &&
                (kKRegions < 4 || k_reg_off(3) == k_reg_off(2) + 8 * k_reg_tile(2)), "K region offsets");
  static_assert(v_reg_off(1) == 8 * v_reg_tile(0) && (kVRegions < 3 || v_reg_off(2) == v_reg_off(1) + 8 * v_reg_tile(1)),
                "V region offsets");
};

constexpr uint32_t kHalf2Magic = 0x64006400u;  // f16 1024.0 in both halves
constexpr uint32_t kByte64x4 = 0x64646464u;    // high byte of f16 1024.0, for byte permutes
constexpr uint32_t kHalf2_1032 = 0x64086408u;  // 1024 + 8
constexpr uint32_t kHalf2_1040 = 0x64106410u;  // 1024 + 16
constexpr uint32_t kHalf2_1152 = 0x64806480u;  // 1024 + 128
constexpr uint32_t kHalf2_1_16 = 0x2C002C00u;  // 1/16
constexpr uint32_t kHalf2_m72 = 0xD480D480u;   // -(64 + 8)
constexpr uint32_t kHalf2_m64 = 0xD400D400u;   // -64
constexpr uint32_t kHalf2_m80 = 0xD500D500u;   // -(64 + 16)
constexpr uint32_t kHalf2_Sign = 0x80008000u;

// B operand (probabilities times a per-token fp16 factor f) as an unevaluated f16 sum hi + lo:
// hi = f16(ph * f); ph * f - hi is an 11 x 11-bit product without its first 11 bits, and lo adds
// pl * f with one rounding.  hi + lo equals (ph + pl) * f to about 2^-22 relative, and to 2^-24 (f16's
// smallest step, once for the remainder and once for lo) where that is more.
__device__ __forceinline__ void split_scaled(uint32_t ph, uint32_t pl, uint32_t f, uint32_t& hi, uint32_t& lo) {
  hi = hmul2(ph, f);
  lo = hfma2(pl, f, hfma2(ph, f, hi ^ kHalf2_Sign));
}

// fp32 pair -> f16 hi part (round to nearest) and f16 lo part (the rounded remainder).
__device__ __forceinline__ void split_pair(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  hi = pack_half2(x0, x1);
  lo = pack_half2(x0 - half_lo(hi), x1 - half_hi(hi));
}

// acc += A B, B in two f16 parts.  SUM: into sums of its own first, added in fp32: the MMA cuts what does not fit
// 24 bits of its sum, always towards zero, which a long stretch of tiles lets grow (about 2^-24 of the sum a step).
template <bool SUM>
__device__ __forceinline__ void mma_parts(float (&acc)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t bh0, uint32_t bh1, uint32_t bl0, uint32_t bl1) {
  if constexpr (SUM) {
    float x[4];
    mma_f16_z(x, a0, a1, a2, a3, bl0, bl1);
    mma_f16(x, a0, a1, a2, a3, bh0, bh1);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] += x[e];
  } else {
    mma_f16(acc, a0, a1, a2, a3, bh0, bh1);
    mma_f16(acc, a0, a1, a2, a3, bl0, bl1);
  }
}

__device__ __forceinline__ void sts_pair(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

__device__ __forceinline__ uint2 lds_pair(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

// Where the parts of a page sit in a shared-memory copy: a whole page (tile G of it is read) ...
template <int KF, int VF>
struct PageLayout {
  using F = TileFormat<KF, VF>;
  static constexpr int kKScale = F::kKScaleOff, kKHigh = kK5HighOffset, kKMinimum = kK5MinOffset;
  static constexpr int kVScale = F::kVScaleOff, kVMinimum = kV41MinOffset;
};

// ... or one tile by itself (G = 0), its part of every region packed: the wide ones first (K codes,
// fifth bits, V codes; multiples of 512 bytes), then the 256-byte ones (scales, minima).  Offsets of
// the V parts are from the V codes, as in a page.
template <int KF, int VF>
struct SingleTileLayout {
  using F = TileFormat<KF, VF>;
  static constexpr int kKCodes = F::k_reg_tile(0), kHigh = F::kK5 ? F::k_reg_tile(1) : 0, kVCodes = F::v_reg_tile(0);
  static constexpr int kKHigh = kKCodes, kV = kKCodes + kHigh;  // from the tile's start
  static constexpr int kSmall = kV + kVCodes, kNarrow = 2 + F::kKMin + F::kVMin;
  static constexpr int kKScale = kSmall, kKMinimum = kSmall + 512;
  static constexpr int kVScale = kSmall + 256 - kV, kVMinimum = kSmall + 512 - kV;
  static_assert(!(F::kKMin && F::kVMin), "one minimum: the third 256 bytes");
  static constexpr int kBytes = kSmall + 256 * kNarrow;
};

// S = K Q^T of one tile of 16 tokens and NR n-tiles of 8 query rows (one warp; g = lane / 4, t = lane %
// 4): sacc[n][e] is token g + 8 (e / 2), row 2t + e % 2 of n-tile n.
//   QP             f16 parts of the query: 2 keeps about 22 bits of it, 1 rounds once
//   qfrag(n, b, f) fills f[k-step] with the B fragments of n-tile n, block b (hi0, hi1, lo0, lo1)
//   qsums(n)       zero-point keys: the query's block sums as a B fragment (hi, lo); with QSUM > 0 divided by
//                  2^QSUM, and lo times 2^11
// The tile is tile G of the copy at kb, arranged as L.
template <typename L, int KF, int VF, int QP, int QSUM, int NR, typename QFrag, typename QSums>
__device__ __forceinline__ void tile_scores(uint32_t kb, int G, int g, int t, QFrag qfrag, QSums qsums,
                                            float (&sacc)[NR][4]) {
  using F = TileFormat<KF, VF>;
  // ---------------- S = K Q^T over the 256 channels ----------------
  // Key codes enter the MMA exactly (integers in f16).  Each 32-channel block is
  // accumulated on its own (two k-steps, each with the query's parts) and then
  // scaled by the block's fp32 scale into S; with a zero point, two more MMAs add the
  // block minima times the query block sums.
#pragma unroll
  for (int n = 0; n < NR; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) sacc[n][e] = 0.f;
  // key scales of rows g (H=0) and g+8 (H=1) for the 8 blocks, fp32; zero-point keys:
  // the minima of blocks 2t, 2t + 1 of the same rows (the A fragment of the MMA that
  // adds the minimum terms)
  float dkf[2][kTileBlocks];
  uint32_t mka[2] = {0u, 0u};
#pragma unroll
  for (int H = 0; H < 2; ++H) {
    const uint32_t sa = kb + L::kKScale + (((G * 8 + g) * 2 + H) * 8) * 2;
    uint32_t w[4];
    const uint4 v = lds128(sa);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    if constexpr (F::kKMin) mka[H] = lds32(sa + (L::kKMinimum - L::kKScale) + 4 * t);
#pragma unroll
    for (int e = 0; e < kTileBlocks / 2; ++e) {
      dkf[H][2 * e] = half_lo(w[e]);
      dkf[H][2 * e + 1] = half_hi(w[e]);
    }
  }
  // one block: an MMA per k-step and query part into xb, then S += d * xb
  auto block_qk = [&](int bl, const uint32_t (&A)[2][4]) {
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      float xb[4];
      uint4 f[2];
      qfrag(n, bl, f);
      mma_f16_z(xb, A[0][0], A[0][1], A[0][2], A[0][3], f[0].x, f[0].y);
      if constexpr (QP == 2) mma_f16(xb, A[0][0], A[0][1], A[0][2], A[0][3], f[0].z, f[0].w);
      mma_f16(xb, A[1][0], A[1][1], A[1][2], A[1][3], f[1].x, f[1].y);
      if constexpr (QP == 2) mma_f16(xb, A[1][0], A[1][1], A[1][2], A[1][3], f[1].z, f[1].w);
#pragma unroll
      for (int e = 0; e < 4; ++e) sacc[n][e] = fmaf(dkf[e >> 1][bl], xb[e], sacc[n][e]);
    }
  };
  if constexpr (KF == kKeyQ8) {
#pragma unroll
    for (int P = 0; P < kTileBlocks / 2; ++P) {
      const uint4 ka = lds128(kb + ((((G * 4 + P) * 2 + 0) * 8 + g) * 4 + t) * 16);
      const uint4 kc = lds128(kb + ((((G * 4 + P) * 2 + 1) * 8 + g) * 4 + t) * 16);
      // code bytes are offset-binary (q + 128)
      const uint32_t wg[4] = {ka.x, ka.y, ka.z, ka.w};
      const uint32_t w8[4] = {kc.x, kc.y, kc.z, kc.w};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t A[2][4];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          // exact code -> f16: 1024 + (q + 128) - 1152
          A[ks][0] = hsub2(prmt(wg[2 * e + ks], kByte64x4, 0x4140u), kHalf2_1152);
          A[ks][2] = hsub2(prmt(wg[2 * e + ks], kByte64x4, 0x4342u), kHalf2_1152);
          A[ks][1] = hsub2(prmt(w8[2 * e + ks], kByte64x4, 0x4140u), kHalf2_1152);
          A[ks][3] = hsub2(prmt(w8[2 * e + ks], kByte64x4, 0x4342u), kHalf2_1152);
        }
        block_qk(2 * P + e, A);
      }
    }
  } else {
    // 4- and 5-bit keys: one 32-bit word per (token, block) and lane holds channels 8t + i,
    // channel i at bit 4 * (i / 2) + 16 * (i % 2); a shift by 8 * ks and two masks give
    // the f16 pairs (4ks, 4ks + 1) and (4ks + 2, 4ks + 3) of k-step ks (1024 + q and
    // 1024 + 16q).  5-bit keys: the fifth bits of the lane's four blocks of one token
    // sit in one word, channel (c, i) at bit 16(i%2) + 4c + i/2, and are shifted to bit 4
    // or bit 8 of each half.  The code (minus 8 for Q4_0, 16 for Q5_0) is exact in f16.
#pragma unroll
    for (int Q = 0; Q < 2; ++Q) {
      const int row0 = (((G * 2 + Q) * 2 + 0) * 8 + g) * 4 + t;
      const int row1 = (((G * 2 + Q) * 2 + 1) * 8 + g) * 4 + t;
      const uint4 ka = lds128(kb + row0 * 16);
      const uint4 kc = lds128(kb + row1 * 16);
      const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w};
      const uint32_t wc[4] = {kc.x, kc.y, kc.z, kc.w};
      uint32_t xa5 = 0, xc5 = 0;
      if constexpr (F::kK5) {
        xa5 = lds32(kb + L::kKHigh + row0 * 4);
        xc5 = lds32(kb + L::kKHigh + row1 * 4);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t A[2][4];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          const uint32_t xa = wa[c] >> (8 * ks), xc = wc[c] >> (8 * ks);
          if constexpr (KF == kKeyQ4) {
            A[ks][0] = hsub2(and_or(xa, 0x000F000Fu, kHalf2Magic), kHalf2_1032);
            A[ks][2] = hfma2(and_or(xa, 0x00F000F0u, kHalf2Magic), kHalf2_1_16, kHalf2_m72);
            A[ks][1] = hsub2(and_or(xc, 0x000F000Fu, kHalf2Magic), kHalf2_1032);
            A[ks][3] = hfma2(and_or(xc, 0x00F000F0u, kHalf2Magic), kHalf2_1_16, kHalf2_m72);
          } else {
            const int slo = 4 - (4 * c + 2 * ks), shi = 7 - (4 * c + 2 * ks);
            const uint32_t ha_lo = slo >= 0 ? xa5 << slo : xa5 >> -slo;
            const uint32_t ha_hi = shi >= 0 ? xa5 << shi : xa5 >> -shi;
            const uint32_t hc_lo = slo >= 0 ? xc5 << slo : xc5 >> -slo;
            const uint32_t hc_hi = shi >= 0 ? xc5 << shi : xc5 >> -shi;
            constexpr uint32_t kSubLo = KF == kKeyQ50 ? kHalf2_1040 : kHalf2Magic;
            constexpr uint32_t kAddHi = KF == kKeyQ50 ? kHalf2_m80 : kHalf2_m64;
            A[ks][0] = hsub2(or_and(and_or(xa, 0x000F000Fu, kHalf2Magic), ha_lo, 0x00100010u), kSubLo);
            A[ks][2] = hfma2(or_and(and_or(xa, 0x00F000F0u, kHalf2Magic), ha_hi, 0x01000100u), kHalf2_1_16,
                             kAddHi);
            A[ks][1] = hsub2(or_and(and_or(xc, 0x000F000Fu, kHalf2Magic), hc_lo, 0x00100010u), kSubLo);
            A[ks][3] = hfma2(or_and(and_or(xc, 0x00F000F0u, kHalf2Magic), hc_hi, 0x01000100u), kHalf2_1_16,
                             kAddHi);
          }
        }
        block_qk(4 * Q + c, A);
      }
    }
  }
  if constexpr (F::kKMin) {
    // S += sum_b m[token][b] qsum[b][row] as one MMA per part of the block sums: A =
    // the minima (tokens g, g + 8 x blocks 2t, 2t + 1; k = 8..15 is zero, exact in f16),
    // B = the block sums of the query rows; the products accumulate in fp32
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const uint2 qs = qsums(n);
      if constexpr (QSUM == 0) {
        mma_f16(sacc[n], mka[0], mka[1], 0u, 0u, qs.x, 0u);
        mma_f16(sacc[n], mka[0], mka[1], 0u, 0u, qs.y, 0u);
      } else {
        float xh[4], xl[4];
        mma_f16_z(xh, mka[0], mka[1], 0u, 0u, qs.x, 0u);
        mma_f16_z(xl, mka[0], mka[1], 0u, 0u, qs.y, 0u);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sacc[n][e] = fmaf(static_cast<float>(1 << QSUM), fmaf(0x1p-11f, xl[e], xh[e]), sacc[n][e]);
      }
    }
  }
}

// The codes of value blocks 2C and 2C + 1 of one tile as A fragments (16 dims x 16 tokens, exact in f16):
// f(block, dims 0-15, dims 16-31, scales of tokens 2t, 2t + 1 and of 2t + 8, 2t + 9).  The scales are those at
// `scales`, the tile's own or its lifted copy.
template <typename L, int KF, int VF, typename Use>
__device__ __forceinline__ void tile_value_pair(uint32_t vb, uint32_t scales, int G, int C, int g, int t, Use f) {
  using F = TileFormat<KF, VF>;
  if constexpr (VF != kValQ8) {
    const uint4 vw = lds128(vb + ((((G * 4 + C) * 8 + g) * 4 + t) * 16));
    const uint4 dv = lds128(scales + (t * 8 + 2 * C) * 8);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t W0 = e ? vw.z : vw.x, W1 = e ? vw.w : vw.y;
      const uint32_t W0s = W0 >> 8, W1s = W1 >> 8;
      // Q4_0: q - 8 (1024 + q - 1032, or (1024 + 16q) / 16 - 72); Q4_1: q
      constexpr uint32_t kSubLo = F::kVMin ? kHalf2Magic : kHalf2_1032;
      constexpr uint32_t kAddHi = F::kVMin ? kHalf2_m64 : kHalf2_m72;
      const uint32_t a0[4] = {hsub2(and_or(W0, 0x000F000Fu, kHalf2Magic), kSubLo),
                              hfma2(and_or(W0, 0x00F000F0u, kHalf2Magic), kHalf2_1_16, kAddHi),
                              hsub2(and_or(W1, 0x000F000Fu, kHalf2Magic), kSubLo),
                              hfma2(and_or(W1, 0x00F000F0u, kHalf2Magic), kHalf2_1_16, kAddHi)};
      const uint32_t a1[4] = {hsub2(and_or(W0s, 0x000F000Fu, kHalf2Magic), kSubLo),
                              hfma2(and_or(W0s, 0x00F000F0u, kHalf2Magic), kHalf2_1_16, kAddHi),
                              hsub2(and_or(W1s, 0x000F000Fu, kHalf2Magic), kSubLo),
                              hfma2(and_or(W1s, 0x00F000F0u, kHalf2Magic), kHalf2_1_16, kAddHi)};
      f(2 * C + e, a0, a1, e ? dv.z : dv.x, e ? dv.w : dv.y);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int b = 2 * C + e;
      const uint4 vw = lds128(vb + ((((G * 8 + b) * 8 + g) * 4 + t) * 16));
      const uint2 dv = lds_pair(scales + (t * 8 + b) * 8);
      const uint32_t w[4] = {vw.x, vw.y, vw.z, vw.w};  // offset-binary code bytes (q + 128)
      uint32_t a[2][4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        a[q >> 1][2 * (q & 1)] = hsub2(prmt(w[q], kByte64x4, 0x4140u), kHalf2_1152);
        a[q >> 1][2 * (q & 1) + 1] = hsub2(prmt(w[q], kByte64x4, 0x4342u), kHalf2_1152);
      }
      f(b, a[0], a[1], dv.x, dv.y);
    }
  }
}

// ---- the powers of two of P x scale.  The second MMA takes P times a value's scale as f16 parts, and f16
// ends at 2^-24: both factors are put as high in it as they fit, by powers of two that the sums carry.
//   P       is relative to a reference of the row, kPTop - k below the row's running maximum (which may
//           lag 2^kGrow behind): the largest P is 2^kPTop to 2^(kPTop + kGrow) = 2^15 for k = 0
//   scales  are multiplied by `mul`, so that the largest so far comes to (1/2, 1]; where it is above 1
//           they stay as they are, and k is its exponent instead (a small scale then keeps its bits)
// The products' two parts so end about 2^37 below the row's largest P times the largest scale.
// (Both are one state of all rows and channels that a warp, or a group of warps, adds up.  It moves when a
// larger scale comes along: seldom after the first tiles.  Single-sequence decode of 131,072 tokens: 47.7 us
// a layer without all this, 48.6 with it.)
constexpr float kPTop = 13.f, kGrow = 2.f;

struct ValueScale {
  uint32_t bound = 0u;          // in both halves, the f16 power of two that no scale so far exceeds (0: none seen)
  float top = kPTop + kGrow;    // how far a score may pass its row's reference: kPTop + kGrow - k
  __device__ __forceinline__ uint32_t mul() const { return 0x78007800u - min(bound, 0x3C003C00u); }
  // the exponent of the bound, + 15 (2^16 is kept as the largest f16 instead, so that infinities exceed it)
  __device__ __forceinline__ int exponent() const { return static_cast<int>((bound & 0xFFFFu) + 0x3FFu) >> 10; }
  // what undoes mul() in a sum
  __device__ __forceinline__ float unit() const { return exp2_int(min(exponent(), 15) - 15); }
  __device__ __forceinline__ static float exp2_int(int e) {
    return __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
  }
  // Takes in scales up to `most` (f16 bits): what the rows' references rise by goes to *dk, the factor of the
  // sums of P x scale beside that to *ratio.
  __device__ __forceinline__ void raise(uint32_t most, int* dk, float* ratio) {
    const int was = exponent();
    int now = was;
    if (most > (bound & 0xFFFFu)) now = most < 0x400u ? 1 : static_cast<int>(most + 0x3FFu) >> 10;
    *dk = max(now - 15, 0) - max(was - 15, 0);
    *ratio = exp2_int(min(was, 15) - min(now, 15));
    bound = min(static_cast<uint32_t>(now) << 10, 0x7BFFu) * 0x00010001u;
    top -= static_cast<float>(*dk);
  }
};

// Whether one of the two f16 pairs has an element whose magnitude exceeds bound's (NaN exceeds all).
__device__ __forceinline__ bool exceeds(uint32_t a, uint32_t b, uint32_t bound) {
  uint32_t over;
  asm("{\n\t.reg .b32 x, y;\n\t.reg .pred p, q;\n\t"
      "abs.f16x2 x, %1;\n\t"
      "abs.f16x2 y, %2;\n\t"
      "max.NaN.f16x2 x, x, y;\n\t"
      "setp.gtu.f16x2 p|q, x, %3;\n\t"
      "or.pred p, p, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(over)
      : "r"(a), "r"(b), "r"(bound));
  return over != 0;
}

// The scales (and minima) of one tile's values as lane (g, t) holds them: block g, tokens 2t, 2t + 1 in the first
// word, 2t + 8, 2t + 9 in the second.
struct TileScales {
  uint2 d, m = {0u, 0u};
  template <typename L, bool VMIN>
  __device__ __forceinline__ void load(uint32_t vb, int G, int g, int t) {
    const uint32_t at = vb + L::kVScale + ((G * 4 + t) * 8 + g) * 8;
    d = lds_pair(at);
    if constexpr (VMIN) m = lds_pair(at + (L::kVMinimum - L::kVScale));
  }
  template <typename L, bool VMIN>
  __device__ __forceinline__ void store(uint32_t vb, int G, int g, int t) const {
    const uint32_t at = vb + L::kVScale + ((G * 4 + t) * 8 + g) * 8;
    sts_pair(at, d.x, d.y);
    if constexpr (VMIN) sts_pair(at + (L::kVMinimum - L::kVScale), m.x, m.y);
  }
  // whether the powers of two have to move, or something here is not finite
  template <bool VMIN>
  __device__ __forceinline__ bool unusual(const ValueScale& vs) const {
    bool x = exceeds(d.x, d.y, vs.bound);
    if constexpr (VMIN) x |= exceeds(m.x, m.y, 0x7BFF7BFFu);
    return x;
  }
  // Zeroes what no row sees (whatever it is) and what is not finite.  lo and hi: whether a row of the lane's sees
  // token g, g + 8 (mma.sync's accumulator layout).  *most: the largest scale left in the tile, as f16 bits.
  // Returns the lane's tokens that some row sees and that are not finite: bit 2H + i for token 2t + i + 8H.
  __device__ __forceinline__ uint32_t clean(bool lo, bool hi, int t, uint32_t* most) {
    const uint32_t vis[2] = {__ballot_sync(0xffffffffu, lo), __ballot_sync(0xffffffffu, hi)};
    uint32_t w[2] = {d.x, d.y}, n[2] = {m.x, m.y}, bad = 0, top = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int H = j >> 1, i = j & 1;
      const uint32_t half = 0xFFFFu << (16 * i), inf = 0x7C00u << (16 * i);
      const bool seen = (vis[H] >> (8 * t + 4 * i)) & 15u, finite = (w[H] & inf) != inf && (n[H] & inf) != inf;
      if (seen && !finite) bad |= 1u << j;
      if (!seen || !finite) w[H] &= ~half, n[H] &= ~half;
      top = max(top, (w[H] >> (16 * i)) & 0x7FFFu);
    }
    d = make_uint2(w[0], w[1]);
    m = make_uint2(n[0], n[1]);
    *most = __reduce_max_sync(0xffffffffu, top);
    return bad;
  }
  // The largest finite scale of the tile, whoever sees it.
  __device__ __forceinline__ uint32_t largest() const {
    const uint32_t w[2] = {d.x, d.y};
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t x = (w[j >> 1] >> (16 * (j & 1))) & 0x7FFFu;
      if (x < 0x7C00u) top = max(top, x);
    }
    return __reduce_max_sync(0xffffffffu, top);
  }
  // The lifted scales, into the tile's copy.
  __device__ __forceinline__ void lift(const ValueScale& vs, uint32_t scales, int g, int t) const {
    const uint32_t mul = vs.mul();
    sts_pair(scales + (t * 8 + g) * 8, hmul2(d.x, mul), hmul2(d.y, mul));
  }
};

// Bit 4b of rows[c]: row 2t + c sees a key whose block b is not finite.  bad: TileScales::clean of every lane; sv:
// the rows' scores, -inf where a key is unseen.
__device__ __forceinline__ void blind_blocks(uint32_t bad, const float (&sv)[4], int t, uint32_t (&rows)[2]) {
  const uint32_t b0 = __ballot_sync(0xffffffffu, bad & 1u), b1 = __ballot_sync(0xffffffffu, bad & 2u);
  const uint32_t b2 = __ballot_sync(0xffffffffu, bad & 4u), b3 = __ballot_sync(0xffffffffu, bad & 8u);
#pragma unroll 1
  for (int tok = 0; tok < 16; ++tok) {
    const uint32_t of = tok < 8 ? (tok & 1 ? b1 : b0) : (tok & 1 ? b3 : b2);
    const uint32_t blocks = (of >> ((tok & 7) >> 1)) & 0x11111111u;
    const int from = (tok & 7) * 4 + t;
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (__shfl_sync(0xffffffffu, tok < 8 ? sv[c] : sv[2 + c], from) != -INFINITY) rows[c] |= blocks;
  }
}

// Adds one tile of 16 tokens to the online softmax of 8 query rows (one warp; g = lane / 4, t =
// lane % 4; the thread's rows are 2t, 2t + 1).
//   QP           f16 parts of the query: 2 keeps about 22 bits of it, 1 rounds once
//   SUM          whether every tile's sums are added by themselves (mma_parts)
//   COPY         the tile's scales are lifted once, into 256 bytes of the warp's own at `copy`, where scales that no
//                row sees are left out and values that are not finite stay with the rows that see them.  Without
//                it they are lifted where they are used (which measured faster in the single-sequence kernel: a
//                131,072-token layer 49.2 us against 50.3) and every finite scale of a tile counts.
//   qfrag(b, f)  fills f[k-step] with the query's B fragments of block b (hi0, hi1, lo0, lo1)
//   qsb_hi, lo   zero-point keys: the query's block sums as a B fragment (tile_scores)
//   crow         turns a dot product with the normalised row into a base-2 softmax score
//   mask(e, x)   x, or -inf where the key is unseen: token g + 8 (e / 2), row 2t + e % 2
//   m_run        the rows' references (above), vs the scales' state; l_run, oacc and racc are sums relative to
//                them: of P, of P x scale x code (x vs.mul()) and of P x minimum
// The tile is tile G of the copy at kb (K) and vb (V), arranged as L.
template <typename L, int KF, int VF, int QP, int QSUM, bool SUM, bool COPY, typename QFrag, typename Mask>
__device__ __forceinline__ void attend_tile(uint32_t kb, uint32_t vb, uint32_t copy, int G, int g, int t, QFrag qfrag,
                                            uint32_t qsb_hi, uint32_t qsb_lo, const float (&crow)[2], Mask mask,
                                            ValueScale& vs, float (&m_run)[2], float (&l_run)[2],
                                            float (&oacc)[2 * kTileBlocks][4], float (&racc)[4]) {
  using F = TileFormat<KF, VF>;
  float sacc[1][4];
  tile_scores<L, KF, VF, QP, QSUM, 1>(
      kb, G, g, t, [&](int, int bl, uint4 (&f)[2]) { qfrag(bl, f); }, [&](int) { return make_uint2(qsb_hi, qsb_lo); },
      sacc);
  // ---------------- online softmax (base 2) ----------------
  // The reference m_run of a row is shared by the 8 lanes that hold the row.  It only has to be
  // within 2^kGrow of what the running maximum asks for, so the exact cross-lane maximum is computed
  // only when some lane sees a score above it: one warp vote per tile (which the scales of the
  // tile's values share) instead of three shuffles per row.
  TileScales ts;
  ts.load<L, F::kVMin>(vb, G, g, t);
  float sv[4], lm[2];
  bool need = ts.unusual<F::kVMin && COPY>(vs);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    sv[e] = mask(e, sacc[0][e] * crow[e & 1]);
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    lm[c] = fmaxf(sv[c], sv[c + 2]);
    need |= lm[c] > m_run[c] + vs.top;
  }
  if (__any_sync(0xffffffffu, need)) {
    uint32_t most;
    if constexpr (COPY) {
      const uint32_t bad = ts.clean(sv[0] != -INFINITY || sv[1] != -INFINITY, sv[2] != -INFINITY || sv[3] != -INFINITY,
                                    t, &most);
      if (__any_sync(0xffffffffu, bad != 0)) {
        uint32_t blind[2] = {0u, 0u};
        blind_blocks(bad, sv, t, blind);
#pragma unroll
        for (int mt = 0; mt < 2 * kTileBlocks; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (blind[e & 1] >> (4 * (mt >> 1)) & 1u) oacc[mt][e] = NAN;
      }
    } else {
      most = ts.largest();
    }
    const float top = vs.top;
    int dk;
    float ratio;
    vs.raise(most, &dk, &ratio);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float mx = lm[c];
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      const float m = mx > m_run[c] + top ? mx + (kGrow - vs.top) : m_run[c] + static_cast<float>(dk);
      const float alpha = m == m_run[c] ? 1.f : fast_exp2(m_run[c] - m);  // 0 when m_run = -inf
      l_run[c] *= alpha;
#pragma unroll
      for (int mt = 0; mt < 2 * kTileBlocks; ++mt) {
        oacc[mt][c] *= alpha * ratio;
        oacc[mt][c + 2] *= alpha * ratio;
      }
      if constexpr (F::kVMin) racc[c] *= alpha;
      m_run[c] = m;
    }
  }
  const uint32_t mul = vs.mul(), scales = COPY ? copy : vb + L::kVScale + G * 256;
  if constexpr (COPY) {
    ts.lift(vs, copy, g, t);
    __syncwarp();
  }
  // P as f16 parts, transposed in registers into B fragments
  uint32_t pbh[2], pbl[2];
  float pr[4];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const float mu = m_run[c] == -INFINITY ? 0.f : m_run[c];
    pr[c] = fast_exp2(sv[c] - mu);
    pr[c + 2] = fast_exp2(sv[c + 2] - mu);
    l_run[c] += pr[c] + pr[c + 2];
  }
  {
    uint32_t h01, l01, h23, l23;
    split_pair(pr[0], pr[1], h01, l01);
    split_pair(pr[2], pr[3], h23, l23);
    pbh[0] = movmatrix_t(h01);
    pbh[1] = movmatrix_t(h23);
    pbl[0] = movmatrix_t(l01);
    pbl[1] = movmatrix_t(l23);
  }
  // ---------------- O^T += V^T P^T ----------------
  // V codes enter the MMA exactly; the per-token block scale multiplies P (in two f16 parts),
  // two MMAs per 16-dimension half.
#pragma unroll
  for (int C = 0; C < kTileBlocks / 2; ++C)
    tile_value_pair<L, KF, VF>(vb, scales, G, C, g, t,
                               [&](int bl, const uint32_t (&a0)[4], const uint32_t (&a1)[4], uint32_t d0, uint32_t d1) {
      uint32_t bh0, bl0, bh1, bl1;
      split_scaled(pbh[0], pbl[0], COPY ? d0 : hmul2(d0, mul), bh0, bl0);
      split_scaled(pbh[1], pbl[1], COPY ? d1 : hmul2(d1, mul), bh1, bl1);
      mma_parts<SUM>(oacc[2 * bl], a0[0], a0[1], a0[2], a0[3], bh0, bh1, bl0, bl1);
      mma_parts<SUM>(oacc[2 * bl + 1], a1[0], a1[1], a1[2], a1[3], bh0, bh1, bl0, bl1);
    });
  if constexpr (F::kVMin) {
    // sum over the tile's tokens of p * m for all 8 blocks at once: A = the minima
    // (block g x tokens 2t, 2t + 1 | 2t + 8, 2t + 9, exact in f16; blocks 8..15 zero),
    // B = P^T as its high and low parts
    mma_parts<SUM>(racc, ts.m.x, 0u, ts.m.y, 0u, pbh[0], pbh[1], pbl[0], pbl[1]);
  }
}

}  // namespace kvattn
