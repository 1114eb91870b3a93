// Ragged batches of sequences over one cache: the parameters that the append, read and decode
// kernels share, and the device helpers that load, store and locate their rows.
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "common.cuh"

namespace kvattn {

// A token array [n_rows][heads][256], strides in elements.
struct RowsView {
  void* data;
  long long row_stride, head_stride;
};

struct BatchParams {
  uint8_t* k_pool;
  uint8_t* v_pool;
  int64_t k_stride, v_stride, n_pages;
  const int32_t* row_start;
  const int32_t* pos_start;
  const int32_t* page_table;  // [n_seqs][n_kv][max_blocks]
  long long n_rows;
  int n_seqs, max_rows, max_blocks, n_kv;
};

// Eight consecutive elements of a row, as they are loaded ...
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Raw8<T> load_raw8(const void* data, long long at) {
  const uint4* s = reinterpret_cast<const uint4*>(static_cast<const T*>(data) + at);
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) r.v[i] = s[i];
  return r;
}

// ... and as fp32 (exact).
template <typename T>
__device__ __forceinline__ void widen8(const Raw8<T>& r, float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[4 * i] = __uint_as_float(r.v[i].x);
      x[4 * i + 1] = __uint_as_float(r.v[i].y);
      x[4 * i + 2] = __uint_as_float(r.v[i].z);
      x[4 * i + 3] = __uint_as_float(r.v[i].w);
    }
  } else {
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same_v<T, __half>) {
        x[2 * i] = half_lo(w[i]);
        x[2 * i + 1] = half_hi(w[i]);
      } else {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ void load8(const void* data, long long at, float (&x)[8]) {
  widen8<T>(load_raw8<T>(data, at), x);
}

// Two fp32 -> two 16-bit elements in one word (lo in the low half), round to nearest.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (std::is_same_v<T, __half>) {
    return pack_half2(lo, hi);
  } else {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
}

template <typename T>
__device__ __forceinline__ void store8(void* data, long long at, const float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(data) + at);
    d[0] = make_float4(x[0], x[1], x[2], x[3]);
    d[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<T*>(data) + at) =
        make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
  }
}

// One sequence of the batch, read and checked (kvattn_batch): rows [r0, r0 + rows) at
// positions pos0 ...  A sequence that breaks a check has rows = 0 and is recorded.
struct BatchSeq {
  int r0, rows, pos0;
};

__device__ __forceinline__ BatchSeq check_seq(const BatchParams& p, int r0, int r1, int pos0, bool check_blocks) {
  BatchSeq q;
  const long long end = static_cast<long long>(pos0) + (static_cast<long long>(r1) - r0);
  const bool ok = r0 >= 0 && r1 >= r0 && r1 <= p.n_rows && static_cast<long long>(r1) - r0 <= p.max_rows && pos0 >= 0 &&
                  end <= INT32_MAX - kPageTokens &&  // positions of a whole page never overflow
                  (!check_blocks || r1 == r0 || end <= static_cast<long long>(p.max_blocks) * kPageTokens);
  q.r0 = r0;
  q.rows = ok ? r1 - r0 : 0;
  q.pos0 = pos0;
  if (!ok) record_error(KVATTN_ERR_INVALID_ARG);
  return q;
}

// Read through L2: the decode's merge grid reads the arrays while the split grid before it still
// runs, when what an earlier kernel wrote is in L2 but a line of this SM's L1 may be older.
__device__ __forceinline__ BatchSeq load_seq(const BatchParams& p, int s, bool check_blocks) {
  return check_seq(p, __ldcg(p.row_start + s), __ldcg(p.row_start + s + 1), __ldcg(p.pos_start + s), check_blocks);
}

}  // namespace kvattn
