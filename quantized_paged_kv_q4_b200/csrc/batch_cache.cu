// The cache of a ragged batch, written and read back (kvattn_append_batch, kvattn_read_batch).
//
// One warp takes one (row, KV head): lane l owns channels [8l, 8l + 8), four lanes form one
// 32-channel block, as in the single-sequence encoder.
#include "batch.cuh"
#include "decode.cuh"

namespace kvattn {

// The value that slot `tok` of a key page holds for channels 8 lane .. 8 lane + 7: the reader's
// side of encode_token.
__device__ __forceinline__ void decode_key8(const uint8_t* pg, int tok, int lane, int fmt, float (&x)[8]) {
  const int G = tok >> 4, H = (tok >> 3) & 1, R = tok & 7;
  const int b = lane >> 2, T = lane & 3;
  const int si = 2 * (((G * 8 + R) * 2 + H) * 8 + b);
  if (fmt == kKeyQ8) {
    const uint2 w = *reinterpret_cast<const uint2*>(
        pg + ((((G * 4 + (lane >> 3)) * 2 + H) * 8 + R) * 4 + T) * 16 + 8 * ((lane & 7) >> 2));
    const float d = __half2float(*reinterpret_cast<const __half*>(pg + kKScaleOffset + si));
#pragma unroll
    for (int e = 0; e < 8; ++e)
      x[e] = (static_cast<int>(((e < 4 ? w.x : w.y) >> (8 * (e & 3))) & 255u) - 128) * d;
    return;
  }
  const int c = b & 3, line = (((G * 2 + (b >> 2)) * 2 + H) * 8 + R) * 4 + T;
  const uint32_t w = *reinterpret_cast<const uint32_t*>(pg + 4 * (line * 4 + c));
  uint32_t hb = 0;
  float d, m = 0.f;
  int off = 0;
  if (fmt == kKeyQ4) {
    d = __half2float(*reinterpret_cast<const __half*>(pg + kK4ScaleOffset + si));
    off = 8;
  } else {
    hb = *reinterpret_cast<const uint32_t*>(pg + kK5HighOffset + 4 * line);
    d = __half2float(*reinterpret_cast<const __half*>(pg + kK5ScaleOffset + si));
    if (fmt == kKeyQ51)
      m = __half2float(*reinterpret_cast<const __half*>(pg + kK5MinOffset + si));
    else
      off = 16;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t lo = (w >> (4 * (e >> 1) + 16 * (e & 1))) & 15u;
    const uint32_t hi = (hb >> (16 * (e & 1) + 4 * c + (e >> 1))) & 1u;
    x[e] = fmaf(static_cast<float>(static_cast<int>(lo | (hi << 4)) - off), d, m);
  }
}

__device__ __forceinline__ void decode_val8(const uint8_t* pg, int tok, int lane, int fmt, float (&x)[8]) {
  const int G = tok >> 4, tl = tok & 15;
  const int T = (tl & 7) >> 1, wlo = tl >> 3, ylo = tl & 1;
  const int b = lane >> 2, cl = lane & 3;
  const int si = 2 * (((G * 4 + T) * 8 + b) * 4 + ylo + 2 * wlo);
  if (fmt == kValQ8) {
    const float d = __half2float(*reinterpret_cast<const __half*>(pg + kV8ScaleOffset + si));
    const uint8_t* at = pg + ((G * 8 + b) * 8 * 4 + T) * 16 + 4 * (2 * (cl >> 1) + wlo) + 2 * (cl & 1) + ylo;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (static_cast<int>(at[64 * e]) - 128) * d;
    return;
  }
  const float d = __half2float(*reinterpret_cast<const __half*>(pg + kV4ScaleOffset + si));
  const float m = fmt == kValQ41 ? __half2float(*reinterpret_cast<const __half*>(pg + kV41MinOffset + si)) : 0.f;
  const int off = fmt == kValQ41 ? 0 : 8;
  const uint8_t* at = pg + ((G * 4 + (b >> 1)) * 8 * 4 + T) * 16 + 4 * (2 * (b & 1) + wlo) + 2 * ylo + (cl >> 1);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    x[e] = fmaf(static_cast<float>(((at[64 * e] >> (4 * (cl & 1))) & 15) - off), d, m);
}

// The page and slot of row `row` for KV head h; false: the row belongs to no sequence, or to
// one that a check left out.  page is -1 where the table's id is out of range.
__device__ __forceinline__ bool locate_row(const BatchParams& p, int row, int h, int lane, int* page, int* slot) {
  const int s = find_seq(p.row_start, p.n_seqs, row, lane);
  if (s < 0) return false;
  const BatchSeq q = load_seq(p, s, true);
  if (row < q.r0 || row >= q.r0 + q.rows) return false;
  const int pos = q.pos0 + (row - q.r0);
  const int pg = p.page_table[(static_cast<long long>(s) * p.n_kv + h) * p.max_blocks + pos / kPageTokens];
  *slot = pos % kPageTokens;
  *page = pg;
  if (pg < 0 || pg >= p.n_pages) {
    record_error(KVATTN_ERR_BAD_PAGE);
    *page = -1;
  }
  return true;
}

template <typename T>
__global__ void __launch_bounds__(256) append_batch_kernel(const BatchParams p, const RowsView k, const RowsView v,
                                                           int k_fmt, int v_fmt) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long item = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int row = static_cast<int>(item / p.n_kv), h = static_cast<int>(item % p.n_kv);
  if (row >= p.n_rows) return;
  int page, slot;
  if (!locate_row(p, row, h, lane, &page, &slot) || page < 0) return;
  float kx[8], vx[8];
  load8<T>(k.data, row * k.row_stride + h * k.head_stride + lane * 8, kx);
  load8<T>(v.data, row * v.row_stride + h * v.head_stride + lane * 8, vx);
  encode_token(kx, vx, lane, p.k_pool + page * p.k_stride, p.v_pool + page * p.v_stride, slot, k_fmt, v_fmt,
               0xffffffffu);
}

template <typename T>
__global__ void __launch_bounds__(256) read_batch_kernel(const BatchParams p, const RowsView k, const RowsView v,
                                                         int k_fmt, int v_fmt) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long item = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int row = static_cast<int>(item / p.n_kv), h = static_cast<int>(item % p.n_kv);
  if (row >= p.n_rows) return;
  int page, slot;
  if (!locate_row(p, row, h, lane, &page, &slot)) return;
  float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (k.data) {
    if (page >= 0) decode_key8(p.k_pool + page * p.k_stride, slot, lane, k_fmt, x);
    store8<T>(k.data, row * k.row_stride + h * k.head_stride + lane * 8, x);
  }
  if (v.data) {
    if (page >= 0) decode_val8(p.v_pool + page * p.v_stride, slot, lane, v_fmt, x);
    store8<T>(v.data, row * v.row_stride + h * v.head_stride + lane * 8, x);
  }
}

using RowsKernel = void (*)(BatchParams, RowsView, RowsView, int, int);

static cudaError_t launch_rows(RowsKernel kernel, const BatchParams& p, const RowsView& k, const RowsView& v,
                               int k_fmt, int v_fmt, cudaStream_t stream) {
  const long long items = p.n_rows * p.n_kv;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((items + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, k, v, k_fmt, v_fmt);
}

cudaError_t launch_append_batch(const BatchParams& p, const RowsView& k, const RowsView& v, int dtype, int k_fmt,
                                int v_fmt, cudaStream_t stream) {
  const RowsKernel f = dtype == KVATTN_F32   ? append_batch_kernel<float>
                       : dtype == KVATTN_F16 ? append_batch_kernel<__half>
                                             : append_batch_kernel<__nv_bfloat16>;
  return launch_rows(f, p, k, v, k_fmt, v_fmt, stream);
}

cudaError_t launch_read_batch(const BatchParams& p, const RowsView& k, const RowsView& v, int dtype, int k_fmt,
                              int v_fmt, cudaStream_t stream) {
  const RowsKernel f = dtype == KVATTN_F32   ? read_batch_kernel<float>
                       : dtype == KVATTN_F16 ? read_batch_kernel<__half>
                                             : read_batch_kernel<__nv_bfloat16>;
  return launch_rows(f, p, k, v, k_fmt, v_fmt, stream);
}

}  // namespace kvattn
