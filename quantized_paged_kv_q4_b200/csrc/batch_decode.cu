// Attention of a ragged batch over its pages (kvattn_decode_batch).
//
// One CTA takes one (row, KV head) and one query head of the group; its warps take the
// visible tokens in turn, each with an online softmax of its own, merged through shared
// memory at the end.
#include "batch.cuh"

namespace kvattn {

struct BatchDecodeParams {
  BatchParams b;
  RowsView q, out;
  float* lse;
  const int32_t* page_logical;  // [n_seqs][n_kv][max_blocks] or null
  const int32_t* n_list;        // [n_seqs][n_kv] or null
  int group, window;
  uint8_t* ws;
};

template <typename T>
__global__ void __launch_bounds__(256) decode_batch_kernel(const BatchDecodeParams p, int k_fmt, int v_fmt) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float sm[8], sl[8], so[8][kHeadDim];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x, hq = blockIdx.y, h = hq / p.group;
  const int s = find_seq(p.b.row_start, p.b.n_seqs, row, lane);
  if (s < 0) return;
  const BatchSeq sq = load_seq(p.b, s, !p.page_logical);
  if (row < sq.r0 || row >= sq.r0 + sq.rows) return;
  const int pos = sq.pos0 + (row - sq.r0);
  const int lowest = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  const long long unit = static_cast<long long>(s) * p.b.n_kv + h;
  const int32_t* table = p.b.page_table + unit * p.b.max_blocks;
  const int32_t* logical = p.page_logical ? p.page_logical + unit * p.b.max_blocks : nullptr;
  const int n = p.n_list ? min(max(p.n_list[unit], 0), p.b.max_blocks)
                : logical ? p.b.max_blocks : (sq.pos0 + sq.rows + kPageTokens - 1) / kPageTokens;
  float qx[8], o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  load8<T>(p.q.data, row * p.q.row_stride + hq * p.q.head_stride + lane * 8, qx);
  float m = -INFINITY, l = 0.f;
  for (int i = 0; i < n; ++i) {
    const int b = logical ? logical[i] : i;
    if (b < 0 || b > pos / kPageTokens || b < lowest / kPageTokens) continue;
    const int page = table[i];
    if (page < 0 || page >= p.b.n_pages) {
      record_error(KVATTN_ERR_BAD_PAGE);
      continue;
    }
    for (int t = warp; t < kPageTokens; t += 8) {
      const int key = b * kPageTokens + t;
      if (key > pos || key < lowest) continue;
      float x[8];
      decode_key8(p.b.k_pool + page * p.b.k_stride, t, lane, k_fmt, x);
      float d = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) d = fmaf(x[e], qx[e], d);
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) d += __shfl_xor_sync(0xffffffffu, d, w);
      d *= 0.0625f;
      const float m1 = fmaxf(m, d), a = expf(m - m1), w = expf(d - m1);
      decode_val8(p.b.v_pool + page * p.b.v_stride, t, lane, v_fmt, x);
      l = l * a + w;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = o[e] * a + w * x[e];
      m = m1;
    }
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) so[warp][lane * 8 + e] = o[e];
  __syncthreads();
  if (warp) return;
  float M = -INFINITY, L = 0.f, r[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int w = 0; w < 8; ++w) M = fmaxf(M, sm[w]);
  for (int w = 0; w < 8 && M != -INFINITY; ++w) {
    const float a = expf(sm[w] - M);
    L += a * sl[w];
    for (int e = 0; e < 8; ++e) r[e] += a * so[w][lane * 8 + e];
  }
  for (int e = 0; e < 8; ++e) r[e] = M == -INFINITY ? 0.f : r[e] / L;
  store8<T>(p.out.data, row * p.out.row_stride + hq * p.out.head_stride + lane * 8, r);
  if (lane == 0) p.lse[static_cast<long long>(row) * (p.b.n_kv * p.group) + hq] = M == -INFINITY ? M : M + logf(L);
}

cudaError_t launch_decode_batch(const BatchDecodeParams& p, int dtype, int k_fmt, int v_fmt, cudaStream_t stream) {
  auto* f = dtype == KVATTN_F32   ? decode_batch_kernel<float>
            : dtype == KVATTN_F16 ? decode_batch_kernel<__half>
                                  : decode_batch_kernel<__nv_bfloat16>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.b.n_rows), p.b.n_kv * p.group);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, f, p, k_fmt, v_fmt);
}

}  // namespace kvattn
