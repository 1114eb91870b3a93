// The cache of a ragged batch, written and read back (kvattn_append_batch, kvattn_read_batch).
//
// One warp takes a quarter (64 channels of K and of V) of one (tile of 16 positions of a sequence, KV
// head).  A page's codes and scales sit in tensor-core fragment order by such tiles, so a tile is a
// few contiguous ranges of the page, and lane (g, t) = (lane / 4, lane % 4) of a warp that holds rows
// 8H + g, channels 32b + 8t .. + 7 of every block b holds, block by block, exactly the key bytes it
// stores: 16 of them per 64 channels.  The four lanes of a quad form one 32-channel block, as in
// the single-sequence encoder.  Values are stored transposed (a lane's bytes belong to four
// tokens), which takes four shuffles per block and eight tokens.
//
// Reading is bound by HBM: 131,072 tokens of 4 KV heads (Q8_0 / Q4_0, 218 MB) into bf16 (537 MB)
// take 123 us, 0.95 of the measured copy bandwidth.  Writing a whole tile costs about 1,250
// instructions a quarter (scales by IEEE division and reciprocal, codes by the format's own fp32
// steps): six prompts of 100 to 4,000 tokens (28 MB of bf16 rows, 8 MB of pages) take 20 us, a
// third of the copy bandwidth.  A warp encodes K and then V, both loaded from the start, so that 39 % of
// the warps are active (64 registers; 91 for fp32 rows) and issue 0.64 instructions a cycle, in one and a
// half waves of CTAs.  One to eight tokens take 3 us a call, latency alone.
// Measured on the way: one warp per (row, head), with its byte stores and strided page reads: 215 us
// for the 131,072 tokens; a whole tile a warp: 49.8 us to write the six prompts and read them back
// (25.7 us in quarters).  Not kept: codes made by adding 2^23 with downward rounding and packed by
// multiply-adds on the biased bits (the same bytes, 25.0 instead of 25.7 us).
//
// A tile that the call's rows fill in part is written token by token with byte stores (its other
// tokens' bits share bytes and words with them, and stay).
#include "batch.cuh"
#include "decode.cuh"

namespace kvattn {

// One warp's share: KV head h, tile `tile` (of the sequence's 16-token tiles) of sequence s, its
// rows [r0, r0 + n) at slots [slot, slot + n) of page `page` (to be checked by page_ok, once other
// loads are on their way).
struct TileRows {
  int s, page, slot, n;
  long long r0;
};

// Tile slots: sequence s owns slots row_start[s] / 16 + 2 s ..., at least as many as its rows touch
// tiles, so a slot's sequence is found by a search without any prefix sum.
__device__ __forceinline__ long long slot_base(int r0, int s) { return (static_cast<long long>(r0) >> 4) + 2ll * s; }

__device__ __forceinline__ bool locate_tile(const BatchParams& p, long long at, int h, int lane, TileRows* out) {
  // the last sequence whose slots start at or before `at`, 32 candidates a step; whatever row_start
  // holds, the answer stays inside [0, n_seqs) and is checked below.  In the last step the lanes
  // load the rest of their candidates too, so that the answer's is there at once.
  int lo = 0, hi = p.n_seqs;
  BatchSeq q;
  long long base;
  while (true) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    int r0 = 0, r1 = 0, pos0 = 0;
    if (i < hi) {
      r0 = p.row_start[i];
      if (step == 1) {
        r1 = p.row_start[i + 1];
        pos0 = p.pos_start[i];
      }
    }
    const uint32_t le = __ballot_sync(0xffffffffu, i < hi && slot_base(r0, i) <= at);
    if (le == 0) return false;
    const int found = 31 - __clz(le);
    lo += found * step;
    hi = min(hi, lo + step);
    if (step == 1) {
      r0 = __shfl_sync(0xffffffffu, r0, found);
      base = slot_base(r0, lo);
      q = check_seq(p, r0, __shfl_sync(0xffffffffu, r1, found), __shfl_sync(0xffffffffu, pos0, found), true);
      break;
    }
  }
  if (q.rows == 0) return false;
  const long long tile = q.pos0 / 16 + (at - base);
  const long long first = max(tile * 16, static_cast<long long>(q.pos0));
  const long long end = min(tile * 16 + 16, static_cast<long long>(q.pos0) + q.rows);
  if (tile < q.pos0 / 16 || first >= end) return false;
  out->s = lo;
  out->slot = static_cast<int>(first % kPageTokens);
  out->n = static_cast<int>(end - first);
  out->r0 = q.r0 + (first - q.pos0);
  out->page = p.page_table[(static_cast<long long>(lo) * p.n_kv + h) * p.max_blocks + first / kPageTokens];
  return true;
}

__device__ __forceinline__ bool page_ok(const BatchParams& p, int page, int lane) {
  const bool ok = page >= 0 && page < p.n_pages;
  if (!ok && lane == 0) record_error(KVATTN_ERR_BAD_PAGE);
  return ok;
}

// ------------------------------------------------------------------------------ writing
// Eight codes of a block (this lane's quarter) of either side's formats, with the scale and minimum
// that every lane of the quad gets.  FMT: 8 (Q8_0, the byte q + 128), 4 / 50 (Q4_0 / Q5_0), 41 / 51.
template <int FMT>
__device__ __forceinline__ void encode8(const float (&x)[8], int lane, uint32_t (&q)[8], uint32_t* d16, uint32_t* m16) {
  float inv, d, mn = 0.f;
  if constexpr (FMT == KVATTN_FMT_Q8_0) {
    d = q8_scale(x, &inv);
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = static_cast<uint32_t>(q8_code(x[e], inv) + 128);
  } else if constexpr (FMT == KVATTN_FMT_Q4_0 || FMT == KVATTN_FMT_Q5_0) {
    constexpr int kHalf = FMT == KVATTN_FMT_Q4_0 ? 8 : 16;
    d = offset_scale<kHalf>(x, lane, &inv);
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = static_cast<uint32_t>(offset_code<kHalf>(x[e], inv));
  } else {
    constexpr int kTop = FMT == KVATTN_FMT_Q4_1 ? 15 : 31;
    d = min_scale<kTop>(x, &mn, &inv);
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = static_cast<uint32_t>(min_code<kTop>(x[e], mn, inv));
  }
  *d16 = __half_as_ushort(__float2half_rn(d));
  *m16 = __half_as_ushort(__float2half_rn(mn));
}

// The rows of a quarter tile, as every lane takes them: row 8H + g, channels 64 part + 32e + 8t ...
template <typename T>
__device__ __forceinline__ void load_quarter(const T* rows, long long row_stride, int part, int lane,
                                             Raw8<T> (&raw)[2][2]) {
#pragma unroll
  for (int H = 0; H < 2; ++H)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      raw[H][e] = load_raw8<T>(rows + (8 * H + (lane >> 2)) * row_stride, 64 * part + 32 * e + 8 * (lane & 3));
}

// Channels 64 P .. + 63 of a whole tile of keys, to their bytes of the page.
template <typename T, int FMT>
__device__ __forceinline__ void write_keys(const Raw8<T> (&raw)[2][2], uint8_t* pg, int G, int P, int lane) {
  const int g = lane >> 2, t = lane & 3;
  constexpr bool k8 = FMT == KVATTN_FMT_Q8_0, k5 = FMT == KVATTN_FMT_Q5_0 || FMT == KVATTN_FMT_Q5_1;
  constexpr int kScale = k8 ? kKScaleOffset : k5 ? kK5ScaleOffset : kK4ScaleOffset;
#pragma unroll
  for (int H = 0; H < 2; ++H) {
    uint32_t q[2][8], d[2], m[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x[8];
      widen8<T>(raw[H][e], x);
      encode8<FMT>(x, lane, q[e], &d[e], &m[e]);
    }
    if constexpr (k8) {
      // the lane's 16 bytes: block 2P in 0-7, block 2P + 1 in 8-15
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t* c = q[i >> 1] + 4 * (i & 1);
        w[i] = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24;
      }
      *reinterpret_cast<uint4*>(pg + G * 4096 + ((((P * 2 + H) * 8 + g) * 4 + t) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      // two of the four words of the lane's 16 bytes; fifth bits: two of the four bytes of its word
      const int line = ((((P >> 1) * 2 + H) * 8 + g) * 4 + t), c0 = 2 * (P & 1);
      uint32_t w[2] = {0u, 0u}, high = 0;
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          w[c] |= (q[c][e] & 15u) << (4 * (e >> 1) + 16 * (e & 1));
          if constexpr (k5) high |= (q[c][e] >> 4) << (16 * (e & 1) + 4 * c + (e >> 1));
        }
      *reinterpret_cast<uint2*>(pg + G * 2048 + 16 * line + 4 * c0) = make_uint2(w[0], w[1]);
      if constexpr (k5) {
        uint8_t* to = pg + kK5HighOffset + G * 512 + 4 * line + (P & 1);
        to[0] = static_cast<uint8_t>(high);
        to[2] = static_cast<uint8_t>(high >> 16);
      }
    }
    if (t == 0) {
      const int si = G * 256 + ((g * 2 + H) * 8 + 2 * P) * 2;
      *reinterpret_cast<uint32_t*>(pg + kScale + si) = d[0] | d[1] << 16;
      if constexpr (FMT == KVATTN_FMT_Q5_1) *reinterpret_cast<uint32_t*>(pg + kK5MinOffset + si) = m[0] | m[1] << 16;
    }
  }
}

// Channels 64 C .. + 63 of a whole tile of values.  Lane (g, t) encodes token 8H + g, channels 32b + 8t
// + e; lane (R, T) stores, per block, the codes of channels R, R + 8, R + 16, R + 24 of tokens 2T,
// 2T + 1 (and + 8).
template <typename T, int FMT>
__device__ __forceinline__ void write_values(const Raw8<T> (&raw)[2][2], uint8_t* pg, int G, int C, int lane) {
  const int g = lane >> 2, t = lane & 3;  // as a source; as a target R = g, T = t
  constexpr bool v8 = FMT == KVATTN_FMT_Q8_0;
  constexpr int kScale = v8 ? kV8ScaleOffset : kV4ScaleOffset;
  const int src = 8 * t + (g >> 2);  // lane (token 2T, channel group R / 4)
  const uint32_t pick = g & 3;       // byte R % 4 of its word
  uint32_t w[2][4];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int b = 2 * C + e;
#pragma unroll
    for (int H = 0; H < 2; ++H) {
      float x[8];
      uint32_t q[8], d, m;
      widen8<T>(raw[H][e], x);
      encode8<FMT>(x, lane, q, &d, &m);
      if (t == 0) {
        const int si = G * 256 + (((g >> 1) * 8 + b) * 4 + (g & 1) + 2 * H) * 2;
        *reinterpret_cast<uint16_t*>(pg + kScale + si) = static_cast<uint16_t>(d);
        if constexpr (FMT == KVATTN_FMT_Q4_1) *reinterpret_cast<uint16_t*>(pg + kV41MinOffset + si) = static_cast<uint16_t>(m);
      }
      if constexpr (v8) {
        const uint32_t lo = q[0] | q[1] << 8 | q[2] << 16 | q[3] << 24, hi = q[4] | q[5] << 8 | q[6] << 16 | q[7] << 24;
        // lane (token, t') holds channels 8t' + 0..3 in lo and + 4..7 in hi; R / 4 picks one
#pragma unroll
        for (int x16 = 0; x16 < 2; ++x16) {
          uint32_t by[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int from = 4 * (2 * t + (y & 1)) + 2 * x16 + (y >> 1);
            const uint32_t a = __shfl_sync(0xffffffffu, lo, from), b2 = __shfl_sync(0xffffffffu, hi, from);
            by[y] = prmt(g >= 4 ? b2 : a, 0u, pick);
          }
          w[e][2 * x16 + H] = prmt(prmt(by[0], by[1], 0x0040u), prmt(by[2], by[3], 0x0040u), 0x5410u);
        }
      } else {
        // eight 4-bit codes; with the neighbour's (channels + 8), lane t makes the bytes of channel
        // group t / 2, elements 4 (t % 2) .. + 3: low nibble channel 16 (t / 2) + e, high + 8
        uint32_t own = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) own |= q[i] << (4 * i);
        const uint32_t other = __shfl_xor_sync(0xffffffffu, own, 1);
        const uint32_t half = (t & 1) * 16;
        const uint32_t lo = ((t & 1) ? other : own) >> half, hi = ((t & 1) ? own : other) >> half;
        // four nibbles over four bytes
        auto spread = [](uint32_t v) {
          v = (v & 0xFFu) | ((v & 0xFF00u) << 8);
          return (v & 0x000F000Fu) | ((v & 0x00F000F0u) << 4);
        };
        const uint32_t word = spread(lo) | spread(hi) << 4;
        // bytes of (2T, x16 = 0), (2T, 1), (2T + 1, 0), (2T + 1, 1) for element R
        const uint32_t b0 = __shfl_sync(0xffffffffu, word, src), b1 = __shfl_sync(0xffffffffu, word, src + 2);
        const uint32_t b2 = __shfl_sync(0xffffffffu, word, src + 4), b3 = __shfl_sync(0xffffffffu, word, src + 6);
        const uint32_t sel = pick | (pick + 4) << 4;
        w[e][H] = prmt(prmt(b0, b1, sel), prmt(b2, b3, sel), 0x5410u);
      }
    }
  }
  if constexpr (v8) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      *reinterpret_cast<uint4*>(pg + G * 4096 + (((2 * C + e) * 8 + g) * 4 + t) * 16) =
          make_uint4(w[e][0], w[e][1], w[e][2], w[e][3]);
  } else {
    *reinterpret_cast<uint4*>(pg + G * 2048 + ((C * 8 + g) * 4 + t) * 16) = make_uint4(w[0][0], w[0][1], w[1][0], w[1][1]);
  }
}

// The warp's share of the grid: quarter of the tile, head, tile slot.
__device__ __forceinline__ bool locate_share(const BatchParams& p, int lane, int* quarter, int* h, TileRows* tr) {
  const long long item = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  *quarter = static_cast<int>(item & 3);
  *h = static_cast<int>((item >> 2) % p.n_kv);
  return locate_tile(p, (item >> 2) / p.n_kv, *h, lane, tr);
}

template <typename T>
__global__ void __launch_bounds__(256) append_batch_kernel(const BatchParams p, const RowsView k, const RowsView v,
                                                           int k_fmt, int v_fmt) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  int part, h;
  TileRows tr;
  if (!locate_share(p, lane, &part, &h, &tr)) return;
  const T* kr = static_cast<const T*>(k.data) + tr.r0 * k.row_stride + h * k.head_stride;
  const T* vr = static_cast<const T*>(v.data) + tr.r0 * v.row_stride + h * v.head_stride;
  uint8_t* kpg = p.k_pool + tr.page * p.k_stride;
  uint8_t* vpg = p.v_pool + tr.page * p.v_stride;
  if (tr.n == 16) {
    const int G = tr.slot >> 4;
    Raw8<T> kraw[2][2], vraw[2][2];
    load_quarter(kr, k.row_stride, part, lane, kraw);
    load_quarter(vr, v.row_stride, part, lane, vraw);
    if (!page_ok(p, tr.page, lane)) return;
    switch (k_fmt) {
      case kKeyQ8: write_keys<T, KVATTN_FMT_Q8_0>(kraw, kpg, G, part, lane); break;
      case kKeyQ4: write_keys<T, KVATTN_FMT_Q4_0>(kraw, kpg, G, part, lane); break;
      case kKeyQ51: write_keys<T, KVATTN_FMT_Q5_1>(kraw, kpg, G, part, lane); break;
      default: write_keys<T, KVATTN_FMT_Q5_0>(kraw, kpg, G, part, lane); break;
    }
    switch (v_fmt) {
      case kValQ4: write_values<T, KVATTN_FMT_Q4_0>(vraw, vpg, G, part, lane); break;
      case kValQ8: write_values<T, KVATTN_FMT_Q8_0>(vraw, vpg, G, part, lane); break;
      default: write_values<T, KVATTN_FMT_Q4_1>(vraw, vpg, G, part, lane); break;
    }
    return;
  }
  // part of a tile: the four warps take its tokens in turn
#pragma unroll 1
  for (int i = part; i < tr.n; i += 4) {
    const Raw8<T> kraw = load_raw8<T>(kr, i * k.row_stride + lane * 8), vraw = load_raw8<T>(vr, i * v.row_stride + lane * 8);
    if (!page_ok(p, tr.page, lane)) return;
    float kx[8], vx[8];
    widen8<T>(kraw, kx);
    widen8<T>(vraw, vx);
    encode_token(kx, vx, lane, kpg, vpg, tr.slot + i, k_fmt, v_fmt, 0xffffffffu);
  }
}

// ------------------------------------------------------------------------------ reading
// Stores a quad's 32 channels of one row, 8 per lane, in whole 32-byte sectors: fp32 lanes exchange
// halves with their neighbour first, so that each of the two stores covers full sectors.
template <typename T>
__device__ __forceinline__ void store_quad8(T* row, int t, const float (&x)[8], bool live) {
  if constexpr (sizeof(T) == 4) {
    const bool odd = t & 1;
    float4 a, b;
    float* pa = &a.x;
    float* pb = &b.x;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float got = __shfl_xor_sync(0xffffffffu, odd ? x[e] : x[4 + e], 1);
      pa[e] = odd ? got : x[e];      // first store: the even lane's eight channels
      pb[e] = odd ? x[4 + e] : got;  // second store: the odd lane's
    }
    if (live) {
      float* at = reinterpret_cast<float*>(row) + 8 * (t & 2) + 4 * odd;
      *reinterpret_cast<float4*>(at) = a;
      *reinterpret_cast<float4*>(at + 8) = b;
    }
  } else {
    if (live) store8<T>(row, 8 * t, x);
  }
}

// Channels 64 P .. + 63 of the tile's rows [lo, lo + n).
template <typename T, int FMT>
__device__ __forceinline__ void read_keys(T* rows, long long row_stride, const uint8_t* pg, int G, int P, int lane,
                                          int lo, int n) {
  const int g = lane >> 2, t = lane & 3;
  constexpr bool k8 = FMT == KVATTN_FMT_Q8_0, k5 = FMT == KVATTN_FMT_Q5_0 || FMT == KVATTN_FMT_Q5_1;
  constexpr int kScale = k8 ? kKScaleOffset : k5 ? kK5ScaleOffset : kK4ScaleOffset;
  uint4 w[2];
  uint32_t d[2], m[2] = {0u, 0u}, high[2] = {0u, 0u};
#pragma unroll
  for (int H = 0; H < 2; ++H) {
    if constexpr (k8) {
      w[H] = *reinterpret_cast<const uint4*>(pg + G * 4096 + (((P * 2 + H) * 8 + g) * 4 + t) * 16);
    } else {
      const int line = (((P >> 1) * 2 + H) * 8 + g) * 4 + t;
      const uint2 u = *reinterpret_cast<const uint2*>(pg + G * 2048 + 16 * line + 8 * (P & 1));
      w[H] = make_uint4(u.x, u.y, 0u, 0u);
      if constexpr (k5)
        high[H] = *reinterpret_cast<const uint32_t*>(pg + kK5HighOffset + G * 512 + 4 * line) >> (8 * (P & 1));
    }
    const int si = G * 256 + ((g * 2 + H) * 8 + 2 * P) * 2;
    d[H] = *reinterpret_cast<const uint32_t*>(pg + kScale + si);
    if constexpr (FMT == KVATTN_FMT_Q5_1) m[H] = *reinterpret_cast<const uint32_t*>(pg + kK5MinOffset + si);
  }
#pragma unroll
  for (int H = 0; H < 2; ++H) {
    const int row = 8 * H + g;
    const bool live = row >= lo && row < lo + n;
    T* to = rows + row * row_stride + 64 * P;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float db = c ? half_hi(d[H]) : half_lo(d[H]);
      float x[8];
      if constexpr (k8) {
        const uint32_t a = c ? w[H].z : w[H].x, b = c ? w[H].w : w[H].y;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          x[e] = static_cast<float>(static_cast<int>(((e < 4 ? a : b) >> (8 * (e & 3))) & 255u) - 128) * db;
      } else {
        const uint32_t a = c ? w[H].y : w[H].x;
        const float mb = c ? half_hi(m[H]) : half_lo(m[H]);
        constexpr int kOff = FMT == KVATTN_FMT_Q4_0 ? 8 : FMT == KVATTN_FMT_Q5_0 ? 16 : 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          uint32_t q = (a >> (4 * (e >> 1) + 16 * (e & 1))) & 15u;
          if constexpr (k5) q |= ((high[H] >> (16 * (e & 1) + 4 * c + (e >> 1))) & 1u) << 4;
          const float v = static_cast<float>(static_cast<int>(q) - kOff);
          x[e] = FMT == KVATTN_FMT_Q5_1 ? fmaf(v, db, mb) : v * db;
        }
      }
      store_quad8<T>(to + 32 * c, t, x, live);
    }
  }
}

// Values come as channels R, R + 8, ... of four tokens a lane; they go through the warp's shared
// rows (16 x 32 channels, a block at a time) to be stored along the channels.
constexpr int kReadStride = 36;  // floats: lane (R, T) writes bank 8T + R (+ const), lane (g, t) reads 16 bytes

template <typename T, int FMT>
__device__ __forceinline__ void read_values(T* rows, long long row_stride, const uint8_t* pg, int G, int C, int lane,
                                            int lo, int n, float* buf) {
  const int g = lane >> 2, t = lane & 3;  // as the page's lane: R = g, T = t
  constexpr bool v8 = FMT == KVATTN_FMT_Q8_0;
  constexpr int kScale = v8 ? kV8ScaleOffset : kV4ScaleOffset;
  uint4 w[2];
  uint2 d[2], m[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (v8 || e == 0)
      w[e] = *reinterpret_cast<const uint4*>(pg + G * (v8 ? 4096 : 2048) + (((v8 ? 2 * C + e : C) * 8 + g) * 4 + t) * 16);
    d[e] = *reinterpret_cast<const uint2*>(pg + kScale + G * 256 + (t * 8 + 2 * C + e) * 8);
    if constexpr (FMT == KVATTN_FMT_Q4_1)
      m[e] = *reinterpret_cast<const uint2*>(pg + kV41MinOffset + G * 256 + (t * 8 + 2 * C + e) * 8);
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    __syncwarp();
#pragma unroll
    for (int H = 0; H < 2; ++H) {
      const uint32_t dw = H ? d[e].y : d[e].x;
      const float ds[2] = {half_lo(dw), half_hi(dw)};  // tokens 2T, 2T + 1 (+ 8H)
      float ms[2] = {0.f, 0.f};
      if constexpr (FMT == KVATTN_FMT_Q4_1) {
        const uint32_t mw = H ? m[e].y : m[e].x;
        ms[0] = half_lo(mw);
        ms[1] = half_hi(mw);
      }
#pragma unroll
      for (int x16 = 0; x16 < 2; ++x16)
#pragma unroll
        for (int x8 = 0; x8 < 2; ++x8)
#pragma unroll
          for (int odd = 0; odd < 2; ++odd) {
            int q;
            if constexpr (v8) {
              const uint32_t word = x16 ? (H ? w[e].w : w[e].z) : (H ? w[e].y : w[e].x);
              q = static_cast<int>((word >> (8 * (2 * x8 + odd))) & 255u) - 128;
            } else {
              const uint32_t word = e ? (H ? w[0].w : w[0].z) : (H ? w[0].y : w[0].x);
              q = static_cast<int>((word >> (8 * (2 * odd + x16) + 4 * x8)) & 15u) - (FMT == KVATTN_FMT_Q4_0 ? 8 : 0);
            }
            buf[(2 * t + odd + 8 * H) * kReadStride + 16 * x16 + 8 * x8 + g] =
                FMT == KVATTN_FMT_Q4_1 ? fmaf(static_cast<float>(q), ds[odd], ms[odd]) : static_cast<float>(q) * ds[odd];
          }
    }
    __syncwarp();
#pragma unroll
    for (int H = 0; H < 2; ++H) {
      const int row = 8 * H + g;
      const float4 a = *reinterpret_cast<const float4*>(buf + row * kReadStride + 8 * t);
      const float4 b = *reinterpret_cast<const float4*>(buf + row * kReadStride + 8 * t + 4);
      const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      store_quad8<T>(rows + row * row_stride + 32 * (2 * C + e), t, x, row >= lo && row < lo + n);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(256) read_batch_kernel(const BatchParams p, const RowsView k, const RowsView v,
                                                         int k_fmt, int v_fmt) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ __align__(16) float bufs[8][16 * kReadStride];
  const int lane = threadIdx.x & 31;
  int part, h;
  TileRows tr;
  if (!locate_share(p, lane, &part, &h, &tr)) return;
  const int G = tr.slot >> 4, lo = tr.slot & 15;
  T* kr = static_cast<T*>(k.data) + (tr.r0 - lo) * k.row_stride + h * k.head_stride;  // row of the tile's first token
  T* vr = static_cast<T*>(v.data) + (tr.r0 - lo) * v.row_stride + h * v.head_stride;
  if (!page_ok(p, tr.page, lane)) {
    const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int i = lo + part; i < lo + tr.n; i += 4) {
      if (k.data) store8<T>(kr, i * k.row_stride + 8 * lane, zero);
      if (v.data) store8<T>(vr, i * v.row_stride + 8 * lane, zero);
    }
    return;
  }
  const uint8_t* kpg = p.k_pool + tr.page * p.k_stride;
  const uint8_t* vpg = p.v_pool + tr.page * p.v_stride;
  if (k.data) {
    switch (k_fmt) {
      case kKeyQ8: read_keys<T, KVATTN_FMT_Q8_0>(kr, k.row_stride, kpg, G, part, lane, lo, tr.n); break;
      case kKeyQ4: read_keys<T, KVATTN_FMT_Q4_0>(kr, k.row_stride, kpg, G, part, lane, lo, tr.n); break;
      case kKeyQ51: read_keys<T, KVATTN_FMT_Q5_1>(kr, k.row_stride, kpg, G, part, lane, lo, tr.n); break;
      default: read_keys<T, KVATTN_FMT_Q5_0>(kr, k.row_stride, kpg, G, part, lane, lo, tr.n); break;
    }
  }
  if (v.data) {
    float* buf = bufs[threadIdx.x >> 5];
    switch (v_fmt) {
      case kValQ4: read_values<T, KVATTN_FMT_Q4_0>(vr, v.row_stride, vpg, G, part, lane, lo, tr.n, buf); break;
      case kValQ8: read_values<T, KVATTN_FMT_Q8_0>(vr, v.row_stride, vpg, G, part, lane, lo, tr.n, buf); break;
      default: read_values<T, KVATTN_FMT_Q4_1>(vr, v.row_stride, vpg, G, part, lane, lo, tr.n, buf); break;
    }
  }
}

using RowsKernel = void (*)(BatchParams, RowsView, RowsView, int, int);

static cudaError_t launch_rows(RowsKernel kernel, const BatchParams& p, const RowsView& k, const RowsView& v,
                               int k_fmt, int v_fmt, cudaStream_t stream) {
  const long long items = (p.n_rows / 16 + 2ll * p.n_seqs) * p.n_kv * 4;  // tile slots x heads x quarters
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
