// Split-KV flash decode of a ragged batch over its pages (kvattn_decode_batch): several sequences
// of different lengths in one grid ([STREAM] method list: paged decode attention over single
// tokens and verify batches).
//
// A unit is one (sequence, KV head): its query rows (group x rows <= 24) against its 16-token
// tiles.  A group of warps works by itself: it streams its own tiles through its own ring of
// stages, keeps its own softmax state and writes its own results.  No group waits for another, so
// what a unit costs beside its tiles (query fragments, output) hides behind the arithmetic of the
// SM's other groups, and the ring runs on from one unit into the next.  The copies are 16 bytes a
// lane (cp.async): a tile has four to six short regions, and a bulk copy of each, issued by the
// warp that also computes, took 700 of the 3,400 cycles a tile.
//
// Up to 8 query rows (one n-tile) a group is one warp (decode_batch_kernel).  With 9 to 24 rows it
// is four (decode_batch_wide_kernel): each takes the scores of one tile of a step of four, for all
// rows, and then a quarter of the channels of all four tiles' values, so that every code is
// decoded once, not once per n-tile; P goes between them through shared memory.
//
// All units form one line, each as long as its tiles and what it costs beside them (kUnitCost),
// and every group takes an equal stretch of it, whatever the lengths are: a group may hold the end
// of one unit, some whole ones and the start of another.  The stretches are found on the device,
// because the lengths live there: every CTA adds up all sequences (one or a few per thread, then a
// scan) and looks its groups' ends up.  A unit inside one group's stretch is written to out at
// once; otherwise each of its groups leaves an (o, lse) partial and a second grid merges them, in
// a fixed order.  A group has at most two partials, its first unit's and its last's, so the
// workspace has two slots per group.
//
// What bounds it.  With 8 rows and bf16 a tile takes a warp about 690 instructions: eight sequences of
// 131,072 tokens (1.745 GB, Q8_0 / Q4_0) take 288 to 293 us in short runs, 0.92 to 0.94 of the measured copy
// bandwidth, and 331 us back to back, 0.82, where the 1,000 W cap lowers the SM clock.  fp32 (the query's second
// part, sums added tile by tile) is bound by its arithmetic: 433 us.  With 24 rows a tile takes 1,500
// instructions at 0.46 a cycle (dependent instructions, the pace of mma.sync, shared-memory latency, two
// barriers a step): eight verify steps of four tokens (149 MB) take 78 us, 0.30 of that bandwidth.  Short batches are bound
// by latency: the plan 2.4 us, pages and queries 3 us, then 1.5 to 2 us a tile and group, and the merge grid.
//
// What precision costs (one run, captured graphs; the three figures are 8 x 131,072, 32 ragged and 8
// verify steps in bf16).  P in one f16 part, P x scale as it comes: 264, 39.8, 64.2 us, with errors of 3e-4
// before the store, and of percents where a dominant key meets small values.  P in two parts: 286,
// 42.9, 75.4.  With the powers of two, and what is not finite told apart: 288, 41.2, 77.8.
//
// Not kept: a CTA of four groups on one stretch, their states merged through shared memory at the
// end of each unit (2 to 4 us of barriers a unit: 32 ragged sequences of up to 16,384 tokens in
// 51.9 us, against 40.4); three warps per tile with 24 rows, one per n-tile (eight verify steps of
// four tokens in 81 us).
#include <algorithm>

#include "batch.cuh"
#include "decode_tile.cuh"

namespace kvattn {

struct BatchDecodeParams {
  BatchParams b;
  RowsView q, out;
  float* lse;
  const int32_t* page_logical;  // [n_seqs][n_kv][max_blocks] or null
  const int32_t* n_list;        // [n_seqs][n_kv] or null
  int group, window;
  // workspace: where each unit's partials are (first slot, last group), and two partials per group
  int2* unit_parts;
  float* part_lse;  // [groups][2][rows_pad], base 2
  float* part_o;    // [groups][2][rows_pad][256]
};

// The query's f16 parts, and the power of two that its row's largest magnitude is scaled to (2^kTop to 2^(kTop
// + 1), as high as f16 holds it: elements far below it keep their bits).  16-bit inputs take one part: every
// fp16 row is exact so, and a bf16 element down to 2^-32 of the row's largest (below that, to 2^-40 of it).
// fp32 takes two, about 22 bits down to 2^-17 of the largest, and 2^-39 of it below.
template <typename T>
struct BatchParts {
  static constexpr int kQ = sizeof(T) == 4 ? 2 : 1, kTop = sizeof(T) == 4 ? 14 : 15;
  static constexpr int kSum = 6;  // block sums (zero-point keys) are 2^5 elements: divided by 2^6 they fit f16
  // mma_parts: with bf16 outputs what the MMA cuts stays below the store's rounding (2,048 tiles in one stretch
  // lose 2.2e-4 of the sum, half a bf16 step is 2e-3 at least), and adding tile by tile costs 2 to 8 %
  static constexpr bool kSums = !std::is_same_v<T, __nv_bfloat16>;
};

// One unit: its n tiles start at tile t0 of its list of pages (n = 0: a sequence without rows).
struct BatchUnit {
  int unit, h, r0, rows, pos0, t0, n;
};

// What a warp's copying keeps between two tiles, in shared memory (registers are the tile's): the
// unit of the next tile, where that starts in the group's numbering, the positions its rows see,
// and either the page at hand (its first position, -1: nothing of it is fetched, and its bytes) or
// the next step's first tile.
struct alignas(16) Producer {
  int unit, start, t0, n;  // read together, as are the next four
  int last, low, key0, next;
  const uint8_t *k, *v;
};

// The CTA's plan, in shared memory.
template <int WARPS, int GROUPS>
struct alignas(16) BatchPlanState {
  int tiles[WARPS], units[WARPS];        // of the warps' sequences
  int from[GROUPS], to[GROUPS];          // the groups' ends on the line of all tiles
  BatchUnit unit[GROUPS];                // each group's first unit ...
  int skip[GROUPS];                      // ... and its tiles that come before the group's
  BatchUnit at_work[WARPS];              // each warp's unit (not in registers while the tiles run)
  Producer producer[WARPS];
};

constexpr int kBatchRoom = 224 * 1024;  // of shared memory, for rings, fragments and P; 3 KB for the plan
constexpr int kBatchMeta = 3 * 1024;

// One CTA per SM, of as many groups (warps) as shared memory holds with two stages each, up to
// twelve (three per scheduler, 168 registers a thread); then as many stages as fit, up to 6.
template <int KF, int VF, typename T>
struct BatchCfg {
  using L = SingleTileLayout<KF, VF>;
  static constexpr int kRowsPad = 8;
  static constexpr int kTileBytes = L::kBytes;
  static constexpr int kQBytes = BatchParts<T>::kQ * 8 * 32 * 16;  // the query's B fragments (load_qfrag)
  static constexpr int kFixed = kQBytes + 256;                     // and a tile's lifted value scales
  static constexpr int kFit = kBatchRoom / (kFixed + 2 * kTileBytes);
  static constexpr int kGroups = kFit < 12 ? kFit : 12;
  static constexpr int kStagesFit = (kBatchRoom / kGroups - kFixed) / kTileBytes;
  static constexpr int kStages = kStagesFit < 6 ? kStagesFit : 6;
  static constexpr int kWarps = kGroups;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kGroupBytes = kStages * kTileBytes + kFixed;
  static constexpr int kMetaOff = kGroups * kGroupBytes;
  static constexpr int kSmemBytes = kMetaOff + kBatchMeta;
  static_assert(kStages >= 2 && kMetaOff <= kBatchRoom && kGroupBytes % 16 == 0, "shared memory");
  static_assert(kWarps * kStages * 4 + sizeof(BatchPlanState<kWarps, kGroups>) <= kBatchMeta, "meta");
  // What a unit costs beside its tiles, and the least a group takes, in tiles (both measured with P in one
  // f16 part).  Units: 32 ragged sequences in 41.3 us with 2, 38.8 with 4.  Shares: 1 x 4,096 tokens in 17.1 us with 4, 15.0 with 2
  // (128 groups of two tiles and a merge of 128 parts).
  static constexpr int kUnitCost = 4, kMinShare = 2;
};

constexpr uint32_t kBlind = 1u << 31;  // some row sees a value of the tile that is not finite

// The wide kernel's state of a unit, per group: rows in order.
template <int NR>
struct alignas(16) WideState {
  float crow[8 * NR];
  int qpos[8 * NR];
  float top[4][8 * NR], sum[4][8 * NR];  // of each warp
  uint32_t most[4];                      // the largest scale of each warp's tile (and kBlind)
  uint32_t blind[4][8 * NR];             // blind_blocks of each warp's tile
  uint2 qsums[NR][32];                   // zero-point keys: block sums as B fragments
};

template <int KF, int VF, int NR, typename T>
struct WideCfg {
  using L = SingleTileLayout<KF, VF>;
  static constexpr int kRowsPad = 8 * NR;
  static constexpr int kTileBytes = L::kBytes;
  static constexpr int kPFragBytes = 16;
  static constexpr int kQTileBytes = BatchParts<T>::kQ * 8 * 32 * 16;  // of one n-tile
  static constexpr int kPTileBytes = NR * 32 * kPFragBytes;   // of one tile of tokens
  static constexpr int kFixed = NR * kQTileBytes + 4 * kPTileBytes + sizeof(WideState<NR>);
  static constexpr int kStepBytes = 4 * kTileBytes;
  static constexpr int kFit = kBatchRoom / (kFixed + 2 * kStepBytes);
  static constexpr int kGroups = kFit < 3 ? kFit : 3;
  static constexpr int kStagesFit = (kBatchRoom / kGroups - kFixed) / kStepBytes;
  static constexpr int kStages = kStagesFit < 4 ? kStagesFit : 4;
  static constexpr int kWarps = 4 * kGroups;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kGroupBytes = kStages * kStepBytes + kFixed;
  static constexpr int kMetaOff = kGroups * kGroupBytes;
  static constexpr int kSmemBytes = kMetaOff + kBatchMeta;
  static_assert(kGroups >= 1 && kStages >= 2 && kMetaOff <= kBatchRoom && kGroupBytes % 16 == 0, "shared memory");
  static_assert(kWarps * kStages * 4 + sizeof(BatchPlanState<kWarps, kGroups>) <= kBatchMeta, "meta");
  // With P in one f16 part: 48 windowed sequences in 38.2, 35.6 and 37.8 us with (3, 4), (6, 8) and (10,
  // 16), eight verify steps in 65.5, 63.5 and 62.2.  With 7 a unit of one tile fills a share: 16 sequences of
  // one to four tokens in 14.5 us, with 8 (two units in some groups) in 21.2
  static constexpr int kUnitCost = 6, kMinShare = 7;
};

__device__ __forceinline__ int lds_int(const int* p) { return static_cast<int>(lds32(smem_u32(p))); }

__device__ __forceinline__ int seq_first_tile(const BatchDecodeParams& p, const BatchSeq& q) {
  return p.window > 0 && !p.page_logical && !p.n_list ? max(0, q.pos0 - p.window + 1) / 16 : 0;
}

// Tiles of one unit of a sequence.  A unit with rows always has one at least (it then has
// something that writes its rows), which may have no page behind it.
__device__ __forceinline__ int unit_tiles(const BatchDecodeParams& p, const BatchSeq& q, long long unit) {
  if (q.rows == 0) return 0;
  if (p.n_list) return max(1, 8 * min(max(__ldcg(p.n_list + unit), 0), p.b.max_blocks));
  if (p.page_logical) return max(1, 8 * p.b.max_blocks);
  return (q.pos0 + q.rows - 1) / 16 + 1 - seq_first_tile(p, q);
}

__device__ __forceinline__ BatchSeq load_decode_seq(const BatchDecodeParams& p, int s) {
  return load_seq(p.b, s, !p.page_logical && !p.n_list);
}

__device__ __forceinline__ BatchUnit load_unit(const BatchDecodeParams& p, int u) {
  BatchUnit w;
  w.unit = u;
  const int s = u / p.b.n_kv;
  w.h = u - s * p.b.n_kv;
  const BatchSeq q = load_decode_seq(p, s);
  w.r0 = q.r0;
  w.rows = q.rows;
  w.pos0 = q.pos0;
  w.t0 = seq_first_tile(p, q);
  w.n = unit_tiles(p, q, u);
  return w;
}

// The next unit that has tiles.  Only called where there is one: a later tile of the CTA's belongs to it.
__device__ __forceinline__ BatchUnit next_unit(const BatchDecodeParams& p, int u) {
  while (true) {
    const BatchUnit w = load_unit(p, ++u);
    if (w.n > 0) return w;
    u = (u / p.b.n_kv + 1) * p.b.n_kv - 1;  // a sequence without rows: none of its heads has any
  }
}

__device__ __forceinline__ const uint8_t* lds_ptr(const uint8_t* const* p) {
  unsigned long long v;
  asm volatile("ld.shared.u64 %0, [%1];" : "=l"(v) : "r"(smem_u32(p)));
  return reinterpret_cast<const uint8_t*>(v);
}

__device__ __forceinline__ void cp16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// The groups' stretches of the line of all units, into shared memory; false: the CTA has none.
template <typename C>
__device__ __forceinline__ bool plan_stretches(const BatchDecodeParams& p, BatchPlanState<C::kWarps, C::kGroups>* plan) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (p.b.n_seqs + C::kThreads - 1) / C::kThreads;
  const int s0 = min(static_cast<int>(threadIdx.x) * per, p.b.n_seqs), s1 = min(s0 + per, p.b.n_seqs);
  int tiles = 0, units = 0;  // of this thread's sequences (the host keeps the whole line below 2^31)
  BatchSeq seq{};            // the last of them (the only one, with few sequences)
  int n_seq = 0;             // its tiles per unit, without n_list
  for (int s = s0; s < s1; ++s) {
    seq = load_decode_seq(p, s);
    if (seq.rows == 0) continue;
    units += p.b.n_kv;
    if (p.n_list) {
      for (int h = 0; h < p.b.n_kv; ++h) tiles += unit_tiles(p, seq, static_cast<long long>(s) * p.b.n_kv + h);
    } else {
      n_seq = unit_tiles(p, seq, 0);
      tiles += p.b.n_kv * n_seq;
    }
  }
  int t_end = tiles, u_end = units;  // inclusive sums over the warp, then the block
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, t_end, d), b = __shfl_up_sync(0xffffffffu, u_end, d);
    if (lane >= d) t_end += a, u_end += b;
  }
  if (lane == 31) plan->tiles[warp] = t_end, plan->units[warp] = u_end;
  __syncthreads();
  int t_all = 0, u_all = 0;
#pragma unroll
  for (int w = 0; w < C::kWarps; ++w) {
    if (w < warp) t_end += plan->tiles[w], u_end += plan->units[w];
    t_all += plan->tiles[w], u_all += plan->units[w];
  }
  const int all = t_all + C::kUnitCost * u_all, takers = static_cast<int>(gridDim.x) * C::kGroups;
  const int share = max((all + takers - 1) / takers, C::kMinShare);
  // Stretch i gridDim.x + blockIdx.x is group i's: the first ones go to different SMs.
  const int stride = share * static_cast<int>(gridDim.x), base = share * static_cast<int>(blockIdx.x);
  if (base >= all) return false;
  if (threadIdx.x < C::kGroups) {
    const long long from = base + static_cast<long long>(threadIdx.x) * stride;
    if (from >= all) plan->from[threadIdx.x] = t_all;
    if (from + share >= all) plan->to[threadIdx.x] = t_all;
  }
  // Every end belongs to the thread whose sequences hold it: end e (0: a stretch's start, 1: its
  // end) of group i sits at base + e share + i stride.
  int at = t_end + C::kUnitCost * u_end - tiles - C::kUnitCost * units, before = t_end - tiles;
  for (int s = s0; s < s1 && units > 0; ++s) {
    if (per > 1) {
      seq = load_decode_seq(p, s);
      if (seq.rows == 0) continue;
      if (!p.n_list) n_seq = unit_tiles(p, seq, 0);
    }
    // units of one length are passed in one go, units with lists one by one
    const int step = p.n_list ? 1 : p.b.n_kv;
    for (int h0 = 0; h0 < p.b.n_kv; h0 += step) {
      const int n = p.n_list ? unit_tiles(p, seq, static_cast<long long>(s) * p.b.n_kv + h0) : n_seq;
      const int len = C::kUnitCost + n, end = at + step * len;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int off = base + e * share;
        int i = at <= off ? 0 : (at - off + stride - 1) / stride;  // the group's first end not before `at`
        for (; i < C::kGroups && off + static_cast<long long>(i) * stride < end; ++i) {
          const int in = off + i * stride - at, hh = in / len, skip = max(in - hh * len - C::kUnitCost, 0);
          if (e == 1) {
            plan->to[i] = before + hh * n + skip;
          } else {
            const int h = h0 + hh;
            plan->from[i] = before + hh * n + skip;
            plan->skip[i] = skip;
            plan->unit[i] =
                BatchUnit{s * p.b.n_kv + h, h, seq.r0, seq.rows, seq.pos0, seq_first_tile(p, seq), n};
          }
        }
      }
      at = end;
      before += step * n;
    }
  }
  __syncthreads();
  return true;
}

__device__ __forceinline__ void sts128(uint32_t to, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// The fragments that query_fragments stored for block bl.
template <int QP>
__device__ __forceinline__ void load_qfrag(uint32_t q_s, int bl, int lane, uint4 (&f)[2]) {
  if constexpr (QP == 2) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) f[ks] = lds128(q_s + ((bl * 2 + ks) * 32 + lane) * 16);
  } else {
    const uint4 v = lds128(q_s + (bl * 32 + lane) * 16);
    f[0] = make_uint4(v.x, v.y, 0u, 0u);
    f[1] = make_uint4(v.z, v.w, 0u, 0u);
  }
}

// The B fragments of query rows 8 nt .. + 7 of the unit, to shared memory (one warp).  A row is scaled by
// the power of two that puts its largest magnitude into [2^kTop, 2^(kTop + 1)), and split into f16 parts.
// Returns what turns a dot product with scaled row g into a base-2 score; zero-point keys: the
// rows' block sums as a B fragment.  `between` runs while the rows are on their way.
template <typename T, int QP, bool KMIN, typename Between>
__device__ __forceinline__ float query_fragments(const BatchDecodeParams& p, const BatchUnit& un, int nt, int lane,
                                                 uint32_t q_s, uint32_t& qsb_hi, uint32_t& qsb_lo, Between between) {
  const int g = lane >> 2, t = lane & 3;
  const int r = nt * 8 + g;
  Raw8<T> raw[kBlocks];
  const bool live = r < un.rows * p.group;
  if (live) {
    const int qi = r / p.group, jj = r - qi * p.group;
    const long long at = (un.r0 + qi) * p.q.row_stride + (un.h * p.group + jj) * p.q.head_stride;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) raw[b] = load_raw8<T>(p.q.data, at + 32 * b + 8 * t);
  }
  between();
  float x[kBlocks][8];
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) {
    if (live) {
      widen8<T>(raw[b], x[b]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[b][e] = 0.f;
    }
  }
  float amax = 0.f;
#pragma unroll
  for (int b = 0; b < kBlocks; ++b)
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[b][e]));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  // 2^e <= amax < 2^(e+1), kept where both 2^(e - kTop) and 2^(kTop - e) are normal numbers
  constexpr int kTop = BatchParts<T>::kTop;
  const int ex = min(max(static_cast<int>(__float_as_uint(amax) >> 23), kTop + 1), 254);
  const float inv = __uint_as_float(static_cast<uint32_t>(254 + kTop - ex) << 23);
  float qs0 = 0.f, qs1 = 0.f;
#pragma unroll
  for (int bl = 0; bl < kBlocks; ++bl) {
    float xv[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) xv[e] = x[bl][e] * inv;
    uint32_t hi[2][2], lo[2][2];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      split_pair(xv[4 * ks], xv[4 * ks + 1], hi[ks][0], lo[ks][0]);
      split_pair(xv[4 * ks + 2], xv[4 * ks + 3], hi[ks][1], lo[ks][1]);
    }
    // 16 bytes a lane: a k-step's high and low parts, or with one part both k-steps'
    if constexpr (QP == 2) {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) sts128(q_s + ((bl * 2 + ks) * 32 + lane) * 16, hi[ks][0], hi[ks][1], lo[ks][0], lo[ks][1]);
    } else {
      sts128(q_s + (bl * 32 + lane) * 16, hi[0][0], hi[0][1], hi[1][0], hi[1][1]);
    }
    if constexpr (KMIN) {
      float sm = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sm += xv[e];
      sm *= 1.f / (1 << BatchParts<T>::kSum);
      sm += __shfl_xor_sync(0xffffffffu, sm, 1);
      sm += __shfl_xor_sync(0xffffffffu, sm, 2);
      if (bl == 2 * t) qs0 = sm;
      if (bl == 2 * t + 1) qs1 = sm;
    }
  }
  if constexpr (KMIN) {
    // the remainders are 2^11 below at least: as much higher they fit f16 too
    qsb_hi = pack_half2(qs0, qs1);
    qsb_lo = pack_half2((qs0 - half_lo(qsb_hi)) * 2048.f, (qs1 - half_hi(qsb_hi)) * 2048.f);
  }
  return __uint_as_float(static_cast<uint32_t>(ex - kTop) << 23) * (1.0f / 16.0f) * 1.4426950408889634f;
}

// Entry i of unit u's list: page and logical block (-1: no such entry).
__device__ __forceinline__ int2 page_of(const BatchDecodeParams& p, int u, int i) {
  const long long at = static_cast<long long>(u) * p.b.max_blocks + i;
  const bool any = i < p.b.max_blocks && (!p.n_list || i < p.n_list[u]);
  return make_int2(any ? p.b.page_table[at] : 0, !any ? -1 : p.page_logical ? p.page_logical[at] : i);
}

// Makes w the unit of the warp's copying, its first tile at `start`.
__device__ __forceinline__ void producer_unit(const BatchDecodeParams& p, Producer* prod, const BatchUnit& w, int start,
                                              int lane) {
  if (lane == 0) {
    prod->unit = w.unit;
    prod->start = start;
    prod->t0 = w.t0;
    prod->n = w.n;
    prod->last = w.pos0 + w.rows - 1;
    prod->low = p.window > 0 ? max(0, w.pos0 - p.window + 1) : 0;
  }
  __syncwarp();
}

// Whether block e.y with page id e.x holds a key that some row sees (a bad id of such a block is recorded).
__device__ __forceinline__ bool fetch_block(const BatchDecodeParams& p, int2 e, int last, int low, int lane) {
  if (e.y < 0 || e.y > last / kPageTokens || e.y < low / kPageTokens) return false;
  if (e.x >= 0 && e.x < p.b.n_pages) return true;
  if (lane == 0) record_error(KVATTN_ERR_BAD_PAGE);
  return false;
}

// Starts the copies of tile G of a page into a stage's tile (one warp, 16 bytes a lane).
template <int KF, int VF>
__device__ __forceinline__ void copy_tile(uint32_t to, const uint8_t* k_page, const uint8_t* v_page, int G, int lane) {
  using F = TileFormat<KF, VF>;
  using L = SingleTileLayout<KF, VF>;
  to += 16 * lane;
  k_page += 16 * lane;
  v_page += 16 * lane;
  const uint8_t* src = k_page + G * L::kKCodes;
#pragma unroll
  for (int i = 0; i < L::kKCodes; i += 512) cp16(to + i, src + i);
  if constexpr (F::kK5) cp16(to + L::kKHigh, k_page + kK5HighOffset + G * 512);
  src = v_page + G * L::kVCodes;
#pragma unroll
  for (int i = 0; i < L::kVCodes; i += 512) cp16(to + L::kV + i, src + i);
  // 256 bytes each: lanes 0-15 the K scales, 16-31 the V scales, then 0-15 the minima
  const uint8_t* narrow = lane < 16 ? k_page + F::kKScaleOff : v_page + (F::kVScaleOff - 256);
  cp16(to + L::kSmall, narrow + G * 256);
  if constexpr (F::kKMin || F::kVMin) {
    const uint8_t* low = F::kKMin ? k_page + kK5MinOffset : v_page + kV41MinOffset;
    if (lane < 16) cp16(to + L::kSmall + 512, low + G * 256);
  }
}

// ---- up to 8 query rows: one warp per group
template <int KF, int VF, typename T>
__global__ void __launch_bounds__(BatchCfg<KF, VF, T>::kThreads, 1) decode_batch_kernel(const BatchDecodeParams p) {
  using C = BatchCfg<KF, VF, T>;
  using F = TileFormat<KF, VF>;
  using L = SingleTileLayout<KF, VF>;
  constexpr int QP = BatchParts<T>::kQ, QSUM = BatchParts<T>::kSum;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int grp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  auto* plan = reinterpret_cast<BatchPlanState<C::kWarps, C::kGroups>*>(smem + C::kMetaOff);
  // first position of the tile in each of the warp's stages, -1: none
  int* key_of = reinterpret_cast<int*>(plan + 1) + grp * C::kStages;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  // only now, so that the merge grid may read the batch's arrays before this grid is done
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (!plan_stretches<C>(p, plan)) return;
  const int n_tiles = plan->to[grp] - plan->from[grp];
  if (n_tiles <= 0) return;

  // ---- the group's ring: its tile k goes to stage k % kStages
  uint8_t* ring = smem + grp * C::kGroupBytes;
  const uint32_t ring_s = smem_u32(ring), q_s = ring_s + C::kStages * C::kTileBytes;
  Producer* prod = &plan->producer[grp];

  // makes entry `e` the page at hand
  auto open_page = [&](int2 e) {
    const bool fetch = fetch_block(p, e, lds_int(&prod->last), lds_int(&prod->low), lane);
    __syncwarp();  // every lane has read the page before (the ring is filled without a barrier between tiles)
    if (lane == 0) {
      prod->key0 = fetch ? e.y * kPageTokens : -1;
      prod->k = p.b.k_pool + e.x * p.b.k_stride;  // used only when fetched
      prod->v = p.b.v_pool + e.x * p.b.v_stride;
    }
    __syncwarp();
  };
  int2 ahead = make_int2(0, -1);  // the entry after the page at hand, loaded when that was opened
  // starts the copies of tile k; one group of copies per call, an empty one past the end
  auto issue = [&](int k) {
    if (k < n_tiles) {
      const uint4 cur = lds128(smem_u32(&prod->unit));  // unit, start, t0, n
      int u = cur.x, start = cur.y;
      int end = start + static_cast<int>(cur.w);
      int j = static_cast<int>(cur.z) + k - start;  // the tile in the unit's list
      if (k >= end) {
        __syncwarp();
        const BatchUnit w = next_unit(p, u);
        producer_unit(p, prod, w, end, lane);
        u = w.unit;
        start = end;
        end += w.n;
        j = w.t0;
        ahead = page_of(p, u, j >> 3);
      }
      const int G = j & 7;
      if (k > 0 && (G == 0 || k == start)) {
        open_page(ahead);
        if (k + 8 - G < end) ahead = page_of(p, u, (j >> 3) + 1);
      }
      const uint4 seen = lds128(smem_u32(&prod->last));  // last, low, key0
      const int key0 = seen.z, key = key0 + 16 * G, st = k % C::kStages;
      const bool fetch = key0 >= 0 && key <= static_cast<int>(seen.x) && key + 15 >= static_cast<int>(seen.y);
      if (lane == 0) *reinterpret_cast<volatile int*>(&key_of[st]) = fetch ? key : -1;
      if (fetch) copy_tile<KF, VF>(ring_s + st * C::kTileBytes, lds_ptr(&prod->k), lds_ptr(&prod->v), G, lane);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  BatchUnit* mine = &plan->at_work[grp];
  int start = -plan->skip[grp];  // first tile of the unit, in the group's numbering
  int k = 0;                     // tiles this group has consumed
  if (lane == 0) *mine = plan->unit[grp];
  __syncwarp();
  producer_unit(p, prod, *mine, start, lane);

  while (true) {
    const BatchUnit un = *mine;
    const int end = min(start + un.n, n_tiles);  // the group's tiles of the unit: [k, end)

    float crow[2];
    uint32_t qsb_hi = 0u, qsb_lo = 0u;
    {
      // every load before any use: the first two pages, then the query rows
      int2 here = make_int2(0, -1);
      if (k == 0) {
        const int i = (un.t0 - start) >> 3;
        here = page_of(p, un.unit, i);
        ahead = page_of(p, un.unit, i + 1);
      }
      const float cr = query_fragments<T, QP, F::kKMin>(p, un, 0, lane, q_s, qsb_hi, qsb_lo, [&]() {
        if (k == 0) {
          open_page(here);
          for (int i = 0; i < C::kStages; ++i) issue(i);
        }
      });
      crow[0] = __shfl_sync(0xffffffffu, cr, (2 * t) * 4);
      crow[1] = __shfl_sync(0xffffffffu, cr, (2 * t + 1) * 4);
    }
    __syncwarp();
    // a fragment is read by the lane that wrote it
    auto qfrag = [&](int bl, uint4 (&f)[2]) { load_qfrag<QP>(q_s, bl, lane, f); };

    // ---- the tiles
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
    float oacc[2 * kTileBlocks][4], racc[4] = {0.f, 0.f, 0.f, 0.f};
    ValueScale vs;
#pragma unroll
    for (int i = 0; i < 2 * kTileBlocks; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) oacc[i][e] = 0.f;
    // positions of the thread's two rows (rows past the last take the last's: never stored)
    int qpos[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) qpos[c] = un.pos0 + min((2 * t + c) / p.group, un.rows - 1);
    const int last = un.pos0 + un.rows - 1;
    const int span = p.window > 0 ? p.window : INT_MAX;
    for (; k < end; ++k) {
      const int st = k % C::kStages;
      asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 1) : "memory");
      __syncwarp();
      const int key = *reinterpret_cast<volatile int*>(&key_of[st]);
      if (key >= 0) {
        const uint32_t kb = ring_s + st * C::kTileBytes;
        const bool need_mask = key + 15 > un.pos0 || key <= last - span;
        attend_tile<L, KF, VF, QP, QSUM, BatchParts<T>::kSums, true>(
            kb, kb + L::kV, q_s + C::kQBytes, 0, g, t, qfrag, qsb_hi, qsb_lo, crow,
            [&](int e, float x) {
              const int at = key + g + 8 * (e >> 1);
              return need_mask && (at > qpos[e & 1] || at <= qpos[e & 1] - span) ? -INFINITY : x;
            },
            vs, m_run, l_run, oacc, racc);
      }
      __syncwarp();
      issue(k + C::kStages);
    }

    // ---- rows 2t, 2t + 1, dims 16 i + g, + 8
    float unit = vs.unit();  // of oacc
    if constexpr (F::kVMin) {
      // zero-point values: the minimum terms of block b for rows 2t, 2t + 1 sit in lane 4b + t
#pragma unroll
      for (int b = 0; b < kTileBlocks; ++b)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float v = __shfl_sync(0xffffffffu, racc[c], 4 * b + t);
#pragma unroll
          for (int hb = 0; hb < 2; ++hb) {
            oacc[2 * b + hb][c] = fmaf(oacc[2 * b + hb][c], unit, v);
            oacc[2 * b + hb][c + 2] = fmaf(oacc[2 * b + hb][c + 2], unit, v);
          }
        }
      unit = 1.f;
    }
    BatchUnit w;  // the unit again
    w.unit = lds_int(&mine->unit);
    w.h = lds_int(&mine->h);
    w.r0 = lds_int(&mine->r0);
    w.n = lds_int(&mine->n);
    const int n_rows = lds_int(&mine->rows) * p.group;
    const bool whole = start >= 0 && start + w.n <= n_tiles;
    const int slot = (grp * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x)) * 2 + (start <= 0 ? 0 : 1);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float l = l_run[c];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      // a row that saw no key: l = 0 (a NaN stays one)
      const float inv = l == 0.f ? 0.f : unit / l;
      const float lse2 = l == 0.f ? -INFINITY : m_run[c] + log2f(l);
      const int row = 2 * t + c;
      if (row >= n_rows) continue;
      if (whole) {
        const int qi = row / p.group, hq = w.h * p.group + row - qi * p.group;
        T* to = static_cast<T*>(p.out.data) + (w.r0 + qi) * p.out.row_stride + hq * p.out.head_stride + g;
#pragma unroll
        for (int i = 0; i < 2 * kTileBlocks; ++i) {
          to[16 * i] = static_cast<T>(oacc[i][c] * inv);
          to[16 * i + 8] = static_cast<T>(oacc[i][c + 2] * inv);
        }
        if (g == 0)
          p.lse[static_cast<long long>(w.r0 + qi) * (p.b.n_kv * p.group) + hq] = lse2 * 0.69314718055994531f;
      } else {
        const long long at = static_cast<long long>(slot) * C::kRowsPad + row;
        float* to = p.part_o + at * kHeadDim + g;
#pragma unroll
        for (int i = 0; i < 2 * kTileBlocks; ++i) {
          to[16 * i] = oacc[i][c] * inv;
          to[16 * i + 8] = oacc[i][c + 2] * inv;
        }
        if (g == 0) p.part_lse[at] = lse2;
      }
    }
    if (lane == 0) {
      int2* parts = p.unit_parts + w.unit;
      if (start >= 0) parts->x = slot;
      if (start + w.n <= n_tiles) parts->y = slot >> 1;
    }
    if (k == n_tiles) break;
    start = k;
    const BatchUnit nx = next_unit(p, w.unit);
    __syncwarp();  // every lane has read the unit and its fragments
    if (lane == 0) *mine = nx;
    __syncwarp();
  }
}

// ---- 9 to 24 query rows: four warps per group.  A step is up to four tiles of a unit.  Warp w takes
// the scores of tile w for all NR n-tiles of rows; the four agree on the rows' running maxima (a
// barrier that also votes: mostly none moves); each puts its P into shared memory as B fragments;
// behind a second barrier warp w adds channels 64 w .. + 63 of all four tiles' values.
template <int KF, int VF, int NR, typename T>
__global__ void __launch_bounds__(WideCfg<KF, VF, NR, T>::kThreads, 1)
    decode_batch_wide_kernel(const BatchDecodeParams p) {
  using C = WideCfg<KF, VF, NR, T>;
  using F = TileFormat<KF, VF>;
  using L = SingleTileLayout<KF, VF>;
  constexpr int QP = BatchParts<T>::kQ, QSUM = BatchParts<T>::kSum;
  constexpr bool SUM = BatchParts<T>::kSums;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int grp = warp >> 2, w = warp & 3;
  auto* plan = reinterpret_cast<BatchPlanState<C::kWarps, C::kGroups>*>(smem + C::kMetaOff);
  // [kStages][4]: first position of each tile of the group's steps, -1: none
  int* key_of = reinterpret_cast<int*>(plan + 1) + grp * 4 * C::kStages;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  // only now, so that the merge grid may read the batch's arrays before this grid is done
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!plan_stretches<C>(p, plan)) return;
  const int n_tiles = plan->to[grp] - plan->from[grp];
  if (n_tiles <= 0) return;  // the whole group

  uint8_t* ring = smem + grp * C::kGroupBytes;
  const uint32_t ring_s = smem_u32(ring), q_s = ring_s + C::kStages * C::kStepBytes;
  const uint32_t p_s = q_s + NR * C::kQTileBytes;
  auto* state = reinterpret_cast<WideState<NR>*>(ring + C::kGroupBytes - sizeof(WideState<NR>));
  Producer* prod = &plan->producer[warp];
  auto group_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(grp + 1) : "memory"); };

  int2 ahead = make_int2(0, -1);  // this warp's entry of the next step to be copied, loaded a step ahead
  // starts the copies of this warp's tile of the next step into stage st, and moves on
  auto issue = [&](int st) {
    const uint4 seen = lds128(smem_u32(&prod->last));  // last, low, -, next
    const int k0 = seen.w;
    if (k0 < n_tiles) {
      const uint4 cur = lds128(smem_u32(&prod->unit));  // unit, start, t0, n
      const int u = cur.x, start = cur.y;
      const int end = min(start + static_cast<int>(cur.w), n_tiles);
      int key = -1;
      if (k0 + w < end) {
        const int last = seen.x, low = seen.y;
        const int G = (static_cast<int>(cur.z) + k0 + w - start) & 7;
        if (fetch_block(p, ahead, last, low, lane)) {
          key = ahead.y * kPageTokens + 16 * G;
          if (key > last || key + 15 < low) key = -1;
        }
        if (key >= 0)
          copy_tile<KF, VF>(ring_s + st * C::kStepBytes + w * C::kTileBytes, p.b.k_pool + ahead.x * p.b.k_stride,
                            p.b.v_pool + ahead.x * p.b.v_stride, G, lane);
      }
      __syncwarp();
      if (lane == 0) *reinterpret_cast<volatile int*>(&key_of[4 * st + w]) = key;
      // the step after it: of this unit, or the first of the next
      int next = k0 + 4, unit = u, unit_start = start, unit_end = end;
      int t0 = cur.z;
      if (next >= end) {
        next = end;
        if (end < n_tiles) {
          const BatchUnit nx = next_unit(p, u);
          producer_unit(p, prod, nx, end, lane);
          unit = nx.unit;
          unit_start = end;
          unit_end = min(end + nx.n, n_tiles);
          t0 = nx.t0;
        }
      }
      if (lane == 0) prod->next = next;
      __syncwarp();
      if (next < n_tiles && next + w < unit_end) ahead = page_of(p, unit, (t0 + next + w - unit_start) >> 3);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  BatchUnit* mine = &plan->at_work[warp];
  int start = -plan->skip[grp];  // first tile of the unit, in the group's numbering
  int k = 0;                     // tiles this group has consumed
  int step = 0;
  if (lane == 0) {
    *mine = plan->unit[grp];
    prod->next = 0;
  }
  __syncwarp();
  producer_unit(p, prod, *mine, start, lane);

  while (true) {
    const BatchUnit un = *mine;
    const int end = min(start + un.n, n_tiles);  // the group's tiles of the unit: [k, end)

    // ---- the query's fragments: warp n those of n-tile n
    {
      if (k == 0 && w < end) ahead = page_of(p, un.unit, (un.t0 + w - start) >> 3);
      auto fill = [&]() {
        if (k == 0)
          for (int i = 0; i < C::kStages - 1; ++i) issue(i);
      };
      if (w < NR) {
        uint32_t qsb_hi = 0u, qsb_lo = 0u;
        const float cr =
            query_fragments<T, QP, F::kKMin>(p, un, w, lane, q_s + w * C::kQTileBytes, qsb_hi, qsb_lo, fill);
        if (t == 0) state->crow[8 * w + g] = cr;
        if constexpr (F::kKMin) state->qsums[w][lane] = make_uint2(qsb_hi, qsb_lo);
      } else {
        fill();
        // positions of the rows (rows past the last take the last's: never stored)
        if (w == 3 && lane < 8 * NR) state->qpos[lane] = un.pos0 + min(lane / p.group, un.rows - 1);
      }
    }
    group_sync();
    float crow[NR][2];
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) crow[n][c] = state->crow[8 * n + 2 * t + c];

    float m_run[NR][2], l_run[NR][2];
    float oacc[4][NR][4], racc[NR][4];  // dims 64 w + 16 i + g (+ 8); zero-point values: all blocks' minimum terms
#pragma unroll
    for (int n = 0; n < NR; ++n) {
#pragma unroll
      for (int c = 0; c < 2; ++c) m_run[n][c] = -INFINITY, l_run[n][c] = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        racc[n][e] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) oacc[i][n][e] = 0.f;
      }
    }
    const int last = un.pos0 + un.rows - 1, pos0 = un.pos0;
    const int span = p.window > 0 ? p.window : INT_MAX;
    ValueScale vs;

    for (; k < end; k += 4, ++step) {
      const int st = step % C::kStages;
      asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 2) : "memory");
      __syncwarp();
      const int key = *reinterpret_cast<volatile int*>(&key_of[4 * st + w]);
      const uint32_t kb = ring_s + st * C::kStepBytes + w * C::kTileBytes;
      const bool live = k + w < end && key >= 0;
      float sv[NR][4];
      TileScales ts;
      ts.d = make_uint2(0u, 0u);
      if (live) {
        ts.load<L, F::kVMin>(kb + L::kV, 0, g, t);
        tile_scores<L, KF, VF, QP, QSUM, NR>(
            kb, 0, g, t,
            [&](int n, int bl, uint4 (&f)[2]) { load_qfrag<QP>(q_s + n * C::kQTileBytes, bl, lane, f); },
            [&](int n) { return state->qsums[n][lane]; }, sv);
        const bool need_mask = key + 15 > pos0 || key <= last - span;
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) sv[n][e] *= crow[n][e & 1];
        if (need_mask) {
#pragma unroll
          for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int at = key + g + 8 * (e >> 1), qpos = state->qpos[8 * n + 2 * t + (e & 1)];
              if (at > qpos || at <= qpos - span) sv[n][e] = -INFINITY;
            }
        }
      } else {
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) sv[n][e] = -INFINITY;
      }
      // ---- the rows' references and the scales' powers of two, as in the one-warp kernel
      uint32_t need = ts.unusual<F::kVMin>(vs);
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) need |= fmaxf(sv[n][c], sv[n][c + 2]) > m_run[n][c] + vs.top;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\t"
          "setp.ne.u32 q, %1, 0;\n\t"
          "bar.red.or.pred p, %2, 128, q;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(need)
          : "r"(need), "r"(grp + 1)
          : "memory");
      // every warp is done with the step before this one: its stage takes the step S - 1 ahead
      issue((step + C::kStages - 1) % C::kStages);
      if (need) {
        bool lo = false, hi = false;
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) lo |= sv[n][c] != -INFINITY, hi |= sv[n][c + 2] != -INFINITY;
        uint32_t most;
        const uint32_t bad = ts.clean(lo, hi, t, &most);
        if (live) ts.store<L, F::kVMin>(kb + L::kV, 0, g, t);  // (behind the next barriers all read them)
        const bool any = __any_sync(0xffffffffu, bad != 0);
        if (lane == 0) state->most[w] = most | (any ? kBlind : 0u);
        if (any) {
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            uint32_t blind[2] = {0u, 0u};
            blind_blocks(bad, sv[n], t, blind);
            if (g == 0) state->blind[w][8 * n + 2 * t] = blind[0], state->blind[w][8 * n + 2 * t + 1] = blind[1];
          }
        }
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float mx = fmaxf(sv[n][c], sv[n][c + 2]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            if (g == 0) state->top[w][8 * n + 2 * t + c] = mx;
          }
        group_sync();
        const uint4 tops = lds128(smem_u32(state->most));
        const uint32_t top4[4] = {tops.x, tops.y, tops.z, tops.w};
        if ((tops.x | tops.y | tops.z | tops.w) & kBlind) {
#pragma unroll 1
          for (int u = 0; u < 4; ++u) {
            if (!(state->most[u] & kBlind)) continue;
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (state->blind[u][8 * n + 2 * t + (e & 1)] >> (8 * w + 4 * (i >> 1)) & 1u) oacc[i][n][e] = NAN;
          }
        }
        uint32_t most_of_all = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) most_of_all = max(most_of_all, top4[u] & ~kBlind);
        const float top = vs.top;
        int dk;
        float ratio;
        vs.raise(most_of_all, &dk, &ratio);
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int row = 8 * n + 2 * t + c;
            const float mx = fmaxf(fmaxf(state->top[0][row], state->top[1][row]),
                                   fmaxf(state->top[2][row], state->top[3][row]));
            const float m = mx > m_run[n][c] + top ? mx + (kGrow - vs.top) : m_run[n][c] + static_cast<float>(dk);
            const float alpha = m == m_run[n][c] ? 1.f : fast_exp2(m_run[n][c] - m);  // 0 when m_run = -inf
            l_run[n][c] *= alpha;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              oacc[i][n][c] *= alpha * ratio;
              oacc[i][n][c + 2] *= alpha * ratio;
            }
            if constexpr (F::kVMin) racc[n][c] *= alpha;
            m_run[n][c] = m;
          }
      }
      // ---- P, as B fragments
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        float pr[4];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float mu = m_run[n][c] == -INFINITY ? 0.f : m_run[n][c];
          pr[c] = fast_exp2(sv[n][c] - mu);
          pr[c + 2] = fast_exp2(sv[n][c + 2] - mu);
          l_run[n][c] += pr[c] + pr[c + 2];
        }
        uint32_t h01, l01, h23, l23;
        split_pair(pr[0], pr[1], h01, l01);
        split_pair(pr[2], pr[3], h23, l23);
        sts128(p_s + w * C::kPTileBytes + (n * 32 + lane) * C::kPFragBytes, movmatrix_t(h01), movmatrix_t(h23),
               movmatrix_t(l01), movmatrix_t(l23));
      }
      group_sync();
      // ---- O^T += V^T P^T for this warp's channels, over the step's tiles
      const uint32_t mul = vs.mul();
      auto add_values = [&](int u) {
        const uint32_t vb = ring_s + st * C::kStepBytes + u * C::kTileBytes + L::kV;
        uint32_t ph[NR][2], pl[NR][2];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          const uint4 v = lds128(p_s + u * C::kPTileBytes + (n * 32 + lane) * C::kPFragBytes);
          ph[n][0] = v.x, ph[n][1] = v.y, pl[n][0] = v.z, pl[n][1] = v.w;
        }
        int e = 0;  // constant in the unrolled code
        tile_value_pair<L, KF, VF>(
            vb, vb + L::kVScale, 0, w, g, t,
            [&](int, const uint32_t (&a0)[4], const uint32_t (&a1)[4], uint32_t d0, uint32_t d1) {
              d0 = hmul2(d0, mul);
              d1 = hmul2(d1, mul);
#pragma unroll
              for (int n = 0; n < NR; ++n) {
                uint32_t bh0, bl0, bh1, bl1;
                split_scaled(ph[n][0], pl[n][0], d0, bh0, bl0);
                split_scaled(ph[n][1], pl[n][1], d1, bh1, bl1);
                mma_parts<SUM>(oacc[2 * e][n], a0[0], a0[1], a0[2], a0[3], bh0, bh1, bl0, bl1);
                mma_parts<SUM>(oacc[2 * e + 1][n], a1[0], a1[1], a1[2], a1[3], bh0, bh1, bl0, bl1);
              }
              ++e;
            });
        if constexpr (F::kVMin) {
          const uint2 m = lds_pair(vb + L::kVMinimum + (t * 8 + g) * 8);
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            mma_parts<SUM>(racc[n], m.x, 0u, m.y, 0u, ph[n][0], ph[n][1], pl[n][0], pl[n][1]);
          }
        }
      };
      int4 keys;  // of the step's tiles
      asm volatile("ld.shared.v4.s32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(keys.x), "=r"(keys.y), "=r"(keys.z), "=r"(keys.w)
                   : "r"(smem_u32(key_of + 4 * st)));
      if (k + 4 <= end && (keys.x | keys.y | keys.z | keys.w) >= 0) {
        // all four are there: their loads and decoding overlap
#pragma unroll
        for (int u = 0; u < 4; ++u) add_values(u);
      } else {
#pragma unroll 1
        for (int u = 0; u < 4 && k + u < end; ++u)
          if (lds_int(&key_of[4 * st + u]) >= 0) add_values(u);
      }
    }
    k = end;

    // ---- rows 8n + 2t (+ 1), dims 64 w + 16 i + g (+ 8)
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float l = l_run[n][c];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (g == 0) state->sum[w][8 * n + 2 * t + c] = l;
      }
    float unit = vs.unit();  // of oacc
    if constexpr (F::kVMin) {
      // the minimum terms of block b for rows 2t, 2t + 1 sit in lane 4b + t
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float v = __shfl_sync(0xffffffffu, racc[n][c], 4 * (2 * w + e) + t);
#pragma unroll
            for (int i = 2 * e; i < 2 * e + 2; ++i) {
              oacc[i][n][c] = fmaf(oacc[i][n][c], unit, v);
              oacc[i][n][c + 2] = fmaf(oacc[i][n][c + 2], unit, v);
            }
          }
      unit = 1.f;
    }
    group_sync();
    BatchUnit wk;  // the unit again
    wk.unit = lds_int(&mine->unit);
    wk.h = lds_int(&mine->h);
    wk.r0 = lds_int(&mine->r0);
    wk.n = lds_int(&mine->n);
    const int n_rows = lds_int(&mine->rows) * p.group;
    const bool whole = start >= 0 && start + wk.n <= n_tiles;
    const int slot = (grp * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x)) * 2 + (start <= 0 ? 0 : 1);
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int row = 8 * n + 2 * t + c;
        if (row >= n_rows) continue;
        const float l = (state->sum[0][row] + state->sum[1][row]) + (state->sum[2][row] + state->sum[3][row]);
        // a row that saw no key: l = 0 (a NaN stays one)
        const float inv = l == 0.f ? 0.f : unit / l;
        const float lse2 = l == 0.f ? -INFINITY : m_run[n][c] + log2f(l);
        if (whole) {
          const int qi = row / p.group, hq = wk.h * p.group + row - qi * p.group;
          T* to = static_cast<T*>(p.out.data) + (wk.r0 + qi) * p.out.row_stride + hq * p.out.head_stride + 64 * w + g;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            to[16 * i] = static_cast<T>(oacc[i][n][c] * inv);
            to[16 * i + 8] = static_cast<T>(oacc[i][n][c + 2] * inv);
          }
          if (w == 0 && g == 0)
            p.lse[static_cast<long long>(wk.r0 + qi) * (p.b.n_kv * p.group) + hq] = lse2 * 0.69314718055994531f;
        } else {
          const long long at = static_cast<long long>(slot) * C::kRowsPad + row;
          float* to = p.part_o + at * kHeadDim + 64 * w + g;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            to[16 * i] = oacc[i][n][c] * inv;
            to[16 * i + 8] = oacc[i][n][c + 2] * inv;
          }
          if (w == 0 && g == 0) p.part_lse[at] = lse2;
        }
      }
    if (w == 0 && lane == 0) {
      int2* parts = p.unit_parts + wk.unit;
      if (start >= 0) parts->x = slot;
      if (start + wk.n <= n_tiles) parts->y = slot >> 1;
    }
    if (k == n_tiles) break;
    start = k;
    const BatchUnit nx = next_unit(p, wk.unit);
    __syncwarp();
    if (lane == 0) *mine = nx;
    group_sync();  // the sums and the fragments, before the next unit's
  }
}

// Merges the partials of the units that more than one group took part in: row blockIdx.y, +
// gridDim.y, ... of unit blockIdx.x.  With few parts a warp takes a row (eight channels a lane, every
// part loaded before any is used); with many the CTA does, its four groups of 64 threads taking
// every fourth part, kMergeAhead loaded ahead (8 with four CTAs per SM, or 16 where the CTAs are few
// and each may have over a hundred parts), combined once through shared memory.
constexpr int kMergeFew = 4;

// The store of a merged row: L = sum of exp2(lse_i - M), 0 where no part saw a key.
__device__ __forceinline__ void store_lse(const BatchDecodeParams& p, const BatchUnit& un, int row, float M, float L) {
  const int qi = row / p.group, hq = un.h * p.group + row - qi * p.group;
  p.lse[static_cast<long long>(un.r0 + qi) * (p.b.n_kv * p.group) + hq] =
      L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

__device__ __forceinline__ long long out_row(const BatchDecodeParams& p, const BatchUnit& un, int row) {
  const int qi = row / p.group, hq = un.h * p.group + row - qi * p.group;
  return (un.r0 + qi) * p.out.row_stride + hq * p.out.head_stride;
}

template <typename T, int kMergeAhead, int kMinBlocks>
__global__ void __launch_bounds__(256, kMinBlocks) merge_batch_kernel(const BatchDecodeParams p, int rows_pad) {
  __shared__ float red_m[4], red_l[4];
  __shared__ float4 red_o[4][kHeadDim / 4];
  const int u = blockIdx.x;
  // the split grid started this one after its own wait: what came before it is there to be read
  const BatchUnit un = load_unit(p, u);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (un.n == 0) return;
  const int2 parts = p.unit_parts[u];
  const int c0 = parts.x >> 1, n_parts = parts.y - c0 + 1;
  if (n_parts == 1) return;  // written by its group
  const int tid = threadIdx.x, n_rows = un.rows * p.group;
  auto part = [&](int i, int row) { return static_cast<long long>(i == 0 ? parts.x : 2 * (c0 + i)) * rows_pad + row; };
  if (n_parts <= kMergeFew) {
    const int lane = tid & 31;
    for (int row = blockIdx.y + gridDim.y * (tid >> 5); row < n_rows; row += 8 * gridDim.y) {
      float v[kMergeFew], x[kMergeFew][8];
#pragma unroll
      for (int i = 0; i < kMergeFew; ++i) {
        v[i] = -INFINITY;
        if (i < n_parts) {
          v[i] = p.part_lse[part(i, row)];
          load8<float>(p.part_o, part(i, row) * kHeadDim + 8 * lane, x[i]);
        }
      }
      float M = -INFINITY, L = 0.f, r[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kMergeFew; ++i) M = fmaxf(M, v[i]);
      const float mu = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int i = 0; i < kMergeFew; ++i) {
        if (i >= n_parts) break;
        const float w = fast_exp2(v[i] - mu);  // 0 for a part that saw no key, NaN for a NaN part
        L += w;
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] += w * x[i][e];
      }
      const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] *= inv;
      store8<T>(p.out.data, out_row(p, un, row) + 8 * lane, r);
      if (lane == 0) store_lse(p, un, row, M, L);
    }
    return;
  }
  const int grp = tid >> 6, d4 = tid & 63;
  for (int row = blockIdx.y; row < n_rows; row += gridDim.y) {
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = grp; i0 < n_parts; i0 += 4 * kMergeAhead) {
      float v[kMergeAhead];
      float4 o[kMergeAhead];
#pragma unroll
      for (int k = 0; k < kMergeAhead; ++k) {
        const int i = i0 + 4 * k;
        v[k] = i < n_parts ? p.part_lse[part(i, row)] : -INFINITY;
        o[k] = i < n_parts ? *reinterpret_cast<const float4*>(p.part_o + part(i, row) * kHeadDim + 4 * d4)
                           : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int k = 0; k < kMergeAhead; ++k) {
        if (v[k] == -INFINITY) continue;  // a part that saw no key
        if (v[k] > m) {
          const float a = fast_exp2(m - v[k]);  // 0 when m = -inf
          l *= a;
          acc.x *= a; acc.y *= a; acc.z *= a; acc.w *= a;
          m = v[k];
        }
        const float w = fast_exp2(v[k] - m);  // a NaN part makes the row NaN
        l += w;
        acc.x += w * o[k].x; acc.y += w * o[k].y; acc.z += w * o[k].z; acc.w += w * o[k].w;
      }
    }
    if (d4 == 0) {
      red_m[grp] = m;
      red_l[grp] = l;
    }
    red_o[grp][d4] = acc;
    __syncthreads();
    if (grp == 0) {
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) M = fmaxf(M, red_m[k]);
      const float mu = M == -INFINITY ? 0.f : M;
      float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float w = fast_exp2(red_m[k] - mu);  // 0 for a group that saw no key
        const float4 o = red_o[k][d4];
        L += w * red_l[k];
        r.x += w * o.x; r.y += w * o.y; r.z += w * o.z; r.w += w * o.w;
      }
      const float inv = L == 0.f ? 0.f : 1.f / L;
      const long long at = out_row(p, un, row) + 4 * d4;
      if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float4*>(static_cast<float*>(p.out.data) + at) =
            make_float4(r.x * inv, r.y * inv, r.z * inv, r.w * inv);
      else
        *reinterpret_cast<uint2*>(static_cast<T*>(p.out.data) + at) =
            make_uint2(pack2<T>(r.x * inv, r.y * inv), pack2<T>(r.z * inv, r.w * inv));
      if (d4 == 0) store_lse(p, un, row, M, L);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------------------
int batch_row_tiles(int rows) { return (rows + 7) / 8; }

// Groups that the split grid can have: the workspace is sized by it.
int batch_group_bound(int sms, int n_tiles8) { return sms * (n_tiles8 == 1 ? 12 : 3); }

template <typename C, typename T>
static cudaError_t launch_batch_t(void (*kernel)(BatchDecodeParams), const BatchDecodeParams& p, int sms,
                                  long long most_tiles, cudaStream_t stream) {
  const long long units = static_cast<long long>(p.b.n_seqs) * p.b.n_kv;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  // every stretch is kMinShare long at least, and the first ones go to different SMs
  const long long stretches = (most_tiles + C::kUnitCost * units) / C::kMinShare + 1;
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(sms, stretches)));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess) return e;
  // as many CTAs per unit as are resident together, between one per row (few units: each may have
  // many parts) and one per eight rows
  const int rows = p.group * p.b.max_rows;
  const long long per_unit = std::max<long long>(8ll * sms / units, (rows + 7) / 8);
  cfg.gridDim = dim3(static_cast<unsigned>(units), static_cast<unsigned>(std::min<long long>(rows, per_unit)));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return units * rows <= sms ? cudaLaunchKernelEx(&cfg, merge_batch_kernel<T, 16, 1>, p, C::kRowsPad)
                             : cudaLaunchKernelEx(&cfg, merge_batch_kernel<T, 8, 4>, p, C::kRowsPad);
}

template <int KF, int VF, typename T>
static cudaError_t launch_batch_rows(const BatchDecodeParams& p, int sms, long long most_tiles, cudaStream_t stream) {
  switch (batch_row_tiles(p.group * p.b.max_rows)) {
    case 1: return launch_batch_t<BatchCfg<KF, VF, T>, T>(decode_batch_kernel<KF, VF, T>, p, sms, most_tiles, stream);
    case 2:
      return launch_batch_t<WideCfg<KF, VF, 2, T>, T>(decode_batch_wide_kernel<KF, VF, 2, T>, p, sms, most_tiles, stream);
    default:
      return launch_batch_t<WideCfg<KF, VF, 3, T>, T>(decode_batch_wide_kernel<KF, VF, 3, T>, p, sms, most_tiles, stream);
  }
}

cudaError_t launch_decode_batch(const BatchDecodeParams& p, int dtype, int k_fmt, int v_fmt, int sms,
                                long long most_tiles, cudaStream_t stream) {
#define KV_LAUNCH(KF, VF)                                                                                 \
  if (k_fmt == KF && v_fmt == VF)                                                                         \
    return dtype == KVATTN_F32   ? launch_batch_rows<KF, VF, float>(p, sms, most_tiles, stream)           \
           : dtype == KVATTN_F16 ? launch_batch_rows<KF, VF, __half>(p, sms, most_tiles, stream)          \
                                 : launch_batch_rows<KF, VF, __nv_bfloat16>(p, sms, most_tiles, stream);
  KVATTN_DECODE_PAIRS(KV_LAUNCH)
#undef KV_LAUNCH
  return cudaErrorInvalidValue;
}

template <int KF, int VF, typename T>
static cudaError_t prepare_batch_t() {
  cudaError_t e = cudaFuncSetAttribute(decode_batch_kernel<KF, VF, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       BatchCfg<KF, VF, T>::kSmemBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(decode_batch_wide_kernel<KF, VF, 2, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             WideCfg<KF, VF, 2, T>::kSmemBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(decode_batch_wide_kernel<KF, VF, 3, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             WideCfg<KF, VF, 3, T>::kSmemBytes);
  return e;
}

cudaError_t prepare_batch_kernels() {
  cudaError_t e;
#define KV_SET1(KF, VF, T) \
  if ((e = prepare_batch_t<KF, VF, T>()) != cudaSuccess) return e;
#define KV_SET(KF, VF) KV_SET1(KF, VF, float) KV_SET1(KF, VF, __half) KV_SET1(KF, VF, __nv_bfloat16)
  KVATTN_DECODE_PAIRS(KV_SET)
#undef KV_SET
#undef KV_SET1
  return cudaSuccess;
}

}  // namespace kvattn
