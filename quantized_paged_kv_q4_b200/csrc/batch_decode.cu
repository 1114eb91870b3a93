// Split-KV flash decode of a ragged batch over its pages (kvattn_decode_batch): several sequences
// of different lengths in one grid ([STREAM] method list: paged decode attention over single
// tokens and verify batches).
//
// A unit is one (sequence, KV head): its query rows (group x rows <= 24) against its 16-token
// tiles.  All units form one line, each as long as its tiles and what a unit costs beside them
// (kUnitCost), and every CTA takes an equal stretch of it, whatever the lengths are: a CTA may
// hold the end of one unit, some whole ones and the start of another.  The stretch is found on
// the device, because the lengths live there: every CTA adds up all sequences (one or a few per
// thread, then a scan) and looks its ends up.
//
// Inside a CTA the warps of a group share each tile, one warp per 8 query rows; the groups take
// the CTA's tiles in turn.  A group streams its own tiles through a ring of stages with bulk
// async copies (one per region of the tile; lane r copies region r), and the ring runs on across
// units, so the next unit's first tiles arrive while the last unit's partial results are merged.
// Two or three CTAs share an SM, so that one CTA's merge and setup hide behind the others'
// arithmetic.  A tile's arithmetic is attend_tile (decode_tile.cuh).
//
// At the end of a unit the groups' states (m, l, o) are merged through shared memory, pairwise,
// in a fixed order.  A unit inside one CTA is written to out at once; otherwise each CTA leaves
// an (o, lse) partial and a second grid merges them.  A CTA has at most two such partials, its
// first unit's and its last's, so the workspace has two slots per CTA.
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
  // workspace: where each unit's partials are (first slot, last CTA), and two partials per CTA
  int2* unit_parts;
  float* part_lse;  // [n_ctas][2][rows_pad], base 2
  float* part_o;    // [n_ctas][2][rows_pad][256]
};

// 16-bit inputs are exact as one f16 part (bf16's 8 bits after scaling by a power of two); fp32
// queries take two.  P keeps two parts unless the output is bf16: one rounding of P and one of
// P x scale to f16 (2^-12 each) are an eighth of the rounding of the store (2^-9).
template <typename T>
struct BatchParts {
  static constexpr int kQ = sizeof(T) == 4 ? 2 : 1;
  static constexpr int kP = std::is_same_v<T, __nv_bfloat16> ? 1 : 2;
};

// One unit: its n tiles start at tile t0 of its list of pages (n = 0: a sequence without rows).
struct BatchUnit {
  int unit, h, r0, rows, pos0, t0, n;
};

// What a group's producer keeps between two tiles, in shared memory (registers are the tile's): the
// unit of the next tile, where that starts in the CTA's numbering, and the positions its rows see.
struct Producer {
  int unit, start, t0, n, last, low;
};

// The CTA's plan and the unit at work, in shared memory.
template <int WARPS>
struct BatchPlanState {
  long long tiles[WARPS], units[WARPS];  // of the warps' sequences
  long long first_tile, end_tile;        // the CTA's tiles on the line of all tiles
  int start;                             // first tile of the first unit, in the CTA's numbering (<= 0)
  int abort;
  BatchUnit unit;
};

template <int KF, int VF, int NT, typename T>
struct BatchCfg {
  using F = TileFormat<KF, VF>;
  using L = SingleTileLayout<KF, VF>;
  static constexpr int kRowsPad = NT * 8;
  static constexpr int kWarps = NT == 3 ? 6 : 4;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kGroups = kWarps / NT;
  static constexpr int kTileBytes = L::kKBytes + L::kVBytes;
  static constexpr int kRegions = F::kKRegions + F::kVRegions;
  // the query's B fragments, and in the same place (never at the same time) the merge slots
  static constexpr int kQFragBytes = BatchParts<T>::kQ == 2 ? 16 : 8;
  static constexpr int kQBytes = 16 * NT * 32 * kQFragBytes;
  static constexpr int kOStride = kHeadDim + 4;       // floats; rows 2t of a quad fall in different banks
  static constexpr int kSlotBytes = 8 * kOStride * 4 + 32 * 16;  // one warp's o, then its (m, l)
  static constexpr int kSlots = kGroups == 4 ? 2 : NT;
  static constexpr int kSharedBytes = kQBytes > kSlots * kSlotBytes ? kQBytes : kSlots * kSlotBytes;
  static constexpr int kMeta = 512;                   // barriers and tags
  static constexpr int budget(int ctas) { return 228 * 1024 / ctas - 1024 - kSharedBytes - kMeta; }
  static constexpr int kStages3 = budget(3) / (kGroups * kTileBytes);
  static constexpr int kCtas = NT < 3 && kStages3 >= 2 ? 3 : 2;  // per SM
  static constexpr int kStagesFit = budget(kCtas) / (kGroups * kTileBytes);
  static constexpr int kStages = kStagesFit < 6 ? kStagesFit : 6;
  static_assert(kStages >= 2, "ring");
  static constexpr int kRingBytes = kGroups * kStages * kTileBytes;
  static constexpr int kSharedOff = kRingBytes;
  static constexpr int kMetaOff = kSharedOff + (kSharedBytes + 15) / 16 * 16;
  static constexpr int kSmemBytes = kMetaOff + kMeta;
  static_assert(kGroups * kStages * (8 + 8 + 4) + sizeof(BatchPlanState<kWarps>) + kGroups * sizeof(Producer) <= kMeta,
                "meta");
  // What a unit costs beside its tiles (setup, merge, output), and the least a CTA takes, in tiles.
  static constexpr int kUnitCost = 6, kMinShare = 8;
};

__device__ __forceinline__ int lds_int(const int* p) { return static_cast<int>(lds32(smem_u32(p))); }

__device__ __forceinline__ int seq_first_tile(const BatchDecodeParams& p, const BatchSeq& q) {
  return p.window > 0 && !p.page_logical && !p.n_list ? max(0, q.pos0 - p.window + 1) / 16 : 0;
}

// Tiles of one unit of a sequence.  A unit with rows always has one at least (it then has
// something that writes its rows), which may have no page behind it.
__device__ __forceinline__ int unit_tiles(const BatchDecodeParams& p, const BatchSeq& q, long long unit) {
  if (q.rows == 0) return 0;
  if (p.n_list) return max(1, 8 * min(max(p.n_list[unit], 0), p.b.max_blocks));
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

// Zeroes the V scales (and minima) of the tokens of a staged tile that lie past the sequence's
// last position: their bytes are whatever the page held, and 0 x NaN would reach the output.
// One lane per (T, block) word of four tokens.
__device__ __noinline__ void blank_tokens(uint8_t* vscale, uint8_t* vmin, int lane, int n_live) {
  const int T = lane >> 3;
  uint32_t keep[2];
#pragma unroll
  for (int w = 0; w < 2; ++w)
    keep[w] = (2 * T + 8 * w < n_live ? 0x0000FFFFu : 0u) | (2 * T + 1 + 8 * w < n_live ? 0xFFFF0000u : 0u);
  uint2* a = reinterpret_cast<uint2*>(vscale) + lane;
  *a = make_uint2(a->x & keep[0], a->y & keep[1]);
  if (vmin) {
    uint2* m = reinterpret_cast<uint2*>(vmin) + lane;
    *m = make_uint2(m->x & keep[0], m->y & keep[1]);
  }
  // the stage is later refilled by the copy engine (async proxy)
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}

template <int KF, int VF, int NT, typename T>
__global__ void __launch_bounds__(BatchCfg<KF, VF, NT, T>::kThreads, BatchCfg<KF, VF, NT, T>::kCtas)
    decode_batch_kernel(const BatchDecodeParams p) {
  using C = BatchCfg<KF, VF, NT, T>;
  using F = TileFormat<KF, VF>;
  using L = SingleTileLayout<KF, VF>;
  constexpr int QP = BatchParts<T>::kQ, PP = BatchParts<T>::kP;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int grp = warp / NT, nt0 = warp % NT;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kMetaOff);   // [kGroups][kStages]
  uint64_t* empty = full + C::kGroups * C::kStages;                   // [kGroups][kStages] (NT > 1)
  int* st_key = reinterpret_cast<int*>(empty + C::kGroups * C::kStages);  // first position of the tile, -1: none
  auto* plan = reinterpret_cast<BatchPlanState<C::kWarps>*>(st_key + C::kGroups * C::kStages);
  Producer* prod = reinterpret_cast<Producer*>(plan + 1) + grp;  // the group's, between two tiles

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kGroups * C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], NT);
    }
    plan->abort = 0;
    fence_barrier_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // only now, so that the merge grid may read the batch's arrays before this grid is done
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- the plan: this CTA's stretch of the line of all units
  {
    const int per = (p.b.n_seqs + C::kThreads - 1) / C::kThreads;
    const int s0 = min(static_cast<int>(threadIdx.x) * per, p.b.n_seqs), s1 = min(s0 + per, p.b.n_seqs);
    long long tiles = 0, units = 0;  // of this thread's sequences
    for (int s = s0; s < s1; ++s) {
      const BatchSeq q = load_decode_seq(p, s);
      if (q.rows == 0) continue;
      const long long u = static_cast<long long>(s) * p.b.n_kv;
      units += p.b.n_kv;
      if (p.n_list)
        for (int h = 0; h < p.b.n_kv; ++h) tiles += unit_tiles(p, q, u + h);
      else
        tiles += static_cast<long long>(p.b.n_kv) * unit_tiles(p, q, u);
    }
    long long t_end = tiles, u_end = units;  // inclusive sums over the warp, then the block
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long a = __shfl_up_sync(0xffffffffu, t_end, d), b = __shfl_up_sync(0xffffffffu, u_end, d);
      if (lane >= d) t_end += a, u_end += b;
    }
    if (lane == 31) plan->tiles[warp] = t_end, plan->units[warp] = u_end;
    __syncthreads();
    long long t_all = 0, u_all = 0;
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w) {
      if (w < warp) t_end += plan->tiles[w], u_end += plan->units[w];
      t_all += plan->tiles[w], u_all += plan->units[w];
    }
    const long long all = t_all + C::kUnitCost * u_all;
    const long long share = max((all + gridDim.x - 1) / gridDim.x, static_cast<long long>(C::kMinShare));
    const long long w0 = share * blockIdx.x, w1 = min(w0 + share, all);
    if (w0 >= all) return;  // past the end of the line
    // the threads whose sequences hold the two ends
    const long long at1 = t_end + C::kUnitCost * u_end, at0 = at1 - tiles - C::kUnitCost * units;
    const bool has0 = w0 >= at0 && w0 < at1, has1 = w1 > at0 && w1 <= at1;
    if (has0 || has1) {
      long long at = at0, before = t_end - tiles;  // where the unit starts, and the tiles before it
      for (int s = s0; s < s1 && at < w1; ++s) {
        const BatchSeq q = load_decode_seq(p, s);
        for (int h = 0; h < p.b.n_kv && q.rows > 0 && at < w1; ++h) {
          const int u = s * p.b.n_kv + h, n = unit_tiles(p, q, u);
          const long long first = at + C::kUnitCost, end = first + n;
          if (has0 && w0 >= at && w0 < end) {
            const int skip = static_cast<int>(max(w0 - first, 0ll));
            plan->first_tile = before + skip;
            plan->start = -skip;
            plan->unit = BatchUnit{u, h, q.r0, q.rows, q.pos0, seq_first_tile(p, q), n};
          }
          if (has1 && w1 > at && w1 <= end) plan->end_tile = before + max(w1 - first, 0ll);
          at = end;
          before += n;
        }
      }
    }
    __syncthreads();
  }
  const int n_tiles = static_cast<int>(plan->end_tile - plan->first_tile);
  if (n_tiles == 0) return;  // nothing but the cost of a unit

  // ---- the group's ring.  Tiles are numbered along the CTA's stretch; group grp takes tiles k with
  // k % kGroups == grp, its j-th being k = grp + j kGroups in stage j % kStages.  The producer is
  // the group's first warp: lane 0 announces a tile, lane r copies region r.
  uint64_t* gfull = full + grp * C::kStages;
  uint64_t* gempty = empty + grp * C::kStages;
  int* gkey = st_key + grp * C::kStages;
  uint8_t* ring = smem + grp * C::kStages * C::kTileBytes;

  // region r of this lane, in units of 256 bytes: where it starts in a page, its bytes per tile, and
  // where it goes in a stage
  uint32_t region = 0;
#pragma unroll
  for (int r = 0; r < F::kKRegions; ++r)
    if (lane == r) region = F::k_reg_off(r) / 256 | F::k_reg_tile(r) / 256 << 8 | L::k_off(r) / 256 << 16;
#pragma unroll
  for (int r = 0; r < F::kVRegions; ++r)
    if (lane == F::kKRegions + r)
      region = F::v_reg_off(r) / 256 | F::v_reg_tile(r) / 256 << 8 | (L::kKBytes + L::v_off(r)) / 256 << 16;

  int p_page = -1, p_block = -1;  // page and logical block of the next tile to issue, loaded a tile ahead
  auto start_unit = [&](const BatchUnit& w, int start) {
    if (lane == 0)
      *prod = Producer{w.unit, start, w.t0, w.n, w.pos0 + w.rows - 1, p.window > 0 ? max(0, w.pos0 - p.window + 1) : 0};
    __syncwarp();
  };
  // page and logical block of tile k of the producer's unit
  auto page_of = [&](int k) -> int2 {
    const int u = lds_int(&prod->unit);
    const int i = (lds_int(&prod->t0) + k - lds_int(&prod->start)) >> 3;
    const long long at = static_cast<long long>(u) * p.b.max_blocks + i;
    const bool any = i < p.b.max_blocks && (!p.n_list || i < p.n_list[u]);
    return make_int2(any ? p.b.page_table[at] : -2, any && p.page_logical ? p.page_logical[at] : i);
  };
  // looks up the page of the group's tile jj (the issue that follows uses it, a tile's arithmetic later)
  auto look_up = [&](int jj) {
    const int k = grp + jj * C::kGroups;
    if (k >= n_tiles) return;
    while (true) {
      const int end = lds_int(&prod->start) + lds_int(&prod->n);
      if (k < end) break;
      const int u = lds_int(&prod->unit);
      __syncwarp();
      start_unit(next_unit(p, u), end);
    }
    const int2 at = page_of(k);
    p_page = at.x;
    p_block = at.y;
  };
  // copies the group's tile jj into its stage
  auto issue = [&](int jj) {
    const int k = grp + jj * C::kGroups;
    if (k >= n_tiles) return;
    const int st = jj % C::kStages;
    const int G = (lds_int(&prod->t0) + k - lds_int(&prod->start)) & 7;
    const int last = lds_int(&prod->last);
    // a tile that no row sees is not fetched
    bool fetch = p_page != -2 && p_block >= 0 && p_block <= last / kPageTokens;
    const int key = fetch ? p_block * kPageTokens + 16 * G : -1;
    fetch = fetch && key <= last && key + 15 >= lds_int(&prod->low);
    if (fetch && (p_page < 0 || p_page >= p.b.n_pages)) {
      if (lane == 0) record_error(KVATTN_ERR_BAD_PAGE);
      fetch = false;
    }
    if (lane == 0) {
      *reinterpret_cast<volatile int*>(&gkey[st]) = fetch ? key : -1;
      if (fetch)
        mbar_arrive_expect_tx(&gfull[st], C::kTileBytes);
      else
        mbar_arrive(&gfull[st]);
    }
    __syncwarp();
    if (fetch && lane < C::kRegions) {
      const uint32_t bytes = (region & 0xFF00u);
      const uint8_t* pool = lane >= F::kKRegions ? p.b.v_pool + p_page * p.b.v_stride : p.b.k_pool + p_page * p.b.k_stride;
      bulk_g2s(ring + st * C::kTileBytes + (region >> 16) * 256, pool + (region & 0xFFu) * 256 + G * bytes, bytes,
               &gfull[st]);
    }
  };
  int j = 0;  // tiles this group has consumed
  int start = plan->start;
  const uint32_t q_s = smem_u32(smem + C::kSharedOff);
  bool ok = true;
  if (nt0 == 0) start_unit(plan->unit, start);

  for (int done = 0; done < n_tiles;) {
    const BatchUnit un = plan->unit;
    const int end = min(start + un.n, n_tiles);  // this CTA's tiles of the unit: [done, end)

    // ---- the query's fragments.  A row is scaled by the power of two that puts its largest
    // magnitude into [1, 2) (exact), and split into f16 parts.
    float crow[2];
    uint32_t qsb_hi = 0u, qsb_lo = 0u;
    {
      // every load before any use: the pages of the ring's first tiles (lane jj the group's tile
      // jj), then the query rows
      int2 ahead = make_int2(-2, 0);
      const int k_ahead = grp + lane * C::kGroups;
      if (done == 0 && nt0 == 0 && lane < C::kStages && k_ahead < end) ahead = page_of(k_ahead);
      const int r = nt0 * 8 + g;
      Raw8<T> raw[kBlocks];
      const bool live = r < un.rows * p.group;
      if (live) {
        const int qi = r / p.group, jj = r - qi * p.group;
        const long long at = (un.r0 + qi) * p.q.row_stride + (un.h * p.group + jj) * p.q.head_stride;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) raw[b] = load_raw8<T>(p.q.data, at + 32 * b + 8 * t);
      }
      if (done == 0 && nt0 == 0) {
        for (int jj = 0; jj < C::kStages; ++jj) {
          p_page = __shfl_sync(0xffffffffu, ahead.x, jj);
          p_block = __shfl_sync(0xffffffffu, ahead.y, jj);
          if (grp + jj * C::kGroups >= end) look_up(jj);  // already another unit's
          issue(jj);
        }
        look_up(C::kStages);
      }
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
      // 2^e <= amax < 2^(e+1), kept where both 2^e and 2^-e are normal numbers
      const int ex = min(max(static_cast<int>(__float_as_uint(amax) >> 23), 1), 253);
      const float inv = __uint_as_float(static_cast<uint32_t>(254 - ex) << 23);
      float qs0 = 0.f, qs1 = 0.f;
#pragma unroll
      for (int bl = 0; bl < kBlocks; ++bl) {
        float xv[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) xv[e] = x[bl][e] * inv;
        if (bl % C::kGroups == grp) {  // the groups hold the same rows: each writes its share
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            uint32_t hi[2], lo[2];
            split_pair(xv[4 * ks], xv[4 * ks + 1], hi[0], lo[0]);
            split_pair(xv[4 * ks + 2], xv[4 * ks + 3], hi[1], lo[1]);
            const uint32_t to = q_s + (((bl * 2 + ks) * NT + nt0) * 32 + lane) * C::kQFragBytes;
            if constexpr (QP == 2)
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(hi[0]), "r"(hi[1]), "r"(lo[0]),
                           "r"(lo[1])
                           : "memory");
            else
              asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(to), "r"(hi[0]), "r"(hi[1]) : "memory");
          }
        }
        if constexpr (F::kKMin) {
          float sm = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) sm += xv[e];
          sm += __shfl_xor_sync(0xffffffffu, sm, 1);
          sm += __shfl_xor_sync(0xffffffffu, sm, 2);
          if (bl == 2 * t) qs0 = sm;
          if (bl == 2 * t + 1) qs1 = sm;
        }
      }
      if constexpr (F::kKMin) split_pair(qs0, qs1, qsb_hi, qsb_lo);
      const float cr = __uint_as_float(static_cast<uint32_t>(ex) << 23) * (1.0f / 16.0f) * 1.4426950408889634f;
      crow[0] = __shfl_sync(0xffffffffu, cr, (2 * t) * 4);
      crow[1] = __shfl_sync(0xffffffffu, cr, (2 * t + 1) * 4);
    }
    __syncthreads();
    auto qfrag = [&](int bl, int ks) -> uint4 {
      const uint32_t from = q_s + (((bl * 2 + ks) * NT + nt0) * 32 + lane) * C::kQFragBytes;
      if constexpr (QP == 2) {
        return lds128(from);
      } else {
        uint2 v;
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(from));
        return make_uint4(v.x, v.y, 0u, 0u);
      }
    };

    // ---- this group's tiles of the unit
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
    float oacc[2 * kTileBlocks][4], racc[4] = {0.f, 0.f, 0.f, 0.f};
    BatchUnit next{};  // the last warp's lane 0: the unit after this one
#pragma unroll
    for (int i = 0; i < 2 * kTileBlocks; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) oacc[i][e] = 0.f;
    // positions of the thread's two rows (rows past the last take the last's: never stored)
    int qpos[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) qpos[c] = un.pos0 + min((nt0 * 8 + 2 * t + c) / p.group, un.rows - 1);
    const int last = un.pos0 + un.rows - 1;
    const int span = p.window > 0 ? p.window : INT_MAX;
    for (; grp + j * C::kGroups < end; ++j) {
      const int st = j % C::kStages;
      const uint32_t par = (j / C::kStages) & 1;
      if (!mbar_wait(&gfull[st], par)) {
        ok = false;
        break;
      }
      const int key = *reinterpret_cast<volatile int*>(&gkey[st]);
      if (key >= 0) {
        uint8_t* tile = ring + st * C::kTileBytes;
        if (key + 15 > last)
          blank_tokens(tile + L::kKBytes + L::kVScale, F::kVMin ? tile + L::kKBytes + L::kVMinimum : nullptr, lane,
                       last - key + 1);
        const bool need_mask = key + 15 > un.pos0 || key <= last - span;
        const uint32_t kb = smem_u32(tile);
        attend_tile<L, KF, VF, QP, PP>(
            kb, kb + L::kKBytes, 0, g, t, qfrag, qsb_hi, qsb_lo, crow, 2.f,
            [&](int e, float x) {
              const int at = key + g + 8 * (e >> 1);
              return need_mask && (at > qpos[e & 1] || at <= qpos[e & 1] - span) ? -INFINITY : x;
            },
            m_run, l_run, oacc, racc);
      }
      __syncwarp();
      if constexpr (NT == 1) {
        issue(j + C::kStages);
        look_up(j + C::kStages + 1);
      } else {
        // the producer refills the stage of the tile before this one: the other warps are done
        // with it, or nearly
        if (lane == 0) mbar_arrive(&gempty[st]);
        if (nt0 == 0 && j > 0) {
          if (!mbar_wait(&gempty[(j - 1) % C::kStages], ((j - 1) / C::kStages) & 1)) {
            ok = false;
            break;
          }
          issue(j - 1 + C::kStages);
          look_up(j + C::kStages);
        }
      }
    }

    // ---- merge the groups' states, pairwise through shared memory
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float l = l_run[c];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      l_run[c] = l;
    }
    if constexpr (F::kVMin) {
      // zero-point values: the minimum terms of block b for rows 2t, 2t + 1 sit in lane 4b + t
#pragma unroll
      for (int b = 0; b < kTileBlocks; ++b)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float v = __shfl_sync(0xffffffffu, racc[c], 4 * b + t);
#pragma unroll
          for (int hb = 0; hb < 2; ++hb) {
            oacc[2 * b + hb][c] += v;
            oacc[2 * b + hb][c + 2] += v;
          }
        }
    }
    if (!ok) *reinterpret_cast<volatile int*>(&plan->abort) = 1;
    float4* slots = reinterpret_cast<float4*>(smem + C::kSharedOff);
    constexpr int kSlot4 = C::kSlotBytes / 16;  // float4s of a slot; (m, l) behind the 16 x 32 of o
#pragma unroll
    for (int half = C::kGroups / 2; half >= 1; half /= 2) {
      __syncthreads();  // the query fragments, or the slots of the round before, are done with
      if (grp >= half && grp < 2 * half) {
        float4* to = slots + ((grp - half) * NT + nt0) * kSlot4 + lane;
#pragma unroll
        for (int i = 0; i < 2 * kTileBlocks; ++i) to[32 * i] = make_float4(oacc[i][0], oacc[i][1], oacc[i][2], oacc[i][3]);
        to[32 * 2 * kTileBlocks] = make_float4(m_run[0], m_run[1], l_run[0], l_run[1]);
        // the last warp, now idle, looks up the next unit and fetches its query rows into L2
        if (warp == C::kWarps - 1 && end < n_tiles) {
          const BatchUnit nx = next_unit(p, un.unit);
          if (lane < nx.rows * p.group) {
            const int qi = lane / p.group;
            const char* row = static_cast<const char*>(p.q.data) +
                              sizeof(T) * ((nx.r0 + qi) * p.q.row_stride +
                                           (nx.h * p.group + lane - qi * p.group) * p.q.head_stride);
#pragma unroll
            for (int b = 0; b < kHeadDim * static_cast<int>(sizeof(T)); b += 128)
              asm volatile("prefetch.global.L2 [%0];" ::"l"(row + b));
          }
          if (lane == 0) next = nx;
        }
      }
      __syncthreads();
      if (grp < half) {
        const float4* from = slots + (grp * NT + nt0) * kSlot4 + lane;
        const float4 ml = from[32 * 2 * kTileBlocks];
        const float om[2] = {ml.x, ml.y}, ol[2] = {ml.z, ml.w};
        float wa[2], wb[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          // a state that saw no key has m = -inf, l = 0 and o = 0: its weight is 0 (and a NaN in l or o stays one)
          const float M = fmaxf(m_run[c], om[c]), mu = M == -INFINITY ? 0.f : M;
          wa[c] = fast_exp2(m_run[c] - mu);
          wb[c] = fast_exp2(om[c] - mu);
          l_run[c] = l_run[c] * wa[c] + ol[c] * wb[c];
          m_run[c] = M;
        }
#pragma unroll
        for (int i = 0; i < 2 * kTileBlocks; ++i) {
          const float4 o = from[32 * i];
          oacc[i][0] = oacc[i][0] * wa[0] + o.x * wb[0];
          oacc[i][1] = oacc[i][1] * wa[1] + o.y * wb[1];
          oacc[i][2] = oacc[i][2] * wa[0] + o.z * wb[0];
          oacc[i][3] = oacc[i][3] * wa[1] + o.w * wb[1];
        }
      }
    }
    __syncthreads();
    if (plan->abort) break;
    if (grp == 0) {
      // rows of 256 through the warp's slot, so that lanes store whole lines
      float* rows = reinterpret_cast<float*>(slots + nt0 * kSlot4);
      float lse2[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float inv = l_run[c] == 0.f ? 0.f : 1.f / l_run[c];
        lse2[c] = l_run[c] == 0.f ? -INFINITY : m_run[c] + log2f(l_run[c]);
#pragma unroll
        for (int i = 0; i < 2 * kTileBlocks; ++i)
#pragma unroll
          for (int hi = 0; hi < 2; ++hi)
            rows[(2 * t + c) * C::kOStride + 16 * i + g + 8 * hi] = oacc[i][c + 2 * hi] * inv;
      }
      __syncwarp();
      const int r0 = lds_int(&plan->unit.r0), n_rows = lds_int(&plan->unit.rows) * p.group;
      const int h = lds_int(&plan->unit.h), unit_n = lds_int(&plan->unit.n);
      const bool whole = start >= 0 && start + unit_n <= n_tiles;
      const int slot = static_cast<int>(blockIdx.x) * 2 + (start <= 0 ? 0 : 1);
      const long long part = static_cast<long long>(slot) * C::kRowsPad;
#pragma unroll 1
      for (int r = 0; r < 8; ++r) {
        const int row = nt0 * 8 + r;
        if (row >= n_rows) break;
        const float* from = rows + r * C::kOStride + 8 * lane;
        const float4 a = *reinterpret_cast<const float4*>(from), b = *reinterpret_cast<const float4*>(from + 4);
        const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        const float l2 = __shfl_sync(0xffffffffu, r & 1 ? lse2[1] : lse2[0], r >> 1);
        if (whole) {
          const int qi = row / p.group, hq = h * p.group + row - qi * p.group;
          store8<T>(p.out.data, (r0 + qi) * p.out.row_stride + hq * p.out.head_stride + 8 * lane, x);
          if (lane == 0)
            p.lse[static_cast<long long>(r0 + qi) * (p.b.n_kv * p.group) + hq] = l2 * 0.69314718055994531f;
        } else {
          store8<float>(p.part_o, (part + row) * kHeadDim + 8 * lane, x);
          if (lane == 0) p.part_lse[part + row] = l2;
        }
      }
      if (threadIdx.x == 0) {
        int2* parts = p.unit_parts + lds_int(&plan->unit.unit);
        if (start >= 0) parts->x = slot;
        if (start + unit_n <= n_tiles) parts->y = static_cast<int>(blockIdx.x);
      }
    }
    done = end;
    start = end;
    __syncthreads();  // the slots and the plan's unit, before the next unit's
    if (done < n_tiles) {
      if (warp == C::kWarps - 1 && lane == 0) plan->unit = next;
      __syncthreads();
    }
  }
  if (plan->abort && nt0 == 0 && lane == 0) {
    // a bounded wait expired: wait (bounded) for the copies still in flight, then leave
    const int issued = min(j + C::kStages, (n_tiles - grp + C::kGroups - 1) / C::kGroups);
    const unsigned long long t0 = global_timer_ns();
    for (int jj = max(0, issued - C::kStages); jj < issued; ++jj)
      while (!mbar_try_wait(&gfull[jj % C::kStages], (jj / C::kStages) & 1))
        if (global_timer_ns() - t0 > kWaitTimeoutNs) break;
  }
}

// Merges the partials of the units that more than one CTA took part in.  One CTA per unit (and
// per row, where there are few units), 256 threads = four groups of 64 (four channels each); a
// group takes every fourth part, loading a batch of them before using any, and the groups are
// combined once through shared memory.
constexpr int kBatchMergeAhead = 8;

template <typename T>
__global__ void __launch_bounds__(256) merge_batch_kernel(const BatchDecodeParams p, int rows_pad) {
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
  if (n_parts == 1) return;  // written by its CTA
  const int tid = threadIdx.x, grp = tid >> 6, d4 = tid & 63;
  for (int row = blockIdx.y; row < un.rows * p.group; row += gridDim.y) {
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = grp; i0 < n_parts; i0 += 4 * kBatchMergeAhead) {
      float v[kBatchMergeAhead];
      float4 o[kBatchMergeAhead];
#pragma unroll
      for (int k = 0; k < kBatchMergeAhead; ++k) {
        const int i = i0 + 4 * k;
        const long long at = static_cast<long long>(i == 0 ? parts.x : 2 * (c0 + i)) * rows_pad + row;
        v[k] = i < n_parts ? p.part_lse[at] : -INFINITY;
        o[k] = i < n_parts ? *reinterpret_cast<const float4*>(p.part_o + at * kHeadDim + 4 * d4)
                           : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int k = 0; k < kBatchMergeAhead; ++k) {
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
      const int qi = row / p.group, hq = un.h * p.group + row - qi * p.group;
      const long long at = (un.r0 + qi) * p.out.row_stride + hq * p.out.head_stride + 4 * d4;
      if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float4*>(static_cast<float*>(p.out.data) + at) =
            make_float4(r.x * inv, r.y * inv, r.z * inv, r.w * inv);
      else
        *reinterpret_cast<uint2*>(static_cast<T*>(p.out.data) + at) =
            make_uint2(pack2<T>(r.x * inv, r.y * inv), pack2<T>(r.z * inv, r.w * inv));
      if (d4 == 0)
        p.lse[static_cast<long long>(un.r0 + qi) * (p.b.n_kv * p.group) + hq] =
            L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------------------
int batch_row_tiles(int rows) { return (rows + 7) / 8; }

// CTAs that the split grid can have: the workspace is sized by it.
int batch_grid_bound(int sms, int n_tiles8) { return sms * (n_tiles8 < 3 ? 3 : 2); }

template <int KF, int VF, int NT, typename T>
static cudaError_t launch_batch_t(const BatchDecodeParams& p, int sms, long long most_tiles, cudaStream_t stream) {
  using C = BatchCfg<KF, VF, NT, T>;
  const long long units = static_cast<long long>(p.b.n_seqs) * p.b.n_kv;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(
      std::min(static_cast<long long>(sms) * C::kCtas, (most_tiles + C::kUnitCost * units) / C::kMinShare + 1)));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, decode_batch_kernel<KF, VF, NT, T>, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(units), units <= 296 ? std::min(p.group * p.b.max_rows, 24) : 1);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, merge_batch_kernel<T>, p, C::kRowsPad);
}

#define KVATTN_BATCH_PAIRS(X)                                                                         \
  X(kKeyQ8, kValQ4) X(kKeyQ8, kValQ8) X(kKeyQ4, kValQ4) X(kKeyQ4, kValQ8) X(kKeyQ51, kValQ4)            \
  X(kKeyQ51, kValQ8) X(kKeyQ50, kValQ41)

template <int KF, int VF, typename T>
static cudaError_t launch_batch_rows(const BatchDecodeParams& p, int sms, long long most_tiles, cudaStream_t stream) {
  switch (batch_row_tiles(p.group * p.b.max_rows)) {
    case 1: return launch_batch_t<KF, VF, 1, T>(p, sms, most_tiles, stream);
    case 2: return launch_batch_t<KF, VF, 2, T>(p, sms, most_tiles, stream);
    default: return launch_batch_t<KF, VF, 3, T>(p, sms, most_tiles, stream);
  }
}

cudaError_t launch_decode_batch(const BatchDecodeParams& p, int dtype, int k_fmt, int v_fmt, int sms,
                                long long most_tiles, cudaStream_t stream) {
#define KV_LAUNCH(KF, VF)                                                                                 \
  if (k_fmt == KF && v_fmt == VF)                                                                         \
    return dtype == KVATTN_F32   ? launch_batch_rows<KF, VF, float>(p, sms, most_tiles, stream)           \
           : dtype == KVATTN_F16 ? launch_batch_rows<KF, VF, __half>(p, sms, most_tiles, stream)          \
                                 : launch_batch_rows<KF, VF, __nv_bfloat16>(p, sms, most_tiles, stream);
  KVATTN_BATCH_PAIRS(KV_LAUNCH)
#undef KV_LAUNCH
  return cudaErrorInvalidValue;
}

template <int KF, int VF, int NT, typename T>
static cudaError_t prepare_batch_t() {
  return cudaFuncSetAttribute(decode_batch_kernel<KF, VF, NT, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              BatchCfg<KF, VF, NT, T>::kSmemBytes);
}

cudaError_t prepare_batch_kernels() {
  cudaError_t e;
#define KV_SET1(KF, VF, NT, T) \
  if ((e = prepare_batch_t<KF, VF, NT, T>()) != cudaSuccess) return e;
#define KV_SET2(KF, VF, T) KV_SET1(KF, VF, 1, T) KV_SET1(KF, VF, 2, T) KV_SET1(KF, VF, 3, T)
#define KV_SET(KF, VF) KV_SET2(KF, VF, float) KV_SET2(KF, VF, __half) KV_SET2(KF, VF, __nv_bfloat16)
  KVATTN_BATCH_PAIRS(KV_SET)
#undef KV_SET
#undef KV_SET2
#undef KV_SET1
  return cudaSuccess;
}

}  // namespace kvattn
