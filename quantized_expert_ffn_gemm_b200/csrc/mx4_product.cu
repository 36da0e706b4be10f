// Product of MXFP4 rows with per-expert MXFP4 weights on the block-scaled tensor cores:
//
//   out[r, n] = sum_k A[r, k] W_g[n, k]   for the rows r of group g, or, with an up matrix,
//   out[r, n] = silu(A W_g^T)[r, n] * (A U_g^T)[r, n]
//
// tcgen05.mma kind::mxf4 multiplies e2m1 codes and applies both operands' block scales itself (one e8m0
// byte for 32 values, read from tensor memory), so the codes go from HBM to shared memory by TMA and from
// there to the MMA untouched; only the scale bytes are rearranged on the way.
//
//   tile    128 weight rows (MMA M, one tensor-memory lane a row: 128 features, or 64 features' gate rows and
//           their up rows) x up to NT = 192 or 96 rows of a group (MMA N, a multiple of 16). A group of 160
//           rows is one tile, so its weights are read once and no MMA works on rows that are not there.
//           (With the rows as M = 128 such a group was two tiles, one a quarter full: 171 us for 8192 tokens
//           over 512 experts, 198 under the power limit, against 156 and 182.)
//   stage   K = 256: 128 bytes of codes a row (one 128-byte swizzle row), four MMAs of K = 64
//   scales  per 128 rows and K = 128 one 512-byte block, row r's four bytes at (r % 32) 16 + (r / 32) 4;
//           tcgen05.cp puts it into 4 columns of all four lane quarters. An MMA reads bytes 0-1 or 2-3.
//   TMEM    384 columns of accumulators (two of 192 or four of 96) and a set of scale columns a stage
//   roles   one CTA an SM, persistent: warp 0 TMA, warp 1 MMA, warp 2 a fence, warps 4-11 epilogue (four warps a
//           tile, in turn), warps 12 on scales.
//
// What bounds it, gate/up of 8192 tokens over 512 experts (K = 2048, N = 512): the 660 MB of weights, codes and
// scales and 84 MB of results take 113 us of HBM time, the kernel 130 at the full clock; run back to back
// it meets the power limit (1.44 GHz). Short groups are bound by the weights' bytes alone, single tokens by
// the chain from launch to the last tile.
//
// Tiles are dealt round-robin with a group's row tiles innermost, so a weight tile is read from HBM once and
// by the group's other row tiles from L2. Every wait on a barrier in shared memory is bounded and reports
// MOE_ERR_TIMEOUT.
#include <type_traits>

#include "block.cuh"
#include "tc.cuh"

namespace moe {

namespace {

constexpr int kMxRows = 128;     // weight rows of a tile
constexpr int kMxBox = 32;       // rows of one TMA box of the group's rows: a short tile loads only those it has
constexpr int kMxStageK = 256;   // K of a stage
constexpr int kMxRowBytes = kMxStageK / 2;
constexpr int kMxTileCache = 128;  // tiles whose place is worked out once, in the prologue
constexpr int kMxAccCols = 384;    // tensor memory columns of the accumulators, the scales behind them

// NT: rows of a group in a tile, at most
template <int NT>
struct MxCfg {
  static constexpr int kRowBlocks = (NT + 127) / 128;  // 128-row scale blocks of the group's rows
  static constexpr int kW = kMxRows * kMxRowBytes, kT = NT * kMxRowBytes;
  static constexpr int kSfW = 2 * 512, kSfT = 2 * kRowBlocks * 512;  // two K = 128 blocks
  static constexpr int kStage = kW + kT + kSfW + kSfT;
  static constexpr int kStages = NT == 96 ? 6 : 4;
  static constexpr int kScaleWarps = kStages / 2, kThreads = 32 * (12 + kScaleWarps);
  static constexpr int kAccs = kMxAccCols / NT, kSfCols = 8 + 8 * kRowBlocks;
  static constexpr int kNumBars = 3 * kStages + 2 * kAccs;
  // shared memory behind the stages: barriers, tiles, gate / up values on their way between lane quarters
  // ([pair of warps][buffer][direction][8 columns][32 lanes] fp32), tiles before each group
  static constexpr int kBar = kStages * kStage;
  static constexpr int kTiles = kBar + (kNumBars * 8 + 16 + 15) / 16 * 16;
  static constexpr int kSwap = kTiles + kMxTileCache * 16;
  static constexpr int smem(int E, bool up) { return kSwap + (up ? 4 * 2 * 2 * 1024 : 0) + (E + 1) * 4 + 1024; }
  static_assert(kStage % 1024 == 0, "stages start on swizzle atoms");
  static_assert(kMxAccCols + kStages * kSfCols <= 512, "tensor memory");
};

struct MxArgs {
  const int32_t *offsets;
  const uint8_t *a_scales, *w_scales, *up_scales;
  void *out;
  int out_type, n_rows, K, N, E, m_tiles;
  Ctrl *ctrl;
};

struct alignas(16) MxTile {
  int group, tok0, toks, m0;  // toks rows from tok0; features from m0
};

__device__ __forceinline__ void tc_mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                            uint32_t sfb, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %6, 0;\n"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
      : "memory");
}
// one 512-byte scale block (32 rows of 16 bytes) to 4 columns, repeated in the four lane quarters
__device__ __forceinline__ void tc_cp_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// unswizzled K-major descriptor: 8-row core matrices of 128 bytes one behind the other
__device__ __forceinline__ uint64_t plain_desc(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(128u >> 4) << 32) | ((uint64_t)1u << 46);
}
// kind::mxf4: A and B e2m1, scales ue8m0, both K-major, M = 128; sf: byte of the scale word (0 or 2)
__device__ __forceinline__ uint32_t idesc_mxf4(int N, uint32_t sf) {
  return (sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(128 >> 7) << 27) |
         (sf << 29);
}
__device__ __forceinline__ void mx_ld16(uint32_t taddr, uint32_t r[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// one lane of a converged warp. The TMA and MMA warps run their loops with all lanes and issue from the
// elected one: addresses and descriptors are then the same in every lane and stay in uniform
// registers. Loops run by lane 0 alone took 180 cycles an MMA instead of its 128.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n.reg .pred q;\nelect.sync _|q, 0xffffffff;\nselp.u32 %0, 1, 0, q;\n}\n" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}
template <bool BF>
__device__ __forceinline__ uint16_t cvt16(float v) {
  if constexpr (BF) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  else return __half_as_ushort(__float2half_rn(v));
}
// gate / (1 + exp(-gate)) with e = exp(-|gate|), so that the divisor stays in (1, 2]: the fast division gives 0 from a
// divisor of 2^126 on, which exp(-gate) passes at a gate of -87, where bf16 still holds the result.
__device__ __forceinline__ float fast_silu(float gate) {
  const float e = __expf(-fabsf(gate));
  return __fdividef(gate < 0.0f ? gate * e : gate, 1.0f + e);
}
// n of a lane's values of C consecutive rows to those rows, N values apart. The type is known at compile time and a
// whole chunk is stored without tests: with both decided value by value a store took 70 cycles. `top` becomes the largest
// magnitude stored as fp16 (one instruction a value), so that what rounds to an infinity is seen once a launch.
template <bool BF, int C>
__device__ __forceinline__ void store_rows(uint16_t *o, int N, const float y[C], int n, float &top) {
  if (n >= C) {
#pragma unroll
    for (int j = 0; j < C; ++j) {
      *o = cvt16<BF>(y[j]);
      if constexpr (!BF) top = fmaxf(top, fabsf(y[j]));
      o += N;
    }
  } else {
#pragma unroll
    for (int j = 0; j < C; ++j) {
      if (j < n) {
        *o = cvt16<BF>(y[j]);
        if constexpr (!BF) top = fmaxf(top, fabsf(y[j]));
      }
      o += N;
    }
  }
}

__device__ __forceinline__ void mx_timeout(Ctrl *ctrl, int where) { set_device_error(ctrl, MOE_ERR_TIMEOUT, where); }

// start and end row of a group, whatever the offsets hold: 0 <= start <= end <= n_rows
__device__ __forceinline__ int2 mx_group(const MxArgs &a, int g) {
  if (!a.offsets) return make_int2(0, a.n_rows);
  const int s = min(max(__ldg(a.offsets + g), 0), a.n_rows);
  return make_int2(s, min(max(__ldg(a.offsets + g + 1), s), a.n_rows));
}

// The scale bytes of the stages whose slots one warp owns: it loads the scales of all rows (lane + 32 i) for a pair
// of stages, waits for their slots, stores them and goes on to its slots' next pair, so that the loads
// are as far ahead as the TMA's. (With every warp on every stage and four loads ahead in registers, the
// oldest were waited for together with the youngest.) A warp sees every use of its slots in order: a
// parity wait that skipped a use would take the phase before the last for the last. Where K % 512 = 0
// a pair is 16 bytes a row, otherwise each stage's 8 are read apart. Four rows 32 apart are 16
// consecutive bytes of a scale block.
template <bool UP, int NT, class TileAt>
struct MxScales {
  static constexpr int kRows = 4 + NT / 32, kFeat = UP ? 64 : 128;
  const MxArgs &a;
  const TileAt &tile_at;
  const int n_my, nk, lane;

  __device__ __forceinline__ const uint8_t *row(const MxTile &t, int i) const {
    const int pitch = a.K / 32;
    if (i >= 4) return a.a_scales + (size_t)(t.tok0 + min(lane + 32 * (i - 4), t.toks - 1)) * pitch;
    const int r = lane + 32 * i;
    const bool up = UP && r >= kFeat;
    const int wr = min(t.group * a.N + t.m0 + (up ? r - kFeat : r), a.E * a.N - 1);
    return (up ? a.up_scales : a.w_scales) + (size_t)wr * pitch;
  }

  __device__ __forceinline__ void load8(const uint8_t *q, int ks, uint32_t v[2]) const {
    const int pitch = a.K / 32;
    if (a.K % 256 == 0) {
      const uint2 w = __ldg(reinterpret_cast<const uint2 *>(q) + ks);
      v[0] = w.x;
      v[1] = w.y;
      return;
    }
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)  // K % 64 == 0: whole pairs of scales
      h[j] = 8 * ks + 2 * j < pitch ? __ldg(reinterpret_cast<const uint16_t *>(q) + 4 * ks + j) : 0x7f7fu;
    v[0] = h[0] | h[1] << 16;
    v[1] = h[2] | h[3] << 16;
  }

  // put(stage, words) stores a stage; false after a time-out
  template <class Put>
  __device__ __forceinline__ void run(int w, const Put &put) const {
    const int total = n_my * nk;
    const bool wide = a.K % 512 == 0;  // nk is even, a pair is in one tile
    for (int g = 2 * w; g < total; g += MxCfg<NT>::kStages) {
      uint32_t v[2][2][kRows];  // [stage][word]
      const bool two = g + 1 < total;
      if (wide) {
        const MxTile t = tile_at(g / nk);
        const int at = 8 * (g % nk);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          if (i > 4 && 32 * (i - 4) >= t.toks) break;
          const uint4 x = __ldg(reinterpret_cast<const uint4 *>(row(t, i) + at));
          v[0][0][i] = x.x;
          v[0][1][i] = x.y;
          v[1][0][i] = x.z;
          v[1][1][i] = x.w;
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h && !two) break;
          const MxTile t = tile_at((g + h) / nk);
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            if (i > 4 && 32 * (i - 4) >= t.toks) break;
            uint32_t x[2];
            load8(row(t, i), (g + h) % nk, x);
            v[h][0][i] = x[0];
            v[h][1][i] = x[1];
          }
        }
      }
      if (!put(g, v[0]) || (two && !put(g + 1, v[1]))) return;
    }
  }
};

template <bool UP, bool BF, int NT>
__global__ void __launch_bounds__(MxCfg<NT>::kThreads, 1)
mx4_product_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                   const __grid_constant__ CUtensorMap tm_u, const MxArgs args) {
  using S = MxCfg<NT>;
  constexpr int kStages = S::kStages, kAccs = S::kAccs, kFeat = UP ? 64 : 128;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t *gbase = smem_raw + (base - smem_u32(smem_raw));
  auto st_w = [&](int s) { return base + s * S::kStage; };
  auto st_t = [&](int s) { return base + s * S::kStage + S::kW; };
  auto st_sf = [&](int s) { return base + s * S::kStage + S::kW + S::kT; };
  auto full = [&](int s) { return base + S::kBar + 8u * s; };
  auto empty = [&](int s) { return base + S::kBar + 8u * (kStages + s); };
  auto sf_in = [&](int s) { return base + S::kBar + 8u * (2 * kStages + s); };
  auto acc_full = [&](int b) { return base + S::kBar + 8u * (3 * kStages + b); };
  auto acc_empty = [&](int b) { return base + S::kBar + 8u * (3 * kStages + kAccs + b); };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + S::kBar + S::kNumBars * 8);
  int32_t *s_pref = reinterpret_cast<int32_t *>(gbase + S::kSwap + (UP ? 4 * 2 * 2 * 1024 : 0));  // [E + 1]
  __shared__ int32_t s_warp[S::kThreads / 32];

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  Ctrl *ctrl = args.ctrl;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), 2);  // TMA's bytes, the scales through the fence warp
      mbar_init(sf_in(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < kAccs; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), 4);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 0 && elect_one()) {
    prefetch_map(&tm_a);
    prefetch_map(&tm_w);
    if (UP) prefetch_map(&tm_u);
  }
  pdl_wait();
  bool good;  // offsets that are no offsets: flagged, and no tile is worked on (groups could overlap without end)
  {  // tiles before each group: every thread sums a run of groups, then a block scan of the runs
    constexpr int kPer = (kMaxE + S::kThreads - 1) / S::kThreads;
    const int per = (args.E + S::kThreads - 1) / S::kThreads, g0 = tid * per;
    int at[kPer + 1], mine = 0, bad = 0;  // a run's offsets, loaded in one round
#pragma unroll
    for (int i = 0; i <= kPer; ++i)
      if (i <= per && g0 + i <= args.E) at[i] = args.offsets ? args.offsets[g0 + i] : i * args.n_rows;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int g = g0 + i;
      if (i >= per || g >= args.E) continue;
      const int s0 = min(max(at[i], 0), args.n_rows), s1 = min(max(at[i + 1], s0), args.n_rows);
      if (s0 != at[i] || s1 != at[i + 1] || (g == 0 && s0 != 0)) {
        set_device_error(ctrl, MOE_ERR_DEVICE_CHECK, g);
        bad = 1;
      }
      at[i] = (s1 - s0 + NT - 1) / NT * args.m_tiles;
      mine += at[i];
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += n;
    }
    if (lane == 31) s_warp[warp] = incl;
    good = !__syncthreads_or(bad);
    int run = incl - mine;
    for (int w = 0; w < warp; ++w) run += s_warp[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int g = g0 + i;
      if (i >= per || g >= args.E) continue;
      s_pref[g] = run;
      run += at[i];
    }
    if (tid == S::kThreads - 1) s_pref[args.E] = run;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const int total = good ? s_pref[args.E] : 0, G = gridDim.x, nk = (args.K + kMxStageK - 1) / kMxStageK;
  const int n_my = total > (int)blockIdx.x ? (total - (int)blockIdx.x + G - 1) / G : 0;

  auto find_tile = [&](int tl) {
    const int ti = blockIdx.x + tl * G;
    int lo = 0, hi = args.E - 1;  // the last group that starts at or before the tile and has one
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_pref[mid] <= ti) lo = mid;
      else hi = mid - 1;
    }
    const int tt = (s_pref[lo + 1] - s_pref[lo]) / args.m_tiles, local = ti - s_pref[lo];
    const int2 r = mx_group(args, lo);
    const int size = ((r.y - r.x + tt - 1) / tt + 15) & ~15;
    MxTile t;
    t.group = lo;
    t.tok0 = r.x + (local % tt) * size;
    t.toks = min(size, r.y - t.tok0);
    t.m0 = (local / tt) * kFeat;
    return t;
  };
  MxTile *s_tiles = reinterpret_cast<MxTile *>(gbase + S::kTiles);
  if (tid < min(n_my, kMxTileCache)) s_tiles[tid] = find_tile(tid);
  __syncthreads();
  auto uniform_tile = [&](MxTile t) {
    t.group = __shfl_sync(0xffffffffu, t.group, 0);
    t.tok0 = __shfl_sync(0xffffffffu, t.tok0, 0);
    t.toks = __shfl_sync(0xffffffffu, t.toks, 0);
    t.m0 = __shfl_sync(0xffffffffu, t.m0, 0);
    return t;
  };
  auto tile_at = [&](int tl) { return tl < kMxTileCache ? s_tiles[tl] : find_tile(tl); };

  if (warp == 0) {
    // ------------------------------------------------ TMA
    bool ok = true;
    int g = 0;
    for (int tl = 0; tl < n_my && ok; ++tl) {
      const MxTile t = uniform_tile(tile_at(tl));
      const int nbox = (t.toks + kMxBox - 1) / kMxBox, wrow = t.group * args.N + t.m0;
      const uint32_t tx = (uint32_t)(nbox * kMxBox + kMxRows) * kMxRowBytes;
      for (int ks = 0; ks < nk; ++ks, ++g) {
        const int s = g % kStages;
        if (!__all_sync(0xffffffffu, mbar_wait(empty(s), ((uint32_t)(g / kStages) & 1u) ^ 1u))) {
          if (lane == 0) mx_timeout(ctrl, 41);
          ok = false;
          break;
        }
        if (elect_one()) {
          mbar_arrive_expect_tx(full(s), tx);
          tma_load_2d(st_w(s), &tm_w, ks * kMxRowBytes, wrow, full(s));
          if (UP) tma_load_2d(st_w(s) + kFeat * kMxRowBytes, &tm_u, ks * kMxRowBytes, wrow, full(s));
          for (int b = 0; b < nbox; ++b)
            tma_load_2d(st_t(s) + b * kMxBox * kMxRowBytes, &tm_a, ks * kMxRowBytes, t.tok0 + b * kMxBox, full(s));
        }
        __syncwarp();
      }
    }
    // after a give-up somewhere: the copies of the last stages have landed before the CTA leaves
    for (int j = max(0, g - kStages); j < g; ++j) (void)mbar_wait(full(j % kStages), (uint32_t)(j / kStages) & 1u);
  } else if (warp == 1) {
    // ------------------------------------------------ MMA
    bool ok = true;
    int g = 0;
    for (int tl = 0; tl < n_my && ok; ++tl) {
      const int b = tl % kAccs, toks = __shfl_sync(0xffffffffu, tile_at(tl).toks, 0);
      if (!__all_sync(0xffffffffu, mbar_wait(acc_empty(b), ((uint32_t)(tl / kAccs) & 1u) ^ 1u))) {
        if (lane == 0) mx_timeout(ctrl, 42);
        break;
      }
      tc_fence_after();
      const uint32_t d = tmem + (uint32_t)(b * NT);
      const int N = (toks + 15) & ~15;
      const uint32_t id0 = idesc_mxf4(N, 0), id2 = idesc_mxf4(N, 2);
      for (int ks = 0; ks < nk; ++ks, ++g) {
        const int s = g % kStages;
        if (!__all_sync(0xffffffffu, mbar_wait(full(s), (uint32_t)(g / kStages) & 1u))) {
          if (lane == 0) mx_timeout(ctrl, 43);
          ok = false;
          break;
        }
        tc_fence_after();
        // the slot's own set of scale columns: its last readers were done when the slot was filled again
        const uint32_t sf = tmem + (uint32_t)(kMxAccCols + s * S::kSfCols);
        const uint64_t dsf = plain_desc(st_sf(s)), da = sw128_desc(st_w(s)), db = sw128_desc(st_t(s));
        const int steps = (args.K - ks * kMxStageK) / 64;
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            tc_cp_scales(sf + 4u * j, dsf + (uint64_t)((512 * j) >> 4));
            tc_cp_scales(sf + 8u + 4u * S::kRowBlocks * j, dsf + (uint64_t)((S::kSfW + 512 * S::kRowBlocks * j) >> 4));
            if (S::kRowBlocks > 1 && toks > 128)
              tc_cp_scales(sf + 12u + 8u * j, dsf + (uint64_t)((S::kSfW + 1024 * j + 512) >> 4));
          }
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (q < steps)
              tc_mma_mxf4(d, da + (uint64_t)((32 * q) >> 4), db + (uint64_t)((32 * q) >> 4), (q & 1) ? id2 : id0,
                          sf + 4u * (q >> 1), sf + 8u + 4u * S::kRowBlocks * (q >> 1), (ks | q) ? 1u : 0u);
          tc_commit(empty(s));
          if (ks == nk - 1) tc_commit(acc_full(b));
        }
        __syncwarp();
      }
    }
    // after a give-up: what was issued is complete before the columns are freed
    if (g > 0) (void)mbar_wait(empty((g - 1) % kStages), (uint32_t)((g - 1) / kStages) & 1u);
  } else if (warp == 2) {
    // ------------------------------------------------ proxy fence
    // The scale warps write through the generic proxy, tcgen05.cp reads through the async one. The fence between
    // them stands on the path from one to the other, in a warp of its own: in the scale warps it waited for
    // their loads in flight as well, in the MMA warp it was a good part of a stage's issue.
    const int total_g = n_my * nk;
    for (int g = 0; g < total_g; ++g) {
      const int s = g % kStages;
      if (!__all_sync(0xffffffffu, mbar_wait(sf_in(s), (uint32_t)(g / kStages) & 1u))) {
        if (lane == 0) mx_timeout(ctrl, 46);
        break;
      }
      if (lane == 0) {
        fence_async_smem();
        mbar_arrive(full(s));
      }
    }
  } else if (warp >= 4 && warp < 12) {
    // ------------------------------------------------ epilogue: four warps, a lane quarter each, every other tile
    const int q = warp & 3, who = (warp - 4) >> 2;
    const uint32_t lane_base = (uint32_t)(32 * q) << 16;
    uint16_t *out = static_cast<uint16_t *>(args.out);
    // With gate and up, quarters 0 and 1 hold 64 features' gate rows, 2 and 3 their up rows. Of 16 columns the gate
    // warp finishes the first 8 and the up warp the others; each hands its partner the 8 values that
    // the partner lacks. Buffers alternate, so one barrier of the pair an exchange is enough.
    const int pair = (q & 1) + 2 * who;
    float *swap = reinterpret_cast<float *>(gbase + S::kSwap) + pair * 4 * 256;
    int turn = 0;
    float top = 0.0f;
    bool ok = true;  // after a time-out a warp goes on through its partner's barriers, without waiting again
    for (int tl = who; tl < n_my; tl += 2) {
      const MxTile t = tile_at(tl);
      const int b = tl % kAccs;
      if (ok && !__all_sync(0xffffffffu, mbar_wait(acc_full(b), (uint32_t)(tl / kAccs) & 1u))) {
        if (lane == 0) mx_timeout(ctrl, 44);
        ok = false;
      }
      tc_fence_after();
      const uint32_t acc = tmem + lane_base + (uint32_t)(b * NT);
      const int f = t.m0 + 32 * (UP ? q & 1 : q) + lane;
      uint16_t *op = out + (size_t)t.tok0 * args.N + f;
      if (UP || f < args.N) {  // a whole warp's rows are there or none are: N % 64 = 0
        uint32_t v[2][16];
        auto finish = [&](int c, const uint32_t x[16]) {
          uint16_t *o = op + (size_t)c * args.N;
          const int left = ok ? t.toks - c : 0;
          if constexpr (UP) {
            const bool up_warp = q >= 2;
            float *w = swap + turn * 512 + (up_warp ? 256 : 0), *r = swap + turn * 512 + (up_warp ? 0 : 256);
            turn ^= 1;
#pragma unroll
            for (int j = 0; j < 8; ++j) w[32 * j + lane] = __uint_as_float(up_warp ? x[j] : x[8 + j]);
            asm volatile("bar.sync %0, 64;" ::"r"(1 + pair) : "memory");
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float other = r[32 * j + lane], own = __uint_as_float(up_warp ? x[8 + j] : x[j]);
              const float gate = up_warp ? other : own, upv = up_warp ? own : other;
              y[j] = fast_silu(gate) * upv;
            }
            store_rows<BF, 8>(up_warp ? o + 8 * (size_t)args.N : o, args.N, y, up_warp ? left - 8 : left, top);
          } else {
            float y[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] = __uint_as_float(x[j]);
            store_rows<BF, 16>(o, args.N, y, left, top);
          }
        };
        mx_ld16(acc, v[0]);
#pragma unroll 1
        for (int c = 0; c < t.toks; c += 32) {  // the next 16 columns are on their way while 16 are stored
          tmem_ld_wait16(v[0]);
          if (c + 16 < t.toks) mx_ld16(acc + c + 16, v[1]);
          finish(c, v[0]);
          if (c + 16 < t.toks) {
            tmem_ld_wait16(v[1]);
            if (c + 32 < t.toks) mx_ld16(acc + c + 32, v[0]);
            finish(c + 16, v[1]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty(b));
    }
    // 65520 is the first magnitude that rounds to an fp16 infinity; a NaN is not larger than anything
    if constexpr (!BF) {
      if (__any_sync(0xffffffffu, top >= 65520.0f) && lane == 0) set_device_error(ctrl, MOE_ERR_RANGE, 47);
    }
    // rows behind the last group
    const int kept = args.offsets ? mx_group(args, args.E - 1).y : args.n_rows;
    const float z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const size_t n8 = (size_t)args.n_rows * (args.N / 8);
    for (size_t i = (size_t)kept * (args.N / 8) + blockIdx.x * 256 + (tid - 128); i < n8; i += (size_t)G * 256)
      store8(args.out, args.out_type, 8 * i, z);
  } else if (warp >= 12) {
    // ------------------------------------------------ scales
    const MxScales<UP, NT, decltype(tile_at)> scales{args, tile_at, n_my, nk, lane};
    auto put = [&](int g, const uint32_t x[2][4 + NT / 32]) {  // stage g's scales of all rows
      const int s = g % kStages;
      if (!__all_sync(0xffffffffu, mbar_wait(empty(s), ((uint32_t)(g / kStages) & 1u) ^ 1u))) {
        if (lane == 0) mx_timeout(ctrl, 45);
        return false;
      }
      uint4 *sf = reinterpret_cast<uint4 *>(gbase + (st_sf(s) - base)) + lane;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        sf[32 * j] = make_uint4(x[j][0], x[j][1], x[j][2], x[j][3]);
        uint4 *sb = sf + S::kSfW / 16 + 32 * S::kRowBlocks * j;
        if constexpr (NT == 96) {
          sb[0] = make_uint4(x[j][4], x[j][5], x[j][6], 0u);
        } else {
          sb[0] = make_uint4(x[j][4], x[j][5], x[j][6], x[j][7]);
          *reinterpret_cast<uint2 *>(sb + 32) = make_uint2(x[j][8], x[j][9]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sf_in(s));
      return true;
    };
    scales.run(warp - 12, put);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

template <bool UP, bool BF, int NT>
cudaError_t launch_tiles(const Mx4ProductArgs &p, cudaStream_t s) {
  constexpr int kFeat = UP ? 64 : 128;
  const uint64_t kb = (uint64_t)p.K / 2, wr = (uint64_t)p.E * p.N;
  CUtensorMap ta, tw, tu;
  auto map = [&](CUtensorMap *m, const uint8_t *ptr, uint64_t rows, int box) {
    return encode_tensor_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, ptr, kb, rows, kMxRowBytes, box,
                                CU_TENSOR_MAP_SWIZZLE_128B);
  };
  if (!map(&ta, p.a_codes, p.n_rows, kMxBox) || !map(&tw, p.w_codes, wr, kFeat)) return cudaErrorInvalidValue;
  if (!UP) tu = tw;
  else if (!map(&tu, p.up_codes, wr, kFeat)) return cudaErrorInvalidValue;
  const int mt = (p.N + kFeat - 1) / kFeat;
  const MxArgs a{p.offsets, p.a_scales, p.w_scales, p.up_scales, p.out, p.out_type, p.n_rows, p.K, p.N, p.E, mt, p.ctrl};
  const int live = p.E < p.n_rows ? p.E : p.n_rows;  // at most: every live group's last tile is partial
  const long long most = ((long long)p.n_rows / NT + live) * mt;
  const int grid = (int)(most < num_sms() ? most : num_sms());
  const cudaError_t e = smem_limit_once(mx4_product_kernel<UP, BF, NT>, MxCfg<NT>::smem(kMaxE, UP));
  if (e != cudaSuccess) return e;
  KTimer kt_(KID_MX4_PRODUCT, s);
  // A short product begins while its predecessor ends (40 rows, four tokens: 0.5 us). A long one gains nothing, and with
  // its blocks waiting beside the quantiser's the two took 173-180 us for 81,920 rows, not 172. The border between
  // the two measurements is not measured.
  if (p.n_rows <= 4096)
    return launch_pdl(mx4_product_kernel<UP, BF, NT>, dim3(grid), dim3(MxCfg<NT>::kThreads), MxCfg<NT>::smem(p.E, UP), s, ta, tw, tu, a);
  mx4_product_kernel<UP, BF, NT><<<grid, MxCfg<NT>::kThreads, MxCfg<NT>::smem(p.E, UP), s>>>(ta, tw, tu, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx4_product(const Mx4ProductArgs &p, cudaStream_t s) {
  // Rows of a tile, by the mean over all experts (the host does not know how many are idle): 192 where
  // groups are long (8192 tokens over 512 experts, 160 rows each, with the quantiser:
  // 156 us, 185 with 96), else 96: a stage is smaller and more are in flight, and four accumulators leave
  // short tiles' epilogues behind (2048 tokens, down, 40 rows each: 67.8 us, 72.2 with 192; ten rows of
  // one token: 12.3 us cold, 13.8).
  const bool long_groups = p.n_rows > 80ll * p.E;
  auto run = [&](auto up, auto bf) {
    return long_groups ? launch_tiles<up.value, bf.value, 192>(p, s) : launch_tiles<up.value, bf.value, 96>(p, s);
  };
  constexpr std::true_type yes{};
  constexpr std::false_type no{};
  if (p.out_type == MOE_BF16) return p.up_codes ? run(yes, yes) : run(no, yes);
  return p.up_codes ? run(yes, no) : run(no, no);
}

}  // namespace moe
