// Product of MXFP4 rows with per-expert MXFP4 weights on the block-scaled tensor cores:
//
//   out[r, n] = sum_k A[r, k] W_g[n, k]   for the rows r of group g, or, with an up matrix,
//   out[r, n] = silu(A W_g^T)[r, n] * (A U_g^T)[r, n]
//
// tcgen05.mma kind::mxf4 multiplies e2m1 codes and applies both operands' block scales itself (one e8m0
// byte for 32 values, read from tensor memory), so the codes go from HBM to shared memory by TMA and from
// there to the MMA untouched; only the scale bytes are rearranged on the way.
//
//   tile    128 rows of a group (MMA M, one tensor-memory lane a row) x NC columns: NC features, or NC / 2
//           gate and NC / 2 up rows of the same features, whose accumulators one thread holds side by side
//   stage   K = 256: 128 bytes of codes a row (one 128-byte swizzle row), four MMAs of K = 64
//   scales  per 128 rows and K = 128 one 512-byte block, row r's four bytes at (r % 32) 16 + (r / 32) 4;
//           tcgen05.cp puts it into 4 columns of all four lane quarters. An MMA reads bytes 0-1 or 2-3.
//   TMEM    two accumulators of NC columns and a set of scale columns a stage in flight. With NC = 256 the
//           accumulators (columns 0 and 208) share 48 columns, which leaves room for two sets: a
//           tile's epilogue first reads the shared ones into registers and lets the next tile begin.
//           (Two sets hold a stage until the one but last has finished, about 1000 cycles from issue to
//           commit: no loss while a stage's MMAs take 512, but 555 cycles a stage of an NC = 64
//           tile, whose MMAs take 128. Three sets and 80 shared columns: the next tile began
//           2000 cycles after a tile's end instead of 600.)
//   roles   one CTA an SM, persistent: warp 0 TMA, warp 1 MMA, warp 2 a fence, warps 4-11 epilogue (two a lane quarter),
//           warps 12 on scales.
//
// Tiles are dealt round-robin with a group's row tiles innermost, so a weight tile is read from HBM once and
// by the group's other row tiles from L2. Every wait is bounded and reports MOE_ERR_TIMEOUT.
#include "block.cuh"
#include "tc.cuh"

namespace moe {

namespace {

constexpr int kMxRows = 128;     // rows of a tile
constexpr int kMxBoxRows = 32;   // rows of one TMA box of A: a short tile loads only the boxes it has rows in
constexpr int kMxStageK = 256;   // K of a stage
constexpr int kMxRowBytes = kMxStageK / 2;
constexpr int kMxTileCache = 128;  // tiles whose place is worked out once, in the prologue

template <int NC>
struct MxSmem {
  static constexpr int kA = kMxRows * kMxRowBytes, kB = NC * kMxRowBytes;
  static constexpr int kRowBlocks = (NC + 127) / 128;               // 128-row scale blocks of B
  static constexpr int kSfA = 2 * 512, kSfB = 2 * kRowBlocks * 512;  // two K = 128 blocks a stage
  static constexpr int kStage = kA + kB + kSfA + kSfB;
  static constexpr int kStages = NC == 256 ? 4 : 6;
  static constexpr int kScaleWarps = kStages / 2, kThreads = 32 * (12 + kScaleWarps);
  // tensor memory: column of the second accumulator, of the scales, columns and number of the scale sets
  static constexpr int kAcc1 = NC == 256 ? 208 : NC, kSf = kAcc1 + NC, kSfCols = 8 + 8 * kRowBlocks;
  static constexpr int kSfSets = NC == 256 ? 2 : kStages;
  static constexpr int kOver = NC - kAcc1;  // columns that both accumulators use
  static_assert(kSf + kSfSets * kSfCols <= 512 && kOver % 16 == 0, "tensor memory");
  static constexpr int kBar = kStages * kStage;
  static constexpr int kNumBars = 3 * kStages + 5;
  static constexpr int kTiles = kBar + (kNumBars * 8 + 16 + 15) / 16 * 16;
  static constexpr int kPrefix = kTiles + kMxTileCache * 16;
  static constexpr int bytes(int E) { return kPrefix + (E + 1) * 4 + 1024; }
  static_assert(kStage % 1024 == 0, "stages start on swizzle atoms");
};

struct MxArgs {
  const int32_t *offsets;
  const uint8_t *a_scales, *w_scales, *up_scales;
  void *out;
  int out_type, n_rows, K, N, E, n_tiles_n;
  Ctrl *ctrl;
};

struct alignas(16) MxTile {
  int group, row0, rows, n0;
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
__device__ __forceinline__ uint32_t pack16(float lo, float hi, int type) {
  if (type == MOE_BF16) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
  }
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
// A lane's 32 bytes of its own row: a warp's store touches 32 lines whatever its width, and their number is
// what the epilogue's stores cost, so one 32-byte store beats two of 16.
__device__ __forceinline__ void store32(void *p, const uint32_t y[8], bool aligned32) {
  if (aligned32) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(y[0]), "r"(y[1]), "r"(y[2]),
                 "r"(y[3]), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
                 : "memory");
    return;
  }
  static_cast<uint4 *>(p)[0] = make_uint4(y[0], y[1], y[2], y[3]);
  static_cast<uint4 *>(p)[1] = make_uint4(y[4], y[5], y[6], y[7]);
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
template <int NC, bool UP, class TileAt>
struct MxScales {
  static constexpr int kRows = 4 + NC / 32, kFeat = UP ? NC / 2 : NC;
  const MxArgs &a;
  const TileAt &tile_at;
  const int n_my, nk, lane;

  __device__ __forceinline__ const uint8_t *row(const MxTile &t, int i) const {
    const int pitch = a.K / 32;
    if (i < 4) return a.a_scales + (size_t)(t.row0 + min(lane + 32 * i, t.rows - 1)) * pitch;
    const int r = lane + 32 * (i - 4);
    const bool up = UP && r >= kFeat;
    const int wr = min(t.group * a.N + t.n0 + (up ? r - kFeat : r), a.E * a.N - 1);
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
    for (int g = 2 * w; g < total; g += MxSmem<NC>::kStages) {
      uint32_t v[2][2][kRows];  // [stage][word]
      const bool two = g + 1 < total;
      if (wide) {
        const MxTile t = tile_at(g / nk);
        const int at = 8 * (g % nk);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
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

template <int NC, bool UP>
__global__ void __launch_bounds__(MxSmem<NC>::kThreads, 1)
mx4_product_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                   const __grid_constant__ CUtensorMap tm_u, const MxArgs args) {
  using S = MxSmem<NC>;
  constexpr int kStages = S::kStages, kFeat = UP ? NC / 2 : NC;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t *gbase = smem_raw + (base - smem_u32(smem_raw));
  auto st_a = [&](int s) { return base + s * S::kStage; };
  auto st_b = [&](int s) { return base + s * S::kStage + S::kA; };
  auto st_sf = [&](int s) { return base + s * S::kStage + S::kA + S::kB; };
  auto full = [&](int s) { return base + S::kBar + 8u * s; };
  auto empty = [&](int s) { return base + S::kBar + 8u * (kStages + s); };
  auto acc_full = [&](int b) { return base + S::kBar + 8u * (2 * kStages + b); };
  auto acc_empty = [&](int b) { return base + S::kBar + 8u * (2 * kStages + 2 + b); };
  const uint32_t acc_over = base + S::kBar + 8u * (2 * kStages + 4);  // the shared columns are read
  auto sf_in = [&](int s) { return base + S::kBar + 8u * (2 * kStages + 5 + s); };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + S::kBar + S::kNumBars * 8);
  int32_t *s_pref = reinterpret_cast<int32_t *>(gbase + S::kPrefix);  // [E + 1] tiles before a group
  __shared__ int32_t s_warp[S::kThreads / 32];

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  Ctrl *ctrl = args.ctrl;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), 2);  // TMA's bytes, the scales through the fence warp
      mbar_init(sf_in(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), 8);
    }
    mbar_init(acc_over, 8);
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
  {  // tiles before each group: every thread sums a run of groups, then a block scan of the runs
    constexpr int kPer = (kMaxE + S::kThreads - 1) / S::kThreads;
    const int per = (args.E + S::kThreads - 1) / S::kThreads, g0 = tid * per;
    int at[kPer + 1], mine = 0;  // a run's offsets, loaded in one round
#pragma unroll
    for (int i = 0; i <= kPer; ++i)
      if (i <= per && g0 + i <= args.E) at[i] = args.offsets ? args.offsets[g0 + i] : i * args.n_rows;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int g = g0 + i;
      if (i >= per || g >= args.E) continue;
      const int s0 = min(max(at[i], 0), args.n_rows), s1 = min(max(at[i + 1], s0), args.n_rows);
      if (s0 != at[i] || s1 != at[i + 1] || (g == 0 && s0 != 0)) set_device_error(ctrl, MOE_ERR_DEVICE_CHECK, g);
      at[i] = (s1 - s0 + kMxRows - 1) / kMxRows * args.n_tiles_n;
      mine += at[i];
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += n;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
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
  const int total = s_pref[args.E], G = gridDim.x, nk = (args.K + kMxStageK - 1) / kMxStageK;
  const int n_my = total > (int)blockIdx.x ? (total - (int)blockIdx.x + G - 1) / G : 0;

  auto find_tile = [&](int tl) {
    const int ti = blockIdx.x + tl * G;
    int lo = 0, hi = args.E - 1;  // the last group that starts at or before the tile and has one
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_pref[mid] <= ti) lo = mid;
      else hi = mid - 1;
    }
    const int mt = (s_pref[lo + 1] - s_pref[lo]) / args.n_tiles_n, local = ti - s_pref[lo];
    const int2 r = mx_group(args, lo);
    MxTile t;
    t.group = lo;
    t.row0 = r.x + (local % mt) * kMxRows;
    t.rows = min(kMxRows, r.y - t.row0);
    t.n0 = (local / mt) * kFeat;
    return t;
  };
  MxTile *s_tiles = reinterpret_cast<MxTile *>(gbase + S::kTiles);
  if (tid < min(n_my, kMxTileCache)) s_tiles[tid] = find_tile(tid);
  __syncthreads();
  auto uniform_tile = [&](MxTile t) {
    t.group = __shfl_sync(0xffffffffu, t.group, 0);
    t.row0 = __shfl_sync(0xffffffffu, t.row0, 0);
    t.rows = __shfl_sync(0xffffffffu, t.rows, 0);
    t.n0 = __shfl_sync(0xffffffffu, t.n0, 0);
    return t;
  };
  auto tile_at = [&](int tl) { return tl < kMxTileCache ? s_tiles[tl] : find_tile(tl); };

  if (warp == 0) {
    // ------------------------------------------------ TMA
    bool ok = true;
    int g = 0;
    for (int tl = 0; tl < n_my && ok; ++tl) {
      const MxTile t = uniform_tile(tile_at(tl));
      const int nbox = (t.rows + kMxBoxRows - 1) / kMxBoxRows, wrow = t.group * args.N + t.n0;
      const uint32_t tx = (uint32_t)(nbox * kMxBoxRows + NC) * kMxRowBytes;
      for (int ks = 0; ks < nk; ++ks, ++g) {
        const int s = g % kStages;
        if (!__all_sync(0xffffffffu, mbar_wait(empty(s), ((uint32_t)(g / kStages) & 1u) ^ 1u))) {
          if (lane == 0) mx_timeout(ctrl, 41);
          ok = false;
          break;
        }
        if (elect_one()) {
          mbar_arrive_expect_tx(full(s), tx);
          tma_load_2d(st_b(s), &tm_w, ks * kMxRowBytes, wrow, full(s));
          if (UP) tma_load_2d(st_b(s) + kFeat * kMxRowBytes, &tm_u, ks * kMxRowBytes, wrow, full(s));
          for (int b = 0; b < nbox; ++b)
            tma_load_2d(st_a(s) + b * kMxBoxRows * kMxRowBytes, &tm_a, ks * kMxRowBytes, t.row0 + b * kMxBoxRows, full(s));
        }
        __syncwarp();
      }
    }
    // after a give-up somewhere: the copies of the last stages have landed before the CTA leaves
    for (int j = max(0, g - kStages); j < g; ++j) (void)mbar_wait(full(j % kStages), (uint32_t)(j / kStages) & 1u);
  } else if (warp == 1) {
    // ------------------------------------------------ MMA
    const uint32_t id0 = idesc_mxf4(NC, 0), id2 = idesc_mxf4(NC, 2);
    bool ok = true;
    int g = 0;
    for (int tl = 0; tl < n_my && ok; ++tl) {
      const int b = tl & 1;
      const bool go = mbar_wait(acc_empty(b), (((uint32_t)tl >> 1) & 1u) ^ 1u) &&
                      (S::kOver == 0 || tl == 0 || mbar_wait(acc_over, (uint32_t)(tl - 1) & 1u));
      if (!__all_sync(0xffffffffu, go)) {
        if (lane == 0) mx_timeout(ctrl, 42);
        break;
      }
      tc_fence_after();
      const uint32_t d = tmem + (uint32_t)(b * S::kAcc1);
      for (int ks = 0; ks < nk; ++ks, ++g) {
        const int s = g % kStages;
        // the scale columns of stage g were read by the MMAs of stage g - kSfSets; with a set a stage
        // the stage's own slot says so
        constexpr int kBack = S::kSfSets;
        const bool in = mbar_wait(full(s), (uint32_t)(g / kStages) & 1u) &&
                        (kBack == kStages || g < kBack ||
                         mbar_wait(empty((g - kBack) % kStages), (uint32_t)((g - kBack) / kStages) & 1u));
        if (!__all_sync(0xffffffffu, in)) {
          if (lane == 0) mx_timeout(ctrl, 43);
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sf = tmem + (uint32_t)(S::kSf + g % kBack * S::kSfCols);
        const uint64_t dsf = plain_desc(st_sf(s)), da = sw128_desc(st_a(s)), db = sw128_desc(st_b(s));
        const int steps = (args.K - ks * kMxStageK) / 64;
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            tc_cp_scales(sf + 4u * j, dsf + (uint64_t)((512 * j) >> 4));
#pragma unroll
            for (int r = 0; r < S::kRowBlocks; ++r)
              tc_cp_scales(sf + 8u + 8u * j + 4u * r,
                           dsf + (uint64_t)((S::kSfA + 512 * (j * S::kRowBlocks + r)) >> 4));
          }
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (q < steps)
              tc_mma_mxf4(d, da + (uint64_t)((32 * q) >> 4), db + (uint64_t)((32 * q) >> 4), (q & 1) ? id2 : id0,
                          sf + 4u * (q >> 1), sf + 8u + 8u * (q >> 1), (ks | q) ? 1u : 0u);
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
    // ------------------------------------------------ epilogue: a lane quarter and every other 16 features
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lane_base = (uint32_t)(32 * q) << 16;
    constexpr int kChunks = kFeat / 16, kIt = kFeat / 32;
    static_assert(S::kOver <= 48, "the shared columns are each warp's first chunk or two");
    const bool out32 = ((uintptr_t)args.out & 31u) == 0;
    for (int tl = 0; tl < n_my; ++tl) {
      const MxTile t = tile_at(tl);
      const int b = tl & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(acc_full(b), ((uint32_t)tl >> 1) & 1u))) {
        if (lane == 0) mx_timeout(ctrl, 44);
        break;
      }
      tc_fence_after();
      const uint32_t acc = tmem + lane_base + (uint32_t)(b * S::kAcc1);
      const int r = 32 * q + lane;
      uint8_t *op = static_cast<uint8_t *>(args.out) + ((size_t)(t.row0 + r) * args.N + t.n0) * 2;
      // from the end that the other accumulator shares, so that those columns are read first
      auto feat = [&](int it) { return 16 * (b ? 2 * it + half : kChunks - 1 - 2 * it - half); };
      uint32_t v[2][16], u[2][16];
      auto load = [&](int it, int p) {
        mx_ld16(acc + feat(it), v[p]);
        if (UP) mx_ld16(acc + kFeat + feat(it), u[p]);
      };
      const bool any = 32 * q < t.rows;  // a quarter without rows has nothing to read
      if (any) {
        load(0, 0);
        if (kIt > 1) load(1, 1);
        tmem_ld_wait16(v[0]);
        tmem_ld_wait16(v[1]);
        if (UP) {
          tmem_ld_wait16(u[0]);
          tmem_ld_wait16(u[1]);
        }
      }
      if (S::kOver) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_over);
      }
#pragma unroll 1
      for (int it0 = 0; any && it0 < kIt; it0 += 2) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int it = it0 + p;
          if (it >= kIt) break;
          const int f = feat(it);
          if (it >= 2) {
            tmem_ld_wait16(v[p]);
            if (UP) tmem_ld_wait16(u[p]);
          }
          uint32_t y[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float a = __uint_as_float(v[p][2 * j]), c = __uint_as_float(v[p][2 * j + 1]);
            if (UP) {
              a = __fdividef(a, 1.0f + __expf(-a)) * __uint_as_float(u[p][2 * j]);
              c = __fdividef(c, 1.0f + __expf(-c)) * __uint_as_float(u[p][2 * j + 1]);
            }
            y[j] = pack16(a, c, args.out_type);
          }
          if (it + 2 < kIt) load(it + 2, p);
          if (r < t.rows && t.n0 + f < args.N) store32(op + 2 * f, y, out32);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty(b));
    }
    // rows behind the last group
    const int kept = args.offsets ? mx_group(args, args.E - 1).y : args.n_rows;
    const float z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const size_t n8 = (size_t)args.n_rows * (args.N / 8);
    for (size_t i = (size_t)kept * (args.N / 8) + blockIdx.x * 256 + (tid - 128); i < n8; i += (size_t)G * 256)
      store8(args.out, args.out_type, 8 * i, z);
  } else if (warp >= 12) {
    // ------------------------------------------------ scales
    const MxScales<NC, UP, decltype(tile_at)> scales{args, tile_at, n_my, nk, lane};
    auto put = [&](int g, const uint32_t x[2][4 + NC / 32]) {  // stage g's scales of all rows
      const int s = g % kStages;
      if (!__all_sync(0xffffffffu, mbar_wait(empty(s), ((uint32_t)(g / kStages) & 1u) ^ 1u))) {
        if (lane == 0) mx_timeout(ctrl, 45);
        return false;
      }
      uint4 *sf = reinterpret_cast<uint4 *>(gbase + (st_sf(s) - base)) + lane;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        sf[32 * j] = make_uint4(x[j][0], x[j][1], x[j][2], x[j][3]);
        uint4 *sb = sf + S::kSfA / 16 + 32 * j * S::kRowBlocks;
        if constexpr (NC < 128) {
          *reinterpret_cast<uint2 *>(sb) = make_uint2(x[j][4], x[j][5]);
        } else {
#pragma unroll
          for (int r = 0; r < S::kRowBlocks; ++r)
            sb[32 * r] = make_uint4(x[j][4 + 4 * r], x[j][5 + 4 * r], x[j][6 + 4 * r], x[j][7 + 4 * r]);
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

template <int NC, bool UP>
cudaError_t launch_nc(const Mx4ProductArgs &p, cudaStream_t s) {
  constexpr int kFeat = UP ? NC / 2 : NC;
  const uint64_t kb = (uint64_t)p.K / 2, wr = (uint64_t)p.E * p.N;
  CUtensorMap ta, tw, tu;
  auto map = [&](CUtensorMap *m, const uint8_t *ptr, uint64_t rows, int box) {
    return encode_tensor_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, ptr, kb, rows, kMxRowBytes, box,
                                CU_TENSOR_MAP_SWIZZLE_128B);
  };
  if (!map(&ta, p.a_codes, p.n_rows, kMxBoxRows) || !map(&tw, p.w_codes, wr, kFeat) ||
      !map(&tu, UP ? p.up_codes : p.w_codes, wr, kFeat))
    return cudaErrorInvalidValue;
  const int nt = (p.N + kFeat - 1) / kFeat;
  const MxArgs a{p.offsets, p.a_scales, p.w_scales, p.up_scales, p.out, p.out_type, p.n_rows, p.K, p.N, p.E, nt, p.ctrl};
  const int live = p.E < p.n_rows ? p.E : p.n_rows;  // at most: every live group's last tile is partial
  const long long most = ((long long)p.n_rows / kMxRows + live) * nt;
  const int grid = (int)(most < num_sms() ? most : num_sms());
  const cudaError_t e = smem_limit_once(mx4_product_kernel<NC, UP>, MxSmem<NC>::bytes(kMaxE));
  if (e != cudaSuccess) return e;
  KTimer kt_(KID_MX4_PRODUCT, s);
  // A short product begins while its predecessor ends (four tokens: 0.5 us). A long one gains nothing, and with
  // its blocks waiting beside the quantiser's the two took 173-180 us for 8192 tokens, not 172.
  if (p.n_rows <= 4096)
    return launch_pdl(mx4_product_kernel<NC, UP>, dim3(grid), dim3(MxSmem<NC>::kThreads), MxSmem<NC>::bytes(p.E), s, ta,
                      tw, tu, a);
  mx4_product_kernel<NC, UP><<<grid, MxSmem<NC>::kThreads, MxSmem<NC>::bytes(p.E), s>>>(ta, tw, tu, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx4_product(const Mx4ProductArgs &p, cudaStream_t s) {
  // Columns of a tile. 256: fewest bytes from L2 and the MMAs' best rate, for groups of many rows (8192 tokens
  // over 512 experts, 160 rows each: 171 us with the quantiser, 189 with 128). 128: less left over at the
  // end and an epilogue of two accumulators, for the others (2048 tokens, down, 40 rows each: 68.5 us, 70.5 with
  // 256; four tokens: 21.0 us cold, 22.6). 64: more SMs at work where 128 leaves some idle (four groups of
  // 64 rows, K = 4096, N = 1024: 14.4 us, 16.0 with 128, 18.5 with 256).
  const bool up = p.up_codes != nullptr;
  const int live = p.E < p.n_rows ? p.E : p.n_rows;
  auto tiles = [&](int nc) {  // at most: every live group's last tile is partial
    const int feat = up ? nc / 2 : nc;
    return ((long long)p.n_rows / kMxRows + live) * ((p.N + feat - 1) / feat);
  };
  if (tiles(256) >= 4ll * num_sms() && p.n_rows >= 64ll * p.E)
    return up ? launch_nc<256, true>(p, s) : launch_nc<256, false>(p, s);
  if (tiles(128) >= num_sms()) return up ? launch_nc<128, true>(p, s) : launch_nc<128, false>(p, s);
  return up ? launch_nc<64, true>(p, s) : launch_nc<64, false>(p, s);
}

}  // namespace moe
