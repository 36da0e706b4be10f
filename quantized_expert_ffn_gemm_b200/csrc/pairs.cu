// (token, slot) pairs sorted by expert, their rows copied there and collected again with the routing
// weights, and the gradients of both.
//
//   sort      row_of[t,j] = place of pair (t,j) among all pairs ordered by (expert, t, j); -1 where
//             idx[t,j] = -1 (a padded token, a slot over an expert's capacity)
//   dispatch  rows[row_of[t,j]] = x[t]
//   collect   y[t] = sum_j w[t,j] rows[row_of[t,j]] (+ residual[t]); without w also dispatch's gradient
//   gradient of collect:  d_rows[row_of[t,j]] = w[t,j] dy[t],   d_w[t,j] = <dy[t], rows[row_of[t,j]]>
//
// The sort is a stable counting sort: each block ranks a chunk of pairs (equal experts of a warp by
// __match_any_sync, warps by a prefix over their counts), so the order is the same in every run.
// Nothing here adds with atomics across blocks; sums run over j in order.
//
// The copies are bound by their bytes. 8192 tokens of ten bf16 rows of 2048: dispatch 60.7 us (369 MB, 56 us of
// measured copy rate), collect 69 us (403 MB, 61 us; it reads rows in 4 KB pieces scattered
// over 335 MB), its gradient 115 us (705 MB, 107 us). The sort before them is a chain of a few
// dependent steps: 8 us for 81,920 pairs in two launches, 2.3 us for 60 in one (in a graph).
#include <type_traits>

#include "block.cuh"

namespace moe {

namespace {

// warps of a chunk's block, 32 pairs each: the per-warp expert counts (16 bits) have to fit shared memory
int chunk_warps(int E) { return E <= 2048 ? 32 : 16; }

// ---------------------------------------------------------------- sort
__device__ __forceinline__ int valid_expert(int e, int E, Ctrl *ctrl) {
  if (e >= 0 && e < E) return e;
  if (e != -1) set_device_error(ctrl, MOE_ERR_DEVICE_CHECK, e);
  return -1;
}

// hist[c][e]: pairs of chunk c that chose expert e
__global__ void __launch_bounds__(1024) pair_hist_kernel(const int32_t *__restrict__ idx, int P, int E,
                                                        int32_t *__restrict__ hist, Ctrl *ctrl) {
  extern __shared__ int32_t s_count[];
  for (int e = threadIdx.x; e < E; e += blockDim.x) s_count[e] = 0;
  pdl_launch_dependents();
  pdl_wait();
  __syncthreads();
  const long long p = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (p < P) {
    const int e = valid_expert(idx[p], E, ctrl);
    if (e >= 0) atomicAdd(&s_count[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) hist[(size_t)blockIdx.x * E + e] = s_count[e];
}

// Many chunks: each expert's counts become the pairs in the chunks before, hist[chunks][e] their total. 32
// experts a block, a warp of lanes apiece over runs of chunks.
__global__ void __launch_bounds__(1024) pair_scan_kernel(int32_t *__restrict__ hist, int chunks, int E) {
  __shared__ int32_t s_run[32][33];
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
  const int per = (chunks + 31) / 32, c0 = run * per, c1 = min(chunks, c0 + per);
  pdl_launch_dependents();
  pdl_wait();
  int sum = 0;
  if (e < E) {
#pragma unroll 8
    for (int c = c0; c < c1; ++c) sum += hist[(size_t)c * E + e];
  }
  s_run[run][lane] = sum;
  __syncthreads();
  int before = 0;
  for (int r = 0; r < run; ++r) before += s_run[r][lane];
  if (e >= E) return;
  for (int c = c0; c < c1; ++c) {
    const int n = hist[(size_t)c * E + e];
    hist[(size_t)c * E + e] = before;
    before += n;
  }
  if (run == 31) hist[(size_t)chunks * E + e] = before;
}

// One chunk a block; with one chunk in all hist is not read, with few (scanned = 0) every block adds up the
// chunks' counts itself, which spares a launch, with many it finds them added up.
__global__ void __launch_bounds__(1024)
pair_place_kernel(const int32_t *__restrict__ idx, int P, int k, int E, const int32_t *__restrict__ hist, int scanned,
                  int32_t *__restrict__ counts, int32_t *__restrict__ offsets, int32_t *__restrict__ row_of,
                  int32_t *__restrict__ src, Ctrl *ctrl) {
  extern __shared__ int32_t s_base[];                         // [E] first row of this chunk's pairs of e
  uint16_t *s_cnt = reinterpret_cast<uint16_t *>(s_base + E);  // [warps][E] pairs of e in a warp, then before it
  __shared__ int32_t s_warp[32];
  __shared__ int32_t s_kept;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5, chunks = gridDim.x;
  const int live = (int)min((long long)nw, (P - (long long)blockIdx.x * blockDim.x + 31) >> 5);  // warps that have pairs
  for (int i = tid; i < (live * E + 1) / 2; i += blockDim.x) reinterpret_cast<uint32_t *>(s_cnt)[i] = 0;  // nw is even
  pdl_launch_dependents();
  pdl_wait();
  __syncthreads();
  const long long p = (long long)blockIdx.x * blockDim.x + tid;
  const int e = p < P ? valid_expert(idx[p], E, ctrl) : -1;
  const unsigned same = __match_any_sync(0xffffffffu, e >= 0 ? e : -1 - lane);
  const int rank = __popc(same & ((1u << lane) - 1u));
  if (e >= 0 && rank == 0) s_cnt[(size_t)warp * E + e] = (uint16_t)__popc(same);
  __syncthreads();
  // counts of each expert: of the warps before (in place), of the chunks before, of all chunks
  const int per = (E + (int)blockDim.x - 1) / (int)blockDim.x;  // consecutive experts a thread, at most 8
  int total[8], mine = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    total[i] = 0;
    const int x = tid * per + i;
    if (i >= per || x >= E) continue;
    int run = 0;
    for (int w0 = 0; w0 < live; w0 += 8) {  // eight counts read before any is replaced
      int n[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) n[j] = w0 + j < live ? s_cnt[(size_t)(w0 + j) * E + x] : 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (w0 + j < live) s_cnt[(size_t)(w0 + j) * E + x] = (uint16_t)run;
        run += n[j];
      }
    }
    int before = 0, all = run;
    if (scanned) {
      before = hist[(size_t)blockIdx.x * E + x];
      all = hist[(size_t)chunks * E + x];
    } else if (chunks > 1) {
      all = 0;
#pragma unroll 16
      for (int c = 0; c < chunks; ++c) {
        const int n = hist[(size_t)c * E + x];
        before += c < (int)blockIdx.x ? n : 0;
        all += n;
      }
    }
    s_base[x] = before;
    total[i] = all;
    mine += all;
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int v = lane < nw ? s_warp[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += n;
    }
    s_warp[lane] = v;
    if (lane == 31) s_kept = v;
  }
  __syncthreads();
  int base = incl - mine + (warp ? s_warp[warp - 1] : 0);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int x = tid * per + i;
    if (i >= per || x >= E) continue;
    if (blockIdx.x == 0) {
      counts[x] = total[i];
      offsets[x] = base;
    }
    s_base[x] += base;
    base += total[i];
  }
  __syncthreads();
  const int kept = s_kept;
  if (blockIdx.x == 0 && tid == 0) offsets[E] = kept;
  if (p < P) {
    int row = -1;
    if (e >= 0) {
      row = s_base[e] + s_cnt[(size_t)warp * E + e] + rank;
      src[row] = (int)p / k;
    }
    row_of[p] = row;
    if (p >= kept) src[p] = -1;  // rows behind the last kept pair
  }
}

// ---------------------------------------------------------------- rows out and back
// zeroes rows kept .. P-1, spread over the grid's warps
__device__ __forceinline__ void zero_tail(void *rows, int type, int P, int H8, const int32_t *kept, long long item,
                                          long long n_items, int lane) {
  if (!kept) return;
  const float z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  const int first = min(max(*kept, 0), P);
  for (long long r = first + item; r < P; r += n_items)
    for (int c = lane; c < H8; c += 32) store8(rows, type, ((size_t)r * H8 + c) * 8, z);
}

// one warp a (token, segment of 32 CH chunks): the segment is loaded once and stored to the token's k rows
template <int CH>
__global__ void __launch_bounds__(256) dispatch_kernel(const void *__restrict__ x, int type, int T, int k, int H,
                                                      const int32_t *__restrict__ row_of,
                                                      const int32_t *__restrict__ kept, void *__restrict__ rows) {
  const int lane = threadIdx.x & 31, H8 = H >> 3, nseg = (H8 + 32 * CH - 1) / (32 * CH), P = T * k;
  const int es = type_bytes(type);
  pdl_launch_dependents();
  pdl_wait();
  const long long n_items = (long long)T * nseg, stride = (long long)gridDim.x * 8;
  const long long first = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  for (long long it = first; it < n_items; it += stride) {
    const int t = (int)(it / nseg), c0 = (int)(it % nseg) * 32 * CH + lane;
    const int my_row = lane < k ? row_of[(size_t)t * k + lane] : -1;
    Raw8 v[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (c0 + 32 * c < H8) v[c] = load_raw8(x, type, ((size_t)t * H8 + c0 + 32 * c) * 8);
    for (int j = 0; j < k; ++j) {
      const int r = __shfl_sync(0xffffffffu, my_row, j);
      if (r < 0 || r >= P) continue;
      uint8_t *d = static_cast<uint8_t *>(rows) + (size_t)r * H * es;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (c0 + 32 * c >= H8) continue;
        store_raw8(d, type, (size_t)(c0 + 32 * c) * 8, v[c]);
      }
    }
  }
  zero_tail(rows, type, P, H8, kept, first, stride, lane);
}

// One warp a (token, segment of 32 CH chunks), the segments of kLoads rows in flight. The rows are scattered over
// memory, so a warp takes 2 KB of each (CH = 4) while that leaves work for every SM: 512 bytes at a time
// read the rows of 8192 tokens at 4.7 TB/s, and eight rows in flight a lane at 3.
template <int CH, int KR, int KY>
__global__ void __launch_bounds__(256) collect_kernel(const void *__restrict__ rows, int rows_type, int T, int k, int H,
                                                     const int32_t *__restrict__ row_of, const float *__restrict__ w,
                                                     const float *residual, void *y, int out_type) {
  const int type = known_type<KR>(rows_type), y_type = known_type<KY>(out_type);
  constexpr int kLoads = CH == 1 ? 4 : 2;
  const int lane = threadIdx.x & 31, H8 = H >> 3, nseg = (H8 + 32 * CH - 1) / (32 * CH), P = T * k;
  pdl_launch_dependents();
  pdl_wait();
  const long long n_items = (long long)T * nseg, stride = (long long)gridDim.x * 8;
  for (long long it = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); it < n_items; it += stride) {
    const int t = (int)(it / nseg), c0 = (int)(it % nseg) * 32 * CH + lane;
    int my_row = lane < k ? row_of[(size_t)t * k + lane] : -1;
    if (my_row >= P) my_row = -1;
    const float my_w = (w && lane < k) ? w[(size_t)t * k + lane] : 1.0f;
    float acc[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[c][q] = 0.0f;
      if (residual && c0 + 32 * c < H8) load8(residual, MOE_F32, ((size_t)t * H8 + c0 + 32 * c) * 8, acc[c]);
    }
    for (int j0 = 0; j0 < k; j0 += kLoads) {
      Raw8 v[kLoads][CH];
      float wj[kLoads];
      int rj[kLoads];
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        rj[u] = __shfl_sync(0xffffffffu, my_row, (j0 + u) & 31);
        wj[u] = __shfl_sync(0xffffffffu, my_w, (j0 + u) & 31);
        if (j0 + u >= k) rj[u] = -1;
        if (rj[u] < 0) continue;
#pragma unroll
        for (int c = 0; c < CH; ++c)
          if (c0 + 32 * c < H8) v[u][c] = load_raw8(rows, type, ((size_t)rj[u] * H8 + c0 + 32 * c) * 8);
      }
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        if (rj[u] < 0) continue;  // a dropped pair adds nothing, whatever its weight is
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          if (c0 + 32 * c >= H8) continue;
          float f[8];
          raw8_to_float(v[u][c], type, f);
#pragma unroll
          for (int q = 0; q < 8; ++q) acc[c][q] = fmaf(wj[u], f[q], acc[c][q]);
        }
      }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (c0 + 32 * c < H8) store8(y, y_type, ((size_t)t * H8 + c0 + 32 * c) * 8, acc[c]);
  }
}

// one warp a pair: dy[t] (from L1 or L2 but for the token's first pair) against the pair's row
template <int KD, int KR>
__global__ void __launch_bounds__(256)
collect_grad_kernel(const void *__restrict__ dy, int in_type, const void *rows, int rows_type, int T, int k, int H,
                    const int32_t *__restrict__ row_of, const float *__restrict__ w, const int32_t *__restrict__ kept,
                    void *d_rows, float *__restrict__ d_w) {
  const int dy_type = known_type<KD>(in_type), type = known_type<KR>(rows_type);
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, H8 = H >> 3, P = T * k;
  const long long stride = (long long)gridDim.x * 8, first = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  for (long long p = first; p < P; p += stride) {
    const int t = (int)(p / k), r = row_of[p];
    float dot = 0.0f;
    if (r >= 0 && r < P) {
      const float wp = w ? w[p] : 1.0f;
      const size_t at_t = (size_t)t * H, at_r = (size_t)r * H;
      auto chunk = [&](int c, const Raw8 &g, const Raw8 &v) {
        float a[8], b[8];
        raw8_to_float(g, dy_type, a);
        if (d_w) {
          raw8_to_float(v, type, b);
#pragma unroll
          for (int q = 0; q < 8; ++q) dot = fmaf(a[q], b[q], dot);
        }
        if (d_rows) {
#pragma unroll
          for (int q = 0; q < 8; ++q) a[q] *= wp;
          store8(d_rows, type, at_r + 8 * c, a);
        }
      };
      int c0 = lane;
      for (; c0 + 96 < H8; c0 += 128) {  // four chunks of each in flight
        Raw8 g[4], v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          g[u] = load_raw8(dy, dy_type, at_t + 8 * (c0 + 32 * u));
          if (d_w) v[u] = load_raw8(rows, type, at_r + 8 * (c0 + 32 * u));
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) chunk(c0 + 32 * u, g[u], v[u]);
      }
      for (; c0 < H8; c0 += 32) {
        Raw8 v;
        const Raw8 g = load_raw8(dy, dy_type, at_t + 8 * c0);
        if (d_w) v = load_raw8(rows, type, at_r + 8 * c0);
        chunk(c0, g, v);
      }
      dot = warp_sum(dot);
    }
    if (d_w && lane == 0) d_w[p] = dot;
  }
  if (d_rows) zero_tail(d_rows, type, P, H8, kept, first, stride, lane);
}

int warp_grid(long long items) {  // eight warps a block
  const long long want = (items + 7) / 8, cap = (long long)num_sms() * 16;
  return (int)(want < cap ? want : cap);
}

}  // namespace

constexpr int kScanChunks = 128;  // chunks from which the scan kernel is worth its launch

size_t sort_pairs_scratch(long long P, int E) {
  const int per = 32 * chunk_warps(E);
  return (size_t)((P + per - 1) / per + 1) * E * 4;
}

cudaError_t launch_sort_pairs(const int32_t *idx, int T, int k, int E, int32_t *counts, int32_t *offsets,
                              int32_t *row_of, int32_t *src, int32_t *hist, Ctrl *ctrl, cudaStream_t s) {
  // One chunk takes no more warps than its pairs and experts (eight a thread) need, eight at least (60 pairs of 512
  // experts 2.4 us in a graph, 3.8 with 32 warps).
  const int P = T * k, most = chunk_warps(E);
  const int nw = P > 32 * most ? most : max(max(8, (P + 63) / 64 * 2), (E + 511) / 512 * 2), threads = 32 * nw;
  const int chunks = (int)(((long long)P + threads - 1) / threads);
  const int scanned = chunks > kScanChunks ? 1 : 0;
  const size_t smem = (size_t)E * 4 + (size_t)nw * E * 2;
  const cudaError_t e = smem_limit_once(pair_place_kernel, smem > 48 * 1024 ? 160 * 1024 : 0);
  if (e != cudaSuccess) return e;
  if (chunks > 1) {
    KTimer kt_(KID_PAIR_HIST, s);
    const cudaError_t eh = launch_pdl(pair_hist_kernel, dim3(chunks), dim3(threads), (size_t)E * 4, s, idx, P, E, hist, ctrl);
    if (eh != cudaSuccess) return eh;
  }
  if (scanned) {
    KTimer kt_(KID_PAIR_SCAN, s);
    const cudaError_t es = launch_pdl(pair_scan_kernel, dim3((E + 31) / 32), dim3(1024), 0, s, hist, chunks, E);
    if (es != cudaSuccess) return es;
  }
  {
    KTimer kt_(KID_PAIR_PLACE, s);
    return launch_pdl(pair_place_kernel, dim3(chunks), dim3(threads), smem, s, idx, P, k, E, (const int32_t *)hist, scanned, counts,
                      offsets, row_of, src, ctrl);
  }
}

cudaError_t launch_dispatch(const void *x, int type, int T, int k, int H, const int32_t *row_of, const int32_t *kept,
                            void *rows, cudaStream_t s) {
  KTimer kt_(KID_DISPATCH, s);
  type = kernel_type(type, (const void *)((uintptr_t)x | (uintptr_t)rows));
  const int H8 = H / 8;
  return launch_pdl(dispatch_kernel<4>, dim3(warp_grid((long long)T * ((H8 + 127) / 128))), dim3(256), 0, s, x, type, T, k,
                    H, row_of, kept, rows);
}

// calls f with two types at compile time (fp32 that is not 32-byte aligned: with types told apart at run time)
template <class F>
cudaError_t by_types(int a, int b, const F &f) {
  using std::integral_constant;
  constexpr integral_constant<int, kAny> any{};
  constexpr integral_constant<int, kF32Wide> w{};
  constexpr integral_constant<int, MOE_F16> h{};
  constexpr integral_constant<int, MOE_BF16> n{};
  if (a == MOE_F32 || b == MOE_F32) return f(any, any);
  auto second = [&](auto x) { return b == kF32Wide ? f(x, w) : b == MOE_F16 ? f(x, h) : f(x, n); };
  return a == kF32Wide ? second(w) : a == MOE_F16 ? second(h) : second(n);
}

cudaError_t launch_collect(const void *rows, int type, int T, int k, int H, const int32_t *row_of, const float *w,
                           const float *residual, void *y, int y_type, cudaStream_t s) {
  KTimer kt_(KID_COLLECT, s);
  type = kernel_type(type, rows);
  y_type = kernel_type(y_type, y);
  const int per = type == kF32Wide || type == MOE_F32 ? 2 : 4;  // chunks a lane for 2 KB of a row
  const long long items = (long long)T * ((H / 8 + 32 * per - 1) / (32 * per));
  const bool wide = items >= 16ll * num_sms();
  return by_types(type, y_type, [&](auto r, auto o) {
    constexpr int CH = r.value == MOE_F16 || r.value == MOE_BF16 ? 4 : 2;
    if (wide)
      return launch_pdl(collect_kernel<CH, r.value, o.value>, dim3(warp_grid(items)), dim3(256), 0, s, rows, type, T, k, H,
                        row_of, w, residual, y, y_type);
    return launch_pdl(collect_kernel<1, r.value, o.value>, dim3(warp_grid((long long)T * ((H / 8 + 31) / 32))), dim3(256),
                      0, s, rows, type, T, k, H, row_of, w, residual, y, y_type);
  });
}

cudaError_t launch_collect_grad(const void *dy, int dy_type, const void *rows, int type, int T, int k, int H,
                                const int32_t *row_of, const float *w, const int32_t *kept, void *d_rows, float *d_w,
                                cudaStream_t s) {
  KTimer kt_(KID_COLLECT_GRAD, s);
  type = kernel_type(type, (const void *)((uintptr_t)rows | (uintptr_t)d_rows));
  dy_type = kernel_type(dy_type, dy);
  return by_types(dy_type, type, [&](auto d, auto r) {
    return launch_pdl(collect_grad_kernel<d.value, r.value>, dim3(warp_grid((long long)T * k)), dim3(256), 0, s, dy,
                      dy_type, rows, type, T, k, H, row_of, w, kept, d_rows, d_w);
  });
}

}  // namespace moe
