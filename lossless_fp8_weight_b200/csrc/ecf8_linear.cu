// Linear layers over decoded E4M3 weights, with low-rank adapters: forward and
// backward, for any size, stride and alignment.
//
//     forward   u[t] = A[a] x[t]            y[t] = s * (W x[t]) + alpha[a] * B[a] u[t]
//     backward  v[t] = B[a]^T dy[t]        dx[t] = W^T (s * dy[t]) + alpha[a] * A[a]^T v[t]
//               da[a] = alpha[a] * sum_t v[t] x[t]^T      db[a] = alpha[a] * sum_t dy[t] u[t]^T
//
// with a the adapter of row t's request.  u and v stay in float32.
//
// The *_simple and route kernels are the formulas as they stand.  They serve
// operands whose rows TMA cannot read and that no workspace has room to copy;
// everything else takes the tensor-core kernels: the projection's in
// ecf8_product.cuh, the others below.  Fractions of measured rates in the
// comments are of 6561 GB/s and 1646 TFLOP/s.
#include "ecf8_linear.cuh"

namespace {

using namespace ecf8_linear_impl;

__device__ inline float e4m3(uint8_t b) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3)));
}

// row_id[t] = the adapter of row t, -1 for none.
__global__ void route_kernel(const int32_t* offsets, const int32_t* ids, uint32_t count, uint32_t n_adapters,
                             uint64_t rows, int32_t* row_id, int32_t* d_status) {
  // every thread owns rows and looks its request up: no two threads write one row
  for (uint64_t t = blockIdx.x * (uint64_t)blockDim.x + threadIdx.x; t < rows; t += (uint64_t)gridDim.x * blockDim.x) {
    uint32_t lo = 0, hi = count;  // the number of offsets[1..count] that are <= t
    while (lo < hi) {
      const uint32_t mid = (lo + hi) / 2;
      if ((int64_t)offsets[mid + 1] <= (int64_t)t) lo = mid + 1;
      else hi = mid;
    }
    int32_t id = -1;
    if (lo < count && (int64_t)offsets[lo] <= (int64_t)t) id = ids[lo];
    row_id[t] = id >= 0 && (uint32_t)id < n_adapters ? id : -1;
  }
  for (uint64_t i = blockIdx.x * (uint64_t)blockDim.x + threadIdx.x; i < count; i += (uint64_t)gridDim.x * blockDim.x) {
    const int32_t b = offsets[i], e = offsets[i + 1], id = ids[i];
    if ((b < 0 || e < b || (int64_t)e > (int64_t)rows || (id >= 0 && (uint32_t)id >= n_adapters)) && d_status)
      atomicOr(d_status, ECF8_STATUS_BAD_REQUEST);
  }
}

// p[t][r] = sum over j of q[t][j] * f[a][r][j], f's element (r, j) at r * sr + j * sj.
// One CTA a row and 8 ranks; the row is read coalesced.
template <class T>
__global__ void __launch_bounds__(128) shrink_simple(const T* q, uint64_t q_stride, const T* f, uint64_t f_adapter,
                                                     uint64_t sr, uint64_t sj, uint64_t len, uint32_t rank,
                                                     const int32_t* row_id, float* p) {
  __shared__ float part[4][8];
  const uint64_t t = blockIdx.x;
  const uint32_t r0 = blockIdx.y * 8, nr = min(8u, rank - r0);
  const int32_t id = row_id[t];
  float acc[8] = {};
  if (id >= 0) {
    const T* row = q + t * q_stride;
    const T* fa = f + (uint64_t)id * f_adapter + r0 * sr;
    for (uint64_t j = threadIdx.x; j < len; j += 128) {
      const float x = to_float(row[j]);
#pragma unroll
      for (uint32_t r = 0; r < 8; ++r)
        if (r < nr) acc[r] = fmaf(x, to_float(fa[r * sr + j * sj]), acc[r]);
    }
  }
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    for (int d = 16; d; d >>= 1) acc[r] += __shfl_xor_sync(~0u, acc[r], d);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32][r] = acc[r];
  }
  __syncthreads();
  if (threadIdx.x < nr)
    p[t * rank + r0 + threadIdx.x] =
        part[0][threadIdx.x] + part[1][threadIdx.x] + part[2][threadIdx.x] + part[3][threadIdx.x];
}

// The shared projection with the adapters' part added before the one rounding.
//   BACK = 0: out[t][c] = scale[c] * sum_j q[t][j] W[c][j]      + alpha * sum_r p[t][r] f[a][c][r]
//   BACK = 1: out[t][c] = sum_j q[t][j] scale[j] W[j][c]        + alpha * sum_r p[t][r] f[a][r][c]
// 64 x 64 tiles, 16 terms at a time through shared memory, 4 x 4 sums a thread.
template <class T, int BACK>
__global__ void __launch_bounds__(256) product_simple(const T* q, uint64_t q_stride, const uint8_t* w,
                                                      uint64_t w_stride, const float* scale, uint64_t n_scale,
                                                      uint64_t rows, uint64_t cols, uint64_t len, const int32_t* row_id,
                                                      const float* p, const T* f, uint64_t f_adapter, uint64_t sr,
                                                      uint64_t sc, const float* alpha, uint32_t rank, T* out,
                                                      uint64_t out_stride) {
  __shared__ float qs[16][65], ws[16][65];
  const uint64_t c0 = (uint64_t)blockIdx.x * 64, t0 = (uint64_t)blockIdx.y * 64;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  for (uint64_t j0 = 0; j0 < len; j0 += 16) {
    for (int i = threadIdx.x; i < 64 * 16; i += 256) {
      const int j = i % 16, t = i / 16;
      float v = 0;
      if (t0 + t < rows && j0 + j < len) {
        v = to_float(q[(t0 + t) * q_stride + j0 + j]);
        if (BACK && n_scale > 1) v *= scale[j0 + j];
      }
      qs[j][t] = v;
      const int jj = BACK ? i / 64 : i % 16, c = BACK ? i % 64 : i / 16;
      float x = 0;
      if (c0 + c < cols && j0 + jj < len)
        x = e4m3(BACK ? w[(j0 + jj) * w_stride + c0 + c] : w[(c0 + c) * w_stride + j0 + jj]);
      ws[jj][c] = x;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      float a[4], b[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) a[k] = qs[j][ty + 16 * k], b[k] = ws[j][tx + 16 * k];
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n) acc[m][n] = fmaf(a[m], b[n], acc[m][n]);
    }
    __syncthreads();
  }
  for (int m = 0; m < 4; ++m) {
    const uint64_t t = t0 + ty + 16 * m;
    if (t >= rows) continue;
    const int32_t id = rank ? row_id[t] : -1;
    for (int n = 0; n < 4; ++n) {
      const uint64_t c = c0 + tx + 16 * n;
      if (c >= cols) continue;
      const float s = n_scale == 0 ? 1.0f : n_scale == 1 ? scale[0] : BACK ? 1.0f : scale[c];
      float y = acc[m][n] * s;
      if (id >= 0) {
        float z = 0;
        const T* fa = f + (uint64_t)id * f_adapter + c * sc;
        for (uint32_t r = 0; r < rank; ++r) z = fmaf(p[t * rank + r], to_float(fa[r * sr]), z);
        y = fmaf(alpha[id], z, y);
      }
      put(out + t * out_stride + c, y);
    }
  }
}

// ---- x A^T of every row's own adapter, on the tensor cores ----
//
//     D[(adapter, r)][t] += sum_j f[adapter][r][j] q[t][j]
//
// Bound: one read of q.  A tile is 16 to 256 rows of q against up to 128 rows of
// adapters: the distinct adapters of the tile's rows, `per` at a time, each
// with its ranks on consecutive lanes.  Sums of a row with an adapter that is
// not its own are dropped: no row sees another request's adapter.  As in the
// projection the reduction is split over a cluster whose sums meet in
// distributed shared memory in a fixed order.
// The kernel also finds the adapter of every row, for itself and for the
// projection, which starts beside it.
//
// Measured: 8192 rows of 8192 at rank 64 37 us, 3.6 TB/s, 55% of the copy rate;
// 32 rows of 4096, 24 adapters of rank 16: 13 us, the latency of its parts.

struct ShrinkArgs {
  uint64_t rows;
  uint32_t blocks;       // 64-wide steps of the reduction
  uint32_t bt, stages, split;
  uint32_t rank, per;    // ranks of an adapter, adapters in a chunk of 128 lanes
  const int32_t* offsets;
  const int32_t* request_ids;
  uint32_t count, n_adapters;
  int32_t* row_id;       // written: the adapter of every row, -1 for none
  float* p;              // rows x rank
  int32_t* status;
  Limits limits;
};

constexpr int kShrinkThreads = 320;

template <class T>
__global__ void __launch_bounds__(kShrinkThreads)
    shrink_tc(const __grid_constant__ CUtensorMap map_f, const __grid_constant__ CUtensorMap map_q,
              const __grid_constant__ ShrinkArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 2];
  __shared__ uint32_t tmem_base;
  __shared__ int failed_s;
  __shared__ int32_t ids[256], runs[256], list[256];
  __shared__ uint32_t count_s, warp_sum[8];
  const Waits waits{&failed_s, a.limits.cycles};

  const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
  const uint32_t f_bytes = 16384, q_bytes = a.bt * 128, stage_bytes = f_bytes + q_bytes;
  const uint32_t full = smem_addr(bars), empty = full + 8 * kMaxStages, done = empty + 8 * kMaxStages,
                 spent = done + 8;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t crank = a.split > 1 ? cluster_rank() : 0;
  const uint32_t chunk = blockIdx.x / a.split;
  const uint64_t t0 = (uint64_t)blockIdx.y * a.bt;
  const uint32_t b0 = (uint32_t)((uint64_t)a.blocks * crank / a.split),
                 b1 = (uint32_t)((uint64_t)a.blocks * (crank + 1) / a.split), nb = b1 - b0;
  const uint32_t columns = a.bt <= 32 ? 32 : a.bt <= 64 ? 64 : a.bt <= 128 ? 128 : 256;
  const uint32_t pad = (a.rank + 7) / 8 * 8;

  const uint32_t n = (uint32_t)(a.rows - t0 < a.bt ? a.rows - t0 : a.bt);
  if (threadIdx.x == 64) {
    tma_prefetch(&map_f);
    tma_prefetch(&map_q);
  }
  if (threadIdx.x < 256) ids[threadIdx.x] = -1;
  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < a.stages; ++i) {
      mbar_init(full + 8 * i, i == 0 ? 1 + a.limits.missing : 1);
      mbar_init(empty + 8 * i, 1);
    }
    mbar_init(done, 1);
    mbar_init(spent, 1);
    failed_s = 0;
    mbar_init_fence();
  }
  if (warp == 1) {
    tmem_alloc<1>(smem_addr(&tmem_base), columns);
    tmem_release_permit<1>();
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_base;
  // Only now: the projection's CTAs hold their tensor memory until this kernel has ended.  Were one to take an SM's while
  // a CTA here still waited for some, neither would go on.
  start_successor();
  // the requests that reach into this tile write their rows' ids
  bool backwards = false;
  for (uint32_t i = threadIdx.x; i < a.count; i += kShrinkThreads) {
    const int32_t b = a.offsets[i], e = a.offsets[i + 1], id = a.request_ids[i];
    const bool known = id < 0 || (uint32_t)id < a.n_adapters;
    if (b < 0 || e < b || (int64_t)e > (int64_t)a.rows || !known) {
      if (a.status && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(a.status, ECF8_STATUS_BAD_REQUEST);
    }
    backwards |= e < b;
    if (id < 0 || !known) continue;
    const int64_t lo = max((int64_t)b - (int64_t)t0, (int64_t)0), hi = min((int64_t)e - (int64_t)t0, (int64_t)n);
    for (int64_t t = lo; t < hi; ++t) ids[t] = id;
  }
  if (__syncthreads_or(backwards)) {
    // Requests of such a table may overlap, and their threads have written shared rows in any order.  The CTAs of a
    // cluster have to agree on every row, since they share its sums and leave together: the last request takes it.
    if (threadIdx.x < 256) ids[threadIdx.x] = -1;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < a.count; i += kShrinkThreads) {
      const int32_t b = a.offsets[i], e = a.offsets[i + 1], id = a.request_ids[i];
      if (id < 0 || (uint32_t)id >= a.n_adapters) continue;
      const int64_t lo = max((int64_t)b - (int64_t)t0, (int64_t)0), hi = min((int64_t)e - (int64_t)t0, (int64_t)n);
      for (int64_t t = lo; t < hi; ++t) atomicMax(&ids[t], (int32_t)i);
    }
    __syncthreads();
    if (threadIdx.x < 256 && ids[threadIdx.x] >= 0) ids[threadIdx.x] = a.request_ids[ids[threadIdx.x]];
    __syncthreads();
  }
  if (chunk == 0 && crank == 0 && threadIdx.x < n) a.row_id[t0 + threadIdx.x] = ids[threadIdx.x];
  distinct(ids, n, runs, list, &count_s, warp_sum);
  // rows without an adapter have zeros
  if (chunk == 0 && crank == 0)
    for (uint32_t t = warp; t < n; t += kShrinkThreads / 32)
      if (ids[t] < 0)
        for (uint32_t r = lane; r < a.rank; r += 32) a.p[(t0 + t) * a.rank + r] = 0.0f;
  const uint32_t first = chunk * a.per;
  if (first >= count_s) {  // the same in every CTA of the cluster
    if (warp == 1) tmem_free<1>(tmem, columns);
    return;
  }
  const uint32_t mine = count_s - first < a.per ? count_s - first : a.per;

  uint32_t next = 0, next_turn = 0;  // warp 0: the next stage to load, and the parity of its use
  if (warp == 0) {
    for (uint32_t i = 0; i < nb; ++i) {
      if (!mbar_wait_lanes(empty + 8 * next, next_turn ^ 1, waits)) break;
      const uint32_t at = base + next * stage_bytes, bar = full + 8 * next;
      const int32_t j = (int32_t)((b0 + i) * 64);
      if (elect_one()) {
        mbar_expect(bar, q_bytes + mine * a.rank * 128);
        tma_load(at + f_bytes, &map_q, j, (int32_t)t0, bar);
      }
      __syncwarp();
      // the lanes share the adapters' loads
      for (uint32_t k = lane; k < mine; k += 32)
        tma_load(at + k * pad * 128, &map_f, j, list[first + k] * (int32_t)a.rank, bar);
      __syncwarp();
      if (++next == a.stages) next = 0, next_turn ^= 1;
    }
  } else if (warp == 1) {
    const uint32_t idesc = idesc_f16(Widen<T>::kBf16, 128, a.bt);
    bool ok = true;
    uint32_t s = 0, turn = 0;
    for (uint32_t i = 0; i < nb; ++i) {
      ok = mbar_wait_lanes(full + 8 * s, turn, waits);
      if (!ok) break;
      fence_after();
      const uint64_t f = desc_k128(base + s * stage_bytes), q = desc_k128(base + s * stage_bytes + f_bytes);
      if (elect_one()) {
#pragma unroll
        for (int m = 0; m < 4; ++m) mma_ss(tmem, f + m * 2, q + m * 2, idesc, i > 0 || m > 0);
        mma_commit<1>(empty + 8 * s, 0);
      }
      __syncwarp();
      if (++s == a.stages) s = 0, turn ^= 1;
    }
    if (ok && elect_one()) mma_commit<1>(done, 0);
    __syncwarp();
  } else {
    const int quarter = warp % 4, half = (warp - 2) / 4;
    const uint32_t row = quarter * 32 + lane;
    const uint32_t slot = row / pad, r = row % pad;
    const bool ok = mbar_wait(done, 0, waits);
    if (ok && quarter * 32 < mine * pad) {
      fence_after();
      const int32_t id = slot < mine && r < a.rank ? list[first + slot] : -2;
      for (uint32_t t = half * 16; t < a.bt; t += 32) {
        float d[16];
        tmem_ld16(tmem + ((uint32_t)(quarter * 32) << 16) + t, d);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          if (a.split > 1)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + ((t + j) * 128 + row) * 4), "f"(d[j]) : "memory");
          else if (ids[t + j] == id) a.p[(t0 + t + j) * a.rank + r] = d[j];
        }
      }
    }
  }
  if (a.split > 1) {
    __syncwarp();
    cluster_sync();
    if (warp >= 2 && !failed_s) {
      // a thread four ranks at a time (of one adapter: pad is a multiple of 8)
      const uint32_t wide = mine * pad / 4, lo = a.bt * crank / a.split, hi = a.bt * (crank + 1) / a.split;
      for (uint32_t i = threadIdx.x - 64; i < (hi - lo) * wide; i += 256) {
        const uint32_t t = lo + i / wide, row = i % wide * 4, slot = row / pad, r = row % pad;
        if (ids[t] != list[first + slot]) continue;
        const float4 d = cluster_sum4(base + (t * 128 + row) * 4, a.split);
        float* p = a.p + (t0 + t) * a.rank + r;
        if (r < a.rank) p[0] = d.x;
        if (r + 1 < a.rank) p[1] = d.y;
        if (r + 2 < a.rank) p[2] = d.z;
        if (r + 3 < a.rank) p[3] = d.w;
      }
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while another reads its sums
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (failed_s) {
    if (warp == 0) drain_loads(full, next, next_turn, a.stages, waits);
    if (warp == 1) drain_products<1>(spent, 0, waits);
  }
  if (warp == 1) tmem_free<1>(tmem, columns);
  if (threadIdx.x == 0 && failed_s && a.status) atomicOr(a.status, ECF8_STATUS_TIMEOUT);
}

// Rows of bytes copied to rows whose bases and distances TMA takes (multiples of 16 bytes), for operands that are
// not laid out so.  A thread writes 16 bytes: the source is read in aligned 4-byte words and shifted into place.
struct Restride {
  const uint8_t* from[3];
  uint8_t* to[3];
  uint64_t rows[3], bytes[3], stride[3], to_stride[3];  // in bytes
};

__global__ void __launch_bounds__(256) restride_kernel(Restride a) {
  const int k = blockIdx.y;
  const uint64_t per = a.to_stride[k] / 16, total = a.rows[k] * per, step = (uint64_t)gridDim.x * 256;
  for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < total; i += step) {
    const uint64_t row = i / per, at = i % per * 16;
    const uint8_t* src = a.from[k] + row * a.stride[k] + at;
    const uint32_t* words = reinterpret_cast<const uint32_t*>((uintptr_t)src & ~(uintptr_t)3);
    const uint32_t shift = ((uintptr_t)src & 3) * 8;
    // bytes of this piece that exist, and the words that hold one of them
    const int64_t left = min((int64_t)16, (int64_t)a.bytes[k] - (int64_t)at), held = (left + shift / 8 + 3) / 4;
    uint32_t w[5], v[4];
#pragma unroll
    for (int j = 0; j < 5; ++j) w[j] = j < held ? words[j] : 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = __funnelshift_r(w[j], w[j + 1], shift);
      if (left < 4 * j + 4) v[j] = left <= 4 * j ? 0 : v[j] & (0xffffffffu >> (32 - 8 * (left - 4 * j)));
    }
    *reinterpret_cast<uint4*>(a.to[k] + row * a.to_stride[k] + at) = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

// out[a][r][j] = in[a][j][r]: B with the reduction of dy B contiguous, as the kernel above reads it.
template <class T>
__global__ void __launch_bounds__(256) transpose_kernel(const T* in, T* out, uint64_t len, uint64_t out_len,
                                                        uint32_t rank) {
  __shared__ T tile[64][ECF8_RANK_MAX + 2];
  const uint64_t j0 = (uint64_t)blockIdx.x * 64, a = blockIdx.y;
  const uint32_t n = (uint32_t)(len - j0 < 64 ? len - j0 : 64);
  const T* from = in + (a * len + j0) * rank;
  for (uint32_t i = threadIdx.x; i < n * rank; i += 256) tile[i / rank][i % rank] = from[i];
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < 64 * rank; i += 256) {
    const uint32_t r = i / 64, j = i % 64;
    if (j < n) out[(a * rank + r) * out_len + j0 + j] = tile[j][r];
  }
}

// ---- the adapters' gradients on the tensor cores ----
//
//     D[c][r] = sum over the adapter's rows of q[t][c] p[t][r]
//
// Bound: one read of q (x for da, dy for db).  A CTA takes one adapter and 128
// columns of da or of db; tiles of 64 rows are read as TMA left them, the
// reduction running across their rows.  p is float32 and has been split into a
// 16-bit part and a 16-bit rest, side by side as columns (2^-17 of a value is
// lost in BF16, 2^-22 in FP16), so the rest costs columns, not another pass.
// (Splitting it here, tile by tile, made the split the bound: 384 us for 8192
// rows of 8192 at rank 64.)  Blocks are 64 rows of one request; rows past its
// end are cleared in shared memory, since the next request's may hold
// infinities.  Few columns split the blocks over a cluster.  A CTA uses half of
// an SM's shared and tensor memory, so that two hide each other's ends.
//
// Measured: both gradients at 8192 rows of 8192x8192, rank 64: 66 us, 4.1 TB/s,
// 62% of the copy rate; the parts before it 10 us, and their peaks (FP16) 17 us.

struct OuterSide {
  uint64_t cols;
  uint32_t tiles;
  const uint32_t* peak;  // FP16: bits of the largest |p| of each adapter
  void* out;
  uint64_t sr, sc;       // element (r, c) of an adapter at r * sr + c * sc
  uint32_t out_vector;   // 8 ranks of a column are one aligned 16-byte store
};
struct OuterArgs {
  uint64_t rows;
  uint32_t stages, split, rank;
  const int32_t* offsets;
  const int32_t* ids;
  uint32_t count;
  const float* alpha;
  OuterSide side[2];
  int32_t* status;
  Limits limits;
};

constexpr int kOuterThreads = 320;
constexpr uint32_t kWindow = 320;  // requests looked through at a time

__host__ __device__ inline uint32_t padded(uint32_t rank) { return (rank + 7) / 8 * 8; }
// Columns of p's parts: the 16-bit values, their rests, and zeros up to whole boxes of 64.
__host__ __device__ inline uint32_t part_columns(uint32_t rank) { return (2 * padded(rank) + 63) / 64 * 64; }

// The power of two by which FP16 parts of p are taken: it brings the largest to [2^13, 2^14).
__device__ inline float unit_of(uint32_t peak) {
  const uint32_t e = peak >> 23;  // the largest is in [2^(e-127), 2^(e-126))
  return __uint_as_float((e > 14 ? 267 - e : 253) << 23);
}

template <class T>
__global__ void __launch_bounds__(kOuterThreads, 2)
    outer_tc(const __grid_constant__ CUtensorMap map_q0, const __grid_constant__ CUtensorMap map_p0,
             const __grid_constant__ CUtensorMap map_q1, const __grid_constant__ CUtensorMap map_p1,
             const __grid_constant__ OuterArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[3 * kMaxStages + 2];
  __shared__ uint32_t tmem_base;
  __shared__ int failed_s;
  __shared__ int32_t begin_s[kWindow], end_s[kWindow];
  __shared__ uint32_t warp_sum[kOuterThreads / 32];
  const Waits waits{&failed_s, a.limits.cycles};

  const uint32_t pad = padded(a.rank), n = part_columns(a.rank);
  const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
  const uint32_t q_bytes = 16384, stage_bytes = q_bytes + n * 128;
  const uint32_t full = smem_addr(bars), empty = full + 8 * kMaxStages, ready = empty + 8 * kMaxStages,
                 done = ready + 8 * kMaxStages, spent = done + 8;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t crank = a.split > 1 ? cluster_rank() : 0;
  const uint32_t tile = blockIdx.x / a.split, which = tile < a.side[0].tiles ? 0 : 1;
  const OuterSide& side = a.side[which];
  const CUtensorMap* map_q = which ? &map_q1 : &map_q0;
  const CUtensorMap* map_p = which ? &map_p1 : &map_p0;
  const uint64_t c0 = (uint64_t)(which ? tile - a.side[0].tiles : tile) * 128;
  const int32_t id = (int32_t)blockIdx.y;
  const uint32_t columns = n <= 64 ? 64 : n <= 128 ? 128 : 256;

  if (threadIdx.x == 64) {
    tma_prefetch(map_q);
    tma_prefetch(map_p);
  }
  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < a.stages; ++i) {
      mbar_init(full + 8 * i, i == 0 ? 1 + a.limits.missing : 1);
      mbar_init(empty + 8 * i, 1);
      mbar_init(ready + 8 * i, 8);
    }
    mbar_init(done, 1);
    mbar_init(spent, 1);
    failed_s = 0;
    mbar_init_fence();
  }
  if (warp == 1) {
    tmem_alloc<1>(smem_addr(&tmem_base), columns);
    tmem_release_permit<1>();
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_base;
  const uint32_t idesc = idesc_f16(Widen<T>::kBf16, 128, n) | kTransposeA | kTransposeB;

  uint32_t seen = 0, used = 0;          // blocks of the adapter so far; those of this CTA
  uint32_t s = 0, turn = 0;     // stage and parity of the next block
  bool ok = true;
  for (uint32_t w0 = 0; w0 < a.count; w0 += kWindow) {
    // this window's requests of the adapter, in order
    const uint32_t i = w0 + threadIdx.x;
    int32_t b = 0, e = 0;
    if (i < a.count && a.ids[i] == id) {
      b = max(0, a.offsets[i]);
      e = (int32_t)min((int64_t)a.offsets[i + 1], (int64_t)a.rows);
    }
    const uint32_t mask = __ballot_sync(~0u, e > b);
    if (lane == 0) warp_sum[warp] = __popc(mask);
    __syncthreads();
    uint32_t before = 0, total = 0;
    for (int w = 0; w < kOuterThreads / 32; ++w) {
      before += w < warp ? warp_sum[w] : 0;
      total += warp_sum[w];
    }
    if (e > b) {
      const uint32_t at = before + __popc(mask & ((1u << lane) - 1));
      begin_s[at] = b;
      end_s[at] = e;
    }
    __syncthreads();
    for (uint32_t k = 0; k < total && ok; ++k) {
      const uint32_t blocks = (uint32_t)(end_s[k] - begin_s[k] + 63) / 64;
      // blocks seen, seen+1, ...: those with number % split == crank are this CTA's
      for (uint32_t j = (crank + a.split - seen % a.split) % a.split; j < blocks; j += a.split) {
        const int64_t t0 = (int64_t)begin_s[k] + 64 * (int64_t)j;
        const uint32_t valid = (uint32_t)min((int64_t)64, (int64_t)end_s[k] - t0);
        const uint32_t at = base + s * stage_bytes, bar = full + 8 * s;
        if (warp == 0) {
          ok = mbar_wait_lanes(empty + 8 * s, turn ^ 1, waits);
          if (!ok) break;
          if (elect_one()) {
            mbar_expect(bar, stage_bytes);
            tma_load(at, map_q, (int32_t)c0, (int32_t)t0, bar);
            tma_load(at + 8192, map_q, (int32_t)c0 + 64, (int32_t)t0, bar);
            for (uint32_t x = 0; x < n; x += 64) tma_load(at + q_bytes + x * 128, map_p, (int32_t)x, (int32_t)t0, bar);
          }
          __syncwarp();
        } else if (warp == 1) {
          ok = mbar_wait_lanes(ready + 8 * s, turn, waits);
          if (!ok) break;
          fence_after();
          const uint64_t q = desc_mn128(at, 8192), p = desc_mn128(at + q_bytes, 8192);
          if (elect_one()) {
#pragma unroll
            for (int m = 0; m < 4; ++m) mma_ss(tmem, q + m * 128, p + m * 128, idesc, used > 0 || m > 0);
            mma_commit<1>(empty + 8 * s, 0);
          }
          __syncwarp();
        } else {
          ok = mbar_wait(bar, turn, waits);
          if (!ok) break;
          if (valid < 64) {
            // whole 128-byte rows, so the swizzle does not matter; boxes of 64 rows follow each other
            const uint32_t boxes = 2 + n / 64;
            for (uint32_t x = threadIdx.x - 64; x < (64 - valid) * boxes * 8; x += 256) {
              const uint32_t box = x / 8 % boxes, r = valid + x / 8 / boxes, to = at + box * 8192 + r * 128 + x % 8 * 16;
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(to), "r"(0) : "memory");
            }
            fence_async();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(ready + 8 * s);
        }
        ++used;
        if (++s == a.stages) s = 0, turn ^= 1;
      }
      seen += blocks;
    }
    __syncwarp();
    __syncthreads();
  }
  if (warp == 1 && used) {
    if (ok && elect_one()) mma_commit<1>(done, 0);
    __syncwarp();
  }
  T* out = static_cast<T*>(side.out) + (uint64_t)id * a.rank * side.cols;
  // an adapter without rows gets zeros, whatever its alpha
  const float alpha = seen ? a.alpha[id] / (Widen<T>::kBf16 ? 1.0f : unit_of(side.peak[id])) : 0.0f;
  if (warp >= 2) {
    const int quarter = warp % 4, half = (warp - 2) / 4;
    const uint32_t row = quarter * 32 + lane;
    const uint64_t c = c0 + row;
    if (used) {
      ok = ok && mbar_wait(done, 0, waits);
      if (ok) fence_after();
    }
    if (ok)
      for (uint32_t r0 = half * 8; r0 < pad; r0 += 16) {
        float d[8] = {}, e[8] = {};
        if (used) {
          tmem_ld8(tmem + ((uint32_t)(quarter * 32) << 16) + r0, d);
          tmem_ld8(tmem + ((uint32_t)(quarter * 32) << 16) + pad + r0, e);
        }
        if (a.split > 1) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + ((r0 + j) * 128 + row) * 4), "f"(d[j] + e[j]) : "memory");
        } else if (c < side.cols) {
          if (side.out_vector) {
            uint4 v;
            v.x = Widen<T>::pack((d[0] + e[0]) * alpha, (d[1] + e[1]) * alpha);
            v.y = Widen<T>::pack((d[2] + e[2]) * alpha, (d[3] + e[3]) * alpha);
            v.z = Widen<T>::pack((d[4] + e[4]) * alpha, (d[5] + e[5]) * alpha);
            v.w = Widen<T>::pack((d[6] + e[6]) * alpha, (d[7] + e[7]) * alpha);
            *reinterpret_cast<uint4*>(out + c * side.sc + r0) = v;
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (r0 + j < a.rank) put(out + (r0 + j) * side.sr + c * side.sc, (d[j] + e[j]) * alpha);
          }
        }
      }
  }
  if (a.split > 1) {
    __syncwarp();
    cluster_sync();
    if (warp >= 2 && !failed_s) {
      const uint32_t k = threadIdx.x - 64, row = k % 32 * 4;
      const uint64_t c = c0 + row;
      const uint32_t lo = a.rank * crank / a.split, hi = a.rank * (crank + 1) / a.split;
      for (uint32_t r = lo + k / 32; r < hi; r += 8) {
        const float4 d = cluster_sum4(base + (r * 128 + row) * 4, a.split);
        const float y[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (c + q < side.cols) put(out + r * side.sr + (c + q) * side.sc, y[q] * alpha);
      }
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while another reads its sums
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (failed_s) {
    if (warp == 0) drain_loads(full, s, turn, a.stages, waits);
    if (warp == 1) drain_products<1>(spent, 0, waits);
  }
  if (warp == 1) tmem_free<1>(tmem, columns);
  if (threadIdx.x == 0 && failed_s && a.status) atomicOr(a.status, ECF8_STATUS_TIMEOUT);
}

// v (blockIdx.y = 0) and u (1), either of which may be absent: what is read, and what is written of it.
struct PartsArgs {
  const float* p[2];
  uint32_t* peak[2];
  void* parts[2];
  uint64_t rows;
  uint32_t rank;
  const int32_t* row_id;
};

// peak[a] = bits of the largest finite |p| of adapter a's rows; peak starts at zero.  The order of the maxima does not
// matter.
__global__ void __launch_bounds__(256) peak_kernel(PartsArgs a) {
  const float* p = a.p[blockIdx.y];
  if (!p) return;
  const uint64_t warps = (uint64_t)gridDim.x * 8;
  for (uint64_t t = blockIdx.x * 8 + threadIdx.x / 32; t < a.rows; t += warps) {
    const int32_t id = a.row_id[t];
    if (id < 0) continue;
    float m = 0;
    for (uint32_t r = threadIdx.x % 32; r < a.rank; r += 32) {
      const float v = fabsf(p[t * a.rank + r]);
      if (isfinite(v)) m = fmaxf(m, v);
    }
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
    if (threadIdx.x % 32 == 0 && m > 0) atomicMax(a.peak[blockIdx.y] + id, __float_as_uint(m));
  }
}

// parts[t] = p[t] as 16-bit values, their rests and zeros; FP16 takes p times its adapter's power of two.
template <class T>
__global__ void __launch_bounds__(256) parts_kernel(PartsArgs a) {
  const float* p = a.p[blockIdx.y];
  if (!p) return;
  const uint32_t pad = padded(a.rank), pairs = part_columns(a.rank) / 2;
  uint32_t* out = static_cast<uint32_t*>(a.parts[blockIdx.y]);
  const uint64_t total = a.rows * pairs, step = (uint64_t)gridDim.x * 256;
  for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < total; i += step) {
    const uint64_t t = i / pairs;
    const uint32_t c = (uint32_t)(i % pairs) * 2, r = c < pad ? c : c - pad;
    const int32_t id = a.row_id[t];
    uint32_t hi = 0, lo = 0;
    if (id >= 0 && c < 2 * pad) {
      const float unit = Widen<T>::kBf16 ? 1.0f : unit_of(a.peak[blockIdx.y][id]);
      const float x = r < a.rank ? p[t * a.rank + r] * unit : 0.0f;
      const float y = r + 1 < a.rank ? p[t * a.rank + r + 1] * unit : 0.0f;
      split_pair<T>(x, y, hi, lo);
    }
    out[i] = c < pad ? hi : lo;
  }
}

// out[a][.] = alpha[a] * sum over a's rows of p[t][r] q[t][c], element (r, c) at r * sr + c * sc.
// One CTA an adapter, 128 columns and 8 ranks; rows in order.
template <class T>
__global__ void __launch_bounds__(128) outer_simple(const float* p, uint32_t rank, const T* q, uint64_t q_stride,
                                                    uint64_t cols, const int32_t* offsets, const int32_t* ids,
                                                    uint32_t count, uint64_t rows, const float* alpha, T* out,
                                                    uint64_t f_adapter, uint64_t sr, uint64_t sc) {
  const uint64_t c = (uint64_t)blockIdx.x * 128 + threadIdx.x;
  const uint32_t r0 = blockIdx.y * 8, nr = min(8u, rank - r0);
  const int32_t a = (int32_t)blockIdx.z;
  float acc[8] = {};
  bool any = false;
  for (uint32_t i = 0; i < count; ++i) {
    if (ids[i] != a) continue;
    const int64_t b = max(0, offsets[i]), e = min((int64_t)offsets[i + 1], (int64_t)rows);
    any |= e > b;
    if (c < cols)
      for (int64_t t = b; t < e; ++t) {
        const float x = to_float(q[(uint64_t)t * q_stride + c]);
#pragma unroll
        for (uint32_t r = 0; r < 8; ++r)
          if (r < nr) acc[r] = fmaf(x, p[(uint64_t)t * rank + r0 + r], acc[r]);
      }
  }
  if (c < cols)
#pragma unroll
    for (uint32_t r = 0; r < 8; ++r)
      if (r < nr) put(out + (uint64_t)a * f_adapter + (r0 + r) * sr + c * sc, any ? alpha[a] * acc[r] : 0.0f);
}

#ifdef ECF8_CHECKED
Limits g_limits[3];  // of the projection, the adapters' first product, their gradients
Limits limits_of(int kernel) { return g_limits[kernel]; }
#else
Limits limits_of(int) { return Limits{}; }
#endif

constexpr uint64_t kGridY = 65535;
constexpr uint64_t kMost = 1ull << 31;  // rows, columns and adapters stay below it

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

bool aligned(const void* p, uint64_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// Whether TMA can read rows of `width`-byte values from here.
bool tma_rows(const void* p, uint64_t stride, uint64_t width) { return aligned(p, 16) && stride * width % 16 == 0; }

// The workspace: sections of a call of this many rows.  Operands whose rows TMA cannot read have a place for a copy
// (x and dy by their length alone: that of rows without gaps).
struct Plan {
  size_t row_id, p, turned, peak, parts, copies, total;
  uint64_t w_stride, x_stride, dy_stride, a_stride, b_stride;  // rows of the copies, in values
  size_t w, x, dy, a;
};

uint64_t up(uint64_t n, uint64_t to) { return (n + to - 1) / to * to; }

Plan plan_of(const ecf8_linear* lin, uint64_t rows) {
  Plan w{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t from = at;
    at += up256(bytes);
    return from;
  };
  w.w_stride = up(lin->k_in, 16);
  w.x_stride = w.a_stride = up(lin->k_in, 8);
  w.dy_stride = w.b_stride = up(lin->n_out, 8);
  const uint64_t factors = (uint64_t)lin->n_adapters * lin->rank;
  if (lin->n_adapters) {
    w.row_id = take(rows * 4);
    w.p = take(rows * lin->rank * 4);
    w.turned = take(factors * w.b_stride * 2);
    w.peak = take((size_t)lin->n_adapters * 8);
    w.parts = take(2 * up256(rows * part_columns(lin->rank) * 2));
  }
  w.copies = at;
  w.w = take(tma_rows(lin->d_w, lin->w_stride, 1) ? 0 : lin->n_out * w.w_stride);
  w.x = take(lin->k_in % 8 ? rows * w.x_stride * 2 : 0);
  w.dy = take(lin->n_out % 8 ? rows * w.dy_stride * 2 : 0);
  if (lin->n_adapters) w.a = take(tma_rows(lin->d_a, lin->k_in, 2) ? 0 : factors * w.a_stride * 2);
  w.total = at;
  return w;
}

int check(const ecf8_linear* l, const ecf8_requests* q, uint64_t rows, const void* ws, size_t ws_bytes,
          const int32_t* d_status) {
  if (!l) return ECF8_ERR_ARG;
  if (l->dtype != ECF8_DTYPE_BF16 && l->dtype != ECF8_DTYPE_FP16) return ECF8_ERR_ARG;
  if (!l->n_out || !l->k_in || l->n_out >= kMost || l->k_in >= kMost || rows >= kMost) return ECF8_ERR_ARG;
  if (l->w_stride < l->k_in || l->w_stride >= kMost * 64) return ECF8_ERR_ARG;
  if (l->n_scale != 0 && l->n_scale != 1 && l->n_scale != l->n_out) return ECF8_ERR_ARG;
  if (!l->d_w || (l->n_scale && !l->d_scale)) return ECF8_ERR_ARG;
  if (((uintptr_t)l->d_scale | (uintptr_t)d_status) & 3) return ECF8_ERR_ALIGN;
  if (l->n_adapters) {
    if (l->n_adapters >= 65536 || l->rank < 1 || l->rank > ECF8_RANK_MAX) return ECF8_ERR_ARG;
    if (!l->d_a || !l->d_b || !l->d_alpha) return ECF8_ERR_ARG;
    if ((((uintptr_t)l->d_a | (uintptr_t)l->d_b) & 1) || ((uintptr_t)l->d_alpha & 3)) return ECF8_ERR_ALIGN;
    if (q && q->count) {
      if (q->count >= kMost || !q->d_offsets || !q->d_ids) return ECF8_ERR_ARG;
      if (((uintptr_t)q->d_offsets | (uintptr_t)q->d_ids) & 3) return ECF8_ERR_ALIGN;
    }
  }
  // without adapters a workspace is for copies alone, and none means no copies
  const size_t need = plan_of(l, rows).total;
  if (ws ? ws_bytes < need : l->n_adapters && need) return ECF8_ERR_WORKSPACE;
  if ((uintptr_t)ws & 15) return ECF8_ERR_ALIGN;
  return ECF8_OK;
}

void route(const ecf8_linear* l, const ecf8_requests* q, uint64_t rows, int32_t* row_id, int32_t* d_status,
           cudaStream_t s) {
  const uint64_t most = rows > q->count ? rows : q->count;
  const unsigned grid = (unsigned)((most + 255) / 256 < 1024 ? (most + 255) / 256 : 1024);
  route_kernel<<<grid, 256, 0, s>>>(q->d_offsets, q->d_ids, q->count, l->n_adapters, rows, row_id, d_status);
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// A map of `rows` rows of `cols` values, `stride` bytes apart, read in boxes of box_rows x box_cols.
bool make_map(CUtensorMap* map, CUtensorMapDataType type, const void* at, uint64_t cols, uint64_t rows,
              uint64_t stride, uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swizzle) {
  const EncodeTiled fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {stride};
  const cuuint32_t box[2] = {box_cols, box_rows}, step[2] = {1, 1};
  return fn(map, type, 2, const_cast<void*>(at), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Where a call's operands are read from: themselves, or copies whose rows TMA can read.
struct Operands {
  ecf8_linear l;         // the weight in place of the caller's
  const void* a;         // A, rows a_stride apart
  uint64_t a_stride;
  const void *x, *dy;
  uint64_t x_stride, dy_stride;
  bool weight, factor;   // TMA can read the weight, A
};

bool small_enough(const ecf8_linear& l) { return l.k_in < (1u << 24) && l.n_out < (1u << 24); }

// Copies what has to be copied and can be.
template <class T>
int lay_out(const ecf8_linear* l, const Plan& w, char* ws, const void* x, uint64_t x_stride, const void* dy,
            uint64_t dy_stride, uint64_t rows, bool use_a, Operands* o, cudaStream_t s) {
  *o = Operands{*l, l->d_a, l->k_in, x, dy, x_stride, dy_stride, tma_rows(l->d_w, l->w_stride, 1),
                use_a && tma_rows(l->d_a, l->k_in, 2)};
  if (!ws || !small_enough(*l)) return ECF8_OK;
  Restride r{};
  int n = 0;
  auto copy = [&](const void* from, uint64_t n_rows, uint64_t len, uint64_t stride, size_t to, uint64_t to_stride,
                  uint64_t width) -> void* {
    r.from[n] = static_cast<const uint8_t*>(from);
    r.to[n] = reinterpret_cast<uint8_t*>(ws + to);
    r.rows[n] = n_rows;
    r.bytes[n] = len * width;
    r.stride[n] = stride * width;
    r.to_stride[n] = to_stride * width;
    return r.to[n++];
  };
  if (!o->weight) {
    o->l.d_w = static_cast<const uint8_t*>(copy(l->d_w, l->n_out, l->k_in, l->w_stride, w.w, w.w_stride, 1));
    o->l.w_stride = w.w_stride;
    o->weight = true;
  }
  if (x && l->k_in % 8 && !tma_rows(x, x_stride, 2)) {
    o->x = copy(x, rows, l->k_in, x_stride, w.x, w.x_stride, 2);
    o->x_stride = w.x_stride;
  }
  if (dy && l->n_out % 8 && !tma_rows(dy, dy_stride, 2)) {
    o->dy = copy(dy, rows, l->n_out, dy_stride, w.dy, w.dy_stride, 2);
    o->dy_stride = w.dy_stride;
  }
  if (use_a && !o->factor && n < 3) {
    o->a = copy(l->d_a, (uint64_t)l->n_adapters * l->rank, l->k_in, l->k_in, w.a, w.a_stride, 2);
    o->a_stride = w.a_stride;
    o->factor = true;
  }
  if (n) {
    uint64_t most = 0;
    for (int i = 0; i < n; ++i) most = most > r.rows[i] * r.to_stride[i] ? most : r.rows[i] * r.to_stride[i];
    const uint64_t blocks = (most / 16 + 255) / 256;
    restride_kernel<<<dim3((unsigned)(blocks < 1184 ? blocks : 1184), n), 256, 0, s>>>(r);
  }
  return ECF8_OK;
}

bool tensor_path(const Operands& o, const void* q, uint64_t q_stride) {
  return o.weight && small_enough(o.l) && tma_rows(q, q_stride, 2);
}

// Two CTAs to a tile of 256 columns where such tiles occupy half of the 148 SMs at least; else single ones, two to an
// SM, on tiles of at most 128 rows, which give more CTAs before the reduction has to be split (256 rows of 1024x4096
// backward: 29 us in pairs, 16 us so; 200 rows of 4096x4096: 33 and 21).
bool in_pairs(uint64_t rows, uint64_t cols) { return rows > 128 && (cols + 255) / 256 * ((rows + 255) / 256) >= 37; }

template <class T, int BACK>
int product_tensor(const ecf8_linear* l, bool adapted, const void* in, uint64_t in_stride, void* out,
                   uint64_t out_stride, uint64_t rows, const int32_t* row_id, const float* p, bool overlap,
                   int32_t* d_status, cudaStream_t s) {
  const uint64_t cols = BACK ? l->k_in : l->n_out, len = BACK ? l->n_out : l->k_in;
  ProductArgs a{};
  a.rows = rows;
  a.cols = cols;
  a.len = len;
  const bool pair = in_pairs(rows, cols);
  const uint64_t tall = pair ? 256 : 128;
  a.bt = (uint32_t)(rows >= tall ? tall : (rows + 15) / 16 * 16);
  const int kb = pair ? 1 : 2, width = pair ? 2 : 1;
  a.blocks = (uint32_t)((len + 64 * kb - 1) / (64 * kb));
  const uint64_t tiles = (cols + 128 * width - 1) / (128 * width), row_tiles = (rows + a.bt - 1) / a.bt;
  if (row_tiles > kGridY) return ECF8_ERR_UNSUPPORTED;
  // Enough CTAs to keep every SM loading, while each still has a few steps to pipeline.  (Pairs are taken where they need
  // no split.)
  a.split = 1;
  while (!pair && a.split < 8 && tiles * row_tiles * a.split * 2 <= 296 && a.blocks / (a.split * 2) >= 2) a.split *= 2;
  const uint32_t here = a.bt / width, stage = 8192 * kb + here * 128 * kb;
  const uint32_t room = (pair ? 216 * 1024 : 106 * 1024) - 1024;
  const uint32_t fit = room / stage, at_most = pair ? kSlots : kMaxStages;
  a.stages = fit < at_most ? fit : at_most;
  size_t smem = (size_t)a.stages * stage + 1024;
  const size_t sums = (size_t)a.bt * 512 + 1024;
  if (a.split > 1 && smem < sums) smem = sums;
  a.scale = l->d_scale;
  a.n_scale = l->n_scale;
  a.row_id = row_id;
  a.p = p;
  a.f = BACK ? l->d_a : l->d_b;
  a.f_adapter = (uint64_t)l->rank * cols;
  a.sr = BACK ? l->k_in : 1;
  a.sc = BACK ? 1 : l->rank;
  a.alpha = l->d_alpha;
  a.rank = adapted ? l->rank : 0;
  a.f_vector = !BACK && l->rank % 8 == 0 && aligned(l->d_b, 16);
  a.p_vector = l->rank % 4 == 0 && aligned(p, 16);
  a.out = out;
  a.out_stride = out_stride;
  a.out_vector = aligned(out, 8) && out_stride % 4 == 0 && cols % 4 == 0;
  a.status = d_status;
  a.limits = limits_of(0);
  const CUtensorMapDataType type =
      Widen<T>::kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap mw, mq;
  const bool made =
      (BACK ? make_map(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, l->d_w, l->k_in, l->n_out, l->w_stride, 128, 64 * kb,
                       CU_TENSOR_MAP_SWIZZLE_NONE)
            : make_map(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, l->d_w, l->k_in, l->n_out, l->w_stride, 64 * kb, 128,
                       kb == 2 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B)) &&
      make_map(&mq, type, in, len, rows, in_stride * 2, 64, here, CU_TENSOR_MAP_SWIZZLE_128B);
  if (!made) return ECF8_ERR_CUDA;
  const dim3 grid((unsigned)(tiles * width * a.split), (unsigned)row_tiles);
  return product_launch<T, BACK>(pair, mw, mq, a, grid, smem, overlap, s);
}

// p = q f^T for every row's own adapter; f is n_adapters x rank rows of `len` values, f_stride apart.
template <class T>
int shrink_tensor(const T* q, uint64_t q_stride, uint64_t rows, const T* f, uint64_t f_stride, uint64_t len,
                  uint32_t n_adapters, uint32_t rank, const ecf8_requests* req, int32_t* row_id, float* p,
                  int32_t* d_status, cudaStream_t s) {
  static bool set[64] = {};
  if (const int rc = allow_smem(shrink_tc<T>, set)) return rc;
  ShrinkArgs a{};
  a.rows = rows;
  a.blocks = (uint32_t)((len + 63) / 64);
  a.rank = rank;
  a.per = 128 / ((rank + 7) / 8 * 8);
  // The largest tiles (q's rows against the adapters' are what is read again) that still give every SM a CTA once
  // the reduction is split, which leaves a CTA two steps at least.
  uint64_t chunks, row_tiles;
  for (a.bt = 256;; a.bt /= 2) {
    const uint64_t most = n_adapters < a.bt ? n_adapters : a.bt;
    chunks = (most + a.per - 1) / a.per;
    row_tiles = (rows + a.bt - 1) / a.bt;
    a.split = 1;
    while (a.split < 8 && chunks * row_tiles * a.split * 2 <= 148 && a.blocks / (a.split * 2) >= 2) a.split *= 2;
    if (a.bt == 32 || chunks * row_tiles * a.split > 74) break;
  }
  if (rows < a.bt) a.bt = (uint32_t)((rows + 15) / 16 * 16);
  if (row_tiles > kGridY) return ECF8_ERR_UNSUPPORTED;
  const uint32_t stage = 16384 + a.bt * 128;
  // small tiles leave room for a CTA of the projection beside them
  a.stages = a.bt <= 64 ? 4 : 216 * 1024 / stage < 8 ? 216 * 1024 / stage : 8;
  size_t smem = (size_t)a.stages * stage + 1024;
  const size_t sums = (size_t)a.bt * 512 + 1024;
  if (a.split > 1 && smem < sums) smem = sums;
  a.offsets = req->d_offsets;
  a.request_ids = req->d_ids;
  a.count = req->count;
  a.n_adapters = n_adapters;
  a.row_id = row_id;
  a.p = p;
  a.status = d_status;
  a.limits = limits_of(1);
  const CUtensorMapDataType type =
      Widen<T>::kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap mf, mq;
  if (!make_map(&mf, type, f, len, (uint64_t)n_adapters * rank, f_stride * 2, 64, rank,
                CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&mq, type, q, len, rows, q_stride * 2, 64, a.bt, CU_TENSOR_MAP_SWIZZLE_128B))
    return ECF8_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(chunks * a.split), (unsigned)row_tiles);
  cfg.blockDim = dim3(kShrinkThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, shrink_tc<T>, mf, mq, a) == cudaSuccess ? ECF8_OK : ECF8_ERR_CUDA;
}

// One of the two gradients: out[a] = alpha[a] * sum over a's rows of p[t] q[t].
struct Outer {
  const void* q;
  uint64_t q_stride, cols;
  const float* p;
  void* out;
  uint64_t sr, sc;
};

template <class T>
int outer_tensor(const Outer* sides, int n_sides, uint32_t rank, uint32_t n_adapters, const ecf8_requests* req,
                 uint64_t rows, const int32_t* row_id, uint32_t* peak, char* parts, const float* alpha,
                 int32_t* d_status, cudaStream_t s) {
  static bool set[64] = {};
  if (const int rc = allow_smem(outer_tc<T>, set)) return rc;
  const CUtensorMapDataType type =
      Widen<T>::kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const uint32_t columns = part_columns(rank);
  const size_t part_bytes = up256(rows * columns * 2);
  OuterArgs a{};
  a.rows = rows;
  a.rank = rank;
  a.offsets = req->d_offsets;
  a.ids = req->d_ids;
  a.count = req->count;
  a.alpha = alpha;
  a.status = d_status;
  a.limits = limits_of(2);
  PartsArgs b{};
  b.rows = rows;
  b.rank = rank;
  b.row_id = row_id;
  CUtensorMap maps[4];
  uint64_t tiles = 0;
  for (int i = 0; i < n_sides; ++i) {
    const Outer& o = sides[i];
    OuterSide& d = a.side[i];
    d.cols = o.cols;
    d.tiles = (uint32_t)((o.cols + 127) / 128);
    d.peak = peak + i * n_adapters;
    d.out = o.out;
    d.sr = o.sr;
    d.sc = o.sc;
    d.out_vector = o.sr == 1 && rank % 8 == 0 && aligned(o.out, 16);
    tiles += d.tiles;
    b.p[i] = o.p;
    b.peak[i] = peak + i * n_adapters;
    b.parts[i] = parts + i * part_bytes;
    if (!make_map(&maps[2 * i], type, o.q, o.cols, rows, o.q_stride * 2, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&maps[2 * i + 1], type, b.parts[i], columns, rows, columns * 2, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B))
      return ECF8_ERR_CUDA;
  }
  for (int i = n_sides; i < 2; ++i) maps[2 * i] = maps[0], maps[2 * i + 1] = maps[1];
  if (!Widen<T>::kBf16) {
    if (cudaMemsetAsync(peak, 0, (size_t)n_adapters * 8, s) != cudaSuccess) return ECF8_ERR_CUDA;
    peak_kernel<<<dim3((unsigned)((rows + 7) / 8 < 592 ? (rows + 7) / 8 : 592), n_sides), 256, 0, s>>>(b);
  }
  const uint64_t blocks = (rows * columns / 2 + 255) / 256;
  parts_kernel<T><<<dim3((unsigned)(blocks < 1184 ? blocks : 1184), n_sides), 256, 0, s>>>(b);
  a.split = 1;
  while (a.split < 8 && tiles * n_adapters * a.split * 2 <= 296 && rows / (64 * a.split * 2) >= 2) a.split *= 2;
  const uint32_t stage = 16384 + columns * 128;
  a.stages = 106 * 1024 / stage < kMaxStages ? 106 * 1024 / stage : kMaxStages;
  const size_t smem = (size_t)a.stages * stage + 1024;  // at least the sums, 512 bytes a rank
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(tiles * a.split), n_adapters);
  cfg.blockDim = dim3(kOuterThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, outer_tc<T>, maps[0], maps[1], maps[2], maps[3], a) == cudaSuccess ? ECF8_OK
                                                                                                     : ECF8_ERR_CUDA;
}

template <class T, int BACK>
int product(const Operands& o, bool adapted, const void* in, uint64_t in_stride, void* out, uint64_t out_stride,
            uint64_t rows, const int32_t* row_id, const float* p, bool overlap, int32_t* d_status, cudaStream_t s) {
  const ecf8_linear* l = &o.l;
  if (tensor_path(o, in, in_stride))
    return product_tensor<T, BACK>(l, adapted, in, in_stride, out, out_stride, rows, row_id, p, overlap, d_status, s);
  const uint64_t cols = BACK ? l->k_in : l->n_out, len = BACK ? l->n_out : l->k_in;
  const uint64_t step = kGridY * 64;
  for (uint64_t t = 0; t < rows; t += step) {
    const uint64_t n = rows - t < step ? rows - t : step;
    product_simple<T, BACK><<<dim3((unsigned)((cols + 63) / 64), (unsigned)((n + 63) / 64)), 256, 0, s>>>(
        static_cast<const T*>(in) + t * in_stride, in_stride, l->d_w, l->w_stride, l->d_scale, l->n_scale, n, cols, len,
        row_id + t, p + t * l->rank, static_cast<const T*>(BACK ? l->d_a : l->d_b),
        (uint64_t)l->rank * cols, BACK ? l->k_in : 1, BACK ? 1 : l->rank, l->d_alpha, adapted ? l->rank : 0,
        static_cast<T*>(out) + t * out_stride, out_stride);
  }
  return ECF8_OK;
}

template <class T>
int forward(const ecf8_linear* l, const ecf8_requests* q, const void* x, uint64_t x_stride, void* y, uint64_t y_stride,
            uint64_t rows, float* u, char* ws, int32_t* d_status, cudaStream_t s) {
  const bool adapted = l->n_adapters && q && q->count;
  const Plan w = plan_of(l, rows);
  int32_t* row_id = reinterpret_cast<int32_t*>(ws);
  const bool keep = u != nullptr;
  bool overlap = false;  // the projection may start beside the kernel before it
  if (l->n_adapters && !u) u = reinterpret_cast<float*>(ws + w.p);
  Operands o;
  if (const int rc = lay_out<T>(l, w, ws, x, x_stride, nullptr, 0, rows, adapted, &o, s)) return rc;
  if (adapted) {
    if (tensor_path(o, o.x, o.x_stride) && o.factor) {
      const int rc = shrink_tensor<T>(static_cast<const T*>(o.x), o.x_stride, rows, static_cast<const T*>(o.a), o.a_stride,
                                      l->k_in, l->n_adapters, l->rank, q, row_id, u, d_status, s);
      if (rc) return rc;
      overlap = true;
    } else {
      route(l, q, rows, row_id, d_status, s);
      shrink_simple<T><<<dim3((unsigned)rows, (l->rank + 7) / 8), 128, 0, s>>>(
          static_cast<const T*>(x), x_stride, static_cast<const T*>(l->d_a), l->rank * l->k_in, l->k_in, 1, l->k_in,
          l->rank, row_id, u);
    }
  } else if (l->n_adapters && keep) {
    if (cudaMemsetAsync(u, 0, rows * l->rank * 4, s) != cudaSuccess) return ECF8_ERR_CUDA;
  }
  const int rc = product<T, 0>(o, adapted, o.x, o.x_stride, y, y_stride, rows, row_id, u, overlap, d_status, s);
  if (rc) return rc;
  return cudaGetLastError() == cudaSuccess ? ECF8_OK : ECF8_ERR_CUDA;
}

template <class T>
int backward(const ecf8_linear* l, const ecf8_requests* q, const void* x, uint64_t x_stride, const void* dy,
             uint64_t dy_stride, const float* u, void* dx, uint64_t dx_stride, void* da, void* db, uint64_t rows,
             char* ws, int32_t* d_status, cudaStream_t s) {
  const bool adapted = l->n_adapters && q && q->count && rows;
  const Plan w = plan_of(l, rows);
  int32_t* row_id = reinterpret_cast<int32_t*>(ws);
  float* v = reinterpret_cast<float*>(ws + w.p);
  bool overlap = false;
  Operands o;
  if (rows)
    if (const int rc = lay_out<T>(l, w, ws, da ? x : nullptr, x_stride, dy, dy_stride, rows, false, &o, s)) return rc;
  if (adapted && (dx || da)) {
    if (tensor_path(o, o.dy, o.dy_stride)) {
      T* turned = reinterpret_cast<T*>(ws + w.turned);
      transpose_kernel<T><<<dim3((unsigned)((l->n_out + 63) / 64), l->n_adapters), 256, 0, s>>>(
          static_cast<const T*>(l->d_b), turned, l->n_out, w.b_stride, l->rank);
      const int rc = shrink_tensor<T>(static_cast<const T*>(o.dy), o.dy_stride, rows, turned, w.b_stride, l->n_out,
                                      l->n_adapters, l->rank, q, row_id, v, d_status, s);
      if (rc) return rc;
      overlap = true;
    } else {
      route(l, q, rows, row_id, d_status, s);
      shrink_simple<T><<<dim3((unsigned)rows, (l->rank + 7) / 8), 128, 0, s>>>(
          static_cast<const T*>(dy), dy_stride, static_cast<const T*>(l->d_b), l->n_out * l->rank, 1, l->rank,
          l->n_out, l->rank, row_id, v);
    }
  } else if (adapted) {
    route(l, q, rows, row_id, d_status, s);
  }
  if (dx && rows) {
    const int rc = product<T, 1>(o, adapted, o.dy, o.dy_stride, dx, dx_stride, rows, row_id, v, overlap, d_status, s);
    if (rc) return rc;
  }
  const uint32_t count = adapted ? q->count : 0;
  const int32_t* offsets = adapted ? q->d_offsets : nullptr;
  const int32_t* ids = adapted ? q->d_ids : nullptr;
  const Outer sides[2] = {{rows ? o.x : x, rows ? o.x_stride : x_stride, l->k_in, v, da, l->k_in, 1},
                          {rows ? o.dy : dy, rows ? o.dy_stride : dy_stride, l->n_out, u, db, 1, l->rank}};
  Outer fast[2];
  int n_fast = 0;
  for (const Outer& side : sides) {
    if (!side.out) continue;
    if (adapted && tensor_path(o, side.q, side.q_stride)) {
      fast[n_fast++] = side;
      continue;
    }
    outer_simple<T><<<dim3((unsigned)((side.cols + 127) / 128), (l->rank + 7) / 8, l->n_adapters), 128, 0, s>>>(
        side.p, l->rank, static_cast<const T*>(side.q), side.q_stride, side.cols, offsets, ids, count, rows,
        l->d_alpha, static_cast<T*>(side.out), l->rank * side.cols, side.sr, side.sc);
  }
  if (n_fast) {
    const int rc = outer_tensor<T>(fast, n_fast, l->rank, l->n_adapters, q, rows, row_id,
                                   reinterpret_cast<uint32_t*>(ws + w.peak), ws + w.parts, l->d_alpha, d_status, s);
    if (rc) return rc;
  }
  return cudaGetLastError() == cudaSuccess ? ECF8_OK : ECF8_ERR_CUDA;
}

}  // namespace

extern "C" {

#ifdef ECF8_CHECKED
// For tests, in this build only: the limit of the waits of one kind of kernel (0 the projection, 1 the adapters' first
// product, 2 their gradients), and arrivals that the first load's barrier waits for in vain.
void ecf8_checked_limits(int kernel, long long cycles, uint32_t missing) {
  g_limits[kernel] = cycles ? Limits{cycles, missing} : Limits{};
}
#endif

size_t ecf8_linear_workspace_size(const ecf8_linear* lin, uint64_t rows) {
  return lin && rows < kMost ? plan_of(lin, rows).total : 0;
}

int ecf8_linear_tile_ctas(const ecf8_linear* lin, uint64_t rows, int backward) {
  if (!lin || !rows || rows >= kMost) return 0;
  return in_pairs(rows, backward ? lin->k_in : lin->n_out) ? 2 : 1;
}

int ecf8_linear_forward(const ecf8_linear* lin, const ecf8_requests* requests, const void* d_x, uint64_t x_stride,
                        void* d_y, uint64_t y_stride, uint64_t rows, float* d_u, void* d_workspace,
                        size_t workspace_bytes, int32_t* d_status, cudaStream_t s) {
  const int rc = check(lin, requests, rows, d_workspace, workspace_bytes, d_status);
  if (rc) return rc;
  if (!rows) return ECF8_OK;
  if (!d_x || !d_y) return ECF8_ERR_ARG;
  if (x_stride < lin->k_in || y_stride < lin->n_out || x_stride >= kMost * 64 || y_stride >= kMost * 64)
    return ECF8_ERR_ARG;
  if ((((uintptr_t)d_x | (uintptr_t)d_y) & 1) || ((uintptr_t)d_u & 3)) return ECF8_ERR_ALIGN;
  char* ws = static_cast<char*>(d_workspace);
  return lin->dtype == ECF8_DTYPE_BF16
             ? forward<__nv_bfloat16>(lin, requests, d_x, x_stride, d_y, y_stride, rows, d_u, ws, d_status, s)
             : forward<__half>(lin, requests, d_x, x_stride, d_y, y_stride, rows, d_u, ws, d_status, s);
}

int ecf8_linear_backward(const ecf8_linear* lin, const ecf8_requests* requests, const void* d_x, uint64_t x_stride,
                         const void* d_dy, uint64_t dy_stride, const float* d_u, void* d_dx, uint64_t dx_stride,
                         void* d_da, void* d_db, uint64_t rows, void* d_workspace, size_t workspace_bytes,
                         int32_t* d_status, cudaStream_t s) {
  const int rc = check(lin, requests, rows, d_workspace, workspace_bytes, d_status);
  if (rc) return rc;
  if (!lin->n_adapters && (d_da || d_db)) return ECF8_ERR_ARG;
  if (rows) {
    if (!d_dy || (d_da && !d_x) || (d_db && !d_u)) return ECF8_ERR_ARG;
    if (dy_stride < lin->n_out || dy_stride >= kMost * 64) return ECF8_ERR_ARG;
    if (d_da && (x_stride < lin->k_in || x_stride >= kMost * 64)) return ECF8_ERR_ARG;
    if (d_dx && (dx_stride < lin->k_in || dx_stride >= kMost * 64)) return ECF8_ERR_ARG;
  }
  if ((((uintptr_t)d_x | (uintptr_t)d_dy | (uintptr_t)d_dx | (uintptr_t)d_da | (uintptr_t)d_db) & 1) ||
      ((uintptr_t)d_u & 3))
    return ECF8_ERR_ALIGN;
  char* ws = static_cast<char*>(d_workspace);
  return lin->dtype == ECF8_DTYPE_BF16
             ? backward<__nv_bfloat16>(lin, requests, d_x, x_stride, d_dy, dy_stride, d_u, d_dx, dx_stride, d_da, d_db,
                                       rows, ws, d_status, s)
             : backward<__half>(lin, requests, d_x, x_stride, d_dy, dy_stride, d_u, d_dx, dx_stride, d_da, d_db, rows,
                                ws, d_status, s);
}

}  // extern "C"
