// Linear layers over decoded E4M3 weights, with low-rank adapters: forward and
// backward, for any size, stride and alignment.
//
//     forward   u[t] = A[a] x[t]            y[t] = s * (W x[t]) + alpha[a] * B[a] u[t]
//     backward  v[t] = B[a]^T dy[t]        dx[t] = W^T (s * dy[t]) + alpha[a] * A[a]^T v[t]
//               da[a] = alpha[a] * sum_t v[t] x[t]^T      db[a] = alpha[a] * sum_t dy[t] u[t]^T
//
// with a the adapter of row t's request.  u and v stay in float32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "ecf8.h"

namespace {

__device__ inline float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ inline float to_float(__half v) { return __half2float(v); }
__device__ inline void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ inline void put(__half* p, float v) { *p = __float2half_rn(v); }

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
  for (uint32_t i = 0; i < count; ++i) {
    if (ids[i] != a) continue;
    const int64_t b = max(0, offsets[i]), e = min((int64_t)offsets[i + 1], (int64_t)rows);
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
      if (r < nr) put(out + (uint64_t)a * f_adapter + (r0 + r) * sr + c * sc, alpha[a] * acc[r]);
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

struct Plan {
  size_t row_id, p, total;
};

Plan plan_of(const ecf8_linear* lin, uint64_t rows) {
  Plan w{};
  if (!lin->n_adapters) return w;
  w.p = up256(rows * 4);
  w.total = w.p + up256(rows * lin->rank * 4);
  return w;
}

constexpr uint64_t kMost = 1ull << 31;  // rows, columns and adapters stay below it

int check(const ecf8_linear* l, const ecf8_requests* q, uint64_t rows, const void* ws, size_t ws_bytes,
          const int32_t* d_status) {
  if (!l) return ECF8_ERR_ARG;
  if (l->dtype != ECF8_DTYPE_BF16 && l->dtype != ECF8_DTYPE_FP16) return ECF8_ERR_ARG;
  if (!l->n_out || !l->k_in || l->n_out >= kMost || l->k_in >= kMost || rows >= kMost) return ECF8_ERR_ARG;
  if (l->w_stride < l->k_in || l->w_stride >= kMost * 64) return ECF8_ERR_ARG;
  if (l->n_scale != 0 && l->n_scale != 1 && l->n_scale != l->n_out) return ECF8_ERR_ARG;
  if (!l->d_w || (l->n_scale && !l->d_scale)) return ECF8_ERR_ARG;
  if (((uintptr_t)l->d_scale | (uintptr_t)d_status) & 3) return ECF8_ERR_ALIGN;
  if (!l->n_adapters) return ECF8_OK;
  if (l->n_adapters >= 65536 || l->rank < 1 || l->rank > ECF8_RANK_MAX) return ECF8_ERR_ARG;
  if (!l->d_a || !l->d_b || !l->d_alpha) return ECF8_ERR_ARG;
  if ((((uintptr_t)l->d_a | (uintptr_t)l->d_b) & 1) || ((uintptr_t)l->d_alpha & 3)) return ECF8_ERR_ALIGN;
  if (q && q->count) {
    if (q->count >= kMost || !q->d_offsets || !q->d_ids) return ECF8_ERR_ARG;
    if (((uintptr_t)q->d_offsets | (uintptr_t)q->d_ids) & 3) return ECF8_ERR_ALIGN;
  }
  const size_t need = plan_of(l, rows).total;
  if (need && (!ws || ws_bytes < need)) return ECF8_ERR_WORKSPACE;
  if ((uintptr_t)ws & 15) return ECF8_ERR_ALIGN;
  return ECF8_OK;
}

void route(const ecf8_linear* l, const ecf8_requests* q, uint64_t rows, int32_t* row_id, int32_t* d_status,
           cudaStream_t s) {
  const uint64_t most = rows > q->count ? rows : q->count;
  const unsigned grid = (unsigned)((most + 255) / 256 < 1024 ? (most + 255) / 256 : 1024);
  route_kernel<<<grid, 256, 0, s>>>(q->d_offsets, q->d_ids, q->count, l->n_adapters, rows, row_id, d_status);
}

constexpr uint64_t kGridY = 65535;

template <class T, int BACK>
void product(const ecf8_linear* l, bool adapted, const void* in, uint64_t in_stride, void* out, uint64_t out_stride,
             uint64_t rows, const int32_t* row_id, const float* p, cudaStream_t s) {
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
}

template <class T>
int forward(const ecf8_linear* l, const ecf8_requests* q, const void* x, uint64_t x_stride, void* y, uint64_t y_stride,
            uint64_t rows, float* u, char* ws, int32_t* d_status, cudaStream_t s) {
  const bool adapted = l->n_adapters && q && q->count;
  const Plan w = plan_of(l, rows);
  int32_t* row_id = reinterpret_cast<int32_t*>(ws);
  const bool keep = u != nullptr;
  if (l->n_adapters && !u) u = reinterpret_cast<float*>(ws + w.p);
  if (adapted) {
    route(l, q, rows, row_id, d_status, s);
    shrink_simple<T><<<dim3((unsigned)rows, (l->rank + 7) / 8), 128, 0, s>>>(
        static_cast<const T*>(x), x_stride, static_cast<const T*>(l->d_a), l->rank * l->k_in, l->k_in, 1, l->k_in,
        l->rank, row_id, u);
  } else if (l->n_adapters && keep) {
    if (cudaMemsetAsync(u, 0, rows * l->rank * 4, s) != cudaSuccess) return ECF8_ERR_CUDA;
  }
  product<T, 0>(l, adapted, x, x_stride, y, y_stride, rows, row_id, u, s);
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
  if (adapted && (dx || da)) {
    route(l, q, rows, row_id, d_status, s);
    shrink_simple<T><<<dim3((unsigned)rows, (l->rank + 7) / 8), 128, 0, s>>>(
        static_cast<const T*>(dy), dy_stride, static_cast<const T*>(l->d_b), l->n_out * l->rank, 1, l->rank, l->n_out,
        l->rank, row_id, v);
  }
  if (dx && rows) product<T, 1>(l, adapted, dy, dy_stride, dx, dx_stride, rows, row_id, v, s);
  const uint32_t count = adapted ? q->count : 0;
  const int32_t* offsets = adapted ? q->d_offsets : nullptr;
  const int32_t* ids = adapted ? q->d_ids : nullptr;
  if (da)
    outer_simple<T><<<dim3((unsigned)((l->k_in + 127) / 128), (l->rank + 7) / 8, l->n_adapters), 128, 0, s>>>(
        v, l->rank, static_cast<const T*>(x), x_stride, l->k_in, offsets, ids, count, rows, l->d_alpha,
        static_cast<T*>(da), l->rank * l->k_in, l->k_in, 1);
  if (db)
    outer_simple<T><<<dim3((unsigned)((l->n_out + 127) / 128), (l->rank + 7) / 8, l->n_adapters), 128, 0, s>>>(
        u, l->rank, static_cast<const T*>(dy), dy_stride, l->n_out, offsets, ids, count, rows, l->d_alpha,
        static_cast<T*>(db), l->rank * l->n_out, 1, l->rank);
  return cudaGetLastError() == cudaSuccess ? ECF8_OK : ECF8_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t ecf8_linear_workspace_size(const ecf8_linear* lin, uint64_t rows) {
  return lin && rows < kMost ? plan_of(lin, rows).total : 0;
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
