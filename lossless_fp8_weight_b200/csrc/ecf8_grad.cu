// The global norm of a set of gradient tensors, and clipping by it.
//
//     norm = sqrt(sum over all tensors, values of x^2)
//     out  = x * min(1, max_norm / (norm + 1e-6))
//
// Bound: HBM.  The norm has to read every value once, the scaled copy reads
// them again (the factor depends on the last value) and writes them once; sets
// that fit in L2 are read from HBM once.  One call takes all tensors, as the
// batched decode does: a set of adapters is hundreds of small tensors, and one
// launch for each would cost more than the data.
//
// A tensor is cut into chunks of kChunk values; each CTA takes a contiguous run
// of the set's chunks, finds its first tensor by a binary search and walks on
// from there.  Squares are summed in float64 (a float32 squared is exact in it,
// and no sum of them overflows), per thread, then per CTA in a fixed
// tree, then over the CTAs' sums in index order, so the result does not vary.
// Conversions to float64 run at a quarter of the rate of other instructions,
// which for 16-bit values is less than memory delivers: four of those are
// squared exactly and added in pairs in float32 first (two roundings, 2^-24 of
// the norm), unless the sum is outside what float32 holds without loss.  The
// second launch sums the CTAs' partial sums in every CTA for itself, which
// needs no barrier across the grid; it starts beside the end of the first and
// takes the chunks from the last one on, which L2 still holds.
//
// Measured: 448 BF16 tensors (84 MB): the norm 26 us (30 with float64 alone),
// with the clipped copy 49 us, 3.4 TB/s of bytes read once and written once,
// 52% of the copy rate, since the second reading comes partly from memory;
// 1120 float32 tensors (828 MB): 152 and 423 us, the norm 83% of the rate and
// the whole, which has to read twice, 89% of what three passes can have.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <vector>

#include "ecf8.h"

namespace {

constexpr uint32_t kMagic = 0x44524745;  // "EGRD"
constexpr int kThreads = 512;
constexpr uint64_t kChunk = 8192;        // values
constexpr uint32_t kMaxCtas = 2048;      // partial sums in the workspace

struct Header {
  uint32_t magic, count;
  uint64_t chunks;
  uint32_t all_out, pad;
  uint64_t pad2;
};

struct Entry {
  const void* in;
  void* out;
  uint64_t n;
  uint64_t first_chunk;
  int32_t dtype;
  uint32_t pad;
};

__host__ __device__ inline uint32_t width(int32_t dtype) { return dtype == ECF8_DTYPE_FP32 ? 4 : 2; }

template <int N> struct Count { static constexpr int value = N; };

template <int DT> struct Type;
template <> struct Type<ECF8_DTYPE_BF16> {
  using T = __nv_bfloat16;
  using U = uint16_t;
  static __device__ float get(T v) { return __bfloat162float(v); }
  static __device__ T put(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Type<ECF8_DTYPE_FP16> {
  using T = __half;
  using U = uint16_t;
  static __device__ float get(T v) { return __half2float(v); }
  static __device__ T put(float v) { return __float2half_rn(v); }
};
template <> struct Type<ECF8_DTYPE_FP32> {
  using T = float;
  using U = uint32_t;
  static __device__ float get(T v) { return v; }
  static __device__ T put(float v) { return v; }
};

// The index of the tensor that holds a chunk: the last entry whose first chunk is not past it.  The threads look at
// every entry at once: a binary search would wait for memory ten times.
__device__ uint32_t find(const Entry* e, uint32_t count, uint64_t chunk) {
  uint32_t upto = 0;
  for (uint32_t i = 0; i < count; i += kThreads)
    upto += __syncthreads_count(i + threadIdx.x < count && e[i + threadIdx.x].first_chunk <= chunk);
  return upto - 1;  // the first entry's is 0
}

// Calls f(entry, begin, end) for run `cta` of chunks, tensor by tensor.
template <class F>
__device__ void walk(const Entry* e, uint32_t count, uint64_t chunks, uint32_t cta, F f) {
  uint64_t c = chunks * cta / gridDim.x;
  const uint64_t last = chunks * (cta + 1) / gridDim.x;
  if (c >= last) return;
  for (uint32_t i = find(e, count, c); i < count && c < last; ++i) {
    const Entry t = e[i];
    const uint64_t own = (t.n + kChunk - 1) / kChunk;
    if (t.first_chunk + own <= c) continue;  // an empty tensor
    const uint64_t stop = min(last, t.first_chunk + own);
    const uint64_t b = (c - t.first_chunk) * kChunk, end = min(t.n, (stop - t.first_chunk) * kChunk);
    f(t, b, end);
    c = stop;
  }
}

// The values before the first 16-byte boundary of a run of values at p.
template <class T>
__device__ uint64_t head_of(const T* p, uint64_t n) {
  const uint64_t to = ((16 - ((uintptr_t)p & 15)) & 15) / sizeof(T);
  return min(to, n);
}

template <int DT>
__device__ double squares(const Entry& t, uint64_t b, uint64_t end) {
  using T = typename Type<DT>::T;
  constexpr int V = 16 / sizeof(T);
  const T* p = static_cast<const T*>(t.in) + b;
  const uint64_t n = end - b, head = head_of(p, n);
  double s = 0;
  auto one = [&](T v) {
    const double d = (double)Type<DT>::get(v);
    s = fma(d, d, s);
  };
  auto vector = [&](const uint4& w) {
    const T* v = reinterpret_cast<const T*>(&w);
    if (V == 4) {
#pragma unroll
      for (int j = 0; j < V; ++j) one(v[j]);
    } else {
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        const float x0 = Type<DT>::get(v[j]), x1 = Type<DT>::get(v[j + 1]), x2 = Type<DT>::get(v[j + 2]),
                    x3 = Type<DT>::get(v[j + 3]);
        const float q = fmaf(x1, x1, x0 * x0) + fmaf(x3, x3, x2 * x2);
        if (q >= 0x1p-90f && q <= 0x1p120f) {
          // a normal float32 as float64, by its bits: the conversion has a quarter of the rate
          const uint32_t bits = __float_as_uint(q);
          s += __hiloint2double((int)((bits >> 3) + 0x38000000u), (int)(bits << 29));
        } else {
          one(v[j]);
          one(v[j + 1]);
          one(v[j + 2]);
          one(v[j + 3]);
        }
      }
    }
  };
  if (threadIdx.x < head) one(p[threadIdx.x]);
  const uint4* q = reinterpret_cast<const uint4*>(p + head);
  const uint64_t nv = (n - head) / V;
  uint64_t i = threadIdx.x;
  for (; i + 3 * kThreads < nv; i += 4 * kThreads) {
    uint4 w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = q[i + k * kThreads];
#pragma unroll
    for (int k = 0; k < 4; ++k) vector(w[k]);
  }
  for (; i < nv; i += kThreads) vector(q[i]);
  const uint64_t tail = head + nv * V;
  if (tail + threadIdx.x < n) one(p[tail + threadIdx.x]);
  return s;
}

template <int DT>
__device__ void scaled(const Entry& t, uint64_t b, uint64_t end, float factor) {
  using T = typename Type<DT>::T;
  constexpr int V = 16 / sizeof(T);
  const T* p = static_cast<const T*>(t.in) + b;
  T* o = static_cast<T*>(t.out) + b;
  const uint64_t n = end - b;
  // A factor of 1 copies the bits, those of a NaN too: as whole numbers, since a
  // compiler may turn a choice between v and v * 1 into v * 1.
  const bool copy = factor == 1.0f;
  auto one = [&](T v) { return Type<DT>::put(Type<DT>::get(v) * factor); };
  using U = typename Type<DT>::U;
  auto single = [&](uint64_t i) {
    if (copy) reinterpret_cast<U*>(o)[i] = reinterpret_cast<const U*>(p)[i];
    else o[i] = one(p[i]);
  };
  if ((((uintptr_t)p ^ (uintptr_t)o) & 15) != 0) {  // in and out never reach a 16-byte boundary together
    for (uint64_t i = threadIdx.x; i < n; i += kThreads) single(i);
    return;
  }
  const uint64_t head = head_of(p, n);
  if (threadIdx.x < head) single(threadIdx.x);
  const uint4* q = reinterpret_cast<const uint4*>(p + head);
  uint4* r = reinterpret_cast<uint4*>(o + head);
  const uint64_t nv = (n - head) / V;
  // read and written for the last time here: other data should stay in L2
  auto vectors = [&](uint64_t i, auto n_vectors) {
    constexpr int N = decltype(n_vectors)::value;
    uint4 w[N];
#pragma unroll
    for (int k = 0; k < N; ++k) w[k] = __ldcs(q + i + k * kThreads);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      T* v = reinterpret_cast<T*>(&w[k]);
      if (!copy)
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = one(v[j]);
      __stcs(r + i + k * kThreads, w[k]);
    }
  };
  uint64_t i = threadIdx.x;
  for (; i + 3 * kThreads < nv; i += 4 * kThreads) vectors(i, Count<4>{});
  for (; i < nv; i += kThreads) vectors(i, Count<1>{});
  const uint64_t tail = head + nv * V;
  if (tail + threadIdx.x < n) single(tail + threadIdx.x);
}

// Sum over the CTA's threads in a fixed tree; the result is in every thread.
__device__ double block_sum(double s) {
  __shared__ double part[kThreads / 32];
  for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = s;
  __syncthreads();
  s = 0;
  for (int i = 0; i < kThreads / 32; ++i) s += part[i];
  return s;
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const Header* table, uint32_t count, uint64_t chunks,
                                                        double* partial) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Entry* e = reinterpret_cast<const Entry*>(table + 1);
  double s = 0;
  walk(e, count, chunks, blockIdx.x, [&](const Entry& t, uint64_t b, uint64_t end) {
    if (t.dtype == ECF8_DTYPE_BF16) s += squares<ECF8_DTYPE_BF16>(t, b, end);
    else if (t.dtype == ECF8_DTYPE_FP16) s += squares<ECF8_DTYPE_FP16>(t, b, end);
    else s += squares<ECF8_DTYPE_FP32>(t, b, end);
  });
  s = block_sum(s);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__global__ void __launch_bounds__(kThreads) clip_kernel(const Header* table, uint32_t count, uint64_t chunks,
                                                        const double* partial, uint32_t n_partial, float max_norm,
                                                        int clip, float* d_norm, int32_t* d_status) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  double s = 0;
  for (uint32_t i = threadIdx.x; i < n_partial; i += kThreads) s += partial[i];
  const double norm = sqrt(block_sum(s));
  const float shown = (float)norm;
  const bool finite = isfinite(shown);  // as the caller sees it
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *d_norm = shown;
    if (!finite && d_status) atomicOr(d_status, ECF8_STATUS_NONFINITE);
  }
  if (!clip) return;
  const float factor = finite ? (float)fmin(1.0, (double)max_norm / (norm + 1e-6)) : 1.0f;
  const Entry* e = reinterpret_cast<const Entry*>(table + 1);
  // what the norm read last is in L2 still: the runs are taken from the end
  walk(e, count, chunks, gridDim.x - 1 - blockIdx.x, [&](const Entry& t, uint64_t b, uint64_t end) {
    if (factor == 1.0f && t.in == t.out) return;  // x * 1 is there already
    if (t.dtype == ECF8_DTYPE_BF16) scaled<ECF8_DTYPE_BF16>(t, b, end, factor);
    else if (t.dtype == ECF8_DTYPE_FP16) scaled<ECF8_DTYPE_FP16>(t, b, end, factor);
    else scaled<ECF8_DTYPE_FP32>(t, b, end, factor);
  });
}

struct Span {
  uintptr_t from, to;
  int tensor;
};

// Whether any output shares bytes with another output, or with an input other than its own in place.
bool outputs_collide(const ecf8_grad* grads, int count) {
  std::vector<Span> outs;
  for (int i = 0; i < count; ++i)
    if (grads[i].n && grads[i].d_out)
      outs.push_back(Span{(uintptr_t)grads[i].d_out, (uintptr_t)grads[i].d_out + grads[i].n * width(grads[i].dtype), i});
  std::sort(outs.begin(), outs.end(), [](const Span& a, const Span& b) { return a.from < b.from; });
  for (size_t i = 1; i < outs.size(); ++i)
    if (outs[i].from < outs[i - 1].to) return true;
  for (int i = 0; i < count; ++i) {
    if (!grads[i].n) continue;
    const uintptr_t from = (uintptr_t)grads[i].d_in, to = from + grads[i].n * width(grads[i].dtype);
    // the outputs do not overlap, so their ends are in order too: the first that ends past `from`
    auto o = std::upper_bound(outs.begin(), outs.end(), from, [](uintptr_t f, const Span& s) { return f < s.to; });
    for (; o != outs.end() && o->from < to; ++o)
      if (o->tensor != i || o->from != from) return true;
  }
  return false;
}

int run(const void* h_table, const void* d_table, int clip, float max_norm, float* d_norm, void* ws, size_t ws_bytes,
        int32_t* d_status, cudaStream_t s) {
  if (!h_table || !d_table || !d_norm) return ECF8_ERR_ARG;
  const Header* h = static_cast<const Header*>(h_table);
  if (h->magic != kMagic) return ECF8_ERR_ARG;
  if (clip && (!h->all_out || !(max_norm >= 0))) return ECF8_ERR_ARG;
  if (((uintptr_t)d_table & 15) || ((uintptr_t)d_norm & 3) || ((uintptr_t)d_status & 3) || ((uintptr_t)ws & 15))
    return ECF8_ERR_ALIGN;
  if (!ws || ws_bytes < ecf8_grad_workspace_size()) return ECF8_ERR_WORKSPACE;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return ECF8_ERR_CUDA;
  // four CTAs of 512 threads fill an SM; a CTA has a chunk at least
  uint64_t grid = (uint64_t)sms * 4;
  if (grid > kMaxCtas) grid = kMaxCtas;
  if (grid > h->chunks) grid = h->chunks;
  const Header* d = static_cast<const Header*>(d_table);
  double* partial = static_cast<double*>(ws);
  if (grid) norm_kernel<<<(unsigned)grid, kThreads, 0, s>>>(d, h->count, h->chunks, partial);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(clip && grid ? (unsigned)grid : 1);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = grid ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, clip_kernel, d, (uint32_t)h->count, (uint64_t)h->chunks, (const double*)partial,
                         (uint32_t)grid, max_norm, (int)(clip && grid), d_norm, d_status) != cudaSuccess)
    return ECF8_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? ECF8_OK : ECF8_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t ecf8_grad_table_bytes(int count) { return count < 0 ? 0 : sizeof(Header) + sizeof(Entry) * (size_t)count; }

size_t ecf8_grad_workspace_size(void) { return kMaxCtas * sizeof(double); }

int ecf8_grad_build_table(const ecf8_grad* grads, int count, void* h_table) {
  if (!h_table || count < 0 || (count && !grads)) return ECF8_ERR_ARG;
  for (int i = 0; i < count; ++i) {
    const ecf8_grad& g = grads[i];
    if (g.dtype != ECF8_DTYPE_BF16 && g.dtype != ECF8_DTYPE_FP16 && g.dtype != ECF8_DTYPE_FP32) return ECF8_ERR_ARG;
    if (g.n > (UINT64_MAX >> 8)) return ECF8_ERR_ARG;
    if (g.n && !g.d_in) return ECF8_ERR_ARG;
    if (((uintptr_t)g.d_in | (uintptr_t)g.d_out) & (width(g.dtype) - 1)) return ECF8_ERR_ALIGN;
  }
  try {
    if (outputs_collide(grads, count)) return ECF8_ERR_ARG;
  } catch (...) {  // no host memory for the check
    return ECF8_ERR_CAPACITY;
  }
  Header* h = static_cast<Header*>(h_table);
  Entry* e = reinterpret_cast<Entry*>(h + 1);
  uint64_t chunks = 0;
  uint32_t all_out = 1;
  for (int i = 0; i < count; ++i) {
    const ecf8_grad& g = grads[i];
    e[i] = Entry{g.d_in, g.d_out, g.n, chunks, g.dtype, 0};
    chunks += (g.n + kChunk - 1) / kChunk;
    if (g.n && !g.d_out) all_out = 0;
  }
  *h = Header{kMagic, (uint32_t)count, chunks, all_out, 0, 0};
  return ECF8_OK;
}

int ecf8_grad_norm(const void* h_table, const void* d_table, float* d_norm, void* d_workspace, size_t workspace_bytes,
                   int32_t* d_status, cudaStream_t s) {
  return run(h_table, d_table, 0, 0.0f, d_norm, d_workspace, workspace_bytes, d_status, s);
}

int ecf8_grad_clip(const void* h_table, const void* d_table, float max_norm, float* d_norm, void* d_workspace,
                   size_t workspace_bytes, int32_t* d_status, cudaStream_t s) {
  return run(h_table, d_table, 1, max_norm, d_norm, d_workspace, workspace_bytes, d_status, s);
}

}  // extern "C"
