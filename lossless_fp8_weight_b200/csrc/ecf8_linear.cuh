// What the kernels of linear layers share: 16-bit types, the rows' adapters, and
// how the projection's kernel is called.  That kernel's four forms (two types,
// forward and input gradient) are compiled one to a file.
#ifndef ECF8_LINEAR_CUH_
#define ECF8_LINEAR_CUH_

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "ecf8.h"
#include "ecf8_tc.cuh"

// hidden: two copies of the library in one process (the bounds-checked one beside the other) share nothing
namespace ecf8_linear_impl __attribute__((visibility("hidden"))) {

using namespace ecf8_tc;

__device__ inline float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ inline float to_float(__half v) { return __half2float(v); }
__device__ inline void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ inline void put(__half* p, float v) { *p = __float2half_rn(v); }

template <class T> struct Widen;
template <> struct Widen<__nv_bfloat16> {
  static __device__ uint32_t pack(float a, float b) {
    __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&x);
  }
  static constexpr bool kBf16 = true;
};
template <> struct Widen<__half> {
  static __device__ uint32_t pack(float a, float b) {
    __half2 x = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&x);
  }
  static constexpr bool kBf16 = false;
};

template <class T> __device__ inline float2 unpack(uint32_t v);
template <> __device__ inline float2 unpack<__nv_bfloat16>(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
template <> __device__ inline float2 unpack<__half>(uint32_t v) {
  return __half22float2(*reinterpret_cast<__half2*>(&v));
}

// The two E4M3 bytes in bits 0-15 as a pair of FP16, as two float32, and as a
// pair of T.  BF16 goes through float32: of the ways tried, the conversions
// (185 clocks of an SM for 128 x 64 weights) beat moving the bits into BF16's
// places and one product by 2^120 (291: integer and multiply pipes both run at
// half rate, and NaN bytes need a check of their own).  FP16 takes 103.
__device__ inline uint32_t widen2_fp16(uint32_t b) {
  uint32_t v;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}" : "=r"(v) : "r"(b));
  return v;
}
__device__ inline float2 widen2_float(uint32_t b) { return unpack<__half>(widen2_fp16(b)); }
template <class T>
__device__ inline uint32_t widen2(uint32_t b) {
  if (!Widen<T>::kBf16) return widen2_fp16(b);
  const float2 w = widen2_float(b);
  return Widen<T>::pack(w.x, w.y);
}

// Two values as a pair of T and the pair of their rests.
template <class T>
__device__ inline void split_pair(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = Widen<T>::pack(x, y);
  const float2 h = unpack<T>(hi);
  // the rest of an infinity is nothing
  lo = Widen<T>::pack(isfinite(h.x) ? x - h.x : 0.0f, isfinite(h.y) ? y - h.y : 0.0f);
}

// The same for scaled weights, with fewer instructions: a rest that is no number (of an infinity) becomes -L, which adds
// nothing to what an infinity makes of a sum.  L is above every rest of FP16 weights, 2^4, and of BF16 weights to 2^68.
template <class T>
__device__ inline void split_scaled(float x, float y, uint32_t& hi, uint32_t& lo) {
  constexpr float L = Widen<T>::kBf16 ? 0x1p60f : 0x1p5f;
  hi = Widen<T>::pack(x, y);
  const float2 h = unpack<T>(hi);
  lo = Widen<T>::pack(fmaxf(x - h.x, -L), fmaxf(y - h.y, -L));
}

// The distinct ids >= 0 of ids[0..n), n <= 256, in the order they first occur, by threads 0..255.
// `runs` is scratch of 256; the list and its length end in `list` and *count.  Every thread of the CTA calls it.
__device__ inline void distinct(const int32_t* ids, uint32_t n, int32_t* runs, int32_t* list, uint32_t* count,
                                uint32_t* warp_sum) {
  const uint32_t t = threadIdx.x, lane = t % 32, warp = t / 32;
  // starts of runs of equal ids
  bool start = t < n && ids[t] >= 0 && (t == 0 || ids[t] != ids[t - 1]);
  uint32_t mask = __ballot_sync(~0u, start);
  if (lane == 0 && warp < 8) warp_sum[warp] = __popc(mask);
  __syncthreads();
  uint32_t before = 0, total = 0;
  for (uint32_t w = 0; w < 8; ++w) {
    before += w < warp ? warp_sum[w] : 0;
    total += warp_sum[w];
  }
  if (start) runs[before + __popc(mask & ((1u << lane) - 1))] = ids[t];
  __syncthreads();
  // runs whose id has not occurred before
  bool first = t < total;
  if (first)
    for (uint32_t j = 0; j < t; ++j)
      if (runs[j] == runs[t]) {
        first = false;
        break;
      }
  __syncwarp();
  mask = __ballot_sync(~0u, first);
  __syncthreads();
  if (lane == 0 && warp < 8) warp_sum[warp] = __popc(mask);
  __syncthreads();
  before = total = 0;
  for (uint32_t w = 0; w < 8; ++w) {
    before += w < warp ? warp_sum[w] : 0;
    total += warp_sum[w];
  }
  if (first) list[before + __popc(mask & ((1u << lane) - 1))] = runs[t];
  if (t == 0) *count = total;
  __syncthreads();
}

// A CTA that has failed does not end before the loads and products that it started.  One warp each: the loads, where
// the next use of a stage would have been `s` with parity `turn` (a wait for the last use of every stage; at once where
// there was none), and the products, whose end arrives on `spent` of the CTA that issued them.
__device__ inline void drain_loads(uint32_t full, uint32_t s, uint32_t turn, uint32_t stages, const Waits& w) {
  for (uint32_t i = 0; i < stages; ++i) mbar_wait_out(full + 8 * i, i < s ? turn : turn ^ 1, w);
}
template <int P>
__device__ inline void drain_products(uint32_t spent, uint32_t rank, const Waits& w) {
  if (elect_one()) mma_commit<P>(spent, 1u << rank);
  __syncwarp();
  mbar_wait_out(spent, 0, w);
}

// How a launch waits.  The bounds-checked build can set it: a short limit, and one arrival more than will come on the
// first load's barrier.
struct Limits {
  long long cycles = kWaitCycles;
  uint32_t missing = 0;
};

struct ProductArgs {
  uint64_t rows, cols, len;
  uint32_t blocks;       // 64 * KB-wide steps of the reduction
  uint32_t bt;           // rows of q in a tile, a multiple of 16, at most 256
  uint32_t stages, split;
  const float* scale;
  uint64_t n_scale;
  const int32_t* row_id;
  const float* p;        // rows x rank
  const void* f;         // the adapters' factor added to the output
  uint64_t f_adapter, sr, sc;
  const float* alpha;
  uint32_t rank;         // 0: no adapters
  uint32_t f_vector;     // 8 ranks of f are one aligned 16-byte load
  uint32_t p_vector;     // and 4 of p
  void* out;
  uint64_t out_stride;
  uint32_t out_vector;   // 4 columns of an output row are one aligned 8-byte store
  int32_t* status;
  Limits limits;
};

constexpr uint32_t kMaxStages = 16, kSlots = 8;

template <class K>
int allow_smem(K kernel, bool (&set)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ECF8_ERR_CUDA;
  if (dev < 64 && set[dev]) return ECF8_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 219 * 1024) != cudaSuccess)
    return ECF8_ERR_CUDA;
  if (dev < 64) set[dev] = true;
  return ECF8_OK;
}
// Launches the projection (BACK = 0) or the input gradient (BACK = 1); `pair`: two CTAs to a tile.
template <class T, int BACK>
int product_launch(bool pair, const CUtensorMap& mw, const CUtensorMap& mq, const ProductArgs& a, dim3 grid,
                   size_t smem, bool overlap, cudaStream_t s);

}  // namespace ecf8_linear_impl

#endif  // ECF8_LINEAR_CUH_
