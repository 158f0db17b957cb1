// The shared projection of a linear layer on the tensor cores, and its input gradient.
//
//     D[c][t] += sum_j W(c, j) q[t][j]        c: output (forward) or input (backward) column
//
// The weight is the 128-row operand and the rows of q are the other (16 to 256
// of them), so a single token costs no more tensor work than it must and one
// kernel serves decoding and prompts.  The tensor cores have no product of E4M3
// by 16-bit values: warps widen the weights, which is exact, and put them
// into tensor memory, from where the matrix unit reads them without passing
// through shared memory again.  One warp loads tiles by TMA, one issues the
// products.
//
// Small calls (up to 128 rows) are bound by reading W: the reduction is split
// over a cluster of up to 8 CTAs, whose sums meet in distributed shared memory
// in a fixed order, so that few columns still occupy every SM and no workspace
// or second launch is needed.  Large calls are bound by the matrix unit and by
// what L2 can deliver: two CTAs act as one on a 256 x 256 tile, each loading
// its own weights and half of q (one CTA on 128 x 256 asked 12 TB/s of L2 and
// stopped there).
//
// Measured without adapters, FP16 and BF16, on a GPU that was idle before.  16
// rows of 28672x8192: 52 and 58 us, 4.6 and 4.1 TB/s, 69 and 62% of the copy
// rate; of 8192x28672: 48 and 53 us.  8192 rows of 14336x4096: 0.82 and 0.84
// ms, 1.17 and 1.14 PFLOP/s, 71 and 69%; the input gradient at 8192 rows of
// 8192x8192: 1.01 and 1.03 ms, 66%; at 4096 rows of 4096x4096 0.152 and 0.158
// ms, 55%.  What bounds it now: the hand-over from load to widening to product
// (forward the matrix unit is active for 59% of the clocks, the warps issue in
// 34%, memory and L2 are below 30%; with the widening left out it ran 15%
// faster), in the input gradient with the byte loads in it that turn a column
// of W into a row (53% and 38%, the shared-memory pipe 28%); in small calls,
// start and end of the CTAs.
//
// The adapters' part of large calls is more terms of the same sum,
//     D[c][t] += sum over the tile's adapters a, ranks r of (f[a][c][r] alpha[a] / s[c]) * [a is t's] p[t][r],
// 32 terms for 16 ranks of an adapter: both factors as a BF16 value and a BF16
// rest (three products; 2^-16 of a term is lost).  Factors of either side that are
// not finite are left out of it and their terms added one by one at the end,
// where they meet their own rows only and no rest; so are columns whose scale
// is zero or extreme.
//
// The input gradient with a scale for every output row needs s W, which no
// 16-bit type holds: it enters as a 16-bit value and a 16-bit rest, two
// products a step (one of them alone made the error up to 1.3 times that of
// the final rounding).  2^-17 of a term is lost in BF16; in FP16 2^-23, or 2^-31
// of the largest scale's where that is more.  8192 rows of 8192x8192: 1.58 and
// 1.56 ms, the matrix unit active for 78% of the clocks at the rate that the
// power cap leaves it (one scale for all, one product: 1.01 and 1.03 ms).
#ifndef ECF8_PRODUCT_CUH_
#define ECF8_PRODUCT_CUH_

#include "ecf8_linear.cuh"

namespace ecf8_linear_impl __attribute__((visibility("hidden"))) {

// sum over r of p[t][r] f[a][c][r] (or f[a][r][c]): the adapter's part of one output.
template <class T>
__device__ inline float adapter_part(const ProductArgs& a, int32_t id, uint64_t t, uint64_t c, uint32_t r0,
                                     uint32_t r1) {
  const float* p = a.p + t * a.rank;
  const T* f = static_cast<const T*>(a.f) + (uint64_t)id * a.f_adapter + c * a.sc;
  float z = 0;
  if (a.f_vector && a.p_vector) {
    for (uint32_t r = r0; r < r1; r += 8) {
      const uint4 w = *reinterpret_cast<const uint4*>(f + r);
      const float4 u = *reinterpret_cast<const float4*>(p + r), v = *reinterpret_cast<const float4*>(p + r + 4);
      float2 x = unpack<T>(w.x);
      z = fmaf(x.x, u.x, fmaf(x.y, u.y, z));
      x = unpack<T>(w.y);
      z = fmaf(x.x, u.z, fmaf(x.y, u.w, z));
      x = unpack<T>(w.z);
      z = fmaf(x.x, v.x, fmaf(x.y, v.y, z));
      x = unpack<T>(w.w);
      z = fmaf(x.x, v.z, fmaf(x.y, v.w, z));
    }
  } else {
    for (uint32_t r = r0; r < r1; ++r) z = fmaf(p[r], to_float(f[r * a.sr]), z);
  }
  return z * a.alpha[id];
}

// 16 ranks of the factor of column c from rank r0 on, times `by`; false if one is not finite.
template <class T>
__device__ inline bool adapter_factor(const ProductArgs& a, int32_t id, uint64_t c, uint32_t r0, float by,
                                      float (&v)[16]) {
  const T* f = static_cast<const T*>(a.f) + (uint64_t)id * a.f_adapter + c * a.sc;
  if (a.f_vector) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (r0 + 8 * h < a.rank) w = *reinterpret_cast<const uint4*>(f + r0 + 8 * h);
      const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 y = unpack<T>(x[k]);
        v[8 * h + 2 * k] = y.x * by;
        v[8 * h + 2 * k + 1] = y.y * by;
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k] = r0 + k < a.rank ? to_float(f[(r0 + k) * a.sr]) * by : 0.0f;
  }
  float m = 0;
#pragma unroll
  for (int k = 0; k < 16; ++k) m = fmaxf(m, v[k] != v[k] ? INFINITY : fabsf(v[k]));
  return m < 3e38f;
}

// 16 of a row's p from rank r0 on; false if one is not finite.
__device__ inline bool row_factor(const ProductArgs& a, uint64_t t, uint32_t r0, float (&y)[16]) {
  const float* p = a.p + t * a.rank;
  if (a.p_vector) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float4 z = make_float4(0, 0, 0, 0);
      if (r0 + 4 * q < a.rank) z = *reinterpret_cast<const float4*>(p + r0 + 4 * q);
      y[4 * q] = z.x;
      y[4 * q + 1] = z.y;
      y[4 * q + 2] = z.z;
      y[4 * q + 3] = z.w;
    }
  } else {
#pragma unroll
    for (int q = 0; q < 16; ++q) y[q] = r0 + q < a.rank ? p[r0 + q] : 0.0f;
  }
  float m = 0;
#pragma unroll
  for (int q = 0; q < 16; ++q) m = fmaxf(m, y[q] != y[q] ? INFINITY : fabsf(y[q]));
  return m < 3e38f;
}

// The ranks of an adapter's part that the tensor cores left out.
template <class T>
__device__ float left_out(const ProductArgs& a, int32_t id, uint64_t t, uint64_t c, float scale, bool divides) {
  float z = 0;
  for (uint32_t r0 = 0; r0 < a.rank; r0 += 16) {
    float f[16], y[16];
    const bool fits = adapter_factor<T>(a, id, c, r0, a.alpha[id] / scale, f);
    if (!row_factor(a, t, r0, y) || !fits || !divides)
      z += adapter_part<T>(a, id, t, c, r0, r0 + 16 < a.rank ? r0 + 16 : a.rank);
  }
  return z;
}

// P: CTAs of a tile.  KB: 64-wide steps in a stage.  G: groups of 4 widening warps.
template <class T, int P, int KB, int G, int BACK>
__global__ void __launch_bounds__(64 + 128 * G, P == 2 ? 1 : 2)
    product_tc(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_q,
               const __grid_constant__ ProductArgs a) {
  // widened steps in tensor memory: as many as there are stages, which they then follow, or four; half of that where
  // a step has two parts
  constexpr uint32_t most_slots = P == 2 ? kSlots : 4, columns = P == 2 ? 512 : 256;
  const bool wide = BACK && a.n_scale > 1;
  const uint32_t slot_bits = (P == 2 ? 3 : 2) - (wide ? 1 : 0), slot_mask = (1u << slot_bits) - 1;
  const uint32_t slot_columns = wide ? 64 : 32;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 2 * kSlots + 2];
  __shared__ uint32_t tmem_base;
  __shared__ int failed_s;
  __shared__ float unit_s;
  __shared__ float max_s[4 * G];
  __shared__ __align__(16) float scale_s[BACK ? 4 * G : 1][64];
  __shared__ int32_t ids[256], runs[256], list[256];
  __shared__ uint32_t count_s, warp_sum[8], apart_s;
  const Waits waits{&failed_s, a.limits.cycles};

  const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
  const uint32_t rows_here = a.bt / P;  // rows of q that this CTA loads
  const uint32_t w_bytes = 8192 * KB, q_bytes = rows_here * 128 * KB, stage_bytes = w_bytes + q_bytes;
  const uint32_t full = smem_addr(bars), empty = full + 8 * kMaxStages, ready = empty + 8 * kMaxStages,
                 freed = ready + 8 * kSlots, done = freed + 8 * kSlots, spent = done + 8;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  // a cluster is a pair, or the parts of a split reduction
  const uint32_t split = P == 2 ? 1 : a.split, cluster = P * split, crank = cluster > 1 ? cluster_rank() : 0;
  const uint32_t side = P == 2 ? crank : 0, part = P == 2 ? 0 : crank;
  const uint64_t c0 = ((uint64_t)(blockIdx.x / cluster) * P + side) * 128, t0 = (uint64_t)blockIdx.y * a.bt;
  const uint32_t b0 = (uint32_t)((uint64_t)a.blocks * part / split),
                 b1 = (uint32_t)((uint64_t)a.blocks * (part + 1) / split), nb = b1 - b0;
  const uint32_t steps = nb * KB;

  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < a.stages; ++i) {
      mbar_init(full + 8 * i, i == 0 ? 1 + a.limits.missing : 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (uint32_t i = 0; i < most_slots; ++i) {
      mbar_init(ready + 8 * i, 4 * P);
      mbar_init(freed + 8 * i, 1);
    }
    mbar_init(done, 1);
    mbar_init(spent, 1);
    failed_s = 0;
    apart_s = 0;
    unit_s = 1.0f;
    count_s = 0;
    mbar_init_fence();
  }
  if (warp == 1) {
    tmem_alloc<P>(smem_addr(&tmem_base), columns);
    tmem_release_permit<P>();
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_base, tmem_a = tmem + (columns - most_slots * 32);
  // where a step is widened to: `at` is its stage with P = 2, its slot else
  auto widened = [&](uint32_t at) { return tmem_a + (at & slot_mask) * slot_columns; };
  uint32_t adapter_steps = 0, units = 0;
  if (P == 2) {
    // the other CTA's barriers are ready before anything arrives on them
    cluster_sync();
  }
  // P = 2, by all threads between the weights' steps and the adapters': what the kernel before this one has written is
  // not needed earlier.
  auto find_adapters = [&] {
    if (P != 2 || !a.rank) return;
    __syncwarp();
    wait_predecessor();
    if (threadIdx.x < 256)
      ids[threadIdx.x] = threadIdx.x < a.bt && t0 + threadIdx.x < a.rows ? a.row_id[t0 + threadIdx.x] : -1;
    __syncthreads();
    distinct(ids, a.bt, runs, list, &count_s, warp_sum);
    units = count_s * ((a.rank + 15) / 16);
    adapter_steps = (units + 1) / 2;
  };

  // P = 2, by all threads: either CTA's apart_s has what both have stored there.  (The products' barriers order the
  // stores of the pair's even CTA for that CTA only.)
  auto share_apart = [&] {
    if (P != 2 || !a.rank) return;
    __syncwarp();
    cluster_sync();
  };

  uint32_t next = 0, next_turn = 0;  // warp 0: the next stage to load, and the parity of its use
  if (warp == 0) {
    if (elect_one()) {
      tma_prefetch(&map_w);
      tma_prefetch(&map_q);
    }
    bool ok = true;
    for (uint32_t i = 0; i < nb; ++i) {
      // a stage is free when its products have ended, and so have the warps that widened for them
      // (a wait for the phase before the first passes at once)
      ok = mbar_wait_lanes(empty + 8 * next, next_turn ^ 1, waits);
      if (!ok) break;
      const uint32_t at = base + next * stage_bytes, bar = full + 8 * next;
      const int32_t j = (int32_t)((b0 + i) * 64 * KB);
      if (elect_one()) {
        mbar_expect(bar, stage_bytes);
        if (BACK) tma_load(at, &map_w, (int32_t)c0, j, bar);
        else tma_load(at, &map_w, j, (int32_t)c0, bar);
#pragma unroll
        for (int k = 0; k < KB; ++k)
          tma_load(at + w_bytes + k * rows_here * 128, &map_q, j + 64 * k, (int32_t)(t0 + side * rows_here), bar);
      }
      __syncwarp();
      if (++next == a.stages) next = 0, next_turn ^= 1;
    }
    find_adapters();
    share_apart();
  } else if (warp == 1) {
    if (side != 0) {
      find_adapters();
    } else {
      const uint32_t mask = 3;
      const uint32_t idesc = idesc_f16(Widen<T>::kBf16, 128 * P, a.bt);
      uint32_t g = 0, s = 0, turn = 0;  // 64-wide steps, stage, parity
      bool ok = true;
      for (uint32_t i = 0; i < nb && ok; ++i) {
#pragma unroll
        for (int k = 0; k < KB && ok; ++k, ++g) {
          // the warps that report a step ready have waited for their CTA's tiles
          const uint32_t slot = P == 2 ? s : g & slot_mask;
          ok = mbar_wait_lanes<P == 2>(ready + 8 * slot, P == 2 ? turn : g >> slot_bits & 1, waits);
          if (!ok) break;
          fence_after();
          const uint64_t b = desc_k128(base + s * stage_bytes + w_bytes + k * rows_here * 128);
          if (elect_one()) {
#pragma unroll
            for (int m = 0; m < 4; ++m) mma_ts<P>(tmem, widened(slot) + m * 8, b + m * 2, idesc, g > 0 || m > 0);
            if (wide)
#pragma unroll
              for (int m = 0; m < 4; ++m) mma_ts<P>(tmem, widened(slot) + 32 + m * 8, b + m * 2, idesc, 1);
            if (P == 1) mma_commit<P>(freed + 8 * slot, mask);
            if (k == KB - 1) mma_commit<P>(empty + 8 * s, mask);
          }
          __syncwarp();
        }
        if (++s == a.stages) s = 0, turn ^= 1;
      }
      find_adapters();
      if (P == 2) {
        const uint32_t idesc_pair = idesc_f16(true, 128 * P, a.bt);
        for (uint32_t i = 0; i < adapter_steps && ok; ++i, ++g) {
          ok = mbar_wait_lanes<true>(ready + 8 * s, turn, waits);
          if (!ok) break;
          fence_after();
          const uint64_t b = desc_k128(base + s * stage_bytes + w_bytes);
          const uint32_t first = i * 2;
          if (elect_one()) {
            for (uint32_t u = 0; u < 2 && first + u < units; ++u) {
              const uint32_t hi = widened(s) + u * 16;
              mma_ts<P>(tmem, hi, b + u * 4, idesc_pair, g > 0 || u > 0);
              mma_ts<P>(tmem, hi, b + u * 4 + 2, idesc_pair, 1);
              mma_ts<P>(tmem, hi + 8, b + u * 4, idesc_pair, 1);
            }
            mma_commit<P>(empty + 8 * s, mask);
          }
          __syncwarp();
          if (++s == a.stages) s = 0, turn ^= 1;
        }
      }
      if (ok && elect_one()) mma_commit<P>(done, mask);
      __syncwarp();
    }
    share_apart();
  } else {
    const int w4 = warp - 2, quarter = warp % 4, group = w4 / 4;
    const uint32_t row = quarter * 32 + lane;
    const uint64_t c = c0 + row;
    // With a scale for each term of the reduction the weights are scaled here, FP16 by a power of two more that brings
    // the largest scale to [64, 128): the largest product, 57344, is in range.
    float unit = 1.0f;
    if (wide && !Widen<T>::kBf16) {
      float m = 0;
#pragma unroll 8
      for (uint32_t i = threadIdx.x - 64; i < (uint32_t)a.n_scale; i += 128 * G) {
        const float s = fabsf(a.scale[i]);
        if (s <= 3e38f) m = fmaxf(m, s);
      }
      for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
      if (lane == 0) max_s[w4] = m;
      asm volatile("bar.sync 1, %0;" ::"n"(128 * G) : "memory");
      for (int i = 0; i < 4 * G; ++i) m = fmaxf(m, max_s[i]);
      const uint32_t e = __float_as_uint(m) >> 23;  // m is in [2^(e-127), 2^(e-126))
      unit = __uint_as_float((e > 6 ? 260 - e : 254) << 23);
      if (threadIdx.x == 64) unit_s = unit;
    }
    // the output's scale, and whether the adapters' factors may be divided by it
    float scale = 1.0f;
    if (c < a.cols) scale = a.n_scale == 0 ? 1.0f : a.n_scale == 1 ? a.scale[0] : BACK ? 1.0f / unit : a.scale[c];
    const bool divides = fabsf(scale) >= 0x1p-40f && fabsf(scale) <= 0x1p40f;

    // Group `group` of 4 warps takes every G-th 64-wide step: a thread one row of the weights.
    auto announce = [&](uint32_t slot) {
      wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) {
        if (P == 2 && side) mbar_arrive_at(ready + 8 * slot, 0);
        else mbar_arrive(ready + 8 * slot);
      }
    };
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    // P = 2: waits until the products of the stage's last use have ended, and where a step takes two slots' columns, those
    // of the group's last step, which lie in them and are later ones.
    static_assert(P == 1 || (kSlots == 8 && G == 4), "a group's last step is four stages back in a ring of eight");
    auto wait_free = [&](uint32_t s, uint32_t turn) {
      return wide ? mbar_wait(empty + 8 * (s ^ 4), s >= 4 ? turn : turn ^ 1, waits)
                  : mbar_wait(empty + 8 * s, turn ^ 1, waits);
    };
    bool ok = true;
    uint32_t g = group, s = group / KB, turn = 0;
    while (s >= a.stages) s -= a.stages, turn ^= 1;
    for (; g < steps; g += G) {
      const uint32_t k = g % KB, at = base + s * stage_bytes, slot = P == 2 ? s : g & slot_mask;
      if (wide) {
        // past the last term the scale is not read; the weights there are zeros
        const uint64_t j = (uint64_t)b0 * 64 * KB + (uint64_t)g * 64 + lane;
        const float x = j < a.n_scale ? a.scale[j] * unit : 0.0f, y = j + 32 < a.n_scale ? a.scale[j + 32] * unit : 0.0f;
        __syncwarp();
        scale_s[BACK ? w4 : 0][lane] = x;
        scale_s[BACK ? w4 : 0][lane + 32] = y;
        __syncwarp();
      }
      // A group skips the stage's uses by the others, and a barrier tells its phases apart by their parity alone: the
      // stage's last products have ended (which no phase can overtake, as this step is still to come), then its
      // load is the one waited for.  In wide steps the group waited for those products before its last step's stores.
      ok = (P == 1 || wide || wait_free(s, turn)) && mbar_wait(full + 8 * s, turn, waits);
      // P = 2: the stage was loaded after its last products ended, and with them the slot's
      if (P == 1 && !wide) ok = ok && mbar_wait(freed + 8 * slot, (g >> slot_bits & 1) ^ 1, waits);
      if (!ok) break;
      fence_after();
      if (!BACK) {
        uint32_t b[16], v[32];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const uint32_t chunk = k * 4 + h;
          const uint32_t off = KB == 2 ? row * 128 + ((chunk ^ (row & 7)) << 4)
                                       : row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(b[4 * h]), "=r"(b[4 * h + 1]), "=r"(b[4 * h + 2]), "=r"(b[4 * h + 3])
                       : "r"(at + off));
        }
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          v[2 * q] = widen2<T>(b[q]);
          v[2 * q + 1] = widen2<T>(b[q] >> 16);
        }
        tmem_st32(widened(slot) + lanes, v);
      } else {
        const uint32_t from = at + k * 64 * 128 + row;
        if (!wide) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t b[32], w[16];
#pragma unroll
            for (int j = 0; j < 32; ++j)
              asm volatile("ld.shared.u8 %0, [%1];" : "=r"(b[j]) : "r"(from + (half * 32 + j) * 128));
#pragma unroll
            for (int j = 0; j < 16; ++j) w[j] = widen2<T>(b[2 * j + 1] * 256u + b[2 * j]);
            tmem_st16(widened(slot) + half * 16 + lanes, w);
          }
        } else {
          // all of the thread's bytes, four to a word, and half of the products before the slot is waited for
          uint32_t b[16], w[16], rest[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            uint32_t x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) asm volatile("ld.shared.u8 %0, [%1];" : "=r"(x[i]) : "r"(from + (4 * j + i) * 128));
            b[j] = __byte_perm(x[1] * 256u + x[0], x[3] * 256u + x[2], 0x5410);
          }
          auto scaled = [&](int half) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 x = *reinterpret_cast<const float4*>(&scale_s[BACK ? w4 : 0][32 * half + 4 * j]);
              const float2 y = widen2_float(b[8 * half + j]), z = widen2_float(b[8 * half + j] >> 16);
              split_scaled<T>(y.x * x.x, y.y * x.y, w[2 * j], rest[2 * j]);
              split_scaled<T>(z.x * x.z, z.y * x.w, w[2 * j + 1], rest[2 * j + 1]);
            }
          };
          scaled(0);
          ok = P == 1 ? mbar_wait(freed + 8 * slot, (g >> slot_bits & 1) ^ 1, waits) : wait_free(s, turn);
          if (!ok) break;
          fence_after();
          tmem_st16(widened(slot) + lanes, w);
          tmem_st16(widened(slot) + 32 + lanes, rest);
          scaled(1);
          tmem_st16(widened(slot) + 16 + lanes, w);
          tmem_st16(widened(slot) + 48 + lanes, rest);
        }
      }
      announce(slot);
      if (KB == 1 || G >= KB) s += G / KB;
      else if (k == KB - 1) ++s;
      if (s >= a.stages) s -= a.stages, turn ^= 1;
    }

    find_adapters();
    if (P == 2) {
      // Adapter steps go on in the ring of stages: a thread widens two units' factors of its column into the slot, and
      // writes its rows' side of both where the stage's rows were.  What they read is fetched before the wait.
      const uint32_t chunks = (a.rank + 15) / 16;
      for (; g < steps + adapter_steps && ok; g += G) {
        const uint32_t first = (g - steps) * 2;
        uint32_t v[32] = {};
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (first + u < units) {
            const int32_t id = list[(first + u) / chunks];
            float f[16];
            bool fits = c < a.cols && divides;
            if (c < a.cols) fits = adapter_factor<T>(a, id, c, (first + u) % chunks * 16, a.alpha[id] / scale, f) && fits;
            if (fits)
#pragma unroll
              for (int q = 0; q < 8; ++q)
                split_pair<__nv_bfloat16>(f[2 * q], f[2 * q + 1], v[16 * u + q], v[16 * u + 8 + q]);
            else if (c < a.cols) apart_s = 1;
          }
        const uint32_t to = base + s * stage_bytes + w_bytes;
        bool waited = false;
        for (uint32_t x = threadIdx.x - 64 - group * 128; x < (rows_here * 2 + 127) / 128 * 128; x += 128) {
          const uint32_t t = x / 2, u = x % 2;
          uint32_t hi[8] = {}, lo[8] = {};
          if (t < rows_here && first + u < units && ids[side * rows_here + t] == list[(first + u) / chunks]) {
            float y[16];
            if (row_factor(a, t0 + side * rows_here + t, (first + u) % chunks * 16, y)) {
#pragma unroll
              for (int q = 0; q < 8; ++q) split_pair<__nv_bfloat16>(y[2 * q], y[2 * q + 1], hi[q], lo[q]);
            } else {
              for (uint32_t r = 0; r < 2; ++r) cluster_stu(smem_addr(&apart_s), r, 1);
            }
          }
          if (!waited) {
            ok = wait_free(s, turn);
            waited = true;
          }
          if (ok && t < rows_here)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t* z = q < 2 ? hi + 4 * q : lo + 4 * (q - 2);
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + t * 128 + (((u * 4 + q) ^ (t & 7)) << 4)),
                           "r"(z[0]), "r"(z[1]), "r"(z[2]), "r"(z[3])
                           : "memory");
            }
        }
        if (!ok) break;
        __syncwarp();
        fence_after();
        tmem_st32(widened(s) + lanes, v);
        fence_async();
        announce(s);
        s += G;
        if (s >= a.stages) s -= a.stages, turn ^= 1;
      }
    }
    ok = ok && mbar_wait(done, 0, waits);
    if (ok) fence_after();
    wait_predecessor();  // row_id and p are there, and nothing before this call reads the output any more
    share_apart();

    const uint32_t from = tmem + ((uint32_t)(quarter * 32) << 16);
    T* out = static_cast<T*>(a.out);
    if (split == 1) {
      const bool apart = P == 2 && apart_s;
      if (ok)
        for (uint32_t t = group * 16; t < a.bt; t += 16 * G) {
          if (t0 + t >= a.rows) break;
          float d[16];
          tmem_ld16(from + t, d);
          if (c >= a.cols) continue;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint64_t tt = t0 + t + j;
            if (tt >= a.rows) break;
            float y = d[j] * scale;
            if (a.rank && (P == 1 || apart)) {
              const int32_t id = P == 1 ? a.row_id[tt] : ids[t + j];
              if (id >= 0) y += P == 1 ? adapter_part<T>(a, id, tt, c, 0, a.rank) : left_out<T>(a, id, tt, c, scale, divides);
            }
            put(out + tt * a.out_stride + c, y);
          }
        }
    } else if (ok) {
      // the tile's sums into this CTA's shared memory: every stage has been consumed
      for (uint32_t t = group * 16; t < a.bt; t += 16 * G) {
        float d[16];
        tmem_ld16(from + t, d);
#pragma unroll
        for (int j = 0; j < 16; ++j)
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + ((t + j) * 128 + row) * 4), "f"(d[j]) : "memory");
      }
    }
  }
  if (split > 1) {
    __syncwarp();
    cluster_sync();
    // each CTA adds up and writes its share of the tile's rows, a thread four columns at a time
    if (warp >= 2 && !failed_s) {
      const uint32_t n = threadIdx.x - 64, row = n % 32 * 4;
      const uint64_t c = c0 + row;
      const uint32_t lo = a.bt * part / split, hi = a.bt * (part + 1) / split;
      float scale[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        scale[k] = 1.0f;
        if (c + k < a.cols)
          scale[k] = a.n_scale == 0 ? 1.0f : a.n_scale == 1 ? a.scale[0] : BACK ? 1.0f / unit_s : a.scale[c + k];
      }
      for (uint32_t t = lo + n / 32; t < hi; t += 4 * G) {
        const uint64_t tt = t0 + t;
        if (tt >= a.rows || c >= a.cols) continue;
        const float4 sum = cluster_sum4(base + (t * 128 + row) * 4, split);
        float y[4] = {sum.x * scale[0], sum.y * scale[1], sum.z * scale[2], sum.w * scale[3]};
        const int32_t id = a.rank ? a.row_id[tt] : -1;
        if (id >= 0)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (c + k < a.cols) y[k] += adapter_part<T>(a, id, tt, c + k, 0, a.rank);
        T* out = static_cast<T*>(a.out) + tt * a.out_stride + c;
        if (a.out_vector) {  // the columns are a multiple of 16
          *reinterpret_cast<uint2*>(out) = make_uint2(Widen<T>::pack(y[0], y[1]), Widen<T>::pack(y[2], y[3]));
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (c + k < a.cols) put(out + k, y[k]);
        }
      }
    }
  }
  __syncthreads();  // no wait of this CTA can fail any more
  if (failed_s) {
    if (warp == 0) drain_loads(full, next, next_turn, a.stages, waits);
    if (warp == 1 && side == 0) drain_products<P>(spent, crank, waits);
  }
  if (cluster > 1) {
    __syncwarp();
    cluster_sync();  // no CTA leaves while another reads its memory or arrives on its barriers
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 1) tmem_free<P>(tmem, columns);
  if (threadIdx.x == 0 && failed_s && a.status) atomicOr(a.status, ECF8_STATUS_TIMEOUT);
}

template <class T, int P, int KB, int G, int BACK>
int launch_form(const CUtensorMap& mw, const CUtensorMap& mq, const ProductArgs& a, dim3 grid, size_t smem,
                   bool overlap, cudaStream_t s) {
  static bool set[64] = {};
  if (const int rc = allow_smem(product_tc<T, P, KB, G, BACK>, set)) return rc;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(64 + 128 * G);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = P * a.split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = overlap ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, product_tc<T, P, KB, G, BACK>, mw, mq, a) == cudaSuccess ? ECF8_OK : ECF8_ERR_CUDA;
}

template <class T, int BACK>
int product_launch(bool pair, const CUtensorMap& mw, const CUtensorMap& mq, const ProductArgs& a, dim3 grid,
                   size_t smem, bool overlap, cudaStream_t s) {
  return pair ? launch_form<T, 2, 1, 4, BACK>(mw, mq, a, grid, smem, overlap, s)
              : launch_form<T, 1, 2, 2, BACK>(mw, mq, a, grid, smem, overlap, s);
}

}  // namespace ecf8_linear_impl

#endif  // ECF8_PRODUCT_CUH_
