// mhc_rows.h - device helpers of the row kernels (norm and write-back;
// internal, not part of the C ABI).
//
//  * chunks of 8 consecutive elements of a row, as fp32 in registers: a full
//    chunk is one 16-byte access (two for fp32) at any element alignment,
//    which gfx950 takes for global memory; the short chunk at the end of a
//    row whose length is no multiple of 8 goes element by element, so
//    nothing outside the row is touched and its missing elements read 0;
//  * fixed-order sums over a block: halving trees in each wave, then the
//    waves' results in ascending order. The order depends on the block size
//    alone.

#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mhc_convert.h"
#include "mhc_lanes.h"

namespace {

// Storage formats (the values of MHC_COEFF_F32 / _BF16 / _F16).
constexpr int kF32 = 0;
constexpr int kBF16 = 1;
constexpr int kF16 = 2;

template <int F>
struct Store {
  typedef uint16_t type;
};
template <>
struct Store<kF32> {
  typedef float type;
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// The same at element alignment, as they lie in a tensor of any width.
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef u32x4 u32x4_at4 __attribute__((aligned(4)));
typedef u32x2 u32x2_at1 __attribute__((aligned(1)));

template <int F>
__device__ __forceinline__ float widen(typename Store<F>::type v) {
  if constexpr (F == kF32) return v;
  else if constexpr (F == kBF16) return bf16_f32(v);
  else return f16_f32(v);
}

template <int F>
__device__ __forceinline__ typename Store<F>::type narrow(float v) {
  if constexpr (F == kF32) return v;
  else if constexpr (F == kBF16) return to_bf16(v);
  else return to_f16(v);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  return static_cast<uint32_t>(to_f16(lo)) | (static_cast<uint32_t>(to_f16(hi)) << 16);
}

// The raw words of one chunk: what a load brings and a later widen() reads,
// so that several chunks can be in flight before the first is used.
template <int F>
struct Chunk {
  u32x4 w[F == kF32 ? 2 : 1];
};

// p: first element of the chunk; count: elements of it that exist (>= 1).
// STREAM: the bytes are not read again (non-temporal).
template <int F, bool STREAM = false>
__device__ __forceinline__ Chunk<F> load_chunk(const typename Store<F>::type* p, int count) {
  Chunk<F> c;
  if (count >= 8) {
    if constexpr (F == kF32) {
      c.w[0] = *reinterpret_cast<const u32x4_at4*>(p);
      c.w[1] = *reinterpret_cast<const u32x4_at4*>(p + 4);
    } else {
      const u32x4_at2* v = reinterpret_cast<const u32x4_at2*>(p);
      c.w[0] = STREAM ? __builtin_nontemporal_load(v) : *v;
    }
    return c;
  }
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    u[i] = 0;
    if (i < count) {
      if constexpr (F == kF32) u[i] = __float_as_uint(p[i]);
      else u[i] = p[i];
    }
  }
  if constexpr (F == kF32) {
    c.w[0] = u32x4{u[0], u[1], u[2], u[3]};
    c.w[1] = u32x4{u[4], u[5], u[6], u[7]};
  } else {
    c.w[0] = u32x4{u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16};
  }
  return c;
}

template <int F>
__device__ __forceinline__ Chunk<F> zero_chunk() {
  Chunk<F> c;
  c.w[0] = u32x4{0, 0, 0, 0};
  if constexpr (F == kF32) c.w[1] = c.w[0];
  return c;
}

template <int F>
__device__ __forceinline__ void widen_chunk(const Chunk<F>& c, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F == kF32) {
      const uint32_t a = c.w[0][i], b = c.w[1][i];
      v[i] = __uint_as_float(a);
      v[4 + i] = __uint_as_float(b);
    } else {
      const uint32_t a = c.w[0][i];
      v[2 * i] = F == kBF16 ? lo_f32(a) : f16_f32(static_cast<uint16_t>(a));
      v[2 * i + 1] = F == kBF16 ? hi_f32(a) : f16_f32(static_cast<uint16_t>(a >> 16));
    }
  }
}

template <int F>
__device__ __forceinline__ void narrow_chunk(const float (&v)[8], Chunk<F>& c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F == kF32) {
      c.w[0][i] = __float_as_uint(v[i]);
      c.w[1][i] = __float_as_uint(v[4 + i]);
    } else if constexpr (F == kBF16) {
      c.w[0][i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    } else {
      c.w[0][i] = pack_f16x2(v[2 * i], v[2 * i + 1]);
    }
  }
}

// Rows are written once and in large part long before they are read: full
// chunks are stored non-temporally. T = 4096, H = 7168: norm forward 46.7 -> 43.5 us,
// streams to mx 66.9 -> 62.0, backward 49.2 -> 47.1; T = 1024 12.1 -> 11.1 and 17.8 -> 16.3;
// non-temporal loads of the same calls are slower (53.8, 70.2, 51.7).
template <int F>
__device__ __forceinline__ void store_chunk(typename Store<F>::type* p, int count,
                                            const Chunk<F>& c) {
  if (count >= 8) {
    if constexpr (F == kF32) {
      __builtin_nontemporal_store(c.w[0], reinterpret_cast<u32x4_at4*>(p));
      __builtin_nontemporal_store(c.w[1], reinterpret_cast<u32x4_at4*>(p + 4));
    } else {
      __builtin_nontemporal_store(c.w[0], reinterpret_cast<u32x4_at2*>(p));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i < count) {
      if constexpr (F == kF32) {
        const uint32_t a = c.w[i / 4][i % 4];
        p[i] = __uint_as_float(a);
      } else {
        p[i] = static_cast<uint16_t>(c.w[0][i / 2] >> (16 * (i % 2)));
      }
    }
  }
}

// Sum over a wave, in lane 0 (other lanes hold values that are not used):
// x[j] += x[j + off] for off = 32, 16, 8, 4, 2, 1.
__device__ __forceinline__ float wave_sum(float x) {
  x += from_lane_plus<32>(x);
  x += from_lane_plus<16>(x);
  x += from_lane_plus<8>(x);
  x += from_lane_plus<4>(x);
  x += from_lane_plus<2>(x);
  x += from_lane_plus<1>(x);
  return x;
}

__device__ __forceinline__ float wave_max(float x) {
  x = fmaxf(x, from_lane_plus<32>(x));
  x = fmaxf(x, from_lane_plus<16>(x));
  x = fmaxf(x, from_lane_plus<8>(x));
  x = fmaxf(x, from_lane_plus<4>(x));
  x = fmaxf(x, from_lane_plus<2>(x));
  x = fmaxf(x, from_lane_plus<1>(x));
  return x;
}

// Sum over the block, in every thread. `part` holds one float for each wave
// and is free for another use only after the block's next barrier.
template <int THREADS>
__device__ __forceinline__ float block_sum(float x, float* part) {
  x = wave_sum(x);
  if constexpr (THREADS == 64) {
    return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(x)));
  } else {
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = x;
    __syncthreads();
    float s = part[0];
#pragma unroll
    for (int w = 1; w < THREADS / 64; ++w) s += part[w];
    return s;
  }
}

template <int THREADS>
__device__ __forceinline__ float block_max(float x, float* part) {
  x = wave_max(x);
  if constexpr (THREADS == 64) {
    return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(x)));
  } else {
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = x;
    __syncthreads();
    float s = part[0];
#pragma unroll
    for (int w = 1; w < THREADS / 64; ++w) s = fmaxf(s, part[w]);
    return s;
  }
}

}  // namespace
