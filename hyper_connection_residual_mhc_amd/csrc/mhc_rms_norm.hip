// mhc_rms_norm.hip - root-mean-square norm with the residual's addition or the
// streams' collapse, 8-bit output with scales, and its backward, for gfx950
// (see include/mhc_rms_norm.h for the operation).

#include "mhc_rms_norm.h"

#include <math.h>

#include "mhc_host.h"
#include "mhc_launch.h"
#include "mhc_rows.h"

#ifdef __FAST_MATH__
#error "this source must not be built with fast-math"
#endif

#pragma clang fp contract(off)

namespace {

constexpr float kE4M3Max = 448.0f;
constexpr float kI8Max = 127.0f;

// Blocks of a launch at most; a block takes every gridDim.x-th row.
constexpr int64_t kMaxBlocks = 1 << 20;

// Rows of up to kHeld columns stay in registers between the two passes (the
// sum of squares, then the output): 2 chunks of 8 in each of 1024 threads.
// Longer rows are read twice.
constexpr int64_t kHeld = 1024 * 2 * 8;

// Where a row comes from: 0 = x, 1 = x + residual, 2 / 4 / 8 = streams.
constexpr int kPlain = 0;
constexpr int kAdd = 1;

// ---------------------------------------------------------------------------
// Pieces of both kernels
// ---------------------------------------------------------------------------

// weight[h .. h+8) as fp32, in the storage type F or in fp32.
template <int F>
__device__ __forceinline__ void load_weight(const void* weight, bool wide, int64_t h, int count,
                                            float (&w)[8]) {
  if (F == kF32 || wide) {
    widen_chunk<kF32>(load_chunk<kF32>(static_cast<const float*>(weight) + h, count), w);
  } else {
    widen_chunk<F>(load_chunk<F>(static_cast<const typename Store<F>::type*>(weight) + h, count),
                   w);
  }
}

// The same, raw: brought before the row's sum is known, widened after.
template <int F>
struct Weight {
  Chunk<kF32> wide;
  Chunk<F> same;
};

template <int F>
__device__ __forceinline__ Weight<F> start_weight(const void* weight, bool wide, int64_t h, int count) {
  Weight<F> w;
  if (F == kF32 || wide) w.wide = load_chunk<kF32>(static_cast<const float*>(weight) + h, count);
  else w.same = load_chunk<F>(static_cast<const typename Store<F>::type*>(weight) + h, count);
  return w;
}

template <int F>
__device__ __forceinline__ void take_weight(const Weight<F>& r, bool wide, float (&w)[8]) {
  if (F == kF32 || wide) widen_chunk<kF32>(r.wide, w);
  else widen_chunk<F>(r.same, w);
}

// Raw chunks of one row source.
template <int F, int SRC>
struct Source {
  Chunk<F> c[SRC >= 2 ? SRC : SRC + 1];
};

template <int F, int SRC>
__device__ __forceinline__ void load_source(const typename Store<F>::type* x,
                                            const typename Store<F>::type* residual, int64_t t,
                                            int64_t H, int64_t h, int count, Source<F, SRC>& s) {
  if constexpr (SRC >= 2) {
#pragma unroll
    for (int i = 0; i < SRC; ++i) s.c[i] = load_chunk<F>(x + (t * SRC + i) * H + h, count);
  } else {
    s.c[0] = load_chunk<F>(x + t * H + h, count);
    if constexpr (SRC == kAdd) s.c[1] = load_chunk<F>(residual + t * H + h, count);
  }
}

// The stored row: the source as one row of the storage type. The streams'
// collapse is that of mhc_h_aggregate.h: separate fp32 products and sums,
// adjacent pairs first.
template <int F, int SRC>
__device__ __forceinline__ Chunk<F> make_stored(const Source<F, SRC>& s, const float* p) {
  if constexpr (SRC == kPlain) {
    return s.c[0];
  } else {
    float a[8], b[8];
    Chunk<F> r;
    if constexpr (SRC == kAdd) {
      widen_chunk<F>(s.c[0], a);
      widen_chunk<F>(s.c[1], b);
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] = a[e] + b[e];
    } else {
      float v[SRC][8];
#pragma unroll
      for (int i = 0; i < SRC; ++i) {
        widen_chunk<F>(s.c[i], v[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = p[i] * v[i][e];
      }
#pragma unroll
      for (int step = 1; step < SRC; step *= 2)
#pragma unroll
        for (int i = 0; i < SRC; i += 2 * step)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] = v[i][e] + v[i + step][e];
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] = v[0][e];
    }
    narrow_chunk<F>(a, r);
    return r;
  }
}

// Eight fp32 values as e4m3 (gfx950's conversion: OCP format, nearest even).
__device__ __forceinline__ u32x2 pack_e4m3(const float (&v)[8]) {
  u32x2 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], w, true);
    r[i] = static_cast<uint32_t>(w);
  }
  return r;
}

// Eight fp32 values of at most 127 as 8-bit integers, nearest even.
__device__ __forceinline__ u32x2 pack_i8(const float (&v)[8]) {
  u32x2 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w |= (static_cast<uint32_t>(static_cast<int>(rintf(v[4 * i + e]))) & 0xFFu) << (8 * e);
    r[i] = w;
  }
  return r;
}

__device__ __forceinline__ void store_codes(uint8_t* p, int count, u32x2 c) {
  if (count >= 8) {
    __builtin_nontemporal_store(c, reinterpret_cast<u32x2_at1*>(p));
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < count) p[i] = static_cast<uint8_t>(c[i / 4] >> (8 * (i % 4)));
}

__device__ __forceinline__ float amax8(const float (&v)[8]) {
  float a = fabsf(v[0]);
#pragma unroll
  for (int e = 1; e < 8; ++e) a = fmaxf(a, fabsf(v[e]));
  return a;
}

// The block's power p: the smallest in [-127, 127] with amax <= 448 * 2^p.
// 448 = 1.75 * 2^8, so p is amax's exponent - 8, one more where its
// significand is over 1.75. Subnormals of amax give the lowest power.
__device__ __forceinline__ int mx_power(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int p = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(-127, min(127, p));
}

// 2^-p for p in [-127, 127].
__device__ __forceinline__ float exp2_neg(int p) {
  return p == 127 ? __uint_as_float(0x00400000u) : __uint_as_float(static_cast<uint32_t>(127 - p) << 23);
}

// ---------------------------------------------------------------------------
// Forward
//
// Bound by memory. One block takes one row and holds it in registers (as
// stored, 16 bytes a chunk) while the sum of squares is joined, so every
// source byte is read once and every output byte written once; ITER chunks of
// a thread are in flight together. ITER = 0 is the form for rows longer than
// the registers hold, which makes the row again from its sources.
// ---------------------------------------------------------------------------
template <int F, int SRC, int FMT, int THREADS, int ITER>
__global__ __launch_bounds__(THREADS) void rms_norm_fwd_kernel(
    const typename Store<F>::type* __restrict__ x,
    const typename Store<F>::type* __restrict__ residual, const float* __restrict__ pre,
    const void* __restrict__ weight, int wide_weight, float eps, void* __restrict__ out,
    void* __restrict__ scales, typename Store<F>::type* __restrict__ stored,
    float* __restrict__ rstd, int64_t T, int64_t H) {
  constexpr int kStep = THREADS * 8;
  constexpr bool kKeep = ITER > 0;
  constexpr int kUnroll = kKeep ? ITER : 1;
  __shared__ float part[2][THREADS / 64];
  const int64_t iters = kKeep ? ITER : (H + kStep - 1) / kStep;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    float p[SRC >= 2 ? SRC : 1];
    if constexpr (SRC >= 2) {
#pragma unroll
      for (int i = 0; i < SRC; ++i) p[i] = pre[t * SRC + i];
    }
    Chunk<F> held[kKeep ? ITER : 1];
    float sum = 0.0f;
    const auto first = [&](int64_t k, const Source<F, SRC>& src, int64_t h, int count) {
      const Chunk<F> c = make_stored<F, SRC>(src, p);
      if (SRC != kPlain && stored != nullptr) store_chunk<F>(stored + t * H + h, count, c);
      float v[8];
      widen_chunk<F>(c, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(v[e], v[e], sum);
      if constexpr (kKeep) held[k] = c;
    };
    if constexpr (kKeep) {
      // all of the thread's loads together, but for eight streams of two chunks
      // (64 registers for them alone)
      constexpr int kSets = SRC >= 8 ? 1 : ITER;
      Source<F, SRC> src[kSets];
#pragma unroll
      for (int k = 0; k < ITER; ++k) {
        const int64_t h = k * kStep + threadIdx.x * 8;
        held[k] = zero_chunk<F>();
        if (kSets == ITER && h < H)
          load_source<F, SRC>(x, residual, t, H, h, static_cast<int>(min(H - h, static_cast<int64_t>(8))), src[k % kSets]);
      }
#pragma unroll
      for (int k = 0; k < ITER; ++k) {
        const int64_t h = k * kStep + threadIdx.x * 8;
        const int count = static_cast<int>(min(H - h, static_cast<int64_t>(8)));
        if (kSets != ITER && h < H) load_source<F, SRC>(x, residual, t, H, h, count, src[0]);
        if (h < H) first(k, src[k % kSets], h, count);
      }
    } else {
      for (int64_t h = threadIdx.x * 8; h < H; h += kStep) {
        const int count = static_cast<int>(min(H - h, static_cast<int64_t>(8)));
        Source<F, SRC> src;
        load_source<F, SRC>(x, residual, t, H, h, count, src);
        first(0, src, h, count);
      }
    }
    Weight<F> kw[kKeep ? ITER : 1];
    if constexpr (kKeep) {
#pragma unroll
      for (int k = 0; k < ITER; ++k) {
        const int64_t h = k * kStep + threadIdx.x * 8;
        if (h < H)
          kw[k] = start_weight<F>(weight, wide_weight != 0, h, static_cast<int>(min(H - h, static_cast<int64_t>(8))));
      }
    }
    sum = block_sum<THREADS>(sum, part[0]);
    const float r = 1.0f / sqrtf(sum / static_cast<float>(H) + eps);
    if (rstd != nullptr && threadIdx.x == 0) rstd[t] = r;

    // The chunk at column h of the row, normed: kept, or made again.
    const auto value = [&](int64_t k, int64_t h, int count, float (&v)[8]) {
      if constexpr (kKeep) {
        widen_chunk<F>(held[k], v);
      } else {
        Source<F, SRC> src;
        load_source<F, SRC>(x, residual, t, H, h, count, src);
        widen_chunk<F>(make_stored<F, SRC>(src, p), v);
      }
      float w[8];
      if constexpr (kKeep) take_weight<F>(kw[k], wide_weight != 0, w);
      else load_weight<F>(weight, wide_weight != 0, h, count, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = v[e] * r * w[e];
    };

    if constexpr (FMT == MHC_NORM_SAME) {
#pragma unroll kUnroll
      for (int64_t k = 0; k < iters; ++k) {
        const int64_t h = k * kStep + threadIdx.x * 8;
        if (h < H) {
          const int count = static_cast<int>(min(H - h, static_cast<int64_t>(8)));
          float v[8];
          value(k, h, count, v);
          Chunk<F> c;
          narrow_chunk<F>(v, c);
          store_chunk<F>(static_cast<typename Store<F>::type*>(out) + t * H + h, count, c);
        }
      }
    } else if constexpr (FMT == MHC_NORM_E4M3_ROW || FMT == MHC_NORM_I8_ROW) {
      // The normed row in registers where it fits them, else computed twice.
      float kept[kKeep ? ITER : 1][8];
      float amax = 0.0f;
#pragma unroll kUnroll
      for (int64_t k = 0; k < iters; ++k) {
        const int64_t h = k * kStep + threadIdx.x * 8;
        float(&v)[8] = kept[kKeep ? k : 0];
        if (h < H) {
          value(k, h, static_cast<int>(min(H - h, static_cast<int64_t>(8))), v);
          amax = fmaxf(amax, amax8(v));
          if constexpr (FMT == MHC_NORM_I8_ROW) {
            // integers have no NaN: the row's scale says that there is one
#pragma unroll
            for (int e = 0; e < 8; ++e) amax = v[e] != v[e] ? INFINITY : amax;
          }
        }
      }
      amax = block_max<THREADS>(amax, part[1]);
      const float scale = fmaxf(amax / (FMT == MHC_NORM_I8_ROW ? kI8Max : kE4M3Max), 0x1p-126f);
      const float inverse = 1.0f / scale;
      if (threadIdx.x == 0) static_cast<float*>(scales)[t] = scale;
#pragma unroll kUnroll
      for (int64_t k = 0; k < iters; ++k) {
        const int64_t h = k * kStep + threadIdx.x * 8;
        if (h < H) {
          const int count = static_cast<int>(min(H - h, static_cast<int64_t>(8)));
          float(&v)[8] = kept[kKeep ? k : 0];
          if constexpr (!kKeep) value(k, h, count, v);
          if constexpr (FMT == MHC_NORM_I8_ROW) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = scale == INFINITY ? 0.0f : v[e] * inverse;
            store_codes(static_cast<uint8_t*>(out) + t * H + h, count, pack_i8(v));
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = v[e] * inverse;
            store_codes(static_cast<uint8_t*>(out) + t * H + h, count, pack_e4m3(v));
          }
        }
      }
    } else {
      const int64_t blocks = (H + 31) / 32;
#pragma unroll kUnroll
      for (int64_t k = 0; k < iters; ++k) {
        const int64_t h = k * kStep + threadIdx.x * 8;
        const bool in = h < H;
        const int count = in ? static_cast<int>(min(H - h, static_cast<int64_t>(8))) : 0;
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (in) value(k, h, count, v);
        // a block is the 32 columns of four neighbouring lanes
        float a = amax8(v);
        a = fmaxf(a, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(a), 0xB1, 0xF, 0xF, false)));
        a = fmaxf(a, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(a), 0x4E, 0xF, 0xF, false)));
        const int power = mx_power(a);
        const float inverse = exp2_neg(power);
        if (in) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = v[e] * inverse;
          store_codes(static_cast<uint8_t*>(out) + t * H + h, count, pack_e4m3(v));
          if (threadIdx.x % 4 == 0)
            static_cast<uint8_t*>(scales)[t * blocks + h / 32] =
                static_cast<uint8_t>(a == INFINITY ? 255 : power + 127);
        }
      }
    }
    if constexpr (THREADS > 64) __syncthreads();  // `part` is written again for the next row
  }
}

// ---------------------------------------------------------------------------
// Backward
//
// Bound by memory: grad_y, s and grad_stored are read once and grad_x written
// once. A block takes every gridDim.x-th row, with the next row's loads under
// this one's sums, and keeps the weight and its part of the weight's gradient
// in registers over all of them (8 ITER each a thread); the blocks' parts go to
// the workspace once, at the end, and a second kernel adds them in ascending
// order of the block. The number of blocks depends on T and H alone (bwd_blocks).
// Rows of up to kFused columns: longer ones leave no room for all this.
// ---------------------------------------------------------------------------
template <int F, int THREADS, int ITER>
__global__ __launch_bounds__(THREADS) void rms_norm_bwd_kernel(
    const typename Store<F>::type* __restrict__ grad_y,
    const typename Store<F>::type* __restrict__ stored, const void* __restrict__ weight,
    int wide_weight, const float* __restrict__ rstd,
    const typename Store<F>::type* __restrict__ grad_stored,
    typename Store<F>::type* __restrict__ grad_x, float* __restrict__ partial, int64_t T,
    int64_t H) {
  constexpr int kStep = THREADS * 8;
  __shared__ float part[2][THREADS / 64];
  // chunk k of a row: its first column, and how many of its 8 exist
  const auto column = [&](int k) { return static_cast<int64_t>(k) * kStep + threadIdx.x * 8; };
  const auto count_of = [&](int k) {
    return static_cast<int>(min(H - column(k), static_cast<int64_t>(8)));
  };
  struct Row {
    Chunk<F> g[ITER], s[ITER], gs[ITER];
    float r;
  };
  float w[ITER][8], dw[ITER][8];
#pragma unroll
  for (int k = 0; k < ITER; ++k) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[k][e] = dw[k][e] = 0.0f;
    if (column(k) < H) load_weight<F>(weight, wide_weight != 0, column(k), count_of(k), w[k]);
  }
  const auto load = [&](int64_t t, Row& row) {
    row.r = rstd[t];
#pragma unroll
    for (int k = 0; k < ITER; ++k) {
      row.g[k] = row.s[k] = row.gs[k] = zero_chunk<F>();
      if (column(k) < H) {
        row.g[k] = load_chunk<F>(grad_y + t * H + column(k), count_of(k));
        row.s[k] = load_chunk<F>(stored + t * H + column(k), count_of(k));
        if (grad_stored != nullptr)
          row.gs[k] = load_chunk<F>(grad_stored + t * H + column(k), count_of(k));
      }
    }
  };
  const auto pass = [&](int64_t t, const Row& row, float* sums) {
    float dot = 0.0f;
#pragma unroll
    for (int k = 0; k < ITER; ++k) {
      float g[8], s[8];
      widen_chunk<F>(row.g[k], g);
      widen_chunk<F>(row.s[k], s);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dot = fmaf(g[e] * w[k][e], s[e], dot);
        dw[k][e] = fmaf(g[e], s[e] * row.r, dw[k][e]);
      }
    }
    dot = block_sum<THREADS>(dot, sums);
    const float c = dot / static_cast<float>(H) * (row.r * row.r);
#pragma unroll
    for (int k = 0; k < ITER; ++k) {
      if (column(k) < H) {
        float g[8], s[8], gs[8], o[8];
        widen_chunk<F>(row.g[k], g);
        widen_chunk<F>(row.s[k], s);
        widen_chunk<F>(row.gs[k], gs);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = row.r * fmaf(-s[e], c, g[e] * w[k][e]);
        if (grad_stored != nullptr) {
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = o[e] + gs[e];
        }
        Chunk<F> q;
        narrow_chunk<F>(o, q);
        store_chunk<F>(grad_x + t * H + column(k), count_of(k), q);
      }
    }
  };
  // Rows in pairs, each row's sums in LDS of its own: a wave that writes a
  // row's finds every wave past the sums of the row two before.
  Row a, b;
  int64_t t = blockIdx.x;
  if (t < T) load(t, a);
  while (t < T) {
    const int64_t t1 = t + gridDim.x, t2 = t1 + gridDim.x;
    if (t1 < T) load(t1, b);
    pass(t, a, part[0]);
    if (t1 >= T) break;
    if (t2 < T) load(t2, a);
    pass(t1, b, part[1]);
    t = t2;
  }
#pragma unroll
  for (int k = 0; k < ITER; ++k) {
    if (column(k) < H) {
      Chunk<kF32> c;
      narrow_chunk<kF32>(dw[k], c);
      store_chunk<kF32>(partial + blockIdx.x * H + column(k), count_of(k), c);
    }
  }
}

// Longer rows: grad_x alone, a block to a row, ITER chunks of a thread held in
// registers between the two passes (ITER = 0: read again) ...
template <int F, int THREADS, int ITER>
__global__ __launch_bounds__(THREADS) void rms_norm_bwd_row_kernel(
    const typename Store<F>::type* __restrict__ grad_y,
    const typename Store<F>::type* __restrict__ stored, const void* __restrict__ weight,
    int wide_weight, const float* __restrict__ rstd,
    const typename Store<F>::type* __restrict__ grad_stored,
    typename Store<F>::type* __restrict__ grad_x, int64_t T, int64_t H) {
  constexpr int kStep = THREADS * 8;
  constexpr bool kKeep = ITER > 0;
  constexpr int kSets = kKeep ? ITER : 1;
  __shared__ float part[THREADS / 64];
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    const float r = rstd[t];
    Chunk<F> cg[kSets], cs[kSets], cgs[kSets];
    const auto load = [&](int64_t h, int k) {
      const int count = static_cast<int>(min(H - h, static_cast<int64_t>(8)));
      cg[k] = load_chunk<F>(grad_y + t * H + h, count);
      cs[k] = load_chunk<F>(stored + t * H + h, count);
    };
    const auto load_more = [&](int64_t h, int k) {
      cgs[k] = zero_chunk<F>();
      if (grad_stored != nullptr)
        cgs[k] = load_chunk<F>(grad_stored + t * H + h, static_cast<int>(min(H - h, static_cast<int64_t>(8))));
    };
    float dot = 0.0f;
    const auto add = [&](int64_t h, int k) {
      float g[8], s[8], w[8];
      widen_chunk<F>(cg[k], g);
      widen_chunk<F>(cs[k], s);
      load_weight<F>(weight, wide_weight != 0, h, static_cast<int>(min(H - h, static_cast<int64_t>(8))), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) dot = fmaf(g[e] * w[e], s[e], dot);
    };
    if constexpr (kKeep) {
#pragma unroll
      for (int k = 0; k < ITER; ++k) {
        const int64_t h = static_cast<int64_t>(k) * kStep + threadIdx.x * 8;
        if (h < H) {
          load(h, k);
          load_more(h, k);
        }
      }
#pragma unroll
      for (int k = 0; k < ITER; ++k) {
        const int64_t h = static_cast<int64_t>(k) * kStep + threadIdx.x * 8;
        if (h < H) add(h, k);
      }
    } else {
      for (int64_t h = threadIdx.x * 8; h < H; h += kStep) {
        load(h, 0);
        add(h, 0);
      }
    }
    dot = block_sum<THREADS>(dot, part);
    const float c = dot / static_cast<float>(H) * (r * r);
    const auto write = [&](int64_t h, int k) {
      const int count = static_cast<int>(min(H - h, static_cast<int64_t>(8)));
      float g[8], s[8], w[8], gs[8], o[8];
      widen_chunk<F>(cg[k], g);
      widen_chunk<F>(cs[k], s);
      widen_chunk<F>(cgs[k], gs);
      load_weight<F>(weight, wide_weight != 0, h, count, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = r * fmaf(-s[e], c, g[e] * w[e]);
      if (grad_stored != nullptr) {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = o[e] + gs[e];
      }
      Chunk<F> q;
      narrow_chunk<F>(o, q);
      store_chunk<F>(grad_x + t * H + h, count, q);
    };
    if constexpr (kKeep) {
#pragma unroll
      for (int k = 0; k < ITER; ++k) {
        const int64_t h = static_cast<int64_t>(k) * kStep + threadIdx.x * 8;
        if (h < H) write(h, k);
      }
    } else {
      for (int64_t h = threadIdx.x * 8; h < H; h += kStep) {
        load(h, 0);
        load_more(h, 0);
        write(h, 0);
      }
    }
    __syncthreads();  // `part` is written again for the next row
  }
}

// ... and parts of the weight's gradient: 2048 columns and `rows` rows to a
// block, each column's rows in ascending order, four rows' loads in flight.
template <int F>
__global__ __launch_bounds__(256) void rms_norm_bwd_weight_kernel(
    const typename Store<F>::type* __restrict__ grad_y,
    const typename Store<F>::type* __restrict__ stored, const float* __restrict__ rstd,
    float* __restrict__ partial, int64_t T, int64_t H, int64_t rows) {
  constexpr int kAhead = 4;
  const int64_t h = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (h >= H) return;
  const int count = static_cast<int>(min(H - h, static_cast<int64_t>(8)));
  const int64_t t0 = blockIdx.y * rows, t1 = min(T, t0 + rows);
  float dw[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int64_t t = t0; t < t1; t += kAhead) {
    Chunk<F> cg[kAhead], cs[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (t + k < t1) {
        cg[k] = load_chunk<F>(grad_y + (t + k) * H + h, count);
        cs[k] = load_chunk<F>(stored + (t + k) * H + h, count);
      }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (t + k < t1) {
        const float r = rstd[t + k];
        float g[8], s[8];
        widen_chunk<F>(cg[k], g);
        widen_chunk<F>(cs[k], s);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[e] = fmaf(g[e], s[e] * r, dw[e]);
      }
  }
  Chunk<kF32> c;
  narrow_chunk<kF32>(dw, c);
  store_chunk<kF32>(partial + blockIdx.y * H + h, count, c);
}

// grad_weight[h] = sum over the blocks' parts: 16 columns to a block, each of 64
// threads of a column adds every 64th part in ascending order, then the 64
// results are added in ascending order, 8 by 8. With no parts the sums are +0.0.
__global__ __launch_bounds__(1024) void rms_norm_bwd_reduce_kernel(const float* __restrict__ partial,
                                                                   float* __restrict__ grad_weight,
                                                                   int64_t parts, int64_t H) {
  __shared__ float sums[64][17];
  __shared__ float groups[8][16];
  const int column = threadIdx.x % 16, lane = threadIdx.x / 16;
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * 16; first < H; first += gridDim.x * 16) {
    const int64_t h = first + column;
    float s = 0.0f;
    if (h < H) {
#pragma unroll 8
      for (int64_t k = lane; k < parts; k += 64) s += partial[k * H + h];
    }
    sums[lane][column] = s;
    __syncthreads();
    if (lane < 8) {
      s = sums[8 * lane][column];
#pragma unroll
      for (int k = 1; k < 8; ++k) s += sums[8 * lane + k][column];
      groups[lane][column] = s;
    }
    __syncthreads();
    if (lane == 0 && h < H) {
      s = groups[0][column];
#pragma unroll
      for (int k = 1; k < 8; ++k) s += groups[k][column];
      grad_weight[h] = s;
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

int64_t size_of(int32_t dtype) { return dtype == MHC_NORM_F32 ? 4 : 2; }

bool known(int32_t dtype) {
  return dtype == MHC_NORM_F32 || dtype == MHC_NORM_BF16 || dtype == MHC_NORM_F16;
}

mhc_status check_sizes(int64_t T, int64_t H, int32_t dtype, int32_t weight_dtype) {
  if (T < 0) return fail(MHC_ERROR_INVALID_VALUE, "T must not be negative");
  if (H < 1 || H > MHC_MAX_H)
    return fail(MHC_ERROR_INVALID_VALUE, "H must be in [1, %lld] (got %lld)", MHC_MAX_H,
                static_cast<long long>(H));
  if (!known(dtype))
    return fail(MHC_ERROR_INVALID_VALUE, "dtype must be MHC_NORM_F32, _BF16 or _F16 (got %d)",
                dtype);
  if (weight_dtype != dtype && weight_dtype != MHC_NORM_F32)
    return fail(MHC_ERROR_INVALID_VALUE, "weight_dtype must be dtype or MHC_NORM_F32 (got %d)",
                weight_dtype);
  return ok();
}

mhc_status validate_fwd(const void* x, const void* residual, const void* pre, int32_t n,
                        const void* weight, int32_t weight_dtype, float eps, const void* out,
                        const void* scales, const void* stored, const void* rstd, int64_t T,
                        int64_t H, int32_t dtype, int32_t out_format) {
  const mhc_status st = check_sizes(T, H, dtype, weight_dtype);
  if (st != MHC_SUCCESS) return st;
  if (out_format != MHC_NORM_SAME && out_format != MHC_NORM_E4M3_ROW &&
      out_format != MHC_NORM_E4M3_MX && out_format != MHC_NORM_I8_ROW)
    return fail(MHC_ERROR_INVALID_VALUE,
                "out_format must be MHC_NORM_SAME, _E4M3_ROW, _E4M3_MX or _I8_ROW (got %d)", out_format);
  if (!(eps >= 0.0f) || !isfinite(eps))
    return fail(MHC_ERROR_INVALID_VALUE, "eps must be finite and not negative (got %g)",
                static_cast<double>(eps));
  if (residual != nullptr && pre != nullptr)
    return fail(MHC_ERROR_INVALID_VALUE, "residual and pre exclude each other");
  if (pre != nullptr ? (n != 2 && n != 4 && n != 8) : n != 0)
    return fail(MHC_ERROR_INVALID_VALUE,
                "the expansion rate n must be 2, 4 or 8 with pre and 0 without (got %d)", n);
  if (pre != nullptr && dtype != MHC_NORM_BF16)
    return fail(MHC_ERROR_INVALID_VALUE, "streams must be bf16");
  if (stored != nullptr && residual == nullptr && pre == nullptr)
    return fail(MHC_ERROR_INVALID_VALUE, "stored needs a residual or pre (the row is x itself)");
  if (T == 0) return ok();
  if (out_format == MHC_NORM_SAME && scales != nullptr)
    return fail(MHC_ERROR_INVALID_VALUE, "MHC_NORM_SAME has no scales");
  const int64_t E = size_of(dtype);
  const bool e8 = out_format != MHC_NORM_SAME;
  const int64_t row = mul_bytes(T, H, E);
  const bool rows = out_format == MHC_NORM_E4M3_ROW || out_format == MHC_NORM_I8_ROW;
  const int64_t scale_bytes = rows                             ? mul_bytes(T, 4, 1)
                              : out_format == MHC_NORM_E4M3_MX ? mul_bytes(T, (H + 31) / 32, 1)
                                                               : 0;
  const Tensor in[] = {{x, mul_bytes(T, H, pre != nullptr ? E * n : E), E, "x"},
                       {residual, residual != nullptr ? row : 0, E, "residual"},
                       {pre, pre != nullptr ? mul_bytes(T, n, 4) : 0, 4, "pre"},
                       {weight, H * size_of(weight_dtype), size_of(weight_dtype), "weight"}};
  const Tensor outs[] = {{out, e8 ? mul_bytes(T, H, 1) : row, e8 ? 1 : E, "out"},
                         {scales, scale_bytes, rows ? 4 : 1, "scales"},
                         {stored, stored != nullptr ? row : 0, E, "stored"},
                         {rstd, rstd != nullptr ? mul_bytes(T, 4, 1) : 0, 4, "rstd"}};
  return check_tensors(in, outs);
}

struct FwdArgs {
  const void *x, *residual;
  const float* pre;
  const void* weight;
  int wide;
  float eps;
  void *out, *scales, *stored;
  float* rstd;
  int64_t T, H;
  hipStream_t s;
  hipEvent_t start, stop;
};

template <int F, int SRC, int FMT, int THREADS, int ITER>
hipError_t launch_fwd(const FwdArgs& a) {
  const int64_t blocks = a.T < kMaxBlocks ? a.T : kMaxBlocks;
  return launch_kernel(rms_norm_fwd_kernel<F, SRC, FMT, THREADS, ITER>,
                       dim3(static_cast<uint32_t>(blocks)), dim3(THREADS), a.s, a.start, a.stop,
                       static_cast<const typename Store<F>::type*>(a.x),
                       static_cast<const typename Store<F>::type*>(a.residual), a.pre, a.weight,
                       a.wide, a.eps, a.out, a.scales,
                       static_cast<typename Store<F>::type*>(a.stored), a.rstd, a.T, a.H);
}

// The block by the row's length alone, so that a row's sums have one order:
// the fewest threads up to 512 that hold it in one chunk each, then 512 and
// 1024 with two, then rows that are read twice. T = 4096, H = 7168: one chunk in each of 1024 threads
// is slower (the sum to e4m3 rows 46.9 us, two in each of 512 35.0).
template <int F, int SRC, int FMT>
hipError_t launch_fwd_h(const FwdArgs& a) {
  if (a.H <= 64 * 8) return launch_fwd<F, SRC, FMT, 64, 1>(a);
  if (a.H <= 128 * 8) return launch_fwd<F, SRC, FMT, 128, 1>(a);
  if (a.H <= 256 * 8) return launch_fwd<F, SRC, FMT, 256, 1>(a);
  if (a.H <= 512 * 8) return launch_fwd<F, SRC, FMT, 512, 1>(a);
  if (a.H <= 512 * 16) return launch_fwd<F, SRC, FMT, 512, 2>(a);
  if (a.H <= kHeld) return launch_fwd<F, SRC, FMT, 1024, 2>(a);
  return launch_fwd<F, SRC, FMT, 512, 0>(a);
}

template <int F, int SRC>
hipError_t launch_fwd_f(const FwdArgs& a, int32_t fmt) {
  if (fmt == MHC_NORM_SAME) return launch_fwd_h<F, SRC, MHC_NORM_SAME>(a);
  if (fmt == MHC_NORM_E4M3_ROW) return launch_fwd_h<F, SRC, MHC_NORM_E4M3_ROW>(a);
  if (fmt == MHC_NORM_I8_ROW) return launch_fwd_h<F, SRC, MHC_NORM_I8_ROW>(a);
  return launch_fwd_h<F, SRC, MHC_NORM_E4M3_MX>(a);
}

template <int F>
hipError_t launch_fwd_s(const FwdArgs& a, int32_t fmt) {
  return a.residual != nullptr ? launch_fwd_f<F, kAdd>(a, fmt) : launch_fwd_f<F, kPlain>(a, fmt);
}

// Blocks of the backward: enough waves for the 256 CUs, each block with its own
// part of the weight's gradient in the workspace (8 MiB in all at most). bf16 with
// grad_stored, blocks against half and twice as many: T = 4096, H = 7168: 256 44.9 us (512 47.8);
// T = 8192, H = 2048: 512 26.1 (1024 28.8); T = 8192, H = 512: 1024 13.5 (512 15.8, 4096 24.0).
int64_t bwd_blocks(int64_t T, int64_t H) {
  const int64_t blocks = H <= 1024 ? 1024 : H <= 4096 ? 512 : 256;
  return T < blocks ? T : blocks;
}

// Rows of up to this many columns have both gradients from one kernel.
constexpr int64_t kFused = 512 * 2 * 8;

// Longer ones: rows of a block of the weight's kernel, about 1024 blocks in all of
// at least 32 rows.
int64_t weight_rows(int64_t T, int64_t H) {
  const int64_t wide = (H + 2047) / 2048;
  const int64_t parts = wide >= 1024 ? 1 : 1024 / wide;
  const int64_t rows = (T + parts - 1) / parts;
  return rows < 32 ? 32 : rows;
}

int64_t workspace_parts(int64_t T, int64_t H) {
  if (H <= kFused) return bwd_blocks(T, H);
  const int64_t rows = weight_rows(T, H);
  return (T + rows - 1) / rows;
}

int64_t workspace_need(int64_t T, int64_t H) { return workspace_parts(T, H) * H * 4; }

mhc_status validate_bwd(const void* grad_y, const void* stored, const void* weight,
                        int32_t weight_dtype, const void* rstd, const void* grad_stored,
                        const void* grad_x, const void* grad_weight, const void* workspace,
                        int64_t workspace_bytes, int64_t T, int64_t H, int32_t dtype) {
  const mhc_status st = check_sizes(T, H, dtype, weight_dtype);
  if (st != MHC_SUCCESS) return st;
  const int64_t need = workspace_need(T, H);
  if (workspace_bytes < need)
    return fail(MHC_ERROR_INVALID_VALUE, "workspace_bytes %lld < %lld needed",
                static_cast<long long>(workspace_bytes), static_cast<long long>(need));
  const int64_t E = size_of(dtype), row = mul_bytes(T, H, E);
  const Tensor in[] = {{grad_y, row, E, "grad_y"},
                       {stored, row, E, "stored"},
                       {weight, T > 0 ? H * size_of(weight_dtype) : 0, size_of(weight_dtype), "weight"},
                       {rstd, mul_bytes(T, 4, 1), 4, "rstd"},
                       {grad_stored, grad_stored != nullptr ? row : 0, E, "grad_stored"}};
  const Tensor outs[] = {{grad_x, row, E, "grad_x"},
                         {grad_weight, H * 4, 4, "grad_weight"},
                         {workspace, need, 4, "workspace"}};
  return check_tensors(in, outs);
}

struct BwdArgs {
  const void *grad_y, *stored, *weight;
  int wide;
  const float* rstd;
  const void* grad_stored;
  void* grad_x;
  float *grad_weight, *partial;
  int64_t T, H;
  hipStream_t s;
  hipEvent_t start, stop;
};

hipError_t launch_reduce(const BwdArgs& a, int64_t parts, hipEvent_t start) {
  const int64_t blocks = (a.H + 15) / 16;
  return launch_kernel(rms_norm_bwd_reduce_kernel,
                       dim3(static_cast<uint32_t>(blocks < kMaxBlocks ? blocks : kMaxBlocks)), dim3(1024), a.s, start, a.stop, a.partial, a.grad_weight, parts, a.H);
}

template <int F, int THREADS, int ITER>
hipError_t launch_bwd(const BwdArgs& a) {
  typedef typename Store<F>::type S;
  const int64_t blocks = bwd_blocks(a.T, a.H);
  const hipError_t e = launch_kernel(
      rms_norm_bwd_kernel<F, THREADS, ITER>, dim3(static_cast<uint32_t>(blocks)), dim3(THREADS),
      a.s, a.start, nullptr, static_cast<const S*>(a.grad_y), static_cast<const S*>(a.stored),
      a.weight, a.wide, a.rstd, static_cast<const S*>(a.grad_stored), static_cast<S*>(a.grad_x),
      a.partial, a.T, a.H);
  return e != hipSuccess ? e : launch_reduce(a, blocks, nullptr);
}

template <int F, int THREADS, int ITER>
hipError_t launch_bwd_row(const BwdArgs& a) {
  typedef typename Store<F>::type S;
  const int64_t blocks = a.T < kMaxBlocks ? a.T : kMaxBlocks;
  hipError_t e = launch_kernel(
      rms_norm_bwd_row_kernel<F, THREADS, ITER>, dim3(static_cast<uint32_t>(blocks)),
      dim3(THREADS), a.s, a.start, nullptr, static_cast<const S*>(a.grad_y),
      static_cast<const S*>(a.stored), a.weight, a.wide, a.rstd,
      static_cast<const S*>(a.grad_stored), static_cast<S*>(a.grad_x), a.T, a.H);
  if (e != hipSuccess) return e;
  const int64_t rows = weight_rows(a.T, a.H), parts = workspace_parts(a.T, a.H);
  e = launch_kernel(rms_norm_bwd_weight_kernel<F>,
                    dim3(static_cast<uint32_t>((a.H + 2047) / 2048), static_cast<uint32_t>(parts)),
                    dim3(256), a.s, nullptr, nullptr, static_cast<const S*>(a.grad_y),
                    static_cast<const S*>(a.stored), a.rstd, a.partial, a.T, a.H, rows);
  return e != hipSuccess ? e : launch_reduce(a, parts, nullptr);
}

template <int F>
hipError_t launch_bwd_h(const BwdArgs& a) {
  if (a.H <= 64 * 8) return launch_bwd<F, 64, 1>(a);
  if (a.H <= 128 * 8) return launch_bwd<F, 128, 1>(a);
  if (a.H <= 256 * 8) return launch_bwd<F, 256, 1>(a);
  if (a.H <= 512 * 8) return launch_bwd<F, 512, 1>(a);
  if (a.H <= kFused) return launch_bwd<F, 512, 2>(a);
  if (a.H <= kHeld) return launch_bwd_row<F, 1024, 2>(a);
  return launch_bwd_row<F, 512, 0>(a);
}

}  // namespace

extern "C" {

int mhc_rms_norm_abi_version(void) { return MHC_NORM_ABI_VERSION; }

const char* mhc_rms_norm_last_error_message(void) { return g_msg; }

int64_t mhc_rms_norm_bwd_workspace_bytes(int64_t T, int64_t H) {
  if (T < 0 || H < 1 || H > MHC_MAX_H) return -1;
  return workspace_need(T, H);
}

mhc_status mhc_rms_norm_validate_fwd(const void* x, const void* residual, const float* pre,
                                     int32_t n, const void* weight, int32_t weight_dtype,
                                     float eps, const void* out, const void* scales,
                                     const void* stored, const float* rstd, int64_t T, int64_t H,
                                     int32_t dtype, int32_t out_format) {
  return validate_fwd(x, residual, pre, n, weight, weight_dtype, eps, out, scales, stored, rstd, T,
                      H, dtype, out_format);
}

mhc_status mhc_rms_norm_validate_bwd(const void* grad_y, const void* stored, const void* weight,
                                     int32_t weight_dtype, const float* rstd,
                                     const void* grad_stored, const void* grad_x,
                                     const float* grad_weight, const void* workspace,
                                     int64_t workspace_bytes, int64_t T, int64_t H,
                                     int32_t dtype) {
  return validate_bwd(grad_y, stored, weight, weight_dtype, rstd, grad_stored, grad_x, grad_weight,
                      workspace, workspace_bytes, T, H, dtype);
}

mhc_status mhc_rms_norm_fwd(const void* x, const void* residual, const float* pre, int32_t n,
                            const void* weight, int32_t weight_dtype, float eps, void* out,
                            void* scales, void* stored, float* rstd, int64_t T, int64_t H,
                            int32_t dtype, int32_t out_format, void* stream, void* start_event,
                            void* stop_event) {
  const mhc_status st = validate_fwd(x, residual, pre, n, weight, weight_dtype, eps, out, scales,
                                     stored, rstd, T, H, dtype, out_format);
  if (st != MHC_SUCCESS) return st;
  if (T == 0) return record_empty(stream, start_event, stop_event);
  const FwdArgs a = {x, residual, pre, weight, weight_dtype == MHC_NORM_F32, eps, out, scales,
                     stored, rstd, T, H, static_cast<hipStream_t>(stream),
                     static_cast<hipEvent_t>(start_event), static_cast<hipEvent_t>(stop_event)};
  hipError_t e;
  if (n == 2) e = launch_fwd_f<kBF16, 2>(a, out_format);
  else if (n == 4) e = launch_fwd_f<kBF16, 4>(a, out_format);
  else if (n == 8) e = launch_fwd_f<kBF16, 8>(a, out_format);
  else if (dtype == MHC_NORM_F32) e = launch_fwd_s<kF32>(a, out_format);
  else if (dtype == MHC_NORM_BF16) e = launch_fwd_s<kBF16>(a, out_format);
  else e = launch_fwd_s<kF16>(a, out_format);
  return launch_status(e, "norm launch");
}

mhc_status mhc_rms_norm_bwd(const void* grad_y, const void* stored, const void* weight,
                            int32_t weight_dtype, const float* rstd, const void* grad_stored,
                            void* grad_x, float* grad_weight, void* workspace,
                            int64_t workspace_bytes, int64_t T, int64_t H, int32_t dtype,
                            void* stream, void* start_event, void* stop_event) {
  const mhc_status st = validate_bwd(grad_y, stored, weight, weight_dtype, rstd, grad_stored,
                                     grad_x, grad_weight, workspace, workspace_bytes, T, H, dtype);
  if (st != MHC_SUCCESS) return st;
  const BwdArgs a = {grad_y, stored, weight, weight_dtype == MHC_NORM_F32, rstd, grad_stored,
                     grad_x, grad_weight, static_cast<float*>(workspace), T, H,
                     static_cast<hipStream_t>(stream), static_cast<hipEvent_t>(start_event),
                     static_cast<hipEvent_t>(stop_event)};
  hipError_t e;
  if (T == 0) e = launch_reduce(a, 0, a.start);
  else if (dtype == MHC_NORM_F32) e = launch_bwd_h<kF32>(a);
  else if (dtype == MHC_NORM_BF16) e = launch_bwd_h<kBF16>(a);
  else e = launch_bwd_h<kF16>(a);
  return launch_status(e, "norm backward launch");
}

}  // extern "C"
