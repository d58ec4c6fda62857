// mhc_cross_entropy.hip - softmax cross entropy of a large vocabulary's logits,
// which are not kept, and its gradients, for gfx950 (see
// include/mhc_cross_entropy.h for the operation).

#include "mhc_cross_entropy.h"

#include <math.h>

#include "mhc_tiles_host.h"

#ifdef __FAST_MATH__
#error "this source must not be built with fast-math"
#endif

#pragma clang fp contract(off)

namespace {

constexpr float kLog2E = 1.44269504f, kLn2 = 0.69314718f;

// exp(a - b), NaN where they are the same infinity. The difference comes before
// the product with log2(e): rounding a log2(e) and b log2(e) apart would put an
// error that grows with |a| into every term of a row (half a step of 1e7 is e^(1/2)),
// and would overflow from 2.36e38 on.
__device__ __forceinline__ float exp_of(float a, float b) {
  return __builtin_amdgcn_exp2f((a - b) * kLog2E);
}

// The same, 1 where they are the same infinity: of sums that are joined.
__device__ __forceinline__ float ratio_of(float a, float b) {
  return __builtin_amdgcn_exp2f((a == b ? 0.0f : a - b) * kLog2E);
}

// A group of columns: its largest logit, and the sum of exp(z - m) 2^15. Of a row:
// the same of all its columns, of which lse is m + log(s / 2^15).
struct Stat {
  float m, s;
};

// The exponentials that the workspace holds between the logits and G are those
// terms, at most 2^15 (the largest logit's is just that, whatever fp32 makes of
// m - 15), in fp16, of either type of x: fp16's rounding is an eighth of
// bf16's, which G then adds (held in bf16 the gradients at 4096 x 131072 x 4096 were
// 0.0027 off by the norm, so 0.0024, with a mean's factor still in G). What is 2^-29
// of a group's largest is a normal number, and what is below 2^-40 of it counts as 0.
constexpr float kHeld = 15.0f;

// The term of z in a group whose largest logit is m, neither of them infinite.
__device__ __forceinline__ float term_of(float z, float m) {
  return __builtin_amdgcn_exp2f(fmaf(z - m, kLog2E, kHeld));
}

// Several groups at once: one exponential each, and one for what was there.
template <int K>
__device__ __forceinline__ Stat join_all(const Stat& a, const Stat (&b)[K]) {
  float m = a.m;
#pragma unroll
  for (int k = 0; k < K; ++k) m = fmaxf(m, b[k].m);
  float s = a.s * ratio_of(a.m, m);
#pragma unroll
  for (int k = 0; k < K; ++k) s = s + b[k].s * ratio_of(b[k].m, m);
  return {m, s};
}

__device__ __forceinline__ Stat join(const Stat& a, const Stat& b) {
  const float m = fmaxf(a.m, b.m);
  return {m, a.s * ratio_of(a.m, m) + b.s * ratio_of(b.m, m)};
}

// What of its row's gradient a probability (a) and the target's place (b) get.
struct Share {
  float a, b;
};

// ---------------------------------------------------------------------------
// Logits
//
// The product's kernels with an epilogue that never writes a logit: each wave
// takes the largest of its 64 (or 32) columns of a row and the sum of exponentials
// under it from its registers, and the target's logit where it is among them. For
// the gradients the exponentials themselves (see kHeld) are written in 16 bits: a
// later pass only has to scale them.
// ---------------------------------------------------------------------------

// Epilogue of the tile kernels. Groups of columns are a wave's; their statistics
// lie [groups][rows], since a wave writes those of 16 rows. The terms go to memory
// from the registers they are made in, 64 consecutive bytes of each of 16 rows at a
// time, while the next rows' are made; through LDS, like other results, they took
// 10 us of a 256 x 256 tile's 112 at K = 4096.
template <bool HOLD>
struct StatEpilogue {
  static constexpr int kW = kOne, kSums = 1, kGroup = 2;
  static constexpr bool kSplits = false, kHalves = false, kTakes = true, kWrites = false, kEarly = false;
  Stat* stats;
  float* target_logit;     // [rows]: written where a target is among the columns
  const int64_t* targets;  // [rows]
  uint16_t* held;          // [rows][ld]
  int64_t ld;

  // Lane l holds in acc[i][j] four columns of row 16 i + l % 16 of the wave's part:
  // of each 32 columns it has 8, and the four lanes of a row have all 16 TJ.
  template <int OP, int TI, int TJ, int WN>
  __device__ __forceinline__ void take(const TileShape& a, const Place& at,
                                       f32x4 (&acc)[TI][TJ]) const {
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const uint32_t lane = threadIdx.x % 64, low = lane % 16, g = lane / 16;
    constexpr int kTiles = TJ < 4 ? TJ : 4;  // of a group
    // 128 x 128 of a wave would be 16 copies of 400 instructions
    constexpr int kCopies = TJ == 8 ? 1 : TI;
#pragma unroll 1
    for (int sub = 0; sub < TJ / kTiles; ++sub) {
      const int64_t first = at.n0 + (wave % WN) * (TJ * 16) + sub * (kTiles * 16);
      if (first >= a.N) return;
      const int32_t left = static_cast<int32_t>(min(a.N - first, static_cast<int64_t>(kTiles * 16)));
      Stat* const out = stats + first / (kTiles * 16) * a.M;
      const int64_t row0 = at.m0 + (wave / WN) * (TI * 16) + low;
#pragma unroll kCopies
      for (int i = 0; i < TI; ++i) {
        f32x4 z[kTiles];
        if constexpr (kCopies == TI) {
#pragma unroll
          for (int j = 0; j < kTiles; ++j) z[j] = acc[i][j];
        } else {
          each_of<TI * 2>(sub * TI + i, [&](auto k) {
#pragma unroll
            for (int j = 0; j < kTiles; ++j) z[j] = acc[k % TI][k / TI * kTiles + j];
          });
        }
        const int64_t row = row0 + i * 16;
        float v[kTiles * 4];
#pragma unroll
        for (int j = 0; j < kTiles; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[j * 4 + e] = z[j][e];
            if (left < kTiles * 16 && column(j, e, g) >= left) v[j * 4 + e] = -INFINITY;
          }
        one_row<kTiles>(a.M, row, first, left, g, v, out);
      }
    }
  }

  // The column of the group that is in v[4 j + e].
  static __device__ __forceinline__ int column(int j, int e, uint32_t g) {
    return (j / 2) * 32 + static_cast<int>(g) * 8 + (j % 2) * 4 + e;
  }

  template <int kTiles>
  __device__ __forceinline__ void one_row(int64_t M, int64_t row, int64_t first, int32_t left, uint32_t g,
                                          float (&v)[kTiles * 4], Stat* out) const {
    float m = v[0];
#pragma unroll
    for (int k = 1; k < kTiles * 4; ++k) m = fmaxf(m, v[k]);
    m = across_max(m);
    if (row < M) {
      const int64_t t = targets[row] - first;
      if (t >= 0 && t < left && t / 8 % 4 == g) {
        float at_t = 0.0f;
#pragma unroll
        for (int k = 0; k < kTiles * 4; ++k) at_t = t == column(k / 4, k % 4, g) ? v[k] : at_t;
        target_logit[row] = at_t;
      }
    }
    float s = 0.0f;
    if (__any(fabsf(m) == INFINITY)) {
      // terms at an infinite maximum count as 2^15, which leaves lse that infinity; exp(inf - inf)
      // has no value, and where it stands NaN is held (ce_grad_kernel sees a row of -inf alone)
#pragma unroll
      for (int k = 0; k < kTiles * 4; ++k) {
        const float t = v[k] == m ? 0x1p15f : term_of(v[k], m);
        s = s + t;
        v[k] = v[k] == INFINITY ? NAN : t;
      }
    } else {
#pragma unroll
      for (int k = 0; k < kTiles * 4; ++k) {
        v[k] = term_of(v[k], m);
        s = s + v[k];
      }
    }
    s = across_sum(s);
    if (g == 0 && row < M) out[row] = {m, s};
    if constexpr (HOLD) {
      if (row < M) {
#pragma unroll
        for (int j = 0; j < kTiles; j += 2) {
          float u[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] = v[j * 4 + e];
          Chunk<kF16> c;
          narrow_chunk<kF16>(u, c);
          // rows of `held` are whole chunks: what is past the last column is read by no one
          if (column(j, 0, g) < left) *reinterpret_cast<u32x4*>(held + row * ld + first + column(j, 0, g)) = c.w[0];
        }
      }
    }
  }

  // Of the four lanes l, l ^ 16, l ^ 32, l ^ 48, in each of them.
  static __device__ __forceinline__ float across_max(float x) {
    uint32_t u = __float_as_uint(x);
    auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const float y = fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
    u = __float_as_uint(y);
    p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
  }
  static __device__ __forceinline__ float across_sum(float x) {
    uint32_t u = __float_as_uint(x);
    auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const float y = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    u = __float_as_uint(y);
    p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
};

// The same of the row kernel: groups are a thread's 8 columns, [rows][groups].
template <bool HOLD>
struct RowStatEpilogue {
  static constexpr int kW = kOne, kSums = 1, kGroup = 0;
  static constexpr bool kSplits = false, kHalves = false, kTakes = false, kWrites = true, kEarly = false;
  Stat* stats;
  float* target_logit;
  const int64_t* targets;
  uint16_t* held;
  int64_t ld, groups;

  template <int OP, class Fn>
  __device__ __forceinline__ void with(const Fn& fn) const {
    fn([&](int64_t m, int64_t n, int count, float(&v)[8]) {
      const int64_t t = targets[m] - n;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (t == e && e < count) target_logit[m] = v[e];
      float top = v[0];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e >= count) v[e] = -INFINITY;
        top = fmaxf(top, v[e]);
      }
      float s = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float t = v[e] == top ? 0x1p15f : term_of(v[e], top);
        s = s + t;
        v[e] = v[e] == INFINITY ? NAN : t;  // see StatEpilogue
      }
      stats[m * groups + n / 8] = {top, s};
      if constexpr (HOLD) {
        Chunk<kF16> c;
        narrow_chunk<kF16>(v, c);
        store_chunk<kF16>(held + m * ld + n, 8, c);
      }
    });
  }
};

// Epilogue of the logits made again: G itself, from the rows' lse and shares.
// Columns V.. of the last piece of a row are zeros (W has no such rows). z - lse is
// at most 0: a rounding of either to the other side (half a step of 1e8 is 4) would
// make a probability of e^4, past all that the shares' scale leaves room for.
struct GradEpilogue {
  static constexpr int kW = kOne, kSums = 1, kGroup = 0;
  static constexpr bool kSplits = false, kHalves = false, kTakes = false, kWrites = true, kEarly = false;
  const float* lse;        // [rows]
  const Share* shares;     // [rows]
  const int64_t* targets;  // [rows]
  void* held;              // [rows][ld]
  int64_t ld, V;

  template <int OP, class Fn>
  __device__ __forceinline__ void with(const Fn& fn) const {
    constexpr int F = out_format(OP);
    typedef typename Store<F>::type S;
    fn([&](int64_t m, int64_t n, int count, float(&v)[8]) {
      const Share w = shares[m];
      const float l = lse[m];
      const int64_t t = targets[m] - n;
      const bool none = w.a == 0.0f && w.b == 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = v[e] - l;
        const float p = __builtin_amdgcn_exp2f((d > 0.0f ? 0.0f : d) * kLog2E) * w.a;
        v[e] = none || n + e >= V ? 0.0f : t == e ? p - w.b : p;
      }
      Chunk<F> c;
      narrow_chunk<F>(v, c);
      store_chunk<F>(static_cast<S*>(held) + m * ld + n, count, c);
    });
  }
};

// ---------------------------------------------------------------------------
// Rows
// ---------------------------------------------------------------------------

// lse and the loss of each row from its groups: R rows to a block of 1024 threads,
// 1024 / R of them to a row, each over every (1024 / R)-th group in ascending
// order, eight at a time, joined by halving. R is 16 where there are rows for all
// CUs (a group's 16 rows are one 128-byte line), and less for fewer rows, which
// need their groups' latency spread over more threads: 8 rows x 8192 groups 14.6 us
// with 8 rows to a block, 5.5 with one.
template <int R>
__global__ __launch_bounds__(1024) void ce_lse_kernel(const Stat* __restrict__ stats,
                                                      const float* __restrict__ target_logit,
                                                      const int64_t* __restrict__ targets,
                                                      float* __restrict__ lse, Stat* __restrict__ whole,
                                                      float* __restrict__ loss, int64_t M, int64_t V, int64_t groups, int64_t up,
                                                      int64_t along, int64_t ignore_index) {
  constexpr int kEach = 1024 / R;
  __shared__ Stat part[1024];
  const int64_t row = static_cast<int64_t>(blockIdx.x) * R + threadIdx.x % R;
  const int k = threadIdx.x / R;
  Stat all = {-INFINITY, 0.0f};
  if (row < M) {
    for (int64_t p = k; p < groups; p += 8 * kEach) {
      Stat some[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t at = p + i * kEach;
        some[i] = at < groups ? stats[at * along + row * up] : Stat{-INFINITY, 0.0f};
      }
      all = join_all(all, some);
    }
  }
  part[threadIdx.x] = all;
  __syncthreads();
#pragma unroll
  for (int off = kEach / 2; off > 0; off /= 2) {
    if (k < off) part[threadIdx.x] = join(part[threadIdx.x], part[threadIdx.x + off * R]);
    __syncthreads();
  }
  if (k == 0 && row < M) {
    all = part[threadIdx.x];
    // with the largest term at 1 the logarithm is small, and rounded as finely; the loss takes
    // it after the logits' difference, which does not see how large they are
    const float log = __log2f(all.s * 0x1p-15f) * kLn2;
    lse[row] = all.m + log;
    whole[row] = all;
    const int64_t t = targets[row];
    loss[row] = t == ignore_index ? 0.0f : t >= 0 && t < V ? (all.m - target_logit[row]) + log : NAN;
  }
}

constexpr int kOneBlock = 1024;

// loss = the rows' sum, over C for a mean: a thread takes every 1024th row.
__global__ __launch_bounds__(kOneBlock) void ce_total_kernel(const float* __restrict__ rows,
                                                             const int64_t* __restrict__ targets,
                                                             float* __restrict__ loss, int64_t M,
                                                             int64_t ignore_index, int mean) {
  __shared__ float part[2][kOneBlock / 64];
  float sum = 0.0f;
  int32_t count = 0;
#pragma unroll 8
  for (int64_t m = threadIdx.x; m < M; m += kOneBlock) {
    sum = sum + rows[m];
    count += targets[m] != ignore_index;
  }
  sum = block_sum<kOneBlock>(sum, part[0]);
  // two exact halves: a count past 2^24 is no fp32 number
  const float low = block_sum<kOneBlock>(static_cast<float>(count & 0xFFF), part[1]);
  __syncthreads();
  const float high = block_sum<kOneBlock>(static_cast<float>(count >> 12), part[0]);
  if (threadIdx.x == 0) loss[0] = mean ? sum / (high * 4096.0f + low) : sum;
}

// The rows' shares, and what they were divided by, which the products' sums take back.
// For a sum or a mean that is |s|, which all rows have alike: left in, its rounding would
// be in every target's G, and not a random part of it (bf16 has 1 / 3870 off by 0.0035, and
// the gradients at 4096 x 131072 x 4096 were 0.0024 to 0.0042 off by the norm with C,
// 0.0028 at 3890, so 0.0019; the output's own rounding is 0.0017). Its power of two
// stays in, so that sums keep their size, and all of it where grad_lse would be more
// than 2^10 of it. For fp16 (`narrow`) then the power of two that
// brings the largest G that the shares allow to [2^14, 2^15): G is a p or, at the target,
// a p - b, with p from 0 to 1, so at most |a|, |b| or |a - b|, which is twice either where
// grad_lse is twice -s.
__global__ __launch_bounds__(kOneBlock) void ce_shares_kernel(
    const int64_t* __restrict__ targets, const float* __restrict__ grad_loss,
    const float* __restrict__ grad_lse, Share* __restrict__ shares, float* __restrict__ inverse,
    int64_t M, int64_t V, int64_t ignore_index, int reduction, int narrow) {
  __shared__ float part[3][kOneBlock / 64];
  float over = 1.0f;
  if (reduction == MHC_REDUCTION_MEAN) {
    int32_t count = 0;
#pragma unroll 8
    for (int64_t m = threadIdx.x; m < M; m += kOneBlock) count += targets[m] != ignore_index;
    const float low = block_sum<kOneBlock>(static_cast<float>(count & 0xFFF), part[0]);
    const float high = block_sum<kOneBlock>(static_cast<float>(count >> 12), part[1]);
    over = high * 4096.0f + low;
  }
  const auto share = [&](int64_t m) {
    const int64_t t = targets[m];
    const float g = grad_loss == nullptr ? 1.0f : grad_loss[reduction == MHC_REDUCTION_NONE ? m : 0];
    const float s = t == ignore_index ? 0.0f : t >= 0 && t < V ? g / over : NAN;
    return Share{grad_lse == nullptr ? s : s + grad_lse[m], s};
  };
  float unit = 1.0f;
  if (reduction != MHC_REDUCTION_NONE) {
    const float s = fabsf((grad_loss == nullptr ? 1.0f : grad_loss[0]) / over);
    if (s >= 0x1p-100f && s < INFINITY) unit = s;
  }
  float most = 0.0f;
  if (narrow || grad_lse != nullptr) {
#pragma unroll 4
    for (int64_t m = threadIdx.x; m < M; m += kOneBlock) {
      const Share w = share(m);
      most = fmaxf(most, fmaxf(fmaxf(fabsf(w.a), fabsf(w.b)), fabsf(w.a - w.b)));
    }
    most = block_max<kOneBlock>(most, part[2]);
    if (most > 0x1p10f * unit) unit = 1.0f;
  }
  int power = narrow ? 0 : ilogbf(unit);
  most = most / unit;
  if (narrow && most > 0.0f && most < INFINITY) power = 14 - ilogbf(most);
  power = power > 126 ? 126 : power;
  const float scale = ldexpf(1.0f, power);
  for (int64_t m = threadIdx.x; m < M; m += kOneBlock) {
    const Share w = share(m);
    shares[m] = {w.a / unit * scale, w.b / unit * scale};
  }
  if (threadIdx.x == 0) *inverse = unit * ldexpf(1.0f, -power);
}

// held -> G in place: the exponentials under their groups' maxima become the
// row's share of the probability, less the target's. A block takes 16 rows x
// `segment` columns, 128 of each row at a time: the groups' 16 rows are one line.
template <int F>
__global__ __launch_bounds__(256) void ce_grad_kernel(
    const Stat* __restrict__ stats, const Stat* __restrict__ whole, const Share* __restrict__ shares,
    const int64_t* __restrict__ targets, typename Store<F>::type* __restrict__ held, int64_t M,
    int64_t V, int64_t ld, int64_t segment, int group_bits, int64_t up, int64_t along) {
  const int64_t row = static_cast<int64_t>(blockIdx.y) * 16 + threadIdx.x / 16;
  if (row >= M) return;
  const Share w = shares[row];
  const Stat all = whole[row];
  const float share = w.a / all.s;
  const int64_t t = targets[row];
  const bool none = w.a == 0.0f && w.b == 0.0f;
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * segment + threadIdx.x % 16 * 8;
  const int64_t end = min(V, static_cast<int64_t>(blockIdx.x + 1) * segment);
#pragma unroll 4
  for (int64_t n = begin; n < end; n += 128) {
    typename Store<F>::type* const p = held + row * ld + n;
    float v[8];
    widen_chunk<kF16>(load_chunk<kF16>(p, 8), v);
    // 1 at an infinite lse, whose terms are 0 or NaN; NaN where all logits are -inf
    const float m = stats[(n >> group_bits) * along + row * up].m;
    const float f = (m == all.m && m == INFINITY ? 1.0f : exp_of(m, all.m)) * share;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = v[e] * f;
      v[e] = none || n + e >= V ? 0.0f : t == n + e ? v[e] - w.b : v[e];
    }
    Chunk<F> c;
    narrow_chunk<F>(v, c);
    store_chunk<F>(p, 8, c);
  }
}

__global__ void ce_fill_kernel(float* p, float v) { *p = v; }

// ---------------------------------------------------------------------------
// The products over G
// ---------------------------------------------------------------------------

// Sums over pieces of V (grad_x) or chunks of rows (grad_weight) are added up in
// fp32, in ascending order, and rounded once, with what the shares were divided by taken back.
struct SumEpilogue {
  static constexpr int kW = kOne, kSums = 1, kGroup = 0;
  static constexpr bool kSplits = true, kHalves = false, kTakes = false, kWrites = true, kEarly = false;
  void* out;
  float* sum;            // where there are several
  const float* inverse;  // what the shares were divided by
  int64_t N;
  int32_t first, last;

  template <int OP, class Fn>
  __device__ __forceinline__ void with(const Fn& fn) const {
    constexpr int F = out_format(OP);
    typedef typename Store<F>::type S;
    // to a scalar register, so that no load is on its way when the next tile begins: that one's loop
    // would wait for it, and with it for its own, in every pass
    float scale = 1.0f;
    if (last != 0)
      scale = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(*inverse)));
    fn([&](int64_t m, int64_t n, int count, float(&v)[8]) {
      if (first == 0) {
        float b[8];
        widen_chunk<kF32>(load_chunk<kF32>(sum + m * N + n, count), b);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = b[e] + v[e];
      }
      if (last != 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] * scale;
        Chunk<F> c;
        narrow_chunk<F>(v, c);
        store_chunk<F>(static_cast<S*>(out) + m * N + n, count, c);
      } else {
        Chunk<kF32> c;
        narrow_chunk<kF32>(v, c);
        store_chunk<kF32>(sum + m * N + n, count, c);
      }
    });
  }
};

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

constexpr int kFwd = 0, kBwd = 1, kGrads = 2;

mhc_status check_sizes(int64_t M, int64_t V, int64_t K, int32_t dtype) {
  if (M < 0 || M > INT32_MAX) return fail(MHC_ERROR_INVALID_VALUE, "M must be in [0, 2^31 - 1]");
  if (V < 1 || V > MHC_CROSS_ENTROPY_MAX_V)
    return fail(MHC_ERROR_INVALID_VALUE, "V must be in [1, %lld] (got %lld)", MHC_CROSS_ENTROPY_MAX_V,
                static_cast<long long>(V));
  if (K < 1 || K > MHC_LINEAR_MAX_K)
    return fail(MHC_ERROR_INVALID_VALUE, "K must be in [1, %lld] (got %lld)", MHC_LINEAR_MAX_K,
                static_cast<long long>(K));
  if (dtype != MHC_LINEAR_BF16 && dtype != MHC_LINEAR_F16)
    return fail(MHC_ERROR_INVALID_VALUE, "dtype must be MHC_LINEAR_BF16 or _F16 (got %d)", dtype);
  return ok();
}

struct Plan {
  int64_t chunk;                 // rows of a chunk
  int64_t ld;                    // columns of a row of G
  int64_t piece;                 // rows of W in one product for grad_x
  mhc_linear_launch logits;
  int group_bits;                // log2 of a group's columns
  int64_t groups;
  bool pad;                      // rows along K are copied whole
  int64_t ldk;                   // their bytes
  mhc_linear_launch px, pw;      // the products over G
  int64_t x, w, stats, target, whole, rows, shares, inverse, held, part, sum_x, sum_w, total;  // places
};

// Rows of a chunk: as many as the held values' bytes allow, evenly, in whole tiles.
int64_t chunk_rows(int64_t M, int64_t ld) {
  int64_t most = MHC_CROSS_ENTROPY_CHUNK_BYTES / (ld * 2) / 256 * 256;
  if (most < 256) most = 256;
  if (most > (1 << 19)) most = 1 << 19;  // a sum's length, and 16 times a grid's height
  if (M <= most) return M;
  return round_up(ceil_div(M, ceil_div(M, most)), 256);
}

// The kernel of the logits: unsplit, since the epilogue needs whole sums.
mhc_status plan_logits(int64_t M, int64_t V, int64_t K, int32_t dtype, int mode,
                       const mhc_linear_launch* launch, mhc_linear_launch* p) {
  if (launch != nullptr && (launch->splits < 0 || launch->splits > 1 || launch->kernel == MHC_LINEAR_NARROW))
    return fail(MHC_ERROR_INVALID_VALUE, "launch: there is no narrow or split kernel here");
  if (mode == kBwd && launch != nullptr && launch->kernel == MHC_LINEAR_ROWS)
    return fail(MHC_ERROR_INVALID_VALUE, "launch: the backward has no row kernel");
  mhc_linear_launch want = {launch != nullptr ? launch->kernel : 0, 1};
  if (mode == kBwd && M <= 16 && want.kernel == 0) want.kernel = MHC_LINEAR_SHORT;
  return best_plan(M, V, K, dtype, false, 1, &want, p);
}

mhc_status make_all(int64_t M, int64_t V, int64_t K, int32_t dtype, int mode,
                    const mhc_linear_launch* launch, Plan* plan) {
  *plan = {};
  Plan& p = *plan;
  mhc_status st = check_sizes(M, V, K, dtype);
  if (st != MHC_SUCCESS) return st;
  p.ld = round_up(V, 64);
  p.chunk = chunk_rows(M, p.ld);
  if ((st = plan_logits(p.chunk, V, K, dtype, mode, launch, &p.logits)) != MHC_SUCCESS) return st;
  if (M == 0) return ok();
  p.group_bits = p.logits.kernel == MHC_LINEAR_ROWS                                            ? 3
                 : p.logits.kernel == MHC_LINEAR_SMALL || p.logits.kernel == MHC_LINEAR_SHORT ? 5
                                                                                              : 6;
  p.groups = ceil_div(V, 1 << p.group_bits);
  // The loss alone has one product, as the forward of mhc_linear.h, and its rule: at few rows a
  // copy of W is three times W's bytes (65536 x 7167 in bf16, 8 rows 619 us and 897 MiB of
  // workspace, so 532 and 0.5; 17 rows 612, 211; 129 rows 638, 404; 16 rows 648, 690). With gradients W is
  // read turned as well, which through registers costs more than the copy.
  const bool few = mode == kFwd && (p.logits.kernel == MHC_LINEAR_ROWS || M < kPadRows || V < kPadRows);
  p.pad = K % 8 != 0 && !few &&
          (M > INT64_MAX / V / K || M * V * K >= (mode == kFwd ? kPadForward : kPadBackward));
  p.ldk = p.pad ? round_up(K * 2, 16) : K * 2;
  Places at;
  if (p.pad) {
    p.x = at.take(mul_bytes(M, p.ldk, 1));
    p.w = at.take(mul_bytes(V, p.ldk, 1));
  }
  if (mode != kBwd) {
    // the launch that the policy chose may go through the medium tiles, whose groups are as wide
    p.stats = at.take(mul_bytes(p.groups, p.chunk, sizeof(Stat)));
    p.target = at.take(mul_bytes(p.chunk, 4, 1));
    p.whole = at.take(mul_bytes(p.chunk, sizeof(Stat), 1));
    p.rows = at.take(mul_bytes(M, 4, 1));
  }
  if (mode != kFwd) {
    p.shares = at.take(mul_bytes(M, sizeof(Share), 1));
    p.inverse = at.take(4);
    p.held = at.take(mul_bytes(p.chunk, p.ld, 2));
    // a turned operand is loaded straight into LDS up to 2^31 bytes
    p.piece = INT32_MAX / p.ldk / 256 * 256;
    if (p.piece < 256) p.piece = 256;
    if (p.piece > V) p.piece = V;
    if (best_plan(p.chunk, K, round_up(p.piece, 8), dtype, true, 32, nullptr, &p.px) != MHC_SUCCESS ||
        best_plan(V, K, p.chunk, dtype, true, 32, nullptr, &p.pw) != MHC_SUCCESS)
      at.total = -1;
    const auto parts = [](int64_t rows, int64_t columns, const mhc_linear_launch& l) {
      return l.splits > 1 ? mul_bytes(mul_bytes(rows, columns, 4), l.splits, 1) : 0;
    };
    const int64_t a = parts(p.chunk, K, p.px), b = parts(V, K, p.pw);
    p.part = at.take(a < 0 || b < 0 ? -1 : a > b ? a : b);
    if (p.piece < V) p.sum_x = at.take(mul_bytes(p.chunk, K, 4));
    // (more than all logits in 16 bits where K > M / 2; the next chunk's part joins it in fp32)
    if (p.chunk < M) p.sum_w = at.take(mul_bytes(V, K, 4));
  }
  p.total = at.total;
  return ok();
}

mhc_status check_call(const Plan& p, int64_t workspace_bytes, int32_t reduction) {
  if (reduction < MHC_REDUCTION_NONE || reduction > MHC_REDUCTION_MEAN)
    return fail(MHC_ERROR_INVALID_VALUE, "unknown reduction %d", reduction);
  if (p.total < 0) return fail(MHC_ERROR_INVALID_VALUE, "the workspace's size does not fit 64 bits");
  if (workspace_bytes < p.total)
    return fail(MHC_ERROR_INVALID_VALUE, "workspace_bytes %lld < %lld needed",
                static_cast<long long>(workspace_bytes), static_cast<long long>(p.total));
  return ok();
}

// With M == 0 only what is no tensor of rows exists.
struct Sizes {
  int64_t x, w, targets, rows, loss, gw;
  Sizes(int64_t M, int64_t V, int64_t K, int32_t reduction)
      : x(mul_bytes(M, K, 2)), w(M > 0 ? mul_bytes(V, K, 2) : 0), targets(mul_bytes(M, 8, 1)),
        rows(mul_bytes(M, 4, 1)), loss(reduction == MHC_REDUCTION_NONE ? rows : 4),
        gw(mul_bytes(V, K, 2)) {}
};

mhc_status validate_fwd(const void* x, const void* w, const void* targets, const void* loss,
                        const void* lse, const void* workspace, int64_t workspace_bytes, int64_t M,
                        int64_t V, int64_t K, int32_t dtype, int32_t reduction,
                        const mhc_linear_launch* launch, Plan* p) {
  mhc_status st = make_all(M, V, K, dtype, kFwd, launch, p);
  if (st != MHC_SUCCESS) return st;
  if ((st = check_call(*p, workspace_bytes, reduction)) != MHC_SUCCESS) return st;
  const Sizes b(M, V, K, reduction);
  const Tensor in[] = {{x, b.x, 2, "x"}, {w, b.w, 2, "weight"}, {targets, b.targets, 8, "targets"}};
  const Tensor out[] = {{loss, b.loss, 4, "loss"},
                        {lse, b.rows, 4, "lse"},
                        {workspace, p->total, 16, "workspace"}};
  return check_tensors(in, out);
}

mhc_status validate_bwd(const void* x, const void* w, const void* targets, const void* lse,
                        const void* grad_loss, const void* grad_lse, const void* gx, const void* gw,
                        const void* workspace, int64_t workspace_bytes, int64_t M, int64_t V,
                        int64_t K, int32_t dtype, int32_t reduction,
                        const mhc_linear_launch* launch, Plan* p) {
  mhc_status st = make_all(M, V, K, dtype, kBwd, launch, p);
  if (st != MHC_SUCCESS) return st;
  if ((st = check_call(*p, workspace_bytes, reduction)) != MHC_SUCCESS) return st;
  const Sizes b(M, V, K, reduction);
  const Tensor in[] = {{x, b.x, 2, "x"},
                       {w, b.w, 2, "weight"},
                       {targets, b.targets, 8, "targets"},
                       {lse, b.rows, 4, "lse"},
                       {grad_loss, grad_loss != nullptr ? b.loss : 0, 4, "grad_loss"},
                       {grad_lse, grad_lse != nullptr ? b.rows : 0, 4, "grad_lse"}};
  const Tensor out[] = {{gx, gx != nullptr ? b.x : 0, 2, "grad_x"},
                        {gw, gw != nullptr ? b.gw : 0, 2, "grad_weight"},
                        {workspace, p->total, 16, "workspace"}};
  return check_tensors(in, out);
}

mhc_status validate_grads(const void* x, const void* w, const void* targets, const void* grad_loss,
                          const void* loss, const void* lse, const void* gx, const void* gw,
                          const void* workspace, int64_t workspace_bytes, int64_t M, int64_t V,
                          int64_t K, int32_t dtype, int32_t reduction,
                          const mhc_linear_launch* launch, Plan* p) {
  mhc_status st = make_all(M, V, K, dtype, kGrads, launch, p);
  if (st != MHC_SUCCESS) return st;
  if ((st = check_call(*p, workspace_bytes, reduction)) != MHC_SUCCESS) return st;
  const Sizes b(M, V, K, reduction);
  const Tensor in[] = {{x, b.x, 2, "x"},
                       {w, b.w, 2, "weight"},
                       {targets, b.targets, 8, "targets"},
                       {grad_loss, grad_loss != nullptr ? b.loss : 0, 4, "grad_loss"}};
  const Tensor out[] = {{loss, b.loss, 4, "loss"},
                        {lse, b.rows, 4, "lse"},
                        {gx, gx != nullptr ? b.x : 0, 2, "grad_x"},
                        {gw, gw != nullptr ? b.gw : 0, 2, "grad_weight"},
                        {workspace, p->total, 16, "workspace"}};
  return check_tensors(in, out);
}

struct Call {
  const void *x, *w;
  const int64_t* targets;
  const float *grad_loss, *grad_lse;
  const float* lse_in;  // kBwd
  float *loss, *lse;
  void *gx, *gw;
  uint8_t* ws;
  int64_t M, V, K;
  int32_t reduction;
  int64_t ignore_index;
};

template <class E>
TileArgs<E> logits_of(const Call& c, const Plan& p, const void* x, const void* w, int64_t rows, const E& e) {
  TileArgs<E> t = {};
  t.x = {x, rows, p.ldk};
  t.w = {w, c.V, p.ldk};
  t.M = rows;
  t.N = c.V;
  t.kbytes = static_cast<uint32_t>(p.ldk);
  t.e = e;
  return t;
}

// The row kernel with groups of 8 columns: 16 or 8 rows of W to a block. bytes: of a row that count.
template <int OP, class E>
hipError_t launch_row_logits(const TileArgs<E>& t, uint32_t bytes, hipStream_t s, hipEvent_t start) {
  const int64_t wide = t.N > 256 * 8 ? 16 : 8;
  // padded or not, a row's sum is that of its K values: the loss alone and the loss with gradients agree
  const RowsArgs<E> a = {static_cast<const uint8_t*>(t.x.p), static_cast<const uint8_t*>(t.w.p), nullptr,
                         nullptr, nullptr, nullptr, t.M, t.N, bytes, t.kbytes, static_cast<uint32_t>(wide), t.e};
  return launch_kernel(linear_rows_kernel<OP, 8, E>, dim3(static_cast<uint32_t>(ceil_div(t.N, wide))),
                       dim3(512), s, start, nullptr, a);
}

// Where the statistics of the next row and of the next group are.
int64_t up_of(const Plan& p) { return p.logits.kernel == MHC_LINEAR_ROWS ? p.groups : 1; }
int64_t along_of(const Plan& p, int64_t rows) { return p.logits.kernel == MHC_LINEAR_ROWS ? 1 : rows; }

// The statistics of a chunk's logits, lse and the rows' losses.
template <int OP, bool HOLD>
hipError_t launch_stats(const Call& c, const Plan& p, const void* x, const void* w, int64_t row0,
                        int64_t rows, hipStream_t s, Marks* marks) {
  Stat* const stats = reinterpret_cast<Stat*>(c.ws + p.stats);
  float* const target = reinterpret_cast<float*>(c.ws + p.target);
  const int64_t* const targets = c.targets + row0;
  uint16_t* const held = HOLD ? reinterpret_cast<uint16_t*>(c.ws + p.held) : nullptr;
  hipError_t e;
  if (p.logits.kernel == MHC_LINEAR_ROWS) {
    const RowStatEpilogue<HOLD> ep = {stats, target, targets, held, p.ld, p.groups};
    e = launch_row_logits<OP>(logits_of(c, p, x, w, rows, ep), static_cast<uint32_t>(c.K * 2), s, marks->first());
  } else {
    const StatEpilogue<HOLD> ep = {stats, target, targets, held, p.ld};
    e = launch_product<OP, false, false>(logits_of(c, p, x, w, rows, ep), p.logits, s, marks->first(), nullptr);
  }
  if (e != hipSuccess) return e;
  float* const loss = c.reduction == MHC_REDUCTION_NONE ? c.loss : reinterpret_cast<float*>(c.ws + p.rows);
  const auto run = [&](auto kernel, int64_t r) {
    return launch_kernel(kernel, dim3(static_cast<uint32_t>(ceil_div(rows, r))), dim3(1024), s, nullptr,
                         nullptr, stats, target, targets, c.lse + row0, reinterpret_cast<Stat*>(c.ws + p.whole),
                         loss + row0, rows, c.V,
                         p.groups, up_of(p), along_of(p, rows), c.ignore_index);
  };
  return rows >= 4096 ? run(ce_lse_kernel<16>, 16) : rows >= 1024 ? run(ce_lse_kernel<4>, 4)
                                                   : run(ce_lse_kernel<1>, 1);
}

template <int OP>
hipError_t launch_total(const Call& c, const Plan& p, hipStream_t s) {
  if (c.reduction == MHC_REDUCTION_NONE) return hipSuccess;
  return launch_kernel(ce_total_kernel, dim3(1), dim3(kOneBlock), s, nullptr, nullptr,
                       reinterpret_cast<const float*>(c.ws + p.rows), c.targets, c.loss, c.M,
                       c.ignore_index, c.reduction == MHC_REDUCTION_MEAN ? 1 : 0);
}

// grad_x and grad_weight's part from a chunk's G.
template <int OP>
hipError_t launch_over_g(const Call& c, const Plan& p, const void* x, const void* w, int64_t row0,
                         int64_t rows, hipStream_t s) {
  const uint8_t* const g = c.ws + p.held;
  const float* const inverse = reinterpret_cast<const float*>(c.ws + p.inverse);
  hipError_t e = hipSuccess;
  if (c.gx != nullptr) {
    for (int64_t v = 0; v < c.V && e == hipSuccess; v += p.piece) {
      // rows of G, with W turned; a row of G has zeros up to a whole piece
      const int64_t n = c.V - v < p.piece ? c.V - v : p.piece;
      TileArgs<SumEpilogue> t = {};
      t.x = {g + v * 2, rows, p.ld * 2};
      t.w = {static_cast<const uint8_t*>(w) + v * p.ldk, c.K, p.ldk};
      t.M = rows; t.N = c.K;
      t.kbytes = static_cast<uint32_t>(round_up(n, 8) * 2);
      t.kturned = static_cast<uint32_t>(n * 2);
      t.partial = reinterpret_cast<float*>(c.ws + p.part);
      t.e = {static_cast<uint8_t*>(c.gx) + row0 * c.K * 2, reinterpret_cast<float*>(c.ws + p.sum_x), inverse,
             c.K, v == 0, v + n == c.V};
      e = launch_product<OP, false, true>(t, p.px, s, nullptr, nullptr);
    }
    if (e != hipSuccess) return e;
  }
  if (c.gw != nullptr) {
    // G and x, both turned
    TileArgs<SumEpilogue> t = {};
    t.x = {g, c.V, p.ld * 2};
    t.w = {x, c.K, p.ldk};
    t.M = c.V; t.N = c.K;
    t.kbytes = t.kturned = static_cast<uint32_t>(rows * 2);
    t.partial = reinterpret_cast<float*>(c.ws + p.part);
    t.e = {c.gw, reinterpret_cast<float*>(c.ws + p.sum_w), inverse, c.K, row0 == 0, row0 + rows == c.M};
    e = launch_product<OP, true, true>(t, p.pw, s, nullptr, nullptr);
  }
  return e;
}

template <int OP, int MODE>
hipError_t launch_all(const Call& c, const Plan& p, hipStream_t s, hipEvent_t start, hipEvent_t stop) {
  constexpr int F = out_format(OP);
  typedef typename Store<F>::type S;
  Marks marks = {start, stop};
  hipError_t e = hipSuccess;
  if (c.M == 0) {
    if (MODE != kBwd && c.reduction != MHC_REDUCTION_NONE)
      e = launch_kernel(ce_fill_kernel, dim3(1), dim3(1), s, marks.first(), nullptr, c.loss,
                        c.reduction == MHC_REDUCTION_MEAN ? NAN : 0.0f);
    if (MODE != kFwd && c.gw != nullptr && e == hipSuccess)
      e = launch_zero(c.gw, c.V * c.K, s, marks.first(), nullptr);
    return marks.end(e, s);
  }
  const uint8_t* x = static_cast<const uint8_t*>(c.x);
  const void* w = c.w;
  if (p.pad) {
    PadJobs jobs = {};
    jobs.job[0] = pad_job(c.x, c.ws + p.x, c.M, c.K * 2, p.ldk, false);
    jobs.job[1] = pad_job(c.w, c.ws + p.w, c.V, c.K * 2, p.ldk, false);
    if ((e = launch_pad(jobs, 2, s, marks.first())) != hipSuccess) return e;
    x = c.ws + p.x;
    w = c.ws + p.w;
  }
  const bool grads = MODE != kFwd && (c.gx != nullptr || c.gw != nullptr);
  Share* const shares = reinterpret_cast<Share*>(c.ws + p.shares);
  if (grads) {
    e = launch_kernel(ce_shares_kernel, dim3(1), dim3(kOneBlock), s, marks.first(), nullptr, c.targets,
                      c.grad_loss, c.grad_lse, shares, reinterpret_cast<float*>(c.ws + p.inverse), c.M, c.V,
                      c.ignore_index, static_cast<int>(c.reduction), F == kF16 ? 1 : 0);
    if (e != hipSuccess) return e;
  }
  for (int64_t row0 = 0; row0 < c.M; row0 += p.chunk) {
    const int64_t rows = c.M - row0 < p.chunk ? c.M - row0 : p.chunk;
    const uint8_t* const xc = x + row0 * p.ldk;
    if constexpr (MODE == kFwd) {
      e = launch_stats<OP, false>(c, p, xc, w, row0, rows, s, &marks);
    } else if constexpr (MODE == kBwd) {
      if (!grads) break;
      const GradEpilogue ep = {c.lse_in + row0, shares + row0, c.targets + row0, c.ws + p.held, p.ld, c.V};
      TileArgs<GradEpilogue> t = logits_of(c, p, xc, w, rows, ep);
      t.N = round_up(c.V, 8);
      e = launch_product<OP, false, false>(t, p.logits, s, marks.first(), nullptr);
    } else {
      if (!grads) {
        e = launch_stats<OP, false>(c, p, xc, w, row0, rows, s, &marks);
      } else {
        e = launch_stats<OP, true>(c, p, xc, w, row0, rows, s, &marks);
        if (e != hipSuccess) return e;
        // 1 to 16 pieces of 128 columns to a block, by what leaves some 2048 blocks
        const int64_t high = ceil_div(rows, 16), pieces = ceil_div(c.V, 128) * high / 2048;
        const int64_t segment = 128 * (pieces < 1 ? 1 : pieces > 16 ? 16 : pieces);
        e = launch_kernel(ce_grad_kernel<F>, dim3(static_cast<uint32_t>(ceil_div(c.V, segment)), static_cast<uint32_t>(high)),
                          dim3(256), s, nullptr, nullptr, reinterpret_cast<const Stat*>(c.ws + p.stats),
                          reinterpret_cast<const Stat*>(c.ws + p.whole), shares + row0, c.targets + row0,
                          reinterpret_cast<S*>(c.ws + p.held), rows, c.V, p.ld, segment, p.group_bits, up_of(p), along_of(p, rows));
      }
    }
    if (e == hipSuccess && grads) e = launch_over_g<OP>(c, p, xc, w, row0, rows, s);
    if (e != hipSuccess) return e;
  }
  if (MODE != kBwd) e = launch_total<OP>(c, p, s);
  return marks.end(e, s);
}

template <int MODE>
mhc_status run(const Call& c, const Plan& p, int32_t dtype, void* stream, void* start, void* stop) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const hipEvent_t b = static_cast<hipEvent_t>(start), f = static_cast<hipEvent_t>(stop);
  const hipError_t e = dtype == MHC_LINEAR_BF16 ? launch_all<kOpBF16, MODE>(c, p, s, b, f)
                                                : launch_all<kOpF16, MODE>(c, p, s, b, f);
  return launch_status(e, "cross entropy launch");
}

int64_t workspace(int64_t M, int64_t V, int64_t K, int32_t dtype, int mode, const mhc_linear_launch* launch) {
  Plan p;
  return make_all(M, V, K, dtype, mode, launch, &p) == MHC_SUCCESS ? p.total : -1;
}

}  // namespace

extern "C" {

int mhc_cross_entropy_abi_version(void) { return MHC_CROSS_ENTROPY_ABI_VERSION; }

const char* mhc_cross_entropy_last_error_message(void) { return g_msg; }

int64_t mhc_cross_entropy_fwd_workspace_bytes(int64_t M, int64_t V, int64_t K, int32_t dtype,
                                              const mhc_linear_launch* launch) {
  return workspace(M, V, K, dtype, kFwd, launch);
}

int64_t mhc_cross_entropy_bwd_workspace_bytes(int64_t M, int64_t V, int64_t K, int32_t dtype,
                                              const mhc_linear_launch* launch) {
  return workspace(M, V, K, dtype, kBwd, launch);
}

int64_t mhc_cross_entropy_grads_workspace_bytes(int64_t M, int64_t V, int64_t K, int32_t dtype,
                                                const mhc_linear_launch* launch) {
  return workspace(M, V, K, dtype, kGrads, launch);
}

mhc_status mhc_cross_entropy_validate_fwd(const void* x, const void* weight,
                                          const int64_t* targets, const float* loss,
                                          const float* lse, const void* workspace,
                                          int64_t workspace_bytes, int64_t M, int64_t V, int64_t K,
                                          int32_t dtype, int32_t reduction,
                                          const mhc_linear_launch* launch) {
  Plan p;
  return validate_fwd(x, weight, targets, loss, lse, workspace, workspace_bytes, M, V, K, dtype,
                      reduction, launch, &p);
}

mhc_status mhc_cross_entropy_validate_bwd(const void* x, const void* weight,
                                          const int64_t* targets, const float* lse,
                                          const float* grad_loss, const float* grad_lse,
                                          const void* grad_x, const void* grad_weight,
                                          const void* workspace, int64_t workspace_bytes,
                                          int64_t M, int64_t V, int64_t K, int32_t dtype,
                                          int32_t reduction, const mhc_linear_launch* launch) {
  Plan p;
  return validate_bwd(x, weight, targets, lse, grad_loss, grad_lse, grad_x, grad_weight, workspace,
                      workspace_bytes, M, V, K, dtype, reduction, launch, &p);
}

mhc_status mhc_cross_entropy_validate_grads(const void* x, const void* weight,
                                            const int64_t* targets, const float* grad_loss,
                                            const float* loss, const float* lse,
                                            const void* grad_x, const void* grad_weight,
                                            const void* workspace, int64_t workspace_bytes,
                                            int64_t M, int64_t V, int64_t K, int32_t dtype,
                                            int32_t reduction, const mhc_linear_launch* launch) {
  Plan p;
  return validate_grads(x, weight, targets, grad_loss, loss, lse, grad_x, grad_weight, workspace,
                        workspace_bytes, M, V, K, dtype, reduction, launch, &p);
}

mhc_status mhc_cross_entropy_fwd(const void* x, const void* weight, const int64_t* targets,
                                 float* loss, float* lse, void* workspace,
                                 int64_t workspace_bytes, int64_t M, int64_t V, int64_t K,
                                 int32_t dtype, int32_t reduction, int64_t ignore_index,
                                 void* stream, const mhc_linear_launch* launch,
                                 void* start_event, void* stop_event) {
  Plan p;
  const mhc_status st = validate_fwd(x, weight, targets, loss, lse, workspace, workspace_bytes, M, V, K,
                                     dtype, reduction, launch, &p);
  if (st != MHC_SUCCESS) return st;
  const Call c = {x, weight, targets, nullptr, nullptr, nullptr, loss, lse, nullptr, nullptr,
                  static_cast<uint8_t*>(workspace), M, V, K, reduction, ignore_index};
  return run<kFwd>(c, p, dtype, stream, start_event, stop_event);
}

mhc_status mhc_cross_entropy_bwd(const void* x, const void* weight, const int64_t* targets,
                                 const float* lse, const float* grad_loss, const float* grad_lse,
                                 void* grad_x, void* grad_weight, void* workspace,
                                 int64_t workspace_bytes, int64_t M, int64_t V, int64_t K,
                                 int32_t dtype, int32_t reduction, int64_t ignore_index,
                                 void* stream, const mhc_linear_launch* launch,
                                 void* start_event, void* stop_event) {
  Plan p;
  const mhc_status st = validate_bwd(x, weight, targets, lse, grad_loss, grad_lse, grad_x, grad_weight,
                                     workspace, workspace_bytes, M, V, K, dtype, reduction, launch, &p);
  if (st != MHC_SUCCESS) return st;
  const Call c = {x, weight, targets, grad_loss, grad_lse, lse, nullptr, nullptr, grad_x, grad_weight,
                  static_cast<uint8_t*>(workspace), M, V, K, reduction, ignore_index};
  return run<kBwd>(c, p, dtype, stream, start_event, stop_event);
}

mhc_status mhc_cross_entropy_grads(const void* x, const void* weight, const int64_t* targets,
                                   const float* grad_loss, float* loss, float* lse, void* grad_x,
                                   void* grad_weight, void* workspace, int64_t workspace_bytes,
                                   int64_t M, int64_t V, int64_t K, int32_t dtype,
                                   int32_t reduction, int64_t ignore_index, void* stream,
                                   const mhc_linear_launch* launch, void* start_event,
                                   void* stop_event) {
  Plan p;
  const mhc_status st = validate_grads(x, weight, targets, grad_loss, loss, lse, grad_x, grad_weight,
                                       workspace, workspace_bytes, M, V, K, dtype, reduction, launch, &p);
  if (st != MHC_SUCCESS) return st;
  const Call c = {x, weight, targets, grad_loss, nullptr, nullptr, loss, lse, grad_x, grad_weight,
                  static_cast<uint8_t*>(workspace), M, V, K, reduction, ignore_index};
  return run<kGrads>(c, p, dtype, stream, start_event, stop_event);
}

}  // extern "C"
