// mhc_tiles_host.h - host half of the matrix products x W^T (internal; not part
// of the C ABI): the choice of a launch, places in a workspace, and the launches.

#pragma once

#include <math.h>

#include "mhc_host.h"
#include "mhc_launch.h"
#include "mhc_tiles.h"

namespace {

// ---------------------------------------------------------------------------
// Rows that are no whole pieces
//
// Operands whose rows are no multiple of 16 bytes cannot be loaded straight into
// LDS. Where the product is long enough they are copied into the workspace
// first, rows padded with zeros: one pass over them, against tiles that go
// through registers (2048 x 2048 x 2047 in bf16: 41 us, a product of the backward 81; with
// copies 37 and 36; 2048 x 2048 x 2048 takes 25 and 26). Where they pay: kPadForward.
// ---------------------------------------------------------------------------

struct PadJob {
  const uint8_t* in;
  uint8_t* out;
  int64_t rows;
  int64_t bytes;   // of a row of `in`
  int64_t pieces;  // 16-byte pieces of a row of `out` (of 4 bytes where `narrow`)
  int32_t narrow;
};

constexpr int kMostJobs = 4;

struct PadJobs {
  PadJob job[kMostJobs];
};

// Job blockIdx.y of four (an index into an argument would put it into scratch
// memory); a thread moves whole pieces of the padded rows.
__global__ __launch_bounds__(256) void linear_pad_kernel(PadJob a, PadJob b, PadJob c, PadJob d) {
  const uint32_t y = blockIdx.y;
  const PadJob j = {y == 0 ? a.in : y == 1 ? b.in : y == 2 ? c.in : d.in,
                    y == 0 ? a.out : y == 1 ? b.out : y == 2 ? c.out : d.out,
                    y == 0 ? a.rows : y == 1 ? b.rows : y == 2 ? c.rows : d.rows,
                    y == 0 ? a.bytes : y == 1 ? b.bytes : y == 2 ? c.bytes : d.bytes,
                    y == 0 ? a.pieces : y == 1 ? b.pieces : y == 2 ? c.pieces : d.pieces,
                    y == 0 ? a.narrow : y == 1 ? b.narrow : y == 2 ? c.narrow : d.narrow};
  const int size = j.narrow ? 4 : 16;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; id < j.rows * j.pieces;
       id += step) {
    const int64_t row = id / j.pieces, at = (id - row * j.pieces) * size;
    const uint8_t* p = j.in + row * j.bytes + at;
    const int64_t left = j.bytes - at;
    typedef u32x4 u32x4_at1 __attribute__((aligned(1)));
    u32x4 v = {0, 0, 0, 0};
    if (left >= size && size == 16) {
      v = *reinterpret_cast<const u32x4_at1*>(p);
    } else {
      uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < left && i < size) u[i / 4] |= static_cast<uint32_t>(p[i]) << (8 * (i % 4));
      v = u32x4{u[0], u[1], u[2], u[3]};
    }
    uint8_t* q = j.out + (row * j.pieces) * size + at;
    if (size == 16) {
      *reinterpret_cast<u32x4*>(q) = v;
    } else {
      const uint32_t w = v[0];
      *reinterpret_cast<uint32_t*>(q) = w;
    }
  }
}

// ---------------------------------------------------------------------------
// Host side: sizes and the choice of a launch
// ---------------------------------------------------------------------------

[[maybe_unused]] bool known_dtype(int32_t d) {
  return (d >= MHC_LINEAR_BF16 && d <= MHC_LINEAR_E4M3_MX) || d == MHC_LINEAR_I8_ROW;
}
int64_t elem(int32_t dtype) { return is8(dtype) ? 1 : 2; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Shape {
  int bm, bn;
};

Shape shape_of(int32_t kernel) {
  switch (kernel) {
    case MHC_LINEAR_SHORT: return {32, 64};
    case MHC_LINEAR_NARROW: return {64, 32};
    case MHC_LINEAR_SMALL: return {64, 64};
    case MHC_LINEAR_MEDIUM: return {128, 128};
    default: return {256, 256};
  }
}

constexpr int32_t kMaxSplits = 64;
constexpr int kMediumStages = 2;  // see the tile kernel

// A launch holds fewer than 2^32 threads along its grid. A large tile's operands
// may send it through four medium ones.
int64_t most_tiles(int32_t kernel) { return 1LL << (kernel == MHC_LINEAR_LARGE ? 21 : 23); }
constexpr int64_t kMaxRowsN = 1LL << 26;  // 16 rows of W to each block of 512 threads

mhc_status make_plan(int64_t M, int64_t N, int64_t K, int32_t dtype,
                     const mhc_linear_launch* launch, mhc_linear_launch* plan) {
  const int32_t want = launch != nullptr ? launch->kernel : 0;
  const int32_t parts = launch != nullptr ? launch->splits : 0;
  if (want < 0 || (want > MHC_LINEAR_LARGE && want != MHC_LINEAR_SHORT) || parts < 0 || parts > kMaxSplits)
    return fail(MHC_ERROR_INVALID_VALUE, "launch: kernel %d with %d splits does not exist", want,
                parts);
  const auto tiles = [&](int32_t k) {
    const Shape s = shape_of(k);
    return ceil_div(M, s.bm) * ceil_div(N, s.bn);
  };
  int32_t k = want;
  if (k == 0) {
    // The row kernel does not split its sum: 1, 4 and 16 rows x 24 columns take it 4.8, 5.3 and 7.0
    // us at K = 4096, the narrow tiles in parts 8.1, 8.4 and 8.7; x 1024 columns 5.5, 6.1 and 8.0 against
    // 10. Over a long sum with few columns the tiles would be ahead, at K = 28672 11.0, 12.1 and
    // 12.6 against 15.5, 19.3 and 32.9 (1024 columns 20 against 24 to 39).
    if (M <= 16) k = MHC_LINEAR_ROWS;
    else if (N <= 32) k = MHC_LINEAR_NARROW;
    else if (tiles(MHC_LINEAR_LARGE) >= 192) k = MHC_LINEAR_LARGE;
    else if (tiles(MHC_LINEAR_MEDIUM) >= 128) k = MHC_LINEAR_MEDIUM;
    else k = MHC_LINEAR_SMALL;
  }
  if (k == MHC_LINEAR_ROWS) {
    if (M > 16 || parts > 1)
      return fail(MHC_ERROR_INVALID_VALUE,
                  "launch: the row kernel takes at most 16 rows and one part");
    if (N > kMaxRowsN)
      return fail(MHC_ERROR_INVALID_VALUE, "N must be at most %lld where M is at most 16",
                  static_cast<long long>(kMaxRowsN));
    *plan = {k, 1};
    return ok();
  }
  if (tiles(k) * (parts > 1 ? parts : 1) > most_tiles(k))
    return fail(MHC_ERROR_INVALID_VALUE, "M, N and splits make more than %lld tiles",
                static_cast<long long>(most_tiles(k)));
  const int64_t all = ceil_div(K * elem(dtype), kTileK);
  int64_t s = parts;
  if (s == 0) {
    // at least 4 tiles of the sum in each part, and at most two blocks for each
    // CU, of the wide tiles one: 2048^3 in bf16 in one part of 256 blocks 25.8 us, in two
    // parts 34; 17 x 7168 x 4096 in four parts of 112 small tiles 14.6, in two 21.9;
    // 2048 x 24 x 28672 in 16 parts of 32 narrow tiles 29.3, in eight 31. More than 32 parts cost the join
    // more than they save: 17 x 24 x 28672 in 32 13.7, in 64 15.4
    s = 1;
    const int64_t slots = k == MHC_LINEAR_MEDIUM || k == MHC_LINEAR_LARGE ? 256 : 512;
    while (s < 32 && M > 0 && tiles(k) * s * 2 <= slots && all / (s * 2) >= 4) s *= 2;
  }
  if (s > all) s = all;
  // no empty part
  s = ceil_div(all, ceil_div(all, s));
  *plan = {k, static_cast<int32_t>(s)};
  return ok();
}

// The launch that takes the least time by a model, for the calls whose sums have no
// older order to keep: products of two weights, those of 8-bit integers (exact in
// any order) and those around a softmax. In us, a kernel takes `pass` for each pass
// of kTileK bytes while every CU has at most one block of it, and a CU with more
// works one off in `busy`; a tile's end takes `end`, a launch 3, and joining s parts 3.5
// and their bytes' way to memory and back. The constants are fitted to 8-bit and bf16
// products of 17 to 4096 rows x 1024 to 28672 x 512 to 28672; of 116 of them this takes
// the fastest launch or one within 5% of it 97 times, and one 10% off or more 11 times
// (36% at worst, 384 x 4096 x 8192 in bf16). 8-bit integers, the rule above
// and this one: 32 x 7168 x 4096 12.5 -> 9.8 us (small tiles in 4 parts, short ones in
// one), 256 x 4096 x 7168 21.9 -> 18.2, 1024 x 1024 x 4096 16.4 -> 11.9; two weights of
// 14336 x 7168 in bf16 and 24 rows 117 -> 74 (medium tiles, short ones).
struct Cost {
  int32_t kernel;
  double pass, busy, end;
};
constexpr Cost kCosts[] = {{MHC_LINEAR_SHORT, 0.21, 0.143, 0.4},
                           {MHC_LINEAR_SMALL, 0.30, 0.197, 0.65},
                           {MHC_LINEAR_MEDIUM, 0.75, 0.54, 2.7},
                           {MHC_LINEAR_LARGE, 1.5, 1.5, 12.0}};

// turned: operands with k down the rows, which have no short form. most: parts.
mhc_status best_plan(int64_t M, int64_t N, int64_t K, int32_t dtype, bool turned, int32_t most,
                     const mhc_linear_launch* launch, mhc_linear_launch* plan) {
  mhc_linear_launch want = {0, most == 1 ? 1 : launch != nullptr ? launch->splits : 0};
  if (launch != nullptr && launch->kernel != 0) want.kernel = launch->kernel;
  if (want.kernel != 0 || M == 0 || (M <= 16 && !turned)) return make_plan(M, N, K, dtype, &want, plan);
  const int64_t all = ceil_div(K * elem(dtype), kTileK);
  double least = INFINITY;
  mhc_linear_launch best = {MHC_LINEAR_SMALL, 1};
  for (const Cost& c : kCosts) {
    if (turned && c.kernel == MHC_LINEAR_SHORT) continue;
    const Shape shape = shape_of(c.kernel);
    const double tiles = static_cast<double>(ceil_div(M, shape.bm)) * static_cast<double>(ceil_div(N, shape.bn));
    for (int32_t s = 1; s <= 32; s *= 2) {
      if (want.splits != 0 ? s != 1 : s > 1 && (s > most || all / s < 4 || tiles * s > 1024)) break;
      const double parts = want.splits != 0 ? want.splits : s;
      double each = tiles * parts / 256;  // blocks of a CU
      if (c.kernel == MHC_LINEAR_LARGE) each = ceil(each);
      if (each < 1) each = 1;
      const double passes = ceil(static_cast<double>(all) / parts);
      double t = 3 + passes * fmax(c.pass, each * c.busy) + each * c.end;
      if (parts > 1) t += 3.5 + parts * static_cast<double>(M) * static_cast<double>(N) * 8 / 4e6;
      if (t < least) {
        least = t;
        best = {c.kernel, static_cast<int32_t>(parts)};
      }
    }
  }
  return make_plan(M, N, K, dtype, &best, plan);
}

int64_t round_up(int64_t v, int64_t to) { return ceil_div(v, to) * to; }

// Products of at least this many terms have operands without whole rows copied
// first. Forward in bf16, with at least kPadRows rows of each, through registers and with
// copies: 512 x 4096 x 2047 31 and 36 us, 2048 x 2048 x 2047 41 and 37, 4096 x 4096 x 2047
// 109 and 76. A product of the backward, where turned operands lose more: 1024 x 1024 x 1023 17.5
// and 19 us, 512 x 2048 x 2047 27 and 26 (x's gradient), 20 and 17 (the weight's), 2048 x 2048 x
// 2047 81 and 36. The rows' length alone decides: operands of whole rows at addresses that are no
// multiples of 16 are not copied (4096 x 7168 x 4096 197 us, so 455).
constexpr int64_t kPadForward = 3LL << 31;
constexpr int64_t kPadRows = 512;
constexpr int64_t kPadBackward = 3LL << 29;

// Places in the workspace, in bytes, each from a multiple of 256 on; `total` is
// -1 where a size does not fit.
struct Places {
  int64_t total = 0;
  int64_t take(int64_t bytes) {
    const int64_t here = total;
    if (total < 0 || bytes < 0 || bytes > INT64_MAX - 256 ||
        __builtin_add_overflow(total, round_up(bytes, 256), &total)) {
      total = -1;
      return 0;
    }
    return here;
  }
};

// Whether an operand can be loaded straight into LDS: whole, aligned 16-byte
// pieces, and where k runs down the rows all of it within a buffer's 31 bits.
template <bool TURNED>
bool whole(const Matrix& m, const TileShape& a) {
  if (reinterpret_cast<uintptr_t>(m.p) % 16 != 0 || m.ld % 16 != 0) return false;
  return TURNED ? static_cast<int64_t>(a.kturned / 2) * m.ld <= INT32_MAX : a.kbytes % 16 == 0;
}

template <int OP, bool TX, bool TW, class E>
bool straight(const TileArgs<E>& a) {
  if (!whole<TX>(a.x, a) || !whole<TW>(a.w, a)) return false;
  if (E::kW != kOne && !whole<TW>(a.w2, a)) return false;
  // the second half's columns of x begin where a piece does
  if (E::kHalves && a.xupper % 8 != 0) return false;
  // block scales come four of a row at a time
  const auto whole_scales = [](const uint8_t* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; };
  return OP != kOpMX || (a.kbytes % kTileK == 0 && whole_scales(a.xs) && whole_scales(a.ws) &&
                         (E::kW != kBoth || whole_scales(a.ws2)));
}

// The grid of tiles of BM x BN results (of either sum BN / kSums columns).
template <int BM, int BN, class E>
dim3 tile_grid(TileArgs<E>& a) {
  a.upper = static_cast<uint32_t>(ceil_div(a.M, BM));
  a.tiles_m = a.upper * (E::kHalves ? 2 : 1);
  a.tiles_n = static_cast<uint32_t>(ceil_div(a.N, BN / E::kSums));
  return dim3(a.tiles_m * a.tiles_n * a.splits);
}

template <int OP, int BM, int BN, int WM, int WN, int STAGES, bool TX, bool TW, class E>
hipError_t launch_tile(TileArgs<E> a, hipStream_t s, hipEvent_t start, hipEvent_t stop) {
  const dim3 grid = tile_grid<BM, BN>(a), block(64 * WM * WN);
  if (straight<OP, TX, TW>(a))
    return launch_kernel(linear_tile_kernel<OP, BM, BN, WM, WN, STAGES, true, TX, TW, E>, grid, block,
                         s, start, stop, a);
  return launch_kernel(linear_tile_kernel<OP, BM, BN, WM, WN, STAGES, false, TX, TW, E>, grid, block,
                       s, start, stop, a);
}

template <int OP, bool TX, bool TW, class E>
hipError_t launch_medium(const TileArgs<E>& a, hipStream_t s, hipEvent_t start, hipEvent_t stop) {
  return launch_tile<OP, 128, 128, 2, 2, kMediumStages, TX, TW>(a, s, start, stop);
}

constexpr uint32_t kUnits = 256;  // compute units: blocks of the wide kernel at once

// The large tiles are loaded straight into LDS only; other operands, and results of
// hardly any or of very many columns, go through the medium tiles, whose sums have
// the same order.
template <int OP, bool TX, bool TW, class E>
hipError_t launch_large(TileArgs<E> a, hipStream_t s, hipEvent_t start, hipEvent_t stop) {
  if (!straight<OP, TX, TW>(a)) return launch_medium<OP, TX, TW>(a, s, start, stop);
  // write_early reads 8 values of a row at a time, and 128 rows within 2^30 bytes
  if (wide_tiles(OP) && E::kEarly && (a.N < 8 || a.N > (1 << 22)))
    return launch_medium<OP, TX, TW>(a, s, start, stop);
  const dim3 grid = tile_grid<256, 256>(a);
  if constexpr (wide_tiles(OP))
    return launch_kernel(linear_wide_kernel<OP, TX, TW, E>, dim3(grid.x < kUnits ? grid.x : kUnits),
                         dim3(256), s, start, stop, a);
  else
    return launch_kernel(linear_large_kernel<OP, E>, grid, dim3(512), s, start, stop, a);
}

// One product and its epilogue, as planned. The backward's products (TW), those
// of two weights and those that are never split have no narrow form.
template <int OP, bool TX, bool TW, class E>
hipError_t launch_product(TileArgs<E> a, const mhc_linear_launch& plan, hipStream_t s,
                          hipEvent_t start, hipEvent_t stop) {
  const int64_t all = ceil_div(a.kbytes, kTileK);
  a.splits = static_cast<uint32_t>(plan.splits);
  a.per_split = static_cast<uint32_t>(ceil_div(all, plan.splits));
  const bool join = a.splits > 1;
  const hipEvent_t end = join ? nullptr : stop;
  hipError_t e;
  switch (plan.kernel) {
    case MHC_LINEAR_NARROW:
      if constexpr (!TW && E::kW == kOne && E::kSplits) {
        e = launch_tile<OP, 64, 32, 4, 1, 3, TX, TW>(a, s, start, end);
        break;
      }
    case MHC_LINEAR_SHORT:
      if constexpr (!TW) {
        e = launch_tile<OP, 32, 64, 2, 2, 4, TX, TW>(a, s, start, end);
        break;
      }
    case MHC_LINEAR_SMALL: e = launch_tile<OP, 64, 64, 2, 2, 3, TX, TW>(a, s, start, end); break;
    case MHC_LINEAR_MEDIUM: e = launch_medium<OP, TX, TW>(a, s, start, end); break;
    default: e = launch_large<OP, TX, TW>(a, s, start, end); break;
  }
  if constexpr (E::kSplits) {
    if (e != hipSuccess || !join) return e;
    const int64_t rows = E::kHalves ? 2 * a.M : a.M;
    const int64_t blocks = ceil_div(rows * ceil_div(a.N, 8), kJoinThreads);
    const auto run = [&](auto kernel) {
      return launch_kernel(kernel, dim3(static_cast<uint32_t>(blocks < 16384 ? blocks : 16384)),
                           dim3(kJoinThreads), s, nullptr, stop, a.partial, a.splits, rows, a.N, a.e);
    };
    if (a.N < 8) return run(linear_join_kernel<OP, E, 4, false>);
    return a.splits <= 4 ? run(linear_join_kernel<OP, E, 4, true>) : run(linear_join_kernel<OP, E, 8 / E::kSums, true>);
  }
  return e;
}

template <int OP, class E>
hipError_t launch_rows(const TileArgs<E>& t, hipStream_t s, hipEvent_t start, hipEvent_t stop) {
  // the fewest blocks for each of 256 CUs, and W's rows spread evenly over them
  const int64_t most = 16 / E::kSums;
  const int64_t wide = ceil_div(t.N, 256 * ceil_div(t.N, 256 * most));
  const RowsArgs<E> a = {static_cast<const uint8_t*>(t.x.p), static_cast<const uint8_t*>(t.w.p),
                         static_cast<const uint8_t*>(t.w2.p), t.xs, t.ws, t.ws2, t.M, t.N, t.kbytes,
                         t.kbytes, static_cast<uint32_t>(wide), t.e};
  const dim3 grid(static_cast<uint32_t>(ceil_div(t.N, wide)));
  return launch_kernel(linear_rows_kernel<OP, 8, E>, grid, dim3(512), s, start, stop, a);
}

PadJob pad_job(const void* in, void* out, int64_t rows, int64_t bytes, int64_t ld, bool narrow) {
  return {static_cast<const uint8_t*>(in), static_cast<uint8_t*>(out), rows, bytes,
          ld / (narrow ? 4 : 16), narrow ? 1 : 0};
}

hipError_t launch_pad(const PadJobs& jobs, int count, hipStream_t s, hipEvent_t start) {
  int64_t most = 1;
  for (int i = 0; i < count; ++i) {
    const int64_t blocks = ceil_div(jobs.job[i].rows * jobs.job[i].pieces, 256);
    if (blocks > most) most = blocks;
  }
  return launch_kernel(linear_pad_kernel, dim3(static_cast<uint32_t>(most < 4096 ? most : 4096), static_cast<uint32_t>(count)),
                       dim3(256), s, start, nullptr, jobs.job[0], jobs.job[1], jobs.job[2], jobs.job[3]);
}

// A product of the backward: the tile kernels from 64 x 64 on.
[[maybe_unused]] mhc_status plan_product(int64_t M, int64_t N, int64_t K, int32_t dtype, mhc_linear_launch* p) {
  const mhc_status st = make_plan(M, N, K, dtype, nullptr, p);
  if (st != MHC_SUCCESS || p->kernel >= MHC_LINEAR_SMALL) return st;
  const mhc_linear_launch small = {MHC_LINEAR_SMALL, 0};
  return make_plan(M, N, K, dtype, &small, p);
}

hipError_t launch_zero(void* p, int64_t count, hipStream_t s, hipEvent_t start, hipEvent_t stop) {
  const int64_t blocks = ceil_div(count, 256);
  return launch_kernel(linear_zero_kernel, dim3(static_cast<uint32_t>(blocks < 4096 ? blocks : 4096)),
                       dim3(256), s, start, stop, static_cast<uint16_t*>(p), count);
}

// Events of a call of several launches: the start goes to the first, the stop
// is recorded by an own (empty) marker after the last.
struct Marks {
  hipEvent_t start, stop;
  hipEvent_t first() {
    const hipEvent_t e = start;
    start = nullptr;
    return e;
  }
  // The events that no launch took, after the call's last.
  hipError_t end(hipError_t e, hipStream_t s) {
    if (e == hipSuccess && start != nullptr) e = hipEventRecord(first(), s);
    if (e == hipSuccess && stop != nullptr) e = hipEventRecord(stop, s);
    return e;
  }
};

}  // namespace
