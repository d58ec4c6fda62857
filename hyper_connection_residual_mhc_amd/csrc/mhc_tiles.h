// mhc_tiles.h - device half of the matrix products x W^T (internal; not part of
// the C ABI): tiles in LDS, the kernels for large, middling and small products and
// for few rows, and the join of split sums. What becomes of the sums is an
// epilogue's: linear, gated and cross-entropy libraries bring their own.

#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mhc_linear.h"
#include "mhc_rows.h"

#pragma clang fp contract(off)

namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef f32x8 f32x8_at4 __attribute__((aligned(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// What the operands of a product are. kOpE4M3 and kOpI8 have their scales applied
// in the epilogue, kOpMX in the matrix instruction. The sums of kOpI8 are 32-bit
// integers, held in the fp32 registers' bits: exact, in any order.
constexpr int kOpBF16 = MHC_LINEAR_BF16;
constexpr int kOpF16 = MHC_LINEAR_F16;
constexpr int kOpE4M3 = MHC_LINEAR_E4M3_ROW;
constexpr int kOpMX = MHC_LINEAR_E4M3_MX;
constexpr int kOpI8 = MHC_LINEAR_I8_ROW;

constexpr bool is8(int op) { return op == kOpE4M3 || op == kOpMX || op == kOpI8; }
// Whether large tiles are four waves' (see linear_wide_kernel).
constexpr bool wide_tiles(int op) { return op == kOpBF16 || op == kOpF16; }
// Scales of a row's, applied in the epilogue.
constexpr bool scaled(int op) { return op == kOpE4M3 || op == kOpI8; }
// Storage format of bias, residual, out and z.
constexpr int out_format(int op) { return op == kOpF16 ? kF16 : kBF16; }
// ---------------------------------------------------------------------------
// Epilogue
// ---------------------------------------------------------------------------

// erfc(x) exp(x^2) for x >= 0 as a polynomial in t = 1 / (1 + 0.44 x) without
// constant term, fitted for least relative error (7e-6 over [0, 14], far below
// the 2^-9 of a bf16 and the 2^-12 of an fp16 result). `half_erfc_sqrt2` gives
// erfc(a / sqrt 2) / 2 = the normal distribution's tail past a.
__device__ __forceinline__ float half_erfc_sqrt2(float a) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.44f * 0.70710678f, a, 1.0f));
  float q = -0.14439557f;
  q = fmaf(q, t, 0.34594810f);
  q = fmaf(q, t, 0.045597363f);
  q = fmaf(q, t, 0.26124406f);
  q = fmaf(q, t, 0.24308856f);
  q = fmaf(q, t, 0.24851908f);
  return 0.5f * q * t * __builtin_amdgcn_exp2f(-0.72134752f * a * a);
}

template <int ACT>
__device__ __forceinline__ float activate(float v) {
  if constexpr (ACT == MHC_ACT_RELU) return v < 0.0f ? 0.0f : v;
  if constexpr (ACT == MHC_ACT_SILU)
    return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * v));
  if constexpr (ACT == MHC_ACT_GELU) {
    // max(v, 0) - |v| tail(|v|); the tail is 0 from 30 on, where an infinite |v| would make 0 * inf
    const float a = fminf(fabsf(v), 30.0f);
    return (v < 0.0f ? 0.0f : v) - a * half_erfc_sqrt2(a);
  }
  return v;
}

// act'(v), for the backward; its limit, 0 or 1, at an infinite v (a z past the
// range of fp16 is stored as one), NaN at NaN alone.
template <int ACT>
__device__ __forceinline__ float slope(float v) {
  if constexpr (ACT == MHC_ACT_RELU) return v > 0.0f ? 1.0f : (v <= 0.0f ? 0.0f : v);
  if constexpr (ACT == MHC_ACT_SILU) {
    // from 200 on the sigmoid is 0 or 1, which times an infinite v would be a NaN
    const float c = v < -200.0f ? -200.0f : (v > 200.0f ? 200.0f : v);
    const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * c));
    return s * fmaf(c, 1.0f - s, 1.0f);
  }
  if constexpr (ACT == MHC_ACT_GELU) {
    const float a = fminf(fabsf(v), 30.0f);
    const float tail = half_erfc_sqrt2(a);
    const float density = 0.39894228f * __builtin_amdgcn_exp2f(-0.72134752f * a * a);
    const float r = (v < 0.0f ? tail : 1.0f - tail) + (v < 0.0f ? -a : a) * density;
    return v != v ? v : r;
  }
  return 1.0f;
}


// f with the activation as a constant.
template <typename Fn>
__device__ __forceinline__ void with_act(int32_t act, const Fn& f) {
  switch (act) {
    case MHC_ACT_RELU: f(std::integral_constant<int, MHC_ACT_RELU>()); break;
    case MHC_ACT_SILU: f(std::integral_constant<int, MHC_ACT_SILU>()); break;
    case MHC_ACT_GELU: f(std::integral_constant<int, MHC_ACT_GELU>()); break;
    default: f(std::integral_constant<int, MHC_ACT_NONE>()); break;
  }
}

// One sum in fp32, and two sums added: see kOpI8.
template <int OP>
__device__ __forceinline__ float sum_value(float v) {
  if constexpr (OP == kOpI8) return static_cast<float>(__float_as_int(v));
  else return v;
}

template <int OP>
__device__ __forceinline__ float sum_add(float a, float b) {
  if constexpr (OP == kOpI8) return __int_as_float(__float_as_int(a) + __float_as_int(b));
  else return a + b;
}

template <int OP>
__device__ __forceinline__ f32x8 sums_added(const f32x8& a, const f32x8& b) {
  if constexpr (OP == kOpI8) return __builtin_bit_cast(f32x8, __builtin_bit_cast(i32x8, a) + __builtin_bit_cast(i32x8, b));
  else return a + b;
}

// ---------------------------------------------------------------------------
// Matrix instructions
// ---------------------------------------------------------------------------

// Bytes of one row that one pass over the tiles in LDS covers: 64 values of 16
// bits or 128 of 8.
constexpr int kTileK = 128;

// One operand's values of one matrix instruction, row l % 16 in lane l. 16
// bits: 8 values from k = 8 (l / 16) on. 8 bits: 16 values from k = 16 (l / 16)
// on and 16 from 64 + 16 (l / 16) on; the lane's scale byte is that of the 32
// values from k = 32 (l / 16) on.
template <int OP>
struct Frag {
  i32x4 w[is8(OP) ? 2 : 1];
};

// acc[i] of lane l: row 4 (l / 16) + i of `a` against row l % 16 of `b`. sa, sb:
// the lane's e8m0 bytes (kMX), in byte BYTE_A and BYTE_B.
template <int OP, int BYTE_A = 0, int BYTE_B = 0>
__device__ __forceinline__ f32x4 mma(const Frag<OP>& a, const Frag<OP>& b, f32x4 acc, int sa,
                                     int sb) {
  const i32x4 a0 = a.w[0], b0 = b.w[0];
  if constexpr (OP == kOpBF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(
        __builtin_bit_cast(bf16x8, a0), __builtin_bit_cast(bf16x8, b0), acc, 0, 0, 0);
  } else if constexpr (OP == kOpF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(
        __builtin_bit_cast(f16x8, a0), __builtin_bit_cast(f16x8, b0), acc, 0, 0, 0);
  } else if constexpr (OP == kOpI8) {
    i32x4 c = __builtin_bit_cast(i32x4, acc);
    c = __builtin_amdgcn_mfma_i32_16x16x64_i8(a0, b0, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_i32_16x16x64_i8(a.w[1], b.w[1], c, 0, 0, 0);
    return __builtin_bit_cast(f32x4, c);
  } else {
    const i32x8 x = __builtin_shufflevector(a0, a.w[1], 0, 1, 2, 3, 4, 5, 6, 7);
    const i32x8 y = __builtin_shufflevector(b0, b.w[1], 0, 1, 2, 3, 4, 5, 6, 7);
    // 0x7F is the scale 1
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
        x, y, acc, 0, 0, BYTE_A, OP == kOpMX ? sa : 0x7F, BYTE_B, OP == kOpMX ? sb : 0x7F);
  }
}

// c += a b^T in place, in the accumulation registers: left to itself the compiler
// gives each result a new place and spends a sixth of a loop of 256 of them moving them
// about. It sees no matrix instruction here, so what it would wait for is waited for
// by hand: acc_ready() stands between these and any other access to c.
template <int OP>
__device__ __forceinline__ void mma_in_place(f32x4& c, const i32x4& a, const i32x4& b) {
  static_assert(OP == kOpBF16 || OP == kOpF16, "16-bit values");
  if constexpr (OP == kOpBF16)
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
  else
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}

// Writes the results of mma_in_place of one row of tiles to LDS, out of the accumulation
// registers (as inputs of the assembly, so that a row's place in a branch costs no copy).
__device__ __forceinline__ void put_row(const f32x4 (&c)[8], const uint32_t (&to)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) asm volatile("ds_write_b128 %0, %1" : : "v"(to[j]), "a"(c[j]) : "memory");
}

template <int TI>
__device__ __forceinline__ void acc_ready(f32x4 (&c)[TI][8]) {
#pragma unroll
  for (int i = 0; i < TI; ++i)
    asm volatile("s_nop 15\n\ts_nop 15"
                 : "+a"(c[i][0]), "+a"(c[i][1]), "+a"(c[i][2]), "+a"(c[i][3]), "+a"(c[i][4]),
                   "+a"(c[i][5]), "+a"(c[i][6]), "+a"(c[i][7]));
}

// The same with the scale bytes named by values that unrolling makes constants.
template <int OP>
__device__ __forceinline__ f32x4 mma_bytes(const Frag<OP>& a, const Frag<OP>& b, f32x4 acc, int sa,
                                           int sb, int byte_a, int byte_b) {
  const auto at = [&](auto i) {
    constexpr int A = decltype(i)::value;
    switch (byte_b) {
      case 0: return mma<OP, A, 0>(a, b, acc, sa, sb);
      case 1: return mma<OP, A, 1>(a, b, acc, sa, sb);
      case 2: return mma<OP, A, 2>(a, b, acc, sa, sb);
      default: return mma<OP, A, 3>(a, b, acc, sa, sb);
    }
  };
  switch (byte_a) {
    case 0: return at(std::integral_constant<int, 0>());
    case 1: return at(std::integral_constant<int, 1>());
    case 2: return at(std::integral_constant<int, 2>());
    default: return at(std::integral_constant<int, 3>());
  }
}

// ---------------------------------------------------------------------------
// Tiles in LDS
//
// A block computes BM x BN outputs from tiles of x and W in LDS, kTileK bytes
// of k at a time. x's rows are the second operand of the matrix instruction and
// W's the first, so a lane's four results are consecutive columns of one row;
// which W row stands at which place is chosen (4 consecutive rows out of every
// 4 G) so that over G tiles a lane's results are 4 G consecutive columns, which
// the epilogue moves in 16-byte accesses.
//
// An operand lies in memory with k along its rows ([rows, k]), or, in the
// backward's products, with k down its columns ([k, columns], TURNED): its tile
// is then 64 rows of k, and gfx950's transposing LDS read hands each lane 4
// consecutive k of one column. Either way the tile is a run of 16-byte pieces
// whose places within a row are exchanged by the row's number (swap), so that
// the lanes of a read spread over all banks:
//   k along the rows: x reads 16 rows at one k: piece ^ (row % 8);
//     W reads 4 consecutive rows of every 4 G: two bits of row % 4, and the
//     row's bit 4 G as the third;
//   k down the columns: a read touches 4 rows (k % 4) at 4 places: bits that
//     keep the 16 apart modulo 256 bytes, by what the places' distance is.
// Pieces are loaded straight into LDS where they are whole and 16-byte aligned
// (DMA: no registers, the range check of the buffer gives the zeros past the
// ends), through registers otherwise.
// ---------------------------------------------------------------------------

// Two loads' operands: where they start, how far their rows are apart, and what
// of them counts.
struct Matrix {
  const void* p;
  int64_t count;  // rows, or columns where k runs down
  int64_t ld;     // bytes from row to row
};

// What a product's W is.
constexpr int kOne = 0;
constexpr int kBoth = 1;   // two weights of N rows: each output has a sum with either
constexpr int kChain = 2;  // two turned weights, one after the other along k

struct TileShape {
  Matrix x, w, w2;     // w2: kBoth, kChain
  const uint8_t* xs;   // kMX
  const uint8_t* ws;   // kMX
  const uint8_t* ws2;  // kMX of kBoth
  int64_t M, N;
  uint32_t kbytes;    // bytes of k that count, in rows that run along it
  uint32_t kturned;   // and in operands where k runs down (no more than kbytes: rows may be padded)
  uint32_t kfirst;    // kChain: tiles of kTileK in the first weight's part of k
  uint32_t tiles_m, tiles_n;
  uint32_t upper, xupper;      // E::kHalves: tiles of M rows in the first half, and x's column where the second begins
  uint32_t splits, per_split;  // parts of the sum, and tiles of kTileK in each
  float* partial;              // [splits][sums][rows][N] where splits > 1
};

// E, the epilogue, says
//   kW       what W is (kOne, kBoth, kChain), kSums how many sums an output has;
//   kGroup   through how many tiles of 16 columns a lane's results are consecutive, 0
//            for as many as there are (of either weight);
//   kSplits  whether sums come in parts, which another kernel joins;
//   kHalves  two products in one launch: x (turned) is two blocks of M columns, and
//            the rows of the second one's results come after the M of the first;
//   kTakes   e.take() has the sums in their registers first;
//   kWrites  e.with<OP>(f) calls f(finish), and finish(m, n, count, v) gets up to 8
//            consecutive columns of a row, v[8 s ...] those of sum s;
//   kEarly   finish reads e.bias, of the columns, and e.residual, both of 16 bits and each
//            absent where it is null, and also takes them loaded (see write_early).
template <class E>
struct TileArgs : TileShape {
  E e;
};

// Offset that lies past every buffer: such a lane loads zeros.
constexpr uint32_t kOutside = 0x80000000u;

template <int V>
constexpr int log2_of() {
  return V <= 1 ? 0 : 1 + log2_of<V / 2>();
}

// How many consecutive tiles of 16 columns a lane's results run through.
template <class E>
constexpr int group_of(int tj) { return E::kGroup != 0 ? E::kGroup : E::kW == kBoth ? tj / 2 : tj < 4 ? tj : 4; }

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void*)p));
}

// Starts a load of BYTES for each lane from `offset` + `at` of the buffer to the
// wave's consecutive places in LDS from `to` on; a lane past the buffer's end
// brings zeros (the check counts `at` too). No vector register is written; the
// loads are waited for by wait_tiles(). m0 is a reserved register, which a list
// of clobbers cannot name: nothing else in this library may use it (a test
// reads the machine code for that). A vector instruction that writes a scalar
// register (a readfirstlane, or the compiler's own readlane of a spilled one) has
// to stand five wait states ahead of a load that reads it. The compiler keeps that
// distance for its own loads and not for these: where it might not be there, safe_load
// waits, and a test reads the machine code of all of them.
template <int BYTES>
__device__ __forceinline__ void load_to_lds(uint32_t offset, i32x4 rsrc, uint32_t at, uint32_t to) {
  if constexpr (BYTES == 16)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(to), "v"(offset), "s"(rsrc), "s"(at)
                 : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
                 :
                 : "s"(to), "v"(offset), "s"(rsrc), "s"(at)
                 : "memory");
}

// The same in two steps, which want something between them: m0 needs a cycle.
__device__ __forceinline__ void set_place(uint32_t to) {
  asm volatile("s_mov_b32 m0, %0" : : "s"(to) : "memory");
}
__device__ __forceinline__ void load_to_place(uint32_t offset, i32x4 rsrc, uint32_t at) {
  asm volatile("buffer_load_dwordx4 %0, %1, %2 offen lds"
               :
               : "v"(offset), "s"(rsrc), "s"(__builtin_amdgcn_readfirstlane(at))
               : "memory");
}

// The same, after the wait states that the buffer and `at` may need, and m0.
__device__ __forceinline__ void safe_load(uint32_t offset, i32x4 rsrc, uint32_t at) {
  asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               :
               : "v"(offset), "s"(rsrc), "s"(__builtin_amdgcn_readfirstlane(at))
               : "memory");
}

// The buffer of up to 2^31 - 1 bytes from p on, in scalar registers.
__device__ __forceinline__ i32x4 buffer_of(const void* p, int64_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(p);
  const int64_t most = 0x7FFFFFFF;
  const int32_t size = static_cast<int32_t>(bytes < 0 ? 0 : bytes < most ? bytes : most);
  return i32x4{__builtin_amdgcn_readfirstlane(static_cast<int32_t>(b)),
               __builtin_amdgcn_readfirstlane(static_cast<int32_t>(b >> 32)),
               __builtin_amdgcn_readfirstlane(size), kRsrcFormat};
}

typedef i32x4 i32x4_at1 __attribute__((aligned(1)));
typedef i32x4 i32x4_at2 __attribute__((aligned(2)));

// 16 bytes from p on, at an element's alignment.
template <int ELEM>
__device__ __forceinline__ i32x4 piece_at(const uint8_t* p) {
  if constexpr (ELEM == 2) return *reinterpret_cast<const i32x4_at2*>(p);
  else return *reinterpret_cast<const i32x4_at1*>(p);
}

// The first 0 < `left` < 16 bytes from p on, zeros after them: the 16 bytes that
// end there, shifted. Where they would begin before the row (`before`: whether 16
// bytes of it are in front of p) byte by byte, which only rows shorter than a
// piece come to: 14 loads one after another are 9 us.
template <int ELEM>
__device__ __forceinline__ i32x4 short_piece(const uint8_t* p, uint32_t left, bool before) {
  uint64_t lo = 0, hi = 0;
  if (before) {
    const i32x4 v = piece_at<ELEM>(p + left - 16);
    const uint64_t a = static_cast<uint32_t>(v[0]) | static_cast<uint64_t>(static_cast<uint32_t>(v[1])) << 32;
    const uint64_t b = static_cast<uint32_t>(v[2]) | static_cast<uint64_t>(static_cast<uint32_t>(v[3])) << 32;
    const uint32_t bits = (16 - left) * 8;
    lo = bits >= 64 ? b >> (bits - 64) : (a >> bits) | (b << (64 - bits));
    hi = bits >= 64 ? 0 : b >> bits;
  } else {
#pragma unroll 1
    for (uint32_t i = left; i-- > 0;) {
      hi = (hi << 8) | (lo >> 56);
      lo = (lo << 8) | p[i];
    }
  }
  return i32x4{static_cast<int32_t>(lo), static_cast<int32_t>(lo >> 32), static_cast<int32_t>(hi),
               static_cast<int32_t>(hi >> 32)};
}

// The part of an operand that a block loads: SPAN rows (or columns) of it. IS_W
// and G choose the places.
template <int SPAN, int THREADS, bool TURNED, bool IS_W, int G, bool DMA, int ELEM, int W = kOne>
struct Operand {
  static constexpr int kSpan = SPAN;
  static constexpr int kRows = W == kBoth ? SPAN / 2 : SPAN;  // of one weight
  static constexpr int Q = SPAN * 8 / THREADS;   // pieces a thread brings of one tile
  static constexpr int P = TURNED ? SPAN / 8 : 8;  // pieces of a row of the tile
  static constexpr int kRowBytes = P * 16;
  static constexpr uint32_t kEach = THREADS / P;   // rows that one round of the threads covers
  static_assert(SPAN * 8 % THREADS == 0 && kEach % (TURNED ? 4 : 32) == 0, "swap() is the same in every round");
  static_assert(kRows % kEach == 0 && (W != kBoth || !TURNED) && (W != kChain || TURNED), "a round is one weight's");
  const uint8_t* base;
  const uint8_t* base2;  // of the second weight
  i32x4 rsrc, rsrc2;
  uint32_t offset;  // of this thread's first piece
  uint32_t row, piece;
  uint32_t ld;
  uint32_t here;    // rows (columns) that exist
  uint32_t kbytes;  // bytes of k that exist
  uint32_t kfirst;
  bool inside;      // TURNED: whether columns are in front of the block's first one
  i32x4 held[2][DMA ? 1 : Q];  // through registers: two tiles on their way

  static __device__ __forceinline__ uint32_t swap(uint32_t row) {
    if constexpr (!TURNED) {
      if constexpr (IS_W) return (row & 3) | (((row >> log2_of<4 * G>()) & 1) << 2);
      return row & 7;
    } else if constexpr (!IS_W) {
      return (row & 3) << 1;
    } else if constexpr (G == 4) {
      return ((row & 1) << 3) | ((row >> 1) & 1);
    } else {
      return P == 8 ? ((row >> 1) & 1) << 2 : 0;
    }
  }

  __device__ __forceinline__ void init(const Matrix& m, int64_t first, const TileShape& a) {
    init(m, first, m.count - first, a);
  }
  // `left` rows (columns) exist from `first` on
  __device__ __forceinline__ void init(const Matrix& m, int64_t first, int64_t left, const TileShape& a) {
    kbytes = TURNED ? a.kturned : a.kbytes;
    here = static_cast<uint32_t>(left < kRows ? left : kRows);
    ld = static_cast<uint32_t>(m.ld);
    inside = first > 0;
    const int64_t at = TURNED ? first * ELEM : first * m.ld;
    const int64_t size = TURNED ? kbytes / ELEM * m.ld - first * ELEM : here * m.ld;
    base = static_cast<const uint8_t*>(m.p) + at;
    rsrc = buffer_of(base, size);
    if constexpr (W != kOne) {
      base2 = static_cast<const uint8_t*>(a.w2.p) + at;
      rsrc2 = buffer_of(base2, size);
      kfirst = a.kfirst;
    }
    row = threadIdx.x / P;
    piece = ((threadIdx.x % P) ^ swap(row)) * 16;
    offset = row * ld + piece;
  }

  // Starts the loads of round q of the tile kt into `to`, the tile's place in LDS.
  template <int SET = 0>
  __device__ __forceinline__ void start(uint32_t kt, uint32_t to, int q) {
    const bool second = W == kBoth ? q * kEach >= kRows : W == kChain && kt >= kfirst;
    const uint32_t rows = q * kEach - (W == kBoth && second ? kRows : 0);
    if (W == kChain && second) kt -= kfirst;
    const i32x4 from = W != kOne && second ? rsrc2 : rsrc;
    if constexpr (DMA) {
      const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
      const uint32_t dst = to + (q * THREADS + wave * 64) * 16;
      // a tile's last rows end inside it where k runs along them; where k runs
      // down, what is past the end is past the buffer's end
      if constexpr (TURNED)
        load_to_lds<16>(offset, from, (kt * (kTileK / ELEM) + rows) * ld, dst);
      else
        load_to_lds<16>(kt * kTileK + piece < kbytes ? offset : kOutside, from,
                        kt * kTileK + rows * ld, dst);
    } else {
      held[SET][q] = i32x4{0, 0, 0, 0};
      uint32_t left;  // bytes of the piece that exist
      const uint8_t* const begin = W != kOne && second ? base2 : base;
      const uint8_t* p = begin;
      if constexpr (TURNED) {
        const uint32_t k = kt * (kTileK / ELEM) + rows + row;
        left = k * ELEM < kbytes && piece < here * ELEM ? here * ELEM - piece : 0;
        p += static_cast<int64_t>(k) * ld + piece;
      } else {
        const uint32_t k = kt * kTileK + piece;
        left = rows + row < here && k < kbytes ? kbytes - k : 0;
        p += (rows + row) * ld + k;  // at most 256 rows of 4 MiB
      }
      if (left >= 16)
        held[SET][q] = piece_at<ELEM>(p);
      else if (left > 0)
        held[SET][q] = short_piece<ELEM>(p, left, TURNED ? piece > 0 || inside : p - begin >= 16);
    }
  }

  // DMA: what the loads of one pass share, and load q of them, whose place is set.
  struct Pass {
    i32x4 from;
    uint32_t offset, at;
  };
  __device__ __forceinline__ Pass pass(uint32_t kt) const {
    Pass p;
    const bool second = W == kChain && kt >= kfirst;
    if (second) kt -= kfirst;
    p.from = W == kChain && second ? rsrc2 : rsrc;
    p.offset = TURNED || kt * kTileK + piece < kbytes ? offset : kOutside;
    p.at = TURNED ? kt * (kTileK / ELEM) * ld : kt * kTileK;
    return p;
  }
  template <bool SAFE = false>
  __device__ __forceinline__ void load(const Pass& p, int q) const {
    const bool second = W == kBoth && q * kEach >= kRows;
    const uint32_t rows = q * kEach - (second ? kRows : 0);
    if constexpr (SAFE) safe_load(p.offset, second ? rsrc2 : p.from, p.at + rows * ld);
    else load_to_place(p.offset, second ? rsrc2 : p.from, p.at + rows * ld);
  }

  // Through registers: writes the loaded tile.
  template <int SET>
  __device__ __forceinline__ void put(uint8_t* to) {
    if constexpr (!DMA) {
#pragma unroll
      for (int q = 0; q < Q; ++q)
        *reinterpret_cast<i32x4*>(to + (q * THREADS + threadIdx.x) * 16) = held[SET][q];
    }
  }
};

// This lane's reads of an operand's tile: `first` is the wave's first row (or
// column) of the SPAN; tile t is 16 rows of x, or 16 of W spread over its group.
template <typename O, bool TURNED, bool IS_W, int G, int W = kOne>
struct Reader {
  // rows from one group of tiles to the next: kBoth has one of either weight
  static constexpr int kGroup = W == kBoth ? O::kRows : 16 * G;
  uint32_t at[2];  // !TURNED: the places of the two pieces of a pass; TURNED: at[0]

  __device__ __forceinline__ void init(uint32_t first) {
    const uint32_t lane = threadIdx.x % 64, low = lane % 16, g = lane / 16;
    if constexpr (!TURNED) {
      const uint32_t row = first + (IS_W ? (low / 4) * (4 * G) + low % 4 : low);
      const uint32_t f = O::swap(row) * 16;
      at[0] = row * kTileK + ((g * 16) ^ f);
      at[1] = row * kTileK + ((64 + g * 16) ^ f);
    } else {
      // rows k = 8 g + low / 4 (and 4 more), 4 columns from `column` on
      const uint32_t r = low / 4, q = low % 4;
      const uint32_t column = first + q * (IS_W ? 4 * G : 4);
      at[0] = (g * 8 + r) * O::kRowBytes + (((column / 8) ^ O::swap(r)) * 16) + column % 8 * 2;
    }
  }

  // Row of the tile that this lane's values of tile t are.
  static __device__ __forceinline__ uint32_t row_of(uint32_t first, int t) {
    const uint32_t low = threadIdx.x % 16;
    return first + (IS_W ? (t / G) * kGroup + (low / 4) * (4 * G) + (t % G) * 4 + low % 4
                         : t * 16 + low);
  }

  // Piece h of tile t: 16 bytes along k, the pass's half h.
  __device__ __forceinline__ i32x4 read(const uint8_t* tile, int t, int h) const {
    if constexpr (!TURNED) {
      const uint32_t row = IS_W ? (t / G) * kGroup + (t % G) * 4 : t * 16;
      return *reinterpret_cast<const i32x4*>(tile + at[h] + row * kTileK);
    } else {
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      typedef int32_t i32x2 __attribute__((ext_vector_type(2)));
      // the tile's columns from the reader's: an XOR where they fall within the
      // pieces that are exchanged
      uint32_t place = at[0];
      if constexpr (!IS_W)
        place = (place ^ ((t % 4) * 32)) + t / 4 * 128;
      else if constexpr (G == 4)
        place = (place ^ (((t % 4) / 2) * 16 + (t / 4) % 2 * 128)) + t % 2 * 8 + t / 8 * 256;
      else
        place += t * 8;
      const uint8_t* p = tile + place + h * 32 * O::kRowBytes;
      i32x2 v[2];
#pragma unroll
      for (int half = 0; half < 2; ++half)
        v[half] = __builtin_bit_cast(
            i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                       (__attribute__((address_space(3))) s16x4*)(p + half * 4 * O::kRowBytes)));
      const i32x2 lo = v[0], hi = v[1];
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3);
    }
  }
};

// At most LEFT of this wave's loads into LDS are still on their way; then so it
// is for every wave, and every wave is done with the tile before this one.
template <int LEFT>
__device__ __forceinline__ void wait_tiles() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(LEFT) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The lanes of a wave see each other's LDS writes (which a wave's own LDS
// instructions do in order; this keeps the compiler's order).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Which tile a block takes: blocks go round the 8 XCDs, so consecutive tiles
// are given to every eighth block, and tiles run down 4 rows of tiles before
// the next column: the blocks of one XCD share rows of x and W in its L2.
struct Place {
  int64_t m0, n0;
  uint32_t part;
  bool second;  // E::kHalves: of the second half
};

template <int BM, int BN, bool HALVES>
__device__ __forceinline__ Place place_of(const TileShape& a, uint32_t id = blockIdx.x) {
  // Quotients are made in vector registers; what is the same in every lane is
  // taken back to scalar ones, or all that follows from it would stay there.
  const uint32_t tiles = a.tiles_m * a.tiles_n;
  const uint32_t part = __builtin_amdgcn_readfirstlane(id / tiles);
  id -= part * tiles;
  const uint32_t each = tiles / 8, more = tiles % 8, xcd = id % 8, k = id / 8;
  id = xcd * each + (xcd < more ? xcd : more) + k;
  const uint32_t band = __builtin_amdgcn_readfirstlane(id / (4 * a.tiles_n));
  const uint32_t high = min(4u, a.tiles_m - 4 * band);
  id -= band * 4 * a.tiles_n;
  const uint32_t column = __builtin_amdgcn_readfirstlane(id / high);
  uint32_t row = 4 * band + id - column * high;
  const bool second = HALVES && row >= a.upper;
  if (second) row -= a.upper;
  return {static_cast<int64_t>(row) * BM, static_cast<int64_t>(column) * BN, part, second};
}

// f(constant) of the one of 0..N-1 that k is, the same in every lane.
template <int N, class F>
__device__ __forceinline__ void each_of(int k, const F& f) {
  if constexpr (N == 1) f(std::integral_constant<int, 0>());
  else if (k == N - 1) f(std::integral_constant<int, N - 1>());
  else each_of<N - 1>(k, f);
}

// The 8 values of 16 bits behind the first `back` (0 to 7) of v.
__device__ __forceinline__ u32x4 values_behind(u32x4 v, int back) {
  v = (back & 4) != 0 ? u32x4{v[2], v[3], 0, 0} : v;
  v = (back & 2) != 0 ? u32x4{v[1], v[2], v[3], 0} : v;
  const u32x4 half = {__builtin_amdgcn_alignbit(v[1], v[0], 16), __builtin_amdgcn_alignbit(v[2], v[1], 16),
                      __builtin_amdgcn_alignbit(v[3], v[2], 16), v[3] >> 16};
  return (back & 1) != 0 ? half : v;
}

// The results of a wide tile, with what the epilogue reads on its way before it is
// needed: one wave to a SIMD has no other to wait under. A lane's columns are the
// same in every row, so their bias is loaded once; a row's residual (ROWS) is loaded as
// soon as the one of the step before is used, a step ahead, without a branch, since one
// around a load in a loop is a wait for it: past the last row from there, and a row's
// short last chunk from the 8 values that end there. The last step starts no load, and
// all are used by name: one on its way there would be waited for in the next tile's passes.
// Waited for chunk by chunk they took 5 us of a tile's end (a bias) and 11 (a residual):
// 8192 x 8192 x 512 with both 148 us, so 96 (eight waves of 128 x 64: 130).
template <int OP, bool ROWS, int TI, int TJ, int WN, class E>
__device__ __forceinline__ void write_early(const TileArgs<E>& a, const Place& at, uint8_t* lds,
                                            f32x4 (&acc)[TI][TJ]) {
  static_assert(TJ == 8 && E::kSums == 1 && E::kSplits && !E::kHalves && out_format(OP) != kF32,
                "a row of 128 columns in 16 lanes");
  constexpr int G = group_of<E>(TJ), kCols = TJ * 16, kChunks = 4;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const uint32_t lane = threadIdx.x % 64, low = lane % 16, g = lane / 16;
  const int64_t m0 = at.m0 + (wave / WN) * (TI * 16), n = at.n0 + (wave % WN) * kCols + low * 8;
  float* const mine = reinterpret_cast<float*>(lds) + wave * (16 * kCols);
  const auto place = [](uint32_t row, uint32_t col) { return row * kCols + (col ^ (row % 8 * 4)); };
  uint32_t to[TJ];
#pragma unroll
  for (int j = 0; j < TJ; ++j)
    to[j] = lds_address(mine) + place(low, (j / G) * (16 * G) + g * (4 * G) + (j % G) * 4) * 4;
  // lane (g, low) has columns n.. of rows g, g + 4, g + 8 and g + 12 of a step
  const bool whole = at.m0 + 256 <= a.M && at.n0 + 256 <= a.N;
  const int count = whole || n + 8 <= a.N ? 8 : n < a.N ? static_cast<int>(a.N - n) : 0;
  const int back = count > 0 ? 8 - count : 0;
  const int64_t from = count > 0 ? n - back : 0;
  // (a wave whose rows are all past the last reads the last one)
  const int64_t m_first = min(m0, a.M - 1);
  const uint8_t* const base = static_cast<const uint8_t*>(a.e.residual) + m_first * a.N * 2;
  const uint32_t ld = static_cast<uint32_t>(a.N * 2), column_at = static_cast<uint32_t>(from * 2);
  const uint32_t last = static_cast<uint32_t>(min(a.M - 1 - m_first, static_cast<int64_t>(TI * 16 - 1))) * ld;
  u32x4 rows[kChunks] = {};
  const auto load = [&](int step, int k) {
    const uint32_t row = min((g + step * 16 + k * 4) * ld, last);
    rows[k] = *reinterpret_cast<const u32x4_at2*>(base + (row + column_at));
  };
  u32x4 bias = {0, 0, 0, 0};
  if (a.e.bias != nullptr) bias = *reinterpret_cast<const u32x4_at2*>(static_cast<const uint8_t*>(a.e.bias) + from * 2);
  if constexpr (ROWS) {
#pragma unroll
    for (int k = 0; k < kChunks; ++k) load(0, k);
    asm volatile("" : : "v"(rows[0]), "v"(rows[1]), "v"(rows[2]), "v"(rows[3]));
  }
  asm volatile("" : : "v"(bias));
  if (!whole) bias = values_behind(bias, back);
  a.e.template with<OP>([&](const auto& finish) {
    const auto one = [&](int step, auto more) {
      each_of<TI>(step, [&](auto i) { put_row(acc[i], to); });
      wave_sync();
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const uint32_t row = g + 4 * k;
        const f32x4 p = *reinterpret_cast<const f32x4*>(mine + place(row, low * 8));
        const f32x4 q = *reinterpret_cast<const f32x4*>(mine + place(row, low * 8 + 4));
        float v[8] = {p[0], p[1], p[2], p[3], q[0], q[1], q[2], q[3]};
        if constexpr (ROWS) asm volatile("" : : "v"(rows[k]));
        const int64_t m = m0 + step * 16 + row;
        if (whole) finish(m, n, 8, v, bias, rows[k]);
        else if (count > 0 && m < a.M) finish(m, n, count, v, bias, values_behind(rows[k], back));
        if constexpr (decltype(more)::value) load(step + 1, k);
      }
      wave_sync();
    };
#pragma unroll 1
    for (int step = 0; step < (ROWS ? TI - 1 : TI); ++step) one(step, std::bool_constant<ROWS>());
    if constexpr (ROWS) one(TI - 1, std::false_type());
  });
}

// The tile's results, written. Lane l of wave (wm, wn) holds in acc[i][j] four
// consecutive columns of row 16 i + l % 16 of the wave's part; over the G tiles
// of a group they are 4 G consecutive ones. LDS: SIZE bytes.
template <int OP, int BM, int BN, int WM, int WN, int SIZE, bool OWN, class E>
__device__ __forceinline__ void write_tile(const TileArgs<E>& a, const Place& at, uint8_t* lds,
                                           f32x4 (&acc)[BM / WM / 16][BN / WN / 16]) {
  constexpr int TI = BM / WM / 16, TJ = BN / WN / 16;
  constexpr int G = group_of<E>(TJ);
  constexpr int kSums = E::kSums;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const uint32_t lane = threadIdx.x % 64, low = lane % 16, g = lane / 16;
  const uint32_t wm = wave / WN, wn = wave % WN;
  // A wave's results go through its own part of LDS, from where its lanes take
  // 8 consecutive columns each of whole rows: one loop for every activation
  // instead of TI * TJ / 2 copies (3% of a 256 x 256 tile's time at K = 4096).
  constexpr int kWide = TJ * 16;
  constexpr int kSteps = BM * BN * 4 > SIZE ? BM * BN * 4 / SIZE : 1;
  constexpr int kRows = TI * 16 / kSteps;
  constexpr int kCols = kWide / kSums;  // outputs: a row holds those of one sum, then of the other
  static_assert(TI % kSteps == 0 && BM * BN * 4 / kSteps <= SIZE, "the results fit");
  if constexpr (!OWN) __syncthreads();  // every wave is done with the tiles
  float* mine = reinterpret_cast<float*>(lds) + wave * (kRows * kWide);
  // four columns, at pieces exchanged by the row, or 16 rows would take turns at four pieces
  const auto place = [](uint32_t row, uint32_t col) { return row * kWide + (col ^ (row % 8 * 4)); };
  const bool whole = at.m0 + BM <= a.M && at.n0 + BN / kSums <= a.N;
  const int64_t top = at.second ? a.M : 0;  // rows in front of this half's
  if constexpr (TJ == 8 && E::kEarly) {
    if (a.splits == 1) {
      if (a.e.residual != nullptr) return write_early<OP, true, TI, TJ, WN>(a, at, lds, acc);
      return write_early<OP, false, TI, TJ, WN>(a, at, lds, acc);
    }
  }
  constexpr bool kByName = TJ == 8;  // one copy of all that follows, and a step's results by name
  constexpr int kCopies = kByName ? 1 : kSteps;
  uint32_t to[TJ];
#pragma unroll
  for (int j = 0; j < TJ; ++j)
    to[j] = lds_address(mine) + place(low, (j / G) * (16 * G) + g * (4 * G) + (j % G) * 4) * 4;
#pragma unroll kCopies
  for (int step = 0; step < kSteps; ++step) {
    if constexpr (kByName) {
      static_assert(TI == kSteps, "a row of tiles in a step");
      each_of<kSteps>(step, [&](auto i) { put_row(acc[i], to); });
    } else {
#pragma unroll
      for (int i = 0; i < TI / kSteps; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j)
          *reinterpret_cast<f32x4*>(mine + place(16 * i + low, (j / G) * (16 * G) + g * (4 * G) + (j % G) * 4)) =
              acc[step * (TI / kSteps) + i][j];
    }
    wave_sync();
    const int64_t m0 = at.m0 + wm * (TI * 16) + step * kRows;
    const int64_t n0 = at.n0 + wn * kCols;
    const auto each = [&](const auto& sink) {
      constexpr int kAhead = TJ == 8 ? 4 : 2;  // chunks whose other inputs are loaded together: four waves have no others to wait under
#pragma unroll kAhead
      for (uint32_t id = lane; id < kRows * kCols / 8; id += 64) {
        const uint32_t row = id / (kCols / 8), col = id % (kCols / 8) * 8;
        const int64_t m = m0 + row, n = n0 + col;
        if (whole || (m < a.M && n < a.N)) {
          float v[8 * kSums];
#pragma unroll
          for (int s = 0; s < kSums; ++s) {
            const f32x4 p = *reinterpret_cast<const f32x4*>(mine + place(row, s * kCols + col));
            const f32x4 q = *reinterpret_cast<const f32x4*>(mine + place(row, s * kCols + col + 4));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[8 * s + e] = p[e];
              v[8 * s + 4 + e] = q[e];
            }
          }
          sink(top + m, n, whole ? 8 : static_cast<int>(min(a.N - n, static_cast<int64_t>(8))), v);
        }
      }
    };
    if (E::kSplits && a.splits > 1) {
      const int64_t rows = E::kHalves ? 2 * a.M : a.M;
      float* partial = a.partial + static_cast<int64_t>(at.part) * kSums * rows * a.N;
      each([&](int64_t m, int64_t n, int count, float(&v)[8 * kSums]) {
#pragma unroll
        for (int s = 0; s < kSums; ++s) {
          Chunk<kF32> c;
          float u[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] = v[8 * s + e];
          narrow_chunk<kF32>(u, c);
          store_chunk<kF32>(partial + (s * rows + m) * a.N + n, count, c);
        }
      });
    } else if constexpr (!(kByName && E::kEarly)) {
      a.e.template with<OP>([&](const auto& finish) { each(finish); });
    }
    wave_sync();
  }
}

// The end of a tile. OWN: its LDS is the results' alone.
template <int OP, int BM, int BN, int WM, int WN, int SIZE, bool OWN = false, class E>
__device__ __forceinline__ void end_tile(const TileArgs<E>& a, const Place& at, uint8_t* lds,
                                         f32x4 (&acc)[BM / WM / 16][BN / WN / 16]) {
  static_assert(!E::kTakes || !E::kSplits, "whole sums");
  if constexpr (E::kTakes) a.e.template take<OP, BM / WM / 16, BN / WN / 16, WN>(a, at, acc);
  if constexpr (E::kWrites) write_tile<OP, BM, BN, WM, WN, SIZE, OWN>(a, at, lds, acc);
}

// ---------------------------------------------------------------------------
// Tile kernel
//
// Small and middling products: blocks are few or the tiles small, so what
// counts is the time from one tile to the next. With DMA, STAGES tiles are in
// LDS and all but one of them on their way; block scales (kMX, where a
// row's come by the four) go the same way. Through registers there are two
// stages, and block scales are read for each tile by the lanes that use them.
//
// 64 x 64 tiles in three stages (three blocks to a CU): 256 x 4096 x 4096 in
// bf16, in the two parts that the policy gives it, 19.8 us, two stages 23.2,
// four 19.9; 512 x 4096 x 4096 by name and in one part 26.1, 32.1 and 27.0.
// 128 x 128 in two stages (two blocks
// to a CU, which fill each other's waits): 1024 x 4096 x 4096 44 us, three or
// four stages and one block 50. Block scales through LDS: 128 x 4096 x 7168 18.3
// us, by each lane 23.9. At least two waves to a SIMD are asked for: with more
// registers than that the compiler moves results between the two register
// files (1024 x 4096 x 4096: 49.6 us).
// ---------------------------------------------------------------------------

template <int OP, int BM, int BN, int WM, int WN, int STAGES, bool DMA, bool TX, bool TW, class E>
__global__ __launch_bounds__(64 * WM * WN, 2) void linear_tile_kernel(TileArgs<E> a) {
  constexpr int kThreads = 64 * WM * WN;
  constexpr int TI = BM / WM / 16, TJ = BN / WN / 16;
  constexpr int G = group_of<E>(TJ);
  constexpr int W = E::kW;
  constexpr int ELEM = is8(OP) ? 1 : 2;
  constexpr int kStages = DMA ? STAGES : 2;
  constexpr uint32_t kBuffer = (BM + BN) * kTileK;
  constexpr bool kScales = OP == kOpMX;
  typedef Operand<BM, kThreads, TX, false, 1, DMA, ELEM> OpX;
  typedef Operand<BN, kThreads, TW, true, G, DMA, ELEM, W> OpW;
  constexpr int kLoads = OpX::Q + OpW::Q;  // of a wave, for a tile
  constexpr uint32_t kWavesX = (BM + 63) / 64;  // that bring the scales of x
  static_assert(!kScales || kWavesX * 64 + BN <= kThreads, "a scale load for each row");
  __shared__ __align__(1024) uint8_t lds[kStages][kBuffer];
  // kMX, DMA: the scales of four passes, of x's rows and then of W's, twice
  constexpr uint32_t kScaleRows = kWavesX * 64 + (W == kBoth ? 2 * 64 : (BN + 63) / 64 * 64);
  __shared__ __align__(1024) uint8_t scales[2][kScales && DMA ? kScaleRows * 16 : 16];

  const Place place = place_of<BM, BN / E::kSums, E::kHalves>(a);
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const uint32_t lane = threadIdx.x % 64, g = lane / 16;
  const uint32_t wm = wave / WN, wn = wave % WN;
  constexpr uint32_t kWaveW = W == kBoth ? TJ * 8 : TJ * 16;  // a wave's rows of a weight
  OpX lx;
  OpW lw;
  if constexpr (E::kHalves) lx.init(a.x, place.m0 + (place.second ? a.xupper : 0), a.M - place.m0, a);
  else lx.init(a.x, place.m0, a);
  lw.init(a.w, place.n0, a);
  Reader<OpX, TX, false, 1> rx;
  Reader<OpW, TW, true, G, W> rw;
  rx.init(wm * (TI * 16));
  rw.init(wn * kWaveW);

  // Block scales. DMA: thread r brings 16 bytes of row r, x's then W's, which are
  // those of four passes: a load of 4 bytes for each pass asks the L2 for as many
  // lines as two thirds of the operands (two weights of 14336 x 7168 and 24
  // rows: 55 -> 43.5 us).
  // Else: each lane the bytes of its own rows; rows past the end read the last
  // row's (their values are zeros), and past the last block of a row any finite
  // scale does (those values are zeros too).
  const uint32_t kblocks = (a.kbytes + 31) / 32;
  i32x4 sr = {0, 0, 0, 0};
  uint32_t so = kOutside;
  uint32_t ox[kScales && !DMA ? TI : 1], ow[kScales && !DMA ? TJ : 1];
  uint32_t sx[kScales ? TI : 1], sw[kScales ? TJ : 1], nx[kScales ? TI : 1], nw[kScales ? TJ : 1];
  const uint8_t* xs = kScales ? a.xs + place.m0 * kblocks : nullptr;
  const uint8_t* ws = kScales ? a.ws + place.n0 * kblocks : nullptr;
  const uint8_t* ws2 = kScales && W == kBoth ? a.ws2 + place.n0 * kblocks : nullptr;
  sx[0] = sw[0] = 0;
  if constexpr (kScales && DMA) {
    // kBoth: one wave brings a weight's rows
    const bool of_x = wave < kWavesX, of_2 = W == kBoth && wave == kWavesX + 1;
    static_assert(W != kBoth || OpW::kRows <= 64, "a weight's scales are one wave's");
    const uint32_t r = threadIdx.x - (of_x ? 0 : of_2 ? (kWavesX + 1) * 64 : kWavesX * 64);
    sr = buffer_of(of_x ? xs : of_2 ? ws2 : ws, static_cast<int64_t>(of_x ? lx.here : lw.here) * kblocks);
    if (r < (of_x ? lx.here : lw.here)) so = r * kblocks;
  } else if constexpr (kScales) {
#pragma unroll
    for (int i = 0; i < TI; ++i) ox[i] = min(rx.row_of(wm * (TI * 16), i), lx.here - 1) * kblocks + g;
#pragma unroll
    for (int j = 0; j < TJ; ++j)
      ow[j] = min(rw.row_of(wn * kWaveW, W == kBoth ? j % G : j), lw.here - 1) * kblocks + g;
  }
  const auto read_scales = [&](uint32_t kt) {
    if constexpr (kScales && !DMA) {
      const bool in = kt * 4 + g < kblocks;
#pragma unroll
      for (int i = 0; i < TI; ++i) nx[i] = in ? xs[ox[i] + kt * 4] : 0;
#pragma unroll
      for (int j = 0; j < TJ; ++j) nw[j] = in ? (W == kBoth && j >= G ? ws2 : ws)[ow[j] + kt * 4] : 0;
    }
  };
  const auto take_scales = [&](uint32_t kt) {
    if constexpr (kScales && DMA) {
      const uint8_t* const from = scales[kt / 4 % 2] + kt % 4 * 4 + g;
#pragma unroll
      for (int i = 0; i < TI; ++i) sx[i] = from[rx.row_of(wm * (TI * 16), i) * 16];
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        const uint32_t r = W == kBoth ? rw.row_of(wn * kWaveW, j % G) + (j / G) * 64 : rw.row_of(wn * kWaveW, j);
        sw[j] = from[(kWavesX * 64 + r) * 16];
      }
    } else if constexpr (kScales) {
#pragma unroll
      for (int i = 0; i < TI; ++i) sx[i] = nx[i];
#pragma unroll
      for (int j = 0; j < TJ; ++j) sw[j] = nw[j];
    }
  };

  f32x4 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  const auto multiply = [&](const uint8_t* tile) {
    constexpr int kHalves = is8(OP) ? 1 : 2;
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      Frag<OP> fw[TJ];
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        fw[j].w[0] = rw.read(tile + BM * kTileK, j, h);
        if constexpr (is8(OP)) fw[j].w[1] = rw.read(tile + BM * kTileK, j, 1);
      }
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        Frag<OP> f;
        f.w[0] = rx.read(tile, i, h);
        if constexpr (is8(OP)) f.w[1] = rx.read(tile, i, 1);
#pragma unroll
        for (int j = 0; j < TJ; ++j)
          acc[i][j] = mma<OP>(fw[j], f, acc[i][j], static_cast<int>(sw[kScales ? j : 0]),
                              static_cast<int>(sx[kScales ? i : 0]));
      }
    }
  };

  const uint32_t all = (a.kbytes + kTileK - 1) / kTileK;
  const uint32_t first = place.part * a.per_split;
  const uint32_t last = min(all, first + a.per_split);
  const uint32_t at0 = lds_address(&lds[0][0]), at1 = lds_address(&scales[0][0]);
  // DMA: past the last tile zeros are loaded, so that each tile is as many loads.
  const auto start = [&](uint32_t kt, uint32_t stage) {
    const uint32_t to = at0 + stage * kBuffer;
#pragma unroll
    for (int q = 0; q < OpX::Q; ++q) lx.start(kt, to, q);
#pragma unroll
    for (int q = 0; q < OpW::Q; ++q) lw.start(kt, to + BM * kTileK, q);
    // (a wait for the tile waits for these too: they are one load more, and before it)
    if constexpr (kScales && DMA)
      if ((kt % 4 == 0 || kt == first) && wave < kScaleRows / 64)
        load_to_lds<16>(kt < all ? so : kOutside, sr, kt / 4 * 16, at1 + kt / 4 % 2 * (kScaleRows * 16) + wave * 1024);
  };
  if constexpr (DMA) {
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) start(first + s, s);
    uint32_t stage = 0;
    for (uint32_t kt = first; kt < last; ++kt) {
      wait_tiles<(kStages - 2) * kLoads>();
      start(kt + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
      take_scales(kt);
      multiply(lds[stage]);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    wait_tiles<0>();  // nothing arrives in LDS any more
  } else {
    // the 8-bit 128 x 128 tile has registers for one tile on its way, not two,
    // and for one pass's block scales
    constexpr int kSets = is8(OP) && TI * TJ >= 16 ? 1 : 2;
    const auto load = [&](uint32_t kt, auto set) {
      constexpr int S = decltype(set)::value % kSets;
      if (kt < last) {
#pragma unroll
        for (int q = 0; q < OpX::Q; ++q) lx.template start<S>(kt, 0, q);
#pragma unroll
        for (int q = 0; q < OpW::Q; ++q) lw.template start<S>(kt, 0, q);
      }
    };
    const auto pass = [&](uint32_t kt, auto set) {
      constexpr int S = decltype(set)::value;
      lx.template put<S % kSets>(lds[S]);
      lw.template put<S % kSets>(lds[S] + BM * kTileK);
      take_scales(S);
      __syncthreads();
      load(kt + kSets, set);
      if (kSets == 2 && kt + 1 < last) read_scales(kt + 1);
      multiply(lds[S]);
      if (kSets == 1 && kt + 1 < last) read_scales(kt + 1);
    };
    typedef std::integral_constant<int, 0> Even;
    typedef std::integral_constant<int, 1> Odd;
    load(first, Even());
    if constexpr (kSets == 2) load(first + 1, Odd());
    read_scales(first);
    uint32_t kt = first;
    for (; kt + 1 < last; kt += 2) {
      pass(kt, Even());
      pass(kt + 1, Odd());
    }
    if (kt < last) pass(kt, Even());
  }
  end_tile<OP, BM, BN, WM, WN, kStages * static_cast<int>(kBuffer)>(a, place, &lds[0][0], acc);
}

// ---------------------------------------------------------------------------
// Large tiles of 8-bit values
//
// 256 x 256 outputs to a block of eight waves, 128 x 64 each, two waves to a
// SIMD. A wave's reads run ahead of its matrix instructions: its W rows and the
// first half of its x rows of a pass are in registers when the pass begins; the
// second half is read under the first half's instructions, and then, once the
// next tile has arrived in the other buffer and every wave has its values of
// this one, the next pass's W rows and first x rows are read under the second
// half's, while this buffer is loaded again, so each load has a whole pass to
// arrive. Reads and loads are spread between the instructions of one W row
// (sched_barrier): a run of other instructions leaves the matrix unit idle.
//
// e4m3 at 8192^3 and 8192 x 4096 x 7168: 2670 TFLOP/s with row scales (the library's 2436
// and 2675), with block scales 2270 and 2460; with a scale byte read for each row and
// pass instead of one word for four tiles 2060. 8-bit integers at 8192 x 4096 x 7168, with
// four waves of 128 x 128 each as below 200 us, so 194. With bf16 at 8192^3 (1373 TFLOP/s on the
// card of these figures): all loads at the start of the half 1140; reads not ahead of
// the pass 1280; without the raised priority of the matrix instructions 1346.
// ---------------------------------------------------------------------------

template <int OP, class E>
__global__ __launch_bounds__(512) void linear_large_kernel(TileArgs<E> a) {
  constexpr int BM = 256, BN = 256, WN = 4, kThreads = 512;
  constexpr int TI = 8, TJ = 4, HALF = TI / 2;
  constexpr int ELEM = 1;
  static_assert(!wide_tiles(OP), "these take linear_wide_kernel");
  constexpr uint32_t kBuffer = (BM + BN) * kTileK;
  constexpr bool kScales = OP == kOpMX;
  constexpr uint32_t kTurned = 8 * 64 + 16;  // words of a pass in `turned`; 16 more, so that four passes are in four banks
  __shared__ __align__(1024) uint8_t lds[2][kBuffer];
  __shared__ __align__(1024) uint8_t scales[kScales ? (BM + BN) * 16 : 16];
  __shared__ uint32_t turned[2][kScales ? 4 * kTurned : 1];
  constexpr int G = group_of<E>(TJ), W = E::kW;
  const Place place = place_of<BM, BN / E::kSums, E::kHalves>(a);
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const uint32_t lane = threadIdx.x % 64, g = lane / 16;
  const uint32_t wm = wave / WN, wn = wave % WN;

  typedef Operand<BM, kThreads, false, false, 1, true, ELEM> OpX;
  typedef Operand<BN, kThreads, false, true, G, true, ELEM, W> OpW;
  static_assert(OpX::Q == TJ && OpW::Q == TJ, "one round of loads for each W tile");
  OpX lx;
  OpW lw;
  lx.init(a.x, place.m0, a);
  lw.init(a.w, place.n0, a);
  Reader<OpX, false, false, 1> rx;
  Reader<OpW, false, true, G, W> rw;
  rx.init(wm * (TI * 16));
  rw.init(wn * (W == kBoth ? TJ * 8 : TJ * 16));

  // kMX: block scales come four passes at a time, 16 bytes of each row into
  // `scales`: the first four waves bring 64 rows of x each, the others of W. A
  // wave then turns its 64 rows: word [pass][wave][lane] of `turned` holds, for the
  // lane group's 32 values of the pass, the bytes of the lane's row in each of
  // four tiles, and the matrix instruction picks the byte of its tile.
  const uint32_t kblocks = a.kbytes / 32;
  uint32_t so = 0;
  i32x4 sr = {0, 0, 0, 0};
  if constexpr (kScales) {
    const bool of_x = wave < 4;
    static_assert(W == kBoth || G == 4, "the order of W's rows in turn_scales");
    const bool of_2 = W == kBoth && wave >= 6;  // two waves bring a weight's 128 rows
    const uint32_t r = threadIdx.x % (W == kBoth && !of_x ? 128 : 256), here = of_x ? lx.here : lw.here;
    sr = buffer_of(of_x ? a.xs + place.m0 * kblocks : (of_2 ? a.ws2 : a.ws) + place.n0 * kblocks,
                   static_cast<int64_t>(here) * kblocks);
    so = r < here ? r * kblocks : kOutside;
  }
  const uint32_t at0 = lds_address(&lds[0][0]), at1 = lds_address(&scales[0]);
  const auto start = [&](uint32_t kt, uint32_t b, int q) {
    lx.start(kt, at0 + b * kBuffer, q);
    lw.start(kt, at0 + b * kBuffer + BM * kTileK, q);
  };
  const auto start_scales = [&](uint32_t kt) {
    if constexpr (kScales) load_to_lds<16>(kt * 4 < kblocks ? so : kOutside, sr, kt * 4, at1 + wave * 1024);
  };
  // Lane (g, low) takes the words of pass g of its four rows.
  const auto turn_scales = [&](uint32_t b) {
    if constexpr (kScales) {
      const uint32_t low = lane % 16;
      uint32_t d[4], e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // the wave's rows: of W those of its wn, in the order of the tiles
        uint32_t row = wave * 64 + (wave < 4 ? i * 16 + low : (low / 4) * 16 + i * 4 + low % 4);
        if (W == kBoth && wave >= 4)
          row = 256 + (i / 2) * 128 + (wave - 4) * 32 + (low / 4) * 8 + (i % 2) * 4 + low % 4;
        d[i] = *reinterpret_cast<const uint32_t*>(&scales[row * 16 + g * 4]);
      }
      const uint32_t lo01 = __builtin_amdgcn_perm(d[1], d[0], 0x05010400), lo23 = __builtin_amdgcn_perm(d[3], d[2], 0x05010400);
      const uint32_t hi01 = __builtin_amdgcn_perm(d[1], d[0], 0x07030602), hi23 = __builtin_amdgcn_perm(d[3], d[2], 0x07030602);
      e[0] = __builtin_amdgcn_perm(lo23, lo01, 0x05040100);
      e[1] = __builtin_amdgcn_perm(lo23, lo01, 0x07060302);
      e[2] = __builtin_amdgcn_perm(hi23, hi01, 0x05040100);
      e[3] = __builtin_amdgcn_perm(hi23, hi01, 0x07060302);
#pragma unroll
      for (int i = 0; i < 4; ++i) turned[b][g * kTurned + wave * 64 + i * 16 + low] = e[i];
    }
  };
  // The scale bytes of a pass: of the W tiles and of each half of the x tiles.
  struct Scales {
    int w, x[2];
  };
  Scales now = {}, next = {};
  const auto read_scales = [&](uint32_t step, Scales& s) {
    if constexpr (kScales) {
      const uint32_t* p = &turned[step / 4 % 2][step % 4 * kTurned + lane];
      s.w = p[(4 + wn) * 64];
      s.x[0] = p[wm * 128];
      s.x[1] = p[wm * 128 + 64];
    }
  };

  struct Row {
    i32x4 w[2];  // both 16-byte pieces of a pass
  };
  Row w[TJ], xa[HALF], xb[HALF];
  const auto read_w = [&](uint32_t b, int j) {
#pragma unroll
    for (int h = 0; h < 2; ++h) w[j].w[h] = rw.read(lds[b] + BM * kTileK, j, h);
  };
  const auto read_x = [&](uint32_t b, int i, Row& r) {
#pragma unroll
    for (int h = 0; h < 2; ++h) r.w[h] = rx.read(lds[b], i, h);
  };

  f32x4 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  const auto multiply = [&](int half, int j, const Row (&x)[HALF]) {
#pragma unroll
    for (int i = 0; i < HALF; ++i) {
      f32x4& c = acc[half * HALF + i][j];
      const Frag<OP> p = {w[j].w[0], w[j].w[1]}, q = {x[i].w[0], x[i].w[1]};
      c = kScales ? mma_bytes<OP>(p, q, c, now.w, now.x[half], j, i) : mma<OP>(p, q, c, 0, 0);
    }
  };

  const uint32_t all = (a.kbytes + kTileK - 1) / kTileK;
  const uint32_t first = place.part * a.per_split;
  const uint32_t last = min(all, first + a.per_split);
#pragma unroll
  for (int q = 0; q < TJ; ++q) start(first, 0, q);
  start_scales(first);
  wait_tiles<0>();
  turn_scales(0);
#pragma unroll
  for (int q = 0; q < TJ; ++q) start(first + 1, 1, q);
#pragma unroll
  for (int j = 0; j < TJ; ++j) read_w(0, j);
#pragma unroll
  for (int i = 0; i < HALF; ++i) read_x(0, i, xa[i]);
  if constexpr (kScales) __syncthreads();  // every wave has turned its rows
  read_scales(0, now);
  for (uint32_t kt = first; kt < last; ++kt) {
    const uint32_t step = kt - first, b = step & 1;
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      if (j < HALF) read_x(b, HALF + j, xb[j]);
      __builtin_amdgcn_s_setprio(1);
      multiply(0, j, xa);
      __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_sched_barrier(0);
    }
    wait_tiles<0>();
    if (kScales && step % 4 == 1) start_scales(kt + 3);
    if (kScales && step % 4 == 2) turn_scales((step + 2) / 4 % 2);
    read_scales(step + 1, next);
    // past the last tile: zeros are loaded and old values read, and neither is used
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      start(kt + 2, b, j);
      __builtin_amdgcn_s_setprio(1);
      multiply(1, j, xb);
      __builtin_amdgcn_s_setprio(0);
      read_w(b ^ 1, j);
      if (j < HALF) read_x(b ^ 1, j, xa[j]);
      __builtin_amdgcn_sched_barrier(0);
    }
    now = next;
  }
  wait_tiles<0>();  // nothing arrives in LDS any more
  end_tile<OP, BM, BN, 2, WN, 2 * static_cast<int>(kBuffer)>(a, place, &lds[0][0], acc);
}

// ---------------------------------------------------------------------------
// Large tiles of 16-bit values
//
// The same tile by four waves, 128 x 128 each and one to a SIMD: two thirds of the
// reads from LDS, and results that never leave the accumulation registers. Nobody
// fills a wave's gaps, so there are none: each of the 128 matrix instructions of a
// pass (16 cycles) has at most one read, one load or one scalar step in front of it,
// held there by sched_barrier. The first half of a pass (k 0..31 of 64) reads the second
// half's values; its last instructions stand behind the barrier after which the
// other buffer has arrived and this one is free, and the second half reads the next
// pass's values there and loads this buffer again.
//
// A block to each compute unit goes through its tiles, and its loads and reads run on
// through their ends: a tile's results are worked on while the next one's first passes
// arrive, and leave through 32 KiB of LDS of their own. Blocks of one tile each had 16 us of
// it without a matrix instruction, as much as a sixth of K = 4096. An output's sums have
// the order that the eight-wave kernel gives them.
//
// 8192^3 in bf16 on one card: 1582 TFLOP/s, blocks of one tile 1502, eight waves 1476, the
// library 1616-1641; 4096 x 16384 x 4096 1465, 1400, 1377, 1605; 4096 x 4096 x 7168 1512, 1450,
// 1437, 1428. What is scalar between two passes in one place (the next pass's addresses) 5% of
// the loop; a load's three steps in a row 1.5%; left to the compiler's registers slower
// than eight waves. Matrix units are busy 85% of the loop, at 1.76 GHz: more of them,
// and the clock gives way.
// ---------------------------------------------------------------------------

template <int OP, bool TX, bool TW, class E>
__global__ __launch_bounds__(256, 1) void linear_wide_kernel(TileArgs<E> a) {
  constexpr int BM = 256, BN = 256, WN = 2, kThreads = 256;
  constexpr int TI = 8, TJ = 8;
  constexpr int ELEM = 2;
  constexpr uint32_t kBuffer = (BM + BN) * kTileK;
  constexpr int G = group_of<E>(TJ), W = E::kW;
  constexpr int kResults = E::kWrites ? 32768 : 0;  // a row of every wave's tiles
  __shared__ __align__(1024) uint8_t lds[2 * kBuffer + kResults];
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const uint32_t wm = wave / WN, wn = wave % WN;
  typedef Operand<BM, kThreads, TX, false, 1, true, ELEM> OpX;
  typedef Operand<BN, kThreads, TW, true, G, true, ELEM, W> OpW;
  static_assert(OpX::Q == 8 && OpW::Q == 8, "16 loads in a pass");
  Reader<OpX, TX, false, 1> rx;
  Reader<OpW, TW, true, G, W> rw;
  rx.init(wm * (TI * 16));
  rw.init(wn * (W == kBoth ? TJ * 8 : TJ * 16));
  const uint32_t tiles = a.tiles_m * a.tiles_n * a.splits;
  const uint32_t all = (a.kbytes + kTileK - 1) / kTileK;
  const auto last_of = [&](uint32_t first) { return min(all, first + a.per_split); };

  // The loads run two passes ahead, through the ends of tiles: `coming` is the tile
  // they are of, ahead its pass, end where its passes end. Behind the block's last tile zeros
  // are loaded, and used by no one.
  const uint32_t blocks = gridDim.x;
  uint32_t coming = blockIdx.x, ahead = all, end = all;
  OpX lx;
  OpW lw;
  const auto aim = [&] {
    const Place p = place_of<BM, BN / E::kSums, E::kHalves>(a, coming);
    if constexpr (E::kHalves) lx.init(a.x, p.m0 + (p.second ? a.xupper : 0), a.M - p.m0, a);
    else lx.init(a.x, p.m0, a);
    lw.init(a.w, p.n0, a);
    ahead = p.part * a.per_split;
    end = last_of(ahead);
  };
  // from the end of a tile's passes to the next tile's first; a part may have none
  const auto next = [&] {
    do {
      coming += blocks;
      if (coming < tiles) {
        aim();
      } else {
        ahead = all;
        end = 0xFFFFFFFFu;  // stays there
      }
    } while (ahead >= end);
  };
  aim();
  if (ahead >= end) next();

  // The values of both halves of a pass: x's tiles, then W's.
  i32x4 xf[2][TI], wf[2][TJ];
  const auto read = [&](uint32_t b, int h, int k) {
    if (k < TI) xf[h][k] = rx.read(lds + b * kBuffer, k, h);
    else wf[h][k - TI] = rw.read(lds + b * kBuffer + BM * kTileK, k - TI, h);
  };
  const uint32_t to_wave = __builtin_amdgcn_readfirstlane(lds_address(lds) + wave * 1024);
  const auto set = [&](uint32_t b, int k) { set_place(to_wave + b * kBuffer + k * (kThreads * 16)); };
  const auto load = [&](const typename OpX::Pass& px, const typename OpW::Pass& pw, int k) {
    if (k < 8) lx.load(px, k);
    else lw.load(pw, k - 8);
  };
  // the block's first loads, whose addresses are only just made
  const auto load_all = [&](uint32_t b) {
    const auto px = lx.pass(ahead);
    const auto pw = lw.pass(ahead);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      set(b, k);
      if (k < 8) lx.template load<true>(px, k);
      else lw.template load<true>(pw, k - 8);
    }
  };
  load_all(0);
  if (++ahead >= end) next();
  wait_tiles<0>();
  load_all(1);
#pragma unroll
  for (int k = 0; k < 16; ++k) read(0, 0, k);
  uint32_t b = 0;
  for (uint32_t id = blockIdx.x; id < tiles; id += blocks) {
    const Place place = place_of<BM, BN / E::kSums, E::kHalves>(a, id);
    f32x4 acc[TI][TJ];
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    acc_ready(acc);
    const uint32_t first = place.part * a.per_split, last = last_of(first);
    for (uint32_t kt = first; kt < last; ++kt, b ^= 1) {
      const auto multiply = [&](int h, int k) {
        mma_in_place<OP>(acc[k % 8][k / 8], wf[h][k / 8], xf[h][k % 8]);
        __builtin_amdgcn_sched_barrier(0);
      };
#pragma unroll
      for (int k = 0; k < 36; ++k) {
        if (k % 2 == 0 && k < 32) read(b, 1, k / 2);
        multiply(0, k);
      }
      if (++ahead >= end) next();
      const auto px = lx.pass(ahead);
      const auto pw = lw.pass(ahead);
#pragma unroll
      for (int k = 36; k < 64; ++k) {
        if (k == 56) wait_tiles<0>();
        multiply(0, k);
      }
#pragma unroll
      for (int k = 0; k < 64; ++k) {
        if (k % 4 == 0) read(b ^ 1, 0, k / 4);
        if (k % 4 == 1) set(b, k / 4);
        if (k % 4 == 2) load(px, pw, k / 4);
        multiply(1, k);
      }
    }
    acc_ready(acc);
    end_tile<OP, BM, BN, 2, WN, kResults, true>(a, place, lds + 2 * kBuffer, acc);
  }
  wait_tiles<0>();  // nothing arrives in LDS any more
}

// The parts of a split sum, added in ascending order, and the epilogue. One wave
// to a block and AHEAD parts' loads in flight, past the last part the last one's
// again: a load in a branch of its own waits for the one before it. 2048 x 24 in 16
// parts 6.3 us, four waves and a part at a time 9.9. WIDE: rows of at least 8
// columns, whose short last chunk comes from the 8 values that end there, shifted
// once they are summed (129 x 1279 in four parts 13 -> 4.4 us: element by element
// it holds up its wave for every part).
constexpr int kJoinThreads = 64;

template <int OP, class E, uint32_t AHEAD, bool WIDE>
__global__ __launch_bounds__(kJoinThreads) void linear_join_kernel(const float* __restrict__ partial,
                                                                   uint32_t splits, int64_t M, int64_t N, E e) {
  constexpr int kSums = E::kSums;
  const int64_t chunks = (N + 7) / 8, all = M * chunks;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kJoinThreads;
  const int64_t part = kSums * M * N;
  for (int64_t id = static_cast<int64_t>(blockIdx.x) * kJoinThreads + threadIdx.x; id < all; id += step) {
    // a division of 64 bits takes as long as a part's load
    const int64_t m = all <= 0xFFFFFFFFLL ? static_cast<uint32_t>(id) / static_cast<uint32_t>(chunks) : id / chunks;
    const int64_t n = (id - m * chunks) * 8;
    const int count = static_cast<int>(min(N - n, static_cast<int64_t>(8)));
    const int back = WIDE ? 8 - count : 0;
    const float* const p = partial + m * N + n - back;
    f32x8 t[kSums];
#pragma unroll
    for (int sum = 0; sum < kSums; ++sum) t[sum] = f32x8{0, 0, 0, 0, 0, 0, 0, 0};
    for (uint32_t s0 = 0; s0 < splits; s0 += AHEAD) {
      f32x8 b[AHEAD][kSums];
#pragma unroll
      for (uint32_t k = 0; k < AHEAD; ++k)
#pragma unroll
        for (int sum = 0; sum < kSums; ++sum) {
          const float* const q = p + min(s0 + k, splits - 1) * part + sum * M * N;
          if constexpr (WIDE) {
            b[k][sum] = *reinterpret_cast<const f32x8_at4*>(q);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) b[k][sum][i] = q[min(i, count - 1)];
          }
        }
#pragma unroll
      for (uint32_t k = 0; k < AHEAD; ++k)
        if (s0 + k < splits) {
#pragma unroll
          for (int sum = 0; sum < kSums; ++sum) t[sum] = s0 + k == 0 ? b[k][sum] : sums_added<OP>(t[sum], b[k][sum]);
        }
    }
    float v[8 * kSums];
#pragma unroll
    for (int sum = 0; sum < kSums; ++sum) {
      f32x8 u = t[sum];
      if constexpr (WIDE) {
        u = (back & 4) != 0 ? __builtin_shufflevector(u, u, 4, 5, 6, 7, 4, 5, 6, 7) : u;
        u = (back & 2) != 0 ? __builtin_shufflevector(u, u, 2, 3, 4, 5, 6, 7, 6, 7) : u;
        u = (back & 1) != 0 ? __builtin_shufflevector(u, u, 1, 2, 3, 4, 5, 6, 7, 7) : u;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[8 * sum + i] = u[i];
    }
    e.template with<OP>([&](const auto& finish) { finish(m, n, count, v); });
  }
}

// ---------------------------------------------------------------------------
// Up to 16 rows of x
//
// Bound by W's bytes: each is read once, straight into registers. A block
// takes up to 16 rows of W; its waves share the sum in units of kTileK bytes of
// each row, four units' loads of a wave in flight, multiply them with x's rows
// as the second operand, and are joined through LDS in ascending order.
//
// Blocks take as many rows of W as leaves every CU as many blocks as any
// other: 16 x 24 x 28672 in bf16 50.4 -> 32.9 us, 1 x 1024 x 4096 6.8 -> 5.3, 1 x 7168 x 7168
// 21.0 -> 19.9 us (5.1 TB/s) against 16 rows always. 1 x 4096 x 7168: 12.7 us (4.6 TB/s);
// 4 or 16 waves 14.8 and 13.3, 32 rows of W to a block 17.8. Lanes without a row of x or
// W load nothing: reading the last row again instead 15.3. Block scales, 16 x 7168 x 4096:
// 11.6 us, one byte a load 13.7.
// ---------------------------------------------------------------------------

template <class E>
struct RowsArgs {
  const uint8_t* x;
  const uint8_t* w;
  const uint8_t* w2;   // kBoth
  const uint8_t* xs;   // kMX
  const uint8_t* ws;   // kMX
  const uint8_t* ws2;  // kMX of kBoth
  int64_t M, N;
  uint32_t kbytes;  // of a row that count, which alone set the order of its sum
  uint32_t ld;      // from row to row, the same in x and W
  uint32_t wide;  // rows of a weight for each block: at most 16, of kBoth 8
  E e;
};

// The lane's values of the unit at byte k of a row; those past kbytes are zeros.
template <int OP, bool FULL>
__device__ __forceinline__ void load_unit(const uint8_t* row, uint32_t k, uint32_t kbytes,
                                          uint32_t g, Frag<OP> (&f)[is8(OP) ? 1 : 2]) {
  constexpr int ELEM = is8(OP) ? 1 : 2;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    // piece p of the unit: the lane group's 16 bytes
    const uint32_t at = k + p * 64 + g * 16;
    i32x4 v = {0, 0, 0, 0};
    if (FULL || at + 16 <= kbytes) {
      v = piece_at<ELEM>(row + at);
    } else if (at < kbytes) {
      v = short_piece<ELEM>(row + at, kbytes - at, at > 0);
    }
    if constexpr (is8(OP)) f[0].w[p] = v;
    else f[p].w[0] = v;
  }
}

template <int OP, int WAVES, class E>
__global__ __launch_bounds__(64 * WAVES) void linear_rows_kernel(RowsArgs<E> a) {
  constexpr int kFrags = is8(OP) ? 1 : 2;
  constexpr int kOf = 16 / E::kSums;  // places for rows of one weight
  __shared__ float sums[WAVES][16][17];
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const uint32_t lane = threadIdx.x % 64, low = lane % 16, g = lane / 16;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * a.wide;
  const bool in_w = low % kOf < a.wide, in_x = low < a.M, of_2 = E::kW == kBoth && low >= kOf;
  const int64_t wrow = min(n0 + (in_w ? low % kOf : 0), a.N - 1);
  const uint32_t xrow = in_x ? low : 0;
  const uint32_t kblocks = (a.kbytes + 31) / 32;
  const uint8_t* w = (of_2 ? a.w2 : a.w) + wrow * a.ld;
  const uint8_t* x = a.x + static_cast<int64_t>(xrow) * a.ld;
  const uint8_t* ws = OP == kOpMX ? (of_2 ? a.ws2 : a.ws) + wrow * kblocks : nullptr;
  const uint8_t* xs = OP == kOpMX ? a.xs + static_cast<int64_t>(xrow) * kblocks : nullptr;
  f32x4 acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};

  const uint32_t full = a.kbytes / kTileK, units = (a.kbytes + kTileK - 1) / kTileK;
  // The waves take turns, unit by unit; with block scales each takes a run of
  // units, so that the scales of four come in one load (byte 4 k + g of 16).
  constexpr bool kRun = OP == kOpMX;
  constexpr uint32_t kStride = kRun ? 1 : WAVES;
  const uint32_t each = (full + WAVES - 1) / WAVES;
  uint32_t u = kRun ? min(full, wave * each) : wave;
  const uint32_t end = kRun ? min(full, u + each) : full;
  const auto some = [&](auto ahead) {
    constexpr int kAhead = decltype(ahead)::value;
    typedef uint32_t Bytes __attribute__((ext_vector_type(kAhead)));
    typedef Bytes Bytes_at1 __attribute__((aligned(1)));
    for (; u + (kAhead - 1) * kStride < end; u += kAhead * kStride) {
      Frag<OP> fw[kAhead][kFrags], fx[kAhead][kFrags];
      Bytes sw = {}, sx = {};
      if constexpr (OP == kOpMX) {
        if (in_w) sw = *reinterpret_cast<const Bytes_at1*>(ws + u * 4);
        if (in_x) sx = *reinterpret_cast<const Bytes_at1*>(xs + u * 4);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const uint32_t at = (u + k * kStride) * kTileK;
        if (in_w) load_unit<OP, true>(w, at, a.kbytes, g, fw[k]);
        else fw[k][0] = fw[k][kFrags - 1] = {};
        if (in_x) load_unit<OP, true>(x, at, a.kbytes, g, fx[k]);
        else fx[k][0] = fx[k][kFrags - 1] = {};
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const uint32_t bw = sw[k], bx = sx[k];
#pragma unroll
        for (int p = 0; p < kFrags; ++p)
          acc[(k + p) % 2] = mma<OP>(fw[k][p], fx[k][p], acc[(k + p) % 2],
                                     static_cast<int>(bw >> (8 * g)), static_cast<int>(bx >> (8 * g)));
      }
    }
  };
  some(std::integral_constant<int, 4>());
  some(std::integral_constant<int, 2>());
  some(std::integral_constant<int, 1>());
  if (full < units && wave == WAVES - 1) {
    Frag<OP> fw[kFrags], fx[kFrags];
    load_unit<OP, false>(w, full * kTileK, a.kbytes, g, fw);
    load_unit<OP, false>(x, full * kTileK, a.kbytes, g, fx);
    int sw = 0, sx = 0;
    if (OP == kOpMX && full * 4 + g < kblocks) {
      sw = ws[full * 4 + g];
      sx = xs[full * 4 + g];
    }
#pragma unroll
    for (int p = 0; p < kFrags; ++p) acc[p % 2] = mma<OP>(fw[p], fx[p], acc[p % 2], sw, sx);
  }
  // sums[wave][row of x][column]
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float s0 = acc[0][i], s1 = acc[1][i];
    sums[wave][low][g * 4 + i] = sum_add<OP>(s0, s1);
  }
  __syncthreads();
  // a thread takes 8 columns of a row (of kBoth, of either sum)
  constexpr int kTakes = 2 / E::kSums;
  const int64_t m = threadIdx.x / kTakes;
  const uint32_t half = threadIdx.x % kTakes;
  const int64_t n = n0 + half * 8;
  if (threadIdx.x < 16 * kTakes && m < a.M && n < a.N && half * 8 < a.wide) {
    float v[8 * E::kSums];
#pragma unroll
    for (int i = 0; i < 8 * E::kSums; ++i) {
      v[i] = sums[0][m][half * 8 + i];
#pragma unroll
      for (int k = 1; k < WAVES; ++k) v[i] = sum_add<OP>(v[i], sums[k][m][half * 8 + i]);
    }
    const int count = static_cast<int>(min(min(a.N - n, static_cast<int64_t>(8)), static_cast<int64_t>(a.wide - half * 8)));
    a.e.template with<OP>([&](const auto& finish) { finish(m, n, count, v); });
  }
}

// Epilogue of the products that are rounded and stored as they are: of one W
// (kOne) or two (kChain), or of two products in one launch (HALVES), whose results
// go to `out` and, from row M on, to `out2`.
template <int W, bool HALVES>
struct StoreEpilogue {
  static constexpr int kW = W, kSums = 1, kGroup = 0;
  static constexpr bool kSplits = true, kHalves = HALVES, kTakes = false, kWrites = true, kEarly = false;
  void* out;
  void* out2;
  int64_t M, N;

  template <int OP, class Fn>
  __device__ __forceinline__ void with(const Fn& fn) const {
    constexpr int F = out_format(OP);
    typedef typename Store<F>::type S;
    fn([&](int64_t m, int64_t n, int count, float(&v)[8]) {
      const bool second = HALVES && m >= M;
      S* const to = static_cast<S*>(second ? out2 : out);
      Chunk<F> c;
      narrow_chunk<F>(v, c);
      store_chunk<F>(to + (second ? m - M : m) * N + n, count, c);
    });
  }
};

// out[n] = the parts' sum, rounded once (+0.0 of none): 64 columns to a block,
// each of four waves every fourth part, joined in ascending order.
template <int F>
__device__ __forceinline__ void sum_parts(const float* __restrict__ partial,
                                          typename Store<F>::type* __restrict__ out, int64_t parts, int64_t N) {
  __shared__ float sums[4][64];
  const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  float s = 0.0f;
  if (n < N) {
#pragma unroll 8
    for (int64_t k = wave; k < parts; k += 4) s = s + partial[k * N + n];
  }
  sums[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && n < N)
    out[n] = narrow<F>(((sums[0][lane] + sums[1][lane]) + sums[2][lane]) + sums[3][lane]);
}

template <int F>
__global__ __launch_bounds__(256) void linear_bias_kernel(const float* __restrict__ partial,
                                                          typename Store<F>::type* __restrict__ out,
                                                          int64_t parts, int64_t N) {
  sum_parts<F>(partial, out, parts, N);
}

__global__ __launch_bounds__(256) void linear_zero_kernel(uint16_t* __restrict__ p, int64_t count) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < count; i += step)
    p[i] = 0;
}

}  // namespace
