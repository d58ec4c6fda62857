// mhc_linear.hip - matrix product with bias, activation and residual in its
// epilogue, and its backward, for gfx950 (see include/mhc_linear.h for the
// operation).

#include "mhc_linear.h"

#include <math.h>

#include <type_traits>

#include "mhc_host.h"
#include "mhc_launch.h"
#include "mhc_rows.h"

#ifdef __FAST_MATH__
#error "this source must not be built with fast-math"
#endif

#pragma clang fp contract(off)

namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// What the operands of a product are. kE4M3 has its scales applied in the
// epilogue, kMX in the matrix instruction.
constexpr int kOpBF16 = MHC_LINEAR_BF16;
constexpr int kOpF16 = MHC_LINEAR_F16;
constexpr int kOpE4M3 = MHC_LINEAR_E4M3_ROW;
constexpr int kOpMX = MHC_LINEAR_E4M3_MX;

constexpr bool is8(int op) { return op == kOpE4M3 || op == kOpMX; }
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

struct Epilogue {
  const void* bias;
  const void* residual;
  void* out;
  void* z;
  const float* x_scales;       // kE4M3 only
  const float* weight_scales;  // kE4M3 only
  int64_t N;                   // row stride of residual, out and z
  int32_t act;
};

// Columns [n, n + count) of row m, count <= 8, from the sums over k.
template <int OP, int ACT>
__device__ __forceinline__ void finish(const Epilogue& e, int64_t m, int64_t n, int count,
                                       float (&v)[8]) {
  constexpr int F = out_format(OP);
  typedef typename Store<F>::type S;
  float b[8];
  if constexpr (OP == kOpE4M3) {
    const float xs = e.x_scales[m];
    widen_chunk<kF32>(load_chunk<kF32>(e.weight_scales + n, count), b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * (xs * b[i]);
  }
  if (e.bias != nullptr) {
    widen_chunk<F>(load_chunk<F>(static_cast<const S*>(e.bias) + n, count), b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] + b[i];
  }
  Chunk<F> c;
  if (e.z != nullptr) {
    narrow_chunk<F>(v, c);
    store_chunk<F>(static_cast<S*>(e.z) + m * e.N + n, count, c);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = activate<ACT>(v[i]);
  if (e.residual != nullptr) {
    widen_chunk<F>(load_chunk<F>(static_cast<const S*>(e.residual) + m * e.N + n, count), b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] + b[i];
  }
  narrow_chunk<F>(v, c);
  store_chunk<F>(static_cast<S*>(e.out) + m * e.N + n, count, c);
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
  } else {
    const i32x8 x = __builtin_shufflevector(a0, a.w[1], 0, 1, 2, 3, 4, 5, 6, 7);
    const i32x8 y = __builtin_shufflevector(b0, b.w[1], 0, 1, 2, 3, 4, 5, 6, 7);
    // 0x7F is the scale 1
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
        x, y, acc, 0, 0, BYTE_A, OP == kOpMX ? sa : 0x7F, BYTE_B, OP == kOpMX ? sb : 0x7F);
  }
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

struct TileArgs {
  Matrix x, w;
  const uint8_t* xs;  // kMX
  const uint8_t* ws;  // kMX
  int64_t M, N;
  uint32_t kbytes;    // bytes of k that count, in rows that run along it
  uint32_t kturned;   // and in operands where k runs down (no more than kbytes: rows may be padded)
  uint32_t tiles_m, tiles_n;
  uint32_t splits, per_split;  // parts of the sum, and tiles of kTileK in each
  float* partial;              // [splits][M][N] where splits > 1
  Epilogue e;
};

// Offset that lies past every buffer: such a lane loads zeros.
constexpr uint32_t kOutside = 0x80000000u;

template <int V>
constexpr int log2_of() {
  return V <= 1 ? 0 : 1 + log2_of<V / 2>();
}

// How many consecutive tiles of 16 columns a lane's results run through.
constexpr int group_of(int tj) { return tj < 4 ? tj : 4; }

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void*)p));
}

// Starts a load of BYTES for each lane from `offset` + `at` of the buffer to the
// wave's consecutive places in LDS from `to` on; a lane past the buffer's end
// brings zeros (the check counts `at` too). No vector register is written; the
// loads are waited for by wait_tiles(). m0 is a reserved register, which a list
// of clobbers cannot name: nothing else in this library may use it (a test
// reads the machine code for that).
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
template <int SPAN, int THREADS, bool TURNED, bool IS_W, int G, bool DMA, int ELEM>
struct Operand {
  static constexpr int Q = SPAN * 8 / THREADS;   // pieces a thread brings of one tile
  static constexpr int P = TURNED ? SPAN / 8 : 8;  // pieces of a row of the tile
  static constexpr int kRowBytes = P * 16;
  static constexpr uint32_t kEach = THREADS / P;   // rows that one round of the threads covers
  static_assert(SPAN * 8 % THREADS == 0 && kEach % (TURNED ? 4 : 32) == 0, "swap() is the same in every round");
  const uint8_t* base;
  i32x4 rsrc;
  uint32_t offset;  // of this thread's first piece
  uint32_t row, piece;
  uint32_t ld;
  uint32_t here;    // rows (columns) that exist
  uint32_t kbytes;  // bytes of k that exist
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

  __device__ __forceinline__ void init(const Matrix& m, int64_t first, const TileArgs& a) {
    const int64_t left = m.count - first;
    kbytes = TURNED ? a.kturned : a.kbytes;
    here = static_cast<uint32_t>(left < SPAN ? left : SPAN);
    ld = static_cast<uint32_t>(m.ld);
    inside = first > 0;
    base = static_cast<const uint8_t*>(m.p) + (TURNED ? first * ELEM : first * m.ld);
    rsrc = buffer_of(base, TURNED ? kbytes / ELEM * m.ld - first * ELEM : here * m.ld);
    row = threadIdx.x / P;
    piece = ((threadIdx.x % P) ^ swap(row)) * 16;
    offset = row * ld + piece;
  }

  // Starts the loads of round q of the tile kt into `to`, the tile's place in LDS.
  template <int SET = 0>
  __device__ __forceinline__ void start(uint32_t kt, uint32_t to, int q) {
    const uint32_t rows = q * kEach;
    if constexpr (DMA) {
      const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
      const uint32_t dst = to + (q * THREADS + wave * 64) * 16;
      // a tile's last rows end inside it where k runs along them; where k runs
      // down, what is past the end is past the buffer's end
      if constexpr (TURNED)
        load_to_lds<16>(offset, rsrc, (kt * (kTileK / ELEM) + rows) * ld, dst);
      else
        load_to_lds<16>(kt * kTileK + piece < kbytes ? offset : kOutside, rsrc,
                        kt * kTileK + rows * ld, dst);
    } else {
      held[SET][q] = i32x4{0, 0, 0, 0};
      uint32_t left;  // bytes of the piece that exist
      const uint8_t* p = base;
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
        held[SET][q] = short_piece<ELEM>(p, left, TURNED ? piece > 0 || inside : p - base >= 16);
    }
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
template <typename O, bool TURNED, bool IS_W, int G>
struct Reader {
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
    return first + (IS_W ? (t / G) * (16 * G) + (low / 4) * (4 * G) + (t % G) * 4 + low % 4
                         : t * 16 + low);
  }

  // Piece h of tile t: 16 bytes along k, the pass's half h.
  __device__ __forceinline__ i32x4 read(const uint8_t* tile, int t, int h) const {
    if constexpr (!TURNED) {
      const uint32_t row = IS_W ? (t / G) * (16 * G) + (t % G) * 4 : t * 16;
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
};

template <int BM, int BN>
__device__ __forceinline__ Place place_of(const TileArgs& a) {
  // Quotients are made in vector registers; what is the same in every lane is
  // taken back to scalar ones, or all that follows from it would stay there.
  const uint32_t tiles = a.tiles_m * a.tiles_n;
  uint32_t id = blockIdx.x;
  const uint32_t part = __builtin_amdgcn_readfirstlane(id / tiles);
  id -= part * tiles;
  const uint32_t each = tiles / 8, more = tiles % 8, xcd = id % 8, k = id / 8;
  id = xcd * each + (xcd < more ? xcd : more) + k;
  const uint32_t band = __builtin_amdgcn_readfirstlane(id / (4 * a.tiles_n));
  const uint32_t high = min(4u, a.tiles_m - 4 * band);
  id -= band * 4 * a.tiles_n;
  const uint32_t column = __builtin_amdgcn_readfirstlane(id / high);
  return {static_cast<int64_t>(4 * band + id - column * high) * BM,
          static_cast<int64_t>(column) * BN, part};
}

// The tile's results, written. Lane l of wave (wm, wn) holds in acc[i][j] four
// consecutive columns of row 16 i + l % 16 of the wave's part; over the G tiles
// of a group they are 4 G consecutive ones. LDS: SIZE bytes.
template <int OP, int BM, int BN, int WM, int WN, int SIZE>
__device__ __forceinline__ void write_tile(const TileArgs& a, const Place& at, uint8_t* lds,
                                           f32x4 (&acc)[BM / WM / 16][BN / WN / 16]) {
  constexpr int TI = BM / WM / 16, TJ = BN / WN / 16;
  constexpr int G = group_of(TJ);
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const uint32_t lane = threadIdx.x % 64, low = lane % 16, g = lane / 16;
  const uint32_t wm = wave / WN, wn = wave % WN;
  // A wave's results go through its own part of LDS, from where its lanes take
  // 8 consecutive columns each of whole rows: one loop for every activation
  // instead of TI * TJ / 2 copies (3% of a 256 x 256 tile's time at K = 4096).
  constexpr int kWide = TJ * 16;
  constexpr int kHalves = BM * BN * 4 > SIZE ? 2 : 1;
  constexpr int kRows = TI * 16 / kHalves;
  static_assert(TI % kHalves == 0 && BM * BN * 4 / kHalves <= SIZE, "the results fit");
  __syncthreads();  // every wave is done with the tiles
  float* mine = reinterpret_cast<float*>(lds) + wave * (kRows * kWide);
  const bool whole = at.m0 + BM <= a.M && at.n0 + BN <= a.N;
#pragma unroll
  for (int half = 0; half < kHalves; ++half) {
#pragma unroll
    for (int i = 0; i < TI / kHalves; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j)
        *reinterpret_cast<f32x4*>(mine + (16 * i + low) * kWide + (j / G) * (16 * G) +
                                  g * (4 * G) + (j % G) * 4) = acc[half * (TI / kHalves) + i][j];
    wave_sync();
    const int64_t m0 = at.m0 + wm * (TI * 16) + half * kRows;
    const int64_t n0 = at.n0 + wn * kWide;
    const auto each = [&](const auto& sink) {
#pragma unroll 2
      for (uint32_t id = lane; id < kRows * kWide / 8; id += 64) {
        const uint32_t row = id / (kWide / 8), col = id % (kWide / 8) * 8;
        const int64_t m = m0 + row, n = n0 + col;
        if (whole || (m < a.M && n < a.N)) {
          const f32x4 p = *reinterpret_cast<const f32x4*>(mine + row * kWide + col);
          const f32x4 q = *reinterpret_cast<const f32x4*>(mine + row * kWide + col + 4);
          float v[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] = p[e];
            v[4 + e] = q[e];
          }
          sink(m, n, whole ? 8 : static_cast<int>(min(a.N - n, static_cast<int64_t>(8))), v);
        }
      }
    };
    if (a.splits > 1) {
      float* partial = a.partial + static_cast<int64_t>(at.part) * a.M * a.N;
      each([&](int64_t m, int64_t n, int count, float(&v)[8]) {
        Chunk<kF32> c;
        narrow_chunk<kF32>(v, c);
        store_chunk<kF32>(partial + m * a.N + n, count, c);
      });
    } else {
      with_act(a.e.act, [&](auto act) {
        each([&](int64_t m, int64_t n, int count, float(&v)[8]) {
          finish<OP, decltype(act)::value>(a.e, m, n, count, v);
        });
      });
    }
    wave_sync();
  }
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

template <int OP, int BM, int BN, int WM, int WN, int STAGES, bool DMA, bool TX, bool TW>
__global__ __launch_bounds__(64 * WM * WN, 2) void linear_tile_kernel(TileArgs a) {
  constexpr int kThreads = 64 * WM * WN;
  constexpr int TI = BM / WM / 16, TJ = BN / WN / 16;
  constexpr int G = group_of(TJ);
  constexpr int ELEM = is8(OP) ? 1 : 2;
  constexpr int kStages = DMA ? STAGES : 2;
  constexpr uint32_t kBuffer = (BM + BN) * kTileK;
  constexpr bool kScales = OP == kOpMX;
  typedef Operand<BM, kThreads, TX, false, 1, DMA, ELEM> OpX;
  typedef Operand<BN, kThreads, TW, true, G, DMA, ELEM> OpW;
  constexpr int kLoads = OpX::Q + OpW::Q + (kScales ? 1 : 0);  // of a wave, for a tile
  static_assert(!kScales || BM + BN <= kThreads, "a scale load for each row");
  __shared__ __align__(1024) uint8_t lds[kStages][kBuffer];
  __shared__ __align__(1024) uint8_t scales[kStages][kScales && DMA ? kThreads * 4 : 16];

  const Place place = place_of<BM, BN>(a);
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const uint32_t lane = threadIdx.x % 64, g = lane / 16;
  const uint32_t wm = wave / WN, wn = wave % WN;
  OpX lx;
  OpW lw;
  lx.init(a.x, place.m0, a);
  lw.init(a.w, place.n0, a);
  Reader<OpX, TX, false, 1> rx;
  Reader<OpW, TW, true, G> rw;
  rx.init(wm * (TI * 16));
  rw.init(wn * (TJ * 16));

  // Block scales. DMA: thread r brings the 4 bytes of row r, x's then W's.
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
  sx[0] = sw[0] = 0;
  if constexpr (kScales && DMA) {
    const bool of_x = wave < BM / 64;
    const uint32_t r = threadIdx.x - (of_x ? 0 : BM);
    sr = buffer_of(of_x ? xs : ws, static_cast<int64_t>(of_x ? lx.here : lw.here) * kblocks);
    if (r < (of_x ? lx.here : lw.here)) so = r * kblocks;
  } else if constexpr (kScales) {
#pragma unroll
    for (int i = 0; i < TI; ++i) ox[i] = min(rx.row_of(wm * (TI * 16), i), lx.here - 1) * kblocks + g;
#pragma unroll
    for (int j = 0; j < TJ; ++j) ow[j] = min(rw.row_of(wn * (TJ * 16), j), lw.here - 1) * kblocks + g;
  }
  const auto read_scales = [&](uint32_t kt) {
    if constexpr (kScales && !DMA) {
      const bool in = kt * 4 + g < kblocks;
#pragma unroll
      for (int i = 0; i < TI; ++i) nx[i] = in ? xs[ox[i] + kt * 4] : 0;
#pragma unroll
      for (int j = 0; j < TJ; ++j) nw[j] = in ? ws[ow[j] + kt * 4] : 0;
    }
  };
  const auto take_scales = [&](uint32_t stage) {
    if constexpr (kScales && DMA) {
#pragma unroll
      for (int i = 0; i < TI; ++i) sx[i] = scales[stage][rx.row_of(wm * (TI * 16), i) * 4 + g];
#pragma unroll
      for (int j = 0; j < TJ; ++j) sw[j] = scales[stage][(BM + rw.row_of(wn * (TJ * 16), j)) * 4 + g];
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
    if constexpr (kScales && DMA)
      load_to_lds<4>(kt < all ? so : kOutside, sr, kt * 4, at1 + stage * (kThreads * 4) + wave * 256);
  };
  if constexpr (DMA) {
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) start(first + s, s);
    uint32_t stage = 0;
    for (uint32_t kt = first; kt < last; ++kt) {
      wait_tiles<(kStages - 2) * kLoads>();
      start(kt + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
      take_scales(stage);
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
  write_tile<OP, BM, BN, WM, WN, kStages * static_cast<int>(kBuffer)>(a, place, &lds[0][0], acc);
}

// ---------------------------------------------------------------------------
// Large tiles
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
// 8192^3 in bf16 (1373 TFLOP/s; the library's product 1430-1465): four waves of 128 x 128, one to a SIMD,
// 1230 (nobody fills a wave's gaps); all loads at the start of the half 1140;
// reads not ahead of the pass 1280; without the raised priority of the
// matrix instructions 1346. Matrix units are busy 57-63% of the cycles, at a clock that the
// load itself brings down to 1.7 GHz (bf16) and 1.95 GHz (e4m3). e4m3 at 8192^3 and 8192 x
// 4096 x 7168: 2670 TFLOP/s with row scales (the library's 2436 and 2675), with block
// scales 2270 and 2460; with a scale byte read for each row and pass instead of
// one word for four tiles 2060.

// ---------------------------------------------------------------------------

template <int OP, bool TX, bool TW>
__global__ __launch_bounds__(512) void linear_large_kernel(TileArgs a) {
  constexpr int BM = 256, BN = 256, WN = 4, kThreads = 512;
  constexpr int TI = 8, TJ = 4, HALF = TI / 2;
  constexpr int kPieces = is8(OP) ? 1 : 2;  // matrix instructions for one result in a pass
  constexpr int ELEM = is8(OP) ? 1 : 2;
  constexpr uint32_t kBuffer = (BM + BN) * kTileK;
  constexpr bool kScales = OP == kOpMX;
  constexpr uint32_t kTurned = 8 * 64 + 16;  // words of a pass in `turned`; 16 more, so that four passes are in four banks
  __shared__ __align__(1024) uint8_t lds[2][kBuffer];
  __shared__ __align__(1024) uint8_t scales[kScales ? (BM + BN) * 16 : 16];
  __shared__ uint32_t turned[2][kScales ? 4 * kTurned : 1];
  const Place place = place_of<BM, BN>(a);
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const uint32_t lane = threadIdx.x % 64, g = lane / 16;
  const uint32_t wm = wave / WN, wn = wave % WN;

  typedef Operand<BM, kThreads, TX, false, 1, true, ELEM> OpX;
  typedef Operand<BN, kThreads, TW, true, 4, true, ELEM> OpW;
  static_assert(OpX::Q == TJ && OpW::Q == TJ, "one round of loads for each W tile");
  OpX lx;
  OpW lw;
  lx.init(a.x, place.m0, a);
  lw.init(a.w, place.n0, a);
  Reader<OpX, TX, false, 1> rx;
  Reader<OpW, TW, true, 4> rw;
  rx.init(wm * (TI * 16));
  rw.init(wn * (TJ * 16));

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
    const uint32_t r = threadIdx.x % 256, here = of_x ? lx.here : lw.here;
    sr = buffer_of(of_x ? a.xs + place.m0 * kblocks : a.ws + place.n0 * kblocks,
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
        const uint32_t row = wave < 4 ? i * 16 + low : (low / 4) * 16 + i * 4 + low % 4;
        d[i] = *reinterpret_cast<const uint32_t*>(&scales[(wave * 64 + row) * 16 + g * 4]);
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
    for (int h = 0; h < kPieces; ++h)
#pragma unroll
      for (int i = 0; i < HALF; ++i) {
        f32x4& c = acc[half * HALF + i][j];
        if constexpr (is8(OP)) {
          const Frag<OP> p = {w[j].w[0], w[j].w[1]}, q = {x[i].w[0], x[i].w[1]};
          c = kScales ? mma_bytes<OP>(p, q, c, now.w, now.x[half], j, i) : mma<OP>(p, q, c, 0, 0);
        } else {
          const Frag<OP> p = {w[j].w[h]}, q = {x[i].w[h]};
          c = mma<OP>(p, q, c, 0, 0);
        }
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
  write_tile<OP, BM, BN, 2, WN, 2 * static_cast<int>(kBuffer)>(a, place, &lds[0][0], acc);
}

// The parts of a split sum, added in ascending order, and the epilogue. One wave
// to a block and eight parts' loads in flight: 2048 x 24 in 16 parts 6.3 us,
// four waves and a part at a time 9.9.
constexpr int kJoinThreads = 64;

template <int OP>
__global__ __launch_bounds__(kJoinThreads) void linear_join_kernel(const float* __restrict__ partial,
                                                                   uint32_t splits, int64_t M, Epilogue e) {
  const int64_t chunks = (e.N + 7) / 8;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kJoinThreads;
  for (int64_t id = static_cast<int64_t>(blockIdx.x) * kJoinThreads + threadIdx.x; id < M * chunks;
       id += step) {
    const int64_t m = id / chunks, n = (id - m * chunks) * 8;
    const int count = static_cast<int>(min(e.N - n, static_cast<int64_t>(8)));
    const float* p = partial + m * e.N + n;
    float v[8], b[8];
    widen_chunk<kF32>(load_chunk<kF32>(p, count), v);
    if (count == 8) {
#pragma unroll 8
      for (uint32_t s = 1; s < splits; ++s) {
        widen_chunk<kF32>(load_chunk<kF32>(p + s * M * e.N, 8), b);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] + b[i];
      }
    } else {
#pragma unroll 4
      for (uint32_t s = 1; s < splits; ++s) {
        widen_chunk<kF32>(load_chunk<kF32>(p + s * M * e.N, count), b);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] + b[i];
      }
    }
    with_act(e.act, [&](auto act) { finish<OP, decltype(act)::value>(e, m, n, count, v); });
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

struct RowsArgs {
  const uint8_t* x;
  const uint8_t* w;
  const uint8_t* xs;  // kMX
  const uint8_t* ws;  // kMX
  int64_t M, N;
  uint32_t kbytes;
  uint32_t wide;  // rows of W for each block, at most 16
  Epilogue e;
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

template <int OP, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void linear_rows_kernel(RowsArgs a) {
  constexpr int kFrags = is8(OP) ? 1 : 2;
  __shared__ float sums[WAVES][16][17];
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const uint32_t lane = threadIdx.x % 64, low = lane % 16, g = lane / 16;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * a.wide;
  const bool in_w = low < a.wide, in_x = low < a.M;
  const int64_t wrow = min(n0 + (in_w ? low : 0), a.N - 1);
  const uint32_t xrow = in_x ? low : 0;
  const uint32_t kblocks = (a.kbytes + 31) / 32;
  const uint8_t* w = a.w + wrow * a.kbytes;
  const uint8_t* x = a.x + static_cast<int64_t>(xrow) * a.kbytes;
  const uint8_t* ws = OP == kOpMX ? a.ws + wrow * kblocks : nullptr;
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
    sums[wave][low][g * 4 + i] = s0 + s1;
  }
  __syncthreads();
  const int64_t m = threadIdx.x / 2;
  const uint32_t half = threadIdx.x % 2;
  const int64_t n = n0 + half * 8;
  if (threadIdx.x < 32 && m < a.M && n < a.N && half * 8 < a.wide) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = sums[0][m][half * 8 + i];
#pragma unroll
      for (int k = 1; k < WAVES; ++k) v[i] = v[i] + sums[k][m][half * 8 + i];
    }
    const int count = static_cast<int>(min(min(a.N - n, static_cast<int64_t>(8)), static_cast<int64_t>(a.wide - half * 8)));
    with_act(a.e.act, [&](auto act) { finish<OP, decltype(act)::value>(a.e, m, n, count, v); });
  }
}

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
// Backward
//
// gz and the bias's sums come from one pass over grad_out and z; the two
// products are tile kernels whose operands are turned on their way out of LDS.
// ---------------------------------------------------------------------------

// gz = rnd(grad_out * act'(z)) where gz is given, and this block's rows of the
// bias's sums (of the products before that rounding) where partial is: 512
// columns to a block, 8 to a lane; each of the four waves takes every fourth
// row, four rows' loads in flight, joined in ascending order.
template <int F, int ACT>
__global__ __launch_bounds__(256) void linear_gz_kernel(
    const typename Store<F>::type* __restrict__ grad_out,
    const typename Store<F>::type* __restrict__ z, typename Store<F>::type* __restrict__ gz,
    float* __restrict__ partial, int64_t M, int64_t N, int64_t ldz, int64_t rows) {
  constexpr int kAhead = 4;
  __shared__ float sums[4][512];
  const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 512 + lane * 8;
  const int64_t m0 = blockIdx.y * rows, m1 = min(M, m0 + rows);
  float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (n < N) {
    const int count = static_cast<int>(min(N - n, static_cast<int64_t>(8)));
    for (int64_t m = m0 + wave; m < m1; m += 4 * kAhead) {
      Chunk<F> cg[kAhead], cz[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (m + 4 * k < m1) {
          cg[k] = load_chunk<F>(grad_out + (m + 4 * k) * N + n, count);
          if constexpr (ACT != MHC_ACT_NONE) cz[k] = load_chunk<F>(z + (m + 4 * k) * N + n, count);
        }
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (m + 4 * k < m1) {
          float v[8], s[8];
          widen_chunk<F>(cg[k], v);
          if constexpr (ACT != MHC_ACT_NONE) {
            widen_chunk<F>(cz[k], s);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = v[i] * slope<ACT>(s[i]);
            Chunk<F> c;
            narrow_chunk<F>(v, c);
            // rows of gz are ldz long, zeros past N
            store_chunk<F>(gz + (m + 4 * k) * ldz + n, static_cast<int>(min(ldz - n, static_cast<int64_t>(8))), c);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[i] = sum[i] + v[i];
        }
    }
  }
  if (partial == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[wave][lane * 8 + i] = sum[i];
  __syncthreads();
  for (int k = threadIdx.x; k < 512; k += 256) {
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 512 + k;
    if (c < N)
      partial[blockIdx.y * N + c] = ((sums[0][k] + sums[1][k]) + sums[2][k]) + sums[3][k];
  }
}

// grad_bias[n] = the parts' sum, rounded once (+0.0 of none): 64 columns to a
// block, each of four waves every fourth part, joined in ascending order.
template <int F>
__global__ __launch_bounds__(256) void linear_bias_kernel(const float* __restrict__ partial,
                                                          typename Store<F>::type* __restrict__ out,
                                                          int64_t parts, int64_t N) {
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

__global__ __launch_bounds__(256) void linear_zero_kernel(uint16_t* __restrict__ p, int64_t count) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < count; i += step)
    p[i] = 0;
}

// ---------------------------------------------------------------------------
// Host side: sizes and the choice of a launch
// ---------------------------------------------------------------------------

bool known_dtype(int32_t d) { return d >= MHC_LINEAR_BF16 && d <= MHC_LINEAR_E4M3_MX; }
int64_t elem(int32_t dtype) { return is8(dtype) ? 1 : 2; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Shape {
  int bm, bn;
};

Shape shape_of(int32_t kernel) {
  switch (kernel) {
    case MHC_LINEAR_NARROW: return {64, 32};
    case MHC_LINEAR_SMALL: return {64, 64};
    case MHC_LINEAR_MEDIUM: return {128, 128};
    default: return {256, 256};
  }
}

mhc_status check_sizes(int64_t M, int64_t N, int64_t K, int32_t dtype) {
  if (M < 0 || M > INT32_MAX) return fail(MHC_ERROR_INVALID_VALUE, "M must be in [0, 2^31 - 1]");
  if (N < 1 || N > INT32_MAX) return fail(MHC_ERROR_INVALID_VALUE, "N must be in [1, 2^31 - 1]");
  if (K < 1 || K > MHC_LINEAR_MAX_K)
    return fail(MHC_ERROR_INVALID_VALUE, "K must be in [1, %lld] (got %lld)", MHC_LINEAR_MAX_K,
                static_cast<long long>(K));
  if (!known_dtype(dtype))
    return fail(MHC_ERROR_INVALID_VALUE,
                "dtype must be MHC_LINEAR_BF16, _F16, _E4M3_ROW or _E4M3_MX (got %d)", dtype);
  return ok();
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
  if (want < 0 || want > MHC_LINEAR_LARGE || parts < 0 || parts > kMaxSplits)
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
    const int64_t slots = k >= MHC_LINEAR_MEDIUM ? 256 : 512;
    while (s < 32 && M > 0 && tiles(k) * s * 2 <= slots && all / (s * 2) >= 4) s *= 2;
  }
  if (s > all) s = all;
  // no empty part
  s = ceil_div(all, ceil_div(all, s));
  *plan = {k, static_cast<int32_t>(s)};
  return ok();
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

struct FwdPlan {
  mhc_linear_launch launch;
  bool pad;
  int64_t ld, scale_ld;               // bytes of padded rows
  int64_t part, x, w, xs, ws, total;  // places
};

FwdPlan plan_fwd(int64_t M, int64_t N, int64_t K, int32_t dtype, const mhc_linear_launch& launch) {
  FwdPlan p = {};
  p.launch = launch;
  if (M == 0) return p;
  Places at;
  p.part = launch.splits > 1 ? at.take(mul_bytes(mul_bytes(M, N, 4), launch.splits, 1)) : 0;
  const int64_t row = K * elem(dtype), whole = dtype == MHC_LINEAR_E4M3_MX ? kTileK : 16;
  p.pad = launch.kernel != MHC_LINEAR_ROWS && row % whole != 0 && M >= kPadRows && N >= kPadRows &&
          (M > INT64_MAX / N / K || M * N * K >= kPadForward);
  if (p.pad) {
    p.ld = round_up(row, whole);
    p.x = at.take(mul_bytes(M, p.ld, 1));
    p.w = at.take(mul_bytes(N, p.ld, 1));
    if (dtype == MHC_LINEAR_E4M3_MX) {
      p.scale_ld = p.ld / 32;
      p.xs = at.take(mul_bytes(M, p.scale_ld, 1));
      p.ws = at.take(mul_bytes(N, p.scale_ld, 1));
    }
  }
  p.total = at.total;
  return p;
}

mhc_status validate_fwd(const void* x, const void* xs, const void* w, const void* ws,
                        const void* bias, const void* residual, const void* out, const void* z,
                        const void* workspace, int64_t workspace_bytes, int64_t M, int64_t N,
                        int64_t K, int32_t dtype, int32_t act, const mhc_linear_launch* launch,
                        FwdPlan* plan) {
  mhc_linear_launch chosen;
  mhc_status st = check_sizes(M, N, K, dtype);
  if (st != MHC_SUCCESS) return st;
  if (act < MHC_ACT_NONE || act > MHC_ACT_GELU)
    return fail(MHC_ERROR_INVALID_VALUE, "unknown activation %d", act);
  if ((st = make_plan(M, N, K, dtype, launch, &chosen)) != MHC_SUCCESS) return st;
  *plan = plan_fwd(M, N, K, dtype, chosen);
  if (!is8(dtype) && (xs != nullptr || ws != nullptr))
    return fail(MHC_ERROR_INVALID_VALUE, "16-bit operands have no scales");
  if (M == 0) return ok();
  const int64_t need = plan->total;
  if (need < 0) return fail(MHC_ERROR_INVALID_VALUE, "the workspace's size does not fit 64 bits");
  if (workspace_bytes < need)
    return fail(MHC_ERROR_INVALID_VALUE, "workspace_bytes %lld < %lld needed",
                static_cast<long long>(workspace_bytes), static_cast<long long>(need));
  const int64_t E = elem(dtype), MN = mul_bytes(M, N, 2);
  const int64_t blocks = ceil_div(K, 32);
  const bool row = dtype == MHC_LINEAR_E4M3_ROW;
  const auto scales = [&](int64_t r) { return !is8(dtype) ? 0 : row ? r * 4 : mul_bytes(r, blocks, 1); };
  const Tensor in[] = {{x, mul_bytes(M, K, E), E, "x"},
                       {xs, scales(M), row ? 4 : 1, "x_scales"},
                       {w, mul_bytes(N, K, E), E, "weight"},
                       {ws, scales(N), row ? 4 : 1, "weight_scales"},
                       {bias, bias != nullptr ? N * 2 : 0, 2, "bias"},
                       {residual, residual != nullptr ? MN : 0, 2, "residual"}};
  const Tensor outs[] = {{out, MN, 2, "out"},
                         {z, z != nullptr ? MN : 0, 2, "z"},
                         {workspace, need, 16, "workspace"}};
  return check_tensors(in, outs);
}

// Whether an operand can be loaded straight into LDS: whole, aligned 16-byte
// pieces, and where k runs down the rows all of it within a buffer's 31 bits.
template <bool TURNED>
bool whole(const Matrix& m, const TileArgs& a) {
  if (reinterpret_cast<uintptr_t>(m.p) % 16 != 0 || m.ld % 16 != 0) return false;
  return TURNED ? static_cast<int64_t>(a.kturned / 2) * m.ld <= INT32_MAX : a.kbytes % 16 == 0;
}

template <int OP, bool TX, bool TW>
bool straight(const TileArgs& a) {
  if (!whole<TX>(a.x, a) || !whole<TW>(a.w, a)) return false;
  // block scales come four of a row at a time
  return OP != kOpMX || (a.kbytes % kTileK == 0 && reinterpret_cast<uintptr_t>(a.xs) % 4 == 0 &&
                         reinterpret_cast<uintptr_t>(a.ws) % 4 == 0);
}

template <int OP, int BM, int BN, int WM, int WN, int STAGES, bool TX, bool TW>
hipError_t launch_tile(TileArgs a, hipStream_t s, hipEvent_t start, hipEvent_t stop) {
  a.tiles_m = static_cast<uint32_t>(ceil_div(a.M, BM));
  a.tiles_n = static_cast<uint32_t>(ceil_div(a.N, BN));
  const dim3 grid(a.tiles_m * a.tiles_n * a.splits), block(64 * WM * WN);
  if (straight<OP, TX, TW>(a))
    return launch_kernel(linear_tile_kernel<OP, BM, BN, WM, WN, STAGES, true, TX, TW>, grid, block,
                         s, start, stop, a);
  return launch_kernel(linear_tile_kernel<OP, BM, BN, WM, WN, STAGES, false, TX, TW>, grid, block,
                       s, start, stop, a);
}

template <int OP, bool TX, bool TW>
hipError_t launch_medium(const TileArgs& a, hipStream_t s, hipEvent_t start, hipEvent_t stop) {
  return launch_tile<OP, 128, 128, 2, 2, kMediumStages, TX, TW>(a, s, start, stop);
}

// The large tiles are loaded straight into LDS only; other operands go through
// the medium tiles, whose sums have the same order.
template <int OP, bool TX, bool TW>
hipError_t launch_large(TileArgs a, hipStream_t s, hipEvent_t start, hipEvent_t stop) {
  if (!straight<OP, TX, TW>(a)) return launch_medium<OP, TX, TW>(a, s, start, stop);
  a.tiles_m = static_cast<uint32_t>(ceil_div(a.M, 256));
  a.tiles_n = static_cast<uint32_t>(ceil_div(a.N, 256));
  return launch_kernel(linear_large_kernel<OP, TX, TW>, dim3(a.tiles_m * a.tiles_n * a.splits),
                       dim3(512), s, start, stop, a);
}

// One product and its epilogue, as planned. The backward's products (TW) have
// no narrow form.
template <int OP, bool TX, bool TW>
hipError_t launch_product(TileArgs a, const mhc_linear_launch& plan, hipStream_t s,
                          hipEvent_t start, hipEvent_t stop) {
  const int64_t all = ceil_div(a.kbytes, kTileK);
  a.splits = static_cast<uint32_t>(plan.splits);
  a.per_split = static_cast<uint32_t>(ceil_div(all, plan.splits));
  const bool join = a.splits > 1;
  const hipEvent_t end = join ? nullptr : stop;
  hipError_t e;
  switch (plan.kernel) {
    case MHC_LINEAR_NARROW:
      if constexpr (!TW) {
        e = launch_tile<OP, 64, 32, 4, 1, 3, TX, TW>(a, s, start, end);
        break;
      }
    case MHC_LINEAR_SMALL: e = launch_tile<OP, 64, 64, 2, 2, 3, TX, TW>(a, s, start, end); break;
    case MHC_LINEAR_MEDIUM: e = launch_medium<OP, TX, TW>(a, s, start, end); break;
    default: e = launch_large<OP, TX, TW>(a, s, start, end); break;
  }
  if (e != hipSuccess || !join) return e;
  const int64_t blocks = ceil_div(a.M * ceil_div(a.N, 8), kJoinThreads);
  return launch_kernel(linear_join_kernel<OP>, dim3(static_cast<uint32_t>(blocks < 16384 ? blocks : 16384)),
                       dim3(kJoinThreads), s, nullptr, stop, a.partial, a.splits, a.M, a.e);
}

template <int OP>
hipError_t launch_rows(const TileArgs& t, hipStream_t s, hipEvent_t start, hipEvent_t stop) {
  // the fewest blocks for each of 256 CUs, and W's rows spread evenly over them
  const int64_t wide = ceil_div(t.N, 256 * ceil_div(t.N, 256 * 16));
  const RowsArgs a = {static_cast<const uint8_t*>(t.x.p), static_cast<const uint8_t*>(t.w.p), t.xs,
                      t.ws, t.M, t.N, t.kbytes, static_cast<uint32_t>(wide), t.e};
  const dim3 grid(static_cast<uint32_t>(ceil_div(t.N, wide)));
  return launch_kernel(linear_rows_kernel<OP, 8>, grid, dim3(512), s, start, stop, a);
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

template <int OP>
hipError_t launch_fwd(TileArgs a, const FwdPlan& p, uint8_t* workspace, hipStream_t s,
                      hipEvent_t start, hipEvent_t stop) {
  if (p.launch.kernel == MHC_LINEAR_ROWS) return launch_rows<OP>(a, s, start, stop);
  a.partial = reinterpret_cast<float*>(workspace + p.part);
  if (p.pad) {
    PadJobs jobs = {};
    int count = 0;
    const int64_t blocks = (a.kbytes + 31) / 32;
    jobs.job[count++] = pad_job(a.x.p, workspace + p.x, a.M, a.kbytes, p.ld, false);
    jobs.job[count++] = pad_job(a.w.p, workspace + p.w, a.N, a.kbytes, p.ld, false);
    if (OP == kOpMX) {
      jobs.job[count++] = pad_job(a.xs, workspace + p.xs, a.M, blocks, p.scale_ld, true);
      jobs.job[count++] = pad_job(a.ws, workspace + p.ws, a.N, blocks, p.scale_ld, true);
      a.xs = workspace + p.xs;
      a.ws = workspace + p.ws;
    }
    const hipError_t e = launch_pad(jobs, count, s, start);
    if (e != hipSuccess) return e;
    start = nullptr;
    a.x = {workspace + p.x, a.M, p.ld};
    a.w = {workspace + p.w, a.N, p.ld};
    a.kbytes = static_cast<uint32_t>(p.ld);
  }
  return launch_product<OP, false, false>(a, p.launch, s, start, stop);
}

// --- backward ---

// Rows of grad_out that one block of linear_gz_kernel takes: about 512 blocks in
// all, of at least 8 rows, in at most 256 parts of the bias's sums.
int64_t bias_rows(int64_t M, int64_t N) {
  const int64_t wide = ceil_div(N, 512);
  const int64_t parts = wide >= 512 ? 1 : 512 / wide < 256 ? 512 / wide : 256;
  const int64_t r = ceil_div(M, parts);
  return r < 8 ? 8 : r;
}

struct BwdPlan {
  bool pad_k, pad_n;               // rows along K (x, W) and along N (gz) are copied whole
  int64_t ldk, ldn;                // their bytes
  int64_t gz, bias, x, w, part, total;  // places; part: split sums
  mhc_linear_launch px, pw;        // the two products
};

// A product of the backward: the tile kernels from 64 x 64 on.
mhc_status plan_product(int64_t M, int64_t N, int64_t K, int32_t dtype, mhc_linear_launch* p) {
  const mhc_status st = make_plan(M, N, K, dtype, nullptr, p);
  if (st != MHC_SUCCESS || p->kernel >= MHC_LINEAR_SMALL) return st;
  const mhc_linear_launch small = {MHC_LINEAR_SMALL, 0};
  return make_plan(M, N, K, dtype, &small, p);
}

BwdPlan plan_bwd(int64_t M, int64_t N, int64_t K, int32_t dtype) {
  BwdPlan p = {};
  if (M == 0) return p;
  Places at;
  const bool large = M > INT64_MAX / N / K || M * N * K >= kPadBackward;
  p.pad_k = large && K % 8 != 0;
  p.pad_n = large && N % 8 != 0;
  p.ldk = p.pad_k ? round_up(K * 2, 16) : K * 2;
  p.ldn = p.pad_n ? round_up(N * 2, 16) : N * 2;
  p.gz = at.take(mul_bytes(M, p.ldn, 1));
  p.bias = at.take(mul_bytes(ceil_div(M, bias_rows(M, N)), N, 4));
  if (p.pad_k) {
    p.x = at.take(mul_bytes(M, p.ldk, 1));
    p.w = at.take(mul_bytes(N, p.ldk, 1));
  }
  if (plan_product(M, K, N, dtype, &p.px) != MHC_SUCCESS ||
      plan_product(N, K, M, dtype, &p.pw) != MHC_SUCCESS)
    at.total = -1;
  const auto parts = [](int64_t rows, int64_t columns, const mhc_linear_launch& l) {
    return l.splits > 1 ? mul_bytes(mul_bytes(rows, columns, 4), l.splits, 1) : 0;
  };
  const int64_t a = parts(M, K, p.px), b = parts(N, K, p.pw);
  p.part = at.take(a < 0 || b < 0 ? -1 : a > b ? a : b);
  p.total = at.total;
  return p;
}

mhc_status check_bwd_sizes(int64_t M, int64_t N, int64_t K, int32_t dtype) {
  const mhc_status st = check_sizes(M, N, K, dtype);
  if (st != MHC_SUCCESS) return st;
  if (is8(dtype)) return fail(MHC_ERROR_INVALID_VALUE, "the backward takes 16-bit types");
  if (M > MHC_LINEAR_MAX_K || N > MHC_LINEAR_MAX_K)
    return fail(MHC_ERROR_INVALID_VALUE, "the backward sums over M and N: at most %lld of each",
                MHC_LINEAR_MAX_K);
  return ok();
}

mhc_status validate_bwd(const void* grad_out, const void* x, const void* w, const void* z,
                        const void* gx, const void* gw, const void* gb, const void* workspace,
                        int64_t workspace_bytes, int64_t M, int64_t N, int64_t K, int32_t dtype,
                        int32_t act) {
  const mhc_status st = check_bwd_sizes(M, N, K, dtype);
  if (st != MHC_SUCCESS) return st;
  if (act < MHC_ACT_NONE || act > MHC_ACT_GELU)
    return fail(MHC_ERROR_INVALID_VALUE, "unknown activation %d", act);
  const int64_t need = plan_bwd(M, N, K, dtype).total;
  if (need < 0) return fail(MHC_ERROR_INVALID_VALUE, "the workspace's size does not fit 64 bits");
  if (workspace_bytes < need)
    return fail(MHC_ERROR_INVALID_VALUE, "workspace_bytes %lld < %lld needed",
                static_cast<long long>(workspace_bytes), static_cast<long long>(need));
  const int64_t MN = mul_bytes(M, N, 2), MK = mul_bytes(M, K, 2);
  // with M == 0 only the gradients of the weight and the bias exist
  const int64_t NK = mul_bytes(N, K, 2);
  const Tensor in[] = {{grad_out, MN, 2, "grad_out"},
                       {x, MK, 2, "x"},
                       {w, M > 0 ? NK : 0, 2, "weight"},
                       {z, act != MHC_ACT_NONE ? MN : 0, 2, "z"}};
  const Tensor outs[] = {{gx, gx != nullptr ? MK : 0, 2, "grad_x"},
                         {gw, gw != nullptr ? NK : 0, 2, "grad_weight"},
                         {gb, gb != nullptr ? N * 2 : 0, 2, "grad_bias"},
                         {workspace, need, 16, "workspace"}};
  return check_tensors(in, outs);
}

struct BwdArgs {
  const void *grad_out, *x, *w, *z;
  void *gx, *gw, *gb;
  uint8_t* ws;
  int64_t M, N, K;
  int32_t act;
};

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
};

template <int OP>
hipError_t launch_bwd(const BwdArgs& a, int32_t dtype, hipStream_t s, hipEvent_t start,
                      hipEvent_t stop) {
  constexpr int F = out_format(OP);
  typedef typename Store<F>::type S;
  Marks marks = {start, stop};
  hipError_t e = hipSuccess;
  if (a.M == 0) {
    if (a.gw != nullptr) e = launch_zero(a.gw, a.N * a.K, s, marks.first(), nullptr);
    if (e == hipSuccess && a.gb != nullptr) e = launch_zero(a.gb, a.N, s, marks.first(), nullptr);
  } else {
    const BwdPlan p = plan_bwd(a.M, a.N, a.K, dtype);
    const S* gz = static_cast<const S*>(a.grad_out);
    const void *x = a.x, *w = a.w;
    PadJobs jobs = {};
    int count = 0;
    if (p.pad_k && a.gw != nullptr) {
      jobs.job[count++] = pad_job(a.x, a.ws + p.x, a.M, a.K * 2, p.ldk, false);
      x = a.ws + p.x;
    }
    if (p.pad_k && a.gx != nullptr) {
      jobs.job[count++] = pad_job(a.w, a.ws + p.w, a.N, a.K * 2, p.ldk, false);
      w = a.ws + p.w;
    }
    const bool products = a.gx != nullptr || a.gw != nullptr;
    if (p.pad_n && a.act == MHC_ACT_NONE && products) {
      jobs.job[count++] = pad_job(a.grad_out, a.ws + p.gz, a.M, a.N * 2, p.ldn, false);
      gz = reinterpret_cast<const S*>(a.ws + p.gz);
    }
    if (count > 0 && (e = launch_pad(jobs, count, s, marks.first())) != hipSuccess) return e;
    if (a.act != MHC_ACT_NONE || a.gb != nullptr) {
      const int64_t rows = bias_rows(a.M, a.N), parts = ceil_div(a.M, rows);
      S* made = a.act != MHC_ACT_NONE ? reinterpret_cast<S*>(a.ws + p.gz) : nullptr;
      float* sums = a.gb != nullptr ? reinterpret_cast<float*>(a.ws + p.bias) : nullptr;
      const auto run = [&](auto kernel) {
        return launch_kernel(kernel, dim3(static_cast<uint32_t>(ceil_div(a.N, 512)), static_cast<uint32_t>(parts)),
                             dim3(256), s, marks.first(), nullptr, static_cast<const S*>(a.grad_out),
                             static_cast<const S*>(a.z), made, sums, a.M, a.N, p.ldn / 2, rows);
      };
      switch (a.act) {
        case MHC_ACT_RELU: e = run(linear_gz_kernel<F, MHC_ACT_RELU>); break;
        case MHC_ACT_SILU: e = run(linear_gz_kernel<F, MHC_ACT_SILU>); break;
        case MHC_ACT_GELU: e = run(linear_gz_kernel<F, MHC_ACT_GELU>); break;
        default: e = run(linear_gz_kernel<F, MHC_ACT_NONE>); break;
      }
      if (e != hipSuccess) return e;
      if (made != nullptr) gz = made;
      if (a.gb != nullptr) {
        e = launch_kernel(linear_bias_kernel<F>, dim3(static_cast<uint32_t>(ceil_div(a.N, 64))), dim3(256),
                          s, nullptr, nullptr, sums, static_cast<S*>(a.gb), parts, a.N);
        if (e != hipSuccess) return e;
      }
    }
    if (a.gx != nullptr) {
      // grad_x [M, K]: rows of gz, with W [N, K] turned
      TileArgs t = {};
      t.x = {gz, a.M, p.ldn};
      t.w = {w, a.K, p.ldk};
      t.M = a.M; t.N = a.K;
      t.kbytes = static_cast<uint32_t>(p.ldn);  // gz's padding is zeros
      t.kturned = static_cast<uint32_t>(a.N * 2);
      t.partial = reinterpret_cast<float*>(a.ws + p.part);
      t.e.out = a.gx; t.e.N = a.K;
      e = launch_product<OP, false, true>(t, p.px, s, marks.first(), nullptr);
      if (e != hipSuccess) return e;
    }
    if (a.gw != nullptr) {
      // grad_weight [N, K]: gz [M, N] and x [M, K], both turned
      TileArgs t = {};
      t.x = {gz, a.N, p.ldn};
      t.w = {x, a.K, p.ldk};
      t.M = a.N; t.N = a.K;
      t.kbytes = t.kturned = static_cast<uint32_t>(a.M * 2);
      t.partial = reinterpret_cast<float*>(a.ws + p.part);
      t.e.out = a.gw; t.e.N = a.K;
      e = launch_product<OP, true, true>(t, p.pw, s, marks.first(), nullptr);
    }
  }
  if (e == hipSuccess && marks.start != nullptr) e = hipEventRecord(marks.first(), s);
  if (e == hipSuccess && stop != nullptr) e = hipEventRecord(stop, s);
  return e;
}

}  // namespace

extern "C" {

int mhc_linear_abi_version(void) { return MHC_LINEAR_ABI_VERSION; }

const char* mhc_linear_last_error_message(void) { return g_msg; }

mhc_status mhc_linear_plan(int64_t M, int64_t N, int64_t K, int32_t dtype,
                           const mhc_linear_launch* launch, mhc_linear_launch* plan) {
  mhc_linear_launch p;
  mhc_status st = check_sizes(M, N, K, dtype);
  if (st == MHC_SUCCESS) st = make_plan(M, N, K, dtype, launch, &p);
  if (st == MHC_SUCCESS && plan != nullptr) *plan = p;
  return st;
}

int64_t mhc_linear_fwd_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t dtype,
                                       const mhc_linear_launch* launch) {
  mhc_linear_launch p;
  if (check_sizes(M, N, K, dtype) != MHC_SUCCESS ||
      make_plan(M, N, K, dtype, launch, &p) != MHC_SUCCESS)
    return -1;
  return plan_fwd(M, N, K, dtype, p).total;
}

int64_t mhc_linear_bwd_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t dtype) {
  if (check_bwd_sizes(M, N, K, dtype) != MHC_SUCCESS) return -1;
  return plan_bwd(M, N, K, dtype).total;
}

mhc_status mhc_linear_validate_fwd(const void* x, const void* x_scales, const void* weight,
                                   const void* weight_scales, const void* bias,
                                   const void* residual, const void* out, const void* z,
                                   const void* workspace, int64_t workspace_bytes, int64_t M,
                                   int64_t N, int64_t K, int32_t dtype, int32_t act,
                                   const mhc_linear_launch* launch) {
  FwdPlan plan;
  return validate_fwd(x, x_scales, weight, weight_scales, bias, residual, out, z, workspace,
                      workspace_bytes, M, N, K, dtype, act, launch, &plan);
}

mhc_status mhc_linear_validate_bwd(const void* grad_out, const void* x, const void* weight,
                                   const void* z, const void* grad_x, const void* grad_weight,
                                   const void* grad_bias, const void* workspace,
                                   int64_t workspace_bytes, int64_t M, int64_t N, int64_t K,
                                   int32_t dtype, int32_t act) {
  return validate_bwd(grad_out, x, weight, z, grad_x, grad_weight, grad_bias, workspace,
                      workspace_bytes, M, N, K, dtype, act);
}

mhc_status mhc_linear_fwd(const void* x, const void* x_scales, const void* weight,
                          const void* weight_scales, const void* bias, const void* residual,
                          void* out, void* z, void* workspace, int64_t workspace_bytes, int64_t M,
                          int64_t N, int64_t K, int32_t dtype, int32_t act, void* stream,
                          const mhc_linear_launch* launch, void* start_event, void* stop_event) {
  FwdPlan plan;
  const mhc_status st = validate_fwd(x, x_scales, weight, weight_scales, bias, residual, out, z,
                                     workspace, workspace_bytes, M, N, K, dtype, act, launch, &plan);
  if (st != MHC_SUCCESS) return st;
  if (M == 0) return record_empty(stream, start_event, stop_event);
  TileArgs a = {};
  const int64_t ld = K * elem(dtype);
  a.x = {x, M, ld};
  a.w = {weight, N, ld};
  if (dtype == MHC_LINEAR_E4M3_MX) {
    a.xs = static_cast<const uint8_t*>(x_scales);
    a.ws = static_cast<const uint8_t*>(weight_scales);
  } else {
    a.e.x_scales = static_cast<const float*>(x_scales);
    a.e.weight_scales = static_cast<const float*>(weight_scales);
  }
  a.M = M;
  a.N = N;
  a.kbytes = static_cast<uint32_t>(ld);
  a.e.bias = bias;
  a.e.residual = residual;
  a.e.out = out;
  a.e.z = z;
  a.e.N = N;
  a.e.act = act;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const hipEvent_t b = static_cast<hipEvent_t>(start_event), f = static_cast<hipEvent_t>(stop_event);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  hipError_t e;
  switch (dtype) {
    case MHC_LINEAR_BF16: e = launch_fwd<kOpBF16>(a, plan, ws, s, b, f); break;
    case MHC_LINEAR_F16: e = launch_fwd<kOpF16>(a, plan, ws, s, b, f); break;
    case MHC_LINEAR_E4M3_ROW: e = launch_fwd<kOpE4M3>(a, plan, ws, s, b, f); break;
    default: e = launch_fwd<kOpMX>(a, plan, ws, s, b, f); break;
  }
  return launch_status(e, "product launch");
}

mhc_status mhc_linear_bwd(const void* grad_out, const void* x, const void* weight, const void* z,
                          void* grad_x, void* grad_weight, void* grad_bias, void* workspace,
                          int64_t workspace_bytes, int64_t M, int64_t N, int64_t K, int32_t dtype,
                          int32_t act, void* stream, void* start_event, void* stop_event) {
  const mhc_status st = validate_bwd(grad_out, x, weight, z, grad_x, grad_weight, grad_bias,
                                     workspace, workspace_bytes, M, N, K, dtype, act);
  if (st != MHC_SUCCESS) return st;
  const BwdArgs a = {grad_out, x, weight, z, grad_x, grad_weight, grad_bias,
                     static_cast<uint8_t*>(workspace), M, N, K, act};
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const hipEvent_t b = static_cast<hipEvent_t>(start_event), f = static_cast<hipEvent_t>(stop_event);
  const hipError_t e = dtype == MHC_LINEAR_BF16 ? launch_bwd<kOpBF16>(a, dtype, s, b, f)
                                                : launch_bwd<kOpF16>(a, dtype, s, b, f);
  return launch_status(e, "product backward launch");
}

}  // extern "C"
