// mhc_post.hip - write-back of a sublayer's output into the residual streams
// and its backward for gfx950 (see include/mhc_post.h for the operation).

#include "mhc_post.h"

#include "mhc_host.h"
#include "mhc_launch.h"
#include "mhc_rows.h"

#ifdef __FAST_MATH__
#error "this source must not be built with fast-math"
#endif

#pragma clang fp contract(off)

namespace {

typedef uint16_t bf16_t;

// Blocks of a launch at most; a block then takes every gridDim.x-th piece of
// work, so any T fits the launch limits.
constexpr int64_t kMaxBlocks = 1 << 20;

// Calls that read more than the 256 MiB of the memory-side cache read
// non-temporally: what an earlier kernel wrote is no longer there, and nothing
// is read twice. n = 4, H = 7168: T = 4096 (294 and 528 MB read) forward 90.0 -> 83.8 us, backward 150.8 ->
// 140.0; T = 1024 (73 and 132 MB) 20.9 -> 22.9 and 32.9 -> 37.1, so not there.
constexpr int64_t kStreamBytes = 256LL << 20;

// ---------------------------------------------------------------------------
// Forward
//
// Bound by memory: (2n + 1) * 2 bytes and n * (n + 1) multiply-adds for each
// (t, h). One wave takes 512 columns of one token, 8 in each lane: n + 1
// loads of 16 bytes in flight, then n stores of 16 bytes, nothing shared with
// any other wave. The gates are the same for the whole wave and come through
// scalar registers.
// ---------------------------------------------------------------------------
constexpr int kSlice = 512;

template <int N, bool STREAM>
__global__ __launch_bounds__(64) void post_fwd_kernel(
    const bf16_t* __restrict__ residual, const float* __restrict__ comb,
    const float* __restrict__ post, const bf16_t* __restrict__ y, bf16_t* __restrict__ out,
    int64_t T, int64_t H, int64_t slices) {
  for (int64_t piece = blockIdx.x; piece < T * slices; piece += gridDim.x) {
    const int64_t t = piece / slices;
    const int64_t h = (piece - t * slices) * kSlice + threadIdx.x * 8;
    if (h >= H) continue;
    const int count = static_cast<int>(min(H - h, static_cast<int64_t>(8)));
    Chunk<kBF16> c[N], cy;
#pragma unroll
    for (int j = 0; j < N; ++j) c[j] = load_chunk<kBF16, STREAM>(residual + (t * N + j) * H + h, count);
    cy = load_chunk<kBF16, STREAM>(y + t * H + h, count);
    float m[N][N], p[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      p[i] = post[t * N + i];
#pragma unroll
      for (int j = 0; j < N; ++j) m[i][j] = comb[(t * N + i) * N + j];
    }
    float r[N][8], v[8];
#pragma unroll
    for (int j = 0; j < N; ++j) widen_chunk<kBF16>(c[j], r[j]);
    widen_chunk<kBF16>(cy, v);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        o[e] = m[i][0] * r[0][e];
#pragma unroll
        for (int j = 1; j < N; ++j) o[e] = fmaf(m[i][j], r[j][e], o[e]);
        o[e] = fmaf(p[i], v[e], o[e]);
      }
      Chunk<kBF16> s;
      narrow_chunk<kBF16>(o, s);
      store_chunk<kBF16>(out + (t * N + i) * H + h, count, s);
    }
  }
}

// ---------------------------------------------------------------------------
// Backward
//
// One block takes one token and reads each of its rows once: for every chunk
// of 8 columns a thread loads the n gradients, the n streams and y, writes
// the n + 1 row gradients and adds to its n * (n + 1) running sums, which the
// block then joins through LDS. Bound by memory: (3n + 2) * 2 bytes for
// 2 n (n + 1) multiply-adds a column.
//
// The block size depends on H alone (and with it the order of the sums).
// ---------------------------------------------------------------------------
template <int N, int THREADS, bool STREAM>
__global__ __launch_bounds__(THREADS) void post_bwd_kernel(
    const bf16_t* __restrict__ grad_out, const bf16_t* __restrict__ residual,
    const float* __restrict__ comb, const float* __restrict__ post, const bf16_t* __restrict__ y,
    bf16_t* __restrict__ grad_residual, float* __restrict__ grad_comb,
    float* __restrict__ grad_post, bf16_t* __restrict__ grad_y, int64_t T, int64_t H) {
  constexpr int kWaves = THREADS / 64;
  constexpr int kSums = N * (N + 1);
  __shared__ float part[kWaves][kSums];
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    float m[N][N], p[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      p[i] = post[t * N + i];
#pragma unroll
      for (int j = 0; j < N; ++j) m[i][j] = comb[(t * N + i) * N + j];
    }
    float sum[N][N + 1];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j <= N; ++j) sum[i][j] = 0.0f;
    for (int64_t h = threadIdx.x * 8; h < H; h += THREADS * 8) {
      const int count = static_cast<int>(min(H - h, static_cast<int64_t>(8)));
      Chunk<kBF16> cg[N], cr[N], cy;
#pragma unroll
      for (int i = 0; i < N; ++i) cg[i] = load_chunk<kBF16, STREAM>(grad_out + (t * N + i) * H + h, count);
#pragma unroll
      for (int j = 0; j < N; ++j) cr[j] = load_chunk<kBF16, STREAM>(residual + (t * N + j) * H + h, count);
      cy = load_chunk<kBF16, STREAM>(y + t * H + h, count);
      float g[N][8], v[8];
#pragma unroll
      for (int i = 0; i < N; ++i) widen_chunk<kBF16>(cg[i], g[i]);
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        o[e] = p[0] * g[0][e];
#pragma unroll
        for (int i = 1; i < N; ++i) o[e] = fmaf(p[i], g[i][e], o[e]);
      }
      Chunk<kBF16> s;
      narrow_chunk<kBF16>(o, s);
      store_chunk<kBF16>(grad_y + t * H + h, count, s);
      widen_chunk<kBF16>(cy, v);
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[i][N] = fmaf(g[i][e], v[e], sum[i][N]);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        widen_chunk<kBF16>(cr[j], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          o[e] = m[0][j] * g[0][e];
#pragma unroll
          for (int i = 1; i < N; ++i) o[e] = fmaf(m[i][j], g[i][e], o[e]);
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[i][j] = fmaf(g[i][e], v[e], sum[i][j]);
        narrow_chunk<kBF16>(o, s);
        store_chunk<kBF16>(grad_residual + (t * N + j) * H + h, count, s);
      }
    }
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j <= N; ++j) {
        const float w = wave_sum(sum[i][j]);
        if (lane == 0) part[wave][i * (N + 1) + j] = w;
      }
    __syncthreads();
    for (int k = threadIdx.x; k < kSums; k += THREADS) {
      float s = part[0][k];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) s += part[w][k];
      const int i = k / (N + 1), j = k % (N + 1);
      if (j < N) grad_comb[(t * N + i) * N + j] = s;
      else grad_post[t * N + i] = s;
    }
    __syncthreads();  // `part` is written again for the next token
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

mhc_status check_sizes(int64_t T, int32_t n, int64_t H) {
  if (n != 2 && n != 4 && n != 8)
    return fail(MHC_ERROR_INVALID_VALUE, "the expansion rate n must be 2, 4 or 8 (got %d)", n);
  if (T < 0) return fail(MHC_ERROR_INVALID_VALUE, "T must not be negative");
  if (H < 1 || H > MHC_MAX_H)
    return fail(MHC_ERROR_INVALID_VALUE, "H must be in [1, %lld] (got %lld)", MHC_MAX_H,
                static_cast<long long>(H));
  return ok();
}

mhc_status validate_fwd(const void* residual, const void* comb, const void* post, const void* y,
                        const void* out, int64_t T, int32_t n, int64_t H) {
  mhc_status st = check_sizes(T, n, H);
  if (st != MHC_SUCCESS || T == 0) return st;
  const int64_t rows = mul_bytes(T, n * 2, H);
  const Tensor in[] = {{residual, rows, 2, "residual"},
                       {comb, mul_bytes(T, n * n, 4), 4, "comb"},
                       {post, mul_bytes(T, n, 4), 4, "post"},
                       {y, mul_bytes(T, 2, H), 2, "y"}};
  const Tensor outs[] = {{out, rows, 2, "out"}};
  return check_tensors(in, outs);
}

mhc_status validate_bwd(const void* grad_out, const void* residual, const void* comb,
                        const void* post, const void* y, const void* grad_residual,
                        const void* grad_comb, const void* grad_post, const void* grad_y,
                        int64_t T, int32_t n, int64_t H) {
  mhc_status st = check_sizes(T, n, H);
  if (st != MHC_SUCCESS || T == 0) return st;
  const int64_t rows = mul_bytes(T, n * 2, H), row = mul_bytes(T, 2, H);
  const int64_t mix = mul_bytes(T, n * n, 4), gates = mul_bytes(T, n, 4);
  const Tensor in[] = {{grad_out, rows, 2, "grad_out"},
                       {residual, rows, 2, "residual"},
                       {comb, mix, 4, "comb"},
                       {post, gates, 4, "post"},
                       {y, row, 2, "y"}};
  const Tensor outs[] = {{grad_residual, rows, 2, "grad_residual"},
                         {grad_comb, mix, 4, "grad_comb"},
                         {grad_post, gates, 4, "grad_post"},
                         {grad_y, row, 2, "grad_y"}};
  return check_tensors(in, outs);
}

template <int N>
hipError_t launch_fwd(const bf16_t* residual, const float* comb, const float* post,
                      const bf16_t* y, bf16_t* out, int64_t T, int64_t H, hipStream_t s,
                      hipEvent_t start, hipEvent_t stop) {
  const int64_t slices = (H + kSlice - 1) / kSlice;
  const int64_t blocks = T > kMaxBlocks / slices ? kMaxBlocks : T * slices;
  const bool stream = T * H * 2 * (N + 1) > kStreamBytes;
  return launch_kernel(stream ? post_fwd_kernel<N, true> : post_fwd_kernel<N, false>,
                       dim3(static_cast<uint32_t>(blocks)), dim3(64), s, start, stop, residual,
                       comb, post, y, out, T, H, slices);
}

template <int N, int THREADS>
hipError_t launch_bwd_t(const bf16_t* grad_out, const bf16_t* residual, const float* comb,
                        const float* post, const bf16_t* y, bf16_t* grad_residual,
                        float* grad_comb, float* grad_post, bf16_t* grad_y, int64_t T, int64_t H,
                        hipStream_t s, hipEvent_t start, hipEvent_t stop) {
  const int64_t blocks = T < kMaxBlocks ? T : kMaxBlocks;
  const bool stream = T * H * 2 * (2 * N + 1) > kStreamBytes;
  return launch_kernel(stream ? post_bwd_kernel<N, THREADS, true> : post_bwd_kernel<N, THREADS, false>,
                       dim3(static_cast<uint32_t>(blocks)), dim3(THREADS), s, start, stop, grad_out, residual, comb, post, y,
                       grad_residual, grad_comb, grad_post, grad_y, T, H);
}

template <int N, typename... A>
hipError_t launch_bwd(int64_t H, A... a) {
  if (H <= 64 * 8) return launch_bwd_t<N, 64>(a...);
  if (H <= 128 * 8) return launch_bwd_t<N, 128>(a...);
  if (H <= 256 * 8 || N == 8) return launch_bwd_t<N, 256>(a...);
  return launch_bwd_t<N, 512>(a...);  // T = 4096, H = 7168, n = 4: 4% less time than 256
}

}  // namespace

extern "C" {

int mhc_post_abi_version(void) { return MHC_POST_ABI_VERSION; }

const char* mhc_post_last_error_message(void) { return g_msg; }

mhc_status mhc_post_validate_fwd(const uint16_t* residual, const float* comb, const float* post,
                                 const uint16_t* y, const uint16_t* out, int64_t T, int32_t n,
                                 int64_t H) {
  return validate_fwd(residual, comb, post, y, out, T, n, H);
}

mhc_status mhc_post_validate_bwd(const uint16_t* grad_out, const uint16_t* residual,
                                 const float* comb, const float* post, const uint16_t* y,
                                 const uint16_t* grad_residual, const float* grad_comb,
                                 const float* grad_post, const uint16_t* grad_y, int64_t T,
                                 int32_t n, int64_t H) {
  return validate_bwd(grad_out, residual, comb, post, y, grad_residual, grad_comb, grad_post,
                      grad_y, T, n, H);
}

mhc_status mhc_post_fwd(const uint16_t* residual, const float* comb, const float* post,
                        const uint16_t* y, uint16_t* out, int64_t T, int32_t n, int64_t H,
                        void* stream, void* start_event, void* stop_event) {
  const mhc_status st = validate_fwd(residual, comb, post, y, out, T, n, H);
  if (st != MHC_SUCCESS) return st;
  if (T == 0) return record_empty(stream, start_event, stop_event);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const hipEvent_t b = static_cast<hipEvent_t>(start_event), e = static_cast<hipEvent_t>(stop_event);
  hipError_t r;
  switch (n) {
    case 2: r = launch_fwd<2>(residual, comb, post, y, out, T, H, s, b, e); break;
    case 4: r = launch_fwd<4>(residual, comb, post, y, out, T, H, s, b, e); break;
    default: r = launch_fwd<8>(residual, comb, post, y, out, T, H, s, b, e); break;
  }
  return launch_status(r, "write-back launch");
}

mhc_status mhc_post_bwd(const uint16_t* grad_out, const uint16_t* residual, const float* comb,
                        const float* post, const uint16_t* y, uint16_t* grad_residual,
                        float* grad_comb, float* grad_post, uint16_t* grad_y, int64_t T,
                        int32_t n, int64_t H, void* stream, void* start_event,
                        void* stop_event) {
  const mhc_status st = validate_bwd(grad_out, residual, comb, post, y, grad_residual, grad_comb,
                                     grad_post, grad_y, T, n, H);
  if (st != MHC_SUCCESS) return st;
  if (T == 0) return record_empty(stream, start_event, stop_event);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const hipEvent_t b = static_cast<hipEvent_t>(start_event), e = static_cast<hipEvent_t>(stop_event);
  hipError_t r;
  switch (n) {
    case 2: r = launch_bwd<2>(H, grad_out, residual, comb, post, y, grad_residual, grad_comb,
                              grad_post, grad_y, T, H, s, b, e); break;
    case 4: r = launch_bwd<4>(H, grad_out, residual, comb, post, y, grad_residual, grad_comb,
                              grad_post, grad_y, T, H, s, b, e); break;
    default: r = launch_bwd<8>(H, grad_out, residual, comb, post, y, grad_residual, grad_comb,
                               grad_post, grad_y, T, H, s, b, e); break;
  }
  return launch_status(r, "write-back backward launch");
}

}  // extern "C"
