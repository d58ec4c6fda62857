// mhc_gated.hip - gated feed-forward block: both projections, the activation and
// the product of the two in one kernel, and its backward, for gfx950 (see
// include/mhc_gated.h for the operation).

#include "mhc_gated.h"

#include <math.h>

#include "mhc_tiles_host.h"

#ifdef __FAST_MATH__
#error "this source must not be built with fast-math"
#endif

#pragma clang fp contract(off)

namespace {

// ---------------------------------------------------------------------------
// Forward
//
// The tile kernels of the product with two weights: half of a tile's W rows are
// Wg's and half are Wu's, for the same columns of out, so that both sums of an
// output stand in one lane's registers, x is read once for both, and neither
// projection is written unless the caller wants it.
// ---------------------------------------------------------------------------

struct GatedEpilogue {
  static constexpr int kW = kBoth, kSums = 2, kGroup = 0;
  static constexpr bool kSplits = true, kHalves = false, kTakes = false, kWrites = true, kEarly = false;
  const void* gate_bias;
  const void* up_bias;
  void* out;
  void* gate;
  void* up;
  const float* x_scales;  // where the type has scales of rows
  const float* gate_scales;
  const float* up_scales;
  int64_t N;  // row stride of out, gate and up
  int32_t act;

  template <int OP, class Fn>
  __device__ __forceinline__ void with(const Fn& fn) const;
};

// Columns [n, n + count) of row m of one projection from its sums over k: scales,
// bias, and the stored value where it is wanted.
template <int OP>
__device__ __forceinline__ void project(const float* x_scales, const float* scales, const void* bias,
                                        void* z, int64_t N, int64_t m, int64_t n, int count,
                                        float (&v)[8]) {
  constexpr int F = out_format(OP);
  typedef typename Store<F>::type S;
  float b[8];
  if constexpr (scaled(OP)) {
    const float xs = x_scales[m];
    widen_chunk<kF32>(load_chunk<kF32>(scales + n, count), b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = sum_value<OP>(v[i]) * (xs * b[i]);
  }
  if (bias != nullptr) {
    widen_chunk<F>(load_chunk<F>(static_cast<const S*>(bias) + n, count), b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] + b[i];
  }
  if (z != nullptr) {
    Chunk<F> c;
    narrow_chunk<F>(v, c);
    store_chunk<F>(static_cast<S*>(z) + m * N + n, count, c);
  }
}

template <int OP, class Fn>
__device__ __forceinline__ void GatedEpilogue::with(const Fn& fn) const {
  constexpr int F = out_format(OP);
  typedef typename Store<F>::type S;
  with_act(act, [&](auto a) {
    fn([&](int64_t m, int64_t n, int count, float(&v)[16]) {
      float g[8], u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        g[i] = v[i];
        u[i] = v[8 + i];
      }
      project<OP>(x_scales, gate_scales, gate_bias, gate, N, m, n, count, g);
      project<OP>(x_scales, up_scales, up_bias, up, N, m, n, count, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = activate<decltype(a)::value>(g[i]) * u[i];
      Chunk<F> c;
      narrow_chunk<F>(g, c);
      store_chunk<F>(static_cast<S*>(out) + m * N + n, count, c);
    });
  });
}

// ---------------------------------------------------------------------------
// Backward
//
// One pass over grad_out, gate and up makes dg and du side by side, [M][dg | du],
// and the biases' sums. grad_x is then one product whose sum runs through dg with
// Wg and on through du with Wu (kChain); both weights' gradients are one launch
// over the columns of dg and du (kHalves), which is loaded straight into LDS while
// it spans no more than 2^31 - 1 bytes: 32768 x 16320 x 4096 7.4 ms, x 16384 through
// registers 12.4.
// ---------------------------------------------------------------------------

// 512 columns to a block, 8 to a lane; each of the four waves takes every fourth
// row, two rows' loads in flight; the biases' sums (of the values before their
// rounding) are joined in ascending order. Columns N..half of dg and of du are
// zeros: a half is whole tiles of the sum.
template <int F, int ACT>
__global__ __launch_bounds__(256) void gated_gz_kernel(
    const typename Store<F>::type* __restrict__ grad_out,
    const typename Store<F>::type* __restrict__ gate,
    const typename Store<F>::type* __restrict__ up, typename Store<F>::type* __restrict__ gz,
    float* __restrict__ partial, int64_t M, int64_t N, int64_t half, int64_t rows, int64_t parts) {
  constexpr int kAhead = 2;
  __shared__ float sums[2][4][512];
  const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 512 + lane * 8;
  const int64_t m0 = blockIdx.y * rows, m1 = min(M, m0 + rows);
  float sg[8] = {0, 0, 0, 0, 0, 0, 0, 0}, su[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (n < half) {
    const int count = n < N ? static_cast<int>(min(N - n, static_cast<int64_t>(8))) : 0;
    for (int64_t m = m0 + wave; m < m1; m += 4 * kAhead) {
      Chunk<F> cd[kAhead], cg[kAhead], cu[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        cd[k] = cg[k] = cu[k] = zero_chunk<F>();
        if (m + 4 * k < m1 && count > 0) {
          const int64_t at = (m + 4 * k) * N + n;
          cd[k] = load_chunk<F>(grad_out + at, count);
          cg[k] = load_chunk<F>(gate + at, count);
          cu[k] = load_chunk<F>(up + at, count);
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (m + 4 * k < m1) {
          float d[8], g[8], u[8];
          widen_chunk<F>(cd[k], d);
          widen_chunk<F>(cg[k], g);
          widen_chunk<F>(cu[k], u);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            u[i] = (d[i] * u[i]) * slope<ACT>(g[i]);
            d[i] = d[i] * activate<ACT>(g[i]);
            sg[i] = sg[i] + u[i];
            su[i] = su[i] + d[i];
          }
          typename Store<F>::type* to = gz + (m + 4 * k) * 2 * half + n;
          Chunk<F> c;
          narrow_chunk<F>(u, c);
          store_chunk<F>(to, 8, c);
          narrow_chunk<F>(d, c);
          store_chunk<F>(to + half, 8, c);
        }
    }
  }
  if (partial == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sums[0][wave][lane * 8 + i] = sg[i];
    sums[1][wave][lane * 8 + i] = su[i];
  }
  __syncthreads();
  for (int k = threadIdx.x; k < 1024; k += 256) {
    const int s = k / 512, i = k % 512;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 512 + i;
    if (c < N)
      partial[(s * parts + blockIdx.y) * N + c] = ((sums[s][0][i] + sums[s][1][i]) + sums[s][2][i]) + sums[s][3][i];
  }
}

// The biases' gradients, of the gate in blockIdx.y 0: the parts' sums, rounded once
// (see linear_bias_kernel).
template <int F>
__global__ __launch_bounds__(256) void gated_bias_kernel(const float* __restrict__ partial,
                                                         typename Store<F>::type* gate,
                                                         typename Store<F>::type* up, int64_t parts, int64_t N) {
  typename Store<F>::type* const out = blockIdx.y == 0 ? gate : up;
  if (out != nullptr) sum_parts<F>(partial + blockIdx.y * parts * N, out, parts, N);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

typedef TileArgs<GatedEpilogue> Args;

mhc_status check_sizes(int64_t M, int64_t N, int64_t K, int32_t dtype) {
  if (M < 0 || M > INT32_MAX) return fail(MHC_ERROR_INVALID_VALUE, "M must be in [0, 2^31 - 1]");
  if (N < 1 || N > INT32_MAX / 2)
    return fail(MHC_ERROR_INVALID_VALUE, "N must be in [1, 2^30 - 1]");
  if (K < 1 || K > MHC_LINEAR_MAX_K)
    return fail(MHC_ERROR_INVALID_VALUE, "K must be in [1, %lld] (got %lld)", MHC_LINEAR_MAX_K,
                static_cast<long long>(K));
  if (!known_dtype(dtype))
    return fail(MHC_ERROR_INVALID_VALUE,
                "dtype must be MHC_LINEAR_BF16, _F16, _E4M3_ROW, _E4M3_MX or _I8_ROW (got %d)", dtype);
  if (dtype == MHC_LINEAR_I8_ROW && K > MHC_LINEAR_MAX_K_I8)
    return fail(MHC_ERROR_INVALID_VALUE, "K must be at most %d with 8-bit integers (got %lld)",
                MHC_LINEAR_MAX_K_I8, static_cast<long long>(K));
  return ok();
}

// The product's plan for 2 N rows of weights; there is no narrow form.
mhc_status plan_gated(int64_t M, int64_t N, int64_t K, int32_t dtype,
                      const mhc_linear_launch* launch, mhc_linear_launch* p) {
  if (launch != nullptr && launch->kernel == MHC_LINEAR_NARROW)
    return fail(MHC_ERROR_INVALID_VALUE, "launch: there is no narrow kernel of two weights");
  return best_plan(M, 2 * N, K, dtype, false, 32, launch, p);
}

struct FwdPlan {
  mhc_linear_launch launch;
  bool pad;
  int64_t ld, scale_ld;                         // bytes of padded rows
  int64_t part, x, wg, wu, xs, gs, us, total;   // places
};

FwdPlan plan_fwd(int64_t M, int64_t N, int64_t K, int32_t dtype, const mhc_linear_launch& launch) {
  FwdPlan p = {};
  p.launch = launch;
  if (M == 0) return p;
  Places at;
  p.part = launch.splits > 1 ? at.take(mul_bytes(mul_bytes(M, 2 * N, 4), launch.splits, 1)) : 0;
  const int64_t row = K * elem(dtype), whole = dtype == MHC_LINEAR_E4M3_MX ? kTileK : 16;
  p.pad = launch.kernel != MHC_LINEAR_ROWS && row % whole != 0 && M >= kPadRows && 2 * N >= kPadRows &&
          (M > INT64_MAX / (2 * N) / K || M * 2 * N * K >= kPadForward);
  if (p.pad) {
    p.ld = round_up(row, whole);
    p.x = at.take(mul_bytes(M, p.ld, 1));
    p.wg = at.take(mul_bytes(N, p.ld, 1));
    p.wu = at.take(mul_bytes(N, p.ld, 1));
    if (dtype == MHC_LINEAR_E4M3_MX) {
      p.scale_ld = p.ld / 32;
      p.xs = at.take(mul_bytes(M, p.scale_ld, 1));
      p.gs = at.take(mul_bytes(N, p.scale_ld, 1));
      p.us = at.take(mul_bytes(N, p.scale_ld, 1));
    }
  }
  p.total = at.total;
  return p;
}

mhc_status check_workspace(int64_t need, int64_t bytes) {
  if (need < 0) return fail(MHC_ERROR_INVALID_VALUE, "the workspace's size does not fit 64 bits");
  if (bytes < need)
    return fail(MHC_ERROR_INVALID_VALUE, "workspace_bytes %lld < %lld needed",
                static_cast<long long>(bytes), static_cast<long long>(need));
  return ok();
}

mhc_status validate_fwd(const void* x, const void* xs, const void* wg, const void* gs,
                        const void* wu, const void* us, const void* gate_bias,
                        const void* up_bias, const void* out, const void* gate, const void* up,
                        const void* workspace, int64_t workspace_bytes, int64_t M, int64_t N,
                        int64_t K, int32_t dtype, int32_t act, const mhc_linear_launch* launch,
                        FwdPlan* plan) {
  mhc_linear_launch chosen;
  mhc_status st = check_sizes(M, N, K, dtype);
  if (st != MHC_SUCCESS) return st;
  if (act < MHC_ACT_NONE || act > MHC_ACT_GELU)
    return fail(MHC_ERROR_INVALID_VALUE, "unknown activation %d", act);
  if ((st = plan_gated(M, N, K, dtype, launch, &chosen)) != MHC_SUCCESS) return st;
  *plan = plan_fwd(M, N, K, dtype, chosen);
  if (!is8(dtype) && (xs != nullptr || gs != nullptr || us != nullptr))
    return fail(MHC_ERROR_INVALID_VALUE, "16-bit operands have no scales");
  if (M == 0) return ok();
  if ((st = check_workspace(plan->total, workspace_bytes)) != MHC_SUCCESS) return st;
  const int64_t E = elem(dtype), MN = mul_bytes(M, N, 2);
  const int64_t blocks = ceil_div(K, 32);
  const bool row = scaled(dtype);
  const auto scales = [&](int64_t r) { return !is8(dtype) ? 0 : row ? r * 4 : mul_bytes(r, blocks, 1); };
  const Tensor in[] = {{x, mul_bytes(M, K, E), E, "x"},
                       {xs, scales(M), row ? 4 : 1, "x_scales"},
                       {wg, mul_bytes(N, K, E), E, "gate_weight"},
                       {gs, scales(N), row ? 4 : 1, "gate_scales"},
                       {wu, mul_bytes(N, K, E), E, "up_weight"},
                       {us, scales(N), row ? 4 : 1, "up_scales"},
                       {gate_bias, gate_bias != nullptr ? N * 2 : 0, 2, "gate_bias"},
                       {up_bias, up_bias != nullptr ? N * 2 : 0, 2, "up_bias"}};
  const Tensor outs[] = {{out, MN, 2, "out"},
                         {gate, gate != nullptr ? MN : 0, 2, "gate"},
                         {up, up != nullptr ? MN : 0, 2, "up"},
                         {workspace, plan->total, 16, "workspace"}};
  return check_tensors(in, outs);
}

template <int OP>
hipError_t launch_fwd(Args a, const FwdPlan& p, uint8_t* workspace, hipStream_t s,
                      hipEvent_t start, hipEvent_t stop) {
  if (p.launch.kernel == MHC_LINEAR_ROWS) return launch_rows<OP>(a, s, start, stop);
  a.partial = reinterpret_cast<float*>(workspace + p.part);
  if (p.pad) {
    PadJobs jobs = {};
    jobs.job[0] = pad_job(a.x.p, workspace + p.x, a.M, a.kbytes, p.ld, false);
    jobs.job[1] = pad_job(a.w.p, workspace + p.wg, a.N, a.kbytes, p.ld, false);
    jobs.job[2] = pad_job(a.w2.p, workspace + p.wu, a.N, a.kbytes, p.ld, false);
    hipError_t e = launch_pad(jobs, 3, s, start);
    if (e != hipSuccess) return e;
    if (OP == kOpMX) {
      const int64_t blocks = (a.kbytes + 31) / 32;
      jobs.job[0] = pad_job(a.xs, workspace + p.xs, a.M, blocks, p.scale_ld, true);
      jobs.job[1] = pad_job(a.ws, workspace + p.gs, a.N, blocks, p.scale_ld, true);
      jobs.job[2] = pad_job(a.ws2, workspace + p.us, a.N, blocks, p.scale_ld, true);
      if ((e = launch_pad(jobs, 3, s, nullptr)) != hipSuccess) return e;
      a.xs = workspace + p.xs;
      a.ws = workspace + p.gs;
      a.ws2 = workspace + p.us;
    }
    start = nullptr;
    a.x = {workspace + p.x, a.M, p.ld};
    a.w = {workspace + p.wg, a.N, p.ld};
    a.w2 = {workspace + p.wu, a.N, p.ld};
    a.kbytes = static_cast<uint32_t>(p.ld);
  }
  return launch_product<OP, false, false>(a, p.launch, s, start, stop);
}

// --- backward ---

// Rows of grad_out that one block of gated_gz_kernel takes: about 1024 blocks in
// all, of at least 8 rows, in at most 256 parts of the biases' sums.
int64_t gz_rows(int64_t M, int64_t half) {
  const int64_t wide = ceil_div(half, 512);
  const int64_t parts = wide >= 1024 ? 1 : 1024 / wide < 256 ? 1024 / wide : 256;
  const int64_t r = ceil_div(M, parts);
  return r < 8 ? 8 : r;
}

struct BwdPlan {
  bool pad;                                  // rows along K are copied whole
  int64_t half, ldk;                         // columns of dg in gz; bytes of x's and the weights' rows
  int64_t rows, parts;                       // of gated_gz_kernel
  int64_t gz, bias, x, wg, wu, part, total;  // places; part: split sums
  mhc_linear_launch px, pw;                  // the two launches
};

BwdPlan plan_bwd(int64_t M, int64_t N, int64_t K, int32_t dtype) {
  BwdPlan p = {};
  if (M == 0) return p;
  Places at;
  p.half = round_up(N, kTileK / 2);
  p.rows = gz_rows(M, p.half);
  p.parts = ceil_div(M, p.rows);
  p.pad = K % 8 != 0 && (M > INT64_MAX / (2 * N) / K || M * 2 * N * K >= kPadBackward);
  p.ldk = p.pad ? round_up(K * 2, 16) : K * 2;
  p.gz = at.take(mul_bytes(M, 2 * p.half, 2));
  p.bias = at.take(mul_bytes(mul_bytes(p.parts, N, 4), 2, 1));
  if (p.pad) {
    p.x = at.take(mul_bytes(M, p.ldk, 1));
    p.wg = at.take(mul_bytes(N, p.ldk, 1));
    p.wu = at.take(mul_bytes(N, p.ldk, 1));
  }
  if (best_plan(M, K, 2 * p.half, dtype, true, 32, nullptr, &p.px) != MHC_SUCCESS ||
      best_plan(2 * N, K, M, dtype, true, 32, nullptr, &p.pw) != MHC_SUCCESS)
    at.total = -1;
  const auto parts = [](int64_t rows, int64_t columns, const mhc_linear_launch& l) {
    return l.splits > 1 ? mul_bytes(mul_bytes(rows, columns, 4), l.splits, 1) : 0;
  };
  const int64_t a = parts(M, K, p.px), b = parts(2 * N, K, p.pw);
  p.part = at.take(a < 0 || b < 0 ? -1 : a > b ? a : b);
  p.total = at.total;
  return p;
}

mhc_status check_bwd_sizes(int64_t M, int64_t N, int64_t K, int32_t dtype) {
  const mhc_status st = check_sizes(M, N, K, dtype);
  if (st != MHC_SUCCESS) return st;
  if (is8(dtype)) return fail(MHC_ERROR_INVALID_VALUE, "the backward takes 16-bit types");
  if (M > MHC_LINEAR_MAX_K || N > MHC_GATED_MAX_BWD_N)
    return fail(MHC_ERROR_INVALID_VALUE, "the backward sums over M and both N: at most %lld and %lld",
                MHC_LINEAR_MAX_K, MHC_GATED_MAX_BWD_N);
  return ok();
}

mhc_status validate_bwd(const void* grad_out, const void* x, const void* wg, const void* wu,
                        const void* gate, const void* up, const void* gx, const void* ggw,
                        const void* guw, const void* ggb, const void* gub, const void* workspace,
                        int64_t workspace_bytes, int64_t M, int64_t N, int64_t K, int32_t dtype,
                        int32_t act) {
  mhc_status st = check_bwd_sizes(M, N, K, dtype);
  if (st != MHC_SUCCESS) return st;
  if (act < MHC_ACT_NONE || act > MHC_ACT_GELU)
    return fail(MHC_ERROR_INVALID_VALUE, "unknown activation %d", act);
  if ((ggw == nullptr) != (guw == nullptr))
    return fail(MHC_ERROR_INVALID_VALUE, "grad_gate_weight and grad_up_weight come together");
  const int64_t need = plan_bwd(M, N, K, dtype).total;
  if ((st = check_workspace(need, workspace_bytes)) != MHC_SUCCESS) return st;
  const int64_t MN = mul_bytes(M, N, 2), MK = mul_bytes(M, K, 2);
  // with M == 0 only the gradients of the weights and the biases exist
  const int64_t NK = mul_bytes(N, K, 2);
  const Tensor in[] = {{grad_out, MN, 2, "grad_out"},
                       {x, MK, 2, "x"},
                       {wg, M > 0 ? NK : 0, 2, "gate_weight"},
                       {wu, M > 0 ? NK : 0, 2, "up_weight"},
                       {gate, MN, 2, "gate"},
                       {up, MN, 2, "up"}};
  const Tensor outs[] = {{gx, gx != nullptr ? MK : 0, 2, "grad_x"},
                         {ggw, ggw != nullptr ? NK : 0, 2, "grad_gate_weight"},
                         {guw, guw != nullptr ? NK : 0, 2, "grad_up_weight"},
                         {ggb, ggb != nullptr ? N * 2 : 0, 2, "grad_gate_bias"},
                         {gub, gub != nullptr ? N * 2 : 0, 2, "grad_up_bias"},
                         {workspace, need, 16, "workspace"}};
  return check_tensors(in, outs);
}

struct BwdArgs {
  const void *grad_out, *x, *wg, *wu, *gate, *up;
  void *gx, *ggw, *guw, *ggb, *gub;
  uint8_t* ws;
  int64_t M, N, K;
  int32_t act;
};

template <int OP>
hipError_t launch_bwd(const BwdArgs& a, int32_t dtype, hipStream_t s, hipEvent_t start,
                      hipEvent_t stop) {
  constexpr int F = out_format(OP);
  typedef typename Store<F>::type S;
  Marks marks = {start, stop};
  hipError_t e = hipSuccess;
  if (a.M == 0) {
    for (void* p : {a.ggw, a.guw})
      if (p != nullptr && e == hipSuccess) e = launch_zero(p, a.N * a.K, s, marks.first(), nullptr);
    for (void* p : {a.ggb, a.gub})
      if (p != nullptr && e == hipSuccess) e = launch_zero(p, a.N, s, marks.first(), nullptr);
    return marks.end(e, s);
  }
  const BwdPlan p = plan_bwd(a.M, a.N, a.K, dtype);
  const void *x = a.x, *wg = a.wg, *wu = a.wu;
  if (p.pad) {
    PadJobs jobs = {};
    int count = 0;
    if (a.ggw != nullptr) {
      jobs.job[count++] = pad_job(a.x, a.ws + p.x, a.M, a.K * 2, p.ldk, false);
      x = a.ws + p.x;
    }
    if (a.gx != nullptr) {
      jobs.job[count++] = pad_job(a.wg, a.ws + p.wg, a.N, a.K * 2, p.ldk, false);
      jobs.job[count++] = pad_job(a.wu, a.ws + p.wu, a.N, a.K * 2, p.ldk, false);
      wg = a.ws + p.wg;
      wu = a.ws + p.wu;
    }
    if (count > 0 && (e = launch_pad(jobs, count, s, marks.first())) != hipSuccess) return e;
  }
  const bool bias = a.ggb != nullptr || a.gub != nullptr;
  if (bias || a.gx != nullptr || a.ggw != nullptr) {
    float* sums = bias ? reinterpret_cast<float*>(a.ws + p.bias) : nullptr;
    const auto run = [&](auto kernel) {
      return launch_kernel(kernel, dim3(static_cast<uint32_t>(ceil_div(p.half, 512)), static_cast<uint32_t>(p.parts)),
                           dim3(256), s, marks.first(), nullptr, static_cast<const S*>(a.grad_out),
                           static_cast<const S*>(a.gate), static_cast<const S*>(a.up),
                           reinterpret_cast<S*>(a.ws + p.gz), sums, a.M, a.N, p.half, p.rows, p.parts);
    };
    switch (a.act) {
      case MHC_ACT_RELU: e = run(gated_gz_kernel<F, MHC_ACT_RELU>); break;
      case MHC_ACT_SILU: e = run(gated_gz_kernel<F, MHC_ACT_SILU>); break;
      case MHC_ACT_GELU: e = run(gated_gz_kernel<F, MHC_ACT_GELU>); break;
      default: e = run(gated_gz_kernel<F, MHC_ACT_NONE>); break;
    }
    if (e != hipSuccess) return e;
    if (bias) {
      e = launch_kernel(gated_bias_kernel<F>, dim3(static_cast<uint32_t>(ceil_div(a.N, 64)), 2), dim3(256),
                        s, nullptr, nullptr, sums, static_cast<S*>(a.ggb), static_cast<S*>(a.gub), p.parts, a.N);
      if (e != hipSuccess) return e;
    }
  }
  if (a.gx != nullptr) {
    // grad_x [M, K]: rows of (dg | du), with Wg and then Wu turned
    TileArgs<StoreEpilogue<kChain, false>> t = {};
    t.x = {a.ws + p.gz, a.M, p.half * 4};
    t.w = {wg, a.K, p.ldk};
    t.w2 = {wu, a.K, p.ldk};
    t.M = a.M; t.N = a.K;
    t.kbytes = static_cast<uint32_t>(p.half * 4);
    t.kturned = static_cast<uint32_t>(a.N * 2);
    t.kfirst = static_cast<uint32_t>(p.half * 2 / kTileK);
    t.partial = reinterpret_cast<float*>(a.ws + p.part);
    t.e = {a.gx, nullptr, a.M, a.K};
    e = launch_product<OP, false, true>(t, p.px, s, marks.first(), nullptr);
    if (e != hipSuccess) return e;
  }
  if (a.ggw != nullptr) {
    // the weights' gradients [N, K]: the columns of dg and of du, and x, all turned
    TileArgs<StoreEpilogue<kOne, true>> t = {};
    t.x = {a.ws + p.gz, 2 * p.half, p.half * 4};
    t.xupper = static_cast<uint32_t>(p.half);
    t.w = {x, a.K, p.ldk};
    t.M = a.N; t.N = a.K;
    t.kbytes = t.kturned = static_cast<uint32_t>(a.M * 2);
    t.partial = reinterpret_cast<float*>(a.ws + p.part);
    t.e = {a.ggw, a.guw, a.N, a.K};
    e = launch_product<OP, true, true>(t, p.pw, s, marks.first(), nullptr);
  }
  return marks.end(e, s);
}

}  // namespace

extern "C" {

int mhc_gated_abi_version(void) { return MHC_GATED_ABI_VERSION; }

const char* mhc_gated_last_error_message(void) { return g_msg; }

mhc_status mhc_gated_plan(int64_t M, int64_t N, int64_t K, int32_t dtype,
                          const mhc_linear_launch* launch, mhc_linear_launch* plan) {
  mhc_linear_launch p;
  mhc_status st = check_sizes(M, N, K, dtype);
  if (st == MHC_SUCCESS) st = plan_gated(M, N, K, dtype, launch, &p);
  if (st == MHC_SUCCESS && plan != nullptr) *plan = p;
  return st;
}

int64_t mhc_gated_fwd_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t dtype,
                                      const mhc_linear_launch* launch) {
  mhc_linear_launch p;
  if (check_sizes(M, N, K, dtype) != MHC_SUCCESS ||
      plan_gated(M, N, K, dtype, launch, &p) != MHC_SUCCESS)
    return -1;
  return plan_fwd(M, N, K, dtype, p).total;
}

int64_t mhc_gated_bwd_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t dtype) {
  if (check_bwd_sizes(M, N, K, dtype) != MHC_SUCCESS) return -1;
  return plan_bwd(M, N, K, dtype).total;
}

mhc_status mhc_gated_validate_fwd(const void* x, const void* x_scales, const void* gate_weight,
                                  const void* gate_scales, const void* up_weight,
                                  const void* up_scales, const void* gate_bias,
                                  const void* up_bias, const void* out, const void* gate,
                                  const void* up, const void* workspace, int64_t workspace_bytes,
                                  int64_t M, int64_t N, int64_t K, int32_t dtype, int32_t act,
                                  const mhc_linear_launch* launch) {
  FwdPlan plan;
  return validate_fwd(x, x_scales, gate_weight, gate_scales, up_weight, up_scales, gate_bias,
                      up_bias, out, gate, up, workspace, workspace_bytes, M, N, K, dtype, act,
                      launch, &plan);
}

mhc_status mhc_gated_validate_bwd(const void* grad_out, const void* x, const void* gate_weight,
                                  const void* up_weight, const void* gate, const void* up,
                                  const void* grad_x, const void* grad_gate_weight,
                                  const void* grad_up_weight, const void* grad_gate_bias,
                                  const void* grad_up_bias, const void* workspace,
                                  int64_t workspace_bytes, int64_t M, int64_t N, int64_t K,
                                  int32_t dtype, int32_t act) {
  return validate_bwd(grad_out, x, gate_weight, up_weight, gate, up, grad_x, grad_gate_weight,
                      grad_up_weight, grad_gate_bias, grad_up_bias, workspace, workspace_bytes, M,
                      N, K, dtype, act);
}

mhc_status mhc_gated_fwd(const void* x, const void* x_scales, const void* gate_weight,
                         const void* gate_scales, const void* up_weight, const void* up_scales,
                         const void* gate_bias, const void* up_bias, void* out, void* gate,
                         void* up, void* workspace, int64_t workspace_bytes, int64_t M, int64_t N,
                         int64_t K, int32_t dtype, int32_t act, void* stream,
                         const mhc_linear_launch* launch, void* start_event, void* stop_event) {
  FwdPlan plan;
  const mhc_status st = validate_fwd(x, x_scales, gate_weight, gate_scales, up_weight, up_scales,
                                     gate_bias, up_bias, out, gate, up, workspace,
                                     workspace_bytes, M, N, K, dtype, act, launch, &plan);
  if (st != MHC_SUCCESS) return st;
  if (M == 0) return record_empty(stream, start_event, stop_event);
  Args a = {};
  const int64_t ld = K * elem(dtype);
  a.x = {x, M, ld};
  a.w = {gate_weight, N, ld};
  a.w2 = {up_weight, N, ld};
  if (dtype == MHC_LINEAR_E4M3_MX) {
    a.xs = static_cast<const uint8_t*>(x_scales);
    a.ws = static_cast<const uint8_t*>(gate_scales);
    a.ws2 = static_cast<const uint8_t*>(up_scales);
  } else {
    a.e.x_scales = static_cast<const float*>(x_scales);
    a.e.gate_scales = static_cast<const float*>(gate_scales);
    a.e.up_scales = static_cast<const float*>(up_scales);
  }
  a.M = M;
  a.N = N;
  a.kbytes = static_cast<uint32_t>(ld);
  a.e.gate_bias = gate_bias;
  a.e.up_bias = up_bias;
  a.e.out = out;
  a.e.gate = gate;
  a.e.up = up;
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
    case MHC_LINEAR_I8_ROW: e = launch_fwd<kOpI8>(a, plan, ws, s, b, f); break;
    default: e = launch_fwd<kOpMX>(a, plan, ws, s, b, f); break;
  }
  return launch_status(e, "gated launch");
}

mhc_status mhc_gated_bwd(const void* grad_out, const void* x, const void* gate_weight,
                         const void* up_weight, const void* gate, const void* up, void* grad_x,
                         void* grad_gate_weight, void* grad_up_weight, void* grad_gate_bias,
                         void* grad_up_bias, void* workspace, int64_t workspace_bytes, int64_t M,
                         int64_t N, int64_t K, int32_t dtype, int32_t act, void* stream,
                         void* start_event, void* stop_event) {
  const mhc_status st = validate_bwd(grad_out, x, gate_weight, up_weight, gate, up, grad_x,
                                     grad_gate_weight, grad_up_weight, grad_gate_bias,
                                     grad_up_bias, workspace, workspace_bytes, M, N, K, dtype, act);
  if (st != MHC_SUCCESS) return st;
  const BwdArgs a = {grad_out, x, gate_weight, up_weight, gate, up, grad_x, grad_gate_weight,
                     grad_up_weight, grad_gate_bias, grad_up_bias,
                     static_cast<uint8_t*>(workspace), M, N, K, act};
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const hipEvent_t b = static_cast<hipEvent_t>(start_event), f = static_cast<hipEvent_t>(stop_event);
  const hipError_t e = dtype == MHC_LINEAR_BF16 ? launch_bwd<kOpBF16>(a, dtype, s, b, f)
                                                : launch_bwd<kOpF16>(a, dtype, s, b, f);
  return launch_status(e, "gated backward launch");
}

}  // extern "C"
