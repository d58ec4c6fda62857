// mhc_linear.hip - matrix product with bias, activation and residual in its
// epilogue, and its backward, for gfx950 (see include/mhc_linear.h for the
// operation).

#include "mhc_linear.h"

#include <math.h>

#include "mhc_tiles_host.h"

#ifdef __FAST_MATH__
#error "this source must not be built with fast-math"
#endif

#pragma clang fp contract(off)

namespace {

// Epilogue: scales, bias, activation and residual.
struct Epilogue {
  static constexpr int kW = kOne, kSums = 1, kGroup = 0;
  static constexpr bool kSplits = true, kHalves = false, kTakes = false, kWrites = true, kEarly = true;
  const void* bias;
  const void* residual;
  void* out;
  void* z;
  const float* x_scales;       // where the type has scales of rows
  const float* weight_scales;
  int64_t N;                   // row stride of residual, out and z
  int32_t act;

  template <int OP, class Fn>
  __device__ __forceinline__ void with(const Fn& fn) const;
};

// The values as they are, in fp32: an instruction that multiplies and rounds to fp16 at
// once, which the compiler takes at the end of a wide tile and nowhere else, rounds once
// where a product in fp32 and its conversion round twice, and a row is to be the same
// from every kernel, bit for bit (elsewhere this would keep loops from being unrolled).
template <int F>
__device__ __forceinline__ void in_fp32(float (&v)[8]) {
  if constexpr (F == kF16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("" : "+v"(v[i]));
  }
}

// Columns [n, n + count) of row m, count <= 8, from the sums over k; bias_of() and
// residual_of() bring those chunks, where there are any. FENCE: see in_fp32.
template <int OP, int ACT, bool FENCE, class B, class R>
__device__ __forceinline__ void finish(const Epilogue& e, int64_t m, int64_t n, int count, float (&v)[8],
                                       const B& bias_of, const R& residual_of) {
  constexpr int F = out_format(OP);
  typedef typename Store<F>::type S;
  float b[8];
  if constexpr (scaled(OP)) {
    const float xs = e.x_scales[m];
    widen_chunk<kF32>(load_chunk<kF32>(e.weight_scales + n, count), b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = sum_value<OP>(v[i]) * (xs * b[i]);
  }
  if (e.bias != nullptr) {
    widen_chunk<F>(bias_of(), b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] + b[i];
  }
  Chunk<F> c;
  if (e.z != nullptr) {
    if constexpr (FENCE) in_fp32<F>(v);
    narrow_chunk<F>(v, c);
    store_chunk<F>(static_cast<S*>(e.z) + m * e.N + n, count, c);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = activate<ACT>(v[i]);
  if (e.residual != nullptr) {
    widen_chunk<F>(residual_of(), b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] + b[i];
  }
  if constexpr (FENCE) in_fp32<F>(v);
  narrow_chunk<F>(v, c);
  store_chunk<F>(static_cast<S*>(e.out) + m * e.N + n, count, c);
}

template <int OP, int ACT>
struct Finish {
  static constexpr int F = out_format(OP);
  typedef typename Store<F>::type S;
  const Epilogue& e;
  __device__ __forceinline__ void operator()(int64_t m, int64_t n, int count, float (&v)[8]) const {
    finish<OP, ACT, false>(e, m, n, count, v, [&] { return load_chunk<F>(static_cast<const S*>(e.bias) + n, count); },
                           [&] { return load_chunk<F>(static_cast<const S*>(e.residual) + m * e.N + n, count); });
  }
  __device__ __forceinline__ void operator()(int64_t m, int64_t n, int count, float (&v)[8], const u32x4& bias,
                                             const u32x4& residual) const {
    finish<OP, ACT, true>(e, m, n, count, v, [&] { return Chunk<F>{{bias}}; }, [&] { return Chunk<F>{{residual}}; });
  }
};

template <int OP, class Fn>
__device__ __forceinline__ void Epilogue::with(const Fn& fn) const {
  with_act(act, [&](auto a) { fn(Finish<OP, decltype(a)::value>{*this}); });
}

typedef TileArgs<Epilogue> Args;

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


mhc_status check_sizes(int64_t M, int64_t N, int64_t K, int32_t dtype) {
  if (M < 0 || M > INT32_MAX) return fail(MHC_ERROR_INVALID_VALUE, "M must be in [0, 2^31 - 1]");
  if (N < 1 || N > INT32_MAX) return fail(MHC_ERROR_INVALID_VALUE, "N must be in [1, 2^31 - 1]");
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


// The forward's launch. Sums of 8-bit integers are the same in every launch, so
// theirs may be the fastest; the narrow kernel has no rival at few columns.
mhc_status plan_launch(int64_t M, int64_t N, int64_t K, int32_t dtype, const mhc_linear_launch* launch,
                       mhc_linear_launch* p) {
  return dtype == MHC_LINEAR_I8_ROW && N > 32 ? best_plan(M, N, K, dtype, false, 32, launch, p)
                                              : make_plan(M, N, K, dtype, launch, p);
}

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
  if ((st = plan_launch(M, N, K, dtype, launch, &chosen)) != MHC_SUCCESS) return st;
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
  const bool row = scaled(dtype);
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

template <int OP>
hipError_t launch_fwd(Args a, const FwdPlan& p, uint8_t* workspace, hipStream_t s,
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
      Args t = {};
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
      Args t = {};
      t.x = {gz, a.N, p.ldn};
      t.w = {x, a.K, p.ldk};
      t.M = a.N; t.N = a.K;
      t.kbytes = t.kturned = static_cast<uint32_t>(a.M * 2);
      t.partial = reinterpret_cast<float*>(a.ws + p.part);
      t.e.out = a.gw; t.e.N = a.K;
      e = launch_product<OP, true, true>(t, p.pw, s, marks.first(), nullptr);
    }
  }
  return marks.end(e, s);
}

}  // namespace

extern "C" {

int mhc_linear_abi_version(void) { return MHC_LINEAR_ABI_VERSION; }

const char* mhc_linear_last_error_message(void) { return g_msg; }

mhc_status mhc_linear_plan(int64_t M, int64_t N, int64_t K, int32_t dtype,
                           const mhc_linear_launch* launch, mhc_linear_launch* plan) {
  mhc_linear_launch p;
  mhc_status st = check_sizes(M, N, K, dtype);
  if (st == MHC_SUCCESS) st = plan_launch(M, N, K, dtype, launch, &p);
  if (st == MHC_SUCCESS && plan != nullptr) *plan = p;
  return st;
}

int64_t mhc_linear_fwd_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t dtype,
                                       const mhc_linear_launch* launch) {
  mhc_linear_launch p;
  if (check_sizes(M, N, K, dtype) != MHC_SUCCESS ||
      plan_launch(M, N, K, dtype, launch, &p) != MHC_SUCCESS)
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
  Args a = {};
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
    case MHC_LINEAR_I8_ROW: e = launch_fwd<kOpI8>(a, plan, ws, s, b, f); break;
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