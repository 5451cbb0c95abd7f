// Entry points of the operators around the recurrent layer (include/kda.h):
// argument checks on the host, then the launches.
#include <cuda_runtime.h>

#include "kda.h"
#include "kda_checks.h"
#include "kda_internal.h"
#include "kda_ops.h"

using namespace kda;

extern "C" kda_status kda_add_rms_norm(const void* x, int64_t ld_x, const void* residual,
                                       int64_t ld_residual, const void* weight, void* h,
                                       int64_t ld_h, void* y, int64_t ld_y, float* y_scale,
                                       int64_t ld_scale, int64_t rows, int32_t dim, float eps,
                                       kda_dtype dtype, kda_dtype weight_dtype, kda_dtype y_dtype,
                                       void* stream) {
  NvtxRange nvtx_range("kda_add_rms_norm");
  if (rows < 0 || dim <= 0)
    return bad(KDA_ERR_INVALID_ARGUMENT, "rows=%lld dim=%d", (long long)rows, dim);
  if (!float_type(dtype) || !float_type(weight_dtype))
    return bad(KDA_ERR_INVALID_ARGUMENT, "x and weight must be bf16 or f32");
  if (y_dtype != dtype && y_dtype != KDA_E4M3)
    return bad(KDA_ERR_INVALID_ARGUMENT, "y must have x's dtype or be e4m3");
  if (!(eps >= 0.0f)) return bad(KDA_ERR_INVALID_ARGUMENT, "eps=%g must not be negative", eps);
  if (dim > kMaxNormDim)
    return bad(KDA_ERR_UNSUPPORTED, "dim=%d exceeds %d", dim, kMaxNormDim);
  if (rows > 0x7fffffffLL)
    return bad(KDA_ERR_UNSUPPORTED, "rows=%lld exceed the grid", (long long)rows);
  if (rows == 0) return KDA_OK;
  const bool quant = y_dtype == KDA_E4M3;
  if (!x || !weight || !y)
    return bad(KDA_ERR_INVALID_ARGUMENT, "%s is NULL", !x ? "x" : !weight ? "weight" : "y");
  if (quant != (y_scale != nullptr))
    return bad(KDA_ERR_INVALID_ARGUMENT,
               quant ? "y_scale is NULL but y is e4m3" : "y_scale is given but y is not e4m3");
  if (residual && !h) return bad(KDA_ERR_INVALID_ARGUMENT, "residual is given but h is NULL");
  const int64_t es = size_of(dtype), ws = size_of(weight_dtype), ys = size_of(y_dtype);
  const int64_t groups = (dim + kScaleGroup - 1) / kScaleGroup;
  KDA_TRY(check_rows("x", x, ld_x, dim, es));
  KDA_TRY(check_rows("residual", residual, ld_residual, dim, es));
  KDA_TRY(check_rows("weight", weight, dim, dim, ws));
  KDA_TRY(check_rows("h", h, ld_h, dim, es));
  KDA_TRY(check_rows("y", y, ld_y, dim, ys));
  KDA_TRY(check_rows("y_scale", y_scale, ld_scale, groups, 4));
  const Rows in[] = {rows_of("x", x, rows, ld_x, dim, es),
                     rows_of("residual", residual, rows, ld_residual, dim, es),
                     rows_of("weight", weight, 1, dim, dim, ws)};
  const Rows out[] = {rows_of("h", h, rows, ld_h, dim, es), rows_of("y", y, rows, ld_y, dim, ys),
                      rows_of("y_scale", y_scale, rows, ld_scale, groups, 4)};
  // a row is read whole before its h or y is written: both may replace x or the residual
  KDA_TRY(check_output(out[0], in, 3, &in[0], &in[1]));
  KDA_TRY(check_output(out[1], in, 3, quant ? nullptr : &in[0], quant ? nullptr : &in[1]));
  KDA_TRY(check_output(out[2], in, 3, nullptr));
  KDA_TRY(check_output(out[1], &out[0], 1, nullptr));
  KDA_TRY(check_output(out[2], &out[0], 2, nullptr));

  NormArgs a;
  a.x = x; a.residual = residual; a.weight = weight; a.h = h; a.y = y; a.y_scale = y_scale;
  a.ld_x = ld_x;
  a.ld_res = residual ? ld_residual : 0;
  a.ld_h = ld_h; a.ld_y = ld_y; a.ld_scale = ld_scale;
  a.rows = rows; a.dim = dim; a.eps = eps;
  a.bf16 = dtype == KDA_BF16; a.w_bf16 = weight_dtype == KDA_BF16; a.quant = quant;
  auto wide = [&](const void* p, int64_t ld, int64_t size, int64_t bytes) {
    return !p || (aligned(p, static_cast<uintptr_t>(bytes)) && (rows == 1 || ld * size % bytes == 0));
  };
  a.vec = dim % 8 == 0 && wide(x, ld_x, es, 16) && wide(residual, ld_residual, es, 16) &&
          wide(h, ld_h, es, 16) && wide(y, ld_y, ys, quant ? 8 : 16) && aligned(weight, 16);
  KDA_TRY(device_sm_count(&a.sm_count));
  KDA_TRY(device_error_word(&a.err));
  return launched(launch_norm(a, static_cast<cudaStream_t>(stream)), "norm launch");
}

// The checks that the convolution's two entry points share.
static kda_status check_conv(const void* x, int64_t ld_x, const void* weight, const void* bias,
                             const void* state_in, const void* state_out, const int32_t* cu,
                             const void* y, int64_t ld_y, int64_t T, int32_t N, int32_t dim,
                             int32_t width, kda_dtype dtype, kda_dtype w_dtype, ConvArgs& a) {
  if (T < 0 || N < 0 || dim <= 0 || width <= 0)
    return bad(KDA_ERR_INVALID_ARGUMENT, "total_tokens=%lld n_seqs=%d dim=%d width=%d", (long long)T,
               N, dim, width);
  if (!float_type(dtype) || !float_type(w_dtype))
    return bad(KDA_ERR_INVALID_ARGUMENT, "x and weight must be bf16 or f32");
  if (width < 2 || width > kMaxConvWidth)
    return bad(KDA_ERR_UNSUPPORTED, "width=%d is not in [2, %d]", width, kMaxConvWidth);
  if (dim > (1 << 24)) return bad(KDA_ERR_UNSUPPORTED, "dim=%d exceeds %d", dim, 1 << 24);
  if (T > 0x7fffffffLL) return bad(KDA_ERR_UNSUPPORTED, "total_tokens=%lld", (long long)T);
  if (N == 0 && T > 0) return bad(KDA_ERR_INVALID_ARGUMENT, "tokens given but n_seqs = 0");
  if (!cu && N > 0 && T % N != 0)
    return bad(KDA_ERR_INVALID_ARGUMENT,
               "cu_seqlens is NULL but total_tokens=%lld is not a multiple of n_seqs=%d",
               (long long)T, N);
  if (N == 0) return KDA_OK;
  const struct { const void* p; const char* n; } req[] = {{x, "x"}, {weight, "weight"}, {y, "y"}};
  if (T > 0)
    for (auto& r : req)
      if (!r.p) return bad(KDA_ERR_INVALID_ARGUMENT, "%s is NULL", r.n);
  const int64_t es = size_of(dtype), ws = size_of(w_dtype), rows = static_cast<int64_t>(N) * (width - 1);
  KDA_TRY(check_rows("x", x, ld_x, dim, es));
  KDA_TRY(check_rows("weight", weight, width, width, ws));
  KDA_TRY(check_rows("bias", bias, dim, dim, ws));
  KDA_TRY(check_rows("state_in", state_in, dim, dim, es));
  KDA_TRY(check_rows("state_out", state_out, dim, dim, es));
  KDA_TRY(check_rows("cu_seqlens", cu, 1, 1, 4));
  KDA_TRY(check_rows("y", y, ld_y, dim, es));
  const Rows in[] = {rows_of("x", x, T, ld_x, dim, es),
                     rows_of("weight", weight, 1, static_cast<int64_t>(dim) * width,
                             static_cast<int64_t>(dim) * width, ws),
                     rows_of("bias", bias, 1, dim, dim, ws),
                     rows_of("state_in", state_in, 1, rows * dim, rows * dim, es),
                     rows_of("cu_seqlens", cu, 1, N + 1LL, N + 1LL, 4)};
  const Rows out[] = {rows_of("state_out", state_out, 1, rows * dim, rows * dim, es),
                      rows_of("y", y, T, ld_y, dim, es)};
  KDA_TRY(check_output(out[0], in, 5, &in[3]));  // the state may be continued in place
  KDA_TRY(check_output(out[1], in, 5, nullptr));
  KDA_TRY(check_output(out[1], &out[0], 1, nullptr));
  a.x = x; a.weight = weight; a.bias = bias; a.state_in = state_in;
  a.state_out = const_cast<void*>(state_out);
  a.cu = cu; a.y = const_cast<void*>(y);
  a.ld_x = ld_x; a.ld_y = ld_y; a.T = T; a.N = N; a.dim = dim; a.width = width;
  a.bf16 = dtype == KDA_BF16; a.w_bf16 = w_dtype == KDA_BF16;
  a.vec = 4;
  auto fits = [&](int v) {
    const uintptr_t to = static_cast<uintptr_t>(v * es);
    return dim % v == 0 && ld_x % v == 0 && ld_y % v == 0 && aligned(x, to) && aligned(y, to) &&
           aligned(state_in, to) && aligned(state_out, to) &&
           aligned(weight, static_cast<uintptr_t>(v * ws));
  };
  while (a.vec > 1 && !fits(a.vec)) a.vec /= 2;
  KDA_TRY(device_sm_count(&a.sm_count));
  return device_error_word(&a.err);
}

extern "C" kda_status kda_short_conv_fwd(const void* x, int64_t ld_x, const void* weight,
                                         const void* bias, const void* state_in, void* state_out,
                                         const int32_t* cu_seqlens, void* y, int64_t ld_y,
                                         int64_t total_tokens, int32_t n_seqs, int32_t dim,
                                         int32_t width, int32_t activation, kda_dtype dtype,
                                         kda_dtype weight_dtype, void* stream) {
  NvtxRange nvtx_range("kda_short_conv_fwd");
  ConvArgs a;
  KDA_TRY(check_conv(x, ld_x, weight, bias, state_in, state_out, cu_seqlens, y, ld_y, total_tokens,
                     n_seqs, dim, width, dtype, weight_dtype, a));
  if (n_seqs == 0) return KDA_OK;
  a.silu = activation != 0;
  return launched(launch_conv(a, static_cast<cudaStream_t>(stream)), "convolution launch");
}

extern "C" kda_status kda_short_conv_step(const void* x, int64_t ld_x, const void* weight,
                                          const void* bias, void* state, void* y, int64_t ld_y,
                                          int32_t n_seqs, int32_t dim, int32_t width,
                                          int32_t activation, kda_dtype dtype,
                                          kda_dtype weight_dtype, void* stream) {
  NvtxRange nvtx_range("kda_short_conv_step");
  if (n_seqs > 0 && !state) return bad(KDA_ERR_INVALID_ARGUMENT, "state is NULL");
  ConvArgs a;
  KDA_TRY(check_conv(x, ld_x, weight, bias, state, state, nullptr, y, ld_y, n_seqs, n_seqs, dim,
                     width, dtype, weight_dtype, a));
  if (n_seqs == 0) return KDA_OK;
  a.silu = activation != 0;
  return launched(launch_conv_step(a, static_cast<cudaStream_t>(stream)), "convolution launch");
}

// The checks that the scan's two entry points share; h_in may be h_out itself.
static kda_status check_ssm(const void* x, int64_t ld_x, const void* dt, int64_t ld_dt,
                            const float* A, const void* B, int64_t ld_b, const void* C,
                            int64_t ld_c, const float* D, const void* z, int64_t ld_z,
                            const float* dt_bias, const float* h_in, const char* h_in_name,
                            float* h_out, const int32_t* cu, void* y, int64_t ld_y, int64_t T,
                            int32_t N, int32_t dim, int32_t state, int32_t groups, kda_dtype dtype,
                            SsmArgs& a) {
  if (T < 0 || N < 0 || dim <= 0 || state <= 0 || groups <= 0)
    return bad(KDA_ERR_INVALID_ARGUMENT, "total_tokens=%lld n_seqs=%d dim=%d state=%d groups=%d",
               (long long)T, N, dim, state, groups);
  if (!float_type(dtype)) return bad(KDA_ERR_INVALID_ARGUMENT, "x must be bf16 or f32");
  if (state != 16 && state != 32 && state != 64 && state != 128)
    return bad(KDA_ERR_UNSUPPORTED, "state=%d is not 16, 32, 64 or 128", state);
  if (dim % groups != 0)
    return bad(KDA_ERR_INVALID_ARGUMENT, "dim=%d is not a multiple of groups=%d", dim, groups);
  if (dim > (1 << 24)) return bad(KDA_ERR_UNSUPPORTED, "dim=%d exceeds %d", dim, 1 << 24);
  if (T > 0x7fffffffLL) return bad(KDA_ERR_UNSUPPORTED, "total_tokens=%lld", (long long)T);
  if (N == 0 && T > 0) return bad(KDA_ERR_INVALID_ARGUMENT, "tokens given but n_seqs = 0");
  if (!cu && N > 0 && T % N != 0)
    return bad(KDA_ERR_INVALID_ARGUMENT,
               "cu_seqlens is NULL but total_tokens=%lld is not a multiple of n_seqs=%d",
               (long long)T, N);
  if (N == 0) return KDA_OK;
  const struct { const void* p; const char* n; } req[] = {
      {x, "x"}, {dt, "dt"}, {A, "A"}, {B, "B"}, {C, "C"}, {y, "y"}};
  if (T > 0)
    for (auto& r : req)
      if (!r.p) return bad(KDA_ERR_INVALID_ARGUMENT, "%s is NULL", r.n);
  const int64_t es = size_of(dtype), gs = static_cast<int64_t>(groups) * state;
  const int64_t rates = static_cast<int64_t>(dim) * state, states = rates * N;
  const Rows in[] = {rows_of("x", x, T, ld_x, dim, es), rows_of("dt", dt, T, ld_dt, dim, es),
                     rows_of("A", A, 1, rates, rates, 4), rows_of("B", B, T, ld_b, gs, es),
                     rows_of("C", C, T, ld_c, gs, es), rows_of("D", D, 1, dim, dim, 4),
                     rows_of("z", z, T, ld_z, dim, es), rows_of("dt_bias", dt_bias, 1, dim, dim, 4),
                     rows_of(h_in_name, h_in, 1, states, states, 4),
                     rows_of("cu_seqlens", cu, 1, N + 1LL, N + 1LL, 4)};
  const Rows out[] = {rows_of("h_final", h_out, 1, states, states, 4), rows_of("y", y, T, ld_y, dim, es)};
  const int64_t lds[] = {ld_x, ld_dt, rates, ld_b, ld_c, dim, ld_z, dim, states, N + 1LL, states, ld_y};
  const int64_t cols[] = {dim, dim, rates, gs, gs, dim, dim, dim, states, N + 1LL, states, dim};
  for (int i = 0; i < 12; ++i) {
    const Rows& r = i < 10 ? in[i] : out[i - 10];
    KDA_TRY(check_rows(r.name, r.p, lds[i], cols[i], cols[i] > 0 ? r.width / cols[i] : 1));
  }
  if (!aligned(h_in, 16) || !aligned(h_out, 16))
    return bad(KDA_ERR_INVALID_ARGUMENT, "%s is not 16-byte aligned",
               !aligned(h_in, 16) ? h_in_name : "h_final");
  KDA_TRY(check_output(out[0], in, 10, &in[8]));  // the states may be continued in place
  KDA_TRY(check_output(out[1], in, 10, nullptr));
  KDA_TRY(check_output(out[1], &out[0], 1, nullptr));
  a.x = x; a.dt = dt; a.z = z; a.B = B; a.C = C; a.A = A; a.D = D; a.dt_bias = dt_bias;
  a.h0 = h_in; a.h_out = h_out; a.cu = cu; a.y = y;
  a.ld_x = ld_x; a.ld_dt = ld_dt; a.ld_z = ld_z; a.ld_b = ld_b; a.ld_c = ld_c; a.ld_y = ld_y;
  a.T = T; a.N = N; a.dim = dim; a.state = state; a.groups = groups;
  a.bf16 = dtype == KDA_BF16;
  a.vec = aligned(A, 16) && aligned(B, static_cast<uintptr_t>(4 * es)) && ld_b % 4 == 0 &&
          aligned(C, static_cast<uintptr_t>(4 * es)) && ld_c % 4 == 0;
  auto even = [&](const void* p, int64_t ld) {
    return !p || (aligned(p, static_cast<uintptr_t>(2 * es)) && ld % 2 == 0);
  };
  a.pairs = a.vec && dim / groups % 2 == 0 && even(x, ld_x) && even(dt, ld_dt) && even(z, ld_z) && even(y, ld_y);
  KDA_TRY(device_sm_count(&a.sm_count));
  return device_error_word(&a.err);
}

extern "C" kda_status kda_ssm_scan_fwd(const void* x, int64_t ld_x, const void* dt, int64_t ld_dt,
                                       const float* A, const void* B, int64_t ld_b, const void* C,
                                       int64_t ld_c, const float* D, const void* z, int64_t ld_z,
                                       const float* dt_bias, const float* h0,
                                       const int32_t* cu_seqlens, void* y, int64_t ld_y,
                                       float* h_final, int64_t total_tokens, int32_t n_seqs,
                                       int32_t dim, int32_t state, int32_t groups,
                                       int32_t dt_softplus, kda_dtype dtype, void* stream) {
  NvtxRange nvtx_range("kda_ssm_scan_fwd");
  SsmArgs a;
  KDA_TRY(check_ssm(x, ld_x, dt, ld_dt, A, B, ld_b, C, ld_c, D, z, ld_z, dt_bias, h0, "h0", h_final,
                    cu_seqlens, y, ld_y, total_tokens, n_seqs, dim, state, groups, dtype, a));
  if (n_seqs == 0) return KDA_OK;
  a.softplus = dt_softplus != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  bool cut = false;
  ssm_chunks(a, cut);
  if (!cut) return launched(launch_ssm_scan(a, false, s), "scan launch");
  // Workspace: the chunks' states and step sums, and, where the states are
  // continued in place, a copy of h0: a block that ends a sequence may write
  // its state before the block that begins it has read the old one.
  const int64_t row = a.dim, chunk_h = a.n_chunks * row * a.state;
  const int64_t dts = (a.n_chunks * row + 3) / 4 * 4;
  const int64_t copy = h0 && h0 == h_final ? static_cast<int64_t>(a.N) * row * a.state : 0;
  void* ws = nullptr;
  KDA_TRY(workspace_alloc(static_cast<size_t>(chunk_h + dts + copy) * sizeof(float), s, &ws));
  a.chunk_h = static_cast<float*>(ws);
  a.chunk_dt = a.chunk_h + chunk_h;
  cudaError_t e = cudaSuccess;
  if (copy) {
    float* old = a.chunk_dt + dts;
    e = cudaMemcpyAsync(old, h0, static_cast<size_t>(copy) * sizeof(float), cudaMemcpyDeviceToDevice, s);
    a.h0 = old;
  }
  if (e == cudaSuccess) e = launch_ssm_scan(a, true, s);
  const cudaError_t ef = cudaFreeAsync(ws, s);
  return launched(e != cudaSuccess ? e : ef, "scan launch");
}

extern "C" kda_status kda_ssm_scan_step(const void* x, int64_t ld_x, const void* dt, int64_t ld_dt,
                                        const float* A, const void* B, int64_t ld_b, const void* C,
                                        int64_t ld_c, const float* D, const void* z, int64_t ld_z,
                                        const float* dt_bias, float* h, void* y, int64_t ld_y,
                                        int32_t n_seqs, int32_t dim, int32_t state, int32_t groups,
                                        int32_t dt_softplus, kda_dtype dtype, void* stream) {
  NvtxRange nvtx_range("kda_ssm_scan_step");
  if (n_seqs > 0 && !h) return bad(KDA_ERR_INVALID_ARGUMENT, "h is NULL");
  SsmArgs a;
  KDA_TRY(check_ssm(x, ld_x, dt, ld_dt, A, B, ld_b, C, ld_c, D, z, ld_z, dt_bias, h, "h", h, nullptr,
                    y, ld_y, n_seqs, n_seqs, dim, state, groups, dtype, a));
  if (n_seqs == 0) return KDA_OK;
  a.softplus = dt_softplus != 0;
  return launched(launch_ssm_step(a, static_cast<cudaStream_t>(stream)), "scan step launch");
}

extern "C" kda_status kda_matmul_fp8(const void* a, int64_t ld_a, const float* a_scale,
                                     int64_t ld_a_scale, const void* b, int64_t ld_b,
                                     const float* b_scale, int64_t ld_b_scale, void* out,
                                     int64_t ld_out, int32_t M, int32_t N, int32_t K,
                                     kda_dtype out_dtype, void* stream) {
  NvtxRange nvtx_range("kda_matmul_fp8");
  if (M < 0 || N < 0 || K <= 0) return bad(KDA_ERR_INVALID_ARGUMENT, "M=%d N=%d K=%d", M, N, K);
  if (!float_type(out_dtype)) return bad(KDA_ERR_INVALID_ARGUMENT, "out must be bf16 or f32");
  if (M == 0 || N == 0) return KDA_OK;
  const struct { const void* p; const char* n; } req[] = {
      {a, "a"}, {a_scale, "a_scale"}, {b, "b"}, {b_scale, "b_scale"}, {out, "out"}};
  for (auto& r : req)
    if (!r.p) return bad(KDA_ERR_INVALID_ARGUMENT, "%s is NULL", r.n);
  const int64_t kb = (K + kScaleGroup - 1) / kScaleGroup, nb = (N + kScaleGroup - 1) / kScaleGroup;
  const int64_t os = size_of(out_dtype);
  KDA_TRY(check_rows("a", a, ld_a, K, 1));
  KDA_TRY(check_rows("a_scale", a_scale, ld_a_scale, kb, 4));
  KDA_TRY(check_rows("b", b, ld_b, K, 1));
  KDA_TRY(check_rows("b_scale", b_scale, ld_b_scale, kb, 4));
  KDA_TRY(check_rows("out", out, ld_out, N, os));
  // (a single row has no next one, whatever its distance)
  if (M == 1) ld_a = (ld_a + 15) / 16 * 16;
  if (N == 1) ld_b = (ld_b + 15) / 16 * 16;
  const struct { const void* p; int64_t ld; const char* n; } wide[] = {{a, ld_a, "a"}, {b, ld_b, "b"}};
  for (auto& w : wide)  // the tensor copies' rule
    if (!aligned(w.p, 16) || w.ld % 16 != 0)
      return bad(KDA_ERR_INVALID_ARGUMENT, "%s: every row must start on a 16-byte boundary", w.n);
  const Rows in[] = {rows_of("a", a, M, ld_a, K, 1), rows_of("a_scale", a_scale, M, ld_a_scale, kb, 4),
                     rows_of("b", b, N, ld_b, K, 1),
                     rows_of("b_scale", b_scale, nb, ld_b_scale, kb, 4)};
  KDA_TRY(check_output(rows_of("out", out, M, ld_out, N, os), in, 4, nullptr));
  MatmulArgs m;
  m.a = a; m.a_scale = a_scale; m.b = b; m.b_scale = b_scale; m.out = out;
  m.ld_a = ld_a; m.ld_as = ld_a_scale; m.ld_b = ld_b; m.ld_bs = ld_b_scale; m.ld_out = ld_out;
  m.M = M; m.N = N; m.K = K;
  m.bf16 = out_dtype == KDA_BF16;
  KDA_TRY(device_sm_count(&m.sm_count));
  KDA_TRY(device_error_word(&m.err));
  return launched(launch_matmul_fp8(m, static_cast<cudaStream_t>(stream)), "product launch");
}
