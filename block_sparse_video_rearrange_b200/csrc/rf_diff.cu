// Host side of the differential-attention calls (checks and workspace layout),
// and lambda with its gradient.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <string>

#include "rf_async.cuh"
#include "rf_device.cuh"

RfDiffLayout rf_diff_layout(const rf_plan* p) {
  const RfGeomDev& g = p->g;
  auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  RfDiffLayout l;
  int longest = 0;
  for (int i = 0; i < g.n_seqs; ++i) {
    const int n = g.seq[i].n_pb + g.seq[i].nb;
    if (n > longest) longest = n;
  }
  l.words = (longest + 31) / 32;
  const int64_t qb = g.t_qblk;
  l.v16 = up(p->ws_bytes);
  l.v_exp = up(l.v16 + (int64_t)g.n2 * qb * RF_BLOCK * g.d * 2);
  l.end_serve = up(l.v_exp + (int64_t)g.n2 * qb * 4);
  l.stats = l.end_serve;
  l.bits = up(l.stats + (int64_t)g.n1 * qb * 4 * RF_BLOCK * 4);
  l.dlam = up(l.bits + (int64_t)g.n1 * qb * l.words * 4);
  l.do_row = up(l.dlam + (int64_t)g.n1 * qb * 4);
  const bool f16 = p->dtype == RF_FP16;
  l.do_blk = up(l.do_row + (f16 ? (int64_t)g.n1 * qb * RF_BLOCK * 4 : 0));
  l.v_blk = up(l.do_blk + (f16 ? (int64_t)g.n1 * qb * 8 : 0));
  l.end = up(l.v_blk + (f16 ? (int64_t)g.n2 * qb * 4 : 0));
  return l;
}

namespace {

bool aligned16(const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15) == 0; }

rf_status_t check_plan(const rf_plan_t* p) {
  if (!p) return rf_fail(RF_ERR_INVALID_ARG, "null plan");
  if (p->precision != RF_PRECISION_NATIVE)
    return rf_fail(RF_ERR_UNSUPPORTED, "differential attention is built for native precision only");
  if (p->g.block_kv != RF_BLOCK)
    return rf_fail(RF_ERR_UNSUPPORTED, "differential attention is built for blockShape 128 x 128 only");
  return RF_OK;
}

rf_status_t check_ws(const void* ws, size_t ws_bytes, int64_t need) {
  if (!ws) return rf_fail(RF_ERR_INVALID_ARG, "null workspace");
  if ((reinterpret_cast<uintptr_t>(ws) & 255) != 0)
    return rf_fail(RF_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if ((uint64_t)ws_bytes < (uint64_t)need)
    return rf_fail(RF_ERR_WORKSPACE_TOO_SMALL, "workspace needs " + std::to_string(need) + " bytes");
  return RF_OK;
}

rf_status_t check_scale(float scale) {
  if (!(scale > 0.0f) || !std::isfinite(scale))
    return rf_fail(RF_ERR_INVALID_ARG, "scale must be finite and > 0");
  return RF_OK;
}

// ---- lambda ---------------------------------------------------------------

__device__ __forceinline__ float load_f(const void* p, int dt, size_t i) {
  if (dt == RF_FP32) return static_cast<const float*>(p)[i];
  if (dt == RF_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void store_f(void* p, int dt, size_t i, float v) {
  if (dt == RF_FP32) static_cast<float*>(p)[i] = v;
  else if (dt == RF_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

struct LambdaArgs {
  const void *a, *b, *c, *d;
  int dt, vec_heads, dim, heads;
  float init;
};

// The two exponentials of vector row `row`, on every lane of the warp.
__device__ __forceinline__ void lambda_exps(const LambdaArgs& x, int row, int lane, float& e1, float& e2) {
  float s1 = 0.f, s2 = 0.f;
  for (int i = lane; i < x.dim; i += 32) {
    const size_t at = (size_t)row * x.dim + i;
    s1 = fmaf(load_f(x.a, x.dt, at), load_f(x.b, x.dt, at), s1);
    s2 = fmaf(load_f(x.c, x.dt, at), load_f(x.d, x.dt, at), s2);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s1 += __shfl_xor_sync(0xffffffffu, s1, o);
    s2 += __shfl_xor_sync(0xffffffffu, s2, o);
  }
  e1 = expf(s1);
  e2 = expf(s2);
}

// One warp per vector row; a row shared by every head writes every lambda.
// Latency-bound: a few kilobytes, one launch.
__global__ void __launch_bounds__(128) rf_diff_lambda_kernel(const __grid_constant__ LambdaArgs x, float* lambda) {
  wait_for_previous();
  const int row = (int)((blockIdx.x * 128 + threadIdx.x) >> 5), lane = threadIdx.x & 31;
  if (row >= x.vec_heads) return;
  float e1, e2;
  lambda_exps(x, row, lane, e1, e2);
  const float lam = e1 - e2 + x.init;
  if (x.vec_heads == x.heads) {
    if (lane == 0) lambda[row] = lam;
  } else {
    for (int h = lane; h < x.heads; h += 32) lambda[h] = lam;
  }
}

// d lambda / d a = e1 b and so on; vectors shared by every head take the sum of
// dlambda over the heads (in a fixed order).
__global__ void __launch_bounds__(128)
    rf_diff_lambda_bwd_kernel(const __grid_constant__ LambdaArgs x, const float* dlambda, void* da,
                              void* db, void* dc, void* dd) {
  wait_for_previous();
  const int row = (int)((blockIdx.x * 128 + threadIdx.x) >> 5), lane = threadIdx.x & 31;
  if (row >= x.vec_heads) return;
  float g = 0.f;
  if (x.vec_heads == x.heads) {
    g = dlambda[row];
  } else {
    for (int h = lane; h < x.heads; h += 32) g += dlambda[h];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) g += __shfl_xor_sync(0xffffffffu, g, o);
  }
  float e1, e2;
  lambda_exps(x, row, lane, e1, e2);
  const float g1 = g * e1, g2 = -g * e2;
  for (int i = lane; i < x.dim; i += 32) {
    const size_t at = (size_t)row * x.dim + i;
    const float a = load_f(x.a, x.dt, at), b = load_f(x.b, x.dt, at);
    const float c = load_f(x.c, x.dt, at), d = load_f(x.d, x.dt, at);
    store_f(da, x.dt, at, g1 * b);
    store_f(db, x.dt, at, g1 * a);
    store_f(dc, x.dt, at, g2 * d);
    store_f(dd, x.dt, at, g2 * c);
  }
}

rf_status_t check_lambda(const void* a, const void* b, const void* c, const void* d, int32_t dtype, int32_t vec_heads,
                         int32_t dim, int32_t heads, float init) {
  if (!a || !b || !c || !d) return rf_fail(RF_ERR_INVALID_ARG, "null vector");
  if (dtype != RF_BF16 && dtype != RF_FP16 && dtype != RF_FP32)
    return rf_fail(RF_ERR_INVALID_ARG, "dtype must be bf16, fp16 or fp32");
  if (heads < 1 || dim < 1) return rf_fail(RF_ERR_INVALID_ARG, "heads and dim must be > 0");
  if (vec_heads != 1 && vec_heads != heads)
    return rf_fail(RF_ERR_INVALID_ARG, "the vectors must have one row, or one per head");
  if (!std::isfinite(init)) return rf_fail(RF_ERR_INVALID_ARG, "lambda_init must be finite");
  return RF_OK;
}

}  // namespace

extern "C" {

rf_status_t rf_diff_lambda(const void* a, const void* b, const void* c, const void* d, rf_dtype_t dtype,
                           int32_t vec_heads, int32_t dim, int32_t heads, float lambda_init, float* lambda,
                           rf_stream_t stream) {
  rf_clear_error();
  rf_status_t st = check_lambda(a, b, c, d, dtype, vec_heads, dim, heads, lambda_init);
  if (st != RF_OK) return st;
  if (!lambda) return rf_fail(RF_ERR_INVALID_ARG, "null lambda");
  if ((st = rf_require_device()) != RF_OK) return st;
  const LambdaArgs x{a, b, c, d, dtype, vec_heads, dim, heads, lambda_init};
  return rf_launch_dependent(rf_diff_lambda_kernel, dim3((unsigned)((vec_heads + 3) / 4)), 128, (cudaStream_t)stream,
                             "rf_diff_lambda_kernel", x, lambda);
}

rf_status_t rf_diff_lambda_backward(const void* a, const void* b, const void* c, const void* d, rf_dtype_t dtype,
                                    int32_t vec_heads, int32_t dim, int32_t heads, const float* dlambda, void* da,
                                    void* db, void* dc, void* dd, rf_stream_t stream) {
  rf_clear_error();
  rf_status_t st = check_lambda(a, b, c, d, dtype, vec_heads, dim, heads, 0.f);
  if (st != RF_OK) return st;
  if (!dlambda || !da || !db || !dc || !dd) return rf_fail(RF_ERR_INVALID_ARG, "null gradient");
  if ((st = rf_require_device()) != RF_OK) return st;
  const LambdaArgs x{a, b, c, d, dtype, vec_heads, dim, heads, 0.f};
  return rf_launch_dependent(rf_diff_lambda_bwd_kernel, dim3((unsigned)((vec_heads + 3) / 4)), 128, (cudaStream_t)stream,
                             "rf_diff_lambda_bwd_kernel", x, dlambda, da, db, dc, dd);
}

rf_status_t rf_diff_attn_workspace_bytes(const rf_plan_t* p, int32_t backward, int64_t* out) {
  rf_clear_error();
  rf_status_t st = check_plan(p);
  if (st != RF_OK) return st;
  if (!out) return rf_fail(RF_ERR_INVALID_ARG, "null out");
  const RfDiffLayout l = rf_diff_layout(p);
  *out = backward ? l.end : l.end_serve;
  return RF_OK;
}

rf_status_t rf_diff_attn(const rf_plan_t* p, const void* q_r, const void* k_r, const void* v_r,
                         const int32_t* select_idx, const int32_t* select_num, const float* lambda, float scale,
                         void* o_r, float* maps, float* lse, void* ws, size_t ws_bytes, rf_stream_t stream) {
  rf_clear_error();
  rf_status_t st = check_plan(p);
  if (st != RF_OK) return st;
  if (!q_r || !k_r || !v_r || !o_r || !select_idx || !select_num || !lambda)
    return rf_fail(RF_ERR_INVALID_ARG, "null tensor");
  if (!aligned16(q_r) || !aligned16(k_r) || !aligned16(v_r) || !aligned16(o_r) || !aligned16(maps))
    return rf_fail(RF_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
  if (o_r == q_r || o_r == k_r || o_r == v_r) return rf_fail(RF_ERR_INVALID_ARG, "o_r aliases an input");
  if (!maps != !lse) return rf_fail(RF_ERR_INVALID_ARG, "maps and lse are kept together or not at all");
  if ((st = check_scale(scale)) != RF_OK) return st;
  if ((st = check_ws(ws, ws_bytes, rf_diff_layout(p).end_serve)) != RF_OK) return st;
  if ((st = rf_require_device()) != RF_OK) return st;
  return rf_launch_diff_attn(p, q_r, k_r, v_r, select_idx, select_num, lambda, scale, o_r, maps, lse, ws,
                             (cudaStream_t)stream);
}

rf_status_t rf_diff_attn_backward(const rf_plan_t* p, const void* q_r, const void* k_r, const void* v_r,
                                  const int32_t* select_idx, const int32_t* select_num, const float* lambda,
                                  float scale, const float* maps, const float* lse, const void* do_r, void* dq_r,
                                  void* dk_r, void* dv_r, float* dlambda, void* ws, size_t ws_bytes,
                                  rf_stream_t stream) {
  rf_clear_error();
  rf_status_t st = check_plan(p);
  if (st != RF_OK) return st;
  const void* in[] = {q_r, k_r, v_r, maps, do_r};
  void* out[] = {dq_r, dk_r, dv_r};
  if (!select_idx || !select_num || !lambda || !lse || !dlambda) return rf_fail(RF_ERR_INVALID_ARG, "null tensor");
  for (const void* x : in)
    if (!x) return rf_fail(RF_ERR_INVALID_ARG, "null tensor");
  for (void* y : out) {
    if (!y) return rf_fail(RF_ERR_INVALID_ARG, "null gradient");
    if (!aligned16(y)) return rf_fail(RF_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
    for (const void* x : in)
      if (x == y) return rf_fail(RF_ERR_INVALID_ARG, "a gradient aliases an input");
  }
  if (dq_r == dk_r || dq_r == dv_r || dk_r == dv_r) return rf_fail(RF_ERR_INVALID_ARG, "two gradients alias");
  for (const void* x : in)
    if (!aligned16(x)) return rf_fail(RF_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
  if ((st = check_scale(scale)) != RF_OK) return st;
  if ((st = check_ws(ws, ws_bytes, rf_diff_layout(p).end)) != RF_OK) return st;
  if ((st = rf_require_device()) != RF_OK) return st;
  return rf_launch_diff_bwd(p, q_r, k_r, v_r, select_idx, select_num, lambda, scale, maps, lse, do_r, dq_r, dk_r,
                            dv_r, dlambda, ws, (cudaStream_t)stream);
}

rf_status_t rf_rearrange_rows(const rf_plan_t* p, int32_t heads, const void* x, void* y, int32_t inverse,
                              rf_stream_t stream) {
  rf_clear_error();
  if (!p) return rf_fail(RF_ERR_INVALID_ARG, "null plan");
  if (heads != p->g.n1 && heads != p->g.n2)
    return rf_fail(RF_ERR_INVALID_ARG, "heads must be the plan's query or key/value heads");
  if (!x || !y) return rf_fail(RF_ERR_INVALID_ARG, "null tensor");
  if (!aligned16(x) || !aligned16(y)) return rf_fail(RF_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
  if (x == y) return rf_fail(RF_ERR_INVALID_ARG, "in-place rearrange");
  rf_status_t st = rf_require_device();
  if (st != RF_OK) return st;
  return rf_launch_gather(p, heads, x, y, inverse != 0, (cudaStream_t)stream);
}

}  // extern "C"
