// Group norm with an activation over channels-last rows, forward and backward.
//
//   mu, var: mean and variance of x over a group's channels, of one row
//            (RF_NORM_ROW: each head of an attention output on its own) or of
//            all rows of a batch element (RF_NORM_SAMPLE)
//   xh = (x - mu) / sqrt(var + eps),  z = gamma xh + beta,  y = act(z)
// and with g = dy act'(z):
//   dgamma = sum g xh,  dbeta = sum g  over the rows,
//   dx = (gamma g - mean(gamma g) - xh mean(gamma g xh)) / sqrt(var + eps).
// Everything is computed in fp32 and rounded once.  Means and variances are
// taken about a value of the data (two-pass in registers for rows; for samples
// sums of x - x_0 per channel and slice, merged by the parallel-variance
// formula), so that a mean far from zero does not cancel the variance away.
// All sums run in a fixed order; there are no atomics.
//
// Bound: HBM.  A row's group is held in registers, so RF_NORM_ROW moves each
// element once; RF_NORM_SAMPLE reads x twice (the second time from L2 where it
// fits).  Measured (bf16): rows of 20 x 128, 33,272 of them: 71 us, 4.8 TB/s;
// 16,640 of them with SiLU, forward and backward: 46 and 82 us.  The backward pass is
// held by its instructions (issue slots 66 % busy, 179 warp instructions for each row
// of a group, against 32 % of the DRAM rate and 26 % of the ex2 and reciprocal unit):
// the sums over lanes, conversions and addresses as much as the activation's
// derivative.  Samples of 16,128 x 320, two of them, with SiLU: 22 us in three
// dependent launches.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <string>
#include <utility>

#include "rf_async.cuh"
#include "rf_device.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kReduceThreads = 1024;  // small sums over many slices: latency, so many in flight
constexpr int kMaxRowWidth = 1024;  // widest group held in one warp's registers

struct NormArgs {
  const void* x;
  const void* gamma;
  const void* beta;
  const void* dy;
  void* y;        // forward: y; backward: dx
  float* stats;   // RF_NORM_SAMPLE: {mean, 1 / sqrt(var + eps)} per (batch, group)
  float* ws;
  long long rows, n_rows;            // rows per batch element, of all
  long long xs_b, xs_r, xs_g, ys_b, ys_r, ys_g;
  int batch, groups, width, pdt, act;
  int slices;                        // row slices (partial sums) per batch element or of all rows
  float eps;
};

__device__ __forceinline__ float load_p(const void* p, int dt, long long i) {
  if (dt == RF_FP32) return static_cast<const float*>(p)[i];
  if (dt == RF_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void store_p(void* p, int dt, long long i, float v) {
  if (dt == RF_FP32) static_cast<float*>(p)[i] = v;
  else if (dt == RF_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <class T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// VEC elements (16 bytes when VEC > 1) as they lie in memory, and to and from fp32.
template <class T, int VEC> struct RawVec { using type = uint4; };
template <class T> struct RawVec<T, 1> { using type = T; };
__device__ __forceinline__ void unpack_word(uint32_t w, float* f, float) { f[0] = __uint_as_float(w); }
__device__ __forceinline__ void unpack_word(uint32_t w, float* f, __nv_bfloat16) {
  f[0] = __uint_as_float(w << 16);
  f[1] = __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ void unpack_word(uint32_t w, float* f, __half) {
  f[0] = __half2float(__ushort_as_half((unsigned short)(w & 0xFFFFu)));
  f[1] = __half2float(__ushort_as_half((unsigned short)(w >> 16)));
}
template <class T, int VEC>
__device__ __forceinline__ void unpack_v(const typename RawVec<T, VEC>::type& u, float* f) {
  if constexpr (VEC == 1) {
    f[0] = to_f(u);
  } else {
    constexpr int kPer = VEC / 4;
    unpack_word(u.x, f, T{});
    unpack_word(u.y, f + kPer, T{});
    unpack_word(u.z, f + 2 * kPer, T{});
    unpack_word(u.w, f + 3 * kPer, T{});
  }
}
__device__ __forceinline__ uint32_t pack_word(const float* f, float) { return __float_as_uint(f[0]); }
__device__ __forceinline__ uint32_t pack_word(const float* f, __nv_bfloat16) { return rf_pack2<true>(f[0], f[1]); }
__device__ __forceinline__ uint32_t pack_word(const float* f, __half) { return rf_pack2<false>(f[0], f[1]); }
template <class T, int VEC>
__device__ __forceinline__ void load_v(const T* p, float* f) {
  using Raw = typename RawVec<T, VEC>::type;
  unpack_v<T, VEC>(*reinterpret_cast<const Raw*>(p), f);
}
template <class T, int VEC>
__device__ __forceinline__ void store_v(T* p, const float* f) {
  if constexpr (VEC == 1) {
    *p = from_f<T>(f[0]);
  } else {
    constexpr int kPer = VEC / 4;
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_word(f, T{}), pack_word(f + kPer, T{}), pack_word(f + 2 * kPer, T{}),
                                              pack_word(f + 3 * kPer, T{}));
  }
}

// gamma or beta of VEC channels from channel i on; vector loads where they are aligned.
template <int VEC>
__device__ __forceinline__ void load_pv(const void* p, int dt, long long i, float* f) {
  if (VEC > 1 && (reinterpret_cast<uintptr_t>(p) & 15) == 0 && i % VEC == 0) {
    if (dt == RF_FP32) {
#pragma unroll
      for (int k = 0; k + 4 <= VEC; k += 4) load_v<float, 4>(static_cast<const float*>(p) + i + k, f + k);
      return;
    }
    if constexpr (VEC == 8) {
      if (dt == RF_BF16) load_v<__nv_bfloat16, 8>(static_cast<const __nv_bfloat16*>(p) + i, f);
      else               load_v<__half, 8>(static_cast<const __half*>(p) + i, f);
      return;
    }
  }
#pragma unroll
  for (int k = 0; k < VEC; ++k) f[k] = load_p(p, dt, i + k);
}
// {mean, 1 / sqrt} (or the backward pass's two means) of the groups of VEC channels.
template <int VEC>
__device__ __forceinline__ void load_stats(const float* st, long long first_group, int c, int width, float* m, float* r) {
  if (width % VEC == 0) {  // one group
    const float2 s = *reinterpret_cast<const float2*>(st + 2 * (first_group + c / width));
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      m[k] = s.x;
      r[k] = s.y;
    }
  } else {
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const float2 s = *reinterpret_cast<const float2*>(st + 2 * (first_group + (c + k) / width));
      m[k] = s.x;
      r[k] = s.y;
    }
  }
}

// 1 / (1 + e^-z) from the ex2 and reciprocal units: off by 2^-21 + |z| 2^-23.7 of
// itself at most (the second part from the fp32 product before ex2), for tensors of
// every type.  z was rounded to fp32 before, which changes e^-z by |z| 2^-24 of
// itself: expf and a division in their place (fp32 rows of 20 x 128, 16,640 of them:
// 70 -> 96 us forward, 119 -> 144 us backward) would not undo that.
__device__ __forceinline__ float sigmoid(float z) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + rf_ex2(-1.4426950408889634f * z)));
  return r;
}
__device__ __forceinline__ float act_f(float z, int act) { return act == RF_ACT_SILU ? z * sigmoid(z) : z; }
// derivative of the activation at z
__device__ __forceinline__ float act_d(float z, int act) {
  if (act != RF_ACT_SILU) return 1.f;
  const float s = sigmoid(z);
  return s * fmaf(z, 1.f - s, 1.f);
}
__device__ __forceinline__ uint64_t pair(float a, float b) { return rf_f2(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ float pair_sum(uint64_t p) {
  float a, b;
  rf_f2_split(p, a, b);
  return a + b;
}

// Sum over the `lanes` (a power of two) neighbouring lanes of a sub-warp.
__device__ __forceinline__ float sub_sum(float v, int lanes) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < lanes) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One row at a time per sub-warp of `lanes` lanes, NV vectors of VEC channels per
// lane; blockIdx.y = group, so that gamma, beta and (backward) the channels' sums
// stay in registers over all rows of the CTA's slice.  kPre rows are on their
// way from memory, unconverted, while one is computed.
template <class T, int VEC, int NV, bool kBwd>
__global__ void __launch_bounds__(kThreads, VEC * NV <= 8 ? (kBwd ? 3 : 4) : 1)
    rf_norm_row_kernel(const __grid_constant__ NormArgs a, int lanes) {
  constexpr int E = VEC * NV;
  constexpr int kPre = E <= 8 && !kBwd ? 2 : 1;
  using Raw = typename RawVec<T, VEC>::type;
  const int g = blockIdx.y, lane = threadIdx.x % lanes, sub = threadIdx.x / lanes, subs = kThreads / lanes;
  const T* x = static_cast<const T*>(a.x) + g * a.xs_g + lane * VEC;
  const T* dy = static_cast<const T*>(a.dy) + g * a.ys_g + lane * VEC;
  T* out = static_cast<T*>(a.y) + (kBwd ? g * a.xs_g : g * a.ys_g) + lane * VEC;
  // channels in pairs for the paired fp32 instructions (a lone channel beside a zero)
  constexpr int P = (E + 1) / 2;
  wait_for_previous();
  uint64_t gm[P], bt[P], sg[kBwd ? P : 1], sb[kBwd ? P : 1];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    float g2[2] = {0.f, 0.f}, b2[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = 2 * p + i, c = (k / VEC * lanes + lane) * VEC + k % VEC;
      if (k < E && c < a.width) {
        g2[i] = load_p(a.gamma, a.pdt, (long long)g * a.width + c);
        b2[i] = load_p(a.beta, a.pdt, (long long)g * a.width + c);
      }
    }
    gm[p] = pair(g2[0], g2[1]);
    bt[p] = pair(b2[0], b2[1]);
    if constexpr (kBwd) sg[p] = sb[p] = 0ull;
  }
  const int mine = (a.width / VEC - lane + lanes - 1) / lanes;  // vectors of this lane (v < mine)
  const float inv = 1.0f / (float)a.width;
  const long long per = (a.n_rows + a.slices - 1) / a.slices;
  const long long first = (long long)blockIdx.x * per, last = min(a.n_rows, first + per);
  const int n_mine = last > first ? (int)(last - first) : 0;  // at most 2^30: check_desc
  const int count = (n_mine + subs - 1) / subs;
  // batch element and row of the next row to load, and of the row to store
  const int n_r = (int)a.rows;
  int lb = (int)((first + sub) / a.rows), lr = (int)((first + sub) - lb * a.rows), sb_ = lb, sr = lr;
  Raw xr[kPre][NV], dr[kBwd ? kPre : 1][kBwd ? NV : 1];
  auto load = [&](int i, int slot) {
    const bool live = sub + i * subs < n_mine;
    const T* px = x + (lb * a.xs_b + lr * a.xs_r);
    const T* pd = dy + (kBwd ? lb * a.ys_b + lr * a.ys_r : 0);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      xr[slot][v] = Raw{};
      if constexpr (kBwd) dr[slot][v] = Raw{};
      if (live && v < mine) {
        xr[slot][v] = *reinterpret_cast<const Raw*>(px + v * lanes * VEC);
        if constexpr (kBwd) dr[slot][v] = *reinterpret_cast<const Raw*>(pd + v * lanes * VEC);
      }
    }
    lr += subs;
    while (lr >= n_r) {
      lr -= n_r;
      ++lb;
    }
  };
#pragma unroll
  for (int i = 0; i < kPre; ++i) load(i, i);
  // every lane of a warp runs the same number of turns (the sums use the whole warp)
  for (int i0 = 0; i0 < count; i0 += kPre) {
#pragma unroll
    for (int w = 0; w < kPre; ++w) {
      const int i = i0 + w;
      const bool live = sub + i * subs < n_mine;
      uint64_t xp[P], dp[kBwd ? P : 1];
      {
        float f[2 * P];
        f[2 * P - 1] = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) unpack_v<T, VEC>(xr[w][v], f + v * VEC);
#pragma unroll
        for (int p = 0; p < P; ++p) xp[p] = pair(f[2 * p], f[2 * p + 1]);
        if constexpr (kBwd) {
#pragma unroll
          for (int v = 0; v < NV; ++v) unpack_v<T, VEC>(dr[w][v], f + v * VEC);
#pragma unroll
          for (int p = 0; p < P; ++p) dp[p] = pair(f[2 * p], f[2 * p + 1]);
        }
      }
      load(i + kPre, w);
      uint64_t s2 = xp[0];
#pragma unroll
      for (int p = 1; p < P; ++p) s2 = rf_add2(s2, xp[p]);
      const float mu = sub_sum(pair_sum(s2), lanes) * inv;
      s2 = 0ull;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        // vectors that this lane does not have stay zero
        const float m0 = 2 * p / VEC < mine ? -mu : 0.f;
        const float m1 = 2 * p + 1 < E && (2 * p + 1) / VEC < mine ? -mu : 0.f;
        xp[p] = rf_add2(xp[p], pair(m0, m1));
        s2 = rf_fma2(xp[p], xp[p], s2);
      }
      float rstd = rsqrtf(sub_sum(pair_sum(s2), lanes) * inv + a.eps);
      if (!live) rstd = 0.f;  // a row past the end counts for nothing, even with eps = 0
      const uint64_t rs2 = pair(rstd, rstd);
      if constexpr (!kBwd) {
#pragma unroll
        for (int p = 0; p < P; ++p) xp[p] = rf_fma2(rf_mul2(xp[p], rs2), gm[p], bt[p]);
        if (a.act == RF_ACT_SILU) {
#pragma unroll
          for (int p = 0; p < P; ++p) {
            float z0, z1;
            rf_f2_split(xp[p], z0, z1);
            xp[p] = pair(z0 * sigmoid(z0), z1 * sigmoid(z1));
          }
        }
      } else {
        uint64_t m1 = 0ull, m2 = 0ull;
        if (a.act == RF_ACT_SILU) {
          const uint64_t one = pair(1.f, 1.f), neg = pair(-1.f, -1.f);
#pragma unroll
          for (int p = 0; p < P; ++p) {
            const uint64_t z = rf_fma2(rf_mul2(xp[p], rs2), gm[p], bt[p]);
            float z0, z1;
            rf_f2_split(z, z0, z1);
            const uint64_t s = pair(sigmoid(z0), sigmoid(z1));
            // act'(z) = s (1 + z (1 - s))
            dp[p] = rf_mul2(dp[p], rf_mul2(s, rf_fma2(z, rf_fma2(s, neg, one), one)));
          }
        }
#pragma unroll
        for (int p = 0; p < P; ++p) {
          xp[p] = rf_mul2(xp[p], rs2);
          sg[p] = rf_fma2(dp[p], xp[p], sg[p]);
          sb[p] = rf_add2(sb[p], dp[p]);
          dp[p] = rf_mul2(dp[p], gm[p]);
          m1 = rf_add2(m1, dp[p]);
          m2 = rf_fma2(dp[p], xp[p], m2);
        }
        const float u1 = -sub_sum(pair_sum(m1), lanes) * inv * rstd, u2 = -sub_sum(pair_sum(m2), lanes) * inv * rstd;
        const uint64_t v1 = pair(u1, u1), v2 = pair(u2, u2);
        // dx = rstd g - rstd mean(g) - xh rstd mean(g xh)
#pragma unroll
        for (int p = 0; p < P; ++p) xp[p] = rf_fma2(xp[p], v2, rf_fma2(dp[p], rs2, v1));
      }
      if (live) {
        T* po = out + (kBwd ? sb_ * a.xs_b + sr * a.xs_r : sb_ * a.ys_b + sr * a.ys_r);
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (v < mine) {
            float f[VEC + 1];
#pragma unroll
            for (int k = 0; k < VEC; k += 2) rf_f2_split(xp[(v * VEC + k) / 2], f[k], f[k + 1]);
            if (VEC == 1 && v % 2) f[0] = f[1];
            store_v<T, VEC>(po + v * lanes * VEC, f);
          }
      }
      sr += subs;
      while (sr >= n_r) {
        sr -= n_r;
        ++sb_;
      }
    }
  }
  if constexpr (kBwd) {
    // this CTA's sums per channel: sub-warps in order, through shared memory
    __shared__ float red[2][kMaxRowWidth];
    for (int turn = 0; turn < subs; ++turn) {
      if (sub == turn) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (v < mine)
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
              const int c = (v * lanes + lane) * VEC + k;
              float g2[2], b2[2];
              rf_f2_split(sg[(v * VEC + k) / 2], g2[0], g2[1]);
              rf_f2_split(sb[(v * VEC + k) / 2], b2[0], b2[1]);
              red[0][c] = (turn ? red[0][c] : 0.f) + g2[(v * VEC + k) % 2];
              red[1][c] = (turn ? red[1][c] : 0.f) + b2[(v * VEC + k) % 2];
            }
      }
      __syncthreads();
    }
    const long long ch = (long long)a.groups * a.width;
    for (int c = threadIdx.x; c < a.width; c += kThreads) {
      float* w = a.ws + (long long)blockIdx.x * 2 * ch + (long long)g * a.width + c;
      w[0] = red[0][c];
      w[ch] = red[1][c];
    }
  }
}

// ---- statistics over a batch element's rows -------------------------------------

// Channel vector `cv` of VEC channels: element offset of its first channel (a
// vector never crosses a group unless the groups are contiguous).
__device__ __forceinline__ long long chan_off(long long c, int width, long long sg) {
  const int g = (int)c / width;  // check_desc keeps groups * width below 2^31
  return g * sg + ((int)c - g * width);
}

// max(v, 0) that keeps a NaN: a group with an infinity has no variance.
__device__ __forceinline__ float not_below_0(float v) { return v < 0.f ? 0.f : v; }

// Per-channel partial sums of one slice of rows.  Forward: {sum(x - x0) as a
// mean, sum of squared deviations}; backward: {sum g, sum g xh}.  A thread owns
// VEC channels; the block's row lanes are merged in order.
template <class T, int VEC, bool kBwd>
__global__ void __launch_bounds__(kThreads) rf_norm_partial_kernel(const __grid_constant__ NormArgs a, int tile) {
  __shared__ float red[2][kThreads][VEC];
  wait_for_previous();
  const int b = blockIdx.z;
  const long long ch = (long long)a.groups * a.width;
  const int lanes = kThreads / tile, rl = threadIdx.x / tile;
  const long long c = ((long long)blockIdx.y * tile + threadIdx.x % tile) * VEC;
  const bool live = rl < lanes && c < ch;
  const long long per = (a.rows + a.slices - 1) / a.slices;
  const long long first = (long long)blockIdx.x * per, last = min(a.rows, first + per);
  float p0[VEC], p1[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) p0[k] = p1[k] = 0.f;
  float n = 0.f;
  if (live && first + rl < last) {
    const T* x = static_cast<const T*>(a.x) + b * a.xs_b + chan_off(c, a.width, a.xs_g);
    float x0[VEC], gm[VEC], bt[VEC], mu[VEC], rs[VEC];
    if constexpr (!kBwd) {
      load_v<T, VEC>(x + (first + rl) * a.xs_r, x0);
    } else {
      load_pv<VEC>(a.gamma, a.pdt, c, gm);
      load_pv<VEC>(a.beta, a.pdt, c, bt);
      load_stats<VEC>(a.stats, b * (long long)a.groups, (int)c, a.width, mu, rs);
    }
    const T* dy = static_cast<const T*>(a.dy) + (kBwd ? b * a.ys_b + chan_off(c, a.width, a.ys_g) : 0);
#pragma unroll 8
    for (long long r = first + rl; r < last; r += lanes) {
      float xv[VEC];
      load_v<T, VEC>(x + r * a.xs_r, xv);
      if constexpr (!kBwd) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float d = xv[k] - x0[k];
          p0[k] += d;
          p1[k] = fmaf(d, d, p1[k]);
        }
        n += 1.f;
      } else {
        float dv[VEC];
        load_v<T, VEC>(dy + r * a.ys_r, dv);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float xh = (xv[k] - mu[k]) * rs[k];
          const float gz = dv[k] * act_d(fmaf(xh, gm[k], bt[k]), a.act);
          p0[k] += gz;
          p1[k] = fmaf(gz, xh, p1[k]);
        }
      }
    }
    if constexpr (!kBwd) {
      const float in = 1.0f / n;
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        p1[k] = not_below_0(p1[k] - p0[k] * p0[k] * in);
        p0[k] = x0[k] + p0[k] * in;
      }
    }
  }
  if (rl < lanes) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      red[0][threadIdx.x][k] = p0[k];
      red[1][threadIdx.x][k] = p1[k];
    }
  }
  __syncthreads();
  if (rl == 0 && c < ch) {
    const long long rows = last > first ? last - first : 0;
    for (int l = 1; l < lanes; ++l) {
      const float nl = (float)((rows - l + lanes - 1) / lanes > 0 && l < rows ? (rows - l + lanes - 1) / lanes : 0);
      if (!kBwd && nl == 0.f) break;
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const float q0 = red[0][threadIdx.x + l * tile][k], q1 = red[1][threadIdx.x + l * tile][k];
        if constexpr (!kBwd) {
          const float d = q0 - p0[k], t = nl / (n + nl);
          p0[k] = fmaf(d, t, p0[k]);
          p1[k] += q1 + d * d * n * t;
        } else {
          p0[k] += q0;
          p1[k] += q1;
        }
      }
      n += nl;
    }
    float* w = a.ws + ((long long)b * a.slices + blockIdx.x) * 2 * ch + c;
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      w[k] = p0[k];
      w[ch + k] = p1[k];
    }
  }
}

__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = red[threadIdx.x & 31];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// Forward: a (batch, group)'s mean and 1 / sqrt(var + eps) from its channels'
// slices, about one of the slices' means (so that what cancels in the variance
// is only how far the channels' means lie apart, which is part of it).
// Backward: {mean(gamma g), mean(gamma g xh)}, behind the slices' sums in the
// workspace.
template <bool kBwd>
__global__ void __launch_bounds__(kReduceThreads) rf_norm_stats_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float red[kReduceThreads / 32];
  wait_for_previous();
  const int b = blockIdx.x / a.groups, g = blockIdx.x % a.groups;
  const long long ch = (long long)a.groups * a.width;
  const float* w = a.ws + (long long)b * a.slices * 2 * ch + (long long)g * a.width;
  const int per = (int)((a.rows + a.slices - 1) / a.slices);
  const float inv = 1.0f / ((float)a.rows * (float)a.width);
  const float ref = kBwd ? 0.f : w[0];
  float s = 0.f, q = 0.f;
  const int wide = min(a.width, kReduceThreads), stride = kReduceThreads / wide;  // channels, slices in parallel
  const int c0 = threadIdx.x % wide, s0 = threadIdx.x / wide;
  if (s0 < stride)
    for (int c = c0; c < a.width; c += kReduceThreads) {
      const float gm = kBwd ? load_p(a.gamma, a.pdt, (long long)g * a.width + c) : 0.f;
#pragma unroll 4
      for (int sl = s0; sl < a.slices; sl += stride) {
        const float v0 = w[sl * 2 * ch + c], v1 = w[sl * 2 * ch + ch + c];
        if constexpr (kBwd) {
          s = fmaf(gm, v0, s);
          q = fmaf(gm, v1, q);
        } else {
          // an empty slice's zeros count for nothing
          const float n = (float)max(0, min((int)a.rows - sl * per, per)), d = v0 - ref;
          s = fmaf(n, d, s);
          q += fmaf(n * d, d, v1);
        }
      }
    }
  s = block_sum(s, red) * inv;
  q = block_sum(q, red) * inv;
  if (threadIdx.x == 0) {
    float* o = kBwd ? a.ws + (long long)a.batch * a.slices * 2 * ch : a.stats;
    o[2 * blockIdx.x] = kBwd ? s : ref + s;
    o[2 * blockIdx.x + 1] = kBwd ? q : rsqrtf(not_below_0(q - s * s) + a.eps);
  }
}

// dgamma and dbeta: the partial sums [parts][2][channels] added in a fixed order.
__global__ void __launch_bounds__(kReduceThreads) rf_norm_params_kernel(const float* ws, int parts,
                                                                        long long ch, int gamma_first, int pdt,
                                                                        void* dgamma, void* dbeta) {
  // 32 channels per block, 32 lanes of parts, merged in order
  __shared__ float red[2][32][33];
  wait_for_previous();
  const int cl = threadIdx.x & 31, pl = threadIdx.x >> 5;
  const long long c = (long long)blockIdx.x * 32 + cl;
  float s0 = 0.f, s1 = 0.f;
  if (c < ch)
#pragma unroll 4
    for (int p = pl; p < parts; p += 32) {
      s0 += ws[p * 2 * ch + c];
      s1 += ws[p * 2 * ch + ch + c];
    }
  red[0][pl][cl] = s0;
  red[1][pl][cl] = s1;
  __syncthreads();
  // warp pl sums channel pl's 32 lanes
  s0 = red[0][cl][pl];
  s1 = red[1][cl][pl];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s0 += __shfl_xor_sync(0xffffffffu, s0, o);
    s1 += __shfl_xor_sync(0xffffffffu, s1, o);
  }
  const long long cc = (long long)blockIdx.x * 32 + pl;
  if (cl == 0 && cc < ch) {
    store_p(dgamma, pdt, cc, gamma_first ? s0 : s1);
    store_p(dbeta, pdt, cc, gamma_first ? s1 : s0);
  }
}

// y (or dx) of every element from the statistics.
template <class T, int VEC, bool kBwd>
__global__ void __launch_bounds__(kThreads) rf_norm_apply_kernel(const __grid_constant__ NormArgs a, int tile) {
  wait_for_previous();
  const int b = blockIdx.z;
  const long long ch = (long long)a.groups * a.width;
  const int lanes = kThreads / tile, rl = threadIdx.x / tile;
  const long long c = ((long long)blockIdx.y * tile + threadIdx.x % tile) * VEC;
  if (rl >= lanes || c >= ch) return;
  float gm[VEC], bt[VEC], mu[VEC], rs[VEC], m1[VEC], m2[VEC];
  load_pv<VEC>(a.gamma, a.pdt, c, gm);
  load_pv<VEC>(a.beta, a.pdt, c, bt);
  load_stats<VEC>(a.stats, b * (long long)a.groups, (int)c, a.width, mu, rs);
  if constexpr (kBwd)
    load_stats<VEC>(a.ws + (long long)a.batch * a.slices * 2 * ch, b * (long long)a.groups, (int)c, a.width, m1, m2);
  const long long xo = b * a.xs_b + chan_off(c, a.width, a.xs_g), yo = b * a.ys_b + chan_off(c, a.width, a.ys_g);
  const T* x = static_cast<const T*>(a.x) + xo;
  const T* dy = static_cast<const T*>(a.dy) + (kBwd ? yo : 0);
  T* out = static_cast<T*>(a.y) + (kBwd ? xo : yo);
  const long long os = kBwd ? a.xs_r : a.ys_r;
  const long long step = (long long)gridDim.x * lanes;
#pragma unroll 4
  for (long long r = (long long)blockIdx.x * lanes + rl; r < a.rows; r += step) {
    float xv[VEC];
    load_v<T, VEC>(x + r * a.xs_r, xv);
    if constexpr (!kBwd) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) xv[k] = act_f(fmaf((xv[k] - mu[k]) * rs[k], gm[k], bt[k]), a.act);
    } else {
      float dv[VEC];
      load_v<T, VEC>(dy + r * a.ys_r, dv);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const float xh = (xv[k] - mu[k]) * rs[k];
        const float gz = dv[k] * act_d(fmaf(xh, gm[k], bt[k]), a.act);
        xv[k] = rs[k] * (gz * gm[k] - m1[k] - xh * m2[k]);
      }
    }
    store_v<T, VEC>(out + r * os, xv);
  }
}

// ---- host -----------------------------------------------------------------------

rf_status_t check_desc(const rf_norm_desc_t* d) {
  if (!d) return rf_fail(RF_ERR_INVALID_ARG, "null descriptor");
  if (d->batch < 0 || d->rows < 0) return rf_fail(RF_ERR_INVALID_ARG, "negative batch or rows");
  if (d->groups < 1 || d->width < 1) return rf_fail(RF_ERR_INVALID_ARG, "groups and width must be > 0");
  if (d->dtype != RF_BF16 && d->dtype != RF_FP16 && d->dtype != RF_FP32)
    return rf_fail(RF_ERR_INVALID_ARG, "dtype must be bf16, fp16 or fp32");
  if (d->param_dtype != RF_BF16 && d->param_dtype != RF_FP16 && d->param_dtype != RF_FP32)
    return rf_fail(RF_ERR_INVALID_ARG, "param_dtype must be bf16, fp16 or fp32");
  if (d->span != RF_NORM_ROW && d->span != RF_NORM_SAMPLE) return rf_fail(RF_ERR_INVALID_ARG, "unknown span");
  if (d->act != RF_ACT_NONE && d->act != RF_ACT_SILU) return rf_fail(RF_ERR_INVALID_ARG, "unknown activation");
  if (!(d->eps >= 0.f) || !(d->eps < INFINITY)) return rf_fail(RF_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (d->span == RF_NORM_ROW && d->width > kMaxRowWidth)
    return rf_fail(RF_ERR_UNSUPPORTED, "groups of more than 1024 channels per row are not built");
  if (d->batch > 65535 && d->span == RF_NORM_SAMPLE)
    return rf_fail(RF_ERR_UNSUPPORTED, "more than 65535 samples");
  if (d->span == RF_NORM_SAMPLE && d->batch * d->groups > 0x7FFFFFFFll)  // one CTA each adds up their statistics
    return rf_fail(RF_ERR_UNSUPPORTED, "too many groups over all samples");
  if (d->groups > 65535) return rf_fail(RF_ERR_UNSUPPORTED, "more than 65535 groups");
  if ((int64_t)d->groups * d->width > (1 << 30)) return rf_fail(RF_ERR_UNSUPPORTED, "too many channels");
  if (d->rows > (1ll << 30) || d->batch > (1ll << 30) || d->batch * d->rows > (1ll << 30)) return rf_fail(RF_ERR_UNSUPPORTED, "too many rows");
  const int64_t st[] = {d->x_stride_b, d->x_stride_r, d->x_stride_g, d->y_stride_b, d->y_stride_r, d->y_stride_g};
  for (int64_t s : st)
    if (s < 0) return rf_fail(RF_ERR_INVALID_ARG, "negative stride");
  return RF_OK;
}

// Whether no two elements of an output with these strides share a place: taken
// from the smallest stride up, each axis steps over all that the smaller ones
// reach (true for every permuted, padded or sliced dense tensor).
bool disjoint(const rf_norm_desc_t* d, int64_t sb, int64_t sr, int64_t sg) {
  std::pair<int64_t, int64_t> ax[3] = {{sb, d->batch}, {sr, d->rows}, {sg, d->groups}};
  std::sort(ax, ax + 3);
  int64_t reach = d->width;
  for (const auto& a : ax) {
    if (a.second <= 1) continue;
    if (a.first < reach) return false;
    reach += (a.second - 1) * a.first;
  }
  return true;
}

int vec_of(const rf_norm_desc_t* d) { return d->dtype == RF_FP32 ? 4 : 8; }

// Channels per thread: 16-byte vectors where every row and group begins on one.
// Samples may have groups that are no whole number of vectors as long as the
// channel axis is contiguous.
bool vector_ok(const rf_norm_desc_t* d, bool rows, const void* a, const void* b, const void* c) {
  const int v = vec_of(d);
  if (d->batch > 1 && (d->x_stride_b % v || d->y_stride_b % v)) return false;
  if (d->rows > 1 && (d->x_stride_r % v || d->y_stride_r % v)) return false;
  const bool split = d->width % v == 0 && d->x_stride_g % v == 0 && d->y_stride_g % v == 0;
  const bool whole = !rows && d->x_stride_g == d->width && d->y_stride_g == d->width &&
                     ((int64_t)d->groups * d->width) % v == 0;
  if (!split && !whole) return false;
  const void* ps[] = {a, b, c};
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) & 15) return false;
  return true;
}

// Row slices: as many CTAs over all groups (channel tiles, samples) as run at
// once, at least 32 rows each.  Rows: four per SM forward, three backward (its
// channel sums take registers); samples: two per SM.
int slices_of(const rf_norm_desc_t* d, bool bwd) {
  if (d->span == RF_NORM_ROW) {
    const int64_t n = d->batch * d->rows;
    const int64_t want = std::max(1, 148 * (bwd ? 3 : 4) / d->groups), most = (n + 31) / 32;
    return (int)std::max<int64_t>(1, std::min(want, most));
  }
  const int64_t b = std::max<int64_t>(1, d->batch);
  const int64_t tiles = ((int64_t)d->groups * d->width + 2047) / 2048;
  const int64_t want = std::max<int64_t>(1, 148 * 2 / (b * tiles)), most = (d->rows + 31) / 32;
  return (int)std::max<int64_t>(1, std::min(want, most));
}

int64_t ws_bytes_of(const rf_norm_desc_t* d) {
  const int64_t ch = (int64_t)d->groups * d->width, sl = slices_of(d, true);
  const int64_t parts = d->span == RF_NORM_ROW ? sl : d->batch * sl;
  return (parts * 2 * ch + 2 * d->batch * d->groups) * 4 + 256;
}

NormArgs make_args(const rf_norm_desc_t* d, const void* x, const void* gamma, const void* beta, const void* dy, void* y,
                   float* stats, void* ws, bool bwd) {
  NormArgs a;
  a.x = x;
  a.gamma = gamma;
  a.beta = beta;
  a.dy = dy;
  a.y = y;
  a.stats = stats;
  a.ws = static_cast<float*>(ws);
  a.rows = d->rows;
  a.n_rows = d->batch * d->rows;
  a.xs_b = d->x_stride_b; a.xs_r = d->x_stride_r; a.xs_g = d->x_stride_g;
  a.ys_b = d->y_stride_b; a.ys_r = d->y_stride_r; a.ys_g = d->y_stride_g;
  a.batch = (int)d->batch;
  a.groups = d->groups;
  a.width = d->width;
  a.pdt = d->param_dtype;
  a.act = d->act;
  a.slices = slices_of(d, bwd);
  a.eps = d->eps;
  return a;
}

template <class T, int VEC, int NV, bool kBwd>
rf_status_t row_launch(const NormArgs& a, int lanes, cudaStream_t st) {
  return rf_launch_dependent(rf_norm_row_kernel<T, VEC, NV, kBwd>, dim3((unsigned)a.slices, (unsigned)a.groups), kThreads,
                             st, "rf_norm_row_kernel", a, lanes);
}

template <class T, bool kBwd>
rf_status_t run_rows(const NormArgs& a, bool vec, cudaStream_t st) {
  constexpr int V = sizeof(T) == 4 ? 4 : 8;
  const int units = vec ? a.width / V : a.width;
  int lanes = 1;
  while (lanes < 32 && lanes < units) lanes <<= 1;
  const int nv = (units + lanes - 1) / lanes;
  if (vec) {
    if (nv <= 1) return row_launch<T, V, 1, kBwd>(a, lanes, st);
    if (nv <= 2) return row_launch<T, V, 2, kBwd>(a, lanes, st);
    return row_launch<T, V, sizeof(T) == 4 ? 8 : 4, kBwd>(a, lanes, st);  // 1,024 channels
  }
  if (nv <= 1) return row_launch<T, 1, 1, kBwd>(a, lanes, st);
  if (nv <= 4) return row_launch<T, 1, 4, kBwd>(a, lanes, st);
  return row_launch<T, 1, 32, kBwd>(a, lanes, st);
}

// Channel vectors of a block: all of them up to 256, so that a row is read in
// one piece; the rest of the threads take further rows.
int tile_of(const NormArgs& a, int vec) {
  const long long cv = ((long long)a.groups * a.width + vec - 1) / vec;
  return (int)std::min<long long>(cv, kThreads);
}

template <class T, int VEC, bool kBwd>
rf_status_t run_samples_v(const NormArgs& a, cudaStream_t st) {
  const int tile = tile_of(a, VEC);
  const long long cv = ((long long)a.groups * a.width + VEC - 1) / VEC;
  const unsigned tiles = (unsigned)((cv + tile - 1) / tile);
  if (tiles > 65535u) return rf_fail(RF_ERR_UNSUPPORTED, "too many channels");
  rf_status_t s = rf_launch_dependent(rf_norm_partial_kernel<T, VEC, kBwd>, dim3((unsigned)a.slices, tiles, (unsigned)a.batch),
                                      kThreads, st, "rf_norm_partial_kernel", a, tile);
  if (s != RF_OK) return s;
  s = rf_launch_dependent(rf_norm_stats_kernel<kBwd>, dim3((unsigned)(a.batch * a.groups)), kReduceThreads, st,
                          "rf_norm_stats_kernel", a);
  if (s != RF_OK) return s;
  const long long lanes = kThreads / tile;
  const long long most = (a.rows + lanes - 1) / lanes, want = std::max<long long>(1, 148ll * 4 / ((long long)tiles * a.batch));
  const unsigned gx = (unsigned)std::max<long long>(1, std::min(most, want));
  return rf_launch_dependent(rf_norm_apply_kernel<T, VEC, kBwd>, dim3(gx, tiles, (unsigned)a.batch), kThreads, st,
                             "rf_norm_apply_kernel", a, tile);
}

template <class T, bool kBwd>
rf_status_t run_t(const rf_norm_desc_t* d, const NormArgs& a, cudaStream_t st) {
  constexpr int V = sizeof(T) == 4 ? 4 : 8;
  const bool rows = d->span == RF_NORM_ROW;
  const bool vec = vector_ok(d, rows, a.x, a.y, kBwd ? a.dy : a.x);
  if (rows) return run_rows<T, kBwd>(a, vec, st);
  return vec ? run_samples_v<T, V, kBwd>(a, st) : run_samples_v<T, 1, kBwd>(a, st);
}

template <bool kBwd>
rf_status_t run(const rf_norm_desc_t* d, const NormArgs& a, cudaStream_t st) {
  if (d->dtype == RF_FP32) return run_t<float, kBwd>(d, a, st);
  if (d->dtype == RF_BF16) return run_t<__nv_bfloat16, kBwd>(d, a, st);
  return run_t<__half, kBwd>(d, a, st);
}

rf_status_t check_norm_ws(const rf_norm_desc_t* d, const void* ws, size_t bytes) {
  if (!ws) return rf_fail(RF_ERR_INVALID_ARG, "null workspace");
  if ((reinterpret_cast<uintptr_t>(ws) & 255) != 0)
    return rf_fail(RF_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if ((uint64_t)bytes < (uint64_t)ws_bytes_of(d))
    return rf_fail(RF_ERR_WORKSPACE_TOO_SMALL, "workspace needs " + std::to_string(ws_bytes_of(d)) + " bytes");
  return RF_OK;
}

}  // namespace

extern "C" {

rf_status_t rf_group_norm_workspace_bytes(const rf_norm_desc_t* d, int64_t* out) {
  rf_clear_error();
  rf_status_t st = check_desc(d);
  if (st != RF_OK) return st;
  if (!out) return rf_fail(RF_ERR_INVALID_ARG, "null out");
  *out = ws_bytes_of(d);
  return RF_OK;
}

rf_status_t rf_group_norm(const rf_norm_desc_t* d, const void* x, const void* gamma, const void* beta, void* y,
                          float* stats, void* ws, size_t ws_bytes, rf_stream_t stream) {
  rf_clear_error();
  rf_status_t st = check_desc(d);
  if (st != RF_OK) return st;
  if (!gamma || !beta) return rf_fail(RF_ERR_INVALID_ARG, "null gamma or beta");
  const bool sample = d->span == RF_NORM_SAMPLE;
  if (d->batch == 0 || d->rows == 0) return RF_OK;
  if (!x || !y || (sample && !stats)) return rf_fail(RF_ERR_INVALID_ARG, "null tensor");
  if (reinterpret_cast<uintptr_t>(stats) & 7) return rf_fail(RF_ERR_INVALID_ARG, "stats must be 8-byte aligned");
  if (x == y) return rf_fail(RF_ERR_INVALID_ARG, "y aliases x");
  if (!disjoint(d, d->y_stride_b, d->y_stride_r, d->y_stride_g))
    return rf_fail(RF_ERR_INVALID_ARG, "elements of y overlap (a broadcast output)");
  if (sample && (st = check_norm_ws(d, ws, ws_bytes)) != RF_OK) return st;
  if ((st = rf_require_device()) != RF_OK) return st;
  return run<false>(d, make_args(d, x, gamma, beta, nullptr, y, stats, ws, false), (cudaStream_t)stream);
}

rf_status_t rf_group_norm_backward(const rf_norm_desc_t* d, const void* x, const void* gamma, const void* beta,
                                   const void* dy, const float* stats, void* dx, void* dgamma, void* dbeta, void* ws,
                                   size_t ws_bytes, rf_stream_t stream) {
  rf_clear_error();
  rf_status_t st = check_desc(d);
  if (st != RF_OK) return st;
  if (!gamma || !beta || !dgamma || !dbeta) return rf_fail(RF_ERR_INVALID_ARG, "null parameter or its gradient");
  const bool sample = d->span == RF_NORM_SAMPLE;
  const int64_t ch = (int64_t)d->groups * d->width;
  if (d->batch == 0 || d->rows == 0) {
    if ((st = rf_require_device()) != RF_OK) return st;
    const size_t bytes = (size_t)ch * (d->param_dtype == RF_FP32 ? 4 : 2);
    if (cudaMemsetAsync(dgamma, 0, bytes, (cudaStream_t)stream) != cudaSuccess ||
        cudaMemsetAsync(dbeta, 0, bytes, (cudaStream_t)stream) != cudaSuccess)
      return rf_check_launch("cudaMemsetAsync(group norm gradients)");
    return RF_OK;
  }
  if (!x || !dy || !dx || (sample && !stats)) return rf_fail(RF_ERR_INVALID_ARG, "null tensor");
  if (reinterpret_cast<uintptr_t>(stats) & 7) return rf_fail(RF_ERR_INVALID_ARG, "stats must be 8-byte aligned");
  if (dx == x || dx == dy) return rf_fail(RF_ERR_INVALID_ARG, "dx aliases an input");
  if (!disjoint(d, d->x_stride_b, d->x_stride_r, d->x_stride_g))
    return rf_fail(RF_ERR_INVALID_ARG, "elements of dx overlap (x is broadcast)");
  if ((st = check_norm_ws(d, ws, ws_bytes)) != RF_OK) return st;
  if ((st = rf_require_device()) != RF_OK) return st;
  const NormArgs a = make_args(d, x, gamma, beta, dy, dx, const_cast<float*>(stats), ws, true);
  if ((st = run<true>(d, a, (cudaStream_t)stream)) != RF_OK) return st;
  return rf_launch_dependent(rf_norm_params_kernel, dim3((unsigned)((ch + 31) / 32)), kReduceThreads, (cudaStream_t)stream,
                             "rf_norm_params_kernel", (const float*)a.ws, sample ? a.batch * a.slices : a.slices,
                             (long long)ch, sample ? 0 : 1, a.pdt, dgamma, dbeta);
}

}  // extern "C"
