// Backward pass of differential attention over the selected key blocks.
//
// With P_w = softmax(scale Q_w K_w^T) (w = 1, 2), A = P_1 - lambda P_2 and
// O = A V per query head, and dO given:
//   dV  = A^T dO                      dA = dO V^T
//   dS_1 = P_1 o (dA - delta_1)       dS_2 = -lambda P_2 o (dA - delta_2)
//   dQ_w = scale dS_w K_w             dK_w = scale dS_w^T Q_w
//   delta_w = rowsum(P_w o dA) = dO . O_w,  dlambda = -sum of delta_2 over rows
// (o: element by element).  P_w is recomputed from S_w and the log2-sum the
// forward pass kept.  delta_w is taken from the fp32 O_w the forward pass kept:
// where a softmax is nearly one-hot, dA - delta cancels almost completely, and
// a 16-bit O_w in its place gave dQ errors of 2e-2 on such rows (fp32: 4e-3, as
// with an exact delta).
//
// Kernels:
//   rf_diff_prep_bwd_kernel  per (query block, head): delta_1, delta_2 and the
//                            kept sums packed per row; the block's part of
//                            dlambda; one bit per listed key block, by key block.
//   rf_diff_dq_kernel        CTA = (query block, head): dQ over the listed blocks.
//   rf_diff_dkv_kernel       CTA = (key block, key/value head): dK and dV over
//                            every (head of the group, query block) that lists
//                            it, in ascending order.
//   rf_diff_dlam_kernel      sums dlambda's parts in block order.
// Two passes (S and dA computed in both, 7 matrix products for 5) need no
// atomic additions, so the gradients are the same bits every time.  dQ does not
// need dK and dV and is launched as their kernel's dependent, into the SMs that
// its last wave leaves free.
//
// A and dS are rounded once, to the inputs' type, for the tensor cores.  fp16
// has no room for their range, so there A and dS carry powers of two (exact to
// undo), one for each accumulation, so that a large value that a gradient does not
// add up costs it no digits.  dQ: one per query row, from its own |dO| and the largest
// |V| of the blocks it lists.  dK, dV: one per key block, from its own |V| and
// the |dO|, |delta| and |lambda| of the (head, query block) pairs that list it.
// The bound on |dS| lands at 2^15; values down to 2^-29 of it stay normal.
#include <cuda.h>
#include <cuda_fp16.h>

#include "rf_async.cuh"
#include "rf_device.cuh"
#include "rf_lists.cuh"
#include "rf_tiles.cuh"

namespace {

constexpr int kThreads = 640;      // four compute warpgroups and one of single-warp roles
constexpr int kCompute = 512;
constexpr int kMmaWarp = 16;       // TMEM allocation and every tcgen05.mma
constexpr int kLoadWarp = 17;      // every load
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kBoxBytes = RF_BLOCK * 128;
constexpr uint32_t kHalfBox = 64 * 128;  // bytes of a 64-row box
constexpr int kQStages = 4;              // dQ: 64-row stages of K and V
constexpr int kKvStages = 3;             // dK/dV: 64-row stages of Q, dO and the rows' numbers
constexpr uint32_t kStatBytes = 4 * 64 * 4;

struct BwdArgs {
  RfGeomDev g;
  RfOrder order;
  const int32_t* sel_idx;
  const int32_t* sel_num;
  const float* lambda;       // [n1]
  const float* stats;        // [n1][t_qblk][2][4][64]: -lse_1, -lse_2, delta_1, delta_2 of 64 rows
  const uint32_t* bits;      // [n1][t_qblk][words]
  const float* do_row;       // fp16: largest |dO| of a row, [n1][t_qblk][128]
  const float2* do_blk;      // fp16: {largest |dO|, |delta|} of a block, [n1][t_qblk]
  const float* v_blk;        // fp16: largest |V| of a block, [n2][t_qblk]
  int words;
  uint16_t* dq;
  uint16_t* dk;
  uint16_t* dv;
  uint32_t* status;
  float scale;
  float sl2;                 // scale * log2(e)
};

// fp16: the power-of-two exponents that A (|A| <= 1 + |lambda| <= 2 ml) and dS (at
// most `bound`) carry through the 16-bit rounding.
__device__ __forceinline__ float lambda_size(float lambda) {
  const float l = fabsf(lambda);
  return l < INFINITY ? fmaxf(1.f, l) : 1.f;
}
__device__ __forceinline__ int carry_a(float ml) { return max(14 - rf_ceil_log2(ml), -100); }
__device__ __forceinline__ int carry_ds(float bound) {
  return bound > 0.f && bound < INFINITY ? min(max(15 - rf_ceil_log2(bound), -100), 100) : 0;
}

template <int D>
struct __align__(1024) DqSmem {
  static constexpr int kTileBytes = RF_BLOCK * D * 2;
  uint8_t q[kTileBytes];
  uint8_t d_o[kTileBytes];
  uint8_t k[kQStages][kTileBytes / 2];
  uint8_t v[kQStages][kTileBytes / 2];
  uint64_t bar_q, bar_aux;
  uint64_t bar_full[kQStages];  // step t's tiles landed, and its TMEM columns free (dQ of t - 2 complete)
  uint64_t bar_empty[kQStages];
  uint64_t bar_sd_full[2];  // S_1, S_2 and dA of a step computed, by parity
  uint64_t bar_ds_full[2];  // dS_1 and dS_2 of it stored, by parity
  uint64_t bar_final, bar_drain;
  uint32_t tmem_base;
  int abort;
  int n_valid;
  int first;  // this CTA's part of the list begins here
  uint32_t v_max;            // fp16: largest |V| of the listed blocks, as fp32 bits
  float f_row[RF_BLOCK];     // what a row of the accumulated dQ is multiplied by
  int list[RF_MAX_KV_LIST];
};

template <int D>
struct __align__(1024) DkvSmem {
  static constexpr int kTileBytes = RF_BLOCK * D * 2;
  uint8_t k[kTileBytes];
  uint8_t v[kTileBytes];
  uint8_t q[kKvStages][kTileBytes / 2];
  uint8_t d_o[kKvStages][kTileBytes / 2];
  uint8_t a[2][RF_BLOCK * 128];  // A^T of a step: 128 keys x 64 queries, K-major, 128-byte swizzle
  float stats[kKvStages][4][64];
  float lam[kKvStages];
  uint64_t bar_kv, bar_aux;
  uint64_t bar_full[kKvStages];  // step t's tiles landed, A's buffer and dS's slot free (products of t - 2), and
                                 // S_1, S_2 and dA of t - 1 read into registers
  uint64_t bar_empty[kKvStages];
  uint64_t bar_sd_full;  // S_1, S_2 and dA of a step computed, the rows' numbers there
  uint64_t bar_ew[2];    // A, dS_1, dS_2 of a step stored, by parity
  uint64_t bar_final, bar_drain;
  uint32_t tmem_base;
  int abort;
  int n_items;
  uint32_t ds_max, lam_max;  // fp16: bound on |dS| and largest |lambda| (at least 1) over the items, as fp32 bits
};

// Zeroes rows [nrows, 64) of a 64-row tile's 128-byte-wide boxes (a row is 128
// bytes of each box whatever the swizzle), by one warp.
__device__ __forceinline__ void zero_tail(uint8_t* tile, int boxes, int nrows, int lane) {
  const int per_box = (64 - nrows) * 8;
  for (int x = 0; x < boxes; ++x)
    for (int i = lane; i < per_box; i += 32)
      *reinterpret_cast<uint4*>(tile + x * kHalfBox + nrows * 128 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
}

// dS of 16 keys of one map for one query row: P = 2^(s * sl2 + nlse), then
// P * (dA * c - dc), rounded to 16 bits and packed.
template <bool kBf16, bool kFull>
__device__ __forceinline__ void ds_chunk(const uint32_t* s, const uint32_t* da, int vr, float sl2,
                                         float nlse, float c, float dc, uint32_t* pk) {
  const uint64_t sl = rf_f2(__float_as_uint(sl2), __float_as_uint(sl2));
  const uint64_t nl = rf_f2(__float_as_uint(nlse), __float_as_uint(nlse));
  const uint64_t cc = rf_f2(__float_as_uint(c), __float_as_uint(c));
  const uint64_t nd = rf_f2(__float_as_uint(-dc), __float_as_uint(-dc));
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    float x0, x1, y0, y1;
    rf_f2_split(rf_fma2(rf_f2(s[i], s[i + 1]), sl, nl), x0, x1);
    const uint64_t p = rf_f2(__float_as_uint(rf_ex2(x0)), __float_as_uint(rf_ex2(x1)));
    rf_f2_split(rf_mul2(p, rf_fma2(rf_f2(da[i], da[i + 1]), cc, nd)), y0, y1);
    if (!kFull) {
      y0 = i < vr ? y0 : 0.f;
      y1 = i + 1 < vr ? y1 : 0.f;
    }
    pk[i >> 1] = rf_pack2<kBf16>(y0, y1);
  }
}

// N consecutive accumulator columns of this thread's row, times f, to 16 bits.
template <int N, bool kBf16>
__device__ __forceinline__ void store_row(uint32_t taddr, bool have, float f, bool live, uint16_t* dst) {
  uint32_t o[N];
  if (have) {
    if constexpr (N == 32) tmem_ld32(taddr, o);
    else                   tmem_ld16(taddr, o);
    tmem_wait_ld();
  }
  if (!live) return;
#pragma unroll
  for (int c = 0; c < N / 8; ++c) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = have ? rf_pack2<kBf16>(f * __uint_as_float(o[8 * c + 2 * i]), f * __uint_as_float(o[8 * c + 2 * i + 1]))
                  : 0u;
    reinterpret_cast<uint4*>(dst)[c] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Rows [rank, rank + 1) * 128 / size of the sum over the cluster's partial
// [128][D] buffers, times factor(row), to 16 bits; by the 512 computing threads.
template <int D, bool kBf16, class Factor, class Row>
__device__ __forceinline__ void merge_rows(uint32_t buf, int size, int rank, int live_rows, Factor factor, Row row_ptr) {
  const int rows = RF_BLOCK / size;
  for (int i = threadIdx.x; i < rows * (D / 4); i += kCompute) {
    const int row = rank * rows + i / (D / 4), c = i % (D / 4);
    if (row >= live_rows) break;  // rows come in order
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < size; ++k) {
      const float4 p = cluster_ld4(cluster_addr(buf + part_off<D>(row, c), k));
      s.x += p.x;
      s.y += p.y;
      s.z += p.z;
      s.w += p.w;
    }
    const float f = factor(row);
    *reinterpret_cast<uint2*>(row_ptr(row) + 4 * c) =
        make_uint2(rf_pack2<kBf16>(f * s.x, f * s.y), rf_pack2<kBf16>(f * s.z, f * s.w));
  }
}

// dQ.  A step is 64 keys of a listed block.  Two sets of TMEM columns (S_1, S_2,
// dA: 64 each at [192 p, +192)) alternate, so that a step's products run while
// the step before is computed.  Thread = query row = TMEM lane; warpgroup e takes
// keys [16 e, +16) of the step, one 16-wide slice of the reduction of dQ, of both
// maps, and writes dS_1 and dS_2 over S_1 and S_2 columns that it alone has read.
// dQ accumulates at [384, 512): 64 columns per map (at D = 64 both maps' columns
// of the product, half of them unused, so that every operand starts at a box).
// A barrier check costs its warp 100 cycles and more: one barrier tells the
// issuing warp that a step's tiles have landed and that its columns are free.
// Bound: per 128 x 128 block the tensor pipe about 2,300 cycles (an N = 64
// product with both operands in shared memory takes 54 cycles, 35 with A in
// TMEM, 32 by its arithmetic); the ex2 unit 2,048.  Measured: about 3,500 (2.70 ms
// for 5 heads of the (21, 30, 52) grid with 512 text rows at s = 0.8; 3.04 ms with
// one map per warpgroup, a barrier each for K, V and dQ, and 128-row stages).
template <int D, bool kBf16>
__global__ void __launch_bounds__(kThreads, 1)
    rf_diff_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                      const __grid_constant__ BwdArgs a) {
  using Smem = DqSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  constexpr int kBoxes = D * 2 / 128;
  constexpr uint32_t kTileBytes = Smem::kTileBytes;
  constexpr uint32_t kDq = 384;

  const RfGeomDev& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int n, tb;
  const int size = (int)cluster_size(), rank = (int)cluster_rank();  // CTAs sharing this list
  rf_cta_item(g, a.order, g.n1, blockIdx.x / size, n, tb);
  const RfSeqDev& s = g.seq[rf_seq_of_qblk(g, tb)];
  const int nblk = s.n_pb + s.nb;
  const int gk = n / (g.n1 / g.n2);
  int q_r0, q_rows;
  rf_block_span(s, tb - s.qblk_off, q_r0, q_rows);
  volatile int* abort = &sm.abort;
  const bool bnsd = g.layout == RF_LAYOUT_BNSD;
  auto coords = [&](int heads, int head, int r0, int& c1, int& c2) {
    if (bnsd) { c1 = r0; c2 = s.batch_idx * heads + head; }
    else      { c1 = head; c2 = (int)s.row_off + r0; }
  };

  if (threadIdx.x == 0) {
    mbar_init(rf_smem_u32(&sm.bar_q), 1);
    mbar_init(rf_smem_u32(&sm.bar_aux), 1);
    for (int i = 0; i < kQStages; ++i) {
      mbar_init(rf_smem_u32(&sm.bar_full[i]), 2);
      mbar_init(rf_smem_u32(&sm.bar_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(rf_smem_u32(&sm.bar_sd_full[i]), 1);
      mbar_init(rf_smem_u32(&sm.bar_ds_full[i]), kCompute);
    }
    mbar_init(rf_smem_u32(&sm.bar_final), 1);
    mbar_init(rf_smem_u32(&sm.bar_drain), 1);
    sm.abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(rf_smem_u32(&sm.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  const size_t row_id = (size_t)tb * g.n1 + n;
  const int32_t* row = a.sel_idx + row_id * g.max_kv;
  const int num_raw = a.sel_num[row_id];
  const int num = num_raw < 0 ? 0 : (num_raw > g.max_kv ? g.max_kv : num_raw);
  const uint32_t expired = *reinterpret_cast<volatile uint32_t*>(a.status + RF_STATUS_TIMEOUT);
  for (int c = threadIdx.x; c < g.max_kv; c += kThreads) sm.list[c] = row[c];
  __syncthreads();
  if (warp == 0) {
    int bad = 0;  // counted by the forward pass and the preparation
    const int cnt = compact_ascending(sm.list, num, nblk, lane, &bad);
    if (lane == 0) {
      const bool stopped = expired != 0;
      sm.first = cnt * rank / size;
      sm.n_valid = stopped ? 0 : cnt * (rank + 1) / size - sm.first;
    }
    if constexpr (!kBf16) {  // over the whole list: the same in every CTA that shares it
      const float* vb = a.v_blk + (size_t)gk * g.t_qblk + s.qblk_off;
      uint32_t top = 0u;
      for (int c = lane; c < cnt; c += 32) top = max(top, __float_as_uint(vb[sm.list[c]]));
      top = __reduce_max_sync(0xffffffffu, top);
      if (lane == 0) sm.v_max = top;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const int nv = sm.n_valid;
  const int* list = sm.list + sm.first;
  const int vr_last = s.Lp - (s.n_pb - 1) * RF_BLOCK;  // valid rows of the last prefix block

  if (warp >= 16) {
    if (warp == kLoadWarp && nv > 0) {
      // ---------------- loads (lane 0; the warp zeroes a partial block's tail) ----------------
      int c1, c2;
      if (lane == 0) {
        coords(g.n1, n, q_r0, c1, c2);
        mbar_arrive_expect_tx(rf_smem_u32(&sm.bar_q), 2 * kTileBytes);
        for (int x = 0; x < kBoxes; ++x) {
          tma_load_3d(rf_smem_u32(sm.q + x * kBoxBytes), &tm_q, rf_smem_u32(&sm.bar_q), x * 64, c1, c2);
          tma_load_3d(rf_smem_u32(sm.d_o + x * kBoxBytes), &tm_do, rf_smem_u32(&sm.bar_q), x * 64, c1, c2);
        }
      }
      volatile int no_abort = 0;
      int issued = 0, tails = 0;
      for (int t = 0; t < 2 * nv; ++t) {  // 64 rows of a key block each
        const int st = t % kQStages;
        if (t >= kQStages && !warp_wait(rf_smem_u32(&sm.bar_empty[st]), ((t / kQStages) & 1) ^ 1, abort)) {
          if (lane == 0) record_timeout(abort, a.status, 4);
          break;
        }
        const int blk = list[t >> 1];
        // K rows past the prefix meet dS = 0 in dQ: they must be finite.
        const int left = blk == s.n_pb - 1 ? vr_last - 64 * (t & 1) : 64;
        const bool tail = left < 64;
        const uint32_t bar = rf_smem_u32(tail ? &sm.bar_aux : &sm.bar_full[st]);
        if (lane == 0) {
          int r0, nr;
          rf_block_span(s, blk, r0, nr);
          coords(g.n2, gk, r0 + 64 * (t & 1), c1, c2);
          mbar_arrive_expect_tx(bar, kTileBytes);
          for (int x = 0; x < kBoxes; ++x) {
            tma_load_3d(rf_smem_u32(sm.v[st] + x * kHalfBox), &tm_v, bar, x * 64, c1, c2);
            tma_load_3d(rf_smem_u32(sm.k[st] + x * kHalfBox), &tm_k, bar, x * 64, c1, c2);
          }
        }
        __syncwarp();
        if (tail) {  // the halves of at most one block
          const bool landed = warp_wait(bar, tails & 1, &no_abort);
          ++tails;
          if (landed) zero_tail(sm.k[st], kBoxes, max(left, 0), lane);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (!landed) record_timeout(abort, a.status, 4);
            mbar_arrive(rf_smem_u32(&sm.bar_full[st]));
          }
          __syncwarp();
        }
        issued = t + 1;
      }
      if (*abort) {
        // Let this warp's own copies land before the shared memory goes away.
        warp_wait(rf_smem_u32(&sm.bar_q), 0, &no_abort);
        for (int t = (issued > kQStages ? issued - kQStages : 0); t < issued; ++t)
          warp_wait(rf_smem_u32(&sm.bar_full[t % kQStages]), (t / kQStages) & 1, &no_abort);
      }
    } else if (warp == kMmaWarp && nv > 0) {
      // ---------------- tcgen05.mma issue ----------------
      const uint32_t fmt = kBf16 ? 1u : 0u;
      const uint32_t id_sd = umma_idesc_f16(fmt, 128, 64, 0);
      const uint32_t id_dq = umma_idesc_f16(fmt, 128, 64, 1);
      const uint64_t dq = umma_desc_sw128(rf_smem_u32(sm.q), 16, 1024);
      const uint64_t ddo = umma_desc_sw128(rf_smem_u32(sm.d_o), 16, 1024);
      const uint64_t dk0 = umma_desc_sw128(rf_smem_u32(sm.k[0]), 16, 1024);
      const uint64_t dv0 = umma_desc_sw128(rf_smem_u32(sm.v[0]), 16, 1024);
      const uint64_t dkn0 = umma_desc_sw128(rf_smem_u32(sm.k[0]), kHalfBox, 1024);
      const int nt = 2 * nv;
      auto issue_sd = [&](int t) {  // S_1, S_2 and dA of step t
        const uint32_t d = tmem + 192 * (t & 1);
        const uint64_t st = (uint64_t)((t % kQStages) * (kTileBytes / 2) >> 4);
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk) {
            const uint32_t byte = w * D + kk * 32, box = byte >> 7, in = byte & 127;
            mma_ss(d + 64 * w, dq + ((box * kBoxBytes + in) >> 4), dk0 + st + ((box * kHalfBox + in) >> 4), id_sd,
                   kk > 0 ? 1u : 0u);
          }
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t in = (kk & 3) * 32, box = kk >> 2;
          mma_ss(d + 128, ddo + ((box * kBoxBytes + in) >> 4), dv0 + st + ((box * kHalfBox + in) >> 4), id_sd,
                 kk > 0 ? 1u : 0u);
        }
        tc_commit(rf_smem_u32(&sm.bar_sd_full[t & 1]));
      };
      // the first two steps' columns are free from the start
      if (lane < 2) mbar_arrive(rf_smem_u32(&sm.bar_full[lane]));
      __syncwarp();
      bool ok = warp_wait<true>(rf_smem_u32(&sm.bar_q), 0, abort) &&
                warp_wait<true>(rf_smem_u32(&sm.bar_full[0]), 0, abort);
      if (ok) {
        tc_fence_after();
        if (elect_one()) issue_sd(0);
        __syncwarp();
      }
      for (int t = 0; ok && t < nt; ++t) {
        const int h = t & 1, st = t % kQStages;
        if (t + 1 < nt) {
          if (!warp_wait<true>(rf_smem_u32(&sm.bar_full[(t + 1) % kQStages]), ((t + 1) / kQStages) & 1, abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) issue_sd(t + 1);
          __syncwarp();
        }
        if (!warp_wait<true>(rf_smem_u32(&sm.bar_ds_full[h]), (t >> 1) & 1, abort)) { ok = false; break; }
        tc_fence_after();
        if (elect_one()) {
          const uint64_t dk = dkn0 + (uint64_t)(st * (kTileBytes / 2) >> 4);
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ts(tmem + kDq + 64 * w, tmem + 192 * h + 64 * w + 16 * kk,
                     dk + (uint64_t)(((D == 128 ? w : 0) * kHalfBox + kk * 2048) >> 4), id_dq,
                     (t > 0 || kk > 0) ? 1u : 0u);
          tc_commit(rf_smem_u32(&sm.bar_empty[st]));
          if (t + 2 < nt) tc_commit(rf_smem_u32(&sm.bar_full[(t + 2) % kQStages]));
        }
        __syncwarp();
      }
      if (!ok && lane == 0) record_timeout(abort, a.status, 6);
      if (elect_one()) {
        tc_commit(rf_smem_u32(&sm.bar_final));
        tc_commit(rf_smem_u32(&sm.bar_drain));
      }
      __syncwarp();
      volatile int no_abort = 0;
      warp_wait(rf_smem_u32(&sm.bar_drain), 0, &no_abort);
    }
  } else {
    // ---------------- dS and epilogue ----------------
    const int e = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float* str = a.stats + ((size_t)n * g.t_qblk + tb) * (4 * RF_BLOCK) + (r >> 6) * 256 + (r & 63);
    const float lam = a.lambda[n];
    int es = 0;  // |dS| <= max(1, |lambda|) (|dA| + |delta|), each of them at most D |dO| |V| of this row and its list
    if constexpr (!kBf16)
      es = carry_ds(2.0f * D * __uint_as_float(sm.v_max) * lambda_size(lam) *
                    a.do_row[((size_t)n * g.t_qblk + tb) * RF_BLOCK + r]);
    const float c1 = kBf16 ? 1.f : rf_pow2(es), c2 = -lam * c1;
    const float nlse1 = str[0], nlse2 = str[64], dc1 = c1 * str[128], dc2 = c2 * str[192];
    bool ok = true;
    for (int t = 0; t < 2 * nv; ++t) {
      if (!warp_wait<true>(rf_smem_u32(&sm.bar_sd_full[t & 1]), (t >> 1) & 1, abort)) { ok = false; break; }
      tc_fence_after();
      const uint32_t base = lane_base + 192 * (t & 1) + 16 * e;
      // valid keys of this thread's 16 (all of them but in the partial prefix block)
      const int vr = (list[t >> 1] == s.n_pb - 1 ? vr_last : RF_BLOCK) - 64 * (t & 1) - 16 * e;
      uint32_t s1[16], s2[16], da[16], pk[8];
      tmem_ld16(base, s1);
      tmem_ld16(base + 64, s2);
      tmem_ld16(base + 128, da);
      tmem_wait_ld();
      tmem_pin16(s1);
      tmem_pin16(s2);
      tmem_pin16(da);
      if (vr >= 16) ds_chunk<kBf16, true>(s1, da, vr, a.sl2, nlse1, c1, dc1, pk);
      else          ds_chunk<kBf16, false>(s1, da, vr, a.sl2, nlse1, c1, dc1, pk);
      tmem_st8(base, pk);
      if (vr >= 16) ds_chunk<kBf16, true>(s2, da, vr, a.sl2, nlse2, c2, dc2, pk);
      else          ds_chunk<kBf16, false>(s2, da, vr, a.sl2, nlse2, c2, dc2, pk);
      tmem_st8(base + 64, pk);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(rf_smem_u32(&sm.bar_ds_full[t & 1]));
    }
    if (!ok) record_timeout(abort, a.status, 7);
    wait_for_previous();  // dK and dV are complete when this kernel is
    const bool have = nv > 0 && !*abort && warp_wait(rf_smem_u32(&sm.bar_final), 0, abort) && !*abort;
    if (have) tc_fence_after();
    constexpr int kN = D / 4;  // columns each warpgroup writes
    const int col = e * kN;
    const uint32_t tcol = lane_base + kDq + (D == 128 ? col : 64 * (col >> 5) + col);
    const float f = a.scale * (kBf16 ? 1.f : rf_pow2(-es));
    if (size == 1) {
      store_row<kN, kBf16>(tcol, have, f, r < q_rows,
                           a.dq + rf_row_offset(g, s, g.n1, n, q_r0 + min(r, q_rows - 1)) + col);
    } else {
      // the partial dQ where the tiles were (every copy and product is complete)
      store_part<D, kN>(rf_smem_u32(sm.q), tcol, have, r, col);
      if (e == 0) sm.f_row[r] = f;
      cluster_sync();
      merge_rows<D, kBf16>(rf_smem_u32(sm.q), size, rank, q_rows, [&](int row) { return sm.f_row[row]; },
                           [&](int row) { return a.dq + rf_row_offset(g, s, g.n1, n, q_r0 + row); });
      cluster_sync();  // the others have read this CTA's part
    }
  }
  if (size > 1 && warp >= 16) {
    cluster_sync();
    cluster_sync();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// dK and dV.  M = the block's 128 keys (thread = key = TMEM lane); a step is 64
// query rows of one (head, query block) that lists the block: S_w^T and dA^T
// with N = 64, A^T, dS_w^T from registers, then dV += A^T dO, dK_w += dS_w^T Q_w.
// TMEM: dV at [256, 256 + D), dK at [384, 512) (per map 64 columns, as dQ), and
// four 64-column slots in which a step's S_1, S_2 and dA take turns: the next
// step's go into the free slot and into dA's and S_1's as soon as this step's
// numbers are in registers, long before they are used up; dS_1 and dS_2 are
// written over S_2, each thread over columns that it alone has read, and A^T goes
// through shared memory (two buffers).  So a step's elements hardly ever wait for
// its products, and the warpgroups drift apart until one's exponentials run under
// another's arithmetic.  A barrier check costs its warp 100 to 200 cycles, so
// there are few: one per step for a computing thread, two for the issuing warp.
// Warpgroup e takes queries [16 e, +16) of the step, which is one 16-wide slice
// of the reduction of dV and dK.
// Rows that a query block does not have carry -lse = -inf (P = 0); their Q and
// dO rows are zeroed in shared memory, so that nothing infinite meets that 0.
// Bound: per 128 x 128 block and head the tensor pipe about 2,800 cycles (S and dA
// at N = 64, see above), the ex2 unit 2,048.  Measured: about 4,400 (3.31 ms on the
// layer above; 5.57 ms when a step's products waited for A and dS of the one
// before, 3.57 ms with the exponentials of all columns before the rest).  The
// issuing warp and the computing threads are both busy nearly all of that time;
// 128-query steps, whose products are fed faster, do not fit: S_1, S_2 and dA
// beside dV and dK would take 640 TMEM columns of 512.
template <int D, bool kBf16>
__global__ void __launch_bounds__(kThreads, 1)
    rf_diff_dkv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                       const __grid_constant__ BwdArgs a) {
  using Smem = DkvSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  constexpr int kBoxes = D * 2 / 128;
  constexpr uint32_t kTileBytes = Smem::kTileBytes;
  constexpr uint32_t kDv = 256, kDk = 384;

  const RfGeomDev& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int gk, tb;  // tb: the key block
  const int size = (int)cluster_size(), rank = (int)cluster_rank();  // CTAs sharing these items
  rf_cta_item(g, a.order, g.n2, blockIdx.x / size, gk, tb);
  const RfSeqDev& s = g.seq[rf_seq_of_qblk(g, tb)];
  wait_for_previous();
  if (threadIdx.x == 0) launch_dependents();  // dQ reads nothing of this kernel: it may fill the last wave
  const int group = g.n1 / g.n2;
  int k_r0, k_rows;
  rf_block_span(s, tb - s.qblk_off, k_r0, k_rows);
  volatile int* abort = &sm.abort;
  const bool bnsd = g.layout == RF_LAYOUT_BNSD;
  auto coords = [&](int heads, int head, int r0, int& c1, int& c2) {
    if (bnsd) { c1 = r0; c2 = s.batch_idx * heads + head; }
    else      { c1 = head; c2 = (int)s.row_off + r0; }
  };

  if (threadIdx.x == 0) {
    mbar_init(rf_smem_u32(&sm.bar_kv), 1);
    mbar_init(rf_smem_u32(&sm.bar_aux), 1);
    for (int i = 0; i < kKvStages; ++i) {
      mbar_init(rf_smem_u32(&sm.bar_full[i]), 2 + kCompute);
      mbar_init(rf_smem_u32(&sm.bar_empty[i]), 1);
    }
    mbar_init(rf_smem_u32(&sm.bar_sd_full), 2);  // the products' commit, and the issuing warp itself
    mbar_init(rf_smem_u32(&sm.bar_ew[0]), kCompute);
    mbar_init(rf_smem_u32(&sm.bar_ew[1]), kCompute);
    mbar_init(rf_smem_u32(&sm.bar_final), 1);
    mbar_init(rf_smem_u32(&sm.bar_drain), 1);
    sm.abort = 0;
    sm.n_items = 0;
    sm.ds_max = 0u;
    sm.lam_max = __float_as_uint(1.f);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(rf_smem_u32(&sm.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  __syncthreads();
  // (head of the group, query block) pairs that list this key block
  int mine = 0;
  float ds_top = 0.f, lam_top = 1.f;
  const float v_top = kBf16 ? 0.f : D * a.v_blk[(size_t)gk * g.t_qblk + tb];
  for (int i = threadIdx.x; i < group * a.words; i += kThreads) {
    const int hh = i / a.words, wd = i - hh * a.words, n = gk * group + hh;
    uint32_t word = a.bits[((size_t)n * g.t_qblk + tb) * a.words + wd];
    mine += __popc(word);
    if constexpr (!kBf16) {
      if (word) {
        const float ml = lambda_size(a.lambda[n]);
        const float2* blk = a.do_blk + (size_t)n * g.t_qblk + s.qblk_off + wd * 32;
        lam_top = fmaxf(lam_top, ml);
        for (; word; word &= word - 1) {
          const float2 m = blk[__ffs(word) - 1];
          ds_top = fmaxf(ds_top, ml * fmaf(v_top, m.x, m.y));  // |dA| + |delta|
        }
      }
    }
  }
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0 && mine) atomicAdd(&sm.n_items, mine);
  if constexpr (!kBf16) {  // positive numbers order as their bits do
    const uint32_t dt = __reduce_max_sync(0xffffffffu, __float_as_uint(ds_top));
    const uint32_t lt = __reduce_max_sync(0xffffffffu, __float_as_uint(lam_top));
    if (lane == 0) {
      atomicMax(&sm.ds_max, dt);
      atomicMax(&sm.lam_max, lt);
    }
  }
  const bool stopped = *reinterpret_cast<volatile uint32_t*>(a.status + RF_STATUS_TIMEOUT) != 0;
  tc_fence_before();
  const int any_stopped = __syncthreads_or(stopped ? 1 : 0);
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const int i0 = sm.n_items * rank / size;  // this CTA's items: [i0, i0 + ni)
  const int ni = any_stopped ? 0 : sm.n_items * (rank + 1) / size - i0;
  const int ea = kBf16 ? 0 : carry_a(__uint_as_float(sm.lam_max)), es = kBf16 ? 0 : carry_ds(__uint_as_float(sm.ds_max));

  if (warp >= 16) {
    if (warp == kLoadWarp && ni > 0) {
      // ---------------- loads: K and V once, then Q, dO and the rows' numbers per item ----------------
      volatile int no_abort = 0;
      int c1, c2;
      if (lane == 0) {
        coords(g.n2, gk, k_r0, c1, c2);
        mbar_arrive_expect_tx(rf_smem_u32(&sm.bar_kv), 2 * kTileBytes);
        for (int x = 0; x < kBoxes; ++x) {
          tma_load_3d(rf_smem_u32(sm.k + x * kBoxBytes), &tm_k, rf_smem_u32(&sm.bar_kv), x * 64, c1, c2);
          tma_load_3d(rf_smem_u32(sm.v + x * kBoxBytes), &tm_v, rf_smem_u32(&sm.bar_kv), x * 64, c1, c2);
        }
      }
      __syncwarp();
      int t = 0, tails = 0, skip = i0;
      bool ok = true;
      for (int hh = 0; ok && hh < group && t < 2 * ni; ++hh) {
        const int n = gk * group + hh;
        const float lam = a.lambda[n];
        const uint32_t* bw = a.bits + ((size_t)n * g.t_qblk + tb) * a.words;
        for (int wd = 0; ok && wd < a.words && t < 2 * ni; ++wd) {
          uint32_t word = bw[wd];
          const int here = __popc(word);
          if (skip >= here) {
            skip -= here;
            continue;
          }
          while (ok && word && t < 2 * ni) {
            const int qb = wd * 32 + __ffs(word) - 1;
            word &= word - 1;
            if (skip > 0) {
              --skip;
              continue;
            }
            int r0, nr;
            rf_block_span(s, qb, r0, nr);
            for (int h = 0; h < 2; ++h, ++t) {  // 64 rows of the query block each
              const int st = t % kKvStages;
              if (t >= kKvStages && !warp_wait(rf_smem_u32(&sm.bar_empty[st]), ((t / kKvStages) & 1) ^ 1, abort)) {
                if (lane == 0) record_timeout(abort, a.status, 8);
                ok = false;
                break;
              }
              const int left = nr - 64 * h;
              const bool tail = left < 64;
              const uint32_t bar = rf_smem_u32(tail ? &sm.bar_aux : &sm.bar_full[st]);
              if (lane == 0) {
                sm.lam[st] = lam;
                coords(g.n1, n, r0 + 64 * h, c1, c2);
                mbar_arrive_expect_tx(bar, kTileBytes + kStatBytes);
                for (int x = 0; x < kBoxes; ++x) {
                  tma_load_3d(rf_smem_u32(sm.q[st] + x * kHalfBox), &tm_q, bar, x * 64, c1, c2);
                  tma_load_3d(rf_smem_u32(sm.d_o[st] + x * kHalfBox), &tm_do, bar, x * 64, c1, c2);
                }
                bulk_load(rf_smem_u32(&sm.stats[st][0][0]),
                          a.stats + (((size_t)n * g.t_qblk + s.qblk_off + qb) * 2 + h) * 256, kStatBytes, bar);
              }
              __syncwarp();
              if (tail) {  // the halves of at most one query block per head
                const bool landed = warp_wait(bar, tails & 1, &no_abort);
                ++tails;
                if (landed) {
                  zero_tail(sm.q[st], kBoxes, max(left, 0), lane);
                  zero_tail(sm.d_o[st], kBoxes, max(left, 0), lane);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                  if (!landed) record_timeout(abort, a.status, 8);
                  mbar_arrive(rf_smem_u32(&sm.bar_full[st]));
                }
                __syncwarp();
              }
            }
          }
        }
      }
      if (*abort) {
        warp_wait(rf_smem_u32(&sm.bar_kv), 0, &no_abort);
        for (int i = (t > kKvStages ? t - kKvStages : 0); i < t; ++i)
          warp_wait(rf_smem_u32(&sm.bar_full[i % kKvStages]), (i / kKvStages) & 1, &no_abort);
      }
    } else if (warp == kMmaWarp && ni > 0) {
      // ---------------- tcgen05.mma issue ----------------
      const uint32_t fmt = kBf16 ? 1u : 0u;
      const uint32_t id_s = umma_idesc_f16(fmt, 128, 64, 0);
      const uint32_t id_dk = umma_idesc_f16(fmt, 128, 64, 1);
      const uint32_t id_dv = umma_idesc_f16(fmt, 128, D, 1);
      const uint64_t dk = umma_desc_sw128(rf_smem_u32(sm.k), 16, 1024);
      const uint64_t dv = umma_desc_sw128(rf_smem_u32(sm.v), 16, 1024);
      const uint64_t dq0 = umma_desc_sw128(rf_smem_u32(sm.q[0]), 16, 1024);
      const uint64_t do0 = umma_desc_sw128(rf_smem_u32(sm.d_o[0]), 16, 1024);
      const uint64_t dqn0 = umma_desc_sw128(rf_smem_u32(sm.q[0]), kHalfBox, 1024);
      const uint64_t don0 = umma_desc_sw128(rf_smem_u32(sm.d_o[0]), kHalfBox, 1024);
      const uint64_t da_t = umma_desc_sw128(rf_smem_u32(sm.a[0]), 16, 1024);
      const int nt = 2 * ni;
      // slots of step t: S_1, S_2, dA (the fourth takes the next S_1)
      auto slot = [&](int t, int which) -> uint32_t {
        const uint32_t tab = which == 0 ? 0x2130u : (which == 1 ? 0x3021u : 0x1302u);
        return tmem + 64u * ((tab >> (4 * (t & 3))) & 15u);
      };
      auto tile_off = [&](int t) -> uint64_t { return (uint64_t)((t % kKvStages) * (kTileBytes / 2) >> 4); };
      auto issue_sd = [&](int t) {  // S_1, S_2 and dA of step t
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint64_t b = dq0 + tile_off(t);
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk) {
            const uint32_t byte = w * D + kk * 32, box = byte >> 7, in = byte & 127;
            mma_ss(slot(t, w), dk + ((box * kBoxBytes + in) >> 4), b + ((box * kHalfBox + in) >> 4), id_s,
                   kk > 0 ? 1u : 0u);
          }
        }
        const uint64_t b = do0 + tile_off(t);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t in = (kk & 3) * 32, box = kk >> 2;
          mma_ss(slot(t, 2), dv + ((box * kBoxBytes + in) >> 4), b + ((box * kHalfBox + in) >> 4), id_s, kk > 0 ? 1u : 0u);
        }
        // The arrival hands on what this thread has seen: the step's numbers in
        // shared memory, and A's buffer read.
        mbar_arrive(rf_smem_u32(&sm.bar_sd_full));
        tc_commit(rf_smem_u32(&sm.bar_sd_full));
      };
      // the first two steps' buffer and slot are free from the start
      if (lane < 2) mbar_arrive(rf_smem_u32(&sm.bar_full[lane]));
      __syncwarp();
      bool ok = warp_wait<true>(rf_smem_u32(&sm.bar_kv), 0, abort) &&
                warp_wait<true>(rf_smem_u32(&sm.bar_full[0]), 0, abort);
      if (ok) {
        tc_fence_after();
        if (elect_one()) issue_sd(0);
        __syncwarp();
      }
      for (int t = 0; ok && t < nt; ++t) {
        if (t + 1 < nt) {
          if (!warp_wait<true>(rf_smem_u32(&sm.bar_full[(t + 1) % kKvStages]), ((t + 1) / kKvStages) & 1, abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) issue_sd(t + 1);
          __syncwarp();
        }
        if (!warp_wait<true>(rf_smem_u32(&sm.bar_ew[t & 1]), (t >> 1) & 1, abort)) { ok = false; break; }
        tc_fence_after();
        if (elect_one()) {
          const uint64_t bo = don0 + tile_off(t), bq = dqn0 + tile_off(t);
          const uint32_t sb = slot(t, 1);
          const uint32_t acc = t > 0 ? 1u : 0u;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss(tmem + kDv, da_t + (uint64_t)(((t & 1) * (RF_BLOCK * 128) + kk * 32) >> 4),
                   bo + (uint64_t)(kk * 2048 >> 4), id_dv, kk > 0 ? 1u : acc);
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ts(tmem + kDk + 64 * w, sb + 16 * kk + 8 * (1 - w),
                     bq + (uint64_t)(((D == 128 ? w : 0) * kHalfBox + kk * 2048) >> 4), id_dk, kk > 0 ? 1u : acc);
          tc_commit(rf_smem_u32(&sm.bar_empty[t % kKvStages]));
          if (t + 2 < nt) tc_commit(rf_smem_u32(&sm.bar_full[(t + 2) % kKvStages]));
        }
        __syncwarp();
      }
      if (!ok && lane == 0) record_timeout(abort, a.status, 9);
      if (elect_one()) {
        tc_commit(rf_smem_u32(&sm.bar_final));
        tc_commit(rf_smem_u32(&sm.bar_drain));
      }
      __syncwarp();
      volatile int no_abort = 0;
      warp_wait(rf_smem_u32(&sm.bar_drain), 0, &no_abort);
    }
  } else {
    // ---------------- A, dS and epilogue ----------------
    const int e = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint64_t sl = rf_f2(__float_as_uint(a.sl2), __float_as_uint(a.sl2));
    const float up_a = (float)ea, up_s = kBf16 ? 1.f : rf_scale_pow2(1.f, es - ea);
    const uint64_t ua = rf_f2(__float_as_uint(up_a), __float_as_uint(up_a));
    const uint64_t us = rf_f2(__float_as_uint(up_s), __float_as_uint(up_s));
    const uint64_t neg1 = rf_f2(__float_as_uint(-1.f), __float_as_uint(-1.f));
    const uint32_t stats0 = rf_smem_u32(&sm.stats[0][0][0]) + 64u * e;
    // this thread's two 16-byte chunks of its key's row of A^T
    const uint32_t a_row = rf_smem_u32(sm.a[0]) + 128u * r;
    const uint32_t a_c0 = a_row + 16u * ((2 * e) ^ (r & 7)), a_c1 = a_row + 16u * ((2 * e + 1) ^ (r & 7));
    bool ok = true;
    if (ni > 0) mbar_arrive(rf_smem_u32(&sm.bar_full[0]));  // nothing to read before the first step
    for (int t = 0; t < 2 * ni; ++t) {
      const uint32_t sh = 4 * (t & 3);
      const uint32_t s1c = lane_base + 64u * ((0x2130u >> sh) & 15u) + 16 * e;
      const uint32_t s2c = lane_base + 64u * ((0x3021u >> sh) & 15u) + 16 * e;
      const uint32_t dac = lane_base + 64u * ((0x1302u >> sh) & 15u) + 16 * e;
      const int st = t % kKvStages;
      // this thread's 16 queries' numbers: -lse_1, -lse_2, delta_1, delta_2, 256 bytes apart
      const uint32_t num = stats0 + (uint32_t)st * kStatBytes;
      if (!warp_wait<true>(rf_smem_u32(&sm.bar_sd_full), t & 1, abort)) { ok = false; break; }
      tc_fence_after();
      uint32_t s1[16], s2[16], da[16];
      tmem_ld16(s1c, s1);
      tmem_ld16(s2c, s2);
      tmem_ld16(dac, da);
      tmem_wait_ld();
      tmem_pin16(s1);
      tmem_pin16(s2);
      tmem_pin16(da);
      tc_fence_before();
      mbar_arrive(rf_smem_u32(&sm.bar_full[(t + 1) % kKvStages]));
      // All of a column group's work together: the exponentials of one group run
      // under the arithmetic of another.
      const float nlam = -lds_f(rf_smem_u32(&sm.lam[0]) + 4u * st);
      const uint64_t nl = rf_f2(__float_as_uint(nlam), __float_as_uint(nlam));
      uint32_t out_a[8], out[16];  // A; dS_2 in [0, 8) and dS_1 in [8, 16)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        uint64_t l1[2], l2[2], d1[2], d2[2];
        lds_2x2(num + 4 * i, l1[0], l1[1]);
        lds_2x2(num + 256 + 4 * i, l2[0], l2[1]);
        lds_2x2(num + 512 + 4 * i, d1[0], d1[1]);
        lds_2x2(num + 768 + 4 * i, d2[0], d2[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int c = i + 2 * k;
          uint64_t x = rf_fma2(rf_f2(s1[c], s1[c + 1]), sl, l1[k]), y = rf_fma2(rf_f2(s2[c], s2[c + 1]), sl, l2[k]);
          if constexpr (!kBf16) {
            x = rf_add2(x, ua);
            y = rf_add2(y, ua);
          }
          float f0, f1;
          rf_f2_split(x, f0, f1);
          const uint64_t p1 = rf_f2(__float_as_uint(rf_ex2(f0)), __float_as_uint(rf_ex2(f1)));
          rf_f2_split(y, f0, f1);
          const uint64_t p2 = rf_mul2(nl, rf_f2(__float_as_uint(rf_ex2(f0)), __float_as_uint(rf_ex2(f1))));
          rf_f2_split(rf_add2(p1, p2), f0, f1);
          out_a[c >> 1] = rf_pack2<kBf16>(f0, f1);
          const uint64_t dd = rf_f2(da[c], da[c + 1]);
          uint64_t t1 = rf_fma2(d1[k], neg1, dd), t2 = rf_fma2(d2[k], neg1, dd);
          if constexpr (!kBf16) {
            t1 = rf_mul2(t1, us);
            t2 = rf_mul2(t2, us);
          }
          rf_f2_split(rf_mul2(p1, t1), f0, f1);
          out[8 + (c >> 1)] = rf_pack2<kBf16>(f0, f1);
          rf_f2_split(rf_mul2(p2, t2), f0, f1);
          out[c >> 1] = rf_pack2<kBf16>(f0, f1);
        }
      }
      sts128(a_c0 + (t & 1) * (RF_BLOCK * 128), out_a);
      sts128(a_c1 + (t & 1) * (RF_BLOCK * 128), out_a + 4);
      fence_async_smem();
      tmem_st16(s2c, out);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(rf_smem_u32(&sm.bar_ew[t & 1]));
    }
    if (!ok) record_timeout(abort, a.status, 10);
    const bool have = ni > 0 && !*abort && warp_wait(rf_smem_u32(&sm.bar_final), 0, abort) && !*abort;
    if (have) tc_fence_after();
    constexpr int kN = D / 4;
    const int col = e * kN;
    const size_t off = rf_row_offset(g, s, g.n2, gk, k_r0 + min(r, k_rows - 1)) + col;
    const bool live = r < k_rows;
    const float fv = kBf16 ? 1.f : rf_pow2(-ea), fk = a.scale * (kBf16 ? 1.f : rf_pow2(-es));
    const uint32_t kcol = lane_base + kDk + (D == 128 ? col : 64 * (col >> 5) + col);
    if (size == 1) {
      store_row<kN, kBf16>(lane_base + kDv + col, have, fv, live, a.dv + off);
      store_row<kN, kBf16>(kcol, have, fk, live, a.dk + off);
    } else {
      // the partial dV and dK where the tiles were (every copy and product is complete)
      const uint32_t bv = rf_smem_u32(sm.k), bk = bv + RF_BLOCK * D * 4;
      store_part<D, kN>(bv, lane_base + kDv + col, have, r, col);
      store_part<D, kN>(bk, kcol, have, r, col);
      cluster_sync();
      merge_rows<D, kBf16>(bv, size, rank, k_rows, [&](int) { return fv; },
                           [&](int row) { return a.dv + rf_row_offset(g, s, g.n2, gk, k_r0 + row); });
      merge_rows<D, kBf16>(bk, size, rank, k_rows, [&](int) { return fk; },
                           [&](int row) { return a.dk + rf_row_offset(g, s, g.n2, gk, k_r0 + row); });
      cluster_sync();  // the others have read this CTA's part
    }
  }
  if (size > 1 && warp >= 16) {
    cluster_sync();
    cluster_sync();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Per (query block, head): packs each row's -lse_1, -lse_2, delta_1 and delta_2
// (rows the block does not have: -inf, -inf, 0, 0), sums delta_2 over the
// block's rows in a fixed order, and sets this query block's bit for every key
// block it lists.  fp16: also the largest finite |dO| of each row, |dO| and |delta|
// of the block, and (CTAs past t_qblk * n1) |V| of each key block.
// 10 D bytes per row and head, read at about half of the copy rate (65 us for 213 MB;
// issue slots 46 % busy).
template <int D, bool kBf16>
__global__ void __launch_bounds__(256, D == 128 && kBf16 ? 8 : 1)
    rf_diff_prep_bwd_kernel(const __grid_constant__ RfGeomDev g, const int32_t* sel_idx,
                            const int32_t* sel_num, const uint16_t* d_o, const uint16_t* v,
                            const float* maps, const float* lse, long long rows_total,
                            int words, float* stats, uint32_t* bits,
                            float* dlam, float* do_row, float2* do_blk, float* v_blk, uint32_t* status) {
  wait_for_previous();
  __shared__ int list[RF_MAX_KV_LIST];
  __shared__ float part[8];
  __shared__ float2 part_top[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kPer = D / 32;  // columns per lane
  const bool is_v = (int)blockIdx.x >= g.t_qblk * g.n1;
  const int bid = is_v ? (int)blockIdx.x - g.t_qblk * g.n1 : (int)blockIdx.x;
  const int n = bid / g.t_qblk, tb = bid % g.t_qblk;
  const RfSeqDev& s = g.seq[rf_seq_of_qblk(g, tb)];
  const int lq = tb - s.qblk_off;
  int r0, nrows;
  rf_block_span(s, lq, r0, nrows);
  auto decode = [](uint32_t u) { return kBf16 ? __uint_as_float(u << 16) : __half2float(__ushort_as_half((unsigned short)u)); };
  float2 top = make_float2(0.f, 0.f);  // of |dO| (or |V|) and |delta|
  auto finite_max = [](float& t, float x) {
    const float m = fabsf(x);
    if (m < INFINITY) t = fmaxf(t, m);
  };
  // the largest over the block's warps, by thread 0 (after a barrier)
  auto block_top = [&]() {
    float2 t = part_top[0];
    for (int i = 1; i < 8; ++i) t = make_float2(fmaxf(t.x, part_top[i].x), fmaxf(t.y, part_top[i].y));
    return t;
  };
  if (is_v) {
    for (int r = warp; r < nrows; r += 8) {
      const uint16_t* p = v + rf_row_offset(g, s, g.n2, n, r0 + r) + lane * kPer;
#pragma unroll
      for (int c = 0; c < kPer; ++c) finite_max(top.x, decode(p[c]));
    }
    top.x = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top.x)));
    if (lane == 0) part_top[warp] = top;
    __syncthreads();
    if (threadIdx.x == 0) v_blk[(size_t)n * g.t_qblk + tb] = block_top().x;
    return;
  }
  const size_t row_id = (size_t)tb * g.n1 + n;
  const int num_raw = sel_num[row_id];
  const int num = num_raw < 0 ? 0 : (num_raw > g.max_kv ? g.max_kv : num_raw);
  for (int c = threadIdx.x; c < num; c += 256) list[c] = sel_idx[row_id * g.max_kv + c];
  __syncthreads();
  float* st = stats + ((size_t)n * g.t_qblk + tb) * (4 * RF_BLOCK);
  const size_t map2 = (size_t)rows_total * g.n1 * D;
  const size_t lrow = (g.layout == RF_LAYOUT_BNSD ? (size_t)s.batch_idx * s.L : (size_t)s.row_off) + r0;
  float sum2 = 0.f;
  for (int r = warp; r < RF_BLOCK; r += 8) {
    float e1 = 0.f, e2 = 0.f, row_top = 0.f;
    if (r < nrows) {
      const size_t off = rf_row_offset(g, s, g.n1, n, r0 + r) + lane * kPer;
      uint16_t u[kPer];
      float m1[kPer], m2[kPer];
      if constexpr (kPer == 4) {
        *reinterpret_cast<uint2*>(u) = *reinterpret_cast<const uint2*>(d_o + off);
        *reinterpret_cast<float4*>(m1) = *reinterpret_cast<const float4*>(maps + off);
        *reinterpret_cast<float4*>(m2) = *reinterpret_cast<const float4*>(maps + map2 + off);
      } else {
        *reinterpret_cast<uint32_t*>(u) = *reinterpret_cast<const uint32_t*>(d_o + off);
        *reinterpret_cast<float2*>(m1) = *reinterpret_cast<const float2*>(maps + off);
        *reinterpret_cast<float2*>(m2) = *reinterpret_cast<const float2*>(maps + map2 + off);
      }
#pragma unroll
      for (int c = 0; c < kPer; ++c) {
        const float x = decode(u[c]);
        e1 = fmaf(x, m1[c], e1);
        e2 = fmaf(x, m2[c], e2);
        if constexpr (!kBf16) finite_max(row_top, x);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        e1 += __shfl_xor_sync(0xffffffffu, e1, d);
        e2 += __shfl_xor_sync(0xffffffffu, e2, d);
      }
    }
    sum2 += e2;
    if constexpr (!kBf16) {
      row_top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(row_top)));
      top.x = fmaxf(top.x, row_top);
      finite_max(top.y, e1);
      finite_max(top.y, e2);
      if (lane == 0) do_row[((size_t)n * g.t_qblk + tb) * RF_BLOCK + r] = row_top;
    }
    if (lane == 0) {
      float* o = st + (r >> 6) * 256 + (r & 63);
      o[0] = r < nrows ? -lse[(size_t)n * rows_total + lrow + r] : -INFINITY;
      o[64] = r < nrows ? -lse[((size_t)g.n1 + n) * rows_total + lrow + r] : -INFINITY;
      o[128] = e1;
      o[192] = e2;
    }
  }
  if (lane == 0) part[warp] = sum2;
  if (!kBf16 && lane == 0) part_top[warp] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += part[i];
    dlam[(size_t)n * g.t_qblk + tb] = sum;
    if constexpr (!kBf16) do_blk[(size_t)n * g.t_qblk + tb] = block_top();
  }
  if (warp == 0) {
    int bad = (lane == 0 && num != num_raw) ? 1 : 0;
    const int cnt = compact_ascending(list, num, s.n_pb + s.nb, lane, &bad);
    bad = __reduce_add_sync(0xffffffffu, bad);
    if (lane == 0 && bad) atomicAdd(status + RF_STATUS_BAD_INDEX, (uint32_t)bad);
    for (int c = lane; c < cnt; c += 32)
      atomicOr(bits + ((size_t)n * g.t_qblk + s.qblk_off + list[c]) * words + (lq >> 5), 1u << (lq & 31));
  }
}

// dlambda[n] = -sum over the query blocks of their sums of delta_2, in a fixed order.
__global__ void __launch_bounds__(256) rf_diff_dlam_kernel(const float* part, int t_qblk, float* dlambda) {
  wait_for_previous();
  __shared__ float red[8];
  float sum = 0.f;
  for (int i = threadIdx.x; i < t_qblk; i += 256) sum += part[(size_t)blockIdx.x * t_qblk + i];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 1; i < 8; ++i) sum += red[i];
    dlambda[blockIdx.x] = -sum;
  }
}

template <int D, bool kBf16>
rf_status_t launch_t(const rf_plan* p, const BwdArgs& a, const void* q_r, const void* k_r, const void* v_r,
                     const void* do_r, const float* maps, const float* lse, float* stats, uint32_t* bits,
                     float* dlam_part, float* dlambda, cudaStream_t st) {
  const RfGeomDev& g = p->g;
  const long long gq = (long long)g.t_qblk * g.n1, gkv = (long long)g.t_qblk * g.n2;
  if (gq + gkv > 0x7FFFFFFFll) return rf_fail(RF_ERR_INVALID_ARG, "grid too large");
  // [0]: 128-row boxes (the tiles a CTA keeps), [1]: 64-row boxes (those it streams)
  CUtensorMap mq[2], mk[2], mv[2], mo[2];
  rf_status_t s;
  for (int i = 0; i < 2; ++i) {
    const int rows = i ? 64 : RF_BLOCK;
    if ((s = make_map(&mq[i], p, q_r, g.n1, kElemPlan, rows)) != RF_OK) return s;
    if ((s = make_map(&mk[i], p, k_r, g.n2, kElemPlan, rows)) != RF_OK) return s;
    if ((s = make_map(&mv[i], p, v_r, g.n2, kElemPlan, rows)) != RF_OK) return s;
    if ((s = make_map(&mo[i], p, do_r, g.n1, kElemPlan, rows)) != RF_OK) return s;
  }
  size_t sq = sizeof(DqSmem<D>) + 1024, skv = sizeof(DkvSmem<D>) + 1024;
  if (sq < 120 * 1024) sq = 120 * 1024;    // each CTA takes all 512 TMEM columns: one per SM
  if (skv < 120 * 1024) skv = 120 * 1024;
  constexpr auto kq = rf_diff_dq_kernel<D, kBf16>;
  constexpr auto kkv = rf_diff_dkv_kernel<D, kBf16>;
  if ((s = rf_prepare_kernel<kq>(sq, "cudaFuncSetAttribute(rf_diff_dq_kernel)")) != RF_OK) return s;
  if ((s = rf_prepare_kernel<kkv>(skv, "cudaFuncSetAttribute(rf_diff_dkv_kernel)")) != RF_OK) return s;
  if (cudaMemsetAsync(bits, 0, (size_t)gq * a.words * 4, st) != cudaSuccess)
    return rf_check_launch("cudaMemsetAsync(rf_diff backward)");
  const unsigned prep = (unsigned)(gq + (kBf16 ? 0 : gkv));
  if ((s = rf_launch_dependent(rf_diff_prep_bwd_kernel<D, kBf16>, dim3(prep), 256, st, "rf_diff_prep_bwd_kernel", g,
                               a.sel_idx, a.sel_num, static_cast<const uint16_t*>(do_r),
                               static_cast<const uint16_t*>(v_r), maps, lse, (long long)p->rows_total, a.words, stats, bits,
                               dlam_part, const_cast<float*>(a.do_row), const_cast<float2*>(a.do_blk),
                               const_cast<float*>(a.v_blk), a.status)) != RF_OK)
    return s;
  if ((s = rf_launch_dependent(rf_diff_dlam_kernel, dim3((unsigned)g.n1), 256, st, "rf_diff_dlam_kernel",
                               (const float*)dlam_part, g.t_qblk, dlambda)) != RF_OK)
    return s;
  if ((s = rf_launch_split(kkv, gkv, rf_split(g, g.n2, g.n1 / g.n2), kThreads, skv, st, "rf_diff_dkv_kernel", mq[1],
                           mk[0], mv[0], mo[1], a)) != RF_OK)
    return s;
  return rf_launch_split(kq, gq, rf_split(g, g.n1, 1), kThreads, sq, st, "rf_diff_dq_kernel", mq[0], mk[1], mv[1],
                         mo[0], a);
}

}  // namespace

rf_status_t rf_launch_diff_bwd(const rf_plan* p, const void* q_r, const void* k_r, const void* v_r,
                               const int32_t* sel_idx, const int32_t* sel_num, const float* lambda,
                               float scale, const float* maps, const float* lse, const void* do_r,
                               void* dq_r, void* dk_r, void* dv_r, float* dlambda, void* ws,
                               cudaStream_t st) {
  const RfDiffLayout lay = rf_diff_layout(p);
  char* w = static_cast<char*>(ws);
  float* stats = reinterpret_cast<float*>(w + lay.stats);
  uint32_t* bits = reinterpret_cast<uint32_t*>(w + lay.bits);
  float* part = reinterpret_cast<float*>(w + lay.dlam);
  BwdArgs a;
  a.g = p->g;
  a.order = rf_order(p->g);
  a.sel_idx = sel_idx;
  a.sel_num = sel_num;
  a.lambda = lambda;
  a.stats = stats;
  a.bits = bits;
  a.do_row = reinterpret_cast<const float*>(w + lay.do_row);
  a.do_blk = reinterpret_cast<const float2*>(w + lay.do_blk);
  a.v_blk = reinterpret_cast<const float*>(w + lay.v_blk);
  a.words = lay.words;
  a.dq = static_cast<uint16_t*>(dq_r);
  a.dk = static_cast<uint16_t*>(dk_r);
  a.dv = static_cast<uint16_t*>(dv_r);
  a.status = reinterpret_cast<uint32_t*>(w + p->off_status);
  a.scale = scale;
  a.sl2 = scale * kLog2e;
  const bool bf = p->dtype == RF_BF16;
  if (p->g.d == 128)
    return bf ? launch_t<128, true>(p, a, q_r, k_r, v_r, do_r, maps, lse, stats, bits, part, dlambda, st)
              : launch_t<128, false>(p, a, q_r, k_r, v_r, do_r, maps, lse, stats, bits, part, dlambda, st);
  return bf ? launch_t<64, true>(p, a, q_r, k_r, v_r, do_r, maps, lse, stats, bits, part, dlambda, st)
            : launch_t<64, false>(p, a, q_r, k_r, v_r, do_r, maps, lse, stats, bits, part, dlambda, st);
}
