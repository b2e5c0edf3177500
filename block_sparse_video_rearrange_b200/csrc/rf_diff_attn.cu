// Differential attention over the selected key blocks on sm_100a tensor cores.
//
// Per query head n, with Q_1, Q_2 the first and second half of the head's
// columns (K_1, K_2 likewise) and one V shared by both maps:
//   P_w = softmax(scale * Q_w K_w^T) over the rows of the listed key blocks,
//   O   = (P_1 - lambda_n P_2) V,
// computed as O_1 - lambda O_2 with O_w = P_w V kept in fp32 until the single
// rounding of the difference: the two maps agree in most of their mass, so a
// rounding of O_1 and O_2 before the subtraction would be magnified in what is
// left.  For the same reason P enters the product as f16 (11 significant bits)
// whatever the input type: with bf16 inputs and near-uniform maps a bf16 P
// gives a relative error of 6e-3, an f16 P under 2e-3, of which 1.65e-3 is the
// output's own rounding (short fp16 lists: see kFineBlocks).  tcgen05.mma takes A
// and B of one type, so V is read from f16 copies by block
// (rf_diff_prep_v_kernel): v * 2^-e, exact for every value down to 2^-29 of the
// block's largest, with the rows past a block's end zero (an unselected row's NaN
// must not meet P = 0).
//
// One CTA = one (query block of 128 rows, query head).  The work
// items of a CTA are (key block b, map w) in the order (0,1), (0,2), (1,1), ...
// so that K_b and V_b are loaded once for both maps; softmax group w of 128
// threads (thread = query row = TMEM lane) owns map w with its own running
// maximum, sum and accumulator.  Roles, barriers, the lazy rescale and the
// register split are those of the single-map kernel (rf_attn.cu):
//   warps 0-3 / 4-7  softmax of map 1 / 2
//   warp 8           TMA producer of Q (once) and K_b, 3-stage ring
//   warp 9           TMEM allocation, S = Q_w K_w^T (the half-width reduction)
//   warp 10          TMA producer of the f16 V_b, 2-stage ring
//   warp 11          O_w += P_w V_b
// TMEM columns: S at [0, 128) (both maps in turn), P_w at [128 + 64 w, +64),
// O_w at [256 + 128 w, +D).
//
// Bound: per 128 x 128 block and head the tensor pipe needs 544 cycles for both S
// and 2 x 512 for P V at D = 128, the ex2 unit 2,048 for 32,768 exponentials.
// Measured: about 3,100 (5 heads of the (21, 30, 52) grid with 512 text rows at
// s = 0.8: 2.33-2.40 ms in isolation, 1,100 TFLOP/s of S and P V products).  Each
// map's softmax is a chain (S, row maximum, exponentials, P) whose parts beside
// the exponentials the other map covers only in part: moving 12 % of the
// exponentials to the FMA pipe gained 1 % on the long lists, 25 % nothing, and 50
// % lost 4 %, so all of them stay on the ex2 unit.  A CTA costs about 11,000
// cycles beside its list; few long lists are shared by a cluster (rf_split).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "rf_async.cuh"
#include "rf_device.cuh"
#include "rf_lists.cuh"
#include "rf_tiles.cuh"

namespace {

constexpr int kThreads = 384;
constexpr int kKWarp = 8;
constexpr int kSWarp = 9;
constexpr int kVWarp = 10;
constexpr int kPvWarp = 11;
constexpr int kLaunchRegs = 168;
constexpr uint32_t kSoftmaxRegs = 216;
constexpr uint32_t kOtherRegs = 72;
static_assert(2 * 128 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs,
              "register split exceeds the launch allocation");
constexpr int kStagesK = 3;
constexpr int kStagesV = 2;
constexpr uint32_t kPCol = 128;
constexpr uint32_t kOCol = 256;
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: P stays below 2^9
constexpr float kNoRow = -1e30f;           // a row's references before its first score
// P of block b is 2^(s + d_b - m_o), d_b <= 0 the block's V exponent below the
// list's largest and m_o the row's running maximum of s + d_b (in steps of one):
// the accumulator's exponent follows what the row adds up, and P's f16 rounding is
// relative to the row's largest product.  The row's sum has a reference m_l of its
// own, the running maximum of s, and gets P times 2^(m_o - d_b - m_l).  Where d_b is
// so low (kFar) that P could leave fp32's range before that, rows whose P is zero in
// f16 all over the block (below 2^-kGone) take their exponentials about the block's
// own maximum instead, for the sum alone.
constexpr int kFar = -60;
constexpr float kGone = 40.0f;
constexpr uint32_t kBoxBytes = RF_BLOCK * 128;
// fp16 lists of up to this many blocks take P in two f16 parts, twice the P V
// products, for fp16 results at their own rounding, 2e-4, instead of 7e-4 where the
// maps are near-uniform: a rounding of P that a short list does not average away.
// It costs (us a call, D = 128, two parts against one): 8 heads of 77, 300 and 1,024
// keys 13.4 / 12.0, 20.2 / 15.9 and 28.8 / 21.9; 160 heads, which fill the GPU, 23.8 /
// 21.2, 70 / 55 and 314 / 206.  On a long list it would cost more (2.48 against
// 4.15 ms, 5 heads of the Wan-shaped grid).
constexpr int kFineBlocks = 8;

template <int D>
struct __align__(1024) DiffSmem {
  static constexpr int kTileBytes = RF_BLOCK * D * 2;
  uint8_t q[kTileBytes];
  uint8_t k[kStagesK][kTileBytes];
  uint8_t v[kStagesV][kTileBytes];
  uint64_t bar_q;
  uint64_t bar_k_full[kStagesK], bar_k_empty[kStagesK];
  uint64_t bar_v_full[kStagesV], bar_v_empty[kStagesV];
  uint64_t bar_s_full[2];                 // S of (b, w) computed, one barrier per map
  uint64_t bar_s_free;                    // S read into registers
  uint64_t bar_p_half[2], bar_p_full[2];  // P of map w stored, first half / all
  uint64_t bar_ph_done[2];                // two parts: the first half's products complete, its P columns free
  uint64_t bar_pv_done[2];                // O_w += P_w V_b complete
  uint64_t bar_final;
  uint64_t bar_drain;
  uint32_t tmem_base;
  int abort;
  int n_valid;
  int first;  // this CTA's part of the list begins here
  int vexp_max;
  int fine;   // P in two f16 parts
  float row_m[2][RF_BLOCK], row_l[2][RF_BLOCK];  // reference m_l and sum of each map's row
  float row_o[2][RF_BLOCK];                      // reference m_o of its accumulator
  int list[RF_MAX_KV_LIST];
  int vexp[RF_MAX_KV_LIST];  // by block of the sequence
};

struct DiffArgs {
  RfGeomDev g;
  RfOrder order;
  const int32_t* sel_idx;
  const int32_t* sel_num;
  const float* lambda;   // [n1]
  uint16_t* o_r;
  float* maps;           // training: O_1 and O_2, fp32 [2][shape of o_r], or null
  float* lse;            // training: log2 of the softmax sums, fp32 [2][n1][rows], or null
  long long rows_total;
  uint32_t* status;
  const int32_t* v_exp;  // [n2][t_qblk]
  float sl2;             // scale * log2(e)
};

__device__ __forceinline__ void softmax_bar_sync() {
  asm volatile("bar.sync 1, 256;" ::: "memory");  // the eight softmax warps
}

// p = 2^(s * sl2 + neg_m) for the 32 scores c0 .. c0 + 31 of a row (the first vr
// valid), rounded to f16 pairs (and masked, unless kFull) in the 16 TMEM columns at
// p_addr; the unrounded values go to the paired fp32 sums.
template <bool kFull>
__device__ __forceinline__ void quarter_exp(const uint32_t* sr, int c0, int vr, float sl2, float neg_m, uint32_t mask,
                                            uint32_t p_addr, uint64_t* acc) {
  const uint64_t sl2x2 = rf_f2(__float_as_uint(sl2), __float_as_uint(sl2));
  const uint64_t negm2 = rf_f2(__float_as_uint(neg_m), __float_as_uint(neg_m));
  uint32_t pk[16];
  if (!kFull && c0 >= vr) {  // nothing valid here (uniform over the CTA)
#pragma unroll
    for (int c = 0; c < 16; ++c) pk[c] = 0u;
    tmem_st16(p_addr, pk);
    return;
  }
#pragma unroll
  for (int c = 0; c < 32; c += 2) {
    float x0, x1;
    rf_f2_split(rf_fma2(rf_f2(sr[c0 + c], sr[c0 + c + 1]), sl2x2, negm2), x0, x1);
    float p0 = rf_ex2(x0), p1 = rf_ex2(x1);
    if (!kFull) {
      p0 = c0 + c < vr ? p0 : 0.f;
      p1 = c0 + c + 1 < vr ? p1 : 0.f;
    }
    acc[(c >> 1) & 3] = rf_add2(acc[(c >> 1) & 3], rf_f2(__float_as_uint(p0), __float_as_uint(p1)));
    pk[c >> 1] = rf_pack2<false>(p0, p1);
    if (!kFull) pk[c >> 1] &= mask;
  }
  tmem_st16(p_addr, pk);
}

// The same for an fp16 list in two parts: the f16 values at p_addr, what their
// rounding left, as f16 too, 32 columns on.
__device__ __forceinline__ void quarter_exp_fine(const uint32_t* sr, int c0, int vr, float sl2, float neg_m,
                                                 uint32_t p_addr, uint64_t* acc) {
  const uint64_t sl2x2 = rf_f2(__float_as_uint(sl2), __float_as_uint(sl2));
  const uint64_t negm2 = rf_f2(__float_as_uint(neg_m), __float_as_uint(neg_m));
  uint32_t pk[16], lo[16];
  if (c0 >= vr) {  // nothing valid here (uniform over the CTA)
#pragma unroll
    for (int c = 0; c < 16; ++c) pk[c] = 0u;
    tmem_st16(p_addr, pk);
    tmem_st16(p_addr + 32, pk);
    return;
  }
#pragma unroll
  for (int c = 0; c < 32; c += 2) {
    float x0, x1;
    rf_f2_split(rf_fma2(rf_f2(sr[c0 + c], sr[c0 + c + 1]), sl2x2, negm2), x0, x1);
    float p0 = rf_ex2(x0), p1 = rf_ex2(x1);
    p0 = c0 + c < vr ? p0 : 0.f;
    p1 = c0 + c + 1 < vr ? p1 : 0.f;
    acc[(c >> 1) & 3] = rf_add2(acc[(c >> 1) & 3], rf_f2(__float_as_uint(p0), __float_as_uint(p1)));
    pk[c >> 1] = rf_pack2<false>(p0, p1);
    const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&pk[c >> 1]));
    lo[c >> 1] = rf_pack2<false>(p0 - r.x, p1 - r.y);
  }
  tmem_st16(p_addr, pk);
  tmem_st16(p_addr + 32, lo);
}

// Exponent of the power of two an accumulator is multiplied by at the end; what is
// cut off below leaves fp32's range either way.
__device__ __forceinline__ int out_exp(float m, int vexp_max) { return max((int)m + max(vexp_max, -252), -252); }

__device__ __forceinline__ float acc_sum(const uint64_t* acc) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    rf_f2_split(acc[i], a, b);
    s += a + b;
  }
  return s;
}

template <int D, bool kBf16, bool kTrain>
__global__ void __launch_bounds__(kThreads, 1)
    rf_diff_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ DiffArgs a) {
  using Smem = DiffSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  constexpr int kBoxes = D * 2 / 128;
  constexpr uint32_t kTileBytes = Smem::kTileBytes;

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

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStagesK; ++i) {
      mbar_init(rf_smem_u32(&sm.bar_k_full[i]), 1);
      mbar_init(rf_smem_u32(&sm.bar_k_empty[i]), 1);
    }
    for (int i = 0; i < kStagesV; ++i) {
      mbar_init(rf_smem_u32(&sm.bar_v_full[i]), 1);
      mbar_init(rf_smem_u32(&sm.bar_v_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(rf_smem_u32(&sm.bar_s_full[i]), 1);
      mbar_init(rf_smem_u32(&sm.bar_p_half[i]), 128);
      mbar_init(rf_smem_u32(&sm.bar_p_full[i]), 128);
      mbar_init(rf_smem_u32(&sm.bar_ph_done[i]), 1);
      mbar_init(rf_smem_u32(&sm.bar_pv_done[i]), 1);
    }
    mbar_init(rf_smem_u32(&sm.bar_s_free), 128);
    mbar_init(rf_smem_u32(&sm.bar_final), 2);  // one commit from each issuing warp
    mbar_init(rf_smem_u32(&sm.bar_drain), 2);
    sm.abort = 0;
    fence_mbar_init();
  }
  const bool bnsd = g.layout == RF_LAYOUT_BNSD;
  auto coords = [&](int heads, int head, int r0, int& c1, int& c2) {
    if (bnsd) { c1 = r0; c2 = s.batch_idx * heads + head; }
    else      { c1 = head; c2 = (int)s.row_off + r0; }
  };
  if (warp == kKWarp && lane == 0) {
    // The Q tile does not depend on the selection: request it first thing.
    mbar_init(rf_smem_u32(&sm.bar_q), 1);
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    int c1, c2;
    coords(g.n1, n, q_r0, c1, c2);
    mbar_arrive_expect_tx(rf_smem_u32(&sm.bar_q), kTileBytes);
#pragma unroll
    for (int x = 0; x < kBoxes; ++x)
      tma_load_3d(rf_smem_u32(sm.q + x * kBoxBytes), &tm_q, rf_smem_u32(&sm.bar_q), x * 64, c1, c2);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == kSWarp) {
    tmem_alloc(rf_smem_u32(&sm.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  const size_t row_id = (size_t)tb * g.n1 + n;
  const int32_t* row = a.sel_idx + row_id * g.max_kv;
  wait_for_previous();  // the copies of V and their exponents, and what came before them
  // The whole row, its length and every block's exponent at once: one round trip.
  const int32_t* ve = a.v_exp + (size_t)gk * g.t_qblk + s.qblk_off;
  const int num_raw = a.sel_num[row_id];
  const float lam = a.lambda[n];
  const uint32_t expired = *reinterpret_cast<volatile uint32_t*>(a.status + RF_STATUS_TIMEOUT);
  for (int c = threadIdx.x; c < g.max_kv; c += kThreads) sm.list[c] = row[c];
  for (int c = threadIdx.x; c < nblk; c += kThreads) sm.vexp[c] = ve[c];
  const int num = num_raw < 0 ? 0 : (num_raw > g.max_kv ? g.max_kv : num_raw);
  __syncthreads();
  if (warp == 0) {
    int bad = (lane == 0 && num != num_raw) ? 1 : 0;
    const int cnt = compact_ascending(sm.list, num, nblk, lane, &bad);
    int vmax = -1000;
    for (int c = lane; c < cnt; c += 32) vmax = max(vmax, sm.vexp[sm.list[c]]);
    vmax = __reduce_max_sync(0xffffffffu, vmax);
    bad = __reduce_add_sync(0xffffffffu, bad);
    if (lane == 0) {
      const bool stopped = expired != 0;  // a wait that already expired in this workspace stops all work
      sm.first = cnt * rank / size;
      sm.n_valid = stopped ? 0 : cnt * (rank + 1) / size - sm.first;
      sm.vexp_max = vmax;
      sm.fine = !kBf16 && cnt <= kFineBlocks;
      if (bad && rank == 0) atomicAdd(a.status + RF_STATUS_BAD_INDEX, (uint32_t)bad);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const int nv = sm.n_valid;
  const int* list = sm.list + sm.first;
  const bool fine = !kBf16 && sm.fine;
  const int vr_last = s.Lp - (s.n_pb - 1) * RF_BLOCK;  // valid rows of the last prefix block
  if (warp >= 8) {
    reg_dealloc<kOtherRegs>();
    if ((warp == kKWarp || warp == kVWarp) && lane == 0 && nv > 0) {
      // ---------------- TMA producers ----------------
      const bool is_k = warp == kKWarp;
      const int stages = is_k ? kStagesK : kStagesV;
      uint8_t* tiles = is_k ? &sm.k[0][0] : &sm.v[0][0];
      uint64_t* full = is_k ? sm.bar_k_full : sm.bar_v_full;
      uint64_t* empty = is_k ? sm.bar_k_empty : sm.bar_v_empty;
      int issued = 0;
      for (int b = 0; b < nv; ++b) {
        const int st = b % stages;
        const uint32_t ph = (b / stages) & 1;
        if (b >= stages && !mbar_wait(rf_smem_u32(&empty[st]), ph ^ 1, abort)) {
          record_timeout(abort, a.status, is_k ? 0 : 1);
          break;
        }
        const uint32_t bar = rf_smem_u32(&full[st]);
        mbar_arrive_expect_tx(bar, kTileBytes);
        int c1, c2;
        if (is_k) {
          int r0, nr;
          rf_block_span(s, list[b], r0, nr);
          coords(g.n2, gk, r0, c1, c2);
        } else {
          c1 = 0;
          c2 = gk * g.t_qblk + s.qblk_off + list[b];
        }
        for (int x = 0; x < kBoxes; ++x)
          tma_load_3d(rf_smem_u32(tiles + st * kTileBytes + x * kBoxBytes),
                      is_k ? static_cast<const void*>(&tm_k) : static_cast<const void*>(&tm_v), bar, x * 64,
                      c1, c2);
        issued = b + 1;
      }
      if (*abort) {
        // Let this thread's own copies land before the shared memory goes away.
        volatile int no_abort = 0;
        if (is_k) mbar_wait(rf_smem_u32(&sm.bar_q), 0, &no_abort);
        for (int b = (issued > stages ? issued - stages : 0); b < issued; ++b)
          mbar_wait(rf_smem_u32(&full[b % stages]), (b / stages) & 1, &no_abort);
      }
    } else if ((warp == kSWarp || warp == kPvWarp) && nv > 0) {
      // ---------------- tcgen05.mma issue ----------------
      bool ok = true;
      if (warp == kSWarp) {
        const uint32_t idesc = umma_idesc_f16(kBf16 ? 1u : 0u, 128, 128, 0);
        const uint64_t dq = umma_desc_sw128(rf_smem_u32(sm.q), 16, 1024);
        const uint64_t dk0 = umma_desc_sw128(rf_smem_u32(sm.k[0]), 16, 1024);
        ok = warp_wait<true>(rf_smem_u32(&sm.bar_q), 0, abort);
        for (int j = 0; ok && j < 2 * nv; ++j) {
          const int b = j >> 1, w = j & 1, st = b % kStagesK;
          if (j > 0 && !warp_wait<true>(rf_smem_u32(&sm.bar_s_free), (j - 1) & 1, abort)) { ok = false; break; }
          if (w == 0 && !warp_wait<true>(rf_smem_u32(&sm.bar_k_full[st]), (b / kStagesK) & 1, abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            // S = Q_w K_w^T: the map's D / 2 columns, 16 per MMA
            const uint64_t dk = dk0 + (uint64_t)(st * (kTileBytes >> 4));
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk) {
              const int byte = w * D + kk * 32;  // of the row's 2 D bytes
              const uint32_t off = ((uint32_t)(byte >> 7) * kBoxBytes + (byte & 127)) >> 4;
              mma_ss(tmem, dq + off, dk + off, idesc, kk > 0 ? 1u : 0u);
            }
            tc_commit(rf_smem_u32(&sm.bar_s_full[w]));
            if (w == 1) tc_commit(rf_smem_u32(&sm.bar_k_empty[st]));
          }
          __syncwarp();
        }
      } else {
        const uint32_t idesc = umma_idesc_f16(0u, 128, D, 1u);
        const uint64_t dv0 = umma_desc_sw128(rf_smem_u32(sm.v[0]), kBoxBytes, 1024);
        for (int j = 0; ok && j < 2 * nv; ++j) {
          const int b = j >> 1, w = j & 1, st = b % kStagesV;
          const uint64_t dv = dv0 + (uint64_t)(st * (kTileBytes >> 4));
          const uint32_t a_p = tmem + kPCol + (uint32_t)(w * 64);
          const uint32_t d_o = tmem + kOCol + (uint32_t)(w * 128);
          // two halves of the key rows, as the softmax releases them
          if (!warp_wait<true>(rf_smem_u32(&sm.bar_p_half[w]), b & 1, abort)) { ok = false; break; }
          if (!warp_wait<true>(rf_smem_u32(&sm.bar_v_full[st]), (b / kStagesV) & 1, abort)) { ok = false; break; }
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ts(d_o, a_p + kk * 8, dv + (uint32_t)(kk * (2048 >> 4)), idesc, (b > 0 || kk > 0) ? 1u : 0u);
            if (fine) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) mma_ts(d_o, a_p + 32 + kk * 8, dv + (uint32_t)(kk * (2048 >> 4)), idesc, 1u);
              tc_commit(rf_smem_u32(&sm.bar_ph_done[w]));
            }
          }
          __syncwarp();
          if (!warp_wait<true>(rf_smem_u32(&sm.bar_p_full[w]), b & 1, abort)) { ok = false; break; }
          tc_fence_after();
          if (elect_one()) {
            const uint32_t a_p2 = fine ? a_p : a_p + 32;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ts(d_o, a_p2 + kk * 8, dv + (uint32_t)((kk + 4) * (2048 >> 4)), idesc, 1u);
            if (fine) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_ts(d_o, a_p + 32 + kk * 8, dv + (uint32_t)((kk + 4) * (2048 >> 4)), idesc, 1u);
            }
            if (w == 1) tc_commit(rf_smem_u32(&sm.bar_v_empty[st]));
            tc_commit(rf_smem_u32(&sm.bar_pv_done[w]));
          }
          __syncwarp();
        }
      }
      if (!ok && lane == 0) record_timeout(abort, a.status, 2);
      if (elect_one()) {
        tc_commit(rf_smem_u32(&sm.bar_final));
        tc_commit(rf_smem_u32(&sm.bar_drain));
      }
      __syncwarp();
      volatile int no_abort = 0;
      warp_wait(rf_smem_u32(&sm.bar_drain), 0, &no_abort);
    }
    if (warp == kKWarp && lane == 0 && nv == 0) {
      // Nothing to compute: the Q copy still has to land before the CTA exits.
      volatile int no_abort = 0;
      mbar_wait(rf_smem_u32(&sm.bar_q), 0, &no_abort);
    }
  } else {
    reg_alloc<kSoftmaxRegs>();
    // ---------------- softmax of map w + epilogue (warps 0-7) ----------------
    const int w = warp >> 2;
    const int r = (warp & 3) * 32 + lane;  // query row = TMEM lane
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t pcol = lane_base + kPCol + (uint32_t)(w * 64);
    const uint32_t ocol = lane_base + kOCol + (uint32_t)(w * 128);
    const float sl2 = a.sl2;
    const int vexp_max = sm.vexp_max;
    float m_o = kNoRow, m_l = kNoRow, l_run = 0.f;  // fp16 has no V exponents: one reference
    int step = 0;                                   // m_o - m_l
    bool ok = true;
    for (int b = 0; b < nv; ++b) {
      if (!warp_wait(rf_smem_u32(&sm.bar_s_full[w]), b & 1, abort)) { ok = false; break; }
      tc_fence_after();
      const int vr = (list[b] == s.n_pb - 1) ? vr_last : RF_BLOCK;
      const int d = kBf16 ? sm.vexp[list[b]] - vexp_max : 0;
      const bool plain = vr == RF_BLOCK && d >= kFar;
      uint32_t sr[128];
      tmem_ld32(lane_base, sr);
      tmem_ld32(lane_base + 32, sr + 32);
      tmem_ld32(lane_base + 64, sr + 64);
      tmem_ld32(lane_base + 96, sr + 96);
      tmem_wait_ld();
      tc_fence_before();
      mbar_arrive(rf_smem_u32(&sm.bar_s_free));
      const float mx = (vr == RF_BLOCK ? row_max<true>(sr, vr) : row_max<false>(sr, vr)) * sl2;
      if (b > 0) {
        if (!warp_wait(rf_smem_u32(&sm.bar_pv_done[w]), (b - 1) & 1, abort)) { ok = false; break; }
        tc_fence_after();
      }
      const float mo = kBf16 ? mx + (float)d : mx;
      if (__any_sync(0xffffffffu, mo > m_o + kRescaleThreshold || (kBf16 && mx > m_l + kRescaleThreshold))) {
        const float o_new = fmaxf(m_o, floorf(mo)), l_new = kBf16 ? fmaxf(m_l, floorf(mx)) : o_new;
        const float alpha = rf_ex2(m_o - o_new);
        l_run *= kBf16 ? rf_ex2(m_l - l_new) : alpha;
        m_o = o_new;
        m_l = l_new;
        step = kBf16 ? (int)(m_o - m_l) : 0;
        if (b > 0) {
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t o[32];
            tmem_ld32(ocol + c0, o);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
            tmem_st32(ocol + c0, o);
          }
        }
      }
      uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
      float neg_m = kBf16 ? (float)d - m_o : -m_o;
      uint32_t mask = ~0u;
      int up = step - d;
      if (fine) {
        // a half's two parts fill the map's P columns: the second half's go there
        // when the first half's products are complete
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 1) {
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(rf_smem_u32(&sm.bar_p_half[w]));
            if (!warp_wait(rf_smem_u32(&sm.bar_ph_done[w]), b & 1, abort)) { ok = false; break; }
            tc_fence_after();
          }
          quarter_exp_fine(sr, 64 * h, vr, sl2, neg_m, pcol, acc);
          quarter_exp_fine(sr, 64 * h + 32, vr, sl2, neg_m, pcol + 16, acc);
        }
        if (!ok) break;
      } else {
        if (plain) {
          quarter_exp<true>(sr, 0, vr, sl2, neg_m, mask, pcol, acc);
          quarter_exp<true>(sr, 32, vr, sl2, neg_m, mask, pcol + 16, acc);
        } else {
          if (d < kFar && mx < m_o - (float)d - kGone) {
            neg_m = -fmaxf(floorf(mx), kNoRow);
            up = (int)(-neg_m - m_l);
            mask = 0u;
          }
          quarter_exp<false>(sr, 0, vr, sl2, neg_m, mask, pcol, acc);
          quarter_exp<false>(sr, 32, vr, sl2, neg_m, mask, pcol + 16, acc);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(rf_smem_u32(&sm.bar_p_half[w]));
        if (plain) {
          quarter_exp<true>(sr, 64, vr, sl2, neg_m, mask, pcol + 32, acc);
          quarter_exp<true>(sr, 96, vr, sl2, neg_m, mask, pcol + 48, acc);
        } else {
          quarter_exp<false>(sr, 64, vr, sl2, neg_m, mask, pcol + 32, acc);
          quarter_exp<false>(sr, 96, vr, sl2, neg_m, mask, pcol + 48, acc);
        }
      }
      // what is below 2^-126 does not count in a sum of at least 2^-9
      l_run = kBf16 ? fmaf(acc_sum(acc), rf_pow2(max(up, -126)), l_run) : l_run + acc_sum(acc);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(rf_smem_u32(&sm.bar_p_full[w]));
    }
    if (!ok) record_timeout(abort, a.status, 3);

    // Epilogue: O_w = 2^(e_max + m_o - m_l) (accumulator) / l, then O_1 - lambda O_2.
    sm.row_m[w][r] = m_l;
    sm.row_l[w][r] = l_run;
    sm.row_o[w][r] = m_o;
    softmax_bar_sync();
    const bool have = nv > 0 && !*abort && warp_wait(rf_smem_u32(&sm.bar_final), 0, abort) && !*abort;
    const size_t lrow = bnsd ? (size_t)s.batch_idx * s.L : (size_t)s.row_off;
    const size_t map2 = (size_t)a.rows_total * g.n1 * D;
    if (have) tc_fence_after();
    const uint32_t parts = rf_smem_u32(sm.q);  // [2][128][D] fp32 where the tiles were
    if (nv == 0) {  // every product is complete, and so is every copy but that of Q where no product waited for it
      volatile int no_abort = 0;
      warp_wait(rf_smem_u32(&sm.bar_q), 0, &no_abort);
    }
    if (size == 1) {
      // Through shared memory, so that whole rows leave in one piece: written by the
      // row's own thread, 16 bytes here and there, the two fp32 maps took 11,000
      // cycles a CTA (now 2,000).
      const float f = have ? 1.0f / l_run : 0.f;
      const int up = out_exp(m_o - m_l, vexp_max);
      const int cols = (warp & 3) * 32 < q_rows ? D : 0;  // none of a warp without rows
#pragma unroll 1
      for (int c0 = 0; c0 < cols; c0 += 32) {
        uint32_t o[32];
        if (have) {
          tmem_ld32(ocol + c0, o);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(rf_scale_pow2(f * __uint_as_float(o[c]), up));
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = 0u;
        }
#pragma unroll
        for (int c = 0; c < 8; ++c)
          sts128(parts + (uint32_t)w * (RF_BLOCK * D * 4) + part_off<D>(r, c0 / 4 + c), o + 4 * c);
      }
      if constexpr (kTrain) {
        if (r < q_rows)
          a.lse[((size_t)w * g.n1 + n) * a.rows_total + lrow + q_r0 + r] = have ? m_l + log2f(l_run) : INFINITY;
      }
      softmax_bar_sync();
#pragma unroll 4
      for (int i = threadIdx.x; i < q_rows * (D / 4); i += 256) {
        const int row = i / (D / 4), c = i % (D / 4);
        const float4 o1 = lds128(parts + part_off<D>(row, c));
        const float4 o2 = lds128(parts + RF_BLOCK * D * 4 + part_off<D>(row, c));
        const size_t off = rf_row_offset(g, s, g.n1, n, q_r0 + row) + 4 * c;
        if constexpr (kTrain) {
          *reinterpret_cast<float4*>(a.maps + off) = o1;
          *reinterpret_cast<float4*>(a.maps + map2 + off) = o2;
        }
        *reinterpret_cast<uint2*>(a.o_r + off) =
            make_uint2(rf_pack2<kBf16>(fmaf(-lam, o2.x, o1.x), fmaf(-lam, o2.y, o1.y)),
                       rf_pack2<kBf16>(fmaf(-lam, o2.z, o1.z), fmaf(-lam, o2.w, o1.w)));
      }
    } else {
      // group w leaves its O_w there
      if (!have) {
        sm.row_m[w][r] = -INFINITY;
        sm.row_l[w][r] = 0.f;
      }
      const uint32_t buf = parts + (uint32_t)w * (RF_BLOCK * D * 4);
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) store_part<D, 32>(buf, ocol + c0, have, r, c0);
    }
    if (size > 1) {
      cluster_sync();
      // this CTA merges rows [rank, rank + 1) * 128 / size: first each part's factor
      // 2^(m_o,k - m_o) / l per row and map and the power of two of their sum (where
      // the V exponents were), then the parts
      const int rows = RF_BLOCK / size;
      const uint32_t buf = parts, am = rf_smem_u32(&sm.row_m[0][0]), al = rf_smem_u32(&sm.row_l[0][0]),
                     ao = rf_smem_u32(&sm.row_o[0][0]);
      float* fac = reinterpret_cast<float*>(sm.vexp);  // [size][2][rows]
      int* ups = sm.vexp + 2 * RF_BLOCK;               // [2][rows]
      if (threadIdx.x < 2 * rows) {
        const int x = threadIdx.x / rows, lr = threadIdx.x - x * rows, row = rank * rows + lr;
        float mk[8], lk[8], ok[8], top = -INFINITY, top_o = -INFINITY, l = 0.f;
        bool any = false;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t at = 4u * (x * RF_BLOCK + row);
          mk[k] = k < size ? cluster_ld(cluster_addr(am + at, k)) : 0.f;
          lk[k] = k < size ? cluster_ld(cluster_addr(al + at, k)) : 0.f;
          ok[k] = k < size ? cluster_ld(cluster_addr(ao + at, k)) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          any |= k < size && mk[k] != -INFINITY;
          if (lk[k] != 0.f) {  // 0: no entries in that part, or none that counts
            top = fmaxf(top, mk[k]);
            top_o = fmaxf(top_o, ok[k]);
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          l = lk[k] != 0.f ? fmaf(rf_ex2(mk[k] - top), lk[k], l) : l;
          ok[k] = lk[k] != 0.f ? rf_ex2(ok[k] - top_o) : 0.f;
        }
        const float inv = !any ? 0.f : 1.0f / l;  // entries whose scores are all -infinity give NaN
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < size) fac[(k * 2 + x) * rows + lr] = ok[k] * inv;
        ups[x * rows + lr] = l == 0.f ? 0 : out_exp(top_o - top, vexp_max);
        if constexpr (kTrain) {
          if (row < q_rows)
            a.lse[((size_t)x * g.n1 + n) * a.rows_total + lrow + q_r0 + row] = !any ? INFINITY : top + log2f(l);
        }
      }
      softmax_bar_sync();
#pragma unroll 2
      for (int i = threadIdx.x; i < rows * (D / 4); i += 256) {
        const int lr = i / (D / 4), row = rank * rows + lr, c = i % (D / 4);
        if (row >= q_rows) break;  // rows come in order
        float o[2][4] = {};
        for (int k = 0; k < size; ++k) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float f = fac[(k * 2 + x) * rows + lr];
            const float4 p = cluster_ld4(cluster_addr(buf + (uint32_t)x * (RF_BLOCK * D * 4) + part_off<D>(row, c), k));
            o[x][0] = fmaf(f, p.x, o[x][0]);
            o[x][1] = fmaf(f, p.y, o[x][1]);
            o[x][2] = fmaf(f, p.z, o[x][2]);
            o[x][3] = fmaf(f, p.w, o[x][3]);
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[x][k] = rf_scale_pow2(o[x][k], ups[x * rows + lr]);
        const size_t off = rf_row_offset(g, s, g.n1, n, q_r0 + row) + 4 * c;
        if constexpr (kTrain) {
          *reinterpret_cast<float4*>(a.maps + off) = make_float4(o[0][0], o[0][1], o[0][2], o[0][3]);
          *reinterpret_cast<float4*>(a.maps + map2 + off) = make_float4(o[1][0], o[1][1], o[1][2], o[1][3]);
        }
        *reinterpret_cast<uint2*>(a.o_r + off) =
            make_uint2(rf_pack2<kBf16>(fmaf(-lam, o[1][0], o[0][0]), fmaf(-lam, o[1][1], o[0][1])),
                       rf_pack2<kBf16>(fmaf(-lam, o[1][2], o[0][2]), fmaf(-lam, o[1][3], o[0][3])));
      }
      cluster_sync();  // the others have read this CTA's part
    }
  }
  if (size > 1 && warp >= 8) {
    cluster_sync();
    cluster_sync();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kSWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// f16 copies of V' by block, [n2][t_qblk][128][D], rows past a block's end
// zero, and their exponents: value = v16 * 2^e.  bf16 inputs: e the smallest
// integer with amax <= 2^(15 + e), amax over the block's finite values (an
// infinity or NaN stays one and must not shrink its neighbours), so that every
// value down to 2^-29 amax is exact; fp16 inputs: e = 0, plain copies.
// One CTA per (block, head): 4 D bytes moved per row, HBM-bound, under 1 % of
// the attention it serves.
template <int D, bool kBf16>
__global__ void __launch_bounds__(256) rf_diff_prep_v_kernel(const __grid_constant__ RfGeomDev g,
                                                             const uint16_t* v, uint4* v16, int32_t* v_exp) {
  constexpr int kChunks = RF_BLOCK * D / 8 / 256;  // 16-byte chunks per thread
  __shared__ uint32_t top_w[8];
  wait_for_previous();
  const int head = blockIdx.x / g.t_qblk, tb = blockIdx.x % g.t_qblk;
  const RfSeqDev& s = g.seq[rf_seq_of_qblk(g, tb)];
  int r0, nrows;
  rf_block_span(s, tb - s.qblk_off, r0, nrows);
  uint4 val[kChunks];
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int ch = threadIdx.x + i * 256, r = ch / (D / 8), c = ch % (D / 8);
    val[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < nrows) val[i] = *reinterpret_cast<const uint4*>(v + rf_row_offset(g, s, g.n2, head, r0 + r) + c * 8);
    if constexpr (kBf16) {
      const uint32_t w[4] = {val[i].x, val[i].y, val[i].z, val[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t lo = w[k] & 0x7FFFu, hi = (w[k] >> 16) & 0x7FFFu;
        if (lo < 0x7F80u) top = max(top, lo);
        if (hi < 0x7F80u) top = max(top, hi);
      }
    }
  }
  uint4* out = v16 + ((size_t)head * g.t_qblk + tb) * (RF_BLOCK * D / 8);
  int e = 0;
  if constexpr (kBf16) {
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) top_w[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, top_w[i]);
    // an all-zero block takes the smallest exponent: it never sets a row's largest
    e = top ? rf_ceil_log2(__uint_as_float(top << 16)) - 15 : -200;
    const int up = top ? -e : 0;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      uint32_t w[4] = {val[i].x, val[i].y, val[i].z, val[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = rf_pack2<false>(rf_scale_pow2(__uint_as_float(w[k] << 16), up),
                               rf_scale_pow2(__uint_as_float(w[k] & 0xFFFF0000u), up));
      val[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
#pragma unroll
  for (int i = 0; i < kChunks; ++i) out[threadIdx.x + i * 256] = val[i];
  if (threadIdx.x == 0) v_exp[(size_t)head * g.t_qblk + tb] = e;
}

// Tensor map over the f16 V copies, [n2 * t_qblk][128][D], 128 x 64 boxes.
rf_status_t make_map_v16(CUtensorMap* m, const rf_plan* p, const void* base) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return rf_fail(RF_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  const RfGeomDev& g = p->g;
  const cuuint64_t d = (cuuint64_t)g.d;
  cuuint64_t dims[3] = {d, (cuuint64_t)RF_BLOCK, (cuuint64_t)g.n2 * (cuuint64_t)g.t_qblk};
  cuuint64_t strides[2] = {d * 2, d * 2 * RF_BLOCK};
  cuuint32_t box[3] = {64, (cuuint32_t)RF_BLOCK, 1}, estr[3] = {1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return rf_fail(RF_ERR_CUDA, "cuTensorMapEncodeTiled (f16 V) failed: " + std::to_string((int)r));
  return RF_OK;
}

template <int D, bool kBf16, bool kTrain>
rf_status_t launch_t(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                     const DiffArgs& args, unsigned grid, cudaStream_t st) {
  size_t smem = sizeof(DiffSmem<D>) + 1024;
  if (smem < 120 * 1024) smem = 120 * 1024;  // each CTA takes all 512 TMEM columns: one per SM
  constexpr auto kern = rf_diff_attn_kernel<D, kBf16, kTrain>;
  int regs = 0;
  rf_status_t s = rf_prepare_kernel<kern>(smem, "cudaFuncSetAttribute(rf_diff_attn_kernel)", &regs);
  if (s != RF_OK) return s;
  // The register split could never be met by a build with fewer registers.
  if (regs != kLaunchRegs)
    return rf_fail(RF_ERR_CUDA, "rf_diff_attn_kernel built with " + std::to_string(regs) +
                                    " registers per thread; the register split needs " +
                                    std::to_string(kLaunchRegs));
  return rf_launch_split(kern, (long long)grid, rf_split(args.g, args.g.n1, 1), kThreads, smem, st,
                         "rf_diff_attn_kernel", mq, mk, mv, args);
}

}  // namespace

rf_status_t rf_launch_diff_attn(const rf_plan* p, const void* q_r, const void* k_r, const void* v_r,
                                const int32_t* sel_idx, const int32_t* sel_num, const float* lambda,
                                float scale, void* o_r, float* maps, float* lse, void* ws,
                                cudaStream_t st) {
  const RfGeomDev& g = p->g;
  const long long grid = (long long)g.t_qblk * g.n1;
  if (grid == 0) return RF_OK;
  if (grid > 0x7FFFFFFFll) return rf_fail(RF_ERR_INVALID_ARG, "grid too large");
  const RfDiffLayout lay = rf_diff_layout(p);
  char* w = static_cast<char*>(ws);
  CUtensorMap mq, mk, mv;
  rf_status_t s;
  if ((s = make_map(&mq, p, q_r, g.n1, kElemPlan)) != RF_OK) return s;
  if ((s = make_map(&mk, p, k_r, g.n2, kElemPlan)) != RF_OK) return s;
  if ((s = make_map_v16(&mv, p, w + lay.v16)) != RF_OK) return s;
  const bool bf = p->dtype == RF_BF16;
  const uint16_t* v = static_cast<const uint16_t*>(v_r);
  uint4* v16 = reinterpret_cast<uint4*>(w + lay.v16);
  int32_t* ve = reinterpret_cast<int32_t*>(w + lay.v_exp);
  const unsigned vgrid = (unsigned)((long long)g.t_qblk * g.n2);
  auto prep = g.d == 128 ? (bf ? rf_diff_prep_v_kernel<128, true> : rf_diff_prep_v_kernel<128, false>)
                         : (bf ? rf_diff_prep_v_kernel<64, true> : rf_diff_prep_v_kernel<64, false>);
  if ((s = rf_launch_dependent(prep, dim3(vgrid), 256, st, "rf_diff_prep_v_kernel", g, v, v16, ve)) != RF_OK) return s;
  DiffArgs a;
  a.g = g;
  a.order = rf_order(g);
  a.sel_idx = sel_idx;
  a.sel_num = sel_num;
  a.lambda = lambda;
  a.o_r = static_cast<uint16_t*>(o_r);
  a.maps = maps;
  a.lse = lse;
  a.rows_total = p->rows_total;
  a.status = reinterpret_cast<uint32_t*>(w + p->off_status);
  a.v_exp = ve;
  a.sl2 = scale * kLog2e;
  const unsigned gr = (unsigned)grid;
  if (g.d == 128) {
    if (maps) return bf ? launch_t<128, true, true>(mq, mk, mv, a, gr, st) : launch_t<128, false, true>(mq, mk, mv, a, gr, st);
    return bf ? launch_t<128, true, false>(mq, mk, mv, a, gr, st) : launch_t<128, false, false>(mq, mk, mv, a, gr, st);
  }
  if (maps) return bf ? launch_t<64, true, true>(mq, mk, mv, a, gr, st) : launch_t<64, false, true>(mq, mk, mv, a, gr, st);
  return bf ? launch_t<64, true, false>(mq, mk, mv, a, gr, st) : launch_t<64, false, false>(mq, mk, mv, a, gr, st);
}
