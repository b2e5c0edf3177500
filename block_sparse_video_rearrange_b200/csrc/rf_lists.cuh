// Selection lists over CTAs: their order in a launch, their sharing by the CTAs of
// a cluster, and their compaction.  Included by the .cu files only.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <string>

#include "rf_async.cuh"
#include "rf_device.cuh"

namespace {

// Order of the CTAs of a launch over (head, block): first the blocks that the
// ranking keeps dense (prefix and first frame; all of a short sequence) of every
// head, then the others, each class head-major.  A dense block's list is several
// times as long as a sparse one's, and one that starts late would run on alone.
struct RfOrder {
  int n_dense;  // dense blocks of all sequences
};
__device__ __forceinline__ int rf_dense_blocks(const RfSeqDev& s) { return s.dense ? s.n_pb + s.nb : s.n_pb + s.ns; }
__device__ __forceinline__ void rf_cta_item(const RfGeomDev& g, const RfOrder& o, int heads, int bid, int& head, int& tb) {
  const bool dense = bid < heads * o.n_dense;
  if (!dense) bid -= heads * o.n_dense;
  const int per = dense ? o.n_dense : g.t_qblk - o.n_dense;
  head = bid / per;
  int i = bid - head * per;
  tb = 0;
#pragma unroll 1
  for (int k = 0; k < g.n_seqs; ++k) {
    const int nd = rf_dense_blocks(g.seq[k]);
    const int here = dense ? nd : g.seq[k].n_pb + g.seq[k].nb - nd;
    if (i < here) {
      tb = g.seq[k].qblk_off + (dense ? i : nd + i);
      break;
    }
    i -= here;
  }
}
inline RfOrder rf_order(const RfGeomDev& g) {
  RfOrder o{0};
  for (int k = 0; k < g.n_seqs; ++k) {
    const RfSeqDev& s = g.seq[k];
    o.n_dense += s.dense ? s.n_pb + s.nb : s.n_pb + s.ns;
  }
  return o;
}

// ---- one list over the CTAs of a cluster ---------------------------------------
// With few (head, block) items the lists are split: the CTAs of a cluster take
// equal consecutive parts of one list, leave their fp32 partial rows in shared
// memory, and each merges 128 / size of the rows from all of them, in rank order.

// Byte offset of 16-byte chunk c of row r in a [128][D] fp32 buffer whose chunks
// are permuted within each row, so that neither a warp writing one chunk of 32
// rows nor one reading a row's chunks meets bank conflicts.
template <int D>
__device__ __forceinline__ uint32_t part_off(int r, int c) {
  return (uint32_t)(r * (D * 4) + ((c ^ (r & (D / 4 - 1))) << 4));
}

// N accumulator columns of this thread's row (TMEM), from column col on, into the
// buffer at `buf`; zeros where there are none.
template <int D, int N>
__device__ __forceinline__ void store_part(uint32_t buf, uint32_t taddr, bool have, int r, int col) {
  uint32_t o[N];
  if (have) {
    if constexpr (N == 32) tmem_ld32(taddr, o);
    else                   tmem_ld16(taddr, o);
    tmem_wait_ld();
  } else {
#pragma unroll
    for (int c = 0; c < N; ++c) o[c] = 0u;
  }
#pragma unroll
  for (int c = 0; c < N / 4; ++c) sts128(buf + part_off<D>(r, col / 4 + c), o + 4 * c);
}

// How many CTAs share a list: the size whose estimated finish is earliest.  The
// launch ends no earlier than its longest CTA and no earlier than the work spread
// over 148 SMs; a CTA counts kFixed blocks beside its list, a merge kMerge more.
// kFixed is a fit, not a measured time: a CTA's start, first loads and epilogue take
// that of about 3.5 blocks (11,000 cycles), and the rest stands for what splitting
// costs otherwise.  Measured with training outputs (us, sizes 1 / 2 / 4 / 8; the
// backward kernels as the time of the whole backward call, one kernel's size varied;
// * the rule's choice, the best in every row):
//                                  forward            dK/dV                   dQ
//   74 items, 37 blocks, d 64      69 43* 47 75       122 87* 89 118          101 87* 98 114
//   148 items, 37 blocks, d 128    72 70* 99 171      151 134* 169 245        143 134* 156 215
//   296 items, 37 blocks, d 128    92* 119 183 340    204* 230 297 451        205* 224 272 392
//   656 items, 82 blocks, d 128    294* 368 528 892   697* 774 910 1,279      727* 775 869 1,140
//   4/1 heads, 37 blocks, d 128    79 73* 101 172     389 232 153 144*        151 145* 172 229
//   8/2 heads, 82 blocks, d 64     277* 323 460 762   905 594* 654 758        594* 638 753 982
inline int rf_split(const RfGeomDev& g, int heads, int group) {
  constexpr double kFixed = 7.0, kMerge = 2.0, kSms = 148.0;
  double dense = 0, sparse = 0, dense_len = 0, sparse_len = 0, longest = 0;
  for (int k = 0; k < g.n_seqs; ++k) {
    const RfSeqDev& s = g.seq[k];
    const double nkv = s.n_pb + s.nb, nd = s.dense ? nkv : s.n_pb + s.ns;
    const double len = s.n_pb + s.ns + (s.nb ? (double)s.k * (s.nb - s.ns) / s.nb : 0.0);
    dense += nd;
    dense_len += nd * nkv;
    sparse += nkv - nd;
    sparse_len += (nkv - nd) * (len < nkv ? len : nkv);
    if (nkv > longest) longest = nkv;
  }
  int best = 1;
  double best_t = 0;
  for (int size = 1; size <= 8; size *= 2) {
    const double fixed = kFixed + (size > 1 ? kMerge : 0.0);
    const double total = heads * ((dense + sparse) * size * fixed + group * (dense_len + sparse_len));
    const double one = fixed + group * longest / size;
    const double t = one > total / kSms ? one : total / kSms;
    if (size == 1 || t < 0.9 * best_t) {
      best = size;
      best_t = t;
    }
  }
  return best;
}

// Sets a kernel's shared-memory limit, once per device (the call takes longer than
// a launch), and gives its registers per thread.
template <auto kern>
inline rf_status_t rf_prepare_kernel(size_t smem, const char* what, int* regs = nullptr) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];  // registers + 1
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return rf_check_launch(what);
  if (dev < 0 || dev >= kDevices) return rf_fail(RF_ERR_UNSUPPORTED_DEVICE, "device ordinal beyond 64");
  int r = known[dev].load(std::memory_order_acquire);
  if (r == 0) {
    cudaFuncAttributes fa;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess ||
        cudaFuncGetAttributes(&fa, kern) != cudaSuccess)
      return rf_check_launch(what);
    r = fa.numRegs + 1;
    known[dev].store(r, std::memory_order_release);
  }
  if (regs) *regs = r - 1;
  return RF_OK;
}

// Launches `kern` with `size` CTAs per cluster for each of `items`, as a dependent of
// the stream's kernel before it: it may start before that one ends and must call
// wait_for_previous() before it touches what that one writes, and in any case
// before it ends.
template <class... Args>
inline rf_status_t rf_launch_split(void (*kern)(Args...), long long items, int size, int threads, size_t smem,
                                   cudaStream_t st, const char* what, Args... args) {
  if (items * size > 0x7FFFFFFFll) return rf_fail(RF_ERR_INVALID_ARG, "grid too large");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items * size));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)size;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = size > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) return rf_check_launch(what);
  return rf_check_launch(what);
}

// Compacts the `num` entries of a selectIdx row in `list` (shared memory) in
// place, by one warp: in-range entries that are larger than every in-range
// entry before them stay, -1 is an unused slot, and anything else (out of
// range, listed twice, out of order) is skipped and counted into *bad.  A lane
// writes at or below its own read position, and every lane reads before the
// ballot.  Returns the entries kept.
__device__ __forceinline__ int compact_ascending(int* list, int num, int nkv, int lane, int* bad) {
  const uint32_t lt = (1u << lane) - 1u;
  int cnt = 0, top = -1;
  for (int c0 = 0; c0 < num; c0 += 32) {
    const int c = c0 + lane;
    const int v = c < num ? list[c] : -1;
    const bool in = v >= 0 && v < nkv;
    int run = in ? v : -1;  // largest in-range entry up to and including this lane's
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, run, d);
      if (lane >= d) run = max(run, o);
    }
    int before = __shfl_up_sync(0xffffffffu, run, 1);
    before = lane == 0 ? top : max(top, before);
    const bool ok = in && v > before;
    if (c < num && v != -1 && !ok) ++*bad;
    const uint32_t ball = __ballot_sync(0xffffffffu, ok);
    if (ok) list[cnt + __popc(ball & lt)] = v;
    cnt += __popc(ball);
    top = max(top, __shfl_sync(0xffffffffu, run, 31));
    __syncwarp();
  }
  return cnt;
}

}  // namespace
