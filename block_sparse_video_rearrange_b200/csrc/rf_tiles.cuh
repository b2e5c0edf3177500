// What the attention kernels share: bounded warp waits, the score row maximum
// and the tensor maps of the rearranged tensors.  Included by the .cu files only.
#pragma once

#include <cuda.h>

#include <atomic>
#include <mutex>
#include <string>

#include "rf_device.cuh"

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// Warp-wide bounded wait: every lane polls the barrier itself (a lane that
// only waits on a warp shuffle for a polling lane 0 wakes far later), then the
// warp agrees on the outcome.  kPoll = true drops the suspend hint: the MMA
// warp's hand-offs (P ready, V and K tiles landed) sit on the critical path,
// and polling them measured about 2% faster overall than sleeping on them.
template <bool kPoll = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  const bool ok = mbar_wait<kPoll>(bar, parity, abort);
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void record_timeout(volatile int* abort, uint32_t* status, int where) {
  *abort = 1;
  atomicOr(status + RF_STATUS_TIMEOUT, 1u << where);
}

// Row max of 128 raw scores (the first vr valid): three-input max, eight chains.
template <bool kFull>
__device__ __forceinline__ float row_max(const uint32_t* sr, int vr) {
  float m[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i] = -INFINITY;
  if (kFull) {
#pragma unroll
    for (int c = 0; c < 128; c += 2)
      m[(c >> 1) & 7] = rf_max3(m[(c >> 1) & 7], __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
  } else {
#pragma unroll
    for (int c = 0; c < 128; ++c)
      if (c < vr) m[c & 7] = fmaxf(m[c & 7], __uint_as_float(sr[c]));
  }
  return rf_max3(rf_max3(m[0], m[1], m[2]), rf_max3(m[3], m[4], m[5]), fmaxf(m[6], m[7]));
}

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

// How many CTAs share a list: the size whose estimated finish is earliest.  A CTA
// costs about kFixed blocks' time beside its list (start, first loads, epilogue);
// a merge two more.  The launch ends no earlier than its longest CTA and no
// earlier than the work spread over 148 SMs.  Measured (forward, us, sizes 1 / 2 /
// 4): 74 items of up to 37 blocks at d = 64: 67 / 41 / 45; 148 such items at
// d = 128: 76 / 68 / 95; 656 items of up to 82 blocks: 259 / 292 / 436.
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

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
    cudaGetLastError();
  });
  return fn;
}

// Element type of a tensor map: the plan's 16-bit type, E4M3 bytes, or f16.
enum MapElem { kElemPlan = 0, kElemByte = 1, kElemF16 = 2 };

// Tensor map over [rows, heads, D] (TND) or [B*heads, rows, D] (BNSD) with a
// box_rows x 128-byte box and 128-byte swizzle: 64 columns of a 16-bit tensor,
// or 128 columns of a one-byte (E4M3) tensor.  box_rows is 128, or 64 for the
// key/value maps of blockShape 128 x 64.
rf_status_t make_map(CUtensorMap* m, const rf_plan* p, const void* base, int heads, MapElem elem,
                     int box_rows = RF_BLOCK) {
  const bool one_byte = elem == kElemByte;
  EncodeTiledFn enc = encode_fn();
  if (!enc) return rf_fail(RF_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  const RfGeomDev& g = p->g;
  const cuuint64_t d = (cuuint64_t)g.d;
  const cuuint64_t esz = one_byte ? 1 : 2;
  const cuuint32_t box_cols = one_byte ? 128 : 64;
  cuuint64_t dims[3], strides[2];
  cuuint32_t box[3], estr[3] = {1, 1, 1};
  if (g.layout == RF_LAYOUT_BNSD) {
    const cuuint64_t L = (cuuint64_t)g.seq[0].L;
    dims[0] = d; dims[1] = L; dims[2] = (cuuint64_t)p->batch * heads;
    strides[0] = d * esz; strides[1] = L * d * esz;
    box[0] = box_cols; box[1] = (cuuint32_t)box_rows; box[2] = 1;
  } else {
    dims[0] = d; dims[1] = (cuuint64_t)heads; dims[2] = (cuuint64_t)p->rows_total;
    strides[0] = d * esz; strides[1] = (cuuint64_t)heads * d * esz;
    box[0] = box_cols; box[1] = 1; box[2] = (cuuint32_t)box_rows;
  }
  const CUtensorMapDataType dt = one_byte ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                 : (p->dtype == RF_BF16 && elem == kElemPlan) ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                                              : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUresult r = enc(m, dt, 3, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return rf_fail(RF_ERR_CUDA, "cuTensorMapEncodeTiled failed: " + std::to_string((int)r));
  return RF_OK;
}

}  // namespace
