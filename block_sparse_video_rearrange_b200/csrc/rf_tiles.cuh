// What the attention kernels share: bounded warp waits, the score row maximum
// and the tensor maps of the rearranged tensors.  Included by the .cu files only.
#pragma once

#include <cuda.h>

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
