// api.cuh -- what the files that define C entry points share (host code only): the calling thread's error
// message, the argument checks that every entry makes, and the profiler range around an entry.
#pragma once

#include <nvtx3/nvToolsExt.h>

#include "common.cuh"

namespace bsva {

// Record the message of a failed call and return its code; ok() clears it. Defined in api.cu.
int fail(int code, const char* fmt, ...);
int ok();
int cuda_fail(cudaError_t e, const char* what);
int check_device();
int check_shape(const bsva_shape& s);
int check_workspace(void* ws, size_t bytes, size_t need);
int get_encoder();   // the driver's tensor-map encoder, looked up once; before the first encode_map
// 3-D map over [heads][rows][inner] with a box of [1][box_rows][box_inner].
int encode_map(CUtensorMap* m, const void* base, CUtensorMapDataType dt, int elem_bytes, uint64_t inner, uint64_t rows,
               uint64_t heads, uint32_t box_inner, uint32_t box_rows, CUtensorMapSwizzle sw, const char* what);
// 4-D bf16 map [n3][n2][n1][inner] with byte strides of n1, n2, n3, boxes of [1][box2][box1][box_inner], 128-byte swizzle.
int encode_map_4d(CUtensorMap* m, const void* base, uint64_t inner, uint64_t n1, uint64_t n2, uint64_t n3,
                  const uint64_t stride[3], uint32_t box_inner, uint32_t box1, uint32_t box2, const char* what);

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// An NVTX range over one entry point (its validation, descriptor encoding and
// launches), named after the entry, so that a profiler timeline shows which
// call issued which kernels. NVTX costs nothing measurable when no tool is attached.
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};
#define BSVA_RANGE(name) NvtxRange bsva_nvtx_range_(name)

#define REQUIRE_PTR(p, align)                                                                          \
  do {                                                                                                 \
    if ((p) == nullptr) return fail(BSVA_ERR_INVALID_ARG, "%s is NULL", #p);                           \
    if (!aligned((p), (align))) return fail(BSVA_ERR_INVALID_ARG, "%s is not %d-byte aligned", #p, (align)); \
  } while (0)

}  // namespace bsva
