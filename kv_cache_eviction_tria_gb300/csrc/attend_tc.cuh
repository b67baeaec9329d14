// Fifth-generation tensor cores and tensor copies, as the attention kernels use
// them (attend_prompt.cu, attend_group.cu): products, accumulators' loads and
// stores, tiles in 128-byte-swizzled shared memory.
#pragma once

#include <cuda.h>

#include <algorithm>

#include "attend_internal.cuh"

namespace tria {

namespace {

constexpr float kLazy = 8.f, kShift = 5.f;   // of the softmax's reference, see attend_prompt.cu
constexpr int kWaitLimit = 1 << 22;          // polls of a wait before it gives up

// ---- PTX -------------------------------------------------------------------

__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// true in one lane of a converged warp (the compiler then knows that the branch
// holds a single thread and keeps descriptors in uniform registers)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xFFFFFFFF;\n selp.b32 %0, 1, 0, q;\n}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define TRIA_R8(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), "=r"(a[i + 5]), "=r"(a[i + 6]), "=r"(a[i + 7])
#define TRIA_S8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), "r"(a[i + 5]), "r"(a[i + 6]), "r"(a[i + 7])
__device__ __forceinline__ void tc_ld32(uint32_t* r, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
      "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : TRIA_R8(r, 0), TRIA_R8(r, 8), TRIA_R8(r, 16), TRIA_R8(r, 24)
      : "r"(addr));
}
__device__ __forceinline__ void tc_ld16(uint32_t* r, uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : TRIA_R8(r, 0), TRIA_R8(r, 8)
               : "r"(addr));
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::TRIA_S8(r, 0),
      TRIA_S8(r, 8), "r"(addr)
      : "memory");
}
// keeps uses of loaded registers behind the wait for them
#define TRIA_P8(a, i) "+r"(a[i]), "+r"(a[i + 1]), "+r"(a[i + 2]), "+r"(a[i + 3]), "+r"(a[i + 4]), "+r"(a[i + 5]), "+r"(a[i + 6]), "+r"(a[i + 7])
__device__ __forceinline__ void tc_pin16(uint32_t* r) { asm volatile("" : TRIA_P8(r, 0), TRIA_P8(r, 8)); }
__device__ __forceinline__ void tc_pin(uint32_t* r) {
  tc_pin16(r);
  tc_pin16(r + 16);
}
#undef TRIA_P8
#undef TRIA_R8
#undef TRIA_S8

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// 128-byte-swizzled tile descriptors: rows of 128 bytes in groups of eight
// (1024 bytes). K-major operands step 32 bytes per 16 dims inside a row; the
// values (dims contiguous, rows along K) step 2048 bytes per 16 rows and
// `blocks` bytes from one 64-dim block to the next.
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr, uint32_t block_bytes) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)(block_bytes >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// fp16 operands, fp32 result, M = 128
__host__ __device__ constexpr uint32_t mma_desc(int n, bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ uint32_t swz(int row, int chunk) { return (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4)); }

__device__ __forceinline__ bool junk_h2(uint32_t w) {     // an infinity or NaN in a pair of fp16
  return (w & 0x7C00u) == 0x7C00u || (w & 0x7C000000u) == 0x7C000000u;
}

__device__ __forceinline__ uint32_t pack_out(int type, float a, float b) {   // a pair of the output's type
  if (type == TRIA_F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Starts the copies of rows row .. row + BN of a plane into a tile, arriving on `bar`.
template <int HD, int BN>
__device__ __forceinline__ void copy_tile(uint8_t* tile, const CUtensorMap* map, int64_t row, uint64_t* bar) {
  mbar_arrive_expect_tx(bar, BN * HD * 2);
#pragma unroll
  for (int c = 0; c < HD / 64; ++c)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_u32(tile) + c * (BN * 128)),
        "l"(map), "r"(c * 64), "r"((int)row), "r"(smem_u32(bar))
        : "memory");
}

// Values past `rows` and those with junk become zeros; the latter's rows are
// marked. By kThreads threads.
template <int HD, int BN, int kThreads>
__device__ __forceinline__ void clean_tile(uint8_t* tile, int rows, uint32_t* marks, int tid) {
  constexpr int per = HD / 8;
#pragma unroll 4
  for (int x = tid; x < BN * per; x += kThreads) {
    const int r = x / per, c = x - r * per;
    uint4* p = reinterpret_cast<uint4*>(tile + (c >> 3) * (BN * 128) + swz(r, c & 7));
    if (r >= rows) {
      *p = make_uint4(0, 0, 0, 0);
      continue;
    }
    const uint4 v = *p;
    if (junk_h2(v.x) || junk_h2(v.y) || junk_h2(v.z) || junk_h2(v.w)) {
      *p = make_uint4(0, 0, 0, 0);
      atomicOr(&marks[r >> 5], 1u << (r & 31));
    }
  }
}

// TMA view of an fp16 plane: boxes of 64 dims x `box` rows, 128-byte swizzle
bool plane_map_f16(CUtensorMap* m, const void* base, int hd, int64_t rows, int box) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return (Encode)fn;
  }();
  if (!encode) return false;
  // (a plane without rows is never read, but a map has one at least)
  const cuuint64_t dims[2] = {(cuuint64_t)hd, (cuuint64_t)std::max<int64_t>(rows, 1)}, strides[1] = {(cuuint64_t)hd * 2};
  const cuuint32_t boxes[2] = {64, (cuuint32_t)box}, steps[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(base), dims, strides, boxes, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

}  // namespace tria
