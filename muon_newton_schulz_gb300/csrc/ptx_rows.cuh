// Inline-PTX wrappers that the feed-forward kernels use besides those of the
// Newton-Schulz phases: tensor maps changed on the device, 32-byte accesses, a left
// operand that is MN-major.
#pragma once

#include "ptx_sm100.cuh"

namespace muon {
namespace ptx {

// Replaces base address and second dimension of a tensor map in shared memory
// (128-byte aligned).
__device__ __forceinline__ void tensormap_replace(const CUtensorMap* smem_map, const void* base, uint32_t dim1) {
  const uint32_t a = smem_u32(smem_map);
  asm volatile("tensormap.replace.tile.global_address.shared::cta.b1024.b64 [%0], %1;" ::"r"(a),
               "l"(reinterpret_cast<uint64_t>(base))
               : "memory");
  asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;" ::"r"(a), "r"(dim1) : "memory");
}

// Copies a tensor map from shared to global memory, for users that acquire it
// (fence_tensormap_acquire).  All threads of a warp.
__device__ __forceinline__ void tensormap_publish(CUtensorMap* dst, const CUtensorMap* smem_map) {
  asm volatile(
      "tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync.aligned [%0], [%1], 128;" ::"l"(
          reinterpret_cast<uint64_t>(dst)),
      "r"(smem_u32(smem_map))
      : "memory");
}

// tma_load_4d (rank 0) and tma_load_4d_pair (rank 1) by shared-memory addresses; the
// last coordinate is 0.
template <int kRank>
__device__ __forceinline__ void tma_load_4d_rank(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
  if constexpr (kRank == 0)
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(0), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(0), "r"(bar)
        : "memory");
}

// 32 bytes at a time, on 32-byte boundaries of global memory, of data that is used
// once: it leaves L2 before the operands do (dh's kernel 482 us with, 515 without).
__device__ __forceinline__ void ld_global_32(const void* p, uint32_t (&v)[8]) {
  asm volatile("ld.global.L1::no_allocate.L2::evict_first.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void st_global_32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.L2::evict_first.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// idesc_bf16_f32 with A K-major or MN-major too.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool a_mn_major, bool b_mn_major) {
  return idesc_bf16_f32(M, N, b_mn_major) | ((a_mn_major ? 1u : 0u) << 15);
}

}  // namespace ptx
}  // namespace muon
