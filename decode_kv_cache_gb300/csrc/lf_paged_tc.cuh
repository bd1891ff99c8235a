// What the tensor-core kernels of the paged cache share: the warps' roles, the ring's layout, the instructions, tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "lf_paged.cuh"

namespace lf {

namespace {

constexpr int kTile = 128;                 // rows of a query tile, tokens of a key tile
constexpr int kBlk = kTile * 128;          // a tile's 64 columns in shared memory (128-byte swizzle)
constexpr int kMmaWarp = 0, kLoadWarp = 1, kScrubWarp = 2, kRestWarp = 3, kSoftWarp = 4;  // softmax: 4 .. 11
constexpr int kThreadsTc = 384;
constexpr uint32_t kDescHigh = (1024 >> 4) | 1u << 14 | 2u << 29;
constexpr float kGrow = 8.f;               // log2 growth of a maximum that is let pass

template <int D>
struct TcPlan {
  static constexpr int kTileBytes = D / 64 * kBlk;
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kOffQ = 1024;
  static constexpr int kOffRing = kOffQ + 2 * kTileBytes;
  static constexpr int kOffOut = kOffRing + kStages * kTileBytes;        // 4 KB per softmax warp
  static constexpr int kSmem = kOffOut + 8 * 4096 + 1024;                // + alignment slack
  static_assert(kSmem <= 232448, "shared memory of one CTA");
};

__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const void* tmap, int x, int y, int z, int w,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}
// D[tmem] (+)= A x B, bf16 inputs, fp32 accumulation, by the lane whose `lead` is set.
// The predicate is on the instruction, not on a branch around it: in straight code the
// descriptors stay in uniform registers, where the instruction wants them.
// Of a descriptor only the low word changes; the high one is the same for all
// operands here (1024 bytes between groups of eight rows, version 1, 128-byte swizzle).
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d_tmem, uint32_t adesc, uint32_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 a, {%1, %6};\n\tmov.b64 b, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(adesc), "r"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead), "n"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint32_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 b, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead), "n"(kDescHigh)
      : "memory");
}
// The largest of three; a NaN among them is passed over.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// This warp's 32 lanes, 16 / 32 consecutive 32-bit columns of tensor memory.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
      "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Wait on, up to kWaitLimitNs or until another wait has expired (`expired`).
__device__ __noinline__ bool wait_longer(uint64_t* bar, uint32_t parity, volatile int* expired) {
  const unsigned long long t0 = global_ns();
  while (!*expired) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (global_ns() - t0 > kWaitLimitNs) *expired = 1;
  }
  return false;
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                             CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                             CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  static std::atomic<void*> fn{nullptr};
  void* p = fn.load();
  if (!p) {
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
            cudaSuccess || q != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      return nullptr;
    }
    fn.store(p);
  }
  return reinterpret_cast<EncodeFn>(p);
}

bool encode(EncodeFn fn, CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A dimension of one entry has no use for its stride, which must still be a legal one.
inline cuuint64_t legal_stride(int64_t s, int64_t n) { return n == 1 && s < 16 ? 16 : (cuuint64_t)s; }

// Tensor maps of the queries (boxes of a query tile's tokens and 64 columns) and of the pools (boxes of 64 columns of
// box_rows tokens of a page).
inline bool encode_maps(const PagedPool& pool, const void* q, int q_heads, int group, int tokens, int head_dim, int box_rows,
                        CUtensorMap* mq, CUtensorMap* mk, CUtensorMap* mv) {
  EncodeFn fn = encoder();
  if (!fn) return false;
  const int ps = pool.page_size;
  const cuuint64_t qd[3] = {(cuuint64_t)head_dim, (cuuint64_t)q_heads, (cuuint64_t)tokens};
  const cuuint64_t qst[2] = {(cuuint64_t)head_dim * 2, (cuuint64_t)q_heads * head_dim * 2};
  const cuuint32_t qb[3] = {64, (cuuint32_t)group, (cuuint32_t)(kTile / group)};
  const cuuint64_t kd[4] = {(cuuint64_t)head_dim, (cuuint64_t)ps, (cuuint64_t)pool.kv_heads, (cuuint64_t)pool.num_pages};
  const cuuint64_t kst[3] = {legal_stride(pool.token_stride, ps), legal_stride(pool.head_stride, pool.kv_heads),
                             legal_stride(pool.page_stride, pool.num_pages)};
  const cuuint32_t kb[4] = {64, (cuuint32_t)box_rows, 1, 1};
  return encode(fn, mq, q, 3, qd, qst, qb) && encode(fn, mk, pool.k, 4, kd, kst, kb) &&
         encode(fn, mv, pool.v, 4, kd, kst, kb);
}

}  // namespace

}  // namespace lf
