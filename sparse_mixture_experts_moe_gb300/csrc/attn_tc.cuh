// What the attention kernels on the 5th-generation tensor cores share: the shape of a CTA, the MMA with its A operand
// in TMEM, and the descriptors of their tensors.
#pragma once
#include <cuda.h>

#include "attn.cuh"
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int BK = 128;       // keys per block
constexpr int TM = 128;       // rows per tile
// 12 warps of 168 registers at launch (64512), which each kernel then shares out among its softmax warps (a row of 128
// scores stays in registers) and the other four.
constexpr int kThreads = 384;
constexpr int kSoftWarps = 8;
constexpr int kMaxSmem = 232448;

// D[tmem] (+)= A[tmem, bf16 pairs] * B[smem desc].
__device__ __forceinline__ void tc_mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};"
      ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

inline bool encode3(EncodeTiledFn enc, CUtensorMap* m, const void* p, int D, int heads, int T, long long stride,
                    int box_heads, int box_rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)T};
  const cuuint64_t str[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  return encode_tmap(enc, m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, 3, dims, str, box);
}
// Q's descriptor, where a tile is a box of whole tokens; *ok says whether there is one.
inline bool encode_q(EncodeTiledFn enc, CUtensorMap* m, const void* p, int D, int H, int G, int T, long long stride,
                     int* ok) {
  *ok = TM % G == 0;
  return !*ok || encode3(enc, m, p, D, H, T, stride, G, TM / G);
}

}  // namespace
}  // namespace moe
