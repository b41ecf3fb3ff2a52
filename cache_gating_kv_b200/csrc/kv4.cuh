// The 4-bit cache format on the device: e2m1 codes (two to a byte) with an
// e4m3 scale for 16 numbers, and the rotation of key rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/flowcache.h"
#include "fc_common.cuh"

namespace fc {

// Strides in elements of a [N][H][L][d] tensor whose rows are contiguous.
// (Kernels that start as programmatic dependents read what the kernels before them
// wrote through plain loads: the compiler may lift a load of the read-only path over
// griddepcontrol.wait.)
struct Strides {
  int64_t n, h, l;
};

namespace kv4 {

// Two e4m3 numbers (the low 16 bits of w) as a float16 pair; exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}\n"
      : "=r"(r)
      : "r"(w));
  return r;
}

// The four code pairs of a word (8 codes) as float16 pairs; exact.  Every result has
// to be used: where two were not, the 12.9 compiler's optimised code gave zeros.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

// 8 numbers to nearest e2m1, ties to even, saturating; element 0 in the low
// four bits.
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float* t) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}\n"
      : "=r"(r)
      : "f"(t[0]), "f"(t[1]), "f"(t[2]), "f"(t[3]), "f"(t[4]), "f"(t[5]), "f"(t[6]), "f"(t[7]));
  return r;
}

// One e4m3 number, to nearest (ties to even), of a float in [0, 448].
__device__ __forceinline__ uint32_t f32_to_e4m3(float x) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %2, %1;\n\tcvt.u32.u16 %0, h;\n\t}\n"
      : "=r"(r)
      : "f"(x), "f"(0.0f));
  return r;
}

// An e4m3 byte that is NaN.
__device__ __forceinline__ bool scale_is_nan(uint32_t b) { return (b & 0x7Fu) == 0x7Fu; }

__device__ __forceinline__ float lo_f16(uint32_t w) {
  return __half2float(__ushort_as_half((unsigned short)(w & 0xffffu)));
}

}  // namespace kv4

// cos and sin of one position and frequency, times m, as the rotation uses
// them: the turn and its functions in float64, one rounding to float32.  The
// turn loses its whole part before the functions see it, so a far position
// costs no accuracy beyond the float64 product.
__device__ __forceinline__ float2 rope_cs(int32_t p, double turns, double m, bool inverse) {
  double u = (double)p * turns;
  u -= rint(u);
  double s, c;
  sincospi(2.0 * u, &s, &c);
  return make_float2((float)(c * m), (float)(inverse ? -(s * m) : s * m));
}

// A row's rotated pair: products and sums rounded one by one.
__device__ __forceinline__ float rope_a(float a, float b, float2 cs) {
  return __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
}
__device__ __forceinline__ float rope_b(float a, float b, float2 cs) {
  return __fadd_rn(__fmul_rn(b, cs.x), __fmul_rn(a, cs.y));
}

// ---- launchers ------------------------------------------------------------------
cudaError_t launch_rope(const void* x, void* y, bool bf16, int N, int H, int L, int d, Strides xs,
                        Strides ys, const int32_t* pos, const fc_rope_plan& plan, bool inverse,
                        cudaStream_t s);
cudaError_t launch_kv4_store(const void* k, const void* v, bool bf16, int L, Strides ks, Strides vs,
                             const int32_t* idx, int rows, int row0, const int32_t* row0_dev,
                             const fc_rope_plan* plan, const int32_t* pos,
                             const fc_kv4_cache& cache, cudaStream_t s);
cudaError_t launch_kv4_load(const fc_kv4_cache& cache, void* k, void* v, bool bf16, int L,
                            Strides ks, Strides vs, int row0, const int32_t* row0_dev,
                            cudaStream_t s);

struct Kv4Attn {
  const void* q;
  void* out;
  float* lse;
  const int32_t* lens;
  Strides qs, os;
  int Hq, Lq, max_len;
  bool bf16, causal;
  float scale;  // of the logits, without 2^k_exp
  // for the self-test of waits that give up: a slot of the ring of key stages whose
  // barrier wants an arrival that nobody makes (-1: none)
  int stuck_slot;
  long long wait_cycles;
};
size_t kv4_attention_ws_bytes(bool bf16, int N, int Hq, int Hkv, int Lq, int max_len, int d);
cudaError_t launch_kv4_attention(const Kv4Attn& a, const fc_kv4_cache& cache, void* ws,
                                 cudaStream_t s);

}  // namespace fc
