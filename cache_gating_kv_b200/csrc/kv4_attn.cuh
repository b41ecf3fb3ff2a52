// What the kernels of the attention over the 4-bit cache share.
#pragma once

#include <cuda.h>

#include "fc_common.cuh"
#include "kv4.cuh"
#include "tc_ptx.cuh"

namespace fc {

struct AttnArgs {
  const void* q;
  void* out;
  float* lse;
  const int32_t* lens;
  Strides qs, os;
  const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  int Hkv, G, R, Lq, max_len, cap;  // R = G * Lq rows of a key head
  int rows_blk, n_rb, n_split, chunk;
  bool causal;
  float scale_log2;  // scale * 2^k_exp * log2 e
  float out_scale;   // 2^v_exp
  int* err;
  float2* part_ml;  // [N Hkv R][n_split] (log2 reference, sum)
  float* part_o;    // [N Hkv R][n_split][d]
};

__device__ __forceinline__ int seq_len(const AttnArgs& a, int n) {
  if (a.lens == nullptr) return a.max_len;
  return max(0, min(__ldg(a.lens + n), a.max_len));
}
// Keys that query i sees.
__device__ __forceinline__ int row_keys(const AttnArgs& a, int len, int i) {
  return a.causal ? max(0, len - a.Lq + i + 1) : len;  // i < Lq, so at most len
}
// Keys that the last of the rows [r0, r0 + rows) sees.
__device__ __forceinline__ int block_keys(const AttnArgs& a, int len, int r0, int rows) {
  return row_keys(a, len, (min(r0 + rows, a.R) - 1) / a.G);
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(reinterpret_cast<const __half2&>(a), reinterpret_cast<const __half2&>(b));
  return reinterpret_cast<const uint32_t&>(r);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 r = __floats2half2_rn(lo, hi);
  return reinterpret_cast<const uint32_t&>(r);
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          tc::smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
      : "memory");
}

// Four outputs of row r from their weighted sums o, the row's log2 reference
// and its sum L of 2^(x - ref).
template <typename T>
__device__ __forceinline__ void write_row(const AttnArgs& a, int n, int hk, int r, int c, float4 o,
                                          float ref, float L) {
  const int i = r / a.G, h = hk * a.G + r % a.G;
  const float f = L == 0.0f ? 0.0f : __fdividef(a.out_scale, L);
  T* p = static_cast<T*>(a.out) + n * a.os.n + h * a.os.h + i * a.os.l + c;
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * f, o.y * f);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(o.z * f, o.w * f);
    *reinterpret_cast<uint2*>(p) = make_uint2(reinterpret_cast<const uint32_t&>(lo),
                                              reinterpret_cast<const uint32_t&>(hi));
  }
  if (c == 0 && a.lse != nullptr) {
    const float v = L == 0.0f ? -INFINITY : (ref + log2f(L)) * 0.6931471805599453f;
    a.lse[((int64_t)n * a.Hkv * a.G + h) * a.Lq + i] = v;
  }
}

// The tensor-core kernel for many query rows (bf16): rows of a block, keys of a
// tile.
constexpr int kTcRows = 256, kTcKeys = 128;
cudaError_t launch_attn_tc(const AttnArgs& a, int N, int d, cudaStream_t s);

}  // namespace fc
