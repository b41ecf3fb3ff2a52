// Rows into and out of the 4-bit cache.
//
// Storing reads 2 x 2 bytes per element pair of K and V (bf16) and writes 4.5
// bits per element, loading the reverse, so both are bound by HBM.  One thread
// owns one group of 16 elements: the group's maximum, its scale and its eight
// bytes of codes then need no exchange between threads, a warp's code stores
// are 256 contiguous bytes and its reads 1 KB.  For keys that are rotated on
// the way the thread also reads the partner elements of its group (the same
// lines, read by another thread of the warp, so they come from L1) instead of
// exchanging numbers through shared memory.
#include "fc_common.cuh"
#include "fc_kernels.h"
#include "kv4.cuh"

namespace fc {

namespace {
constexpr int kThreads = 256;

// 16 consecutive elements as float32.
template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&f)[16]) {
  constexpr int V = 16 / (int)sizeof(T);
#pragma unroll
  for (int i = 0; i < 16 / V; ++i)
    Vec16<T>::to_float(__ldg(reinterpret_cast<const uint4*>(p) + i), f + i * V);
}

template <typename T>
__device__ __forceinline__ float load1(const T* p) {
  if constexpr (sizeof(T) == 4)
    return __ldg(p);
  else
    return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p)) << 16);
}

// One group of 16 numbers to its scale byte and its eight code bytes.
__device__ __forceinline__ uint2 quantise16(float (&y)[16], uint32_t& scale) {
  uint32_t top = 0;  // bits of max |y|: NaN counts above infinity
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(y[i]) & 0x7fffffffu);
  const float amax = __uint_as_float(top);
  if (top > 0x7f800000u) {  // a NaN: the group reads as NaN
    scale = 0x7Fu;
    return make_uint2(0u, 0u);
  }
  // Numbers beyond 6 * 448 saturate whatever they are; cutting them there
  // keeps the quotients below finite (their scale is 448).
  if (amax > 4096.0f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = fminf(fmaxf(y[i], -4096.0f), 4096.0f);
  }
  scale = kv4::f32_to_e4m3(fminf(__fdiv_rn(amax, 6.0f), 448.0f));
  const float s = kv4::lo_f16(kv4::e4m3x2_to_f16x2(scale));
  // y / s rounded to nearest, so that a number half way between two codes is
  // seen as such: from the correctly rounded reciprocal r, q = y r is within an
  // ulp and q - r (q s - y) is the rounded quotient (Markstein, "Computation of
  // elementary functions on the IBM RISC System/6000 processor", 1990); with the
  // remainder in this order a zero keeps its sign.
  const float r = s > 0.0f ? __frcp_rn(s) : 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float q = __fmul_rn(y[i], r);
    y[i] = __fmaf_rn(-__fmaf_rn(q, s, -y[i]), r, q);
  }
  return make_uint2(kv4::f32x8_to_e2m1(y), kv4::f32x8_to_e2m1(y + 8));
}

struct StoreArgs {
  const uint8_t* src[2];
  Strides st[2];
  uint8_t* codes[2];
  uint8_t* scales[2];
  float down[2];  // 2^-exp
  const int32_t* idx;
  const int32_t* row0_dev;
  const int32_t* pos;
  int N, H, L, rows, row0, cap;
  int T, log_t, HG, n_hg, n_lt;
};

// Source row of result row r (-1: zeros).
__device__ __forceinline__ int source_row(const StoreArgs& a, int64_t nh, int r) {
  if (a.idx == nullptr) return r;
  const int j = __ldg(a.idx + nh * a.rows + r);
  return j >= 0 && j < a.L ? j : -1;
}

// kRope: 0 none, 1 half layout, 2 interleaved.
template <typename T, int D, int kRope>
__global__ void __launch_bounds__(kThreads)
    store_kernel(const StoreArgs a, const __grid_constant__ fc_rope_plan plan) {
  extern __shared__ float2 cs[];
  constexpr int G = D / 16;  // groups (and threads) of a row
  constexpr int kRowsPerPass = kThreads / G;
  const int kv = blockIdx.y;  // 0 keys, 1 values
  int b = blockIdx.x;
  const int hg = b % a.n_hg;
  b /= a.n_hg;
  const int l0 = (b % a.n_lt) * a.T;
  const int n = b / a.n_lt;
  const int nt = min(a.T, a.rows - l0);
  grid_dep_wait();
  const bool rotate = kRope != 0 && kv == 0;
  const int half = plan.rot_dim / 2;
  if (rotate) {
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
      const int t = i / half, f = i - t * half;
      const int32_t p = __ldg(a.pos + ((int64_t)plan.axis[f] * a.N + n) * a.L + l0 + t);
      cs[i] = rope_cs(p, plan.turns[f], plan.m, false);
    }
    __syncthreads();
  }
  const int first = a.row0_dev != nullptr ? __ldg(a.row0_dev + n) : a.row0;
  const int h0 = hg * a.HG, nh = min(a.HG, a.H - h0);
  const int g = threadIdx.x % G;
  const Strides st = a.st[kv];
  const T* src = reinterpret_cast<const T*>(a.src[kv]) + n * st.n;
  const int rows = nh << a.log_t;
  for (int r = threadIdx.x / G; r < rows; r += kRowsPerPass) {
    const int t = r & (a.T - 1), h = h0 + (r >> a.log_t);
    const int64_t dst = (int64_t)first + l0 + t;
    if (t >= nt || dst < 0 || dst >= a.cap) continue;
    const int64_t nhi = (int64_t)n * a.H + h;
    const int j = source_row(a, nhi, l0 + t);
    float y[16];
    if (j >= 0) {
      const T* row = src + h * st.h + (int64_t)j * st.l;
      load16(row + g * 16, y);
      if (rotate && g * 16 < plan.rot_dim) {
        const float2* c = cs + t * half;
        if constexpr (kRope == 1) {
          if (half % 16 == 0) {  // the group and its partners are whole groups
            float z[16];
            const bool low = g * 16 < half;
            load16(row + g * 16 + (low ? half : -half), z);
            c += low ? g * 16 : g * 16 - half;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              y[i] = low ? rope_a(y[i], z[i], c[i]) : rope_b(z[i], y[i], c[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int e = g * 16 + i;
              if (e < half)
                y[i] = rope_a(y[i], load1(row + e + half), c[e]);
              else if (e < plan.rot_dim)
                y[i] = rope_b(load1(row + e - half), y[i], c[e - half]);
            }
          }
        } else {
          c += g * 8;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (g * 8 + i < half) {
              const float y0 = y[2 * i];
              y[2 * i] = rope_a(y0, y[2 * i + 1], c[i]);
              y[2 * i + 1] = rope_b(y0, y[2 * i + 1], c[i]);
            }
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = 0.0f;
    }
    const float down = a.down[kv];
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = __fmul_rn(y[i], down);
    uint32_t scale;
    const uint2 codes = quantise16(y, scale);
    const int64_t at = (nhi * a.cap + dst) * G + g;
    reinterpret_cast<uint2*>(a.codes[kv])[at] = codes;
    a.scales[kv][at] = (uint8_t)scale;
  }
}

template <typename T, int D>
cudaError_t run_store(StoreArgs a, const fc_rope_plan* plan, cudaStream_t s) {
  constexpr int kRowsPerPass = kThreads / (D / 16);
  a.log_t = 0;
  while (a.log_t < 4 && (1 << a.log_t) < a.rows) ++a.log_t;
  a.T = 1 << a.log_t;
  a.n_lt = (int)ceil_div(a.rows, a.T);
  a.HG = a.H;
  // as for the rotation alone: split the heads while SMs would be idle, and
  // without angles to share down to one pass of a block
  const int64_t want = plan != nullptr ? 6ll * sm_count() : INT64_MAX;
  const int64_t tiles = (int64_t)a.N * a.n_lt;
  while (a.HG > 1 && tiles * ceil_div(a.H, a.HG) < want && (a.HG + 1) / 2 * a.T >= kRowsPerPass)
    a.HG = (a.HG + 1) / 2;
  a.n_hg = (int)ceil_div(a.H, a.HG);
  const int64_t blocks = tiles * a.n_hg;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  fc_rope_plan none = {};
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, 2);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  if (plan == nullptr) {
    e = cudaLaunchKernelEx(&cfg, store_kernel<T, D, 0>, a, none);
  } else {
    cfg.dynamicSmemBytes = (size_t)a.T * (plan->rot_dim / 2) * sizeof(float2);
    e = plan->layout == FC_ROPE_HALF ? cudaLaunchKernelEx(&cfg, store_kernel<T, D, 1>, a, *plan)
                                     : cudaLaunchKernelEx(&cfg, store_kernel<T, D, 2>, a, *plan);
  }
  if (e != cudaSuccess) return e;
  add_launches(1);
  return cudaGetLastError();
}

struct LoadArgs {
  const uint8_t* codes[2];
  const uint8_t* scales[2];
  uint8_t* dst[2];
  Strides st[2];
  float up[2];  // 2^exp
  const int32_t* row0_dev;
  int H, L, row0, cap;
  int n_lt;  // row tiles of a head
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) load_kernel(const LoadArgs a) {
  constexpr int G = D / 16;
  constexpr int V = 16 / (int)sizeof(T);
  constexpr int kRowsPerPass = kThreads / G;
  grid_dep_wait();
  const int kv = blockIdx.y;
  const int nh = blockIdx.x / a.n_lt;
  const int l = (blockIdx.x % a.n_lt) * kRowsPerPass + threadIdx.x / G;
  const int g = threadIdx.x % G;
  if (l >= a.L) return;
  const int n = nh / a.H, h = nh % a.H;
  const int64_t src = (int64_t)(a.row0_dev != nullptr ? __ldg(a.row0_dev + n) : a.row0) + l;
  float f[16];
  if (src >= 0 && src < a.cap) {
    const int64_t at = ((int64_t)nh * a.cap + src) * G + g;
    const uint2 c = __ldg(reinterpret_cast<const uint2*>(a.codes[kv]) + at);
    const uint32_t sb = __ldg(a.scales[kv] + at);
    const float s = __fmul_rn(kv4::lo_f16(kv4::e4m3x2_to_f16x2(sb)), a.up[kv]);
    uint32_t p[8];
    kv4::e2m1x8_to_f16x2(c.x, reinterpret_cast<uint32_t(&)[4]>(p[0]));
    kv4::e2m1x8_to_f16x2(c.y, reinterpret_cast<uint32_t(&)[4]>(p[4]));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f[2 * i] = kv4::lo_f16(p[i]) * s;
      f[2 * i + 1] = kv4::lo_f16(p[i] >> 16) * s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = 0.0f;
  }
  const Strides st = a.st[kv];
  T* out = reinterpret_cast<T*>(a.dst[kv]) + n * st.n + h * st.h + (int64_t)l * st.l + g * 16;
#pragma unroll
  for (int i = 0; i < 16 / V; ++i) {
    uint4 w;
    if constexpr (sizeof(T) == 4) {
      w = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                     __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3]));
    } else {  // exact: the products have at most 6 significant bits
      uint32_t u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[8 * i + 2 * j], f[8 * i + 2 * j + 1]);
        u[j] = reinterpret_cast<const uint32_t&>(b);
      }
      w = make_uint4(u[0], u[1], u[2], u[3]);
    }
    reinterpret_cast<uint4*>(out)[i] = w;
  }
}

template <typename T, int D>
cudaError_t run_load(LoadArgs a, int N, cudaStream_t s) {
  a.n_lt = (int)ceil_div(a.L, kThreads / (D / 16));
  const int64_t blocks = (int64_t)N * a.H * a.n_lt;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, 2);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, load_kernel<T, D>, a);
  if (e != cudaSuccess) return e;
  add_launches(1);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_kv4_store(const void* k, const void* v, bool bf16, int L, Strides ks, Strides vs,
                             const int32_t* idx, int rows, int row0, const int32_t* row0_dev,
                             const fc_rope_plan* plan, const int32_t* pos,
                             const fc_kv4_cache& c, cudaStream_t s) {
  StoreArgs a = {};
  a.src[0] = static_cast<const uint8_t*>(k);
  a.src[1] = static_cast<const uint8_t*>(v);
  a.st[0] = ks;
  a.st[1] = vs;
  a.codes[0] = static_cast<uint8_t*>(c.k_codes);
  a.codes[1] = static_cast<uint8_t*>(c.v_codes);
  a.scales[0] = static_cast<uint8_t*>(c.k_scales);
  a.scales[1] = static_cast<uint8_t*>(c.v_scales);
  a.down[0] = ldexpf(1.0f, -c.k_exp);
  a.down[1] = ldexpf(1.0f, -c.v_exp);
  a.idx = idx;
  a.row0_dev = row0_dev;
  a.pos = pos;
  a.N = c.N;
  a.H = c.H;
  a.L = L;
  a.rows = rows;
  a.row0 = row0;
  a.cap = c.cap;
  if (c.d == 128)
    return bf16 ? run_store<__nv_bfloat16, 128>(a, plan, s) : run_store<float, 128>(a, plan, s);
  return bf16 ? run_store<__nv_bfloat16, 64>(a, plan, s) : run_store<float, 64>(a, plan, s);
}

cudaError_t launch_kv4_load(const fc_kv4_cache& c, void* k, void* v, bool bf16, int L, Strides ks,
                            Strides vs, int row0, const int32_t* row0_dev, cudaStream_t s) {
  LoadArgs a = {};
  a.codes[0] = static_cast<const uint8_t*>(c.k_codes);
  a.codes[1] = static_cast<const uint8_t*>(c.v_codes);
  a.scales[0] = static_cast<const uint8_t*>(c.k_scales);
  a.scales[1] = static_cast<const uint8_t*>(c.v_scales);
  a.dst[0] = static_cast<uint8_t*>(k);
  a.dst[1] = static_cast<uint8_t*>(v);
  a.st[0] = ks;
  a.st[1] = vs;
  a.up[0] = ldexpf(1.0f, c.k_exp);
  a.up[1] = ldexpf(1.0f, c.v_exp);
  a.row0_dev = row0_dev;
  a.H = c.H;
  a.L = L;
  a.row0 = row0;
  a.cap = c.cap;
  if (c.d == 128)
    return bf16 ? run_load<__nv_bfloat16, 128>(a, c.N, s) : run_load<float, 128>(a, c.N, s);
  return bf16 ? run_load<__nv_bfloat16, 64>(a, c.N, s) : run_load<float, 64>(a, c.N, s);
}

}  // namespace fc
