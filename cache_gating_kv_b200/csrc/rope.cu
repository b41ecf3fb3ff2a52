// Rotary positions of queries and keys.
//
// For the pair (a, b) of frequency i at position p the kernel writes
// (a c - b s, b c + a s) with c = m cos(2 pi p w_i), s = m sin(2 pi p w_i).
// Per element that is 3 flops on 2 x 2 bytes (bf16), so the bound is HBM; the
// angles are the only costly arithmetic (a float64 sine and cosine), and all
// heads of a token share them.  A block therefore takes T tokens, writes their
// T x rot/2 (c, s) pairs to shared memory once, and streams the rows of a
// group of heads through them with 16-byte vectors, a thread's pairs in registers.
// 40 heads x 8190 tokens x 128 bf16: 31 us, 168 MB at 5.3 TB/s (82 % of the measured
// copy rate); with frequencies read by lane from the constant bank 46, with 16
// tokens to a block 33, with two rows in flight 34.  A rotated part that does not end
// on a vector (24 of 128 in the half layout, 6 in both) goes element by element and
// takes 91 us, float32 96.
#include "fc_common.cuh"
#include "fc_kernels.h"
#include "kv4.cuh"

namespace fc {

namespace {
constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // rows a thread loads before it stores the first
constexpr int kLogTokens = 3;  // tokens of a block: at most 8

struct RopeArgs {
  const uint8_t* x;
  uint8_t* y;
  Strides xs, ys;
  const int32_t* pos;
  int N, H, L, d;
  int T, log_t;        // tokens of a block, a power of two
  int HG, n_hg, n_lt;  // heads of a block, head groups, token tiles
  int upr, rpi;        // units of a row, rows of a pass
  bool inverse;
};

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f(float v) { return v; }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) {
  return __float2bfloat16_rn(v);
}

template <typename T>
__device__ __forceinline__ uint4 pack16(const float* f) {
  if constexpr (sizeof(T) == 4) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = reinterpret_cast<const uint32_t&>(h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// kVec: a unit is a pair of 16-byte vectors (half layout) or one vector
// (interleaved); without it, for rotated parts that do not end on a vector, a
// unit is one pair of elements.
template <typename T, bool kHalf, bool kVec>
__global__ void __launch_bounds__(kThreads)
    rope_kernel(const RopeArgs a, const __grid_constant__ fc_rope_plan plan) {
  extern __shared__ float2 cs[];  // [T][rot/2], behind the turns and the axes
  double* turns = reinterpret_cast<double*>(cs + a.T * (plan.rot_dim / 2));
  uint8_t* axes = reinterpret_cast<uint8_t*>(turns + plan.rot_dim / 2);
  constexpr int V = 16 / (int)sizeof(T);
  const int half = plan.rot_dim / 2;
  int b = blockIdx.x;
  const int hg = b % a.n_hg;
  b /= a.n_hg;
  const int l0 = (b % a.n_lt) * a.T;
  const int n = b / a.n_lt;
  const int nt = min(a.T, a.L - l0);
  // Lanes of a warp want different frequencies, which the constant bank would hand
  // out one at a time.
  for (int f = threadIdx.x; f < half; f += kThreads) {
    turns[f] = plan.turns[f];
    axes[f] = plan.axis[f];
  }
  __syncthreads();
  grid_dep_wait();
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int t = i / half, f = i - t * half;
    const int32_t p = a.pos[((int64_t)axes[f] * a.N + n) * a.L + l0 + t];
    cs[i] = rope_cs(p, turns[f], plan.m, a.inverse);
  }
  __syncthreads();
  const int h0 = hg * a.HG, nh = min(a.HG, a.H - h0);
  const int rpi = a.rpi;  // a multiple of T: a thread keeps its token and its angles
  const int u = threadIdx.x % a.upr;
  const int r0 = threadIdx.x / a.upr;
  if (r0 >= rpi) return;
  const T* x = reinterpret_cast<const T*>(a.x) + n * a.xs.n + (int64_t)h0 * a.xs.h;
  T* y = reinterpret_cast<T*>(a.y) + n * a.ys.n + (int64_t)h0 * a.ys.h;
  const int rows = nh << a.log_t;  // row r: token r % T, head r / T

  if constexpr (kVec) {
    // element offsets of the unit's vectors; a unit that only copies has one
    const int pu = kHalf ? half / V : plan.rot_dim / V;  // units that rotate
    const bool rot = u < pu;
    const int e0 = rot ? u * V : plan.rot_dim + (u - pu) * V;
    const int t = r0 & (a.T - 1);
    if (t >= nt) return;
    constexpr int kPairs = kHalf ? V : V / 2;
    float2 c[kPairs];
    if (rot) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) c[i] = cs[t * half + u * kPairs + i];
    }
    x += (int64_t)(l0 + t) * a.xs.l + e0;
    y += (int64_t)(l0 + t) * a.ys.l + e0;
    for (int r = r0; r < rows; r += rpi * kUnroll) {
      uint4 va[kUnroll], vb[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int q = r + k * rpi;
        if (q < rows) {
          const T* p = x + (int64_t)(q >> a.log_t) * a.xs.h;
          va[k] = *reinterpret_cast<const uint4*>(p);
          if (kHalf && rot) vb[k] = *reinterpret_cast<const uint4*>(p + half);
        }
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int q = r + k * rpi;
        if (q >= rows) continue;
        T* p = y + (int64_t)(q >> a.log_t) * a.ys.h;
        if (rot) {
          float f[V], g[V];
          Vec16<T>::to_float(va[k], f);
          if constexpr (kHalf) {
            Vec16<T>::to_float(vb[k], g);
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float f0 = f[i];
              f[i] = rope_a(f0, g[i], c[i]);
              g[i] = rope_b(f0, g[i], c[i]);
            }
            *reinterpret_cast<uint4*>(p + half) = pack16<T>(g);
          } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
              const float f0 = f[2 * i];
              f[2 * i] = rope_a(f0, f[2 * i + 1], c[i]);
              f[2 * i + 1] = rope_b(f0, f[2 * i + 1], c[i]);
            }
          }
          *reinterpret_cast<uint4*>(p) = pack16<T>(f);
        } else {
          *reinterpret_cast<uint4*>(p) = va[k];
        }
      }
    }
  } else {
    const bool rot = u < half;
    const int ea = kHalf && rot ? u : 2 * u;
    const int eb = kHalf && rot ? u + half : 2 * u + 1;
    for (int r = r0; r < rows; r += rpi) {
      const int t = r & (a.T - 1);
      if (t >= nt) continue;
      const T* p = x + (int64_t)(r >> a.log_t) * a.xs.h + (int64_t)(l0 + t) * a.xs.l;
      T* w = y + (int64_t)(r >> a.log_t) * a.ys.h + (int64_t)(l0 + t) * a.ys.l;
      const T xa = p[ea], xb = p[eb];
      if (rot) {
        const float2 c = cs[t * half + u];
        w[ea] = from_f<T>(rope_a(to_f(xa), to_f(xb), c));
        w[eb] = from_f<T>(rope_b(to_f(xa), to_f(xb), c));
      } else {
        w[ea] = xa;
        w[eb] = xb;
      }
    }
  }
}

template <typename T, bool kHalf, bool kVec>
cudaError_t run(RopeArgs a, const fc_rope_plan& plan, cudaStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  const int half = plan.rot_dim / 2;
  a.upr = !kVec ? a.d / 2 : kHalf ? half / V + (a.d - plan.rot_dim) / V : a.d / V;
  a.rpi = kThreads / a.upr;
  a.log_t = 0;
  while (a.log_t < kLogTokens && (1 << a.log_t) < a.L && (2 << a.log_t) <= a.rpi) ++a.log_t;
  a.T = 1 << a.log_t;
  a.rpi &= ~(a.T - 1);
  a.n_lt = (int)ceil_div(a.L, a.T);
  // Fewer heads to a block (each block computes its angles anew) only while the grid
  // would leave SMs without work and a block keeps a full pass.
  a.HG = a.H;
  const int64_t want = 4ll * sm_count(), tiles = (int64_t)a.N * a.n_lt;
  while (a.HG > 1 && tiles * ceil_div(a.H, a.HG) < want && (a.HG + 1) / 2 * a.T >= a.rpi)
    a.HG = (a.HG + 1) / 2;
  a.n_hg = (int)ceil_div(a.H, a.HG);
  const int64_t blocks = tiles * a.n_hg;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)half * (a.T * sizeof(float2) + sizeof(double) + 1);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, rope_kernel<T, kHalf, kVec>, a, plan);
  if (e != cudaSuccess) return e;
  add_launches(1);
  return cudaGetLastError();
}

template <typename T>
cudaError_t pick(const RopeArgs& a, const fc_rope_plan& plan, cudaStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  if (plan.layout == FC_ROPE_HALF)
    return plan.rot_dim % (2 * V) == 0 ? run<T, true, true>(a, plan, s)
                                       : run<T, true, false>(a, plan, s);
  return plan.rot_dim % V == 0 ? run<T, false, true>(a, plan, s)
                               : run<T, false, false>(a, plan, s);
}
}  // namespace

cudaError_t launch_rope(const void* x, void* y, bool bf16, int N, int H, int L, int d, Strides xs,
                        Strides ys, const int32_t* pos, const fc_rope_plan& plan, bool inverse,
                        cudaStream_t s) {
  RopeArgs a = {};
  a.x = static_cast<const uint8_t*>(x);
  a.y = static_cast<uint8_t*>(y);
  a.xs = xs;
  a.ys = ys;
  a.pos = pos;
  a.N = N;
  a.H = H;
  a.L = L;
  a.d = d;
  a.inverse = inverse;
  return bf16 ? pick<__nv_bfloat16>(a, plan, s) : pick<float>(a, plan, s);
}

}  // namespace fc
