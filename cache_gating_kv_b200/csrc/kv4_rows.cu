// Rows into and out of the 4-bit cache.
//
// Storing reads 2 x 2 bytes per element pair of K and V (bf16) and writes 4.5
// bits per element, loading the reverse, so both are bound by HBM.  In storing one
// thread owns one group of 16 elements: the group's maximum, its scale and its eight
// bytes of codes then need no exchange between threads, a warp's code stores
// are 256 contiguous bytes and its reads 1 KB.  (In loading a thread takes half a
// group: see there.)  For keys that are rotated on
// the way the thread also reads the partner elements of its group (the same
// lines, read by another thread of the warp, so they come from L1) instead of
// exchanging numbers through shared memory.  16380 selected rows of 40 heads, d = 128,
// bf16, stored and read back: 159 us for 768 MB (74 % of the measured copy rate), of
// which reading back is 69 (95 %); storing issues about 230 instructions to a group
// and waits for its loads in turn.  4096 rows of 24 heads with rotated keys: 37 us for
// 115 MB; storing (29 of them with cold caches) issues in half of the cycles, and of the
// 13.7 from one instruction of a warp to its next 6.2 wait for loads from memory and 2.0
// for shared memory: the angles come before a block's first row is asked for, and one
// row of a thread is under way at a time.
#include <cuda.h>

#include "fc_common.cuh"
#include "fc_kernels.h"
#include "kv4.cuh"
#include "tc_ptx.cuh"

namespace fc {

namespace {
constexpr int kThreads = 256;
constexpr int kLoadRows = 4;  // rows of a thread that reads the cache

// 16 consecutive elements as float32.
template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&f)[16]) {
  constexpr int V = 16 / (int)sizeof(T);
#pragma unroll
  for (int i = 0; i < 16 / V; ++i)
    Vec16<T>::to_float(reinterpret_cast<const uint4*>(p)[i], f + i * V);
}

template <typename T>
__device__ __forceinline__ float load1(const T* p) {
  if constexpr (sizeof(T) == 4)
    return *p;
  else
    return __uint_as_float((uint32_t)*reinterpret_cast<const unsigned short*>(p) << 16);
}

// The largest |x| of 16 raw elements; NaN if one of them is.
__device__ __forceinline__ float absmax16(const uint4 (&w)[2], __nv_bfloat16) {
  __nv_bfloat162 m = __habs2(reinterpret_cast<const __nv_bfloat162&>(w[0].x));
  const uint32_t u[7] = {w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
  for (int i = 0; i < 7; ++i)
    m = __hmax2_nan(m, __habs2(reinterpret_cast<const __nv_bfloat162&>(u[i])));
  return __bfloat162float(__hmax_nan(m.x, m.y));
}
__device__ __forceinline__ float absmax16(const float (&x)[16]) {
  uint32_t top = 0;  // as bits: NaN counts above infinity
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
  return __uint_as_float(top);
}

// One group of 16 numbers, given as their negatives x with the largest |x|, to its
// scale byte and its eight code bytes; `down` and `up` are 2^-exp and 2^exp, powers of two that are multiplied into
// the scale and its reciprocal instead of every element.
__device__ __forceinline__ uint2 quantise16(float (&x)[16], float amax, float down, float up,
                                            uint32_t& scale) {
  amax *= down;
  if (!(amax <= 4096.0f)) {
    if (amax != amax) {  // the group reads as NaN
      scale = 0x7Fu;
      return make_uint2(0u, 0u);
    }
    // Numbers beyond 6 * 448 saturate whatever they are; cutting them here keeps
    // the quotients below finite (their scale is 448).
    const float cut = 4096.0f * up;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = fminf(fmaxf(x[i], -cut), cut);
  }
  // (rounded quotients as below, the reciprocal of 6 being a constant)
  constexpr float kSixth = 1.0f / 6.0f;
  const float a6 = __fmul_rn(amax, kSixth);
  scale = kv4::f32_to_e4m3(fminf(__fmaf_rn(-__fmaf_rn(a6, 6.0f, -amax), kSixth, a6), 448.0f));
  float s = kv4::lo_f16(kv4::e4m3x2_to_f16x2(scale));
  // y / s rounded to nearest, so that a number half way between two codes is
  // seen as such: from the correctly rounded reciprocal r, q = y r is within an
  // ulp and q - r (q s - y) is the rounded quotient (Markstein, "Computation of
  // elementary functions on the IBM RISC System/6000 processor", 1990).  Two
  // numbers to an instruction, from -y and -r; in this order a zero keeps its sign.
  const float nr = s > 0.0f ? __frcp_rn(s) * -down : -0.0f;
  s *= up;
  const float2 rr = make_float2(nr, nr), ss = make_float2(s, s);
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const float2 y = make_float2(x[i], x[i + 1]);  // negative
    const float2 q = tc::fmul2(y, rr);
    const float2 t = tc::ffma2(tc::ffma2(q, ss, y), rr, q);
    x[i] = t.x;
    x[i + 1] = t.y;
  }
  return make_uint2(kv4::f32x8_to_e2m1(x), kv4::f32x8_to_e2m1(x + 8));
}

struct StoreArgs {
  const uint8_t* src[2];
  Strides st[2];
  uint8_t* codes[2];
  uint8_t* scales[2];
  float down[2], up[2];  // 2^-exp, 2^exp
  const int32_t* idx;
  const int32_t* row0_dev;
  const int32_t* pos;
  int N, H, L, rows, row0, cap;
  int T, log_t, HG, n_hg, n_lt;
};

// kRope: 0 none, 1 half layout, 2 interleaved.
template <typename T, int D, int kRope>
__global__ void __launch_bounds__(kThreads, 4)
    store_kernel(const StoreArgs a, const __grid_constant__ fc_rope_plan plan) {
  extern __shared__ float2 cs[];  // [T][rot/2], behind the turns and the axes
  constexpr int G = D / 16;       // groups (and threads) of a row
  constexpr int kRowsPerPass = kThreads / G;
  constexpr int kRaw = (int)sizeof(T);  // 16-byte vectors of a group: 2 (bf16), 4
  constexpr int kUnroll = kRope == 0 ? 2 : 1;  // rows loaded before the first is stored
  const int kv = blockIdx.y;  // 0 keys, 1 values
  int b = blockIdx.x;
  const int hg = b % a.n_hg;
  b /= a.n_hg;
  const int l0 = (b % a.n_lt) * a.T;
  const int n = b / a.n_lt;
  const int nt = min(a.T, a.rows - l0);
  const bool rotate = kRope != 0 && kv == 0;
  const int half = plan.rot_dim / 2;
  double* turns = reinterpret_cast<double*>(cs + a.T * half);
  uint8_t* axes = reinterpret_cast<uint8_t*>(turns + half);
  if (rotate) {  // (lanes want different frequencies: see the rotation's kernel)
    for (int f = threadIdx.x; f < half; f += kThreads) {
      turns[f] = plan.turns[f];
      axes[f] = plan.axis[f];
    }
    __syncthreads();
  }
  grid_dep_wait();
  if (rotate) {
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
      const int t = i / half, f = i - t * half;
      const int32_t p = a.pos[((int64_t)axes[f] * a.N + n) * a.L + l0 + t];
      cs[i] = rope_cs(p, turns[f], plan.m, false);
    }
    __syncthreads();
  }
  const int h0 = hg * a.HG, nh = min(a.HG, a.H - h0);
  const int g = threadIdx.x % G;
  const Strides st = a.st[kv];
  const float down = a.down[kv], up = a.up[kv];
  // Pass by pass a thread goes on either by tokens of one head (T over the rows of a
  // pass) or by heads of one token.
  const bool by_token = a.T > kRowsPerPass;
  const int step_t = by_token ? kRowsPerPass : 0;
  const int step_h = by_token ? 0 : kRowsPerPass >> a.log_t;
  int t = threadIdx.x / G & (a.T - 1), h = threadIdx.x / G >> a.log_t;
  const int64_t nhi = (int64_t)n * a.H + h0 + h;
  // tokens whose row lies in the cache
  const int64_t row0 = (int64_t)(a.row0_dev != nullptr ? a.row0_dev[n] : a.row0) + l0;
  const int t_min = (int)max((int64_t)0, min((int64_t)nt, -row0));
  const int t_max = (int)max((int64_t)0, min((int64_t)nt, a.cap - row0));
  // group of the cache, element of the source: of this pass, and on to the next
  int64_t o = (nhi * a.cap + row0 + t) * G + g;
  const int64_t o_step = ((int64_t)step_h * a.cap + step_t) * G;
  const T* src = reinterpret_cast<const T*>(a.src[kv]) + n * st.n + (h0 + h) * st.h + g * 16;
  const int32_t* idx = a.idx != nullptr ? a.idx + nhi * a.rows + l0 + t : nullptr;
  const int64_t idx_step = (int64_t)step_h * a.rows + step_t;
  const int64_t src_step = step_h * st.h + (idx == nullptr ? step_t * st.l : 0);
  if (idx == nullptr) src += (int64_t)(l0 + t) * st.l;
  uint2* const codes_out = reinterpret_cast<uint2*>(a.codes[kv]);
  uint8_t* const scales_out = a.scales[kv];
  const int64_t src_l = st.l;
  const int L = a.L;
  // The next pass's indices are loaded a pass ahead: they are the only load that
  // another one waits for.
  int ahead[kUnroll];
#pragma unroll
  for (int k = 0; k < kUnroll; ++k)
    ahead[k] = idx != nullptr && t + k * step_t < nt && h + k * step_h < nh ? idx[k * idx_step] : 0;
  while (t < t_max && h < nh) {
    bool put[kUnroll];
    const T* from[kUnroll]; // nullptr: zeros
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      put[k] = t >= t_min && t < t_max && h < nh;
      from[k] = src;
      if (idx != nullptr)
        from[k] = (unsigned)ahead[k] < (unsigned)L ? src + ahead[k] * src_l : nullptr;
      t += step_t;
      h += step_h;
      src += src_step;
    }
    if (idx != nullptr) {
      idx += kUnroll * idx_step;
#pragma unroll
      for (int k = 0; k < kUnroll; ++k)
        ahead[k] = t + k * step_t < nt && h + k * step_h < nh ? idx[k * idx_step] : 0;
    }
    uint4 raw[kUnroll][kRaw];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
#pragma unroll
      for (int i = 0; i < kRaw; ++i) {
        raw[k][i] = make_uint4(0u, 0u, 0u, 0u);
        if (put[k] && from[k] != nullptr) raw[k][i] = reinterpret_cast<const uint4*>(from[k])[i];
      }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k, o += o_step) {
      if (!put[k]) continue;
      float y[16];
      const bool turn = rotate && g * 16 < plan.rot_dim && from[k] != nullptr;
#pragma unroll
      for (int i = 0; i < kRaw; ++i) {
        // to the negatives: of what is rotated only behind it, since a zero that a
        // rotation of negatives gives has not the sign of the zero that it stands for
        const uint32_t flip = turn ? 0u : sizeof(T) == 2 ? 0x80008000u : 0x80000000u;
        raw[k][i].x ^= flip;
        raw[k][i].y ^= flip;
        raw[k][i].z ^= flip;
        raw[k][i].w ^= flip;
        Vec16<T>::to_float(raw[k][i], y + i * (16 / kRaw));
      }
      if (turn) {
        const float2* c = cs + (threadIdx.x / G & (a.T - 1)) * half;  // (by heads)
        if constexpr (kRope == 1) {
          const T* row = from[k] - g * 16;
          if (half % 16 == 0) {  // the group and its partners are whole groups
            float z[16];
            const bool low = g * 16 < half;
            load16(from[k] + (low ? half : -half), z);
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
        } else if constexpr (kRope == 2) {
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
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = -y[i];
      }
      float amax;
      if constexpr (sizeof(T) == 2)
        amax = turn ? absmax16(y) : absmax16(raw[k], T());
      else
        amax = absmax16(y);
      uint32_t scale;
      const uint2 codes = quantise16(y, amax, down, up, scale);
      codes_out[o] = codes;
      scales_out[o] = (uint8_t)scale;
    }
  }
}

template <typename T, int D>
cudaError_t run_store(StoreArgs a, const fc_rope_plan* plan, cudaStream_t s) {
  constexpr int kRowsPerPass = kThreads / (D / 16);
  // Rotated keys: few tokens and many heads to a block, which share the angles.
  // Otherwise a run of tokens, whose rows (or kept rows) lie close together.
  const int most = plan != nullptr ? 3 : 9;
  a.log_t = 0;
  while (a.log_t < most && (1 << a.log_t) < a.rows) ++a.log_t;
  a.T = 1 << a.log_t;
  a.n_lt = (int)ceil_div(a.rows, a.T);
  // Heads of a block: with rotated keys as many as share the angles, unless that
  // leaves SMs idle; else one, or what two loads of the block's threads reach.
  a.HG = a.H;
  const int64_t want = plan != nullptr ? 3ll * sm_count() : INT64_MAX;
  const int64_t tiles = (int64_t)a.N * a.n_lt;
  const int least = plan != nullptr ? kRowsPerPass : 2 * kRowsPerPass;
  while (a.HG > 1 && tiles * ceil_div(a.H, a.HG) < want && (a.HG + 1) / 2 * a.T >= least)
    a.HG = (a.HG + 1) / 2;
  if (a.T > kRowsPerPass) a.HG = 1;
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
    cfg.dynamicSmemBytes =
        (size_t)(plan->rot_dim / 2) * (a.T * sizeof(float2) + sizeof(double) + 1);
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

// A thread takes 8 codes, for bf16 16 bytes of numbers, so that a warp's stores are
// whole lines (with 16 numbers to a thread every store covered half sectors: 4.7 of
// 6.6 TB/s).
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) load_kernel(const LoadArgs a) {
  constexpr int TPR = D / 8;  // threads of a row
  constexpr int kRowsPerPass = kThreads / TPR;
  grid_dep_wait();
  const int kv = blockIdx.y;
  const int nh = blockIdx.x / a.n_lt;
  const int l0 = (blockIdx.x % a.n_lt) * (kRowsPerPass * kLoadRows) + threadIdx.x / TPR;
  const int c = threadIdx.x % TPR;
  const int n = nh / a.H, h = nh % a.H;
  const int64_t first = a.row0_dev != nullptr ? a.row0_dev[n] : a.row0;
  const Strides st = a.st[kv];
  T* out = reinterpret_cast<T*>(a.dst[kv]) + n * st.n + h * st.h + c * 8;
  const float up = a.up[kv];
  uint32_t code[kLoadRows], sb[kLoadRows];
#pragma unroll
  for (int k = 0; k < kLoadRows; ++k) {
    const int l = l0 + k * kRowsPerPass;
    const int64_t src = first + l;
    code[k] = sb[k] = 0;
    if (l < a.L && src >= 0 && src < a.cap) {
      const int64_t row = (int64_t)nh * a.cap + src;
      code[k] = reinterpret_cast<const uint32_t*>(a.codes[kv] + row * (D / 2))[c];
      sb[k] = a.scales[kv][row * (D / 16) + (c >> 1)];
    }
  }
#pragma unroll
  for (int k = 0; k < kLoadRows; ++k) {
    const int l = l0 + k * kRowsPerPass;
    if (l >= a.L) return;
    const float s = kv4::lo_f16(kv4::e4m3x2_to_f16x2(sb[k])) * up;
    uint32_t p[4];
    kv4::e2m1x8_to_f16x2(code[k], p);
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = kv4::lo_f16(p[i]) * s;
      f[2 * i + 1] = kv4::lo_f16(p[i] >> 16) * s;
    }
    uint4* w = reinterpret_cast<uint4*>(out + (int64_t)l * st.l);
    if constexpr (sizeof(T) == 4) {
      w[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                        __float_as_uint(f[3]));
      w[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                        __float_as_uint(f[7]));
    } else {  // exact: the products have at most 6 significant bits
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        u[i] = reinterpret_cast<const uint32_t&>(b);
      }
      *w = make_uint4(u[0], u[1], u[2], u[3]);
    }
  }
}

template <typename T, int D>
cudaError_t run_load(LoadArgs a, int N, cudaStream_t s) {
  a.n_lt = (int)ceil_div(a.L, kThreads * 8 / D * kLoadRows);
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
  a.up[0] = ldexpf(1.0f, c.k_exp);
  a.up[1] = ldexpf(1.0f, c.v_exp);
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
