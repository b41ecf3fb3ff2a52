// Attention over the 4-bit cache for few query rows per key head (decoding), and
// for float32 queries.
//
//   out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j)
//
// The R = (Hq/Hkv) Lq query rows of a key head read the same keys, so they share
// one pass over them: row r is query r / G of head r % G in the group.  The
// bound is HBM: a key and its value are 144 bytes at d = 128 (72 at 64) for 4 R d
// flops.  What has to keep up with it is the conversion of the codes, so
//   - the codes go from shared memory straight into the B fragments of
//     mma.m16n8k16 and are never written back as float16: a thread reads 32
//     consecutive codes of a key (16 bytes), and the order in which the MMA
//     steps see the elements of d is whatever that makes it, since the queries
//     are loaded in the same order.  Values need pairs of keys instead of pairs
//     of elements: two shift-and-select instructions interleave the nibbles of
//     two keys' words before the conversion.  Which output column a thread's
//     element is follows from the same freedom: each thread ends with 32
//     consecutive outputs of a row;
//   - code * scale is exact in float16 (at most 6 significant bits), so one
//     packed multiplication per pair finishes the conversion;
//   - each warp walks its own keys (steps of 32, in turn with the other warps of
//     the block) behind its own ring of bulk copies, with its own running
//     maximum, sum and output; there is no barrier in the loop.  The warps are
//     joined at the end, and the shares of a long axis by a second, small kernel.
// The running maximum only moves when a step exceeds it by 2^8 (float16
// probabilities, offset by 2^5, keep 11 bits over that range); for float32
// queries it is exact, and queries and probabilities are sums of two float16
// (22 bits and the sign of the second).
#include <cuda.h>

#include "fc_common.cuh"
#include "fc_kernels.h"
#include "kv4.cuh"
#include "kv4_attn.cuh"
#include "tc_ptx.cuh"

namespace fc {

namespace {
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStep = 32;  // keys of a warp's step

template <int D> constexpr int step_bytes() { return kStep * (D + D / 8); }
template <int D> constexpr int stages() { return D == 128 ? 3 : 5; }
template <int D> constexpr int ring_bytes() { return step_bytes<D>() * stages<D>(); }
template <int D, int MT> constexpr int merge_bytes() { return MT * 16 * (D + 2) * 4; }
template <int D, int MT> constexpr int warp_bytes() {
  return ring_bytes<D>() > merge_bytes<D, MT>() ? ring_bytes<D>() : merge_bytes<D, MT>();
}
template <int D, int MT> constexpr int smem_bytes() {
  return kWarps * warp_bytes<D, MT>() + kWarps * stages<D>() * 8;
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// What float16 rounding left of (lo, hi).
__device__ __forceinline__ uint32_t rest_f16(uint32_t h, float lo, float hi) {
  const float2 f = __half22float2(reinterpret_cast<const __half2&>(h));
  return pack_f16(lo - f.x, hi - f.y);
}

// D/4 consecutive elements of a query row as float32; zeros for a missing row.
template <typename T, int E>
__device__ __forceinline__ void load_q(const T* p, bool have, float (&f)[E]) {
  constexpr int V = 16 / (int)sizeof(T);
#pragma unroll
  for (int i = 0; i < E / V; ++i) {
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (have) w = __ldg(reinterpret_cast<const uint4*>(p) + i);
    Vec16<T>::to_float(w, f + i * V);
  }
}

// Two scale bytes (keys a and b, one group) as a float16 pair, zero where a key
// is not used or its scale is NaN (the keys carry the NaN instead).
__device__ __forceinline__ uint32_t value_scales(uint32_t a, uint32_t b, bool use_a, bool use_b) {
  a = use_a && !kv4::scale_is_nan(a) ? a : 0u;
  b = use_b && !kv4::scale_is_nan(b) ? b : 0u;
  return kv4::e4m3x2_to_f16x2(a | (b << 8));
}

template <typename T, int D, int MT>
__global__ void __launch_bounds__(kThreads) attn_mma_kernel(const AttnArgs a) {
  constexpr bool kF32 = sizeof(T) == 4;
  constexpr int KS = D / 16;        // k16 steps of a logit
  constexpr int NT = D / 8;         // n8 tiles of the output
  constexpr int E = D / 4;          // elements of d that a thread holds of a key
  constexpr int CB = D / 2, SB = D / 16;
  constexpr int S = stages<D>();
  constexpr int P = kF32 ? 2 : 1;   // float16 terms of queries and probabilities
  constexpr float kShift = kF32 ? 14.0f : 5.0f;
  constexpr float kSlack = kF32 ? 0.0f : 8.0f;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * warp_bytes<D, MT>();
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kWarps * warp_bytes<D, MT>()) + warp * S;

  int b = blockIdx.x;
  const int split = b % a.n_split;
  b /= a.n_split;
  const int rb = b % a.n_rb;
  const int unit = b / a.n_rb;  // n * Hkv + key head
  const int n = unit / a.Hkv, hk = unit % a.Hkv;

  if (lane == 0) {
    for (int s = 0; s < S; ++s) tc::mbar_init(&full[s], 1);
    tc::fence_barrier_init();
  }
  __syncwarp();
  grid_dep_wait();
  grid_dep_launch();

  const int len = seq_len(a, n);
  const int r_base = rb * 16 * MT;
  const int k_top = block_keys(a, len, r_base, 16 * MT);
  const int k_begin = split * a.chunk;
  const int k_end = min(k_top, k_begin + a.chunk);
  if (a.n_split > 1 && k_begin >= k_end) return;  // the join does not look for it
  const int n_steps = k_begin < k_end ? (k_end - k_begin + kStep - 1) / kStep : 0;
  const int k_pad = (k_end + 15) & ~15;  // rows are copied in sixteens (cap is a multiple)

  const int64_t head = (int64_t)unit * a.cap;
  auto fetch = [&](int step) {  // lane 0: the copies of one of the warp's steps
    const int s = (step / kWarps) % S;
    const int k0 = k_begin + step * kStep;
    const int rows = min(kStep, k_pad - k0);
    uint8_t* dst = ring + s * step_bytes<D>();
    tc::mbar_expect_tx(&full[s], rows * 2 * (CB + SB));
    bulk_load(dst, a.k_codes + (head + k0) * CB, rows * CB, &full[s]);
    bulk_load(dst + kStep * CB, a.v_codes + (head + k0) * CB, rows * CB, &full[s]);
    bulk_load(dst + 2 * kStep * CB, a.k_scales + (head + k0) * SB, rows * SB, &full[s]);
    bulk_load(dst + kStep * (2 * CB + SB), a.v_scales + (head + k0) * SB, rows * SB, &full[s]);
  };
  if (lane == 0)
    for (int i = 0; i < S; ++i)
      if (warp + i * kWarps < n_steps) fetch(warp + i * kWarps);

  // Queries: the fragment of k16 step s holds elements t E + 4 s .. + 3 of rows
  // g and g + 8, times a power of two that brings the row's largest to 2^13.
  uint32_t qa[MT][P][KS][4];
  float fac[MT][2];   // of a logit, to base 2
  int lim[MT][2];     // keys that the row sees
  int lim_min = k_end;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int hrow = 0; hrow < 2; ++hrow) {
      const int r = r_base + m * 16 + hrow * 8 + g;
      const bool have = r < a.R;
      const int i = r / a.G, hq = hk * a.G + r % a.G;
      lim[m][hrow] = have ? min(k_end, row_keys(a, len, i)) : 0;
      lim_min = min(lim_min, have ? lim[m][hrow] : k_end);
      float f[E];
      load_q<T, E>(reinterpret_cast<const T*>(a.q) + n * a.qs.n + hq * a.qs.h + i * a.qs.l + t * E,
                   have, f);
      float top = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) top = fmaxf(top, fabsf(f[e]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      int ex = (int)(__float_as_uint(top) >> 23) - 127;
      ex = top == 0.0f ? 0 : max(-100, min(ex, 127));
      const float down = __uint_as_float((uint32_t)(127 + 13 - ex) << 23);
      fac[m][hrow] = fmaxf(ldexpf(a.scale_log2, ex - 13), 1.2e-38f);  // never 0 * -inf
#pragma unroll
      for (int s = 0; s < KS; ++s) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const float lo = f[4 * s + 2 * w] * down, hi = f[4 * s + 2 * w + 1] * down;
          const uint32_t h = pack_f16(lo, hi);
          qa[m][0][s][2 * w + hrow] = h;
          if constexpr (kF32) qa[m][P - 1][s][2 * w + hrow] = rest_f16(h, lo, hi);
        }
      }
    }
  }
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, o));

  float acc[MT][NT][4];
  float mref[MT][2], lsum[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[m][j][c] = 0.0f;
    mref[m][0] = mref[m][1] = -INFINITY;
    lsum[m][0] = lsum[m][1] = 0.0f;
  }

  bool ok = true;
  for (int step = warp, it = 0; step < n_steps; step += kWarps, ++it) {
    const int s = it % S;
    if (!__all_sync(0xffffffffu, tc::mbar_wait(&full[s], (it / S) & 1))) {
      ok = false;
      for (int j = it; j < it + S && warp + j * kWarps < n_steps; ++j)  // copies under way
        tc::mbar_wait(&full[j % S], (j / S) & 1);
      break;
    }
    const uint8_t* kc = ring + s * step_bytes<D>();
    const uint8_t* vc = kc + kStep * CB;
    const uint8_t* ks = kc + 2 * kStep * CB;
    const uint8_t* vs = ks + kStep * SB;
    const int k0 = k_begin + step * kStep;

    // ---- logits: n8 tile j holds keys 8 j + kappa(column)
    float sc[MT][4][4];
    const int kap = (g & 1) ? 4 + ((g >> 1) ^ 1) : g >> 1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int key = 8 * j + kap;
      uint32_t kw[E / 8];
      uint32_t s0, s1;  // float16 scale pairs of the thread's groups
      if constexpr (D == 128) {
        const uint4 w = *reinterpret_cast<const uint4*>(kc + key * CB + t * 16);
        kw[0] = w.x, kw[1] = w.y, kw[2] = w.z, kw[3] = w.w;
        uint32_t sb = *reinterpret_cast<const uint16_t*>(ks + key * SB + t * 2);
        const uint32_t vb = *reinterpret_cast<const uint16_t*>(vs + key * SB + t * 2);
        if (((vb & 0x7F7Fu) + 0x0101u) & 0x8080u) sb = 0x7F7Fu;
        const uint32_t h = kv4::e4m3x2_to_f16x2(sb);
        s0 = __byte_perm(h, h, 0x1010);
        s1 = __byte_perm(h, h, 0x3232);
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(kc + key * CB + t * 8);
        kw[0] = w.x, kw[1] = w.y;
        uint32_t sb = ks[key * SB + t];
        if (kv4::scale_is_nan(vs[key * SB + t])) sb = 0x7Fu;
        const uint32_t h = kv4::e4m3x2_to_f16x2(sb);
        s0 = s1 = __byte_perm(h, h, 0x1010);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[m][j][c] = 0.0f;
#pragma unroll
      for (int w = 0; w < E / 8; ++w) {
        uint32_t p[4];
        kv4::e2m1x8_to_f16x2(kw[w], p);
        const uint32_t sg = D == 128 && w >= 2 ? s1 : s0;
#pragma unroll
        for (int x = 0; x < 4; ++x) p[x] = hmul2(p[x], sg);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int q = 0; q < P; ++q) {
            mma16816(sc[m][j], qa[m][q][2 * w], p[0], p[1]);
            mma16816(sc[m][j], qa[m][q][2 * w + 1], p[2], p[3]);
          }
      }
    }

    // ---- running maximum and probabilities
    uint32_t pa[MT][P][2][4];  // A fragments of the two k16 steps over keys
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (k0 + kStep > lim_min) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int key = k0 + 8 * j + ((c & 1) ? 4 + (t ^ 1) : t);
            if (key >= lim[m][c >> 1]) sc[m][j][c] = -INFINITY;
          }
      }
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) mx[c >> 1] = fmaxf(mx[c >> 1], sc[m][j][c]);
      bool move = false;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2)) * fac[m][h];
        move |= mx[h] > mref[m][h] + kSlack;
      }
      if (__any_sync(0xffffffffu, move)) {
        float al[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float to = fmaxf(mref[m][h], mx[h]);
          al[h] = to == mref[m][h] ? 1.0f : tc::ex2(mref[m][h] - to);
          mref[m][h] = to;
          lsum[m][h] *= al[h];
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[m][j][c] *= al[c >> 1];
      }
      const float off[2] = {kShift - (mref[m][0] == -INFINITY ? 0.0f : mref[m][0]),
                            kShift - (mref[m][1] == -INFINITY ? 0.0f : mref[m][1])};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float p[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          p[c] = tc::ex2(fmaf(sc[m][j][c], fac[m][c >> 1], off[c >> 1]));
          lsum[m][c >> 1] += p[c];
        }
        const int u = j >> 1, w = (j & 1) * 2;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t x = pack_f16(p[2 * h], p[2 * h + 1]);
          pa[m][0][u][w + h] = x;
          if constexpr (kF32) pa[m][P - 1][u][w + h] = rest_f16(x, p[2 * h], p[2 * h + 1]);
        }
      }
    }

    // ---- values: column g of n8 tile j is element g D/8 + j
    const int left = k_end - k0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      constexpr int W = D / 64;  // words of D/8 codes
      uint32_t w[4][W];
      uint32_t sb[4];
      const int key[4] = {16 * u + t, 16 * u + 4 + (t ^ 1), 16 * u + 8 + t, 16 * u + 12 + (t ^ 1)};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if constexpr (D == 128) {
          const uint2 v = *reinterpret_cast<const uint2*>(vc + key[x] * CB + g * 8);
          w[x][0] = v.x, w[x][W - 1] = v.y;
          sb[x] = vs[key[x] * SB + g];
        } else {
          w[x][0] = *reinterpret_cast<const uint32_t*>(vc + key[x] * CB + g * 4);
          sb[x] = vs[key[x] * SB + (g >> 1)];
        }
      }
      const uint32_t sab = value_scales(sb[0], sb[1], key[0] < left, key[1] < left);
      const uint32_t scd = value_scales(sb[2], sb[3], key[2] < left, key[3] < left);
#pragma unroll
      for (int x = 0; x < W; ++x) {
        uint32_t e0[4], o0[4], e1[4], o1[4];  // even and odd elements of the word
        kv4::e2m1x8_to_f16x2((w[0][x] & 0x0F0F0F0Fu) | ((w[1][x] << 4) & 0xF0F0F0F0u), e0);
        kv4::e2m1x8_to_f16x2(((w[0][x] >> 4) & 0x0F0F0F0Fu) | (w[1][x] & 0xF0F0F0F0u), o0);
        kv4::e2m1x8_to_f16x2((w[2][x] & 0x0F0F0F0Fu) | ((w[3][x] << 4) & 0xF0F0F0F0u), e1);
        kv4::e2m1x8_to_f16x2(((w[2][x] >> 4) & 0x0F0F0F0Fu) | (w[3][x] & 0xF0F0F0F0u), o1);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint32_t be0 = hmul2(e0[y], sab), be1 = hmul2(e1[y], scd);
          const uint32_t bo0 = hmul2(o0[y], sab), bo1 = hmul2(o1[y], scd);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int q = 0; q < P; ++q) {
              mma16816(acc[m][8 * x + 2 * y], pa[m][q][u], be0, be1);
              mma16816(acc[m][8 * x + 2 * y + 1], pa[m][q][u], bo0, bo1);
            }
        }
      }
    }
    __syncwarp();  // every lane has read the stage
    if (lane == 0 && step + S * kWarps < n_steps) fetch(step + S * kWarps);
  }

  // ---- join the warps: each leaves (maximum, sum) and its outputs per row
  if (!ok) atomicExch(a.err, 1);
  float* mine = reinterpret_cast<float*>(ring);
  __syncwarp();
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float l = lsum[m][h];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      const int row = m * 16 + h * 8 + g;
      if (t == 0) {
        mine[row * 2] = mref[m][h];
        mine[row * 2 + 1] = l;
      }
      // thread t holds elements t D/4 .. of the row: columns 2t (first half)
      // and 2t + 1
      float* o = mine + MT * 32 + row * D + t * E;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        o[j] = acc[m][j][2 * h];
        o[NT + j] = acc[m][j][2 * h + 1];
      }
    }
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(smem);
  constexpr int WB = warp_bytes<D, MT>() / 4;
  for (int i = threadIdx.x; i < MT * 16 * (D / 4); i += kThreads) {
    const int row = i / (D / 4), c = (i % (D / 4)) * 4;
    const int r = r_base + row;
    if (r >= a.R) break;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, all[w * WB + row * 2]);
    const float ref = M == -INFINITY ? 0.0f : M;
    float L = 0.0f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = tc::ex2(all[w * WB + row * 2] - ref);
      L += f * all[w * WB + row * 2 + 1];
      const float4 x = *reinterpret_cast<const float4*>(all + w * WB + MT * 32 + row * D + c);
      o.x += f * x.x, o.y += f * x.y, o.z += f * x.z, o.w += f * x.w;
    }
    if (a.n_split == 1) {
      write_row<T>(a, n, hk, r, c, o, M == -INFINITY ? M : M - kShift, L);
    } else {
      const int64_t at = ((int64_t)unit * a.R + r) * a.n_split + split;
      if (c == 0) a.part_ml[at] = make_float2(M == -INFINITY ? M : M - kShift, L);
      *reinterpret_cast<float4*>(a.part_o + at * D + c) = o;
    }
  }
}

// Join the shares of a row: one block per row, its warps over the shares.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) attn_join_kernel(const AttnArgs a) {
  __shared__ float4 part[kWarps][32];
  __shared__ float part_l[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;  // unit * R + r
  const int unit = (int)(row / a.R), r = (int)(row % a.R);
  const int n = unit / a.Hkv, hk = unit % a.Hkv;
  grid_dep_wait();
  grid_dep_launch();
  const int len = seq_len(a, n);
  const int k_top = block_keys(a, len, r / a.rows_blk * a.rows_blk, a.rows_blk);
  const int ns = (k_top + a.chunk - 1) / a.chunk;
  const float2* ml = a.part_ml + row * a.n_split;
  float M = -INFINITY;
  for (int s = lane; s < ns; s += 32) M = fmaxf(M, ml[s].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float ref = M == -INFINITY ? 0.0f : M;
  float L = 0.0f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  const bool col = lane < D / 4;
#pragma unroll 4
  for (int s = warp; s < ns; s += kWarps) {
    const float2 x = ml[s];
    const float f = tc::ex2(x.x - ref);
    L += f * x.y;
    if (col) {
      const float4 v = *reinterpret_cast<const float4*>(a.part_o + (row * a.n_split + s) * D + lane * 4);
      o.x += f * v.x, o.y += f * v.y, o.z += f * v.z, o.w += f * v.w;
    }
  }
  part[warp][lane] = o;
  if (lane == 0) part_l[warp] = L;
  __syncthreads();
  if (warp == 0 && col) {
    L = part_l[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 v = part[w][lane];
      o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
      L += part_l[w];
    }
    write_row<T>(a, n, hk, r, lane * 4, o, M, L);
  }
}

// Shares of the key axis: enough blocks to fill the SMs, at least `least` keys to
// a share.  With as many units as slots, or one short history, there is nothing to
// split and the join is not launched.  n_most bounds n_split and does not fall
// with max_len: the workspace goes by it, so one made for a length serves every
// shorter one.
struct Shares {
  int n_split, chunk;
  int64_t n_most;
};
Shares choose_split(int64_t units, int max_len, int64_t slots, int least, int64_t waves) {
  Shares s = {1, max_len > 0 ? (int)align_up((size_t)max_len, 128) : 128, 1};
  if (max_len <= 2 * least || units >= (waves > 1 ? 4 * slots : slots)) return s;
  // few units: one wave; many: several, so that unlike lengths even out
  const int64_t want = waves == 1 || units * 4 <= slots ? slots / units : ceil_div(waves * slots, units);
  if (want <= 1) return s;
  const int64_t c = ceil_div(max_len, want);
  s.chunk = (int)align_up((size_t)(c < least ? least : c), 128);
  s.n_split = (int)ceil_div(max_len, s.chunk);
  s.n_most = ceil_div(max_len, least);
  if (s.n_most > want) s.n_most = want;
  return s;
}

template <typename T, int D, int MT>
cudaError_t run(AttnArgs a, int N, cudaStream_t s) {
  constexpr int smem = smem_bytes<D, MT>();
  cudaError_t e = cudaFuncSetAttribute(attn_mma_kernel<T, D, MT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (int64_t)N * a.Hkv * a.n_rb * a.n_split;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, attn_mma_kernel<T, D, MT>, a);
  if (e != cudaSuccess) return e;
  add_launches(1);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t join(const AttnArgs& a, int N, cudaStream_t s) {
  const int64_t rows = (int64_t)N * a.Hkv * a.R;
  if (rows > 0x7fffffffll) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, attn_join_kernel<T, D>, a);
  if (e != cudaSuccess) return e;
  add_launches(1);
  return cudaGetLastError();
}

// The tensor-core kernel takes over where its 256-row blocks are worth filling.
bool use_tc(bool bf16, int R) { return bf16 && R > 64; }

struct Layout {
  int rows_blk, n_rb, n_split, chunk;
  size_t ml, o, total;
};
Layout layout(bool bf16, int N, int Hq, int Hkv, int Lq, int max_len, int d) {
  Layout l;
  const int R = Hq / Hkv * Lq;
  const bool tc = use_tc(bf16, R);
  l.rows_blk = tc ? kTcRows : bf16 && R > 16 ? 32 : 16;
  l.n_rb = (int)ceil_div(R, l.rows_blk);
  const int64_t units = (int64_t)N * Hkv * l.n_rb;
  const Shares sh = tc ? choose_split(units, max_len, sm_count(), 512, 1)
                       : choose_split(units, max_len, 3ll * sm_count(), 256, 3);
  l.n_split = sh.n_split;
  l.chunk = sh.chunk;
  const size_t parts = sh.n_most > 1 ? (size_t)N * Hkv * R * sh.n_most : 0;
  l.ml = 256;
  l.o = align_up(l.ml + parts * sizeof(float2), 256);
  l.total = align_up(l.o + parts * d * sizeof(float), 256);
  return l;
}

template <int D>
cudaError_t run_all(const AttnArgs& a, bool bf16, int N, cudaStream_t s) {
  cudaError_t e;
  if (!bf16)
    e = run<float, D, 1>(a, N, s);
  else if (a.rows_blk == kTcRows)
    e = launch_attn_tc(a, N, D, s);
  else if (a.rows_blk == 16)
    e = run<__nv_bfloat16, D, 1>(a, N, s);
  else
    e = run<__nv_bfloat16, D, 2>(a, N, s);
  if (e != cudaSuccess || a.n_split == 1) return e;
  return bf16 ? join<__nv_bfloat16, D>(a, N, s) : join<float, D>(a, N, s);
}
}  // namespace

size_t kv4_attention_ws_bytes(bool bf16, int N, int Hq, int Hkv, int Lq, int max_len, int d) {
  return layout(bf16, N, Hq, Hkv, Lq, max_len, d).total;
}

cudaError_t launch_kv4_attention(const Kv4Attn& p, const fc_kv4_cache& c, void* ws,
                                 cudaStream_t s) {
  AttnArgs a = {};
  a.q = p.q;
  a.out = p.out;
  a.lse = p.lse;
  a.lens = p.lens;
  a.qs = p.qs;
  a.os = p.os;
  a.k_codes = static_cast<const uint8_t*>(c.k_codes);
  a.k_scales = static_cast<const uint8_t*>(c.k_scales);
  a.v_codes = static_cast<const uint8_t*>(c.v_codes);
  a.v_scales = static_cast<const uint8_t*>(c.v_scales);
  a.Hkv = c.H;
  a.G = p.Hq / c.H;
  a.R = a.G * p.Lq;
  a.Lq = p.Lq;
  a.max_len = p.max_len;
  a.cap = c.cap;
  a.causal = p.causal;
  a.scale_log2 = ldexpf(p.scale * 1.4426950408889634f, c.k_exp);
  a.out_scale = ldexpf(1.0f, c.v_exp);
  const Layout l = layout(p.bf16, c.N, p.Hq, c.H, p.Lq, p.max_len, c.d);
  a.rows_blk = l.rows_blk;
  a.n_rb = l.n_rb;
  a.n_split = l.n_split;
  a.chunk = l.chunk;
  char* w = static_cast<char*>(ws);
  a.err = reinterpret_cast<int*>(w);
  a.part_ml = reinterpret_cast<float2*>(w + l.ml);
  a.part_o = reinterpret_cast<float*>(w + l.o);
  return c.d == 128 ? run_all<128>(a, p.bf16, c.N, s) : run_all<64>(a, p.bf16, c.N, s);
}

}  // namespace fc
