// Attention over the 4-bit cache for few query rows per key head (decoding), and
// for float32 queries.
//
//   out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j)
//
// The R = (Hq/Hkv) Lq query rows of a key head read the same keys, so they share
// one pass over them: row r is query r / G of head r % G in the group.  The
// bound is HBM: a key and its value are 144 bytes at d = 128 (72 at 64) for 4 R d
// flops.  What has to keep up with it is the conversion of the codes, so
//   - keys and values are the A operand of mma.m16n8k16 and the rows its columns: up
//     to 8 rows cost one n8 tile (as A operand, 16 whatever there are: twice the
//     MMA, exponentials and accumulators; 110 -> 83 us for 32 sequences of up to
//     16384 keys);
//   - the codes go from shared memory straight into fragments and are never written
//     back as float16: a thread reads 32 consecutive codes of a key (16 bytes), and
//     the order in which the MMA steps see the elements of d is whatever that makes
//     it, since the queries are stored in the same order.  Values need pairs of keys
//     instead of pairs of elements: two shift-and-select instructions interleave the
//     nibbles of two keys' words before the conversion;
//   - code * scale is exact in float16 (at most 6 significant bits), so one
//     packed multiplication per pair finishes the conversion;
//   - probabilities come out with keys on the rows and are wanted with keys on the K
//     axis: one 8 x 8 transposition (movmatrix) for eight keys;
//   - blocks of 8 warps take equal shares of all sequences' keys (StreamShare), in
//     stages of 128 keys that bulk copies bring, four warps to a stage with 32 keys
//     each and two stages at a time; a warp has its own running maximum, sum and
//     output, so there is no barrier in the loop.  The logits of the next stage are
//     computed beside the values of this one (81 -> 78 us).  The warps are joined at
//     the end of a unit, and units that blocks share by a second, small kernel.
// Per 32 keys a warp issues about 520 instructions, 128 of them conversions and 128
// multiplications, at 16 warps an SM (120 registers; 24 warps of 80 spill and take
// 92 us for 76).  No unit is full: with four warps to a scheduler it issues in half of
// the cycles, and of the 7.4 cycles from one instruction of a warp to its next 1.1 go to
// other warps, 1.0 each to the latency of arithmetic, to full math pipes and to fetching
// instructions, 0.7 to the block's barriers between units and 0.5 to dispatch (loads
// are hardly among them).  72 to 78 us for 312 MB, over several GPUs (61 to 66 % of
// the measured copy rate), 36 to 38 us for one sequence of 131072 keys and 8 key heads
// (62 %); the same without any arithmetic takes 55 and 28.  16 rows to a key head (two
// n8 tiles, 128 registers with some spilled): 63 us for 151 MB, which 8 rows take 40 for.
// The running maximum only moves when a step exceeds it by 2^8 (float16
// probabilities, offset by 2^5, keep 11 bits over that range); for float32
// queries it is exact, and queries and probabilities are sums of two float16
// (22 bits and the sign of the second).  8 sequences of 8 heads and 8192 keys, float32,
// take 31 us for 75 MB, 8 heads x 256 queries x 4096 keys 42.
#include <cuda.h>

#include "fc_common.cuh"
#include "fc_kernels.h"
#include "kv4.cuh"
#include "kv4_attn.cuh"
#include "kv4_ring.cuh"
#include "tc_ptx.cuh"

namespace fc {

namespace {
constexpr int kStep = kRingKeys;    // keys of a warp's step
constexpr int kU = kStep / 16;      // m16 tiles of a step
constexpr int kGroup = kRingWarps;  // warps that work on one stage
constexpr int kGroups = kRingGroups;
constexpr int kWarps = kGroups * kGroup;
constexpr int kThreads = 32 * kWarps;
constexpr int kStage = kGroup * kStep;
static_assert(kStage == kStageKeys, "stages are the unit of the shares");
constexpr int kJoinWarps = 8;
constexpr int kLeastStages = 2;  // of a block's share

template <int D> constexpr int stage_bytes() { return kStage * (D + D / 8); }
template <int D> constexpr int stages() { return ring_slots(D); }
// Outputs of a row at the end, with two numbers beside them and an odd stride.
template <int D, int NR> constexpr int warp_result_bytes() { return NR * 8 * (D + 4) * 4; }
template <int D, int NR> constexpr int ring_bytes() {
  const int ring = stages<D>() * stage_bytes<D>(), join = kWarps * warp_result_bytes<D, NR>();
  return ring > join ? ring : join;
}
template <int D, int NR> constexpr int smem_bytes() {
  return ring_bytes<D, NR>() + 2 * stages<D>() * 8;
}

// c = a b (+ c): m16n8k16, float16 operands, float32 sums.
__device__ __forceinline__ void mma_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_add(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit numbers (thread 4 r + c / 2 holds row r, columns c, c + 1)
// transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t both_low(uint32_t x) {
  const __half2 r = __low2half2(reinterpret_cast<const __half2&>(x));
  return reinterpret_cast<const uint32_t&>(r);
}
__device__ __forceinline__ uint32_t both_high(uint32_t x) {
  const __half2 r = __high2half2(reinterpret_cast<const __half2&>(x));
  return reinterpret_cast<const uint32_t&>(r);
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
    if (have) w = reinterpret_cast<const uint4*>(p)[i];
    Vec16<T>::to_float(w, f + i * V);
  }
}

// Bit 7 of each byte of the result: that byte of e4m3 is NaN.
__device__ __forceinline__ uint32_t nan_bits(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// NR: tiles of 8 query rows.
template <typename T, int D, int NR>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 || NR == 1 ? 2 : 1)
    attn_mma_kernel(const AttnArgs a) {
  constexpr bool kF32 = sizeof(T) == 4;
  constexpr int KS = D / 16;        // k16 steps of a logit
  constexpr int MT = D / 16;        // m16 tiles of the output
  constexpr int E = D / 4;          // elements of d that a thread holds of a key
  constexpr int CB = D / 2, SB = D / 16;
  constexpr int S = stages<D>();
  constexpr int P = kF32 ? 2 : 1;   // float16 terms of queries and probabilities
  constexpr float kShift = kF32 ? 14.0f : 5.0f;
  constexpr float kSlack = kF32 ? 0.0f : 8.0f;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + ring_bytes<D, NR>());
  uint64_t* empty = full + S;

  __shared__ StreamShare<kThreads> share;
  __shared__ Piece piece;
  __shared__ struct {
    uint4 q[NR][P][KS / 2][32];
    float fac[NR * 8];
    int lim[NR * 8];
  } qs;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      tc::mbar_init(&full[s], s == a.stuck_slot ? 2 : 1);
      tc::mbar_init(&empty[s], kGroup);
    }
    tc::fence_barrier_init();
  }
  grid_dep_wait();
  if (a.stream) grid_dep_launch();  // the join

  // The block's share: one unit, or a run of stages over units.
  if (a.stream) share.begin(a, kLeastStages);
  bool ok = true;
  int base = 0;  // stages of the units before: slots and phases go on
  for (;;) {
  if (threadIdx.x == 0) {
    if (!a.stream)
      whole_unit(a, piece);
    else if (!share.next(a, share.first, piece))
      piece.n_unit = -1;
  }
  __syncthreads();
  if (piece.n_unit < 0) return;
  const int len = seq_len(a, piece.n);
  const int r_base = piece.rb * 8 * NR;
  const int k_begin = piece.s_begin * kStage;
  const int k_end = min(block_keys(a, len, r_base, 8 * NR), piece.s_end * kStage);
  const int n_stages = piece.s_end - piece.s_begin;
  const int k_pad = (k_end + 15) & ~15;  // rows are copied in sixteens (cap is a multiple)

  const int64_t head = (int64_t)(piece.n * a.Hkv + piece.hk) * a.cap;
  auto fetch = [&](int i, int s) {  // one thread: the copies of stage i into slot s
    const int k0 = k_begin + i * kStage;
    const int rows = min(kStage, k_pad - k0);
    uint8_t* dst = smem + s * stage_bytes<D>();
    tc::mbar_expect_tx(&full[s], rows * 2 * (CB + SB));
    bulk_load(dst, a.k_codes + (head + k0) * CB, rows * CB, &full[s]);
    bulk_load(dst + kStage * CB, a.v_codes + (head + k0) * CB, rows * CB, &full[s]);
    bulk_load(dst + 2 * kStage * CB, a.k_scales + (head + k0) * SB, rows * SB, &full[s]);
    bulk_load(dst + kStage * (2 * CB + SB), a.v_scales + (head + k0) * SB, rows * SB, &full[s]);
  };
  if (threadIdx.x == 0) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // behind the last unit's join
    for (int i = 0; i < S && i < n_stages; ++i) fetch(i, (base + i) % S);
    if (a.stream && piece.s_begin == 0)
      a.part_of[(int64_t)(piece.n * a.Hkv + piece.hk) * a.n_rb + piece.rb] =
          make_int2(blockIdx.x, piece.n_parts);
  }

  // Queries are the B operand: in k16 step s thread (g, t) holds elements
  // t E + 4 s .. + 3 of row g, times a power of two that brings the row's largest
  // to 2^13.  Logits come out with the rows on the columns, 2 t and 2 t + 1.  One warp
  // to eight rows converts them for all; they are read from shared memory at every
  // step, since the 16 registers that they would take cost more.
  if (warp >= 1 && warp <= NR) {
    const int m = warp - 1;
    const int r = r_base + m * 8 + g;
    const bool have = r < a.R;
    const int i = r / a.G, hq = piece.hk * a.G + r % a.G;
    float f[E];
    load_q<T, E>(reinterpret_cast<const T*>(a.q) + piece.n * a.qs.n + hq * a.qs.h + i * a.qs.l + t * E,
                 have, f);
    float top = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) top = fmaxf(top, fabsf(f[e]));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    int ex = (int)(__float_as_uint(top) >> 23) - 127;
    ex = top == 0.0f ? 0 : max(-100, min(ex, 127));
    const float down = __uint_as_float((uint32_t)(127 + 13 - ex) << 23);
    if (t == 0) {
      qs.fac[m * 8 + g] = fmaxf(ldexpf(a.scale_log2, ex - 13), 1.2e-38f);  // never 0 * -inf
      qs.lim[m * 8 + g] = have ? min(k_end, row_keys(a, len, i)) : k_end;
    }
#pragma unroll
    for (int w = 0; w < KS / 2; ++w) {
      uint32_t q[4], rest[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float lo = f[8 * w + 2 * x] * down, hi = f[8 * w + 2 * x + 1] * down;
        q[x] = pack_f16(lo, hi);
        if constexpr (kF32) rest[x] = rest_f16(q[x], lo, hi);
      }
      qs.q[m][0][w][lane] = make_uint4(q[0], q[1], q[2], q[3]);
      if constexpr (kF32) qs.q[m][P - 1][w][lane] = make_uint4(rest[0], rest[1], rest[2], rest[3]);
    }
  }

  float acc[NR][MT][4];  // (element g or g + 8 of the m16 tile, row 2 t or 2 t + 1)
  float mref[NR][2], lsum[NR][2];
#pragma unroll
  for (int m = 0; m < NR; ++m) {
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[m][j][c] = 0.0f;
    mref[m][0] = mref[m][1] = -INFINITY;
    lsum[m][0] = lsum[m][1] = 0.0f;
  }
  __syncthreads();  // the barriers and the queries are there
  float fac[NR][2];  // of a logit, to base 2
  int lim[NR][2];    // keys that the row sees
  int lim_min = k_end;
#pragma unroll
  for (int m = 0; m < NR; ++m) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      fac[m][c] = qs.fac[m * 8 + 2 * t + c];
      lim[m][c] = qs.lim[m * 8 + 2 * t + c];
    }
    lim_min = min(lim_min, qs.lim[m * 8 + g]);
  }
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, o));

  // Row g of the 8 keys j is key 8 j + kap: with this order neither the loads of
  // keys nor those of values (four rows at once) meet a bank twice.
  const int kap = (g & 1) ? 4 + ((g >> 1) ^ 1) : g >> 1;
  const int w_off = (warp % kGroup) * kStep;  // the warp's keys of a stage

  // Logits of the warp's keys of stage i: m16 tile u holds keys 16 u + kap (rows g)
  // and 16 u + 8 + kap.
  float sc[NR][kU][4];
  auto logits = [&](int s) {
    const uint8_t* st = smem + s * stage_bytes<D>();
    const uint8_t* kc = st + (w_off + kap) * CB + t * (CB / 4);
    const uint8_t* ks = st + 2 * kStage * CB + (w_off + kap) * SB + t * (SB / 4);
    uint32_t kw[2 * kU][E / 8];
    uint32_t s0[2 * kU], s1[2 * kU];  // float16 scale pairs of the thread's groups
#pragma unroll
    for (int h = 0; h < 2 * kU; ++h) {
      if constexpr (D == 128) {
        const uint4 w = *reinterpret_cast<const uint4*>(kc + 8 * h * CB);
        kw[h][0] = w.x, kw[h][1] = w.y, kw[h][2] = w.z, kw[h][3] = w.w;
        const uint32_t x =
            kv4::e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(ks + 8 * h * SB));
        s0[h] = both_low(x);
        s1[h] = both_high(x);
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(kc + 8 * h * CB);
        kw[h][0] = w.x, kw[h][1] = w.y;
        const uint32_t x = kv4::e4m3x2_to_f16x2(ks[8 * h * SB]);
        s0[h] = s1[h] = both_low(x);
      }
    }
#pragma unroll
    for (int w = 0; w < E / 8; ++w) {
      uint4 qw[NR][P];
#pragma unroll
      for (int m = 0; m < NR; ++m)
#pragma unroll
        for (int q = 0; q < P; ++q) qw[m][q] = qs.q[m][q][w][lane];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        uint32_t p[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          kv4::e2m1x8_to_f16x2(kw[2 * u + h][w], p[h]);
#pragma unroll
          for (int x = 0; x < 4; ++x)
            p[h][x] = hmul2(p[h][x], D == 128 && w >= 2 ? s1[2 * u + h] : s0[2 * u + h]);
        }
        const uint32_t a0[4] = {p[0][0], p[1][0], p[0][1], p[1][1]};
        const uint32_t a1[4] = {p[0][2], p[1][2], p[0][3], p[1][3]};
#pragma unroll
        for (int m = 0; m < NR; ++m)
#pragma unroll
          for (int q = 0; q < P; ++q) {
            if (w == 0 && q == 0)
              mma_first(sc[m][u], a0, qw[m][q].x, qw[m][q].y);
            else
              mma_add(sc[m][u], a0, qw[m][q].x, qw[m][q].y);
            mma_add(sc[m][u], a1, qw[m][q].z, qw[m][q].w);
          }
      }
    }
  };

  // Probabilities of stage i from its logits, and the scales of its values: byte x
  // of vsc[u] is key 16 u + 4 x + (t, t^1, t, t^1), the group of the thread's
  // elements.
  uint32_t pb[NR][P][kU][2];  // B fragments of the k16 steps over keys
  uint32_t vsc[kU];
  auto softmax = [&](int i, int s) {
    const int k0 = k_begin + i * kStage + w_off;
    const uint8_t* vs = smem + s * stage_bytes<D>() + kStage * (2 * CB + SB) + w_off * SB +
                        (D == 128 ? g : g >> 1);
    const uint8_t *p0 = vs + t * SB, *p1 = vs + (4 + (t ^ 1)) * SB;
    uint32_t odd = 0;  // something to look after: NaN scales, a row to rescale
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      vsc[u] = p0[16 * u * SB] + 0x100u * p1[16 * u * SB] + 0x10000u * p0[(16 * u + 8) * SB] +
               0x1000000u * p1[(16 * u + 8) * SB];
      odd |= nan_bits(vsc[u]);
    }
    if (k0 + kStep > lim_min) {  // keys that a row does not see, rows behind the last key
#pragma unroll
      for (int u = 0; u < kU; ++u) {
#pragma unroll
        for (int m = 0; m < NR; ++m)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (k0 + 16 * u + 8 * (c >> 1) + kap >= lim[m][c & 1]) sc[m][u][c] = -INFINITY;
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (k0 + 16 * u + 4 * x + ((x & 1) ? t ^ 1 : t) >= k_end) vsc[u] &= ~(0xFFu << (8 * x));
      }
    }
    float mx[NR][2];  // of the thread's own keys
#pragma unroll
    for (int m = 0; m < NR; ++m)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        mx[m][c] = fmaxf(sc[m][0][c], sc[m][0][2 + c]);
#pragma unroll
        for (int u = 1; u < kU; ++u) mx[m][c] = tc::fmax3(mx[m][c], sc[m][u][c], sc[m][u][2 + c]);
        odd |= mx[m][c] * fac[m][c] > mref[m][c] + kSlack ? 1u : 0u;
      }
    if (__any_sync(0xffffffffu, odd != 0)) {
      uint32_t nans = 0;
#pragma unroll
      for (int u = 0; u < kU; ++u) nans |= nan_bits(vsc[u]);
      if (__any_sync(0xffffffffu, nans != 0)) {
        // a NaN among a key's values goes with its logits, and reads as zero
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          // the lanes of one t hold the groups of four keys
          uint32_t bad = nan_bits(vsc[u]);
          vsc[u] &= ~((bad >> 7) * 0xFFu);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) bad |= __shfl_xor_sync(0xffffffffu, bad, o);
          // the thread's own keys, 16 u + kap and + 8: bytes of lane g / 2
          bad = __shfl_sync(0xffffffffu, bad, g >> 1) >> ((g & 1) ? 8 : 0);
#pragma unroll
          for (int m = 0; m < NR; ++m) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (bad & (c < 2 ? 0x80u : 0x800000u) &&
                  k0 + 16 * u + 8 * (c >> 1) + kap < lim[m][c & 1])
                sc[m][u][c] = __int_as_float(0x7fffffff);
          }
        }
      }
      // the row's largest, and everything of the row so far relative to it
#pragma unroll
      for (int m = 0; m < NR; ++m) {
        float al[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float top = mx[m][c];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          top *= fac[m][c];
          const float to = top > mref[m][c] + kSlack ? top : mref[m][c];
          al[c] = to == mref[m][c] ? 1.0f : tc::ex2(mref[m][c] - to);
          mref[m][c] = to;
          lsum[m][c] *= al[c];
        }
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[m][j][c] *= al[c & 1];
      }
    }
#pragma unroll
    for (int m = 0; m < NR; ++m) {
      const float off[2] = {kShift - (mref[m][0] == -INFINITY ? 0.0f : mref[m][0]),
                            kShift - (mref[m][1] == -INFINITY ? 0.0f : mref[m][1])};
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float p[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            p[c] = tc::ex2(fmaf(sc[m][u][2 * h + c], fac[m][c], off[c]));
            lsum[m][c] += p[c];
          }
          // (keys on the lanes' rows, query rows on the columns) to the B operand
          const uint32_t x = pack_f16(p[0], p[1]);
          pb[m][0][u][h] = transpose8x8(x);
          if constexpr (kF32) pb[m][P - 1][u][h] = transpose8x8(rest_f16(x, p[0], p[1]));
        }
    }
  };

  // Values of stage i are the A operand: rows g and g + 8 of m16 tile j are elements
  // g D/8 + 2 j and + 2 j + 1.
  auto values = [&](int s) {
    const uint8_t* vc = smem + s * stage_bytes<D>() + kStage * CB + w_off * CB + g * (CB / 8);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      constexpr int VW = D / 64;  // words of D/8 codes
      uint32_t w[4][VW];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint8_t* at = vc + (16 * u + 4 * x + ((x & 1) ? t ^ 1 : t)) * CB;
        if constexpr (D == 128) {
          const uint2 v = *reinterpret_cast<const uint2*>(at);
          w[x][0] = v.x, w[x][VW - 1] = v.y;
        } else {
          w[x][0] = *reinterpret_cast<const uint32_t*>(at);
        }
      }
      const uint32_t sab = kv4::e4m3x2_to_f16x2(vsc[u]), scd = kv4::e4m3x2_to_f16x2(vsc[u] >> 16);
#pragma unroll
      for (int x = 0; x < VW; ++x) {
        uint32_t e0[4], o0[4], e1[4], o1[4];  // even and odd elements of the word
        kv4::e2m1x8_to_f16x2((w[0][x] & 0x0F0F0F0Fu) | ((w[1][x] << 4) & 0xF0F0F0F0u), e0);
        kv4::e2m1x8_to_f16x2(((w[0][x] >> 4) & 0x0F0F0F0Fu) | (w[1][x] & 0xF0F0F0F0u), o0);
        kv4::e2m1x8_to_f16x2((w[2][x] & 0x0F0F0F0Fu) | ((w[3][x] << 4) & 0xF0F0F0F0u), e1);
        kv4::e2m1x8_to_f16x2(((w[2][x] >> 4) & 0x0F0F0F0Fu) | (w[3][x] & 0xF0F0F0F0u), o1);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint32_t av[4] = {hmul2(e0[y], sab), hmul2(o0[y], sab), hmul2(e1[y], scd),
                                  hmul2(o1[y], scd)};
#pragma unroll
          for (int m = 0; m < NR; ++m) {
            if constexpr (kF32) {
              // The tensor cores cut what they add to (2^-23 of it, always downwards: 2e-6
              // of a result over 40000 keys), so 16 keys are added by themselves and
              // their sum to nearest.
              float part[4];
              mma_first(part, av, pb[m][P - 1][u][0], pb[m][P - 1][u][1]);
              mma_add(part, av, pb[m][0][u][0], pb[m][0][u][1]);
#pragma unroll
              for (int c = 0; c < 4; ++c) acc[m][4 * x + y][c] += part[c];
            } else {
              mma_add(acc[m][4 * x + y], av, pb[m][0][u][0], pb[m][0][u][1]);
            }
          }
        }
      }
    }
  };
  auto arrived = [&](int i, int s, uint32_t parity) {
    const bool in = __all_sync(0xffffffffu, tc::mbar_wait(&full[s], parity, a.wait_cycles));
    if (!in) {
      ok = false;
      for (int x = base + i; x < base + min(i + S, n_stages); ++x)  // copies under way
        tc::mbar_wait(&full[x % S], (x / S) & 1, tc::kDrainCycles);
    }
    return in;
  };
  auto release = [&](int s) {
    __syncwarp();  // every lane has read the stage
    if (lane == 0) tc::mbar_arrive(&empty[s]);
  };
  auto refill = [&](int i, int s, uint32_t parity) {
    if (lane == 0 && ring_refills<S>(i, warp % kGroup, n_stages)) {
      if (tc::mbar_wait(&empty[s], parity, a.wait_cycles))
        fetch(i + S, s);
      else
        ok = false;
    }
  };

  // Slots stay with their group of warps.  The waits of refill() are one lane's, so the
  // lanes agree on whether a wait has given up before they go on together.
  ring_walk<S>(base, (warp / kGroup + base) % kGroups,
               ring_own_stages(k_end - k_begin, warp % kGroup), n_stages, arrived, logits, softmax,
               values, release, refill, [&] { return __all_sync(0xffffffffu, ok) != 0; });
  if (!ok) atomicExch(a.err, 1);
  __syncthreads();

  // ---- join the warps: each leaves (maximum, sum) and its outputs per row
  constexpr int RS = D + 4;  // floats of a row: D outputs, maximum, sum
  float* mine = reinterpret_cast<float*>(smem + warp * warp_result_bytes<D, NR>());
#pragma unroll
  for (int m = 0; m < NR; ++m)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float l = lsum[m][c];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      float* row = mine + (m * 8 + 2 * t + c) * RS;
      if (g == 0) {
        row[D] = mref[m][c];
        row[D + 1] = l;
      }
#pragma unroll
      for (int j = 0; j < MT; ++j)
        *reinterpret_cast<float2*>(row + g * (D / 8) + 2 * j) =
            make_float2(acc[m][j][c], acc[m][j][2 + c]);
    }
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(smem);
  constexpr int WB = warp_result_bytes<D, NR>() / 4;
  for (int i = threadIdx.x; i < NR * 8 * (D / 4); i += kThreads) {
    const int row = i / (D / 4), c = (i % (D / 4)) * 4;
    const int r = r_base + row;
    if (r >= a.R) break;
    const float* at_row = all + row * RS;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, at_row[w * WB + D]);
    const float ref = M == -INFINITY ? 0.0f : M;
    float L = 0.0f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = tc::ex2(at_row[w * WB + D] - ref);
      L += f * at_row[w * WB + D + 1];
      const float4 x = *reinterpret_cast<const float4*>(at_row + w * WB + c);
      o.x += f * x.x, o.y += f * x.y, o.z += f * x.z, o.w += f * x.w;
    }
    if (n_stages == piece.n_unit) {
      write_row<T>(a, piece.n, piece.hk, r, c, o, M == -INFINITY ? M : M - kShift, L);
    } else {
      const int64_t at = ((int64_t)blockIdx.x * 2 + (piece.s_begin == 0 ? 1 : 0)) * (8 * NR) + row;
      if (c == 0) a.part_ml[at] = make_float2(M == -INFINITY ? M : M - kShift, L);
      *reinterpret_cast<float4*>(a.part_o + at * D + c) = o;
    }
  }
  if (!a.stream) return;
  base += n_stages;
  if (__syncthreads_or(!ok)) return;  // the results have been read: the stages are free
  }
}

// Join the parts of a row.  What this costs is latency, so everything that does not
// wait for the parts comes before the wait for them, and a warp's first loads do not
// wait for the reference.  A row of few parts takes one warp (kRowWarps = 1, eight
// rows to a block), one of many takes a block's eight: with a block to each of 1280
// rows of three parts the whole call takes 80.1 us, with a warp 77.3.
template <typename T, int D, int kRowWarps>
__global__ void __launch_bounds__(32 * kJoinWarps) attn_join_kernel(const AttnArgs a) {
  constexpr int kAhead = 5;
  __shared__ float4 part[kJoinWarps][32];
  __shared__ float part_l[kJoinWarps];
  const int lane = threadIdx.x & 31;
  const int warp = kRowWarps == 1 ? 0 : threadIdx.x >> 5;
  // rows of the units that blocks share
  const int64_t i = kRowWarps == 1 ? (int64_t)blockIdx.x * kJoinWarps + (threadIdx.x >> 5) : blockIdx.x;
  const int64_t at_unit = i / a.rows_blk;
  if (a.n_whole + at_unit >= (int64_t)a.N * a.Hkv * a.n_rb) return;
  int n, hk, rb;
  unit_at(a, a.n_whole + at_unit, n, hk, rb);
  const int in_blk = (int)(i - at_unit * a.rows_blk), r = rb * a.rows_blk + in_blk;
  if (r >= a.R) return;
  // Lengths are older than the kernel that this one depends on, which waited for
  // them itself before it let this one start.
  const bool some = entry_stages(a, n * a.n_rb + rb) > 0;
  const bool col = lane < D / 4;
  grid_dep_wait();
  // (a share of equal work has no block for a unit without keys)
  int2 of = make_int2(0, 0);
  if (some || !a.stream) of = a.part_of[(int64_t)(n * a.Hkv + hk) * a.n_rb + rb];
  // What a block that gave up a wait did not write is whatever the workspace held: no
  // parts then (the error word is set), and no access by it.
  const int leaving = a.blocks - a.n_whole;  // blocks that leave parts
  if (of.x < 0 || of.x >= leaving || of.y < 1 || of.y > leaving - of.x) of = make_int2(0, 0);
  if (of.y == 1) return;  // one block had it all
  const int ns = of.y;
  // of equal shares: slot 1 of the first block, slot 0 of the others
  const int64_t at0 = (a.stream ? (int64_t)of.x * 2 + 1 : of.x) * a.rows_blk + in_blk;
  const float2* ml = a.part_ml + at0;
  const float4* po = reinterpret_cast<const float4*>(a.part_o + at0 * D) + lane;
  auto place = [&](int s) { return (int64_t)(a.stream && s > 0 ? 2 * s - 1 : s) * a.rows_blk; };
  float2 x[kAhead];
  float4 v[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int s = warp + k * kRowWarps;
    x[k] = s < ns ? ml[place(s)] : make_float2(-INFINITY, 0.0f);
    v[k] = s < ns && col ? po[place(s) * (D / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float M = -INFINITY;
  for (int s = lane; s < ns; s += 32) M = fmaxf(M, ml[place(s)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float ref = M == -INFINITY ? 0.0f : M;
  float L = 0.0f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float2 xs, float4 vs) {
    const float f = tc::ex2(xs.x - ref);
    L += f * xs.y;
    o.x += f * vs.x, o.y += f * vs.y, o.z += f * vs.z, o.w += f * vs.w;
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (warp + k * kRowWarps < ns) add(x[k], v[k]);
#pragma unroll 4
  for (int s = warp + kAhead * kRowWarps; s < ns; s += kRowWarps)
    add(ml[place(s)], col ? po[place(s) * (D / 4)] : make_float4(0.f, 0.f, 0.f, 0.f));
  if constexpr (kRowWarps > 1) {
    part[warp][lane] = o;
    if (lane == 0) part_l[warp] = L;
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int w = 1; w < kRowWarps; ++w) {
      const float4 y = part[w][lane];
      o.x += y.x, o.y += y.y, o.z += y.z, o.w += y.w;
      L += part_l[w];
    }
  }
  if (col) write_row<T>(a, n, hk, r, lane * 4, o, M, L);
}

template <typename T, int D, int NR>
cudaError_t run(const AttnArgs& a, int N, cudaStream_t s) {
  constexpr int smem = smem_bytes<D, NR>();
  cudaError_t e = cudaFuncSetAttribute(attn_mma_kernel<T, D, NR>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, attn_mma_kernel<T, D, NR>, a);
  if (e != cudaSuccess) return e;
  add_launches(1);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t join(const AttnArgs& a, int N, cudaStream_t s) {
  const int64_t units = (int64_t)N * a.Hkv * a.n_rb, rows = (units - a.n_whole) * a.rows_blk;
  const int64_t parts = a.stream ? a.blocks / units + 2 : a.n_split;  // of a row, about
  const bool one = parts <= 5;
  const int64_t blocks = one ? ceil_div(rows, kJoinWarps) : rows;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = one ? cudaLaunchKernelEx(&cfg, attn_join_kernel<T, D, 1>, a)
                            : cudaLaunchKernelEx(&cfg, attn_join_kernel<T, D, kJoinWarps>, a);
  if (e != cudaSuccess) return e;
  add_launches(1);
  return cudaGetLastError();
}

// The tcgen05 kernel computes 128 rows whatever there are, this one reads the keys
// once more for every 16.  Measured at 128 key heads x 8192 keys: d = 128, 32 rows
// 106 us here and 134 there, 48 rows 152 and 136; d = 64, 24 rows 59 and 112, and
// 24 heads x 1000 keys with 64 rows 15 and 21.  (The bytes alone take 23 and 11.5 us:
// between 9 and 64 rows both kernels are four to six times from them, this one for
// converting every key again, the other for computing rows that there are not.)
bool use_tc(bool bf16, int R, int d) { return bf16 && R > (d == 128 ? 32 : 64); }

struct Layout {
  int rows_blk, n_rb, blocks, n_whole, n_split, chunk;
  bool stream;
  size_t of, ml, o, total;
};
// causal, unlike: only for the choice of parts (the workspace does not go by them).
bool layout(bool bf16, bool causal, bool unlike, int N, int Hq, int Hkv, int Lq, int max_len, int d, Layout& l) {
  const int R = Hq / Hkv * Lq;
  const bool tc = use_tc(bf16, R, d);
  l.rows_blk = tc ? kTcRows : R > 8 ? 16 : 8;
  l.n_rb = (int)ceil_div(R, l.rows_blk);
  const int64_t units = (int64_t)N * Hkv * l.n_rb, sms = sm_count();
  l.stream = false;
  l.n_split = l.chunk = 1;
  int64_t blocks = units, n_whole = units, parts = 0;
  if (tc) {
    // One block to an SM.  Whole waves of units have a block each; those of the last
    // wave are split along the keys into s parts, with s such that the parts' own
    // waves take least, counted in key tiles: a part costs about 4 beside its own, the
    // join 6, and a causal unit has half of the longest's on average.  At most three
    // waves of parts, of 512 keys or more.  (384 units of 160 tiles: 1108 us without,
    // 1047 with; 192 causal units of up to 16: 41 without, 48 with.)
    const int64_t rem = units % sms;
    const int64_t tiles = ceil_div(max_len, kTcKeys);
    int64_t most = rem > 0 ? 3 * sms / rem : 1;
    if (most > max_len / 512) most = max_len / 512;
    int64_t best = INT64_MAX, s = 1;
    for (int64_t x = 1; x <= most || x == 1; ++x) {
      const int64_t own = ceil_div(causal ? ceil_div(tiles, 2) : tiles, x);
      const int64_t cost = ceil_div(rem * x, sms) * (own + 4) + (x > 1 ? 6 : 0);
      if (cost < best) {
        best = cost;
        s = x;
      }
    }
    if (s > 1) {
      l.chunk = (int)ceil_div(tiles, s) * kTcKeys;
      l.n_split = (int)ceil_div(max_len, l.chunk);
    }
    if (l.n_split > 1) {
      n_whole = units - rem;
      blocks = n_whole + rem * l.n_split;
    }
    // (a workspace made for a longer history serves this one)
    parts = most > 1 ? rem * most : 0;
  } else {
    // Equal shares, or a block for each unit.  In stages (0.5 us each), with S of the
    // longest unit and half of them on average where the lengths come from the device:
    // blocks of their own take S in one wave, or all work and half of S in several;
    // equal shares take all work, 3 for a unit (kUnitCost), and the join, 7 and one for
    // 16 units.  Measured, own block / share, in us: 8 units of 768 keys 7.0 / 7.4, of
    // 1024 8.1 / 7.5, of 4096 21 / 8.2; 64 units of 1536 keys 10.5 / 11.5, of 2048 12.9 /
    // 12.3; 256 of 4096 33.9 / 37.3, but of up to 16384, half on average, 104 / 77.
    const int64_t slots = (bf16 || l.rows_blk == 8 ? 2 : 1) * sms;
    const bool may = max_len > 512 && units < 16 * slots;
    const double S = (double)ceil_div(max_len, kStageKeys), mean = unlike ? 0.5 * S : S;
    const double fill = (double)units / (double)slots;
    const double own = units <= slots ? S : fill * mean + 0.5 * S;
    l.stream = may && own > fill * (mean + 3.0) + 7.0 + (double)units / 16.0;
    if (may) parts = slots * 2;
    if (l.stream) {
      blocks = slots;
      n_whole = 0;
    }
  }
  if (blocks > 0x7fffffffll) return false;
  l.blocks = (int)blocks;
  l.n_whole = (int)n_whole;
  l.of = 256;
  l.ml = align_up(l.of + (parts > 0 ? (size_t)units * sizeof(int2) : 0), 256);
  l.o = align_up(l.ml + (size_t)parts * l.rows_blk * sizeof(float2), 256);
  l.total = align_up(l.o + (size_t)parts * l.rows_blk * d * sizeof(float), 256);
  return true;
}

template <int D>
cudaError_t run_all(const AttnArgs& a, bool bf16, int N, cudaStream_t s) {
  cudaError_t e;
  if (a.rows_blk == kTcRows)
    e = launch_attn_tc(a, N, D, s);
  else if (a.rows_blk == 8)
    e = bf16 ? run<__nv_bfloat16, D, 1>(a, N, s) : run<float, D, 1>(a, N, s);
  else
    e = bf16 ? run<__nv_bfloat16, D, 2>(a, N, s) : run<float, D, 2>(a, N, s);
  if (e != cudaSuccess || (!a.stream && a.n_split == 1)) return e;
  return bf16 ? join<__nv_bfloat16, D>(a, N, s) : join<float, D>(a, N, s);
}
}  // namespace

size_t kv4_attention_ws_bytes(bool bf16, int N, int Hq, int Hkv, int Lq, int max_len, int d) {
  Layout l;
  return layout(bf16, false, false, N, Hq, Hkv, Lq, max_len, d, l) ? l.total : 0;
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
  a.N = c.N;
  a.Hkv = c.H;
  a.G = p.Hq / c.H;
  a.R = a.G * p.Lq;
  a.Lq = p.Lq;
  a.max_len = p.max_len;
  a.cap = c.cap;
  a.causal = p.causal;
  a.scale_log2 = ldexpf(p.scale * 1.4426950408889634f, c.k_exp);
  a.out_scale = ldexpf(1.0f, c.v_exp);
  Layout l;
  if (!layout(p.bf16, p.causal, p.lens != nullptr, c.N, p.Hq, c.H, p.Lq, p.max_len, c.d, l)) return cudaErrorInvalidValue;
  a.rows_blk = l.rows_blk;
  a.n_rb = l.n_rb;
  a.stream = l.stream;
  a.n_whole = l.n_whole;
  a.n_split = l.n_split;
  a.chunk = l.chunk;
  a.blocks = l.blocks;
  a.stuck_slot = p.stuck_slot;
  a.wait_cycles = (uint32_t)p.wait_cycles;
  char* w = static_cast<char*>(ws);
  a.err = reinterpret_cast<int*>(w);
  a.part_of = reinterpret_cast<int2*>(w + l.of);
  a.part_ml = reinterpret_cast<float2*>(w + l.ml);
  a.part_o = reinterpret_cast<float*>(w + l.o);
  return c.d == 128 ? run_all<128>(a, p.bf16, c.N, s) : run_all<64>(a, p.bf16, c.N, s);
}

}  // namespace fc
