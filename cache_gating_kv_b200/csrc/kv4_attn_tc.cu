// Attention over the 4-bit cache for many query rows per key head (a prompt, a
// chunk being denoised), on the 5th-generation tensor cores.
//
// 4 R L d flops per key head: bound by the tensor cores and, one exponential per
// logit, by the special-function units, not by HBM.  A block holds 256 query rows
// (two tiles of 128, kept in shared memory as float16 after a power of two per
// row) and walks the keys in tiles of 128:
//   S_j = Q_j K^T      tcgen05.mma, both operands in shared memory, into TMEM
//   P_j = 2^(c S_j - ref)   softmax warps, from TMEM to registers and back as
//                      float16 into the columns that S_j held
//   O_j += P_j V       tcgen05.mma with P_j read from TMEM
// for the two tiles j in turn, so that the tensor cores work on one tile while
// the softmax warps work on the other.  TMEM (512 columns at d = 128): S_0, S_1,
// O_0, O_1.
//
// Keys and values stay 4 bits up to shared memory: bulk copies bring codes and
// scales (contiguous for a run of rows), four warps write code * scale, exact in
// float16, into 128-byte-swizzled operand tiles.  K is a K-major operand and V an
// MN-major one, so both are written as they come, row by row.  A converting thread
// takes 16 bytes of codes (a quarter of a row at d = 128) and the quarters of a row
// start at different chunks, which leaves neither its loads nor its stores a bank
// conflict.
//
// The running reference of a row moves only when a tile exceeds it by 2^8, and
// then the softmax warps scale O_j themselves: S_j of a tile is issued after
// P_j V of the one before, so its arrival means that O_j is at rest.
//
// What bounds it: at N = 128 a tcgen05.mma with both operands in shared memory reads
// 8 KB for 64 cycles of work, all that shared memory gives, and S_j -> P_j -> O_j is a
// chain through three units.  4096 queries x 20480 keys x 24 heads, d = 128: 0.97-1.0
// ms (0.63 ms at the measured GEMM rate).  In clocks a tile of 128 keys takes a softmax
// warp 3700: 200 for the load, 470 for the maximum, 1400 for the exponentials (1024 at
// the units' rate), 100 for the store and 1500 of waiting, in which the tensor cores
// have 500 of P V and 700 of Q K^T for each of the two query tiles.  So P goes out in
// halves, and P V starts behind the first (972 us for 988).
// Measured and not kept: a quarter of the exponentials on the FMA pipes (+5 %), one
// read of S in two parts to save registers (+10 %), a persistent loop over equal shares
// (+10 %: its state makes the softmax warps spill), S in halves of 64 keys computed one
// ahead (+10 %: at N = 64 the tensor cores take 90 clocks for 16 of K in P V, 64 in
// Q K^T), six converting warps (0).
//
// Roles (512 threads): warps 0-3 and 4-7 softmax of tile 0 and 1 (a thread owns a
// row), 8-11 conversion, 12 bulk copies, 13 MMA issue, 14 TMEM allocation.  Every
// wait is bounded; one that gives up sets the workspace's error word.
#include "fc_common.cuh"
#include "fc_kernels.h"
#include "kv4.cuh"
#include "kv4_attn.cuh"
#include "tc_ptx.cuh"

namespace fc {

namespace {
constexpr int kThreads = 512;
constexpr int kM = 128;       // rows of a query tile
constexpr int kN = kTcKeys;   // keys of a tile
constexpr int kOps = 4;       // operand stages: K and V tiles in turn
constexpr int kCodes = 3;     // code stages
constexpr float kShift = 5.0f, kSlack = 8.0f;
// Registers of the softmax, converting and remaining warps; their sum over 512
// threads is within the 65,536 that 512 x 128 at launch hold.
constexpr int kRegSoftmax = 200, kRegConvert = 56, kRegRest = 48;
static_assert(256 * kRegSoftmax + 128 * kRegConvert + 128 * kRegRest <= 512 * 128, "registers");

template <int D> constexpr int op_bytes() { return kN * D * 2; }
template <int D> constexpr int code_bytes() { return kN * (D / 2 + D / 8); }  // codes, scales, V scales
constexpr int kBarBytes = 512;
template <int D> constexpr int smem_bytes() {
  return 1024 + 2 * kM * D * 2 + kOps * op_bytes<D>() + kCodes * code_bytes<D>() + kBarBytes;
}

struct Bars {
  uint64_t code_full[kCodes], code_empty[kCodes];
  uint64_t op_full[kOps], op_empty[kOps];
  uint64_t q_full;
  uint64_t s_full[2], p_full[2][2], o_full[2];  // of the query tiles; P in halves
  uint64_t drained;
  uint32_t tmem_slot;
};
static_assert(sizeof(Bars) <= kBarBytes, "barriers");

// Offset of 16-byte chunk c (of D/8) of row r in a tile of kN swizzled rows.
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return (uint32_t)((c >> 3) * (kN * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// One arrival for the warp, behind what all its lanes did.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) tc::mbar_arrive(bar);
}

template <int J> struct Tile { static constexpr int value = J; };

__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ float2 f2(uint32_t a, uint32_t b) {
  return make_float2(__uint_as_float(a), __uint_as_float(b));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_tc_kernel(const AttnArgs a) {
  constexpr int CB = D / 2, SB = D / 16;
  constexpr int kOp = op_bytes<D>(), kCode = code_bytes<D>();
  constexpr int kQ = kM * D * 2;
  constexpr uint32_t kIdescQK = tc::idesc_f16_f32(kM, kN, false);
  constexpr uint32_t kIdescPV = tc::idesc_f16_f32(kM, D, true);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  uint8_t* sQ = base;
  uint8_t* sOp = sQ + 2 * kQ;
  uint8_t* sCode = sOp + kOps * kOp;
  Bars* bars = reinterpret_cast<Bars*>(sCode + kCodes * kCode);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // The first n_whole units have a block each, the others n_split.
  const int b = blockIdx.x, part = b - a.n_whole;
  const bool shared_unit = part >= 0;
  const int split = shared_unit ? part % a.n_split : 0;
  int n, hk, rb;
  unit_at(a, shared_unit ? a.n_whole + part / a.n_split : b, n, hk, rb);
  const int unit = n * a.Hkv + hk;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kCodes; ++i) {
      tc::mbar_init(&bars->code_full[i], i == a.stuck_slot ? 2 : 1);
      tc::mbar_init(&bars->code_empty[i], 4);
    }
    for (int i = 0; i < kOps; ++i) {
      tc::mbar_init(&bars->op_full[i], 4);
      tc::mbar_init(&bars->op_empty[i], 1);
    }
    tc::mbar_init(&bars->q_full, 8);
    for (int j = 0; j < 2; ++j) {
      tc::mbar_init(&bars->s_full[j], 1);
      tc::mbar_init(&bars->p_full[j][0], 4);
      tc::mbar_init(&bars->p_full[j][1], 4);
      tc::mbar_init(&bars->o_full[j], 1);
    }
    tc::mbar_init(&bars->drained, 1);
    tc::fence_barrier_init();
  }
  if (warp == 14) tc::tmem_alloc(&bars->tmem_slot, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem_slot, 0);  // known as uniform
  grid_dep_wait();
  if (a.n_split > 1) grid_dep_launch();  // the join

  const int len = seq_len(a, n);
  const int r_base = rb * kTcRows;
  const int chunk = shared_unit ? a.chunk : a.max_len;
  const int k_begin = split * chunk;
  // keys and key tiles of each query tile
  int k_end[2], nt[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int r0 = r_base + j * kM;
    k_end[j] = r0 < a.R ? min(block_keys(a, len, r0, kM), k_begin + chunk) : 0;
    nt[j] = k_end[j] > k_begin ? (k_end[j] - k_begin + kN - 1) / kN : 0;
  }
  const int T = max(nt[0], nt[1]);
  const int k_top = max(k_end[0], k_end[1]);
  // The unit is joined from its parts if it has more than one with keys; parts without
  // are not written.
  const int keys = block_keys(a, len, r_base, kTcRows);
  const int n_parts = shared_unit ? max(1, (keys + chunk - 1) / chunk) : 1;
  const bool idle = split >= n_parts;
  if (shared_unit && split == 0 && threadIdx.x == 0)
    a.part_of[(int64_t)unit * a.n_rb + rb] = make_int2(part, n_parts);
  const int64_t head = (int64_t)unit * a.cap;
  bool ok = true;

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegSoftmax));
    const int j = warp >> 2;                       // query tile
    const int rloc = (warp & 3) * 32 + lane;       // row of the tile, TMEM lane
    const int r = r_base + j * kM + rloc;
    const bool have = r < a.R;
    const int i = r / a.G, hq = hk * a.G + r % a.G;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = lanes + j * kN, tO = lanes + 2 * kN + j * D;
    float fac;
    if (T > 0) {
      // the row as float16, its largest number brought to 2^13
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                        n * a.qs.n + hq * a.qs.h + i * a.qs.l);
      uint4 w[D / 8];
      uint32_t top2 = 0;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        w[c] = have ? src[c] : make_uint4(0u, 0u, 0u, 0u);
        top2 = __vmaxu2(top2, __vmaxu2(__vmaxu2(w[c].x & 0x7fff7fffu, w[c].y & 0x7fff7fffu),
                                       __vmaxu2(w[c].z & 0x7fff7fffu, w[c].w & 0x7fff7fffu)));
      }
      const uint32_t top = max(top2 & 0xffffu, top2 >> 16);  // bf16 bits
      int ex = (int)(top >> 7) - 127;
      ex = top == 0 ? 0 : max(-100, min(ex, 127));
      const float down = __uint_as_float((uint32_t)(127 + 13 - ex) << 23);
      fac = fmaxf(ldexpf(a.scale_log2, ex - 13), 1.2e-38f);  // never 0 * -inf
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        float f[8];
        Vec16<__nv_bfloat16>::to_float(w[c], f);
        *reinterpret_cast<uint4*>(sQ + j * kQ + chunk_at(rloc, c)) =
            make_uint4(pack_f16(f[0] * down, f[1] * down), pack_f16(f[2] * down, f[3] * down),
                       pack_f16(f[4] * down, f[5] * down), pack_f16(f[6] * down, f[7] * down));
      }
      fence_async();
      warp_arrive(&bars->q_full);
    }
    const int lim = have ? min(k_top, row_keys(a, len, i)) : k_top;  // keys of the row
    int lim_min = lim;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, o));

    float ref = -INFINITY;
    float2 l2 = make_float2(0.f, 0.f);
    for (int t = 0; t < nt[j]; ++t) {
      if (!__all_sync(0xffffffffu, tc::mbar_sleep(&bars->s_full[j], t & 1, a.wait_cycles))) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      uint32_t s[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tc::tmem_ld32(tS + c * 32, s[c]);
#pragma unroll
      for (int c = 0; c < 4; ++c) tc::tmem_ld_wait(s[c]);
      const int k0 = k_begin + t * kN;
      if (k0 + kN > lim_min) {  // some row of the warp does not see all of the tile
        const int left = lim - k0;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (c * 32 + e >= left) s[c][e] = 0xff800000u;  // -inf
      }
      float mx[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        mx[c] = __uint_as_float(s[c][0]);
#pragma unroll
        for (int e = 1; e < 31; e += 2)
          mx[c] = tc::fmax3_nan(mx[c], __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
        mx[c] = tc::fmax3_nan(mx[c], __uint_as_float(s[c][31]), __uint_as_float(s[c][31]));
      }
      const float top = tc::fmax3_nan(tc::fmax3_nan(mx[0], mx[1], mx[2]), mx[3], mx[3]) * fac;
      const bool move = !(top <= ref + kSlack);
      if (__any_sync(0xffffffffu, move)) {
        // a NaN in the row makes the reference and with it the sum NaN
        const float to = move ? top : ref;
        const float al = to == ref ? 1.0f : tc::ex2(ref - to);
        if (move) ref = to;
        l2.x *= al;
        l2.y *= al;
        if (t > 0) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tc::tmem_ld32(tO + c * 32, o);
            tc::tmem_ld_wait(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
            tc::tmem_st32(tO + c * 32, o);
          }
        }
      }
      const float off = kShift - (ref == -INFINITY ? 0.0f : ref);
      const float2 ff = make_float2(fac, fac), oo = make_float2(off, off);
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int hp = 0; hp < 2; ++hp) {
        uint32_t p[32];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const uint32_t* v = s[2 * hp + c] + 2 * e;
            const float2 x = tc::ffma2(f2(v[0], v[1]), ff, oo);
            const float2 y = make_float2(tc::ex2(x.x), tc::ex2(x.y));
            sum = tc::fadd2(sum, y);
            p[c * 16 + e] = pack_f16(y.x, y.y);
          }
        }
        tc::tmem_st32(tS + hp * 32, p);
        tc::tmem_st_wait();
        tc::fence_before_sync();
        warp_arrive(&bars->p_full[j][hp]);
      }
      l2 = tc::fadd2(l2, sum);
    }
    // ---- the row's result
    if (ok && nt[j] > 0) {
      ok = __all_sync(0xffffffffu, tc::mbar_sleep(&bars->o_full[j], 0, a.wait_cycles));
      tc::fence_after_sync();
    }
    if (!idle) {
      const float L = ref == -INFINITY ? 0.0f : l2.x + l2.y;
      const float at_ref = ref == -INFINITY ? ref : ref - kShift;
      const int64_t at = (int64_t)part * kTcRows + j * kM + rloc;
      if (n_parts > 1 && have) a.part_ml[at] = make_float2(at_ref, L);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (ok && nt[j] > 0) {
          tc::tmem_ld32(tO + c * 32, o);
          tc::tmem_ld_wait(o);
        }
        if (!ok || ref == -INFINITY) {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        if (have) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 v = make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                         __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
            if (n_parts > 1)
              *reinterpret_cast<float4*>(a.part_o + at * D + c * 32 + e) = v;
            else
              write_row<__nv_bfloat16>(a, n, hk, r, c * 32 + e, v, at_ref, L);
          }
        }
      }
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegConvert));
    // ---- conversion: a thread takes 16 bytes of codes (32 numbers) of a row
    constexpr int TPR = CB / 16;          // threads of a row: 4 or 2
    constexpr int kPass = 128 / TPR;      // rows of a pass
    const int tid = threadIdx.x - 256;
    const int part = tid % TPR, r0 = tid / TPR;
    // The lanes of a store phase are 8 / TPR rows of TPR parts; starting the
    // upper parts (the second 128-byte block of a row) two chunks later makes
    // them meet no bank twice.
    const int turn = (part >> 1) * 2;
    for (int h = 0; h < 2 * T; ++h) {
      const int cs = h % kCodes, os = h % kOps;
      // the lanes go on together or not at all: a warp split between its own barrier and
      // the block's might wait for ever
      ok = __all_sync(0xffffffffu,
                      tc::mbar_sleep(&bars->code_full[cs], (h / kCodes) & 1, a.wait_cycles) &&
                          tc::mbar_sleep(&bars->op_empty[os], ((h / kOps) & 1) ^ 1, a.wait_cycles));
      if (!ok) break;
      const bool key = (h & 1) == 0;
      const uint8_t* codes = sCode + cs * kCode;
      const uint8_t* scales = codes + kN * CB;
      uint8_t* op = sOp + os * kOp;
      const int left = k_top - (k_begin + (h >> 1) * kN);
#pragma unroll 1
      for (int p = 0; p < kN / kPass; ++p) {
        const int r = p * kPass + r0;
        const uint4 w = *reinterpret_cast<const uint4*>(codes + r * CB + part * 16);
        uint32_t sb = *reinterpret_cast<const uint16_t*>(scales + r * SB + part * 2);
        if (key) {  // a NaN among the row's values goes with the key (see value_scales)
          const uint32_t vb = *reinterpret_cast<const uint16_t*>(scales + kN * SB + r * SB + part * 2);
          if (((vb & 0x7F7Fu) + 0x0101u) & 0x8080u) sb = 0x7F7Fu;
        } else {
          if (((sb & 0x7Fu) == 0x7Fu) || r >= left) sb &= 0xFF00u;
          if (((sb & 0x7F00u) == 0x7F00u) || r >= left) sb &= 0x00FFu;
        }
        const uint32_t hs = kv4::e4m3x2_to_f16x2(sb);
        const uint32_t s0 = __byte_perm(hs, hs, 0x1010), s1 = __byte_perm(hs, hs, 0x3232);
        // chunk i of the part is word i; the turned order starts at word 2
        const bool up = turn != 0;
        const uint32_t x[4] = {up ? w.z : w.x, up ? w.w : w.y, up ? w.x : w.z, up ? w.y : w.w};
        const uint32_t sa = up ? s1 : s0, sc = up ? s0 : s1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t v[4];
          kv4::e2m1x8_to_f16x2(x[i], v);
          const uint32_t sg = i < 2 ? sa : sc;
          *reinterpret_cast<uint4*>(op + chunk_at(r, part * 4 + (i ^ turn))) =
              make_uint4(hmul2(v[0], sg), hmul2(v[1], sg), hmul2(v[2], sg), hmul2(v[3], sg));
        }
      }
      fence_async();
      warp_arrive(&bars->op_full[os]);
      if ((threadIdx.x & 31) == 0) tc::mbar_arrive(&bars->code_empty[cs]);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegRest));
    if (warp == 12 && lane == 0) {
      // ---- bulk copies: K tile t is stage 2 t, V tile t stage 2 t + 1
      const int k_pad = (k_top + 15) & ~15;  // cap is a multiple of 16
      int h = 0;
      for (; h < 2 * T; ++h) {
        const int cs = h % kCodes;
        if (!tc::mbar_sleep(&bars->code_empty[cs], ((h / kCodes) & 1) ^ 1, a.wait_cycles)) {
          ok = false;
          break;
        }
        const int k0 = k_begin + (h >> 1) * kN;
        const int rows = min(kN, k_pad - k0);
        uint8_t* dst = sCode + cs * kCode;
        uint64_t* bar = &bars->code_full[cs];
        if ((h & 1) == 0) {
          tc::mbar_expect_tx(bar, rows * (CB + 2 * SB));
          bulk_load(dst, a.k_codes + (head + k0) * CB, rows * CB, bar);
          bulk_load(dst + kN * CB, a.k_scales + (head + k0) * SB, rows * SB, bar);
          bulk_load(dst + kN * (CB + SB), a.v_scales + (head + k0) * SB, rows * SB, bar);
        } else {
          tc::mbar_expect_tx(bar, rows * (CB + SB));
          bulk_load(dst, a.v_codes + (head + k0) * CB, rows * CB, bar);
          bulk_load(dst + kN * CB, a.v_scales + (head + k0) * SB, rows * SB, bar);
        }
      }
      for (int x = max(0, h - kCodes); x < h; ++x)  // no copy outlives the block
        ok &= tc::mbar_sleep(&bars->code_full[x % kCodes], (x / kCodes) & 1, tc::kDrainCycles);
    } else if (warp == 13 && T > 0) {
      // ---- MMA issue.  The logits of a tile wait for this warp twice a step, so it
      // keeps no arrays and finds its descriptors by additions.  The warp stays together
      // and one elected thread issues: with the loop in a single thread of a divergent
      // warp an MMA took some 120 clocks to issue (1013 us for 996; 40.5 for 38.6 for 4
      // causal prompts).
      const uint64_t q_desc = tc::desc_k_sw128(tc::smem_u32(sQ));
      const uint64_t k_desc = tc::desc_k_sw128(tc::smem_u32(sOp));
      const uint64_t v_desc = tc::desc_mn_sw128(tc::smem_u32(sOp), kN * 128);
      auto wait = [&](uint64_t* bar, int phase) {
        return __all_sync(0xffffffffu, tc::mbar_sleep(bar, phase & 1, a.wait_cycles)) != 0;
      };
      auto qk = [&](auto jc, int os) {
        constexpr int j = decltype(jc)::value;
        const uint64_t q = q_desc + j * (kQ >> 4), k = k_desc + os * (kOp >> 4);
        if (!tc::elect()) return;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t o = ((kk >> 2) * (kN * 128) + (kk & 3) * 32) >> 4;
          tc::mma_bf16(tmem + j * kN, q + o, k + o, kIdescQK, kk > 0 ? 1u : 0u);
        }
        tc::mma_commit(&bars->s_full[j]);
      };
      auto pv = [&](auto jc, int os, int t) -> bool {
        constexpr int j = decltype(jc)::value;
        const uint64_t v = v_desc + os * (kOp >> 4);
#pragma unroll
        for (int hp = 0; hp < 2; ++hp) {
          if (!wait(&bars->p_full[j][hp], t)) return false;
          tc::fence_after_sync();
          if (tc::elect()) {
#pragma unroll
            for (int kk = hp * kN / 32; kk < (hp + 1) * kN / 32; ++kk)
              tc::mma_f16_ts(tmem + 2 * kN + j * D, tmem + j * kN + kk * 8, v + (kk * 2048 >> 4),
                             kIdescPV, t > 0 || kk > 0 ? 1u : 0u);
          }
        }
        return true;
      };
      auto stage_in = [&](int x) { return wait(&bars->op_full[x % kOps], x / kOps); };
      auto commit = [&](uint64_t* bar) {
        if (tc::elect()) tc::mma_commit(bar);
      };
      constexpr Tile<0> t0;
      constexpr Tile<1> t1;
      const int nt0 = nt[0], nt1 = nt[1];
      ok = wait(&bars->q_full, 0) && stage_in(0);
      if (ok) {
        tc::fence_after_sync();
        if (nt0 > 0) qk(t0, 0);
        if (nt1 > 0) qk(t1, 0);
        commit(&bars->op_empty[0]);
      }
#pragma unroll 1
      for (int t = 0; ok && t < T; ++t) {
        const int sv = (2 * t + 1) % kOps, sk = (2 * t + 2) % kOps;
        if (!(ok = stage_in(2 * t + 1))) break;
        if (t + 1 < T && !(ok = stage_in(2 * t + 2))) break;
        if (t < nt0) {
          if (!(ok = pv(t0, sv, t))) break;
          if (t + 1 == nt0) commit(&bars->o_full[0]);
        }
        if (t + 1 < nt0) qk(t0, sk);
        if (t < nt1) {
          if (!(ok = pv(t1, sv, t))) break;
          if (t + 1 == nt1) commit(&bars->o_full[1]);
        }
        commit(&bars->op_empty[sv]);
        if (t + 1 < nt1) qk(t1, sk);
        if (t + 1 < T) commit(&bars->op_empty[sk]);
      }
      if (!ok) {  // no MMA outlives the allocation
        commit(&bars->drained);
        tc::mbar_sleep(&bars->drained, 0);
      }
    }
  }
  if (!ok) atomicExch(a.err, 1);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 14) tc::tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t run(const AttnArgs& a, int N, cudaStream_t s) {
  constexpr int smem = smem_bytes<D>();
  static_assert(smem <= 232448, "shared memory of a block");
  cudaError_t e = cudaFuncSetAttribute(attn_tc_kernel<D>,
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
  e = cudaLaunchKernelEx(&cfg, attn_tc_kernel<D>, a);
  if (e != cudaSuccess) return e;
  add_launches(1);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_attn_tc(const AttnArgs& a, int N, int d, cudaStream_t s) {
  return d == 128 ? run<128>(a, N, s) : run<64>(a, N, s);
}

}  // namespace fc
