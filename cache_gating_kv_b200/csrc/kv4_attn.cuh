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
  int N, Hkv, G, R, Lq, max_len, cap;  // R = G * Lq rows of a key head
  int rows_blk, n_rb;                  // query rows of a block, row blocks of a key head
  bool stream;                         // shares of equal work (StreamShare)
  int n_whole, n_split, chunk;         // without: units with a block of their own, blocks
                                       // of each other one and their keys
  int blocks;                          // of the grid that computes
  bool causal;
  float scale_log2;  // scale * 2^k_exp * log2 e
  float out_scale;   // 2^v_exp
  int* err;
  uint32_t wait_cycles;  // limit of a wait
  int stuck_slot;         // of the ring: its barrier never completes (self-test; -1: none)
  // what blocks that share a unit leave for the join: by block (stream: two slots to a
  // block) and row
  float2* part_ml;  // [..][rows_blk] (log2 reference, sum)
  float* part_o;    // [..][rows_blk][d]
  int2* part_of;    // [N Hkv][n_rb] (first block, blocks) of a unit
};

__device__ __forceinline__ int seq_len(const AttnArgs& a, int n) {
  if (a.lens == nullptr) return a.max_len;
  return max(0, min(a.lens[n], a.max_len));
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

// Shares of equal work.  A unit is one key head of one sequence with one block of
// query rows; its work is its key stages (of kStageKeys) and kUnitCost more for what
// a unit costs whatever its length (loading its queries, filling and emptying the
// pipeline, joining the warps).  Units lie one behind the other in the order
// (sequence, row block, key head), the fixed cost first, and block c of C takes the
// work from floor(T c / C) to floor(T (c + 1) / C) of all T, whatever the lengths are:
// it ends the unit that an earlier block began, takes whole ones, and begins one.  A
// unit whose stages several blocks share leaves one part for each, in slot 1 of the
// block with its first stage and slot 0 of the others, and a second kernel joins
// them.  The lengths are on the device, so every block adds up the work itself.  (32
// sequences of unlike lengths, 8 key heads: 97 us with a unit cost of 0, 75 with 3; 82
// with a fixed split of every unit.)
constexpr int kStageKeys = 128;
constexpr int kUnitCost = 3;

__device__ __forceinline__ int entry_stages(const AttnArgs& a, int e) {
  const int n = a.n_rb == 1 ? e : e / a.n_rb;
  const int rb = e - n * a.n_rb;
  const int keys = block_keys(a, seq_len(a, n), rb * a.rows_blk, a.rows_blk);
  return (keys + kStageKeys - 1) / kStageKeys;
}
// Work of one key head of an entry (sequence, row block).
__device__ __forceinline__ int entry_work(const AttnArgs& a, int e) {
  const int s = entry_stages(a, e);
  return s > 0 ? s + kUnitCost : 0;
}
// x / y for x >= 0, y > 0, mostly small.
__device__ __forceinline__ int64_t div_small(int64_t x, int64_t y) {
  if (((x | y) >> 32) == 0) return (int64_t)((uint32_t)x / (uint32_t)y);
  return x / y;
}

// A piece of a share: stages [s_begin, s_end) of n_unit of a unit.
struct Piece {
  int n, hk, rb, n_unit, s_begin, s_end;
  int n_parts;  // blocks that share the unit, where this one has its first stage
};

// Where a walk through a share stands.
struct Walk {
  int64_t pos;    // work done
  int64_t start;  // the work before entry e
  int e;          // entry (sequence, row block) at pos
};

// A block's share, in shared memory.  begin() is called by the whole block.
template <int kThreads>
struct StreamShare {
  int64_t warp_sum[kThreads / 32];
  int64_t total, end;  // all work, the end of the share
  int C;               // blocks
  Walk first;

  __device__ __forceinline__ void begin(const AttnArgs& a, int least) {
    const int E = a.N * a.n_rb;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (E + kThreads - 1) / kThreads;
    const int e0 = threadIdx.x * per, e1 = min(E, e0 + per);
    int64_t own = 0;
    for (int i = e0; i < e1; ++i) own += entry_work(a, i);
    own *= a.Hkv;
    int64_t upto = own;  // inclusive
    if (E > 1) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
    }
    int64_t all = upto;
    if (E > per * 32) {  // over more than the first warp
      if (lane == 31) warp_sum[warp] = upto;
      __syncthreads();
      all = 0;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) upto += warp_sum[w];
        all += warp_sum[w];
      }
    } else if (E > 1) {
      all = __shfl_sync(0xffffffffu, upto, 31);
    }
    if (E > per * 32 || warp == 0) {
      const int64_t most = all / least;  // a constant
      const int blocks = most < 1 ? 1 : most < (int64_t)gridDim.x ? (int)most : (int)gridDim.x;
      const int c = blockIdx.x;
      const int64_t lo = c < blocks ? div_small(all * c, blocks) : 0;
      const int64_t hi = c < blocks ? div_small(all * (c + 1), blocks) : 0;
      if (lo >= hi) {
        if (threadIdx.x == 0) first.pos = end = 0;
      } else if (upto - own <= lo && lo < upto) {
        int64_t at = upto - own;
        int i = e0;
        for (;; ++i) {
          const int64_t w = (int64_t)entry_work(a, i) * a.Hkv;
          if (lo < at + w) break;
          at += w;
        }
        total = all;
        end = hi;
        C = blocks;
        first.pos = lo;
        first.start = at;
        first.e = i;
      }
    }
    __syncthreads();
  }

  // The next piece with stages; false at the end of the share.
  __device__ __forceinline__ bool next(const AttnArgs& a, Walk& at, Piece& p) const {
    while (at.pos < end) {
      int w;
      while ((w = entry_work(a, at.e)) == 0) ++at.e;
      p.n = a.n_rb == 1 ? at.e : at.e / a.n_rb;
      p.rb = at.e - p.n * a.n_rb;
      p.n_unit = w - kUnitCost;
      p.hk = (int)div_small(at.pos - at.start, w);
      const int64_t unit0 = at.start + (int64_t)p.hk * w;
      const int from = (int)(at.pos - unit0), to = (int)min((int64_t)w, from + (end - at.pos));
      p.s_begin = max(0, from - kUnitCost);
      p.s_end = max(0, to - kUnitCost);
      // the block with the unit's last stage: the largest c with T c / C <= it
      p.n_parts = 1;
      if (p.s_begin == 0 && p.s_end > 0 && p.s_end < p.n_unit)
        p.n_parts = (int)div_small((unit0 + w) * C - 1, total) - (int)blockIdx.x + 1;
      at.pos += to - from;
      if (to == w && p.hk == a.Hkv - 1) {
        at.start = at.pos;
        ++at.e;
      }
      if (p.s_end > p.s_begin) return true;
    }
    return false;
  }
};
// Without shares: unit i, by sequence, key head and row block, the last rows first
// (where the mask is causal they see the most keys).
__device__ __forceinline__ void unit_at(const AttnArgs& a, int64_t i, int& n, int& hk, int& rb) {
  const int unit = (int)(i / a.n_rb);
  rb = a.n_rb - 1 - (int)(i - (int64_t)unit * a.n_rb);
  n = unit / a.Hkv;
  hk = unit - n * a.Hkv;
}
__device__ __forceinline__ void whole_unit(const AttnArgs& a, Piece& p) {
  unit_at(a, blockIdx.x, p.n, p.hk, p.rb);
  p.s_begin = 0;
  p.s_end = p.n_unit = entry_stages(a, p.n * a.n_rb + p.rb);
  p.n_parts = 1;
}

// Four outputs of row r from their weighted sums o, the row's log2 reference
// and its sum L of 2^(x - ref).
template <typename T>
__device__ __forceinline__ void write_row(const AttnArgs& a, int n, int hk, int r, int c, float4 o,
                                          float ref, float L) {
  const int i = r / a.G, h = hk * a.G + r % a.G;
  T* p = static_cast<T*>(a.out) + n * a.os.n + h * a.os.h + i * a.os.l + c;
  if constexpr (sizeof(T) == 4) {  // each quotient rounds once
    const float by = L == 0.0f ? 1.0f : L, up = L == 0.0f ? 0.0f : a.out_scale;
    *reinterpret_cast<float4*>(p) = make_float4(__fdiv_rn(o.x, by) * up, __fdiv_rn(o.y, by) * up,
                                                __fdiv_rn(o.z, by) * up, __fdiv_rn(o.w, by) * up);
  } else {
    // 2 ulps of float32 here, in front of a rounding to 8 bits (L is far below the 2^126
    // from which this quotient would be zero)
    const float f = L == 0.0f ? 0.0f : __fdividef(a.out_scale, L);
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
