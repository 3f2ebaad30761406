// fd_int4.cuh — a KV cache held in 4 bits: quantising rows into it, reading it
// back as bf16, and decode attention over it.
//
// A row (one token of one KV head, D entries) has two groups of D / 2 entries.
// Entry x of a group is held as a code c in 0..15 with the group's bf16 scale s
// and bias b, and stands for s (c - 8) + b.  The codes of K and V are D / 2
// bytes each, entry 2j in the low nibble of byte j; the scales and biases of
// both are one 16-byte record, ks0 kb0 ks1 kb1 vs0 vb0 vs1 vb1.  The same
// record size for D = 64 and 128 keeps a row's record one aligned 16-byte
// load; a bf16 scale has the range of the bf16 rows it comes from.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "fd_kernels.cuh"
#include "fd_ptx.cuh"

namespace fd {

struct Int4Cache {
  uint8_t* k4;          // [planes, Hkv, rows, D/2], or [planes, rows, Hkv, D/2]
  uint8_t* v4;
  uint8_t* params;      // the same order, 16 bytes per row
  int planes;           // sequences (contiguous) or pages (paged)
  int rows;             // rows per plane and KV head
  int Hkv;
  bool nhd;             // token-major
};

// Index of a row among the cache's rows.
__device__ __forceinline__ size_t int4_row(const Int4Cache& c, int plane, int head, int row) {
  return c.nhd ? (static_cast<size_t>(plane) * c.rows + row) * c.Hkv + head
               : (static_cast<size_t>(plane) * c.Hkv + head) * c.rows + row;
}

__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// ---------------------------------------------------------------- append

struct AppendArgs {
  Int4Cache c;
  const __nv_bfloat16* k;    // token i, head h: k + i * k_stride + h * D
  const __nv_bfloat16* v;
  int64_t k_stride, v_stride;
  const int64_t* slots;      // [n_tokens]
  int n_tokens;
};

// Quantises the 8 entries that this lane holds of a row; LPG neighbouring
// lanes hold a group.  Returns the lane's codes, entry i in bits 4i .. 4i+3,
// and the group's record (scale in the low half, bias in the high half).
//   s = bf16((mx - mn) / 15), b = bf16(mn + 8 s),
//   c = clamp(rint((x - b) / s), -8, 7) + 8
// in fp32 (ties to even).  (mx - mn) / 15 is taken as (mx/2 - mn/2) / 7.5 and
// mn + 8 s with one rounding, so that no bf16 input overflows.  A group with
// s = 0 gets the code 8; one with a NaN or an infinity gets s = b = NaN.
template <int LPG>
__device__ __forceinline__ uint32_t int4_quantise(uint4 raw, uint32_t& record) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  float x[8];
  float mn = INFINITY, mx = -INFINITY;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
    mn = fminf(mn, fminf(x[2 * i], x[2 * i + 1]));
    mx = fmaxf(mx, fmaxf(x[2 * i], x[2 * i + 1]));
    top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
  }
#pragma unroll
  for (int off = 1; off < LPG; off <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
  }
  const float half_range = __fsub_rn(__fmul_rn(mx, 0.5f), __fmul_rn(mn, 0.5f));
  const float s = round_to_bf16(__fdiv_rn(half_range, 7.5f));
  const float b = round_to_bf16(__fmaf_rn(8.f, s, mn));
  const bool finite = top < 0x7f80u;
  record = finite ? pack_bf16x2(s, b) : 0x7fc07fc0u;
  if (!finite || !(s > 0.f)) return 0x88888888u;
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = rintf(__fdiv_rn(__fsub_rn(x[i], b), s));
    codes |= static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(y, -8.f), 7.f)) + 8) << (4 * i);
  }
  return codes;
}

// D / 8 lanes per row; the rows of a token are its K heads, then its V heads.
template <int D>
__global__ void __launch_bounds__(256) fd_append_int4_kernel(const AppendArgs a) {
  grid_dependency_wait();
  grid_dependents_launch();
  constexpr int LPR = D / 8;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * (256 / LPR) + threadIdx.x / LPR;
  const int part = threadIdx.x % LPR;
  const int64_t n_rows = static_cast<int64_t>(a.n_tokens) * 2 * a.c.Hkv;
  const int64_t row = at < n_rows ? at : n_rows - 1;      // whole warps take part in the shuffles
  const int token = static_cast<int>(row / (2 * a.c.Hkv));
  const int unit = static_cast<int>(row - static_cast<int64_t>(token) * 2 * a.c.Hkv);
  const bool is_v = unit >= a.c.Hkv;
  const int head = is_v ? unit - a.c.Hkv : unit;
  const __nv_bfloat16* src = is_v ? a.v + token * a.v_stride : a.k + token * a.k_stride;
  const uint4 raw = *reinterpret_cast<const uint4*>(src + head * D + part * 8);
  uint32_t record;
  const uint32_t codes = int4_quantise<LPR / 2>(raw, record);
  const int64_t slot = a.slots[token];
  if (at >= n_rows || slot < 0 || slot >= static_cast<int64_t>(a.c.planes) * a.c.rows) return;
  const int plane = static_cast<int>(slot / a.c.rows);
  const size_t to = int4_row(a.c, plane, head, static_cast<int>(slot - static_cast<int64_t>(plane) * a.c.rows));
  uint8_t* dst = is_v ? a.c.v4 : a.c.k4;
  *reinterpret_cast<uint32_t*>(dst + to * (D / 2) + part * 4) = codes;
  if (part % (LPR / 2) == 0)
    *reinterpret_cast<uint32_t*>(a.c.params + to * 16 + (is_v ? 8 : 0) + (part / (LPR / 2)) * 4) = record;
}

// ---------------------------------------------------------------- expand

struct ExpandArgs {
  Int4Cache c;
  const int32_t* seqlens;
  const int32_t* block_table;
  int log2_block_size, max_blocks;
  int max_len;
  __nv_bfloat16* k;          // [B, Hkv, max_len, D], or [B, max_len, Hkv, D]
  __nv_bfloat16* v;
};

// The 8 codes of a word as the bf16 values they stand for.
__device__ __forceinline__ uint4 int4_values(uint32_t codes, uint32_t record) {
  const float s = bf16_lo(record), b = bf16_hi(record);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c0 = static_cast<int>((codes >> (8 * i)) & 15u) - 8;
    const int c1 = static_cast<int>((codes >> (8 * i + 4)) & 15u) - 8;
    w[i] = pack_bf16x2(__fmaf_rn(s, static_cast<float>(c0), b), __fmaf_rn(s, static_cast<float>(c1), b));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kExpandTokens = 32;

// One CTA per 32 tokens of one KV head of one sequence; D / 8 lanes per row.
template <int D>
__global__ void __launch_bounds__(256) fd_expand_int4_kernel(const ExpandArgs a) {
  grid_dependency_wait();
  grid_dependents_launch();
  constexpr int LPR = D / 8;
  const int b = blockIdx.z, head = blockIdx.y;
  const int n = seq_length(a.seqlens, b, a.max_len);
  const int t0 = blockIdx.x * kExpandTokens;
  const int part = threadIdx.x % LPR;
  for (int t = t0 + threadIdx.x / LPR; t < min(n, t0 + kExpandTokens); t += 256 / LPR) {
    int plane = b, row = t;
    if (a.block_table) {
      plane = a.block_table[static_cast<size_t>(b) * a.max_blocks + (t >> a.log2_block_size)];
      row = t & ((1 << a.log2_block_size) - 1);
    }
    uint4 kv = make_uint4(0, 0, 0, 0), vv = kv;
    if (plane >= 0 && plane < a.c.planes) {
      const size_t from = int4_row(a.c, plane, head, row);
      const uint8_t* rec = a.c.params + from * 16 + (part / (LPR / 2)) * 4;
      kv = int4_values(*reinterpret_cast<const uint32_t*>(a.c.k4 + from * (D / 2) + part * 4),
                       *reinterpret_cast<const uint32_t*>(rec));
      vv = int4_values(*reinterpret_cast<const uint32_t*>(a.c.v4 + from * (D / 2) + part * 4),
                       *reinterpret_cast<const uint32_t*>(rec + 8));
    }
    const size_t to = a.c.nhd ? (static_cast<size_t>(b) * a.max_len + t) * a.c.Hkv + head
                              : (static_cast<size_t>(b) * a.c.Hkv + head) * a.max_len + t;
    *reinterpret_cast<uint4*>(a.k + to * D + part * 8) = kv;
    *reinterpret_cast<uint4*>(a.v + to * D + part * 8) = vv;
  }
}

// ---------------------------------------------------------------- decode

struct Int4DecodeArgs {
  SplitArgs a;     // as fd_split_kernel's; k_scale and v_scale do not apply
  Int4Cache c;
};

constexpr int kInt4Warps = 4;

// The log-sum-exp of a split as the merge takes it.  The merge reads a row
// whose partials are all NaN as empty; +inf makes it NaN, as NaN rows have to.
__device__ __forceinline__ float part_lse_of(float lse) { return lse != lse ? INFINITY : lse; }

// Split kernel of a 4-bit cache: one CTA per (split, KV head, sequence), as
// fd_split_kernel; each warp takes every fourth token, its lanes the entries
// of the head dimension.
template <int D, int G>
__global__ void __launch_bounds__(kInt4Warps * 32) fd_split_int4_kernel(const Int4DecodeArgs p) {
  const SplitArgs& a = p.a;
  grid_dependency_wait();
  constexpr int VPL = D / 32;
  const int split = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = seq_length(a.seqlens, b, a.max_len);
  const int start = split_first_tile(a, split) * kTile;
  const int end = min(split_first_tile(a, split + 1) * kTile, n);
  const int h0 = kvh * G;
  const int n_parts = (a.n_splits == 1 || (n + kTile - 1) / kTile <= a.tile_q) ? 1 : 2;
  if (start >= end) {
    grid_dependents_launch();
    if (split == 0) {
      const size_t base = (static_cast<size_t>(b) * a.Hq + h0) * D;
      for (int i = threadIdx.x; i < G * D; i += kInt4Warps * 32) a.out[base + i] = __float2bfloat16_rn(0.f);
      if (a.lse && threadIdx.x < G) a.lse[static_cast<size_t>(b) * a.Hq + h0 + threadIdx.x] = -INFINITY;
    }
    return;
  }
  float q[G][VPL], acc[G][VPL], m[G], l[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      q[g][i] = __bfloat162float(a.q[(static_cast<size_t>(b) * a.Hq + h0 + g) * D + lane * VPL + i]);
      acc[g][i] = 0.f;
    }
  }
  for (int t = start + warp; t < end; t += kInt4Warps) {
    int plane = b, row = t;
    if (a.block_table) {
      plane = a.block_table[static_cast<size_t>(b) * a.max_blocks_per_seq + (t >> a.log2_block_size)];
      row = t & (a.block_size - 1);
    }
    float k[VPL], v[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) k[i] = v[i] = 0.f;
    if (plane >= 0 && plane < p.c.planes) {
      const size_t from = int4_row(p.c, plane, kvh, row);
      const uint32_t* rec = reinterpret_cast<const uint32_t*>(p.c.params + from * 16) + lane / 16;
      const uint32_t kr = rec[0], vr = rec[2];
#pragma unroll
      for (int i = 0; i < VPL; i += 2) {
        const uint32_t kc = p.c.k4[from * (D / 2) + (lane * VPL + i) / 2];
        const uint32_t vc = p.c.v4[from * (D / 2) + (lane * VPL + i) / 2];
        k[i] = __fmaf_rn(bf16_lo(kr), static_cast<float>(static_cast<int>(kc & 15u) - 8), bf16_hi(kr));
        k[i + 1] = __fmaf_rn(bf16_lo(kr), static_cast<float>(static_cast<int>(kc >> 4) - 8), bf16_hi(kr));
        v[i] = __fmaf_rn(bf16_lo(vr), static_cast<float>(static_cast<int>(vc & 15u) - 8), bf16_hi(vr));
        v[i + 1] = __fmaf_rn(bf16_lo(vr), static_cast<float>(static_cast<int>(vc >> 4) - 8), bf16_hi(vr));
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) s += q[g][i] * k[i];
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      s *= a.scale_log2;
      const float mn = fmaxf(m[g], s);
      const float mu = mn == -INFINITY ? 0.f : mn;
      const float al = ex2(m[g] - mu), e = ex2(s - mu);
      m[g] = mn;
      l[g] = l[g] * al + e;
#pragma unroll
      for (int i = 0; i < VPL; ++i) acc[g][i] = acc[g][i] * al + e * v[i];
    }
  }
  grid_dependents_launch();
  // Merge of the warps' states.
  __shared__ float s_m[kInt4Warps][G], s_l[kInt4Warps][G], s_o[kInt4Warps][D];
  if (lane == 0) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      s_m[warp][g] = m[g];
      s_l[warp][g] = l[g];
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) s_o[warp][lane * VPL + i] = acc[g][i];
    __syncthreads();
    float M = -INFINITY, L = 0.f, o = 0.f;
    const int d = threadIdx.x;
#pragma unroll
    for (int w = 0; w < kInt4Warps; ++w) M = fmaxf(M, s_m[w][g]);
    const float mu = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int w = 0; w < kInt4Warps; ++w) {
      const float wt = ex2(s_m[w][g] - mu);
      L += wt * s_l[w][g];
      if (d < D) o += wt * s_o[w][d];
    }
    const size_t r = static_cast<size_t>(b) * a.Hq + h0 + g;
    const float lse = (M + log2f(L)) * 0.69314718055994530942f;
    if (n_parts == 1) {
      if (d < D) a.out[r * D + d] = __float2bfloat16_rn(o / L);
      if (a.lse && d == 0) a.lse[r] = lse;
    } else {
      if (d < D) a.part_o[(r * a.n_splits + split) * D + d] = o / L;
      if (d == 0) a.part_lse[r * a.n_splits + split] = part_lse_of(lse);
    }
    __syncthreads();
  }
}

}  // namespace fd
