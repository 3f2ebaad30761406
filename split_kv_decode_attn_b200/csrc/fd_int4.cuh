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
  uint32_t n_rows;           // n_tokens Hkv < 2^31
  uint32_t head_mul;         // x / Hkv = x head_mul >> (31 + head_shift) for x < 2^31
  int head_shift;
  int log2_rows;             // rows = 2^log2_rows, or -1
};

__device__ __forceinline__ uint32_t min2_nan(uint32_t x, uint32_t y) {   // of two bf16
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t max2_nan(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// The codes of eight entries as defined: clamp(rint((x - b) / s), -8, 7) + 8.
__device__ __noinline__ uint32_t int4_divided(uint4 raw, float s, float b) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = __fdiv_rn(__fsub_rn((i & 1) ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]), b), s);
    codes |= static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(rintf(y), -8.f), 7.f)) + 8) << (4 * i);
  }
  return codes;
}

// Quantises the 16 entries that this lane holds of a row (two words of 8 codes,
// entry i in bits 4i .. 4i+3); LPG neighbouring lanes hold a group.  Returns the
// group's record (scale in the low half, bias in the high half).
//   s = bf16((mx - mn) / 15), b = bf16(mn + 8 s),
//   c = clamp(rint((x - b) / s), -8, 7) + 8
// in fp32 (ties to even).  (mx - mn) / 15 is taken as (mx/2 - mn/2) / 7.5 and
// mn + 8 s with one rounding, so that no bf16 input overflows.  A group with
// s = 0 gets the code 8; one with a NaN or an infinity gets s = b = NaN.
//
// A division per entry made this kernel twice as slow as its copies, so the codes
// come from two products with reciprocals just below and just above 1 / s
// (rcp.approx is within 2^-23, they are 2^-22 to either side).  Adding
// M = 1.5 2^23 + 8 to a product rounds it to an integer, ties to even, in the low
// bits of the sum.
//  * Both agree: so does everything between them.
//  * They differ by one at a tie, Q = d / s = k + 1/2, or next to it.  With x and b
//    zero or at least 2^-9 s in size, d is a multiple of 2^-17 s and
//    exact, (k + 1/2) s a multiple of 2^-9 s, and |Q| < 9 puts the two products
//    within 9 (2^-22 + 2^-23 + 2^-24) < 2^-17 of Q: then it is a tie.  The sum of
//    the two results is odd, twice the tie, and beyond 2^24, where fp32 holds only
//    even numbers: the addition itself rounds half to even.  It is exact when they
//    agree, so it is used for all entries.
//    (A smaller entry, |x| < 2^-9 s, comes next to a tie only when -b / s does,
//    within 2^-9 + 2^-17: looking at b saves a look at every entry, 8 us of 34.)
//  * Otherwise (b of that kind, a bias so large that codes have to be clamped, a
//    scale whose reciprocal overflows) the lane divides.
template <int LPG>
__device__ __forceinline__ uint32_t int4_quantise(const uint4 (&raw)[2], uint32_t (&codes)[2]) {
  const uint32_t w[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
  uint32_t lo2 = w[0], hi2 = w[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo2 = min2_nan(lo2, w[i]);
    hi2 = max2_nan(hi2, w[i]);
  }
  // The smallest entry and minus the largest: one minimum for both.
  uint32_t ends = min2_nan(__byte_perm(lo2, hi2 ^ 0x80008000u, 0x5410), __byte_perm(lo2, hi2 ^ 0x80008000u, 0x7632));
#pragma unroll
  for (int off = 1; off < LPG; off <<= 1) ends = min2_nan(ends, __shfl_xor_sync(0xffffffffu, ends, off));
  const float mn = bf16_lo(ends), mx = -bf16_hi(ends);
  const float half_range = __fsub_rn(__fmul_rn(mx, 0.5f), __fmul_rn(mn, 0.5f));
  codes[0] = codes[1] = 0x88888888u;
  if (!(half_range < INFINITY)) return 0x7fc07fc0u;
  // half_range / 7.5: the product with the reciprocal and one correction by its
  // exact residue (Markstein 1990; right for all 2^23 significands), or the
  // division where the residue could underflow.
  constexpr float kInv = 1.f / 7.5f;
  float q = __fmul_rn(half_range, kInv);
  q = __fmaf_rn(__fmaf_rn(-q, 7.5f, half_range), kInv, q);
  if (half_range < 0x1p-90f) q = __fdiv_rn(half_range, 7.5f);
  const float s = round_to_bf16(q);
  const float b = round_to_bf16(__fmaf_rn(8.f, s, mn));
  const uint32_t record = pack_bf16x2(s, b);
  if (!(s > 0.f)) return record;

  constexpr float kM = 12582920.f;                     // 1.5 2^23 + 8
  constexpr uint32_t kBase = 0x4bc00000u * 0x11111111u;   // 2 kM - 16, in every code's place
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  const float below = __fmul_rn(r, 1.f - 0x1p-22f), above = __fmul_rn(r, 1.f + 0x1p-22f);
  auto entry = [&](int i) { return (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]); };
  uint32_t differ = 0;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    uint32_t c = 0;
#pragma unroll
    for (int i = 7; i >= 0; --i) {
      const float d = __fsub_rn(entry(8 * x + i), b);
      const float t0 = __fmaf_rn(d, below, kM), t1 = __fmaf_rn(d, above, kM);
      differ |= __float_as_uint(t0) ^ __float_as_uint(t1);
      c = c * 16u + __float_as_uint(__fadd_rn(t0, t1));
    }
    codes[x] = c - kBase;
  }
  const float y0 = __fmul_rn(__fsub_rn(mn, b), above), y1 = __fmul_rn(__fsub_rn(mx, b), above);
  bool divide = y0 < -8.25f || y1 > 7.25f || s < 0x1p-100f;
  if (differ) {
    const float y = __fmul_rn(b, r), off = fabsf(y - rintf(y));
    divide |= off > 0.5f - 0x1p-8f || (b != 0.f && fabsf(b) < s * 0x1p-9f);
  }
  if (divide) {
    codes[0] = int4_divided(raw[0], s, b);
    codes[1] = int4_divided(raw[1], s, b);
  }
  return record;
}

// D / 16 lanes take the K and the V row of one (token, KV head), so that the
// record leaves as one 16-byte store; rows of whole warps of lanes need neither
// shared memory nor a barrier.  26,313 tokens of 8 heads (D = 128, 138 MB): 28 us,
// 4.9 TB/s, bound by instruction issue (12 per entry; 24 us without the rules for
// ties).  With a division per entry and 64-bit divisions for the addresses it took
// about 50 us.
template <int D>
__global__ void __launch_bounds__(256) fd_append_int4_kernel(const AppendArgs a) {
  constexpr int LPR = D / 16, LPG = LPR / 2;
  const uint32_t at = blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
  const int part = threadIdx.x % LPR;
  const uint32_t unit = min(at, a.n_rows - 1);         // whole warps take part in the shuffles
  const uint32_t token = static_cast<uint32_t>((static_cast<uint64_t>(unit) * a.head_mul) >> (31 + a.head_shift));
  const int head = static_cast<int>(unit - token * a.c.Hkv);
  const uint4* k = reinterpret_cast<const uint4*>(a.k + token * a.k_stride + head * D) + 2 * part;
  const uint4* v = reinterpret_cast<const uint4*>(a.v + token * a.v_stride + head * D) + 2 * part;
  grid_dependency_wait();
  grid_dependents_launch();
  const uint4 kr[2] = {__ldcs(k), __ldcs(k + 1)}, vr[2] = {__ldcs(v), __ldcs(v + 1)};
  const int64_t slot = __ldcg(a.slots + token);
  uint32_t kc[2], vc[2];
  const uint32_t krec = int4_quantise<LPG>(kr, kc), vrec = int4_quantise<LPG>(vr, vc);
  const uint32_t krec1 = __shfl_down_sync(0xffffffffu, krec, LPG), vrec1 = __shfl_down_sync(0xffffffffu, vrec, LPG);
  const uint64_t s = static_cast<uint64_t>(slot);
  if (at >= a.n_rows || s >= static_cast<uint64_t>(a.c.planes) * a.c.rows) return;
  size_t to;
  if (a.c.nhd) {
    to = s * a.c.Hkv + head;
  } else {
    const uint32_t plane = a.log2_rows >= 0 ? static_cast<uint32_t>(s >> a.log2_rows)
                           : s >> 32        ? static_cast<uint32_t>(s / static_cast<uint32_t>(a.c.rows))
                                            : static_cast<uint32_t>(s) / static_cast<uint32_t>(a.c.rows);
    to = s + (static_cast<size_t>(plane) * (a.c.Hkv - 1) + head) * a.c.rows;
  }
  reinterpret_cast<uint2*>(a.c.k4 + to * (D / 2))[part] = make_uint2(kc[0], kc[1]);
  reinterpret_cast<uint2*>(a.c.v4 + to * (D / 2))[part] = make_uint2(vc[0], vc[1]);
  if (part == 0) reinterpret_cast<uint4*>(a.c.params)[to] = make_uint4(krec, krec1, vrec, vrec1);
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

// The 8 codes of a word as the bf16 values they stand for.  128 + c is a bf16
// number with c in its low bits; taking 136 off is exact, and the fused multiply-
// add rounds s (c - 8) + b once.
__device__ __forceinline__ uint4 int4_values(uint32_t codes, uint32_t record) {
  const uint32_t s = __byte_perm(record, record, 0x1010), b = __byte_perm(record, record, 0x3232);
  uint32_t v[4];                                       // entries i and i + 4
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = ((codes >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(v[i]) : "r"(c), "r"(0x43084308u));
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v[i]) : "r"(s), "r"(v[i]), "r"(b));
  }
  return make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                    __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
}

constexpr int kExpandTokens = 64;

// One CTA per 64 tokens of one KV head of one sequence; D / 8 lanes per row, and
// a thread's rows are all requested before the first is used.  26,313 tokens of 8
// heads (D = 128, 138 MB): 22 us, 6.3 TB/s, bound by HBM.  (32 tokens per CTA 25.6
// us, 128 26.7 against 25.4 at 64, all with plain stores; the streaming stores gave
// the rest, as the output leaves the small input in L2 alone.  With conversions
// from integers and a multiply-add per entry in fp32 it took about 50 us.)
template <int D>
__global__ void __launch_bounds__(256) fd_expand_int4_kernel(const ExpandArgs a) {
  grid_dependency_wait();
  grid_dependents_launch();
  constexpr int LPR = D / 8, STEP = 256 / LPR, N = kExpandTokens / STEP;
  const int b = blockIdx.z, head = blockIdx.y;
  const int n = seq_length(a.seqlens, b, a.max_len);
  const int t0 = blockIdx.x * kExpandTokens + threadIdx.x / LPR;
  const int part = threadIdx.x % LPR;
  if (t0 >= n) return;
  int plane[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    plane[i] = b;
    if (a.block_table)
      plane[i] = t0 + i * STEP < n ? __ldcg(a.block_table + static_cast<size_t>(b) * a.max_blocks + ((t0 + i * STEP) >> a.log2_block_size)) : -1;
  }
  uint32_t kc[N], vc[N], kr[N], vr[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int t = t0 + i * STEP;
    kc[i] = vc[i] = kr[i] = vr[i] = 0;                 // a page outside the pool: zeros
    if (t < n && plane[i] >= 0 && plane[i] < a.c.planes) {
      const size_t from = int4_row(a.c, plane[i], head, a.block_table ? t & (a.c.rows - 1) : t);
      const uint32_t* rec = reinterpret_cast<const uint32_t*>(a.c.params + from * 16) + part / (LPR / 2);
      kc[i] = reinterpret_cast<const uint32_t*>(a.c.k4 + from * (D / 2))[part];
      vc[i] = reinterpret_cast<const uint32_t*>(a.c.v4 + from * (D / 2))[part];
      kr[i] = rec[0];
      vr[i] = rec[2];
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int t = t0 + i * STEP;
    if (t >= n) break;
    const size_t to = a.c.nhd ? (static_cast<size_t>(b) * a.max_len + t) * a.c.Hkv + head
                              : (static_cast<size_t>(b) * a.c.Hkv + head) * a.max_len + t;
    __stcs(reinterpret_cast<uint4*>(a.k + to * D) + part, int4_values(kc[i], kr[i]));
    __stcs(reinterpret_cast<uint4*>(a.v + to * D) + part, int4_values(vc[i], vr[i]));
  }
}

// ---------------------------------------------------------------- decode

// A warp streams units of tokens through a ring of its own: it issues its
// copies, waits for them and computes, with no other warp to wait for.
//   WARPS   warps per CTA        CTAS    CTAs per SM the registers allow
//   UNIT    tokens per unit      STAGES  units per ring
template <int WARPS_, int CTAS_, int UNIT_, int STAGES_>
struct Int4Shape {
  static constexpr int WARPS = WARPS_, CTAS = CTAS_, UNIT = UNIT_, STAGES = STAGES_;
};
constexpr float kRescaleLog2 = 8.f;   // a score may pass the reference by 2^8 ...
constexpr float kWeightLog2 = 7.f;    // ... whose own weight is 2^7
constexpr float kBiasRoom = 0x1p-64f;  // a bias of V may pass R by 2^64 (see P V below)

// 1 / x of a power of two within 2^+-126.
__device__ __forceinline__ float power_inverse(float x) { return __uint_as_float(0x7f000000u - __float_as_uint(x)); }

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// 4-D tile load: {byte, head, row, plane}.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* tm, uint32_t bar,
                                            int head, int row, int plane, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(bar), "r"(0), "r"(head), "r"(row), "r"(plane),
      "l"(policy)
      : "memory");
}

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int threads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

template <int N>
__device__ __forceinline__ void set_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Between the CTAs of a cluster: what was written to shared memory before the arrival
// is there for all after the wait (threads that have ended count as arrived).
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// The address of this CTA's `at` in CTA `rank` of the cluster, and loads from there.
__device__ __forceinline__ uint32_t cluster_address(uint32_t at, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
  return r;
}
__device__ __forceinline__ float cluster_load(uint32_t at) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}

template <class T>
__device__ __forceinline__ T smem_at(const uint8_t* p) {
  return *reinterpret_cast<const T*>(p);
}

constexpr int kInt4MaxCluster = 8;    // the portable limit
constexpr int kInt4MaxCtas = 256;     // that the batch is dealt to, a power of two

struct Int4DecodeArgs {
  SplitArgs a;            // part_o [2 ctas heads, G, D] and part_lse [2 ctas heads, G]: see
                          // below; the fields of the split cut, k_scale and v_scale do not apply
  int B;
  int ctas;               // CTAs the batch is dealt to (by_row: not used)
  int groups;             // rows that the cut sees per sequence: KV heads, or eighths of them
  int heads;              // KV heads per row of the cut: 1, or 8 (a warp each)
  bool by_row;            // one cluster per (sequence, KV head), no partial results
  int cluster;            // its CTAs (by_row), at most kInt4MaxCluster
  bool evict_first;       // what is read leaves L2 first
  float scale_m;          // scale log2(e) = scale_m 2^scale_e, scale_m in [1/2, 1]: the
  int scale_e;            // product may be beyond fp32 where the scores are not
};

// D = A B, m16n8k16, f16 inputs, fp32 result.
__device__ __forceinline__ void mma_f16_16816_zero(float (&d)[4], const uint32_t (&a)[4],
                                                   uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// ---- the cut.  The tokens of a (sequence, KV head) row are taken in units of U.
// A row of n units costs n + 1: its end takes about as long as a unit (measured,
// D = 128, G = 8: 1.9-2.0 us a unit, 2.2 us for the end of a row and the start of
// the next).  The costs of all rows, one row after another, are dealt to the CTAs
// in equal ranges, and a CTA's range to its warps.  A warp works through its
// range alone, its copies running ahead over the ends of rows; nothing waits for
// another warp before the range ends.  So the load is even whatever the lengths.
// (One CTA per split of a row, as fd_split_kernel, left a ragged batch of 32 x up
// to 8,192 tokens at 55-58 us whatever the split count and the CTAs' shape.)
// CTA c of C begins at c T / C of the total cost T.
//
// Eight heads at a time (the KV heads a multiple of 8, and a workspace for the
// partial results): the rows of eight neighbouring KV heads, which are equally
// long, are dealt as one, and each warp of a CTA takes its head through the CTA's
// whole range.  The heads' rows of a token-major cache, neighbours of 64 bytes,
// are then read at about the same time (8 x 40,000 tokens in pages of 16 at 32/8
// heads: 42.0 us, 49.4 with the range dealt to the warps; 64 x 4,096 in pages
// of 32 at 64/8: 50.4, 61.8), and no warp's state is merged with another's.
//
// Every warp works the cut out for itself from the lengths, whose first
// kInt4Lens a CTA keeps in shared memory.  Costs stay below 2^31 (checked on the
// host), so that c T / C = c (T / C) + c (T mod C) / C stays in 32 bits.
constexpr int kInt4Lens = 512;

__device__ __forceinline__ int int4_length(const SplitArgs& a, int b) {
  return a.seqlens ? min(max(__ldcg(a.seqlens + b), 0), a.max_len) : a.max_len;
}
__device__ __forceinline__ int int4_length(const SplitArgs& a, const int* lens, int b) {
  return b < kInt4Lens ? lens[b] : int4_length(a, b);
}

struct Int4Cut {
  uint32_t total, ctas;     // cost; CTAs that get any
  __device__ __forceinline__ uint32_t begin(uint32_t c) const {
    return c * (total / ctas) + c * (total % ctas) / ctas;
  }
  // The CTA that holds place x: near x C / T, which is rounded in fp32.
  __device__ __forceinline__ uint32_t holder(uint32_t x) const {
    uint32_t c = min(static_cast<uint32_t>(static_cast<float>(x) * ctas / static_cast<float>(total)), ctas - 1);
    while (begin(c) > x) --c;
    while (begin(c + 1) <= x) ++c;
    return c;
  }
};

// Where a warp stands: unit u of the `units` of row (sequence b, group h of KV
// heads), whose sequence holds n tokens.
struct Int4Walk {
  int b, h, u, units, n;
};

// The place `at` (below the total): u == units at the end of a row.  rows: the
// rows with a token before it.
template <int U>
__device__ __forceinline__ Int4Walk int4_locate(const SplitArgs& a, const int* lens, int B, int groups, int lane,
                                                uint32_t at, uint32_t& rows) {
  uint32_t before = 0, seqs = 0;
  for (int b0 = 0;; b0 += 32) {
    const int n = b0 + lane < B ? int4_length(a, lens, b0 + lane) : 0;
    const int units = (n + U - 1) / U;
    uint32_t sum = n > 0 ? static_cast<uint32_t>(units + 1) * groups : 0u;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, sum, off);
      if (lane >= off) sum += x;
    }
    const unsigned held = __ballot_sync(0xffffffffu, n > 0);
    const unsigned hit = __ballot_sync(0xffffffffu, before + sum > at);
    if (hit || b0 + 32 >= B) {
      const int l = hit ? __ffs(hit) - 1 : 31;
      Int4Walk w;
      w.b = b0 + l;
      w.n = __shfl_sync(0xffffffffu, n, l);
      w.units = __shfl_sync(0xffffffffu, units, l);
      const uint32_t off = at - (before + __shfl_sync(0xffffffffu, sum, l) - (w.units + 1) * groups);
      w.h = static_cast<int>(off / (w.units + 1));
      w.u = static_cast<int>(off) - w.h * (w.units + 1);
      rows = (seqs + __popc(held & ((1u << l) - 1u))) * groups + w.h;
      return w;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
    seqs += __popc(held);
  }
}

// To the next unit; from the last one of a row to the next row that has any.
template <int U>
__device__ __forceinline__ void int4_advance(const SplitArgs& a, const int* lens, int B, int groups, Int4Walk& w) {
  if (++w.u < w.units) return;
  w.u = 0;
  if (++w.h < groups) return;
  w.h = 0;
  do {
    if (++w.b >= B) return;
    w.n = int4_length(a, lens, w.b);
  } while (w.n == 0);
  w.units = (w.n + U - 1) / U;
}

// A state that a warp left: of row b Hkv + h (-1: none), which begins at place
// `begin` of the batch's costs.
struct Int4Piece {
  long long row;
  uint32_t begin, units;
};
static_assert(sizeof(Int4Piece) == 16, "as laid out in shared memory");

// What a warp has to copy: `units` units from where the walk stands.
struct Int4Range {
  Int4Walk from;
  int units;
};
static_assert(sizeof(Int4Range) <= 32, "as laid out in shared memory");

// Registers per thread: 4 copying warps and 8 computing ones share what the CTA
// starts with, 384 x 168 (the host checks that the kernel was built with these).
constexpr int kInt4CopyWarps = 4, kInt4StartRegs = 168, kInt4CopyRegs = 40, kInt4ComputeRegs = 232;

template <int D, int NB, class SH>
struct Int4Smem {
  static constexpr int kUnit = SH::UNIT, kInt4Warps = SH::WARPS, kInt4Stages = SH::STAGES;
  static constexpr int kRowBytes = D / 2;
  static constexpr int kCodeBytes = kUnit * kRowBytes;
  static constexpr int kV = kCodeBytes;                 // offsets within a stage
  static constexpr int kP = 2 * kCodeBytes;
  static constexpr int kStageBytes = 2 * kCodeBytes + kUnit * 16;
  static constexpr int kWarpBytes = kInt4Stages * kStageBytes;
  // V's part of a unit's records, unpacked: vs0 / R, vs1 / R in fp32 per token,
  // then vb0 / R, vb1 / R in bf16.  (K's part, in fp32, takes the records' place.)
  static constexpr int kVRecOffset = kInt4Warps * kWarpBytes;
  static constexpr int kVRecBytes = kUnit * 12;
  // A softmax state (floats): [column][kAccStride] outputs over R, the columns'
  // references and sums, R of both groups.  A warp leaves up to two: that of the row its range
  // begins in, in a place of its own, and that of the row its range ends in, over
  // its drained ring.
  static constexpr int kNcol = NB * 8;
  static constexpr int kAccStride = D + 4;
  static constexpr int kM = kNcol * kAccStride;
  static constexpr int kL = kM + kNcol;
  static constexpr int kR = kL + kNcol;
  static constexpr int kStateFloats = kR + 4;
  static_assert(kStateFloats * 4 <= kWarpBytes, "the state of a warp fits its ring");
  static constexpr int kFirstOffset = kVRecOffset + kInt4Warps * kVRecBytes;
  static constexpr int kRowOffset = kFirstOffset + kInt4Warps * kStateFloats * 4;   // Int4Piece[2 warps]
  static constexpr int kLenOffset = kRowOffset + 2 * kInt4Warps * 16;
  static constexpr int kRangeOffset = kLenOffset + 4 * kInt4Lens;             // Int4Range[warps]
  static constexpr int kBarOffset = kRangeOffset + 32 * kInt4Warps;   // filled, then free, [warps][stages]
  static constexpr int kFreeBars = 8 * kInt4Warps * kInt4Stages;
  static constexpr int kErrorOffset = kBarOffset + 2 * kFreeBars;
  static constexpr int kDynamicBytes = kErrorOffset + 16 + 1024;   // room to align to 1 KB
  static_assert(kDynamicBytes <= 227 * 1024, "shared memory per CTA");
};

// Row of a unit's 16-token block that takes slot s (0..7) of the MMAs, 8..15
// likewise.  A 64-byte code row (D = 128) covers half the banks, chosen by its
// parity, and its two 32-byte groups lie there as the copy's swizzle puts them,
// by bit 2 of the row.  The four rows of slots 4i .. 4i+3 (loads of K) and of
// slots i, i+2, i+4, i+6 (loads of V) are in four different places, so that no
// load has a bank conflict.  The 32-byte rows of D = 64 need no reordering.
template <int D>
__device__ __forceinline__ uint32_t int4_slot_row(uint32_t s) {
  if constexpr (D == 64) return s;
  return ((s & 2) << 1) | ((s & 4) >> 1) | ((s ^ (s >> 2)) & 1);
}

// Offset of byte `col` of code row r (0..7) of a unit; the copy's swizzle (64
// bytes for D = 128, 32 for D = 64) exchanges 16-byte chunks and repeats every
// 8 rows, so that rows r + 8 i are i * kEightRows further.
template <int D>
__device__ __forceinline__ uint32_t int4_code_offset(uint32_t r, uint32_t col) {
  const uint32_t a = r * (D / 2) + col;
  return D == 128 ? a ^ ((r << 3) & 0x30u) : a ^ ((r << 2) & 0x10u);
}

// The copying warps.  Each fills the rings of two computing warps, one per half of
// its lanes, running ahead over the ends of rows: a warp that issued its own copies
// spent 450 cycles of a unit's 3,650 on it, and 950 of 4,200 with two pages per
// unit.
template <int D, class SH, class L>
__device__ __forceinline__ void int4_copy_warp(const Int4DecodeArgs& p, const CUtensorMap* tmK,
                                               const CUtensorMap* tmV, const CUtensorMap* tmP,
                                               uint8_t* smem, const Int4Range* ranges, const int* lens,
                                               int copy_warp, int lane) {
  constexpr int kUnit = SH::UNIT, kStages = SH::STAGES;
  constexpr int kHalf = 32 * kInt4CopyWarps / SH::WARPS;   // lanes per ring
  static_assert(kHalf == 16 && kUnit / 8 <= kHalf, "a lane per page of a unit");
  set_regs_down<kInt4CopyRegs>();
  const SplitArgs& a = p.a;
  const int lbs = a.log2_block_size;
  const bool paged = a.block_size != 0;
  const int pages_per_unit = paged && a.block_size < kUnit ? kUnit >> lbs : 1;
  const int box_rows = kUnit / pages_per_unit;
  // A head-major row's codes are read once and in order.  Token-major ones lie 64
  // bytes between those of other heads, whose warps want the rest of the line.
  uint64_t policy;
  if (p.evict_first)
    policy = policy_evict_first();
  else
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
  const int sub = lane & (kHalf - 1), of = 2 * copy_warp + (lane >> 4);
  const uint32_t ring = smem_u32(smem) + of * L::kWarpBytes;
  const uint32_t bar = smem_u32(smem) + L::kBarOffset + 8 * kStages * of;
  bar_sync(1, (SH::WARPS + kInt4CopyWarps) * 32);
  Int4Walk at = ranges[of].from;
  const int units = ranges[of].units;
  // The page of this lane's box in the next unit (lanes past the boxes: none).
  auto page_at = [&]() {
    const int pg = ((at.u * kUnit) >> lbs) + sub;
    return paged && sub < pages_per_unit && pg < ((at.n + a.block_size - 1) >> lbs)
               ? __ldcg(a.block_table + static_cast<size_t>(at.b) * a.max_blocks_per_seq + pg)
               : 0;
  };
  const int head = p.heads == 1 ? 0 : of;              // within the group
  int issued = 0, stage = 0;
  uint32_t phase = 1;                  // a fresh barrier counts as passed in this phase
  int page = units > 0 ? page_at() : at.b;
  uint64_t since = 0;
  bool failed = false;
  while (__any_sync(0xffffffffu, issued < units && !failed)) {
    const bool more = issued < units && !failed;
    const uint32_t full = bar + 8 * stage;
    // The lanes of a ring go on together: each has seen its stage free, or none goes.
    const unsigned seen = __ballot_sync(0xffffffffu, more && mbar_test(full + L::kFreeBars, phase));
    const bool ready = ((seen >> (lane & kHalf)) & 0xffffu) == 0xffffu;
    if (ready) {
      const int t0 = at.u * kUnit;
      const uint32_t st = ring + stage * L::kStageBytes;
      const int boxes = paged ? min(pages_per_unit, ((at.n + a.block_size - 1) >> lbs) - (t0 >> lbs)) : 1;
      const int row = paged ? t0 & (a.block_size - 1) : t0;
      const int plane = paged ? page : at.b;
      if (sub == 0) mbar_arrive_expect_tx(full, boxes * box_rows * (D + 16));
      __syncwarp(0xffffu << (lane & 16));
      if (sub < boxes) {
        const uint32_t r = sub * box_rows;
        tma_load_4d(st + r * L::kRowBytes, tmK, full, at.h * p.heads + head, row, plane, policy);
        tma_load_4d(st + L::kV + r * L::kRowBytes, tmV, full, at.h * p.heads + head, row, plane, policy);
        tma_load_4d(st + L::kP + r * 16, tmP, full, at.h * p.heads + head, row, plane, policy);
      }
      if (++issued < units) {
        int4_advance<kUnit>(a, lens, p.B, p.groups, at);
        page = page_at();
      }
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
      since = 0;
    } else if (more) {
      const uint64_t now = global_timer_ns();
      if (since == 0) since = now;
      failed = now - since > kWaitLimitNs;
    }
    if (seen == 0) __nanosleep(100);                   // leave the issue slots to the others
    __syncwarp();
  }
  volatile int* cta_error = reinterpret_cast<volatile int*>(smem + L::kErrorOffset);
  if (failed && sub == 0) {
    raise_device_error(1u);
    *cta_error = 1;
  }
  __syncthreads();
  if (!*cta_error || sub != 0) return;
  // After an error copies may be under way that no warp waits for, the last in
  // each stage; none may land when the CTA has gone.
  for (int i = max(issued - kStages, 0); i < issued; ++i)
    if (!mbar_wait(bar + 8 * (i % kStages), (i / kStages) & 1, kWaitLimitNs)) raise_device_error(2u);
}

// A row that a cluster shares: each CTA merges its warps' states, one per warp, into
// one at the start of its (drained) rings, and the entries of the result are dealt to
// the CTAs, which read the states of all.  Two arrivals and a read of the neighbours'
// shared memory take about 1 us where the partial results in device memory and the
// second kernel take 4.4 (64/8 heads, D = 128: 1 x 2,048 tokens 8.0 us against 11.4
// from graph replays; 5 x 3,001, 8/8, D = 64: 9.4 against 12.5).  A unit costs its warp
// about 2 us, the same with fewer warps at work, so that a row gains from more CTAs
// until each warp has one.
template <int D, class L>
__device__ __forceinline__ void int4_cluster_merge(const Int4DecodeArgs& p, uint8_t* smem, const Int4Piece* pieces,
                                                   bool good, int b, int h, int lane) {
  constexpr int kWarps = L::kInt4Warps, kChunks = D / 4;
  const SplitArgs& a = p.a;
  const unsigned held = __ballot_sync(0xffffffffu, lane < kWarps && pieces[2 * min(lane, kWarps - 1)].row >= 0);
  float* own = reinterpret_cast<float*>(smem);         // as a warp's state, kAccStride apart
  const int items = a.G * kChunks;
  if (good) {
    for (int c = threadIdx.x; c < items; c += kWarps * 32) {
      const int hd = c / kChunks, d = (c % kChunks) * 4;
      const int group = d / (D / 2);
      const float* states = reinterpret_cast<const float*>(smem + L::kFirstOffset);
      float m[kWarps], r[kWarps], M = -INFINITY, R = 0x1p-126f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        m[k] = (held >> k) & 1u ? states[k * L::kStateFloats + L::kM + hd] : -INFINITY;
        r[k] = (held >> k) & 1u ? states[k * L::kStateFloats + L::kR + group] : 0.f;
        M = fmaxf(M, m[k]);
        R = fmaxf(R, r[k]);
      }
      const float inv_r = power_inverse(R);
      float l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kWarps; ++k)
        if ((held >> k) & 1u) {
          const float wt = M == -INFINITY ? 0.f : ex2(m[k] - M), wr = wt * (r[k] * inv_r);
          const float4 v = *reinterpret_cast<const float4*>(states + k * L::kStateFloats + hd * L::kAccStride + d);
          l += wt * states[k * L::kStateFloats + L::kL + hd];
          o.x += wr * v.x;
          o.y += wr * v.y;
          o.z += wr * v.z;
          o.w += wr * v.w;
        }
      *reinterpret_cast<float4*>(own + hd * L::kAccStride + d) = o;
      if (d == 0) {
        own[L::kM + hd] = M;
        own[L::kL + hd] = l;
      }
      if (hd == 0 && d % (D / 2) == 0) own[L::kR + group] = R;
    }
  }
  cluster_arrive();
  cluster_wait();
  const int share = (items + p.cluster - 1) / p.cluster;
  const int first = static_cast<int>(blockIdx.x % p.cluster) * share;
  const uint32_t base = smem_u32(smem);
  for (int c = first + threadIdx.x; good && c < min(first + share, items); c += kWarps * 32) {
    const int hd = c / kChunks, d = (c % kChunks) * 4;
    const int group = d / (D / 2);
    float m[kInt4MaxCluster], l[kInt4MaxCluster], r[kInt4MaxCluster], M = -INFINITY, R = 0x1p-126f, sum = 0.f;
    float4 v[kInt4MaxCluster], o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kInt4MaxCluster; ++k)
      if (k < p.cluster) {
        const uint32_t at = cluster_address(base, k);
        m[k] = cluster_load(at + 4 * (L::kM + hd));
        l[k] = cluster_load(at + 4 * (L::kL + hd));
        r[k] = cluster_load(at + 4 * (L::kR + group));
        v[k] = cluster_load4(at + 4 * (hd * L::kAccStride + d));
        M = fmaxf(M, m[k]);
        R = fmaxf(R, r[k]);
      }
    const float inv_r = power_inverse(R);
#pragma unroll
    for (int k = 0; k < kInt4MaxCluster; ++k)
      if (k < p.cluster) {
        const float wt = M == -INFINITY ? 0.f : ex2(m[k] - M), wr = wt * (r[k] * inv_r);
        sum += wt * l[k];
        o.x += wr * v[k].x;
        o.y += wr * v[k].y;
        o.z += wr * v[k].z;
        o.w += wr * v[k].w;
      }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const size_t orow = static_cast<size_t>(b) * a.Hq + h * a.G + hd;
    *reinterpret_cast<uint2*>(a.out + orow * D + d) =
        make_uint2(pack_bf16x2(o.x * inv * R, o.y * inv * R), pack_bf16x2(o.z * inv * R, o.w * inv * R));
    if (d == 0 && a.lse) a.lse[orow] = (M + log2f(sum)) * 0.69314718055994530942f;
  }
  cluster_arrive();                                    // a CTA's memory stays until all have read it
  cluster_wait();
}

// Decode attention over a 4-bit cache.  A row that lies within a warp's range is
// finished by the warp, one within a CTA's by the CTA; of a row that goes over
// the end of CTA c's range each CTA leaves one partial result (with eight heads at
// a time one per head), at index 2 c of part_o and part_lse if the row began
// before the CTA's range (or with it), otherwise at 2 c + 1, and
// fd_combine_int4_kernel merges them.
//
// No code is converted.  A nibble in the low four bits of a half word is the f16
// subnormal c 2^-24 as it stands, one in the next four bits c 2^-20, which the
// tensor cores multiply as they are: masks and shifts unpack the codes, 5 operations per 8
// codes of K and 6 of V (whose pairs run along the tokens, so that two tokens'
// words are merged first).  The e4m3 reading of a nibble, c 2^-9, takes 3, but
// mma.sync spends 6 conversions on each e4m3 instruction here (measured: 105 a
// unit, and 38.0 us against 29.7 us at 64K tokens of the CodeLlama-34B heads).
// What it costs: a subnormal's products are aligned as if it were 2^-14.  Beside a
// product 8 c w of one MMA another of c w 2^-16 is lost (measured) where c is 2^-24, of
// c w 2^-20 where it is 2^-20, and of c w 2^-21, fp32's own end, from 2^-18 on.  So a code
// step counts to 2^-15 of the largest factor of its 16: weights within 2^5 of the
// largest, and entries of q within 2^8, are taken exactly.  (Codes at 2^-20 alone would
// take 64 more shifts a unit.)
// Scores.  S^T = c q^T on m16n8k16 f16 MMAs (16 tokens by up to 8 heads), one
// fp32 sum per group of channels.  q is scaled by a power of two that brings its
// largest entry to [2^14, 2^15), for the channels in odd nibbles 2^4 less, and
// enters exactly down to 2^-24 of the largest.  Then, per token,
//   t = ks0 S0 + ks1 S1 + (kb0 - 8 ks0) sum_0(q) + (kb1 - 8 ks1) sum_1(q),
// so that no scale touches an entry; the sum starts at minus the reference.
// P V.  O^T += c^T w on the same MMAs, w = f16(p vs / R) with R a power of
// two above every |vs| (and 2^-64 of every |vb|) that the warp has seen: f16's 11
// bits for V of any size.  One more MMA per group sums 8 w as the tensor core sees
// it, which the end takes off: c - 8, with no rounding of w to f16 left in it.  The
// biases' part sum_j p_j vb_j / R is summed in fp32 beside it; the factor R comes
// in once the row's sum is divided by that of the weights, so that nothing on the
// way is larger than the result.  (1 x 65,536 tokens at 64/8 heads 25.3 us, 25.0
// with the plain sums, which overflowed from |V| = 1e31 on.)
// The running maximum is only moved when a score passes it by 2^8 (a vote per
// unit in place of shuffles), and the weights are 2^7 p, so that they use f16's
// range: up to 2^15, and down to 2^-31 of the largest before one is lost.
template <int D, int NB, class SH>
__global__ void __launch_bounds__((SH::WARPS + kInt4CopyWarps) * 32, SH::CTAS)
    fd_split_int4_kernel(const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV,
                         const __grid_constant__ CUtensorMap tmP, const Int4DecodeArgs p) {
  using L = Int4Smem<D, NB, SH>;
  constexpr int kUnit = SH::UNIT, kInt4Warps = SH::WARPS, kInt4Stages = SH::STAGES;
  constexpr int BB = kUnit / 16;      // 16-token blocks per unit
  constexpr int KW = D / 64;          // words of K's codes a lane holds per row and group
  constexpr int MB = D / 32;          // m-blocks of a group's P V MMA
  const SplitArgs& a = p.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  // The warp's number from a shuffle: the compiler then keeps what follows from
  // it, the addresses of copies and barriers, in uniform registers.
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int g = lane >> 2, t4 = lane & 3;
  uint8_t* ring = smem + warp * L::kWarpBytes;
  const uint32_t ring_at = smem_u32(ring);
  const uint32_t bar = smem_u32(smem) + L::kBarOffset + 8 * kInt4Stages * warp;
  volatile int* cta_error = reinterpret_cast<volatile int*>(smem + L::kErrorOffset);
  Int4Piece* pieces = reinterpret_cast<Int4Piece*>(smem + L::kRowOffset);
  const int B = p.B;

  static_assert(SH::CTAS == 1 && kInt4Warps == 8 &&
                    (kInt4Warps + kInt4CopyWarps) * kInt4StartRegs ==
                        kInt4Warps * kInt4ComputeRegs + kInt4CopyWarps * kInt4CopyRegs,
                "the warps' shares are what the CTA starts with");
  if (lane == 0 && warp < kInt4Warps) {
    for (int s = 0; s < kInt4Stages; ++s) {
      mbar_init(bar + 8 * s, 1);
      mbar_init(bar + L::kFreeBars + 8 * s, 1);
    }
    fence_mbar_init();
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
    prefetch_tensormap(&tmP);
    pieces[2 * warp].row = pieces[2 * warp + 1].row = -1;
  }
  if (threadIdx.x == 0) *cta_error = 0;

  __syncthreads();

  grid_dependency_wait();

  // The lengths, and from them the range of this CTA and this warp's part of it.
  // (Working it out ahead of the wait on the lengths as they stood, to pull the
  // first units into L2, and again if they had changed, gained 0.7 us on batches
  // of a few short sequences and lost 0.8-1.4 us on every larger one.)
  int* lens = reinterpret_cast<int*>(smem + L::kLenOffset);
  Int4Walk cur;
  Int4Cut cut{0u, 0u};
  uint32_t cta_begin = 0, cta_end = 0;
  uint32_t row_begin = 0;              // where cur's row begins
  int mine = 0;
  if (!p.by_row) {
    for (int b = threadIdx.x; b < min(B, kInt4Lens); b += (kInt4Warps + kInt4CopyWarps) * 32)
      lens[b] = int4_length(a, b);
    __syncthreads();
  }
  Int4Range* ranges = reinterpret_cast<Int4Range*>(smem + L::kRangeOffset);
  if (warp >= kInt4Warps) {
    int4_copy_warp<D, SH, L>(p, &tmK, &tmV, &tmP, smem, ranges, lens, warp - kInt4Warps, lane);
    return;
  }

  if (p.by_row) {
    cur.b = blockIdx.y;
    cur.h = blockIdx.x / p.cluster;
    cur.n = int4_length(a, cur.b);
    cur.units = (cur.n + kUnit - 1) / kUnit;
    cta_end = cur.units;
    const int warps = kInt4Warps * p.cluster, at = static_cast<int>(blockIdx.x % p.cluster) * kInt4Warps + warp;
    cur.u = static_cast<int>(static_cast<long long>(cur.units) * at / warps);
    mine = static_cast<int>(static_cast<long long>(cur.units) * (at + 1) / warps) - cur.u;
  } else {
    uint32_t total = 0, rows = 0;
    for (int b = lane; b < B; b += 32) {
      const int n = int4_length(a, lens, b);
      if (n > 0) {
        total += static_cast<uint32_t>((n + kUnit - 1) / kUnit + 1) * p.groups;
        rows += p.groups;
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      total += __shfl_xor_sync(0xffffffffu, total, off);
      rows += __shfl_xor_sync(0xffffffffu, rows, off);
    }
    cut = Int4Cut{total, min(static_cast<uint32_t>(p.ctas), total)};
    if (blockIdx.x < cut.ctas) {
      cta_begin = cut.begin(blockIdx.x);
      cta_end = cut.begin(blockIdx.x + 1);
    }
    const uint32_t cost = cta_end - cta_begin, each = cost / kInt4Warps, rest = cost % kInt4Warps;
    const uint32_t lo = p.heads > 1 ? cta_begin : cta_begin + each * warp + rest * warp / kInt4Warps;
    const uint32_t hi =
        p.heads > 1 ? cta_end : cta_begin + each * (warp + 1) + rest * (warp + 1) / kInt4Warps;
    if (lo < hi) {
      // Units before a place: its cost less the rows before it.
      uint32_t rows_lo, rows_hi = rows;
      cur = int4_locate<kUnit>(a, lens, B, p.groups, lane, lo, rows_lo);
      if (hi < total) int4_locate<kUnit>(a, lens, B, p.groups, lane, hi, rows_hi);
      mine = static_cast<int>((hi - rows_hi) - (lo - rows_lo));
      row_begin = lo - cur.u;
      if (cur.u == cur.units && mine > 0) {            // the end of a row: begin with the next
        row_begin += cur.units + 1;
        --cur.u;
        int4_advance<kUnit>(a, lens, B, p.groups, cur);
      }
    }
  }

  if (lane == 0) ranges[warp] = Int4Range{cur, mine};
  __syncwarp();
  bar_arrive(1, (kInt4Warps + kInt4CopyWarps) * 32);    // to the copying warps
  set_regs_up<kInt4ComputeRegs>();

  const int head = p.heads == 1 ? 0 : warp;             // within the group
  // Word w of q of lane t4 in group h holds channels h D/2 + t4 D/8 + 8 w ..
  uint4 raw[NB][2][KW];
  auto load_q = [&]() {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const bool live = nb * 8 + g < a.G;
      const __nv_bfloat16* qrow =
          a.q + (static_cast<size_t>(cur.b) * a.Hq + (cur.h * p.heads + head) * a.G + (live ? nb * 8 + g : 0)) * D;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          raw[nb][h][w] = *reinterpret_cast<const uint4*>(qrow + h * (D / 2) + t4 * (D / 8) + 8 * w);
          if (!live) raw[nb][h][w] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
  };
  if (mine > 0) load_q();

  // Offsets within a unit of this lane's loads: codes of K (slot g), of V
  // (slots 2 t4 and 2 t4 + 1) and the records of slot g.
  constexpr uint32_t kEight = 8 * L::kRowBytes;        // 8 rows further
  const uint32_t k_row = int4_slot_row<D>(g);
  uint32_t k_at[2], v_at[2][2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    k_at[h] = int4_code_offset<D>(k_row, h * (D / 4) + t4 * (D / 16));
    v_at[h][0] = L::kV + int4_code_offset<D>(int4_slot_row<D>(2 * t4), h * (D / 4) + g * (D / 32));
    v_at[h][1] = L::kV + int4_code_offset<D>(int4_slot_row<D>(2 * t4 + 1), h * (D / 4) + g * (D / 32));
  }
  const uint32_t k_rec = L::kP + k_row * 16;           // within the unit
  uint8_t* v_recs = smem + L::kVRecOffset + warp * L::kVRecBytes;
  const uint8_t* vs_rec = v_recs + k_row * 8;
  const uint8_t* vb_rec = v_recs + kUnit * 8 + k_row * 4;
  bool failed = false;
  uint32_t stage = 0, phase = 0;

  for (int done = 0; done < mine && !failed;) {        // the rows of the range
  const int u_first = cur.u;
  const int count = min(cur.units - cur.u, mine - done);
  // ---- q in f16, in the order of K's codes: k-step s of a word takes nibbles
  // 2s, 2s+4 (slots 2 t4, 2 t4 + 1) and 2s+1, 2s+5 (slots 2 t4 + 8, + 9).
  uint32_t qf[NB][2][KW][2][2];
  float sq[NB][2][2], scl[NB][2];      // per column 2 t4 + c: sum of q per group, scale
  int exps[NB], top_exp = -1024;       // of lane g's heads: the power of two in scl
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    float mx = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        const uint32_t x[4] = {raw[nb][h][w].x, raw[nb][h][w].y, raw[nb][h][w].z, raw[nb][h][w].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(x[i])), fabsf(bf16_hi(x[i]))));
      }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // mx 2^-e in [1, 2) (rows below 2^-112 stay below 1).
    const int e = min(max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -112), 127);
    const float down = __uint_as_float(static_cast<uint32_t>(141 - e) << 23);    // 2^(14 - e)
    float sum[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      sum[h] = 0.f;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        const uint32_t x[4] = {raw[nb][h][w].x, raw[nb][h][w].y, raw[nb][h][w].z, raw[nb][h][w].w};
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          y[i] = ((i & 1) ? bf16_hi(x[i / 2]) : bf16_lo(x[i / 2])) * down;
          sum[h] += y[i];
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          qf[nb][h][w][s][0] = pack_f16x2(y[2 * s], y[2 * s + 4]);
          qf[nb][h][w][s][1] = pack_f16x2(y[2 * s + 1] * 0.0625f, y[2 * s + 5] * 0.0625f);
        }
      }
#pragma unroll
      for (int off = 1; off < 4; off <<= 1) sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], off);
    }
    // S holds q 2^(14 - e) (c 2^-24): the sums of q take the same factor, and
    // the scale its inverse, 2^(e + 10).
    exps[nb] = e + 10 + p.scale_e;
    if (mx > 0.f) top_exp = max(top_exp, exps[nb]);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h) sq[nb][h][c] = __shfl_sync(0xffffffffu, sum[h] * 0x1p-24f, 8 * t4 + 4 * c);
  }
  // Where the largest of the heads' powers is not within 2^+-100 (q next to bf16's ends),
  // K takes the rest of it.
  top_exp = __reduce_max_sync(0xffffffffu, top_exp);
  const int k_exp = top_exp == -1024 ? 0 : min(max(top_exp - min(max(top_exp, -100), 100), -126), 127);
  const uint32_t k_power = static_cast<uint32_t>(127 + k_exp) * 0x00800080u;     // 2^k_exp, two bf16
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const float sc = p.scale_m * __uint_as_float(static_cast<uint32_t>(127 + min(max(exps[nb] - k_exp, -125), 127)) << 23);
#pragma unroll
    for (int c = 0; c < 2; ++c) scl[nb][c] = __shfl_sync(0xffffffffu, sc, 8 * t4 + 4 * c);   // a lane of head 2 t4 + c
  }

  // ---- softmax state.  Per column: the reference, a t whose weight is 2^7, and how far
  // beyond it t may be before it moves.  t is taken relative to it (a weight is
  // 2^(t scl + 7)), so that no weight passes 2^15 however large the scores are: the
  // difference of two rounded numbers of 2^23 and more would.
  float ref[NB][2], bound[NB][2], l_run[NB][2], bias[NB][2][2];
  float acc[NB][2][MB][4], eight[NB][4];              // c w; 8 w of group 0 and of group 1
  float inv_r[2] = {0x1p126f, 0x1p126f};              // 1 / R per group
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      bound[nb][c] = -INFINITY;
      ref[nb][c] = l_run[nb][c] = bias[nb][0][c] = bias[nb][1][c] = 0.f;
    }
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      eight[nb][i] = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < MB; ++j) acc[nb][h][j][i] = 0.f;
    }

  for (int i = 0; i < count; ++i) {
    uint8_t* st = ring + stage * L::kStageBytes;
    const bool ok = mbar_wait(bar + 8 * stage, phase, kWaitLimitNs);
    if (!__all_sync(0xffffffffu, ok)) {
      failed = true;
      break;
    }
    const int valid = cur.n - (u_first + i) * kUnit;   // tokens of the unit that count

    // Records unpacked, one token per lane and 32 tokens: K's as ks0, kb0 - 8 ks0,
    // ks1, kb1 - 8 ks1 in fp32 over the record, V's beside the ring; zeros for a
    // token that does not count (its record and codes may be anything).  The four
    // lanes of a token read them afterwards: unpacking there took 29 more
    // instructions per 32 tokens.
    {
      uint4 rec[kUnit / 32];
      float vtop[2] = {0.f, 0.f}, btop[2] = {0.f, 0.f};
#pragma unroll
      for (int x = 0; x < kUnit / 32; ++x) {
        rec[x] = smem_at<uint4>(st + L::kP + (32 * x + lane) * 16);
        if (32 * x + lane >= valid) rec[x] = make_uint4(0u, 0u, 0u, 0u);
        vtop[0] = fmaxf(vtop[0], fabsf(bf16_lo(rec[x].z)));
        vtop[1] = fmaxf(vtop[1], fabsf(bf16_lo(rec[x].w)));
        // The bias is the high half; as fp32 the word is at most a bf16 step larger.
        btop[0] = fmaxf(btop[0], fabsf(__uint_as_float(rec[x].z)));
        btop[1] = fmaxf(btop[1], fabsf(__uint_as_float(rec[x].w)));
      }
      if (__any_sync(0xffffffffu, fmaxf(fmaxf(vtop[0] * inv_r[0], vtop[1] * inv_r[1]),
                                        fmaxf(btop[0] * (inv_r[0] * kBiasRoom), btop[1] * (inv_r[1] * kBiasRoom))) > 1.f)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          vtop[h] = fmaxf(vtop[h], btop[h] * kBiasRoom);
#pragma unroll
          for (int off = 1; off < 32; off <<= 1) vtop[h] = fmaxf(vtop[h], __shfl_xor_sync(0xffffffffu, vtop[h], off));
          if (vtop[h] * inv_r[h] > 1.f) {
            // R becomes the power of two above vtop (scales are below 2^126).
            const uint32_t e = min((__float_as_uint(vtop[h]) >> 23) + 1u, 253u);
            const float r = __uint_as_float((254u - e) << 23), keep = r / inv_r[h];   // old R / new R
            inv_r[h] = r;
            if (i == 0) continue;                      // nothing is summed yet
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              bias[nb][h][0] *= keep;
              bias[nb][h][1] *= keep;
              eight[nb][2 * h] *= keep;
              eight[nb][2 * h + 1] *= keep;
#pragma unroll
              for (int j = 0; j < MB; ++j)
#pragma unroll
                for (int x = 0; x < 4; ++x) acc[nb][h][j][x] *= keep;
            }
          }
        }
      }
      const uint32_t inv_r2 = __byte_perm(__float_as_uint(inv_r[0]), __float_as_uint(inv_r[1]), 0x7632);
#pragma unroll
      for (int x = 0; x < kUnit / 32; ++x) {
        const uint32_t k0 = mul_bf16x2(rec[x].x, k_power), k1 = mul_bf16x2(rec[x].y, k_power);
        const float ks0 = bf16_lo(k0), ks1 = bf16_lo(k1);
        const int at = 32 * x + lane;
        *reinterpret_cast<float4*>(st + L::kP + at * 16) =
            make_float4(ks0, fmaf(-8.f, ks0, bf16_hi(k0)), ks1, fmaf(-8.f, ks1, bf16_hi(k1)));
        *reinterpret_cast<float2*>(v_recs + at * 8) =
            make_float2(bf16_lo(rec[x].z) * inv_r[0], bf16_lo(rec[x].w) * inv_r[1]);
        *reinterpret_cast<uint32_t*>(v_recs + kUnit * 8 + at * 4) =
            mul_bf16x2(__byte_perm(rec[x].z, rec[x].w, 0x7632), inv_r2);
      }
      __syncwarp();
    }

    // Scores less the reference, t[..][row][column].
    float t[NB][BB][2][2], scs[BB][NB][2][4];
#pragma unroll
    for (int bb = 0; bb < BB; ++bb) {
      auto& sc = scs[bb];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w[2][KW];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint8_t* at = st + k_at[h] + (2 * bb + r) * kEight;
          if constexpr (D == 128) {
            const uint2 v = smem_at<uint2>(at);
            w[r][0] = v.x;
            w[r][1] = v.y;
          } else {
            w[r][0] = smem_at<uint32_t>(at);
          }
        }
#pragma unroll
        for (int k = 0; k < KW; ++k)
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const uint32_t y0 = w[0][k] >> (8 * s), y1 = w[1][k] >> (8 * s);
            const uint32_t af[4] = {y0 & 0x000f000fu, y1 & 0x000f000fu, y0 & 0x00f000f0u, y1 & 0x00f000f0u};
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              if (k == 0 && s == 0)
                mma_f16_16816_zero(sc[nb][h], af, qf[nb][h][k][s][0], qf[nb][h][k][s][1]);
              else
                mma_f16_16816(sc[nb][h], af, qf[nb][h][k][s][0], qf[nb][h][k][s][1]);
            }
          }
      }
    }
#pragma unroll
    for (int bb = 0; bb < BB; ++bb) {
      auto& sc = scs[bb];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float4 rec = smem_at<float4>(st + k_rec + (16 * bb + 8 * r) * 16);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x = fmaf(rec.y, sq[nb][0][c], -ref[nb][c]);
            x = fmaf(rec.w, sq[nb][1][c], x);
            x = fmaf(rec.x, sc[nb][0][2 * r + c], x);
            t[nb][bb][r][c] = fmaf(rec.z, sc[nb][1][2 * r + c], x);
          }
      }
    }
    if (valid < kUnit) {
#pragma unroll
      for (int bb = 0; bb < BB; ++bb)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (16 * bb + 8 * r + static_cast<int>(k_row) >= valid) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) t[nb][bb][r][0] = t[nb][bb][r][1] = -INFINITY;
          }
    }

    // Does a score pass its bound?
    float top[NB][2];
    bool move = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        top[nb][c] = -INFINITY;
#pragma unroll
        for (int bb = 0; bb < BB; ++bb) top[nb][c] = fmaxf(top[nb][c], fmaxf(t[nb][bb][0][c], t[nb][bb][1][c]));
        move |= top[nb][c] > bound[nb][c];
      }
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1)
            top[nb][c] = fmaxf(top[nb][c], __shfl_xor_sync(0xffffffffu, top[nb][c], off));
          if (top[nb][c] > bound[nb][c]) {
            const float al = bound[nb][c] == -INFINITY ? 0.f : ex2(-top[nb][c] * scl[nb][c]);
            ref[nb][c] += top[nb][c];
            bound[nb][c] = fminf(kRescaleLog2 / scl[nb][c], 3e38f);
#pragma unroll
            for (int bb = 0; bb < BB; ++bb) {
              t[nb][bb][0][c] -= top[nb][c];
              t[nb][bb][1][c] -= top[nb][c];
            }
            if (i == 0) continue;
            l_run[nb][c] *= al;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              bias[nb][h][c] *= al;
              eight[nb][2 * h + c] *= al;
#pragma unroll
              for (int j = 0; j < MB; ++j) {
                acc[nb][h][j][c] *= al;
                acc[nb][h][j][c + 2] *= al;
              }
            }
          }
        }
    }

    // Weights, and P V for the 16 tokens of each block.
    uint32_t pbs[BB][NB][2][2];    // [group][slots 0-7, 8-15]
#pragma unroll
    for (int bb = 0; bb < BB; ++bb) {
      auto& pb = pbs[bb];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float2 vs = smem_at<float2>(vs_rec + (16 * bb + 8 * r) * 8);
        const uint32_t vb = smem_at<uint32_t>(vb_rec + (16 * bb + 8 * r) * 4);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float e[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            e[c] = ex2(fmaf(t[nb][bb][r][c], scl[nb][c], kWeightLog2));
            l_run[nb][c] += e[c];
            bias[nb][0][c] = fmaf(e[c], bf16_lo(vb), bias[nb][0][c]);
            bias[nb][1][c] = fmaf(e[c], bf16_hi(vb), bias[nb][1][c]);
          }
          pb[nb][0][r] = movmatrix_trans(pack_f16x2(e[0] * vs.x, e[1] * vs.x));
          pb[nb][1][r] = movmatrix_trans(pack_f16x2(e[0] * vs.y, e[1] * vs.y));
        }
      }
    }
#pragma unroll
    for (int bb = 0; bb < BB; ++bb) {
      auto& pb = pbs[bb];
      // Slots 2 t4, 2 t4 + 1 and 8 more: this lane's tokens in V.
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t x[2][2];          // [slots 0-7, 8-15][low, high half of the words]: two tokens' halves
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint8_t* a0 = st + v_at[h][0] + (2 * bb + r) * kEight;
          const uint8_t* a1 = st + v_at[h][1] + (2 * bb + r) * kEight;
          if constexpr (D == 128) {
            const uint32_t w0 = smem_at<uint32_t>(a0), w1 = smem_at<uint32_t>(a1);
            x[r][0] = __byte_perm(w0, w1, 0x5410);
            x[r][1] = __byte_perm(w0, w1, 0x7632);
          } else {
            x[r][0] = __byte_perm(smem_at<uint16_t>(a0), smem_at<uint16_t>(a1), 0x5410);
            x[r][1] = 0u;
          }
        }
        // Nibbles 2j and 2j + 1 of the two tokens' halves, as f16 subnormals.
#pragma unroll
        for (int j = 0; j < MB; ++j) {
          const uint32_t y0 = x[0][j / 2] >> (8 * (j & 1)), y1 = x[1][j / 2] >> (8 * (j & 1));
          const uint32_t vf[4] = {y0 & 0x000f000fu, y0 & 0x00f000f0u, y1 & 0x000f000fu, y1 & 0x00f000f0u};
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma_f16_16816(acc[nb][h][j], vf, pb[nb][h][0], pb[nb][h][1]);
        }
        // The code 8 in 8 rows: sums of 8 w, group 0 in rows 0-7, group 1 in 8-15.
        const uint32_t v8[4] = {h == 0 ? 0x00080008u : 0u, h == 1 ? 0x00080008u : 0u,
                                h == 0 ? 0x00080008u : 0u, h == 1 ? 0x00080008u : 0u};
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) mma_f16_16816(eight[nb], v8, pb[nb][h][0], pb[nb][h][1]);
      }
    }
    // The stage is read (and its records were written to): it may be refilled.
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar + L::kFreeBars + 8 * stage);
    if (++stage == kInt4Stages) {
      stage = 0;
      phase ^= 1;
    }
  }
  if (failed) break;

  // ---- the row's end within the range.  Row g of m-block j of group h is entry
  // h D/2 + g D/16 + 2 j, row g + 8 the next one.
  const bool whole = u_first == 0 && count == cur.units && p.cluster == 1;
  const bool is_first = done == 0;
  float* f = reinterpret_cast<float*>(is_first ? smem + L::kFirstOffset + warp * L::kStateFloats * 4 : ring);
  if (!whole && !is_first) __syncwarp();               // the ring is drained, and read by every lane
  const bool alone = p.heads > 1;                      // no other warp of the CTA has this row
  const size_t part = (2 * static_cast<size_t>(blockIdx.x) + (row_begin > cta_begin ? 1 : 0)) * p.heads + head;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        l_run[nb][c] += __shfl_xor_sync(0xffffffffu, l_run[nb][c], off);
        bias[nb][0][c] += __shfl_xor_sync(0xffffffffu, bias[nb][0][c], off);
        bias[nb][1][c] += __shfl_xor_sync(0xffffffffu, bias[nb][1][c], off);
      }
      const int col = nb * 8 + 2 * t4 + c;
      const size_t orow = static_cast<size_t>(cur.b) * a.Hq + (cur.h * p.heads + head) * a.G + col;
      const size_t prow = part * a.G + col;
      const bool state = !whole && !alone;
      const float inv = l_run[nb][c] == 0.f ? 0.f : 1.f / l_run[nb][c];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float r = power_inverse(inv_r[h]);
        const float w8 = eight[nb][2 * h + c];
        const int d = h * (D / 2) + g * (D / 16);
        float o[2 * MB];
#pragma unroll
        for (int j = 0; j < MB; ++j) {
          o[2 * j] = fmaf(acc[nb][h][j][c] - w8, 0x1p24f, bias[nb][h][c]);
          o[2 * j + 1] = fmaf(acc[nb][h][j][c + 2] - 16.f * w8, 0x1p20f, bias[nb][h][c]);
        }
        if (state) {
#pragma unroll
          for (int j = 0; j < 2 * MB; j += 4)
            *reinterpret_cast<float4*>(f + col * L::kAccStride + d + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
        } else if (!whole) {
          if (col < a.G)
#pragma unroll
            for (int j = 0; j < 2 * MB; j += 4)
              *reinterpret_cast<float4*>(a.part_o + prow * D + d + j) =
                  make_float4(o[j] * inv * r, o[j + 1] * inv * r, o[j + 2] * inv * r, o[j + 3] * inv * r);
        } else if (col < a.G) {
          uint32_t w[MB];
#pragma unroll
          for (int j = 0; j < MB; ++j) w[j] = pack_bf16x2(o[2 * j] * inv * r, o[2 * j + 1] * inv * r);
          if constexpr (MB == 4)
            *reinterpret_cast<uint4*>(a.out + orow * D + d) = make_uint4(w[0], w[1], w[2], w[3]);
          else
            *reinterpret_cast<uint2*>(a.out + orow * D + d) = make_uint2(w[0], w[1]);
        }
      }
      if (g == 0) {
        const float at0 = fmaf(ref[nb][c], scl[nb][c], -kWeightLog2);     // the score of weight 1
        const float lse = (at0 + log2f(l_run[nb][c])) * 0.69314718055994530942f;
        if (state) {
          f[L::kM + col] = l_run[nb][c] == 0.f ? -INFINITY : at0;
          f[L::kL + col] = l_run[nb][c];
        } else if (!whole) {
          if (col < a.G) a.part_lse[prow] = lse;
        } else if (col < a.G && a.lse) {
          a.lse[orow] = lse;
        }
      }
    }
  if (!whole && !alone && lane == 0) {
    Int4Piece& pc = pieces[2 * warp + (is_first ? 0 : 1)];
    pc.row = static_cast<long long>(cur.b) * a.Hkv + cur.h;
    pc.begin = row_begin;
    pc.units = cur.units;
    f[L::kR] = power_inverse(inv_r[0]);
    f[L::kR + 1] = power_inverse(inv_r[1]);
  }
  done += count;
  if (done < mine) {
    row_begin += cur.units + 1;
    cur.u += count - 1;
    int4_advance<kUnit>(a, lens, B, p.groups, cur);
    load_q();
  }
  }
  grid_dependents_launch();
  if (failed && lane == 0) {
    raise_device_error(1u);
    *cta_error = 1;
  }
  // Sequences without a token belong to no range.
  if (!p.by_row || cta_end == 0) {
    for (int b = p.by_row ? blockIdx.y : blockIdx.x; b < B; b += p.by_row ? B : gridDim.x) {
      if ((p.by_row ? cur.n : int4_length(a, lens, b)) > 0) continue;
      const int rows = p.by_row ? a.G : a.Hq;
      const size_t row = static_cast<size_t>(b) * a.Hq + (p.by_row ? blockIdx.x / p.cluster * a.G : 0);
      for (int i = threadIdx.x; i < rows * D; i += kInt4Warps * 32) a.out[row * D + i] = __float2bfloat16_rn(0.f);
      if (a.lse)
        for (int i = threadIdx.x; i < rows; i += kInt4Warps * 32) a.lse[row + i] = -INFINITY;
    }
  }
  __syncthreads();
  if (p.cluster > 1) {
    // Without a token the zeros above are the result (written by every CTA alike).
    if (cur.n > 0) int4_cluster_merge<D, L>(p, smem, pieces, *cta_error == 0, cur.b, cur.h, lane);
    return;
  }
  if (*cta_error) return;

  // ---- rows that several warps share, one after another.  Lane k of each warp
  // looks at piece k; the pieces of a row are neighbours.
  constexpr int kPieces = 2 * kInt4Warps;
  static_assert(kPieces <= 32, "a lane per piece");
  const long long my_row = lane < kPieces ? pieces[lane].row : -1;
  unsigned todo = __ballot_sync(0xffffffffu, my_row >= 0);
  while (todo) {
    const int k0 = __ffs(todo) - 1;
    const long long row = __shfl_sync(0xffffffffu, my_row, k0);
    const unsigned held = __ballot_sync(0xffffffffu, my_row == row);
    todo &= ~held;
    const uint32_t begin = pieces[k0].begin, end = begin + pieces[k0].units;
    const bool whole = begin >= cta_begin && end <= cta_end;
    const int slot = 2 * static_cast<int>(blockIdx.x) + (begin > cta_begin ? 1 : 0);
    constexpr int kChunks = D / 4;
    for (int c = threadIdx.x; c < a.G * kChunks; c += kInt4Warps * 32) {
      const int hd = c / kChunks, d = (c % kChunks) * 4;
      const int group = d / (D / 2);
      const float* states = reinterpret_cast<const float*>(smem);
      float m[kPieces], r[kPieces], M = -INFINITY, R = 0x1p-126f;
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int at = (k & 1) ? (k >> 1) * (L::kWarpBytes / 4) : L::kFirstOffset / 4 + (k >> 1) * L::kStateFloats;
        m[k] = (held >> k) & 1u ? states[at + L::kM + hd] : -INFINITY;
        r[k] = (held >> k) & 1u ? states[at + L::kR + group] : 0.f;
        M = fmaxf(M, m[k]);
        R = fmaxf(R, r[k]);
      }
      const float inv_r = power_inverse(R);
      float l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int at = (k & 1) ? (k >> 1) * (L::kWarpBytes / 4) : L::kFirstOffset / 4 + (k >> 1) * L::kStateFloats;
        if ((held >> k) & 1u) {
          const float wt = M == -INFINITY ? 0.f : ex2(m[k] - M), wr = wt * (r[k] * inv_r);
          const float4 v = *reinterpret_cast<const float4*>(states + at + hd * L::kAccStride + d);
          l += wt * states[at + L::kL + hd];
          o.x += wr * v.x;
          o.y += wr * v.y;
          o.z += wr * v.z;
          o.w += wr * v.w;
        }
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      o.x = o.x * inv * R;
      o.y = o.y * inv * R;
      o.z = o.z * inv * R;
      o.w = o.w * inv * R;
      const float lse = (M + log2f(l)) * 0.69314718055994530942f;
      if (whole) {
        // Rows are numbered b Hkv + h, queries b Hq + h G + head.
        const size_t orow = static_cast<size_t>(row) * a.G + hd;
        *reinterpret_cast<uint2*>(a.out + orow * D + d) =
            make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
        if (d == 0 && a.lse) a.lse[orow] = lse;
      } else {
        const size_t prow = static_cast<size_t>(slot) * a.G + hd;
        *reinterpret_cast<float4*>(a.part_o + prow * D + d) = o;
        if (d == 0) a.part_lse[prow] = lse;
      }
    }
  }
}

constexpr int kInt4CombineWarps = 4;

// Merges the partial results of rows that several CTAs share: SHARE warps (one or
// the CTA's four) per query head of a row, their lanes over D.  The candidates are
// the rows themselves or, when there are fewer CTAs than rows, the row that begins
// in each CTA's range and goes on beyond.  A warp requests BATCH partial results at
// once.
template <int D, int U, int SHARE, int BATCH>
__global__ void __launch_bounds__(kInt4CombineWarps * 32) fd_combine_int4_kernel(const Int4DecodeArgs p) {
  constexpr int VPL = D / 32;
  constexpr float kLog2e = 1.4426950408889634074f;
  constexpr float kPart = 1.f / kInt4MaxCtas;          // of a weight: sums of finite parts stay finite
  __shared__ int lens[kInt4Lens];
  const SplitArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  const int w = blockIdx.x * (kInt4CombineWarps / SHARE) + (threadIdx.x >> 5) / SHARE;
  const int share = (threadIdx.x >> 5) % SHARE;        // this warp takes parts share + i SHARE
  const int per = p.heads * a.G;       // query heads of a candidate
  const int cand = w / per, head = w - cand * per;
  // The lengths may be read before the wait, as fd_combine_kernel reads them.
  for (int b = threadIdx.x; b < min(p.B, kInt4Lens); b += kInt4CombineWarps * 32) lens[b] = int4_length(a, b);
  __syncthreads();
  const bool by_rows = p.B * p.groups <= p.ctas;
  const int cand_b = by_rows ? cand / p.groups : 0;
  uint32_t total = 0, before = 0;      // costs of all rows, of the sequences before cand_b
  for (int b = lane; b < p.B; b += 32) {
    const int n = int4_length(a, lens, b);
    const uint32_t cost = n > 0 ? static_cast<uint32_t>((n + U - 1) / U + 1) * p.groups : 0u;
    total += cost;
    if (b < cand_b) before += cost;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, off);
    before += __shfl_xor_sync(0xffffffffu, before, off);
  }
  const Int4Cut cut{total, min(static_cast<uint32_t>(p.ctas), total)};
  int parts = 0, row_b = cand_b, row_h = cand - cand_b * p.groups;
  uint32_t first = 0;                  // the CTA with the row's first part
  bool begins = false;                 // with that CTA's range
  if (by_rows) {
    const int n = cand_b < p.B ? int4_length(a, lens, cand_b) : 0;
    if (n > 0) {
      const uint32_t units = (n + U - 1) / U, begin = before + row_h * (units + 1);
      first = cut.holder(begin);
      parts = static_cast<int>(cut.holder(begin + units - 1) - first) + 1;
      begins = begin == cut.begin(first);
      if (begin + units <= cut.begin(first + 1)) parts = 0;   // one CTA's, finished there
    }
  } else if (cand + 1 < static_cast<int>(cut.ctas)) {
    uint32_t rows;
    first = cand;
    const uint32_t at = cut.begin(first + 1), from = cut.begin(first);
    const Int4Walk row = int4_locate<U>(a, lens, p.B, p.groups, lane, at, rows);
    const uint32_t begin = at - row.u;
    if (row.u > 0 && row.u < row.units && begin >= from) {
      parts = static_cast<int>(cut.holder(begin + row.units - 1) - first) + 1;
      begins = begin == from;
      row_b = row.b;
      row_h = row.h;
    }
  }
  grid_dependency_wait();     // partial results come from the kernel before
  grid_dependents_launch();
  if (parts == 0) return;
  const size_t r = static_cast<size_t>(row_b) * a.Hq + row_h * per + head;
  auto index = [&](int i) {            // of part i
    return static_cast<size_t>(i == 0 && !begins ? 2 * first + 1 : 2 * (first + i)) * per + head;
  };
  // The first parts are requested at once, with their log-sum-exps.
  float lb[BATCH], ob[BATCH][VPL];
  auto load = [&](int s) {
#pragma unroll
    for (int j = 0; j < BATCH; ++j)
      if (s + j * SHARE < parts) {
        const size_t x = index(s + j * SHARE);
        lb[j] = __ldcg(a.part_lse + x);
        if constexpr (VPL == 4) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part_o + x * D) + lane);
          ob[j][0] = v.x; ob[j][1] = v.y; ob[j][2] = v.z; ob[j][3] = v.w;
        } else {
          const float2 v = __ldcg(reinterpret_cast<const float2*>(a.part_o + x * D) + lane);
          ob[j][0] = v.x; ob[j][1] = v.y;
        }
      }
  };
  load(share);
  float mx = -INFINITY;
  bool nan = false;
  for (int i = lane; i < parts; i += 32) {
    const float l = __ldcg(a.part_lse + index(i));
    nan |= l != l;
    mx = fmaxf(mx, l);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
  if (__any_sync(0xffffffffu, nan)) mx = NAN;          // rows of NaN give NaN
  float W = 0.f, acc[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) acc[i] = 0.f;
  for (int s = share; s < parts; s += BATCH * SHARE) {
    if (s > share) load(s);
#pragma unroll
    for (int j = 0; j < BATCH; ++j)
      if (s + j * SHARE < parts) {
        const float wt = mx == -INFINITY ? 0.f : ex2((lb[j] - mx) * kLog2e) * kPart;
        W += wt;
#pragma unroll
        for (int i = 0; i < VPL; ++i) acc[i] += wt * ob[j][i];
      }
  }
  if constexpr (SHARE > 1) {
    __shared__ float sums[SHARE][D + 1];
#pragma unroll
    for (int i = 0; i < VPL; ++i) sums[share][lane * VPL + i] = acc[i];
    if (lane == 0) sums[share][D] = W;
    __syncthreads();
    if (share > 0) return;
    for (int s = 1; s < SHARE; ++s) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) acc[i] += sums[s][lane * VPL + i];
      W += sums[s][D];
    }
  }
  const float inv = W == 0.f ? 0.f : 1.f / W;
  if constexpr (VPL == 4)
    *reinterpret_cast<uint2*>(a.out + r * D + lane * 4) =
        make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(a.out + r * D + lane * 2) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
  if (a.lse && lane == 0) a.lse[r] = mx + logf(W * kInt4MaxCtas);
}

}  // namespace fd
