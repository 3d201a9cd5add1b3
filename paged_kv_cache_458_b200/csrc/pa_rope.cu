// pa_rope.cu -- appends with the rotary position embedding applied on the way,
// the 4-bit (E2M1) append, and the gather of cached rows.
//
// Rotary embedding: the pair (a, b) of a head's dims with angle theta(p) at
// position p becomes (a cos - b sin, b cos + a sin).  cos and sin come from the
// caller's table; every product and sum is one fp32 rounding, and the result
// is rounded once to the element type, before any quantisation: a cache of any
// format is built from the same rotated rows.
//
// Append.  A task is some of a token's q rows, or k and v rows of some of its kv
// heads, 4 KB at most.  The tasks are split evenly into a span per warp, and a warp
// runs its own ring of bulk copies: a task's rows are contiguous, and the token's row of
// the table comes along, so reads are in flight without registers, three tasks
// deep.  A lane takes two units of 8 dims of a row: with the half pairing a unit
// and its partner, so that each element is widened once and no shuffle is
// needed; else neighbours, which are one block of an E2M1 row.  (Before: rows in
// registers, a unit a lane, the partner by shuffle, the next token prefetched:
// 129 instructions per 32 units.)  On a B200: 8191 tokens of 32/8 heads of 128 into a 16-bit
// cache 38.5 us (201 MB read and written: 30.7 us at the copy rate of 6551
// GB/s; before, 47); 16384 tokens of 32/32 heads into an E4M3 cache 128 us (102
// at the copy rate; before, 152), where instructions and reads share the time;
// 20011 tokens of 8 kv heads into an E2M1 cache without rotation 31.5 us (16),
// bound by instructions: two reciprocals, a scale and 16 conversions per 16 dims.
//
// Gather.  A lane takes one unit; a warp walks over tokens with one group of
// rows, four tokens in flight and the next ones' slots ahead.  65536 tokens of 8 kv heads out
// of an E2M1 cache: 70 us (344 MB, 52 us at the copy rate).
//
// Divisions by a head scale h are x * (1 / h) corrected by one residual: with
// y = RN(1 / h), q = RN(x y) and r = x - q h (exact in an fma), RN(q + r y) is the
// correctly rounded quotient (P. Markstein, 1990) as long as nothing overflows or
// falls below fp32's normal range; outside of a safe range the plain division runs.
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "pa_common.cuh"
#include "pa_fp4.cuh"
#include "pa_internal.h"

namespace pa {

enum : int { kFmt16 = 0, kFmtFp8 = 1, kFmtFp4 = 2 };

// Division of 0 <= n < 2^31 by a fixed d >= 2 as a product and a shift: with
// 2^s >= d and m = ceil(2^(31 + s) / d), n m exceeds n 2^(31 + s) / d by less
// than 2^(31 + s) / d, so the floor is exact (Granlund and Montgomery, 1994).
struct FastDiv {
  uint32_t m;
  int shift;
  explicit FastDiv(int d) {
    int s = 1;
    while ((1LL << s) < d) ++s;
    m = (uint32_t)(((1ULL << (31 + s)) + d - 1) / d);
    shift = s - 1;
  }
  __device__ __forceinline__ int div(int n) const { return (int)(__umulhi((uint32_t)n, m) >> shift); }
};

// Two floats rounded to two packed elements, in one conversion.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  uint32_t r;
  if constexpr (std::is_same<T, __half>::value) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// x / h by the corrected reciprocal y = RN(1 / h); see above.  Without a
// residual q is the quotient: -0 keeps its sign, an infinity or a NaN stays.
__device__ __forceinline__ float div_by(float x, float h, float y) {
  const float q = __fmul_rn(x, y);
  const float r = __fmaf_rn(-q, h, x);
  return fabsf(r) > 0.f ? __fmaf_rn(r, y, q) : q;
}

// The larger magnitude of two pairs of packed elements, NaN if one is NaN; the signs come out mixed.
template <typename T>
__device__ __forceinline__ uint32_t top2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (std::is_same<T, __half>::value) asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <typename T>
__device__ __forceinline__ uint32_t top8(const uint32_t (&w)[4]) {
  return top2<T>(top2<T>(w[0], w[1]), top2<T>(w[2], w[3]));
}
// The largest magnitude in a pair.
template <typename T>
__device__ __forceinline__ float magnitude(uint32_t pair) {
  return Elem<T>::to_f2(top2<T>(pair, __byte_perm(pair, 0, 0x1032)) & 0x7fffu).x;
}

// A kv head's scale, its reciprocal, and whether that and the products with it stay well inside fp32's range.
struct HeadScale {
  float h, y;
  bool safe;
};
__device__ __forceinline__ HeadScale head_scale(float h) {
  return HeadScale{h, __frcp_rn(h), h > 0x1p-60f && h < 0x1p60f};
}

// 8 elements -> 8 E4M3 codes of x / h, in two words.
template <typename T>
__device__ __forceinline__ uint2 e4m3x8_of(const uint32_t (&w)[4], const HeadScale& s) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 v = Elem<T>::to_f2(w[j]);
    f[2 * j] = v.x;
    f[2 * j + 1] = v.y;
  }
  // a quotient beyond fp32 (a bf16 row) must come out infinite, not NaN, also beside a NaN; fp16's are below 2^77
  bool safe = s.safe;
  if (!std::is_same<T, __half>::value) safe = safe && magnitude<T>(top8<T>(w)) * s.y < 0x1p100f;
  if (safe) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = div_by(f[j], s.h, s.y);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __fdiv_rn(f[j], s.h);
  }
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o[j] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(f[2 * j], f[2 * j + 1]), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
}

// The scale code of a block of 16 dims with largest magnitude `amax` (NaN: a
// dim is NaN): the E4M3 value nearest to (amax / 6) / h, 6 being E2M1's largest,
// at most 448.  *r is the factor that takes a value to the codes' range.
__device__ __forceinline__ uint8_t block_scale(float amax, const HeadScale& s, float* r) {
  float want;
  if (s.safe && amax < 0x1p60f)  // what is too small for the correction gives a zero scale either way
    want = div_by(div_by(amax, 6.f, 0.16666667163372039795f), s.h, s.y);
  else
    want = __fdiv_rn(__fdiv_rn(amax, 6.f), s.h);
  const uint8_t code = amax != amax ? 0x7f : (uint8_t)__nv_cvt_float_to_fp8(want, __NV_SATFINITE, __NV_E4M3);
  const float f = e4m3_to_f(code);
  *r = f > 0.f ? __frcp_rn(__fmul_rn(f, s.h)) : 0.f;
  return code;
}

// 8 elements times r -> 8 E2M1 codes: nearest, ties to the even code, saturating at 6.
template <typename T>
__device__ __forceinline__ uint32_t e2m1x8_of(const uint32_t (&w)[4], float r) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 v = Elem<T>::to_f2(w[j]);
    f[2 * j] = __fmul_rn(v.x, r);
    f[2 * j + 1] = __fmul_rn(v.y, r);
  }
  uint32_t o;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(o)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return o;
}

constexpr int kRowWarps = 4, kRowStages = 3, kRowCtas = 4;
constexpr int kTaskBytes = 4096, kStageBytes = kTaskBytes + 512;  // rows, then the table's row

// ROT: whether anything rotates.
template <typename T, int FMT, int D, bool ROT>
__global__ void __launch_bounds__(kRowWarps * 32, kRowCtas)
rope_append_kernel(const RopeArgs a, const int num_tokens, const FastDiv by_block) {
  constexpr int LANES = D / 16, RW = 32 / LANES;   // lanes per row, rows per step
  constexpr int PR = kTaskBytes / (2 * D);         // rows of a task
  extern __shared__ __align__(128) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, p = lane % LANES;
  unsigned char* stages = smem + warp * kRowStages * kStageBytes;
  const uint32_t bar0 = smem_addr(smem) + kRowWarps * kRowStages * kStageBytes + warp * kRowStages * 8;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < kRowStages; ++i) mbar_init(bar0 + i * 8, 1);
    mbar_init_fence();
  }
  __syncwarp();
  pdl_wait();  // a copy-on-write of this slot's block must land first
  pdl_launch_dependents();

  const int num_slots = (int)a.num_slots;  // below 2^31
  // tasks of a token: PR of its q rows, or half as many of k and of v
  const int q_tasks = (a.num_q_heads + PR - 1) / PR;
  const int per_token = q_tasks + (a.num_kv_heads + PR / 2 - 1) / (PR / 2);
  const long long total = (long long)num_tokens * per_token, warps = (long long)gridDim.x * kRowWarps;
  const long long w = (long long)blockIdx.x * kRowWarps + warp;
  const long long begin = total * w / warps;
  const int n_mine = (int)(total * (w + 1) / warps - begin);
  if (n_mine == 0) return;

  // The copies run kRowStages tasks ahead: their cursor, and the slots of the tasks in flight (negative: skip).
  int f_t = (int)(begin / per_token), f_part = (int)(begin % per_token), f_stage = 0;
  int slots[kRowStages];
  // first head of a task, and the number of heads
  auto head_of = [&](int part) { return part < q_tasks ? part * PR : (part - q_tasks) * (PR / 2); };
  auto heads_of = [&](int part) {
    return part < q_tasks ? min(PR, a.num_q_heads - part * PR) : min(PR / 2, a.num_kv_heads - (part - q_tasks) * (PR / 2));
  };
  // Starts the next task's copies and returns its slot, or -1 where the token is
  // skipped; what is wrong with a token is reported with its first task.
  auto issue = [&](int slot, int pos) {
    const bool padding = slot < 0, bad_slot = slot >= num_slots;
    const bool bad_pos = ROT && (unsigned)pos >= (unsigned)a.max_position;
    if (padding || bad_slot || bad_pos) {
      if (!padding && f_part == 0 && lane == 0) report(a.err, bad_slot ? kErrSlot : kErrPosition);
      slot = -1;
    }
    const bool is_q = f_part < q_tasks;
    const uint32_t bytes = slot < 0 ? 0 : heads_of(f_part) * D * 2;
    const uint32_t table_bytes = !ROT || slot < 0 ? 0 : a.rotary_dim * 4;
    if (lane == 0) {
      const uint32_t bar = bar0 + f_stage * 8, dst = smem_addr(stages + f_stage * kStageBytes);
      const int from = head_of(f_part) * D;
      mbar_arrive_expect_tx(bar, (is_q ? bytes : 2 * bytes) + table_bytes);
      if (bytes) {
        if (is_q) {
          bulk_load(dst, a.q + f_t * a.q_stride + from, bytes, bar);
        } else {
          bulk_load(dst, a.k + f_t * a.k_stride + from, bytes, bar);
          bulk_load(dst + kTaskBytes / 2, a.v + f_t * a.v_stride + from, bytes, bar);
        }
        if (table_bytes) bulk_load(dst + kTaskBytes, a.cos_sin + (long long)pos * a.rotary_dim, table_bytes, bar);
      }
    }
    if (++f_part == per_token) { f_part = 0; ++f_t; }
    if (++f_stage == kRowStages) f_stage = 0;
    return slot;
  };
  auto slot_of = [&](int t) { return __ldg(a.slot_mapping + t); };
  auto pos_of = [&](int t) { return ROT ? __ldg(a.positions + t) : 0; };
  int t = f_t, part = f_part, stage_at = 0, phase = 0;  // the task at work
#pragma unroll
  for (int k = 0; k < kRowStages; ++k) slots[k] = k < n_mine ? issue(slot_of(f_t), pos_of(f_t)) : -1;
  int next_slot = 0, next_pos = 0;
  if (kRowStages < n_mine) next_slot = slot_of(f_t), next_pos = pos_of(f_t);

  // bytes from a token, a block, or a head to the next
  const long long kv_row = (long long)a.num_kv_heads * D * (FMT == kFmt16 ? 2 : 1);
  const long long run = fp4_head_bytes(a.block_size, D), block_bytes = run * a.num_kv_heads;
  for (int k = 0; k < n_mine; ++k) {
    if (!mbar_wait_warp(bar0 + stage_at * 8, phase, a.err)) {
      for (int i = k + 1; i < min(n_mine, k + kRowStages); ++i) {  // let the copies in flight land
        if (++stage_at == kRowStages) { stage_at = 0; phase ^= 1; }
        mbar_wait(bar0 + stage_at * 8, phase, a.err);
      }
      return;
    }
    const int slot = slots[0];
    const unsigned char* stage = stages + stage_at * kStageBytes;
    if (slot >= 0) {
      const bool is_q = part < q_tasks;
      const int head0 = head_of(part), heads = heads_of(part);
#pragma unroll 1
      for (int is_v = 0; is_v < (is_q ? 1 : 2); ++is_v) {
        // this lane's two units: a unit and its partner (half pairing), else neighbours
        const int hu = !ROT || is_v || a.interleaved ? 0 : a.rotary_dim / 16;  // units per half
        const bool split = p < hu, turn = split || (ROT && !is_v && a.interleaved && p * 16 < a.rotary_dim);
        const int u0 = split ? p : hu + p + (p - hu), u1 = split ? p + hu : u0 + 1;
        // half pairing: cos and sin of the pairs (unit, partner); interleaved: of the 4 pairs of u0, then of u1
        alignas(16) float cs[8], sn[8];
        if (turn) {
          const float* tab = reinterpret_cast<const float*>(stage + kTaskBytes) + p * 8;
#pragma unroll
          for (int i = 0; i < 8; i += 4) {
            *reinterpret_cast<float4*>(cs + i) = *reinterpret_cast<const float4*>(tab + i);
            *reinterpret_cast<float4*>(sn + i) = *reinterpret_cast<const float4*>(tab + a.rotary_dim / 2 + i);
          }
        }
        // this lane's row of the first step: in the stage, its head's scale, and where it goes (rows; block scales)
        const int row = lane / LANES, head = head0 + row;
        const unsigned char* rows = stage + is_v * (kTaskBytes / 2) + row * (2 * D);
        const float* scale = (is_v ? a.v_scale : a.k_scale) + head;
        unsigned char* to = static_cast<unsigned char*>(is_v ? a.v_cache : a.k_cache);
        unsigned char* to_scale = nullptr;
        long long to_step;
        if (is_q) {
          to = reinterpret_cast<unsigned char*>(a.q_out + t * a.q_out_stride + head * D);
          to_step = RW * D * 2;
        } else if constexpr (FMT == kFmtFp4) {
          const int block = by_block.div(slot), off = slot - block * a.block_size;
          to += block * block_bytes + head * run;
          to_scale = to + a.block_size * (D / 2) + off * (D / 16);
          to += off * (D / 2);
          to_step = RW * run;
        } else {
          to += slot * kv_row + head * (FMT == kFmt16 ? 2 * D : D);
          to_step = RW * (FMT == kFmt16 ? 2 * D : D);
        }
        // all lanes take every step (the shuffles below need them); rows past the task's are computed and dropped
#pragma unroll 2
        for (int i = 0; i < heads; i += RW, rows += RW * 2 * D, scale += RW, to += to_step) {
          const bool live = i + row < heads;
          const uint4 x0 = *reinterpret_cast<const uint4*>(rows + u0 * 16);
          const uint4 x1 = *reinterpret_cast<const uint4*>(rows + u1 * 16);
          uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w}, w1[4] = {x1.x, x1.y, x1.z, x1.w};
          if (turn) {
            if (a.interleaved) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 v = Elem<T>::to_f2(w0[j]), z = Elem<T>::to_f2(w1[j]);
                w0[j] = pack2<T>(__fsub_rn(__fmul_rn(v.x, cs[j]), __fmul_rn(v.y, sn[j])),
                                 __fadd_rn(__fmul_rn(v.y, cs[j]), __fmul_rn(v.x, sn[j])));
                w1[j] = pack2<T>(__fsub_rn(__fmul_rn(z.x, cs[4 + j]), __fmul_rn(z.y, sn[4 + j])),
                                 __fadd_rn(__fmul_rn(z.y, cs[4 + j]), __fmul_rn(z.x, sn[4 + j])));
              }
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 v = Elem<T>::to_f2(w0[j]), z = Elem<T>::to_f2(w1[j]);
                w0[j] = pack2<T>(__fsub_rn(__fmul_rn(v.x, cs[2 * j]), __fmul_rn(z.x, sn[2 * j])),
                                 __fsub_rn(__fmul_rn(v.y, cs[2 * j + 1]), __fmul_rn(z.y, sn[2 * j + 1])));
                w1[j] = pack2<T>(__fadd_rn(__fmul_rn(z.x, cs[2 * j]), __fmul_rn(v.x, sn[2 * j])),
                                 __fadd_rn(__fmul_rn(z.y, cs[2 * j + 1]), __fmul_rn(v.y, sn[2 * j + 1])));
              }
            }
          }
          if (FMT == kFmt16 || is_q) {
            uint4* out = reinterpret_cast<uint4*>(to);
            if (live) {
              out[u0] = make_uint4(w0[0], w0[1], w0[2], w0[3]);
              out[u1] = make_uint4(w1[0], w1[1], w1[2], w1[3]);
            }
          } else if constexpr (FMT == kFmtFp8) {
            const HeadScale s = head_scale(live ? __ldg(scale) : 1.f);
            const uint2 o0 = e4m3x8_of<T>(w0, s), o1 = e4m3x8_of<T>(w1, s);
            uint2* out = reinterpret_cast<uint2*>(to);
            if (live) {
              out[u0] = o0;
              out[u1] = o1;
            }
          } else if constexpr (FMT == kFmtFp4) {
            const HeadScale s = head_scale(live ? __ldg(scale) : 1.f);
            const uint32_t m0 = top8<T>(w0), m1 = top8<T>(w1);
            uint32_t* codes = reinterpret_cast<uint32_t*>(to);
            if (hu == 0) {  // neighbours: one block
              float f;
              const uint8_t sc = block_scale(magnitude<T>(top2<T>(m0, m1)), s, &f);
              const uint32_t o0 = e2m1x8_of<T>(w0, f), o1 = e2m1x8_of<T>(w1, f);
              if (live) {
                *reinterpret_cast<uint2*>(codes + u0) = make_uint2(o0, o1);
                to_scale[p] = sc;
              }
            } else {
              // the other unit of each unit's block: in lane `l` of this row, as its first or second unit
              auto mate = [&](int u) {
                const int v = u ^ 1, l = v < hu ? v : v < 2 * hu ? v - hu : hu + (v - 2 * hu) / 2;
                const int src = lane - p + l;
                const uint32_t f0 = __shfl_sync(0xffffffffu, m0, src), f1 = __shfl_sync(0xffffffffu, m1, src);
                return v < hu || (v >= 2 * hu && (v & 1) == 0) ? f0 : f1;
              };
              const uint32_t n0 = mate(u0), n1 = mate(u1);
              float f0, f1;
              const uint8_t s0 = block_scale(magnitude<T>(top2<T>(m0, n0)), s, &f0);
              const uint8_t s1 = block_scale(magnitude<T>(top2<T>(m1, n1)), s, &f1);
              const uint32_t o0 = e2m1x8_of<T>(w0, f0), o1 = e2m1x8_of<T>(w1, f1);
              if (live) {
                codes[u0] = o0;
                codes[u1] = o1;
                if ((u0 & 1) == 0) to_scale[u0 / 2] = s0;
                if ((u1 & 1) == 0) to_scale[u1 / 2] = s1;
              }
            }
            to_scale += to_step;
          }
        }
      }
    }
    __syncwarp();
    // the stage is free again: refill it
    int refill = -1;
    if (k + kRowStages < n_mine) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      refill = issue(next_slot, next_pos);
      if (k + kRowStages + 1 < n_mine) next_slot = slot_of(f_t), next_pos = pos_of(f_t);
    }
#pragma unroll
    for (int i = 0; i + 1 < kRowStages; ++i) slots[i] = slots[i + 1];
    slots[kRowStages - 1] = refill;
    if (++part == per_token) { part = 0; ++t; }
    if (++stage_at == kRowStages) { stage_at = 0; phase ^= 1; }
  }
}

// Rows of a cache back into 16-bit rows: stored value = code * block scale *
// head scale (one fp32 rounding), rounded to the element type; a 16-bit
// cache is copied bit by bit.  A warp takes one group of rows of U tokens at a time.
template <typename T, int FMT, int D, int U>
__global__ void __launch_bounds__(256, 5)
cache_gather_kernel(const GatherArgs a, const int num_tokens, const int groups, const FastDiv by_block) {
  constexpr int UNITS = D / 8, RW = 32 / UNITS;
  const int lane = threadIdx.x & 31, u = lane % UNITS;
  const int warp = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int step = gridDim.x * (blockDim.x >> 5) / groups * U, t_first = warp / groups * U;
  const int r = warp % groups * RW + lane / UNITS;
  pdl_wait();
  pdl_launch_dependents();
  if (t_first >= step || r >= 2 * a.num_kv_heads) return;
  const bool is_v = r >= a.num_kv_heads;
  const int h = is_v ? r - a.num_kv_heads : r;
  const unsigned char* pool = static_cast<const unsigned char*>(is_v ? a.v_cache : a.k_cache);
  const float hs = FMT == kFmt16 ? 1.f : __ldg((is_v ? a.v_scale : a.k_scale) + h);
  const long long kv_bytes = (long long)a.num_kv_heads * D;
  if (FMT == kFmtFp4) pool += h * fp4_head_bytes(a.block_size, D);
  else pool += (h * D + u * 8) * (FMT == kFmt16 ? 2 : 1);
  unsigned char* out = reinterpret_cast<unsigned char*>((is_v ? a.v_out : a.k_out) + h * D + u * 8);

  int ahead[U];  // the next tokens' slots
#pragma unroll
  for (int i = 0; i < U; ++i) ahead[i] = t_first + i < num_tokens ? __ldg(a.slot_mapping + t_first + i) : -1;
  for (int t0 = t_first; t0 < num_tokens; t0 += step) {
    int slot[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      slot[i] = ahead[i];
      ahead[i] = t0 + step + i < num_tokens ? __ldg(a.slot_mapping + t0 + step + i) : -1;
    }
    uint4 x[U];
    uint8_t sc[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      x[i] = make_uint4(0, 0, 0, 0);  // a slot beyond the pool reads as zeros
      sc[i] = 0;
      if (slot[i] >= a.num_slots) {
        if (r == 0 && u == 0) report(a.err, kErrSlot);
      } else if (slot[i] >= 0) {
        if constexpr (FMT == kFmtFp4) {
          const int block = by_block.div(slot[i]), off = slot[i] - block * a.block_size;
          const unsigned char* run = pool + block * (kv_bytes * a.block_size / 16 * 9);
          x[i].x = __ldg(reinterpret_cast<const uint32_t*>(run + off * (D / 2) + u * 4));
          sc[i] = __ldg(run + fp4_code_bytes(a.block_size, D) + off * (D / 16) + u / 2);
        } else if constexpr (FMT == kFmt16) {
          x[i] = __ldg(reinterpret_cast<const uint4*>(pool + slot[i] * (2 * kv_bytes)));
        } else {
          const uint2 w = __ldg(reinterpret_cast<const uint2*>(pool + slot[i] * kv_bytes));
          x[i].x = w.x;
          x[i].y = w.y;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (slot[i] < 0) continue;
      uint4 y = x[i];
      if constexpr (FMT != kFmt16) {
        float2 f[4];
        if constexpr (FMT == kFmtFp8) {
          f[0] = e4m3x2_to_f2((uint16_t)y.x);
          f[1] = e4m3x2_to_f2((uint16_t)(y.x >> 16));
          f[2] = e4m3x2_to_f2((uint16_t)y.y);
          f[3] = e4m3x2_to_f2((uint16_t)(y.y >> 16));
        } else {
          // code times block scale is exact in f16: 2 significant bits times 4, from 2^-10 to 2688
          const uint32_t s = e4m3x2_to_h2((uint16_t)(sc[i] | (sc[i] << 8)));
          uint32_t hv[4];
          e2m1x8_to_h2(y.x, hv);
#pragma unroll
          for (int j = 0; j < 4; ++j) f[j] = h2_to_f2(hmul2(hv[j], s));
        }
        y = make_uint4(pack2<T>(__fmul_rn(f[0].x, hs), __fmul_rn(f[0].y, hs)),
                       pack2<T>(__fmul_rn(f[1].x, hs), __fmul_rn(f[1].y, hs)),
                       pack2<T>(__fmul_rn(f[2].x, hs), __fmul_rn(f[2].y, hs)),
                       pack2<T>(__fmul_rn(f[3].x, hs), __fmul_rn(f[3].y, hs)));
      }
      *reinterpret_cast<uint4*>(out + (t0 + i) * (2 * kv_bytes)) = y;
    }
  }
}

namespace {

// CTAs of 8 warps: as many as a B200 holds at `per_sm`, fewer where the work
// (warps that have something to do) runs out, and never less than one token's.
unsigned row_ctas(long long warps, int warps_per_token, int per_sm) {
  const long long most = (warps + 7) / 8, least = (warps_per_token + 7) / 8, n = most < 148 * per_sm ? most : 148 * per_sm;
  return (unsigned)(n > least ? n : least);
}

template <typename T, int FMT, int D, bool ROT>
cudaError_t launch_append(const RopeArgs& a, int num_tokens, cudaStream_t stream) {
  constexpr int smem = kRowWarps * kRowStages * (kStageBytes + 8), PR = kTaskBytes / (2 * D);
  auto* kern = rope_append_kernel<T, FMT, D, ROT>;
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = allow_smem(kern, smem, &configured);
  if (e != cudaSuccess) return e;
  const long long tasks =
      (long long)num_tokens * ((a.num_q_heads + PR - 1) / PR + (a.num_kv_heads + PR / 2 - 1) / (PR / 2));
  const long long ctas = (tasks + kRowWarps - 1) / kRowWarps, wave = 148 * kRowCtas;  // what a B200 holds at once
  return launch_pdl(kern, dim3((unsigned)(ctas < wave ? ctas : wave)), dim3(kRowWarps * 32), smem, stream, a, num_tokens,
                    FastDiv(a.block_size));
}

template <typename T, int FMT, int D>
cudaError_t launch_gather(const GatherArgs& a, int num_tokens, cudaStream_t stream) {
  constexpr int U = 4;
  const int rw = 256 / D, groups = (2 * a.num_kv_heads + rw - 1) / rw;
  return launch_pdl(cache_gather_kernel<T, FMT, D, U>,
                    dim3(row_ctas((num_tokens + U - 1LL) / U * groups, groups, 5)), dim3(256), 0, stream, a, num_tokens,
                    groups, FastDiv(a.block_size));
}

// Calls f(T, format, D) for the run-time values.
template <typename F>
cudaError_t dispatch(int dtype, int head_dim, int format, F f) {
  auto fmt = [&](auto t, auto d) {
    if (format == kFmt16) return f(t, std::integral_constant<int, kFmt16>{}, d);
    if (format == kFmtFp8) return f(t, std::integral_constant<int, kFmtFp8>{}, d);
    return f(t, std::integral_constant<int, kFmtFp4>{}, d);
  };
  auto dim = [&](auto t) {
    return head_dim == 128 ? fmt(t, std::integral_constant<int, 128>{}) : fmt(t, std::integral_constant<int, 64>{});
  };
  return dtype == 0 ? dim(__half{}) : dim(__nv_bfloat16{});
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs& a, int dtype, int head_dim, int format, int num_tokens,
                               cudaStream_t stream, int* launches) {
  const cudaError_t e = dispatch(dtype, head_dim, format, [&](auto t, auto fmt, auto d) {
    using T = decltype(t);
    constexpr int F = decltype(fmt)::value, D = decltype(d)::value;
    if constexpr (F == kFmtFp4)
      if (a.rotary_dim == 0) return launch_append<T, F, D, false>(a, num_tokens, stream);
    return launch_append<T, F, D, true>(a, num_tokens, stream);
  });
  if (e == cudaSuccess) ++*launches;
  return e;
}

cudaError_t launch_cache_gather(const GatherArgs& a, int dtype, int head_dim, int format, int num_tokens,
                                cudaStream_t stream, int* launches) {
  const cudaError_t e = dispatch(dtype, head_dim, format, [&](auto t, auto fmt, auto d) {
    return launch_gather<decltype(t), decltype(fmt)::value, decltype(d)::value>(a, num_tokens, stream);
  });
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace pa
