// pa_rope.cu -- appends with the rotary position embedding applied on the way,
// the 4-bit (E2M1) append, and the gather of cached rows.
//
// Rotary embedding: the pair (a, b) of a head's dims with angle theta(p) at
// position p becomes (a cos - b sin, b cos + a sin).  cos and sin come from the
// caller's table; every product and sum is one fp32 rounding, and the result
// is rounded once to the element type, before any quantisation: a cache of any
// format is built from the same rotated rows.
//
// Work split: a head's row of D elements is D / 8 units of 16 bytes, one lane
// each, so that a warp holds 2 (D 128) or 4 (D 64) whole rows: the partner unit
// of the half pairing comes by shuffle, and a row may be rotated in place.  A
// warp walks over tokens with a fixed slice of the token's rows: where a row comes from and
// goes to, its head's scale and the scale's reciprocal are worked out once, and per token
// only the slot's and the position's offsets are left.  An append has the next
// token's rows, slot and position in flight while it works on this one's; a
// gather has four tokens in flight.
//
// Divisions by a head scale h are x * (1 / h) corrected by one residual: with
// y = RN(1 / h), q = RN(x y) and r = x - q h (exact in an fma), RN(q + r y) is the
// correctly rounded quotient (P. Markstein, 1990) as long as nothing overflows or
// falls below fp32's normal range; outside of a safe range the plain division runs.
#include <cuda_runtime.h>

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

// Largest magnitude of 8 elements, NaN if one is NaN.
template <typename T>
__device__ __forceinline__ float amax8(const uint32_t (&w)[4]) {
  constexpr bool kHalf = std::is_same<T, __half>::value;
  auto top = [](uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (kHalf) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  };
  constexpr uint32_t kAbs = 0x7fff7fffu;
  const uint32_t m = top(top(w[0] & kAbs, w[1] & kAbs), top(w[2] & kAbs, w[3] & kAbs));
  const float2 f = Elem<T>::to_f2(top(m, __byte_perm(m, 0, 0x1032)));
  return f.x;
}

// Head scales whose reciprocal and the products with it stay well inside fp32's range.
__device__ __forceinline__ bool safe_scale(float h) { return h > 0x1p-60f && h < 0x1p60f; }

// 8 elements -> 8 E4M3 codes of x / h, in two words.
template <typename T>
__device__ __forceinline__ uint2 e4m3x8_of(const uint32_t (&w)[4], float h, float y, bool safe) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 v = Elem<T>::to_f2(w[j]);
    f[2 * j] = v.x;
    f[2 * j + 1] = v.y;
  }
  // a quotient beyond fp32 (a bf16 row) must come out infinite, not NaN; fp16's are below 2^77
  if (!std::is_same<T, __half>::value) safe = safe && !(amax8<T>(w) * y >= 0x1p100f);
  if (safe) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = div_by(f[j], h, y);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __fdiv_rn(f[j], h);
  }
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o[j] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(f[2 * j], f[2 * j + 1]), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
}

// 8 elements of a block of 16 (two adjacent lanes) -> their E2M1 codes in a word, and the block's scale code.
template <typename T>
__device__ __forceinline__ uint32_t e2m1x8_of(const uint32_t (&w)[4], float h, float y, bool safe, uint8_t* scale) {
  float amax = amax8<T>(w);
  const float other = __shfl_xor_sync(0xffffffffu, amax, 1);
  const bool nan = amax != amax || other != other;
  amax = fmaxf(amax, other);
  float want;
  if (safe && amax < 0x1p60f)  // below 2^-60 the scale is 0 either way
    want = div_by(div_by(amax, 6.f, 0.16666667163372039795f), h, y);
  else
    want = __fdiv_rn(__fdiv_rn(amax, 6.f), h);
  *scale = nan ? 0x7f : (uint8_t)__nv_cvt_float_to_fp8(want, __NV_SATFINITE, __NV_E4M3);
  const float f = e4m3_to_f(*scale);
  const float r = f > 0.f ? __frcp_rn(__fmul_rn(f, h)) : 0.f;
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 v = Elem<T>::to_f2(w[j]);
    o[j] = e2m1x2_of(__fmul_rn(v.x, r), __fmul_rn(v.y, r));
  }
  return (o[0] | (o[1] << 8)) | ((o[2] | (o[3] << 8)) << 16);
}

template <typename T, int FMT, int D, int U>
__global__ void __launch_bounds__(256, 3)
rope_append_kernel(const RopeArgs a, const int num_tokens, const int slices, const FastDiv by_block) {
  constexpr int UNITS = D / 8;        // lanes per row
  constexpr int RW = 32 / UNITS;      // rows per warp and group
  const int lane = threadIdx.x & 31, u = lane % UNITS;
  const int kv_rows = a.num_q_heads + a.num_kv_heads, rows = kv_rows + a.num_kv_heads;
  const int warp = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int step = gridDim.x * (blockDim.x >> 5) / slices;  // tokens between a warp's
  const int slice = warp % slices;
  int t = warp / slices;
  if (t >= step) t = num_tokens;  // a warp over
  pdl_wait();  // a copy-on-write of this slot's block must land first
  pdl_launch_dependents();
  if (t >= num_tokens) return;

  // this thread's rows: 16 bytes of one head's row of q, k or v
  struct Row {
    const uint16_t* src;
    unsigned char* dst;  // of token 0 (q) or slot 0 (k, v); null: no such row
    long long src_step;
    float h, y;          // head scale and its reciprocal
    bool is_q, is_v;
  } row[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int r = (slice * U + i) * RW + lane / UNITS;
    Row& w = row[i];
    w.is_q = r < a.num_q_heads;
    w.is_v = r >= kv_rows;
    const int head = w.is_q ? r : w.is_v ? r - kv_rows : r - a.num_q_heads;
    const bool live = r < rows;
    const long long stride = w.is_q ? a.q_stride : w.is_v ? a.v_stride : a.k_stride;
    w.src = (w.is_q ? a.q : w.is_v ? a.v : a.k) + t * stride + (live ? head * D + u * 8 : 0);
    w.src_step = step * stride;
    unsigned char* pool = static_cast<unsigned char*>(w.is_v ? a.v_cache : a.k_cache);
    if (w.is_q) w.dst = reinterpret_cast<unsigned char*>(a.q_out + head * D + u * 8);
    else if (FMT == kFmt16) w.dst = pool + (head * D + u * 8) * 2;
    else if (FMT == kFmtFp8) w.dst = pool + head * D + u * 8;
    else w.dst = pool + head * fp4_head_bytes(a.block_size, D);
    if (!live) w.dst = nullptr;
    w.h = FMT == kFmt16 || w.is_q || !live ? 1.f : __ldg((w.is_v ? a.v_scale : a.k_scale) + head);
    w.y = __frcp_rn(w.h);
  }
  const bool rot_unit = u * 8 < a.rotary_dim;
  const long long kv_bytes = (long long)a.num_kv_heads * D;
  struct Token {
    uint4 x[U];
    int slot, pos;
  };
  auto load = [&](int at) {
    Token n;
    n.slot = __ldg(a.slot_mapping + at);
    n.pos = a.rotary_dim > 0 ? __ldg(a.positions + at) : 0;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      n.x[i] = *reinterpret_cast<const uint4*>(row[i].src);
      row[i].src += row[i].src_step;
    }
    return n;
  };

  for (Token next = load(t); t < num_tokens; t += step) {
    const Token now = next;
    bool skip = now.slot < 0;  // padding
    if (now.slot >= a.num_slots) {
      if (slice == 0 && lane == 0) report(a.err, kErrSlot);
      skip = true;
    } else if (!skip && a.rotary_dim > 0 && (unsigned)now.pos >= (unsigned)a.max_position) {
      if (slice == 0 && lane == 0) report(a.err, kErrPosition);
      skip = true;
    }
    // cos and (signed) sin of this thread's 8 dims, and the lane of its partner unit
    float cs[8], sn[8];
    int partner = lane;
    if (!skip && rot_unit) {
      const float* tab = a.cos_sin + (long long)now.pos * a.rotary_dim;
      const int half = a.rotary_dim / 2;
      if (a.interleaved) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(tab + u * 4));
        const float4 s = __ldg(reinterpret_cast<const float4*>(tab + half + u * 4));
        cs[0] = cs[1] = c.x; cs[2] = cs[3] = c.y; cs[4] = cs[5] = c.z; cs[6] = cs[7] = c.w;
        sn[0] = -s.x; sn[1] = s.x; sn[2] = -s.y; sn[3] = s.y;
        sn[4] = -s.z; sn[5] = s.z; sn[6] = -s.w; sn[7] = s.w;
      } else {
        const int hu = half / 8;      // units per half
        const bool lower = u < hu;
        partner = lower ? lane + hu : lane - hu;
        const float* c = tab + (lower ? u : u - hu) * 8;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const float4 cv = __ldg(reinterpret_cast<const float4*>(c + i));
          const float4 sv = __ldg(reinterpret_cast<const float4*>(c + half + i));
          cs[i] = cv.x; cs[i + 1] = cv.y; cs[i + 2] = cv.z; cs[i + 3] = cv.w;
          sn[i] = lower ? -sv.x : sv.x; sn[i + 1] = lower ? -sv.y : sv.y;
          sn[i + 2] = lower ? -sv.z : sv.z; sn[i + 3] = lower ? -sv.w : sv.w;
        }
      }
    }
    if (t + step < num_tokens) next = load(t + step);
    if (skip) continue;
    // where the token's rows start: q's, and the pools' (codes and scales apart in an E2M1 pool)
    const long long q_at = t * a.q_out_stride * 2;
    long long kv_at, sc_at = 0;
    if constexpr (FMT == kFmtFp4) {
      const int block = by_block.div(now.slot), off = now.slot - block * a.block_size;
      kv_at = block * (kv_bytes * a.block_size / 16 * 9);
      sc_at = kv_at + (long long)a.block_size * (D / 2) + off * (D / 16) + u / 2;
      kv_at += off * (D / 2) + u * 4;
    } else {
      kv_at = now.slot * (FMT == kFmt16 ? 2 * kv_bytes : kv_bytes);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const Row& w = row[i];
      uint4 y = now.x[i];
      if (a.rotary_dim > 0) {
        uint4 p;
        if (a.interleaved) {
          p = make_uint4(__byte_perm(y.x, 0, 0x1032), __byte_perm(y.y, 0, 0x1032), __byte_perm(y.z, 0, 0x1032),
                         __byte_perm(y.w, 0, 0x1032));
        } else {
          p = make_uint4(__shfl_sync(0xffffffffu, y.x, partner), __shfl_sync(0xffffffffu, y.y, partner),
                         __shfl_sync(0xffffffffu, y.z, partner), __shfl_sync(0xffffffffu, y.w, partner));
        }
        if (rot_unit && !w.is_v) {
          const uint32_t xw[4] = {y.x, y.y, y.z, y.w}, pw[4] = {p.x, p.y, p.z, p.w};
          uint32_t yw[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 xf = Elem<T>::to_f2(xw[j]), pf = Elem<T>::to_f2(pw[j]);
            yw[j] = pack2<T>(__fadd_rn(__fmul_rn(xf.x, cs[2 * j]), __fmul_rn(pf.x, sn[2 * j])),
                             __fadd_rn(__fmul_rn(xf.y, cs[2 * j + 1]), __fmul_rn(pf.y, sn[2 * j + 1])));
          }
          y = make_uint4(yw[0], yw[1], yw[2], yw[3]);
        }
      }
      if (w.is_q) *reinterpret_cast<uint4*>(w.dst + q_at) = y;
      if (__all_sync(0xffffffffu, w.is_q)) continue;
      const bool store = w.dst && !w.is_q;
      if constexpr (FMT == kFmt16) {
        if (store) *reinterpret_cast<uint4*>(w.dst + kv_at) = y;
      } else {
        const uint32_t yw[4] = {y.x, y.y, y.z, y.w};
        if constexpr (FMT == kFmtFp8) {
          const uint2 o = e4m3x8_of<T>(yw, w.h, w.y, safe_scale(w.h));
          if (store) *reinterpret_cast<uint2*>(w.dst + kv_at) = o;
        } else {
          uint8_t sc;
          const uint32_t o = e2m1x8_of<T>(yw, w.h, w.y, safe_scale(w.h), &sc);
          if (store) {
            *reinterpret_cast<uint32_t*>(w.dst + kv_at) = o;
            if ((u & 1) == 0) w.dst[sc_at] = sc;
          }
        }
      }
    }
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

template <typename T, int FMT, int D>
cudaError_t launch_append(const RopeArgs& a, int num_tokens, cudaStream_t stream) {
  constexpr int U = 2;
  const int rw = 256 / D, groups = (a.num_q_heads + 2 * a.num_kv_heads + rw - 1) / rw, slices = (groups + U - 1) / U;
  return launch_pdl(rope_append_kernel<T, FMT, D, U>, dim3(row_ctas((long long)num_tokens * slices, slices, 3)), dim3(256),
                    0, stream, a, num_tokens, slices, FastDiv(a.block_size));
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
    return launch_append<decltype(t), decltype(fmt)::value, decltype(d)::value>(a, num_tokens, stream);
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
