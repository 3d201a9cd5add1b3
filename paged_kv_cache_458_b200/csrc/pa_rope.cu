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
// of the half pairing comes by shuffle, and a row may be rotated in place.  An
// append's CTA takes one token, a warp U groups of rows whose loads are in flight
// together with those of the slot and the position; a thread's unit, and
// with it its cos and sin, are the same in all of them.  A gather's warp
// takes one group of rows of U tokens.
#include <cuda_runtime.h>

#include <type_traits>

#include "pa_common.cuh"
#include "pa_fp4.cuh"
#include "pa_internal.h"

namespace pa {

enum : int { kFmt16 = 0, kFmtFp8 = 1, kFmtFp4 = 2 };

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return (uint32_t)Elem<T>::from_f(a) | ((uint32_t)Elem<T>::from_f(b) << 16);
}

template <typename T, int FMT, int D, int U>
__global__ void __launch_bounds__(256)
rope_append_kernel(const RopeArgs a) {
  constexpr int UNITS = D / 8;        // lanes per row
  constexpr int RW = 32 / UNITS;      // rows per warp and group
  pdl_wait();  // a copy-on-write of this slot's block must land first
  pdl_launch_dependents();
  const int t = blockIdx.x, lane = threadIdx.x & 31, u = lane % UNITS, warps = blockDim.x >> 5;
  const int rows = a.num_q_heads + 2 * a.num_kv_heads;
  const uint16_t* q_row = a.q + (long long)t * a.q_stride;
  const uint16_t* k_row = a.k + (long long)t * a.k_stride;
  const uint16_t* v_row = a.v + (long long)t * a.v_stride;
  const long long slot = __ldg(a.slot_mapping + t);
  const int pos = a.rotary_dim > 0 ? __ldg(a.positions + t) : 0;
  const bool rot_unit = u * 8 < a.rotary_dim;
  float cs[8], sn[8];                 // cos and (signed) sin of this thread's 8 dims
  int partner = lane;                 // the lane of its partner unit

  for (int r0 = (threadIdx.x >> 5) * RW + lane / UNITS, first = true; r0 - lane / UNITS < rows;
       r0 += U * warps * RW, first = false) {
    uint4 x[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int r = r0 + i * warps * RW;
      const uint16_t* src = r < a.num_q_heads ? q_row + r * D
                            : r < a.num_q_heads + a.num_kv_heads ? k_row + (r - a.num_q_heads) * D
                                                                 : v_row + (r - a.num_q_heads - a.num_kv_heads) * D;
      x[i] = r < rows ? *reinterpret_cast<const uint4*>(src + u * 8) : make_uint4(0, 0, 0, 0);
    }
    if (first) {
      if (slot < 0) return;           // padding
      if (slot >= a.num_slots) {
        if (threadIdx.x == 0) report(a.err, kErrSlot);
        return;
      }
      if (a.rotary_dim > 0 && (pos < 0 || pos >= a.max_position)) {
        if (threadIdx.x == 0) report(a.err, kErrPosition);
        return;
      }
      if (rot_unit) {
        const float* row = a.cos_sin + (long long)pos * a.rotary_dim;
        const int half = a.rotary_dim / 2;
        if (a.interleaved) {
          const float4 c = __ldg(reinterpret_cast<const float4*>(row + u * 4));
          const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + u * 4));
          cs[0] = cs[1] = c.x; cs[2] = cs[3] = c.y; cs[4] = cs[5] = c.z; cs[6] = cs[7] = c.w;
          sn[0] = -s.x; sn[1] = s.x; sn[2] = -s.y; sn[3] = s.y;
          sn[4] = -s.z; sn[5] = s.z; sn[6] = -s.w; sn[7] = s.w;
        } else {
          const int hu = half / 8;    // units per half
          const bool lower = u < hu;
          partner = lower ? lane + hu : lane - hu;
          const float* c = row + (lower ? u : u - hu) * 8;
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
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int r = r0 + i * warps * RW;
      const bool live = r < rows, is_q = r < a.num_q_heads, is_v = r >= a.num_q_heads + a.num_kv_heads;
      const int h = is_q ? r : r - a.num_q_heads - (is_v ? a.num_kv_heads : 0);
      uint4 y = x[i];
      if (a.rotary_dim > 0) {
        uint4 p;
        if (a.interleaved) {
          p = make_uint4(__byte_perm(y.x, 0, 0x1032), __byte_perm(y.y, 0, 0x1032), __byte_perm(y.z, 0, 0x1032),
                         __byte_perm(y.w, 0, 0x1032));
        } else {
          p = make_uint4(__shfl_sync(0xffffffffu, y.x, partner), __shfl_sync(0xffffffffu, y.y, partner),
                         __shfl_sync(0xffffffffu, y.z, partner), __shfl_sync(0xffffffffu, y.w, partner));
        }
        if (rot_unit && !is_v) {
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
      if (is_q) *reinterpret_cast<uint4*>(a.q_out + (long long)t * a.q_out_stride + h * D + u * 8) = y;
      const bool store = live && !is_q;
      // no row of this warp's group goes to the cache: nothing to quantise
      if (r - lane / UNITS + RW <= a.num_q_heads) continue;
      unsigned char* pool = static_cast<unsigned char*>(is_v ? a.v_cache : a.k_cache);
      if constexpr (FMT == kFmt16) {
        if (store) *reinterpret_cast<uint4*>(pool + ((slot * a.num_kv_heads + h) * D + u * 8) * 2) = y;
      } else {
        const float hs = store ? __ldg((is_v ? a.v_scale : a.k_scale) + h) : 1.f;
        const uint32_t yw[4] = {y.x, y.y, y.z, y.w};
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 v = Elem<T>::to_f2(yw[j]);
          f[2 * j] = v.x;
          f[2 * j + 1] = v.y;
        }
        if constexpr (FMT == kFmtFp8) {
          uint32_t o[2] = {0, 0};
#pragma unroll
          for (int j = 0; j < 8; j += 2)
            o[j / 4] |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(f[j], hs), __fdiv_rn(f[j + 1], hs)),
                                                           __NV_SATFINITE, __NV_E4M3)
                        << (8 * (j % 4));
          if (store)
            *reinterpret_cast<uint2*>(pool + (slot * a.num_kv_heads + h) * D + u * 8) = make_uint2(o[0], o[1]);
        } else {
          float amax = 0.f;
          bool nan = false;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            amax = fmaxf(amax, fabsf(f[j]));
            nan |= f[j] != f[j];
          }
          // a block of 16 dims is two adjacent lanes
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
          nan |= __shfl_xor_sync(0xffffffffu, (int)nan, 1) != 0;
          float rs;
          const uint8_t s = fp4_block_scale(amax, nan, hs, &rs);
          uint32_t o = 0;
#pragma unroll
          for (int j = 0; j < 8; j += 2) o |= e2m1x2_of(__fmul_rn(f[j], rs), __fmul_rn(f[j + 1], rs)) << (4 * j);
          if (store) {
            const int block = (int)slot / a.block_size, off = (int)slot - block * a.block_size;  // slots are below 2^31
            unsigned char* run = pool + ((long long)block * a.num_kv_heads + h) * fp4_head_bytes(a.block_size, D);
            *reinterpret_cast<uint32_t*>(run + off * (D / 2) + u * 4) = o;
            if ((u & 1) == 0) run[fp4_code_bytes(a.block_size, D) + off * (D / 16) + u / 2] = s;
          }
        }
      }
    }
  }
}

// Rows of a cache back into 16-bit rows: stored value = code * block scale *
// head scale (one fp32 rounding), rounded to the element type; a 16-bit
// cache is copied bit by bit.  Same split as above, over the 2 Hkv rows of a token.
template <typename T, int FMT, int D, int U>
__global__ void __launch_bounds__(256)
cache_gather_kernel(const GatherArgs a, const int num_tokens) {
  constexpr int UNITS = D / 8, RW = 32 / UNITS;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, u = lane % UNITS, t0 = blockIdx.x * U;
  const int r = (blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5)) * RW + lane / UNITS;
  if (r >= 2 * a.num_kv_heads) return;
  const bool is_v = r >= a.num_kv_heads;
  const int h = is_v ? r - a.num_kv_heads : r;
  const unsigned char* pool = static_cast<const unsigned char*>(is_v ? a.v_cache : a.k_cache);
  const float hs = FMT == kFmt16 ? 1.f : __ldg((is_v ? a.v_scale : a.k_scale) + h);
  long long slot[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    slot[i] = t0 + i < num_tokens ? __ldg(a.slot_mapping + t0 + i) : -1;
    if (slot[i] >= a.num_slots) {  // such a row reads as zeros
      if (threadIdx.x == 0 && blockIdx.y == 0) report(a.err, kErrSlot);
      slot[i] = -2;
    }
  }
  uint4 x[U];
  uint8_t sc[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    x[i] = make_uint4(0, 0, 0, 0);
    sc[i] = 0;
    if (slot[i] >= 0) {
      if constexpr (FMT == kFmt16) {
        x[i] = __ldg(reinterpret_cast<const uint4*>(pool + ((slot[i] * a.num_kv_heads + h) * D + u * 8) * 2));
      } else if constexpr (FMT == kFmtFp8) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(pool + (slot[i] * a.num_kv_heads + h) * D + u * 8));
        x[i].x = w.x;
        x[i].y = w.y;
      } else {
        const int block = (int)slot[i] / a.block_size, off = (int)slot[i] - block * a.block_size;
        const unsigned char* run = pool + ((long long)block * a.num_kv_heads + h) * fp4_head_bytes(a.block_size, D);
        x[i].x = __ldg(reinterpret_cast<const uint32_t*>(run + off * (D / 2) + u * 4));
        sc[i] = __ldg(run + fp4_code_bytes(a.block_size, D) + off * (D / 16) + u / 2);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (slot[i] == -2 || slot[i] >= 0) {
      uint4 y = x[i];
      if constexpr (FMT != kFmt16) {
        float2 f[4];
        if constexpr (FMT == kFmtFp8) {
          f[0] = e4m3x2_to_f2((uint16_t)y.x);
          f[1] = e4m3x2_to_f2((uint16_t)(y.x >> 16));
          f[2] = e4m3x2_to_f2((uint16_t)y.y);
          f[3] = e4m3x2_to_f2((uint16_t)(y.y >> 16));
        } else {
          const float s = e4m3_to_f(sc[i]);
          uint32_t hv[4];
          e2m1x8_to_h2(y.x, hv);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            f[j] = h2_to_f2(hv[j]);
            f[j].x *= s;  // exact: 2 significant bits times 4
            f[j].y *= s;
          }
        }
        y = make_uint4(pack2<T>(__fmul_rn(f[0].x, hs), __fmul_rn(f[0].y, hs)),
                       pack2<T>(__fmul_rn(f[1].x, hs), __fmul_rn(f[1].y, hs)),
                       pack2<T>(__fmul_rn(f[2].x, hs), __fmul_rn(f[2].y, hs)),
                       pack2<T>(__fmul_rn(f[3].x, hs), __fmul_rn(f[3].y, hs)));
      }
      uint16_t* out = (is_v ? a.v_out : a.k_out) + ((long long)(t0 + i) * a.num_kv_heads + h) * D + u * 8;
      *reinterpret_cast<uint4*>(out) = y;
    }
  }
}

namespace {

constexpr int kGatherTokens = 4;

template <typename T, int FMT, int D>
cudaError_t launch_append(const RopeArgs& a, int num_tokens, cudaStream_t stream) {
  const int rw = 256 / D, groups = (a.num_q_heads + 2 * a.num_kv_heads + rw - 1) / rw;
  const dim3 grid(num_tokens), block(32 * (groups < 8 ? groups : 8));
  if (groups <= 8) return launch_pdl(rope_append_kernel<T, FMT, D, 1>, grid, block, 0, stream, a);
  if (groups <= 16) return launch_pdl(rope_append_kernel<T, FMT, D, 2>, grid, block, 0, stream, a);
  return launch_pdl(rope_append_kernel<T, FMT, D, 3>, grid, block, 0, stream, a);
}

template <typename T, int FMT, int D>
cudaError_t launch_gather(const GatherArgs& a, int num_tokens, cudaStream_t stream) {
  const int rw = 256 / D, groups = (2 * a.num_kv_heads + rw - 1) / rw, warps = groups < 8 ? groups : 8;
  const dim3 grid((num_tokens + kGatherTokens - 1) / kGatherTokens, (groups + warps - 1) / warps);
  return launch_pdl(cache_gather_kernel<T, FMT, D, kGatherTokens>, grid, dim3(32 * warps), 0, stream, a, num_tokens);
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
