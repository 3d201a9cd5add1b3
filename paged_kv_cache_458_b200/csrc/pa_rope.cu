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
// CTA takes one token: a thread's unit index, and with it its cos and sin, are
// the same for all rows it walks over.
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

template <typename T, int FMT, int D>
__global__ void __launch_bounds__(256)
rope_append_kernel(const RopeArgs a) {
  constexpr int UNITS = D / 8;        // lanes per row
  constexpr int RW = 32 / UNITS;      // rows per warp and step
  pdl_wait();  // a copy-on-write of this slot's block must land first
  pdl_launch_dependents();
  const int t = blockIdx.x;
  const long long slot = __ldg(a.slot_mapping + t);
  if (slot < 0) return;               // padding
  if (slot >= a.num_slots) {
    if (threadIdx.x == 0 && blockIdx.y == 0) report(a.err, kErrSlot);
    return;
  }
  const int lane = threadIdx.x & 31, u = lane % UNITS;
  const bool rot_unit = u * 8 < a.rotary_dim;

  // cos and (signed) sin of this thread's 8 dims, and the lane of its partner unit
  float cs[8], sn[8];
  int partner = lane;
  if (a.rotary_dim > 0) {
    const int pos = __ldg(a.positions + t);
    if (pos < 0 || pos >= a.max_position) {
      if (threadIdx.x == 0 && blockIdx.y == 0) report(a.err, kErrPosition);
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
        const int hu = half / 8;       // units per half
        const bool first = u < hu;
        partner = first ? lane + hu : lane - hu;
        const float* c = row + (first ? u : u - hu) * 8;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const float4 cv = __ldg(reinterpret_cast<const float4*>(c + i));
          const float4 sv = __ldg(reinterpret_cast<const float4*>(c + half + i));
          cs[i] = cv.x; cs[i + 1] = cv.y; cs[i + 2] = cv.z; cs[i + 3] = cv.w;
          sn[i] = first ? -sv.x : sv.x; sn[i + 1] = first ? -sv.y : sv.y;
          sn[i + 2] = first ? -sv.z : sv.z; sn[i + 3] = first ? -sv.w : sv.w;
        }
      }
    }
  }

  const int rows = a.num_q_heads + 2 * a.num_kv_heads;
  const int step = gridDim.y * (blockDim.x >> 5) * RW;
  const int w0 = (blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5)) * RW;
  for (int r0 = w0; r0 < rows; r0 += step) {
    const int r = r0 + lane / UNITS;
    const bool live = r < rows;
    const bool is_q = r < a.num_q_heads;
    const int h = is_q ? r : (r - a.num_q_heads) % a.num_kv_heads;
    const bool is_v = r >= a.num_q_heads + a.num_kv_heads;
    const uint16_t* src = is_q   ? a.q + (long long)t * a.q_stride
                          : is_v ? a.v + (long long)t * a.v_stride
                                 : a.k + (long long)t * a.k_stride;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (live) x = *reinterpret_cast<const uint4*>(src + h * D + u * 8);
    const bool rotate = rot_unit && !is_v;
    if (a.rotary_dim > 0) {
      uint4 p;
      if (a.interleaved) {
        p = make_uint4(__byte_perm(x.x, 0, 0x1032), __byte_perm(x.y, 0, 0x1032),
                       __byte_perm(x.z, 0, 0x1032), __byte_perm(x.w, 0, 0x1032));
      } else {
        p = make_uint4(__shfl_sync(0xffffffffu, x.x, partner), __shfl_sync(0xffffffffu, x.y, partner),
                       __shfl_sync(0xffffffffu, x.z, partner), __shfl_sync(0xffffffffu, x.w, partner));
      }
      if (rotate) {
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, pw[4] = {p.x, p.y, p.z, p.w};
        uint32_t yw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 xf = Elem<T>::to_f2(xw[i]), pf = Elem<T>::to_f2(pw[i]);
          yw[i] = pack2<T>(__fadd_rn(__fmul_rn(xf.x, cs[2 * i]), __fmul_rn(pf.x, sn[2 * i])),
                           __fadd_rn(__fmul_rn(xf.y, cs[2 * i + 1]), __fmul_rn(pf.y, sn[2 * i + 1])));
        }
        x = make_uint4(yw[0], yw[1], yw[2], yw[3]);
      }
    }
    if (is_q) {
      if (live) *reinterpret_cast<uint4*>(a.q_out + (long long)t * a.q_out_stride + h * D + u * 8) = x;
    }
    unsigned char* pool = static_cast<unsigned char*>(is_v ? a.v_cache : a.k_cache);
    const bool store = live && !is_q;
    if constexpr (FMT == kFmt16) {
      if (store)
        *reinterpret_cast<uint4*>(pool + ((slot * a.num_kv_heads + h) * D + u * 8) * 2) = x;
    } else {
      const float hs = store ? __ldg((is_v ? a.v_scale : a.k_scale) + h) : 1.f;
      const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
      float f[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = Elem<T>::to_f2(xw[i]);
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
      }
      if constexpr (FMT == kFmtFp8) {
        uint32_t o[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 8; i += 2)
          o[i / 4] |= (uint32_t)__nv_cvt_float2_to_fp8x2(
                          make_float2(__fdiv_rn(f[i], hs), __fdiv_rn(f[i + 1], hs)), __NV_SATFINITE,
                          __NV_E4M3)
                      << (8 * (i % 4));
        if (store)
          *reinterpret_cast<uint2*>(pool + (slot * a.num_kv_heads + h) * D + u * 8) =
              make_uint2(o[0], o[1]);
      } else {
        float amax = 0.f;
        bool nan = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          amax = fmaxf(amax, fabsf(f[i]));
          nan |= f[i] != f[i];
        }
        // a block of 16 dims is two adjacent lanes
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        nan |= __shfl_xor_sync(0xffffffffu, (int)nan, 1) != 0;
        float rs;
        const uint8_t s = fp4_block_scale(amax, nan, hs, &rs);
        uint32_t o = 0;
#pragma unroll
        for (int i = 0; i < 8; i += 2)
          o |= e2m1x2_of(__fmul_rn(f[i], rs), __fmul_rn(f[i + 1], rs)) << (4 * i);
        if (store) {
          const long long block = slot / a.block_size;
          const int off = (int)(slot % a.block_size);
          unsigned char* run =
              pool + (block * a.num_kv_heads + h) * fp4_head_bytes(a.block_size, D);
          *reinterpret_cast<uint32_t*>(run + off * (D / 2) + u * 4) = o;
          if ((u & 1) == 0) run[fp4_code_bytes(a.block_size, D) + off * (D / 16) + u / 2] = s;
        }
      }
    }
  }
}

// Rows of a cache back into 16-bit rows: stored value = code * block scale *
// head scale (one fp32 rounding), rounded to the element type; a 16-bit
// cache is copied bit by bit.  Same split as above, over the 2 Hkv rows of a token.
template <typename T, int FMT, int D>
__global__ void __launch_bounds__(256)
cache_gather_kernel(const GatherArgs a) {
  constexpr int UNITS = D / 8, RW = 32 / UNITS;
  pdl_wait();
  pdl_launch_dependents();
  const int t = blockIdx.x;
  const long long slot = __ldg(a.slot_mapping + t);
  if (slot < 0) return;
  const bool bad = slot >= a.num_slots;  // such a row reads as zeros
  if (bad && threadIdx.x == 0 && blockIdx.y == 0) report(a.err, kErrSlot);
  const int lane = threadIdx.x & 31, u = lane % UNITS;
  const int rows = 2 * a.num_kv_heads;
  const int step = gridDim.y * (blockDim.x >> 5) * RW;
  for (int r = (blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5)) * RW + lane / UNITS; r < rows; r += step) {
    const bool is_v = r >= a.num_kv_heads;
    const int h = is_v ? r - a.num_kv_heads : r;
    const unsigned char* pool = static_cast<const unsigned char*>(is_v ? a.v_cache : a.k_cache);
    uint4 x = make_uint4(0, 0, 0, 0);
    if (!bad) {
      if constexpr (FMT == kFmt16) {
        x = __ldg(reinterpret_cast<const uint4*>(pool + ((slot * a.num_kv_heads + h) * D + u * 8) * 2));
      } else {
        const float hs = __ldg((is_v ? a.v_scale : a.k_scale) + h);
        float2 f[4];
        if constexpr (FMT == kFmtFp8) {
          const uint2 w = __ldg(reinterpret_cast<const uint2*>(pool + (slot * a.num_kv_heads + h) * D + u * 8));
          f[0] = e4m3x2_to_f2((uint16_t)w.x);
          f[1] = e4m3x2_to_f2((uint16_t)(w.x >> 16));
          f[2] = e4m3x2_to_f2((uint16_t)w.y);
          f[3] = e4m3x2_to_f2((uint16_t)(w.y >> 16));
        } else {
          const long long block = slot / a.block_size;
          const int off = (int)(slot % a.block_size);
          const unsigned char* run = pool + (block * a.num_kv_heads + h) * fp4_head_bytes(a.block_size, D);
          const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(run + off * (D / 2) + u * 4));
          const float s = e4m3_to_f(__ldg(run + fp4_code_bytes(a.block_size, D) + off * (D / 16) + u / 2));
          uint32_t hv[4];
          e2m1x8_to_h2(w, hv);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f[i] = h2_to_f2(hv[i]);
            f[i].x *= s;  // exact: 2 significant bits times 4
            f[i].y *= s;
          }
        }
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack2<T>(__fmul_rn(f[i].x, hs), __fmul_rn(f[i].y, hs));
        x = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    uint16_t* out = (is_v ? a.v_out : a.k_out) + ((long long)t * a.num_kv_heads + h) * D + u * 8;
    *reinterpret_cast<uint4*>(out) = x;
  }
}

namespace {

template <typename Args, typename Kern>
cudaError_t launch_rows(Kern kern, const Args& a, int num_tokens, int rows, int head_dim,
                        cudaStream_t stream, int* launches) {
  const int rw = 256 / head_dim, warp_rows = (rows + rw - 1) / rw;
  const int warps = warp_rows < 8 ? warp_rows : 8;
  cudaError_t e = launch_pdl(kern, dim3(num_tokens), dim3(32 * warps), 0, stream, a);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs& a, int dtype, int head_dim, int format, int num_tokens,
                               cudaStream_t stream, int* launches) {
  auto go = [&](auto kern) {
    return launch_rows(kern, a, num_tokens, a.num_q_heads + 2 * a.num_kv_heads, head_dim, stream, launches);
  };
  auto fmt = [&](auto t, auto d) {
    using T = decltype(t);
    constexpr int D = decltype(d)::value;
    if (format == kFmt16) return go(rope_append_kernel<T, kFmt16, D>);
    if (format == kFmtFp8) return go(rope_append_kernel<T, kFmtFp8, D>);
    return go(rope_append_kernel<T, kFmtFp4, D>);
  };
  auto dim = [&](auto t) {
    return head_dim == 128 ? fmt(t, std::integral_constant<int, 128>{}) : fmt(t, std::integral_constant<int, 64>{});
  };
  return dtype == 0 ? dim(__half{}) : dim(__nv_bfloat16{});
}

cudaError_t launch_cache_gather(const GatherArgs& a, int dtype, int head_dim, int format, int num_tokens,
                                cudaStream_t stream, int* launches) {
  auto go = [&](auto kern) {
    return launch_rows(kern, a, num_tokens, 2 * a.num_kv_heads, head_dim, stream, launches);
  };
  auto fmt = [&](auto t, auto d) {
    using T = decltype(t);
    constexpr int D = decltype(d)::value;
    if (format == kFmt16) return go(cache_gather_kernel<T, kFmt16, D>);
    if (format == kFmtFp8) return go(cache_gather_kernel<T, kFmtFp8, D>);
    return go(cache_gather_kernel<T, kFmtFp4, D>);
  };
  auto dim = [&](auto t) {
    return head_dim == 128 ? fmt(t, std::integral_constant<int, 128>{}) : fmt(t, std::integral_constant<int, 64>{});
  };
  return dtype == 0 ? dim(__half{}) : dim(__nv_bfloat16{});
}

}  // namespace pa
