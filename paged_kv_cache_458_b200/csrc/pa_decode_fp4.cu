// pa_decode_fp4.cu -- single-token decode attention over an E2M1 cache.
//
// One CTA per (partition, sequence, kv head), as pa_decode.cu.  Warp w takes
// tokens w, w + NW, ... of the partition; a lane holds D / 32 consecutive dims of
// the group's queries, widens its codes of a K row, and a butterfly completes
// the logits.  Online softmax per warp in the log2 domain (the K head scale
// folded into the query, the V head scale into the output), the warps merged in
// shared memory, partitions by the merge kernel of pa_decode.cu.  All sums fp32.
#include <cuda_runtime.h>

#include "pa_common.cuh"
#include "pa_fp4.cuh"
#include "pa_internal.h"

namespace pa {

constexpr int kFp4Warps = 4;

// This lane's D / 32 stored values of row `off` of one (block, head) run, without the head scale.
template <int D>
__device__ __forceinline__ void load_fp4_slice(const unsigned char* run, int off, int block_size, int lane,
                                               float (&x)[D / 32]) {
  const float s = e4m3_to_f(__ldg(run + fp4_code_bytes(block_size, D) + off * (D / 16) + lane / (512 / D)));
  const unsigned char* codes = run + off * (D / 2) + lane * (D / 64);
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const float2 v = e2m1x2_to_f2(__ldg(codes + i));
    x[2 * i] = v.x * s;
    x[2 * i + 1] = v.y * s;
  }
}

template <typename T, int D, int G>
__global__ void __launch_bounds__(kFp4Warps * 32)
decode_fp4_kernel(const DecodeArgs a, const unsigned char* __restrict__ k_pool,
                  const unsigned char* __restrict__ v_pool) {
  constexpr int VEC = D / 32, NW = kFp4Warps;
  __shared__ float mg_m[NW][G], mg_l[NW][G], mg_acc[NW][G][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_launch_dependents();

  int bid = blockIdx.x;
  const int kvh = bid % a.num_kv_heads;
  bid /= a.num_kv_heads;
  const int s = bid % a.num_seqs, part = bid / a.num_seqs;
  int ctx = __ldg(a.context_lens + s);
  if (ctx < 0 || ctx > a.max_context_len) {
    if (part == 0 && kvh == 0 && threadIdx.x == 0) report(a.err, kErrContextLen);
    ctx = max(0, min(ctx, a.max_context_len));
  }
  const size_t head0 = (size_t)s * a.num_q_heads + kvh * G;
  if (ctx == 0) {
    if (part == 0)
      for (int i = threadIdx.x; i < G * D; i += NW * 32) a.out[head0 * D + i] = 0;
    return;
  }
  const int t_begin = part * a.own_tokens;
  if (t_begin >= ctx) return;
  const int t_end = min(ctx, t_begin + a.own_tokens);

  const float qs = a.scale_log2 * __ldg(a.k_scale + kvh);
  float q[G][VEC], acc[G][VEC], m[G], l[G];
#pragma unroll
  for (int h = 0; h < G; ++h) {
#pragma unroll
    for (int v = 0; v < VEC; v += 2) {
      const float2 x = Elem<T>::to_f2(
          *reinterpret_cast<const uint32_t*>(a.q + (head0 + h) * D + lane * VEC + v));
      q[h][v] = x.x * qs;
      q[h][v + 1] = x.y * qs;
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) acc[h][v] = 0.f;
    m[h] = -INFINITY;
    l[h] = 0.f;
  }
  const long long run_bytes = fp4_head_bytes(a.block_size, D);
  for (int tok = t_begin + warp; tok < t_end; tok += NW) {
    const int blk = __ldg(a.block_tables + (size_t)s * a.max_blocks_per_seq + tok / a.block_size);
    const bool bad = blk < 0 || blk >= a.num_blocks;
    if (bad && lane == 0) report(a.err, kErrBlockId);
    const long long run = ((long long)blk * a.num_kv_heads + kvh) * run_bytes;
    const int off = tok % a.block_size;
    float kf[VEC] = {}, vf[VEC] = {};
    if (!bad) {  // a row outside the pool reads as zeros
      load_fp4_slice<D>(k_pool + run, off, a.block_size, lane, kf);
      load_fp4_slice<D>(v_pool + run, off, a.block_size, lane, vf);
    }
#pragma unroll
    for (int h = 0; h < G; ++h) {
      float x = 0.f;
#pragma unroll
      for (int v = 0; v < VEC; ++v) x = fmaf(q[h][v], kf[v], x);
#pragma unroll
      for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      const float mn = fmaxf(m[h], x), al = exp2f(m[h] - mn), p = exp2f(x - mn);
      l[h] = l[h] * al + p;
      m[h] = mn;
#pragma unroll
      for (int v = 0; v < VEC; ++v) acc[h][v] = fmaf(p, vf[v], acc[h][v] * al);
    }
  }
#pragma unroll
  for (int h = 0; h < G; ++h) {
    mg_m[warp][h] = m[h];
    mg_l[warp][h] = l[h];
#pragma unroll
    for (int v = 0; v < VEC; ++v) mg_acc[warp][h][lane * VEC + v] = acc[h][v];
  }
  __syncthreads();
  const bool direct = ctx <= a.own_tokens;
  const float vs = __ldg(a.v_scale + kvh);
  for (int i = threadIdx.x; i < G * D; i += NW * 32) {
    const int h = i / D, d = i % D;
    float M = -INFINITY, num = 0.f, den = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, mg_m[w][h]);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float wt = mg_l[w][h] == 0.f ? 0.f : exp2f(mg_m[w][h] - M);  // a warp without tokens
      num = fmaf(wt, mg_acc[w][h][d], num);
      den = fmaf(wt, mg_l[w][h], den);
    }
    num *= vs;
    if (direct) {
      a.out[(head0 + h) * D + d] = Elem<T>::from_f(num / den);
    } else {
      const size_t slot = (head0 + h) * a.num_parts + part;
      a.ws_acc[slot * D + d] = num;
      if (d == 0) {
        a.ws_ml[2 * slot] = M;
        a.ws_ml[2 * slot + 1] = den;
      }
    }
  }
}

namespace {

template <typename T, int D, int G>
cudaError_t launch_fp4(const DecodeArgs& a, const void* k, const void* v, cudaStream_t stream, int* launches) {
  const long long grid = (long long)a.grid_parts * a.num_seqs * a.num_kv_heads;
  if (grid <= 0) return cudaSuccess;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaError_t e = launch_pdl(decode_fp4_kernel<T, D, G>, dim3((unsigned)grid), dim3(kFp4Warps * 32), 0, stream, a,
                             static_cast<const unsigned char*>(k), static_cast<const unsigned char*>(v));
  if (e == cudaSuccess) ++*launches;
  return e;
}

template <typename T, int D>
cudaError_t launch_fp4_group(const DecodeArgs& a, int group, const void* k, const void* v, cudaStream_t st, int* n) {
  switch (group) {
    case 1: return launch_fp4<T, D, 1>(a, k, v, st, n);
    case 2: return launch_fp4<T, D, 2>(a, k, v, st, n);
    case 4: return launch_fp4<T, D, 4>(a, k, v, st, n);
    case 8: return launch_fp4<T, D, 8>(a, k, v, st, n);
    case 16: return launch_fp4<T, D, 16>(a, k, v, st, n);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_decode_fp4(const DecodeArgs& a, int dtype, int head_dim, int group, const void* k_pool,
                              const void* v_pool, cudaStream_t stream, int* launches) {
  cudaError_t e;
  if (dtype == 0)
    e = head_dim == 128 ? launch_fp4_group<__half, 128>(a, group, k_pool, v_pool, stream, launches)
                        : launch_fp4_group<__half, 64>(a, group, k_pool, v_pool, stream, launches);
  else
    e = head_dim == 128 ? launch_fp4_group<__nv_bfloat16, 128>(a, group, k_pool, v_pool, stream, launches)
                        : launch_fp4_group<__nv_bfloat16, 64>(a, group, k_pool, v_pool, stream, launches);
  if (e != cudaSuccess) return e;
  return launch_decode_merge(a, dtype, head_dim, stream, launches);
}

}  // namespace pa
