// pa_decode_fp4.cu -- single-token decode attention over an E2M1 cache.
//
// One CTA per (partition, sequence, kv head), as in pa_decode.cu.  A warp owns every
// NW-th chunk of 32 tokens and runs its own ring of bulk copies: a (block, head)
// run is contiguous, so a chunk of K is one copy per block (two where a block
// holds more than the chunk: codes, then block scales), one lane each, and
// table entries are read one chunk ahead.  Warps meet only at the end, to merge.
//
// Both products run as m16n8k16 matrix instructions in f16 with fp32 sums, the
// cache always on the 16-row side and the group's query heads on the 8-column side:
//   S^T (tokens x heads) = K q^T,   O^T (dims x heads) += V^T P^T.
// A code times its block scale has at most 6 significant bits and lies in
// [2^-10, 2688], so the widened operands are exact in f16, and the warp builds them
// from codes in registers: no second pass through shared memory.  A thread
// takes 16-byte (K) and 8-byte (V) pieces of rows as they lie; the order of dims within
// a contraction, of tokens within a tile and of output rows is free, and is
// chosen so that a thread's fragment is what it loaded:
//   K: thread (g, t) = (lane / 4, lane % 4) holds dims [t D/4, (t + 1) D/4) of
//      the tile's tokens perm(g) and perm(g) + 8;
//   V: thread (g, t) holds dims [g D/8, (g + 1) D/8) of tokens t, t + 4, t + 8, t + 12;
//      nibbles of two tokens are paired into bytes (one shift and one 3-input
//      logic op per four) before widening, since a register pairs tokens.
// The 8 x 8 transposes from S^T's layout to P^T's are one movmatrix each.
//
// Softmax per warp in the log2 domain.  The reference m of a head moves only when a
// logit exceeds it by more than 2^8: p <= 256 stays within f16, and the warp-wide
// maximum and rescaling are rare.  Any m gives the same quotient.
//
// Roundings: q is bf16 or f16; a bf16 row is scaled by a power of two to a
// largest magnitude in [2^14, 2^15) and is then exact in f16 down to 2^-29 of it.
// p enters the second product as one f16 for bf16 outputs (2^-11 relative, against
// the output's 2^-8) and as hi + lo, 22 bits, for f16 outputs.  Sums, the
// softmax statistics and the partial results are fp32.
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "pa_common.cuh"
#include "pa_fp4.cuh"
#include "pa_internal.h"

namespace pa {

constexpr int kFp4Warps = 4;
constexpr int kFp4Stages = 4;
constexpr int kFp4Chunk = 32;  // tokens a stage holds

template <int D>
struct Fp4Smem {
  static constexpr int kTokenBytes = D * 9 / 16;
  static constexpr int kPoolBytes = kFp4Chunk * kTokenBytes;  // K or V of one stage
  static constexpr int kStageBytes = 2 * kPoolBytes;
  static constexpr int kBars = kFp4Warps * kFp4Stages * kStageBytes;
  static constexpr int kTotal = kBars + kFp4Warps * kFp4Stages * 8;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// Untiled bulk copy global -> shared, completion counted on an mbarrier; addresses and size in 16 bytes.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// NT: column tiles of 8 query heads (group <= 8 NT).
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kFp4Warps * 32, 3)
decode_fp4_kernel(const DecodeArgs a, const unsigned char* __restrict__ k_pool,
                  const unsigned char* __restrict__ v_pool, const int copy_tokens) {
  using L = Fp4Smem<D>;
  constexpr bool kLo = std::is_same<T, __half>::value;  // p as hi + lo
  constexpr int NW = kFp4Warps, NST = kFp4Stages, CT = kFp4Chunk, TILES = CT / 16;
  constexpr int KW = D / 32;   // words of K codes a thread takes per row
  constexpr int VW = D / 64;   // words of V codes a thread takes per row
  constexpr int MT = VW * 4;   // 16-row tiles of output dims
  extern __shared__ __align__(128) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t stage0 = smem_addr(smem) + warp * NST * L::kStageBytes;
  const uint32_t bar0 = smem_addr(smem) + L::kBars + warp * NST * 8;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < NST; ++i) mbar_init(bar0 + i * 8, 1);
    mbar_init_fence();
  }
  __syncwarp();
  pdl_wait();  // the append before this decode must have landed
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
  const int G = a.group;
  const size_t head0 = (size_t)s * a.num_q_heads + kvh * G;
  if (ctx == 0) {
    if (part == 0)
      for (int i = threadIdx.x; i < G * D; i += NW * 32) a.out[head0 * D + i] = 0;
    return;
  }
  const int t_begin = part * a.own_tokens;
  if (t_begin >= ctx) return;
  const int t_end = min(ctx, t_begin + a.own_tokens);
  const int n_chunks = (t_end - t_begin + CT - 1) / CT;
  const int n_mine = warp < n_chunks ? (n_chunks - warp + NW - 1) / NW : 0;

  // ---- copies: lane (sub, piece, pool) moves one piece of one group of
  // copy_tokens (8, 16 or 32) tokens, which never crosses a block
  const int R = copy_tokens, bs = a.block_size;
  const bool whole = R == bs;  // codes and scales of the group are one run
  const int c_sub = lane >> 2, c_piece = (lane >> 1) & 1;
  const bool c_lane = c_sub * R < CT && (c_piece == 0 || !whole);
  const uint32_t c_bytes = whole ? R * L::kTokenBytes : c_piece ? R * (D / 16) : R * (D / 2);
  const unsigned char* c_pool = (lane & 1) ? v_pool : k_pool;
  const uint32_t c_dst = ((lane & 1) ? L::kPoolBytes : 0) + c_sub * R * L::kTokenBytes + (c_piece ? R * (D / 2) : 0);
  const long long run_bytes = fp4_head_bytes(bs, D);
  const int32_t* table = a.block_tables + (size_t)s * a.max_blocks_per_seq;
  // First token of this lane's group in chunk k (its own chunks), or -1.
  auto group_token = [&](int k) {
    const int tok = t_begin + (warp + k * NW) * CT + c_sub * R;
    return c_lane && k < n_mine && tok < t_end ? tok : -1;
  };
  auto entry = [&](int k) {
    const int tok = group_token(k);
    return tok >= 0 ? __ldg(table + tok / bs) : 0;
  };
  auto issue = [&](int k, int blk) {
    const int tok = group_token(k);
    const uint32_t bar = bar0 + (k % NST) * 8, dst = stage0 + (k % NST) * L::kStageBytes + c_dst;
    bool copy = tok >= 0;
    if (copy && (blk < 0 || blk >= a.num_blocks)) {  // rows outside the pool read as zeros
      report(a.err, kErrBlockId);
      for (uint32_t i = 0; i < c_bytes; i += 16)
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + i), "r"(0) : "memory");
      copy = false;
    }
    const uint32_t total = __reduce_add_sync(0xffffffffu, copy ? c_bytes : 0u);
    if (lane == 0) mbar_arrive_expect_tx(bar, total);
    __syncwarp();
    if (copy) {
      const int off = tok % bs;
      const unsigned char* src = c_pool + ((long long)blk * a.num_kv_heads + kvh) * run_bytes +
                                 (c_piece ? bs * (D / 2) + off * (D / 16) : off * (D / 2));
      bulk_load(dst, src, c_bytes, bar);
    }
  };
  {
    int e[NST];
#pragma unroll
    for (int k = 0; k < NST; ++k) e[k] = entry(k);
#pragma unroll
    for (int k = 0; k < NST; ++k)
      if (k < n_mine) issue(k, e[k]);
  }
  int next_entry = entry(NST);

  // ---- queries as column fragments: thread (g, t) holds dims [t D/4, (t + 1) D/4) of heads g, g + 8
  const float cscale = a.scale_log2 * __ldg(a.k_scale + kvh);
  uint32_t bq[NT][KW * 4];
  float xs[NT][2];  // logit scale of this thread's columns 2t, 2t + 1
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int h = n * 8 + g;
    uint32_t w[KW * 4];
#pragma unroll
    for (int i = 0; i < KW; ++i) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (h < G) v = *reinterpret_cast<const uint4*>(a.q + (head0 + h) * D + t * (D / 4) + i * 8);
      w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
    }
    if constexpr (kLo) {
#pragma unroll
      for (int i = 0; i < KW * 4; ++i) bq[n][i] = w[i];
      xs[n][0] = xs[n][1] = cscale;
    } else {
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < KW * 4; ++i) {
        const float2 f = Elem<T>::to_f2(w[i]);
        top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = max((int)(__float_as_uint(top) >> 23), 15);  // 2^(e - 127) <= top
      const float up = __uint_as_float((uint32_t)(268 - e) << 23);     // 2^(141 - e)
      const float down = __uint_as_float((uint32_t)(e - 14) << 23);
#pragma unroll
      for (int i = 0; i < KW * 4; ++i) {
        const float2 f = Elem<T>::to_f2(w[i]);
        bq[n][i] = f16x2_of(f.x * up, f.y * up);
      }
      xs[n][0] = cscale * __shfl_sync(0xffffffffu, down, 8 * t);
      xs[n][1] = cscale * __shfl_sync(0xffffffffu, down, 8 * t + 4);
    }
  }

  // ---- where this thread's pieces of a tile lie: a tile is 16 tokens, its rows
  // 8 .. 15 in a group of their own when R is 8, two tiles share a group when R is 32
  const uint32_t code_tile = R == 32 ? 16 * (D / 2) : 16 * L::kTokenBytes;
  const uint32_t scale_tile = R == 32 ? 16 * (D / 16) : 16 * L::kTokenBytes;
  const uint32_t code_half = R == 8 ? 8 * L::kTokenBytes : 8 * (D / 2);
  const uint32_t scale_half = R == 8 ? 8 * L::kTokenBytes : 8 * (D / 16);
  const uint32_t scale_base = R * (D / 2);
  const int k_row = (g >> 1) + 4 * (g & 1);  // token of the tile's row g (row g + 8: 8 tokens on)
  const uint32_t k_code = k_row * (D / 2) + t * (D / 8);
  const uint32_t k_sc = scale_base + k_row * (D / 16) + t * (D / 64);
  const uint32_t v_code = L::kPoolBytes + t * (D / 2) + g * (D / 16);
  const uint32_t v_sc = L::kPoolBytes + scale_base + t * (D / 16) + g * (D / 64) / 2;

  float o[MT][NT][4], m[NT][2], l[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][n][j] = 0.f;
    m[n][0] = m[n][1] = -1e30f;
    l[n][0] = l[n][1] = 0.f;
  }

  bool ok = true;
  int k = 0;
  for (; k < n_mine; ++k) {
    if (!mbar_wait(bar0 + (k % NST) * 8, (k / NST) & 1, a.err)) { ok = false; break; }
    const uint32_t st = stage0 + (k % NST) * L::kStageBytes;
    const int n_valid = t_end - (t_begin + (warp + k * NW) * CT);  // of this chunk's 32 tokens
    const bool tail = n_valid < CT;

    // ---- logits
    float x[TILES][NT][4];
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
      uint32_t ca[KW], cb[KW], sa, sb;
      const uint32_t ka = st + k_code + i * code_tile, kb = ka + code_half;
      const uint32_t ks = st + k_sc + i * scale_tile;
      if constexpr (D == 128) {
        const uint4 u = lds128(ka), w = lds128(kb);
        ca[0] = u.x; ca[1] = u.y; ca[2] = u.z; ca[3] = u.w;
        cb[0] = w.x; cb[1] = w.y; cb[2] = w.z; cb[3] = w.w;
        sa = e4m3x2_to_h2((uint16_t)lds16(ks));
        sb = e4m3x2_to_h2((uint16_t)lds16(ks + scale_half));
      } else {
        const uint2 u = lds64(ka), w = lds64(kb);
        ca[0] = u.x; ca[1] = u.y;
        cb[0] = w.x; cb[1] = w.y;
        sa = e4m3x2_to_h2((uint16_t)lds8(ks));
        sb = e4m3x2_to_h2((uint16_t)lds8(ks + scale_half));
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][n][j] = 0.f;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        const uint32_t pick = w < 2 ? 0x1010 : 0x3232;  // scale of this word's 16 dims, twice
        const uint32_t da = __byte_perm(sa, 0, pick), db = __byte_perm(sb, 0, pick);
        uint32_t fa[4], fb[4];
        e2m1x8_to_h2(ca[w], fa);
        e2m1x8_to_h2(cb[w], fb);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          fa[j] = hmul2(fa[j], da);
          fb[j] = hmul2(fb[j], db);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_f16(x[i][n], fa[0], fb[0], fa[1], fb[1], bq[n][4 * w], bq[n][4 * w + 1]);
          mma_f16(x[i][n], fa[2], fb[2], fa[3], fb[3], bq[n][4 * w + 2], bq[n][4 * w + 3]);
        }
      }
    }

    // ---- softmax
    bool grow = false;
    float top[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      top[n][0] = top[n][1] = -INFINITY;
#pragma unroll
      for (int i = 0; i < TILES; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float v = x[i][n][j] * xs[n][j & 1];
          if (tail && i * 16 + k_row + (j >> 1) * 8 >= n_valid) v = -INFINITY;
          x[i][n][j] = v;
          top[n][j & 1] = fmaxf(top[n][j & 1], v);
        }
      grow |= top[n][0] > m[n][0] + 8.f || top[n][1] > m[n][1] + 8.f;
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float v = top[n][j];
#pragma unroll
          for (int d = 4; d <= 16; d <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
          const float mn = fmaxf(m[n][j], v), al = ex2(m[n][j] - mn);
          m[n][j] = mn;
          l[n][j] *= al;
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            o[i][n][j] *= al;
            o[i][n][j + 2] *= al;
          }
        }
    }

    // ---- probabilities as column fragments, and O^T += V^T P^T
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
      uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float p0 = ex2(x[i][n][2 * j] - m[n][0]), p1 = ex2(x[i][n][2 * j + 1] - m[n][1]);
          l[n][0] += p0;
          l[n][1] += p1;
          const uint32_t h = f16x2_of(p0, p1);
          hi[n][j] = transpose_8x8(h);
          if constexpr (kLo) {
            const float2 f = h2_to_f2(h);
            lo[n][j] = transpose_8x8(f16x2_of(p0 - f.x, p1 - f.y));
          }
        }
      const uint32_t va = st + v_code + i * code_tile, vs = st + v_sc + i * scale_tile;
      uint32_t c[4][VW], sc[2];
#pragma unroll
      for (int r = 0; r < 4; ++r) {  // tokens t, t + 4, t + 8, t + 12 of the tile
        const uint32_t at = va + (r & 1) * 4 * (D / 2) + (r >> 1) * code_half;
        if constexpr (D == 128) {
          const uint2 u = lds64(at);
          c[r][0] = u.x; c[r][1] = u.y;
        } else {
          c[r][0] = lds32(at);
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t s0 = lds8(vs + r * scale_half), s1 = lds8(vs + 4 * (D / 16) + r * scale_half);
        if (tail) {  // what lies behind the last token may be anything: codes are finite, scales need not be
          if (i * 16 + t + 8 * r >= n_valid) s0 = 0;
          if (i * 16 + t + 4 + 8 * r >= n_valid) s1 = 0;
        }
        sc[r] = e4m3x2_to_h2((uint16_t)(s0 | (s1 << 8)));
      }
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        uint32_t ev[2][4], od[2][4];  // [token pair][j]: dims 2j and 2j + 1 of the word
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t u0 = c[2 * r][w], u1 = c[2 * r + 1][w];
          e2m1x8_to_h2((u0 & 0x0f0f0f0fu) | ((u1 << 4) & 0xf0f0f0f0u), ev[r]);
          e2m1x8_to_h2(((u0 >> 4) & 0x0f0f0f0fu) | (u1 & 0xf0f0f0f0u), od[r]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            ev[r][j] = hmul2(ev[r][j], sc[r]);
            od[r][j] = hmul2(od[r][j], sc[r]);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_f16(o[4 * w + j][n], ev[0][j], od[0][j], ev[1][j], od[1][j], hi[n][0], hi[n][1]);
            if constexpr (kLo)
              mma_f16(o[4 * w + j][n], ev[0][j], od[0][j], ev[1][j], od[1][j], lo[n][0], lo[n][1]);
          }
      }
    }
    __syncwarp();
    // the stage is free again: refill it
    if (k + NST < n_mine) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      issue(k + NST, next_entry);
      next_entry = entry(k + NST + 1);
    }
  }
  if (!ok)  // let every copy in flight land before the CTA exits
    for (int i = k; i < min(n_mine, k + NST); ++i) mbar_wait(bar0 + (i % NST) * 8, (i / NST) & 1, a.err);

  // ---- merge the warps (the stages are all consumed)
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int d = 4; d <= 16; d <<= 1) l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], d);
  const int any_failed = __syncthreads_or(!ok);
  float* mg_m = reinterpret_cast<float*>(smem);  // [NW][G] m, [NW][G] l, [NW][G][D] o
  float* mg_l = mg_m + NW * G;
  float* mg_o = mg_l + NW * G;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int h = n * 8 + 2 * t + j;
      if (h < G) {
        if (g == 0) {
          mg_m[warp * G + h] = m[n][j];
          mg_l[warp * G + h] = l[n][j];
        }
        float* row = mg_o + (warp * G + h) * D + g * (D / 8);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          row[2 * i] = o[i][n][j];
          row[2 * i + 1] = o[i][n][j + 2];
        }
      }
    }
  __syncthreads();
  const bool direct = ctx <= a.own_tokens;
  const float v_scale = __ldg(a.v_scale + kvh);
  for (int i = threadIdx.x; i < G * D; i += NW * 32) {
    const int h = i / D, d = i % D;
    float M = -INFINITY, num = 0.f, den = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, mg_m[w * G + h]);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float wt = exp2f(mg_m[w * G + h] - M);  // a warp without tokens: l and o are 0
      num = fmaf(wt, mg_o[(w * G + h) * D + d], num);
      den = fmaf(wt, mg_l[w * G + h], den);
    }
    num *= v_scale;
    if (any_failed) num = __int_as_float(0x7fc00000), den = 1.f;
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

template <typename T, int D, int NT>
cudaError_t launch_fp4(const DecodeArgs& a, const void* k, const void* v, cudaStream_t stream, int* launches) {
  static_assert(kFp4Warps * 8 * NT * (D + 2) * 4 <= Fp4Smem<D>::kBars, "the merge must fit the stages");
  const long long grid = (long long)a.grid_parts * a.num_seqs * a.num_kv_heads;
  if (grid <= 0) return cudaSuccess;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  auto* kern = decode_fp4_kernel<T, D, NT>;
  constexpr int smem = Fp4Smem<D>::kTotal;
  static std::atomic<uint64_t> configured{0};  // a bit per device; setting the attribute twice is harmless
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(configured.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) configured.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  // a copy's tokens lie in one block, and partitions start at whole copies
  int copy = 32;
  while (a.block_size % copy || a.own_tokens % copy) copy /= 2;
  e = launch_pdl(kern, dim3((unsigned)grid), dim3(kFp4Warps * 32), smem, stream, a,
                 static_cast<const unsigned char*>(k), static_cast<const unsigned char*>(v), copy);
  if (e == cudaSuccess) ++*launches;
  return e;
}

template <typename T, int D>
cudaError_t launch_fp4_group(const DecodeArgs& a, int group, const void* k, const void* v, cudaStream_t st, int* n) {
  return group <= 8 ? launch_fp4<T, D, 1>(a, k, v, st, n) : launch_fp4<T, D, 2>(a, k, v, st, n);
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
