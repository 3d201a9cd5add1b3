// pa_decode_fp4.cu -- single-token decode attention over an E2M1 cache.
//
// Work split.  An item is a (sequence, kv head) pair; its context is cut into chunks of
// 32 tokens.  The chunks of all items, in order, are split evenly into one
// span per CTA, CTAs filling the device once: long and short contexts
// balance, and only an item cut by a span's border needs merging.  Every CTA finds its
// span itself, by a scan over the context lengths.  In a span warp w takes
// every NW-th chunk, across items, through its own ring of bulk copies: a (block, head)
// run is contiguous, so a chunk of K is one copy per block (two where a block
// holds more than the copy: codes, then block scales), one lane each, and
// table entries are read one chunk ahead.  At an item's end the warps merge
// their states through shared memory, while the copies of the next items run.
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
constexpr int kFp4Chunk = 32;  // tokens a stage holds

template <int D, int NT>
struct Fp4Smem {
  // stages per warp and CTAs per SM: what registers and shared memory allow
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kCtas = NT == 1 ? 4 : 3;
  static constexpr int kTokenBytes = D * 9 / 16;
  static constexpr int kPoolBytes = kFp4Chunk * kTokenBytes;  // K or V of one stage
  static constexpr int kStageBytes = 2 * kPoolBytes;
  static constexpr int kMerge = kFp4Warps * kStages * kStageBytes;  // 3 warp states
  static constexpr int kStateBytes = (D / 16 + 1) * NT * 32 * 16;
  static constexpr int kBars = kMerge + 3 * kStateBytes;
  static constexpr int kScan = kBars + kFp4Warps * kStages * 8;
  static constexpr int kTotal = kScan + 32;
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

__device__ __forceinline__ float4 lds_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts_f4(uint32_t a, float x, float y, float z, float w) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(x), "f"(y), "f"(z), "f"(w) : "memory");
}

// NT: column tiles of 8 query heads (group <= 8 NT).
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kFp4Warps * 32, Fp4Smem<D, NT>::kCtas)
decode_fp4_kernel(const DecodeArgs a, const unsigned char* __restrict__ k_pool,
                  const unsigned char* __restrict__ v_pool, const int copy_tokens, int2* item_parts) {
  using L = Fp4Smem<D, NT>;
  constexpr bool kLo = std::is_same<T, __half>::value;  // p as hi + lo
  constexpr int NW = kFp4Warps, NST = L::kStages, CT = kFp4Chunk, TILES = CT / 16;
  constexpr int KW = D / 32;   // words of K codes a thread takes per row
  constexpr int VW = D / 64;   // words of V codes a thread takes per row
  constexpr int MT = VW * 4;   // 16-row tiles of output dims
  extern __shared__ __align__(128) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t stage0 = smem_addr(smem) + warp * NST * L::kStageBytes;
  const uint32_t bar0 = smem_addr(smem) + L::kBars + warp * NST * 8;
  const uint32_t states = smem_addr(smem) + L::kMerge + lane * 16;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < NST; ++i) mbar_init(bar0 + i * 8, 1);
    mbar_init_fence();
  }
  __syncwarp();
  pdl_wait();  // the append before this decode must have landed
  pdl_launch_dependents();

  // ---- this CTA's span of chunks, and the sequence it starts in
  const int S = a.num_seqs, Hkv = a.num_kv_heads, G = a.group;
  auto context = [&](int s) { return max(0, min(__ldg(a.context_lens + s), a.max_context_len)); };
  int span_begin = 0, span_end = 0, chunks, ctas, seq, seq_base;  // seq_base: the number of the sequence's first chunk
  {
    int* sh = reinterpret_cast<int*>(smem + L::kScan);
    const int per = (S + NW * 32 - 1) / (NW * 32), lo = min(S, (int)threadIdx.x * per), hi = min(S, lo + per);
    int sum = 0;
    bool bad = false;
    for (int s = lo; s < hi; ++s) {
      sum += (context(s) + CT - 1) / CT;
      const int c = __ldg(a.context_lens + s);
      bad |= c < 0 || c > a.max_context_len;
    }
    if (bad && blockIdx.x == 0) report(a.err, kErrContextLen);
    int upto = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += v;
    }
    if (lane == 31) sh[warp] = upto;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w < warp) upto += sh[w];
      total += sh[w];
    }
    chunks = total * Hkv;            // below 2^31
    ctas = min((int)gridDim.x, chunks);  // so that no span among them is empty
    if ((int)blockIdx.x < ctas) {
      span_begin = (int)((long long)chunks * blockIdx.x / ctas);
      span_end = (int)((long long)chunks * (blockIdx.x + 1) / ctas);
    }
    int before = upto - sum;
    if (span_begin < span_end && before * Hkv <= span_begin && span_begin < upto * Hkv) {
      int s = lo;
      for (;; ++s) {
        const int n = (context(s) + CT - 1) / CT;
        if (span_begin < (before + n) * Hkv) break;
        before += n;
      }
      sh[4] = s;
      sh[5] = before * Hkv;
    }
    __syncthreads();
    seq = sh[4];
    seq_base = sh[5];
  }
  // sequences without tokens: zero rows
  for (int s = blockIdx.x; s < S; s += gridDim.x)
    if (context(s) == 0) {
      uint4* o = reinterpret_cast<uint4*>(a.out + (size_t)s * a.num_q_heads * D);
      for (int i = threadIdx.x; i < a.num_q_heads * D / 8; i += NW * 32) o[i] = make_uint4(0, 0, 0, 0);
    }
  if (span_begin >= span_end) return;
  const int n_mine = max(0, (span_end - span_begin - warp + NW - 1) / NW);  // chunks of this warp

  // ---- copies: lane (sub, piece, pool) moves one piece of one group of
  // copy_tokens (8, 16 or 32) tokens, which never crosses a block
  const int R = copy_tokens, bs = a.block_size;
  const bool whole = R == bs;  // codes and scales of the group are one run
  const int c_sub = lane >> 2, c_piece = (lane >> 1) & 1;
  const bool c_lane = c_sub * R < CT && (c_piece == 0 || !whole);
  const uint32_t c_bytes = whole ? R * L::kTokenBytes : c_piece ? R * (D / 16) : R * (D / 2);
  const uint32_t c_dst = ((lane & 1) ? L::kPoolBytes : 0) + c_sub * R * L::kTokenBytes + (c_piece ? R * (D / 2) : 0);
  const long long run_bytes = fp4_head_bytes(bs, D);
  const unsigned char* c_base = ((lane & 1) ? v_pool : k_pool) + (c_piece ? bs * (D / 2) : 0);
  const int c_unit = c_piece ? D / 16 : D / 2;
  // The copies' cursor: the next chunk to fetch, its item and chunk number there;
  // this lane's group in it: table index and offset in the block.
  int f_left = n_mine, f_seq = seq, f_head = 0, f_chunk = 0, f_ctx = context(seq), f_idx = 0, f_off = 0;
  const int step_idx = NW * CT / bs, step_off = NW * CT - step_idx * bs;
  {
    int rel = span_begin + warp - seq_base;
    int n = (f_ctx + CT - 1) / CT;
    while (f_left > 0 && rel >= n * Hkv) {
      rel -= n * Hkv;
      f_ctx = context(++f_seq);
      n = (f_ctx + CT - 1) / CT;
    }
    f_head = n ? rel / n : 0;
    f_chunk = rel - f_head * n;
    f_idx = (f_chunk * CT + c_sub * R) / bs;
    f_off = f_chunk * CT + c_sub * R - f_idx * bs;
  }
  struct Group {
    int blk, off, head;  // table entry, first token in the block (negative: nothing to copy), kv head
  };
  auto fetch = [&]() {
    Group e{0, -1, f_head};
    if (f_left > 0) {
      if (c_lane && f_chunk * CT + c_sub * R < f_ctx) {
        e.off = f_off;
        e.blk = __ldg(a.block_tables + (size_t)f_seq * a.max_blocks_per_seq + f_idx);
      }
      if (--f_left > 0) {
        int n = (f_ctx + CT - 1) / CT;
        f_chunk += NW;
        f_idx += step_idx;
        f_off += step_off;
        if (f_off >= bs) { f_off -= bs; ++f_idx; }
        if (f_chunk >= n) {
          do {
            f_chunk -= n;
            if (++f_head == Hkv) {
              f_head = 0;
              do {
                f_ctx = context(++f_seq);
              } while (f_ctx == 0);
              n = (f_ctx + CT - 1) / CT;
            }
          } while (f_chunk >= n);
          f_idx = (f_chunk * CT + c_sub * R) / bs;
          f_off = f_chunk * CT + c_sub * R - f_idx * bs;
        }
      }
    }
    return e;
  };
  auto issue = [&](int k, Group e) {
    const uint32_t bar = bar0 + (k % NST) * 8, dst = stage0 + (k % NST) * L::kStageBytes + c_dst;
    bool copy = e.off >= 0;
    if (copy && (unsigned)e.blk >= (unsigned)a.num_blocks) {  // rows outside the pool read as zeros
      report(a.err, kErrBlockId);
      for (uint32_t i = 0; i < c_bytes; i += 16)
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + i), "r"(0) : "memory");
      copy = false;
    }
    const uint32_t total = __reduce_add_sync(0xffffffffu, copy ? c_bytes : 0u);
    if (lane == 0) mbar_arrive_expect_tx(bar, total);
    __syncwarp();
    if (copy) bulk_load(dst, c_base + ((long long)e.blk * Hkv + e.head) * run_bytes + e.off * c_unit, c_bytes, bar);
  };
  {
    Group e[NST];
#pragma unroll
    for (int k = 0; k < NST; ++k) e[k] = fetch();
#pragma unroll
    for (int k = 0; k < NST; ++k)
      if (k < n_mine) issue(k, e[k]);
  }
  Group next = fetch();

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

  // ---- the items of the span, each from its chunk `first` to its end or the span's
  int failed_at = n_mine;     // the chunk whose wait ran out
  int k = 0, at = span_begin;  // this warp's chunk count; the segment's first chunk
  int ctx = context(seq), kvh = (span_begin - seq_base) / ((ctx + CT - 1) / CT);
  int first = span_begin - seq_base - kvh * ((ctx + CT - 1) / CT);
  for (;;) {
    const int item_chunks = (ctx + CT - 1) / CT, len = min(item_chunks - first, span_end - at);
    const size_t head0 = (size_t)seq * a.num_q_heads + kvh * G;

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

    for (; span_begin + warp + k * NW < at + len; ++k) {
      if (failed_at < n_mine) continue;
      if (!mbar_wait(bar0 + (k % NST) * 8, (k / NST) & 1, a.err)) {
        failed_at = k;
        continue;
      }
      const uint32_t st = stage0 + (k % NST) * L::kStageBytes;
      const int n_valid = ctx - (first + span_begin + warp + k * NW - at) * CT;  // of this chunk's 32 tokens
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
        issue(k + NST, next);
        next = fetch();
      }
    }

    // ---- merge the warps: 2 and 3 into 0 and 1, then 1 into 0
    auto dump = [&](int slot) {
      const uint32_t to = states + slot * L::kStateBytes;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < MT; ++i) sts_f4(to + (n * (MT + 1) + i) * 512, o[i][n][0], o[i][n][1], o[i][n][2], o[i][n][3]);
        sts_f4(to + (n * (MT + 1) + MT) * 512, m[n][0], m[n][1], l[n][0], l[n][1]);
      }
    };
    auto absorb = [&](int slot) {
      const uint32_t from = states + slot * L::kStateBytes;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float4 s4 = lds_f4(from + (n * (MT + 1) + MT) * 512);
        const float m0 = fmaxf(m[n][0], s4.x), m1 = fmaxf(m[n][1], s4.y);
        const float a0 = ex2(m[n][0] - m0), a1 = ex2(m[n][1] - m1), b0 = ex2(s4.x - m0), b1 = ex2(s4.y - m1);
        m[n][0] = m0;
        m[n][1] = m1;
        l[n][0] = l[n][0] * a0 + s4.z * b0;
        l[n][1] = l[n][1] * a1 + s4.w * b1;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const float4 v = lds_f4(from + (n * (MT + 1) + i) * 512);
          o[i][n][0] = o[i][n][0] * a0 + v.x * b0;
          o[i][n][1] = o[i][n][1] * a1 + v.y * b1;
          o[i][n][2] = o[i][n][2] * a0 + v.z * b0;
          o[i][n][3] = o[i][n][3] * a1 + v.w * b1;
        }
      }
    };
    if (warp >= 2) dump(warp - 2);
    const bool failed = __syncthreads_or(failed_at < n_mine);
    if (warp < 2) absorb(warp);
    if (warp == 1) dump(2);
    __syncthreads();
    if (warp == 0) {
      absorb(2);
      // an item within the span is finished; else a partial result: slot 2 i + 1 of
      // CTA i for an item that starts here, 2 i for one that started before
      const bool direct = first == 0 && len == item_chunks;
      const int slot = 2 * blockIdx.x + (first == 0);
      const float v_scale = __ldg(a.v_scale + kvh);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int h = n * 8 + 2 * t + j;
          float den = l[n][j];
#pragma unroll
          for (int d = 4; d <= 16; d <<= 1) den += __shfl_xor_sync(0xffffffffu, den, d);
          if (failed) den = __int_as_float(0x7fc00000);
          if (h >= G) continue;
          if (direct) {
            const float f = v_scale / den;
            uint32_t w[MT];
#pragma unroll
            for (int i = 0; i < MT; ++i)
              w[i] = (uint32_t)Elem<T>::from_f(o[i][n][j] * f) | ((uint32_t)Elem<T>::from_f(o[i][n][j + 2] * f) << 16);
            uint4* to = reinterpret_cast<uint4*>(a.out + (head0 + h) * D + g * (D / 8));
#pragma unroll
            for (int i = 0; i < VW; ++i) to[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          } else {
            const size_t row = (size_t)slot * G + h;
            float4* to = reinterpret_cast<float4*>(a.ws_acc + row * D + g * (D / 8));
#pragma unroll
            for (int i = 0; i < MT; i += 2)
              to[i / 2] = make_float4(o[i][n][j] * v_scale, o[i][n][j + 2] * v_scale, o[i + 1][n][j] * v_scale,
                                      o[i + 1][n][j + 2] * v_scale);
            if (g == 0) *reinterpret_cast<float2*>(a.ws_ml + 2 * row) = make_float2(m[n][j], den);
          }
        }
      // the CTAs whose spans this item lies in: the merge reads their partials
      if (first == 0 && lane == 0) {
        // chunk e lies in the span of CTA ceil((e + 1) ctas / chunks) - 1
        const int last = (int)(((long long)(at + item_chunks) * ctas - 1) / chunks);
        item_parts[(size_t)seq * Hkv + kvh] = make_int2(blockIdx.x, last);
      }
    }
    at += len;
    if (at >= span_end) break;
    first = 0;
    if (++kvh == Hkv) {
      kvh = 0;
      do {
        ctx = context(++seq);
      } while (ctx == 0);
    }
  }
  // after a failed wait let every copy in flight land before the CTA exits
  for (int i = failed_at; i < min(n_mine, failed_at + NST); ++i)
    mbar_wait(bar0 + (i % NST) * 8, (i / NST) & 1, a.err);
}

// Merge of the items that span borders cut: a warp per (sequence, query head).
template <typename T, int D>
__global__ void __launch_bounds__(128) decode_fp4_merge_kernel(const DecodeArgs a, const int2* item_parts) {
  constexpr int VEC = D / 32;
  pdl_wait();  // every partial is written
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, G = a.group;
  const int row = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= a.num_seqs * a.num_q_heads) return;
  const int s = row / a.num_q_heads, h = row % a.num_q_heads;
  if (__ldg(a.context_lens + s) <= 0 || a.max_context_len == 0) return;
  const int2 parts = item_parts[(size_t)s * a.num_kv_heads + h / G];
  if (parts.x == parts.y) return;  // written directly
  float M = -INFINITY, den = 0.f, num[VEC] = {};
  for (int p = parts.x; p <= parts.y; ++p) {
    const size_t r = (size_t)(2 * p + (p == parts.x)) * G + h % G;
    const float2 ml = *reinterpret_cast<const float2*>(a.ws_ml + 2 * r);
    float v[VEC];
    if constexpr (VEC == 4) {
      const float4 x = *reinterpret_cast<const float4*>(a.ws_acc + r * D + lane * 4);
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else {
      const float2 x = *reinterpret_cast<const float2*>(a.ws_acc + r * D + lane * 2);
      v[0] = x.x; v[1] = x.y;
    }
    const float Mn = fmaxf(M, ml.x), al = exp2f(M - Mn), be = exp2f(ml.x - Mn);
    M = Mn;
    den = den * al + ml.y * be;
#pragma unroll
    for (int i = 0; i < VEC; ++i) num[i] = num[i] * al + v[i] * be;
  }
  uint32_t w[VEC / 2];
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i)
    w[i] = (uint32_t)Elem<T>::from_f(num[2 * i] / den) | ((uint32_t)Elem<T>::from_f(num[2 * i + 1] / den) << 16);
  uint32_t* to = reinterpret_cast<uint32_t*>(a.out + (size_t)row * D) + lane * (VEC / 2);
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) to[i] = w[i];
}

namespace {

template <typename T, int D, int NT>
cudaError_t launch_fp4(const DecodeArgs& a, const void* k, const void* v, int2* parts, cudaStream_t stream,
                       int* launches) {
  auto* kern = decode_fp4_kernel<T, D, NT>;
  constexpr int smem = Fp4Smem<D, NT>::kTotal;
  static std::atomic<uint64_t> configured{0};  // a bit per device; setting the attribute twice is harmless
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(configured.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) configured.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  int copy = kFp4Chunk;  // a copy's tokens lie in one block
  while (a.block_size % copy) copy /= 2;
  e = launch_pdl(kern, dim3(a.grid_parts), dim3(kFp4Warps * 32), smem, stream, a,
                 static_cast<const unsigned char*>(k), static_cast<const unsigned char*>(v), copy, parts);
  if (e == cudaSuccess) ++*launches;
  if (e != cudaSuccess || a.grid_parts == 1) return e;  // one span cuts no item
  const long long rows = (long long)a.num_seqs * a.num_q_heads;
  e = launch_pdl(decode_fp4_merge_kernel<T, D>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, stream, a,
                 static_cast<const int2*>(parts));
  if (e == cudaSuccess) ++*launches;
  return e;
}

template <typename T, int D>
cudaError_t launch_fp4_group(const DecodeArgs& a, const void* k, const void* v, int2* parts, cudaStream_t st, int* n) {
  return a.group <= 8 ? launch_fp4<T, D, 1>(a, k, v, parts, st, n) : launch_fp4<T, D, 2>(a, k, v, parts, st, n);
}

}  // namespace

int fp4_decode_ctas(int num_seqs, int num_kv_heads, int group, int max_context_len, int partition_tokens) {
  if (max_context_len > 1 << 30) return 0;
  const long long per_item = (max_context_len + kFp4Chunk - 1) / kFp4Chunk;
  const long long chunks = (per_item > 0 ? per_item : 1) * num_seqs * num_kv_heads;
  if (chunks > 0x7fffffffLL) return 0;
  // one wave of a B200's 148 SMs; no CTA with less than its four warps' chunks or
  // the caller's partition
  const long long wave = 148 * (group <= 8 ? Fp4Smem<128, 1>::kCtas : Fp4Smem<128, 2>::kCtas);
  const long long least = partition_tokens > 0 ? (partition_tokens + kFp4Chunk - 1) / kFp4Chunk : kFp4Warps;
  const long long n = (chunks + least - 1) / least;
  return (int)(n < wave ? n : wave);
}

cudaError_t launch_decode_fp4(const DecodeArgs& a, int dtype, int head_dim, const void* k_pool, const void* v_pool,
                              int2* item_parts, cudaStream_t stream, int* launches) {
  if (dtype == 0)
    return head_dim == 128 ? launch_fp4_group<__half, 128>(a, k_pool, v_pool, item_parts, stream, launches)
                           : launch_fp4_group<__half, 64>(a, k_pool, v_pool, item_parts, stream, launches);
  return head_dim == 128 ? launch_fp4_group<__nv_bfloat16, 128>(a, k_pool, v_pool, item_parts, stream, launches)
                         : launch_fp4_group<__nv_bfloat16, 64>(a, k_pool, v_pool, item_parts, stream, launches);
}

}  // namespace pa
