// pa_decode_fp4.cu -- single-token decode attention over an E2M1 cache.
//
// Work split.  An item is a (sequence, kv head) pair; its context is cut into chunks of
// 64 tokens.  The chunks of all items, in order, are split evenly into one span
// per worker: long and short contexts balance, and only an item cut by a
// span's border needs merging.  Every CTA finds its spans itself, by a scan
// over the context lengths.  A worker is a warp, or (few long items) the four
// warps of a CTA, which take a span's chunks in turn and merge through shared
// memory at an item's end.  A warp runs its own ring of bulk copies, across
// items: a (block, head) run is contiguous, so a chunk of K is one copy per
// block (two where a block holds more than the copy: codes, then block scales),
// one lane each, and table entries are read one chunk ahead.
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
#ifndef FP4_CT
#define FP4_CT 64
#define FP4_NST 2
#endif
constexpr int kFp4Chunk = FP4_CT;  // tokens a stage holds
#ifndef FP4_CTAS
#define FP4_CTAS 3
#endif
#ifndef FP4_TEAM
#define FP4_TEAM 1000
#endif
constexpr int kFp4Ctas = FP4_CTAS;    // per SM, by registers and (D = 128) shared memory

template <int D, int GT>
struct Fp4Smem {
  static constexpr int kStages = FP4_NST;
  static constexpr int kTokenBytes = D * 9 / 16;
  static constexpr int kPoolBytes = kFp4Chunk * kTokenBytes;  // K or V of one stage
  static constexpr int kStageBytes = 2 * kPoolBytes;
  static constexpr int kBars = kFp4Warps * kStages * kStageBytes;
  static constexpr int kScan = kBars + kFp4Warps * kStages * 8;
  static constexpr int kTotal = kScan + 32;
  static constexpr int kStateBytes = ((GT == 4 ? D / 32 : D / 16) + 1) * (GT == 16 ? 2 : 1) * 32 * 16;  // one warp's, to merge
  static constexpr int kMerge = kScan + 32;
  static constexpr int kTotalMerge = kMerge + 3 * kStateBytes;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The first product of a sum: c = a b.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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
// GT: the group's query heads, at most: 4, 8 or 16.  R: tokens of one copy.
template <typename T, int D, int GT, int R>
__global__ void __launch_bounds__(kFp4Warps * 32, kFp4Ctas)
decode_fp4_kernel(const DecodeArgs a, const unsigned char* __restrict__ k_pool,
                  const unsigned char* __restrict__ v_pool, const int num_workers, const int team, int2* item_parts) {
  constexpr int NT = GT == 16 ? 2 : 1;  // column tiles of 8
  constexpr bool kPairs = GT == 4;      // V registers hold pairs of dims (see above), else pairs of tokens
  using L = Fp4Smem<D, GT>;
  constexpr bool kLo = std::is_same<T, __half>::value;  // p as hi + lo
  constexpr int NW = kFp4Warps, NST = L::kStages, CT = kFp4Chunk, TILES = 2;
  constexpr int KW = D / 32;   // words of K codes a thread takes per row
  constexpr int VW = D / 64;   // words of V codes a thread takes per row
  constexpr int MT = kPairs ? VW * 2 : VW * 4;  // 16-row tiles of output dims, or of pairs of dims
  extern __shared__ __align__(128) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  unsigned char* stages = smem + warp * NST * L::kStageBytes;
  const uint32_t stage0 = smem_addr(stages);
  const uint32_t bar0 = smem_addr(smem) + L::kBars + warp * NST * 8;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < NST; ++i) mbar_init(bar0 + i * 8, 1);
    mbar_init_fence();
  }
  __syncwarp();
  pdl_wait();  // the append before this decode must have landed
  pdl_launch_dependents();

  // ---- this worker's span of chunks, and the sequence it starts in
  const int S = a.num_seqs, Hkv = a.num_kv_heads, G = a.group;
  const bool alone = team == 1;
  const int rank = alone ? 0 : warp, worker = alone ? blockIdx.x + gridDim.x * warp : blockIdx.x;
  auto context = [&](int s) { return max(0, min(__ldg(a.context_lens + s), a.max_context_len)); };
  int span_begin = 0, span_end = 0, chunks, workers, seq = 0, seq_base = 0;  // seq_base: number of seq's first chunk
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
    chunks = total * Hkv;                // below 2^31
    workers = min(num_workers, chunks);  // so that no span among them is empty
    // every thread looks for the spans that start in its sequences
    __syncthreads();
    for (int w = 0; w < NW / team; ++w) {
      const int id = alone ? blockIdx.x + gridDim.x * w : blockIdx.x;
      if (id >= workers) break;
      const int begin = (int)((long long)chunks * id / workers);
      int before = upto - sum;
      if (before * Hkv <= begin && begin < upto * Hkv) {
        int s = lo;
        for (;; ++s) {
          const int n = (context(s) + CT - 1) / CT;
          if (begin < (before + n) * Hkv) break;
          before += n;
        }
        sh[2 * w] = s;
        sh[2 * w + 1] = before * Hkv;
      }
    }
    __syncthreads();
    if (worker < workers) {
      span_begin = (int)((long long)chunks * worker / workers);
      span_end = (int)((long long)chunks * (worker + 1) / workers);
      seq = sh[alone ? 2 * warp : 0];
      seq_base = sh[alone ? 2 * warp + 1 : 1];
    }
  }
  // sequences without tokens: zero rows
  for (int s = blockIdx.x; s < S; s += gridDim.x)
    if (context(s) == 0) {
      uint4* o = reinterpret_cast<uint4*>(a.out + (size_t)s * a.num_q_heads * D);
      for (int i = threadIdx.x; i < a.num_q_heads * D / 8; i += NW * 32) o[i] = make_uint4(0, 0, 0, 0);
    }
  if (span_begin >= span_end) return;  // a whole team returns
  const int n_mine = max(0, (span_end - span_begin - rank + team - 1) / team);  // chunks of this warp

  // ---- copies: lane (sub, piece, pool) moves one piece of one group of R tokens, which never crosses a block
  const int bs = a.block_size;
  const bool whole = R == bs;  // codes and scales of the group are one run
  const int c_sub = lane >> 2, c_piece = (lane >> 1) & 1;
  const bool c_lane = c_sub * R < CT && (c_piece == 0 || !whole);
  const uint32_t c_bytes = whole ? R * L::kTokenBytes : c_piece ? R * (D / 16) : R * (D / 2);
  const uint32_t c_dst = ((lane & 1) ? L::kPoolBytes : 0) + c_sub * R * L::kTokenBytes + (c_piece ? R * (D / 2) : 0);
  const long long run_bytes = fp4_head_bytes(bs, D);
  const unsigned char* c_base = ((lane & 1) ? v_pool : k_pool) + (c_piece ? bs * (D / 2) : 0);
  const int c_unit = c_piece ? D / 16 : D / 2;
  // The copies' cursor: the next chunk to fetch, its item and chunk number there;
  // this lane's group in it: first token, its table index and offset in the block.
  int f_left = n_mine, f_seq = seq, f_head = 0, f_chunk = 0, f_ctx = context(seq), f_idx = 0, f_off = 0;
  const int step_idx = team * CT / bs, step_off = team * CT - step_idx * bs;
  {
    int rel = span_begin + rank - seq_base;
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
      f_chunk += team;
      f_idx += step_idx;
      f_off += step_off;
      if (f_off >= bs) { f_off -= bs; ++f_idx; }
      if (--f_left > 0 && f_chunk * CT >= f_ctx) {  // on to a later item, which exists
        int n = (f_ctx + CT - 1) / CT;
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

  // ---- where a tile of 16 tokens lies in the stage: its rows 8 .. 15 are in a
  // group of their own when R is 8, two tiles share a group when R is 32
  constexpr int kCodeTile = R == 32 ? 16 * (D / 2) : 16 * L::kTokenBytes;
  constexpr int kScaleTile = R == 32 ? 16 * (D / 16) : 16 * L::kTokenBytes;
  constexpr int kCodeHalf = R == 8 ? 8 * L::kTokenBytes : 8 * (D / 2);
  constexpr int kScaleHalf = R == 8 ? 8 * L::kTokenBytes : 8 * (D / 16);
  constexpr int kScaleBase = R * (D / 2);
  const int k_row = (g >> 1) + 4 * (g & 1);  // token of the tile's row g (row g + 8: 8 tokens on)
  const int k_code = k_row * (D / 2) + t * (D / 8);
  const int k_sc = kScaleBase + k_row * (D / 16) + t * (D / 64);
  // pairs: where a transposed probability of token t (or t + 4) goes: the even dim's
  // place in columns 0 .. 3, the odd dim's in columns 4 .. 7
  [[maybe_unused]] const uint32_t pair_lo = g < 4 ? 0x4410 : 0x1044, pair_hi = g < 4 ? 0x4432 : 0x3244;
  const int v_code = L::kPoolBytes + t * (D / 2) + g * (D / 16);
  const int v_sc = L::kPoolBytes + kScaleBase + t * (D / 16) + g * (D / 64) / 2;

  // ---- the items of the span, each from its chunk `first` to its end or the span's
  int failed_at = n_mine;      // the chunk whose wait ran out
  int k = 0, at = span_begin;  // this warp's chunk count; the item's first chunk in the span
  int ctx = context(seq), kvh = (span_begin - seq_base) / ((ctx + CT - 1) / CT);
  int first = span_begin - seq_base - kvh * ((ctx + CT - 1) / CT);
  for (;;) {
    const int item_chunks = (ctx + CT - 1) / CT, len = min(item_chunks - first, span_end - at);
    const size_t head0 = (size_t)seq * a.num_q_heads + kvh * G;

    // queries as column fragments: thread (g, t) holds dims [t D/4, (t + 1) D/4) of heads g, g + 8
    const float cscale = a.scale_log2 * __ldg(a.k_scale + kvh);
    uint32_t bq[NT][KW * 4];
    float xs[NT][2];  // logit scale of this thread's columns 2t, 2t + 1
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int h = kPairs ? g & 3 : n * 8 + g;  // pairs: columns 4 .. 7 repeat the heads
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
        const float up = __uint_as_float((uint32_t)(268 - e) << 23);  // 2^(141 - e)
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

    for (; span_begin + rank + k * team < at + len; ++k) {
      if (failed_at < n_mine) continue;
      if (!mbar_wait(bar0 + (k % NST) * 8, (k / NST) & 1, a.err)) {
        failed_at = k;
        continue;
      }
      unsigned char* stage = stages + (k % NST) * L::kStageBytes;
      const int n_valid = ctx - (first + span_begin + rank + k * team - at) * CT;  // of this chunk's tokens
      if (n_valid < CT) {
        // what lies behind the last token may be anything: codes are finite, V's scales need not be
        for (int tok = n_valid + lane; tok < CT; tok += 32) {
          unsigned char* sc = stage + L::kPoolBytes + tok / R * R * L::kTokenBytes + kScaleBase + tok % R * (D / 16);
          if constexpr (D == 128) *reinterpret_cast<uint2*>(sc) = make_uint2(0, 0);
          else *reinterpret_cast<uint32_t*>(sc) = 0;
        }
        __syncwarp();
      }
#pragma unroll 1
      for (int half = 0; half < min(n_valid, CT); half += 32) {
        const unsigned char* st = stage + half * L::kTokenBytes;

        // ---- logits
        float x[TILES][NT][4];
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
          uint32_t ca[KW], cb[KW], sa, sb;
          const unsigned char* ka = st + k_code + i * kCodeTile;
          const unsigned char* ks = st + k_sc + i * kScaleTile;
          if constexpr (D == 128) {
            const uint4 u = *reinterpret_cast<const uint4*>(ka), w = *reinterpret_cast<const uint4*>(ka + kCodeHalf);
            ca[0] = u.x; ca[1] = u.y; ca[2] = u.z; ca[3] = u.w;
            cb[0] = w.x; cb[1] = w.y; cb[2] = w.z; cb[3] = w.w;
            sa = e4m3x2_to_h2(*reinterpret_cast<const uint16_t*>(ks));
            sb = e4m3x2_to_h2(*reinterpret_cast<const uint16_t*>(ks + kScaleHalf));
          } else {
            const uint2 u = *reinterpret_cast<const uint2*>(ka), w = *reinterpret_cast<const uint2*>(ka + kCodeHalf);
            ca[0] = u.x; ca[1] = u.y;
            cb[0] = w.x; cb[1] = w.y;
            sa = e4m3x2_to_h2(ks[0]);
            sb = e4m3x2_to_h2(ks[kScaleHalf]);
          }
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
              if (w == 0) mma_f16_first(x[i][n], fa[0], fb[0], fa[1], fb[1], bq[n][0], bq[n][1]);
              else mma_f16(x[i][n], fa[0], fb[0], fa[1], fb[1], bq[n][4 * w], bq[n][4 * w + 1]);
              mma_f16(x[i][n], fa[2], fb[2], fa[3], fb[3], bq[n][4 * w + 2], bq[n][4 * w + 3]);
            }
          }
        }

        // ---- softmax
        bool grow = false;
        float top[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < TILES; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[i][n][j] *= xs[n][j & 1];
        if (half + 32 > n_valid) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < TILES; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (half + i * 16 + k_row + (j >> 1) * 8 >= n_valid) x[i][n][j] = -INFINITY;
          __syncwarp();
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          top[n][0] = fmaxf(fmaxf(x[0][n][0], x[0][n][2]), fmaxf(x[1][n][0], x[1][n][2]));
          top[n][1] = fmaxf(fmaxf(x[0][n][1], x[0][n][3]), fmaxf(x[1][n][1], x[1][n][3]));
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
          const unsigned char* va = st + v_code + i * kCodeTile;
          const unsigned char* vs = st + v_sc + i * kScaleTile;
          uint32_t c[4][VW], sc[2];
#pragma unroll
          for (int r = 0; r < 4; ++r) {  // tokens t, t + 4, t + 8, t + 12 of the tile
            const unsigned char* from = va + (r & 1) * 4 * (D / 2) + (r >> 1) * kCodeHalf;
            if constexpr (D == 128) {
              const uint2 u = *reinterpret_cast<const uint2*>(from);
              c[r][0] = u.x; c[r][1] = u.y;
            } else {
              c[r][0] = *reinterpret_cast<const uint32_t*>(from);
            }
          }
#pragma unroll
          for (int r = 0; r < 2; ++r)
            sc[r] = e4m3x2_to_h2((uint16_t)(vs[r * kScaleHalf] | (vs[4 * (D / 16) + r * kScaleHalf] << 8)));
          if constexpr (kPairs) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {  // 8 tokens a product: t and t + 4, then t + 8 and t + 12
              const uint32_t s0 = __byte_perm(sc[r], 0, 0x1010), s1 = __byte_perm(sc[r], 0, 0x3232);
              const uint32_t b0 = __byte_perm(hi[0][r], 0, pair_lo), b1 = __byte_perm(hi[0][r], 0, pair_hi);
              uint32_t d0 = 0, d1 = 0;
              if constexpr (kLo) {
                d0 = __byte_perm(lo[0][r], 0, pair_lo);
                d1 = __byte_perm(lo[0][r], 0, pair_hi);
              }
#pragma unroll
              for (int w = 0; w < VW; ++w) {
                uint32_t f0[4], f1[4];
                e2m1x8_to_h2(c[2 * r][w], f0);
                e2m1x8_to_h2(c[2 * r + 1][w], f1);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  f0[j] = hmul2(f0[j], s0);
                  f1[j] = hmul2(f1[j], s1);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  mma_f16(o[2 * w + j][0], f0[2 * j], f0[2 * j + 1], f1[2 * j], f1[2 * j + 1], b0, b1);
                  if constexpr (kLo)
                    mma_f16(o[2 * w + j][0], f0[2 * j], f0[2 * j + 1], f1[2 * j], f1[2 * j + 1], d0, d1);
                }
              }
            }
          } else {
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

    // ---- a team merges its warps: 2 and 3 into 0 and 1, then 1 into 0
    bool failed = failed_at < n_mine;
    if (!alone) {
      float4* states = reinterpret_cast<float4*>(smem + L::kMerge) + lane;
      constexpr int kSlot = L::kStateBytes / 16;
      auto dump = [&](int slot) {
        float4* to = states + slot * kSlot;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int i = 0; i < MT; ++i)
            to[(n * (MT + 1) + i) * 32] = make_float4(o[i][n][0], o[i][n][1], o[i][n][2], o[i][n][3]);
          to[(n * (MT + 1) + MT) * 32] = make_float4(m[n][0], m[n][1], l[n][0], l[n][1]);
        }
      };
      auto absorb = [&](int slot) {
        const float4* from = states + slot * kSlot;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float4 s4 = from[(n * (MT + 1) + MT) * 32];
          const float m0 = fmaxf(m[n][0], s4.x), m1 = fmaxf(m[n][1], s4.y);
          const float a0 = ex2(m[n][0] - m0), a1 = ex2(m[n][1] - m1), b0 = ex2(s4.x - m0), b1 = ex2(s4.y - m1);
          m[n][0] = m0;
          m[n][1] = m1;
          l[n][0] = l[n][0] * a0 + s4.z * b0;
          l[n][1] = l[n][1] * a1 + s4.w * b1;
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            const float4 v = from[(n * (MT + 1) + i) * 32];
            o[i][n][0] = o[i][n][0] * a0 + v.x * b0;
            o[i][n][1] = o[i][n][1] * a1 + v.y * b1;
            o[i][n][2] = o[i][n][2] * a0 + v.z * b0;
            o[i][n][3] = o[i][n][3] * a1 + v.w * b1;
          }
        }
      };
      if (warp >= 2) dump(warp - 2);
      failed = __syncthreads_or(failed);
      if (warp < 2) absorb(warp);
      if (warp == 1) dump(2);
      __syncthreads();
      if (warp == 0) absorb(2);
    }
    if (rank == 0) {
      // an item within the span is finished; else a partial result: slot 2 i + 1 of
      // worker i for an item that starts here, 2 i for one that started before
      const bool direct = first == 0 && len == item_chunks;
      const int slot = 2 * worker + (first == 0);
      const float v_scale = __ldg(a.v_scale + kvh);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int h = kPairs ? 2 * (t & 1) + j : n * 8 + 2 * t + j;
          float den = l[n][j];
#pragma unroll
          for (int d = 4; d <= 16; d <<= 1) den += __shfl_xor_sync(0xffffffffu, den, d);
          if (failed) den = __int_as_float(0x7fc00000);
          float f = v_scale;
          if (direct) f /= den;
          // this thread's D / 8 dims of head h, two at a time
          float v[D / 8];
          if constexpr (kPairs) {
            // threads t < 2 hold the even dims, t >= 2 the odd ones: each takes half of both
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              const float send = t < 2 ? o[i][0][j + 2] : o[i][0][j], keep = t < 2 ? o[i][0][j] : o[i][0][j + 2];
              const float got = __shfl_xor_sync(0xffffffffu, send, 2);
              v[2 * i] = (t < 2 ? keep : got) * f;  // pair 2i + (t >= 2) of the thread's D / 16
              v[2 * i + 1] = (t < 2 ? got : keep) * f;
            }
          } else {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              v[2 * i] = o[i][n][j] * f;
              v[2 * i + 1] = o[i][n][j + 2] * f;
            }
          }
          if (h >= G) continue;
          const size_t row = direct ? head0 + h : (size_t)slot * G + h;
          // pairs: v[2i], v[2i + 1] are dims 4i + 2 (t >> 1) and the next; else dims 2i and 2i + 1
          const size_t dim0 = row * D + g * (D / 8) + (kPairs ? 2 * (t >> 1) : 0);
          constexpr int kStep = kPairs ? 4 : 2;
          if (direct) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
              *reinterpret_cast<uint32_t*>(a.out + dim0 + i * kStep) =
                  (uint32_t)Elem<T>::from_f(v[2 * i]) | ((uint32_t)Elem<T>::from_f(v[2 * i + 1]) << 16);
          } else {
#pragma unroll
            for (int i = 0; i < MT; ++i)
              *reinterpret_cast<float2*>(a.ws_acc + dim0 + i * kStep) = make_float2(v[2 * i], v[2 * i + 1]);
            if (g == 0 && (!kPairs || t < 2)) *reinterpret_cast<float2*>(a.ws_ml + 2 * row) = make_float2(m[n][j], den);
          }
        }
      // the workers whose spans this item lies in: the merge reads their partials
      if (first == 0 && lane == 0) {
        // chunk e lies in the span of worker ceil((e + 1) workers / chunks) - 1
        const int last = (int)(((long long)(at + item_chunks) * workers - 1) / chunks);
        item_parts[(size_t)seq * Hkv + kvh] = make_int2(worker, last);
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

// Merge of the items that span borders cut: a CTA per (sequence, query head), warp w
// the partials w, w + 4, ..., several loads in flight.
template <typename T, int D>
__global__ void __launch_bounds__(128) decode_fp4_merge_kernel(const DecodeArgs a, const int2* item_parts) {
  constexpr int VEC = D / 32, UN = 4;
  __shared__ float sm[4][2 + D];
  pdl_wait();  // every partial is written
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = a.group;
  const int s = blockIdx.x / a.num_q_heads, h = blockIdx.x % a.num_q_heads;
  if (__ldg(a.context_lens + s) <= 0 || a.max_context_len == 0) return;
  const int2 parts = item_parts[(size_t)s * a.num_kv_heads + h / G];
  if (parts.x == parts.y) return;  // written directly
  float M = -INFINITY, den = 0.f, num[VEC] = {};
  for (int p0 = parts.x + warp; p0 <= parts.y; p0 += 4 * UN) {
    float2 ml[UN];
    float v[UN][VEC], top = M;
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int p = min(p0 + 4 * u, parts.y);
      const size_t r = (size_t)(2 * p + (p == parts.x)) * G + h % G;
      ml[u] = *reinterpret_cast<const float2*>(a.ws_ml + 2 * r);
      if constexpr (VEC == 4) {
        const float4 x = *reinterpret_cast<const float4*>(a.ws_acc + r * D + lane * 4);
        v[u][0] = x.x; v[u][1] = x.y; v[u][2] = x.z; v[u][3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(a.ws_acc + r * D + lane * 2);
        v[u][0] = x.x; v[u][1] = x.y;
      }
      top = fmaxf(top, ml[u].x);
    }
    const float al = exp2f(M - top);
    M = top;
    den *= al;
#pragma unroll
    for (int i = 0; i < VEC; ++i) num[i] *= al;
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const float wt = p0 + 4 * u <= parts.y ? exp2f(ml[u].x - M) : 0.f;
      den += ml[u].y * wt;
#pragma unroll
      for (int i = 0; i < VEC; ++i) num[i] += v[u][i] * wt;
    }
  }
  if (lane == 0) {
    sm[warp][0] = M;
    sm[warp][1] = den;
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) sm[warp][2 + lane * VEC + i] = num[i];
  __syncthreads();
  if (threadIdx.x < D) {
    const float top = fmaxf(fmaxf(sm[0][0], sm[1][0]), fmaxf(sm[2][0], sm[3][0]));
    float d = 0.f, n = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float wt = exp2f(sm[w][0] - top);  // 0 for a warp without partials
      d += sm[w][1] * wt;
      n += sm[w][2 + threadIdx.x] * wt;
    }
    a.out[(size_t)blockIdx.x * D + threadIdx.x] = Elem<T>::from_f(n / d);
  }
}

namespace {

template <typename T, int D, int GT, int R>
cudaError_t launch_fp4(const DecodeArgs& a, const void* k, const void* v, const Fp4Split& w, int2* parts,
                       cudaStream_t stream, int* launches) {
  using L = Fp4Smem<D, GT>;
  auto* kern = decode_fp4_kernel<T, D, GT, R>;
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = allow_smem(kern, L::kTotalMerge, &configured);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3(w.ctas), dim3(kFp4Warps * 32), w.team == 1 ? L::kTotal : L::kTotalMerge, stream, a,
                 static_cast<const unsigned char*>(k), static_cast<const unsigned char*>(v), w.workers, w.team, parts);
  if (e == cudaSuccess) ++*launches;
  if (e != cudaSuccess || w.workers == 1) return e;  // one span cuts no item
  const long long rows = (long long)a.num_seqs * a.num_q_heads;
  e = launch_pdl(decode_fp4_merge_kernel<T, D>, dim3((unsigned)rows), dim3(128), 0, stream, a,
                 static_cast<const int2*>(parts));
  if (e == cudaSuccess) ++*launches;
  return e;
}

template <typename T, int D, int GT>
cudaError_t launch_fp4_copy(const DecodeArgs& a, const void* k, const void* v, const Fp4Split& w, int2* parts,
                            cudaStream_t st, int* n) {
  // a copy's tokens lie in one block
  if (a.block_size % 32 == 0) return launch_fp4<T, D, GT, 32>(a, k, v, w, parts, st, n);
  if (a.block_size % 16 == 0) return launch_fp4<T, D, GT, 16>(a, k, v, w, parts, st, n);
  return launch_fp4<T, D, GT, 8>(a, k, v, w, parts, st, n);
}

template <typename T, int D>
cudaError_t launch_fp4_group(const DecodeArgs& a, const void* k, const void* v, const Fp4Split& w, int2* parts,
                             cudaStream_t st, int* n) {
  if (a.group <= 4) return launch_fp4_copy<T, D, 4>(a, k, v, w, parts, st, n);
  if (a.group <= 8) return launch_fp4_copy<T, D, 8>(a, k, v, w, parts, st, n);
  return launch_fp4_copy<T, D, 16>(a, k, v, w, parts, st, n);
}

}  // namespace

bool fp4_decode_split(int num_seqs, int num_kv_heads, int max_context_len, int partition_tokens, Fp4Split* w) {
  *w = Fp4Split{1, 1, 1};
  if (num_seqs == 0) return true;
  if (max_context_len > 1 << 30) return false;
  const long long per_item = (max_context_len + kFp4Chunk - 1) / kFp4Chunk, items = (long long)num_seqs * num_kv_heads;
  if (items > 0x7fffffff || per_item * items > 0x7fffffffLL) return false;
  const int wave = 148 * kFp4Ctas;  // CTAs that a B200 holds at once
  w->team = items >= FP4_TEAM ? 1 : kFp4Warps;
  const long long least = (long long)w->team * (partition_tokens > 0 ? (partition_tokens + kFp4Chunk - 1) / kFp4Chunk : 1);
  const long long most = (per_item * items + least - 1) / least;  // workers that have something to do
  const long long all = (long long)wave * (kFp4Warps / w->team);
  w->workers = (int)(most < 1 ? 1 : most < all ? most : all);
  w->ctas = w->workers < wave ? w->workers : wave;
  return true;
}

cudaError_t launch_decode_fp4(const DecodeArgs& a, int dtype, int head_dim, const void* k_pool, const void* v_pool,
                              const Fp4Split& split, int2* item_parts, cudaStream_t stream, int* launches) {
  if (dtype == 0)
    return head_dim == 128 ? launch_fp4_group<__half, 128>(a, k_pool, v_pool, split, item_parts, stream, launches)
                           : launch_fp4_group<__half, 64>(a, k_pool, v_pool, split, item_parts, stream, launches);
  return head_dim == 128 ? launch_fp4_group<__nv_bfloat16, 128>(a, k_pool, v_pool, split, item_parts, stream, launches)
                         : launch_fp4_group<__nv_bfloat16, 64>(a, k_pool, v_pool, split, item_parts, stream, launches);
}

}  // namespace pa
