// pa_decode_fp4.cu -- single-token decode attention over an E2M1 cache.
//
// Work split.  An item is a (sequence, kv head) pair; its context is cut into
// chunks of 64 tokens.  The chunks of all items, in order, are split evenly into
// one span per worker: long and short contexts balance, and only an item cut by
// a span's border needs merging.  A worker finds its span by a scan over the
// context lengths.  A worker is a warp; or, at groups of more than 8 heads of 64
// where there are fewer items than CTAs, a team: the four warps of a CTA, which take a span's
// chunks in turn and merge through shared memory at an item's end; whole items
// of few chunks (kFp4Solo) go to one warp, without a merge.  Which warp takes what is
// fixed: chunks claimed by whoever came first gave other bits from call to call.  A team cuts
// an item into a quarter of the parts, and its warps share the merges: 32 sequences of 8000 to
// 8192 tokens, 64/4 heads of 64, take 45.6 us against 48.7 by warps, 8 of 50 to 8000 20 against
// 26, one of 1000 9.7 against 13.9; where all items are short its uneven end costs more (40 of 20
// to 300 16.2 against 11.2).  At heads of 128 and at smaller groups it costs more than it saves
// (both sides with p as one f16, see below: 4 sequences of 300 to 40000 tokens, 128/8 heads of
// 128, 63 us by teams and 52 by warps; one of 300 tokens, 32/8 heads, 13.7 and 9.1; 18 of 300 to
// 16000 63 and 48; 6 of 40000 to 131071 with 64/8 heads 125 and 128; one of 60000 30.5 and 32.4).
//
// Copies.  A warp runs its own ring of two stages of bulk copies, across items: a
// (block, head) run is contiguous, so a chunk of K is one copy per block (two
// where a block holds more than the copy: codes, then block scales), one lane
// each, and table entries are read one chunk ahead.
//
// A cut item's parts are merged as they arrive: the parts form a tree (see
// kFp4Radix); a worker publishes its partial result, counts itself in at
// the node, and the last one in combines the children, in order, and goes on to
// the node above with the result, so the outcome does not depend on who came
// last.  Nobody waits.  (A kernel of its own for this cost 8 to 12 us at 64 to
// 128 sequences: its loads start only when the last span has ended.)
//
// What bounds it, on a B200 (128 sequences of 1024 to 4096 tokens, 32/8 heads of
// 128, bf16; 380 MB, 58 us at 6551 GB/s): 94 us, 4.05 TB/s.  It is latency.  No pipe is full:
// issue slots 56 %, the pipe of conversions and logic 51 %, matrix 22 %, DRAM 47 % (6 long
// sequences, 64/8 heads: 53, 48, 31 and 42 %), 320 instructions a warp for 16 tokens; 2.7 warps a
// scheduler do not cover a warp's chain of products, maximum, exponentials, transposes, products.
// The same copies without the arithmetic take 70 us: 2 us of launch and scan, 61 of streaming at
// 6.2 TB/s, the rest the first copies' latency and the last warp's lead; of the other 24 us some 5
// are the merges of cut items.  Measured and not kept (when the whole
// took 87 us, p being one f16): 16 warps per SM with chunks of
// 32 tokens (the work per chunk doubles: 98 us), producer warps that issue the
// copies for twelve others (111 us), one lane issuing all of a warp's copies (93 us),
// small spans claimed at the end (103 us).
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
//      A register holds two neighbours of the contraction, two tokens here: nibbles of
//      both are paired into bytes (one shift and one 3-input logic op per four) before
//      widening.  (Pairing the two dims of a byte instead, against a column that holds p for
//      one and 0 for the other, needs no such step, but a column per head and parity: with p in
//      two parts (below) 96.1 us against 94.4 at 4 heads, 150 against 132 at 8.)
// The 8 x 8 transposes from S^T's layout to P^T's are one movmatrix each.
//
// Softmax per warp in the log2 domain.  The reference m of a head lies 7 below a
// maximum and moves only when a logit exceeds it by more than 15: p <= 2^15 stays
// within f16, the warp-wide maximum and rescaling are rare, and with a sum of 2^7 at
// least f16's smallest step, 2^-24, is 2^-31 of it: what many tiny p lose to
// rounding stays below 2^-12 up to a million tokens.  Any m gives the same quotient.
//
// Roundings: q is bf16 or f16; a bf16 row is scaled by a power of two to a
// largest magnitude in [2^14, 2^15) and is then exact in f16 down to 2^-29 of it.
// p enters the second product as hi + lo, two f16 of 22 bits together, so that the product
// keeps what the sums keep: as one f16 p is 2^-12 off, which shows where V's cancel.  Up to
// groups of 4 the columns 4 .. 7 of a tile repeat the heads and take the lo parts; beyond, lo is a
// product of its own (one f16 against two: 128 sequences, 32/8 heads 88 us and 94; 6 long ones,
// 64/8 heads 126 and 132).  Sums, the softmax statistics and the partial results are fp32.
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "pa_common.cuh"
#include "pa_fp4.cuh"
#include "pa_internal.h"

namespace pa {

constexpr int kFp4Warps = 4;
constexpr int kFp4Chunk = 64;   // tokens a stage holds
constexpr int kFp4Stages = 2;   // per warp
// CTAs per SM: 3, by registers and (D = 128) shared memory; 2 where the state of 16 heads of 128 takes 64 registers of a thread,
// which at 168 spills in the products' loop (128 sequences of 1024 to 4096 tokens, 128/8 heads: 141 us against 210).
constexpr int fp4_ctas(int head_dim, int group) { return head_dim == 128 && group > 8 ? 2 : 3; }
// Children of a merge node, at most: 8; but with a state small enough for four children in flight (GT = 4), all parts of an
// item of up to 24, so that one level does: a level costs some 2 us, a child 0.15 (16 parts of 64 tokens, 8 heads: 10.5 us
// against 11.5 with nodes of 8; 64 parts: nodes of 8 15.5, of 16 16.2, of 32 18.2; GT = 8, 25 parts: 26.3, 28.0, 31.9).
constexpr int kFp4Wide = 24, kFp4Radix = 8;
constexpr int kFp4Solo = 4;     // chunks of an item that a team leaves to one warp, at most (8 measured slower)

constexpr float kFp4Lowest = -3.402823466e38f;  // reference before the first logit: fp32's lowest, so that any finite one raises it

template <int D>
struct Fp4Smem {
  static constexpr int kTokenBytes = D * 9 / 16;
  static constexpr int kPoolBytes = kFp4Chunk * kTokenBytes;  // K or V of one stage
  static constexpr int kStageBytes = 2 * kPoolBytes;
  static constexpr int kBars = kFp4Warps * kFp4Stages * kStageBytes;
  static constexpr int kTeam = kBars + kFp4Warps * kFp4Stages * 8;  // a team's merge verdict
  static constexpr int kTotal = kTeam + 16;
};

// A warp's state as it is stored: output tiles, then maxima and sums.
template <int D, int GT>
struct Fp4State {
  static constexpr int NS = GT == 16 ? 2 : 1;            // tiles of 8 columns of logits
  static constexpr bool kFolded = GT == 4;               // columns 0 .. 3 hold the heads' hi parts, 4 .. 7 their lo parts
  static constexpr int MT = D / 16;                      // 16-row tiles of output dims
  static constexpr int MS = kFolded ? MT / 2 : MT;       // as stored: hi and lo added up, each thread keeps half of the rows
  static constexpr int kBytes = (MS + 1) * NS * 32 * 16;
};
int fp4_state_bytes(int head_dim, int group) {
  if (head_dim == 128) return group <= 4 ? Fp4State<128, 4>::kBytes : group <= 8 ? Fp4State<128, 8>::kBytes : Fp4State<128, 16>::kBytes;
  return group <= 4 ? Fp4State<64, 4>::kBytes : group <= 8 ? Fp4State<64, 8>::kBytes : Fp4State<64, 16>::kBytes;
}

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
// (x, y) *= (a, b) and += (a, b), each one packed instruction.
__device__ __forceinline__ void mul_f32x2(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 u, v;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\tmul.rn.f32x2 u, u, v;\n\t"
      "mov.b64 {%0, %1}, u;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
__device__ __forceinline__ void add_f32x2(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 u, v;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\tadd.rn.f32x2 u, u, v;\n\t"
      "mov.b64 {%0, %1}, u;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// GT: the group's query heads, at most: 4, 8 or 16.  R: tokens of one copy.  TEAM: the CTA's warps share a span.
template <typename T, int D, int GT, int R, bool TEAM>
__global__ void __launch_bounds__(kFp4Warps * 32, fp4_ctas(D, GT))
decode_fp4_kernel(const DecodeArgs a, const unsigned char* __restrict__ k_pool,
                  const unsigned char* __restrict__ v_pool, const int num_workers, const int least, float4* partials,
                  unsigned long long* arrivals) {
  constexpr int NS = Fp4State<D, GT>::NS, MT = Fp4State<D, GT>::MT, MS = Fp4State<D, GT>::MS;
  constexpr bool kFolded = Fp4State<D, GT>::kFolded;
  static_assert(!TEAM || !kFolded, "a team merges states whose hi and lo parts share columns");
  using L = Fp4Smem<D>;
  constexpr int NW = kFp4Warps, NST = kFp4Stages, CT = kFp4Chunk, TILES = 2;
  constexpr int KW = D / 32;   // words of K codes a thread takes per row
  constexpr int VW = D / 64;   // words of V codes a thread takes per row
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

  // ---- this warp's span of chunks, and the sequence it starts in
  const int S = a.num_seqs, Hkv = a.num_kv_heads, G = a.group;
  const int worker = TEAM ? blockIdx.x : blockIdx.x + gridDim.x * warp;
  auto context = [&](int s) { return max(0, min(__ldg(a.context_lens + s), a.max_context_len)); };
  // lane i counts the chunks of the sequences [i run, (i + 1) run)
  const int run = (S - 1) / 1024 * 32 + 32;
  int run_sum = 0, run_at = 0, run_left = run;
  bool bad = false;
  for (int s0 = 0; s0 < S; s0 += 4 * 32) {
    int n[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int s = s0 + j * 32 + lane, c = s < S ? __ldg(a.context_lens + s) : 0;
      bad |= c < 0 || c > a.max_context_len;
      n[j] = (max(0, min(c, a.max_context_len)) + CT - 1) / CT;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int sum = (int)__reduce_add_sync(0xffffffffu, (unsigned)n[j]);
      if (lane == run_at) run_sum += sum;
      if ((run_left -= 32) == 0) { ++run_at; run_left = run; }
    }
  }
  if (bad && blockIdx.x == 0 && warp == 0) report(a.err, kErrContextLen);
  run_sum *= Hkv;
  int run_end = run_sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, run_end, d);
    if (lane >= d) run_end += v;
  }
  const int chunks = __shfl_sync(0xffffffffu, run_end, 31);  // below 2^31
  const int workers = max(1, min(num_workers, chunks / least));  // spans of `least` chunks or more, where there are as many
  // sequences without tokens: zero rows
  for (int s = blockIdx.x + gridDim.x * warp; s < S; s += gridDim.x * NW)
    if (context(s) == 0) {
      uint4* o = reinterpret_cast<uint4*>(a.out + (size_t)s * a.num_q_heads * D);
      for (int i = lane; i < a.num_q_heads * D / 8; i += 32) o[i] = make_uint4(0, 0, 0, 0);
    }
  if (worker >= workers || chunks == 0) return;
  const int span_begin = (int)((long long)chunks * worker / workers);
  const int span_end = (int)((long long)chunks * (worker + 1) / workers);
  // opens this span's arrival word: no count of another call is above the tag, and one of this call's stays
  const unsigned long long tag = a.epoch << 8;
  if (lane == 0) atomicMax(arrivals + worker, tag);
  // Team: a span's chunks go to its warps by number, all of a short whole item's to one warp, items in turn: which warp
  // adds what up is fixed, and with it every bit of the sums.
  auto one_warps = [&](int start, int n) { return TEAM && n <= kFp4Solo && start >= span_begin && start + n <= span_end; };
  auto owner = [&](int s, int head) { return (s * Hkv + head) % NW; };
  // the sequence of chunk span_begin, and the number of its first chunk: its run, then 32 sequences at a time
  const int in_run = __ffs(__ballot_sync(0xffffffffu, span_begin < run_end)) - 1;
  int seq = in_run * run, seq_base = __shfl_sync(0xffffffffu, run_end - run_sum, in_run);
  for (;; seq += 32) {
    const int n = seq + lane < S ? (context(seq + lane) + CT - 1) / CT * Hkv : 0;
    int upto = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += v;
    }
    const unsigned after = __ballot_sync(0xffffffffu, span_begin < seq_base + upto);
    if (after) {
      const int l = __ffs(after) - 1;
      seq += l;
      seq_base += __shfl_sync(0xffffffffu, upto - n, l);
      break;
    }
    seq_base += __shfl_sync(0xffffffffu, upto, 31);
  }

  // ---- copies: lane (sub, piece, pool) moves one piece of one group of R tokens, which never crosses a block
  const int bs = a.block_size;
  const bool whole = R == bs;  // codes and scales of the group are one run
  const int c_sub = lane >> 2, c_piece = (lane >> 1) & 1;
  const bool c_lane = c_sub * R < CT && (c_piece == 0 || !whole);
  const uint32_t c_bytes = whole ? R * L::kTokenBytes : c_piece ? R * (D / 16) : R * (D / 2);
  const uint32_t c_dst = ((lane & 1) ? L::kPoolBytes : 0) + c_sub * R * L::kTokenBytes + (c_piece ? R * (D / 2) : 0);
  const int run_bytes = (int)fp4_head_bytes(bs, D);  // a block's bytes are below 2^31
  const unsigned block_bytes = (unsigned)run_bytes * Hkv;
  const unsigned char* c_base = ((lane & 1) ? v_pool : k_pool) + (c_piece ? bs * (D / 2) : 0);
  const int c_unit = c_piece ? D / 16 : D / 2;
  // The copies' cursor: the next chunk to fetch, its item, chunk number there and context;
  // this lane's group in it: its table entry and its offset in the block.
  int f_at = span_begin, f_seq = seq, f_head, f_chunk, f_ctx = context(seq), f_off;
  const int32_t* f_entry;          // of the group in the block table
  const int step_idx = CT / bs, step_off = CT - step_idx * bs;
  auto place = [&]() {
    const int idx = (f_chunk * CT + c_sub * R) / bs;
    f_off = f_chunk * CT + c_sub * R - idx * bs;
    f_entry = a.block_tables + (size_t)f_seq * a.max_blocks_per_seq + idx;
  };
  {
    const int rel = span_begin - seq_base, n = (f_ctx + CT - 1) / CT;
    f_head = rel / n;
    f_chunk = rel - f_head * n;
    place();
  }
  // on to the first chunk of the next item, which exists
  auto next_item = [&]() {
    f_chunk = 0;
    if (++f_head == Hkv) {
      f_head = 0;
      do {
        f_ctx = context(++f_seq);
      } while (f_ctx == 0);
    }
  };
  // the cursor's item's queries will be wanted in a moment
  auto warm = [&]() {
    const char* q = reinterpret_cast<const char*>(a.q + ((size_t)f_seq * a.num_q_heads + f_head * G) * D);
    if (lane * 128 < G * D * 2) asm volatile("prefetch.global.L1 [%0];" ::"l"(q + lane * 128));
  };
  struct Group {
    int chunk, blk, off, head;  // chunk (the span's end: none), table entry, first token in the block (negative:
                                // nothing to copy), kv head
  };
  auto fetch = [&]() {
    Group e{span_end, 0, -1, 0};
    if constexpr (TEAM) {  // from the cursor on, this warp's next chunk
      bool moved = false;
      for (;;) {
        const int n = (f_ctx + CT - 1) / CT, start = f_at - f_chunk;
        if (!one_warps(start, n)) f_chunk += (warp - (f_at - span_begin)) & (NW - 1);
        else if (owner(f_seq, f_head) != warp) f_chunk = n;
        f_at = start + min(f_chunk, n);
        if (f_at >= span_end) return e;
        if (f_chunk < n) break;
        next_item();
        moved = true;
      }
      place();
      if (moved) warm();
    }
    if (TEAM || f_at < span_end) {
      e.chunk = f_at;
      e.head = f_head;
      if (c_lane && f_chunk * CT + c_sub * R < f_ctx) {
        e.off = f_off;
        e.blk = __ldg(f_entry);
      }
      ++f_at;
      ++f_chunk;
      if (!TEAM && f_at < span_end) {
        f_entry += step_idx;
        f_off += step_off;
        if (f_off >= bs) { f_off -= bs; ++f_entry; }
        if (f_chunk * CT >= f_ctx) {
          next_item();
          place();
          warm();
        }
      }
    }
    return e;
  };
  int ids[NST], issued = 0;  // chunks in flight
  auto issue = [&](const Group& e) {
    const int k = issued++;
#pragma unroll
    for (int i = 0; i < NST; ++i)
      if (k % NST == i) ids[i] = e.chunk;
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
    if (copy)
      bulk_load(dst, c_base + (unsigned long long)(unsigned)e.blk * block_bytes + (unsigned)(e.head * run_bytes + e.off * c_unit),
                c_bytes, bar);
  };
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
  const int v_code = L::kPoolBytes + t * (D / 2) + g * (D / 16);
  const int v_sc = L::kPoolBytes + kScaleBase + t * (D / 16) + g * (D / 64) / 2;

  // ---- the items of the span, each from its chunk `first` to its end or the span's
  bool failed = false;         // a wait ran out
  int k = 0, at = span_begin;  // this warp's chunk count; the item's first chunk in the span
  int ctx = context(seq), kvh = f_head, first = f_chunk;
  Group next = fetch();
  for (;;) {
    const int item_chunks = (ctx + CT - 1) / CT, len = min(item_chunks - first, span_end - at);
    const bool solo = one_warps(at - first, item_chunks);
    if (!solo || owner(seq, kvh) == warp) {
      // what may be copied by now: a team's stages are free for its merge at the item's end
      const int copy_end = TEAM ? at + len : span_end;
      while (issued - k < NST && next.chunk < copy_end) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        issue(next);
        next = fetch();
      }
      const size_t head0 = (size_t)seq * a.num_q_heads + kvh * G;

      // queries as column fragments: thread (g, t) holds dims [t D/4, (t + 1) D/4) of heads g, g + 8
      // The logit scale is kept positive: its sign goes into the queries, and a zero scale zeroes
      // them (but for NaN and infinity, which become NaN).
      const float cscale = a.scale_log2 * __ldg(a.k_scale + kvh);
      uint32_t bq[NS][KW * 4];
      float xs[NS][2];  // logit scale of this thread's columns 2t, 2t + 1
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        const int h = kFolded ? g & 3 : n * 8 + g;  // folded: columns 4 .. 7 repeat the heads
        uint32_t w[KW * 4];
#pragma unroll
        for (int i = 0; i < KW; ++i) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (h < G) v = *reinterpret_cast<const uint4*>(a.q + (head0 + h) * D + t * (D / 4) + i * 8);
          w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        }
        float down = 1.f;
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
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
          down = __uint_as_float((uint32_t)(e - 14) << 23);
#pragma unroll
          for (int i = 0; i < KW * 4; ++i) {
            const float2 f = Elem<T>::to_f2(w[i]);
            w[i] = f16x2_of(f.x * up, f.y * up);
          }
        }
        const float c = cscale * down;
        const uint32_t sign = c == 0.f ? 0u : c < 0.f ? 0xbc00bc00u : 0x3c003c00u;  // 0, -1 or 1, twice
#pragma unroll
        for (int i = 0; i < KW * 4; ++i) bq[n][i] = hmul2(w[i], sign);
        const float pos = c == 0.f ? 1.f : fabsf(c);
        xs[n][0] = __shfl_sync(0xffffffffu, pos, 8 * t);
        xs[n][1] = __shfl_sync(0xffffffffu, pos, 8 * t + 4);
      }

      float o[MT][NS][4], m[NS][2], l[NS][2];
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[i][n][j] = 0.f;
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        m[n][0] = m[n][1] = kFp4Lowest;
        l[n][0] = l[n][1] = 0.f;
      }

      for (; k < issued; ++k) {
        int chunk = ids[0];
#pragma unroll
        for (int i = 1; i < NST; ++i)
          if (k % NST == i) chunk = ids[i];
        if (chunk >= at + len) break;
        if (failed) continue;
        if (!mbar_wait_warp(bar0 + (k % NST) * 8, (k / NST) & 1, a.err)) {
          // let the copies in flight land, and start no more
          for (int i = k + 1; i < issued; ++i) mbar_wait(bar0 + (i % NST) * 8, (i / NST) & 1, a.err);
          next.chunk = span_end;
          failed = true;
          continue;
        }
        unsigned char* stage = stages + (k % NST) * L::kStageBytes;
        const int n_valid = ctx - (first + chunk - at) * CT;  // of this chunk's tokens
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
          float x[TILES][NS][4];
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
              for (int n = 0; n < NS; ++n) {
                if (w == 0) mma_f16_first(x[i][n], fa[0], fb[0], fa[1], fb[1], bq[n][0], bq[n][1]);
                else mma_f16(x[i][n], fa[0], fb[0], fa[1], fb[1], bq[n][4 * w], bq[n][4 * w + 1]);
                mma_f16(x[i][n], fa[2], fb[2], fa[3], fb[3], bq[n][4 * w + 2], bq[n][4 * w + 3]);
              }
            }
          }

          // ---- softmax
          bool grow = false;
          float top[NS][2];
          if (half + 32 > n_valid) {
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
              for (int i = 0; i < TILES; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  if (half + i * 16 + k_row + (j >> 1) * 8 >= n_valid) x[i][n][j] = -INFINITY;
            __syncwarp();
          }
          // Scaled and rounded before the reference is taken off: fused, a logit of 2^28 or more would differ from its
          // own rounded maximum by more than the exponentials' range.
#pragma unroll
          for (int n = 0; n < NS; ++n) {
#pragma unroll
            for (int i = 0; i < TILES; ++i)
#pragma unroll
              for (int j = 0; j < 4; j += 2) mul_f32x2(x[i][n][j], x[i][n][j + 1], xs[n][0], xs[n][1]);
            top[n][0] = fmaxf(fmaxf(x[0][n][0], x[0][n][2]), fmaxf(x[1][n][0], x[1][n][2]));
            top[n][1] = fmaxf(fmaxf(x[0][n][1], x[0][n][3]), fmaxf(x[1][n][1], x[1][n][3]));
            grow |= top[n][0] - m[n][0] > 15.f || top[n][1] - m[n][1] > 15.f;
          }
          if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                float v = top[n][j];
#pragma unroll
                for (int d = 4; d <= 16; d <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
                const float mn = fmaxf(m[n][j], v - 7.f), al = ex2(m[n][j] - mn);
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
            uint32_t hi[NS][2], lo[NS][2];
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                add_f32x2(x[i][n][2 * j], x[i][n][2 * j + 1], -m[n][0], -m[n][1]);
                const float p0 = ex2(x[i][n][2 * j]), p1 = ex2(x[i][n][2 * j + 1]);
                l[n][0] += p0;
                l[n][1] += p1;
                const uint32_t h = f16x2_of(p0, p1);
                const float2 f = h2_to_f2(h);
                const uint32_t r = f16x2_of(p0 - f.x, p1 - f.y);
                hi[n][j] = transpose_8x8(kFolded && t >= 2 ? r : h);
                if constexpr (!kFolded) lo[n][j] = transpose_8x8(r);
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
                for (int n = 0; n < NS; ++n) {
                  mma_f16(o[4 * w + j][n], ev[0][j], od[0][j], ev[1][j], od[1][j], hi[n][0], hi[n][1]);
                  if constexpr (!kFolded)
                    mma_f16(o[4 * w + j][n], ev[0][j], od[0][j], ev[1][j], od[1][j], lo[n][0], lo[n][1]);
                }
            }
          }
        }
        __syncwarp();
        // the stage is free again: refill it
        if (next.chunk < copy_end) {
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          issue(next);
          next = fetch();
        }
      }

#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int d = 4; d <= 16; d <<= 1) l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], d);
          if (failed) l[n][j] = __int_as_float(0x7fc00000);
        }

      // Writes row `row` of the state's outputs: x[n] are its tiles, f the columns' factors.
      auto emit = [&](int row, const float4 (&x)[NS], const float (&f)[NS][2]) {
        auto pair = [](float v0, float v1) {
          return (uint32_t)Elem<T>::from_f(v0) | ((uint32_t)Elem<T>::from_f(v1) << 16);
        };
        // this thread's dims of head 0: from the tile's rows g and g + 8
        uint16_t* out = a.out + head0 * D + g * (D / 8) + 2 * (kFolded && t >= 2 ? row + MS : row);
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          const int h = n * 8 + (kFolded ? 2 * (t & 1) : 2 * t);  // and h + 1
          if (h < G) *reinterpret_cast<uint32_t*>(out + h * D) = pair(x[n].x * f[n][0], x[n].z * f[n][0]);
          if (h + 1 < G) *reinterpret_cast<uint32_t*>(out + (h + 1) * D) = pair(x[n].y * f[n][1], x[n].w * f[n][1]);
        }
      };
      auto factors = [&](float (&f)[NS][2]) {
        const float v_scale = __ldg(a.v_scale + kvh);
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          f[n][0] = v_scale / l[n][0];
          f[n][1] = v_scale / l[n][1];
        }
      };
      if (solo) {
        float f[NS][2];
        factors(f);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          float4 y[NS];
#pragma unroll
          for (int n = 0; n < NS; ++n) y[n] = make_float4(o[i][n][0], o[i][n][1], o[i][n][2], o[i][n][3]);
          emit(i, y, f);
        }
      } else {

        // From here a warp holds the rows i = row0, row0 + rows_step, ... of the
        // stored state (all of them, or a team's warp every fourth) and every m and l.
        const int row0 = TEAM ? warp : 0;
        constexpr int rows_step = TEAM ? NW : 1, ROWS = (MS + rows_step - 1) / rows_step;
        float4 x[ROWS][NS];
        auto has = [&](int i) { return !TEAM || row0 + i * rows_step < MS; };
        auto at_row = [&](int i, int n) { return (n * MS + row0 + i * rows_step) * 32; };  // in a stored state
        auto at_ml = [&](int n) { return (MS * NS + n) * 32; };
        // adds w0, w1 (columns 2t, 2t + 1) times a stored state's rows
        auto add = [](float4& to, const float4& v, float w0, float w1) {
          to.x = fmaf(v.x, w0, to.x);
          to.y = fmaf(v.y, w1, to.y);
          to.z = fmaf(v.z, w0, to.z);
          to.w = fmaf(v.w, w1, to.w);
        };
        if constexpr (TEAM) {
          float4* state = reinterpret_cast<float4*>(stages) + lane;  // every warp's, in its own stages
#pragma unroll
          for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < MT; ++i) state[(n * MT + i) * 32] = make_float4(o[i][n][0], o[i][n][1], o[i][n][2], o[i][n][3]);
#pragma unroll
          for (int n = 0; n < NS; ++n) state[at_ml(n)] = make_float4(m[n][0], m[n][1], l[n][0], l[n][1]);
          __syncthreads();
          const float4* of[NW];
          float w0[NS][NW], w1[NS][NW];
#pragma unroll
          for (int w = 0; w < NW; ++w) of[w] = reinterpret_cast<const float4*>(smem + w * NST * L::kStageBytes) + lane;
#pragma unroll
          for (int n = 0; n < NS; ++n) {
            float4 ml[NW];
            m[n][0] = m[n][1] = kFp4Lowest;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
              ml[w] = of[w][at_ml(n)];
              m[n][0] = fmaxf(m[n][0], ml[w].x);
              m[n][1] = fmaxf(m[n][1], ml[w].y);
            }
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
              w0[n][w] = ex2(ml[w].x - m[n][0]);
              w1[n][w] = ex2(ml[w].y - m[n][1]);
              l[n][0] = fmaf(ml[w].z, w0[n][w], l[n][0]);
              l[n][1] = fmaf(ml[w].w, w1[n][w], l[n][1]);
            }
          }
#pragma unroll
          for (int i = 0; i < ROWS; ++i)
#pragma unroll
            for (int n = 0; n < NS; ++n) {
              x[i][n] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (!has(i)) continue;
#pragma unroll
              for (int w = 0; w < NW; ++w) add(x[i][n], of[w][at_row(i, n)], w0[n][w], w1[n][w]);
            }
        } else {
#pragma unroll
          for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
              float y[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                y[j] = o[i][n][j];
                if constexpr (kFolded) {  // threads t < 2 keep the first half of the rows, t >= 2 the second
                  const float other = __shfl_xor_sync(0xffffffffu, t < 2 ? o[i + MS][n][j] : y[j], 2);
                  y[j] = (t < 2 ? y[j] : o[i + MS][n][j]) + other;
                }
              }
              x[i][n] = make_float4(y[0], y[1], y[2], y[3]);
            }
        }

        // ---- an item cut by span borders: merge what has arrived
        bool whole_item = first == 0 && len == item_chunks;
        if (!whole_item) {
          // chunk e lies in the span of worker ceil((e + 1) workers / chunks) - 1
          const int item_at = at - first;  // the item's first chunk
          const int lead = (int)(((long long)(item_at + 1) * workers - 1) / chunks);
          const int parts = (int)(((long long)(item_at + item_chunks) * workers - 1) / chunks) - lead + 1;
          const int radix = GT == 4 && parts <= kFp4Wide ? kFp4Wide : kFp4Radix;
          constexpr int kState = Fp4State<D, GT>::kBytes / 16;
          // part p: slot 2 i + 1 of worker i = lead for the item's first part, 2 i for those that started before span i
          auto slot = [&](int p) { return partials + (size_t)(2 * (lead + p) + (p == 0)) * kState + lane; };
          int node = worker - lead, width = 1;  // this result stands for the parts [node, node + width)
          for (;;) {
            float4* mine = slot(node);
#pragma unroll
            for (int n = 0; n < NS; ++n)
#pragma unroll
              for (int i = 0; i < ROWS; ++i)
                if (has(i)) __stcg(mine + at_row(i, n), x[i][n]);
            if (row0 == 0) {
#pragma unroll
              for (int n = 0; n < NS; ++n) __stcg(mine + at_ml(n), make_float4(m[n][0], m[n][1], l[n][0], l[n][1]));
            }
            // the node above: up to `radix` children of this width, from part `up` on
            int up, kids;
            for (;;) {
              up = node / (width * radix) * (width * radix);
              kids = min(radix, (parts - up + width - 1) / width);
              if (kids > 1) break;
              width *= radix;  // an only child: nothing to merge at this level
            }
            __threadfence();
            if constexpr (TEAM) __syncthreads();
            else __syncwarp();
            bool last = false;
            if (TEAM ? threadIdx.x == 0 : lane == 0) {
              // counted in the word of the second child's first span, under this call's tag
              unsigned long long* word = arrivals + lead + up + width;
              unsigned long long old = atomicAdd(word, 1ull);
              if ((old & ~0xffull) != tag) {  // not opened yet: this call's first count replaces what was there
                unsigned long long now = old + 1;
                for (;;) {
                  const bool open = (now & ~0xffull) == tag;
                  old = atomicCAS(word, now, open ? now + 1 : tag | 1);
                  if (old == now) break;
                  now = old;
                }
                if ((old & ~0xffull) != tag) old = tag;
              }
              last = (int)(old & 0xff) + 1 == kids;
              if (last) __stcg(word, 0ull);  // for a replay of the same call
              // Orders the count before the reads below: here, then for the other threads by the barrier (a shuffle orders nothing).
              __threadfence();
              if constexpr (TEAM) *reinterpret_cast<volatile int*>(smem + L::kTeam) = last;
            }
            if constexpr (TEAM) {
              __syncthreads();
              last = *reinterpret_cast<volatile int*>(smem + L::kTeam) != 0;
            } else {
              last = __shfl_sync(0xffffffffu, (int)last, 0);
              __syncwarp();
            }
            if (!last) break;
            // all children, in order, kBatch of them in flight
            constexpr int kBatch = TEAM ? 4 : GT == 4 ? 4 : GT == 8 ? 2 : 1;
            for (int c0 = 0; c0 < kids; c0 += kBatch) {
              float4 y[kBatch][ROWS][NS], ml[kBatch][NS];
#pragma unroll
              for (int b = 0; b < kBatch; ++b) {
                const float4* from = slot(up + min(c0 + b, kids - 1) * width);
#pragma unroll
                for (int n = 0; n < NS; ++n) ml[b][n] = __ldcg(from + at_ml(n));
#pragma unroll
                for (int i = 0; i < ROWS; ++i)
#pragma unroll
                  for (int n = 0; n < NS; ++n)
                    if (has(i)) y[b][i][n] = __ldcg(from + at_row(i, n));
              }
              float a0[NS], a1[NS];  // weights of what has been added up so far
#pragma unroll
              for (int n = 0; n < NS; ++n) {
                float m0 = c0 ? m[n][0] : kFp4Lowest, m1 = c0 ? m[n][1] : kFp4Lowest;
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                  m0 = fmaxf(m0, ml[b][n].x);
                  m1 = fmaxf(m1, ml[b][n].y);
                }
                a0[n] = ex2(m[n][0] - m0);
                a1[n] = ex2(m[n][1] - m1);
                m[n][0] = m0;
                m[n][1] = m1;
                l[n][0] = c0 ? l[n][0] * a0[n] : 0.f;
                l[n][1] = c0 ? l[n][1] * a1[n] : 0.f;
              }
#pragma unroll
              for (int i = 0; i < ROWS; ++i)
#pragma unroll
                for (int n = 0; n < NS; ++n) {
                  const float w0 = a0[n], w1 = a1[n];
                  x[i][n] = c0 ? make_float4(x[i][n].x * w0, x[i][n].y * w1, x[i][n].z * w0, x[i][n].w * w1)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
              for (int b = 0; b < kBatch; ++b)
                if (c0 + b < kids) {
                  float w0[NS], w1[NS];
#pragma unroll
                  for (int n = 0; n < NS; ++n) {
                    w0[n] = ex2(ml[b][n].x - m[n][0]);
                    w1[n] = ex2(ml[b][n].y - m[n][1]);
                    l[n][0] = fmaf(ml[b][n].z, w0[n], l[n][0]);
                    l[n][1] = fmaf(ml[b][n].w, w1[n], l[n][1]);
                  }
#pragma unroll
                  for (int i = 0; i < ROWS; ++i)
#pragma unroll
                    for (int n = 0; n < NS; ++n)
                      if (has(i)) add(x[i][n], y[b][i][n], w0[n], w1[n]);
                }
            }
            node = up;
            width *= radix;
            if (width >= parts) {
              whole_item = true;
              break;
            }
            if constexpr (TEAM) __syncthreads();  // the children are read before the result takes the first one's slot
          }
        }

        if (whole_item) {
          float f[NS][2];
          factors(f);
#pragma unroll
          for (int i = 0; i < ROWS; ++i)
            if (has(i)) emit(row0 + i * rows_step, x[i], f);
        }
        if constexpr (TEAM) __syncthreads();  // the stages are free for copies again
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
}

namespace {

struct Fp4Launch {
  const unsigned char* k;
  const unsigned char* v;
  Fp4Split split;
  float4* partials;
  unsigned long long* arrivals;
  cudaStream_t stream;
};

template <typename T, int D, int GT, int R, bool TEAM>
cudaError_t launch_fp4(const DecodeArgs& a, const Fp4Launch& w) {
  static_assert(Fp4State<D, GT>::kBytes <= kFp4Stages * Fp4Smem<D>::kStageBytes, "a team's warp merges from its stages");
  auto* kern = decode_fp4_kernel<T, D, GT, R, TEAM>;
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = allow_smem(kern, Fp4Smem<D>::kTotal, &configured);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(w.split.ctas), dim3(kFp4Warps * 32), Fp4Smem<D>::kTotal, w.stream, a, w.k, w.v,
                    w.split.workers, w.split.least, w.partials, w.arrivals);
}

template <typename T, int D, int GT, int R>
cudaError_t launch_fp4_team(const DecodeArgs& a, const Fp4Launch& w) {
  if constexpr (GT == 16 && D == 64)
    if (w.split.team) return launch_fp4<T, D, GT, R, true>(a, w);
  return launch_fp4<T, D, GT, R, false>(a, w);
}

template <typename T, int D, int GT>
cudaError_t launch_fp4_copy(const DecodeArgs& a, const Fp4Launch& w) {
  // a copy's tokens lie in one block
  if (a.block_size % 32 == 0) return launch_fp4_team<T, D, GT, 32>(a, w);
  if (a.block_size % 16 == 0) return launch_fp4_team<T, D, GT, 16>(a, w);
  return launch_fp4_team<T, D, GT, 8>(a, w);
}

template <typename T, int D>
cudaError_t launch_fp4_group(const DecodeArgs& a, const Fp4Launch& w) {
  if (a.group <= 4) return launch_fp4_copy<T, D, 4>(a, w);
  if (a.group <= 8) return launch_fp4_copy<T, D, 8>(a, w);
  return launch_fp4_copy<T, D, 16>(a, w);
}

template <typename T>
cudaError_t launch_fp4_dim(const DecodeArgs& a, int head_dim, const Fp4Launch& w) {
  return head_dim == 128 ? launch_fp4_group<T, 128>(a, w) : launch_fp4_group<T, 64>(a, w);
}

}  // namespace

bool fp4_decode_split(int num_seqs, int num_kv_heads, int group, int head_dim, int max_context_len, int partition_tokens,
                      Fp4Split* w) {
  *w = Fp4Split{1, 1, 1, false};
  if (num_seqs == 0) return true;
  if (num_seqs > 1 << 30 || max_context_len > 1 << 30) return false;  // sums with a chunk or a scan's step stay in 31 bits
  const long long per_item = (max_context_len + kFp4Chunk - 1) / kFp4Chunk, items = (long long)num_seqs * num_kv_heads;
  if (items > 0x7fffffff || per_item * items > 0x7fffffffLL) return false;
  const int wave = 148 * fp4_ctas(head_dim, group);  // CTAs that a B200 holds at once
  w->team = head_dim == 64 && group > 8 && items < wave;  // see the top of this file
  // a warp takes a chunk at least, or the caller's partition
  w->least = (partition_tokens > 0 ? (partition_tokens + kFp4Chunk - 1) / kFp4Chunk : 1) * (w->team ? kFp4Warps : 1);
  const long long most = per_item * items / w->least, all = w->team ? wave : wave * kFp4Warps;
  w->workers = (int)(most < 1 ? 1 : most < all ? most : all);
  w->ctas = w->workers < wave ? w->workers : wave;
  return true;
}

cudaError_t launch_decode_fp4(const DecodeArgs& a, int dtype, int head_dim, const void* k_pool, const void* v_pool,
                              const Fp4Split& split, void* partials, unsigned long long* arrivals, cudaStream_t stream,
                              int* launches) {
  const Fp4Launch w{static_cast<const unsigned char*>(k_pool), static_cast<const unsigned char*>(v_pool), split,
                    static_cast<float4*>(partials), arrivals, stream};
  const cudaError_t e = dtype == 0 ? launch_fp4_dim<__half>(a, head_dim, w) : launch_fp4_dim<__nv_bfloat16>(a, head_dim, w);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace pa
