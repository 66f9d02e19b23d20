// Linear attention with a decay per head, over padded or packed variable-length batches:
// chunked kernels for whole sequences (forward and backward) and a kernel for single tokens.
//
//   S_t = lambda S_{t-1} + k_t v_t^T   (d x d, fp32),   o_t = scale S_t^T q_t,   lambda = exp(g)
//
// Chunks of 128 tokens, i and j counting inside a chunk of m valid tokens, R the state that
// the tokens before it leave:
//   o_i = scale (lambda^(i+1) R^T q_i + sum_{j <= i} lambda^(i-j) (q_i . k_j) v_j)
//   R  <- lambda^m R + sum_j lambda^(m-1-j) k_j v_j^T
// so a chunk is four matrix products: P = Q K^T (weighted and masked), P V, Q R, and K^T V'
// with V' the decayed values.  The state of a sequence stays in fp32 registers.
//
// Backward: with dS_t = lambda dS_{t+1} + scale q_t do_t^T,
//   dq_t = scale S_t do_t,   dv_t = dS_t^T k_t,   dk_t = dS_t v_t,   dS_{-1} = lambda dS_0.
// Each of the three is the forward's recurrence again with other tensors in its places:
//   dq: (q, k, v) := (dO, V, K), state S^T;  dk: (V, dO, Q), dv: (K, Q, dO), time reversed.
// So one kernel serves all four, and the backward's three passes share one launch.  Reversed,
// the carried state is kept already decayed to the next token (index r = m - 1 - i):
//   o_i = lambda^r R^T q_i + sum_{j >= i} lambda^(j-i) (..),  R <- lambda^m R + sum_j lambda^(j+1) k_j v_j^T
//
// What it has to move: q, k, v and o once (the backward seven tensors; its passes read ten, the
// two that run side by side sharing their reads through L2).  What bounds it is waiting: with full
// lengths (16 x 2048, 16 heads of 128) DRAM is 56 % busy, the tensor pipe 37 %, shared memory's
// banks 24 % (reads) and 15 % (writes), the issue slots 51 %.  A chunk's jobs hang on each other
// (the weights of a warp whose rows see all keys take 2300 of a chunk's 3600 cycles), and its
// loads, 2200 to 5600 cycles, on the products that free their stage.  With Q R in two buffers, so
// that it need not wait for the outputs of the chunk before, and the issuer's tests side by side,
// the long ragged batch (8 x 4096..16384, 16 heads of 128) went from 303 to 292 us and the
// gradients of the documents below from 335 to 316; 287 us is 3500 cycles a chunk on the SM with
// the most, 153, and the copy of its tensors 233.  (All times here are of 20 calls in a row at
// 1965 MHz.  After a second of them the power cap holds the clock at 1400 to 1550 MHz: the long
// batch then takes 337 us, the documents' gradients 377.)
// Layout: 128 tokens a chunk are the M of every product; d = 128 is cut into two items of 64
// value columns, because all of its operands fit shared memory twice that way (one item of 128
// columns leaves K and Q single stages, whose copies nothing hides: 553 us).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <initializer_list>

#include "internal.h"
#include "sm100.cuh"

namespace sigattn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kChunk = 128;
constexpr int kCols = 64;       // value columns of a work item
constexpr int kSms = 148;       // B200
constexpr int kMaxSorted = 256;  // batches up to this size are walked longest-first
constexpr int kRing = 8;         // work items decoded ahead
constexpr int kMaxSegs = 16;     // of a sequence
constexpr int kThreads = 768;
// first warps of P (4), V' (4), the outputs (4), the state (8); last, those of the items and of
// the zero rows
constexpr int kWarpP = 2, kWarpV = 6, kWarpO = 10, kWarpS = 14, kWarpI = 22;

struct LinPass {
  int q, k, v;     // which of the tensor maps stand in the places of q, k, v
  int reverse;
  float o1, o2;    // factors of Q R and of P V in the output
  float vs;        // factor of V' (what the state accumulates)
  int o;           // tensor map of the output
  __nv_bfloat16* out;
  int64_t o_sb, o_sn, o_sh;
  const float* init;    // state before the first chunk, nullptr: 0; element (row, col) of
  int init_sr, init_sc;  // (b, h) at (b H + h) D D + row init_sr + col init_sc
  float* fin;            // state after the last chunk [B, H, D, D], nullptr: not wanted
  float* seg;            // [B, H, nseg, D, D]: see sigattn_linear_workspace_size
  int rest;              // packed: rows of no sequence are written as 0
};

struct LinParams {
  CUtensorMap map[7];  // inputs (boxes of 128 rows), then outputs (32 rows)
  LinPass pass[3];
  int npass, B, H, N, T, nseg, seg_chunks, nitems;
  const int32_t* lengths;
  const int32_t* cu;
  const float* log_decay;
  int* status;
  unsigned long long wait_ns;
};

// log2 of the decay: log_decay above 0 counts as 0, and below -1e4 as -1e4 (lambda = 0 in
// fp32 either way), so that 0 * log2(lambda) = 0 and lambda^0 = 1 for a decay of exp(-inf).
__device__ __forceinline__ float clamped_decay(const LinParams& p, int h) {
  return fmaxf(fminf(__ldg(p.log_decay + h), 0.0f), -1e4f);
}

struct Seq {
  int n, row0, tma_b;  // tokens, first row in the tensors' token dimension, batch coordinate
};

// Lengths and offsets are device data: clamped, so that no value of theirs reaches outside
// the tensors.
__device__ __forceinline__ Seq sequence(const LinParams& p, int b) {
  Seq s;
  if (p.cu) {
    s.row0 = max(0, min(__ldg(p.cu + b), p.T));
    const int end = max(s.row0, min(__ldg(p.cu + b + 1), p.T));
    s.n = min(end - s.row0, p.N);
    s.tma_b = 0;
  } else {
    s.n = p.lengths ? max(0, min(__ldg(p.lengths + b), p.N)) : p.N;
    s.row0 = 0;
    s.tma_b = b;
  }
  return s;
}

struct alignas(16) Item {
  Seq s;
  int pass;     // -1: no more items
  int b, h, slice, seg;
  int c0, cn;   // its chunks [c0, c0 + cn)
  float l2;     // log2 lambda
  float full;   // lambda^128, and lambda^m for the last chunk of the sequence.  exp in 64 bits:
  float part;   // the state is multiplied by them once a chunk, so their errors add up
};

// Work item w: sequences longest-first (order), then segment, head, pass and slice of value
// columns, so that the items that read the same rows run side by side.
template <int D>
__device__ __forceinline__ Item decode(const LinParams& p, const uint8_t* order, int w) {
  Item it;
  it.slice = w % (D / kCols);
  w /= D / kCols;
  it.pass = w % p.npass;
  w /= p.npass;
  it.h = w % p.H;
  w /= p.H;
  it.seg = w % p.nseg;
  w /= p.nseg;
  it.b = p.B <= kMaxSorted ? order[w] : w;
  it.s = sequence(p, it.b);
  it.c0 = it.seg * p.seg_chunks;
  const int chunks = (it.s.n + kChunk - 1) / kChunk;
  it.cn = max(0, min(p.seg_chunks, chunks - it.c0));
  return it;
}

// The j-th chunk of an item in its pass's direction, and its valid tokens.
__device__ __forceinline__ int chunk_of(const Item& it, bool reverse, int j) {
  return reverse ? it.c0 + it.cn - 1 - j : it.c0 + j;
}
__device__ __forceinline__ int valid_of(const Item& it, int c) {
  return min(kChunk, it.s.n - c * kChunk);
}

// Waits for the last of n phases of a ring of `len` barriers that falls to its x-th (none if there
// is no such barrier, or no phase of it).
__device__ __forceinline__ void wait_last(uint64_t* bars, int x, int n, int len,
                                          const WaitCtx& w) {
  if (x < len && x < n) mbar_wait(bars + x, (n - 1 - x) / len & 1, w);
  __syncwarp();
}

template <int D, bool OUT, bool TWO>
struct LinLayout {
  static constexpr int kBoxes = D / 64;
  static constexpr int kBox = 128 * 128;            // 128 tokens x 64 bf16
  static constexpr int kTile = kBoxes * kBox;       // a Q or K tile
  // Stages of Q and K, and of V.  Without the outputs there are no Q, R and O, and their room
  // goes to stages and a second V'.
  static constexpr int kSt = OUT ? (D == 64 ? 3 : 2) : (D == 64 ? 4 : 3);
  static constexpr int kVs = OUT ? (D == 64 ? 4 : TWO ? 2 : 3) : (D == 64 ? 4 : 3);
  static constexpr int kNu = OUT ? 1 : 2;           // buffers of V' and U
  static constexpr int kNo = TWO ? 1 : 2;           // buffers of Q R
  static constexpr int kK = 0;
  static constexpr int kQ = kK + kSt * kTile;
  static constexpr int kV = kQ + (OUT ? kSt * kTile : 0);
  static constexpr int kVp = kV + kVs * kBox;       // V' and (TWO) behind it its rounding error
  static constexpr int kVpSize = TWO ? 2 * kBox : kBox;
  static constexpr int kR = kVp + kNu * kVpSize;   // bf16 state, D rows of 64
  static constexpr int kO = kR + (OUT ? D * 128 : 0);  // outputs on their way, 4 KB per warp
  static constexpr int kBar = kO + (OUT ? kBox : 0);
  // qk_full[St] qk_empty[St] v_full[Vs] pv_done[Vs] s_full[2] p_full[2]
  // u_full[2] u_empty[2] vp_full[2] o_empty[2] r_full done item_full[8] item_empty[8]
  static constexpr int kNumBars = 2 * kSt + 2 * kVs + 14 + 2 * kRing;
  static constexpr int kMisc = (kBar + 8 * kNumBars + 15) / 16 * 16;  // tmem base, flags
  static constexpr int kPow = kMisc + 16;            // powers of lambda, 32 per warp of P
  static constexpr int kItems = kPow + 4 * 32 * 4;   // work items decoded ahead
  static constexpr int kOrder = kItems + kRing * sizeof(Item);
  static constexpr int kBytes = kOrder + kMaxSorted;
  static constexpr int kAlloc = kBytes + 1024;       // slack for 1024-byte alignment
  // TMEM columns
  static constexpr int kTS = 0;     // two S / P buffers of 128
  static constexpr int kTO2 = 256;  // P V
  static constexpr int kTO1 = 320;  // Q R
  // K^T V' and (TWO) K^T times its rounding error
  static constexpr int kTU = kTO1 + kNo * kCols;
};

// Products of a chunk with the commit behind them, all issued under one elect.sync (see
// mma_ss_lh_w): these loops are unrolled in full, and four roles' code has to stay in the
// instruction cache together, so a product is kept to a handful of instructions.
#define SIGATTN_LIN_STEP(OA, OB)                                               \
  "add.u32 la, %1, " #OA ";\n\tadd.u32 lb, %2, " #OB ";\n\t"                   \
  "mov.b64 da, {la, %3};\n\tmov.b64 db, {lb, %3};\n\t"                        \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, q;\n\t"
#define SIGATTN_LIN_HEAD                                                        \
  "{\n\t.reg .pred p, q, e;\n\t.reg .b64 da, db;\n\t.reg .b32 la, lb;\n\t"     \
  "setp.ne.b32 p, %6, 1;\n\tsetp.ne.b32 q, %6, 0;\n\telect.sync _|e, 0xffffffff;\n\t" \
  "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"                        \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t"
#define SIGATTN_LIN_TAIL \
  "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t}\n"

// D = Q R: A K-major (32 bytes a step, boxes of 64 columns), B MN-major (2048 bytes a step).
template <int kSteps>
__device__ __forceinline__ void mma_qr_commit_w(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                                uint32_t hi, uint32_t idesc, uint64_t* bar) {
  static_assert(kSteps == 4 || kSteps == 8, "d = 64 or 128");
  if constexpr (kSteps == 4) {
    asm volatile(SIGATTN_LIN_HEAD SIGATTN_LIN_STEP(2, 128) SIGATTN_LIN_STEP(4, 256)
                     SIGATTN_LIN_STEP(6, 384) SIGATTN_LIN_TAIL ::"r"(d_tmem),
                 "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(smem_u32(bar)), "r"(1u)
                 : "memory");
  } else {
    asm volatile(SIGATTN_LIN_HEAD SIGATTN_LIN_STEP(2, 128) SIGATTN_LIN_STEP(4, 256)
                     SIGATTN_LIN_STEP(6, 384) SIGATTN_LIN_STEP(1024, 512)
                         SIGATTN_LIN_STEP(1026, 640) SIGATTN_LIN_STEP(1028, 768)
                             SIGATTN_LIN_STEP(1030, 896) SIGATTN_LIN_TAIL ::"r"(d_tmem),
                 "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(smem_u32(bar)), "r"(1u)
                 : "memory");
  }
}

// D = K^T V' over 128 tokens: A and B MN-major, 16 tokens (2048 bytes) a step.
__device__ __forceinline__ void mma_kv_commit_w(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                                uint32_t hi, uint32_t idesc, uint64_t* bar) {
  asm volatile(SIGATTN_LIN_HEAD SIGATTN_LIN_STEP(128, 128) SIGATTN_LIN_STEP(256, 256)
                   SIGATTN_LIN_STEP(384, 384) SIGATTN_LIN_STEP(512, 512)
                       SIGATTN_LIN_STEP(640, 640) SIGATTN_LIN_STEP(768, 768)
                           SIGATTN_LIN_STEP(896, 896) SIGATTN_LIN_TAIL ::"r"(d_tmem),
               "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(smem_u32(bar)), "r"(1u)
               : "memory");
}
#undef SIGATTN_LIN_STEP
#undef SIGATTN_LIN_HEAD
#undef SIGATTN_LIN_TAIL

// lambda^|i - j| in blocks of 32 columns is the product of a row's power f up to the block's
// near end and a column's power pow[c] from there.  Off the diagonal both are at most 1 for any
// decay; in the diagonal block f is lambda^-31 at most, 2^62 where lambda is 1/4 or more; below
// that each element takes an exp2 of its own (weigh_near).

// Waits for the reads of TMEM; r, one of them, is not used before (which the compiler could not
// know when the read and its use are in different steps of a loop).
__device__ __forceinline__ void tmem_wait_ld_of(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}

// 16 columns of a row of S.  masked: bit c of keep says whether column c counts.
__device__ __forceinline__ void weigh(const uint32_t (&s)[16], float f, const float* pow,
                                      bool masked, uint32_t keep, uint32_t (&pk)[8]) {
  const float2 f2 = make_float2(f, f);
#pragma unroll
  for (int c = 0; c < 16; c += 4) {
    const float4 q = *reinterpret_cast<const float4*>(pow + c);
    const float2 a = mul2(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])),
                          mul2(f2, make_float2(q.x, q.y)));
    const float2 b = mul2(make_float2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])),
                          mul2(f2, make_float2(q.z, q.w)));
    pk[c / 2] = pack_bf16x2(a.x, a.y);
    pk[c / 2 + 1] = pack_bf16x2(b.x, b.y);
  }
  if (masked) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
      pk[c] &= (keep >> 2 * c & 1u ? 0xFFFFu : 0u) | (keep >> 2 * c & 2u ? 0xFFFF0000u : 0u);
  }
}

// 16 columns of row i of S in the diagonal block; at = j - i of the first.
__device__ __forceinline__ void weigh_near(const uint32_t (&s)[16], float l2, bool rev, int at,
                                           int last, uint32_t (&pk)[8]) {
  const float x0 = l2 * static_cast<float>(rev ? at : -at), dx = rev ? l2 : -l2;
#pragma unroll
  for (int c = 0; c < 16; c += 2) {
    float f[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const bool keep = rev ? at + c + y >= 0 && c + y < last : at + c + y <= 0;
      const float x = ex2_approx(fmaf(dx, static_cast<float>(c + y), x0));
      f[y] = keep ? __uint_as_float(s[c + y]) * x : 0.0f;
    }
    pk[c / 2] = pack_bf16x2(f[0], f[1]);
  }
}

// OUT: the whole computation.  Otherwise only the state that each segment of a sequence
// leaves from a zero start is computed, into pass.seg.
// TWO: V' is carried as the sum of two bf16 numbers, because a state is handed out, whose fp32
// accuracy a rounded V' would cost (2^-9 instead of 2^-18).  Where the state only serves the
// outputs, for which it is rounded to bf16 anyway, V' is rounded once: the outputs are 2.6e-3
// off instead of 2.3e-3 (relative, 2-norm; their own rounding is 1.7e-3), the long ragged batch
// took 303 us instead of 328 when it was changed, gradients of 64 documents (32768 tokens, 16
// heads of 128) 357 instead of 430.
//
// Warps: 0 copies, 1 issues the products, the last two decode the work items and zero the pad
// rows (at their own pace: written by the outputs' warps after an item's last chunk they held
// the next item back, 341 us instead of 330 on the long ragged batch); and four jobs on a chunk,
// each with warps of its own so that none waits for another's turn:
//   P       S from TMEM, decayed, masked and rounded into the A operand of P V
//   V'      the decayed values, rounded once or as the sum of two bf16 numbers
//   O       lambda^(i+1) Q R + P V to bf16 and out, a tensor-map store of 32 rows per warp
//   state   R <- lambda^m R + K^T V' in registers; its bf16 copy is the B operand of Q R
template <int D, bool OUT, bool TWO>
__global__ void __launch_bounds__(kThreads, 1)
    linear_kernel(const __grid_constant__ LinParams p) {
  using L = LinLayout<D, OUT, TWO>;
  constexpr int ST = L::kSt, VS = L::kVs;
  constexpr int NU = L::kNu;
  extern __shared__ uint8_t smem_raw[];
  // (an offset, not a cast of the rounded address, which would lose its address space)
  uint8_t* smem = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);
  const int warp = warp_id(), lane = lane_id();
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* qk_full = bars;
  uint64_t* qk_empty = qk_full + ST;   // S, K^T V' and Q R of the chunk complete
  uint64_t* v_full = qk_empty + ST;
  uint64_t* pv_done = v_full + VS;     // P V of the chunk complete: outputs ready, V free
  uint64_t* s_full = pv_done + VS;
  uint64_t* p_full = s_full + 2;
  uint64_t* u_full = p_full + 2;       // K^T V' complete: U ready, V' free
  uint64_t* u_empty = u_full + 2;
  uint64_t* vp_full = u_empty + 2;
  uint64_t* o_empty = vp_full + 2;     // outputs read from TMEM
  uint64_t* r_full = o_empty + 2;
  uint64_t* done = r_full + 1;
  uint64_t* item_full = done + 1;
  uint64_t* item_empty = item_full + kRing;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  volatile int* drain_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 8);
  Item* items = reinterpret_cast<Item*>(smem + L::kItems);
  uint8_t* order = smem + L::kOrder;
  const WaitCtx wctx{p.status, p.wait_ns, abort_flag}, drain{p.status, kDrainWaitNs, drain_flag};

  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(qk_full + i, 1);
      mbar_init(qk_empty + i, 1);
    }
    for (int i = 0; i < VS; ++i) {
      mbar_init(v_full + i, 1);
      mbar_init(pv_done + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4);
      mbar_init(u_full + i, 1);
      mbar_init(u_empty + i, 8);
      mbar_init(vp_full + i, 4);
      mbar_init(o_empty + i, 4);
    }
    mbar_init(r_full, 8);
    mbar_init(done, 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(item_full + i, 1);
      mbar_init(item_empty + i, OUT ? (p.cu ? 21 : 22) : 17);  // the warps that take items
    }
    *abort_flag = 0;
    *drain_flag = 0;
    fence_barrier_init();
  }
  __syncwarp();
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  if (p.B <= kMaxSorted) {
    // ranks by length, ties by index: every CTA derives the same order
    int* len = reinterpret_cast<int*>(smem);  // before any tile arrives here
    for (int b = threadIdx.x; b < p.B; b += kThreads) len[b] = sequence(p, b).n;
    __syncthreads();
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
      int rank = 0;
      for (int x = 0; x < p.B; ++x) rank += len[x] > len[b] || (len[x] == len[b] && x < b);
      order[rank] = static_cast<uint8_t>(b);
    }
    // the copies that overwrite len go through the async proxy
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // The k-th work item of this CTA, from the ring; false at the end of the list (and after a
  // wait that gave up).  Called by whole warps; every one of them takes every item.
  auto take = [&](int k, Item& it) -> bool {
    if (!mbar_wait_w(item_full + k % kRing, (k / kRing) & 1, wctx)) return false;
    it = items[k % kRing];
    __syncwarp();
    if (lane == 0) mbar_arrive(item_empty + k % kRing);
    return it.pass >= 0;
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    int t = 0, tv = 0;  // chunks whose Q and K, whose V copies are issued
    bool ok = true;
    Item it;
    for (int k = 0; ok && take(k, it); ++k) {
      if (lane == 0) {
        const LinPass& ps = p.pass[it.pass];
        const CUtensorMap* mq = p.map + ps.q;
        const CUtensorMap* mk = p.map + ps.k;
        const CUtensorMap* mv = p.map + ps.v;
        for (int j = 0; j < it.cn; ++j) {
          const int s = t % ST, vs = tv % VS;
          const int row = it.s.row0 + chunk_of(it, ps.reverse, j) * kChunk;
          if (t >= ST && !(ok = mbar_wait(qk_empty + s, ((t / ST) - 1) & 1, wctx))) break;
          mbar_arrive_expect_tx(qk_full + s, (OUT ? 2 : 1) * L::kTile);
          for (int x = 0; x < L::kBoxes; ++x) {
            tma_load_4d(smem + L::kK + s * L::kTile + x * L::kBox, mk, qk_full + s, x * 64, row,
                        it.h, it.s.tma_b);
            if (OUT)
              tma_load_4d(smem + L::kQ + s * L::kTile + x * L::kBox, mq, qk_full + s, x * 64, row,
                          it.h, it.s.tma_b);
          }
          ++t;
          if (tv >= VS && !(ok = mbar_wait(pv_done + vs, ((tv / VS) - 1) & 1, wctx))) break;
          mbar_arrive_expect_tx(v_full + vs, L::kBox);
          tma_load_4d(smem + L::kV + vs * L::kBox, mv, v_full + vs, it.slice * kCols, row, it.h,
                      it.s.tma_b);
          ++tv;
        }
      }
      ok = __all_sync(0xFFFFFFFFu, ok);
    }
    // Let the copies still in flight land before the CTA's shared memory goes away: always, as the
    // warps that wait for them may give up after this one has issued its last.  A lane for each
    // barrier, which waits for its last phase.
    t = __shfl_sync(0xFFFFFFFFu, t, 0);
    tv = __shfl_sync(0xFFFFFFFFu, tv, 0);
    const bool v = lane >= ST;
    wait_last(v ? v_full : qk_full, v ? lane - ST : lane, v ? tv : t, v ? VS : ST, drain);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    // Four streams of products, each in chunk order; whichever has its operands goes next.
    // The tensor pipe runs in issue order, so a buffer may be overwritten by a product that
    // is issued after the last one that reads it.  A test after a product waits some 500 cycles
    // behind it, so U comes before Q R, which may then follow it at once (287 us; the other way
    // round 292 on the long ragged batch).
    constexpr uint32_t kHi = sw128_desc_hi(1024);
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, false);
    constexpr uint32_t idesc_o = idesc_bf16_f32(128, kCols, true);
    constexpr uint32_t idesc_u = idesc_bf16_f32(128, TWO ? 2 * kCols : kCols, true, true);
    int total = 0;
    for (int k = lane; snake_item(k) < p.nitems; k += 32)
      total += decode<D>(p, order, snake_item(k)).cn;
    total = __reduce_add_sync(0xFFFFFFFFu, total);
    // Seven lanes hold one barrier each that the streams' next products wait for, so that one
    // test answers for all of them (one after another the tests took as long as the products).
    // A barrier that frees a buffer starts at parity 1, as if its first phase had passed; P V has
    // one buffer, so that it waits for the outputs of the chunk before, in the other barrier.
    enum { kP, kPe, kR, kOe, kVf, kUe, kQk, kTests };
    uint64_t* const base[kTests] = {p_full, o_empty, r_full, o_empty, vp_full, u_empty, qk_full};
    constexpr int kLen[kTests] = {2, 2, 1, 2, NU, NU, ST};
    uint64_t* mine = p_full;
    int ring = 1;
#pragma unroll
    for (int x = 0; x < kTests; ++x)
      if (lane == x) mine = base[x], ring = kLen[x];
    int at = lane == kPe || (lane == kOe && L::kNo == 1);
    uint32_t parity = lane == kPe || lane == kOe || lane == kUe;
    const uint32_t stream = lane <= kPe ? 1u : lane <= kOe ? 2u : lane <= kUe || !OUT ? 4u : 8u;
    int ts = 0, tu = 0, to = 0, tp = 0, idle = 0;  // next chunk of each stream
    long long t0 = clock64();
    const long long limit = static_cast<long long>(p.wait_ns) * 2;
    while ((OUT ? tp : tu) < total) {
      const uint32_t ready = __ballot_sync(0xFFFFFFFFu, mbar_test_wait(mine + at, parity));
      __syncwarp();  // what one lane's test has seen the issuing lane sees
      tc_fence_after();
      uint32_t issued = 0u;
      if (OUT && tp < to && (~ready & (1u << kP | 1u << kPe)) == 0u) {
        // O2 = P V (P from TMEM)
        const uint32_t v_base = smem_u32(smem + L::kV + (tp % VS) * L::kBox);
        mma_pv8_commit_w(tmem + L::kTO2, tmem + L::kTS + (tp & 1) * 128,
                         sw128_desc_lo(v_base, L::kBox), kHi, idesc_o, 0u, pv_done + tp % VS);
        ++tp;
        issued |= 1u;
      }
      if (tu < (OUT ? ts : total) &&
          (~ready & (1u << kVf | 1u << kUe | (OUT ? 0u : 1u << kQk))) == 0u) {
        // U = K^T (V' | its rounding error).  A holds the K columns as rows: 128 for d = 128;
        // for d = 64 the chunk stride of 0 gives them twice, lanes 64-127 a copy of 0-63.
        const uint32_t k_base = smem_u32(smem + L::kK + (tu % ST) * L::kTile);
        const uint32_t v_base = smem_u32(smem + L::kVp + tu % NU * L::kVpSize);
        mma_kv_commit_w(tmem + (tu % NU == 0 ? L::kTU : L::kTS),
                        sw128_desc_lo(k_base, D == 128 ? L::kBox : 0),
                        sw128_desc_lo(v_base, L::kBox), kHi, idesc_u, u_full + tu % NU);
        if (!OUT) {
          mma_commit_w(qk_empty + tu % ST);
          mma_commit_w(pv_done + tu % VS);
        }
        ++tu;
        issued |= 4u;
      }
      if (OUT && to < tu && (~ready & (1u << kR | 1u << kOe)) == 0u) {
        // O1 = Q R; with S and U of the chunk issued before, Q and K are free after it
        const uint32_t q_base = smem_u32(smem + L::kQ + (to % ST) * L::kTile);
        const uint32_t r_base = smem_u32(smem + L::kR);
        mma_qr_commit_w<D / 16>(tmem + L::kTO1 + to % L::kNo * kCols, sw128_desc_lo(q_base, 16),
                                sw128_desc_lo(r_base, L::kBox), kHi, idesc_o,
                                qk_empty + to % ST);
        ++to;
        issued |= 2u;
      }
      if (OUT && ts < total && ts < tp + 2 && (ready >> kQk & 1u)) {
        // S = Q K^T
        const uint32_t q_base = smem_u32(smem + L::kQ + (ts % ST) * L::kTile);
        const uint32_t k_base = smem_u32(smem + L::kK + (ts % ST) * L::kTile);
        mma_s_commit_w<D / 16>(tmem + L::kTS + (ts & 1) * 128, sw128_desc_lo(q_base, 16),
                               sw128_desc_lo(k_base, 16), kHi, idesc_s, s_full + (ts & 1));
        ++ts;
        issued |= 8u;
      }
      if (issued & stream) {
        at = at + 1 == ring ? 0 : at + 1;
        parity ^= at == 0;
      }
      if (issued) {
        idle = 0;
      } else if (++idle == 1) {
        t0 = clock64();
      } else if (idle % 32 == 0) {
        const bool late = __any_sync(0xFFFFFFFFu, clock64() - t0 > limit);
        if (__any_sync(0xFFFFFFFFu, late || *abort_flag)) {
          if (lane == 0 && late) atomicOr(p.status, kStatusTimeout);
          *abort_flag = 1;
          break;
        }
      }
    }
    // every MMA complete before the TMEM is released (also after an abort)
    mma_commit_w(done);
    mbar_wait_w(done, 0, drain);
    // ... and every commit's arrival seen, as none may come when the CTA's shared memory is
    // another's: nobody else waits for the last ones of qk_empty and pv_done, and after an abort
    // the warps that would have waited for s_full and u_full are gone.  A lane for each barrier.
    int x = lane, n = OUT ? to : tu, len = ST;
    uint64_t* bar = qk_empty;
    if (x >= ST) x -= ST, n = OUT ? tp : tu, len = VS, bar = pv_done;
    if (bar == pv_done && x >= VS) x -= VS, n = ts, len = 2, bar = s_full;
    if (bar == s_full && x >= 2) x -= 2, n = tu, len = NU, bar = u_full;
    wait_last(bar, x, n, len, drain);
  } else if (warp < kWarpV) {
    // ---------------------------------------------------------------- P = decayed, masked S
    if (OUT) {
      const int wq = warp & 3, i = wq * 32 + lane;
      const uint32_t t_lane = tmem + (static_cast<uint32_t>(wq * 32) << 16);
      float* pow = reinterpret_cast<float*>(smem + L::kPow) + wq * 32;
      int t = 0;
      bool ok = true;
      Item it;
      for (int k = 0; ok && take(k, it); ++k) {
        const bool rev = p.pass[it.pass].reverse != 0;
        const float l2 = it.l2;
        const int steep = l2 < -2.0f;  // see weigh
        __syncwarp();
        pow[lane] = ex2_approx(l2 * static_cast<float>(rev ? lane : 31 - lane));
        __syncwarp();
        for (int j = 0; j < it.cn; ++j, ++t) {
          const int m = valid_of(it, chunk_of(it, rev, j));
          const uint32_t sb = t_lane + L::kTS + (t & 1) * 128;
          if (!(ok = mbar_wait_w(s_full + (t & 1), (t >> 1) & 1, wctx))) break;
          tc_fence_after();
          // P of keys c0.. goes to column (c0 / 64) 64 + (c0 % 64) / 2, where S has been read
          // by then.  Blocks [b0, b1) are weighed, 16 columns while the next 16 are read.
          const int b0 = rev ? wq + steep : 0, b1 = rev ? 4 : wq + 1 - steep;
          uint32_t sa[16], se[16], pk[8];
          const auto near = [&] {
#pragma unroll 1
            for (int c0 = 0; c0 < 32; c0 += 16) {
              tmem_ld16(sb + wq * 32 + c0, sa);
              tmem_wait_ld();
              weigh_near(sa, l2, rev, c0 - lane, m - wq * 32 - c0, pk);
              tmem_st8(sb + (wq & 2) * 32 + (wq & 1) * 16 + c0 / 2, pk);
            }
          };
          if (steep && rev) near();
          if (b0 < b1) tmem_ld16(sb + b0 * 32, sa);
#pragma unroll 1
          for (int blk = b0; blk < b1; ++blk) {
            const uint32_t src = sb + blk * 32, dst = sb + (blk & 2) * 32 + (blk & 1) * 16;
            const int last = m - blk * 32;
            const bool masked = blk == wq || last < 32;
            uint32_t keep = blk != wq ? ~0u : rev ? ~0u << lane : ~0u >> (31 - lane);
            if (last < 32) keep &= last <= 0 ? 0u : (1u << last) - 1u;
            const float f =
                ex2_approx(l2 * static_cast<float>(rev ? blk * 32 - i : i - blk * 32 - 31));
            tmem_wait_ld_of(sa);
            tmem_ld16(src + 16, se);
            weigh(sa, f, pow, masked, keep, pk);
            tmem_st8(dst, pk);
            tmem_wait_ld_of(se);
            if (blk + 1 < b1) tmem_ld16(src + 32, sa);
            weigh(se, f, pow + 16, masked, keep >> 16, pk);
            tmem_st8(dst + 8, pk);
          }
          if (steep && !rev) near();
#pragma unroll
          for (int c = 0; c < 8; ++c) pk[c] = 0u;
#pragma unroll 1
          for (int blk = rev ? 0 : wq + 1; blk < (rev ? wq : 4); ++blk) {
            tmem_st8(sb + (blk & 2) * 32 + (blk & 1) * 16, pk);
            tmem_st8(sb + (blk & 2) * 32 + (blk & 1) * 16 + 8, pk);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full + (t & 1));
        }
      }
    }
  } else if (warp < (OUT ? kWarpO : kWarpS)) {
    // ---------------------------------------------------------------- V'
    // (without the outputs their warps take every other chunk)
    const int tid = (threadIdx.x - kWarpV * 32) % 128, odd = warp >= kWarpO;
    int t = 0;
    bool ok = true;
    Item it;
    for (int k = 0; ok && take(k, it); ++k) {
      const LinPass& ps = p.pass[it.pass];
      const bool rev = ps.reverse != 0;
      const float l2 = it.l2;
      for (int j = 0; j < it.cn; ++j, ++t) {
        const int m = valid_of(it, chunk_of(it, rev, j));
        if (!OUT && t % 2 != odd) continue;
        const int vs = t % VS, s = t % ST;
        if (!(ok = mbar_wait_w(v_full + vs, (t / VS) & 1, wctx))) break;
        if (m < kChunk && !(ok = mbar_wait_w(qk_full + s, (t / ST) & 1, wctx))) break;
        // 16 bytes a step, at the address they have in the swizzled tile: only its row counts
        uint8_t* v = smem + L::kV + vs * L::kBox + tid * 16;
        uint8_t* vp = smem + L::kVp + t % NU * L::kVpSize + tid * 16;
        const int row0 = tid / 8;
        if (m < kChunk) {
          // Behind the sequence: whatever these rows hold (NaN among it) must not reach the
          // products over tokens, in which 0 times it would still be NaN.
          for (int x = 0; x < 8; ++x) {
            if (row0 + x * 16 < m) continue;
            *reinterpret_cast<uint4*>(v + x * 2048) = make_uint4(0u, 0u, 0u, 0u);
            for (int y = 0; y < L::kBoxes; ++y)
              *reinterpret_cast<uint4*>(smem + L::kK + s * L::kTile + y * L::kBox + tid * 16 +
                                        x * 2048) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        if (t >= NU && !(ok = mbar_wait_w(u_full + t % NU, (t / NU - 1) & 1, wctx))) break;
#pragma unroll 1
        for (int x0 = 0; x0 < 8; x0 += 2) {
          uint4 in[2];
#pragma unroll
          for (int x = 0; x < 2; ++x)
            in[x] = *reinterpret_cast<const uint4*>(v + (x0 + x) * 2048);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int row = row0 + (x0 + x) * 16;
            const float f = ps.vs * ex2_approx(l2 * static_cast<float>(
                                                        rev ? row + 1 : max(0, m - 1 - row)));
            uint32_t hi[4], lo[4];
            const uint32_t wds[4] = {in[x].x, in[x].y, in[x].z, in[x].w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const float2 a = mul2(make_float2(__uint_as_float(wds[y] << 16),
                                                __uint_as_float(wds[y] & 0xFFFF0000u)),
                                    make_float2(f, f));
              hi[y] = pack_bf16x2(a.x, a.y);
              if constexpr (TWO) {
                const float2 b = fma2(make_float2(__uint_as_float(hi[y] << 16),
                                                  __uint_as_float(hi[y] & 0xFFFF0000u)),
                                      make_float2(-1.0f, -1.0f), a);
                lo[y] = pack_bf16x2(b.x, b.y);
              }
            }
            uint8_t* dst = vp + (x0 + x) * 2048;
            *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if constexpr (TWO)
              *reinterpret_cast<uint4*>(dst + L::kBox) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(vp_full + t % NU);
      }
    }
  } else if (warp < kWarpS) {
    // ---------------------------------------------------------------- the outputs
    if (OUT) {
      const int wq = warp & 3, i = wq * 32 + lane;
      const uint32_t t_lane = tmem + (static_cast<uint32_t>(wq * 32) << 16);
      uint8_t* box = smem + L::kO + wq * 4096;  // 32 rows of 128 swizzled bytes
      int t = 0;
      bool ok = true;
      Item it;
      for (int k = 0; ok && take(k, it); ++k) {
        const LinPass& ps = p.pass[it.pass];
        const bool rev = ps.reverse != 0;
        const float l2 = it.l2;
        for (int j = 0; j < it.cn; ++j, ++t) {
          const int c = chunk_of(it, rev, j), m = valid_of(it, c);
          const float f = ps.o1 * ex2_approx(l2 * static_cast<float>(rev ? m - 1 - i : i + 1));
          const float2 f1 = make_float2(f, f), f2 = make_float2(ps.o2, ps.o2);
          if (lane == 0) bulk_wait_read_0();  // the box's last store has read it
          __syncwarp();
          if (!(ok = mbar_wait_w(pv_done + t % VS, (t / VS) & 1, wctx))) break;
          tc_fence_after();
#pragma unroll 1
          for (int x = 0; x < 4; ++x) {
            uint32_t a[16], b[16], pk[8];
            tmem_ld16(t_lane + L::kTO1 + t % L::kNo * kCols + x * 16, a);
            tmem_ld16(t_lane + L::kTO2 + x * 16, b);
            tmem_wait_ld();
#pragma unroll
            for (int y = 0; y < 8; ++y) {
              const float2 o = fma2(
                  make_float2(__uint_as_float(a[2 * y]), __uint_as_float(a[2 * y + 1])), f1,
                  mul2(make_float2(__uint_as_float(b[2 * y]), __uint_as_float(b[2 * y + 1])),
                       f2));
              pk[y] = i < m ? pack_bf16x2(o.x, o.y) : 0u;
            }
#pragma unroll
            for (int y = 0; y < 2; ++y)
              *reinterpret_cast<uint4*>(box + lane * 128 + (((2 * x + y) ^ (lane & 7)) << 4)) =
                  make_uint4(pk[4 * y], pk[4 * y + 1], pk[4 * y + 2], pk[4 * y + 3]);
          }
          tc_fence_before();
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(o_empty + (t & 1));
          const int row = c * kChunk + wq * 32;  // of the sequence
          if (!p.cu || wq * 32 + 32 <= m) {
            // padded: rows behind the sequence are 0, rows behind the tensor not written
            if (lane == 0 && (p.cu || row < p.N)) {
              tma_store_4d(p.map + ps.o, box, it.slice * kCols, it.s.row0 + row, it.h,
                           it.s.tma_b);
              bulk_commit_group();
            }
          } else {
            // packed: the rows behind belong to the next sequence
            __nv_bfloat16* out = ps.out + (it.s.row0 + row) * ps.o_sn + it.h * ps.o_sh +
                                 it.slice * kCols;
            for (int r = lane / 8; r < 32 && wq * 32 + r < m; r += 4)
              *reinterpret_cast<uint4*>(out + r * ps.o_sn + (lane % 8) * 8) =
                  *reinterpret_cast<const uint4*>(box + r * 128 + (((lane % 8) ^ (r & 7)) << 4));
            __syncwarp();
          }
        }
      }
      if (lane == 0) bulk_wait_all();
      __syncwarp();
    }
  } else if (warp < kWarpI) {
    // ---------------------------------------------------------------- the state
    // Eight warps: d = 128, a thread holds 32 columns of one row; d = 64, 16 columns, half of
    // the warps reading the copy of the rows in lanes 64-127 of U.
    constexpr int kHold = D == 128 ? 32 : 16;
    const int wq = warp & 3, g = (warp - kWarpS) / 4;
    const int row = D == 128 ? wq * 32 + lane : (wq & 1) * 32 + lane;
    const int col0 = D == 128 ? g * 32 : g * 32 + (wq >> 1) * 16;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(wq * 32) << 16) + col0;
    float r[kHold];
    int t = 0;
    bool ok = true;
    Item it;
    for (int k = 0; ok && take(k, it); ++k) {
      const LinPass& ps = p.pass[it.pass];
      const bool rev = ps.reverse != 0;
      const int64_t bh = static_cast<int64_t>(it.b) * p.H + it.h;
      float* seg = ps.seg + ((bh * p.nseg + it.seg) * D + row) * D + it.slice * kCols + col0;
      if (!TWO && p.nseg > 1) {
        if (it.cn > 0)
#pragma unroll
          for (int c = 0; c < kHold; c += 4) {
            const float4 x = *reinterpret_cast<const float4*>(seg + c);
            r[c] = x.x, r[c + 1] = x.y, r[c + 2] = x.z, r[c + 3] = x.w;
          }
      } else if (OUT && ps.init) {
        const float* at = ps.init + bh * D * D + row * ps.init_sr +
                          static_cast<int64_t>(it.slice * kCols + col0) * ps.init_sc;
#pragma unroll
        for (int c = 0; c < kHold; ++c) r[c] = at[c * ps.init_sc];
      } else {
#pragma unroll
        for (int c = 0; c < kHold; ++c) r[c] = 0.0f;
      }
      for (int j = 0; j < it.cn; ++j, ++t) {
        const int m = valid_of(it, chunk_of(it, rev, j));
        if (OUT) {
          // the state as the B operand of Q R: row by row, 128 swizzled bytes each
          if (t > 0 && !(ok = mbar_wait_w(qk_empty + (t - 1) % ST, ((t - 1) / ST) & 1, wctx)))
            break;
          uint8_t* dst = smem + L::kR + row * 128;
#pragma unroll
          for (int c = 0; c < kHold / 8; ++c)
            *reinterpret_cast<uint4*>(dst + (((col0 / 8 + c) ^ (row & 7)) << 4)) =
                make_uint4(pack_bf16x2(r[8 * c], r[8 * c + 1]),
                           pack_bf16x2(r[8 * c + 2], r[8 * c + 3]),
                           pack_bf16x2(r[8 * c + 4], r[8 * c + 5]),
                           pack_bf16x2(r[8 * c + 6], r[8 * c + 7]));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(r_full);
        }
        if (!(ok = mbar_wait_w(u_full + t % NU, (t / NU) & 1, wctx))) break;
        tc_fence_after();
        const float f = m == kChunk ? it.full : it.part;
        const int at = t % NU == 0 ? L::kTU : L::kTS;
#pragma unroll
        for (int c = 0; c < kHold; c += 8) {
          uint32_t u[8], e[8];
          tmem_ld8(t_lane + at + c, u);
          if constexpr (TWO) tmem_ld8(t_lane + at + kCols + c, e);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 8; ++x)
            r[c + x] = fmaf(f, r[c + x],
                            TWO ? __uint_as_float(u[x]) + __uint_as_float(e[x])
                                : __uint_as_float(u[x]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(u_empty + t % NU);
      }
      if constexpr (!TWO) continue;
      float* dst = !OUT ? (it.cn > 0 ? seg : nullptr)
                   : ps.fin ? ps.fin + (bh * D + row) * D + it.slice * kCols + col0 : nullptr;
      if (ok && dst) {
#pragma unroll
        for (int c = 0; c < kHold; c += 4)
          *reinterpret_cast<float4*>(dst + c) = make_float4(r[c], r[c + 1], r[c + 2], r[c + 3]);
      }
    }
  } else if (warp == kWarpI + 1) {
    // ---------------------------------------------------------------- zero rows
    // Rows behind a padded sequence's last chunk, within the item's segment, are written as 0
    // (those inside it come out of the chunk as 0).
    if (OUT && !p.cu) {
      Item it;
      for (int k = 0; take(k, it); ++k) {
        const LinPass& ps = p.pass[it.pass];
        const int lo = max(it.c0 * kChunk, (it.s.n + kChunk - 1) / kChunk * kChunk);
        const int hi = it.seg == p.nseg - 1 ? p.N : min(p.N, (it.c0 + p.seg_chunks) * kChunk);
        __nv_bfloat16* out =
            ps.out + it.b * ps.o_sb + it.h * ps.o_sh + it.slice * kCols + lane % 8 * 8;
        for (int r = lo + lane / 8; r < hi; r += 4)
          *reinterpret_cast<uint4*>(out + r * ps.o_sn) = make_uint4(0u, 0u, 0u, 0u);
      }
    } else if (OUT) {
      // Packed rows of no sequence, where asked: before the first, from each one's end to the next
      // one's start, behind the last.  Every CTA looks through all of them, a lane for each, and
      // takes its share of rows, four at a time.  Following the items instead cost the other
      // warps issue slots by its waits (gradients of documents without such rows 393 us, so 380);
      // padded rows done this way come all at once (gradients of the padded batch 209 us, by
      // the items 87).
      int any = 0;
      for (int i = 0; i < p.npass; ++i) any |= p.pass[i].rest;
      for (int b0 = -1; any && b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        int lo = 0, hi = 0;
        if (b < 0) {
          hi = sequence(p, 0).row0;
        } else if (b < p.B) {
          const Seq s = sequence(p, b);
          lo = s.row0 + s.n;
          hi = b + 1 < p.B ? sequence(p, b + 1).row0 : p.T;
        }
        for (uint32_t left = __ballot_sync(0xFFFFFFFFu, lo < hi); left != 0u; left &= left - 1) {
          const int from = __ffs(left) - 1;
          const int end = __shfl_sync(0xFFFFFFFFu, hi, from);
          int r = __shfl_sync(0xFFFFFFFFu, lo, from) + lane / 8;
          for (r += blockIdx.x * 4; r < end; r += gridDim.x * 4)
            for (int i = 0; i < p.npass; ++i) {
              const LinPass& ps = p.pass[i];
              __nv_bfloat16* out = ps.out + r * ps.o_sn + lane % 8 * 8;
              for (int h = 0; ps.rest && h < p.H; ++h)
                for (int x = 0; x < D; x += 64)
                  *reinterpret_cast<uint4*>(out + h * ps.o_sh + x) = make_uint4(0u, 0u, 0u, 0u);
            }
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- the work items
    // 32 at a time, one per lane, and into the ring as its places get free.
    bool more = true;
    for (int k0 = 0; more; k0 += 32) {
      const int w = snake_item(k0 + lane);
      Item it{};
      it.pass = -1;
      if (w < p.nitems) {
        it = decode<D>(p, order, w);
        const float g = clamped_decay(p, it.h);
        it.l2 = g * kLog2e;
        it.full = static_cast<float>(exp(static_cast<double>(g) * kChunk));
        it.part = static_cast<float>(exp(static_cast<double>(g) * (it.s.n % kChunk)));
      }
      for (int u = 0; u < 32 && more; ++u) {
        const int k = k0 + u;
        bool go = true;
        if (lane == u) {
          if (k >= kRing) go = mbar_wait(item_empty + k % kRing, (k / kRing - 1) & 1, wctx);
          if (go) {
            items[k % kRing] = it;
            mbar_arrive(item_full + k % kRing);
          }
          go = go && it.pass >= 0;
        }
        more = __all_sync(0xFFFFFFFFu, go);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The states that the segments start from, in place of what each leaves from a zero start, and
// the final state.  Four state columns per thread; all of a thread's reads are issued before
// the first is used.
template <int D>
__global__ void __launch_bounds__(128) k_linear_join(const __grid_constant__ LinParams p) {
  __shared__ float factor[2];  // lambda to the tokens of a whole segment, of the last one
  const int e = (blockIdx.x * 128 + threadIdx.x) * 4;
  const int bh = blockIdx.y, b = bh / p.H, h = bh % p.H;
  const LinPass& ps = p.pass[blockIdx.z];
  const int n = sequence(p, b).n, rows = p.seg_chunks * kChunk;
  const int segs = (n + rows - 1) / rows;
  float* seg = ps.seg + static_cast<int64_t>(bh) * p.nseg * D * D + e;
  const auto at = [&](int x) {
    const int s = ps.reverse ? segs - 1 - x : x;
    return reinterpret_cast<float4*>(seg + static_cast<int64_t>(s) * D * D);
  };
  float4 u[kMaxSegs];
#pragma unroll
  for (int x = 0; x < kMaxSegs; ++x)
    if (x < segs) u[x] = *at(x);
  float4 r = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (ps.init) {
    const float* from = ps.init + static_cast<int64_t>(bh) * D * D + (e / D) * ps.init_sr +
                        (e % D) * ps.init_sc;
    r = make_float4(from[0], from[ps.init_sc], from[2 * ps.init_sc], from[3 * ps.init_sc]);
  }
  if (threadIdx.x < 2)
    factor[threadIdx.x] = static_cast<float>(
        exp(static_cast<double>(clamped_decay(p, h)) *
            (threadIdx.x == 0 ? rows : n - (segs - 1) * rows)));
  __syncthreads();
#pragma unroll
  for (int x = 0; x < kMaxSegs; ++x) {
    if (x >= segs) break;
    *at(x) = r;
    const float f = factor[x == (ps.reverse ? 0 : segs - 1)];
    r = make_float4(fmaf(f, r.x, u[x].x), fmaf(f, r.y, u[x].y), fmaf(f, r.z, u[x].z),
                    fmaf(f, r.w, u[x].w));
  }
  if (ps.fin) *reinterpret_cast<float4*>(ps.fin + static_cast<int64_t>(bh) * D * D + e) = r;
}

// ------------------------------------------------------------------------------------
// Single tokens: one pass over the state, read, updated, written, and contracted with q: 8 d^2
// bytes per head, 82.8 us for 256 x 16 states of 128 x 128 (99.5 % of the copy rate); one
// sequence's 16 heads take 4.2 us, a launch.
// A CTA takes 32 columns of one (b, h): 8 lanes of 16 bytes cover a row's 128 bytes, a warp
// four rows, and every load of a thread (d / 32 of them) is issued before the first is used.
// ------------------------------------------------------------------------------------
struct StepParams {
  int H;
  const int32_t* lengths;
  const float* log_decay;
  float scale;
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* o;
  int64_t q_sb, q_sh, k_sb, k_sh, v_sb, v_sh, o_sb, o_sh;
  const float* in;
  float* out;
};

template <int D>
__global__ void __launch_bounds__(256) k_linear_step(const StepParams p) {
  __shared__ float sums[8][32];
  const int bh = blockIdx.x / (D / 32), c0 = (blockIdx.x % (D / 32)) * 32;
  const int b = bh / p.H, h = bh % p.H;
  const int col = c0 + (threadIdx.x % 8) * 4, row0 = threadIdx.x / 8;
  const int64_t base = static_cast<int64_t>(bh) * D * D + col;
  float4 s[D / 32];
#pragma unroll
  for (int x = 0; x < D / 32; ++x)
    s[x] = *reinterpret_cast<const float4*>(p.in + base + (row0 + 32 * x) * D);
  const bool active = !p.lengths || __ldg(p.lengths + b) > 0;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (active) {
    const float f = expf(fminf(__ldg(p.log_decay + h), 0.0f));
    const __nv_bfloat16* v = p.v + b * p.v_sb + h * p.v_sh + col;
    const float v0 = __bfloat162float(v[0]), v1 = __bfloat162float(v[1]),
                v2 = __bfloat162float(v[2]), v3 = __bfloat162float(v[3]);
#pragma unroll
    for (int x = 0; x < D / 32; ++x) {
      const int row = row0 + 32 * x;
      const float k = __bfloat162float(p.k[b * p.k_sb + h * p.k_sh + row]);
      const float q = __bfloat162float(p.q[b * p.q_sb + h * p.q_sh + row]);
      s[x] = make_float4(fmaf(f, s[x].x, k * v0), fmaf(f, s[x].y, k * v1),
                         fmaf(f, s[x].z, k * v2), fmaf(f, s[x].w, k * v3));
      o = make_float4(fmaf(q, s[x].x, o.x), fmaf(q, s[x].y, o.y), fmaf(q, s[x].z, o.z),
                      fmaf(q, s[x].w, o.w));
    }
  }
  if (active || p.out != p.in) {
#pragma unroll
    for (int x = 0; x < D / 32; ++x)
      *reinterpret_cast<float4*>(p.out + base + (row0 + 32 * x) * D) = s[x];
  }
#pragma unroll
  for (int m = 8; m <= 16; m <<= 1) {
    o.x += __shfl_xor_sync(0xFFFFFFFFu, o.x, m);
    o.y += __shfl_xor_sync(0xFFFFFFFFu, o.y, m);
    o.z += __shfl_xor_sync(0xFFFFFFFFu, o.z, m);
    o.w += __shfl_xor_sync(0xFFFFFFFFu, o.w, m);
  }
  if (threadIdx.x % 32 < 8)
    *reinterpret_cast<float4*>(&sums[threadIdx.x / 32][(threadIdx.x % 8) * 4]) = o;
  __syncthreads();
  if (threadIdx.x < 32) {
    float a = 0.0f;
#pragma unroll
    for (int x = 0; x < 8; ++x) a += sums[x][threadIdx.x];
    p.o[b * p.o_sb + h * p.o_sh + c0 + threadIdx.x] = __float2bfloat16(active ? p.scale * a : 0.0f);
  }
}

// ------------------------------------------------------------------------------------
// Launches
// ------------------------------------------------------------------------------------
// How a sequence is cut when there are fewer (pass, batch, head, slice) items than SMs: into
// segments whose states are computed first, from their keys and values alone, and joined.
void segments(int npass, int B, int N, int H, int d, int* nseg, int* seg_chunks) {
  const int64_t items = static_cast<int64_t>(npass) * B * H * (d / kCols);
  const int chunks = (N + kChunk - 1) / kChunk;
  int want = items >= kSms ? 1 : static_cast<int>(kSms / items);
  want = std::max(1, std::min({want, chunks / 4, kMaxSegs}));
  *seg_chunks = (chunks + want - 1) / want;
  *nseg = (chunks + *seg_chunks - 1) / *seg_chunks;
}

template <int D, bool OUT, bool TWO>
int launch_one(const LinParams& p, cudaStream_t stream) {
  using L = LinLayout<D, OUT, TWO>;
  static_assert(L::kAlloc <= 227 * 1024, "shared memory");
  auto kern = linear_kernel<D, OUT, TWO>;
  static std::atomic<unsigned long long> opted{0};
  const int rc = opt_in_shared(kern, L::kAlloc, &opted);
  if (rc != SIGATTN_OK) return rc;
  kern<<<std::min(p.nitems, kSms), kThreads, L::kAlloc, stream>>>(p);
  return cuda_status(cudaGetLastError());
}

template <int D>
int launch(const LinParams& p, cudaStream_t stream) {
  if (p.nseg > 1) {
    int rc = launch_one<D, false, true>(p, stream);
    if (rc != SIGATTN_OK) return rc;
    k_linear_join<D><<<dim3(D * D / 512, p.B * p.H, p.npass), 128, 0, stream>>>(p);
    if ((rc = cuda_status(cudaGetLastError())) != SIGATTN_OK) return rc;
  }
  bool two = false;
  for (int i = 0; i < p.npass; ++i) two = two || (p.nseg == 1 && p.pass[i].fin);
  return two ? launch_one<D, true, true>(p, stream) : launch_one<D, true, false>(p, stream);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Whether two state arrays of n floats share memory (absent ones share none).
bool overlap(const float* a, const float* b, int64_t n) {
  const intptr_t x = reinterpret_cast<intptr_t>(a), y = reinterpret_cast<intptr_t>(b);
  return a && b && std::abs(x - y) < n * static_cast<int64_t>(sizeof(float));
}

// Whether an output is the very tensor that one of the others is: what reads them is not done
// when the first output is written (two items share the rows of q and k, passes the inputs).
bool same_as_any(const void* out, std::initializer_list<const void*> others) {
  return std::find(others.begin(), others.end(), out) != others.end();
}

int check_tensor(const void* ptr, const int64_t* strides, int rows, TensorDesc* t) {
  if (!ptr || !strides) return SIGATTN_ERR_INVALID;
  for (int i = 0; i < 3; ++i)
    if (strides[i] < 0) return SIGATTN_ERR_INVALID;
  if (!aligned16(ptr)) return SIGATTN_ERR_ALIGNMENT;
  for (int i = 0; i < 3; ++i)
    if (strides[i] % 8 != 0) return SIGATTN_ERR_ALIGNMENT;
  *t = TensorDesc{ptr, strides[0], strides[1], strides[2], rows};
  return SIGATTN_OK;
}

int check_sizes(int B, int N, int64_t T, int H, int d, bool packed) {
  if (B < 1 || N < 1 || H < 1 || (packed && T < 1)) return SIGATTN_ERR_INVALID;
  if (d != 64 && d != 128) return SIGATTN_ERR_UNSUPPORTED;
  // row indices, item counts (six items per batch, head and segment at most, fewer than
  // 148 segments where items are few) and the join's grid stay below their limits
  if (N > 0x7FFFFF00 || (packed && T > 0x7FFFFF00)) return SIGATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(B) * H > 0x0FFFFFFF) return SIGATTN_ERR_UNSUPPORTED;
  return SIGATTN_OK;
}

// Fills what the passes share; the tensor maps are those of t[0..n).
int fill(LinParams* p, int npass, int B, int N, int64_t T, int H, int d, const int32_t* lengths,
         const int32_t* cu, const float* log_decay, const TensorDesc* t, int n,
         const TensorDesc* out) {
  int rc;
  if ((rc = status_ptr(&p->status)) != SIGATTN_OK) return rc;
  for (int i = 0; i < n; ++i)
    if ((rc = make_tmap_bf16(&p->map[i], t[i], cu ? 1 : B, H, d)) != SIGATTN_OK) return rc;
  for (int i = 0; i < npass; ++i) {
    if ((rc = make_tmap_bf16(&p->map[n + i], out[i], cu ? 1 : B, H, d, 32)) != SIGATTN_OK)
      return rc;
    LinPass& ps = p->pass[i];
    ps.o = n + i;
    ps.out = static_cast<__nv_bfloat16*>(const_cast<void*>(out[i].ptr));
    ps.o_sb = out[i].sb;
    ps.o_sn = out[i].sn;
    ps.o_sh = out[i].sh;
  }
  p->npass = npass;
  p->B = B;
  p->H = H;
  p->N = N;
  p->T = static_cast<int>(T);
  segments(npass, B, N, H, d, &p->nseg, &p->seg_chunks);
  p->nitems = npass * B * p->nseg * H * (d / kCols);
  p->lengths = lengths;
  p->cu = cu;
  p->log_decay = log_decay;
  p->wait_ns = wait_limit_ns();
  return SIGATTN_OK;
}

size_t workspace_bytes_of(int npass, int B, int N, int H, int d) {
  int nseg, seg_chunks;
  segments(npass, B, N, H, d, &nseg, &seg_chunks);
  return nseg == 1 ? 0 : sizeof(float) * npass * B * H * nseg * d * d;
}

}  // namespace
}  // namespace sigattn

using namespace sigattn;

extern "C" int sigattn_linear_workspace_size(int B, int N, int H, int d, int backward,
                                             size_t* bytes) {
  if (!bytes || (backward != 0 && backward != 1)) return SIGATTN_ERR_INVALID;
  const int rc = check_sizes(B, N, 1, H, d, false);
  if (rc != SIGATTN_OK) return rc;
  *bytes = workspace_bytes_of(backward ? 3 : 1, B, N, H, d);
  return SIGATTN_OK;
}

extern "C" int sigattn_linear_fwd(int B, int N, int64_t T, int H, int d, const int32_t* lengths,
                                  const int32_t* cu_seqlens, const float* log_decay, float scale,
                                  const void* q, const int64_t q_strides[3], const void* k,
                                  const int64_t k_strides[3], const void* v,
                                  const int64_t v_strides[3], const float* state, void* o,
                                  const int64_t o_strides[3], float* final_state, void* workspace,
                                  size_t workspace_bytes, sigattn_stream s) {
  return sigattn_linear_fwd_ex(B, N, T, H, d, lengths, cu_seqlens, log_decay, scale, q, q_strides, k,
                               k_strides, v, v_strides, state, o, o_strides, final_state, 0,
                               workspace, workspace_bytes, s);
}

extern "C" int sigattn_linear_fwd_ex(int B, int N, int64_t T, int H, int d, const int32_t* lengths,
                                     const int32_t* cu_seqlens, const float* log_decay,
                                     float scale, const void* q, const int64_t q_strides[3],
                                     const void* k, const int64_t k_strides[3], const void* v,
                                     const int64_t v_strides[3], const float* state, void* o,
                                     const int64_t o_strides[3], float* final_state, int zero_rest,
                                     void* workspace, size_t workspace_bytes, sigattn_stream s) {
  const bool packed = cu_seqlens != nullptr;
  int rc = check_sizes(B, N, T, H, d, packed);
  if (rc != SIGATTN_OK) return rc;
  if (zero_rest & ~1) return SIGATTN_ERR_INVALID;
  if (!log_decay || !std::isfinite(scale) || (packed && lengths)) return SIGATTN_ERR_INVALID;
  const int rows = packed ? static_cast<int>(T) : N;
  TensorDesc t[3], to;
  if ((rc = check_tensor(q, q_strides, rows, &t[0])) != SIGATTN_OK) return rc;
  if ((rc = check_tensor(k, k_strides, rows, &t[1])) != SIGATTN_OK) return rc;
  if ((rc = check_tensor(v, v_strides, rows, &t[2])) != SIGATTN_OK) return rc;
  if ((rc = check_tensor(o, o_strides, rows, &to)) != SIGATTN_OK) return rc;
  const size_t need = workspace_bytes_of(1, B, N, H, d);
  if (need && (!workspace || workspace_bytes < need)) return SIGATTN_ERR_INVALID;
  if (!aligned16(state) || !aligned16(final_state) || !aligned16(workspace))
    return SIGATTN_ERR_ALIGNMENT;
  // in place is fine: what writes an element of the state has read it before
  if (state != final_state && overlap(state, final_state, static_cast<int64_t>(B) * H * d * d))
    return SIGATTN_ERR_INVALID;
  if (same_as_any(o, {q, k, v})) return SIGATTN_ERR_INVALID;
  LinParams p;
  std::memset(&p, 0, sizeof(p));
  if ((rc = fill(&p, 1, B, N, T, H, d, lengths, cu_seqlens, log_decay, t, 3, &to)) !=
      SIGATTN_OK)
    return rc;
  LinPass& ps = p.pass[0];
  ps.q = 0, ps.k = 1, ps.v = 2;
  ps.o1 = ps.o2 = scale;
  ps.vs = 1.0f;
  ps.init = state;
  ps.init_sr = d;
  ps.init_sc = 1;
  ps.fin = final_state;
  ps.seg = static_cast<float*>(workspace);
  ps.rest = zero_rest;
  const cudaStream_t stream = static_cast<cudaStream_t>(s);
  return d == 64 ? launch<64>(p, stream) : launch<128>(p, stream);
}

extern "C" int sigattn_linear_bwd(int B, int N, int64_t T, int H, int d, const int32_t* lengths,
                                  const int32_t* cu_seqlens, const float* log_decay, float scale,
                                  const void* q, const int64_t q_strides[3], const void* k,
                                  const int64_t k_strides[3], const void* v,
                                  const int64_t v_strides[3], const void* dout,
                                  const int64_t do_strides[3], const float* state,
                                  const float* dfinal_state, void* dq, const int64_t dq_strides[3],
                                  void* dk, const int64_t dk_strides[3], void* dv,
                                  const int64_t dv_strides[3], float* dstate, void* workspace,
                                  size_t workspace_bytes, sigattn_stream s) {
  return sigattn_linear_bwd_ex(B, N, T, H, d, lengths, cu_seqlens, log_decay, scale, q, q_strides, k,
                               k_strides, v, v_strides, dout, do_strides, state, dfinal_state, dq,
                               dq_strides, dk, dk_strides, dv, dv_strides, dstate, 0, workspace,
                               workspace_bytes, s);
}

extern "C" int sigattn_linear_bwd_ex(int B, int N, int64_t T, int H, int d, const int32_t* lengths,
                                     const int32_t* cu_seqlens, const float* log_decay,
                                     float scale, const void* q, const int64_t q_strides[3],
                                     const void* k, const int64_t k_strides[3], const void* v,
                                     const int64_t v_strides[3], const void* dout,
                                     const int64_t do_strides[3], const float* state,
                                     const float* dfinal_state, void* dq,
                                     const int64_t dq_strides[3], void* dk,
                                     const int64_t dk_strides[3], void* dv,
                                     const int64_t dv_strides[3], float* dstate, int zero_rest,
                                     void* workspace, size_t workspace_bytes, sigattn_stream s) {
  const bool packed = cu_seqlens != nullptr;
  int rc = check_sizes(B, N, T, H, d, packed);
  if (rc != SIGATTN_OK) return rc;
  if (zero_rest & ~7) return SIGATTN_ERR_INVALID;
  if (!log_decay || !std::isfinite(scale) || (packed && lengths)) return SIGATTN_ERR_INVALID;
  const int rows = packed ? static_cast<int>(T) : N;
  TensorDesc t[4], out[3];
  if ((rc = check_tensor(q, q_strides, rows, &t[0])) != SIGATTN_OK) return rc;
  if ((rc = check_tensor(k, k_strides, rows, &t[1])) != SIGATTN_OK) return rc;
  if ((rc = check_tensor(v, v_strides, rows, &t[2])) != SIGATTN_OK) return rc;
  if ((rc = check_tensor(dout, do_strides, rows, &t[3])) != SIGATTN_OK) return rc;
  if ((rc = check_tensor(dq, dq_strides, rows, &out[0])) != SIGATTN_OK) return rc;
  if ((rc = check_tensor(dk, dk_strides, rows, &out[1])) != SIGATTN_OK) return rc;
  if ((rc = check_tensor(dv, dv_strides, rows, &out[2])) != SIGATTN_OK) return rc;
  const size_t need = workspace_bytes_of(3, B, N, H, d);
  if (need && (!workspace || workspace_bytes < need)) return SIGATTN_ERR_INVALID;
  if (!aligned16(state) || !aligned16(dfinal_state) || !aligned16(dstate) || !aligned16(workspace))
    return SIGATTN_ERR_ALIGNMENT;
  // the other passes read them while this one is written
  const int64_t n = static_cast<int64_t>(B) * H * d * d;
  if (overlap(dstate, state, n) || overlap(dstate, dfinal_state, n)) return SIGATTN_ERR_INVALID;
  if (same_as_any(dq, {q, k, v, dout, dk, dv}) || same_as_any(dk, {q, k, v, dout, dv}) ||
      same_as_any(dv, {q, k, v, dout}))
    return SIGATTN_ERR_INVALID;
  LinParams p;
  std::memset(&p, 0, sizeof(p));
  if ((rc = fill(&p, 3, B, N, T, H, d, lengths, cu_seqlens, log_decay, t, 4, out)) !=
      SIGATTN_OK)
    return rc;
  const size_t part = need / 3 / sizeof(float);
  for (int i = 0; i < 3; ++i) {
    p.pass[i].seg = workspace ? static_cast<float*>(workspace) + i * part : nullptr;
    p.pass[i].rest = zero_rest >> i & 1;
  }
  // dq_t = scale S_t do_t: the forward's direction over (dO, V, K), state transposed
  LinPass& a = p.pass[0];
  a.q = 3, a.k = 2, a.v = 1;
  a.o1 = a.o2 = scale;
  a.vs = 1.0f;
  a.init = state;
  a.init_sr = 1;
  a.init_sc = d;
  // dk_t = dS_t v_t: reversed over (V, dO, Q), state dS^T
  LinPass& b = p.pass[1];
  b.q = 2, b.k = 3, b.v = 0;
  b.reverse = 1;
  b.o1 = 1.0f;
  b.o2 = b.vs = scale;
  b.init = dfinal_state;
  b.init_sr = 1;
  b.init_sc = d;
  // dv_t = dS_t^T k_t: reversed over (K, Q, dO), state dS
  LinPass& c = p.pass[2];
  c.q = 1, c.k = 0, c.v = 3;
  c.reverse = 1;
  c.o1 = 1.0f;
  c.o2 = c.vs = scale;
  c.init = dfinal_state;
  c.init_sr = d;
  c.init_sc = 1;
  c.fin = dstate;
  const cudaStream_t stream = static_cast<cudaStream_t>(s);
  return d == 64 ? launch<64>(p, stream) : launch<128>(p, stream);
}

extern "C" int sigattn_linear_step(int B, int H, int d, const int32_t* lengths,
                                   const float* log_decay, float scale, const void* q,
                                   const int64_t q_strides[2], const void* k,
                                   const int64_t k_strides[2], const void* v,
                                   const int64_t v_strides[2], const float* state,
                                   float* state_out, void* o, const int64_t o_strides[2],
                                   sigattn_stream s) {
  if (B < 1 || H < 1 || !log_decay || !std::isfinite(scale)) return SIGATTN_ERR_INVALID;
  if (!q || !k || !v || !o || !state || !state_out) return SIGATTN_ERR_INVALID;
  if (!q_strides || !k_strides || !v_strides || !o_strides) return SIGATTN_ERR_INVALID;
  for (int i = 0; i < 2; ++i)
    if (q_strides[i] < 0 || k_strides[i] < 0 || v_strides[i] < 0 || o_strides[i] < 0)
      return SIGATTN_ERR_INVALID;
  if (d != 64 && d != 128) return SIGATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(B) * H * (d / 32) > 0x7FFFFFFF) return SIGATTN_ERR_UNSUPPORTED;
  if (!aligned16(state) || !aligned16(state_out)) return SIGATTN_ERR_ALIGNMENT;
  if (state != state_out && overlap(state, state_out, static_cast<int64_t>(B) * H * d * d))
    return SIGATTN_ERR_INVALID;
  if (same_as_any(o, {q, k, v})) return SIGATTN_ERR_INVALID;
  const auto bf = [](const void* x) { return static_cast<const __nv_bfloat16*>(x); };
  StepParams p{H,
               lengths,
               log_decay,
               scale,
               bf(q),
               bf(k),
               bf(v),
               static_cast<__nv_bfloat16*>(o),
               q_strides[0],
               q_strides[1],
               k_strides[0],
               k_strides[1],
               v_strides[0],
               v_strides[1],
               o_strides[0],
               o_strides[1],
               state,
               state_out};
  const unsigned grid = static_cast<unsigned>(B) * H * (d / 32);
  const cudaStream_t stream = static_cast<cudaStream_t>(s);
  if (d == 64)
    k_linear_step<64><<<grid, 256, 0, stream>>>(p);
  else
    k_linear_step<128><<<grid, 256, 0, stream>>>(p);
  return cuda_status(cudaGetLastError());
}
