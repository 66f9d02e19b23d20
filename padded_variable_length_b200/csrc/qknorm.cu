// Norm of each query and key head with the position rotation in the same pass, forward and
// backward (sigattn_qk_norm_rope, sigattn_qk_norm_rope_bwd).
//
// One valid row x of d values (a token's head), weight w:
//   r = 1 / sqrt(mean(x^2) + eps),  u = r x,  z = w u,  y = R z
// R turns pair p of the first rot_dim values by the angle position * inv_freq[p]; the other
// values pass.  Backward, from g = R^T dy:
//   dw = sum over rows of g u,   h = w g,   dx = r (h - u mean(h u))
// Nothing is kept from the forward: r is recomputed from x, which the backward reads anyway.
//
// Layout of the work: d / 16 lanes share a row and each lane holds the two 8-value pieces
// whose pairs it turns (halves: pieces c and c + rot_dim/16; side by side: any two), so that
// the rotation needs no exchange between lanes and the norm two or three shuffles.  A warp
// takes one token of q or of k at a time and walks its heads, 512 / d of them per step.  The
// lanes of a step's rows compute the sines and cosines of a token together, one or two pairs
// each, and exchange them: they serve every head.
//
// What bounds it is the memory, 4 bytes an element forward and 6 backward, if enough loads are
// in flight and few enough instructions are issued: each lane keeps the pieces of its next
// kDepth - 1 steps on their way into shared memory slots of its own (cp.async; nobody else
// reads them, so a step waits for its own copies alone), and arithmetic is done on pairs.
// Measured (20 calls in a row, 1965 MHz): 16 + 16 heads of 128 at 32768 tokens, backward, 138 us
// (5.8 TB/s, 89 % of the copy rate; 155 us once the power cap holds the clock at 1717 MHz; with
// plain loads one step ahead at most 303); 8 + 8 heads of 64 on a padded batch of 32 x 2048 with
// 23676 valid rows, forward without rotation, 35 us (5.2 TB/s, 79 %: 18.6 for these rows packed,
// as long as torch.neg over them, and the rest for the zero rows); 64 single tokens 4.3 us, a
// launch.
//
// Angles: with inv_freq / 2 pi kept as a 64-bit fraction F of a turn, position * F modulo
// 2^64 is the angle modulo one turn.  F is taken from a product in twice double's bits, so it is
// off by 2^-63 of a turn at most and the angle of any int32 position by 2^-32, which is where
// the sines take it: far positions are as exact as near ones (a 32-bit product is off by 1e-2
// radians at 2e5; a double's, rounded, by 5e-7 inv_freq at the ends of int32).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "sm100.cuh"

namespace sigattn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxAxes = 4;
// a warp's token index steps past the last one by at most the grid's warps (148 * 3 * 8)
constexpr int64_t kMaxTokens = 0x7FFFFFFF - 16384;
constexpr int kDepth = 4;         // slots of a warp: kDepth - 1 steps' loads are in flight
enum Turn { kNone, kHalves, kPairs };  // rotation: none, halves, pairs side by side
constexpr int kSms = 148;         // B200
// Resident blocks.  Three pay where a token is one step without angles (single-cell batch,
// 35.4 us against 37.0); else what every warp does before its first step weighs more (image
// patches: 38.3 against 34.6), and the backward needs the registers.
constexpr int per_sm(bool grad, bool turns) { return !grad && !turns ? 3 : 2; }
constexpr int kGradBlocks = kSms * per_sm(true, true);  // most blocks of a backward

struct QkTensor {
  const uint4* x;
  const uint4* dy;  // backward only
  uint4* y;         // forward: y; backward: dx
  // strides in 8-value pieces; a head's is below 2^31 / H, so that offsets within a token
  // are 32-bit numbers
  int64_t x_sb, x_sn, dy_sb, dy_sn, y_sb, y_sn;
  int x_sh, dy_sh, y_sh;
  const float* w;
  int H;
};

struct QkParams {
  QkTensor t[2];  // queries, keys (H = 0: absent)
  int N, d;
  int tokens;  // B N
  const int32_t* lengths;
  float eps, inv_d;
  int norm;
  int rot_dim, interleaved, axes;
  int axis_end[kMaxAxes];  // pair p belongs to the first axis a with p < axis_end[a]
  const double* inv_freq;
  const int32_t* pos;
  int64_t pos_sa, pos_sb;
  int blocks0;     // blocks [0, blocks0) take the queries, the others the keys
  float* partial;  // backward: [gridDim.x][d] sums of g u, nullptr without weights
};

// Values travel as pairs of neighbours: the packed fp32 instructions take one issue slot for
// two, and issue slots are what these kernels run out of before the memory does.
__device__ __forceinline__ void unpack8(const uint4& v, float2* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

__device__ __forceinline__ uint4 pack8(const float2* f) {
  return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y),
                    pack_bf16x2(f[2].x, f[2].y), pack_bf16x2(f[3].x, f[3].y));
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// cos and sin of 2 pi turns / 2^32.  The nearest quarter turn is taken off in integers, which
// leaves an angle of at most pi / 4 for the Taylor polynomials of degree 9 and 8 (remainders
// below 2e-9 and 3e-8), and decides which of the two is which, and their signs.
__device__ __forceinline__ void cos_sin(uint32_t turns, float* c, float* s) {
  const uint32_t quarter = (turns + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int32_t>(turns - (quarter << 30))) *
                  (6.283185307179586f * 0x1p-32f);
  const float q = x * x;
  float a = fmaf(q, 1.0f / 362880.0f, -1.0f / 5040.0f);
  a = fmaf(q, a, 1.0f / 120.0f);
  a = fmaf(q, a, -1.0f / 6.0f);
  const float sn = fmaf(x * q, a, x);
  float b = fmaf(q, 1.0f / 40320.0f, -1.0f / 720.0f);
  b = fmaf(q, b, 1.0f / 24.0f);
  b = fmaf(q, b, -0.5f);
  const float cs = fmaf(q, b, 1.0f);
  const float c0 = quarter & 1 ? sn : cs, s0 = quarter & 1 ? cs : sn;
  *c = quarter == 1 || quarter == 2 ? -c0 : c0;
  *s = quarter & 2 ? -s0 : s0;
}

// What a lane knows of its place in a row: its two pieces and the pairs that they form.
template <int D, int TURN>
struct Lane {
  static constexpr int kLanes = D / 16;      // lanes of a row
  static constexpr int kRows = 32 / kLanes;  // rows of a warp's step
  static constexpr int kOwn = 8 / kRows;     // pairs of the lane's eight that it computes
  int c0, c1;           // pieces
  int sub;              // row of the step
  bool turn0, turn1;    // whether the pieces' pairs turn
  uint64_t frac[kOwn];  // turns per position of the pairs it computes, in 2^-64
  int axis[kOwn];       // their axes
  // The token's rotation.  Halves: cosines, sines and negated sines of pairs 2x, 2x + 1.
  // Side by side: (cos, cos) and (-sin, sin) of pair x.
  float2 cs[TURN == kPairs ? 8 : 4], sn[TURN == kPairs ? 8 : 4], ms[4];

  __device__ Lane(const QkParams& p) {
    const int l = threadIdx.x % 32 % kLanes;
    sub = threadIdx.x % 32 / kLanes;
    const int r = p.rot_dim / 16;  // turned pieces of a half
    // (halves: behind the 2 r turned pieces the rest follow, so that neighbouring lanes hold
    // neighbouring pieces and 32-byte sectors are moved whole)
    c0 = TURN != kHalves || l < r ? l : l + r;
    c1 = TURN == kHalves && l < r ? l + r : l + kLanes;
    turn0 = TURN == kPairs ? 8 * c0 < p.rot_dim : l < r;
    turn1 = TURN == kPairs ? 8 * c1 < p.rot_dim : l < r;
    if constexpr (TURN != kNone) {
#pragma unroll
      for (int x = 0; x < kOwn; ++x) {
        const int i = sub * kOwn + x;  // of the lane's eight pairs
        const int pair = TURN == kHalves ? 8 * l + i : i < 4 ? 4 * c0 + i : 4 * c1 + i - 4;
        frac[x] = 0;
        axis[x] = 0;
        if (i < 4 ? turn0 : turn1) {
          // inv_freq / 2 pi as a sum of two doubles f + e (1 / 2 pi is one too), each without
          // its whole turns; scaling by 2^64 is exact
          const double v = p.inv_freq[pair], one = 0.15915494309189535, rest = -9.839338337591243e-18;
          double f = v * one, e = fma(v, rest, fma(v, one, -f));
          f -= floor(f);
          e -= rint(e);
          if (f < 1.0)  // (not of an infinity or a NaN)
            frac[x] = static_cast<uint64_t>(f * 18446744073709551616.0) +
                      static_cast<uint64_t>(__double2ll_rn(e * 18446744073709551616.0));
          while (axis[x] + 1 < p.axes && pair >= p.axis_end[axis[x]]) ++axis[x];
        }
      }
    }
  }

  // Takes the token's positions pos[axis]; way -1 turns back.
  __device__ __forceinline__ void place(const int32_t* pos, float way) {
    float c[kOwn], s[kOwn];
#pragma unroll
    for (int x = 0; x < kOwn; ++x) {
      const uint64_t turns = frac[x] * static_cast<uint64_t>(static_cast<int64_t>(pos[axis[x]]));
      cos_sin(static_cast<uint32_t>(turns >> 32), &c[x], &s[x]);
      s[x] *= way;
    }
    const int l = threadIdx.x % 32 % kLanes;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float cj = __shfl_sync(0xFFFFFFFFu, c[j % kOwn], j / kOwn * kLanes + l);
      const float sj = __shfl_sync(0xFFFFFFFFu, s[j % kOwn], j / kOwn * kLanes + l);
      if constexpr (TURN == kPairs) {
        cs[j] = both(cj);
        sn[j] = make_float2(-sj, sj);
      } else if (j % 2 == 0) {
        cs[j / 2].x = cj;
        sn[j / 2].x = sj;
        ms[j / 2].x = -sj;
      } else {
        cs[j / 2].y = cj;
        sn[j / 2].y = sj;
        ms[j / 2].y = -sj;
      }
    }
  }

  // z <- R z on the lane's two pieces z[0..3], z[4..7] (pairs of neighbours).  Values outside
  // the rotation pass untouched: a product with a sine of 0 would spread their infinities.
  __device__ __forceinline__ void turn(float2* z) const {
    if constexpr (TURN == kPairs) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (x == 0 ? turn0 : turn1)
#pragma unroll
          for (int j = 4 * x; j < 4 * x + 4; ++j)
            z[j] = fma2(z[j], cs[j], mul2(make_float2(z[j].y, z[j].x), sn[j]));
    } else if constexpr (TURN == kHalves) {
      if (turn0)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 a = z[j], b = z[j + 4];
          z[j] = fma2(a, cs[j], mul2(b, ms[j]));
          z[j + 4] = fma2(b, cs[j], mul2(a, sn[j]));
        }
    }
  }

  // sum over the lanes of a row
  __device__ __forceinline__ static float row_sum(float2 v2) {
    float v = v2.x + v2.y;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
  }
};

__device__ __forceinline__ void copy16(void* dst, const uint4* src, bool have) {
  // without a source 16 zero bytes are written
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src), "r"(have ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy4(void* dst, const int32_t* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}

// One step of a warp: its slot in shared memory.  piece[x][lane]: the lane's two pieces of x,
// and of dy in the backward.
template <int PIECES>
struct Slot {
  uint4 piece[PIECES][32];
  int32_t pos[kMaxAxes];
};

// A warp's walk over the steps of its tokens: every stride-th token, its heads kRows at a
// time.  (b, i) move by the stride's whole batch entries and rows, without divisions.
struct Walk {
  int tok, h, b, i;
  bool valid;
  __device__ __forceinline__ void enter(const QkParams& p) {
    valid = tok < p.tokens && (!p.lengths || i < __ldg(p.lengths + b));
  }
  __device__ __forceinline__ void next(const QkParams& p, int H, int rows, int stride,
                                       int stride_b, int stride_i) {
    h += rows;
    if (h >= H) {
      h = 0;
      tok += stride;
      b += stride_b;
      i += stride_i;
      if (i >= p.N) {
        i -= p.N;
        ++b;
      }
      enter(p);
    }
  }
  // offset of the token in a tensor with these strides, in pieces
  __device__ __forceinline__ int64_t token(int64_t sb, int64_t sn) const {
    return b * sb + i * sn;
  }
};

// Forward (GRAD false) and backward.  In the backward y takes the gradient of x.
template <int D, int TURN, bool GRAD>
__global__ void __launch_bounds__(kThreads, per_sm(GRAD, TURN != kNone)) k_qk(const QkParams p) {
  using L = Lane<D, TURN>;
  constexpr int kPieces = GRAD ? 4 : 2;
  extern __shared__ uint4 smem[];
  const int warp = threadIdx.x / 32, ln = threadIdx.x % 32;
  Slot<kPieces>* slots = reinterpret_cast<Slot<kPieces>*>(smem) + warp * kDepth;
  const bool keys = static_cast<int>(blockIdx.x) >= p.blocks0;
  const QkTensor& t = p.t[keys];
  const int block = keys ? blockIdx.x - p.blocks0 : blockIdx.x;
  const int stride = (keys ? gridDim.x - p.blocks0 : p.blocks0) * kWarps;
  const int stride_b = stride / p.N, stride_i = stride % p.N;
  L lane(p);

  const int first = block * kWarps + warp;
  Walk ahead{first, 0, first / p.N, first % p.N, false};
  ahead.enter(p);
  Walk at = ahead;
  // the tokens' places in x and dy (ahead) and in y (at), the lane's row in a step
  int64_t x_at = ahead.token(t.x_sb, t.x_sn), y_at = ahead.token(t.y_sb, t.y_sn);
  int64_t g_at = GRAD ? ahead.token(t.dy_sb, t.dy_sn) : 0;
  auto fetch = [&](Slot<kPieces>& s) {
    if (ahead.tok < p.tokens) {
      if (ahead.valid) {
        const int h = ahead.h + lane.sub;
        const bool have = h < t.H;
        const uint4* x = t.x + x_at + (have ? h : 0) * t.x_sh;
        copy16(&s.piece[0][ln], x + lane.c0, have);
        copy16(&s.piece[1][ln], x + lane.c1, have);
        if constexpr (GRAD) {
          const uint4* g = t.dy + g_at + (have ? h : 0) * t.dy_sh;
          copy16(&s.piece[2][ln], g + lane.c0, have);
          copy16(&s.piece[3][ln], g + lane.c1, have);
        }
        if (TURN != kNone && ahead.h == 0 && ln < p.axes)
          copy4(&s.pos[ln], p.pos + ln * p.pos_sa + ahead.b * p.pos_sb + ahead.i);
      }
      ahead.next(p, t.H, L::kRows, stride, stride_b, stride_i);
      if (ahead.h == 0) {
        x_at = ahead.token(t.x_sb, t.x_sn);
        if (GRAD) g_at = ahead.token(t.dy_sb, t.dy_sn);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < kDepth - 1; ++s) fetch(slots[s]);

  float2 w[8], dw[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float* at_w = t.w + (j < 4 ? lane.c0 : lane.c1) * 8 + 2 * (j & 3);
    w[j] = t.w ? make_float2(__ldg(at_w), __ldg(at_w + 1)) : both(1.0f);
    dw[j] = both(0.0f);
  }

  for (int n = 0; at.tok < p.tokens; n = n + 1 == kDepth ? 0 : n + 1) {
    Slot<kPieces>& s = slots[n];
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
    const int h = at.h + lane.sub;
    const bool have = h < t.H;
    uint4* y = t.y + y_at + (have ? h : 0) * t.y_sh;
    uint4 out0 = make_uint4(0u, 0u, 0u, 0u), out1 = out0;
    if (at.valid) {
      if (TURN != kNone && at.h == 0) {
        __syncwarp();  // the positions were copied by other lanes
        lane.place(s.pos, GRAD ? -1.0f : 1.0f);
      }
      float2 z[8];
      unpack8(s.piece[0][ln], z);
      unpack8(s.piece[1][ln], z + 4);
      float r = 1.0f;
      if (p.norm) {
        float2 sum = mul2(z[0], z[0]);
#pragma unroll
        for (int j = 1; j < 8; ++j) sum = fma2(z[j], z[j], sum);
        r = rsqrtf(fmaf(L::row_sum(sum), p.inv_d, p.eps));
      }
      if constexpr (!GRAD) {
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = mul2(mul2(z[j], both(r)), w[j]);
        lane.turn(z);
        out0 = pack8(z);
        out1 = pack8(z + 4);
      } else {
        float2 g[8];
        unpack8(s.piece[2][ln], g);
        unpack8(s.piece[3][ln], g + 4);
        lane.turn(g);
        // a lane without a row has u = g = 0 and, with r = 0 (not rsqrt(eps)), adds nothing
        if (!have) r = 0.0f;
        float2 dot = both(0.0f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          z[j] = mul2(z[j], both(r));
          dw[j] = fma2(g[j], z[j], dw[j]);
          g[j] = mul2(g[j], w[j]);
          dot = fma2(g[j], z[j], dot);
        }
        const float mean = p.norm ? -L::row_sum(dot) * p.inv_d : 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = mul2(fma2(z[j], both(mean), g[j]), both(r));
        out0 = pack8(g);
        out1 = pack8(g + 4);
      }
    }
    if (have) {
      y[lane.c0] = out0;
      y[lane.c1] = out1;
    }
    at.next(p, t.H, L::kRows, stride, stride_b, stride_i);
    if (at.h == 0) y_at = at.token(t.y_sb, t.y_sn);
    if (TURN != kNone) __syncwarp();  // every lane has read the positions of the next slot
    fetch(slots[n == 0 ? kDepth - 1 : n - 1]);
  }
  if (!GRAD || !p.partial) return;
  // The block's sums, in a fixed order: the rows of each warp by shuffles, the warps one
  // after another from shared memory.
  __shared__ float sums[kWarps][D];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float v = j % 2 ? dw[j / 2].y : dw[j / 2].x;
#pragma unroll
    for (int o = 16; o >= L::kLanes; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (lane.sub == 0) sums[warp][(j < 8 ? lane.c0 : lane.c1) * 8 + (j & 7)] = v;
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float v = 0.0f;
#pragma unroll
    for (int x = 0; x < kWarps; ++x) v += sums[x][threadIdx.x];
    p.partial[blockIdx.x * D + threadIdx.x] = v;
  }
}

// dwq, dwk from the blocks' partial sums [rows][d], the first rows0 of them of the queries:
// one block per 32 columns of one of the two, its warps take the rows in turn (coalesced
// 128-byte reads) and are added in a fixed order.
__global__ void __launch_bounds__(1024) k_qk_dw(const float* __restrict__ partial, int rows0,
                                                int rows, int d, float* __restrict__ dwq,
                                                float* __restrict__ dwk) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const bool keys = static_cast<int>(blockIdx.x) >= d / 32;
  const int c0 = (blockIdx.x % (d / 32)) * 32;
  float* out = keys ? dwk : dwq;
  if (!out) return;
  constexpr int kMost = (kGradBlocks + 1 + 31) / 32;  // rows of a warp, all read at once
  const int end = keys ? rows : rows0;
  float in[kMost], v = 0.0f;
#pragma unroll
  for (int x = 0; x < kMost; ++x) {
    const int r = (keys ? rows0 : 0) + warp + 32 * x;
    in[x] = r < end ? partial[r * d + c0 + lane] : 0.0f;
  }
#pragma unroll
  for (int x = 0; x < kMost; ++x) v += in[x];
  sums[warp][lane] = v;
  __syncthreads();
  v = sums[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (lane == 0) out[c0 + warp] = v;
}

// Blocks of the queries and of the keys: a warp per token of each, or as many as the GPU
// holds at once, shared out by the work of a token: its steps, and about one more for the
// angles (by heads alone, 4 key heads beside 16 query heads took a third longer than these).
void blocks_for(const QkParams& p, bool grad, int* q, int* k) {
  const int Hq = p.t[0].H, Hk = p.t[1].H;
  const int need = (p.tokens + kWarps - 1) / kWarps;
  const int rows = 512 / p.d, more = p.rot_dim > 0 ? 1 : 0;
  const int64_t wq = Hq == 0 ? 0 : (Hq + rows - 1) / rows + more;
  const int64_t wk = Hk == 0 ? 0 : (Hk + rows - 1) / rows + more;
  const int64_t most = kSms * per_sm(grad, p.rot_dim > 0);
  *q = Hq == 0 ? 0 : std::max<int>(1, std::min<int64_t>(need, most * wq / (wq + wk)));
  *k = Hk == 0 ? 0 : std::max<int>(1, std::min<int64_t>(need, most * wk / (wq + wk)));
}

template <int D, int TURN, bool GRAD>
int launch_turn(const QkParams& p, int blocks, cudaStream_t stream) {
  constexpr int bytes = kWarps * kDepth * sizeof(Slot<GRAD ? 4 : 2>);
  const auto kern = k_qk<D, TURN, GRAD>;
  static std::atomic<unsigned long long> opted{0};
  const int rc = bytes > 48 * 1024 ? opt_in_shared(kern, bytes, &opted) : SIGATTN_OK;
  if (rc != SIGATTN_OK) return rc;
  kern<<<blocks, kThreads, bytes, stream>>>(p);
  return cuda_status(cudaGetLastError());
}

template <bool GRAD>
int launch_qk(QkParams& p, cudaStream_t stream) {
  int q, k;
  blocks_for(p, GRAD, &q, &k);
  p.blocks0 = q;
  if (p.d == 64)
    return p.rot_dim == 0  ? launch_turn<64, kNone, GRAD>(p, q + k, stream)
           : p.interleaved ? launch_turn<64, kPairs, GRAD>(p, q + k, stream)
                           : launch_turn<64, kHalves, GRAD>(p, q + k, stream);
  return p.rot_dim == 0  ? launch_turn<128, kNone, GRAD>(p, q + k, stream)
         : p.interleaved ? launch_turn<128, kPairs, GRAD>(p, q + k, stream)
                         : launch_turn<128, kHalves, GRAD>(p, q + k, stream);
}

int check_strided(const void* ptr, const int64_t* strides, int H, int64_t s[3]) {
  if (!ptr || !strides) return SIGATTN_ERR_INVALID;
  for (int i = 0; i < 3; ++i)
    if (strides[i] < 0) return SIGATTN_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(ptr) & 15u) return SIGATTN_ERR_ALIGNMENT;
  for (int i = 0; i < 3; ++i) {
    if (strides[i] % 8 != 0) return SIGATTN_ERR_ALIGNMENT;
    s[i] = strides[i] / 8;
  }
  if (s[2] > 0x7FFFFFFF / H) return SIGATTN_ERR_UNSUPPORTED;
  return SIGATTN_OK;
}

// The checks that both directions share; fills all of p but the tensors.
int check_common(int B, int N, int Hq, int Hk, int d, const int32_t* lengths, float eps, int norm,
                 int rot_dim, int interleaved, int axes, const int32_t* sections,
                 const double* inv_freq, const int32_t* positions, int64_t pos_sa, int64_t pos_sb,
                 QkParams* p) {
  if (B < 1 || N < 1 || Hq < 0 || Hk < 0 || Hq + static_cast<int64_t>(Hk) < 1)
    return SIGATTN_ERR_INVALID;
  if (norm != 0 && norm != 1) return SIGATTN_ERR_INVALID;
  if (norm && !(std::isfinite(eps) && eps >= 0.0f)) return SIGATTN_ERR_INVALID;
  if (rot_dim < 0 || (interleaved != 0 && interleaved != 1)) return SIGATTN_ERR_INVALID;
  if (d != 64 && d != 128) return SIGATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(B) * N > kMaxTokens) return SIGATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(Hq) + Hk > 0x3FFFFFFF) return SIGATTN_ERR_UNSUPPORTED;
  if (rot_dim > d || rot_dim % 16 != 0) return SIGATTN_ERR_UNSUPPORTED;
  *p = QkParams{};
  if (rot_dim > 0) {
    if (!inv_freq || !positions || !sections || pos_sa < 0 || pos_sb < 0) return SIGATTN_ERR_INVALID;
    if (axes < 1) return SIGATTN_ERR_INVALID;
    if (axes > kMaxAxes) return SIGATTN_ERR_UNSUPPORTED;
    int64_t end = 0;
    for (int a = 0; a < axes; ++a) {
      if (sections[a] < 0) return SIGATTN_ERR_INVALID;
      end += sections[a];
      if (end > rot_dim / 2) return SIGATTN_ERR_INVALID;
      p->axis_end[a] = static_cast<int>(end);
    }
    if (end != rot_dim / 2) return SIGATTN_ERR_INVALID;
    p->axes = axes;
    p->inv_freq = inv_freq;
    p->pos = positions;
    p->pos_sa = pos_sa;
    p->pos_sb = pos_sb;
  }
  p->N = N;
  p->d = d;
  p->tokens = B * N;
  p->lengths = lengths;
  p->eps = eps;
  p->inv_d = 1.0f / static_cast<float>(d);
  p->norm = norm;
  p->rot_dim = rot_dim;
  p->interleaved = interleaved;
  return SIGATTN_OK;
}

int check_one(int H, const void* x, const int64_t* xs, const void* dy, const int64_t* dys,
              bool grad, void* y, const int64_t* ys, const float* w, QkTensor* t) {
  t->H = H;
  if (H == 0) return SIGATTN_OK;
  int64_t s[3];
  int rc;
  if ((rc = check_strided(x, xs, H, s)) != SIGATTN_OK) return rc;
  t->x = static_cast<const uint4*>(x);
  t->x_sb = s[0], t->x_sn = s[1], t->x_sh = static_cast<int>(s[2]);
  if (grad) {
    if ((rc = check_strided(dy, dys, H, s)) != SIGATTN_OK) return rc;
    t->dy = static_cast<const uint4*>(dy);
    t->dy_sb = s[0], t->dy_sn = s[1], t->dy_sh = static_cast<int>(s[2]);
  }
  if ((rc = check_strided(y, ys, H, s)) != SIGATTN_OK) return rc;
  t->y = static_cast<uint4*>(y);
  t->y_sb = s[0], t->y_sn = s[1], t->y_sh = static_cast<int>(s[2]);
  t->w = w;
  return SIGATTN_OK;
}

// Whether an output is another tensor than the ones it is computed from, which it may be: the
// queries' blocks and the keys' run side by side, so neither side's output may be the other's
// input or output, nor a tensor of its own side with other strides.
bool in_anothers_place(const QkParams& p) {
  for (int i = 0; i < 2; ++i) {
    const QkTensor &t = p.t[i], &other = p.t[1 - i];
    if (t.H == 0) continue;
    const auto moved = [&](int64_t sb, int64_t sn, int64_t sh) {  // (of steps that are taken)
      return (p.tokens > p.N && sb != t.y_sb) || (p.N > 1 && sn != t.y_sn) ||
             (t.H > 1 && sh != t.y_sh);
    };
    if (t.y == t.x && moved(t.x_sb, t.x_sn, t.x_sh)) return true;
    if (t.y == t.dy && moved(t.dy_sb, t.dy_sn, t.dy_sh)) return true;
    if (other.H > 0 && (t.y == other.x || t.y == other.dy || t.y == other.y)) return true;
  }
  return false;
}

}  // namespace
}  // namespace sigattn

using namespace sigattn;

extern "C" int sigattn_qk_norm_rope(int B, int N, int Hq, int Hk, int d, const int32_t* lengths,
                                    const void* q, const int64_t q_strides[3], const void* k,
                                    const int64_t k_strides[3], const float* wq, const float* wk,
                                    int norm, float eps, int rot_dim, int interleaved, int axes,
                                    const int32_t* sections, const double* inv_freq,
                                    const int32_t* positions, int64_t pos_stride_axis,
                                    int64_t pos_stride_b, void* yq, const int64_t yq_strides[3],
                                    void* yk, const int64_t yk_strides[3], sigattn_stream s) {
  QkParams p;
  int rc;
  if ((rc = check_common(B, N, Hq, Hk, d, lengths, eps, norm, rot_dim, interleaved, axes, sections,
                         inv_freq, positions, pos_stride_axis, pos_stride_b, &p)) != SIGATTN_OK)
    return rc;
  if ((rc = check_one(Hq, q, q_strides, nullptr, nullptr, false, yq, yq_strides, wq, &p.t[0])) !=
      SIGATTN_OK)
    return rc;
  if ((rc = check_one(Hk, k, k_strides, nullptr, nullptr, false, yk, yk_strides, wk, &p.t[1])) !=
      SIGATTN_OK)
    return rc;
  if (in_anothers_place(p)) return SIGATTN_ERR_INVALID;
  return launch_qk<false>(p, static_cast<cudaStream_t>(s));
}

extern "C" int sigattn_qk_norm_rope_bwd_workspace_size(int B, int N, int d, size_t* bytes) {
  if (!bytes || B < 1 || N < 1) return SIGATTN_ERR_INVALID;
  if ((d != 64 && d != 128) || static_cast<int64_t>(B) * N > kMaxTokens)
    return SIGATTN_ERR_UNSUPPORTED;
  // of any head counts: the queries' and the keys' blocks, one more where a share rounds up
  const size_t most = std::min<size_t>(2 * ((static_cast<size_t>(B) * N + kWarps - 1) / kWarps),
                                       kGradBlocks + 1);
  *bytes = sizeof(float) * d * most;
  return SIGATTN_OK;
}

extern "C" int sigattn_qk_norm_rope_bwd(
    int B, int N, int Hq, int Hk, int d, const int32_t* lengths, const void* q,
    const int64_t q_strides[3], const void* k, const int64_t k_strides[3], const void* dyq,
    const int64_t dyq_strides[3], const void* dyk, const int64_t dyk_strides[3], const float* wq,
    const float* wk, int norm, float eps, int rot_dim, int interleaved, int axes,
    const int32_t* sections, const double* inv_freq, const int32_t* positions,
    int64_t pos_stride_axis, int64_t pos_stride_b, void* dq, const int64_t dq_strides[3], void* dk,
    const int64_t dk_strides[3], float* dwq, float* dwk, void* workspace, size_t workspace_bytes,
    sigattn_stream s) {
  QkParams p;
  int rc;
  if ((rc = check_common(B, N, Hq, Hk, d, lengths, eps, norm, rot_dim, interleaved, axes, sections,
                         inv_freq, positions, pos_stride_axis, pos_stride_b, &p)) != SIGATTN_OK)
    return rc;
  if ((rc = check_one(Hq, q, q_strides, dyq, dyq_strides, true, dq, dq_strides, wq, &p.t[0])) !=
      SIGATTN_OK)
    return rc;
  if ((rc = check_one(Hk, k, k_strides, dyk, dyk_strides, true, dk, dk_strides, wk, &p.t[1])) !=
      SIGATTN_OK)
    return rc;
  if (dwq || dwk) {
    size_t need = 0;
    if ((rc = sigattn_qk_norm_rope_bwd_workspace_size(B, N, d, &need)) != SIGATTN_OK) return rc;
    if (!workspace || workspace_bytes < need) return SIGATTN_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(workspace) & 15u) return SIGATTN_ERR_ALIGNMENT;
    p.partial = static_cast<float*>(workspace);
  }
  if (in_anothers_place(p)) return SIGATTN_ERR_INVALID;
  const cudaStream_t stream = static_cast<cudaStream_t>(s);
  rc = launch_qk<true>(p, stream);
  if (rc != SIGATTN_OK || !p.partial) return rc;
  int nq, nk;
  blocks_for(p, true, &nq, &nk);
  k_qk_dw<<<2 * d / 32, 1024, 0, stream>>>(p.partial, nq, nq + nk, d, dwq, dwk);
  return cuda_status(cudaGetLastError());
}
