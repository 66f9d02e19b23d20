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
// What bounds it is the memory, 4 bytes an element forward and 6 backward, if enough loads
// are in flight: each lane keeps the pieces of its next kDepth steps on their way into shared
// memory slots of its own (cp.async; nobody else reads them, so a step waits for its own
// copies alone).
//
// Angles: with inv_freq / 2 pi kept as a 64-bit fraction F of a turn, position * F modulo
// 2^64 is the angle modulo one turn with no rounding that grows with the position, so far
// positions are as exact as near ones (a 32-bit product is off by 1e-2 radians at 2e5).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "internal.h"

namespace sigattn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxAxes = 4;
// a warp's token index steps past the last one by at most the grid's warps (148 * 3 * 8)
constexpr int64_t kMaxTokens = 0x7FFFFFFF - 16384;
constexpr int kDepth = 4;         // steps whose loads are in flight
constexpr int kSms = 148;         // B200
constexpr int kPerSm[2] = {3, 2};  // resident blocks, forward and backward

struct QkTensor {
  const uint4* x;
  const uint4* dy;  // backward only
  uint4* y;         // forward: y; backward: dx
  int64_t x_sb, x_sn, x_sh, dy_sb, dy_sn, dy_sh, y_sb, y_sn, y_sh;  // in 8-value pieces
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

__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// What a lane knows of its place in a row: its two pieces and the pairs that they form.
template <int D>
struct Lane {
  static constexpr int kLanes = D / 16;      // lanes of a row
  static constexpr int kRows = 32 / kLanes;  // rows of a warp's step
  static constexpr int kOwn = 8 / kRows;     // pairs of the lane's eight that it computes
  int c0, c1;           // pieces
  int sub;              // row of the step
  uint64_t frac[kOwn];  // turns per position of the pairs it computes, in 2^-64
  int axis[kOwn];       // their axes

  __device__ Lane(const QkParams& p) {
    const int l = threadIdx.x % 32 % kLanes;
    sub = threadIdx.x % 32 / kLanes;
    const int r = p.rot_dim / 16;  // turned pieces of a half
    c0 = p.interleaved || l < r ? l : 2 * l;  // halves: behind 2 r pieces the rest pair up
    c1 = p.interleaved ? l + kLanes : l < r ? l + r : 2 * l + 1;
#pragma unroll
    for (int x = 0; x < kOwn; ++x) {
      const int i = sub * kOwn + x;  // of the lane's eight pairs
      const int pair = !p.interleaved ? 8 * l + i : i < 4 ? 4 * c0 + i : 4 * c1 + i - 4;
      frac[x] = 0;
      axis[x] = 0;
      if (p.interleaved ? 2 * pair < p.rot_dim : l < r) {
        // inv_freq / 2 pi without its whole turns; scaling by 2^64 is exact
        double f = p.inv_freq[pair] * 0.15915494309189533577;
        f -= floor(f);
        frac[x] = f < 1.0 ? static_cast<uint64_t>(f * 18446744073709551616.0) : 0;
        while (axis[x] + 1 < p.axes && pair >= p.axis_end[axis[x]]) ++axis[x];
      }
    }
  }

  // cos and sin of the lane's eight angles at the positions pos[axis]
  __device__ __forceinline__ void angles(const int32_t* pos, float* cs, float* sn) const {
    float c[kOwn], s[kOwn];
#pragma unroll
    for (int x = 0; x < kOwn; ++x) {
      const uint64_t turn = frac[x] * static_cast<uint64_t>(static_cast<int64_t>(pos[axis[x]]));
      // the high word as a signed fraction of half turns in [-1, 1)
      sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &s[x], &c[x]);
    }
    const int l = threadIdx.x % 32 % kLanes;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      cs[j] = __shfl_sync(0xFFFFFFFFu, c[j % kOwn], j / kOwn * kLanes + l);
      sn[j] = __shfl_sync(0xFFFFFFFFu, s[j % kOwn], j / kOwn * kLanes + l);
    }
  }

  // y = R z, or R^T z with the sines negated, on the lane's two pieces z[0..7], z[8..15]
  __device__ __forceinline__ static void turn(bool interleaved, const float* cs, const float* sn,
                                              float* z) {
    if (interleaved) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float a = z[2 * j], b = z[2 * j + 1];
        z[2 * j] = a * cs[j] - b * sn[j];
        z[2 * j + 1] = a * sn[j] + b * cs[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float a = z[j], b = z[j + 8];
        z[j] = a * cs[j] - b * sn[j];
        z[j + 8] = a * sn[j] + b * cs[j];
      }
    }
  }

  // sum over the lanes of a row
  __device__ __forceinline__ static float row_sum(float v) {
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

// A warp's walk over the steps of its tokens.
struct Walk {
  int tok, h, b, i;  // token, first head of the step, batch entry and row
  bool valid;
  __device__ __forceinline__ void enter(const QkParams& p) {
    b = tok / p.N;
    i = tok - b * p.N;
    valid = tok < p.tokens && (!p.lengths || i < __ldg(p.lengths + b));
  }
  __device__ __forceinline__ void next(const QkParams& p, int H, int rows, int stride) {
    h += rows;
    if (h >= H) {
      h = 0;
      tok += stride;
      if (tok < p.tokens) enter(p);
    }
  }
};

// Forward (GRAD false) and backward.  In the backward y takes the gradient of x.
template <int D, bool GRAD>
__global__ void __launch_bounds__(kThreads, kPerSm[GRAD]) k_qk(const QkParams p) {
  using L = Lane<D>;
  constexpr int kPieces = GRAD ? 4 : 2;
  extern __shared__ uint4 smem[];
  const int warp = threadIdx.x / 32, ln = threadIdx.x % 32;
  Slot<kPieces>* slots = reinterpret_cast<Slot<kPieces>*>(smem) + warp * kDepth;
  const bool keys = static_cast<int>(blockIdx.x) >= p.blocks0;
  const QkTensor& t = p.t[keys];
  const int block = keys ? blockIdx.x - p.blocks0 : blockIdx.x;
  const int stride = (keys ? gridDim.x - p.blocks0 : p.blocks0) * kWarps;
  const L lane(p);

  Walk ahead{block * kWarps + warp, 0, 0, 0, false};
  ahead.enter(p);
  Walk at = ahead;
  auto fetch = [&](Slot<kPieces>& s) {
    if (ahead.tok < p.tokens) {
      if (ahead.valid) {
        const int h = ahead.h + lane.sub;
        const bool have = h < t.H;
        const uint4* x = t.x + ahead.b * t.x_sb + ahead.i * t.x_sn + (have ? h : 0) * t.x_sh;
        copy16(&s.piece[0][ln], x + lane.c0, have);
        copy16(&s.piece[1][ln], x + lane.c1, have);
        if constexpr (GRAD) {
          const uint4* g = t.dy + ahead.b * t.dy_sb + ahead.i * t.dy_sn + (have ? h : 0) * t.dy_sh;
          copy16(&s.piece[2][ln], g + lane.c0, have);
          copy16(&s.piece[3][ln], g + lane.c1, have);
        }
        if (ahead.h == 0 && ln < p.axes)
          copy4(&s.pos[ln], p.pos + ln * p.pos_sa + ahead.b * p.pos_sb + ahead.i);
      }
      ahead.next(p, t.H, L::kRows, stride);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < kDepth - 1; ++s) fetch(slots[s]);

  float w[16], dw[16], cs[8], sn[8];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    w[j] = t.w ? __ldg(t.w + (j < 8 ? lane.c0 : lane.c1) * 8 + (j & 7)) : 1.0f;
    dw[j] = 0.0f;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) cs[j] = 1.0f, sn[j] = 0.0f;

  for (int n = 0; at.tok < p.tokens; ++n) {
    Slot<kPieces>& s = slots[n % kDepth];
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
    const int h = at.h + lane.sub;
    const bool have = h < t.H;
    uint4* y = t.y + at.b * t.y_sb + at.i * t.y_sn + (have ? h : 0) * t.y_sh;
    if (at.valid) {
      if (at.h == 0 && p.rot_dim > 0) {
        __syncwarp();  // the positions were copied by other lanes
        lane.angles(s.pos, cs, sn);
        if (GRAD)
#pragma unroll
          for (int j = 0; j < 8; ++j) sn[j] = -sn[j];
      }
      float z[16], g[16];
      unpack8(s.piece[0][ln], z);
      unpack8(s.piece[1][ln], z + 8);
      if constexpr (GRAD) {
        unpack8(s.piece[2][ln], g);
        unpack8(s.piece[3][ln], g + 8);
        L::turn(p.interleaved, cs, sn, g);
      }
      float r = 1.0f;
      if (p.norm) {
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) sum = fmaf(z[j], z[j], sum);
        r = rsqrtf(fmaf(L::row_sum(sum), p.inv_d, p.eps));
      }
      if constexpr (!GRAD) {
#pragma unroll
        for (int j = 0; j < 16; ++j) z[j] *= r * w[j];
        L::turn(p.interleaved, cs, sn, z);
        if (have) {
          y[lane.c0] = pack8(z);
          y[lane.c1] = pack8(z + 8);
        }
      } else {
        // a lane without a row has u = g = 0 and, with r = 0 (not rsqrt(eps)), adds nothing
        if (!have) r = 0.0f;
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          z[j] *= r;
          dw[j] = fmaf(g[j], z[j], dw[j]);
          g[j] *= w[j];
          dot = fmaf(g[j], z[j], dot);
        }
        dot = p.norm ? L::row_sum(dot) * p.inv_d : 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) g[j] = r * fmaf(-z[j], dot, g[j]);
        if (have) {
          y[lane.c0] = pack8(g);
          y[lane.c1] = pack8(g + 8);
        }
      }
    } else if (have) {
      y[lane.c0] = make_uint4(0u, 0u, 0u, 0u);
      y[lane.c1] = make_uint4(0u, 0u, 0u, 0u);
    }
    at.next(p, t.H, L::kRows, stride);
    __syncwarp();  // every lane has read the positions of the slot that is filled next
    fetch(slots[(n + kDepth - 1) % kDepth]);
  }
  if (!GRAD || !p.partial) return;
  // The block's sums, in a fixed order: the rows of each warp by shuffles, the warps one
  // after another from shared memory.
  __shared__ float sums[kWarps][D];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float v = dw[j];
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
  float v = 0.0f;
  for (int r = (keys ? rows0 : 0) + warp; r < (keys ? rows : rows0); r += 32)
    v += partial[r * d + c0 + lane];
  sums[warp][lane] = v;
  __syncthreads();
  v = sums[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (lane == 0) out[c0 + warp] = v;
}

// Blocks of the queries and of the keys: a warp per token of each, or as many as the GPU
// holds at once, shared out by their heads.
void blocks_for(int tokens, int Hq, int Hk, int most, int* q, int* k) {
  const int need = (tokens + kWarps - 1) / kWarps;
  const int64_t heads = static_cast<int64_t>(Hq) + Hk;
  *q = Hq == 0 ? 0 : std::max<int>(1, std::min<int64_t>(need, static_cast<int64_t>(most) * Hq / heads));
  *k = Hk == 0 ? 0 : std::max<int>(1, std::min<int64_t>(need, static_cast<int64_t>(most) * Hk / heads));
}

template <int D, bool GRAD>
int launch_qk(QkParams& p, cudaStream_t stream) {
  constexpr int bytes = kWarps * kDepth * sizeof(Slot<GRAD ? 4 : 2>);
  int q, k;
  blocks_for(p.tokens, p.t[0].H, p.t[1].H, kSms * kPerSm[GRAD], &q, &k);
  p.blocks0 = q;
  const auto kern = k_qk<D, GRAD>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return cuda_status(e);
  kern<<<q + k, kThreads, bytes, stream>>>(p);
  return cuda_status(cudaGetLastError());
}

int check_strided(const void* ptr, const int64_t* strides, int64_t s[3]) {
  if (!ptr || !strides) return SIGATTN_ERR_INVALID;
  for (int i = 0; i < 3; ++i)
    if (strides[i] < 0) return SIGATTN_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(ptr) & 15u) return SIGATTN_ERR_ALIGNMENT;
  for (int i = 0; i < 3; ++i) {
    if (strides[i] % 8 != 0) return SIGATTN_ERR_ALIGNMENT;
    s[i] = strides[i] / 8;
  }
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
  if ((rc = check_strided(x, xs, s)) != SIGATTN_OK) return rc;
  t->x = static_cast<const uint4*>(x);
  t->x_sb = s[0], t->x_sn = s[1], t->x_sh = s[2];
  if (grad) {
    if ((rc = check_strided(dy, dys, s)) != SIGATTN_OK) return rc;
    t->dy = static_cast<const uint4*>(dy);
    t->dy_sb = s[0], t->dy_sn = s[1], t->dy_sh = s[2];
  }
  if ((rc = check_strided(y, ys, s)) != SIGATTN_OK) return rc;
  t->y = static_cast<uint4*>(y);
  t->y_sb = s[0], t->y_sn = s[1], t->y_sh = s[2];
  t->w = w;
  return SIGATTN_OK;
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
  const cudaStream_t stream = static_cast<cudaStream_t>(s);
  return d == 64 ? launch_qk<64, false>(p, stream) : launch_qk<128, false>(p, stream);
}

extern "C" int sigattn_qk_norm_rope_bwd_workspace_size(int B, int N, int d, size_t* bytes) {
  if (!bytes || B < 1 || N < 1) return SIGATTN_ERR_INVALID;
  if ((d != 64 && d != 128) || static_cast<int64_t>(B) * N > kMaxTokens)
    return SIGATTN_ERR_UNSUPPORTED;
  // of any head counts: the queries' and the keys' blocks, one more where a share rounds up
  const size_t most = std::min<size_t>(2 * ((static_cast<size_t>(B) * N + kWarps - 1) / kWarps),
                                       kSms * kPerSm[1] + 1);
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
  const cudaStream_t stream = static_cast<cudaStream_t>(s);
  rc = d == 64 ? launch_qk<64, true>(p, stream) : launch_qk<128, true>(p, stream);
  if (rc != SIGATTN_OK || !p.partial) return rc;
  int nq, nk;
  blocks_for(p.tokens, Hq, Hk, kSms * kPerSm[1], &nq, &nk);
  k_qk_dw<<<2 * d / 32, 1024, 0, stream>>>(p.partial, nq, nq + nk, d, dwq, dwk);
  return cuda_status(cudaGetLastError());
}
