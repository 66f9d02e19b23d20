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
// takes one token at a time and walks its heads, 512 / d of them per step; the angles'
// sines and cosines are computed once per token and serve every head.
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
constexpr int kMaxBlocks = 148 * 8;  // also the rows of the backward's partial weight sums

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
  float* partial;  // backward: [gridDim.x][2][d] sums of g u, nullptr without weights
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
  static constexpr int kLanes = D / 16;     // lanes of a row
  static constexpr int kRows = 32 / kLanes;  // rows of a warp's step
  int c0, c1;       // pieces
  int sub;          // row of the step
  bool turns[2];    // halves: both the same; side by side: of each piece
  uint64_t frac[8];  // turns per position of the lane's pairs, in 2^-64
  uint32_t axis;    // their axes, 4 bits each

  __device__ Lane(const QkParams& p) {
    const int l = threadIdx.x % 32 % kLanes;
    sub = threadIdx.x % 32 / kLanes;
    int pair[8];
    if (p.interleaved) {
      c0 = l;
      c1 = l + kLanes;
      turns[0] = c0 * 8 < p.rot_dim;
      turns[1] = c1 * 8 < p.rot_dim;
#pragma unroll
      for (int i = 0; i < 8; ++i) pair[i] = i < 4 ? 4 * c0 + i : 4 * c1 + i - 4;
    } else {
      const int r = p.rot_dim / 16;
      turns[0] = turns[1] = l < r;
      c0 = l < r ? l : 2 * l;  // behind the 2r turned pieces the rest pair up in order
      c1 = l < r ? l + r : 2 * l + 1;
#pragma unroll
      for (int i = 0; i < 8; ++i) pair[i] = 8 * l + i;
    }
    axis = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      frac[i] = 0;
      if (turns[i / 4]) {
        // inv_freq / 2 pi without its whole turns; scaling by 2^64 is exact
        double f = p.inv_freq[pair[i]] * 0.15915494309189533577;
        f -= floor(f);
        frac[i] = f < 1.0 ? static_cast<uint64_t>(f * 18446744073709551616.0) : 0;
        uint32_t a = 0;
        while (a + 1 < static_cast<uint32_t>(p.axes) && pair[i] >= p.axis_end[a]) ++a;
        axis |= a << (4 * i);
      }
    }
  }

  // cos and sin of the lane's eight angles at token (b, i)
  __device__ void angles(const QkParams& p, int b, int i, float* cs, float* sn) const {
    if (p.rot_dim == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) cs[j] = 1.0f, sn[j] = 0.0f;
      return;
    }
    const int32_t* at = p.pos + b * p.pos_sb + i;
    int32_t x[kMaxAxes];
#pragma unroll
    for (int a = 0; a < kMaxAxes; ++a) x[a] = a < p.axes ? at[a * p.pos_sa] : 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t a = (axis >> (4 * j)) & 15u;
      const int32_t pos = a == 0 ? x[0] : a == 1 ? x[1] : a == 2 ? x[2] : x[3];
      const uint64_t turn = frac[j] * static_cast<uint64_t>(static_cast<int64_t>(pos));
      // the high word as a signed fraction of half turns in [-1, 1)
      sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &sn[j], &cs[j]);
    }
  }

  // y = R z (way = 1) or R^T z (way = -1) on the lane's two pieces z[0..7], z[8..15]
  __device__ __forceinline__ static void turn(bool interleaved, float way, const float* cs,
                                              const float* sn, float* z) {
    if (interleaved) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float a = z[2 * j], b = z[2 * j + 1], s = way * sn[j];
        z[2 * j] = a * cs[j] - b * s;
        z[2 * j + 1] = a * s + b * cs[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float a = z[j], b = z[j + 8], s = way * sn[j];
        z[j] = a * cs[j] - b * s;
        z[j + 8] = a * s + b * cs[j];
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

__device__ __forceinline__ void load_weights(const float* w, int c0, int c1, float* f) {
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] = w ? __ldg(w + (i < 8 ? c0 : c1) * 8 + (i & 7)) : 1.0f;
}

template <int D>
__global__ void __launch_bounds__(kThreads) k_qk_fwd(const QkParams p) {
  using L = Lane<D>;
  const L lane(p);
  float w[2][16];
  load_weights(p.t[0].w, lane.c0, lane.c1, w[0]);
  load_weights(p.t[1].w, lane.c0, lane.c1, w[1]);
  const int step = gridDim.x * kWarps;
  for (int tok = blockIdx.x * kWarps + threadIdx.x / 32; tok < p.tokens; tok += step) {
    const int b = tok / p.N, i = tok % p.N;
    const bool valid = !p.lengths || i < __ldg(p.lengths + b);
    float cs[8], sn[8];
    if (valid) lane.angles(p, b, i, cs, sn);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const QkTensor& t = p.t[m];
      const uint4* x = t.x + b * t.x_sb + i * t.x_sn;
      uint4* y = t.y + b * t.y_sb + i * t.y_sn;
      for (int h0 = 0; h0 < t.H; h0 += L::kRows) {
        const int h = h0 + lane.sub;
        const bool have = h < t.H;
        if (!valid) {
          if (have) {
            y[h * t.y_sh + lane.c0] = make_uint4(0u, 0u, 0u, 0u);
            y[h * t.y_sh + lane.c1] = make_uint4(0u, 0u, 0u, 0u);
          }
          continue;
        }
        uint4 r0 = make_uint4(0u, 0u, 0u, 0u), r1 = r0;
        if (have) {
          r0 = x[h * t.x_sh + lane.c0];
          r1 = x[h * t.x_sh + lane.c1];
        }
        float z[16];
        unpack8(r0, z);
        unpack8(r1, z + 8);
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) s = fmaf(z[j], z[j], s);
        s = L::row_sum(s);
        const float r = p.norm ? rsqrtf(fmaf(s, p.inv_d, p.eps)) : 1.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) z[j] *= r * w[m][j];
        L::turn(p.interleaved, 1.0f, cs, sn, z);
        if (have) {
          y[h * t.y_sh + lane.c0] = pack8(z);
          y[h * t.y_sh + lane.c1] = pack8(z + 8);
        }
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) k_qk_bwd(const QkParams p) {
  using L = Lane<D>;
  const L lane(p);
  float w[2][16], dw[2][16];
  load_weights(p.t[0].w, lane.c0, lane.c1, w[0]);
  load_weights(p.t[1].w, lane.c0, lane.c1, w[1]);
#pragma unroll
  for (int j = 0; j < 16; ++j) dw[0][j] = dw[1][j] = 0.0f;
  const int step = gridDim.x * kWarps;
  for (int tok = blockIdx.x * kWarps + threadIdx.x / 32; tok < p.tokens; tok += step) {
    const int b = tok / p.N, i = tok % p.N;
    const bool valid = !p.lengths || i < __ldg(p.lengths + b);
    float cs[8], sn[8];
    if (valid) lane.angles(p, b, i, cs, sn);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const QkTensor& t = p.t[m];
      const uint4* x = t.x + b * t.x_sb + i * t.x_sn;
      const uint4* dy = t.dy + b * t.dy_sb + i * t.dy_sn;
      uint4* dx = t.y + b * t.y_sb + i * t.y_sn;
      for (int h0 = 0; h0 < t.H; h0 += L::kRows) {
        const int h = h0 + lane.sub;
        const bool have = h < t.H;
        if (!valid) {
          if (have) {
            dx[h * t.y_sh + lane.c0] = make_uint4(0u, 0u, 0u, 0u);
            dx[h * t.y_sh + lane.c1] = make_uint4(0u, 0u, 0u, 0u);
          }
          continue;
        }
        uint4 r0 = make_uint4(0u, 0u, 0u, 0u), r1 = r0, g0 = r0, g1 = r0;
        if (have) {
          r0 = x[h * t.x_sh + lane.c0];
          r1 = x[h * t.x_sh + lane.c1];
          g0 = dy[h * t.dy_sh + lane.c0];
          g1 = dy[h * t.dy_sh + lane.c1];
        }
        float u[16], g[16];
        unpack8(r0, u);
        unpack8(r1, u + 8);
        unpack8(g0, g);
        unpack8(g1, g + 8);
        L::turn(p.interleaved, -1.0f, cs, sn, g);
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) s = fmaf(u[j], u[j], s);
        s = L::row_sum(s);
        // a lane without a row has u = g = 0 and, with r = 0 (not rsqrt(eps)), adds nothing
        const float r = !have ? 0.0f : p.norm ? rsqrtf(fmaf(s, p.inv_d, p.eps)) : 1.0f;
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          u[j] *= r;
          dw[m][j] = fmaf(g[j], u[j], dw[m][j]);
          g[j] *= w[m][j];
          dot = fmaf(g[j], u[j], dot);
        }
        dot = p.norm ? L::row_sum(dot) * p.inv_d : 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) g[j] = r * fmaf(-u[j], dot, g[j]);
        if (have) {
          dx[h * t.y_sh + lane.c0] = pack8(g);
          dx[h * t.y_sh + lane.c1] = pack8(g + 8);
        }
      }
    }
  }
  if (!p.partial) return;
  // The block's sums, in a fixed order: the rows of each warp by shuffles, the warps one
  // after another from shared memory.
  __shared__ float sums[kWarps][2][D];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      float v = dw[m][j];
#pragma unroll
      for (int o = 16; o >= L::kLanes; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      if (lane.sub == 0) sums[threadIdx.x / 32][m][(j < 8 ? lane.c0 : lane.c1) * 8 + (j & 7)] = v;
    }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * D; c += kThreads) {
    float v = 0.0f;
#pragma unroll
    for (int x = 0; x < kWarps; ++x) v += sums[x][c / D][c % D];
    p.partial[static_cast<int64_t>(blockIdx.x) * 2 * D + c] = v;
  }
}

// dwq, dwk from the blocks' partial sums [rows][2 d]: one block per 32 columns, its warps
// take the rows in turn (coalesced 128-byte reads) and are added in a fixed order.
__global__ void __launch_bounds__(1024) k_qk_dw(const float* __restrict__ partial, int rows,
                                                int d, float* __restrict__ dwq,
                                                float* __restrict__ dwk) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
  float v = 0.0f;
  for (int r = warp; r < rows; r += 32) v += partial[static_cast<int64_t>(r) * 2 * d + c];
  sums[warp][lane] = v;
  __syncthreads();
  v = sums[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (lane == 0) {
    const int col = blockIdx.x * 32 + warp;
    float* out = col < d ? dwq : dwk;
    if (out) out[col % d] = v;
  }
}

int blocks_for(int tokens) { return std::min((tokens + kWarps - 1) / kWarps, kMaxBlocks); }

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
  if (static_cast<int64_t>(B) * N > 0x7FFFFFFF - kMaxBlocks * kWarps) return SIGATTN_ERR_UNSUPPORTED;
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
  const auto kern = d == 64 ? k_qk_fwd<64> : k_qk_fwd<128>;
  kern<<<blocks_for(p.tokens), kThreads, 0, static_cast<cudaStream_t>(s)>>>(p);
  return cuda_status(cudaGetLastError());
}

extern "C" int sigattn_qk_norm_rope_bwd_workspace_size(int B, int N, int d, size_t* bytes) {
  if (!bytes || B < 1 || N < 1) return SIGATTN_ERR_INVALID;
  if ((d != 64 && d != 128) || static_cast<int64_t>(B) * N > 0x7FFFFFFF - kMaxBlocks * kWarps)
    return SIGATTN_ERR_UNSUPPORTED;
  *bytes = sizeof(float) * 2 * d * blocks_for(B * N);
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
  const int blocks = blocks_for(p.tokens);
  if (dwq || dwk) {
    if (!workspace || workspace_bytes < sizeof(float) * 2 * d * static_cast<size_t>(blocks))
      return SIGATTN_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(workspace) & 15u) return SIGATTN_ERR_ALIGNMENT;
    p.partial = static_cast<float*>(workspace);
  }
  const cudaStream_t stream = static_cast<cudaStream_t>(s);
  const auto kern = d == 64 ? k_qk_bwd<64> : k_qk_bwd<128>;
  kern<<<blocks, kThreads, 0, stream>>>(p);
  rc = cuda_status(cudaGetLastError());
  if (rc != SIGATTN_OK || !p.partial) return rc;
  k_qk_dw<<<2 * d / 32, 1024, 0, stream>>>(p.partial, blocks, d, dwq, dwk);
  return cuda_status(cudaGetLastError());
}
