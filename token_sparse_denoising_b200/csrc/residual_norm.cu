// residual_norm.cu -- the residual update after a block and the norm before the next one, in one
// pass over the rows (hsa_residual_norm):
//   z  = post(y + b)                      none, RMSNorm * g or LayerNorm * g + c
//   X' = a X + gate * z                   a scalar, gate from the row's modulation row
//   h  = pre(X') * (1 + mul) + add        or pre(X') * mul + add
//
// Bound by memory: X read and X' written in float32, y read and h written in their own types, 12 to 16
// bytes an element, each once.  hsa_gated_residual followed by hsa_layernorm_rows moves X' twice more
// (written, read again) and has no post-norm.
//
// A row lives in the registers of W warps, 8 columns (16 or 32 bytes) per thread and chunk, so both
// norms see all of it without a second read.  W = 1 up to 1536 columns (48 values a thread); wider rows
// take one block of 2, 4 or 8 warps, and each reduction crosses the warps through shared memory.  All
// sums are float32, variances of centred values.  The modulation vectors of neighbouring rows are
// mostly the same, so they come from L1.
#include "common.cuh"

namespace hsa {

constexpr int kResNormWarpD = 1536;                // widest row of one warp
constexpr int kResNormMaxD = 8 * kResNormWarpD;

struct ResNormArgs {
  const float* X;
  float* X_out;                 // may be X
  const float* b;               // nullable from here on
  const float* post_g;
  const float* post_b;
  const float* gate;
  const float* mul;
  const float* add;
  const int* mod_row;
  const int* idx;
  float res_scale;
  int M, D, N, n_mod, post, pre, modulate;
  int64_t mod_stride;
};

// 8 consecutive elements as floats
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = ld4(p), b = ld4(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  st4(p, make_float4(v[0], v[1], v[2], v[3]));
  st4(p + 4, make_float4(v[4], v[5], v[6], v[7]));
}
// one rounding to bf16, of the finished value
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint4 u;
  u.x = pack_bf16x2(v[0], v[1]);
  u.y = pack_bf16x2(v[2], v[3]);
  u.z = pack_bf16x2(v[4], v[5]);
  u.w = pack_bf16x2(v[6], v[7]);
  *reinterpret_cast<uint4*>(p) = u;
}

// Sum over the W warps of a row.  W > 1: one row per block; the two halves of `part` alternate, so
// one barrier a reduction is enough.
template <int W>
__device__ __forceinline__ float row_sum(float v, float* part, int& turn) {
  v = warp_sum(v);
  if constexpr (W > 1) {
    float* p = part + (turn & 1) * W;
    ++turn;
    if ((threadIdx.x & 31) == 0) p[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += p[w];
  }
  return v;
}

// v <- normalised row (no gain): LayerNorm when `layer`, else RMSNorm
template <int W, int C>
__device__ __forceinline__ void normalise(float (&v)[C][8], int D, int l, bool layer, float* part, int& turn) {
  const float inv_d = 1.0f / (float)D;
  if (layer) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[c][e];          // columns beyond D hold 0
    const float mean = row_sum<W>(s, part, turn) * inv_d;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] = (8 * (l + c * 32 * W) < D) ? v[c][e] - mean : 0.f;
  }
  float q = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) q = fmaf(v[c][e], v[c][e], q);
  const float r = rsqrtf(fmaf(row_sum<W>(q, part, turn), inv_d, kNormEps));
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[c][e] *= r;
}

template <int W, int C, typename TY, typename TO>
__global__ void __launch_bounds__(W == 1 ? 256 : 32 * W)
    k_residual_norm(const ResNormArgs a, const TY* y, TO* out) {
  pdl_prologue();
  __shared__ float part[W > 1 ? 2 * W : 1];
  int turn = 0;
  const int r = W == 1 ? (int)((blockIdx.x * blockDim.x + threadIdx.x) >> 5) : (int)blockIdx.x;
  const int l = W == 1 ? (threadIdx.x & 31) : threadIdx.x;
  if (r >= a.M) return;
  const int D = a.D;
  // modulation row of this token
  int64_t m_off = 0;
  if (a.mod_row) {
    const int n = a.idx ? a.idx[r] : r;
    const int m = (n >= 0 && n < a.N) ? a.mod_row[n] : -1;
    if (m < 0 || m >= a.n_mod) {
      if (l == 0) flag_error(HSA_EINDEX);
      return;                                            // the same for every thread of the row
    }
    m_off = m * a.mod_stride;
  }
  const size_t base = (size_t)r * D;
  float z[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = 8 * (l + c * 32 * W);
    if (col < D) {
      load8(y + base + col, z[c]);
      if (a.b) {
        float t[8];
        load8(a.b + col, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[c][e] += t[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) z[c][e] = 0.f;
    }
  }
  if (a.post != HSA_NORM_NONE) {
    normalise<W, C>(z, D, l, a.post == HSA_NORM_LAYER, part, turn);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = 8 * (l + c * 32 * W);
      if (col < D) {
        float t[8];
        if (a.post_g) {
          load8(a.post_g + col, t);
#pragma unroll
          for (int e = 0; e < 8; ++e) z[c][e] *= t[e];
        }
        if (a.post_b) {
          load8(a.post_b + col, t);
#pragma unroll
          for (int e = 0; e < 8; ++e) z[c][e] += t[e];
        }
      }
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = 8 * (l + c * 32 * W);
    if (col < D) {
      float x[8], t[8];
      load8(a.X + base + col, x);
      if (a.gate) {
        load8(a.gate + m_off + col, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[c][e] *= t[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) z[c][e] = fmaf(a.res_scale, x[e], z[c][e]);
      store8(a.X_out + base + col, z[c]);
    }
  }
  if (a.pre == HSA_NORM_NONE) return;
  normalise<W, C>(z, D, l, a.pre == HSA_NORM_LAYER, part, turn);
  const float one = a.modulate ? 1.0f : 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = 8 * (l + c * 32 * W);
    if (col < D) {
      float t[8];
      if (a.mul) {
        load8(a.mul + m_off + col, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[c][e] *= one + t[e];
      }
      if (a.add) {
        load8(a.add + m_off + col, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[c][e] += t[e];
      }
      store8(out + base + col, z[c]);
    }
  }
}

template <int W, int C, typename TY, typename TO>
static void launch_resnorm(const ResNormArgs& a, const void* y, void* out, cudaStream_t st) {
  const unsigned rows_per_block = W == 1 ? 8 : 1;
  launch(k_residual_norm<W, C, TY, TO>, ((unsigned)a.M + rows_per_block - 1) / rows_per_block, W == 1 ? 256 : 32 * W, 0,
         st, a, static_cast<const TY*>(y), static_cast<TO*>(out));
}

// W: the fewest warps whose threads hold at most 48 values; C: chunks of 8 columns a thread
template <typename TY, typename TO>
static void dispatch_resnorm(const ResNormArgs& a, const void* y, void* out, cudaStream_t st) {
  const int D = a.D;
  const int W = D <= kResNormWarpD ? 1 : D <= 2 * kResNormWarpD ? 2 : D <= 4 * kResNormWarpD ? 4 : 8;
  const int C = (D + 256 * W - 1) / (256 * W);
  if (W == 1) {
    if (C <= 2) launch_resnorm<1, 2, TY, TO>(a, y, out, st);
    else if (C <= 4) launch_resnorm<1, 4, TY, TO>(a, y, out, st);
    else launch_resnorm<1, 6, TY, TO>(a, y, out, st);
  } else if (W == 2) {
    launch_resnorm<2, 6, TY, TO>(a, y, out, st);
  } else if (W == 4) {
    if (C <= 5) launch_resnorm<4, 5, TY, TO>(a, y, out, st);
    else launch_resnorm<4, 6, TY, TO>(a, y, out, st);
  } else {
    launch_resnorm<8, 6, TY, TO>(a, y, out, st);
  }
}

}  // namespace hsa

using namespace hsa;

extern "C" int hsa_residual_norm(const hsa_residual_norm_args* p, void* stream) {
  if (!p) return set_error(HSA_EINVAL, "residual_norm: null arguments");
  const bool y_bf = p->dtype_y == HSA_BF16, o_bf = p->dtype_out == HSA_BF16;
  if ((!y_bf && p->dtype_y != HSA_F32) || (!o_bf && p->dtype_out != HSA_F32))
    return set_error(HSA_EINVAL, "residual_norm: unknown dtype");
  if (p->post < HSA_NORM_NONE || p->post > HSA_NORM_LAYER || p->pre < HSA_NORM_NONE || p->pre > HSA_NORM_LAYER)
    return set_error(HSA_EINVAL, "residual_norm: unknown norm");
  if (p->M < 0 || p->D <= 0 || p->D % 8 || p->D > kResNormMaxD)
    return set_error(HSA_EINVAL, "residual_norm: need M >= 0, D % 8 == 0 and D <= 12288");
  if (p->d_mod_row && (p->n_mod < 1 || p->N < 1 || (!p->d_idx && p->N < p->M)))
    return set_error(HSA_EINVAL, "residual_norm: modulation rows need n_mod >= 1 and N table entries");
  if (p->d_mod_row && (p->mod_stride < p->D || p->mod_stride % 4))
    return set_error(HSA_EINVAL, "residual_norm: need mod_stride >= D and mod_stride % 4 == 0");
  if (p->post == HSA_NORM_NONE && (p->d_post_g || p->d_post_b))
    return set_error(HSA_EINVAL, "residual_norm: a post-norm gain without a post-norm");
  if (p->pre == HSA_NORM_NONE && (p->d_mul || p->d_add || p->d_out))
    return set_error(HSA_EINVAL, "residual_norm: an output without a pre-norm");
  if (p->M == 0) return HSA_OK;
  if (!p->d_X || !p->d_X_out || !p->d_y || (p->pre != HSA_NORM_NONE && !p->d_out))
    return set_error(HSA_EINVAL, "residual_norm: null pointer");
  const void* ptrs[] = {p->d_X, p->d_X_out, p->d_y, p->d_out, p->d_b, p->d_post_g, p->d_post_b, p->d_gate, p->d_mul,
                        p->d_add};
  for (const void* q : ptrs)
    if (!aligned16(q)) return set_error(HSA_EINVAL, "residual_norm: misaligned pointer");
  cudaStream_t st = as_stream(stream);
  ResNormArgs a{p->d_X, p->d_X_out, p->d_b, p->d_post_g, p->d_post_b, p->d_gate, p->d_mul, p->d_add, p->d_mod_row,
                p->d_idx, p->res_scale, p->M, p->D, p->N, p->n_mod, p->post, p->pre, p->modulate, p->mod_stride};
  ScopedTiming timing(HSA_KCLASS_OTHER, st);
  using bf16 = __nv_bfloat16;
  if (y_bf && o_bf) dispatch_resnorm<bf16, bf16>(a, p->d_y, p->d_out, st);
  else if (y_bf) dispatch_resnorm<bf16, float>(a, p->d_y, p->d_out, st);
  else if (o_bf) dispatch_resnorm<float, bf16>(a, p->d_y, p->d_out, st);
  else dispatch_resnorm<float, float>(a, p->d_y, p->d_out, st);
  count_launch(1);
  return check_launch("residual_norm launch");
}
