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
// A row lives in the registers of W warps, 4 columns (one 16-byte access) per thread and chunk, so both
// norms see all of it without a second read.  W = 1 up to 768 columns (24 values a thread), wider rows
// take 2 to 16 warps, and each reduction crosses them through shared memory.  All sums are float32,
// variances of centred values.
// One block of 32 warps per SM walks the rows.  Each group of W warps has its own ring of row slots in
// shared memory, filled by bulk copies (one elected lane, an mbarrier per slot), so the next row's X
// and y travel while this row is reduced and written; the copies bypass L1, which keeps the
// modulation vectors that neighbouring rows share.
// Measured, 32760 x 1536 (bf16 in and out) / 8190 x 5120 (float32 in, bf16 out), one set of buffers again and
// again: 103 / 97 us (before the barrier ahead of a refill also told of waits that gave up, 0.5 %); 16 warps of 48
// values a thread 111 / 102, 8 warps 127 / 119; a warp per row with plain loads and no ring 150 / 122.  With sets
// that take turns, so that nothing is left in L2: 108 / 108 us, 5.6 / 5.5 TB/s of the 6.56 a copy reaches; cache
// hints on the loads or stores and larger rings change that by 2 % at most.
#include "common.cuh"

namespace hsa {

constexpr int kResNormWarpD = 768;                // widest row of one warp
constexpr int kResNormMaxD = 16 * kResNormWarpD;

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

// Bulk copy global -> shared, `bytes` (a multiple of 16) completing on `bar`
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

constexpr int kRnWarps = 32;        // per block, one block per SM
constexpr int kRnSlots = 4;         // most row slots a group may have
constexpr int kRnSmem = 200 * 1024; // of row slots

// The W warps of group g
template <int W>
__device__ __forceinline__ void group_sync(int g) {
  if constexpr (W == 1) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(g), "r"(32 * W) : "memory");
}

// The same, and whether `x` holds in all of their threads
template <int W>
__device__ __forceinline__ bool group_all(int g, bool x) {
  if constexpr (W == 1) {
    x = __all_sync(0xffffffffu, x);
    __syncwarp();
    return x;
  } else {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.and.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(r)
        : "r"((uint32_t)x), "r"(g), "r"(32 * W)
        : "memory");
    return r != 0;
  }
}

// Sum over the W warps of a row; the two halves of `part` alternate, so one barrier a sum is enough
template <int W>
__device__ __forceinline__ float row_sum(float v, float* part, int& turn, int g) {
  v = warp_sum(v);
  if constexpr (W > 1) {
    float* p = part + (turn & 1) * W;
    ++turn;
    if ((threadIdx.x & 31) == 0) p[(threadIdx.x >> 5) % W] = v;
    group_sync<W>(g);
    v = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += p[w];
  }
  return v;
}

// v <- normalised row (no gain): LayerNorm when `layer`, else RMSNorm.  Columns beyond D hold 0.
template <int W, int C>
__device__ __forceinline__ void normalise(float4 (&v)[C], int D, int l, bool layer, float* part, int& turn, int g) {
  const float inv_d = 1.0f / (float)D;
  if (layer) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) s += (v[c].x + v[c].y) + (v[c].z + v[c].w);
    const float mean = row_sum<W>(s, part, turn, g) * inv_d;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (4 * (l + c * 32 * W) < D) {
        v[c].x -= mean; v[c].y -= mean; v[c].z -= mean; v[c].w -= mean;
      }
  }
  float q = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c)
    q = fmaf(v[c].x, v[c].x, fmaf(v[c].y, v[c].y, fmaf(v[c].z, v[c].z, fmaf(v[c].w, v[c].w, q))));
  const float r = rsqrtf(fmaf(row_sum<W>(q, part, turn, g), inv_d, kNormEps));
#pragma unroll
  for (int c = 0; c < C; ++c) {
    v[c].x *= r; v[c].y *= r; v[c].z *= r; v[c].w *= r;
  }
}

__device__ __forceinline__ float4 fma4(float4 a, float4 b, float4 c) {
  return make_float4(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y), fmaf(a.z, b.z, c.z), fmaf(a.w, b.w, c.w));
}
__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
__device__ __forceinline__ float4 mul4(float4 a, float4 b) {
  return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}

// f(z[c], v[col]) for the thread's chunks of a row vector, `kRnBatch` loads in flight at a time (a load
// that waits for the use before it costs an L1 round trip per chunk: 221 against 111 us at 32760 x 1536,
// 16 warps; with 32 warps three, four and six in flight take 109, 107 and 103 us)
constexpr int kRnBatch = 6;
template <int W, int C, typename F>
__device__ __forceinline__ void with_vector(float4 (&z)[C], const float* v, int D, int l, F&& f) {
#pragma unroll
  for (int c0 = 0; c0 < C; c0 += kRnBatch) {
    float4 t[kRnBatch];
#pragma unroll
    for (int i = 0; i < kRnBatch; ++i) {
      const int col = 4 * (l + (c0 + i) * 32 * W);
      t[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c0 + i < C && col < D) t[i] = ld4(v + col);
    }
#pragma unroll
    for (int i = 0; i < kRnBatch; ++i)
      if (c0 + i < C) z[c0 + i < C ? c0 + i : 0] = f(z[c0 + i < C ? c0 + i : 0], t[i]);
  }
}

template <int W, int C, typename TY, typename TO>
__global__ void __launch_bounds__(32 * kRnWarps, 1) k_residual_norm(const ResNormArgs a, const TY* y, TO* out, int slots) {
  pdl_prologue();
  constexpr int G = kRnWarps / W;
  extern __shared__ __align__(128) uint8_t rn_smem[];
  __shared__ uint64_t full[G][kRnSlots];
  __shared__ float parts[G][2 * W];
  const int D = a.D, M = a.M;
  const int g = threadIdx.x / (32 * W), l = threadIdx.x % (32 * W);
  const size_t slot_bytes = (size_t)D * (4 + sizeof(TY));
  uint8_t* ring = rn_smem + (size_t)g * slots * slot_bytes;
  float* part = parts[g];
  if (l == 0) {
    for (int s = 0; s < slots; ++s) mbar_init(&full[g][s], 1);
    fence_mbar_init();
  }
  group_sync<W>(g);
  // the group's rows: first, first + step, ...: consecutive rows go to different SMs
  const int first = g * (int)gridDim.x + (int)blockIdx.x, step = G * (int)gridDim.x;
  auto load_row = [&](int64_t r, int s) {
    uint8_t* p = ring + s * slot_bytes;
    mbar_expect_tx(&full[g][s], (uint32_t)slot_bytes);
    bulk_load(p, a.X + (size_t)r * D, (uint32_t)D * 4, &full[g][s]);
    bulk_load(p + (size_t)D * 4, y + (size_t)r * D, (uint32_t)D * sizeof(TY), &full[g][s]);
  };
  if (l == 0)
    for (int s = 0; s < slots; ++s) {
      const int64_t r = first + (int64_t)s * step;
      if (r < M) load_row(r, s);
    }
  int turn = 0, s = 0;
  uint32_t phase = 0;
  bool filled = true;
  const float one = a.modulate ? 1.0f : 0.0f;
  for (int64_t r = first; r < M; r += step) {
    // modulation row of this token; `good` is the same for the whole group
    int64_t m_off = 0;
    bool good = true;
    if (a.mod_row) {
      const int n = a.idx ? a.idx[r] : (int)r;
      const int m = (n >= 0 && n < a.N) ? a.mod_row[n] : -1;
      good = m >= 0 && m < a.n_mod;
      if (good) m_off = m * a.mod_stride;
      else if (l == 0) flag_error(HSA_EINDEX);
    }
    const float* xs = reinterpret_cast<const float*>(ring + s * slot_bytes);
    const TY* ys = reinterpret_cast<const TY*>(xs + D);
    filled = mbar_wait(&full[g][s], phase) && filled;     // gives up only once the library has stalled
    __syncwarp();
    const size_t base = (size_t)r * D;
    float4 z[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = 4 * (l + c * 32 * W);
      z[c] = col < D ? load4(ys + col) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (a.b) with_vector<W, C>(z, a.b, D, l, add4);
    if (a.post != HSA_NORM_NONE) {
      normalise<W, C>(z, D, l, a.post == HSA_NORM_LAYER, part, turn, g);
      if (a.post_g) with_vector<W, C>(z, a.post_g, D, l, mul4);
      if (a.post_b) with_vector<W, C>(z, a.post_b, D, l, add4);
    }
    if (a.gate) with_vector<W, C>(z, a.gate + m_off, D, l, mul4);
    const float4 scale = make_float4(a.res_scale, a.res_scale, a.res_scale, a.res_scale);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = 4 * (l + c * 32 * W);
      if (col < D) z[c] = fma4(scale, ld4(xs + col), z[c]);
    }
    // The row is in registers: its slot takes the row `slots` further on.  Where a thread's wait gave up, none of
    // the group stores this row or a later one, and no copy is sent to a slot whose last one may not have landed.
    // (Joined to the barrier: 0.6 % of the whole; a flag in shared memory or leaving the loop 1 to 4 %.)
    filled = group_all<W>(g, filled);
    good = good && filled;
    if (l == 0 && filled && r + (int64_t)slots * step < M) load_row(r + (int64_t)slots * step, s);
    if (++s == slots) {
      s = 0;
      phase ^= 1;
    }
    if (good) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int col = 4 * (l + c * 32 * W);
        if (col < D) st4(a.X_out + base + col, z[c]);
      }
    }
    if (a.pre == HSA_NORM_NONE) continue;
    normalise<W, C>(z, D, l, a.pre == HSA_NORM_LAYER, part, turn, g);
    if (!good) continue;
    if (a.mul) {
      with_vector<W, C>(z, a.mul + m_off, D, l, [one](float4 v, float4 t) {
        return mul4(v, make_float4(one + t.x, one + t.y, one + t.z, one + t.w));
      });
    }
    if (a.add) with_vector<W, C>(z, a.add + m_off, D, l, add4);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = 4 * (l + c * 32 * W);
      if (col < D) store4(out + base + col, z[c]);        // one rounding, of the finished value
    }
  }
  if (!filled) stall_drain();
}

template <int W, int C, typename TY, typename TO>
static int launch_resnorm(const ResNormArgs& a, const void* y, void* out, cudaStream_t st) {
  static PerContextOnce attr;
  int rc = attr.ensure([](void**) {
    if (cudaFuncSetAttribute(k_residual_norm<W, C, TY, TO>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRnSmem) !=
        cudaSuccess)
      return check_launch("residual_norm: shared-memory attribute");
    return (int)HSA_OK;
  });
  if (rc) return rc;
  constexpr int G = kRnWarps / W;
  const size_t slot = (size_t)a.D * (4 + sizeof(TY)) * G;
  int slots = (int)(kRnSmem / slot);
  slots = slots < 1 ? 1 : slots > kRnSlots ? kRnSlots : slots;
  const int blocks = a.M < num_sms() ? a.M : num_sms();
  launch(k_residual_norm<W, C, TY, TO>, (unsigned)blocks, 32 * kRnWarps, slots * slot, st, a,
         static_cast<const TY*>(y), static_cast<TO*>(out), slots);
  return HSA_OK;
}

// W: the fewest warps whose threads hold at most 24 values; C: chunks of 4 columns a thread: six, or four (for one
// warp two or one) where the row fits them (50 million elements in rows of 1664 / 2048 / 8192: 145 / 118 / 129 us
// with six, 124 / 106 / 115 with four), and five for eight warps alone (4097 to 5120 columns; the other widths
// between two thirds and five sixths of six chunks take six)
template <typename TY, typename TO>
static int dispatch_resnorm(const ResNormArgs& a, const void* y, void* out, cudaStream_t st) {
  const int D = a.D;
  if (D <= 128) return launch_resnorm<1, 1, TY, TO>(a, y, out, st);
  if (D <= 256) return launch_resnorm<1, 2, TY, TO>(a, y, out, st);
  if (D <= 512) return launch_resnorm<1, 4, TY, TO>(a, y, out, st);
  if (D <= kResNormWarpD) return launch_resnorm<1, 6, TY, TO>(a, y, out, st);
  if (D <= 2 * 512) return launch_resnorm<2, 4, TY, TO>(a, y, out, st);
  if (D <= 2 * kResNormWarpD) return launch_resnorm<2, 6, TY, TO>(a, y, out, st);
  if (D <= 4 * 512) return launch_resnorm<4, 4, TY, TO>(a, y, out, st);
  if (D <= 4 * kResNormWarpD) return launch_resnorm<4, 6, TY, TO>(a, y, out, st);
  if (D <= 8 * 512) return launch_resnorm<8, 4, TY, TO>(a, y, out, st);
  if (D <= 8 * 640) return launch_resnorm<8, 5, TY, TO>(a, y, out, st);
  if (D <= 8 * kResNormWarpD) return launch_resnorm<8, 6, TY, TO>(a, y, out, st);
  if (D <= 16 * 512) return launch_resnorm<16, 4, TY, TO>(a, y, out, st);
  return launch_resnorm<16, 6, TY, TO>(a, y, out, st);
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
  const int rc = y_bf ? (o_bf ? dispatch_resnorm<bf16, bf16>(a, p->d_y, p->d_out, st)
                              : dispatch_resnorm<bf16, float>(a, p->d_y, p->d_out, st))
                      : (o_bf ? dispatch_resnorm<float, bf16>(a, p->d_y, p->d_out, st)
                              : dispatch_resnorm<float, float>(a, p->d_y, p->d_out, st));
  if (rc) return rc;
  count_launch(1);
  return check_launch("residual_norm launch");
}
