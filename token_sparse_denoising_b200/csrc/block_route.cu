// block_route.cu -- which key blocks each query tile attends to: the cheap scores
// (hsa_block_scores) and the choice of the best blocks (hsa_block_select).
//
// Scores.  The dot product is linear, so the mean logit of a 128-row query tile against a block of
// keys is the product of their mean rows:
//   s[h][t][b] = (1/|t| sum_{r in t} q_r) . (1/|b| sum_{j in b} k_j) / sqrt(128)
// and the (M + L) rows are read once.  k_block_means is bound by that read; k_block_product is a
// small float32 product of the means.
//
// Selection.  Total order of a row's blocks: (score descending, index ascending), scores compared as
// float32 with -0 equal to 0 and NaN as +inf; -inf closes a block, forced blocks come first.  The
// result is unique, so it does not depend on how the kernel finds it.
#include "common.cuh"

namespace hsa {

constexpr int kRouteTile = HSA_QUERY_TILE;

// Mean rows: CTA = one head of one block of rows; 16 threads cover the head's 128 channels, 16 row
// groups walk the block's rows, joined by a shuffle and through shared memory.  Blocks [0, T) are the
// query tiles, [T, T + B) the key blocks.  Sums in float32 (at most 128 terms).
template <typename T>
__global__ void __launch_bounds__(256) k_block_means(const T* __restrict__ q, int M, const T* __restrict__ k, int L,
                                                     int H, int block_k, int n_tiles, float* __restrict__ means) {
  pdl_prologue();
  __shared__ float part[8][128];
  const int h = blockIdx.x, j = blockIdx.y;
  const bool key = j >= n_tiles;
  const int size = key ? block_k : kRouteTile;
  const int r0 = (key ? j - n_tiles : j) * size;
  const int n = min(size, (key ? L : M) - r0);
  const size_t D = (size_t)H * 128;
  const int c = (threadIdx.x & 15) * 8, g = threadIdx.x >> 4;
  const T* src = (key ? k : q) + (size_t)r0 * D + h * 128 + c;
  float s[8] = {};
#pragma unroll 8
  for (int i = 0; i < 8; ++i) {
    const int r = g + 16 * i;
    if (r < n) {
      float v[8];
      load8(src + (size_t)r * D, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] += v[e];
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] += __shfl_xor_sync(0xffffffffu, s[e], 16);
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 16) == 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) part[warp][c + e] = s[e];
  }
  __syncthreads();
  if (threadIdx.x < 128) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += part[w][threadIdx.x];
    means[(size_t)j * D + h * 128 + threadIdx.x] = t / (float)n;
  }
}

// scores[h] = Qm[h] Km[h]^T / sqrt(128) in float32: 64 x 64 tile per CTA, 4 x 4 per thread.
__global__ void __launch_bounds__(256) k_block_product(const float* __restrict__ means, int n_tiles, int n_blocks,
                                                       int H, float* __restrict__ scores) {
  pdl_prologue();
  __shared__ float Qs[32][68], Ks[32][68];
  const int h = blockIdx.z, t0 = blockIdx.y * 64, b0 = blockIdx.x * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const size_t D = (size_t)H * 128;
  const float* qm = means + h * 128;
  const float* km = means + (size_t)n_tiles * D + h * 128;
  float acc[4][4] = {};
  for (int c0 = 0; c0 < 128; c0 += 32) {
    for (int i = threadIdx.x; i < 64 * 8; i += 256) {
      const int row = i >> 3, c4 = (i & 7) * 4;
      const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
      const float4 a = t0 + row < n_tiles ? ld4(qm + (size_t)(t0 + row) * D + c0 + c4) : z;
      const float4 b = b0 + row < n_blocks ? ld4(km + (size_t)(b0 + row) * D + c0 + c4) : z;
      Qs[c4][row] = a.x; Qs[c4 + 1][row] = a.y; Qs[c4 + 2][row] = a.z; Qs[c4 + 3][row] = a.w;
      Ks[c4][row] = b.x; Ks[c4 + 1][row] = b.y; Ks[c4 + 2][row] = b.z; Ks[c4 + 3][row] = b.w;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      const float4 a = *reinterpret_cast<const float4*>(&Qs[c][ty * 4]);
      const float4 b = *reinterpret_cast<const float4*>(&Ks[c][tx * 4]);
      const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
    }
    __syncthreads();
  }
  const float scale = 0.08838834764831845f;              // 1 / sqrt(128)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + ty * 4 + i;
    if (t >= n_tiles) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int b = b0 + tx * 4 + j;
      if (b < n_blocks) scores[((size_t)h * n_tiles + t) * n_blocks + b] = acc[i][j] * scale;
    }
  }
}

// ------------------------------------------------------------------ selection
// Order key: ascending in the score; -inf (closed) maps to kRouteClosed, all ones = forced (above +inf,
// 0xFF800000).  fminf turns NaN into +inf, adding +0 turns -0 into +0.
constexpr uint32_t kRouteClosed = 0x007FFFFFu;
__device__ __forceinline__ uint32_t route_key(float s) {
  const uint32_t u = __float_as_uint(fminf(s, INFINITY) + 0.0f);
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}

constexpr int kRouteMaxBlocks = 16384;

// float of an order key, the largest finite one for keys at or above +inf (interpolation only)
__device__ __forceinline__ float route_value(uint32_t k) {
  k = min(k, 0xFF7FFFFFu);
  return __uint_as_float(k ^ ((uint32_t)((int)~k >> 31) | 0x80000000u));
}

constexpr int kRouteFew = 32;      // keys a warp ranks against each other to finish the search

// One row of scores per group of W warps (W = 1: 8 rows a block; W = 8: one).  Warp w of the group
// holds blocks [w 32 V, (w + 1) 32 V) in registers, 32 consecutive ones at a time.
// The cut is searched between keys lo and hi with count(key >= lo) > keep > count(key >= hi): a pass counts
// the keys at or above a candidate and replaces one bound, and the search ends when the count is `keep`
// (a distinct cut) or hi = lo + 1 (ties at lo, given to the lowest index).  Scores are spread smoothly, so
// the first candidates interpolate between the bounds' values (about 5 passes until 32 of 1182 normal
// scores are left, against 11 by halving); every third one, and all after the sixth, halve the key
// interval, which bounds the passes whatever the scores.  Once at most 32 keys are left between the
// bounds, a warp with many registers of keys moves them to one register a lane and ranks them.
// Then the chosen blocks are written in index order.  Bound by instructions: a row of 1182 scores
// takes a warp about 1500, against 4.7 KB read.
template <int W, int V>
__global__ void __launch_bounds__(256, V > 40 ? 1 : V > 16 ? 3 : 4)
    k_block_select(const float* __restrict__ scores, int rows, int n_blocks, int keep,
                   const uint8_t* __restrict__ forced, int* __restrict__ list, int* __restrict__ count) {
  pdl_prologue();
  __shared__ uint32_t part[2][3][8];
  __shared__ uint32_t fbits[W * V];
  __shared__ __align__(16) uint32_t few[W == 1 && V > 8 ? 8 : 1][kRouteFew];
  int turn = 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = W == 1 ? (int)blockIdx.x * 8 + warp : (int)blockIdx.x;
  if (forced) {
    // one bit per block, read by every row of the CTA
    for (int i = warp; i < W * V; i += 8) {
      const int b = 32 * i + lane;
      const uint32_t m = __ballot_sync(0xffffffffu, b < n_blocks && forced[b] != 0);
      if (lane == 0) fbits[i] = m;
    }
    __syncthreads();
  }
  if (row >= rows) return;
  const int base = W == 1 ? 0 : warp * 32 * V;
  const float* src = scores + (size_t)row * n_blocks;
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int b = base + 32 * i + lane;
    key[i] = __float_as_uint(b < n_blocks ? __ldcs(src + b) : -INFINITY);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = route_key(__uint_as_float(key[i]));
  // sum over the group of one count per lane
  auto group_sum = [&](uint32_t x) -> uint32_t {
    x = __reduce_add_sync(0xffffffffu, x);
    if constexpr (W > 1) {
      uint32_t* p = part[turn & 1][0];
      ++turn;
      if (lane == 0) p[warp] = x;
      __syncthreads();
      x = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) x += p[w];
    }
    return x;
  };
  // bounds of the open scores (a forced block's own score may widen them, which is harmless)
  uint32_t n_open = 0, n_forced = 0, hi = 0u, lo = 0xFFFFFFFFu;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    lo = min(lo, key[i] - (kRouteClosed + 1u));           // closed: all ones
    hi = max(hi, key[i]);
  }
  if (forced) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t m = fbits[(W == 1 ? 0 : warp * V) + i];
      if (m) {                                            // the same for the whole warp
        if ((m >> lane) & 1u) key[i] = 0xFFFFFFFFu;
        n_forced += __popc(m);
      }
    }
    n_forced = group_sum(lane == 0 ? n_forced : 0u);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) n_open += key[i] > kRouteClosed;
  n_open = group_sum(n_open);
  hi = __reduce_max_sync(0xffffffffu, hi);
  lo = __reduce_min_sync(0xffffffffu, lo);
  if constexpr (W > 1) {
    uint32_t(*p)[8] = part[turn & 1];
    ++turn;
    if (lane == 0) {
      p[1][warp] = hi;
      p[2][warp] = lo;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) {
      hi = max(hi, p[1][w]);
      lo = min(lo, p[2][w]);
    }
  }
  lo += kRouteClosed + 1u;
  const uint32_t want = (uint32_t)keep;
  uint32_t cut = kRouteClosed + 1u, ties = 0u;                           // chosen: key >= cut, or > cut and `ties` of == cut
  bool tied = false;
  if (n_forced >= want) {
    cut = 0xFFFFFFFFu;
    ties = want;
    tied = true;
  } else if (n_open > want) {
    uint32_t n_lo = n_open, n_hi = n_forced;
    hi += 1u;                                             // above every key that is not forced
    bool exact = false;
    for (int pass = 0; hi - lo > 1u; ++pass) {
      if (W == 1 && V > 8 && n_lo - n_hi <= kRouteFew) break;
      uint32_t cand = lo + ((hi - lo) >> 1);
      if (pass < 6 && pass % 3 != 2) {
        // aim a tenth past the target, so that the bound on the larger side moves
        float f = (float)(n_lo - want) / (float)(n_lo - n_hi);
        f = f > 0.5f ? fmaxf(0.5f, f - 0.1f) : fminf(0.5f, f + 0.1f);
        const float a = route_value(lo), b = route_value(hi);
        cand = min(max(route_key(fmaf(b - a, f, a)), lo + 1u), hi - 1u);
      }
      uint32_t n = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) n += key[i] >= cand;
      n = group_sum(n);
      if (n >= want) {
        lo = cand;
        n_lo = n;
      } else {
        hi = cand;
        n_hi = n;
      }
      if (n == want) {
        exact = true;
        break;
      }
    }
    if (W == 1 && V > 8 && !exact && hi - lo > 1u) {
      // the keys in [lo, hi), in any order, one a lane
      uint32_t c = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) c += key[i] - lo < hi - lo;
      uint32_t at = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += t;
      }
      at -= c;
      uint32_t* buf = few[warp];
      buf[lane] = 0u;                                     // below every key
      __syncwarp();
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (key[i] - lo < hi - lo) buf[at++] = key[i];
      __syncwarp();
      // rank of the lane's key among them: the one with fewer than the missing number of keys above it,
      // and at least as many at or above, is the cut
      const uint32_t mine = buf[lane], need = want - n_hi;
      uint32_t above = 0, from = 0;
#pragma unroll
      for (int j = 0; j < kRouteFew; j += 4) {
        const uint4 o = *reinterpret_cast<const uint4*>(buf + j);
        above += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
        from += (o.x >= mine) + (o.y >= mine) + (o.z >= mine) + (o.w >= mine);
      }
      const uint32_t who = __ballot_sync(0xffffffffu, above < need && need <= from);
      const int first = __ffs(who) - 1;
      lo = __shfl_sync(0xffffffffu, mine, first);
      n_hi += __shfl_sync(0xffffffffu, above, first);
      exact = __shfl_sync(0xffffffffu, from, first) == need;
    }
    cut = lo;
    if (!exact) {                                         // n_hi keys above lo, too few; the rest are lo
      ties = want - n_hi;
      tied = true;
    }
  }
  // positions in index order
  const uint32_t below = (1u << lane) - 1u;
  uint32_t pos = 0, tie = 0;                              // chosen and tied blocks before this warp's
  if constexpr (W > 1) {
    uint32_t n_above = 0, n_tie = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      n_above += tied ? key[i] > cut : key[i] >= cut;
      n_tie += tied && key[i] == cut;
    }
    n_above = __reduce_add_sync(0xffffffffu, n_above);
    n_tie = __reduce_add_sync(0xffffffffu, n_tie);
    uint32_t(*p)[8] = part[turn & 1];
    if (lane == 0) {
      p[1][warp] = n_above;
      p[2][warp] = n_tie;
    }
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
      tie += p[2][w];
      pos += p[1][w];
    }
    pos += min(tie, ties);
  }
  int* dst = list + (size_t)row * keep;
  if (tied) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool t = key[i] == cut;
      const uint32_t tm = __ballot_sync(0xffffffffu, t);
      const bool sel = t ? tie + __popc(tm & below) < ties : key[i] > cut;
      const uint32_t sm = __ballot_sync(0xffffffffu, sel);
      if (sel) dst[pos + __popc(sm & below)] = base + 32 * i + lane;
      pos += __popc(sm);
      tie += __popc(tm);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool sel = key[i] >= cut;
      const uint32_t sm = __ballot_sync(0xffffffffu, sel);
      if (sel) dst[pos + __popc(sm & below)] = base + 32 * i + lane;
      pos += __popc(sm);
    }
  }
  const uint32_t total = min(n_open, want);
  const int group_lane = W == 1 ? lane : (int)threadIdx.x;
  for (uint32_t i = total + group_lane; i < want; i += 32 * W) dst[i] = -1;
  if (group_lane == 0) count[row] = (int)total;
}

template <int W, int V>
static void launch_select(const float* s, int rows, int n_blocks, int keep, const uint8_t* f, int* list, int* count,
                          cudaStream_t st) {
  launch(k_block_select<W, V>, W == 1 ? (unsigned)(rows + 7) / 8 : (unsigned)rows, 256, 0, st, s, rows, n_blocks, keep,
         f, list, count);
}

}  // namespace hsa

using namespace hsa;

static inline int blocks_of(int n, int size) { return (n + size - 1) / size; }

extern "C" size_t hsa_block_scores_workspace_size(int M, int L, int H, int block_k) {
  if (M <= 0 || L <= 0 || H <= 0 || (block_k != 64 && block_k != 128)) return 0;
  return align256(((size_t)blocks_of(M, kRouteTile) + blocks_of(L, block_k)) * H * 128 * sizeof(float));
}

extern "C" int hsa_block_scores(const void* d_q, int M, const void* d_k, int L, int H, int dtype, int block_k,
                                float* d_scores, void* d_ws, size_t ws_bytes, void* stream) {
  if (dtype != HSA_BF16 && dtype != HSA_F32) return set_error(HSA_EINVAL, "block_scores: unknown dtype");
  if (M < 0 || L <= 0 || H <= 0 || H > 65535) return set_error(HSA_EINVAL, "block_scores: need M >= 0, L > 0 and H > 0");
  if (block_k != 64 && block_k != 128) return set_error(HSA_EINVAL, "block_scores: need block_k = 64 or 128");
  const int T = blocks_of(M, kRouteTile), B = blocks_of(L, block_k);
  if ((long long)T + B > 65535) return set_error(HSA_EINVAL, "block_scores: more than 65535 blocks");
  if (M == 0) return HSA_OK;
  if (!d_q || !d_k || !d_scores || !d_ws || !aligned16(d_q) || !aligned16(d_k) || !aligned16(d_ws))
    return set_error(HSA_EINVAL, "block_scores: null or misaligned pointer");
  if (ws_bytes < hsa_block_scores_workspace_size(M, L, H, block_k))
    return set_error(HSA_EWORKSPACE, "block_scores: workspace smaller than hsa_block_scores_workspace_size");
  cudaStream_t st = as_stream(stream);
  float* means = static_cast<float*>(d_ws);
  ScopedTiming timing(HSA_KCLASS_OTHER, st);
  const dim3 g1((unsigned)H, (unsigned)(T + B));
  if (dtype == HSA_BF16)
    launch(k_block_means<__nv_bfloat16>, g1, 256, 0, st, static_cast<const __nv_bfloat16*>(d_q), M,
           static_cast<const __nv_bfloat16*>(d_k), L, H, block_k, T, means);
  else
    launch(k_block_means<float>, g1, 256, 0, st, static_cast<const float*>(d_q), M, static_cast<const float*>(d_k), L,
           H, block_k, T, means);
  count_launch(1);
  int rc = check_launch("block means launch");
  if (rc) return rc;
  launch(k_block_product, dim3((unsigned)blocks_of(B, 64), (unsigned)blocks_of(T, 64), (unsigned)H), 256, 0, st, means,
         T, B, H, d_scores);
  count_launch(1);
  return check_launch("block product launch");
}

extern "C" int hsa_block_select(const float* d_scores, int rows, int n_blocks, int keep, const uint8_t* d_forced,
                                int32_t* d_list, int32_t* d_count, void* stream) {
  if (rows < 0 || n_blocks < 1 || n_blocks > kRouteMaxBlocks)
    return set_error(HSA_EINVAL, "block_select: need rows >= 0 and 1 <= n_blocks <= 16384");
  if (keep < 1 || keep > HSA_SPARSE_MAX_KEEP) return set_error(HSA_EINVAL, "block_select: need 1 <= keep <= 4096");
  if (rows == 0) return HSA_OK;
  if (!d_scores || !d_list || !d_count) return set_error(HSA_EINVAL, "block_select: null pointer");
  cudaStream_t st = as_stream(stream);
  ScopedTiming timing(HSA_KCLASS_OTHER, st);
  const int v = blocks_of(n_blocks, 32);
  if (v <= 4) launch_select<1, 4>(d_scores, rows, n_blocks, keep, d_forced, d_list, d_count, st);
  else if (v <= 8) launch_select<1, 8>(d_scores, rows, n_blocks, keep, d_forced, d_list, d_count, st);
  else if (v <= 16) launch_select<1, 16>(d_scores, rows, n_blocks, keep, d_forced, d_list, d_count, st);
  else if (v <= 40) launch_select<1, 40>(d_scores, rows, n_blocks, keep, d_forced, d_list, d_count, st);
  else if (v <= 64) launch_select<1, 64>(d_scores, rows, n_blocks, keep, d_forced, d_list, d_count, st);
  else if (v <= 128) launch_select<8, 16>(d_scores, rows, n_blocks, keep, d_forced, d_list, d_count, st);
  else launch_select<8, 64>(d_scores, rows, n_blocks, keep, d_forced, d_list, d_count, st);
  count_launch(1);
  return check_launch("block_select launch");
}
