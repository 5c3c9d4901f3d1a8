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
#include "tcgen05.cuh"

namespace hsa {

constexpr int kRouteTile = HSA_QUERY_TILE;

// 8 bf16 values as floats
__device__ __forceinline__ void widen8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// Mean rows.  Bound by the one read of Q and K, so the reads are TMA boxes of 64 rows x 512 bytes through a
// ring of six slots, one CTA per SM, 192 KB in flight.  An item is one block of rows x 512 bytes of columns,
// one or two boxes; the SMs walk the items side by side, so rows are read whole.  Warp 8 issues the loads;
// warps 0-7 take every eighth row of a box, 16 bytes of columns a lane, and leave their sums in shared
// memory; warps 9-10 join them and write the means while the next item is summed.  (Joined by the summing
// warps behind a barrier, every item cost them its latency: 79 against 72 us for 40950 rows of 5120 in blocks
// of 64; plain loads with eight in flight per warp: 42 us for 65520 rows of 1536, this 37, a bare TMA read
// without sums 33.)  Rows and columns beyond the matrix arrive as zeros.  Items [0, T) x columns are the
// query tiles, then the key blocks.  Sums in float32 (at most 128 terms).
constexpr int kMeanSlots = 6, kMeanBox = 64 * 512, kMeanParts = 3;
constexpr int kMeanThreads = 11 * 32;
struct MeanShared {
  uint64_t full[kMeanSlots], empty[kMeanSlots], part_full[kMeanParts], part_empty[kMeanParts];
  float part[kMeanParts][8][256];
};
constexpr int kMeanSmem = kMeanSlots * kMeanBox + 128 + (int)sizeof(MeanShared);

template <typename T>
__global__ void __launch_bounds__(kMeanThreads, 1)
    k_block_means(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK, int M, int L, int D,
                  int block_k, int n_tiles, int n_blocks, int n_items, int cols, __nv_bfloat16* __restrict__ means) {
  pdl_prologue();
  constexpr int V = 16 / (int)sizeof(T);                  // columns a lane
  extern __shared__ uint8_t mean_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(mean_raw) + 127) & ~uintptr_t(127));
  MeanShared* sh = reinterpret_cast<MeanShared*>(ring + kMeanSlots * kMeanBox);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMeanSlots; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], 8);
    }
    for (int s = 0; s < kMeanParts; ++s) {
      mbar_init(&sh->part_full[s], 8);
      mbar_init(&sh->part_empty[s], 2);
    }
    fence_mbar_init();
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
  }
  __syncthreads();
  int s = 0, ps = 0;
  uint32_t phase = 0, pphase = 0;
  bool good = true;
  for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
    const int j = item / cols, x = (item - j * cols) * 32 * V;
    const bool key = j >= n_tiles;
    const int size = key ? block_k : kRouteTile;
    const int r0 = (key ? j - n_tiles : j) * size;
    const int n = min(size, (key ? L : M) - r0);
    const int boxes = (n + 63) >> 6;
    if (warp == 8) {
      for (int b = 0; b < boxes; ++b) {
        good = mbar_wait_warp(&sh->empty[s], phase ^ 1u);
        if (!good) break;
        if (lane == 0) {
          mbar_expect_tx(&sh->full[s], kMeanBox);
          tma_load_2d(ring + s * kMeanBox, key ? &tmK : &tmQ, &sh->full[s], x, r0 + 64 * b);
        }
        __syncwarp();
        if (++s == kMeanSlots) {
          s = 0;
          phase ^= 1u;
        }
      }
    } else if (warp < 8) {
      float sum[V] = {};
      for (int b = 0; b < boxes; ++b) {
        good = mbar_wait_warp(&sh->full[s], phase);
        if (!good) break;
        const uint8_t* box = ring + s * kMeanBox + warp * 512 + lane * 16;
        uint4 raw[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) raw[i] = *reinterpret_cast<const uint4*>(box + i * 8 * 512);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float v[V];
          if constexpr (V == 8) {
            widen8(raw[i], v);
          } else {
            v[0] = __uint_as_float(raw[i].x); v[1] = __uint_as_float(raw[i].y);
            v[2] = __uint_as_float(raw[i].z); v[3] = __uint_as_float(raw[i].w);
          }
#pragma unroll
          for (int e = 0; e < V; ++e) sum[e] += v[e];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->empty[s]);
        if (++s == kMeanSlots) {
          s = 0;
          phase ^= 1u;
        }
      }
      if (good) good = mbar_wait_warp(&sh->part_empty[ps], pphase ^ 1u);
      if (!good) break;
#pragma unroll
      for (int e = 0; e < V; e += 4)
        st4(&sh->part[ps][warp][lane * V + e], make_float4(sum[e], sum[e + 1], sum[e + 2], sum[e + 3]));
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->part_full[ps]);
    } else {
      good = mbar_wait_warp(&sh->part_full[ps], pphase);
      if (!good) break;
      const int c = ((warp - 9) * 32 + lane) * 4;
      if (c < 32 * V) {
        float4 t = ld4(&sh->part[ps][0][c]);
#pragma unroll
        for (int w = 1; w < 8; ++w) {
          const float4 o = ld4(&sh->part[ps][w][c]);
          t = make_float4(t.x + o.x, t.y + o.y, t.z + o.z, t.w + o.w);
        }
        if (x + c < D) {
          // the mean as three bf16 terms, each the rounding of what the ones before leave (exact differences)
          const float cnt = (float)n;
          t = make_float4(t.x / cnt, t.y / cnt, t.z / cnt, t.w / cnt);
          const size_t plane = (size_t)(n_tiles + n_blocks) * D;
          __nv_bfloat16* dst = means + (size_t)j * D + x + c;
#pragma unroll
          for (int p = 0; p < 3; ++p) {
            uint2 u;
            u.x = pack_bf16x2(t.x, t.y);
            u.y = pack_bf16x2(t.z, t.w);
            *reinterpret_cast<uint2*>(dst + p * plane) = u;
            const float4 r = widen4(u);
            t = make_float4(t.x - r.x, t.y - r.y, t.z - r.z, t.w - r.w);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->part_empty[ps]);
    }
    if (!good) break;                                     // the loads' warp
    if (++ps == kMeanParts) {
      ps = 0;
      pphase ^= 1u;
    }
  }
  if (!good) stall_drain();
}

template <typename T>
static int launch_means(const void* q, int M, const void* k, int L, int H, int block_k, int n_tiles, int n_blocks,
                        __nv_bfloat16* means, cudaStream_t st) {
  constexpr bool bf = sizeof(T) == 2;
  const int D = H * 128, box_cols = 512 / (int)sizeof(T);
  CUtensorMap tq, tk;
  int rc = make_tmap_2d(&tq, q, bf, (uint64_t)D, (uint64_t)M, (uint64_t)D * sizeof(T), (uint32_t)box_cols, 64, false);
  if (!rc)
    rc = make_tmap_2d(&tk, k, bf, (uint64_t)D, (uint64_t)L, (uint64_t)D * sizeof(T), (uint32_t)box_cols, 64, false);
  if (rc) return rc;
  static PerContextOnce attr;
  rc = attr.ensure([](void**) {
    if (cudaFuncSetAttribute(k_block_means<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMeanSmem) != cudaSuccess)
      return check_launch("block_scores: shared-memory attribute");
    return (int)HSA_OK;
  });
  if (rc) return rc;
  const int cols = (D + box_cols - 1) / box_cols, items = cols * (n_tiles + n_blocks);
  launch(k_block_means<T>, (unsigned)(items < num_sms() ? items : num_sms()), kMeanThreads, kMeanSmem, st, tq, tk, M, L,
         D, block_k, n_tiles, n_blocks, items, cols, means);
  return HSA_OK;
}

// scores[h] = Qm[h] Km[h]^T / sqrt(128) on the tensor cores, with float32 accuracy: a mean x is kept as three
// bf16 terms, x = x0 + x1 + x2 with |x1| <= 2^-8 |x| and |x2| <= 2^-16 |x|, and the product takes the six
// pairs (i, j) with i + j <= 2; what is left out is below 2^-22 of the magnitudes.  A CUDA-core product
// (8 x 8 values a thread) took 12-19 us for the same sizes, and more with T x B.  CTA = 128 query tiles of a
// head against a range of its 64-block tiles: the three terms of the query side stay in shared memory, warp
// 0 loads the block tiles' terms (two buffers of 48 KB), warp 1 issues 48 MMAs a tile into one of two
// 64-column accumulators, warps 2-5 stage the other one in shared memory and write whole rows.
// A mean that is not finite gives NaN.
constexpr int kProdB = 3 * 64 * 128 * 2;                  // one block tile, three terms
constexpr int kProdStage = 32 * 65 * 4;                   // per epilogue warp
constexpr int kProdSmem = 3 * kTileBytes + 2 * kProdB + 4 * kProdStage + 1024;
__global__ void __launch_bounds__(192, 1)
    k_block_product(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, int n_tiles,
                    int n_blocks, float* __restrict__ scores) {
  pdl_prologue();
  extern __shared__ uint8_t prod_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(prod_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sB = smem + 3 * kTileBytes;
  __shared__ uint64_t a_full, b_full[2], b_empty[2], d_full[2], d_empty[2];
  __shared__ uint32_t tmem;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.z, t0 = blockIdx.y * 128;
  const int nb = (n_blocks + 63) >> 6;
  const int j0 = (int)((long long)blockIdx.x * nb / gridDim.x);
  const int nj = (int)((long long)(blockIdx.x + 1) * nb / gridDim.x) - j0;
  if (threadIdx.x == 0) {
    mbar_init(&a_full, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&b_full[b], 1);
      mbar_init(&b_empty[b], 1);
      mbar_init(&d_full[b], 1);
      mbar_init(&d_empty[b], 128);
    }
    fence_mbar_init();
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(&tmem, 128);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem;
  bool good = true;
  if (warp == 0) {
    const bool leader = elect_one();
    const int rows = n_tiles + n_blocks, x = h * 128;
    if (leader) {
      mbar_expect_tx(&a_full, 3 * kTileBytes);
      for (int p = 0; p < 3; ++p)
        for (int c = 0; c < 2; ++c)
          tma_load_2d(smem + p * kTileBytes + c * (kTileBytes / 2), &tmA, &a_full, x + 64 * c, p * rows + t0);
    }
    __syncwarp();
    for (int i = 0; i < nj; ++i) {
      const int b = i & 1;
      good = mbar_wait_warp(&b_empty[b], ((i >> 1) & 1) ^ 1);
      if (!good) break;
      if (leader) {
        mbar_expect_tx(&b_full[b], kProdB);
        for (int p = 0; p < 3; ++p)
          for (int c = 0; c < 2; ++c)
            tma_load_2d(sB + b * kProdB + p * (kProdB / 3) + c * (kProdB / 6), &tmB, &b_full[b], x + 64 * c,
                        p * rows + n_tiles + (j0 + i) * 64);
      }
      __syncwarp();
    }
  } else if (warp == 1) {
    const bool leader = elect_one();
    constexpr uint32_t idesc = idesc_bf16_f32(128, 64, false);
    const uint64_t ad = sdesc_sw128(smem_u32(smem), 16, 1024), bd = sdesc_sw128(smem_u32(sB), 16, 1024);
    good = mbar_wait_warp(&a_full, 0);
    for (int i = 0; good && i < nj; ++i) {
      const int b = i & 1;
      good = mbar_wait_warp(&b_full[b], (i >> 1) & 1) && mbar_wait_warp(&d_empty[b], ((i >> 1) & 1) ^ 1);
      if (!good) break;
      tc_fence_after();
      if (leader) {
        // smallest pairs first: (2,0) (1,1) (0,2) (1,0) (0,1) (0,0)
#pragma unroll
        for (int e = 0; e < 6; ++e) {
          constexpr int kP[6] = {2, 1, 0, 1, 0, 0}, kR[6] = {0, 1, 2, 0, 1, 0};
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_ss(tm + b * 64,
                    ad + (uint64_t)((kP[e] * kTileBytes + (kk >> 2) * (kTileBytes / 2) + (kk & 3) * 32) >> 4),
                    bd + (uint64_t)((b * kProdB + kR[e] * (kProdB / 3) + (kk >> 2) * (kProdB / 6) + (kk & 3) * 32) >> 4),
                    idesc, e > 0 || kk > 0);
        }
        umma_commit(&d_full[b]);
        umma_commit(&b_empty[b]);
      }
      __syncwarp();
    }
  } else {
    // thread = row of the tile; rows staged 65 floats apart, free of bank conflicts in both directions
    const int quarter = warp & 3;
    const float scale = 0.08838834764831845f;            // 1 / sqrt(128)
    float* stage = reinterpret_cast<float*>(sB + 2 * kProdB + quarter * kProdStage);
    const int rows = min(32, n_tiles - t0 - quarter * 32);
    for (int i = 0; i < nj; ++i) {
      const int b = i & 1, b0 = (j0 + i) * 64;
      good = mbar_wait_warp(&d_full[b], (i >> 1) & 1);
      if (!good) break;
      tc_fence_after();
      uint32_t v[64];
      tmem_ld32(tm + ((uint32_t)(quarter * 32) << 16) + b * 64, *reinterpret_cast<uint32_t(*)[32]>(v));
      tmem_ld32(tm + ((uint32_t)(quarter * 32) << 16) + b * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive(&d_empty[b]);
#pragma unroll
      for (int e = 0; e < 64; ++e) stage[lane * 65 + e] = __uint_as_float(v[e]) * scale;
      __syncwarp();
      float* dst = scores + ((size_t)h * n_tiles + t0 + quarter * 32) * n_blocks + b0;
      const bool in0 = b0 + lane < n_blocks, in1 = b0 + 32 + lane < n_blocks;
#pragma unroll 4
      for (int r = 0; r < rows; ++r) {
        if (in0) dst[(size_t)r * n_blocks + lane] = stage[r * 65 + lane];
        if (in1) dst[(size_t)r * n_blocks + 32 + lane] = stage[r * 65 + 32 + lane];
      }
      __syncwarp();
    }
  }
  if (!good) stall_drain();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tm, 128);
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

// One row of scores per group of W warps (W = 1: 8 rows a block; else the block is one group).  Warp w of the group
// holds blocks [w 32 V, (w + 1) 32 V) in registers, 32 consecutive ones at a time.
// The cut is searched between keys lo and hi with count(key >= lo) > keep > count(key >= hi): a pass counts
// the keys at or above a candidate and replaces one bound, and the search ends when the count is `keep`
// (a distinct cut) or hi = lo + 1 (ties at lo, given to the lowest index).  Scores are spread smoothly, so
// the first candidates interpolate between the bounds' values (about 5 passes until 32 of 1182 normal
// scores are left, against 11 by halving); every third one, and all after the sixth, halve the key
// interval, which bounds the passes whatever the scores.  Once at most 32 keys are left between the
// bounds, a warp with many registers of keys moves them to one register a lane and ranks them.
// Then the chosen blocks are written in index order.  Bound by instructions: a row of 1182 scores
// takes a warp about 3100, against 4.7 KB read (80 us for 23640 such rows; 309 by halving from keys loaded one
// by one).
template <int W, int V>
__global__ void __launch_bounds__(W == 1 ? 256 : 32 * W, W == 1 ? (V > 16 ? 3 : 4) : (V > 40 ? 8 : 24) / W)
    k_block_select(const float* __restrict__ scores, int rows, int n_blocks, int keep,
                   const uint8_t* __restrict__ forced, int* __restrict__ list, int* __restrict__ count) {
  pdl_prologue();
  __shared__ uint32_t part[2][3][W];
  __shared__ uint32_t fbits[W * V];
  __shared__ __align__(16) uint32_t few[W == 1 && V > 8 ? 8 : 1][kRouteFew];
  int turn = 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = W == 1 ? (int)blockIdx.x * 8 + warp : (int)blockIdx.x;
  if (forced) {
    // one bit per block, read by every row of the CTA
    for (int i = warp; i < W * V; i += (W == 1 ? 8 : W)) {
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
    uint32_t(*p)[W] = part[turn & 1];
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
    uint32_t(*p)[W] = part[turn & 1];
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
  launch(k_block_select<W, V>, W == 1 ? ((unsigned)rows + 7) / 8 : (unsigned)rows, W == 1 ? 256 : 32 * W, 0, st, s, rows,
         n_blocks, keep, f, list, count);
}

}  // namespace hsa

using namespace hsa;

static inline int blocks_of(int n, int size) { return n / size + (n % size != 0); }   // n + size may overflow

extern "C" size_t hsa_block_scores_workspace_size(int M, int L, int H, int block_k) {
  if (M <= 0 || L <= 0 || H <= 0 || (block_k != 64 && block_k != 128)) return 0;
  return align256(((size_t)blocks_of(M, kRouteTile) + blocks_of(L, block_k)) * H * 128 * 3 * sizeof(__nv_bfloat16));
}

extern "C" int hsa_block_scores(const void* d_q, int M, const void* d_k, int L, int H, int dtype, int block_k,
                                float* d_scores, void* d_ws, size_t ws_bytes, void* stream) {
  if (dtype != HSA_BF16 && dtype != HSA_F32) return set_error(HSA_EINVAL, "block_scores: unknown dtype");
  if (M < 0 || L <= 0 || H <= 0 || H > 4096) return set_error(HSA_EINVAL, "block_scores: need M >= 0, L > 0 and 0 < H <= 4096");
  if (block_k != 64 && block_k != 128) return set_error(HSA_EINVAL, "block_scores: need block_k = 64 or 128");
  const int T = blocks_of(M, kRouteTile), B = blocks_of(L, block_k);
  if ((long long)T + B > 65535) return set_error(HSA_EINVAL, "block_scores: more than 65535 blocks");
  if (M == 0) return HSA_OK;
  if (!d_q || !d_k || !d_scores || !d_ws || !aligned16(d_q) || !aligned16(d_k) || !aligned16(d_ws))
    return set_error(HSA_EINVAL, "block_scores: null or misaligned pointer");
  if (ws_bytes < hsa_block_scores_workspace_size(M, L, H, block_k))
    return set_error(HSA_EWORKSPACE, "block_scores: workspace smaller than hsa_block_scores_workspace_size");
  cudaStream_t st = as_stream(stream);
  __nv_bfloat16* means = static_cast<__nv_bfloat16*>(d_ws);
  ScopedTiming timing(HSA_KCLASS_OTHER, st);
  static PerContextOnce attr;
  int rc = attr.ensure([](void**) {
    if (cudaFuncSetAttribute(k_block_product, cudaFuncAttributeMaxDynamicSharedMemorySize, kProdSmem) != cudaSuccess)
      return check_launch("block_scores: shared-memory attribute");
    return (int)HSA_OK;
  });
  if (rc) return rc;
  rc = dtype == HSA_BF16 ? launch_means<__nv_bfloat16>(d_q, M, d_k, L, H, block_k, T, B, means, st)
                         : launch_means<float>(d_q, M, d_k, L, H, block_k, T, B, means, st);
  if (rc) return rc;
  count_launch(1);
  rc = check_launch("block means launch");
  if (rc) return rc;
  CUtensorMap ta, tb;
  const uint64_t planes = 3 * (uint64_t)(T + B);
  rc = make_tmap_2d(&ta, means, true, (uint64_t)H * 128, planes, (uint64_t)H * 256, 64, 128, true);
  if (!rc) rc = make_tmap_2d(&tb, means, true, (uint64_t)H * 128, planes, (uint64_t)H * 256, 64, 64, true);
  if (rc) return rc;
  // ranges of block tiles: as many CTAs as SMs while a head's 128 query tiles leave some idle (one range a
  // head: 48.8 against 42.8 us for the whole call at 32760 x 32760, 12 heads), else ranges of about twelve
  // tiles, the query side being loaded once per range (three / six / twelve: 366 / 354 / 345 us at 75600 x
  // 75600, 40 heads)
  const int tiles_b = blocks_of(B, 64), units = blocks_of(T, 128) * H, few = blocks_of(tiles_b, 12);
  int ranges = num_sms() / units > few ? num_sms() / units : few;
  ranges = ranges > tiles_b ? tiles_b : ranges;
  launch(k_block_product, dim3((unsigned)ranges, (unsigned)blocks_of(T, 128), (unsigned)H), 192, kProdSmem, st, ta, tb,
         T, B, d_scores);
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
  // Warps a row and keys a lane: one warp up to 1280 blocks, two up to 2560, four up to 4096, with at most 40 keys
  // a lane (64 leave an SM too few warps: 24 million scores in rows of 1500 122 us, with two warps of 24 79) and
  // the next size of the register array; beyond that eight warps, of 32 keys up to 8192 blocks and of 64 above.
  // At 80 registers a thread the arrays of 40 spill 96 to 148 bytes a thread, the smaller ones at most 64.
  const int v = blocks_of(n_blocks, 32);
  if (v <= 2) launch_select<1, 2>(d_scores, rows, n_blocks, keep, d_forced, d_list, d_count, st);
  else if (v <= 4) launch_select<1, 4>(d_scores, rows, n_blocks, keep, d_forced, d_list, d_count, st);
  else if (v <= 8) launch_select<1, 8>(d_scores, rows, n_blocks, keep, d_forced, d_list, d_count, st);
  else if (v <= 12) launch_select<1, 12>(d_scores, rows, n_blocks, keep, d_forced, d_list, d_count, st);
  else if (v <= 16) launch_select<1, 16>(d_scores, rows, n_blocks, keep, d_forced, d_list, d_count, st);
  else if (v <= 24) launch_select<1, 24>(d_scores, rows, n_blocks, keep, d_forced, d_list, d_count, st);
  else if (v <= 32) launch_select<1, 32>(d_scores, rows, n_blocks, keep, d_forced, d_list, d_count, st);
  else if (v <= 40) launch_select<1, 40>(d_scores, rows, n_blocks, keep, d_forced, d_list, d_count, st);
  else if (v <= 2 * 24) launch_select<2, 24>(d_scores, rows, n_blocks, keep, d_forced, d_list, d_count, st);
  else if (v <= 2 * 32) launch_select<2, 32>(d_scores, rows, n_blocks, keep, d_forced, d_list, d_count, st);
  else if (v <= 2 * 40) launch_select<2, 40>(d_scores, rows, n_blocks, keep, d_forced, d_list, d_count, st);
  else if (v <= 4 * 24) launch_select<4, 24>(d_scores, rows, n_blocks, keep, d_forced, d_list, d_count, st);
  else if (v <= 4 * 32) launch_select<4, 32>(d_scores, rows, n_blocks, keep, d_forced, d_list, d_count, st);
  else if (v <= 8 * 32) launch_select<8, 32>(d_scores, rows, n_blocks, keep, d_forced, d_list, d_count, st);
  else launch_select<8, 64>(d_scores, rows, n_blocks, keep, d_forced, d_list, d_count, st);
  count_launch(1);
  return check_launch("block_select launch");
}
