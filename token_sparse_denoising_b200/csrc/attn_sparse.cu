// attn_sparse.cu -- attention of compacted queries over listed blocks of the KV cache
// (hsa_sparse_attention): for the rows of query tile t (128 compacted rows) and head h
//   o = softmax(q K_S^T / sqrt(128)) V_S,   S = the keys of blocks list[h][t][0 .. count[h][t]),
// 0 for a row whose list is empty.  Blocks are 64 or 128 consecutive cache rows.
//
// bf16 kernel: CTA = one (query tile, head) unit, or one range of its list.  The tile
// schedule is that of the full-context kernel (attn_tc.cu): warp 0 loads tiles by TMA, warp 1 issues
// the MMAs, warps 2-5 and 6-9 run the softmax of the even and the odd tiles, each parity with its own
// running max, sum and O accumulator in TMEM.  What differs is where a tile's 128 keys come from: one
// listed 128-row block (two 64-column boxes) or two listed 64-row blocks (four 64 x 64 boxes), so a
// finer list costs only more TMA instructions, and the tensor-core shapes stay 128 x 128 x 128.
// The CTA's part of the list is staged in shared memory as first rows of blocks before the pipeline
// starts; L stands for "no block" (padding of an odd list, an index outside [0, blocks)), which TMA
// fills with zeros and the softmax masks to -inf.  The stages' row numbers also tell the softmax which
// tiles need a mask at all (the ragged last block may stand anywhere in a list).
//
// Rounding: logits, running max and sum, and O are float32; p is rounded to bf16 for the second
// product (its sum is taken before the rounding, relative error 2^-9 per term), and O once at the end.
#include "tcgen05.cuh"

namespace hsa {

struct SparseShared {
  uint64_t q_full;
  uint64_t k_full[2], k_empty[3];
  uint64_t v_empty[2];
  uint64_t s_full[2], p_full[2][2], o_done;
  uint32_t tmem;
  float xm[2][128], xl[2][128];
};

constexpr int kSpThreads = 64 + 256;
constexpr int kSpKSlots = 3, kSpVSlots = 2;
constexpr uint32_t kSpColS = 0, kSpColO = 256, kSpCols = 512;
constexpr int kSpTilesBytes = kTileBytes * (1 + kSpKSlots + kSpVSlots);
constexpr int kSpSmemFixed = kSpTilesBytes + 1024 + (int)sizeof(SparseShared);
static_assert(kSpSmemFixed + 4 * (HSA_SPARSE_MAX_KEEP + 2) <= 227 * 1024, "the longest list must fit shared memory");

struct SparseList {
  const int* list;    // [H][QT][keep]
  const int* count;   // [H][QT]
  int keep, block, n_blocks;
};

// Blocks listed for a unit (clamped to [0, keep])
__device__ __forceinline__ int listed_blocks(const SparseList& s, size_t unit) {
  const int n = s.count[unit];
  if (n < 0 || n > s.keep) {
    if (threadIdx.x == 0) flag_error(HSA_EINDEX);
    return n < 0 ? 0 : s.keep;
  }
  return n;
}

// First cache row of each listed block of [first, first + n) into rows[0, n), L for a bad index
__device__ __forceinline__ void stage_rows(const SparseList& s, size_t unit, int first, int n, int L, int* rows) {
  const int* src = s.list + unit * s.keep + first;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int b = src[i];
    const bool ok = b >= 0 && b < s.n_blocks;
    if (!ok) flag_error(HSA_EINDEX);
    rows[i] = ok ? b * s.block : L;
  }
}

__global__ void __launch_bounds__(kSpThreads, 1)
    k_attn_sparse(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, int M, int L, int H, __nv_bfloat16* __restrict__ O,
                  const AttnGrid grid, const SparseList sl) {
  pdl_prologue();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = smem + kTileBytes;
  uint8_t* sV = sK + kSpKSlots * kTileBytes;
  SparseShared* sh = reinterpret_cast<SparseShared*>(sV + kSpVSlots * kTileBytes);
  int* rows = reinterpret_cast<int*>(sh + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int u = blockIdx.x, split = 0, n_split = 1, slot = -1;
  if (u >= grid.u_full) {
    const int t = u - grid.u_full;
    u = grid.u_full + t / grid.s_tail;
    split = t % grid.s_tail;
    n_split = grid.s_tail;
    if (n_split > 1) slot = t;
  }
  const int m0 = (u % grid.QT) * kAttnBM, h = u / grid.QT;
  const bool halves = sl.block == 64;                     // two blocks per 128-key tile
  const int n_list = listed_blocks(sl, (size_t)u);
  const int nt_all = halves ? (n_list + 1) >> 1 : n_list;
  const int j0 = (int)((long long)split * nt_all / n_split);
  const int nt = (int)((long long)(split + 1) * nt_all / n_split) - j0;

  if (nt == 0) {                                          // nothing listed: the rows are 0 (or add nothing)
    if (slot >= 0) {
      if (threadIdx.x < kAttnBM) grid.part_ml[(size_t)slot * kAttnBM + threadIdx.x] = make_float2(-INFINITY, 0.f);
    } else {
      const uint4 z = make_uint4(0u, 0u, 0u, 0u);
      for (int i = threadIdx.x; i < kAttnBM * 16; i += kSpThreads) {
        const int r = m0 + (i >> 4);
        if (r < M) *reinterpret_cast<uint4*>(O + (size_t)r * (H * 128) + h * 128 + (i & 15) * 8) = z;
      }
    }
    return;
  }

  if (threadIdx.x == 0) {
    mbar_init(&sh->q_full, 1);
    for (int s = 0; s < kSpKSlots; ++s) mbar_init(&sh->k_empty[s], 1);
    for (int s = 0; s < kSpVSlots; ++s) mbar_init(&sh->v_empty[s], 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh->k_full[b], 1);
      mbar_init(&sh->s_full[b], 1);
      mbar_init(&sh->p_full[b][0], 129);   // the parity's 128 softmax threads + the producer
      mbar_init(&sh->p_full[b][1], 129);
    }
    mbar_init(&sh->o_done, 1);
    fence_mbar_init();
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  {
    const int per = halves ? 2 : 1, first = j0 * per;
    const int n = min(nt * per, n_list - first);
    stage_rows(sl, (size_t)u, first, n, L, rows);
    if (threadIdx.x == 0 && n < nt * per) rows[n] = L;
  }
  if (warp == 1) {
    tmem_alloc(&sh->tmem, kSpCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = sh->tmem;

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    const int x0 = h * 128;
    const bool leader = elect_one();
    // the 128 keys of local tile t, 32 KB completing on `bar`
    auto load_tile = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int t) {
      mbar_expect_tx(bar, kTileBytes);
      if (halves) {
        const int r0 = rows[2 * t], r1 = rows[2 * t + 1];
        tma_load_2d(dst, map, bar, x0, r0);
        tma_load_2d(dst + kTileBytes / 4, map, bar, x0, r1);
        tma_load_2d(dst + kTileBytes / 2, map, bar, x0 + 64, r0);
        tma_load_2d(dst + 3 * (kTileBytes / 4), map, bar, x0 + 64, r1);
      } else {
        tma_load_2d(dst, map, bar, x0, rows[t]);
        tma_load_2d(dst + kTileBytes / 2, map, bar, x0 + 64, rows[t]);
      }
    };
    if (leader) {
      mbar_expect_tx(&sh->q_full, kTileBytes);
      tma_load_2d(sQ, &tmQ, &sh->q_full, x0, m0);
      tma_load_2d(sQ + kTileBytes / 2, &tmQ, &sh->q_full, x0 + 64, m0);
    }
    auto load_k = [&](int j, uint64_t* bar) -> bool {
      const int sk = j % kSpKSlots;
      const bool ok = __shfl_sync(0xffffffffu, mbar_wait(&sh->k_empty[sk], ((j / kSpKSlots) & 1) ^ 1), 0);
      __syncwarp();
      if (ok && leader) load_tile(sK + sk * kTileBytes, &tmK, bar, j);
      return ok;
    };
    bool ok = load_k(0, &sh->k_full[0]);
    if (ok && nt > 1) ok = load_k(1, &sh->k_full[1]);
    // Phase order of the p_full arrivals: the producer arrives on phase t / 2 of p_full[t % 2][*] only
    // after waiting for a ring slot that the MMA warp releases after it waited on the previous phase
    // of the same barrier, so no arrival lands a phase early
    for (int t = 0; ok && t < nt; ++t) {
      const int b = t & 1, sv = t % kSpVSlots;
      ok = __shfl_sync(0xffffffffu, mbar_wait(&sh->v_empty[sv], ((t / kSpVSlots) & 1) ^ 1), 0);
      __syncwarp();
      if (!ok) break;
      if (leader) load_tile(sV + sv * kTileBytes, &tmV, &sh->p_full[b][0], t);
      if (t + 2 < nt) {
        ok = load_k(t + 2, &sh->p_full[b][1]);
      } else {
        if (leader) mbar_arrive(&sh->p_full[b][1]);
        __syncwarp();
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, false);
    constexpr uint32_t idesc_o = idesc_bf16_f32(128, 128, true);
    const bool leader = elect_one();
    const uint64_t q_desc = sdesc_sw128(smem_u32(sQ), 16, 1024);
    const uint64_t k_desc = sdesc_sw128(smem_u32(sK), 16, 1024);
    const uint64_t v_desc = sdesc_sw128(smem_u32(sV), kTileBytes / 2, 1024);
    auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
      const bool r = __shfl_sync(0xffffffffu, mbar_wait(bar, parity), 0);
      __syncwarp();
      return r;
    };
    auto issue_qk = [&](int t) -> bool {
      const int sk = t % kSpKSlots, b = t & 1;
      if (t < 2 && !wait_all(&sh->k_full[t], 0)) return false;
      tc_fence_after();
      const uint64_t kd = k_desc + (uint64_t)((sk * kTileBytes) >> 4);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = ((kk >> 2) * (kTileBytes / 2) + (kk & 3) * 32) >> 4;
          umma_ss(tm + kSpColS + b * 128, q_desc + off, kd + off, idesc_s, kk > 0);
        }
        umma_commit(&sh->s_full[b]);
        umma_commit(&sh->k_empty[sk]);
      }
      __syncwarp();
      return true;
    };
    bool ok = wait_all(&sh->q_full, 0);
    if (ok) ok = issue_qk(0);
    if (ok && nt > 1) ok = issue_qk(1);
    for (int t = 0; ok && t < nt; ++t) {
      const int b = t & 1, sv = t % kSpVSlots;
      const uint64_t vd = v_desc + (uint64_t)((sv * kTileBytes) >> 4);
      bool got = true;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (!wait_all(&sh->p_full[b][q], (t / 2) & 1)) { got = false; break; }
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int kk = q * 4; kk < q * 4 + 4; ++kk)
            umma_ts(tm + kSpColO + b * 128, tm + kSpColS + b * 128 + kk * 8, vd + (uint64_t)(kk * 2048 >> 4), idesc_o,
                    (t >= 2 || kk > 0));
          if (q == 1) umma_commit(&sh->v_empty[sv]);
        }
        __syncwarp();
      }
      if (!got) break;
      if (t + 2 < nt) ok = issue_qk(t + 2);
    }
    if (leader) umma_commit(&sh->o_done);
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax warps
    const int quarter = warp & 3;
    const int par = (warp - 2) >> 2;
    const int row = quarter * 32 + lane;
    const uint32_t lane_base = tm + ((uint32_t)(quarter * 32) << 16);
    const uint32_t s_col = lane_base + kSpColS + par * 128, o_col = lane_base + kSpColO + par * 128;
    const float sc = 0.12751743074680484f;               // log2(e) / sqrt(128)
    float m = -INFINITY, l = 0.f;
    for (int t = par; t < nt; t += 2) {
      // keys of the tile's two 64-key halves that exist (64 or more: all)
      const int v0 = L - (halves ? rows[2 * t] : rows[t]);
      const int v1 = halves ? L - rows[2 * t + 1] : v0 - 64;
      mbar_wait(&sh->s_full[par], (t / 2) & 1);
      __syncwarp();
      tc_fence_after();
      uint32_t sr[128];
#pragma unroll
      for (int q4 = 0; q4 < 4; ++q4)
        tmem_ld32(s_col + q4 * 32, *reinterpret_cast<uint32_t(*)[32]>(sr + q4 * 32));
      tmem_ld_wait();
      if (v0 < 64 || v1 < 64) {
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          if (c >= v0) sr[c] = __float_as_uint(-INFINITY);
          if (c >= v1) sr[64 + c] = __float_as_uint(-INFINITY);
        }
      }
      float mx8[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) mx8[e] = __uint_as_float(sr[e]);
#pragma unroll
      for (int c = 8; c < 128; c += 2)
        mx8[(c >> 1) & 7] = fmax3(mx8[(c >> 1) & 7], __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
      const float m_tile = sc * fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                                      fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
      // lazy rescale: the max moves only when it grew by more than 2^8
      bool need = false;
      float corr = 1.0f;
      if (t == par) {
        m = m_tile;
      } else if (m_tile > m + 8.0f) {
        need = true;
        corr = ex2_approx(m - m_tile);
        l *= corr;
        m = m_tile;
      }
      const bool any_need = __any_sync(0xffffffffu, need);
      const float neg_m = m == -INFINITY ? 0.f : -m;      // no key so far: every p is 2^-inf = 0
      const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(neg_m, neg_m);
      float2 rs4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        uint32_t pk[32];
#pragma unroll
        for (int c = hh * 64; c < hh * 64 + 64; c += 2) {
          const float2 x = ffma2(make_float2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), sc2, nm2);
          const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
          rs4[(c >> 1) & 3] = fadd2(rs4[(c >> 1) & 3], make_float2(p0, p1));
          pk[(c >> 1) & 31] = pack_bf16x2(p0, p1);
          if ((c & 31) == 30) tmem_st16(s_col + (c >> 5) * 16, pk + ((c >> 1) & 31) - 15);
          if (hh == 1 && c == 66 && !any_need) {
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&sh->p_full[par][0]);
          }
        }
      }
      l += ((rs4[0].x + rs4[0].y) + (rs4[1].x + rs4[1].y)) + ((rs4[2].x + rs4[2].y) + (rs4[3].x + rs4[3].y));
      if (any_need) {
        // O of this parity holds the PV of its previous tiles, complete: S was written by an MMA issued
        // after them, and PV of this tile starts only after the p_full arrivals below
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          tmem_ld32(o_col + c * 32, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
          tmem_st32(o_col + c * 32, o);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      if (any_need) mbar_arrive(&sh->p_full[par][0]);
      mbar_arrive(&sh->p_full[par][1]);
    }
    // ---------------------------------------------------------------- epilogue: merge the parities
    sh->xm[par][row] = m;
    sh->xl[par][row] = l;
    named_bar_sync(1 + quarter, 64);
    const bool two = nt >= 2;
    const float m0v = sh->xm[0][row], m1v = sh->xm[1][row];
    const float mm = two ? fmaxf(m0v, m1v) : m0v;
    const float ms = mm == -INFINITY ? 0.f : mm;          // no key at all: weights 0
    const float a0 = ex2_approx(m0v - ms);
    const float a1 = two ? ex2_approx(m1v - ms) : 0.f;
    const float den = a0 * sh->xl[0][row] + (two ? a1 * sh->xl[1][row] : 0.f);
    const float inv_l = den > 0.f ? 1.0f / den : 0.f;
    const float w0 = slot >= 0 ? a0 : a0 * inv_l, w1 = slot >= 0 ? a1 : a1 * inv_l;
    mbar_wait(&sh->o_done, 0);
    __syncwarp();
    tc_fence_after();
    const int grow = m0 + row;
    if (slot >= 0 && par == 0) grid.part_ml[(size_t)slot * kAttnBM + row] = make_float2(mm, den);
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
      const uint32_t col = (uint32_t)(par * 64 + c * 32);
      uint32_t o0[32], o1[32];
      __syncwarp();
      tmem_ld32(lane_base + kSpColO + col, o0);
      if (two) tmem_ld32(lane_base + kSpColO + 128 + col, o1);
      tmem_ld_wait();
      if (!two) {
#pragma unroll
        for (int e = 0; e < 32; ++e) o1[e] = 0u;
      }
      float f[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) f[e] = fmaf(__uint_as_float(o0[e]), w0, __uint_as_float(o1[e]) * w1);
      if (slot >= 0) {
        float* dst = grid.part_o + ((size_t)slot * kAttnBM + row) * 128 + col;
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          *reinterpret_cast<float4*>(dst + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
      } else if (grow < M) {
        __nv_bfloat16* dst = O + (size_t)grow * (H * 128) + h * 128 + col;
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          uint4 pk4;
          pk4.x = pack_bf16x2(f[e], f[e + 1]);
          pk4.y = pack_bf16x2(f[e + 2], f[e + 3]);
          pk4.z = pack_bf16x2(f[e + 4], f[e + 5]);
          pk4.w = pack_bf16x2(f[e + 6], f[e + 7]);
          *reinterpret_cast<uint4*>(dst + e) = pk4;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tm, kSpCols);
  }
}

// Merge of the list ranges of the split units, as k_attn_combine; a range without keys has sum 0 and
// wrote no O.  One warp per (unit, row), lane = 4 channels.
__global__ void __launch_bounds__(256) k_attn_sparse_combine(const float* __restrict__ part_o,
                                                             const float2* __restrict__ part_ml, int n_tail,
                                                             int s_tail, int u_full, int QT, int M, int H,
                                                             __nv_bfloat16* __restrict__ O) {
  pdl_prologue();
  const int w = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
  const int tu = w / kAttnBM, row = w % kAttnBM;
  if (tu >= n_tail) return;
  const int u = u_full + tu, grow = (u % QT) * kAttnBM + row, h = u / QT;
  if (grow >= M) return;
  float mx = -INFINITY;
  for (int sp = 0; sp < s_tail; ++sp) mx = fmaxf(mx, part_ml[(size_t)(tu * s_tail + sp) * kAttnBM + row].x);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float den = 0.f;
  for (int sp = 0; sp < s_tail; ++sp) {
    const size_t r = (size_t)(tu * s_tail + sp) * kAttnBM + row;
    const float2 ml = part_ml[r];
    if (ml.y == 0.f) continue;
    const float a = exp2f(ml.x - mx);
    den = fmaf(a, ml.y, den);
    const float4 o = ld4(part_o + r * 128 + lane * 4);
    acc = make_float4(fmaf(a, o.x, acc.x), fmaf(a, o.y, acc.y), fmaf(a, o.z, acc.z), fmaf(a, o.w, acc.w));
  }
  const float inv = den > 0.f ? 1.0f / den : 0.f;
  store4(O + (size_t)grow * (H * 128) + h * 128 + lane * 4,
         make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
}

// ------------------------------------------------------------------ float32, CUDA cores
// The full-context fp32 kernel's tiling (k_attn_f32: 32 query rows per CTA, 64-key tiles) over the list
// of the rows' query tile; a 128-row block is two tiles.
__global__ void __launch_bounds__(256, 2)
    k_attn_sparse_f32(const float* __restrict__ Q, int M, const float* __restrict__ K, const float* __restrict__ V,
                      int L, int H, int n_split, const SparseList sl, float* __restrict__ O,
                      float* __restrict__ part_o, float2* __restrict__ part_ml) {
  pdl_prologue();
  extern __shared__ float4 sm4[];
  float* Qs = reinterpret_cast<float*>(sm4);
  float* Ks = Qs + kF32BQ * kF32Ld;
  float* Vs = Ks + kF32BK * kF32Ld;
  float* Ps = Vs + kF32BK * kF32Ld;
  constexpr int kPsLd = kF32BK + 4;
  int* rows = reinterpret_cast<int*>(Ps + kF32BQ * kPsLd);
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int QB = (M + kF32BQ - 1) / kF32BQ, QT = (M + HSA_QUERY_TILE - 1) / HSA_QUERY_TILE;
  int b = blockIdx.x;
  const int split = b % n_split;
  b /= n_split;
  const int qb = b % QB, h = b / QB;
  const int D = H * 128, m0 = qb * kF32BQ;
  const size_t unit = (size_t)h * QT + m0 / HSA_QUERY_TILE;
  const int n_list = listed_blocks(sl, unit);
  const int per = sl.block / kF32BK;                      // tiles per block
  const int i0 = (int)((long long)split * n_list / n_split);
  const int i1 = (int)((long long)(split + 1) * n_list / n_split);
  stage_rows(sl, unit, i0, i1 - i0, L, rows);
  for (int i = tid; i < kF32BQ * 32; i += 256) {
    const int r = i >> 5, c4 = i & 31;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (m0 + r < M) v = ld4(Q + (size_t)(m0 + r) * D + h * 128 + 4 * c4);
    st4(Qs + r * kF32Ld + 4 * c4, v);
  }
  const float scale = 0.08838834764831845f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float o[2][8];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int c = 0; c < 8; ++c) o[i][c] = 0.f;
  const float* q0r = Qs + (2 * ty) * kF32Ld;
  const float* q1r = q0r + kF32Ld;
  const int nt = (i1 - i0) * per;
  for (int t = 0; t < nt; ++t) {
    __syncthreads();                                      // rows staged; the previous tile's reads are done
    const int k0 = per == 1 ? rows[t] : rows[t >> 1] + (t & 1) * kF32BK;
    for (int i = tid; i < kF32BK * 32; i += 256) {
      const int key = i >> 5, c4 = i & 31;
      float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
      if (k0 + key < L) {
        kv = ld4(K + (size_t)(k0 + key) * D + h * 128 + 4 * c4);
        vv = ld4(V + (size_t)(k0 + key) * D + h * 128 + 4 * c4);
      }
      st4(Ks + key * kF32Ld + 4 * c4, kv);
      st4(Vs + key * kF32Ld + 4 * c4, vv);
    }
    __syncthreads();
    float s[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int c = 0; c < 128; c += 4) {
      const float4 a0 = ld4(q0r + c), a1 = ld4(q1r + c);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 kk = ld4(Ks + (tx + 16 * j) * kF32Ld + c);
        s[0][j] = fmaf(a0.x, kk.x, fmaf(a0.y, kk.y, fmaf(a0.z, kk.z, fmaf(a0.w, kk.w, s[0][j]))));
        s[1][j] = fmaf(a1.x, kk.x, fmaf(a1.y, kk.y, fmaf(a1.z, kk.z, fmaf(a1.w, kk.w, s[1][j]))));
      }
    }
    float corr[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = (k0 + tx + 16 * j < L) ? s[i][j] * scale : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float m_new = fmaxf(m[i], mx);
      const float m_ref = m_new == -INFINITY ? 0.f : m_new;   // no key so far: every weight is 0
      corr[i] = expf(m[i] - m_ref);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = expf(s[i][j] - m_ref);
        sum += p;
        Ps[(2 * ty + i) * kPsLd + tx + 16 * j] = p;
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      l[i] = l[i] * corr[i] + sum;
      m[i] = m_new;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < 8; ++c) o[i][c] *= corr[i];
    const float* p0r = Ps + (2 * ty) * kPsLd;
    const float* p1r = p0r + kPsLd;
#pragma unroll 4
    for (int key = 0; key < kF32BK; ++key) {
      const float p0 = p0r[key], p1 = p1r[key];
      const float4 va = ld4(Vs + key * kF32Ld + 8 * tx), vb = ld4(Vs + key * kF32Ld + 8 * tx + 4);
      const float vv[8] = {va.x, va.y, va.z, va.w, vb.x, vb.y, vb.z, vb.w};
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        o[0][c] = fmaf(p0, vv[c], o[0][c]);
        o[1][c] = fmaf(p1, vv[c], o[1][c]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = 2 * ty + i, grow = m0 + row;
    if (grow >= M) continue;
    if (n_split == 1) {
      const float inv = l[i] > 0.f ? 1.0f / l[i] : 0.f;
      float* dst = O + (size_t)grow * D + h * 128 + 8 * tx;
      st4(dst, make_float4(o[i][0] * inv, o[i][1] * inv, o[i][2] * inv, o[i][3] * inv));
      st4(dst + 4, make_float4(o[i][4] * inv, o[i][5] * inv, o[i][6] * inv, o[i][7] * inv));
    } else {
      const size_t slot = (size_t)blockIdx.x * kF32BQ + row;
      float* dst = part_o + slot * 128 + 8 * tx;
      st4(dst, make_float4(o[i][0], o[i][1], o[i][2], o[i][3]));
      st4(dst + 4, make_float4(o[i][4], o[i][5], o[i][6], o[i][7]));
      if (tx == 0) part_ml[slot] = make_float2(m[i], l[i]);
    }
  }
}

__global__ void __launch_bounds__(256) k_attn_sparse_f32_combine(const float* __restrict__ part_o,
                                                                 const float2* __restrict__ part_ml, int M, int H,
                                                                 int n_split, float* __restrict__ O) {
  pdl_prologue();
  const int w = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
  const int QB = (M + kF32BQ - 1) / kF32BQ;
  const int row = w % kF32BQ, unit = w / kF32BQ;
  if (unit >= QB * H) return;
  const int qb = unit % QB, h = unit / QB, grow = qb * kF32BQ + row;
  if (grow >= M) return;
  float mx = -INFINITY;
  for (int s = 0; s < n_split; ++s) mx = fmaxf(mx, part_ml[((size_t)unit * n_split + s) * kF32BQ + row].x);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float den = 0.f;
  for (int s = 0; s < n_split; ++s) {
    const size_t slot = ((size_t)unit * n_split + s) * kF32BQ + row;
    const float2 ml = part_ml[slot];
    if (ml.y == 0.f) continue;
    const float a = expf(ml.x - mx);
    den = fmaf(a, ml.y, den);
    const float4 v = ld4(part_o + slot * 128 + 4 * lane);
    acc = make_float4(fmaf(a, v.x, acc.x), fmaf(a, v.y, acc.y), fmaf(a, v.z, acc.z), fmaf(a, v.w, acc.w));
  }
  const float inv = den > 0.f ? 1.0f / den : 0.f;
  st4(O + (size_t)grow * (H * 128) + h * 128 + 4 * lane,
      make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
}

// ------------------------------------------------------------------ host
namespace {
int sparse_tiles(int keep, int block) { return block == 64 ? (keep + 1) / 2 : keep; }

int sparse_bf16(const void* Q, int M, const void* K, const void* V, int L, int H, const SparseList& sl, void* O,
                void* ws, size_t ws_bytes, cudaStream_t st) {
  const uint64_t D = (uint64_t)H * 128;
  CUtensorMap tq, tk, tv;
  int rc = make_tmap_2d(&tq, Q, true, D, (uint64_t)M, D * 2, 64, kAttnBM, true);
  if (!rc) rc = make_tmap_2d(&tk, K, true, D, (uint64_t)L, D * 2, 64, (uint32_t)sl.block, true);
  if (!rc) rc = make_tmap_2d(&tv, V, true, D, (uint64_t)L, D * 2, 64, (uint32_t)sl.block, true);
  if (rc) return rc;
  static PerContextOnce attr;
  rc = attr.ensure([](void**) {
    if (cudaFuncSetAttribute(k_attn_sparse, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSpSmemFixed + 4 * (HSA_SPARSE_MAX_KEEP + 2)) != cudaSuccess)
      return check_launch("sparse attention: shared-memory attribute");
    return (int)HSA_OK;
  });
  if (rc) return rc;
  const int QT = (M + kAttnBM - 1) / kAttnBM, U = QT * H;
  TailSplit ts = plan_tail(U, sparse_tiles(sl.keep, sl.block), num_sms());
  const size_t need = tail_split_bytes(ts);
  if (need == 0 || !ws || ws_bytes < need) ts = TailSplit{U, 1, 0};
  AttnGrid g{QT, ts.u_full, ts.s_tail, nullptr, nullptr};
  if (ts.s_tail > 1) {
    const size_t slots = (size_t)ts.n_tail * ts.s_tail * kAttnBM;
    g.part_o = static_cast<float*>(ws);
    g.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + align256(slots * 128 * sizeof(float)));
  }
  ScopedTiming timing(HSA_KCLASS_ATTENTION, st);
  launch(k_attn_sparse, (unsigned)(ts.u_full + ts.n_tail * ts.s_tail), kSpThreads, kSpSmemFixed + 4 * (sl.keep + 2), st,
         tq, tk, tv, M, L, H, reinterpret_cast<__nv_bfloat16*>(O), g, sl);
  count_launch(1);
  rc = check_launch("sparse attention launch");
  if (rc || ts.s_tail == 1) return rc;
  launch(k_attn_sparse_combine, (unsigned)((ts.n_tail * kAttnBM + 7) / 8), 256, 0, st, g.part_o, g.part_ml, ts.n_tail,
         ts.s_tail, ts.u_full, QT, M, H, reinterpret_cast<__nv_bfloat16*>(O));
  count_launch(1);
  return check_launch("sparse attention combine launch");
}

int sparse_f32(const float* Q, int M, const float* K, const float* V, int L, int H, const SparseList& sl, float* O,
               void* ws, size_t ws_bytes, cudaStream_t st) {
  static PerContextOnce attr;
  int rc = attr.ensure([](void**) {
    if (cudaFuncSetAttribute(k_attn_sparse_f32, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kF32AttnSmem + 4 * HSA_SPARSE_MAX_KEEP) != cudaSuccess)
      return check_launch("sparse attention (fp32): shared-memory attribute");
    return (int)HSA_OK;
  });
  if (rc) return rc;
  const int QB = (M + kF32BQ - 1) / kF32BQ;
  int S = ws ? f32_attn_splits(M, sl.keep * sl.block, H, ws_bytes) : 1;
  const size_t slots = (size_t)QB * H * S * kF32BQ;
  const size_t o_bytes = align256(slots * 128 * sizeof(float));
  if (S > 1 && o_bytes + slots * sizeof(float2) > ws_bytes) S = 1;
  float* part_o = S > 1 ? static_cast<float*>(ws) : nullptr;
  float2* part_ml = S > 1 ? reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + o_bytes) : nullptr;
  ScopedTiming timing(HSA_KCLASS_ATTENTION, st);
  launch(k_attn_sparse_f32, (unsigned)(QB * H * S), 256, kF32AttnSmem + 4 * sl.keep, st, Q, M, K, V, L, H, S, sl, O,
         part_o, part_ml);
  count_launch(1);
  rc = check_launch("sparse attention (fp32) launch");
  if (rc || S == 1) return rc;
  const long long warps = (long long)QB * H * kF32BQ;
  launch(k_attn_sparse_f32_combine, (unsigned)((warps + 7) / 8), 256, 0, st, part_o, part_ml, M, H, S, O);
  count_launch(1);
  return check_launch("sparse attention (fp32) combine launch");
}
}  // namespace

}  // namespace hsa

using namespace hsa;

extern "C" size_t hsa_sparse_attention_workspace_size(int M, int L, int H, int dtype, int block_k, int keep) {
  if (M <= 0 || L <= 0 || H <= 0 || keep < 1 || keep > HSA_SPARSE_MAX_KEEP || (block_k != 64 && block_k != 128)) return 0;
  if (dtype == HSA_F32) return attention_f32_split_bytes(M, keep * block_k, H);
  if (dtype != HSA_BF16) return 0;
  return tail_split_bytes(plan_tail((M + kAttnBM - 1) / kAttnBM * H, sparse_tiles(keep, block_k), num_sms()));
}

extern "C" int hsa_sparse_attention(const void* d_q, int M, const void* d_k, const void* d_v, int L, int H, int dtype,
                                    int block_k, const int32_t* d_list, int keep, const int32_t* d_count, void* d_o,
                                    void* d_ws, size_t ws_bytes, void* stream) {
  if (dtype != HSA_BF16 && dtype != HSA_F32) return set_error(HSA_EINVAL, "sparse_attention: unknown dtype");
  if (M < 0 || L <= 0 || H <= 0) return set_error(HSA_EINVAL, "sparse_attention: need M >= 0, L > 0 and H > 0");
  if (block_k != 64 && block_k != 128) return set_error(HSA_EINVAL, "sparse_attention: need block_k = 64 or 128");
  if (keep < 1 || keep > HSA_SPARSE_MAX_KEEP)
    return set_error(HSA_EINVAL, "sparse_attention: need 1 <= keep <= 4096");
  if (M == 0) return HSA_OK;
  if (!d_q || !d_k || !d_v || !d_o || !d_list || !d_count || !aligned16(d_q) || !aligned16(d_k) || !aligned16(d_v) ||
      !aligned16(d_o) || (d_ws && !aligned16(d_ws)))
    return set_error(HSA_EINVAL, "sparse_attention: null or misaligned pointer");
  const SparseList sl{d_list, d_count, keep, block_k, (L + block_k - 1) / block_k};
  cudaStream_t st = as_stream(stream);
  if (dtype == HSA_BF16) return sparse_bf16(d_q, M, d_k, d_v, L, H, sl, d_o, d_ws, ws_bytes, st);
  return sparse_f32(static_cast<const float*>(d_q), M, static_cast<const float*>(d_k), static_cast<const float*>(d_v), L,
                    H, sl, static_cast<float*>(d_o), d_ws, ws_bytes, st);
}
