// attn_sparse.cu -- attention of compacted queries over listed blocks of the KV cache
// (hsa_sparse_attention): for the rows of query tile t (128 compacted rows) and head h
//   o = softmax(q K_S^T / sqrt(128)) V_S,   S = the keys of blocks list[h][t][0 .. count[h][t]),
// 0 for a row whose list is empty.  Blocks are 64 or 128 consecutive cache rows.
//
// bf16 kernel.  A work unit is one (query tile, head), or one range of its list; lists are short (tens of
// 128-key tiles), so filling and draining the pipeline per unit is what costs: with a CTA per unit it
// took 6.3 us beside 0.96 us per tile.  Here the CTAs stay (one per SM) and see one endless
// stream of tiles, g = 0, 1, 2, ..., in which a unit's first tile follows the last one of the unit before:
//   warp 2      scheduler: takes the next CTA of the grid that has not started yet (cluster launch control,
//               so units go to the SM that is free whatever their lists' lengths, without a counter in
//               memory), reads its count and list, and hands units on through a ring of three slots
//   warp 0      TMA producer: V_g, then K_{g+2}, of whichever unit they belong to; Q of a unit once the
//               last QK^T of the one before is done
//   warp 1      TMEM owner and MMA issuer: for each g  O_b (+)= P_g V_g in two halves of 64 keys, then
//               S_b = Q K_{g+2}^T, b = g % 2
//   warps 4-7   softmax of the even tiles of the stream, warps 8-11 of the odd ones, one thread per
//               query row; the two parities keep their own max, sum and O, merged at a unit's end.  The next
//               unit's first two QK^T run during that epilogue.
// V_g and K_{g+2} complete on the barriers that count the softmax warps' P_g, so the MMA warp waits twice
// per tile.  V has one slot per parity: the producer's arrival on p_full[b] for tile g follows its wait for
// the slot, which the MMA warp releases after it has waited for both halves of P_{g-2}; so no arrival lands
// a phase early, whatever the unit boundaries.  The softmax warpgroups take the registers that the control
// warpgroup gives up (208 + 208 + 88 = 3 x 168 a thread at launch; 56 or 72 for the control warps spill or
// are 1 % slower, and spills in the softmax, as with all of O in registers at once, cost 15 %).
// A tile's 128 keys are one listed 128-row block (two 64-column boxes) or two listed 64-row blocks (four
// 64 x 64 boxes), so a finer list costs only more TMA instructions, and the tensor-core shapes stay
// 128 x 128 x 128.  A unit's list is staged in shared memory as 16-bit block numbers; kNoBlock stands for
// "no block" (padding of an odd list, an index outside [0, blocks)), which TMA fills with zeros and the
// softmax masks to -inf.  The numbers also tell the softmax which tiles need a mask at all (the ragged
// last block may stand anywhere in a list).
//
// Rounding: logits, running max and sum, and O are float32; p is rounded to bf16 for the second
// product (its sum is taken before the rounding; at most 2^-8 of each term), and O once at the end.
#include <climits>

#include "tcgen05.cuh"

namespace hsa {

constexpr int kSpThreads = 384;
constexpr int kSpKSlots = 3, kSpUnits = 3;
constexpr uint32_t kSpColS = 0, kSpColO = 256, kSpCols = 512;
constexpr uint32_t kNoBlock = 0xFFFFu;
constexpr int kSpMaxBlocks = 65535;
constexpr int kSpCtrlRegs = 88, kSpSoftRegs = 208;       // per thread; (88 + 2 * 208) * 128 = 168 * 384
// The next unit is claimed when this many tiles of the current one are left (a long one; shorter ones are
// claimed up to the ring's capacity): enough to read its list meanwhile, and late enough that an SM does
// not sit on a whole unit while others run out (lists of 0 to 77 blocks of 64: 388 us with a unit claimed
// ahead, 381 us so)
constexpr int kSpAheadTiles = 6;

struct SparseUnit {
  int u, nt, slot;      // unit, its tiles (0: the end of the stream), partial-result slot or -1
};
struct SparseShared {
  uint64_t q_full, q_empty;
  uint64_t k_full[2], k_empty[kSpKSlots];   // k_full: the first two tiles of the stream only
  uint64_t v_empty[2];
  uint64_t s_full[2], p_full[2][2], o_done, o_free;
  uint64_t unit_full[kSpUnits], unit_empty[kSpUnits];
  uint64_t near_end;                        // the V stream is kSpAheadTiles before the end of a long unit
  uint64_t merge[4];                        // a lane quarter's two softmax warps, at a unit's end
  uint64_t clc;
  uint4 clc_answer;
  SparseUnit unit[kSpUnits];
  uint32_t tmem;
  float xm[2][2][128], xl[2][2][128];       // [unit % 2][parity][row]
};
constexpr int kSpSmemFixed = kTileBytes * (1 + kSpKSlots + 2) + 1024 + (int)sizeof(SparseShared);
__host__ __device__ constexpr int sparse_list_stride(int keep) { return (keep + 1 + 7) & ~7; }   // 16-bit entries
constexpr int sparse_smem(int keep) { return kSpSmemFixed + kSpUnits * 2 * sparse_list_stride(keep); }
static_assert(sparse_smem(HSA_SPARSE_MAX_KEEP) <= 227 * 1024, "three of the longest lists must fit shared memory");

struct SparseList {
  const int* list;    // [H][QT][keep]
  const int* count;   // [H][QT]
  int keep, block, n_blocks;
};

// Blocks listed for a unit (clamped to [0, keep])
__device__ __forceinline__ int listed_blocks(const SparseList& s, size_t unit) {
  const int n = s.count[unit];
  if (n < 0 || n > s.keep) {
    flag_error(HSA_EINDEX);
    return n < 0 ? 0 : s.keep;
  }
  return n;
}

template <int R>
__device__ __forceinline__ void regs_give() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_take() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }

// Ask for a CTA of this grid that has not started: 16 bytes into `answer`, completing on `bar`
__device__ __forceinline__ void clc_request(uint4* answer, uint64_t* bar) {
  mbar_expect_tx(bar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
               ::"r"(smem_u32(answer)), "r"(smem_u32(bar))
               : "memory");
}
// The CTA's index, or -1 when every CTA has started
__device__ __forceinline__ int clc_answer_cta(const uint4* answer) {
  int x = -1;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t.reg .b32 x;\n\t"
      "ld.shared.b128 r, [%1];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "mov.b32 x, 0xFFFFFFFF;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 x, r;\n\t"
      "mov.b32 %0, x;\n\t}\n"
      : "=r"(x)
      : "r"(smem_u32(answer))
      : "memory");
  return x;
}

// A role's position in the ring of units
struct UnitCursor {
  int s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void advance() {
    if (++s == kSpUnits) {
      s = 0;
      phase ^= 1u;
    }
  }
};

// Chunk j of lane 4 q + i  <->  chunk i of lane 4 q + j, i, j < 4
__device__ __forceinline__ uint4 shfl_xor_u4(uint4 v, int m) {
  return make_uint4(__shfl_xor_sync(0xffffffffu, v.x, m), __shfl_xor_sync(0xffffffffu, v.y, m),
                    __shfl_xor_sync(0xffffffffu, v.z, m), __shfl_xor_sync(0xffffffffu, v.w, m));
}
__device__ __forceinline__ void quad_transpose(uint4 (&c)[4], int lane) {
#pragma unroll
  for (int m = 1; m <= 2; m <<= 1) {
    const bool up = (lane & m) != 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & m) continue;
      const uint4 got = shfl_xor_u4(up ? c[i] : c[i | m], m);
      if (up) c[i] = got;
      else c[i | m] = got;
    }
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
  SparseShared* sh = reinterpret_cast<SparseShared*>(sV + 2 * kTileBytes);
  uint16_t* lists = reinterpret_cast<uint16_t*>(sh + 1);  // [kSpUnits][stride]
  const int stride = sparse_list_stride(sl.keep);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool halves = sl.block == 64;                     // two blocks per 128-key tile

  if (threadIdx.x == 0) {
    mbar_init(&sh->q_full, 1);
    mbar_init(&sh->q_empty, 1);
    for (int s = 0; s < kSpKSlots; ++s) mbar_init(&sh->k_empty[s], 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh->k_full[b], 1);
      mbar_init(&sh->v_empty[b], 1);
      mbar_init(&sh->s_full[b], 1);
      mbar_init(&sh->p_full[b][0], 129);   // the parity's 128 softmax threads + the producer
      mbar_init(&sh->p_full[b][1], 129);
    }
    mbar_init(&sh->o_done, 1);
    mbar_init(&sh->o_free, 256);
    for (int s = 0; s < kSpUnits; ++s) {
      mbar_init(&sh->unit_full[s], 1);
      mbar_init(&sh->unit_empty[s], 10);   // producer, MMA issuer, eight softmax warps
    }
    for (int q = 0; q < 4; ++q) mbar_init(&sh->merge[q], 64);
    mbar_init(&sh->clc, 1);
    mbar_init(&sh->near_end, 1);
    fence_mbar_init();
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(&sh->tmem, kSpCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = sh->tmem;

  if (warp < 4) {
    regs_give<kSpCtrlRegs>();
    if (warp == 2) {
      // ---------------------------------------------------------------- scheduler
      UnitCursor at;
      uint32_t clc_phase = 0, end_phase = 0;
      int cta = blockIdx.x, staged = 0;
      bool ok = true;
      while (true) {
        int nt = 0, slot = -1, u = -1;
        if (cta >= 0) {
          int split = 0, n_split = 1;
          u = cta;
          if (u >= grid.u_full) {
            const int t = u - grid.u_full;
            u = grid.u_full + t / grid.s_tail;
            split = t % grid.s_tail;
            n_split = grid.s_tail;
            if (n_split > 1) slot = t;
          }
          const int n_list = listed_blocks(sl, (size_t)u);
          const int nt_all = halves ? (n_list + 1) >> 1 : n_list;
          const int j0 = (int)((long long)split * nt_all / n_split);
          nt = (int)((long long)(split + 1) * nt_all / n_split) - j0;
          if (nt > 0 && ok) {
            // slot free: the unit kSpUnits before it is finished everywhere
            if (staged >= kSpUnits) ok = mbar_wait_warp(&sh->unit_empty[at.s], at.phase ^ 1u);
            const int per = halves ? 2 : 1, first = j0 * per, n = min(nt * per, n_list - first);
            const int* src = sl.list + (size_t)u * sl.keep + first;
            uint16_t* dst = lists + at.s * stride;
            for (int i = lane; i < nt * per; i += 32) {
              int b = (int)kNoBlock;
              if (i < n) {
                b = src[i];
                if (b < 0 || b >= sl.n_blocks) {
                  flag_error(HSA_EINDEX);
                  b = (int)kNoBlock;
                }
              }
              dst[i] = (uint16_t)b;
            }
          } else if (nt == 0) {
            // nothing listed: the rows are 0 (or this range adds nothing)
            if (slot >= 0) {
              for (int r = lane; r < kAttnBM; r += 32)
                grid.part_ml[(size_t)slot * kAttnBM + r] = make_float2(-INFINITY, 0.f);
            } else {
              const int m0 = (u % grid.QT) * kAttnBM, h = u / grid.QT;
              for (int i = lane; i < kAttnBM * 16; i += 32) {
                const int r = m0 + (i >> 4);
                if (r < M)
                  *reinterpret_cast<uint4*>(O + (size_t)r * (H * 128) + h * 128 + (i & 15) * 8) =
                      make_uint4(0u, 0u, 0u, 0u);
              }
            }
          }
        } else if (staged >= kSpUnits && ok) {
          ok = mbar_wait_warp(&sh->unit_empty[at.s], at.phase ^ 1u);
        }
        if (ok && (nt > 0 || cta < 0)) {
          if (lane == 0) sh->unit[at.s] = SparseUnit{u, nt, slot};
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->unit_full[at.s]);
          at.advance();
          ++staged;
          if (nt >= kSpAheadTiles) {
            ok = mbar_wait_warp(&sh->near_end, end_phase);
            end_phase ^= 1u;
          }
        }
        if (cta < 0 || !ok) break;
        if (lane == 0) clc_request(&sh->clc_answer, &sh->clc);
        ok = mbar_wait_warp(&sh->clc, clc_phase);
        if (!ok) break;
        clc_phase ^= 1u;
        cta = clc_answer_cta(&sh->clc_answer);
        __syncwarp();
        if (lane == 0) fence_proxy_async_smem();          // read before the next answer is written
      }
      if (!ok) stall_drain();
    } else if (warp == 0) {
      // ---------------------------------------------------------------- TMA producer
      const bool leader = elect_one();
      // the 128 keys of tile t of the list in ring slot s, 32 KB completing on `bar`
      auto load_tile = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int s, int t, int x0) {
        const uint16_t* l = lists + s * stride;
        mbar_expect_tx(bar, kTileBytes);
        auto row = [&](uint32_t b) { return b == kNoBlock ? L : (int)b * sl.block; };
        if (halves) {
          const int r0 = row(l[2 * t]), r1 = row(l[2 * t + 1]);
          tma_load_2d(dst, map, bar, x0, r0);
          tma_load_2d(dst + kTileBytes / 4, map, bar, x0, r1);
          tma_load_2d(dst + kTileBytes / 2, map, bar, x0 + 64, r0);
          tma_load_2d(dst + 3 * (kTileBytes / 4), map, bar, x0 + 64, r1);
        } else {
          const int r = row(l[t]);
          tma_load_2d(dst, map, bar, x0, r);
          tma_load_2d(dst + kTileBytes / 2, map, bar, x0 + 64, r);
        }
      };
      UnitCursor kc, vc;
      int k_t = 0, k_nt = 0, k_x0 = 0, k_m0 = 0, k_slot = 0, n_q = 0;
      uint32_t k_phase = 1;
      bool ok = true, k_end = false, k_first = true;
      // the stream's next K tile, completing on `bar`; false at the stream's end
      auto load_k = [&](uint64_t* bar) -> bool {
        if (k_t == k_nt) {
          if (!k_first) kc.advance();
          k_first = false;
          ok = mbar_wait_warp(&sh->unit_full[kc.s], kc.phase);
          const SparseUnit unit = sh->unit[kc.s];
          if (!ok || unit.nt == 0) {
            k_end = true;
            return false;
          }
          k_t = 0;
          k_nt = unit.nt;
          k_x0 = unit.u / grid.QT * 128;
          k_m0 = unit.u % grid.QT * kAttnBM;
        }
        ok = mbar_wait_warp(&sh->k_empty[k_slot], k_phase);
        if (!ok) return false;
        if (leader) load_tile(sK + k_slot * kTileBytes, &tmK, bar, kc.s, k_t, k_x0);
        __syncwarp();
        ++k_t;
        if (++k_slot == kSpKSlots) {
          k_slot = 0;
          k_phase ^= 1u;
        }
        if (k_t == 1) {
          // a unit's Q follows its first K: the buffer is free once the last QK^T of the unit before is done,
          // and that wait must not hold up the P barrier that this K completes on
          if (n_q > 0) ok = mbar_wait_warp(&sh->q_empty, (n_q - 1) & 1);
          if (ok && leader) {
            mbar_expect_tx(&sh->q_full, kTileBytes);
            tma_load_2d(sQ, &tmQ, &sh->q_full, k_x0, k_m0);
            tma_load_2d(sQ + kTileBytes / 2, &tmQ, &sh->q_full, k_x0 + 64, k_m0);
          }
          __syncwarp();
          ++n_q;
        }
        return true;
      };
      if (load_k(&sh->k_full[0])) load_k(&sh->k_full[1]);
      uint32_t g = 0;
      while (ok) {
        ok = mbar_wait_warp(&sh->unit_full[vc.s], vc.phase);
        if (!ok) break;
        const int nt = sh->unit[vc.s].nt, x0 = sh->unit[vc.s].u / grid.QT * 128;
        if (nt == 0) break;
        for (int t = 0; ok && t < nt; ++t, ++g) {
          const uint32_t b = g & 1u;
          if (t == nt - kSpAheadTiles && lane == 0) mbar_arrive(&sh->near_end);
          ok = mbar_wait_warp(&sh->v_empty[b], ((g >> 1) & 1u) ^ 1u);
          if (!ok) break;
          if (leader) load_tile(sV + b * kTileBytes, &tmV, &sh->p_full[b][0], vc.s, t, x0);
          __syncwarp();
          if (k_end || !load_k(&sh->p_full[b][1])) {
            if (ok && leader) mbar_arrive(&sh->p_full[b][1]);
            __syncwarp();
          }
        }
        if (ok && lane == 0) mbar_arrive(&sh->unit_empty[vc.s]);
        __syncwarp();
        vc.advance();
      }
      if (!ok) stall_drain();
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, false);
      constexpr uint32_t idesc_o = idesc_bf16_f32(128, 128, true);
      const bool leader = elect_one();
      const uint64_t q_desc = sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t k_desc = sdesc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t v_desc = sdesc_sw128(smem_u32(sV), kTileBytes / 2, 1024);
      UnitCursor qc, pc;
      int q_t = 0, q_nt = 0, q_slot = 0, n_q = 0, n_o = 0;
      bool ok = true, q_end = false, q_first = true;
      // QK^T of the stream's next tile into S_b; its K has arrived (the first two wait here)
      auto issue_qk = [&](uint32_t g) -> bool {
        if (q_t == q_nt) {
          if (!q_first) qc.advance();
          q_first = false;
          ok = mbar_wait_warp(&sh->unit_full[qc.s], qc.phase);
          q_nt = ok ? sh->unit[qc.s].nt : 0;
          if (q_nt == 0) {
            q_end = true;
            return false;
          }
          q_t = 0;
          ok = mbar_wait_warp(&sh->q_full, n_q & 1);
          ++n_q;
          if (!ok) return false;
        }
        if (g < 2) {
          ok = mbar_wait_warp(&sh->k_full[g], 0);
          if (!ok) return false;
        }
        const uint32_t b = g & 1u;
        ++q_t;
        tc_fence_after();
        const uint64_t kd = k_desc + (uint64_t)((q_slot * kTileBytes) >> 4);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t off = ((kk >> 2) * (kTileBytes / 2) + (kk & 3) * 32) >> 4;
            umma_ss(tm + kSpColS + b * 128, q_desc + off, kd + off, idesc_s, kk > 0);
          }
          umma_commit(&sh->s_full[b]);
          umma_commit(&sh->k_empty[q_slot]);
          if (q_t == q_nt) umma_commit(&sh->q_empty);
        }
        __syncwarp();
        if (++q_slot == kSpKSlots) q_slot = 0;
        return true;
      };
      if (issue_qk(0)) issue_qk(1);
      uint32_t g = 0;
      while (ok) {
        ok = mbar_wait_warp(&sh->unit_full[pc.s], pc.phase);
        if (!ok) break;
        const int nt = sh->unit[pc.s].nt;
        if (nt == 0) break;
        // the first PV of a unit overwrites O: the epilogue of the one before has read it
        if (n_o > 0) ok = mbar_wait_warp(&sh->o_free, (n_o - 1) & 1);
        for (int t = 0; ok && t < nt; ++t, ++g) {
          const uint32_t b = g & 1u;
          const uint64_t vd = v_desc + (uint64_t)((b * kTileBytes) >> 4);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            if (!ok) break;
            ok = mbar_wait_warp(&sh->p_full[b][q], (g >> 1) & 1u);
            if (!ok) break;
            tc_fence_after();
            if (leader) {
#pragma unroll
              for (int kk = q * 4; kk < q * 4 + 4; ++kk)
                umma_ts(tm + kSpColO + b * 128, tm + kSpColS + b * 128 + kk * 8, vd + (uint64_t)(kk * 2048 >> 4),
                        idesc_o, (t >= 2 || kk > 0));
              if (q == 1) umma_commit(&sh->v_empty[b]);
            }
            __syncwarp();
          }
          if (!ok) break;
          if (t == nt - 1) {
            if (leader) umma_commit(&sh->o_done);
            __syncwarp();
          }
          if (!q_end) issue_qk(g + 2);
        }
        ++n_o;
        if (ok && lane == 0) mbar_arrive(&sh->unit_empty[pc.s]);
        __syncwarp();
        pc.advance();
      }
      if (!ok) stall_drain();
    }
  } else {
    // ---------------------------------------------------------------- softmax warps
    regs_take<kSpSoftRegs>();
    const int quarter = warp & 3;
    const uint32_t par = (warp >> 2) - 1;
    const int row = quarter * 32 + lane;
    const uint32_t lane_base = tm + ((uint32_t)(quarter * 32) << 16);
    const uint32_t s_col = lane_base + kSpColS + par * 128, o_col = lane_base + kSpColO + par * 128;
    const float sc = 0.12751743074680484f;               // log2(e) / sqrt(128)
    UnitCursor at;
    uint32_t s_phase = 0, first = 0, n_unit = 0;          // first: parity of the unit's first tile
    // The unit whose tiles are done and whose rows are still to be written.  The parity of its last tile
    // writes at once; the other one, whose next S is ready before that last PV is done, first takes the
    // softmax of its first tile of the next unit, so that P is there when O comes free.
    int done_u = -1, done_slot = -1;
    bool done_two = false;
    uint32_t done_first = 0, done_last = 0;               // parities of its first and last tile
    bool ok = true;
    while (ok) {
      ok = mbar_wait_warp(&sh->unit_full[at.s], at.phase);
      if (!ok) break;
      const int nt = sh->unit[at.s].nt;                   // 0: the end
      const uint16_t* blk = lists + at.s * stride;
      float m = -INFINITY, l = 0.f;
      int t = (int)(par ^ first);
      bool write = t >= nt || done_last == par;
      do {
        if (done_u >= 0 && write) {
          // -------------------------------------------------------------- merge the parities, write the rows
          // F: the parity of the unit's first tile, G: the other one, without a tile in a unit of one
          const uint32_t pb = (n_unit & 1u) ^ 1u;
          const float(*xm)[128] = sh->xm[pb];
          const float(*xl)[128] = sh->xl[pb];
          ok = mbar_wait_warp(&sh->merge[quarter], pb);
          if (!ok) break;
          const float mF = xm[done_first][row], mG = xm[done_first ^ 1u][row];
          const float mm = fmaxf(mF, mG);
          const float ms = mm == -INFINITY ? 0.f : mm;    // no key at all: weights 0
          const float aF = ex2_approx(mF - ms), aG = ex2_approx(mG - ms);
          const float den = aF * xl[done_first][row] + aG * xl[done_first ^ 1u][row];
          const float inv_l = den > 0.f ? 1.0f / den : 0.f;
          const float wF = done_slot >= 0 ? aF : aF * inv_l, wG = done_slot >= 0 ? aG : aG * inv_l;
          const int m0 = (done_u % grid.QT) * kAttnBM;
          const bool part = done_slot >= 0 && m0 + row < M;
          if (part && par == 0) grid.part_ml[(size_t)done_slot * kAttnBM + row] = make_float2(mm, den);
          ok = mbar_wait_warp(&sh->o_done, pb);
          if (!ok) break;
          tc_fence_after();
          // this warp writes output columns [64 par, 64 par + 64) of its 32 rows, 32 at a time
          uint4 ch[2][4];                                 // the row's 64 columns in bf16, chunks of 8
#pragma unroll
          for (int hc = 0; hc < 2; ++hc) {
            const uint32_t col = par * 64 + (uint32_t)hc * 32;
            uint32_t oF[32], oG[32];
            tmem_ld32(lane_base + kSpColO + done_first * 128 + col, oF);
            if (done_two) tmem_ld32(lane_base + kSpColO + (done_first ^ 1u) * 128 + col, oG);
            tmem_ld_wait();
            if (hc == 1) {
              tc_fence_before();
              mbar_arrive(&sh->o_free);
            }
            float f[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float g = done_two ? __uint_as_float(oG[e]) : 0.f;
              f[e] = fmaf(__uint_as_float(oF[e]), wF, g * wG);
            }
            if (part) {
              float* dst = grid.part_o + ((size_t)done_slot * kAttnBM + row) * 128 + col;
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4*>(dst + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
              ch[hc][i] = make_uint4(pack_bf16x2(f[8 * i], f[8 * i + 1]), pack_bf16x2(f[8 * i + 2], f[8 * i + 3]),
                                     pack_bf16x2(f[8 * i + 4], f[8 * i + 5]), pack_bf16x2(f[8 * i + 6], f[8 * i + 7]));
          }
          if (done_slot < 0) {
            // chunks transposed among the four lanes of a quad, so that a store covers 64 consecutive
            // bytes of 8 rows instead of 16 bytes of 32
            const int r0 = m0 + quarter * 32 + (lane & ~3);
            __nv_bfloat16* dst = O + (size_t)r0 * (H * 128) + (done_u / grid.QT) * 128 + par * 64 + (lane & 3) * 8;
#pragma unroll
            for (int hc = 0; hc < 2; ++hc) {
              quad_transpose(ch[hc], lane);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (r0 + i < M) *reinterpret_cast<uint4*>(dst + (size_t)i * (H * 128) + hc * 32) = ch[hc][i];
            }
          }
          __syncwarp();
          done_u = -1;
        }
        write = true;
        if (t < nt) {
        // keys of the tile's two 64-key halves that exist (64 or more: all)
        int v0, v1;
        {
          const uint32_t b0 = blk[halves ? 2 * t : t], b1 = halves ? blk[2 * t + 1] : b0;
          v0 = b0 == kNoBlock ? 0 : L - (int)b0 * sl.block;
          v1 = b1 == kNoBlock ? 0 : L - (int)b1 * sl.block;
          if (!halves) v1 -= 64;
        }
        ok = mbar_wait_warp(&sh->s_full[par], s_phase);
        if (!ok) break;
        s_phase ^= 1u;
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
        if (t < 2) {
          m = m_tile;
        } else if (m_tile > m + 8.0f) {
          need = true;
          corr = ex2_approx(m - m_tile);
          l *= corr;
          m = m_tile;
        }
        const bool any_need = __any_sync(0xffffffffu, need);
        const float neg_m = m == -INFINITY ? 0.f : -m;    // no key so far: every p is 2^-inf = 0
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
          // O of this parity holds the PV of the unit's earlier tiles, complete: S was written by an MMA
          // issued after them, and PV of this tile starts only after the p_full arrivals below
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
        t += 2;
      } while (t < nt || done_u >= 0);
      if (!ok || nt == 0) break;
      done_u = sh->unit[at.s].u;
      done_slot = sh->unit[at.s].slot;
      done_two = nt >= 2;
      done_first = first;
      done_last = first ^ ((uint32_t)(nt - 1) & 1u);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->unit_empty[at.s]);  // done with the list
      sh->xm[n_unit & 1][par][row] = m;
      sh->xl[n_unit & 1][par][row] = l;
      mbar_arrive(&sh->merge[quarter]);
      first ^= (uint32_t)nt & 1u;
      ++n_unit;
      at.advance();
    }
    if (!ok) stall_drain();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tm, kSpCols);
  }
}

// Row of a split unit from its S <= 32 list ranges, by one warp: lane s holds range s's max and sum, then
// every lane 4 channels, eight ranges' loads in flight (one after the other they cost the row S trips to
// L2).  A range without keys has sum 0 and wrote no O.  EX: exponential of the ranges' logit units.
template <typename EX>
__device__ __forceinline__ float4 merge_ranges(const float* __restrict__ part_o, const float2* __restrict__ part_ml,
                                               size_t first, size_t stride, int S, int lane, EX ex) {
  const float2 ml = lane < S ? part_ml[first + (size_t)lane * stride] : make_float2(-INFINITY, 0.f);
  float mx = ml.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float a = ml.y != 0.f ? ex(ml.x - mx) : 0.f;      // a sum that is NaN stays one
  const float den = warp_sum(a * ml.y);
  const float w = den != 0.f ? a / den : 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < S; s0 += 8) {
    float4 v[8];
    float ws[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      ws[i] = __shfl_sync(0xffffffffu, w, (s0 + i) & 31);
      v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s0 + i < S && ws[i] != 0.f) v[i] = ld4(part_o + (first + (size_t)(s0 + i) * stride) * 128 + lane * 4);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (s0 + i < S)
        acc = make_float4(fmaf(ws[i], v[i].x, acc.x), fmaf(ws[i], v[i].y, acc.y), fmaf(ws[i], v[i].z, acc.z),
                          fmaf(ws[i], v[i].w, acc.w));
  }
  return acc;
}

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
  const float4 o = merge_ranges(part_o, part_ml, (size_t)tu * s_tail * kAttnBM + row, kAttnBM, s_tail, lane,
                                [](float x) { return exp2f(x); });
  store4(O + (size_t)grow * (H * 128) + h * 128 + lane * 4, o);
}

// ------------------------------------------------------------------ float32, CUDA cores
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

// CTA = BQ query rows of one head x a range of their tile's list, 64 keys at a time (a 128-row block is two
// tiles).  2 BQ threads; thread (ty, tx) has rows 8 ty .. 8 ty + 7, logits of keys tx + 16 j (j < 4) and
// output channels 4 tx .. and 64 + 4 tx ...  Bound by shared-memory reads, so the thread tiles are 8 x 4 and
// 8 x 8, products run in packed pairs, and P is kept key by key so that a thread's eight weights are two reads
// (2 x 4 and 2 x 8 tiles with P row by row, as in k_attn_f32, read three times as much: 22.7 against 16.1 us
// for 512 rows x 8 of 16 blocks of 64, 2 heads).  Tiles come by 16-byte asynchronous copies: K of the next
// tile travels while this one's softmax and P V run, V while the next Q K^T does.  BQ = 128 gives an SM eight
// warps to hide the reads' latency with (2000 x 16 of 63 blocks of 64, 8 heads: 264 us, with 64 rows 307);
// BQ = 64 makes twice the CTAs, for calls that would leave SMs idle (the rule: sparse_f32_rows).
constexpr int kSp32BK = 64, kSp32Ld = 132;
constexpr int sparse_f32_smem(int bq) { return ((bq + 2 * kSp32BK) * kSp32Ld + kSp32BK * (bq + 4)) * 4; }
static_assert(sparse_f32_smem(128) + 4 * HSA_SPARSE_MAX_KEEP <= 227 * 1024, "the longest list must fit shared memory");

__device__ __forceinline__ void copy16_async(float* dst, const float* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
               ::"r"(smem_u32(dst)), "l"(src), "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int BQ>
__global__ void __launch_bounds__(2 * BQ, 1)
    k_attn_sparse_f32(const float* __restrict__ Q, int M, const float* __restrict__ K, const float* __restrict__ V,
                      int L, int H, int n_split, const SparseList sl, float* __restrict__ O,
                      float* __restrict__ part_o, float2* __restrict__ part_ml) {
  pdl_prologue();
  constexpr int kWarps = BQ / 16;
  extern __shared__ float4 sm4[];
  float* Qs = reinterpret_cast<float*>(sm4);              // [BQ][132]
  float* Ks = Qs + BQ * kSp32Ld;                     // [64][132]
  float* Vs = Ks + kSp32BK * kSp32Ld;                     // [64][132]
  float* Ps = Vs + kSp32BK * kSp32Ld;                     // [64 keys][BQ + 4]
  int* rows = reinterpret_cast<int*>(Ps + kSp32BK * (BQ + 4));
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int QB = (M + BQ - 1) / BQ, QT = (M + HSA_QUERY_TILE - 1) / HSA_QUERY_TILE;
  int b = blockIdx.x;
  const int split = b % n_split;
  b /= n_split;
  const int qb = b % QB, h = b / QB;
  const int D = H * 128, m0 = qb * BQ;
  const size_t unit = (size_t)h * QT + m0 / HSA_QUERY_TILE;
#pragma unroll
  for (int i = 0; i < BQ / kWarps; ++i) {
    const int r = (tid >> 5) + kWarps * i, c4 = tid & 31;
    const bool ok = m0 + r < M;
    copy16_async(Qs + r * kSp32Ld + 4 * c4, Q + (size_t)(ok ? m0 + r : m0) * D + h * 128 + 4 * c4, ok);
  }
  const int n_list = listed_blocks(sl, unit);
  const int per = sl.block / kSp32BK;                     // tiles per block
  const int i0 = (int)((long long)split * n_list / n_split);
  const int i1 = (int)((long long)(split + 1) * n_list / n_split);
  stage_rows(sl, unit, i0, i1 - i0, L, rows);
  __syncthreads();
  const int nt = (i1 - i0) * per;
  auto tile_row = [&](int t) { return per == 1 ? rows[t] : rows[t >> 1] + (t & 1) * kSp32BK; };
  // the 64 keys from cache row k0, zeros beyond the cache
  auto load_tile = [&](float* dst, const float* src, int k0) {
#pragma unroll
    for (int i = 0; i < kSp32BK / kWarps; ++i) {
      const int key = (tid >> 5) + kWarps * i, c4 = tid & 31;
      const bool ok = k0 + key < L;
      copy16_async(dst + key * kSp32Ld + 4 * c4, src + (size_t)(ok ? k0 + key : 0) * D + h * 128 + 4 * c4, ok);
    }
    copy_group();
  };
  if (nt > 0) {
    load_tile(Ks, K, tile_row(0));                        // with Q
    load_tile(Vs, V, tile_row(0));
  }
  const float scale = 0.08838834764831845f;
  float m[8], l[8];
  float2 o[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) o[i][c] = make_float2(0.f, 0.f);
  }
  const float* qr = Qs + (8 * ty) * kSp32Ld;
  for (int t = 0; t < nt; ++t) {
    const int k0 = tile_row(t);
    copy_wait<1>();                                       // K_t; V_t may still travel
    __syncthreads();
    float2 s2[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s2[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int c = 0; c < 128; c += 4) {
      float4 kk[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) kk[j] = ld4(Ks + (tx + 16 * j) * kSp32Ld + c);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 a = ld4(qr + i * kSp32Ld + c);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s2[i][j] = ffma2(make_float2(a.z, a.w), make_float2(kk[j].z, kk[j].w),
                           ffma2(make_float2(a.x, a.y), make_float2(kk[j].x, kk[j].y), s2[i][j]));
      }
    }
    __syncthreads();                                      // K is read: the next one may come
    if (t + 1 < nt) load_tile(Ks, K, tile_row(t + 1));
    float p[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[i][j] = (k0 + tx + 16 * j < L) ? (s2[i][j].x + s2[i][j].y) * scale : -INFINITY;
        mx = fmaxf(mx, p[i][j]);
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float m_new = fmaxf(m[i], mx);
      const float m_ref = m_new == -INFINITY ? 0.f : m_new;   // no key so far: every weight is 0
      const float corr = expf(m[i] - m_ref);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[i][j] = expf(p[i][j] - m_ref);
        sum += p[i][j];
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      l[i] = l[i] * corr + sum;
      m[i] = m_new;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        o[i][c].x *= corr;
        o[i][c].y *= corr;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float* dst = Ps + (tx + 16 * j) * (BQ + 4) + 8 * ty;
      st4(dst, make_float4(p[0][j], p[1][j], p[2][j], p[3][j]));
      st4(dst + 4, make_float4(p[4][j], p[5][j], p[6][j], p[7][j]));
    }
    if (t + 1 < nt) copy_wait<1>();                       // V_t; K_{t+1} may still travel
    else copy_wait<0>();
    __syncthreads();
#pragma unroll 4
    for (int key = 0; key < kSp32BK; ++key) {
      const float4 pa = ld4(Ps + key * (BQ + 4) + 8 * ty), pb = ld4(Ps + key * (BQ + 4) + 8 * ty + 4);
      const float4 va = ld4(Vs + key * kSp32Ld + 4 * tx), vb = ld4(Vs + key * kSp32Ld + 64 + 4 * tx);
      const float pw[8] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
      const float2 vv[4] = {make_float2(va.x, va.y), make_float2(va.z, va.w), make_float2(vb.x, vb.y),
                            make_float2(vb.z, vb.w)};
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[i][c] = ffma2(make_float2(pw[i], pw[i]), vv[c], o[i][c]);
    }
    if (t + 1 < nt) {
      __syncthreads();                                    // V and P are read
      load_tile(Vs, V, tile_row(t + 1));
    }
  }
  if (nt == 0) copy_wait<0>();                            // Q
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = 8 * ty + i, grow = m0 + row;
    if (grow >= M) continue;
    const size_t slot = (size_t)blockIdx.x * BQ + row;
    const bool whole = n_split == 1;
    const float w = whole ? (l[i] > 0.f ? 1.0f / l[i] : 0.f) : 1.0f;
    float* dst = (whole ? O + (size_t)grow * D + h * 128 : part_o + slot * 128) + 4 * tx;
    st4(dst, make_float4(o[i][0].x * w, o[i][0].y * w, o[i][1].x * w, o[i][1].y * w));
    st4(dst + 64, make_float4(o[i][2].x * w, o[i][2].y * w, o[i][3].x * w, o[i][3].y * w));
    if (!whole && tx == 0) part_ml[slot] = make_float2(m[i], l[i]);
  }
}

__global__ void __launch_bounds__(256) k_attn_sparse_f32_combine(const float* __restrict__ part_o,
                                                                 const float2* __restrict__ part_ml, int M, int H,
                                                                 int n_split, int BQ, float* __restrict__ O) {
  pdl_prologue();
  const int w = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
  const int QB = (M + BQ - 1) / BQ;
  const int row = w % BQ, unit = w / BQ;
  if (unit >= QB * H) return;
  const int qb = unit % QB, h = unit / QB, grow = qb * BQ + row;
  if (grow >= M) return;
  const float4 o = merge_ranges(part_o, part_ml, (size_t)unit * n_split * BQ + row, BQ, n_split, lane,
                                [](float x) { return expf(x); });
  st4(O + (size_t)grow * (H * 128) + h * 128 + 4 * lane, o);
}

// ------------------------------------------------------------------ host
namespace {
// Sizes whose work units, rows and columns the kernels can count in an int (the float32 kernel has up to two
// units per query tile and head)
bool sparse_sizes_ok(int M, int H) {
  return M <= INT_MAX - 127 && H <= INT_MAX / 128 && 2LL * ((M + 127) / 128) * H <= INT_MAX;
}

int sparse_tiles(int keep, int block) { return block == 64 ? (keep + 1) / 2 : keep; }

// Ranges of the lists of an incomplete last wave's units.  Few units (a handful of query rows) against long
// lists wait for memory, and the more SMs fetch the better: as many ranges as fill one wave.  Otherwise as
// for the full-context kernel.
TailSplit sparse_plan(int M, int H, int keep, int block) {
  const int U = (M + kAttnBM - 1) / kAttnBM * H, tiles = sparse_tiles(keep, block), sms = num_sms();
  if (2 * U <= sms) {
    int S = sms / U < tiles ? sms / U : tiles;
    if (S > 32) S = 32;
    return S > 1 ? TailSplit{0, S, U} : TailSplit{U, 1, 0};
  }
  return plan_tail(U, tiles, sms);
}

// The fp32 kernel's query rows per CTA: 128 where the units, cut into at most 32 ranges of a block or more, could
// make a CTA for every SM.  Ranges are SMs / units rounded down, so 75 to 147 units are not split, and nothing is
// without a workspace.  Measured with 128 against 64 rows (16 of 63 blocks of 64): 80 or 125 units 263 us against
// 307, 32 units 72 / 82; 8 units of 20 blocks 41 / 36, of 8 blocks, where the rule says 64, 23 / 16.  Without a
// workspace 64 rows are faster below 75 units (32 units: 263 / 154), which the rule does not look at.
int sparse_f32_rows(int M, int H, int keep) {
  const long long units = (long long)((M + 127) / 128) * H;
  return units * (keep < 32 ? keep : 32) >= num_sms() ? 128 : 64;
}

// Its list ranges: one block or more each, one CTA per SM, partials within the workspace
int sparse_f32_splits(int M, int H, int keep, int BQ, size_t ws_bytes) {
  const long long units = (long long)((M + BQ - 1) / BQ) * H;
  long long S = num_sms() / units;
  if (S > keep) S = keep;
  if (S > 32) S = 32;
  const size_t per = (size_t)units * BQ * (128 * sizeof(float) + sizeof(float2));
  if ((size_t)S * per + 256 > ws_bytes) S = ws_bytes < 256 ? 1 : (long long)((ws_bytes - 256) / per);
  return S < 1 ? 1 : (int)S;
}

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
                             sparse_smem(HSA_SPARSE_MAX_KEEP)) != cudaSuccess)
      return check_launch("sparse attention: shared-memory attribute");
    return (int)HSA_OK;
  });
  if (rc) return rc;
  const int QT = (M + kAttnBM - 1) / kAttnBM, U = QT * H;
  TailSplit ts = sparse_plan(M, H, sl.keep, sl.block);
  const size_t need = tail_split_bytes(ts);
  if (need == 0 || !ws || ws_bytes < need) ts = TailSplit{U, 1, 0};
  AttnGrid g{QT, ts.u_full, ts.s_tail, nullptr, nullptr};
  if (ts.s_tail > 1) {
    const size_t slots = (size_t)ts.n_tail * ts.s_tail * kAttnBM;
    g.part_o = static_cast<float*>(ws);
    g.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + align256(slots * 128 * sizeof(float)));
  }
  ScopedTiming timing(HSA_KCLASS_ATTENTION, st);
  launch(k_attn_sparse, (unsigned)(ts.u_full + ts.n_tail * ts.s_tail), kSpThreads, sparse_smem(sl.keep), st, tq,
          tk, tv, M, L, H, reinterpret_cast<__nv_bfloat16*>(O), g, sl);
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
    if (cudaFuncSetAttribute(k_attn_sparse_f32<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             sparse_f32_smem(64) + 4 * HSA_SPARSE_MAX_KEEP) != cudaSuccess ||
        cudaFuncSetAttribute(k_attn_sparse_f32<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             sparse_f32_smem(128) + 4 * HSA_SPARSE_MAX_KEEP) != cudaSuccess)
      return check_launch("sparse attention (fp32): shared-memory attribute");
    return (int)HSA_OK;
  });
  if (rc) return rc;
  const int BQ = sparse_f32_rows(M, H, sl.keep), QB = (M + BQ - 1) / BQ;
  const int S = ws ? sparse_f32_splits(M, H, sl.keep, BQ, ws_bytes) : 1;
  const size_t o_bytes = align256((size_t)QB * H * S * BQ * 128 * sizeof(float));
  float* part_o = S > 1 ? static_cast<float*>(ws) : nullptr;
  float2* part_ml = S > 1 ? reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + o_bytes) : nullptr;
  ScopedTiming timing(HSA_KCLASS_ATTENTION, st);
  const unsigned ctas = (unsigned)(QB * H * S);
  const size_t smem = sparse_f32_smem(BQ) + 4 * (size_t)sl.keep;
  if (BQ == 128) launch(k_attn_sparse_f32<128>, ctas, 256, smem, st, Q, M, K, V, L, H, S, sl, O, part_o, part_ml);
  else launch(k_attn_sparse_f32<64>, ctas, 128, smem, st, Q, M, K, V, L, H, S, sl, O, part_o, part_ml);
  count_launch(1);
  rc = check_launch("sparse attention (fp32) launch");
  if (rc || S == 1) return rc;
  const long long warps = (long long)QB * H * BQ;
  launch(k_attn_sparse_f32_combine, (unsigned)((warps + 7) / 8), 256, 0, st, part_o, part_ml, M, H, S, BQ, O);
  count_launch(1);
  return check_launch("sparse attention (fp32) combine launch");
}
}  // namespace

}  // namespace hsa

using namespace hsa;

extern "C" size_t hsa_sparse_attention_workspace_size(int M, int L, int H, int dtype, int block_k, int keep) {
  if (M <= 0 || L <= 0 || H <= 0 || keep < 1 || keep > HSA_SPARSE_MAX_KEEP || (block_k != 64 && block_k != 128) ||
      !sparse_sizes_ok(M, H))
    return 0;
  if (dtype == HSA_F32) {
    const int BQ = sparse_f32_rows(M, H, keep), S = sparse_f32_splits(M, H, keep, BQ, ~size_t(0));
    if (S <= 1) return 0;
    const size_t slots = (size_t)((M + BQ - 1) / BQ) * H * S * BQ;
    return align256(slots * 128 * sizeof(float)) + align256(slots * sizeof(float2)) + 256;
  }
  if (dtype != HSA_BF16) return 0;
  return tail_split_bytes(sparse_plan(M, H, keep, block_k));
}

extern "C" int hsa_sparse_attention(const void* d_q, int M, const void* d_k, const void* d_v, int L, int H, int dtype,
                                    int block_k, const int32_t* d_list, int keep, const int32_t* d_count, void* d_o,
                                    void* d_ws, size_t ws_bytes, void* stream) {
  if (dtype != HSA_BF16 && dtype != HSA_F32) return set_error(HSA_EINVAL, "sparse_attention: unknown dtype");
  if (M < 0 || L <= 0 || H <= 0) return set_error(HSA_EINVAL, "sparse_attention: need M >= 0, L > 0 and H > 0");
  if (block_k != 64 && block_k != 128) return set_error(HSA_EINVAL, "sparse_attention: need block_k = 64 or 128");
  if (keep < 1 || keep > HSA_SPARSE_MAX_KEEP)
    return set_error(HSA_EINVAL, "sparse_attention: need 1 <= keep <= 4096");
  if ((L - 1) / block_k >= kSpMaxBlocks)
    return set_error(HSA_EINVAL, "sparse_attention: more than 65535 blocks");
  if (!sparse_sizes_ok(M, H)) return set_error(HSA_EINVAL, "sparse_attention: M or H too large");
  if (M == 0) return HSA_OK;
  if (!d_q || !d_k || !d_v || !d_o || !d_list || !d_count || !aligned16(d_q) || !aligned16(d_k) || !aligned16(d_v) ||
      !aligned16(d_o) || (d_ws && !aligned16(d_ws)))
    return set_error(HSA_EINVAL, "sparse_attention: null or misaligned pointer");
  const SparseList sl{d_list, d_count, keep, block_k, (L - 1) / block_k + 1};
  cudaStream_t st = as_stream(stream);
  if (dtype == HSA_BF16) return sparse_bf16(d_q, M, d_k, d_v, L, H, sl, d_o, d_ws, ws_bytes, st);
  return sparse_f32(static_cast<const float*>(d_q), M, static_cast<const float*>(d_k), static_cast<const float*>(d_v), L,
                    H, sl, static_cast<float*>(d_o), d_ws, ws_bytes, st);
}
