"""Block-sparse self-attention inside the layer step, the models, a recorded run and the head-parallel
block.  The oracle chooses its own lists, so every case asserts that no choice is near: the scores of the
last block kept and the first one left are further apart than the bf16 path's q and k can move them."""
import ctypes as C

import numpy as np
import pytest
import torch

from oracle import hsa_oracle as O
from tests._util import assert_bf16_close, assert_f32_close, dev, host
from token_sparse_denoising_b200 import hsa, pipeline
from token_sparse_denoising_b200 import synthetic as S
from token_sparse_denoising_b200.sharded import EmulatedGroup, HeadParallelBlock, HeadShard, gather_block_output

# A mean logit averages the roundings of a tile's q rows and a block's k rows.  For full tiles: errors of at
# most 2^-7 of unit-scale values (normalised input, product, norm and rotation, each rounded to bf16) with
# random signs, 64 rows or more, 128 channels: a standard deviation below 2^-7 / 8 = 0.001 of the mean rows'
# products, which are themselves below 0.5 here; 0.003 is six of them.
GAP = 0.003


def _case(seed, grid, H, F, cross, M, bf16):
    N, D = grid.N, 128 * H
    bw = S.perturb_vectors(S.block_weights(seed, S.BlockShape(D, H, F, cross, 16), bf16, 0.05), seed + 1)
    idx = np.arange(N, dtype=np.int32) if M == N else S.scattered_mask(seed + 2, N, M)
    Kc, Vc = S.normal(seed + 3, (N, D), 1.0, bf16), S.normal(seed + 4, (N, D), 1.0, bf16)
    # blocks that differ in their means, so that scores are spread
    Kc = Kc + 0.7 * np.repeat(S.normal(seed + 5, (-(-N // 64), D)), 64, 0)[:N]
    Kc = S.round_bf16(Kc) if bf16 else Kc.astype(np.float32)
    ctx = S.normal(seed + 6, (16, D), 1.0, bf16) if cross else None
    return bw, idx, S.normal(seed + 7, (N, D)), Kc, Vc, ctx


def sparse_block(bw, x, idx, pos, Kc, Vc, ctx, H, block, keep, forced=None):
    """The oracle's block with block-sparse self-attention, and the smallest gap between a score kept and one
    left (infinite where nothing is left)."""
    q, k, v = O.qkv_projection(bw, x[idx], np.asarray(pos)[idx])
    Kc, Vc = np.array(Kc, float), np.array(Vc, float)
    Kc[idx], Vc[idx] = k, v
    s = O.block_scores(q, Kc, H, block)
    lists, counts = O.block_select(s, keep, forced)
    free = np.ones(s.shape[-1], bool) if forced is None else np.asarray(forced) == 0
    gap = np.inf
    for h in range(s.shape[0]):
        for t in range(s.shape[1]):
            kept = np.zeros(s.shape[-1], bool)
            kept[lists[h, t, :counts[h, t]]] = True
            if (kept & free).any() and (~kept).any():
                gap = min(gap, s[h, t][kept & free].min() - s[h, t][~kept].max())
    o = O.sparse_attention(q, Kc, Vc, H, block, lists, counts)
    return O.block_tail(bw, x[idx], o, None if ctx is None else O.context_kv(bw, ctx)), Kc, gap


CASES = [(S.Grid(3, 10, 10), 300, 64, 2, True), (S.Grid(3, 10, 10), 150, 64, 2, False),
         (S.Grid(3, 10, 10), 1, 64, 1, True), (S.Grid(4, 12, 12), 576, 128, 3, False),
         (S.Grid(4, 12, 12), 70, 128, 2, True)]


def _seed(case, bf16):
    """The first seed of a fixed row whose choices are far from each other."""
    grid, M, block, keep, cross = case
    for seed in range(100, 700, 10):
        bw, idx, x, Kc, Vc, ctx = _case(seed, grid, 2, 512, cross, M, bf16)
        if sparse_block(bw, x, idx, S.token_positions(grid), Kc, Vc, ctx, 2, block, keep)[2] > GAP:
            return seed
    raise AssertionError("no seed with clear choices")


@pytest.mark.parametrize("case", CASES)
def test_cases_have_clear_choices(case):
    assert _seed(case, True) is not None and _seed(case, False) is not None


def _run_step(bw, bf16, grid, idx, x, Kc, Vc, ctx, sp):
    N, D = x.shape
    dt = torch.bfloat16 if bf16 else torch.float32
    w = hsa.LayerWeights(bw, "cuda", bf16)
    kc, vc, xA = dev(Kc, dt), dev(Vc, dt), torch.empty((len(idx), D), device="cuda")
    ws = torch.full((hsa.layer_step_workspace_size(len(idx), D, bw.w_1.shape[0], w.dtype, N, sp),), 255,
                    dtype=torch.uint8, device="cuda")
    ck = cv = None
    if ctx is not None:
        ck, cv = (torch.empty((ctx.shape[0], D), dtype=dt, device="cuda") for _ in range(2))
        cws = torch.empty(hsa.context_kv_workspace_size(ctx.shape[0], D), dtype=torch.uint8, device="cuda")
        hsa.context_kv(dev(ctx, dt), w.t["w_kv2"], w.t["b_kv2"], w.t["g_k2"], ck, cv, cws)
    hsa.layer_step(w, kc, vc, xA, dev(idx), dev(S.token_positions(grid)), ws, x_src=dev(x), ctx_k=ck, ctx_v=cv,
                   sparsity=sp)
    assert hsa.device_status() == 0
    return host(xA), host(kc)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("bf16", [True, False])
def test_layer_step_sparse_matches_oracle(cuda_lib, case, bf16):
    grid, M, block, keep, cross = case
    bw, idx, x, Kc, Vc, ctx = _case(_seed(case, bf16), grid, 2, 512, cross, M, bf16)
    want, Kw, _ = sparse_block(bw, x, idx, S.token_positions(grid), Kc, Vc, ctx, 2, block, keep)
    got, kc = _run_step(bw, bf16, grid, idx, x, Kc, Vc, ctx, hsa.BlockSparsity(keep, block))
    close = assert_bf16_close if bf16 else assert_f32_close
    close(got - x[idx], want - x[idx], "block output delta")
    close(kc[idx], Kw[idx], "fresh K rows")


@pytest.mark.gpu
@pytest.mark.parametrize("bf16", [True, False])
def test_layer_step_sparse_with_every_block_is_the_dense_step(cuda_lib, bf16):
    grid = S.Grid(3, 10, 10)
    bw, idx, x, Kc, Vc, ctx = _case(200, grid, 2, 512, True, 140, bf16)
    want, _, _ = O.dit_block_active(bw, x[idx], idx, S.token_positions(grid), Kc, Vc, O.context_kv(bw, ctx))
    for block, keep in ((64, 5), (128, 40)):
        got, _ = _run_step(bw, bf16, grid, idx, x, Kc, Vc, ctx, hsa.BlockSparsity(keep, block))
        (assert_bf16_close if bf16 else assert_f32_close)(got - x[idx], want - x[idx], "block output delta")


@pytest.mark.gpu
@pytest.mark.parametrize("bf16", [True, False])
def test_run_with_sparsity_and_its_recording(cuda_lib, bf16):
    """An HSA run whose blocks attend sparsely, the conditioning frame's blocks forced: the recorded run
    equals the eager one bit for bit, a sparse run differs from the dense one, and one that lists every
    block agrees with it."""
    grid, T = S.Grid(3, 16, 16), 4
    N = grid.N
    shape = S.BlockShape(256, 2, 512, False)
    pm = S.patch_model_weights(5, shape, 64, 2, bf16)
    pos = S.token_positions(grid)
    x0, vh0 = S.normal(6, (N, 64)), S.normal(7, (N, 64))
    forced = pipeline.forced_blocks(pipeline.conditioning_frame_mask(pos), 64)
    assert forced.tolist() == [1] * 4 + [0] * 8

    def run(sp, record=False):
        model = pipeline.PatchModel(pm, pos, N, bf16, sparsity=sp)
        r = pipeline.HSARun(model, x0, vh0, T, (4, 2), [N // 2, N - N // 2], 1, 1, 3.0)
        if record:
            r.replay(r.capture())
        else:
            r.run()
        assert hsa.device_status() == 0
        return host(r.x)

    dense, full = run(None), run(hsa.BlockSparsity(12, 64))
    sparse = run(hsa.BlockSparsity(6, 64, forced))
    assert np.array_equal(sparse, run(hsa.BlockSparsity(6, 64, forced), record=True))
    (assert_bf16_close if bf16 else assert_f32_close)(full - x0, dense - x0, "latent update")
    assert np.all(np.isfinite(sparse)) and not np.allclose(sparse, dense, atol=1e-4)


@pytest.mark.gpu
def test_head_parallel_block_with_sparsity(cuda_lib):
    case = CASES[1]
    grid, M, block, keep, cross = case
    H, N = 2, grid.N
    bw, idx, x, Kc, Vc, ctx = _case(_seed(case, True), grid, H, 512, cross, M, True)
    want, _, _ = sparse_block(bw, x, idx, S.token_positions(grid), Kc, Vc, ctx, H, block, keep)
    blocks = [HeadParallelBlock(bw, HeadShard(g, 2, H, 512, M), N, "cuda", cache_init=(Kc, Vc),
                                sparsity=hsa.BlockSparsity(keep, block)) for g in range(2)]
    EmulatedGroup.run(b.step(dev(x), dev(idx), dev(S.token_positions(grid))) for b in blocks)
    assert hsa.device_status() == 0
    assert_bf16_close(host(gather_block_output(blocks)) - x[idx], want - x[idx], "block output delta")


# ------------------------------------------------------------------ refusals (no GPU)

def test_layer_step_sparse_refusals():
    from token_sparse_denoising_b200 import build
    build.build_library()
    lib, fake = hsa.load(), 1 << 20
    w = hsa.LayerWeightsC(256, 2, 512, hsa.HSA_BF16)
    for name, _ in hsa.LayerWeightsC._fields_[4:15]:
        setattr(w, name, fake)
    ok = hsa.BlockSparsityC(64, 4, None)
    need = lib.hsa_layer_step_sparse_workspace_size(100, 300, 256, 512, hsa.HSA_BF16, C.byref(ok))
    assert need > lib.hsa_layer_step_workspace_size(100, 256, 512, hsa.HSA_BF16)
    call = lambda sp, bytes_: lib.hsa_layer_step_sparse(C.byref(w), fake, fake, 300, fake, fake, fake, 100, fake, None,
                                                        None, 0, sp, fake, bytes_, None)
    assert call(None, 1 << 30) == hsa.HSA_EINVAL
    assert call(C.byref(ok), need - 1) == hsa.HSA_EWORKSPACE
    for bad in (hsa.BlockSparsityC(32, 4, None), hsa.BlockSparsityC(64, 0, None), hsa.BlockSparsityC(64, 4097, None)):
        assert call(C.byref(bad), 1 << 30) == hsa.HSA_EINVAL
        assert lib.hsa_layer_step_sparse_workspace_size(100, 300, 256, 512, hsa.HSA_BF16, C.byref(bad)) == 0
    assert lib.hsa_layer_step_sparse_workspace_size(100, 300, 256, 512, 7, C.byref(ok)) == 0
    assert lib.hsa_layer_step_sparse_workspace_size(301, 300, 256, 512, hsa.HSA_BF16, C.byref(ok)) == 0
    with pytest.raises(ValueError):
        hsa.BlockSparsity(4, 100)
    with pytest.raises(ValueError):
        hsa.BlockSparsity(0)
    with pytest.raises(TypeError):
        hsa.BlockSparsity(4, 64, torch.ones(5))
    with pytest.raises(ValueError):
        hsa.BlockSparsity(4, 64, torch.ones(4, dtype=torch.uint8)).check(300)
    with pytest.raises(ValueError):
        pipeline._step_workspace(300, 256, 512, hsa.HSA_BF16, hsa.BlockSparsity(4, 64, torch.ones(4, dtype=torch.uint8)))


def test_step_workspace_covers_every_row_count():
    from token_sparse_denoising_b200 import build
    build.build_library()
    hsa.load()
    for H, dt, sp in ((2, hsa.HSA_BF16, hsa.BlockSparsity(9, 64)), (40, hsa.HSA_F32, hsa.BlockSparsity(40, 128)),
                      (5, hsa.HSA_F32, hsa.BlockSparsity(300, 64))):
        N, D, F = 2100, 128 * H, 64
        have = pipeline._step_workspace(N, D, F, dt, sp)
        assert all(hsa.layer_step_workspace_size(M, D, F, dt, N, sp) <= have for M in range(1, N + 1, 7))
