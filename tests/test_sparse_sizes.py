"""Sizes at the ends of their types: refused, or counted right, before anything reaches a GPU."""
import ctypes as C

import pytest

from token_sparse_denoising_b200 import build, hsa

FAKE, MAX = 1 << 20, 2 ** 31 - 1                           # aligned stand-in, never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return hsa.load()


@pytest.mark.parametrize("M,L,H", [(MAX, 1000, 2), (MAX - 100, 1000, 2), (300, MAX, 2), (MAX, MAX, 4096)])
@pytest.mark.parametrize("block", [64, 128])
def test_block_scores_of_the_largest_counts(lib, M, L, H, block):
    rows = -(-M // 128) + -(-L // block)
    assert lib.hsa_block_scores_workspace_size(M, L, H, block) == rows * H * 128 * 3 * 2     # a multiple of 256
    assert lib.hsa_block_scores(FAKE, M, FAKE, L, H, hsa.HSA_BF16, block, FAKE, FAKE, 1 << 62, None) == hsa.HSA_EINVAL


@pytest.mark.parametrize("M,H", [(MAX, 2), (MAX - 100, 1), (300, MAX // 128 + 1), (1 << 27, 4000), (1, MAX)])
@pytest.mark.parametrize("dtype", [hsa.HSA_BF16, hsa.HSA_F32])
def test_sparse_attention_refuses_what_it_cannot_count(lib, M, H, dtype):
    assert lib.hsa_sparse_attention_workspace_size(M, 1000, H, dtype, 64, 4) == 0
    assert lib.hsa_sparse_attention(FAKE, M, FAKE, FAKE, 1000, H, dtype, 64, FAKE, 4, FAKE, FAKE, None, 0,
                                    None) == hsa.HSA_EINVAL


def test_layer_step_sparse_refuses_heads_that_its_scores_would(lib):
    """Before the cache rows are written: the scores take at most 4096 heads."""
    sp, H = hsa.BlockSparsityC(64, 4, None), 4097
    w = hsa.LayerWeightsC(128 * H, H, 512, hsa.HSA_BF16)
    for name, _ in hsa.LayerWeightsC._fields_[4:15]:
        setattr(w, name, FAKE)
    assert lib.hsa_layer_step_sparse_workspace_size(10, 300, 128 * H, 512, hsa.HSA_BF16, C.byref(sp)) == 0
    assert lib.hsa_layer_step_sparse(C.byref(w), FAKE, FAKE, 300, FAKE, FAKE, FAKE, 10, FAKE, None, None, 0, C.byref(sp),
                                     FAKE, 1 << 62, None) == hsa.HSA_EINVAL
