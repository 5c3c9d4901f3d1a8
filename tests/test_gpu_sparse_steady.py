"""The block-sparse and residual-norm kernels beyond their first wave of work: CTAs and warp groups that take
unit after unit and row after row, and what they leave behind when a wait on the device gives up there."""
import numpy as np
import pytest
import torch

from oracle import hsa_oracle as O
from tests._util import dev, host
from token_sparse_denoising_b200 import synthetic as S

pytestmark = pytest.mark.gpu


def uneven_lists(seed, H, T, B, keep):
    """Lists of 0, 1, 2, 5, 6, 7 and many blocks in turn, each of distinct blocks in ascending order."""
    r = np.random.default_rng(seed)
    lists, counts = np.full((H * T, keep), -1, np.int32), np.zeros(H * T, np.int32)
    for u in range(H * T):
        n = min([0, 1, keep, 2, 5, int(r.integers(0, keep + 1)), 6, 7, keep - 1, 3][u % 10], keep)
        lists[u, :n] = np.sort(r.choice(B, n, replace=False))
        counts[u] = n
    return lists.reshape(H, T, keep), counts.reshape(H, T)


# ------------------------------------------------------------------ waits that give up in the middle

@pytest.mark.parametrize("M,D", [(23700, 256), (9000, 1536), (2000, 5120), (700, 8200)])
def test_residual_norm_rows_are_whole_or_untouched_after_a_stall(cuda_lib, M, D):
    """With the abort flag raised the waits for rows give up: in place, each row of X and its output are
    finished, bit for bit, or as they were; afterwards the same call finishes all of them."""
    X, y = dev(S.normal(201, (M, D))), dev(S.normal(202, (M, D), 2.0))
    want, out = X.clone(), torch.full((M, D), 9.0, device="cuda")
    cuda_lib.residual_norm(want, y, out=out, post="rms", pre="layer")
    want_out = out.clone()
    cuda_lib.selftest_wait_timeout()
    got, out = X.clone(), torch.full((M, D), 9.0, device="cuda")
    cuda_lib.residual_norm(got, y, out=out, post="rms", pre="layer")
    assert cuda_lib.device_status() == cuda_lib.HSA_ETIMEOUT
    done, kept = (got == want).all(1), (got == X).all(1)
    assert bool((done | kept).all())
    assert bool(((out == want_out).all(1) == done).all()) and bool(((out == 9.0).all(1) == kept).all())
    cuda_lib.residual_norm(X, y, out=out, post="rms", pre="layer")
    assert torch.equal(X, want) and torch.equal(out, want_out) and cuda_lib.device_status() == 0


@pytest.mark.parametrize("M,L,H,dtype", [(20000, 9000, 4, torch.bfloat16), (3000, 9000, 5, torch.float32)])
def test_block_scores_return_after_a_stall_in_the_middle(cuda_lib, M, L, H, dtype):
    """Several items a CTA and several tiles a range, with the abort flag raised: the call returns, writes its
    scores and nothing beside them, and the next one is right."""
    q, k = (dev(S.normal(211 + i, (n, 128 * H)), dtype) for i, n in enumerate((M, L)))
    shape = (H, -(-M // 128), -(-L // 64))
    want, guarded = torch.empty(shape, device="cuda"), torch.full((H + 2, *shape[1:]), 9.0, device="cuda")
    cuda_lib.block_scores(q, k, H, 64, want)
    cuda_lib.selftest_wait_timeout()
    cuda_lib.block_scores(q, k, H, 64, guarded[1:-1])
    assert cuda_lib.device_status() == cuda_lib.HSA_ETIMEOUT
    assert bool((guarded[0] == 9.0).all()) and bool((guarded[-1] == 9.0).all())
    cuda_lib.block_scores(q, k, H, 64, guarded[1:-1])
    assert torch.equal(guarded[1:-1], want) and cuda_lib.device_status() == 0


@pytest.mark.parametrize("block", [64, 128])
def test_sparse_attention_rows_are_whole_or_untouched_after_a_stall(cuda_lib, block):
    """480 units on 148 SMs, lists run whole, with the abort flag raised: each 64 columns of a row are right, bit
    for bit, or as they were (the two halves of a head's channels are written by two warps)."""
    M, L, H, keep, bf = 5000, 4000, 12, 30, torch.bfloat16
    q, k, v = (dev(S.normal(221 + i, (n, 128 * H), 1.0, True), bf) for i, n in enumerate((M, L, L)))
    lists, counts = (dev(a) for a in uneven_lists(1, H, 40, -(-L // block), keep))
    want = torch.empty_like(q)
    cuda_lib.sparse_attention(q, k, v, H, block, lists, counts, want)
    cuda_lib.selftest_wait_timeout()
    got = torch.full_like(q, 7.0)
    cuda_lib.sparse_attention(q, k, v, H, block, lists, counts, got)
    assert cuda_lib.device_status() == cuda_lib.HSA_ETIMEOUT
    piece = lambda a: a.view(M, 2 * H, 64)
    assert bool(((piece(got) == piece(want)).all(2) | (piece(got) == 7.0).all(2)).all())
    cuda_lib.sparse_attention(q, k, v, H, block, lists, counts, got)
    assert torch.equal(got, want) and cuda_lib.device_status() == 0
