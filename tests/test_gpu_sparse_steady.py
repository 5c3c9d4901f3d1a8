"""The block-sparse and residual-norm kernels beyond their first wave of work: CTAs and warp groups that take
unit after unit and row after row, and what they leave behind when a wait on the device gives up there."""
import numpy as np
import pytest
import torch

from oracle import hsa_oracle as O
from tests._util import dev, host
from token_sparse_denoising_b200 import synthetic as S

pytestmark = pytest.mark.gpu


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
