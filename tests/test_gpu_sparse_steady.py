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
