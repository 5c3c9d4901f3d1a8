"""The block-sparse and residual-norm kernels beyond their first wave of work: CTAs and warp groups that take
unit after unit and row after row, lists of the greatest length, and what the kernels leave behind when a wait
on the device gives up there.  Bounds of attention, scores and norms are those of test_gpu_sparse."""
import numpy as np
import pytest
import torch

from oracle import hsa_oracle as O
from tests._util import dev, host
from tests.test_gpu_sparse import DTYPES, U, _mean_magnitudes, attention_bound, cdiv, residual_bounds, run_attention
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


# ------------------------------------------------------------------ several units, rows and items each

def heads(seed, n, H, bf16):
    return S.normal(seed, (n, 128 * H), 1.0, bf16)


# 480 units on 148 SMs (a tail of 36), 301 (a tail of 5, split into many ranges), 100 (less than one wave)
@pytest.mark.parametrize("M,H,L,keep", [(5000, 12, 2000, 30), (5430, 7, 4100, 60), (2500, 5, 4100, 50)])
@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sparse_attention_over_several_waves(cuda_lib, M, H, L, keep, block, dtype):
    q, k, v = (heads(231 + i, n, H, dtype == "bf16") for i, n in enumerate((M, L, L)))
    B = cdiv(L, block)
    keep = min(keep, B - 1)
    lists, counts = uneven_lists(M, H, cdiv(M, 128), B, keep)
    want = O.sparse_attention(q, k, v, H, block, lists, counts)
    bound = attention_bound(q, k, v, H, block, lists, counts, dtype)
    for split in (True, False):
        got = run_attention(cuda_lib, q, k, v, H, block, lists, counts, dtype, split)
        assert cuda_lib.device_status() == 0
        assert np.all(np.abs(got - want) <= bound), (split, np.max(np.abs(got - want) - bound))


@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_entry_of_the_longest_lists_counts(cuda_lib, block, dtype):
    """Lists of 4096 and 4095 distinct blocks in any order, and one with an entry in another's place.  With q = 0
    every weight is 1, the sums count keys, below 2^24, and are exact; block b adds to channel b % 128 only, which
    32 blocks share, so an entry too few or too many moves a channel by 3 %.  Rounded: the weights of at most 32 ranges
    and their sums (3 u a range), the quotient, and the output to its type."""
    H, keep, M = 2, 4096, 3
    L, t = keep * block - 5, DTYPES[dtype][0]
    key = torch.arange(L, device="cuda")
    v = torch.zeros((L, 128 * H), dtype=t, device="cuda")
    for h in range(H):
        v[key, 128 * h + key // block % 128] = 1.0
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    k = torch.randn((L, 128 * H), generator=g, device="cuda").to(t)
    q, o = (torch.zeros((M, 128 * H), dtype=t, device="cuda") for _ in range(2))
    r = np.random.default_rng(11)
    lists = np.stack([r.permutation(keep), r.permutation(keep)]).astype(np.int32).reshape(H, 1, keep)
    lists[1, 0, 3000] = lists[1, 0, 5]
    ws = torch.empty(cuda_lib.sparse_attention_workspace_size(M, L, H, DTYPES[dtype][1], block, keep),
                     dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    size = np.full(keep, block)
    size[-1] -= 5
    for n in (keep, keep - 1):
        want = np.zeros((H, 128))
        for h in range(H):
            listed = lists[h, 0, :n]
            np.add.at(want[h], listed % 128, size[listed])
            want[h] /= size[listed].sum()
        tol = (3 * 32 + 3) * U + (2.0 ** -8 if dtype == "bf16" else 0.0)
        for w in (ws, None):
            o.fill_(float("nan"))
            cuda_lib.sparse_attention(q, k, v, H, block, dev(lists), dev(np.full((H, 1), n, np.int32)), o, ws=w)
            assert cuda_lib.device_status() == 0
            assert np.all(np.abs(host(o).reshape(M, H, 128) - want) <= tol * want)


@pytest.mark.parametrize("M,L,H,block,dtype", [(16500, 19200, 40, 64, "bf16"), (16500, 3000, 4, 128, "f32")])
def test_block_scores_over_several_waves(cuda_lib, M, L, H, block, dtype):
    """More than 128 query tiles, several block tiles a range, and many blocks of rows for every SM."""
    t = DTYPES[dtype][0]
    q, k = (heads(241 + i, n, H, dtype == "bf16") for i, n in enumerate((M, L)))
    out = torch.full((H, cdiv(M, 128), cdiv(L, block)), float("nan"), device="cuda")
    cuda_lib.block_scores(dev(q, t), dev(k, t), H, block, out)
    assert cuda_lib.device_status() == 0
    assert np.all(np.abs(host(out) - O.block_scores(q, k, H, block)) <= 388 * U * _mean_magnitudes(q, k, H, block))


# more rows than (slots + 1) x groups x 148, so that every slot is filled again: one, two, four, eight, sixteen warps a row
@pytest.mark.parametrize("M,D", [(24000, 128), (19500, 256), (7200, 1000), (4900, 1536), (3700, 2048), (1300, 5120),
                                 (930, 8192), (620, 12288)])
@pytest.mark.parametrize("ydt,post,pre", [("bf16", "rms", "layer"), ("f32", "layer", "rms"), ("f32", "none", "none")])
def test_residual_norm_over_many_rows(cuda_lib, M, D, ydt, post, pre):
    """In place, with modulation rows and an index out of range in the middle and in the last row."""
    X, y = S.normal(251, (M, D)), S.normal(252, (M, D), 3.0, ydt == "bf16")
    tab = S.normal(253, (5, 3, D), 0.5)
    r = np.random.default_rng(M)
    mod_row = r.integers(0, 5, M).astype(np.int32)
    bad = np.array([M // 2, M - 1])
    mod_row[bad] = 5, -1
    part = lambda i: None if i and pre == "none" else tab[np.clip(mod_row, 0, 4), i]
    c = dict(b=S.normal(254, (D,), 0.5), post=post, post_g=S.normal(255, (D,)) if post != "none" else None,
             post_b=None, res_scale=0.5, gate=part(0), pre=pre, mul=part(1), add=part(2), modulate=True)
    want_X, want_h = O.residual_norm(X, y, **c)
    bX, bh = residual_bounds(X, y, c, want_X, want_h)
    Xd, t = dev(X), dev(tab)
    out = None if pre == "none" else torch.full((M, D), 9.0, device="cuda")
    view = lambda i: None if i and pre == "none" else t[:, i]
    d = lambda a: None if a is None else dev(a)
    cuda_lib.residual_norm(Xd, dev(y, DTYPES[ydt][0]), out=out, b=d(c["b"]), post=post, post_g=d(c["post_g"]), res_scale=0.5,
                           gate=view(0), pre=pre, mul=view(1), add=view(2), mod_row=dev(mod_row))
    assert cuda_lib.device_status() == cuda_lib.HSA_EINDEX
    good = np.ones(M, bool)
    good[bad] = False
    got = host(Xd)
    assert np.array_equal(got[bad], X[bad])
    assert np.all(np.abs(got - want_X)[good] <= bX[good])
    if pre != "none":
        h = host(out)
        assert np.all(h[bad] == 9.0) and np.all(np.abs(h - want_h)[good] <= bh[good])


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
    shape = (H, cdiv(M, 128), cdiv(L, 64))
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
    lists, counts = (dev(a) for a in uneven_lists(1, H, 40, cdiv(L, block), keep))
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
