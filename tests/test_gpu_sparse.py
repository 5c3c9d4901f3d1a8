"""Block scores, block selection, block-sparse attention and the fused residual norm on the GPU, each
against the fp64 oracle through the C ABI, at the sizes and inputs where they can go wrong.

Tolerances count roundings (u = 2^-24 for float32, 2^-8 for bf16 values) and are taken per element:
  scores      a mean of n <= 128 terms is within n u of the sum of magnitudes in any order of adding, its
              division one more; the product of two means over 128 channels 128 u; the scale 1 u: at most
              388 u times the product of the mean magnitudes
  attention   see attention_bound
  residual    see residual_bounds
"""
import numpy as np
import pytest
import torch

from oracle import hsa_oracle as O
from tests._util import dev, host
from token_sparse_denoising_b200 import synthetic as S

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DTYPES = {"bf16": (torch.bfloat16, 1), "f32": (torch.float32, 0)}


def cdiv(a, b):
    return -(-a // b)


def qkv(seed, M, L, H, bf16):
    return (S.normal(seed, (M, 128 * H), 1.0, bf16), S.normal(seed + 1, (L, 128 * H), 1.0, bf16),
            S.normal(seed + 2, (L, 128 * H), 1.0, bf16))


# ------------------------------------------------------------------ scores

@pytest.mark.parametrize("M,L,H,block", [(1, 1, 1, 64), (1, 64, 2, 64), (127, 129, 2, 128), (128, 128, 1, 128),
                                         (129, 65, 3, 64), (300, 1000, 2, 64), (640, 5000, 5, 128), (3, 9001, 2, 64),
                                         (8190, 130, 1, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_block_scores(cuda_lib, M, L, H, block, dtype):
    t = DTYPES[dtype][0]
    q, k, _ = qkv(11, M, L, H, dtype == "bf16")
    k += np.float32(2.0) * (np.arange(L) // block % 3 == 1)[:, None]           # exact in both types up to rounding
    k = S.round_bf16(k) if dtype == "bf16" else k
    out = torch.full((H, cdiv(M, 128), cdiv(L, block)), float("nan"), device="cuda")
    ws = torch.full((cuda_lib.block_scores_workspace_size(M, L, H, block),), 255, dtype=torch.uint8, device="cuda")
    cuda_lib.block_scores(dev(q, t), dev(k, t), H, block, out, ws=ws)
    assert cuda_lib.device_status() == 0
    want = O.block_scores(q, k, H, block)
    bound = 388 * U * _mean_magnitudes(q, k, H, block)
    assert np.all(np.abs(host(out) - want) <= bound)


def _mean_magnitudes(q, k, H, block):
    return O.block_scores(np.abs(q), np.abs(k), H, block)


def test_block_scores_keep_infinities_and_nan_to_their_blocks(cuda_lib):
    q, k, _ = qkv(12, 200, 500, 2, True)
    k[70, 5], k[300, 200] = np.nan, np.inf
    out = torch.empty((2, 2, 8), device="cuda")
    cuda_lib.block_scores(dev(q, torch.bfloat16), dev(k, torch.bfloat16), 2, 64, out)
    got = host(out)
    bad = ~np.isfinite(got)
    want = np.zeros((2, 2, 8), bool)
    want[0, :, 1] = True
    want[1, :, 4] = True
    assert np.array_equal(bad, want)


# ------------------------------------------------------------------ selection: bit-exact

def score_rows(seed, rows, B, kind):
    r = np.random.default_rng(seed)
    if kind == "ties":
        return r.choice(np.float32([0.0, -0.0, 0.5, 0.50000006, -1.5, np.nan, np.inf, -np.inf, 1e-40]), size=(rows, B))
    if kind == "const":
        return np.full((rows, B), -0.25, np.float32)
    if kind == "closed":
        s = r.standard_normal((rows, B)).astype(np.float32)
        s[r.random((rows, B)) < 0.9] = -np.inf
        s[rows // 2] = -np.inf
        return s
    return (r.standard_normal((rows, B)) * r.choice([1e-3, 1.0, 1e30], size=(rows, B))).astype(np.float32)


@pytest.mark.parametrize("rows,B,keep", [(1, 1, 1), (3, 1, 5), (9, 31, 4), (7, 128, 128), (8, 129, 17), (5, 256, 255),
                                         (20, 500, 33), (17, 1182, 177), (4, 1281, 1280), (3, 2048, 1), (3, 2049, 300),
                                         (2, 4097, 4096), (2, 16384, 1000), (1, 100, 4096), (7, 300, 40),
                                         (5, 700, 90), (6, 1000, 150), (3, 2700, 400), (2, 4000, 600)])
@pytest.mark.parametrize("kind", ["rand", "ties", "const", "closed"])
@pytest.mark.parametrize("forced", [None, "some", "all"])
def test_block_select_bit_exact(cuda_lib, rows, B, keep, kind, forced):
    s = score_rows(rows * B + keep, rows, B, kind)
    f = None if forced is None else np.ones(B, np.uint8) if forced == "all" else \
        (np.random.default_rng(B).random(B) < 0.05).astype(np.uint8) * 7
    lists = torch.full((rows, keep), -9, dtype=torch.int32, device="cuda")
    counts = torch.full((rows,), -9, dtype=torch.int32, device="cuda")
    cuda_lib.block_select(dev(s), keep, lists, counts, forced=None if f is None else dev(f))
    want_l, want_c = O.block_select(s, keep, f)
    assert np.array_equal(host(counts), want_c)
    assert np.array_equal(host(lists), want_l)


# ------------------------------------------------------------------ attention

def attention_bound(q, k, v, H, block, lists, counts, dtype):
    """Per element, with w the softmax weights and A = sum w |v|:
      logits      off by at most e = 130 u max(sum |q||k|) / sqrt(128) absolutely, so each weight by 2 e
      exp, sums   exp within 2^-21; n products and sums at 2 u each (a tensor core may truncate)
      bf16        the weight rounded once (2^-8) and the output once (2^-8)
    """
    n = max(1, int(counts.max()) * block)
    e = 0.0
    for h in range(H):
        c = slice(128 * h, 128 * h + 128)
        e = max(e, np.linalg.norm(q[:, c], axis=1).max() * np.linalg.norm(k[:, c], axis=1).max())
    rel = 2 * 130 * U * e / np.sqrt(128) + 2.0 ** -21 + 2 * n * 2 * U
    if dtype == "bf16":
        rel += 2 * 2.0 ** -8
    return rel * O.sparse_attention(q, k, v, H, block, lists, counts, absolute=True) + 1e-30


def random_lists(seed, H, T, B, keep, kind):
    r = np.random.default_rng(seed)
    lists = np.full((H, T, keep), -1, np.int32)
    counts = np.zeros((H, T), np.int32)
    for h in range(H):
        for t in range(T):
            n = {"full": min(keep, B), "uneven": int(r.integers(0, min(keep, B) + 1)), "empty": 0,
                 "one": 1, "twice": keep, "backwards": min(keep, B)}[kind]
            b = r.integers(0, B, n) if kind == "twice" else np.sort(r.choice(B, n, replace=False))
            lists[h, t, :n] = b[::-1] if kind == "backwards" else b
            counts[h, t] = n
    if kind in ("full", "one", "backwards") and counts.max() > 0:
        lists[0, 0, 0] = B - 1                            # the ragged last block first in a list
        if counts[0, 0] > 1 and B - 1 in lists[0, 0, 1:counts[0, 0]]:
            lists[0, 0, 1:counts[0, 0]][lists[0, 0, 1:counts[0, 0]] == B - 1] = 0 if B > 1 else B - 1
    return lists, counts


def run_attention(hsa, q, k, v, H, block, lists, counts, dtype, split=True, stream=None):
    t, code = DTYPES[dtype]
    M = q.shape[0]
    guard = torch.full((M + 3, 128 * H), 7.0, dtype=t, device="cuda")
    ws = None
    if split:
        n = hsa.sparse_attention_workspace_size(M, k.shape[0], H, code, block, lists.shape[2])
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")              # NaN bit patterns
    hsa.sparse_attention(dev(q, t), dev(k, t), dev(v, t), H, block, dev(lists), dev(counts), guard[:M], ws=ws,
                         stream=stream)
    assert torch.all(guard[M:] == 7.0)                    # rows behind the last query stay as they were
    return host(guard[:M])


SHAPES = [(1, 1, 1, 1), (1, 64, 1, 1), (1, 5000, 2, 40), (127, 63, 2, 1), (128, 128, 1, 2), (129, 200, 2, 3),
          (300, 1000, 2, 9), (257, 4100, 3, 17), (520, 1111, 5, 5)]


@pytest.mark.parametrize("M,L,H,keep", SHAPES)
@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("kind", ["full", "uneven", "backwards"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sparse_attention(cuda_lib, M, L, H, keep, block, kind, dtype):
    q, k, v = qkv(21, M, L, H, dtype == "bf16")
    q *= np.float32(2.0)
    lists, counts = random_lists(M + L, H, cdiv(M, 128), cdiv(L, block), keep, kind)
    bound = attention_bound(q, k, v, H, block, lists, counts, dtype)
    want = O.sparse_attention(q, k, v, H, block, lists, counts)
    for split in (True, False):
        got = run_attention(cuda_lib, q, k, v, H, block, lists, counts, dtype, split)
        assert cuda_lib.device_status() == 0
        assert np.all(np.abs(got - want) <= bound), (split, np.max(np.abs(got - want) - bound))


@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["empty", "one", "twice"])
def test_sparse_attention_list_kinds(cuda_lib, block, dtype, kind):
    """Empty lists give rows of exactly 0, one block alone, and an index listed twice counts twice."""
    M, L, H, keep = 200, 700, 2, 5
    q, k, v = qkv(31, M, L, H, dtype == "bf16")
    lists, counts = random_lists(5, H, 2, cdiv(L, block), keep, kind)
    got = run_attention(cuda_lib, q, k, v, H, block, lists, counts, dtype)
    assert cuda_lib.device_status() == 0
    want = O.sparse_attention(q, k, v, H, block, lists, counts)
    assert np.all(np.abs(got - want) <= attention_bound(q, k, v, H, block, lists, counts, dtype))
    if kind == "empty":
        assert np.all(got == 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("order", [1, -1])
def test_sparse_attention_growing_and_falling_maxima(cuda_lib, dtype, order):
    """Logits that rise (or fall) steeply from block to block: every tile moves the running maximum, or
    none after the first does."""
    M, L, H, block = 140, 1200, 1, 64
    q, k, v = qkv(41, M, L, H, True)
    k = S.round_bf16(k + q.mean(0) * (np.arange(L) // block)[:, None])
    q = S.round_bf16(q + 1.0)
    B = cdiv(L, block)
    lists = np.tile(np.arange(B, dtype=np.int32)[::order], (H, 2, 1)).copy()
    counts = np.full((H, 2), B, np.int32)
    want = O.sparse_attention(q, k, v, H, block, lists, counts)
    for split in (True, False):
        got = run_attention(cuda_lib, q, k, v, H, block, lists, counts, dtype, split)
        assert np.all(np.abs(got - want) <= attention_bound(q, k, v, H, block, lists, counts, dtype))


@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sparse_attention_reads_only_what_is_listed(cuda_lib, block, dtype):
    """NaN and infinity in unlisted blocks, and wild numbers behind the counts, change nothing."""
    M, L, H, keep = 150, 900, 2, 4
    q, k, v = qkv(51, M, L, H, dtype == "bf16")
    B = cdiv(L, block)
    lists, counts = random_lists(6, H, 2, B - 1, keep, "uneven")
    counts[0, 0] = max(counts[0, 0], 1)
    clean = run_attention(cuda_lib, q, k, v, H, block, lists, counts, dtype)
    for h in range(H):
        unlisted = np.ones(L, bool)
        for t in range(2):
            for b in lists[h, t, :counts[h, t]]:
                unlisted[b * block:(b + 1) * block] = False
        k[unlisted, 128 * h:128 * h + 128] = np.nan
        v[unlisted, 128 * h:128 * h + 128] = np.inf
        for t in range(2):
            lists[h, t, counts[h, t]:] = 2 ** 31 - 1
    dirty = run_attention(cuda_lib, q, k, v, H, block, lists, counts, dtype)
    assert cuda_lib.device_status() == 0
    assert np.array_equal(clean, dirty)


@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sparse_attention_skips_and_flags_bad_lists(cuda_lib, block, dtype):
    """A listed index outside the blocks is skipped (the other entries count), a count beyond the list is
    clamped; both flag HSA_EINDEX.  A list of nothing but bad indices gives 0."""
    M, L, H, keep = 200, 700, 1, 4
    q, k, v = qkv(61, M, L, H, dtype == "bf16")
    B = cdiv(L, block)
    good = np.int32([[[1, 3, 0, 2], [2, 4, 1, 0]]])
    counts = np.int32([[4, 4]])
    bad = good.copy()
    bad[0, 0, 1], bad[0, 1, 0] = -5, B
    keepers = np.int32([[[1, 0, 2, -1], [4, 1, 0, -1]]])
    want = O.sparse_attention(q, k, v, H, block, keepers, np.int32([[3, 3]]))
    bound = attention_bound(q, k, v, H, block, keepers, np.int32([[3, 3]]), dtype)
    got = run_attention(cuda_lib, q, k, v, H, block, bad, counts, dtype)
    assert cuda_lib.device_status() == cuda_lib.HSA_EINDEX
    assert np.all(np.abs(got - want) <= bound)
    got = run_attention(cuda_lib, q, k, v, H, block, good, np.int32([[9, -2]]), dtype)
    assert cuda_lib.device_status() == cuda_lib.HSA_EINDEX
    want = O.sparse_attention(q, k, v, H, block, good, np.int32([[4, 0]]))
    assert np.all(np.abs(got - want) <= attention_bound(q, k, v, H, block, good, np.int32([[4, 0]]), dtype))
    got = run_attention(cuda_lib, q, k, v, H, block, np.full_like(good, 2 ** 30), counts, dtype)
    assert cuda_lib.device_status() == cuda_lib.HSA_EINDEX and np.all(got == 0)
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sparse_attention_passes_nan_on(cuda_lib, dtype, split):
    """NaN in a listed block reaches exactly the rows whose tile and head list it (also through the joining
    of list ranges), everything else stays as it was."""
    M, L, H, keep, block = 200, 1000, 2, 9, 64
    q, k, v = qkv(65, M, L, H, dtype == "bf16")
    lists, counts = random_lists(8, H, 2, cdiv(L, block), keep, "full")
    lists[1, 1] = np.sort(np.setdiff1d(np.arange(cdiv(L, block)), [5])[:keep])
    lists[0, 0, :] = np.arange(keep)                       # lists block 5
    clean = run_attention(cuda_lib, q, k, v, H, block, lists, counts, dtype, split)
    k[5 * block + 3, :] = np.nan
    got = run_attention(cuda_lib, q, k, v, H, block, lists, counts, dtype, split)
    for h in range(H):
        for t in range(2):
            r, c = slice(128 * t, min(128 * t + 128, M)), slice(128 * h, 128 * h + 128)
            if 5 in lists[h, t]:
                assert np.all(np.isnan(got[r, c]))
            else:
                assert np.array_equal(got[r, c], clean[r, c])
    assert np.all(np.isnan(got[:128, :128])) and not np.any(np.isnan(got[128:, 128:]))


@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sparse_attention_longest_lists(cuda_lib, block, dtype):
    """Lists of 4096 entries, far more than there are blocks, every index many times, one of them odd."""
    M, L, H, keep = 3, 300, 1, 4096
    q, k, v = qkv(75, M, L, H, dtype == "bf16")
    B = cdiv(L, block)
    lists = np.random.default_rng(3).integers(0, B, (H, 1, keep)).astype(np.int32)
    for n in (keep, keep - 1):
        counts = np.full((H, 1), n, np.int32)
        want = _by_multiplicity(q, k, v, block, lists[0, 0, :n])
        bound = attention_bound(q, k, v, H, block, lists[:, :, :1], np.ones((H, 1), np.int32), dtype)
        rel = 4 * keep * block * U * np.abs(want).max() + bound.max()
        for split in (True, False):
            got = run_attention(cuda_lib, q, k, v, H, block, lists, counts, dtype, split)
            assert np.all(np.abs(got - want) <= rel)


def _by_multiplicity(q, k, v, block, listed):
    times = np.bincount(listed, minlength=cdiv(k.shape[0], block))[np.arange(k.shape[0]) // block]
    x = q.astype(float) @ k.astype(float).T / np.sqrt(128)
    e = np.exp(x - x.max(1, keepdims=True)) * times
    return e @ v.astype(float) / e.sum(1, keepdims=True)


def test_operators_return_after_a_stall_and_run_again(cuda_lib):
    """With the library's abort flag raised every wait gives up: the calls return, and after the status has been
    read the same calls give their results."""
    M, L, H, keep, block = 300, 3000, 2, 12, 64
    q, k, v = qkv(77, M, L, H, True)
    lists, counts = random_lists(9, H, 3, cdiv(L, block), keep, "uneven")
    bf = torch.bfloat16
    scores = torch.empty((H, 3, cdiv(L, block)), device="cuda")
    X, y = torch.zeros((50, 1536), device="cuda"), torch.ones((50, 1536), device="cuda")
    want = run_attention(cuda_lib, q, k, v, H, block, lists, counts, "bf16")
    cuda_lib.block_scores(dev(q, bf), dev(k, bf), H, block, scores)
    want_s = host(scores).copy()
    cuda_lib.selftest_wait_timeout()
    run_attention(cuda_lib, q, k, v, H, block, lists, counts, "bf16")
    cuda_lib.block_scores(dev(q, bf), dev(k, bf), H, block, scores)
    cuda_lib.residual_norm(X, y)
    assert cuda_lib.device_status() == cuda_lib.HSA_ETIMEOUT
    assert np.array_equal(run_attention(cuda_lib, q, k, v, H, block, lists, counts, "bf16"), want)
    cuda_lib.block_scores(dev(q, bf), dev(k, bf), H, block, scores)
    assert np.array_equal(host(scores), want_s)
    X.zero_()
    cuda_lib.residual_norm(X, y)
    assert torch.equal(X, y) and cuda_lib.device_status() == 0


def test_sparse_attention_far_offsets(cuda_lib):
    """A cache of more than 2^31 elements (32 heads x 560000 rows): the last blocks of the last head."""
    H, L, M, block = 32, 560000, 40, 64
    k = torch.zeros((L, 128 * H), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    tail = 500
    kt, vt = S.normal(71, (tail, 128 * H), 1.0, True), S.normal(72, (tail, 128 * H), 1.0, True)
    q = S.normal(73, (M, 128 * H), 1.0, True)
    k[L - tail:], v[L - tail:] = dev(kt, torch.bfloat16), dev(vt, torch.bfloat16)
    B = cdiv(L, block)
    first = (L - tail) // block + 1
    lists = np.tile(np.arange(first, B, dtype=np.int32), (H, 1, 1))
    counts = np.full((H, 1), B - first, np.int32)
    o = torch.empty((M, 128 * H), dtype=torch.bfloat16, device="cuda")
    cuda_lib.sparse_attention(dev(q, torch.bfloat16), k, v, H, block, dev(lists), dev(counts), o)
    assert cuda_lib.device_status() == 0
    cut = first * block - (L - tail)
    small = np.tile(np.arange(B - first, dtype=np.int32), (H, 1, 1))
    want = O.sparse_attention(q, kt[cut:], vt[cut:], H, block, small, counts)
    assert np.all(np.abs(host(o) - want) <= attention_bound(q, kt[cut:], vt[cut:], H, block, small, counts, "bf16"))
    scores = torch.empty((H, 1, B), device="cuda")
    cuda_lib.block_scores(dev(q, torch.bfloat16), k, H, block, scores)
    got = host(scores)[:, :, first:]
    assert np.all(np.abs(got - O.block_scores(q, kt[cut:], H, block)) <=
                  388 * U * _mean_magnitudes(q, kt[cut:], H, block))


# ------------------------------------------------------------------ residual norm

def residual_bounds(X, y, c, want_X, want_h):
    """(bound of X', bound of h), first order in u.  A norm's sums of at most D terms are added in at most
    64 + 13 steps (a thread's 48 values one after the other, then trees), so a mean is within 80 u of the mean magnitude
    and a normalised value within r 160 u (|t| + mean |t|) of the exact one, r = 1 / rms (of the centred
    row), for inputs t that are themselves off by e: another r (e + mean e) + |n| r rms(e)."""
    def norm_err(t, e, kind):
        if kind == "none":
            return e + U * np.abs(t)
        if kind == "layer":
            cen = t - t.mean(1, keepdims=True)
        else:
            cen = t
        r = 1.0 / np.sqrt((cen * cen).mean(1, keepdims=True) + 1e-6)
        mag = np.abs(t) + np.abs(t).mean(1, keepdims=True)
        e = e + 160 * U * mag
        return r * (e + e.mean(1, keepdims=True)) + np.abs(cen * r) * r * np.sqrt((e * e).mean(1, keepdims=True)) + \
            160 * U * np.abs(cen * r)

    one = lambda a: 1.0 if a is None else np.abs(a.astype(float))
    t = y.astype(float) + (0.0 if c["b"] is None else c["b"])
    e = norm_err(t, U * np.abs(t), c["post"])
    z = O._norm_rows(t, c["post"])
    ez = one(c["post_g"]) * (e + 4 * U * np.abs(z)) + (0.0 if c["post_b"] is None else 4 * U * np.abs(c["post_b"]))
    zg = np.abs(z * (1.0 if c["post_g"] is None else c["post_g"]) + (0.0 if c["post_b"] is None else c["post_b"]))
    eX = one(c["gate"]) * (ez + 4 * U * zg) + 4 * U * (np.abs(c["res_scale"] * X) + np.abs(want_X))
    if c["pre"] == "none":
        return eX + 1e-30, None
    n = O._norm_rows(want_X, c["pre"])
    eh = norm_err(want_X, eX, c["pre"])
    m = 1.0 if c["mul"] is None else np.abs((1.0 if c["modulate"] else 0.0) + c["mul"].astype(float))
    return eX + 1e-30, m * (eh + 4 * U * np.abs(n)) + 4 * U * (np.abs(want_h) + (0.0 if c["add"] is None else np.abs(c["add"]))) + 1e-30


def norm_case(seed, M, D, ydt, post, pre, gains, modulate=True, rows=False, scale=1.0):
    X, y = S.normal(seed, (M, D)), S.normal(seed + 1, (M, D), 3.0, ydt == "bf16") + np.float32(0.5)
    y = S.round_bf16(y) if ydt == "bf16" else y
    n = 5 if rows else 1
    v = lambda k, s=0.5: S.normal(seed + k, (D,), s) if gains else None
    tab = S.normal(seed + 9, (n, 3, D), 0.5) if gains or rows else None
    c = dict(b=v(2), post=post, post_g=v(3) if post != "none" else None, post_b=v(4) if post != "none" else None,
             res_scale=scale, pre=pre, modulate=modulate)
    return X, y, tab, c


@pytest.mark.parametrize("M,D", [(1, 8), (1, 1536), (5, 24), (9, 128), (33, 264), (7, 512), (6, 1032), (17, 1536),
                                 (3, 1544), (4, 2304), (3, 4104), (6, 5120), (2, 6144), (3, 8192), (2, 12288)])
@pytest.mark.parametrize("ydt,odt", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("post,pre", [("none", "layer"), ("rms", "rms"), ("layer", "none"), ("rms", "layer"),
                                      ("none", "none"), ("layer", "rms")])
@pytest.mark.parametrize("rows", [False, True])
def test_residual_norm(cuda_lib, M, D, ydt, odt, post, pre, rows):
    gains = (M + D) % 3 != 0 or rows
    modulate = D % 16 == 0
    X, y, tab, c = norm_case(M + D, M, D, ydt, post, pre, gains, modulate, rows, scale=0.75 if rows else 1.0)
    N = 2 * M + 3
    r = np.random.default_rng(D)
    idx = r.permutation(N)[:M].astype(np.int32)
    mod_row = r.integers(0, 5, N).astype(np.int32)
    pick = np.zeros(M, int) if not rows else mod_row[idx]
    part = lambda i: None if tab is None or (i and pre == "none") else tab[pick, i]
    c.update(gate=part(0), mul=part(1), add=part(2))
    want_X, want_h = O.residual_norm(X, y, **c)
    t = None if tab is None else dev(tab)
    view = lambda i: None if t is None or (i and pre == "none") else t[:, i]
    Xd, Xo = dev(X), torch.full((M, D), float("nan"), device="cuda")
    out = None if pre == "none" else torch.full((M, D), float("nan"), dtype=DTYPES[odt][0], device="cuda")
    d = lambda a: None if a is None else dev(a)
    kw = dict(out=out, b=d(c["b"]), post=post, post_g=d(c["post_g"]), post_b=d(c["post_b"]), res_scale=c["res_scale"],
              gate=view(0), pre=pre, mul=view(1), add=view(2), modulate=modulate,
              mod_row=dev(mod_row) if rows else None, idx=dev(idx) if rows else None)
    yd = dev(y, DTYPES[ydt][0])
    cuda_lib.residual_norm(Xd, yd, X_out=Xo, **kw)
    assert cuda_lib.device_status() == 0
    bX, bh = residual_bounds(X, y, c, want_X, want_h)
    assert np.array_equal(host(Xd), X)                    # the input stays
    assert np.all(np.abs(host(Xo) - want_X) <= bX)
    if pre != "none":
        bh = bh + (2.0 ** -8 * (np.abs(want_h) + bh) if odt == "bf16" else 0.0)
        assert np.all(np.abs(host(out) - want_h) <= bh)
    keep = None if out is None else out.clone()
    cuda_lib.residual_norm(Xd, yd, **kw)                  # in place: the same bits
    assert torch.equal(Xd, Xo) and (out is None or torch.equal(out, keep))


def test_residual_norm_constant_rows(cuda_lib):
    """Rows without variance (the norm is 0 / sqrt(eps)) and rows of zeros stay finite."""
    D = 1536
    X = np.zeros((4, D), np.float32)
    y = np.stack([np.zeros(D), np.full(D, 3.0), np.full(D, -1e4), np.ones(D)]).astype(np.float32)
    Xd, out = dev(X), torch.empty((4, D), device="cuda")
    cuda_lib.residual_norm(Xd, dev(y), out=out, post="layer", pre="layer")
    # a constant row's mean is exact to 80 u of the value, centred to that, times 1 / sqrt(1e-6)
    bound = 160 * U * np.abs(y) * 1e3
    assert np.all(np.abs(host(Xd)) <= bound)
    assert np.all(np.isfinite(host(out)))


def test_residual_norm_leaves_rows_with_bad_indices(cuda_lib):
    M, D, n = 6, 1544, 3
    X, y = S.normal(81, (M, D)), S.normal(82, (M, D))
    tab = dev(S.normal(83, (n, D)))
    mod_row = dev(np.int32([0, 3, 1, -1, 2, 0]))
    idx = dev(np.int32([0, 1, 2, 3, 6, -1]))
    Xd, out = dev(X), torch.full((M, D), 9.0, device="cuda")
    cuda_lib.residual_norm(Xd, dev(y), out=out, gate=tab, pre="rms", mod_row=mod_row, idx=idx)
    assert cuda_lib.device_status() == cuda_lib.HSA_EINDEX
    got, o = host(Xd), host(out)
    for r in (1, 3, 4, 5):
        assert np.array_equal(got[r], X[r]) and np.all(o[r] == 9.0)
    for r in (0, 2):
        assert not np.array_equal(got[r], X[r]) and np.all(o[r] != 9.0)


# ------------------------------------------------------------------ together, streams, graphs

@pytest.mark.parametrize("M,N,block,keep", [(700, 1500, 64, 6), (130, 1500, 128, 3), (1, 900, 64, 5)])
def test_operators_together(cuda_lib, M, N, block, keep):
    """Scores, selection, sparse attention, output projection and the fused residual norm in a row, as a
    block runs them: each step against the oracle on what the step before it gave."""
    hsa, H = cuda_lib, 2
    D, bf = 128 * H, torch.bfloat16
    q, k, v = qkv(91, M, N, H, True)
    forced = np.zeros(cdiv(N, block), np.uint8)
    forced[0] = 1
    scores = torch.empty((H, cdiv(M, 128), cdiv(N, block)), device="cuda")
    lists = torch.empty((H, cdiv(M, 128), keep), dtype=torch.int32, device="cuda")
    counts = torch.empty((H, cdiv(M, 128)), dtype=torch.int32, device="cuda")
    o, y = torch.empty((M, D), dtype=bf, device="cuda"), torch.empty((M, D), device="cuda")
    w = S.normal(95, (D, D), 0.06, True)
    X, tab = S.normal(96, (M, D)), S.normal(97, (3, D), 0.3)
    Xd, out, t = dev(X), torch.empty((M, D), dtype=bf, device="cuda"), dev(tab)
    dq, dk, dv = dev(q, bf), dev(k, bf), dev(v, bf)
    hsa.block_scores(dq, dk, H, block, scores)
    hsa.block_select(scores, keep, lists, counts, forced=dev(forced))
    ws = torch.empty(hsa.sparse_attention_workspace_size(M, N, H, hsa.HSA_BF16, block, keep), dtype=torch.uint8,
                     device="cuda")
    hsa.sparse_attention(dq, dk, dv, H, block, lists, counts, o, ws=ws)
    hsa.linear(o, dev(w, bf), None, hsa.EPI_F32, y)
    hsa.residual_norm(Xd, y, out=out, post="rms", gate=t[0], pre="layer", mul=t[1], add=t[2])
    assert hsa.device_status() == 0
    assert np.all(np.abs(host(scores) - O.block_scores(q, k, H, block)) <= 388 * U * _mean_magnitudes(q, k, H, block))
    wl, wc = O.block_select(host(scores), keep, forced)
    assert np.array_equal(host(lists), wl) and np.array_equal(host(counts), wc)
    want = O.sparse_attention(q, k, v, H, block, wl, wc)
    assert np.all(np.abs(host(o) - want) <= attention_bound(q, k, v, H, block, wl, wc, "bf16"))
    c = dict(b=None, post="rms", post_g=None, post_b=None, res_scale=1.0, gate=tab[0], pre="layer", mul=tab[1],
             add=tab[2], modulate=True)
    want_X, want_h = O.residual_norm(X, host(y), **c)
    bX, bh = residual_bounds(X, host(y), c, want_X, want_h)
    assert np.all(np.abs(host(Xd) - want_X) <= bX)
    assert np.all(np.abs(host(out) - want_h) <= bh + 2.0 ** -8 * (np.abs(want_h) + bh))


@pytest.mark.parametrize("M", [1, 300])
def test_captured_graph_follows_new_inputs(cuda_lib, M):
    """One recording of scores -> selection -> attention, replayed on other contents of the same buffers,
    equals the eager calls bit for bit; two recordings that share the workspaces alternate."""
    hsa, H, N, block, keep = cuda_lib, 2, 2000, 64, 12
    bf = torch.bfloat16
    T, B = cdiv(M, 128), cdiv(N, block)
    q = torch.zeros((M, 256), dtype=bf, device="cuda")
    k, v = torch.zeros((N, 256), dtype=bf, device="cuda"), torch.zeros((N, 256), dtype=bf, device="cuda")
    scores = torch.empty((H, T, B), device="cuda")
    lists = torch.empty((H, T, keep), dtype=torch.int32, device="cuda")
    counts = torch.empty((H, T), dtype=torch.int32, device="cuda")
    o = torch.empty((M, 256), dtype=bf, device="cuda")
    sws = torch.empty(hsa.block_scores_workspace_size(M, N, H, block), dtype=torch.uint8, device="cuda")
    ws = torch.empty(hsa.sparse_attention_workspace_size(M, N, H, hsa.HSA_BF16, block, keep), dtype=torch.uint8,
                     device="cuda")

    def calls():
        hsa.block_scores(q, k, H, block, scores, ws=sws)
        hsa.block_select(scores, keep, lists, counts)
        hsa.sparse_attention(q, k, v, H, block, lists, counts, o, ws=ws)

    calls()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            calls()
    for i in range(4):
        a, b, c = qkv(100 + i, M, N, H, True)
        q.copy_(dev(a, bf)), k.copy_(dev(b, bf)), v.copy_(dev(c, bf))
        o.fill_(float("nan"))
        graphs[i % 2].replay()
        got = o.clone()
        calls()
        assert torch.equal(got, o)
    assert hsa.device_status() == 0


def test_two_streams_at_once(cuda_lib):
    """The same calls on two streams with their own buffers, started together, give what they give alone."""
    hsa, bf, H, N, block, keep = cuda_lib, torch.bfloat16, 2, 6000, 64, 20
    sets = []
    for i in range(2):
        M = (2100, 700)[i]
        a, b, c = qkv(130 + i, M, N, H, True)
        d = dict(q=dev(a, bf), k=dev(b, bf), v=dev(c, bf), scores=torch.empty((H, cdiv(M, 128), cdiv(N, block)),
                                                                                device="cuda"),
                 lists=torch.empty((H, cdiv(M, 128), keep), dtype=torch.int32, device="cuda"),
                 counts=torch.empty((H, cdiv(M, 128)), dtype=torch.int32, device="cuda"),
                 X=torch.zeros((M, 256), device="cuda"), stream=torch.cuda.Stream(),
                 sws=torch.empty(hsa.block_scores_workspace_size(M, N, H, block), dtype=torch.uint8, device="cuda"),
                 ws=torch.empty(hsa.sparse_attention_workspace_size(M, N, H, hsa.HSA_BF16, block, keep),
                                dtype=torch.uint8, device="cuda"))
        d["o"] = torch.empty_like(d["q"])
        sets.append(d)

    def calls(d, stream):
        hsa.block_scores(d["q"], d["k"], H, block, d["scores"], ws=d["sws"], stream=stream)
        hsa.block_select(d["scores"], keep, d["lists"], d["counts"], stream=stream)
        hsa.sparse_attention(d["q"], d["k"], d["v"], H, block, d["lists"], d["counts"], d["o"], ws=d["ws"],
                             stream=stream)
        hsa.residual_norm(d["X"], d["o"], post="rms", stream=stream)

    want = []
    for d in sets:
        calls(d, None)
        torch.cuda.synchronize()
        want.append((d["o"].clone(), d["X"].clone()))
    for _ in range(5):
        for d in sets:
            d["o"].fill_(float("nan"))
            d["X"].zero_()
        torch.cuda.synchronize()
        for d in sets:
            calls(d, d["stream"])
        torch.cuda.synchronize()
        for d, (o, X) in zip(sets, want):
            assert torch.equal(d["o"], o) and torch.equal(d["X"], X)
    assert hsa.device_status() == 0


def test_calls_without_rows_do_nothing(cuda_lib):
    hsa, bf = cuda_lib, torch.bfloat16
    q, k = torch.empty((0, 256), dtype=bf, device="cuda"), torch.ones((100, 256), dtype=bf, device="cuda")
    lists, counts = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((2, 0, 3), (2, 0)))
    scores = torch.empty((2, 0, 2), device="cuda")
    before = hsa.launch_count()
    hsa.block_scores(q, k, 2, 64, scores)
    hsa.block_select(scores, 3, lists, counts)
    hsa.sparse_attention(q, k, k, 2, 64, lists, counts, torch.empty_like(q))
    X = torch.empty((0, 256), device="cuda")
    hsa.residual_norm(X, q, out=torch.empty_like(q), pre="layer")
    assert hsa.launch_count() == before and hsa.device_status() == 0


def test_binding_refuses_mixed_devices_types_and_shapes(cuda_lib):
    hsa, bf = cuda_lib, torch.bfloat16
    q, k = torch.ones((130, 256), dtype=bf, device="cuda"), torch.ones((100, 256), dtype=bf, device="cuda")
    scores = torch.empty((2, 2, 2), device="cuda")
    with pytest.raises(ValueError, match="shape"):
        hsa.block_scores(q, k, 2, 64, scores[:, :1])
    with pytest.raises(ValueError, match="device"):
        hsa.block_scores(q, k.cpu(), 2, 64, scores)
    with pytest.raises(TypeError):
        hsa.block_scores(q, k.float(), 2, 64, scores)
    with pytest.raises(ValueError, match="block"):
        hsa.block_scores(q, k, 2, 32, scores)
    with pytest.raises(ValueError, match="device"):
        hsa.block_scores(q, k, 2, 64, scores, ws=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(hsa.HsaError):
        hsa.block_scores(q, k, 2, 64, scores, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    lists, counts = torch.zeros((2, 2, 3), dtype=torch.int32, device="cuda"), torch.zeros((2, 2), dtype=torch.int32,
                                                                                          device="cuda")
    with pytest.raises(ValueError, match="shape"):
        hsa.block_select(scores, 4, lists, counts)
    with pytest.raises(TypeError):
        hsa.block_select(scores, 3, lists, counts.long())
    with pytest.raises(ValueError, match="shape"):
        hsa.block_select(scores, 3, lists, counts, forced=torch.zeros(3, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        hsa.sparse_attention(q, k, torch.ones((256, 100), dtype=bf, device="cuda").t(), 2, 64, lists, counts,
                             torch.empty_like(q))
    with pytest.raises(hsa.HsaError):
        hsa.sparse_attention(q, k, k, 2, 96, lists, counts, torch.empty_like(q))
    X, tab = torch.zeros((130, 256), device="cuda"), torch.zeros((4, 3, 256), device="cuda")
    with pytest.raises(ValueError, match="mod_row"):
        hsa.residual_norm(X, q, gate=tab[:, 0])
    with pytest.raises(ValueError, match="stride"):
        hsa.residual_norm(X, q, gate=tab[0, 0], pre="rms", out=q, mul=tab[:, 1])
    with pytest.raises(ValueError, match="rows of"):
        hsa.residual_norm(X, q, gate=tab[0, 0].bfloat16())
    with pytest.raises(hsa.HsaError):
        hsa.residual_norm(X, q, out=q.clone())             # an output without a norm
    assert hsa.device_status() == 0


def test_calls_use_the_stream_they_are_given(cuda_lib):
    """Inputs written late on a side stream: calls given that stream wait for them."""
    hsa, M, N, H = cuda_lib, 200, 600, 1
    bf = torch.bfloat16
    q, k, v = qkv(111, M, N, H, True)
    lists, counts = random_lists(1, H, 2, 10, 4, "full")
    want = run_attention(hsa, q, k, v, H, 64, lists, counts, "bf16", split=False)
    side = torch.cuda.Stream()
    dq, dk, dv, dl, dc = (torch.zeros_like(t) for t in (dev(q, bf), dev(k, bf), dev(v, bf), dev(lists), dev(counts)))
    o = torch.empty_like(dq)
    src = [dev(q, bf), dev(k, bf), dev(v, bf), dev(lists), dev(counts)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        for a, b in zip((dq, dk, dv, dl, dc), src):
            a.copy_(b)
    hsa.sparse_attention(dq, dk, dv, H, 64, dl, dc, o, stream=side)
    side.synchronize()
    assert np.array_equal(host(o), want)
