"""Block-sparse attention and the fused residual norm on the CPU: refusals of the C ABI and of the
binding before anything reaches a GPU, struct layout, and the oracle's own functions against worked cases."""
import ctypes as C

import numpy as np
import pytest
import torch

from oracle import hsa_oracle as O
from tests.test_abi import HEADER, _struct_fields
from token_sparse_denoising_b200 import build, hsa
from token_sparse_denoising_b200 import synthetic as S

FAKE = 1 << 20                                             # aligned stand-in, never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return hsa.load()


# ------------------------------------------------------------------ refusals of the C ABI

@pytest.mark.parametrize("change,code", [
    (dict(dtype=7), "EINVAL"), (dict(M=-1), "EINVAL"), (dict(L=0), "EINVAL"), (dict(H=0), "EINVAL"),
    (dict(block=32), "EINVAL"), (dict(block=0), "EINVAL"), (dict(q=None), "EINVAL"), (dict(k=None), "EINVAL"),
    (dict(scores=None), "EINVAL"), (dict(ws=None), "EINVAL"), (dict(q=FAKE + 8), "EINVAL"),
    (dict(ws_bytes=100), "EWORKSPACE"), (dict(L=64 * 70000), "EINVAL"), (dict(M=0), "OK")])
def test_block_scores_refusals(lib, change, code):
    a = dict(q=FAKE, M=300, k=FAKE, L=1000, H=2, dtype=hsa.HSA_BF16, block=64, scores=FAKE, ws=FAKE, ws_bytes=1 << 20)
    a.update(change)
    assert lib.hsa_block_scores(a["q"], a["M"], a["k"], a["L"], a["H"], a["dtype"], a["block"], a["scores"], a["ws"],
                                a["ws_bytes"], None) == getattr(hsa, "HSA_" + code)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), "EINVAL"), (dict(n_blocks=0), "EINVAL"), (dict(n_blocks=16385), "EINVAL"), (dict(keep=0), "EINVAL"),
    (dict(keep=4097), "EINVAL"), (dict(scores=None), "EINVAL"), (dict(lists=None), "EINVAL"),
    (dict(counts=None), "EINVAL"), (dict(rows=0, scores=None), "OK")])
def test_block_select_refusals(lib, change, code):
    a = dict(scores=FAKE, rows=4, n_blocks=100, keep=10, lists=FAKE, counts=FAKE)
    a.update(change)
    assert lib.hsa_block_select(a["scores"], a["rows"], a["n_blocks"], a["keep"], None, a["lists"], a["counts"],
                                None) == getattr(hsa, "HSA_" + code)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=2), "EINVAL"), (dict(M=-1), "EINVAL"), (dict(L=0), "EINVAL"), (dict(H=-3), "EINVAL"),
    (dict(block=96), "EINVAL"), (dict(keep=0), "EINVAL"), (dict(keep=4097), "EINVAL"), (dict(q=None), "EINVAL"),
    (dict(v=FAKE + 4), "EINVAL"), (dict(o=None), "EINVAL"), (dict(lists=None), "EINVAL"), (dict(counts=None), "EINVAL"),
    (dict(ws=FAKE + 8), "EINVAL"), (dict(L=64 * 65535 + 1), "EINVAL"), (dict(M=0, q=None), "OK")])
@pytest.mark.parametrize("dtype", [hsa.HSA_BF16, hsa.HSA_F32])
def test_sparse_attention_refusals(lib, change, code, dtype):
    a = dict(q=FAKE, M=300, k=FAKE, v=FAKE, L=1000, H=2, dtype=dtype, block=64, lists=FAKE, keep=4, counts=FAKE, o=FAKE,
             ws=None, ws_bytes=0)
    a.update(change)
    assert lib.hsa_sparse_attention(a["q"], a["M"], a["k"], a["v"], a["L"], a["H"], a["dtype"], a["block"], a["lists"],
                                    a["keep"], a["counts"], a["o"], a["ws"], a["ws_bytes"],
                                    None) == getattr(hsa, "HSA_" + code)


def _norm_args(**change):
    a = hsa.ResidualNormArgsC()
    a.d_X = a.d_X_out = a.d_y = a.d_out = FAKE
    a.dtype_y, a.dtype_out, a.M, a.D, a.pre, a.res_scale, a.n_mod, a.mod_stride = hsa.HSA_BF16, 0, 4, 256, 2, 1.0, 1, 256
    for k, v in change.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,code", [
    (dict(dtype_y=5), "EINVAL"), (dict(dtype_out=-1), "EINVAL"), (dict(post=3), "EINVAL"), (dict(pre=-1), "EINVAL"),
    (dict(M=-1), "EINVAL"), (dict(D=0), "EINVAL"), (dict(D=100), "EINVAL"), (dict(D=12296), "EINVAL"),
    (dict(d_X=None), "EINVAL"), (dict(d_X_out=None), "EINVAL"), (dict(d_y=None), "EINVAL"), (dict(d_out=None), "EINVAL"),
    (dict(d_y=FAKE + 8), "EINVAL"), (dict(d_gate=FAKE + 4), "EINVAL"), (dict(d_post_g=FAKE), "EINVAL"),
    (dict(pre=0), "EINVAL"), (dict(pre=0, d_out=None, d_mul=FAKE), "EINVAL"), (dict(d_mod_row=FAKE, N=3), "EINVAL"),
    (dict(d_mod_row=FAKE, N=4, n_mod=0), "EINVAL"), (dict(d_mod_row=FAKE, N=4, mod_stride=128), "EINVAL"),
    (dict(d_mod_row=FAKE, N=4, mod_stride=258), "EINVAL"), (dict(M=0, d_X=None), "OK")])
def test_residual_norm_refusals(lib, change, code):
    assert lib.hsa_residual_norm(C.byref(_norm_args(**change)), None) == getattr(hsa, "HSA_" + code)


def test_residual_norm_refuses_null_arguments(lib):
    assert lib.hsa_residual_norm(None, None) == hsa.HSA_EINVAL


def test_residual_norm_struct_matches_the_c_compiler(tmp_path):
    import shutil
    import subprocess
    fields = _struct_fields("hsa_residual_norm_args")
    assert fields == [f[0] for f in hsa.ResidualNormArgsC._fields_]
    packed = hsa.ResidualNormArgsC.PACKED
    values = [(i + 1) * 8 for i in range(len(fields))]
    a = hsa.ResidualNormArgsC.from_buffer_copy(packed.pack(*values))
    assert packed.size == C.sizeof(a) and [getattr(a, f) for f in fields] == values
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "%s"\nint main(void) {\n' % HEADER +
                   "".join(f'  printf("%zu\\n", offsetof(hsa_residual_norm_args, {f}));\n' for f in fields) +
                   '  printf("%zu\\n", sizeof(hsa_residual_norm_args));\n  return 0;\n}\n')
    subprocess.run([cc, "-std=c99", "-o", str(exe), str(src)], check=True, capture_output=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [getattr(hsa.ResidualNormArgsC, f).offset for f in fields] + [C.sizeof(hsa.ResidualNormArgsC)]


def test_workspace_sizes(lib):
    assert hsa.block_scores_workspace_size(300, 1000, 2, 64) >= (3 + 16) * 256 * 4
    assert hsa.block_scores_workspace_size(0, 1000, 2, 64) == 0
    assert hsa.block_scores_workspace_size(300, 1000, 2, 100) == 0
    # one query tile per head against a long list is split; a single listed tile is not
    assert hsa.sparse_attention_workspace_size(1, 75600, 12, hsa.HSA_BF16, 64, 118) > 0
    assert hsa.sparse_attention_workspace_size(1, 75600, 12, hsa.HSA_BF16, 64, 2) == 0
    assert hsa.sparse_attention_workspace_size(1, 1024, 2, hsa.HSA_F32, 64, 16) > 0
    assert hsa.sparse_attention_workspace_size(1, 75600, 12, hsa.HSA_BF16, 64, 5000) == 0


# ------------------------------------------------------------------ refusals of the binding

def test_binding_refuses_tensors_that_do_not_fit(lib):
    """Shapes, types, strides and devices are checked before the call (these are CPU tensors)."""
    q, k = torch.zeros(300, 256), torch.zeros(1000, 256)
    s = torch.zeros(2, 3, 16)
    with pytest.raises(ValueError, match="shape"):
        hsa.block_scores(q, k, 3, 64, s)
    with pytest.raises(ValueError, match="contiguous"):
        hsa.block_scores(torch.zeros(256, 300).t(), k, 2, 64, s)
    with pytest.raises(TypeError):
        hsa.block_scores(q.half(), k.half(), 2, 64, s)
    with pytest.raises(ValueError, match="device"):
        hsa.block_scores(q, k, 2, 64, s)
    lists, counts = torch.zeros(2, 3, 4, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(TypeError):
        hsa.block_select(s.double(), 4, lists, counts)
    with pytest.raises(ValueError, match="device"):
        hsa.block_select(s, 4, lists, counts)
    with pytest.raises(ValueError, match="shape"):
        hsa.sparse_attention(q[:, :128], k, k, 2, 64, lists, counts, torch.empty_like(q))
    with pytest.raises(ValueError, match="device"):
        hsa.sparse_attention(q, k, k, 2, 64, lists, counts, torch.empty_like(q))
    with pytest.raises(ValueError, match="post and pre"):
        hsa.residual_norm(q, q, post="batch")
    with pytest.raises(ValueError, match="device"):
        hsa.residual_norm(q, q)


# ------------------------------------------------------------------ the oracle against worked cases

def test_oracle_selection_worked_case():
    nan, inf = float("nan"), float("inf")
    s = np.float32([[3, 1, 1, -inf, 2, nan], [0.0, -0.0, -1, inf, nan, -inf], [-inf] * 6])
    lists, counts = O.block_select(s, 3)
    assert lists.tolist() == [[0, 4, 5], [0, 3, 4], [-1, -1, -1]] and counts.tolist() == [3, 3, 0]
    lists, counts = O.block_select(s, 2, forced=np.uint8([0, 0, 0, 1, 0, 0]))
    assert lists.tolist() == [[3, 5], [3, 4], [3, -1]] and counts.tolist() == [2, 2, 1]
    lists, counts = O.block_select(s, 4)
    assert lists[0].tolist() == [0, 1, 4, 5] and counts[2] == 0


def test_oracle_sparse_attention_is_attention_where_every_block_is_listed():
    q, k, v = S.normal(1, (130, 256)), S.normal(2, (200, 256)), S.normal(3, (200, 256))
    lists = np.tile(np.arange(4, dtype=np.int32), (2, 2, 1))
    counts = np.full((2, 2), 4, np.int32)
    full = O.attention(q, k, v)
    assert np.allclose(O.sparse_attention(q, k, v, 2, 64, lists, counts), full, rtol=1e-12, atol=1e-12)
    counts[1, 1] = 0
    part = O.sparse_attention(q, k, v, 2, 64, lists, counts)
    assert np.all(part[128:, 128:] == 0) and np.allclose(part[:128], full[:128])
    # scores are the mean logits
    logits = q[:128, :128].astype(float) @ k[64:128, :128].T / np.sqrt(128)
    assert O.block_scores(q, k, 2, 64)[0, 0, 1] == pytest.approx(logits.mean(), rel=1e-10)


def test_oracle_residual_norm_reduces_to_the_pieces():
    X, y, g = S.normal(4, (5, 256)), S.normal(5, (5, 256)), S.normal(6, (256,))
    mod = S.normal(7, (3, 256), 0.3)
    Xn, h = O.residual_norm(X, y, post="rms", post_g=g, gate=mod[0], pre="layer", mul=mod[1], add=mod[2])
    mod = mod.astype(float)
    want = X + mod[0] * O.rms_norm(y, g)
    assert np.allclose(Xn, want, rtol=1e-12)
    assert np.allclose(h, O.layer_norm(want) * (1 + mod[1]) + mod[2], rtol=1e-10)
