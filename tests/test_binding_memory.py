"""Memory that the binding takes or is given, on the CPU: whose stream a call's own scratch belongs to, and
buffers that a kernel could not use as they are.  A recorder stands in for libhsa; nothing is launched."""
import contextlib
import types

import pytest
import torch

from token_sparse_denoising_b200 import hsa, pipeline


class Recorder:
    """Every function of the library: notes its name and arguments and returns 0, or a size that is set."""

    def __init__(self, **sizes):
        self.sizes, self.calls = sizes, []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return self.sizes.get(name, 0)
        return call

    def launches(self):
        return [c for c in self.calls if not c[0].endswith("_size")]


class Stream:
    cuda_stream = 77


@pytest.fixture
def streams(monkeypatch):
    """The stream that is current while each tensor is allocated, in order (None: the caller's own)."""
    current, seen = [None], []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    def empty(*args, _empty=torch.empty, **kw):
        seen.append(current[-1])
        return _empty(*args, **kw)

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream())
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(hsa, "_current", lambda dev, s: 0 if s is None else s.cuda_stream)
    return seen


def use(monkeypatch, **sizes):
    lib = Recorder(**sizes)
    monkeypatch.setattr(hsa, "_lib", lib)
    return lib


@pytest.mark.parametrize("side", [True, False])
def test_block_scores_takes_its_scratch_on_the_calls_stream(monkeypatch, streams, side):
    lib = use(monkeypatch, hsa_block_scores_workspace_size=4096)
    q, k, scores = torch.zeros(300, 256), torch.zeros(1000, 256), torch.zeros(2, 3, 16)
    s = Stream() if side else None
    hsa.block_scores(q, k, 2, 64, scores, stream=s)
    assert streams == [s] and [c[0] for c in lib.launches()] == ["hsa_block_scores"]
    assert lib.launches()[0][1][-1] == (77 if side else 0)


@pytest.mark.parametrize("side", [True, False])
@pytest.mark.parametrize("pinned", [True, False])
def test_select_tokens_takes_its_scratch_on_the_calls_stream(monkeypatch, streams, side, pinned):
    lib = use(monkeypatch, hsa_select_tokens_workspace_size=512)
    s = Stream() if side else None
    hsa.select_tokens(torch.zeros(100), [40, 60], torch.zeros(100, dtype=torch.int8), torch.zeros(100, dtype=torch.int32),
                      stream=s, pinned=torch.zeros(100, dtype=torch.uint8) if pinned else None)
    assert streams == [s] and len(lib.launches()) == 1 and lib.launches()[0][1][-1] == 77


class Elsewhere:
    """As much of a device tensor as a check looks at."""
    is_cuda, device, shape = True, torch.device("cuda", 1), (5,)


def test_forced_blocks_have_to_be_on_the_steps_device(monkeypatch):
    """The layer step hands their address on: a CPU tensor's would be read by the kernel, another GPU's too."""
    lib = use(monkeypatch)
    mask = torch.ones(5, dtype=torch.uint8)
    idx, cache = torch.arange(4, dtype=torch.int32), torch.zeros(300, 256)
    w = types.SimpleNamespace(c=hsa.LayerWeightsC())
    monkeypatch.setattr(hsa, "_stream", lambda s: 0)
    with pytest.raises(ValueError, match="device"):
        hsa.layer_step(w, cache, cache, cache, idx, idx, cache, sparsity=hsa.BlockSparsity(4, 64, mask))
    with pytest.raises(ValueError, match="device"):
        pipeline._step_workspace(300, 256, 512, hsa.HSA_BF16, hsa.BlockSparsity(4, 64, mask))
    monkeypatch.setattr(hsa, "_need", lambda *a: None)
    monkeypatch.setattr(hsa, "_ptr", lambda t: None)
    sp = hsa.BlockSparsity(4, 64, Elsewhere())
    sp.check(300)
    sp.check(300, torch.device("cuda", 1))
    with pytest.raises(ValueError, match="device"):
        sp.check(300, torch.device("cuda", 0))
    assert not lib.launches()


@pytest.mark.parametrize("name,value", [("keep", 8), ("block", 128), ("forced", torch.zeros(5, dtype=torch.uint8))])
def test_block_sparsity_does_not_change_behind_its_struct(name, value):
    """The layer step reads the C struct: an attribute set later would leave it with the old numbers, and with
    the address of a mask that may have been freed."""
    sp = hsa.BlockSparsity(4, 64, torch.ones(5, dtype=torch.uint8))
    with pytest.raises(AttributeError):
        setattr(sp, name, value)
    assert (sp.c.keep, sp.c.block_k, sp.c.d_forced) == (sp.keep, sp.block, sp.forced.data_ptr())


GAPS = torch.zeros(1 << 16, dtype=torch.uint8)[::2]
W = types.SimpleNamespace(c=hsa.LayerWeightsC())
I32 = dict(dtype=torch.int32)


@pytest.mark.parametrize("call", [
    lambda x, v, i: hsa.block_scores(x, x, 2, 64, torch.zeros(2, 3, 5), ws=GAPS),
    lambda x, v, i: hsa.sparse_attention(x, x, x, 2, 64, torch.zeros(2, 3, 4, **I32), torch.zeros(2, 3, **I32), x, ws=GAPS),
    lambda x, v, i: hsa.select_tokens(v, [300], i, i, ws=GAPS),
    lambda x, v, i: hsa.attention(x, x, x, 2, x, ws=GAPS),
    lambda x, v, i: hsa.context_kv(x, x, v, v, x, x, GAPS),
    lambda x, v, i: hsa.layer_step(W, x, x, x, i, i, GAPS),
    lambda x, v, i: hsa.layer_step(W, x, x, x, i, i, GAPS, sparsity=hsa.BlockSparsity(4)),
    lambda x, v, i: hsa.patch_embed(x, i, x, v, x, GAPS),
    lambda x, v, i: hsa.velocity_head(x, v, x, v, x, GAPS),
    lambda x, v, i: hsa.iteration_host(W, x, x, i, i, x, x, 0.1, x, x, types.SimpleNamespace(c=hsa.HostSlotC()), GAPS),
    lambda x, v, i: hsa.iteration_host(W, x, x, i, i, x, x, 0.1, x, x, types.SimpleNamespace(c=hsa.HostSlotC()), v,
                                       sel_ws=GAPS)])
def test_workspaces_without_gaps(monkeypatch, streams, call):
    """The kernels write `bytes of ws` consecutive bytes: in a strided view they would run over what lies between."""
    lib = use(monkeypatch)
    with pytest.raises(ValueError, match="ws must be contiguous"):
        call(torch.zeros(300, 256), torch.zeros(300), torch.zeros(300, **I32))
    assert not lib.launches()


@pytest.mark.gpu
def test_block_scores_on_a_side_stream_keep_their_scratch(cuda_lib):
    """Scratch of a call that waits on a side stream is not handed out meanwhile, nor taken from memory that
    the current stream still uses: the scores are the current stream's own, and so is the other tensor."""
    M, L, H, block = 2000, 3000, 4, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    q, k = (torch.randn((n, 128 * H), generator=g, device="cuda").bfloat16() for n in (M, L))
    want, got = (torch.empty((H, 16, 47), device="cuda") for _ in range(2))
    n = cuda_lib.block_scores_workspace_size(M, L, H, block)
    cuda_lib.block_scores(q, k, H, block, want)
    side = torch.cuda.Stream()
    for late in (True, False):
        got.fill_(float("nan"))
        torch.cuda.synchronize()
        if late:                                          # the call waits, the current stream goes on
            with torch.cuda.stream(side):
                torch.cuda._sleep(20_000_000)
            cuda_lib.block_scores(q, k, H, block, got, stream=side)
            others = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        else:                                             # the current stream still writes what it has given back
            torch.cuda._sleep(20_000_000)
            others = [torch.full((n,), 255, dtype=torch.uint8, device="cuda")]
            kept = others[0].clone()
            del others[0]
            cuda_lib.block_scores(q, k, H, block, got, stream=side)
            others = [kept]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        assert all(bool((t == 255).all()) for t in others)
    assert cuda_lib.device_status() == 0
