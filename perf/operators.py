"""Workloads of the block-sparse attention and fused residual operators, with their plain forms.

Four operators of a video DiT block (heads of 128 channels, Q compacted rows, K and V cache rows):

  block_scores      s[h, t, b] = mean(Q rows of 128-row tile t) . mean(K rows of block b) / sqrt(128)
  block_select      per score row the `keep` best blocks: (score descending, index ascending), NaN as
                    +inf, -inf never, forced blocks ahead of all; the list ascending, filled with -1
  sparse_attention  o = softmax(q K_S^T / sqrt(128)) V_S over the keys S of the blocks listed for the
                    row's tile; a row whose list is empty gives 0
  residual_norm     X' = a X + gate * post(y + b);  h = pre(X') * (1 + mul) + add, the modulation row
                    of each token taken from a table

`run` computes them in elementary torch operations in 32 bits, or, where `own` is true, through the
framework's binding.
"""
import math

import torch

own = False

TILE = 128          # rows of a query tile
HEAD = 128          # channels of a head
EPS = 1e-6          # of the norms
FRAMES = 21         # latent frames of the video grids: one modulation row per frame


# ---------------------------------------------------------------- cases

def listed():
    return [
        # routing scores of a Wan-1.3B block, every token active
        dict(name="scores_full", op="scores", M=32760, L=32760, H=12, dtype="bf16", block=128),
        # a Wan-14B block at a quarter of the tokens, finer key blocks
        dict(name="scores_quarter_wide", op="scores", M=8190, L=32760, H=40, dtype="bf16", block=64),
        # the small float32 loop: a few rows active
        dict(name="scores_f32_few", op="scores", M=300, L=1024, H=2, dtype="f32", block=64),
        # lists of the first case: 32 of 256 blocks
        dict(name="select_full", op="select", H=12, tiles=256, blocks=256, keep=32, forced=0, closed=0.0),
        # the longest grid (75600 tokens), 64-key blocks, the conditioning frame's blocks forced and
        # a tenth of the blocks closed by the caller
        dict(name="select_long_forced", op="select", H=40, tiles=591, blocks=1182, keep=177, forced=57, closed=0.1),
        # self-attention of a Wan-1.3B block over an eighth of the cache
        dict(name="attn_full", op="attention", M=32760, L=32760, H=12, dtype="bf16", block=128, keep=32, uneven=False),
        # a Wan-14B block at a quarter of the tokens, lists of every length from 0 to 77
        dict(name="attn_quarter_uneven", op="attention", M=8190, L=32760, H=40, dtype="bf16", block=64, keep=77,
             uneven=True),
        # one new row against the longest cache: latency
        dict(name="attn_one_row", op="attention", M=1, L=75600, H=12, dtype="bf16", block=64, keep=118, uneven=False),
        # the small float32 loop
        dict(name="attn_f32_loop", op="attention", M=512, L=1024, H=2, dtype="f32", block=64, keep=8, uneven=False),
        # attention residual and the FFN's modulated LayerNorm, Wan-1.3B, one modulation row per frame
        dict(name="norm_full", op="norm", M=32760, D=1536, y="bf16", out="bf16", post="none", pre="layer", table=FRAMES,
             bias=True, scale=1.0),
        # sandwich norms with a residual scale at the Wan-14B width, y from a float32 reduction
        dict(name="norm_sandwich_wide", op="norm", M=8190, D=5120, y="f32", out="bf16", post="rms", pre="rms", table=1,
             bias=False, scale=0.5),
        # one row: latency
        dict(name="norm_one_row", op="norm", M=1, D=1536, y="f32", out="f32", post="layer", pre="layer", table=1,
             bias=True, scale=1.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scores", "select", "attention", "attention", "norm"])
    if op == "scores":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        H = rng.randint(1, 40)
        rows = min(75600, int((100e6 if dtype == "bf16" else 50e6) / (H * HEAD)))     # rows of Q and K together
        L = _log(rng, 60, rows * 3 // 4)
        return dict(op=op, M=_log(rng, 1, rows - L), L=L, H=H, dtype=dtype, block=rng.choice([64, 128]))
    if op == "select":
        H = rng.randint(1, 40)
        blocks = _log(rng, 3, 3000)
        tiles = _log(rng, 1, max(1, min(600, 28000000 // (H * blocks))))
        return dict(op=op, H=H, tiles=tiles, blocks=blocks, keep=_log(rng, 1, max(2, blocks // 2)),
                    forced=rng.choice([0, 0, max(1, blocks // 20)]), closed=rng.choice([0.0, 0.1, 0.6]))
    if op == "attention":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        H = rng.randint(1, 40 if dtype == "bf16" else 8)
        block = rng.choice([64, 128])
        L = _log(rng, 100, min(75600, int(150e6 / (H * HEAD))))
        keep = _log(rng, 1, max(1, (L + block - 1) // block // 2))
        most = (0.8e12 if dtype == "bf16" else 0.02e12) / (4.0 * keep * block * H * HEAD)
        M = _log(rng, 1, max(1, int(min(L, most))))
        return dict(op=op, M=M, L=L, H=H, dtype=dtype, block=block, keep=keep, uneven=rng.random() < 0.4)
    D = HEAD * rng.randint(1, 64)
    return dict(op=op, M=_log(rng, 1, min(75600, 50000000 // D)), D=D, y=rng.choice(["bf16", "f32"]),
                out=rng.choice(["bf16", "f32"]), post=rng.choice(["none", "rms", "layer"]),
                pre=rng.choice(["none", "rms", "layer"]), table=rng.choice([1, FRAMES]), bias=rng.random() < 0.5,
                scale=rng.choice([1.0, 0.5]))


# ---------------------------------------------------------------- inputs

_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _cdiv(a, b):
    return -(-a // b)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _rows(g, n, H, dtype):
    """n rows of H heads as RMSNorm leaves them: unit scale, with the part neighbouring tokens share."""
    base = _normal(g, _cdiv(n, 64), H * HEAD).repeat_interleave(64, 0)[:n]
    return (0.8 * _normal(g, n, H * HEAD) + 0.6 * base).to(_DTYPE[dtype])


def _counts(case):
    """Blocks listed for each (head, tile): `keep`, or every length from 0 to keep in turn."""
    H, T = case["H"], _cdiv(case["M"], TILE)
    if not case["uneven"]:
        return torch.full((H, T), case["keep"], dtype=torch.int32)
    return ((torch.arange(H * T) * 7 + 3) % (case["keep"] + 1)).to(torch.int32).view(H, T)


def prepare(case, seed):
    g, op, s = _gen(seed), case["op"], {"op": case["op"], "case": case}
    if op == "scores":
        H, T, B = case["H"], _cdiv(case["M"], TILE), _cdiv(case["L"], case["block"])
        s.update(q=_rows(g, case["M"], H, case["dtype"]), k=_rows(g, case["L"], H, case["dtype"]))
        if own:
            from token_sparse_denoising_b200 import hsa
            s["scores"] = torch.empty((H, T, B), device="cuda")
            s["ws"] = torch.empty(hsa.block_scores_workspace_size(case["M"], case["L"], H, case["block"]),
                                  dtype=torch.uint8, device="cuda")
    elif op == "select":
        H, T, B = case["H"], case["tiles"], case["blocks"]
        x = 0.3 * _normal(g, H, T, B) + 0.3 * _normal(g, H, 1, B)
        if case["closed"]:
            x[torch.rand((H, T, B), generator=g, device="cuda") < case["closed"]] = -math.inf
            x[:, T // 2] = -math.inf                     # a tile with nothing open
        s["x"] = x
        s["forced"] = None
        if case["forced"]:
            s["forced"] = (torch.arange(B, device="cuda") < case["forced"]).to(torch.uint8)
        if own:
            s["lists"] = torch.empty((H, T, case["keep"]), dtype=torch.int32, device="cuda")
            s["counts"] = torch.empty((H, T), dtype=torch.int32, device="cuda")
    elif op == "attention":
        M, L, H, keep = case["M"], case["L"], case["H"], case["keep"]
        T, B = _cdiv(M, TILE), _cdiv(L, case["block"])
        s.update(q=_rows(g, M, H, case["dtype"]), k=_rows(g, L, H, case["dtype"]), v=_rows(g, L, H, case["dtype"]))
        # lists as a selection leaves them: neighbouring tiles of a head share part of their blocks
        x = _normal(g, H, T, B) + _normal(g, H, 1, B)
        lists = torch.sort(torch.topk(x, keep, dim=2).indices, dim=2).values.to(torch.int32)
        s["counts"] = _counts(case).cuda()
        dead = torch.arange(keep, device="cuda") >= s["counts"][..., None]
        s["lists"] = torch.where(dead, torch.full_like(lists, -1), lists)
        if own:
            from token_sparse_denoising_b200 import hsa
            s["o"] = torch.empty_like(s["q"])
            n = hsa.sparse_attention_workspace_size(M, L, H, hsa.HSA_BF16 if case["dtype"] == "bf16" else hsa.HSA_F32,
                                                    case["block"], keep)
            s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    else:
        M, D, table = case["M"], case["D"], case["table"]
        s.update(X=_normal(g, M, D), y=(2.0 * _normal(g, M, D) + 0.3).to(_DTYPE[case["y"]]),
                 mod=0.3 * _normal(g, table, 3, D),      # rows (gate, mul, add) of each modulation row
                 b=0.1 * _normal(g, D) if case["bias"] else None,
                 post_g=1.0 + 0.1 * _normal(g, D) if case["post"] != "none" else None,
                 rows=None)
        if table > 1:
            s["rows"] = (torch.arange(M, device="cuda") * table // M).to(torch.int32)
        if own:
            s["X_out"] = torch.empty_like(s["X"])
            s["out"] = None if case["pre"] == "none" else torch.empty((M, D), dtype=_DTYPE[case["out"]], device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state, state["case"])


def _own_scores(s, c):
    from token_sparse_denoising_b200 import hsa
    hsa.block_scores(s["q"], s["k"], c["H"], c["block"], s["scores"], ws=s["ws"])
    return s["scores"]


def _own_select(s, c):
    from token_sparse_denoising_b200 import hsa
    hsa.block_select(s["x"], c["keep"], s["lists"], s["counts"], forced=s["forced"])
    return s["lists"], s["counts"]


def _own_attention(s, c):
    from token_sparse_denoising_b200 import hsa
    hsa.sparse_attention(s["q"], s["k"], s["v"], c["H"], c["block"], s["lists"], s["counts"], s["o"], ws=s["ws"])
    return s["o"]


def _own_norm(s, c):
    from token_sparse_denoising_b200 import hsa
    mod, D = s["mod"], c["D"]
    none = c["pre"] == "none"
    hsa.residual_norm(s["X"], s["y"], X_out=s["X_out"], out=s["out"], b=s["b"], post=c["post"], post_g=s["post_g"],
                      res_scale=c["scale"], gate=mod[:, 0], pre=c["pre"], mul=None if none else mod[:, 1],
                      add=None if none else mod[:, 2], modulate=True, mod_row=s["rows"])
    return (s["X_out"],) if none else (s["X_out"], s["out"])


def _block_means(x, H, size):
    """(H, blocks, 128) mean of each block of `size` rows (the last over the rows it has)."""
    n = x.shape[0]
    full = n // size * size
    parts = []
    if full:
        parts.append(x[:full].float().view(-1, size, H * HEAD).mean(1))
    if full < n:
        parts.append(x[full:].float().mean(0, keepdim=True))
    return torch.cat(parts).view(-1, H, HEAD).transpose(0, 1)


def _plain_scores(s, c):
    q, k = _block_means(s["q"], c["H"], TILE), _block_means(s["k"], c["H"], c["block"])
    return torch.matmul(q, k.transpose(1, 2)) / math.sqrt(HEAD)


def _plain_select(s, c):
    x = torch.where(torch.isnan(s["x"]), torch.full_like(s["x"], math.inf), s["x"])
    B, keep = c["blocks"], c["keep"]
    open_ = x > -math.inf
    order = torch.sort(x, dim=2, descending=True, stable=True).indices
    if s["forced"] is not None:
        f = s["forced"] != 0
        open_ = open_ | f
        first = f[order]
        order = torch.gather(order, 2, torch.sort((~first).to(torch.uint8), dim=2, stable=True).indices)
        nf = int(c["forced"])                            # forced blocks among themselves by index
        head = torch.sort(order[..., :nf], dim=2).values
        order = torch.cat([head, order[..., nf:]], dim=2)
    counts = torch.clamp(open_.sum(2), max=keep).to(torch.int32)
    lists = order[..., :keep]
    if keep > B:
        lists = torch.cat([lists, lists.new_full((*lists.shape[:2], keep - B), B)], dim=2)
    live = torch.arange(keep, device=lists.device) < counts[..., None]
    lists = torch.sort(torch.where(live, lists, torch.full_like(lists, B)), dim=2).values
    return torch.where(live, lists, torch.full_like(lists, -1)).to(torch.int32), counts


def _plain_attention(s, c):
    M, L, H, keep, size = c["M"], c["L"], c["H"], c["keep"], c["block"]
    T, B = _cdiv(M, TILE), _cdiv(L, size)
    q, k, v = s["q"], s["k"], s["v"]
    if M < T * TILE:
        q = torch.cat([q, q.new_zeros(T * TILE - M, H * HEAD)])
    if L < B * size:
        k = torch.cat([k, k.new_zeros(B * size - L, H * HEAD)])
        v = torch.cat([v, v.new_zeros(B * size - L, H * HEAD)])
    q = q.view(T, TILE, H, HEAD).permute(2, 0, 1, 3).reshape(H * T, TILE, HEAD)
    k, v = k.view(B, size, H, HEAD), v.view(B, size, H, HEAD)
    lists, counts = s["lists"].view(H * T, keep).long(), s["counts"].view(H * T)
    live = torch.arange(keep, device=q.device) < counts[:, None]
    lists = torch.where(live, lists, torch.zeros_like(lists))
    inside = live[..., None] & (lists[..., None] * size + torch.arange(size, device=q.device) < L)
    head = torch.arange(H, device=q.device).repeat_interleave(T)
    o = torch.empty((H * T, TILE, HEAD), dtype=q.dtype, device=q.device)
    step = max(1, int(2e8 / (keep * size * HEAD)))       # tiles at a time: 0.8 GB of gathered float32 keys
    for a in range(0, H * T, step):
        b = slice(a, a + step)
        n = lists[b].shape[0]
        kk = k[lists[b], :, head[b, None]].reshape(n, keep * size, HEAD).float()
        x = torch.matmul(q[b].float(), kk.transpose(1, 2)) / math.sqrt(HEAD)
        ok = inside[b].reshape(n, 1, keep * size)
        x = torch.where(ok, x, torch.full_like(x, -math.inf))
        m = x.amax(2, keepdim=True)
        p = torch.exp(x - torch.where(m > -math.inf, m, torch.zeros_like(m)))
        l = p.sum(2, keepdim=True)
        vv = v[lists[b], :, head[b, None]].reshape(n, keep * size, HEAD).float()
        w = torch.matmul(p, vv)
        o[b] = (w / torch.where(l > 0, l, torch.ones_like(l))).to(o.dtype)
    return o.view(H, T * TILE, HEAD).transpose(0, 1).reshape(T * TILE, H * HEAD)[:M].contiguous()


def _plain_norm_rows(x, kind):
    if kind == "layer":
        d = x - x.mean(1, keepdim=True)
        return d * torch.rsqrt((d * d).mean(1, keepdim=True) + EPS)
    return x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)


def _plain_norm(s, c):
    mod = s["mod"] if s["rows"] is None else s["mod"][s["rows"].long()]
    z = s["y"].float()
    if s["b"] is not None:
        z = z + s["b"]
    if c["post"] != "none":
        z = _plain_norm_rows(z, c["post"]) * s["post_g"]
    X = c["scale"] * s["X"] + mod[:, 0] * z
    if c["pre"] == "none":
        return (X,)
    h = _plain_norm_rows(X, c["pre"]) * (1.0 + mod[:, 1]) + mod[:, 2]
    return X, h.to(_DTYPE[c["out"]])


_PLAIN = {"scores": _plain_scores, "select": _plain_select, "attention": _plain_attention, "norm": _plain_norm}
_OWN = {"scores": _own_scores, "select": _own_select, "attention": _own_attention, "norm": _own_norm}


# ---------------------------------------------------------------- definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](s, case)


def _membership(n, size):
    """(blocks, n) matrix that averages the rows of each block."""
    w = (torch.arange(n, device="cuda") // size == torch.arange(_cdiv(n, size), device="cuda")[:, None]).double()
    return w / w.sum(1, keepdim=True)


def _exact_scores(s, c):
    out = []
    wq, wk = _membership(c["M"], TILE), _membership(c["L"], c["block"])
    for h in range(c["H"]):
        cols = slice(h * HEAD, (h + 1) * HEAD)
        q, k = wq @ s["q"][:, cols].double(), wk @ s["k"][:, cols].double()
        out.append(torch.einsum("td,bd->tb", q, k) / HEAD ** 0.5)
    return torch.stack(out)


def _exact_select(s, c):
    """Rank of a block = how many blocks come before it; the ones of rank below keep are listed."""
    H, T, B, keep = c["H"], c["tiles"], c["blocks"], c["keep"]
    x = s["x"].double()
    x = torch.where(torch.isnan(x), torch.full_like(x, math.inf), x).view(H * T, B)
    forced = torch.zeros(B, dtype=torch.bool, device="cuda") if s["forced"] is None else s["forced"] != 0
    lower = torch.arange(B, device="cuda")[None, :] < torch.arange(B, device="cuda")[:, None]     # [i, j]: j < i
    lists = torch.full((H * T, keep), -1, dtype=torch.int64, device="cuda")
    counts = torch.zeros(H * T, dtype=torch.int64, device="cuda")
    step = max(1, int(2e8 / (B * B)))
    for a in range(0, H * T, step):
        r = x[a:a + step]
        xi, xj, fi, fj = r[:, :, None], r[:, None, :], forced[:, None], forced[None, :]
        by_score = (xj > xi) | ((xj == xi) & lower)
        before = (fj & ~fi) | (fj & fi & lower) | (~fj & ~fi & by_score)
        rank = before.sum(2)
        chosen = (rank < keep) & ((r > -math.inf) | forced)
        place = torch.cumsum(chosen, 1) - 1
        row, col = torch.nonzero(chosen, as_tuple=True)
        lists[a + row, place[row, col]] = col
        counts[a:a + step] = chosen.sum(1)
    return lists.view(H, T, keep).to(torch.int32), counts.view(H, T).to(torch.int32)


def _exact_attention(s, c):
    """Attention over the whole cache with each key weighted by how often the row's tile lists its block."""
    M, L, H, size, keep = c["M"], c["L"], c["H"], c["block"], c["keep"]
    T, B = _cdiv(M, TILE), _cdiv(L, size)
    if 4.0 * M * L * H * HEAD > 60e12:
        return None
    times = torch.zeros((H * T, B + 1), dtype=torch.float64, device="cuda")
    use = torch.arange(keep, device="cuda") < s["counts"].view(-1, 1)
    where = torch.where(use, s["lists"].view(H * T, keep).long(), torch.full((1, 1), B, device="cuda"))
    times.scatter_add_(1, where, torch.ones_like(where, dtype=torch.float64))
    times = times[:, :B].view(H, T, B)
    key_block = torch.arange(L, device="cuda") // size
    out = torch.zeros((M, H * HEAD), dtype=torch.float64, device="cuda")
    rows = max(1, int(1.2e8 / (L * TILE))) * TILE
    for h in range(H):
        cols = slice(h * HEAD, (h + 1) * HEAD)
        k, v = s["k"][:, cols].double(), s["v"][:, cols].double()
        for a in range(0, M, rows):
            q = s["q"][a:a + rows, cols].double()
            tile = torch.arange(a, a + q.shape[0], device="cuda") // TILE
            weight = times[h][tile][:, key_block]
            logit = (q @ k.T) * HEAD ** -0.5
            logit = logit.masked_fill(weight == 0, -math.inf)
            top = logit.max(1, keepdim=True).values.clamp(min=-1e300)
            e = weight * torch.exp(logit - top)
            den = e.sum(1, keepdim=True)
            out[a:a + rows, cols] = (e @ v) / den.clamp(min=1e-300)
    return out


def _exact_norm(s, c):
    D = c["D"]
    row = torch.zeros(c["M"], dtype=torch.int64, device="cuda") if s["rows"] is None else s["rows"].to(torch.int64)
    gate, mul, add = (s["mod"][:, i].double().index_select(0, row) for i in range(3))

    def norm(t, kind):
        if kind == "none":
            return t
        if kind == "layer":
            t = t - t.sum(1, keepdim=True) / D
        return t / torch.sqrt(t.square().sum(1, keepdim=True) / D + EPS)

    z = s["y"].double() + (0.0 if s["b"] is None else s["b"].double())
    z = norm(z, c["post"]) * (1.0 if s["post_g"] is None else s["post_g"].double())
    X = s["X"].double() * c["scale"] + gate * z
    return (X,) if c["pre"] == "none" else (X, norm(X, c["pre"]) * (mul + 1.0) + add)


_EXACT = {"scores": _exact_scores, "select": _exact_select, "attention": _exact_attention, "norm": _exact_norm}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c, op = case, case["op"]
    if op == "scores":
        e = 2 if c["dtype"] == "bf16" else 4
        T, B, D = _cdiv(c["M"], TILE), _cdiv(c["L"], c["block"]), c["H"] * HEAD
        return {"bytes": (c["M"] + c["L"]) * D * e + 4 * c["H"] * T * B,
                "flops": (c["M"] + c["L"]) * D + 2 * T * B * D}
    if op == "select":
        n = c["H"] * c["tiles"]
        return {"bytes": 4 * n * (c["blocks"] + c["keep"] + 1), "flops": n * c["blocks"]}
    if op == "attention":
        e = 2 if c["dtype"] == "bf16" else 4
        counts, M, L, D = _counts(c), c["M"], c["L"], c["H"] * HEAD
        rows = torch.full((counts.shape[1],), TILE)
        rows[-1] = M - (counts.shape[1] - 1) * TILE
        pairs = int((counts.long() * rows).sum()) * c["block"]
        keys = min(L * c["H"], int(counts.sum()) * c["block"])       # K and V rows of all heads, each read once
        return {"bytes": 2 * M * D * e + 2 * keys * HEAD * e + 4 * (int(counts.sum()) + counts.numel()),
                "flops": 4 * pairs * HEAD}
    per = 8 + (2 if c["y"] == "bf16" else 4) + (0 if c["pre"] == "none" else 2 if c["out"] == "bf16" else 4)
    vec = 3 * c["table"] + (1 if c["bias"] else 0) + (0 if c["post"] == "none" else 1)
    return {"bytes": c["M"] * c["D"] * per + 4 * vec * c["D"], "flops": 12 * c["M"] * c["D"]}
