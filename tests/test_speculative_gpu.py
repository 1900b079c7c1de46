"""GPU tests of the speculative-step calls against plain 64-bit formulas:
rtp_qk_norm_rope, rtp_tree_attn, rtp_kv_accept, and TreeDecodeLayer, which runs
them together.

Tolerances (u = 2^-24, half a step of fp32)
  * qk_norm_rope: a pair (a, b) of normed values of size r = |a| + |b|: the sum of
    squares, its root and the weight cost fewer than 40 roundings of a term, the
    cosine and sine are within pi u of the angle's rounding plus 4 u, two more
    roundings in the turn: 48 u r; plus half a step of a bf16 output.
  * tree_attn: scores are fp32 dots of 128 terms, so a logit is within 128 u S of
    its value, S = scale * sum |q_d k_d|, which moves every softmax weight by at
    most 2 * 128 u S (numerator and denominator); P as bf16 hi + lo keeps 2^-16;
    sums of n/16 partial products, truncated: n/16 * 2^-23; 32 u for the rest.
    All of it against the largest |v|; plus half a step of a bf16 output.
"""
import numpy as np
import pytest
import torch

from long_context_sparse_dim_b200 import rtp
from long_context_sparse_dim_b200 import workloads as wl
from long_context_sparse_dim_b200.layer import CachedDecodeLayer, TreeDecodeLayer

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = torch.bfloat16
D = 128


def _half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ---- qk_norm_rope --------------------------------------------------------------------

def _freqs(dev):
    return torch.tensor([500000.0 ** (-2.0 * i / D) for i in range(64)], dtype=torch.float64, device=dev)


def _norm_rope_ref(x, w, eps, where, freq, pairing):
    """(y, r) in fp64: rotated rows, and |a| + |b| of each value's pair."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()[None, :, None, :]
    ang = where.double()[:, None, :, None] * freq
    c, s = torch.cos(ang), torch.sin(ang)
    i = torch.arange(64, device=x.device)
    ia, ib = (i, i + 64) if pairing == "half" else (2 * i, 2 * i + 1)
    a, b = y[..., ia], y[..., ib]
    out, r = torch.empty_like(y), torch.empty_like(y)
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    r[..., ia] = r[..., ib] = a.abs() + b.abs()
    return out, r


def _check_norm_rope(got, ref, r, name):
    tol = 48 * U * r + (_half_step(got.dtype) * ref.abs() if got.dtype == BF else 0)
    bad = (got.double() - ref).abs() > tol
    assert not bool(bad.any()), f"{name}: {int(bad.sum())} values off, worst " \
                                f"{float(((got.double() - ref).abs() / tol.clamp_min(1e-300)).max()):.3g} x tolerance"


@pytest.mark.parametrize("B,Hq,Hk,T", [(1, 1, 1, 1), (3, 5, 1, 1), (2, 8, 2, 33), (1, 32, 8, 257), (7, 3, 3, 70)])
@pytest.mark.parametrize("pairing", ["half", "adjacent"])
@pytest.mark.parametrize("din,dout", [(BF, BF), (BF, torch.float32), (torch.float32, torch.float32),
                                      (torch.float32, BF)])
def test_norm_rope(B, Hq, Hk, T, pairing, din, dout):
    torch.manual_seed(B * 1000 + T)
    dev = "cuda"
    qkv = torch.randn(B, T, Hq + 2 * Hk, D, device=dev).to(din).transpose(1, 2)  # heads side by side
    q, k = qkv[:, :Hq], qkv[:, Hq: Hq + Hk]
    qw = (1 + 0.3 * torch.randn(Hq, D, device=dev)).to(BF if T % 2 else torch.float32)
    kw = 1 + 0.3 * torch.randn(1, D, device=dev)
    pos = torch.randint(0, 1 << 20, (B,), dtype=torch.int32, device=dev)
    offs = torch.randint(0, 90, (B, T), dtype=torch.int32, device=dev) if Hq % 2 else None
    where = pos[:, None] + (torch.arange(T, device=dev) if offs is None else offs)
    freq = _freqs(dev)
    qo, ko = torch.empty(B, Hq, T, D, dtype=dout, device=dev), torch.empty(B, Hk, T, D, dtype=dout, device=dev)
    rtp.qk_norm_rope(q, k, qw, kw, 1e-6, pos, freq, qo, ko, offs=offs, pairing=pairing)
    for x, w, o in ((q, qw, qo), (k, kw, ko)):
        _check_norm_rope(o, *_norm_rope_ref(x, w, 1e-6, where, freq, pairing), "both")
    # rotation alone, queries only, in place
    x = q.clone()
    rtp.qk_norm_rope(x, None, None, None, 0.0, pos, freq, x if din == dout else qo, None, offs=offs, pairing=pairing)
    _check_norm_rope(x if din == dout else qo, *_norm_rope_ref(q, None, 0.0, where, freq, pairing), "rotation only")
    # norm of the keys only
    rtp.qk_norm_rope(q, k, None, kw, 1e-6, pos, freq, qo, ko, offs=offs, pairing=pairing)
    _check_norm_rope(qo, *_norm_rope_ref(q, None, 0.0, where, freq, pairing), "q unnormed")
    _check_norm_rope(ko, *_norm_rope_ref(k, kw, 1e-6, where, freq, pairing), "k normed")


def test_norm_rope_extreme_rows():
    """Sums of squares outside fp32, zero rows, negative and far positions, a frequency of 0."""
    dev = "cuda"
    torch.manual_seed(5)
    x = torch.randn(1, 6, 4, D, device=dev)
    for h, scale in enumerate((1e18, 1e25, 1e-22, 1e-30, 0.0, 1.0)):
        x[:, h] *= scale
    w = torch.randn(1, D, device=dev)
    freq = _freqs(dev)
    freq[7] = 0.0
    for start in (-100, 0, 2 ** 31 - 4):
        pos = torch.tensor([start], dtype=torch.int32, device=dev)
        where = start + torch.arange(4, device=dev, dtype=torch.int64)[None]
        for eps in (1e-6, 1e-38):
            o = torch.empty_like(x)
            rtp.qk_norm_rope(x, None, w, None, eps, pos, freq, o, None)
            # the call's eps is fp32
            _check_norm_rope(o, *_norm_rope_ref(x, w, float(np.float32(eps)), where, freq, "half"), f"{start} {eps}")
    # an infinity or a NaN stays in its row
    x[0, 5, 1, 3], x[0, 5, 2, 100] = float("inf"), float("nan")
    rtp.qk_norm_rope(x, None, w, None, 1e-6, pos, freq, o, None)
    assert bool(torch.isfinite(o[0, 5, 0]).all()) and bool(torch.isfinite(o[0, 5, 3]).all())
    assert bool(torch.isnan(o[0, 5, 2]).all())


def test_norm_rope_rows_behind_an_empty_batch_stay():
    dev = "cuda"
    q = torch.zeros(2, 4, 0, D, dtype=BF, device=dev)
    i = torch.zeros(2, dtype=torch.int32, device=dev)
    rtp.qk_norm_rope(q, None, None, None, 1e-6, i, _freqs(dev), q.clone(), None)


# ---- tree_attn -------------------------------------------------------------------------

def _trees(B, T, kind, seed):
    rng = np.random.default_rng(seed)
    anc, depth = np.zeros((B, T, T), bool), np.zeros((B, T), np.int32)
    for b in range(B):
        for t in range(T):
            if t:
                par = t - 1 if kind == "chain" else int(rng.integers(max(0, t - 6), t))
                anc[b, t] = anc[b, par]
                depth[b, t] = depth[b, par] + 1
            anc[b, t, t] = True
    return anc, depth


def _bits(x):
    """bool array [..., n] -> int32 words [..., ceil(n / 32)] on the GPU."""
    n = x.shape[-1]
    words = max((n + 31) // 32, 1)
    full = np.zeros(x.shape[:-1] + (words * 32,), bool)
    full[..., :n] = x
    w = np.packbits(full, axis=-1, bitorder="little").view(np.int32)
    return torch.from_numpy(np.ascontiguousarray(w)).cuda()


def _tree_ref(q, k, v, lens, kn, vn, anc, depth, W, ring, sel, scale):
    """(o, tolerance without the output's rounding) in fp64, [B, Hq, T, D] and [B, Hq, T, 1]."""
    B, Hq, T, _ = q.shape
    Hk, N = k.shape[1], k.shape[2]
    G = Hq // Hk
    o = torch.zeros(B, Hq, T, D, dtype=torch.float64, device=q.device)
    tol = torch.zeros(B, Hq, T, 1, dtype=torch.float64, device=q.device)
    for b in range(B):
        n = max(int(lens[b]), 0) if ring else min(max(int(lens[b]), 0), N)
        position = torch.arange(max(0, n - N), n, device=q.device)
        rows = position % N if ring else position
        at = n + torch.as_tensor(depth[b], device=q.device).long().clamp_min(0)
        ok = torch.ones(T, len(position), dtype=torch.bool, device=q.device)
        okd = torch.as_tensor(anc[b], device=q.device)
        if W:
            ok = position[None] > at[:, None] - W
            okd = okd & (at[None] > at[:, None] - W)
        for h in range(Hq):
            a = ok if sel is None else ok & torch.as_tensor(sel[b, h], device=q.device)[:, rows]
            a = torch.cat((a, okd), 1)
            K = torch.cat((k[b, h // G][rows], kn[b, h // G])).double()
            V = torch.cat((v[b, h // G][rows], vn[b, h // G])).double()
            # a key that nobody attends may hold anything
            dead = ~a.any(0)
            K[dead], V[dead] = 0, 0
            x = (q[b, h].double() @ K.T) * scale
            S = (q[b, h].double().abs() @ K.abs().T).amax(1, keepdim=True) * abs(scale)
            x = x.masked_fill(~a, -float("inf"))
            m = x.amax(1, keepdim=True) if x.shape[1] else torch.full((T, 1), -float("inf"), device=q.device)
            p = torch.exp(x - torch.where(torch.isinf(m), 0.0, m))
            z = p.sum(1, keepdim=True)
            o[b, h] = (p @ V) / torch.where(z > 0, z, 1.0)
            tol[b, h] = V.abs().amax() * (2 * 128 * U * S + 2.0 ** -16 + a.shape[1] / 16 * 2.0 ** -23 + 32 * U)
    return o, tol


def _check_tree(got, ref, tol, name):
    t = tol + (_half_step(BF) * ref.abs() if got.dtype == BF else 0)
    assert bool(torch.isfinite(got).all()), name
    err = (got.double() - ref).abs()
    assert bool((err <= t).all()), f"{name}: worst {float((err / t.clamp_min(1e-300)).max()):.3g} x tolerance"


def _inputs(B, Hq, Hk, N, T, seed, layout="bhnd", dead=float("nan"), lens=None, ring=False):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda").to(BF)

    q, kn, vn = randn(B, Hq, T, D), randn(B, Hk, T, D), randn(B, Hk, T, D)
    if layout == "bnhd":
        k, v = randn(B, N, Hk, D).transpose(1, 2), randn(B, N, Hk, D).transpose(1, 2)
    else:
        k, v = randn(B, Hk, N, D), randn(B, Hk, N, D)
    for b in range(B):  # rows that hold no token
        n = max(int(lens[b]), 0)
        if n < N:
            k[b, :, n:], v[b, :, n:] = dead, dead
    return q, k, v, kn, vn


def _run_tree(q, k, v, lens, kn, vn, anc, depth, W, ring, sel, scale, out, ws=None):
    B, Hq, T, _ = q.shape
    Hk, N = k.shape[1], k.shape[2]
    o = torch.full((B, Hq, T, D), 7.0, dtype=out, device="cuda")
    s = None
    if sel is not None:
        m = _bits(sel).view(B * Hq * T, -1)
        s = rtp.Selection(tau_bits=m[:, 0], tiepos=m[:, 0], count=m[:, 0], mask=m)
    if ws is None:
        ws = rtp.workspace(rtp.tree_attn_workspace_size(B, Hq, T, Hk, N), "cuda")
    args = (q, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), kn, vn, _bits(anc), scale, o, ws)
    kw = dict(depth=torch.from_numpy(depth).cuda(), W=W, ring=ring, sel=s)
    rtp.tree_attn(*args, **kw)
    torch.cuda.synchronize()
    assert rtp.poll_device_error() == 0
    first = o.clone()
    o.fill_(3.0)
    rtp.tree_attn(*args, **kw)  # the workspace is ready again, and the bits are the same
    torch.cuda.synchronize()
    assert torch.equal(o.view(torch.uint8), first.view(torch.uint8))
    return o


TREE_CASES = [
    # B, Hq, Hk, N, lens, T, W, ring, kind, out
    (1, 1, 1, 1, [1], 1, 0, False, "chain", torch.float32),
    (1, 4, 1, 0, [0], 3, 0, False, "wide", BF),
    (2, 4, 2, 100, [0, 100], 5, 0, False, "wide", torch.float32),
    (3, 8, 2, 130, [127, 128, 129], 16, 0, False, "wide", BF),
    (2, 32, 8, 1000, [1000, 333], 8, 0, False, "wide", BF),
    (1, 8, 8, 700, [650], 27, 0, False, "chain", torch.float32),
    (2, 6, 2, 515, [515, 16], 31, 0, False, "wide", torch.float32),
    (1, 12, 3, 2000, [1999], 32, 0, False, "wide", BF),
    (1, 8, 2, 300, [300], 33, 0, False, "wide", torch.float32),      # 132 rows per KV head
    (1, 5, 1, 400, [390], 64, 0, False, "wide", BF),                 # 320 rows
    (1, 8, 1, 260, [255], 16, 0, False, "wide", torch.float32),      # 8 heads, 128 rows
    (1, 2, 1, 64, [40], 130, 0, False, "wide", torch.float32),       # tree rows of five words
    (1, 1, 1, 50, [50], 300, 0, False, "chain", BF),                 # more drafts than rows of a block
    (40, 2, 2, 90, list(range(50, 90)), 4, 0, False, "wide", torch.float32),
    (2, 8, 2, 6000, [6000, 5000], 16, 0, False, "wide", torch.float32),
    # windows inside a cache by position
    (2, 8, 2, 1000, [1000, 700], 16, 100, False, "chain", torch.float32),
    (2, 8, 2, 1000, [1000, 30], 16, 1, False, "wide", torch.float32),
    (1, 4, 2, 600, [599], 40, 20, False, "chain", torch.float32),    # the window also cuts the drafts
    (1, 4, 2, 600, [599], 9, 5000, False, "wide", BF),
    # rings
    (3, 8, 2, 128, [5, 128, 100000], 16, 128, True, "wide", torch.float32),
    (2, 6, 2, 100, [99, 101], 8, 100, True, "chain", torch.float32),
    (2, 6, 2, 103, [250, 64], 8, 60, True, "wide", BF),              # more rows than the window
    (1, 4, 1, 1, [9], 3, 1, True, "wide", torch.float32),
    (2, 24, 6, 1024, [5000, 1024], 16, 1024, True, "wide", torch.float32),
]


@pytest.mark.parametrize("i", range(len(TREE_CASES)))
def test_tree_attn(i):
    B, Hq, Hk, N, lens, T, W, ring, kind, out = TREE_CASES[i]
    q, k, v, kn, vn = _inputs(B, Hq, Hk, N, T, i, "bnhd" if i % 2 else "bhnd", lens=lens, ring=ring)
    anc, depth = _trees(B, T, kind, i)
    o = _run_tree(q, k, v, lens, kn, vn, anc, depth, W, ring, None, D ** -0.5, out)
    _check_tree(o, *_tree_ref(q, k, v, lens, kn, vn, anc, depth, W, ring, None, D ** -0.5), f"case {i}")


@pytest.mark.parametrize("density", [0.0, 0.01, 0.3, 1.0])
@pytest.mark.parametrize("B,Hq,Hk,N,lens,T,W", [(2, 8, 2, 1500, [1500, 900], 16, 0), (1, 4, 1, 64, [33], 1, 0),
                                                (1, 6, 2, 700, [700], 35, 0), (1, 8, 1, 9000, [8999], 16, 0),
                                                (1, 4, 2, 500, [500], 6, 77)])
def test_tree_attn_selected(B, Hq, Hk, N, lens, T, W, density):
    """Only selected committed keys; what no query of a KV head selects may hold NaN."""
    q, k, v, kn, vn = _inputs(B, Hq, Hk, N, T, 3, lens=lens)
    anc, depth = _trees(B, T, "wide", 3)
    rng = np.random.default_rng(8)
    runs = np.repeat(rng.random((B, Hq, T, (N + 24) // 25)) < density, 25, axis=-1)[..., :N]
    sel = runs | (rng.random((B, Hq, T, N)) < density / 20)
    sel[:, :, T // 2] = False  # a query that keeps nothing
    live = torch.from_numpy(sel.reshape(B, Hk, -1, N).any(2)).cuda()
    k[~live] = float("nan")
    v[~live] = float("inf")
    o = _run_tree(q, k, v, lens, kn, vn, anc, depth, W, False, sel, D ** -0.5, torch.float32)
    _check_tree(o, *_tree_ref(q, k, v, lens, kn, vn, anc, depth, W, False, sel, D ** -0.5), "selected")


def test_tree_attn_empty_rows_are_zero():
    """No committed token, a selection of nothing, an empty tree row: 0."""
    q, k, v, kn, vn = _inputs(2, 4, 2, 70, 4, 1, lens=[0, 70])
    anc, depth = _trees(2, 4, "wide", 1)
    anc[:, 2] = False
    sel = np.zeros((2, 4, 4, 70), bool)
    o = _run_tree(q, k, v, [0, 70], kn, vn, anc, depth, 0, False, sel, D ** -0.5, torch.float32)
    assert bool((o[:, :, 2] == 0).all())
    o = _run_tree(q, k, v, [-3, 70], kn, vn, anc, depth, 0, False, None, D ** -0.5, torch.float32)
    assert bool((o[0, :, 2] == 0).all()) and bool((o[1, :, 2] != 0).any())


def test_tree_attn_nan_in_a_key_that_another_query_attends():
    """A NaN value reaches the queries that attend its key, and no others (nor other heads or sequences)."""
    q, k, v, kn, vn = _inputs(2, 8, 2, 300, 8, 2, lens=[300, 300])
    anc, depth = _trees(2, 8, "wide", 2)
    sel = np.ones((2, 8, 8, 300), bool)
    sel[0, 1, 3:, 77] = False
    k2, v2 = k.clone(), v.clone()
    v2[0, 0, 77, 5] = float("nan")
    k2[0, 0, 78] = float("inf")
    sel[0, :4, :, 78] = False
    ref, tol = _tree_ref(q, k, v, [300, 300], kn, vn, anc, depth, 0, False, sel, D ** -0.5)
    m = _bits(sel).view(2 * 8 * 8, -1)
    s = rtp.Selection(tau_bits=m[:, 0], tiepos=m[:, 0], count=m[:, 0], mask=m)
    o = torch.empty(2, 8, 8, D, device="cuda")
    ws = rtp.workspace(rtp.tree_attn_workspace_size(2, 8, 8, 2, 300), "cuda")
    rtp.tree_attn(q, k2, v2, None, kn, vn, _bits(anc), D ** -0.5, o, ws, sel=s)
    torch.cuda.synchronize()
    hit = torch.from_numpy(sel[..., 77]).cuda()
    hit[1], hit[0, 4:] = False, False
    assert bool(torch.isnan(o[..., 5][hit]).all())
    clean = ~hit
    assert bool(torch.isfinite(o[clean]).all())
    err = (o.double() - ref).abs()
    assert bool((err <= tol)[clean.unsqueeze(-1).expand_as(err)].all())
    others = torch.arange(D, device="cuda") != 5  # the other dims of a hit row
    assert bool((err <= tol)[..., others].all())


@pytest.mark.parametrize("scale,mag", [(-0.05, 1.0), (0.0, 1.0), (1.0, 3.0), (0.0883, 30.0)])
def test_tree_attn_scales(scale, mag):
    """Negative and zero scales, peaked softmaxes with maxima far apart along the keys."""
    lens = [1200, 40]
    q, k, v, kn, vn = _inputs(2, 8, 2, 1200, 12, 4, lens=lens)
    k = (k.float() * torch.linspace(0.1, mag, 1200, device="cuda")[:, None]).to(BF)
    anc, depth = _trees(2, 12, "wide", 4)
    o = _run_tree(q, k, v, lens, kn, vn, anc, depth, 0, False, None, scale, torch.float32)
    sc = float(np.float32(scale))
    _check_tree(o, *_tree_ref(q, k, v, lens, kn, vn, anc, depth, 0, False, None, sc), f"{scale} {mag}")


def test_tree_attn_strided_rows_streams_and_graph():
    """Queries and outputs as views, another stream, one workspace for two shapes, a captured call replayed
    with other inputs."""
    lens = [900, 650]
    q, k, v, kn, vn = _inputs(2, 8, 2, 900, 10, 6, lens=lens)
    anc, depth = _trees(2, 10, "wide", 6)
    mask = _bits(anc)
    big = torch.full((2, 10, 16, D), 5.0, dtype=BF, device="cuda")
    o = big.transpose(1, 2)[:, 4:12]
    qv = torch.zeros(2, 10, 8, D, dtype=BF, device="cuda").transpose(1, 2).copy_(q)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = rtp.workspace(rtp.tree_attn_workspace_size(2, 8, 10, 2, 900), "cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    rtp.tree_attn(qv, k, v, lt, kn, vn, mask, D ** -0.5, o, ws, stream=stream)
    rtp.tree_attn(qv[:, :, :1], k, v, lt, kn[:, :, :1], vn[:, :, :1], mask[:, :1].contiguous(), D ** -0.5,
                  torch.empty(2, 8, 1, D, device="cuda"), ws, stream=stream)
    torch.cuda.synchronize()
    ref = _tree_ref(q, k, v, lens, kn, vn, anc, depth, 0, False, None, D ** -0.5)
    _check_tree(o, *ref, "views")
    assert bool((big[:, :, :4] == 5).all()) and bool((big[:, :, 12:] == 5).all())
    graph = torch.cuda.CUDAGraph()
    call = rtp.bind_tree_attn(qv, k, v, lt, kn, vn, mask, D ** -0.5, o, ws, stream=stream)
    with torch.cuda.graph(graph, stream=stream):
        call()
    lt.copy_(torch.tensor([13, 899], dtype=torch.int32))
    kn.copy_(torch.randn_like(kn, dtype=torch.float32).to(BF))
    v[0, :, :13] = 2.0
    v[1] = torch.randn(2, 900, D, device="cuda").to(BF)
    k[1] = torch.randn(2, 900, D, device="cuda").to(BF)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    _check_tree(o, *_tree_ref(q, k, v, [13, 899], kn, vn, anc, depth, 0, False, None, D ** -0.5), "replayed")


# ---- kv_accept ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("B,H,R,T,A,N,W", [(1, 1, 1, 1, 1, 1, 1), (3, 5, 2, 9, 6, 70, 16), (2, 4, 0, 20, 20, 8, 7),
                                           (2, 9, 9, 5, 5, 33, 1), (33, 8, 2, 40, 33, 200, 64)])
def test_kv_accept_equals_appending_the_rows(dtype, B, H, R, T, A, N, W):
    """Bit for bit what rtp_kv_append writes for the accepted rows, nothing else."""
    g = torch.Generator(device="cuda").manual_seed(B * 100 + T)
    rng = np.random.default_rng(T)
    L = H - R

    def rand(*s):
        return torch.randn(*s, generator=g, device="cuda").to(dtype)

    kn, vn = rand(B, H, T, D), rand(B, H, T, D)
    P = torch.randn(R, 16, D, generator=g, device="cuda") if R else None
    init = [rand(B, R, N, D), rand(B, R, N, D), rand(B, R, N, 16), rand(B, L, W, D), rand(B, L, W, D)]
    pos = rng.integers(-2, N + 1, B).astype(np.int32)
    count = rng.integers(0, A + 1, B).astype(np.int32)
    count[0] = A + 3  # clamped
    path = np.stack([np.sort(rng.permutation(T)[:A]) for _ in range(B)]).astype(np.int32)
    got, want = [x.clone() for x in init], [x.clone() for x in init]
    lens, rlens = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    dpos, dpath, dcount = (torch.from_numpy(x).cuda() for x in (pos, path, count))

    def caches(c):
        return (c[0] if R else None, c[1] if R else None, c[2] if R else None, c[3] if L else None, c[4] if L else None)

    rtp.kv_accept(kn, vn, dpos, dpath, dcount, R, P, *caches(got), lens, rlens if L else None)
    for b in range(B):
        n = min(int(count[b]), A)
        rows = torch.from_numpy(path[b, :n]).long().cuda()
        one, rone = torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
        rtp.kv_append(kn[b: b + 1, :, rows].contiguous(), vn[b: b + 1, :, rows].contiguous(), dpos[b: b + 1].clone(),
                      R, P, *(None if c is None else c[b: b + 1] for c in caches(want)), one, rone if L else None)
        assert int(lens[b]) == int(one)
        if L:
            assert int(rlens[b]) == int(rone)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_kv_accept_bad_rows_write_nothing():
    kn = torch.randn(1, 2, 4, D, device="cuda").to(BF)
    cache, ring = torch.zeros(1, 1, 10, D, dtype=BF, device="cuda"), torch.zeros(1, 1, 8, D, dtype=BF, device="cuda")
    idx, v = torch.zeros(1, 1, 10, 16, dtype=BF, device="cuda"), torch.zeros(1, 1, 10, D, dtype=BF, device="cuda")
    P = torch.randn(1, 16, D, device="cuda")
    path = torch.tensor([[2, -1, 4, 2 ** 31 - 1, 0]], dtype=torch.int32, device="cuda")
    i = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.zeros(1, dtype=torch.int32, device="cuda")
    rtp.kv_accept(kn, kn, i, path, i + 5, 1, P, cache, v, idx, ring, ring.clone(), out)
    assert int(out) == 5
    assert torch.equal(cache[0, 0, 0], kn[0, 0, 2]) and torch.equal(cache[0, 0, 4], kn[0, 0, 0])
    assert bool((cache[0, 0, 1:4] == 0).all()) and bool((ring[0, 0, 1:4] == 0).all())
    assert torch.equal(ring[0, 0, 4], kn[0, 1, 0])


# ---- together: the layer ---------------------------------------------------------------

@pytest.mark.parametrize("R,side", [(2, False), (2, True), (0, False), (4, False)])
def test_tree_steps_equal_plain_decode_steps(R, side):
    """A chain of drafts verified in one pass gives every token what decoding it step by step gives (with p >= 1,
    where the selection keeps every committed key), and accepting part of a tree leaves the caches as if the
    accepted tokens had been decoded one by one; then the next tree starts from there."""
    B, Hq, Hkv, N, W, T = 2, 16, 4, 600, 48, 12
    dev = "cuda"
    torch.manual_seed(11)
    P = torch.randn(max(R, 1), 16, D, device=dev)[:R] / 8
    freq = _freqs(dev)
    qw, kw = 1 + 0.2 * torch.randn(1, D, device=dev), 1 + 0.2 * torch.randn(1, D, device=dev)
    layer = TreeDecodeLayer(B, Hq, Hkv, N, R, W, 1.0, P, T, q_weight=qw, k_weight=kw, inv_freq=freq)
    plain = CachedDecodeLayer(B, Hq, Hkv, N, R, W, 1.0, P)
    n0 = 300
    ctx = [torch.randn(B, Hkv, n0, D, device=dev).to(BF) for _ in range(2)]
    layer.append(*ctx)
    plain.append(*ctx)
    lens = [n0] * B
    side_stream = torch.cuda.Stream() if side else None
    for step in range(3):
        raw = [torch.randn(B, H, T, D, device=dev).to(BF) for H in (Hq, Hkv, Hkv)]
        anc, depth = _trees(B, T, "chain" if step == 0 else "wide", step)
        mask, dep = _bits(anc), torch.from_numpy(depth).cuda()
        before = [x.clone() for x in (layer.k_cache, layer.k_ring)]
        o = layer.tree_step(*raw, mask, dep, side_stream=side_stream).clone()
        torch.cuda.synchronize()
        assert rtp.poll_device_error() == 0
        assert all(torch.equal(a, b) for a, b in zip(before, (layer.k_cache, layer.k_ring)))  # nothing taken yet
        # accept a root-to-leaf path, cut short differently per sequence
        path, count = np.zeros((B, T), np.int32), np.zeros(B, np.int32)
        for b in range(B):
            leaf = T - 1 if b == 0 else T // 2
            line = np.flatnonzero(anc[b, leaf])
            keep = max(1, len(line) - b * step)
            path[b, :keep], count[b] = line[:keep], keep
        steps = int(count.max())
        for i in range(steps):
            # one plain step; sequences that accepted fewer tokens step a token that is dropped again below
            pick = torch.from_numpy(path[:, i]).long().cuda()
            tok = torch.arange(B, device=dev)
            keep_lens = plain.lens.clone()
            saved = [x.clone() for x in (plain.k_cache, plain.v_cache, plain.k_idx, plain.k_ring, plain.v_ring)]
            q1, k1, v1 = (x[tok, :, pick][:, :, None] for x in (layer.tree_q, layer.tree_k, layer.tree_v))
            po = plain.step(q1, k1, v1).clone()
            for b in range(B):
                if i < count[b]:
                    got, want = o[b, :, path[b, i]].double(), po[b, :, 0].double()
                    vmax = float(max(plain.v_cache.abs().max() if R else 0, plain.v_ring.abs().max() if R < Hkv else 0))
                    # both sides are within the tolerance above of the same value: S <= |q| |k| scale
                    S = float(q1.float().norm(dim=-1).max() * max(ctx[0].float().norm(dim=-1).max(),
                                                                 layer.tree_k.float().norm(dim=-1).max()) * D ** -0.5)
                    tol = 2 * vmax * (2 * 128 * U * S + 2.0 ** -16 + (N + T) / 16 * 2.0 ** -23 + 32 * U)
                    assert float((got - want).abs().max()) <= tol, (step, i, b)
                else:  # undo this sequence's step
                    for x, s in zip((plain.k_cache, plain.v_cache, plain.k_idx, plain.k_ring, plain.v_ring), saved):
                        x[b] = s[b]
                    plain.lens[b] = keep_lens[b]
                    plain.ring_lens[b] = min(int(keep_lens[b]), W)
        layer.accept(torch.from_numpy(path).cuda(), torch.from_numpy(count).cuda())
        lens = [n + int(c) for n, c in zip(lens, count)]
        assert layer.lens.tolist() == lens == plain.lens.tolist()
        for a, b in ((layer.k_cache, plain.k_cache), (layer.v_cache, plain.v_cache), (layer.k_idx, plain.k_idx),
                     (layer.k_ring, plain.k_ring), (layer.v_ring, plain.v_ring)):
            assert torch.equal(a, b)
        if R < Hkv:
            assert torch.equal(layer.ring_lens, plain.ring_lens)


def test_tree_step_selects_by_top_p():
    """The retrieval heads' drafts attend the keys that rtp_topp_select keeps for each of them."""
    w = wl.DECODE_B8_N32K.replace(name="tree", B=2, N=3000, W=256, needles=8)
    inst = wl.generate(w)
    dev = torch.device("cuda")
    k, v = (torch.from_numpy(x).to(dev, BF) for x in (inst.k, inst.v))
    P = torch.from_numpy(inst.P).to(dev, torch.float32)
    T, R, G = 4, w.R, w.Hq // w.Hkv
    layer = TreeDecodeLayer(w.B, w.Hq, w.Hkv, w.N, R, w.W, 0.7, P, T)
    layer.append(k, v)
    q = torch.from_numpy(inst.q).to(dev, BF).expand(-1, -1, T, -1) * torch.tensor([1, -1, 2, 0.5], device=dev)[:, None]
    q = q.to(BF)
    kn, vn = torch.randn(2, w.B, w.Hkv, T, D, device=dev).to(BF)
    anc, depth = _trees(w.B, T, "wide", 0)
    o = layer.tree_step(q, kn, vn, _bits(anc), torch.from_numpy(depth).cuda())
    torch.cuda.synchronize()
    words = layer.tree_sel.mask.cpu().numpy().view(np.uint8)
    sel = np.unpackbits(words, axis=-1, bitorder="little")[:, : w.N].astype(bool).reshape(w.B, R * G, T, w.N)
    frac = sel.mean()
    assert 0.05 < frac < 0.9 and np.array_equal(sel.sum(-1).reshape(-1), layer.tree_sel.count.cpu().numpy())
    lens = [w.N] * w.B
    ref = _tree_ref(q[:, : R * G], k[:, :R], v[:, :R], lens, kn[:, :R], vn[:, :R], anc, depth, 0, False, sel, D ** -0.5)
    _check_tree(o[:, : R * G], *ref, "retrieval")
    ref = _tree_ref(q[:, R * G:], k[:, R:], v[:, R:], lens, kn[:, R:], vn[:, R:], anc, depth, w.W, False, None,
                    D ** -0.5)
    _check_tree(o[:, R * G:], *ref, "local")


# ---- the binding -------------------------------------------------------------------------

def test_binding_refuses_wrong_arrays():
    """Plain device arrays are described by their address alone, so the binding checks type, shape and layout."""
    z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    i32 = lambda *s: z(*s, dtype=torch.int32)  # noqa: E731
    q, kv, freq = z(2, 4, 3, D), z(2, 2, 3, D), _freqs("cuda")

    def rope(pos=i32(2), f=freq, offs=None, eps=1e-6):
        rtp.qk_norm_rope(q, kv, None, None, eps, pos, f, q, kv, offs=offs)

    for bad in (dict(pos=i32(3)), dict(pos=i32(2).long()), dict(pos=i32(2, 2)[:, 0]), dict(f=freq.float()),
                dict(f=freq[:63]), dict(offs=i32(2, 2)), dict(offs=i32(2, 6)[:, ::2])):
        with pytest.raises(ValueError, match="need a contiguous"):
            rope(**bad)
    with pytest.raises(TypeError):
        rope(eps="x")
    with pytest.raises(rtp.RtpError):
        rope(eps=-1.0)
    with pytest.raises(ValueError, match="current CUDA device"):
        rope(pos=torch.zeros(2, dtype=torch.int32))
    ws = rtp.workspace(rtp.tree_attn_workspace_size(2, 4, 3, 2, 8), "cuda")

    def attn(lens=None, mask=i32(2, 3, 1), depth=None, sel=None, ws=ws, o=q, W=0):
        s = None if sel is None else rtp.Selection(tau_bits=sel, tiepos=sel, count=sel, mask=sel)
        rtp.tree_attn(q, z(2, 2, 8, D), z(2, 2, 8, D), lens, kv, kv, mask, 0.1, o, ws, depth=depth, sel=s, W=W)

    for bad in (dict(lens=i32(1)), dict(mask=i32(2, 2, 1)), dict(depth=i32(2, 4), W=1), dict(sel=i32(23, 1)),
                dict(ws=ws[::2]), dict(ws=ws.cpu()), dict(mask=i32(2, 3)), dict(o=z(2, 4, 3))):
        with pytest.raises(ValueError):
            attn(**bad)
    with pytest.raises(TypeError, match="unsupported dtype"):
        attn(o=q.half())
    with pytest.raises(rtp.RtpError):
        attn(ws=None)
    for bad in (dict(path=i32(2)), dict(path=i32(1, 2)), dict(count=i32(3)), dict(lens_out=i32(2).float())):
        a = dict(path=i32(2, 2), count=i32(2), lens_out=i32(2))
        a.update(bad)
        with pytest.raises(ValueError):
            rtp.kv_accept(kv, kv, i32(2), a["path"], a["count"], 0, k_ring=z(2, 2, 4, D), v_ring=z(2, 2, 4, D),
                          lens_out=a["lens_out"])
