"""GPU tests of the speculative-step calls at the sizes where their kernels change
form: tree attention over few tiles (a CTA per tile), over many with up to 64 query
rows per KV head, with up to 128 and with more; selections; references that have to
move; workspaces and streams shared between them; long batches of rows and of
accepted drafts.  Formulas and tolerances are those of test_speculative_gpu.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from long_context_sparse_dim_b200 import rtp
from long_context_sparse_dim_b200.layer import TreeDecodeLayer
from test_speculative_gpu import (BF, D, _bits, _check_norm_rope, _check_tree, _freqs, _inputs, _norm_rope_ref,
                                  _run_tree, _tree_ref, _trees)

pytestmark = pytest.mark.gpu

F32 = torch.float32
SCALE = D ** -0.5

CASES = [
    # B, Hq, Hk, N, lens, T, W, ring, kind, out
    # few tiles: the sizes around the form's limit, rows of one, two and four groups of 16
    (1, 4, 4, 6950, [6950], 1, 0, False, "wide", F32),
    (1, 4, 4, 6976, [6976], 1, 0, False, "wide", F32),
    (1, 4, 4, 7100, [7000], 17, 0, False, "wide", BF),
    (2, 4, 2, 2000, [0, 1999], 8, 0, False, "chain", F32),
    (2, 2, 2, 500, [500, 1], 32, 31, False, "wide", F32),
    (3, 3, 1, 70, [64, 65, 63], 65, 0, False, "wide", F32),
    (2, 4, 1, 200, [200, 130], 50, 64, True, "chain", F32),
    (1, 1, 1, 20000, [20000], 5, 0, False, "wide", F32),
    # up to 64 rows per KV head: several tiles of 128 in a CTA's range, groups that end inside one
    (4, 16, 4, 9000, [9000, 8999, 0, 4500], 16, 0, False, "wide", F32),
    (3, 64, 8, 12001, [12001, 1, 11900], 8, 0, False, "wide", BF),
    (5, 8, 8, 15000, [15000, 14000, 13000, 127, 128], 64, 0, False, "chain", F32),
    (70, 4, 2, 700, [(37 * i) % 701 for i in range(70)], 9, 0, False, "wide", F32),
    (300, 2, 2, 150, [i % 151 for i in range(300)], 3, 0, False, "wide", BF),
    (33, 8, 2, 2048, [60 * i + 100 for i in range(33)], 16, 700, False, "chain", F32),
    (16, 16, 4, 4096, [256 * i + 5 for i in range(16)], 16, 4096, True, "wide", F32),
    (16, 16, 4, 1000, [125 * i for i in range(16)], 16, 1000, True, "chain", F32),
    (9, 4, 4, 3000, [3000] * 9, 27, 2999, False, "wide", F32),
    # 65 to 128 rows
    (2, 16, 4, 9001, [9001, 8000], 17, 0, False, "wide", F32),
    (5, 8, 1, 6000, [6000, 5000, 0, 3, 129], 16, 0, False, "wide", BF),
    (1, 20, 4, 70000, [69999], 25, 0, False, "wide", F32),
    (7, 10, 2, 4000, [4000, 3999, 4, 1000, 2000, 3000, 0], 24, 900, False, "chain", F32),
    # more than 128
    (4, 10, 2, 9999, [9999, 9000, 128, 7777], 27, 0, False, "wide", F32),
    (2, 8, 2, 5000, [5000, 4800], 64, 0, False, "wide", BF),
    (5, 40, 8, 3000, [3000, 2900, 2800, 0, 7], 33, 512, False, "chain", F32),
    (2, 8, 1, 4097, [4097, 4000], 80, 0, False, "wide", F32),        # three row blocks
    (2, 3, 1, 9000, [9000, 8500], 200, 0, False, "chain", F32),      # drafts of two tiles
    (6, 16, 4, 2000, [100000, 1999, 2000, 2001, 0, 12], 40, 1500, True, "chain", F32),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_tree_attn_forms(i):
    B, Hq, Hk, N, lens, T, W, ring, kind, out = CASES[i]
    q, k, v, kn, vn = _inputs(B, Hq, Hk, N, T, 50 + i, "bnhd" if i % 2 else "bhnd", lens=lens, ring=ring)
    anc, depth = _trees(B, T, kind, i)
    anc[:, T // 3] = False  # a draft that attends committed keys only
    o = _run_tree(q, k, v, lens, kn, vn, anc, depth, W, ring, None, SCALE, out)
    _check_tree(o, *_tree_ref(q, k, v, lens, kn, vn, anc, depth, W, ring, None, SCALE), f"case {i}")


@pytest.mark.parametrize("rows", [(16, 16, 4), (25, 20, 4), (50, 16, 2)])  # T, Hq, Hk: 64, 125 and 400 rows
def test_tree_attn_long_ranges(rows):
    """Ranges of more than 32 tiles, so that outputs leave the accumulator on the way."""
    T, Hq, Hk = rows
    N = 100000 if T < 50 else 120000
    lens = [N, N - 333]
    q, k, v, kn, vn = _inputs(2, Hq, Hk, N, T, 5, lens=lens)
    anc, depth = _trees(2, T, "wide", 5)
    o = _run_tree(q, k, v, lens, kn, vn, anc, depth, 0, False, None, SCALE, F32)
    _check_tree(o, *_tree_ref(q, k, v, lens, kn, vn, anc, depth, 0, False, None, SCALE), "long")


# T, Hq, Hk, N: few tiles; 64, 128 and 256 rows per KV head over long ranges
FORMS = [(8, 8, 2, 900), (16, 16, 4, 40000), (16, 8, 1, 60000), (32, 16, 2, 60000)]


@pytest.mark.parametrize("form", range(len(FORMS)))
@pytest.mark.parametrize("kind", ["rising", "jumps", "falling", "masked_top"])
def test_tree_attn_references(form, kind):
    """Logits that climb by thousands along the keys, jump, fall, or whose first (masked) draft lies far above."""
    T, Hq, Hk, N = FORMS[form]
    lens = [N, N - 77]
    q, k, v, kn, vn = _inputs(2, Hq, Hk, N, T, 9, lens=lens, dead=0.0)
    one = torch.randn(D, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    one /= one.norm()
    q = (q.float() * 0.3 + 6 * one).to(BF)                  # every query leans on `one`
    if kind == "rising":
        lean = torch.linspace(-300, 300, N, device="cuda")
    elif kind == "falling":
        lean = torch.linspace(300, -300, N, device="cuda")
    elif kind == "jumps":
        lean = torch.zeros(N, device="cuda")
        for i, at in enumerate((N // 7, N // 3, N // 2, 3 * N // 4)):
            lean[at:] += 120 * (i + 1)
    else:
        lean = torch.zeros(N, device="cuda")
    k = (k.float() + lean[:, None] * one).to(BF)
    anc, depth = _trees(2, T, "wide", 9)
    if kind == "masked_top":
        anc[:, 1:, 0] = False
        kn[:, :, 0] = (2000 * one).to(BF)
    sc = 1.0 if kind != "masked_top" else 0.25
    o = _run_tree(q, k, v, lens, kn, vn, anc, depth, 0, False, None, sc, F32)
    _check_tree(o, *_tree_ref(q, k, v, lens, kn, vn, anc, depth, 0, False, None, sc), kind)


@pytest.mark.parametrize("density", [0.0, 0.02, 1.0])
@pytest.mark.parametrize("B,Hq,Hk,N,T,W", [(4, 16, 4, 9000, 16, 0), (3, 20, 4, 5001, 25, 0), (40, 4, 2, 1300, 8, 0),
                                           (5, 8, 4, 4000, 16, 1100), (2, 8, 2, 12000, 40, 0), (2, 8, 2, 3500, 4, 50),
                                           (4, 16, 4, 8192, 16, 0), (3, 8, 2, 12800, 20, 5000)])
def test_tree_attn_selected_forms(B, Hq, Hk, N, T, W, density):
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, N + 1, B)]
    lens[0] = N
    q, k, v, kn, vn = _inputs(B, Hq, Hk, N, T, 13, "bnhd", lens=lens)
    anc, depth = _trees(B, T, "wide", 13)
    runs = np.repeat(rng.random((B, Hq, T, (N + 24) // 25)) < density, 25, axis=-1)[..., :N]
    sel = runs | (rng.random((B, Hq, T, N), dtype=np.float32) < density / 20)
    sel[:, :, T // 2] = False
    sel[:, 0] = False
    live = torch.from_numpy(sel.reshape(B, Hk, -1, N).any(2)).cuda()
    k[~live] = float("inf")
    v[~live] = float("nan")
    o = _run_tree(q, k, v, lens, kn, vn, anc, depth, W, False, sel, SCALE, F32)
    _check_tree(o, *_tree_ref(q, k, v, lens, kn, vn, anc, depth, W, False, sel, SCALE), "selected")


@pytest.mark.parametrize("T,Hq,Hk,N", [(8, 8, 2, 900), (16, 16, 4, 9000), (25, 20, 4, 9000), (50, 16, 2, 9000)])
def test_tree_attn_nan_goes_where_it_is_attended(T, Hq, Hk, N):
    """A NaN among the drafts reaches the drafts below it and no other row, in every form; an infinite V, too."""
    lens = [N, N - 300]
    q, k, v, kn, vn = _inputs(2, Hq, Hk, N, T, 21, lens=lens)
    anc, depth = _trees(2, T, "wide", 21)
    anc[:, :, 2] = np.arange(T) % 3 == 2  # who attends draft 2
    G = Hq // Hk
    for what in ("k", "v"):
        bad_k, bad_v = kn.clone(), vn.clone()
        (bad_k if what == "k" else bad_v)[0, Hk - 1, 2, 7] = float("nan")
        o = torch.empty(2, Hq, T, D, device="cuda")
        ws = rtp.workspace(rtp.tree_attn_workspace_size(2, Hq, T, Hk, N), "cuda")
        rtp.tree_attn(q, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), bad_k, bad_v, _bits(anc), SCALE, o,
                      ws)
        torch.cuda.synchronize()
        hit = torch.zeros(2, Hq, T, dtype=torch.bool, device="cuda")
        hit[0, Hq - G:, 2::3] = True
        dims = torch.ones(D, dtype=torch.bool, device="cuda") if what == "k" else torch.arange(D, device="cuda") == 7
        assert bool(torch.isnan(o[hit][:, dims]).all())
        ref, tol = _tree_ref(q, k, v, lens, kn, vn, anc, depth, 0, False, None, SCALE)
        free = ~hit[..., None] | ~dims
        assert bool(((o.double() - ref).abs() <= tol)[free].all())


@pytest.mark.parametrize("T,Hq,Hk,N", [(16, 16, 4, 500), (25, 20, 4, 500), (50, 32, 4, 300)])
def test_tree_attn_rows_computed_anew_in_whole_groups(T, Hq, Hk, N):
    """Groups that one CTA works on alone: a NaN among the drafts, and a reference far above all that is attended."""
    B, G = 50, Hq // Hk
    lens = [N - 3 * b for b in range(B)]
    q, k, v, kn, vn = _inputs(B, Hq, Hk, N, T, 23, lens=lens)
    one = torch.randn(D, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    one /= one.norm()
    q[1:] = (q[1:].float() * 0.3 + 6 * one).to(BF)
    kn[1:, :, 0] = (2000 * one).to(BF)
    anc, depth = _trees(B, T, "wide", 23)
    anc[1:, 1:, 0] = False
    anc[0, :, 2] = np.arange(T) % 3 == 2
    bad_v = vn.clone()
    bad_v[0, :, 2, 7] = float("nan")
    for out in (F32, BF):
        o = torch.empty(B, Hq, T, D, dtype=out, device="cuda")
        ws = rtp.workspace(rtp.tree_attn_workspace_size(B, Hq, T, Hk, N), "cuda")
        rtp.tree_attn(q, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), kn, bad_v, _bits(anc), 0.25, o, ws)
        torch.cuda.synchronize()
        assert rtp.poll_device_error() == 0
        assert bool(torch.isnan(o[0, :, 2::3, 7]).all())
        o[0, :, 2::3, 7] = 0
        ref, tol = _tree_ref(q, k, v, lens, kn, vn, anc, depth, 0, False, None, 0.25)
        ref[0, :, 2::3, 7] = 0
        _check_tree(o, ref, tol, "anew")


@pytest.mark.parametrize("T,Hq,Hk,N", [(4, 8, 2, 700), (16, 16, 4, 9000), (25, 20, 4, 9000), (50, 16, 2, 9000)])
def test_tree_attn_shared_prefix(T, Hq, Hk, N):
    """One cache for all sequences and all KV heads (strides of 0)."""
    lens = [N, N - 5]
    q, k, v, kn, vn = _inputs(1, Hq, 1, N, T, 31, lens=lens[:1])
    q = torch.cat((q, -q))
    k, v = k.expand(2, Hk, N, D), v.expand(2, Hk, N, D)
    kn, vn = kn.expand(2, Hk, T, D), vn.expand(2, Hk, T, D)
    anc, depth = _trees(2, T, "wide", 31)
    o = _run_tree(q, k, v, lens, kn, vn, anc, depth, 0, False, None, SCALE, F32)
    _check_tree(o, *_tree_ref(q, k, v, lens, kn, vn, anc, depth, 0, False, None, SCALE), "shared")


def _call(B, Hq, Hk, N, T, seed, lens, sel=None):
    q, k, v, kn, vn = _inputs(B, Hq, Hk, N, T, seed, lens=lens)
    anc, _ = _trees(B, T, "wide", seed)
    o = torch.empty(B, Hq, T, D, device="cuda")
    s = None
    if sel is not None:
        rng = np.random.default_rng(seed)
        m = _bits(rng.random((B, Hq, T, N)) < sel).view(B * Hq * T, -1)
        s = rtp.Selection(tau_bits=m[:, 0], tiepos=m[:, 0], count=m[:, 0], mask=m)
    size = rtp.tree_attn_workspace_size(B, Hq, T, Hk, N)
    args = (q, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), kn, vn, _bits(anc), SCALE, o)
    return args, o, s, size


SHAPES = [(2, 8, 2, 900, 8, 1, [900, 100]), (3, 16, 4, 9000, 16, 2, [9000, 8000, 0]),
          (2, 20, 4, 9000, 25, 3, [9000, 70]), (2, 16, 2, 6000, 50, 4, [6000, 5000]),
          (2, 16, 4, 9000, 16, 5, [9000, 8000], 0.1), (1, 4, 1, 300, 40, 6, [299])]


def test_tree_attn_one_workspace_for_all_forms():
    """Calls of every form in turn through one workspace leave what each leaves with its own."""
    calls = [_call(*s[:7], sel=s[7] if len(s) > 7 else None) for s in SHAPES]
    own = []
    for args, o, s, size in calls:
        rtp.tree_attn(*args, rtp.workspace(size, "cuda"), sel=s)
        torch.cuda.synchronize()
        own.append(o.clone())
    ws = rtp.workspace(max(c[3] for c in calls), "cuda")
    ws.fill_(255)
    for order in (range(len(calls)), reversed(range(len(calls)))):
        order = list(order)
        for i in order:
            calls[i][1].fill_(9.0)
        for i in order:
            rtp.tree_attn(*calls[i][0], ws, sel=calls[i][2])
        torch.cuda.synchronize()
        for i in order:
            assert torch.equal(calls[i][1], own[i]), i


def test_tree_attn_on_two_streams():
    """Calls of two streams, each with its own workspace, at the same time; and captured ones."""
    calls = [_call(*s[:7], sel=s[7] if len(s) > 7 else None) for s in SHAPES]
    ws = [rtp.workspace(c[3], "cuda") for c in calls]
    own = []
    for (args, o, s, _), w in zip(calls, ws):
        rtp.tree_attn(*args, w, sel=s)
        torch.cuda.synchronize()
        own.append(o.clone())
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):
        for (args, o, s, _), w, st in zip(calls, ws, streams):
            rtp.tree_attn(*args, w, sel=s, stream=st)
    torch.cuda.synchronize()
    assert rtp.poll_device_error() == 0
    for (args, o, s, _), w in zip(calls, own):
        assert torch.equal(o, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        for (args, o, s, _), w in zip(calls, ws):
            rtp.tree_attn(*args, w, sel=s, stream=streams[0])
    for (args, o, s, _) in calls:
        o.fill_(9.0)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for (args, o, s, _), w in zip(calls, own):
        assert torch.equal(o, w)


@pytest.mark.parametrize("T", [7103, 7105, 18950, 40001])
def test_norm_rope_many_rows(T):
    """Batches so large that a row has fewer lanes."""
    dev = "cuda"
    torch.manual_seed(T)
    q, k = (torch.randn(1, T, h, D, device=dev).to(BF).transpose(1, 2) for h in (3, 1))
    w = 1 + 0.3 * torch.randn(3, D, device=dev)
    pos = torch.tensor([7], dtype=torch.int32, device=dev)
    where = 7 + torch.arange(T, device=dev)[None]
    freq = _freqs(dev)
    for pairing in ("half", "adjacent"):
        for out in (BF, F32):
            qo, ko = (torch.empty(*x.shape, dtype=out, device=dev) for x in (q, k))
            rtp.qk_norm_rope(q, k, w, None, 1e-6, pos, freq, qo, ko, pairing=pairing)
            _check_norm_rope(qo, *_norm_rope_ref(q, w, 1e-6, where, freq, pairing), "q")
            _check_norm_rope(ko, *_norm_rope_ref(k, None, 0.0, where, freq, pairing), "k")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,R,T,A,N,W", [(2, 4, 2, 5, 0, 20, 8), (1, 3, 1, 3, 200, 250, 16), (70, 6, 2, 70, 65, 90, 33),
                                           (300, 2, 1, 2, 2, 6, 3), (1, 2, 1, 1500, 1030, 1100, 256)])
def test_kv_accept_repeated_rows(dtype, B, H, R, T, A, N, W):
    """No columns, the same row at several steps, more steps than drafts, rings that wrap several times."""
    g = torch.Generator(device="cuda").manual_seed(B)
    rng = np.random.default_rng(B)
    kn, vn = (torch.randn(B, H, T, D, generator=g, device="cuda").to(dtype) for _ in range(2))
    P = torch.randn(R, 16, D, generator=g, device="cuda")

    def fresh():
        return [torch.full(s, 3.0, dtype=dtype, device="cuda") for s in
                ((B, R, N, D), (B, R, N, D), (B, R, N, 16), (B, H - R, W, D), (B, H - R, W, D))]

    got, want = fresh(), fresh()
    pos = torch.from_numpy(rng.integers(0, N, B).astype(np.int32)).cuda()
    pos[0] = 5
    path = rng.integers(0, T, (B, A)).astype(np.int32)
    count = torch.from_numpy(rng.integers(0, A + 1, B).astype(np.int32)).cuda()
    count[0] = A
    lens, rlens = (torch.full((B,), -1, dtype=torch.int32, device="cuda") for _ in range(2))
    rtp.kv_accept(kn, vn, pos, torch.from_numpy(path).cuda(), count, R, P, *got, lens, rlens)
    for b in range(B):
        rows = torch.from_numpy(path[b, :int(count[b])]).long().cuda()
        one, rone = (torch.empty(1, dtype=torch.int32, device="cuda") for _ in range(2))
        if len(rows):
            rtp.kv_append(kn[b: b + 1, :, rows].contiguous(), vn[b: b + 1, :, rows].contiguous(), pos[b: b + 1].clone(),
                          R, P, *(c[b: b + 1] for c in want), one, rone)
        else:
            one.fill_(min(int(pos[b]), N)), rone.fill_(min(int(pos[b]), W))
        assert int(lens[b]) == int(one) and int(rlens[b]) == int(rone)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("B,T", [(2, 0), (0, 3), (0, 0)])
def test_tree_attn_of_nothing(B, T):
    q, kv = torch.zeros(B, 4, T, D, dtype=BF, device="cuda"), torch.zeros(B, 2, T, D, dtype=BF, device="cuda")
    cache = torch.zeros(B, 2, 64, D, dtype=BF, device="cuda")
    mask = torch.zeros(B, T, 1, dtype=torch.int32, device="cuda")
    for W in (0, 5):
        rtp.tree_attn(q, cache, cache, None, kv, kv, mask, SCALE, torch.empty_like(q), rtp.workspace(0, "cuda"),
                      depth=mask[..., 0], W=W)
    torch.cuda.synchronize()


def test_tree_step_refuses_other_shapes():
    """Rows of another shape would be spread over the layer's drafts."""
    layer = TreeDecodeLayer(2, 4, 2, 64, 1, 16, 0.9, torch.randn(1, 16, D, device="cuda"), 5)
    q, kv = torch.zeros(2, 4, 5, D, dtype=BF, device="cuda"), torch.zeros(2, 2, 5, D, dtype=BF, device="cuda")
    mask, depth = torch.zeros(2, 5, 1, dtype=torch.int32, device="cuda"), torch.zeros(2, 5, dtype=torch.int32, device="cuda")
    for bad in ((q[:, :, :1], kv, kv), (q, kv[:, :1], kv), (q, kv, kv[:1])):
        with pytest.raises(ValueError, match="need"):
            layer.tree_step(*bad, mask, depth)
    assert layer.tree_step(q, kv, kv, mask, depth).shape == q.shape


@pytest.mark.parametrize("shape", SHAPES[1:5])
def test_tree_attn_wait_budget_runs_out(shape):
    """Waits given up (a budget of a few cycles) are reported, read nothing that was not written for them, and leave
    the next call as it should be."""
    args, o, s, size = _call(*shape[:7], sel=shape[7] if len(shape) > 7 else None)
    ws = rtp.workspace(size, "cuda")
    rtp.tree_attn(*args, ws, sel=s)
    torch.cuda.synchronize()
    want = o.clone()
    for fill in (255, 127, 0):
        ws.fill_(fill)
        try:
            rtp.set_wait_budget_cycles(4)
            rtp.tree_attn(*args, ws, sel=s)
            torch.cuda.synchronize()
        finally:
            rtp.set_wait_budget_cycles(0)
        assert rtp.poll_device_error() == 1
        rtp.tree_attn(*args, ws, sel=s)
        torch.cuda.synchronize()
        assert rtp.poll_device_error() == 0
        assert torch.equal(o, want)


_FIRST = """
import torch
from long_context_sparse_dim_b200 import rtp
D, dev = 128, "cuda"
q, kv = torch.randn(1, 8, 16, D, device=dev).bfloat16(), torch.randn(1, 2, N, D, device=dev).bfloat16()
new, mask = torch.randn(1, 2, 16, D, device=dev).bfloat16(), torch.full((1, 16, 1), 65535, dtype=torch.int32, device=dev)
i, path = torch.zeros(1, dtype=torch.int32, device=dev), torch.arange(4, dtype=torch.int32, device=dev).view(1, 4)
freq, o = torch.rand(64, dtype=torch.float64, device=dev), torch.zeros(1, 8, 16, D, device=dev)
turned, ring = torch.zeros_like(q), torch.zeros(1, 2, 32, D, device=dev).bfloat16()
ws = rtp.workspace(rtp.tree_attn_workspace_size(1, 8, 16, 2, N), dev)
graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
torch.cuda.synchronize()
with torch.cuda.graph(graph, stream=st):
    rtp.qk_norm_rope(q, None, None, None, 1e-6, i, freq, turned, None, stream=st)
    rtp.tree_attn(turned, kv, kv, None, new, new, mask, 0.1, o, ws, stream=st)
    rtp.kv_accept(new, new, i, path, i + 4, 0, k_ring=ring, v_ring=ring.clone(), stream=st)
graph.replay()
torch.cuda.synchronize()
got = o.clone()
rtp.qk_norm_rope(q, None, None, None, 1e-6, i, freq, turned, None)
rtp.tree_attn(turned, kv, kv, None, new, new, mask, 0.1, o, ws)
torch.cuda.synchronize()
assert torch.equal(got, o) and bool((got != 0).any()) and torch.equal(ring[0, :, :4], new[0, :, :4])
"""


@pytest.mark.parametrize("N", [500, 30000])
def test_first_calls_of_a_process_are_captured(N):
    subprocess.run([sys.executable, "-c", f"N = {N}\n" + _FIRST], check=True, timeout=300,
                   cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


@pytest.mark.parametrize("form", range(len(FORMS)))
def test_tree_attn_logits_at_the_end_of_fp32(form):
    """All logits the same and near fp32's lowest value: the mean of the attended rows.  (The key-by-key pass adds
    n terms of weight 1 in fp32: n u of the largest value, and a division.)"""
    T, Hq, Hk, _ = FORMS[form]
    N = 900 if form == 0 else 9000
    q, k, v, kn, vn = _inputs(2, Hq, Hk, N, T, 77, lens=[N, N - 5], dead=0.0)
    q.zero_(), k.zero_(), kn.zero_()
    q[..., 0], k[..., 0], kn[..., 0] = 2.0 ** 60, -2.0 ** 60, -2.0 ** 60
    anc, depth = _trees(2, T, "wide", 77)
    o = _run_tree(q, k, v, [N, N - 5], kn, vn, anc, depth, 0, False, None, 128.0, F32)
    for b, n in enumerate((N, N - 5)):
        a = torch.from_numpy(anc[b]).cuda().double()
        total = v[b, :, None, :n].double().sum(2) + torch.einsum("tj,hjd->htd", a, vn[b].double())
        want = (total / (n + a.sum(1))[None, :, None]).repeat_interleave(Hq // Hk, 0)
        tol = float(v[b].abs().max()) * (n + T + 8) * 2.0 ** -24
        assert bool(((o[b].double() - want).abs() <= tol).all())


def test_tree_attn_selects_from_an_empty_cache():
    q, k, v, kn, vn = _inputs(2, 4, 2, 0, 5, 3, lens=[0, 0])
    anc, depth = _trees(2, 5, "wide", 3)
    o = _run_tree(q, k, v, [0, 0], kn, vn, anc, depth, 0, False, None, SCALE, F32)
    none = torch.zeros(2 * 4 * 5, 0, dtype=torch.int32, device="cuda")
    got, one = torch.empty_like(o), torch.zeros(40, dtype=torch.int32, device="cuda")
    rtp.tree_attn(q, k, v, torch.zeros(2, dtype=torch.int32, device="cuda"), kn, vn, _bits(anc), SCALE, got,
                  rtp.workspace(rtp.tree_attn_workspace_size(2, 4, 5, 2, 0), "cuda"),
                  sel=rtp.Selection(tau_bits=one, tiepos=one, count=one, mask=none))
    torch.cuda.synchronize()
    assert torch.equal(got, o)
