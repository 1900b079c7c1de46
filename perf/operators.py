"""Cases, plain forms and exact values of the operators of a speculative decoding step.

A model drafts a tree of T tokens per sequence and the layer verifies the tree in
one pass.  Three operators:

  norm_rope  per-head RMS norm of queries and keys and the position rotation, one pass
             (rtp.qk_norm_rope): y = rot(x / sqrt(mean x^2 + eps) * w)
  tree       attention of the drafted tokens over the committed cache and their own
             ancestors (rtp.tree_attn): over the whole cache, over a ring of the last W
             keys (local heads), or over each query's selected keys (retrieval heads)
  accept     the accepted drafts go into the caches, the projected-key cache and the
             rings, and the lengths move on (rtp.kv_accept)

``run`` with ``own`` false computes them from elementary torch operations in fp32
(angles in fp64); with ``own`` true it makes the framework's calls.
"""
import numpy as np
import torch

own = False

D = 128  # head dim of every layer here


# ---- cases ---------------------------------------------------------------------

def listed():
    # layer shapes: 32 query heads, 8 KV heads (2 retrieval, 6 local), as the decode and prefill workloads
    return [
        # one token per sequence out of a packed qkv projection: the smallest call, latency only
        dict(name="norm_rope_b8_t1", op="norm_rope", B=8, Hq=32, Hk=8, T=1, dtype="bf16", pairing="half",
             norm=True, offs=False, maxpos=32768),
        # a tree of 24 drafts per sequence in a million-token context: positions by depth
        dict(name="norm_rope_b16_t24_tree", op="norm_rope", B=16, Hq=32, Hk=8, T=24, dtype="bf16", pairing="half",
             norm=True, offs=True, maxpos=1048576),
        # odd sizes, neighbouring pairs, fp32 activations, per-head weights
        dict(name="norm_rope_b3_t1001_f32", op="norm_rope", B=3, Hq=15, Hk=5, T=1001, dtype="f32", pairing="adjacent",
             norm=True, offs=False, maxpos=131072),
        # the projections of a whole 32768-token prompt: the largest call
        dict(name="norm_rope_b1_t32768", op="norm_rope", B=1, Hq=32, Hk=8, T=32768, dtype="bf16", pairing="half",
             norm=True, offs=False, maxpos=1),
        # a short chat turn, 8 drafts: the smallest attention call
        dict(name="tree_b1_n1000_t8", op="tree", B=1, Hq=32, Hk=8, ctx=1000, spread=0, N=1024, T=8, W=0, ring=False,
             sel=0.0, tree="wide", out="bf16"),
        # a batch at 32k context with ragged lengths, 16 drafts: the ordinary call
        dict(name="tree_b8_n32768_t16", op="tree", B=8, Hq=32, Hk=8, ctx=32768, spread=20000, N=32768, T=16, W=0,
             ring=False, sel=0.0, tree="wide", out="bf16"),
        # the local heads of the same layer over their rings of 4096 rows, fp32 output (the layer's default)
        dict(name="tree_b8_ring4096_t16", op="tree", B=8, Hq=24, Hk=6, ctx=32768, spread=20000, N=4096, T=16, W=4096,
             ring=True, sel=0.0, tree="wide", out="f32"),
        # the retrieval heads over keys selected in runs (about 8% of the context), fp32 output
        dict(name="tree_b8_n32768_t16_selected", op="tree", B=8, Hq=8, Hk=2, ctx=32768, spread=20000, N=32768, T=16,
             W=0, ring=False, sel=0.08, tree="wide", out="f32"),
        # one group of 5 query heads, an odd chain of 27 drafts, a sliding window inside a longer cache
        dict(name="tree_b5_n9999_t27_window", op="tree", B=5, Hq=15, Hk=3, ctx=9999, spread=3333, N=10007, T=27, W=1500,
             ring=False, sel=0.0, tree="chain", out="bf16"),
        # 64 drafts at 131072 keys, 256 query rows per KV head: the largest call
        dict(name="tree_b4_n131072_t64", op="tree", B=4, Hq=32, Hk=8, ctx=131072, spread=0, N=131072, T=64, W=0,
             ring=False, sel=0.0, tree="wide", out="bf16"),
        # up to 8 of 16 drafts accepted per sequence: latency only
        dict(name="accept_b8_t16", op="accept", B=8, Hk=8, R=2, T=16, A=8, N=8192, W=4096, dtype="bf16"),
        # a large batch of long chains
        dict(name="accept_b64_t256", op="accept", B=64, Hk=8, R=2, T=256, A=256, N=4096, W=1024, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["norm_rope", "tree", "tree", "accept"])
    if op == "norm_rope":
        Hk = rng.choice([1, 2, 3, 4, 5, 8])
        Hq = Hk * rng.choice([1, 2, 3, 4, 5, 8])
        B = _log(rng, 1, 64)
        T = _log(rng, 1, max(1, 32768 * 40 // (B * (Hq + Hk) * 2)))
        return dict(op=op, B=B, Hq=Hq, Hk=Hk, T=min(T, 32768), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    pairing=rng.choice(["half", "half", "adjacent"]), norm=rng.random() < 0.8,
                    offs=rng.random() < 0.4, maxpos=_log(rng, 1, 1048576))
    if op == "tree":
        Hk = rng.choice([1, 2, 3, 6, 8])
        G = rng.choice([1, 2, 3, 4, 4, 5, 8])
        B = _log(rng, 1, 16)
        T = _log(rng, 1, 80)
        kind = rng.choice(["full", "full", "ring", "window", "selected"])
        ctx = _log(rng, 8, max(8, min(131072, 1000000 // (B * Hk))))
        spread = rng.randint(0, ctx)
        N, W = ctx + rng.randint(0, 40), 0
        if kind == "ring":
            W = max(1, min(_log(rng, 16, 8192), ctx))
            N = W + rng.choice([0, 0, 5])
        elif kind == "window":
            W = _log(rng, 1, ctx)
        return dict(op=op, B=B, Hq=Hk * G, Hk=Hk, ctx=ctx, spread=spread, N=N, T=T, W=W, ring=kind == "ring",
                    sel=rng.choice([0.03, 0.1, 0.18]) if kind == "selected" else 0.0, tree=rng.choice(["wide", "chain"]),
                    out=rng.choice(["bf16", "f32"]))
    Hk = rng.choice([1, 2, 5, 8])
    T = _log(rng, 1, 256)
    return dict(op=op, B=_log(rng, 1, 64), Hk=Hk, R=rng.randint(0, Hk), T=T, A=rng.randint(1, T), N=rng.randint(300, 4096),
                W=rng.randint(257, 1024), dtype=rng.choice(["bf16", "bf16", "f32"]))


# ---- what follows from a case alone ----------------------------------------------

def _lens(c):
    """Committed tokens of each sequence."""
    return [c["ctx"] - c["spread"] * ((5 * b + 1) % 8) // 8 for b in range(c["B"])]


def _tree(c):
    """Ancestor matrix [B, T, T] (token itself included) and depths [B, T] of the drafted trees."""
    B, T = c["B"], c["T"]
    rng = np.random.default_rng(12345)
    anc = np.zeros((B, T, T), dtype=bool)
    depth = np.zeros((B, T), dtype=np.int64)
    for b in range(B):
        for t in range(T):
            if t:
                par = t - 1 if c["tree"] == "chain" else int(rng.integers(max(0, t - 8), t))
                anc[b, t] = anc[b, par]
                depth[b, t] = depth[b, par] + 1
            anc[b, t, t] = True
    return anc, depth


def _counts(c):
    return [1 + (7 * b + c["A"] - 1) % c["A"] for b in range(c["B"])]


_RUN = 24  # keys per selected run, one run in a cell of 128 keys


def _cells(c, n):
    """Cells of 128 keys that hold a selected run, of a sequence of n keys."""
    cells = n // 128
    return min(cells, max(1, int(round(c["sel"] * n / _RUN)))) if cells else 0


_PICK = 0.6  # share of the runs that one query takes


def work(c):
    if c["op"] == "norm_rope":
        es = 2 if c["dtype"] == "bf16" else 4
        n = c["B"] * (c["Hq"] + c["Hk"]) * c["T"] * D
        return {"bytes": 2 * n * es, "flops": 8 * n}
    if c["op"] == "accept":
        es = 2 if c["dtype"] == "bf16" else 4
        tok, R, L = sum(_counts(c)), c["R"], c["Hk"] - c["R"]
        rows = 2 * D * es
        return {"bytes": tok * (2 * rows * (R + L) + 16 * es * R) + R * 16 * D * 4, "flops": tok * R * 2 * 16 * D}
    B, Hq, Hk, T, W = c["B"], c["Hq"], c["Hk"], c["T"], c["W"]
    anc, depth = _tree(c)
    es = 2 if c["out"] == "bf16" else 4
    byt = B * Hq * T * D * (2 + es) + 2 * B * Hk * T * D * 2
    pairs = 0.0
    for b, n in enumerate(_lens(c)):
        if W:
            union = min(n, W - 1)
            seen = np.minimum(n, np.maximum(W - 1 - depth[b], 0))
            drafts = np.sum(anc[b] & (depth[b][None, :] > depth[b][:, None] - W))
            pairs += Hq * (int(seen.sum()) + int(drafts))
        elif c["sel"] > 0:
            union = _cells(c, n) * _RUN
            pairs += Hq * (T * union * _PICK + int(anc[b].sum()))
            byt += Hq * T * ((n + 31) // 32) * 4
        else:
            union = n
            pairs += Hq * (T * n + int(anc[b].sum()))
        byt += Hk * union * 2 * D * 2
    return {"bytes": int(byt), "flops": int(4 * D * pairs)}


# ---- inputs ------------------------------------------------------------------------

def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _inv_freq(dev):
    return torch.tensor([500000.0 ** (-2.0 * i / D) for i in range(D // 2)], dtype=torch.float64, device=dev)


def _pack_bits(bits):
    """bool [..., n] -> int32 words [..., ceil(n / 32)], bit j % 32 of word j // 32."""
    n = bits.shape[-1]
    words = max((n + 31) // 32, 1)
    full = torch.zeros(*bits.shape[:-1], words * 32, dtype=torch.int64, device=bits.device)
    full[..., :n] = bits
    w = (full.view(*bits.shape[:-1], words, 32) << torch.arange(32, device=bits.device)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    r = np.random.default_rng(seed)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev).to(dtype)

    s = dict(case=c)
    if c["op"] == "norm_rope":
        B, Hq, Hk, T, dt = c["B"], c["Hq"], c["Hk"], c["T"], _dt(c["dtype"])
        qkv = randn(B, T, (Hq + 2 * Hk) * D, dtype=dt)  # the projection's output, heads side by side
        heads = qkv.view(B, T, Hq + 2 * Hk, D).transpose(1, 2)
        s["q"], s["k"] = heads[:, :Hq], heads[:, Hq: Hq + Hk]
        s["qw"] = s["kw"] = None
        if c["norm"]:
            per_head = c["pairing"] == "adjacent"
            s["qw"] = 1 + 0.3 * randn(Hq if per_head else 1, D)
            s["kw"] = 1 + 0.3 * randn(Hk if per_head else 1, D)
        s["eps"] = 1e-6
        s["pos"] = torch.from_numpy(r.integers(0, c["maxpos"], B).astype(np.int32)).to(dev)
        s["offs"] = torch.from_numpy(r.integers(0, T, (B, T)).astype(np.int32)).to(dev) if c["offs"] else None
        s["inv_freq"] = _inv_freq(dev)
        s["q_out"] = torch.empty(B, Hq, T, D, dtype=dt, device=dev)
        s["k_out"] = torch.empty(B, Hk, T, D, dtype=dt, device=dev)
        return s
    if c["op"] == "accept":
        B, Hk, R, T, A, N, W, dt = (c[x] for x in ("B", "Hk", "R", "T", "A", "N", "W", "dtype"))
        dt, L = _dt(dt), c["Hk"] - c["R"]
        s["k_new"], s["v_new"] = randn(B, Hk, T, D, dtype=dt), randn(B, Hk, T, D, dtype=dt)
        s["pos"] = torch.from_numpy(r.integers(0, N - A + 1, B).astype(np.int32)).to(dev)
        s["path"] = torch.from_numpy(np.stack([np.sort(r.permutation(T)[:A]) for _ in range(B)]).astype(np.int32)).to(dev)
        s["count"] = torch.tensor(_counts(c), dtype=torch.int32, device=dev)
        s["P"] = randn(R, 16, D) / D ** 0.5 if R else None
        for name, shape in (("k_cache", (B, R, N, D)), ("v_cache", (B, R, N, D)), ("k_idx", (B, R, N, 16)),
                            ("k_ring", (B, L, W, D)), ("v_ring", (B, L, W, D))):
            s[name] = randn(*shape, dtype=dt) if shape[1] else None
        s["lens_out"] = torch.zeros(B, dtype=torch.int32, device=dev)
        s["ring_lens"] = torch.zeros(B, dtype=torch.int32, device=dev) if L else None
        return s
    B, Hq, Hk, T, N = c["B"], c["Hq"], c["Hk"], c["T"], c["N"]
    bf = torch.bfloat16
    lens = _lens(c)
    s["q"] = randn(B, Hq, T, D, dtype=bf)
    s["k_new"], s["v_new"] = randn(B, Hk, T, D, dtype=bf), randn(B, Hk, T, D, dtype=bf)
    s["k"], s["v"] = torch.zeros(B, Hk, N, D, dtype=bf, device=dev), torch.zeros(B, Hk, N, D, dtype=bf, device=dev)
    for b, n in enumerate(lens):
        n = min(n, N)
        s["k"][b, :, :n], s["v"][b, :, :n] = randn(Hk, n, D, dtype=bf), randn(Hk, n, D, dtype=bf)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    anc, depth = _tree(c)
    s["tree_mask"] = _pack_bits(torch.from_numpy(anc).to(dev))
    s["depth"] = torch.from_numpy(depth.astype(np.int32)).to(dev)
    s["scale"] = D ** -0.5
    s["mask"] = None
    if c["sel"] > 0:
        # runs of neighbouring keys that a KV head's queries share; each query takes most of them
        G = Hq // Hk
        words = max((N + 31) // 32, 1)
        s["mask"] = torch.zeros(B, Hq, T, words, dtype=torch.int32, device=dev)
        for b, n in enumerate(lens):
            m = _cells(c, n)
            if not m:
                continue
            for h in range(Hk):
                start = 128 * r.permutation(n // 128)[:m] + r.integers(0, 128 - _RUN + 1, m)
                pick = r.random((G * T, m)) < _PICK
                pick[r.integers(0, G * T, m), np.arange(m)] = True  # every run is some query's
                keys = torch.from_numpy((start[:, None] + np.arange(_RUN)[None, :]).reshape(-1)).to(dev)
                bits = torch.zeros(G * T, words * 32, dtype=torch.bool, device=dev)
                bits[:, keys] = torch.from_numpy(np.repeat(pick, _RUN, axis=1)).to(dev)
                s["mask"][b, h * G: (h + 1) * G] = _pack_bits(bits).view(G, T, words)
    s["o"] = torch.empty(B, Hq, T, D, dtype=_dt(c["out"]), device=dev)
    if own:
        from long_context_sparse_dim_b200 import rtp
        s["sel"] = None
        if s["mask"] is not None:
            rows = B * Hq * T
            none = torch.zeros(rows, dtype=torch.int32, device=dev)
            s["sel"] = rtp.Selection(tau_bits=none, tiepos=none, count=none, mask=s["mask"].view(rows, -1))
        s["ws"] = rtp.workspace(rtp.tree_attn_workspace_size(B, Hq, T, Hk, N), dev)
    return s


# ---- one pass ------------------------------------------------------------------------

def run(s):
    return {"norm_rope": _run_norm_rope, "tree": _run_tree, "accept": _run_accept}[s["case"]["op"]](s)


def _run_norm_rope(s):
    c = s["case"]
    if own:
        from long_context_sparse_dim_b200 import rtp
        rtp.qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["eps"], s["pos"], s["inv_freq"], s["q_out"], s["k_out"],
                         offs=s["offs"], pairing=c["pairing"])
        return s["q_out"], s["k_out"]
    T = c["T"]
    step = s["offs"] if s["offs"] is not None else torch.arange(T, device=s["pos"].device)[None, :]
    ang = (s["pos"][:, None] + step).double()[:, None, :, None] * s["inv_freq"]  # [B, 1, T, 64]
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    out = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * w[None, :, None, :]
        if c["pairing"] == "half":
            a, b = y[..., : D // 2], y[..., D // 2:]
            y = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
        else:
            a, b = y[..., 0::2], y[..., 1::2]
            y = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
        out.append(y.to(x.dtype))
    return tuple(out)


def _key_positions(c, n, dev):
    """Position held by each cache row of a sequence of n committed tokens (-1: none)."""
    row = torch.arange(c["N"], device=dev)
    if not c["ring"]:
        return torch.where(row < n, row, -1)
    return torch.where(row < n, n - 1 - torch.remainder(n - 1 - row, c["N"]), -1)


def _run_tree(s):
    c = s["case"]
    if own:
        from long_context_sparse_dim_b200 import rtp
        rtp.tree_attn(s["q"], s["k"], s["v"], s["lens"], s["k_new"], s["v_new"], s["tree_mask"], s["scale"], s["o"], s["ws"],
                      depth=s["depth"] if c["W"] else None, W=c["W"], ring=c["ring"], sel=s["sel"])
        return s["o"]
    B, Hq, Hk, T, W = c["B"], c["Hq"], c["Hk"], c["T"], c["W"]
    G, dev = Hq // Hk, s["q"].device
    bit = torch.arange(32, device=dev)
    outs = []
    for b, n in enumerate(_lens(c)):
        pos = _key_positions(c, n, dev)
        used = min(n, c["N"])  # rows behind it hold nothing
        allow = (pos[None, :used] >= 0).expand(T, used)
        tree = ((s["tree_mask"][b][:, :, None] >> bit) & 1).flatten(1)[:, :T].bool()
        if W:
            lo = n + s["depth"][b].long() - W + 1
            allow = allow & (pos[None, :used] >= lo[:, None])
            tree = tree & ((n + s["depth"][b].long())[None, :] >= lo[:, None])
        allow = allow[None].expand(Hq, T, used)
        if s["mask"] is not None:
            allow = allow & ((s["mask"][b][..., None] >> bit) & 1).flatten(-2)[..., :used].bool()
        allow = torch.cat((allow, tree[None].expand(Hq, T, T)), dim=-1).view(Hk, G * T, used + T)
        keys = torch.cat((s["k"][b, :, :used], s["k_new"][b]), dim=1).float()
        vals = torch.cat((s["v"][b, :, :used], s["v_new"][b]), dim=1).float()
        x = torch.matmul(s["q"][b].float().view(Hk, G * T, D) * s["scale"], keys.transpose(1, 2))
        x = torch.where(allow, x, float("-inf"))
        m = x.amax(-1, keepdim=True)
        x = torch.exp(x - torch.where(m == float("-inf"), 0.0, m))
        z = x.sum(-1, keepdim=True)
        o = torch.matmul(x, vals) / torch.where(z > 0, z, 1.0)
        outs.append(o.view(Hq, T, D))
    return torch.stack(outs).to(_dt(c["out"]))


def _run_accept(s):
    c = s["case"]
    R, T, A, N, W, B = (c[x] for x in ("R", "T", "A", "N", "W", "B"))
    L = c["Hk"] - R
    outs = ["k_cache", "v_cache", "k_idx"] * (R > 0) + ["k_ring", "v_ring", "ring_lens"] * (L > 0) + ["lens_out"]
    if own:
        from long_context_sparse_dim_b200 import rtp
        rtp.kv_accept(s["k_new"], s["v_new"], s["pos"], s["path"], s["count"], R, s["P"], s["k_cache"], s["v_cache"],
                      s["k_idx"], s["k_ring"], s["v_ring"], s["lens_out"], s["ring_lens"])
        return {x: s[x] for x in outs}
    dev = s["pos"].device
    step = torch.arange(A, device=dev)
    keep = (step[None, :] < s["count"][:, None])[:, :, None]  # [B, A, 1]
    b = torch.arange(B, device=dev)[:, None]
    at = s["pos"][:, None].long() + step

    def put(dst, src, rows):  # dst [B, H, rows, d] at rows [B, A] receives src [B, A, H, d] where kept
        view = dst.transpose(1, 2)
        view[b, rows] = torch.where(keep[..., None], src, view[b, rows])

    taken = [x.transpose(1, 2)[b, s["path"].long()] for x in (s["k_new"], s["v_new"])]  # [B, A, Hk, D]
    if R:
        put(s["k_cache"], taken[0][:, :, :R], at)
        put(s["v_cache"], taken[1][:, :, :R], at)
        proj = (taken[0][:, :, :R, None, :].float() * s["P"]).sum(-1)
        put(s["k_idx"], proj.to(s["k_idx"].dtype), at)
    if L:
        put(s["k_ring"], taken[0][:, :, R:], at % W)
        put(s["v_ring"], taken[1][:, :, R:], at % W)
        s["ring_lens"].copy_(torch.clamp(s["pos"] + s["count"], 0, W))
    end = s["pos"] + s["count"]
    s["lens_out"].copy_(torch.clamp(end, 0, N) if R else end)
    return {x: s[x] for x in outs}


# ---- the definitions in 64 bits ---------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_rope": _exact_norm_rope, "tree": _exact_tree, "accept": _exact_accept}[case["op"]](case, s)


def _exact_norm_rope(c, s):
    B, T = c["B"], c["T"]
    out = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        H = x.shape[1]
        y = torch.empty(B, H, T, D, dtype=torch.float64, device=x.device)
        for b in range(B):
            z = x[b].double()
            if w is not None:
                z = z / torch.sqrt(torch.sum(z ** 2, dim=-1, keepdim=True) / D + s["eps"]) * w.double().unsqueeze(1)
            where = torch.arange(T, device=x.device) if s["offs"] is None else s["offs"][b]
            phase = torch.polar(torch.ones(T, D // 2, dtype=torch.float64, device=x.device),
                                (int(s["pos"][b]) + where).double()[:, None] * s["inv_freq"][None, :])
            if c["pairing"] == "half":
                z = torch.complex(z[..., :64].contiguous(), z[..., 64:].contiguous()) * phase
                y[b, ..., :64], y[b, ..., 64:] = z.real, z.imag
            else:
                z = torch.complex(z[..., 0::2].contiguous(), z[..., 1::2].contiguous()) * phase
                y[b, ..., 0::2], y[b, ..., 1::2] = z.real, z.imag
        out.append(y)
    return tuple(out)


def _exact_tree(c, s):
    B, Hq, Hk, T, W, N = (c[x] for x in ("B", "Hq", "Hk", "T", "W", "N"))
    G, dev = Hq // Hk, s["q"].device
    anc, depth = _tree(c)
    o = torch.zeros(B, Hq, T, D, dtype=torch.float64, device=dev)
    for b, n in enumerate(_lens(c)):
        first = max(0, n - N) if c["ring"] else 0  # oldest committed position still held
        position = torch.arange(first, n, device=dev)
        rows = position % N if c["ring"] else position
        at = n + torch.from_numpy(depth[b]).to(dev)  # positions of the drafts
        ok = torch.ones(T, n - first, dtype=torch.bool, device=dev)
        okd = torch.from_numpy(anc[b]).to(dev)
        if W:
            ok = at[:, None] - position[None, :] < W
            okd = okd & (at[:, None] - at[None, :] < W)
        for h in range(Hk):
            K = torch.cat((s["k"][b, h][rows], s["k_new"][b, h])).double()
            V = torch.cat((s["v"][b, h][rows], s["v_new"][b, h])).double()
            for e in range(h * G, (h + 1) * G):
                allowed = ok
                if s["mask"] is not None:
                    word = s["mask"][b, e][:, torch.div(rows, 32, rounding_mode="floor")]
                    allowed = ok & (torch.bitwise_and(torch.bitwise_right_shift(word, (rows % 32).int()[None, :]), 1) == 1)
                allowed = torch.cat((allowed, okd), dim=1)
                logit = (s["q"][b, e].double() @ K.T) * s["scale"]
                logit[~allowed] = -float("inf")
                some = allowed.any(dim=1)
                o[b, e, some] = torch.softmax(logit[some], dim=1) @ V
    return o


def _exact_accept(c, s):
    R, N, W, B = (c[x] for x in ("R", "N", "W", "B"))
    pos, count, path = s["pos"].tolist(), s["count"].tolist(), s["path"].long()
    out = {x: s[x].double() for x in ("k_cache", "v_cache", "k_idx", "k_ring", "v_ring") if s[x] is not None}
    for b in range(B):
        src = path[b, : count[b]]
        at = torch.arange(pos[b], pos[b] + count[b], device=src.device)
        if R:
            out["k_cache"][b][:, at] = s["k_new"][b, :R][:, src].double()
            out["v_cache"][b][:, at] = s["v_new"][b, :R][:, src].double()
            out["k_idx"][b][:, at] = torch.einsum("rjd,rnd->rnj", s["P"].double(), s["k_new"][b, :R][:, src].double())
        if R < c["Hk"]:
            out["k_ring"][b][:, at % W] = s["k_new"][b, R:][:, src].double()
            out["v_ring"][b][:, at % W] = s["v_new"][b, R:][:, src].double()
    end = [p + n for p, n in zip(pos, count)]
    if R < c["Hk"]:
        out["ring_lens"] = torch.tensor([min(e, W) for e in end], dtype=torch.int32, device=s["pos"].device)
    out["lens_out"] = torch.tensor([min(e, N) if R else e for e in end], dtype=torch.int32, device=s["pos"].device)
    return out
