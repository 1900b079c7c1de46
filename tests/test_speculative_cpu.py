"""Refusals of the speculative-step calls (rtp_qk_norm_rope, rtp_tree_attn,
rtp_kv_accept), without a GPU: every call below fails validation, so nothing is
launched (the pointers are fake)."""
import ctypes

import pytest
import torch

from test_library_cpu import _desc, _lib, _sel

by = ctypes.byref


def _norm_rope(q=None, k=0, qw=None, kw=None, eps=1e-6, pos=0x1000, offs=None, freq=0x2000, pairing=0, qo=None, ko=0):
    rtp = _lib()
    q = _desc(rtp, [2, 8, 5, 128]) if q is None else q
    k = _desc(rtp, [2, 2, 5, 128], data=0x20000) if k == 0 else k
    qo = _desc(rtp, [2, 8, 5, 128], data=0x30000) if qo is None else qo
    ko = _desc(rtp, [2, 2, 5, 128], data=0x40000) if ko == 0 else ko
    ref = lambda t: None if t is None else by(t)  # noqa: E731
    return rtp.lib().rtp_qk_norm_rope(ref(q), ref(k), ref(qw), ref(kw), eps, pos, offs, freq, pairing, ref(qo),
                                      ref(ko), None)


def test_qk_norm_rope_refusals():
    rtp = _lib()
    d = lambda *a, **kw: _desc(rtp, *a, **kw)  # noqa: E731
    assert _norm_rope(pos=None) == 1
    assert _norm_rope(freq=None) == 1
    assert _norm_rope(freq=0x2004) == 4
    for eps in (-1e-6, float("nan"), float("inf")):
        assert _norm_rope(eps=eps) == 1
    for pairing in (-1, 2):
        assert _norm_rope(pairing=pairing) == 1
    assert _norm_rope(k=None) == 1                                          # k without k_out and the other way round
    assert _norm_rope(ko=None) == 1
    assert _norm_rope(k=None, ko=None, kw=d([1, 128])) == 1                 # a weight for no keys
    assert _norm_rope(q=d([2, 8, 5, 64])) == 2
    assert _norm_rope(qo=d([2, 8, 4, 128])) == 2
    assert _norm_rope(k=d([2, 2, 4, 128]), ko=d([2, 2, 4, 128], data=0x40000)) == 2
    assert _norm_rope(k=d([2, 2, 5, 128], dtype=0)) == 3                    # q and k of one type
    assert _norm_rope(ko=d([2, 2, 5, 128], dtype=0, data=0x40000)) == 3
    assert _norm_rope(q=d([2, 8, 5, 128], data=0x10008)) == 4
    assert _norm_rope(qw=d([3, 128])) == 2                                  # neither 1 row nor one per head
    assert _norm_rope(qw=d([1, 64])) == 2
    assert _norm_rope(qw=d([1, 128], dtype=5)) == 3
    assert _norm_rope(qw=d([1, 128], data=0)) == 1
    assert _norm_rope(qw=d([1, 128], data=0x10004)) == 4
    assert _norm_rope(kw=d([2, 128], strides=[130, 1])) == 4
    # in place only with the input's own strides and type
    assert _norm_rope(qo=d([2, 8, 5, 128], strides=[8 * 5 * 128, 128, 8 * 128, 1])) == 1
    assert _norm_rope(qo=d([2, 8, 5, 128], dtype=0), ko=d([2, 2, 5, 128], dtype=0, data=0x40000)) == 1


def _tree_attn(q=None, k=None, v=None, lens=None, kn=None, vn=None, mask=0x1000, words=1, depth=0x2000, W=0, ring=0,
               sel=None, scale=0.1, o=None, ws=0x100000, nb=1 << 40, tree=True):
    rtp = _lib()
    q = _desc(rtp, [2, 8, 5, 128]) if q is None else q
    k = _desc(rtp, [2, 2, 64, 128]) if k is None else k
    v = _desc(rtp, list(k.shape)) if v is None else v
    kn = _desc(rtp, [2, 2, 5, 128]) if kn is None else kn
    vn = _desc(rtp, list(kn.shape)) if vn is None else vn
    o = _desc(rtp, [2, 8, 5, 128]) if o is None else o
    t = rtp.RtpTree()
    t.mask, t.mask_words, t.depth = mask, words, depth
    return rtp.lib().rtp_tree_attn(by(q), by(k), by(v), lens, by(kn), by(vn), by(t) if tree else None, W, ring,
                                   None if sel is None else by(sel), scale, by(o), ws, nb, None)


def test_tree_attn_refusals():
    rtp = _lib()
    d = lambda *a, **kw: _desc(rtp, *a, **kw)  # noqa: E731
    assert _tree_attn(tree=False) == 1
    assert _tree_attn(mask=None) == 1
    assert _tree_attn(words=0) == 2
    assert _tree_attn(W=-1) == 1
    assert _tree_attn(W=3, depth=None) == 1
    assert _tree_attn(ring=2, W=3) == 1
    assert _tree_attn(ring=1, W=0) == 1                                     # a ring needs its window
    assert _tree_attn(ring=1, W=65) == 1                                    # which fits into it
    assert _tree_attn(ring=1, W=64, sel=_sel(rtp)) == 1
    assert _tree_attn(sel=_sel(rtp, mask=False)) == 1
    assert _tree_attn(sel=_sel(rtp, words=1)) == 2
    for scale in (float("nan"), float("inf")):
        assert _tree_attn(scale=scale) == 1
    assert _tree_attn(kn=d([2, 2, 6, 128])) == 2
    assert _tree_attn(kn=d([2, 1, 5, 128])) == 2
    assert _tree_attn(vn=d([2, 2, 4, 128])) == 2
    assert _tree_attn(o=d([2, 8, 4, 128])) == 2
    assert _tree_attn(q=d([2, 7, 5, 128]), o=d([2, 7, 5, 128])) == 2        # Hq % Hk
    assert _tree_attn(q=d([2, 18, 5, 128]), o=d([2, 18, 5, 128])) == 2      # more than 8 heads in a group
    f32 = dict(q=d([2, 8, 5, 128], dtype=0), k=d([2, 2, 64, 128], dtype=0), v=d([2, 2, 64, 128], dtype=0),
               kn=d([2, 2, 5, 128], dtype=0), vn=d([2, 2, 5, 128], dtype=0))
    assert _tree_attn(**f32) == 3                                           # bf16 tiles
    assert _tree_attn(kn=f32["kn"], vn=f32["vn"]) == 3
    assert _tree_attn(k=d([2, 2, 64, 128], data=0x10004)) == 4


def test_tree_attn_refuses_more_rows_than_it_numbers():
    rtp = _lib()
    d = lambda *a, **kw: _desc(rtp, *a, **kw)  # noqa: E731
    B, T = 1 << 16, 1 << 13
    assert _tree_attn(q=d([B, 4, T, 128]), o=d([B, 4, T, 128]), k=d([B, 1, 64, 128]), kn=d([B, 1, T, 128]),
                      words=T // 32) == 7


def test_tree_attn_workspace_is_checked():
    rtp = _lib()
    need = rtp.tree_attn_workspace_size(2, 8, 5, 2, 64)
    if need:
        assert _tree_attn(ws=None, nb=0) == 5
        assert _tree_attn(nb=need - 1) == 5
        assert _tree_attn(ws=0x100010) == 4
    assert rtp.tree_attn_workspace_size(0, 8, 5, 2, 64) == 0
    assert rtp.tree_attn_workspace_size(2, 8, 0, 2, 64) == 0


def _kv_accept(path=0x1000, A=3, count=0x2000, pos=0x3000, lens_out=0x4000, ring_lens=0x5000, R=1, kn=None, **kw):
    rtp = _lib()
    d = lambda s, **k: _desc(rtp, s, **k)  # noqa: E731
    kn = d([2, 3, 5, 128]) if kn is None else kn
    a = dict(P=d([1, 16, 128], dtype=0), kc=d([2, 1, 64, 128]), vc=d([2, 1, 64, 128]), ki=d([2, 1, 64, 16]),
             kr=d([2, 2, 8, 128]), vr=d([2, 2, 8, 128]))
    a.update(kw)
    return rtp.lib().rtp_kv_accept(by(kn), by(kn), pos, path, A, count, R, *(by(a[x]) for x in
                                   ("P", "kc", "vc", "ki", "kr", "vr")), lens_out, ring_lens, None)


def test_kv_accept_refusals():
    rtp = _lib()
    d = lambda s, **k: _desc(rtp, s, **k)  # noqa: E731
    assert _kv_accept(path=None) == 1
    assert _kv_accept(count=None) == 1
    assert _kv_accept(pos=None) == 1
    assert _kv_accept(A=-1) == 1
    assert _kv_accept(lens_out=0x1000) == 1                                 # a length output over path, count or pos
    assert _kv_accept(ring_lens=0x2000) == 1
    assert _kv_accept(lens_out=0x3000) == 1
    assert _kv_accept(lens_out=0x5000) == 1
    assert _kv_accept(R=4) == 1
    assert _kv_accept(ki=d([2, 1, 63, 16])) == 2
    assert _kv_accept(kr=d([2, 3, 8, 128])) == 2
    assert _kv_accept(kc=d([2, 1, 64, 128], dtype=0)) == 3


def test_binding_refuses_host_tensors():
    rtp = _lib()
    bf = torch.bfloat16
    q, kv = torch.zeros(1, 2, 3, 128, dtype=bf), torch.zeros(1, 1, 3, 128, dtype=bf)
    i1, mask = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 3, 1, dtype=torch.int32)
    freq = torch.zeros(64, dtype=torch.float64)
    with pytest.raises(ValueError, match="current CUDA device"):
        rtp.qk_norm_rope(q, kv, None, None, 1e-6, i1, freq, q, kv)
    with pytest.raises(ValueError, match="current CUDA device"):
        rtp.tree_attn(q, kv, kv, None, kv, kv, mask, 0.1, q)
    with pytest.raises(ValueError, match="current CUDA device"):
        rtp.kv_accept(kv, kv, i1, torch.zeros(1, 2, dtype=torch.int32), i1, 0, k_ring=kv, v_ring=kv)
    with pytest.raises(TypeError, match="need a tensor"):
        rtp.qk_norm_rope([1.0], kv, None, None, 1e-6, i1, freq, q, kv)
    with pytest.raises(ValueError, match="pairing"):
        rtp.qk_norm_rope(q, kv, None, None, 1e-6, i1, freq, q, kv, pairing="both")
    none = rtp.Selection(tau_bits=i1, tiepos=i1, count=i1, mask=None)
    with pytest.raises(ValueError, match="mask"):
        rtp.tree_attn(q, kv, kv, None, kv, kv, mask, 0.1, q, sel=none)
