"""The draft-tree calls and the log probabilities without a GPU: what they refuse, their
sizing helper, and the oracle's pins on closed forms."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

import decode_step_attention_gb300 as dsa
from oracle import brute
from oracle import decode_ref as O
from oracle import tree as OT


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(dsa.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return dsa.lib()


def _st(L, name, *args):
    st = getattr(L, name)(*args)
    return st, L.dec_last_error().decode()


def at(mib, off=0):  # a dummy address; never dereferenced
    return ctypes.c_void_p((mib << 26) + off)


def test_rope_tree_rejects(L):
    def call(B=2, N=4, Hq=8, Hkv=2, D=128, theta=1e4, layout=0, eps=1e-6, q=at(1), qo=at(2),
             kn=at(3), vn=at(4), qw=None, kw=None, kt=at(5), vt=at(6), pos=at(7), err=None):
        return _st(L, "dec_qknorm_rope_tree", q, qo, kn, vn, qw, kw, kt, vt, pos, None, B, N, Hq,
                   Hkv, D, theta, layout, None, eps, err, None)
    for bad, st in ((dict(B=-1), 1), (dict(B=8193), 2), (dict(N=0), 1), (dict(N=65), 2),
                    (dict(Hq=7), 1), (dict(Hkv=0), 1), (dict(D=96), 2), (dict(theta=-1.0), 1),
                    (dict(layout=2), 1), (dict(eps=-1.0), 1), (dict(qw=at(9)), 1),
                    (dict(q=None), 1), (dict(pos=None), 1), (dict(kt=None), 1),
                    (dict(q=at(1, 8)), 1), (dict(pos=at(7, 2)), 1), (dict(qo=at(1, 256)), 1),
                    (dict(vt=at(5, 1024)), 1), (dict(kt=at(3, 512)), 1), (dict(err=at(9, 1)), 1)):
        got, msg = call(**bad)
        assert got == st and msg, (bad, got, msg)
    assert call(B=0, q=None)[0] == 0


def test_tree_attn_rejects(L):
    def call(B=2, N=4, Hq=8, Hkv=2, D=128, T=256, max_len=256, scale=0.0, cap=0.0, window=0,
             parts=3, q=at(1), kc=at(2), vc=at(3), lens=at(4), kt=at(5), vt=at(6), mask=at(7),
             pos=None, slopes=None, out=at(8), ws=at(9), ws_bytes=1 << 40):
        return _st(L, "dec_gqa_tree_attn", q, kc, vc, lens, kt, vt, mask, None, pos, slopes, out,
                   B, N, Hq, Hkv, D, T, max_len, scale, cap, window, parts, ws, ws_bytes, None)
    for bad, st in ((dict(B=-1), 1), (dict(B=8193), 2), (dict(N=0), 1), (dict(N=65), 2),
                    (dict(Hq=7), 1), (dict(Hq=18), 2), (dict(D=32), 2), (dict(T=0), 1),
                    (dict(max_len=257), 1), (dict(max_len=-1), 1), (dict(parts=-1), 1),
                    (dict(parts=1 << 20), 2), (dict(window=-1), 1),
                    (dict(scale=float("nan")), 1), (dict(cap=-1.0), 1),
                    (dict(cap=float("inf")), 1), (dict(cap=1e-38), 1), (dict(q=None), 1),
                    (dict(mask=None), 1), (dict(kt=None), 1), (dict(window=8), 1), (dict(slopes=at(10)), 1),
                    (dict(kc=at(2, 8)), 1), (dict(mask=at(7, 4)), 1), (dict(lens=at(4, 2)), 1),
                    (dict(out=at(1, 256)), 1), (dict(ws=None), 3), (dict(ws=at(9, 16)), 3),
                    (dict(ws_bytes=16), 3), (dict(B=8000, T=1 << 20, max_len=1), 2)):
        got, msg = call(**bad)
        assert got == st and msg, (bad, got, msg)
    assert call(B=0, q=None)[0] == 0
    need = L.dec_tree_attn_workspace_bytes(2, 4, 8, 2, 128, 256, 3)
    assert need >= 256 and call(ws_bytes=need - 1)[0] == 3
    assert L.dec_tree_attn_workspace_bytes(2, 65, 8, 2, 128, 256, 3) == 0
    assert L.dec_tree_attn_workspace_bytes(2, 4, 7, 2, 128, 256, 3) == 0


def test_tree_attn_rejects_caps_beyond_the_float_range(L):
    for cap, st in ((1.1e30, 1), (3e38, 1), (float("nan"), 1)):
        got, msg = _st(L, "dec_gqa_tree_attn", at(1), at(2), at(3), at(4), at(5), at(6), at(7), None,
                       None, None, at(8), 2, 4, 8, 2, 128, 256, 256, 0.0, cap, 0, 3, at(9), 1 << 40,
                       None)
        assert got == st and "softcap" in msg, (cap, got, msg)
    # a cap that is allowed is refused for something else
    got, msg = _st(L, "dec_gqa_tree_attn", at(1), at(2), at(3), at(4), at(5), at(6), at(7), None, None,
                   None, at(8), 2, 4, 8, 2, 128, 256, 256, 0.0, 1e30, 0, 3, None, 1 << 40, None)
    assert got == 3 and "workspace" in msg


def test_tree_commit_rejects(L):
    def call(B=2, N=4, Hkv=2, D=128, T=256, kt=at(1), vt=at(2), path=at(3), n=at(4), kc=at(5),
             vc=at(6), lens=at(7), err=None):
        return _st(L, "dec_tree_commit", kt, vt, path, n, kc, vc, lens, B, N, Hkv, D, T, err, None)
    for bad, st in ((dict(B=-1), 1), (dict(N=0), 1), (dict(N=65), 2), (dict(Hkv=0), 1),
                    (dict(D=80), 2), (dict(T=0), 1), (dict(kt=None), 1), (dict(path=None), 1),
                    (dict(lens=None), 1), (dict(kc=at(5, 8)), 1), (dict(n=at(4, 2)), 1),
                    (dict(vc=at(5, 4096)), 1), (dict(kc=at(1, 1024)), 1)):
        got, msg = call(**bad)
        assert got == st and msg, (bad, got, msg)
    assert call(B=0, kt=None)[0] == 0


def test_token_logprobs_rejects(L):
    def call(B=2, V=1000, ld=1000, C=1, K=2, T=1.0, ty=0, z=at(1), ids=at(2), lp=at(3), ent=None,
             ti=at(4), tl=at(5)):
        return _st(L, "dec_token_logprobs", z, ty, ld, ids, C, lp, ent, ti, tl, K, B, V, T, None)
    for bad, st in ((dict(B=-1), 1), (dict(B=1 << 21), 2), (dict(V=0), 1),
                    (dict(V=262145, ld=262145), 2), (dict(ld=999), 1), (dict(ty=2), 1),
                    (dict(C=-1), 1), (dict(C=65537), 2), (dict(K=-1), 1), (dict(K=33), 2),
                    (dict(V=1, K=2), 1), (dict(T=0.0), 1), (dict(T=float("nan")), 1),
                    (dict(T=float("inf")), 1), (dict(z=None), 1), (dict(ids=None), 1),
                    (dict(lp=None), 1), (dict(ti=None), 1), (dict(tl=None), 1),
                    (dict(z=at(1, 2)), 1), (dict(ty=1, z=at(1, 1)), 1), (dict(ids=at(2, 2)), 1)):
        got, msg = call(**bad)
        assert got == st and msg, (bad, got, msg)
    assert call(B=0, z=None)[0] == 0
    assert call(C=0, K=0, z=None)[0] == 0  # nothing asked for


def test_python_refusals():
    bf = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dsa.gqa_tree_attn(bf[0], bf, bf, None, bf, bf, None)
    with pytest.raises(TypeError):
        dsa.gqa_tree_attn(bf, bf, bf, None, bf, bf, None, workspace=bf, out=bf)
    with pytest.raises(ValueError):
        dsa.qknorm_rope_tree(bf, bf, bf, bf, bf, None, 1e4)
    with pytest.raises(ValueError):
        dsa.tree_commit(bf, bf, None, None, bf, bf, None)
    with pytest.raises(TypeError):
        dsa.token_logprobs(torch.zeros(2, 8, dtype=torch.float16))
    with pytest.raises(ValueError):
        dsa.token_logprobs(torch.zeros(2, 8))


# ---- the oracle's pins ----------------------------------------------------------------
def _rand(rng, *shape):
    return rng.standard_normal(shape)


def test_oracle_single_node_is_decode_attention():
    rng = np.random.default_rng(0)
    B, Hq, Hkv, D, T = 2, 4, 2, 64, 9
    q, kc, vc = _rand(rng, B, 1, Hq, D), _rand(rng, B, Hkv, T, D), _rand(rng, B, Hkv, T, D)
    kt, vt = _rand(rng, B, Hkv, 1, D), _rand(rng, B, Hkv, 1, D)
    lens = np.array([8, 3])
    out, _ = OT.tree_attention(q, kc, vc, lens, kt, vt, np.ones((B, 1), np.int64), np.ones(B))
    k2, v2 = kc.copy(), vc.copy()
    for b in range(B):
        k2[b, :, lens[b]], v2[b, :, lens[b]] = kt[b, :, 0], vt[b, :, 0]
    want = brute.gqa_decode_attention(q[:, 0], k2, v2, lens + 1)
    assert np.allclose(out[:, 0], want, rtol=1e-12)


def test_oracle_chain_is_sequential_decoding():
    """A chain of nodes gives what decoding them one after the other gives."""
    rng = np.random.default_rng(1)
    N, Hq, Hkv, D, L0 = 4, 2, 1, 64, 5
    q, kt, vt = _rand(rng, 1, N, Hq, D), _rand(rng, 1, Hkv, N, D), _rand(rng, 1, Hkv, N, D)
    kc, vc = _rand(rng, 1, Hkv, L0 + N, D), _rand(rng, 1, Hkv, L0 + N, D)
    mask = np.array([[(1 << (n + 1)) - 1 for n in range(N)]])
    pos = L0 + np.arange(N)[None]
    for window in (0, 1, 3, 100):
        out, _ = OT.tree_attention(q, kc, vc, [L0], kt, vt, mask, [N], pos=pos, window=window)
        k2, v2 = kc.copy(), vc.copy()
        k2[0, :, L0:], v2[0, :, L0:] = kt[0], vt[0]
        for n in range(N):
            want = brute.gqa_decode_attention(q[:, n], k2, v2, [L0 + n + 1],
                                              window=window or None)
            assert np.allclose(out[:, n], want, rtol=1e-12)


def test_oracle_score_options():
    rng = np.random.default_rng(2)
    q, kc, vc = _rand(rng, 1, 1, 1, 64), _rand(rng, 1, 1, 6, 64), _rand(rng, 1, 1, 6, 64)
    none = np.zeros((1, 1), np.int64)
    args = (q, kc, vc, [6], kc[:, :, :1], vc[:, :, :1], none, [1])
    flat, _ = OT.tree_attention(*args, softcap=1e-9)   # all scores squeezed to zero
    assert np.allclose(flat[0, 0, 0], vc[0, 0].mean(0), rtol=1e-6)
    steep, _ = OT.tree_attention(*args, pos=np.array([[6]]), slopes=np.array([1e4]))
    assert np.allclose(steep[0, 0, 0], vc[0, 0, 5], rtol=1e-12)  # the nearest key alone
    empty, _ = OT.tree_attention(q, kc, vc, [0], kc[:, :, :1], vc[:, :, :1], none, [1])
    assert np.all(empty == 0)


def test_oracle_logprobs_closed_forms():
    lp, ent, top, tl = OT.logprobs(np.zeros(8), [0, 7, 8, -1], 3)
    assert np.allclose(lp[:2], -math.log(8)) and np.all(np.isneginf(lp[2:]))
    assert abs(ent - math.log(8)) < 1e-12 and list(top) == [0, 1, 2]
    lp, ent, top, _ = OT.logprobs([1.0, -np.inf, 1.0, 5.0], [1], 2)
    assert np.isneginf(lp[0]) and list(top) == [3, 0]
    z = np.array([0.3, -1.0, 2.0])
    assert np.allclose(OT.logprobs(z, [0], 0, 0.5)[0], 0.6 - math.log(np.exp(2 * z).sum()))


def test_oracle_commit_moves_the_path():
    kt = np.arange(8.0).reshape(1, 1, 4, 2)
    kc = -np.ones((1, 1, 5, 2))
    k, v = OT.commit(kt, kt + 10, np.array([[0, 3, 9, 0]]), [3], kc, kc, [2])
    assert np.array_equal(k[0, 0, 2:4], kt[0, 0, [0, 3]]) and np.all(k[0, 0, 4] == -1)
    assert np.array_equal(v[0, 0, 3], kt[0, 0, 3] + 10) and np.all(k[0, 0, :2] == -1)


def test_oracle_rope_tree_keeps_norms_and_dead_nodes():
    rng = np.random.default_rng(3)
    q, k, v = _rand(rng, 1, 3, 2, 64), _rand(rng, 1, 3, 1, 64), _rand(rng, 1, 3, 1, 64)
    kt = np.zeros((1, 1, 3, 64))
    qr, kr, vr = OT.rope_tree(q, k, v, None, None, kt, kt, np.array([[0, 5, 7]]), [2], 1e4,
                              O.NEOX, 1e-6)
    assert np.allclose(qr[0, 0], q[0, 0]) and np.array_equal(qr[0, 2], q[0, 2])
    assert np.allclose(np.linalg.norm(kr[0, 0, 1]), np.linalg.norm(k[0, 1, 0]))
    assert np.all(kr[0, 0, 2] == 0) and np.array_equal(vr[0, 0, 0], v[0, 0, 0])


def test_rope_tree_rejects_overlaps(L):
    def call(q=at(1), qo=at(2), kn=at(3), vn=at(4), qw=None, kw=None, kt=at(5), vt=at(6), pos=at(7),
             n=at(8), err=at(9)):
        return _st(L, "dec_qknorm_rope_tree", q, qo, kn, vn, qw, kw, kt, vt, pos, n, 2, 4, 8, 2, 128,
                   1e4, 0, None, 1e-6, err, None)
    kv, q = 2 * 4 * 2 * 128 * 2, 2 * 4 * 8 * 128 * 2
    for bad in (dict(qo=at(3, kv - 16)), dict(qo=at(4)), dict(qo=at(5, 16)), dict(qo=at(6)),
                dict(q=at(5), qo=at(2)), dict(q=at(6, 256)), dict(kt=at(4)), dict(vt=at(3, 512)),
                dict(kt=at(1, q - 16)), dict(vt=at(2, q - 16)), dict(qw=at(2, 256), kw=at(10)),
                dict(qw=at(10), kw=at(5)), dict(pos=at(6, 64)), dict(n=at(2)), dict(err=at(7)),
                dict(err=at(5, 4))):
        got, msg = call(**bad)
        assert got == 1 and "overlap" in msg, (bad, got, msg)
    for fine in ({}, dict(qo=at(1)), dict(qo=at(3, kv)), dict(kt=at(1, q)), dict(vt=at(5, kv))):
        got, msg = call(**fine)  # refused for what the addresses are, if at all
        assert "overlap" not in msg, (fine, got, msg)


def test_tree_attn_rejects_overlaps(L):
    need = L.dec_tree_attn_workspace_bytes(2, 4, 8, 2, 128, 256, 3)

    def call(q=at(1), kc=at(2), vc=at(3), lens=at(4), kt=at(5), vt=at(6), mask=at(7), n=at(10),
             pos=at(11), slopes=at(12), out=at(8), ws=at(9)):
        return _st(L, "dec_gqa_tree_attn", q, kc, vc, lens, kt, vt, mask, n, pos, slopes, out, 2, 4,
                   8, 2, 128, 256, 256, 0.0, 0.0, 0, 3, ws, 1 << 40, None)
    row, cache = 2 * 4 * 8 * 128 * 2, 2 * 2 * 256 * 128 * 2
    for bad in (dict(out=at(1, row - 16)), dict(out=at(2, cache - 16)), dict(out=at(3)),
                dict(out=at(5)), dict(out=at(6, 16)), dict(out=at(9, 256)), dict(lens=at(8, 4)),
                dict(mask=at(8, 64)), dict(n=at(8)), dict(pos=at(8)), dict(slopes=at(8, row - 4)),
                dict(ws=at(2)), dict(ws=at(1, 256)), dict(ws=at(8, 256)), dict(kt=at(9, need - 16)),
                dict(pos=at(9, 128)), dict(mask=at(9))):
        got, msg = call(**bad)
        assert got == 1 and "overlap" in msg, (bad, got, msg)
    for fine in ({}, dict(out=at(1, row)), dict(out=at(2, cache)), dict(kt=at(2), vt=at(2))):
        got, msg = call(**fine)
        assert "overlap" not in msg, (fine, got, msg)


def test_commit_and_logprobs_reject_overlaps(L):
    def commit(kt=at(1), vt=at(2), path=at(3), n=at(4), kc=at(5), vc=at(6), lens=at(7), err=at(8)):
        return _st(L, "dec_tree_commit", kt, vt, path, n, kc, vc, lens, 2, 4, 2, 128, 256, err, None)
    cache = 2 * 2 * 256 * 128 * 2
    for bad in (dict(kt=at(6, cache - 16)), dict(vt=at(5)), dict(vc=at(5, 4096)), dict(path=at(5)),
                dict(n=at(6, 8)), dict(lens=at(5, cache - 4)), dict(err=at(5)), dict(err=at(7, 4))):
        got, msg = commit(**bad)
        assert got == 1 and "overlap" in msg, (bad, got, msg)
    assert "overlap" not in commit()[1] and "overlap" not in commit(vc=at(5, cache))[1]

    def logprobs(z=at(1), ids=at(2), lp=at(3), ent=at(4), ti=at(5), tl=at(6), C=3, K=2, ty=0):
        return _st(L, "dec_token_logprobs", z, ty, 1000, ids, C, lp, ent, ti, tl, K, 2, 900, 1.0, None)
    for bad in (dict(lp=at(2)), dict(lp=at(2, 20)), dict(ent=at(1, 1000 * 4 + 900 * 4 - 4)),
                dict(ti=at(6, 12)), dict(tl=at(1)), dict(ent=at(3, 8)), dict(lp=at(5)),
                dict(ti=at(2))):
        got, msg = logprobs(**bad)
        assert got == 1 and "overlap" in msg, (bad, got, msg)
    for fine in ({}, dict(ent=at(1, 7600)), dict(ty=1, ent=at(1, 3800)), dict(lp=at(2), C=0),
                 dict(ti=at(2), K=0)):
        got, msg = logprobs(**fine)
        assert "overlap" not in msg, (fine, got, msg)


def test_tree_workspace_of_refused_shapes_is_nothing(L):
    ws = L.dec_tree_attn_workspace_bytes
    for bad in ((8193, 4, 8, 2, 128, 256, 0), (1 << 20, 64, 1 << 16, 1 << 13, 128, 256, 0),
                (2, 4, 18, 2, 128, 256, 0), (2, 4, 65536, 65536, 128, 256, 0),
                (2, 4, 8, 2, 128, 256, 4097), (2, 64, 1 << 30, 1, 128, 256, 3)):
        assert ws(*bad) == 0, bad
    assert ws(8192, 64, 64, 8, 128, 131072, 0) > ws(2, 64, 64, 8, 128, 131072, 0) > 0


def test_tree_attn_rejects_scales_beyond_the_float_range(L):
    def call(scale, ws):
        return _st(L, "dec_gqa_tree_attn", at(1), at(2), at(3), at(4), at(5), at(6), at(7), None, None,
                   None, at(8), 2, 4, 8, 2, 128, 256, 256, scale, 0.0, 0, 3, ws, 1 << 40, None)
    for scale in (1.1e30, 3e38, float("inf"), float("nan")):
        got, msg = call(scale, at(9))
        assert got == 1 and "scale" in msg, (scale, got, msg)
    for scale in (1e30, 0.0, -3e38):  # allowed, and refused for something else
        got, msg = call(scale, None)
        assert got == 3 and "workspace" in msg
