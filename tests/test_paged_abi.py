"""The paged cache's calls without a GPU: what they refuse, the sizing helper, and the oracle's
pins on closed forms."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

import decode_step_attention_gb300 as dsa
from oracle import brute
from oracle import paged as OP


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


def append_call(L, B=2, n=2, Hq=8, Hkv=2, D=128, P=10, page=16, M=4, ty=2, rot=128, theta=1e4, layout=0,
                eps=1e-6, q=at(1), q_ld=1024, qo=at(2), qo_ld=1024, k=at(3), k_ld=256, v=at(4),
                v_ld=256, qw=None, kw=None, kp=at(5), vp=at(6), ks=at(7), vs=at(8), table=at(9),
                start=at(10), cu=None, err=None, inv=None):
    return _st(L, "dec_qknorm_rope_paged_append", q, q_ld, qo, qo_ld, k, k_ld, v, v_ld, qw, kw, kp,
               vp, ty, ks, vs, table, M, start, cu, n, B, Hq, Hkv, D, P, page, rot, theta, layout,
               inv, eps, err, None)


def attn_call(L, B=2, Hq=8, Hkv=2, D=128, P=10, page=16, M=4, ty=2, max_len=64, scale=0.0, window=0,
              parts=3, q=at(1), kp=at(5), vp=at(6), ks=at(7), vs=at(8), table=at(9), lens=at(10),
              out=at(2), ws=at(11), ws_bytes=1 << 40):
    return _st(L, "dec_gqa_paged_attn", q, kp, vp, ty, ks, vs, table, M, lens, out, B, Hq, Hkv, D, P,
               page, max_len, scale, window, parts, ws, ws_bytes, None)


def gather_call(L, B=2, Hkv=2, D=128, P=10, page=16, M=4, ty=2, rows=40, kp=at(5), vp=at(6), ks=at(7),
                vs=at(8), table=at(9), start=None, lens=at(10), ko=at(1), vo=at(2), err=None):
    return _st(L, "dec_paged_gather", kp, vp, ty, ks, vs, table, M, start, lens, ko, vo, B, Hkv, D, P,
               page, rows, err, None)


def step_call(L, B=2, Hq=8, Hkv=2, D=128, P=10, page=16, M=4, ty=2, max_len=64, rot=128, hidden=256,
              x=at(12), res=at(13), nw=at(14), y=at(15), q=at(1), k=at(3), v=at(4), kp=at(5), vp=at(6),
              ks=at(7), vs=at(8), table=at(9), pos=at(10), lens=at(16), out=at(2), ws=at(11),
              eps=1e-6, theta=1e4, window=0):
    return _st(L, "dec_paged_decode_step", x, res, nw, y, hidden, eps, q, k, v, None, None, kp, vp, ty,
               ks, vs, table, M, pos, lens, out, B, Hq, Hkv, D, P, page, max_len, rot, theta, 0, None,
               0.0, window, 3, ws, 1 << 40, None)


CACHE = ((dict(B=-1), 1), (dict(B=8193), 2), (dict(Hkv=0), 1), (dict(D=96), 2), (dict(page=8), 2),
         (dict(page=48), 2), (dict(page=256), 2), (dict(P=0), 1), (dict(M=0), 1), (dict(ty=0), 1),
         (dict(ty=3), 1), (dict(P=1 << 30), 2), (dict(M=1 << 27), 2), (dict(kp=None), 1),
         (dict(vp=None), 1), (dict(table=None), 1), (dict(ks=None), 1), (dict(vs=None), 1),
         (dict(ty=1), 1), (dict(kp=at(5, 8)), 1), (dict(ks=at(7, 2)), 1), (dict(table=at(9, 1)), 1))


def test_append_rejects(L):
    for bad, st in CACHE + (
            (dict(Hq=7), 1), (dict(n=-1), 1), (dict(n=3), 1), (dict(n=1 << 24, cu=at(11)), 2),
            (dict(rot=8), 1), (dict(rot=144), 1), (dict(rot=-16), 1), (dict(theta=0.0), 1),
            (dict(theta=float("inf")), 1), (dict(layout=2), 1), (dict(eps=-1.0), 1), (dict(qw=at(11)), 1),
            (dict(q_ld=1016), 1), (dict(q_ld=1028), 1), (dict(k_ld=248), 1), (dict(v_ld=260), 1),
            (dict(qo_ld=0), 1), (dict(q_ld=1 << 31), 2), (dict(q=None), 1), (dict(qo=None), 1),
            (dict(k=None), 1), (dict(v=None), 1), (dict(start=None), 1), (dict(q=at(1, 8)), 1),
            (dict(start=at(10, 2)), 1), (dict(cu=at(11, 2)), 1), (dict(err=at(11, 1)), 1)):
        got, msg = append_call(L, **bad)
        assert got == st and msg, (bad, got, msg)
    assert append_call(L, B=0, n=0, q=None)[0] == 0
    assert append_call(L, n=0, cu=at(11), q=None)[0] == 0
    assert append_call(L, rot=0, theta=0.0, n=0, cu=at(11))[0] == 0  # nothing turns: theta is not read


def test_append_rejects_overlaps(L):
    pages, row = 10 * 2 * 16 * 128, 1024 * 2
    for bad in (dict(qo=at(1, 256)), dict(qo=at(1), qo_ld=2048), dict(qo=at(3)), dict(qo=at(4, 256)),
                dict(qo=at(5)), dict(q=at(6, 256)), dict(k=at(5, pages - 16)), dict(v=at(7)),
                dict(vp=at(5, 1024)), dict(ks=at(8, 4)), dict(ks=at(5)), dict(table=at(7)),
                dict(start=at(8, 8)), dict(start=at(2)), dict(cu=at(2, 16)), dict(err=at(10)),
                dict(err=at(7)), dict(qw=at(2), kw=at(11)), dict(qw=at(11), kw=at(6)),
                dict(table=at(2, 2 * row - 4))):
        got, msg = append_call(L, **bad)
        assert got == 1 and "overlap" in msg, (bad, got, msg)
    for fine in ({}, dict(qo=at(1)), dict(qo=at(1, 2 * row)), dict(k=at(1, 2 * row), v=at(1, 2 * row))):
        got, msg = append_call(L, **fine)
        assert "overlap" not in msg, (fine, got, msg)
    # column blocks of one packed projection [n, (8 + 2 + 2) 128], q in place
    packed = dict(q=at(1), qo=at(1), k=at(1, 2048), v=at(1, 2560), q_ld=1536, qo_ld=1536, k_ld=1536,
                  v_ld=1536)
    assert "overlap" not in append_call(L, **packed)[1]
    for off in (2032, 1536 * 2 - 496):  # into the heads of q, of this token's or the next one's
        got, msg = append_call(L, **dict(packed, k=at(1, off)))
        assert got == 1 and "overlap" in msg, off


def test_attn_rejects(L):
    for bad, st in CACHE + (
            (dict(Hq=7), 1), (dict(Hq=18), 2), (dict(max_len=65), 1), (dict(max_len=-1), 1),
            (dict(parts=-1), 1), (dict(parts=1 << 20), 2), (dict(window=-1), 1),
            (dict(scale=float("nan")), 1), (dict(scale=2e30), 1), (dict(q=None), 1),
            (dict(lens=None), 1), (dict(out=None), 1), (dict(ws=None), 3), (dict(ws=at(11, 16)), 3),
            (dict(ws_bytes=1), 3), (dict(q=at(1, 8)), 1), (dict(lens=at(10, 2)), 1)):
        got, msg = attn_call(L, **bad)
        assert got == st and msg, (bad, got, msg)
    assert attn_call(L, B=0, q=None)[0] == 0


def test_attn_rejects_overlaps(L):
    need = L.dec_paged_attn_workspace_bytes(2, 8, 2, 128, 64, 3)
    rows = 2 * 8 * 128 * 2
    for bad in (dict(out=at(1)), dict(out=at(1, rows - 16)), dict(out=at(5)), dict(out=at(6, 256)),
                dict(out=at(8)), dict(out=at(11)), dict(table=at(2)), dict(lens=at(2, 4)),
                dict(ws=at(5)), dict(ws=at(1, 256)), dict(kp=at(11, need - 16)), dict(lens=at(11))):
        got, msg = attn_call(L, **bad)
        assert got == 1 and "overlap" in msg, (bad, got, msg)
    for fine in ({}, dict(out=at(1, rows)), dict(vp=at(5)), dict(vs=at(7))):
        got, msg = attn_call(L, **fine)
        assert "overlap" not in msg, (fine, got, msg)


def test_gather_rejects(L):
    for bad, st in CACHE + ((dict(rows=0), 1), (dict(lens=None), 1), (dict(ko=None), 1),
                            (dict(vo=None), 1), (dict(ko=at(1, 8)), 1), (dict(lens=at(10, 2)), 1),
                            (dict(start=at(11, 2)), 1), (dict(err=at(11, 2)), 1),
                            (dict(ko=at(5)), 1), (dict(vo=at(1)), 1), (dict(lens=at(1)), 1),
                            (dict(start=at(2, 64)), 1), (dict(table=at(1, 64)), 1),
                            (dict(ks=at(2)), 1)):
        got, msg = gather_call(L, **bad)
        assert got == st and msg, (bad, got, msg)
    assert gather_call(L, B=0, ko=None)[0] == 0


def test_step_rejects(L):
    for bad, st in CACHE + ((dict(hidden=4), 2), (dict(hidden=260), 2), (dict(x=None), 1),
                            (dict(nw=None), 1), (dict(y=None), 1), (dict(pos=None), 1),
                            (dict(lens=None), 1), (dict(q=None), 1), (dict(max_len=65), 1),
                            (dict(rot=8), 1), (dict(eps=-1.0), 1), (dict(theta=-1.0), 1),
                            (dict(window=-1), 1), (dict(ws=None), 3), (dict(y=at(12)), 1),
                            (dict(y=at(13, 16)), 1), (dict(res=at(12, 256)), 1), (dict(y=at(1)), 1),
                            (dict(res=at(5)), 1), (dict(out=at(3)), 1), (dict(x=at(2)), 1),
                            (dict(ws=at(14)), 1), (dict(q=at(3)), 1), (dict(lens=at(1, 4)), 1)):
        got, msg = step_call(L, **bad)
        assert got == st and msg, (bad, got, msg)
    assert step_call(L, B=0, x=None)[0] == 0


def test_workspace_of_refused_shapes_is_nothing(L):
    ws = L.dec_paged_attn_workspace_bytes
    for bad in ((8193, 8, 2, 128, 256, 0), (-1, 8, 2, 128, 256, 0), (2, 18, 2, 128, 256, 0),
                (2, 7, 2, 128, 256, 0), (2, 8, 0, 128, 256, 0), (2, 8, 2, 96, 256, 0),
                (2, 8, 2, 128, -1, 0), (2, 8, 2, 128, 256, -1), (2, 8, 2, 128, 256, 4097),
                (8192, 65536, 65536, 64, 64, 0)):
        assert ws(*bad) == 0, bad
    assert ws(8192, 64, 8, 128, 131072, 0) >= ws(2, 64, 8, 128, 131072, 0) > 0
    assert ws(1, 1, 1, 64, 0, 0) > 0


@pytest.mark.parametrize("D", [64, 128])
def test_workspace_of_the_longest_contexts(L, D):
    """Lengths up to 2^31 - 1 are as many tiles as they are: no less workspace than half of them."""
    ws = L.dec_paged_attn_workspace_bytes
    for max_len in (2 ** 31 - 1, 2 ** 31 - 16, 2 ** 31 - 128, 2 ** 31 - 256):
        assert ws(1, 1, 1, D, max_len, 0) == ws(1, 1, 1, D, 2 ** 30, 0) > ws(1, 1, 1, D, 0, 0), max_len


@pytest.mark.parametrize("D", [64, 128])
def test_workspace_of_few_parts_for_very_many_tiles(L, D):
    """A piece's ring goes by 32-bit numbers, two to a tile: parts asked for are raised until a piece has some
    2^28 tiles at most, and left alone where it has fewer."""
    ws = L.dec_paged_attn_workspace_bytes
    for max_len, least in ((2 ** 31 - 1, 8), (2 ** 30, 4), (2 ** 28, 1), (4096, 1)):
        for parts in (1, 2, 3, 5, 8, 300):
            # (bf16's tiles of 128 tokens, more than e4m3's; 15 of the largest: B Hkv max_len / 128 < 2^31)
            assert ws(15, 8, 8, D, max_len, parts) == ws(1, 8, 8, D, 0, max(parts, least)), (max_len, parts)


def test_binding_checks():
    bf = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    q, i = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    table = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError):  # bf16 pages have no scales
        dsa.gqa_paged_attn(q, bf, bf, table, i, k_scale=torch.ones(4, 2), v_scale=torch.ones(4, 2))
    with pytest.raises(ValueError):  # e4m3 ones do
        dsa.gqa_paged_attn(q, bf.to(dsa.E4M3), bf.to(dsa.E4M3), table, i)
    with pytest.raises(TypeError):
        dsa.gqa_paged_attn(q, bf.half(), bf.half(), table, i)
    with pytest.raises(ValueError):  # no CPU path
        dsa.gqa_paged_attn(q, bf, bf, table, i)
    with pytest.raises(ValueError):
        dsa.gqa_paged_attn(q, bf, bf, table[0], i)
    with pytest.raises(ValueError):
        dsa.gqa_paged_attn(q[0], bf, bf, table, i)
    with pytest.raises(ValueError):
        dsa.paged_gather(bf, bf, table, i, q, q)
    with pytest.raises(TypeError):
        dsa.qknorm_rope_paged_append(q, q, q, bf, bf, table, None, 1e4)
    with pytest.raises(TypeError):
        dsa.alloc_paged_cache(4, 16, 2, 64, torch.float16, "cpu")
    k, v, ks, vs = dsa.alloc_paged_cache(4, 16, 2, 64, device="cpu")
    assert k.shape == (4, 2, 16, 64) and k.dtype == v.dtype == dsa.E4M3 and ks.shape == (4, 2)
    assert bool((ks == 1).all()) and dsa.alloc_paged_cache(4, 16, 2, 64, dsa.BF16, "cpu")[2] is None


# ---- the oracle's pins ----------------------------------------------------------------
def test_oracle_e4m3_is_the_format():
    assert OP.E4M3.size == 127 and OP.E4M3[-1] == 448 and OP.E4M3[1] == 2.0 ** -9 and OP.E4M3[8] == 2.0 ** -6
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(every[:127], OP.E4M3.astype(np.float32))
    x = np.concatenate([OP.E4M3, (OP.E4M3[1:] + OP.E4M3[:-1]) / 2, np.linspace(0, 448, 9999)])
    x = np.concatenate([x, -x])
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(OP.to_e4m3(x.astype(np.float32)), want)
    assert OP.to_e4m3(1e9) == 448 and OP.to_e4m3(-np.inf) == -448 and np.isnan(OP.to_e4m3(np.nan))


def test_oracle_scale_is_the_smallest_power():
    for top, want in ((448.0, 1.0), (448.0001, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8), (0.0, 2.0 ** -64),
                      (1e-30, 2.0 ** -64)):
        assert OP.scale_for(np.array([0.0, -top])) == want
    assert OP.scale_for(np.array([np.inf, np.nan, 1.75])) == 2.0 ** -8


def test_oracle_partial_rotation():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 64))
    for layout in ("neox", "interleaved"):
        y = OP.rotated(x, None, 7, 1e4, layout, 32, 0.0)
        assert np.array_equal(y[:, 32:], x[:, 32:])
        full = OP.rotated(x[:, :32], None, 7, 1e4, layout, 32, 0.0)
        assert np.allclose(y[:, :32], full)
        assert np.array_equal(OP.rotated(x, None, 7, 1e4, layout, 0, 0.0), x)
    y = OP.rotated(x, None, 1, 1e4, "neox", 16, 0.0)  # pair 0 turns by one radian
    assert np.allclose(y[:, 0], x[:, 0] * math.cos(1) - x[:, 8] * math.sin(1))


def test_oracle_paged_attention_is_contiguous_attention():
    rng = np.random.default_rng(1)
    P, Hkv, page, D = 7, 2, 16, 64
    cache = dict(k=rng.standard_normal((P, Hkv, page, D)), v=rng.standard_normal((P, Hkv, page, D)),
                 ks=None, vs=None)
    table = np.array([[3, 0, 6], [5, 99, 99]])
    q, lens = rng.standard_normal((2, 4, D)), [40, 3]
    K = np.stack([cache["k"][np.clip(t, 0, 6)].transpose(1, 0, 2, 3).reshape(Hkv, -1, D) for t in table])
    V = np.stack([cache["v"][np.clip(t, 0, 6)].transpose(1, 0, 2, 3).reshape(Hkv, -1, D) for t in table])
    for window in (0, 2, 17):
        out = OP.attention(q, cache, table, lens, window=window)[0]
        assert np.allclose(out, brute.gqa_decode_attention(q, K, V, lens, window=window or None))
    cache["ks"], cache["vs"] = np.full((P, Hkv), 2.0), np.full((P, Hkv), 3.0)
    twice = OP.attention(q / 2, cache, table, lens)[0]
    assert np.allclose(twice, 3 * OP.attention(q, dict(cache, ks=None, vs=None), table, lens)[0])


def test_oracle_append_grows_a_page():
    cache = dict(k=np.zeros((3, 1, 16, 64)), v=np.zeros((3, 1, 16, 64)), ks=np.ones((3, 1)),
                 vs=np.ones((3, 1)))
    x = np.full((2, 1, 64), 0.5)
    table = np.array([[2, 0]])
    _, c = OP.append(np.zeros((2, 1, 64)), x, x, cache, table, [0], [0, 2], 1e4, "neox", 0)
    assert c["vs"][2, 0] == 2.0 ** -9 and np.all(c["v"][2, 0, :2] == 256) and np.all(c["v"][2, 0, 2:] == 0)
    _, d = OP.append(np.zeros((1, 1, 64)), 64 * x[:1], x[:1] / 4, c, table, [2], None, 1e4, "neox", 0)
    assert d["ks"][2, 0] == 2.0 ** -3 and np.all(d["k"][2, 0, :2] == 4) and np.all(d["k"][2, 0, 2] == 256)
    assert d["vs"][2, 0] == 2.0 ** -9 and np.all(d["v"][2, 0, 2] == 64)
    _, e = OP.append(np.zeros((20, 1, 64)), np.ones((20, 1, 64)), np.ones((20, 1, 64)), d, table, [10],
                     [0, 20], 1e4, "neox", 0)
    assert e["vs"][0, 0] == 2.0 ** -8 and np.all(e["v"][0, 0, :14] == 256) and np.all(e["v"][0, 0, 14:] == 0)
